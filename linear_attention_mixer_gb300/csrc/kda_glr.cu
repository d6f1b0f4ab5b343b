// kda_glr.cu - the gated linear recurrence: token by token (decode), and the host side of its entry points.
#include <climits>
#include <cstdarg>
#include <cstdio>

#include "kda_colsum.cuh"
#include "kda_glr.cuh"
#include "kda_glr_scan.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace glr {
namespace {

// Decode: one thread has four channels of one row through its n <= N tokens, all of which it asks for before it begins. 256 rows of
// 12288 channels, four tokens, BF16 with an output gate: 26.4 us, 5.7 TB/s, 60% of the issue slots taken (two channels a thread: 28.0,
// 74%; asking for a token at a time: 47).
template <typename T, bool G, int N>
__global__ void __launch_bounds__(128) glr_decode_kernel(const __grid_constant__ Args p)
{
    using Q = Quad<T>;
    const int quarter = p.D / 4, unit = blockIdx.x * 128 + threadIdx.x;
    const int row = unit / quarter, c = 4 * (unit - row * quarter);
    if (row >= p.N) return;
    int src, dst;
    const bool ok = slots_ok(p, row, src, dst);
    const int64_t t0 = (int64_t)row * p.n;
    const T *xp = static_cast<const T *>(p.rows.x) + t0 * p.rows.x_stride + c, *ap = static_cast<const T *>(p.rows.a) + t0 * p.rows.a_stride + c;
    const T *bp = static_cast<const T *>(p.rows.b) + t0 * p.rows.b_stride + c, *gp = G ? static_cast<const T *>(p.rows.g) + t0 * p.rows.g_stride + c : nullptr;
    T *op = static_cast<T *>(p.rows.out) + t0 * p.rows.out_stride + c;
    typename Q::Raw x[N], a[N], b[N], g[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < p.n) {
            x[i] = ld_quad(xp + i * p.rows.x_stride);
            a[i] = ld_quad(ap + i * p.rows.a_stride);
            b[i] = ld_quad(bp + i * p.rows.b_stride);
            if (G) g[i] = ld_quad(gp + i * p.rows.g_stride);
        }
    if (!ok) {
        if (c == 0) set_err(p.err);
        return;
    }
    const float4 S = src >= 0 ? *reinterpret_cast<const float4 *>(p.S + (size_t)src * p.D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    float2 h[2] = {make_float2(S.x, S.y), make_float2(S.z, S.w)};
    Chan ch[2];
    ch[0].load(p.A_log, p.a_bias, p.b_bias, c);
    ch[1].load(p.A_log, p.a_bias, p.b_bias, c + 2);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < p.n) {
            float2 o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 e, u;
                gates(ch[j], Q::get(x[i], j), Q::get(a[i], j), Q::get(b[i], j), e, u);
                h[j] = step(h[j], e, u);
                o[j] = G ? f2_mul(h[j], silu2(Q::get(g[i], j))) : h[j];
            }
            *reinterpret_cast<typename Q::Raw *>(op + i * p.rows.out_stride) = Q::put(o[0], o[1]);
        }
    *reinterpret_cast<float4 *>(p.S + (size_t)dst * p.D + c) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
}

template <typename T, bool G>
void launch_decode(const Args &p, unsigned blocks, cudaStream_t s)
{
    if (p.n == 1) glr_decode_kernel<T, G, 1><<<blocks, 128, 0, s>>>(p);
    else if (p.n == 2) glr_decode_kernel<T, G, 2><<<blocks, 128, 0, s>>>(p);
    else if (p.n <= 4) glr_decode_kernel<T, G, 4><<<blocks, 128, 0, s>>>(p);
    else glr_decode_kernel<T, G, 8><<<blocks, 128, 0, s>>>(p);
}

__global__ void __launch_bounds__(kSumCols *kSumGroups) glr_param_sums_kernel(const float *part, int rows, int D, float *dA_log, float *da_bias, float *db_bias)
{
    __shared__ float sh[kSumGroups][kSumCols];
    wait_for_previous();
    float *out = blockIdx.y == 0 ? dA_log : blockIdx.y == 1 ? da_bias : db_bias;
    if (!out) return;
    const float s = column_sum(part + (size_t)blockIdx.y * D, rows, 3 * (int64_t)D, blockIdx.x * kSumCols, D, sh);
    const int c = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.y == 0 && c < D) out[c] = s;
}

// ---------------------------------------------------------------- host side
thread_local char g_msg[256];

kda_status fail(kda_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return record_error(s, g_msg);
}

bool cfg_ok(const kda_glr_config_t *c)
{
    if (!c) return fail(KDA_ERR_INVALID, "config is NULL"), false;
    if (c->io_dtype != KDA_F32 && c->io_dtype != KDA_BF16) return fail(KDA_ERR_INVALID, "io_dtype must be KDA_F32 or KDA_BF16"), false;
    const int unit = c->io_dtype == KDA_BF16 ? 8 : 4;
    if (c->dim < unit || c->dim % unit || c->dim > KDA_GLR_MAX_DIM)
        return fail(KDA_ERR_INVALID, "dim must be a positive multiple of %d up to %d (got %d)", unit, KDA_GLR_MAX_DIM, c->dim), false;
    return true;
}

bool row_ok(const char *name, const void *ptr, int64_t stride, int64_t T, const kda_glr_config_t *c)
{
    const int e = c->io_dtype == KDA_BF16 ? 2 : 4;
    if (!ptr) return fail(KDA_ERR_INVALID, "%s is NULL", name), false;
    if (reinterpret_cast<uintptr_t>(ptr) % 16) return fail(KDA_ERR_INVALID, "%s must be 16-byte aligned", name), false;
    if (T == 1) return true;  // the distance between tokens is not used
    if (stride < c->dim)
        return fail(KDA_ERR_INVALID, "%s_stride must be >= %d (got %lld)", name, c->dim, (long long)stride), false;
    if (stride > ((int64_t)1 << 38) || T > ((int64_t)1 << 60) / stride) return fail(KDA_ERR_INVALID, "%s_stride out of range (%lld)", name, (long long)stride), false;
    if ((stride * e) % 16) return fail(KDA_ERR_INVALID, "%s_stride must be a multiple of %d elements (got %lld)", name, 16 / e, (long long)stride), false;
    return true;
}

bool f32_ok(const char *name, const void *ptr)
{
    if (!ptr || (reinterpret_cast<uintptr_t>(ptr) & 15u)) return fail(KDA_ERR_INVALID, "%s is NULL or not 16-byte aligned", name), false;
    return true;
}
bool f32_or_null_ok(const char *name, const void *ptr) { return !ptr || f32_ok(name, ptr); }

bool params_ok(const kda_glr_params *p)
{
    if (!p) return fail(KDA_ERR_INVALID, "params is NULL"), false;
    return f32_ok("A_log", p->A_log) && f32_ok("a_bias", p->a_bias) && f32_ok("b_bias", p->b_bias);
}

bool call_ok(const kda_glr_config_t *c, const kda_glr_params *prm, const float *S, int32_t max_slots, const int32_t *src,
             const int32_t *dst, const kda_glr_rows *r, int64_t T)
{
    if (!params_ok(prm) || !f32_ok("S", S)) return false;
    if (max_slots < 1) return fail(KDA_ERR_INVALID, "max_slots must be >= 1 (got %d)", max_slots), false;
    if (!src || !dst) return fail(KDA_ERR_INVALID, "src_slots or dst_slots is NULL"), false;
    if (!r) return fail(KDA_ERR_INVALID, "rows is NULL"), false;
    if (T == 0) return true;
    return row_ok("x", r->x, r->x_stride, T, c) && row_ok("a", r->a, r->a_stride, T, c) && row_ok("b", r->b, r->b_stride, T, c) &&
           (!r->g || row_ok("g", r->g, r->g_stride, T, c)) && row_ok("out", r->out, r->out_stride, T, c);
}

Args make_args(const kda_glr_config_t *c, const kda_glr_params *prm, float *S, int32_t max_slots, const int32_t *src, const int32_t *dst,
               int32_t N, const kda_glr_rows *r, int32_t *err)
{
    Args p = {};
    p.S = S; p.max_slots = max_slots; p.src = src; p.dst = dst; p.err = err; p.N = N; p.D = c->dim;
    p.A_log = prm->A_log; p.a_bias = prm->a_bias; p.b_bias = prm->b_bias;
    p.rows = *r;
    return p;
}

// Checks the host's cu_seqlens.
bool lengths_ok(const int32_t *cu, int32_t N)
{
    if (N < 0) return fail(KDA_ERR_INVALID, "N must be >= 0 (got %d)", N), false;
    if (N == 0) return true;
    if (!cu) return fail(KDA_ERR_INVALID, "cu_seqlens or cu_seqlens_host is NULL"), false;
    if (cu[0] != 0) return fail(KDA_ERR_INVALID, "cu_seqlens[0] must be 0 (got %d)", cu[0]), false;
    for (int32_t i = 0; i < N; ++i) {
        if (cu[i + 1] < cu[i]) return fail(KDA_ERR_INVALID, "cu_seqlens decreases at %d", i + 1), false;
    }
    if (cu[N] > KDA_GLR_MAX_TOKENS) return fail(KDA_ERR_INVALID, "at most %d tokens (got %d)", KDA_GLR_MAX_TOKENS, cu[N]), false;
    return true;
}

int64_t slabs_of(int32_t D) { return (D + kSlab - 1) / kSlab; }

bool workspace_ok(const void *ws, size_t bytes, size_t need)
{
    if (ws && !(reinterpret_cast<uintptr_t>(ws) & 15u) && bytes >= need) return true;
    return fail(KDA_ERR_INVALID, "workspace is NULL, not 16-byte aligned, or holds %zu bytes of %zu needed", bytes, need), false;
}

// The workspace: a backward's partial sums, then what split sequences need.
size_t sums_bytes(int32_t N, int32_t D) { return N == 0 ? 0 : ((size_t)back_parts(N, slabs_of(D)) * 3 * D * sizeof(float) + 255) / 256 * 256; }
size_t need_bytes(int32_t N, int32_t D) { return N == 0 ? 256 : 256 + sums_bytes(N, D) + split_bytes(N, slabs_of(D)); }
void lay_out(Split &split, void *workspace, int32_t N, int32_t D)
{
    char *at = static_cast<char *>(workspace) + sums_bytes(N, D);
    split.pairs = reinterpret_cast<float4 *>(at);
    split.S0 = reinterpret_cast<float *>(at + split_pairs_bytes(N, slabs_of(D)));
}

}  // namespace
}  // namespace glr
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_glr_config(kda_glr_config_t *cfg, int32_t dim, int32_t io_dtype)
{
    if (!cfg) return glr::fail(KDA_ERR_INVALID, "cfg is NULL");
    const kda_glr_config_t c = {dim, io_dtype};
    if (!glr::cfg_ok(&c)) return KDA_ERR_INVALID;
    *cfg = c;
    return KDA_OK;
}

kda_status kda_glr_decode(const kda_glr_config_t *cfg, const kda_glr_params *params, float *S, int32_t max_slots, const int32_t *src_slots,
                          const int32_t *dst_slots, int32_t B, int32_t n, const kda_glr_rows *rows, int32_t *err, void *stream)
{
    if (!glr::cfg_ok(cfg)) return KDA_ERR_INVALID;
    if (B < 0) return glr::fail(KDA_ERR_INVALID, "B must be >= 0 (got %d)", B);
    if (n < 1 || n > KDA_DECODE_MAX_TOKENS) return glr::fail(KDA_ERR_INVALID, "n must be in 1 .. %d (got %d)", KDA_DECODE_MAX_TOKENS, n);
    if (B == 0) return KDA_OK;
    if (!glr::call_ok(cfg, params, S, max_slots, src_slots, dst_slots, rows, (int64_t)B * n)) return KDA_ERR_INVALID;
    glr::Args p = glr::make_args(cfg, params, S, max_slots, src_slots, dst_slots, B, rows, err);
    p.n = n;
    p.total_T = (int64_t)B * n;
    if ((int64_t)B * (cfg->dim / 4) > INT_MAX - 128) return glr::fail(KDA_ERR_INVALID, "B * dim is too large");
    const int64_t blocks = ((int64_t)B * (cfg->dim / 4) + 127) / 128;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = cfg->io_dtype == KDA_F32;
    if (rows->g) {
        if (f32) glr::launch_decode<float, true>(p, (unsigned)blocks, s);
        else glr::launch_decode<__nv_bfloat16, true>(p, (unsigned)blocks, s);
    } else {
        if (f32) glr::launch_decode<float, false>(p, (unsigned)blocks, s);
        else glr::launch_decode<__nv_bfloat16, false>(p, (unsigned)blocks, s);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KDA_OK : glr::fail(KDA_ERR_CUDA, "kda_glr_decode: %s", cudaGetErrorString(e));
}

size_t kda_glr_workspace_bytes(const kda_glr_config_t *cfg, const int32_t *cu_seqlens_host, int32_t N)
{
    if (!glr::cfg_ok(cfg) || !glr::lengths_ok(cu_seqlens_host, N)) return 0;
    return glr::need_bytes(N, cfg->dim);
}

int64_t kda_glr_chunks(const int32_t *cu_seqlens_host, int32_t N)
{
    if (!glr::lengths_ok(cu_seqlens_host, N)) return -1;
    return N == 0 ? 0 : (int64_t)(cu_seqlens_host[N] / glr::kChunk) + N;
}

kda_status kda_glr_prefill(const kda_glr_config_t *cfg, const kda_glr_params *params, float *S, int32_t max_slots, const int32_t *src_slots,
                           const int32_t *dst_slots, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int32_t N,
                           const kda_glr_rows *rows, float *starts, void *workspace, size_t workspace_bytes, int32_t *err, void *stream)
{
    if (!glr::cfg_ok(cfg) || !glr::lengths_ok(cu_seqlens_host, N)) return KDA_ERR_INVALID;
    if (N == 0) return KDA_OK;
    if (!cu_seqlens) return glr::fail(KDA_ERR_INVALID, "cu_seqlens or cu_seqlens_host is NULL");
    const int64_t T = cu_seqlens_host[N];
    if (!glr::call_ok(cfg, params, S, max_slots, src_slots, dst_slots, rows, T) || !glr::f32_or_null_ok("starts", starts)) return KDA_ERR_INVALID;
    if (N * glr::slabs_of(cfg->dim) > INT_MAX / 16) return glr::fail(KDA_ERR_INVALID, "N * dim is too large");
    if (!glr::workspace_ok(workspace, workspace_bytes, glr::need_bytes(N, cfg->dim))) return KDA_ERR_INVALID;
    glr::Args p = glr::make_args(cfg, params, S, max_slots, src_slots, dst_slots, N, rows, err);
    p.cu = cu_seqlens;
    p.total_T = T;
    p.starts = starts;
    glr::lay_out(p.split, workspace, N, cfg->dim);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int dev = 0, sms = 0;
    cudaError_t e = current_sms(&dev, &sms);
    if (e == cudaSuccess) e = glr::launch_scan(p, cfg->io_dtype == KDA_F32, cu_seqlens_host, dev, sms, s);
    return e == cudaSuccess ? KDA_OK : glr::fail(KDA_ERR_CUDA, "kda_glr_prefill: %s", cudaGetErrorString(e));
}

kda_status kda_glr_backward(const kda_glr_config_t *cfg, const kda_glr_params *params, const int32_t *cu_seqlens,
                            const int32_t *cu_seqlens_host, int32_t N, const float *starts, const kda_glr_grad_rows *rows,
                            const float *dS_last, float *dS_first, float *dA_log, float *da_bias, float *db_bias, void *workspace,
                            size_t workspace_bytes, int32_t *err, void *stream)
{
    if (!glr::cfg_ok(cfg) || !glr::lengths_ok(cu_seqlens_host, N)) return KDA_ERR_INVALID;
    if (!glr::f32_or_null_ok("dA_log", dA_log) || !glr::f32_or_null_ok("da_bias", da_bias) || !glr::f32_or_null_ok("db_bias", db_bias)) return KDA_ERR_INVALID;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int32_t D = cfg->dim;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (N > 0) {
        if (!cu_seqlens) return glr::fail(KDA_ERR_INVALID, "cu_seqlens or cu_seqlens_host is NULL");
        if (!rows) return glr::fail(KDA_ERR_INVALID, "rows is NULL");
        if (!glr::params_ok(params) || !glr::f32_ok("starts", starts) || !glr::f32_or_null_ok("dS_last", dS_last) ||
            !glr::f32_or_null_ok("dS_first", dS_first)) return KDA_ERR_INVALID;
        const int64_t T = cu_seqlens_host[N];
        const kda_glr_grad_rows *r = rows;
        if (T > 0) {
            if (!glr::row_ok("x", r->x, r->x_stride, T, cfg) || !glr::row_ok("a", r->a, r->a_stride, T, cfg) ||
                !glr::row_ok("b", r->b, r->b_stride, T, cfg) || !glr::row_ok("dout", r->dout, r->dout_stride, T, cfg) ||
                !glr::row_ok("dx", r->dx, r->dx_stride, T, cfg) || !glr::row_ok("da", r->da, r->da_stride, T, cfg) ||
                !glr::row_ok("db", r->db, r->db_stride, T, cfg)) return KDA_ERR_INVALID;
            if (!r->g != !r->dg) return glr::fail(KDA_ERR_INVALID, "g and dg must both be given or both be NULL");
            if (r->g && (!glr::row_ok("g", r->g, r->g_stride, T, cfg) || !glr::row_ok("dg", r->dg, r->dg_stride, T, cfg))) return KDA_ERR_INVALID;
        }
        if (N * glr::slabs_of(D) > INT_MAX / 16) return glr::fail(KDA_ERR_INVALID, "N * dim is too large");
        if (!glr::workspace_ok(workspace, workspace_bytes, glr::need_bytes(N, D))) return KDA_ERR_INVALID;
        glr::BackArgs p = {};
        p.err = err; p.cu = cu_seqlens; p.N = N; p.total_T = T; p.D = D;
        p.A_log = params->A_log; p.a_bias = params->a_bias; p.b_bias = params->b_bias;
        p.starts = starts; p.rows = *rows; p.dS_last = dS_last; p.dS_first = dS_first;
        p.part = static_cast<float *>(workspace);
        glr::lay_out(p.split, workspace, N, D);
        p.groups = glr::back_groups(N, glr::slabs_of(D));
        int dev = 0, sms = 0;
        if ((e = current_sms(&dev, &sms)) == cudaSuccess) e = glr::launch_scan_back(p, cfg->io_dtype == KDA_F32, cu_seqlens_host, &parts, dev, sms, s);
    }
    if (e == cudaSuccess && (dA_log || da_bias || db_bias)) {  // without sequences: zeros
        const dim3 grid((D + kSumCols - 1) / kSumCols, 3);
        const float *part = static_cast<const float *>(workspace);
        // without sequences no kernel of this call comes before it
        if (parts > 0) e = launch_after(glr::glr_param_sums_kernel, grid, sum_block(parts), 0, s, part, parts, D, dA_log, da_bias, db_bias);
        else glr::glr_param_sums_kernel<<<grid, sum_block(0), 0, s>>>(part, 0, D, dA_log, da_bias, db_bias), e = cudaGetLastError();
    }
    return e == cudaSuccess ? KDA_OK : glr::fail(KDA_ERR_CUDA, "kda_glr_backward: %s", cudaGetErrorString(e));
}

}  // extern "C"
