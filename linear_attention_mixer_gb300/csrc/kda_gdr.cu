// kda_gdr.cu - the gated delta rule, token by token (decode, and prefill of FP32 rows), and the
// host side of its entry points.
//
// One warp owns 16 value columns of one (row, head) state: columns of S do not interact, so a warp
// runs its tokens alone, with no barrier and no shared memory. Lane (rg, cg) = (lane / 4, lane % 4)
// holds the 16 key rows 16 rg .. 16 rg + 15 of the 4 columns 4 cg .. 4 cg + 3 in registers from the
// first token to the last. With the raw k, q and the scalars rk = 1 / sqrt(|k|^2 + eps),
// rq = q_scale / sqrt(|q|^2 + eps) a token is
//   p = S^T k, r = S^T q                       8 partial sums a lane, added over rg by halving exchanges
//   u = beta (v - alpha rk p)
//   o = rq (alpha r + rk (k . q) u),  S = alpha S + k (rk u)^T
// so that the normalised vectors are never formed.
//
// Decode is bound by the states' way through HBM: one read and one write of 64 KB a (row, head), 3.25 GB and
// 458 us for 256 rows of 96 heads, 7.0 TB/s, the rate of a copy. With n > 1 tokens a row the FP32 instructions
// of the later tokens add up (64 rows of 32 heads: 44 us for one token, 93 us for eight).
#include <climits>
#include <cstdarg>
#include <cstdio>

#include "kda_gdr.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace gdr {
namespace {

constexpr int kRecWarps = 2;  // warps a block, of the 8 of one (row, head): 458 us at B = 256 and 96 heads; 4: 463, 8: 642

// Decode: n tokens for each row.
template <typename T>
__global__ void __launch_bounds__(32 * kRecWarps)
gdr_decode_kernel(const __grid_constant__ Args p, int64_t n_units)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kRecWarps + (threadIdx.x >> 5);  // (row, head, 16 columns)
    if (unit >= n_units) return;
    const int cb = (int)(unit & 7);
    const int64_t rh = unit >> 3;
    const int h = (int)(rh % p.H), row = (int)(rh / p.H);
    int src, dst;
    if (!slots_ok(p, row, src, dst)) {
        if (lane == 0) set_err(p.err);
        return;
    }
    walk_tokens<T>(p, src, dst, h, cb, (int64_t)row * p.n, p.n);
}

// FP32 prefill: the same walk over whole sequences. A block has half of a (sequence, head); its rows come by
// eight tokens through a ring of three stages in shared memory, two ahead. What is the same for every column
// of a token (the gates, the norms, k . q) each warp works out for eight tokens at once, four lanes a token.
// Bound by the latency of a token's chain (two sums over the rows, an exchange, the update): 0.36 us a token
// (three sequences of up to 1024 tokens, 8 heads: 371 us; 744 us with every warp loading its own rows).
constexpr int kStep = 8, kSeqStages = 3;
constexpr int kSqK = 0, kSqQ = kStep * 512, kSqV = 2 * kStep * 512, kSqA = kSqV + kStep * 256, kSqB = kSqA + kStep * 4;
constexpr int kSqStage = kSqB + kStep * 4;

__global__ void __launch_bounds__(128)
gdr_sequence_kernel(const __grid_constant__ Args p)
{
    __shared__ __align__(16) unsigned char ring[kSeqStages][kSqStage];
    __shared__ __align__(16) float scal[4][kStep][8];  // per warp and token: alpha, beta, -beta alpha rk, rq alpha, rq rk k.q, rk
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = blockIdx.x & 1;
    const int h = (int)((blockIdx.x >> 1) % (unsigned)p.H), row = (int)((blockIdx.x >> 1) / (unsigned)p.H);
    const int rg = lane >> 2, cg = lane & 3, hk = h / p.G;
    int src, dst;
    // Every block looks at the whole cu_seqlens, so that one that is wrong anywhere leaves every sequence alone. (A
    // vote over the block in place of the shared word costs the walk below 32 registers, and a block an SM.)
    __shared__ int bad;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int s = tid; s < p.N; s += 128) {
        const int b = __ldg(p.cu + s), e = __ldg(p.cu + s + 1);
        if (!(b >= 0 && e >= b && e <= p.total_T && (s > 0 || b == 0) && (s < p.N - 1 || e == p.total_T))) bad = 1;
    }
    __syncthreads();
    const bool ok = bad == 0;
    const int64_t t0 = __ldg(p.cu + row), t1 = __ldg(p.cu + row + 1);
    if (!ok || !slots_ok(p, row, src, dst)) {  // the same for every thread
        if (tid == 0) set_err(p.err);
        return;
    }
    const int n = (int)(t1 - t0), steps = (n + kStep - 1) / kStep;
    const float *kg = static_cast<const float *>(p.rows.k) + (size_t)hk * kD + t0 * p.rows.k_stride;
    const float *qg = static_cast<const float *>(p.rows.q) + (size_t)hk * kD + t0 * p.rows.q_stride;
    const float *vg = static_cast<const float *>(p.rows.v) + (size_t)h * kD + 64 * half + t0 * p.rows.v_stride;
    const float *ag = static_cast<const float *>(p.rows.a) + h + t0 * p.rows.a_stride;
    const float *bg = static_cast<const float *>(p.rows.b) + h + t0 * p.rows.b_stride;
    auto fetch = [&](int st) {
        if (st < steps) {
            unsigned char *d = ring[st % kSeqStages];
            const int t = st * kStep, left = n - t;  // tokens past the end read the last one, and are not used
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = tid + 128 * i, r = x >> 5, c = x & 31, rr = t + min(r, left - 1);
                cp_async16(d + kSqK + r * 512 + c * 16, kg + rr * p.rows.k_stride + 4 * c, 16);
                cp_async16(d + kSqQ + r * 512 + c * 16, qg + rr * p.rows.q_stride + 4 * c, 16);
            }
            const int r = tid >> 4, rr = t + min(r, left - 1);
            cp_async16(d + kSqV + r * 256 + (tid & 15) * 16, vg + rr * p.rows.v_stride + 4 * (tid & 15), 16);
            if (tid < 2 * kStep) {
                const int r2 = tid & (kStep - 1), r3 = t + min(r2, left - 1);
                const float *g = tid < kStep ? ag + r3 * p.rows.a_stride : bg + r3 * p.rows.b_stride;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(d + (tid < kStep ? kSqA : kSqB) + 4 * r2)), "l"(g) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    fetch(1);
    const int col = 16 * warp + 4 * cg + (rg & 3);  // of this block's 64
    const size_t at = (size_t)(16 * rg) * kD + 64 * half + 16 * warp + 4 * cg;
    float4 s[16];
    load_state(s, p, src, h, at);
    const float expA = expf(__ldg(p.A_log + h)), dt_bias = __ldg(p.dt_bias + h);
    float *op = static_cast<float *>(p.rows.out) + (size_t)h * kD + 64 * half + col + t0 * p.rows.out_stride;
#pragma unroll 1
    for (int st = 0; st < steps; ++st) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // this stage has arrived; the one before it has been read
        fetch(st + 2);
        const unsigned char *d = ring[st % kSeqStages];
        const float *ks = reinterpret_cast<const float *>(d + kSqK), *qs = reinterpret_cast<const float *>(d + kSqQ);
        const float *vs = reinterpret_cast<const float *>(d + kSqV);
        {  // lane / 4: token, lane % 4: 32 of its elements (in an order that spreads the lanes over the banks)
            float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int x = rg * 128 + cg * 32 + 4 * ((i + lane) & 7);
                const float4 a = *reinterpret_cast<const float4 *>(ks + x), b = *reinterpret_cast<const float4 *>(qs + x);
                kk = fmaf(a.x, a.x, fmaf(a.y, a.y, fmaf(a.z, a.z, fmaf(a.w, a.w, kk))));
                qq = fmaf(b.x, b.x, fmaf(b.y, b.y, fmaf(b.z, b.z, fmaf(b.w, b.w, qq))));
                kq = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, kq))));
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                kk += __shfl_xor_sync(0xFFFFFFFFu, kk, o);
                qq += __shfl_xor_sync(0xFFFFFFFFu, qq, o);
                kq += __shfl_xor_sync(0xFFFFFFFFu, kq, o);
            }
            const float rk = p.l2norm ? rsqrtf(kk + p.l2_eps) : 1.f;
            const float rq = p.l2norm ? p.q_scale * rsqrtf(qq + p.l2_eps) : p.q_scale;
            const float alpha = expf(log_decay(reinterpret_cast<const float *>(d + kSqA)[rg], dt_bias, expA));
            const float beta = sigmoidf_(reinterpret_cast<const float *>(d + kSqB)[rg]);
            if (cg == 0) {
                *reinterpret_cast<float4 *>(scal[warp][rg]) = make_float4(alpha, beta, -beta * alpha * rk, rq * alpha);
                *reinterpret_cast<float2 *>(scal[warp][rg] + 4) = make_float2(rq * rk * kq, rk);
            }
            __syncwarp();
        }
        const int tn = min(kStep, n - st * kStep);
        float k[16], q[16];
        auto load = [&](int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(ks + t * 128 + 16 * rg + 4 * i);
                const float4 b = *reinterpret_cast<const float4 *>(qs + t * 128 + 16 * rg + 4 * i);
                k[4 * i] = a.x; k[4 * i + 1] = a.y; k[4 * i + 2] = a.z; k[4 * i + 3] = a.w;
                q[4 * i] = b.x; q[4 * i + 1] = b.y; q[4 * i + 2] = b.z; q[4 * i + 3] = b.w;
            }
        };
#pragma unroll 2
        for (int t = 0; t < tn; ++t) {
            load(t);
            const float4 c0 = *reinterpret_cast<const float4 *>(scal[warp][t]);
            const float2 c1 = *reinterpret_cast<const float2 *>(scal[warp][t] + 4);
            const float v = vs[t * 64 + col];
            float2 p01, p23, r01, r23;
            column_partials(s, k, q, p01, p23, r01, r23);
            float ps, rs;
            column_sums(p01, p23, r01, r23, lane, ps, rs);
            const float u = fmaf(c0.z, ps, c0.y * v);
            if (!(lane & 16)) op[(int64_t)(st * kStep + t) * p.rows.out_stride] = fmaf(c1.x, u, c0.w * rs);
            column_update(s, k, c0.x, c1.y * u, cg);
        }
        __syncwarp();  // the scalars have been read
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    store_state(s, p, dst, h, at);
}

thread_local char g_msg[256];

kda_status fail(kda_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return record_error(s, g_msg);
}

bool cfg_ok(const kda_gdr_config_t *c)
{
    if (!c) return fail(KDA_ERR_INVALID, "config is NULL"), false;
    if (c->num_heads < 1 || c->num_qk_heads < 1 || c->num_heads % c->num_qk_heads != 0)
        return fail(KDA_ERR_INVALID, "num_heads must be a positive multiple of num_qk_heads (got %d, %d)", c->num_heads,
                    c->num_qk_heads), false;
    if (c->num_heads > 65536) return fail(KDA_ERR_INVALID, "num_heads must be <= 65536 (got %d)", c->num_heads), false;
    if (c->head_dim != kD) return fail(KDA_ERR_INVALID, "head_dim must be %d (got %d)", kD, c->head_dim), false;
    if (c->io_dtype != KDA_F32 && c->io_dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID, "io_dtype must be KDA_F32 or KDA_BF16"), false;
    if (c->qk_l2norm && !(c->l2_eps > 0.f && c->l2_eps < INFINITY))
        return fail(KDA_ERR_INVALID, "l2_eps must be finite and > 0"), false;
    if (!(fabsf(c->q_scale) < INFINITY)) return fail(KDA_ERR_INVALID, "q_scale must be finite"), false;
    return true;
}

bool row_ok(const char *name, const void *ptr, int64_t stride, int64_t width, int64_t T, int esize, bool vec)
{
    if (!ptr) return fail(KDA_ERR_INVALID, "%s is NULL", name), false;
    if (T > 1 && stride < width)
        return fail(KDA_ERR_INVALID, "%s_stride must be >= %lld (got %lld)", name, (long long)width, (long long)stride), false;
    if (stride < 0 || stride > ((int64_t)1 << 38))
        return fail(KDA_ERR_INVALID, "%s_stride out of range (%lld)", name, (long long)stride), false;
    const uintptr_t u = reinterpret_cast<uintptr_t>(ptr);
    if (u % (vec ? 16 : esize)) return fail(KDA_ERR_INVALID, "%s must be %d-byte aligned", name, vec ? 16 : esize), false;
    if (vec && (stride * esize) % 16)
        return fail(KDA_ERR_INVALID, "%s_stride must be a multiple of %d elements (got %lld)", name, 16 / esize,
                    (long long)stride), false;
    return true;
}

// Everything but the token counts. T: rows of q, k, v, a, b and out.
bool call_ok(const kda_gdr_config_t *c, const kda_gdr_params *prm, const float *S, int32_t max_slots,
             const int32_t *src, const int32_t *dst, const kda_gdr_rows *r, int64_t T)
{
    if (!prm || !prm->A_log || !prm->dt_bias) return fail(KDA_ERR_INVALID, "params (or one of its pointers) is NULL"), false;
    if (!S || (reinterpret_cast<uintptr_t>(S) & 15u)) return fail(KDA_ERR_INVALID, "S is NULL or not 16-byte aligned"), false;
    if (max_slots < 1) return fail(KDA_ERR_INVALID, "max_slots must be >= 1 (got %d)", max_slots), false;
    if (!src || !dst) return fail(KDA_ERR_INVALID, "src_slots or dst_slots is NULL"), false;
    if (!r) return fail(KDA_ERR_INVALID, "rows is NULL"), false;
    if (T == 0) return true;
    const int e = c->io_dtype == KDA_BF16 ? 2 : 4;
    const int64_t Dk = (int64_t)c->num_qk_heads * kD, Dv = (int64_t)c->num_heads * kD;
    return row_ok("q", r->q, r->q_stride, Dk, T, e, true) && row_ok("k", r->k, r->k_stride, Dk, T, e, true) &&
           row_ok("v", r->v, r->v_stride, Dv, T, e, true) && row_ok("a", r->a, r->a_stride, c->num_heads, T, e, false) &&
           row_ok("b", r->b, r->b_stride, c->num_heads, T, e, false) && row_ok("out", r->out, r->out_stride, Dv, T, e, true);
}

Args make_args(const kda_gdr_config_t *c, const kda_gdr_params *prm, float *S, int32_t max_slots, const int32_t *src,
               const int32_t *dst, int32_t N, const kda_gdr_rows *r, int32_t *err)
{
    Args p;
    p.S = S; p.max_slots = max_slots; p.src = src; p.dst = dst; p.err = err;
    p.cu = nullptr; p.N = N; p.n = 0; p.total_T = 0;
    p.H = c->num_heads; p.G = c->num_heads / c->num_qk_heads;
    p.A_log = prm->A_log; p.dt_bias = prm->dt_bias;
    p.rows = *r;
    p.l2norm = c->qk_l2norm != 0; p.l2_eps = c->l2_eps; p.q_scale = c->q_scale;
    return p;
}

// host cu_seqlens: total chunks (or -1 with the error set), and those of the longest sequence
int64_t count_chunks(const int32_t *cu, int32_t N, int64_t *longest = nullptr)
{
    if (cu[0] != 0) return fail(KDA_ERR_INVALID, "cu_seqlens[0] must be 0 (got %d)", cu[0]), -1;
    int64_t n = 0;
    for (int32_t i = 0; i < N; ++i) {
        if (cu[i + 1] < cu[i]) return fail(KDA_ERR_INVALID, "cu_seqlens decreases at %d", i + 1), -1;
        const int64_t c = ((int64_t)cu[i + 1] - cu[i] + kC - 1) / kC;
        n += c;
        if (longest && c > *longest) *longest = c;
    }
    return n;
}

}  // namespace

cudaError_t launch_decode_rows(const Args &p, bool f32, cudaStream_t stream)
{
    const int64_t units = (int64_t)p.N * p.H * (kD / 16);
    const unsigned grid = (unsigned)((units + kRecWarps - 1) / kRecWarps);
    if (f32) gdr_decode_kernel<float><<<grid, 32 * kRecWarps, 0, stream>>>(p, units);
    else gdr_decode_kernel<__nv_bfloat16><<<grid, 32 * kRecWarps, 0, stream>>>(p, units);
    return cudaGetLastError();
}

cudaError_t launch_sequences(const Args &p, cudaStream_t stream)
{
    gdr_sequence_kernel<<<(unsigned)((int64_t)p.N * p.H * 2), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdr
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_gdr_config(kda_gdr_config_t *cfg, int32_t num_heads, int32_t num_qk_heads, int32_t head_dim,
                          int32_t io_dtype)
{
    if (!cfg) return gdr::fail(KDA_ERR_INVALID, "cfg is NULL");
    kda_gdr_config_t c;
    c.num_heads = num_heads;
    c.num_qk_heads = num_qk_heads;
    c.head_dim = head_dim;
    c.io_dtype = io_dtype;
    c.qk_l2norm = 1;
    c.l2_eps = 1e-6f;
    c.q_scale = 0.08838834764831845f;  // 128^-1/2
    if (!gdr::cfg_ok(&c)) return KDA_ERR_INVALID;
    *cfg = c;
    return KDA_OK;
}

kda_status kda_gdr_decode(const kda_gdr_config_t *cfg, const kda_gdr_params *params, float *S, int32_t max_slots,
                          const int32_t *src_slots, const int32_t *dst_slots, int32_t B, int32_t n,
                          const kda_gdr_rows *rows, int32_t *err, void *stream)
{
    if (!gdr::cfg_ok(cfg)) return KDA_ERR_INVALID;
    if (B < 0) return gdr::fail(KDA_ERR_INVALID, "B must be >= 0 (got %d)", B);
    if (n < 1 || n > KDA_DECODE_MAX_TOKENS)
        return gdr::fail(KDA_ERR_INVALID, "n must be in 1 .. %d (got %d)", KDA_DECODE_MAX_TOKENS, n);
    if (B == 0) return KDA_OK;
    if ((int64_t)B * cfg->num_heads > INT_MAX / 8) return gdr::fail(KDA_ERR_INVALID, "B * num_heads is too large");
    if (!gdr::call_ok(cfg, params, S, max_slots, src_slots, dst_slots, rows, (int64_t)B * n)) return KDA_ERR_INVALID;
    gdr::Args p = gdr::make_args(cfg, params, S, max_slots, src_slots, dst_slots, B, rows, err);
    p.n = n;
    p.total_T = (int64_t)B * n;
    const cudaError_t e = gdr::launch_decode_rows(p, cfg->io_dtype == KDA_F32, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : gdr::fail(KDA_ERR_CUDA, "kda_gdr_decode: %s", cudaGetErrorString(e));
}

size_t kda_gdr_workspace_bytes(const kda_gdr_config_t *cfg, const int32_t *cu_seqlens_host, int32_t N)
{
    if (!gdr::cfg_ok(cfg)) return 0;
    if (N < 0 || (N > 0 && !cu_seqlens_host)) return gdr::fail(KDA_ERR_INVALID, "cu_seqlens_host is NULL or N < 0"), 0;
    if (N == 0 || cfg->io_dtype == KDA_F32) return 256;
    const int64_t nc = gdr::count_chunks(cu_seqlens_host, N);
    return nc < 0 ? 0 : gdr::chunked_workspace_bytes(nc, cfg->num_heads);
}

kda_status kda_gdr_prefill(const kda_gdr_config_t *cfg, const kda_gdr_params *params, float *S, int32_t max_slots,
                           const int32_t *src_slots, const int32_t *dst_slots, const int32_t *cu_seqlens,
                           const int32_t *cu_seqlens_host, int32_t N, const kda_gdr_rows *rows, void *workspace,
                           size_t workspace_bytes, int32_t *err, void *stream)
{
    if (!gdr::cfg_ok(cfg)) return KDA_ERR_INVALID;
    if (N < 0) return gdr::fail(KDA_ERR_INVALID, "N must be >= 0 (got %d)", N);
    if (N == 0) return KDA_OK;
    if (!cu_seqlens || !cu_seqlens_host) return gdr::fail(KDA_ERR_INVALID, "cu_seqlens or cu_seqlens_host is NULL");
    if ((int64_t)N * cfg->num_heads > INT_MAX / 8) return gdr::fail(KDA_ERR_INVALID, "N * num_heads is too large");
    int64_t longest = 0;
    const int64_t nc = gdr::count_chunks(cu_seqlens_host, N, &longest);
    if (nc < 0) return KDA_ERR_INVALID;
    if (nc * cfg->num_heads > INT_MAX / 8) return gdr::fail(KDA_ERR_INVALID, "chunks * num_heads is too large");
    const int64_t T = cu_seqlens_host[N];
    if (!gdr::call_ok(cfg, params, S, max_slots, src_slots, dst_slots, rows, T)) return KDA_ERR_INVALID;
    gdr::Args p = gdr::make_args(cfg, params, S, max_slots, src_slots, dst_slots, N, rows, err);
    p.cu = cu_seqlens;
    p.total_T = T;
    cudaError_t e;
    if (cfg->io_dtype == KDA_F32) {
        e = gdr::launch_sequences(p, static_cast<cudaStream_t>(stream));
    } else {
        const size_t need = gdr::chunked_workspace_bytes(nc, cfg->num_heads);
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need)
            return gdr::fail(KDA_ERR_INVALID, "workspace is NULL, not 16-byte aligned, or holds %zu bytes of %zu needed",
                             workspace_bytes, need);
        int dev = 0, sms = 0;
        if ((e = current_sms(&dev, &sms)) == cudaSuccess)
            e = gdr::launch_chunked(p, nc, longest, workspace, dev, sms, static_cast<cudaStream_t>(stream));
    }
    return e == cudaSuccess ? KDA_OK : gdr::fail(KDA_ERR_CUDA, "kda_gdr_prefill: %s", cudaGetErrorString(e));
}

}  // extern "C"
