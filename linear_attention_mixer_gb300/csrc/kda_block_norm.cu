// kda_block_norm.cu - the norms around a block of a stack, fused with its residual: from the stream x and the block's
// output y
//   x' = x + scale sigmoid(g) post_w y / rms(y),  h = pre_w x' / rms(x'),  rms(z) = sqrt(mean(z^2) + eps)
// h (the next block's input) in the rows' type or in E4M3 with a power-of-two scale for each 128 columns. And the
// gradients of that.
#include <climits>
#include <cstdarg>
#include <cstdio>

#include "kda_colsum.cuh"
#include "kda_internal.cuh"
#include "kda_launch.cuh"
#include "kda_ptx.cuh"
#include "kda_q8.cuh"

namespace kda {
namespace bn {
namespace {

struct Args {
    int64_t M;
    int32_t D;
    float eps;
    const float *post_w, *scale, *pre_w;
    kda_block_norm_rows r;
};
struct BackArgs {
    int64_t M;
    int32_t D;
    float eps;
    const float *post_w, *scale, *pre_w;
    kda_block_norm_grad_rows r;
    float *part;  // [parts][2][D]
};

// 8 channels of a row
template <typename T> struct V8;
template <> struct V8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const void *p, int64_t at) { r = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at)); }
    __device__ __forceinline__ float2 get(int i) const
    {
        const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(int i, float2 f)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        (i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w) = *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ __forceinline__ void store(void *p, int64_t at) const { *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at) = r; }
};
template <> struct V8<float> {
    float4 r[2];
    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        r[0] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at));
        r[1] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at) + 1);
    }
    __device__ __forceinline__ float2 get(int i) const { return i & 1 ? make_float2(r[i >> 1].z, r[i >> 1].w) : make_float2(r[i >> 1].x, r[i >> 1].y); }
    __device__ __forceinline__ void set(int i, float2 f)
    {
        if (i & 1) r[i >> 1].z = f.x, r[i >> 1].w = f.y;
        else r[i >> 1].x = f.x, r[i >> 1].y = f.y;
    }
    __device__ __forceinline__ void store(void *p, int64_t at) const
    {
        reinterpret_cast<float4 *>(static_cast<float *>(p) + at)[0] = r[0];
        reinterpret_cast<float4 *>(static_cast<float *>(p) + at)[1] = r[1];
    }
};
// A row of FP32 channels need not be a multiple of 8: its last vector then has 4.
template <typename T> __device__ __forceinline__ void load8(V8<T> &v, const void *p, int64_t at, int c, int D) { v.load(p, at); }
template <> __device__ __forceinline__ void load8(V8<float> &v, const void *p, int64_t at, int c, int D)
{
    v.r[0] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at));
    v.r[1] = c + 4 < D ? __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
}
template <typename T> __device__ __forceinline__ void store8(const V8<T> &v, void *p, int64_t at, int c, int D) { v.store(p, at); }
template <> __device__ __forceinline__ void store8(const V8<float> &v, void *p, int64_t at, int c, int D)
{
    reinterpret_cast<float4 *>(static_cast<float *>(p) + at)[0] = v.r[0];
    if (c + 4 < D) reinterpret_cast<float4 *>(static_cast<float *>(p) + at)[1] = v.r[1];
}
// 8 parameters from channel c on (0 past the end)
struct W8 {
    float4 r[2];
    __device__ __forceinline__ void load(const float *p, int c, int D)
    {
        r[0] = __ldg(reinterpret_cast<const float4 *>(p + c));
        r[1] = c + 4 < D ? __ldg(reinterpret_cast<const float4 *>(p + c) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ float2 get(int i) const { return i & 1 ? make_float2(r[i >> 1].z, r[i >> 1].w) : make_float2(r[i >> 1].x, r[i >> 1].y); }
};

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 sigmoid2(float2 g) { return make_float2(sigmoid_ftz(g.x), sigmoid_ftz(g.y)); }

// Sums over the NT threads that have a row; each thread gets them. A block of more than one warp has one row.
template <int NT, int K>
__device__ __forceinline__ void row_sum(float (&s)[K], float (*sh)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = warp_sum(s[k]);
    if (NT == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) sh[warp][k] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v = lane < NT / 32 ? sh[lane][k] : 0.f;
#pragma unroll
        for (int o = NT / 64; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        s[k] = __shfl_sync(0xFFFFFFFFu, v, 0);
    }
}

template <typename T, int NT, int VPT, bool F8>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) block_norm_kernel(const __grid_constant__ Args p)
{
    constexpr int kRows = NT == 32 ? 4 : 1;
    __shared__ float sh[2][32][1];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * kRows + (NT == 32 ? threadIdx.x >> 5 : 0);
    if (row >= p.M) return;  // a whole warp
    V8<T> x[VPT], y[VPT], g[VPT];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (tid + i * NT);
        if (c < p.D) {
            load8(x[i], p.r.x, row * p.r.x_stride + c, c, p.D);
            if (p.r.y) load8(y[i], p.r.y, row * p.r.y_stride + c, c, p.D);
            if (p.r.g) load8(g[i], p.r.g, row * p.r.g_stride + c, c, p.D);
        }
    }
    const float inv_D = 1.f / p.D;
    if (p.r.y) {
        float2 q = f2(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (8 * (tid + i * NT) < p.D)
#pragma unroll
                for (int j = 0; j < 4; ++j) q = f2_fma(y[i].get(j), y[i].get(j), q);
        s[0] = q.x + q.y;
        row_sum<NT, 1>(s, sh[0]);
    }
    const float ry = rsqrtf(fmaf(s[0], inv_D, p.eps));
    float2 f[VPT][4], q = f2(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (tid + i * NT);
        if (c >= p.D) continue;
        W8 w, sc;
        if (p.r.y) w.load(p.post_w, c, p.D), sc.load(p.scale, c, p.D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[i][j] = x[i].get(j);
            if (p.r.y) {
                float2 t = f2_mul(sc.get(j), f2_mul(w.get(j), f2_mul(y[i].get(j), f2(ry))));
                if (p.r.g) t = f2_mul(t, sigmoid2(g[i].get(j)));
                f[i][j] = f2_add(f[i][j], t);
                x[i].set(j, f[i][j]);
            }
            q = f2_fma(f[i][j], f[i][j], q);
        }
        if (p.r.x_out) store8(x[i], p.r.x_out, row * p.r.x_out_stride + c, c, p.D);
    }
    if (!p.r.h) return;
    s[0] = q.x + q.y;
    row_sum<NT, 1>(s, sh[1]);
    const float rx = rsqrtf(fmaf(s[0], inv_D, p.eps));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (tid + i * NT);
        if (!F8 && c >= p.D) continue;
        W8 w;
        if (c < p.D) w.load(p.pre_w, c, p.D);
        if (!F8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i].set(j, f2_mul(w.get(j), f2_mul(f[i][j], f2(rx))));
            store8(x[i], p.r.h, row * p.r.h_stride + c, c, p.D);
        } else {  // 16 lanes have 128 columns; every lane of the warp takes part
            Q8<float> v;
            v.zero();
            if (c < p.D) {
                float2 o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = f2_mul(w.get(j), f2_mul(f[i][j], f2(rx)));
                v.r[0] = make_uint4(__float_as_uint(o[0].x), __float_as_uint(o[0].y), __float_as_uint(o[1].x), __float_as_uint(o[1].y));
                v.r[1] = make_uint4(__float_as_uint(o[2].x), __float_as_uint(o[2].y), __float_as_uint(o[3].x), __float_as_uint(o[3].y));
            }
            uint32_t m = q8_max(v);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const bool odd = m >= kQInf;
            if (__any_sync(0xFFFFFFFFu, odd)) {
                m = q8_max_finite(v);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            }
            float sc, inv;
            q8_scale(m, sc, inv);
            if (c < p.D) {
                *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.r.h) + row * p.r.h_stride + c) = q8_codes(v, inv, odd);
                if ((threadIdx.x & 15) == 0) p.r.hs[row * ((p.D + kQb - 1) / kQb) + c / kQb] = sc;
            }
        }
    }
}

// Gradients, a row at a time: with n = z / rms(z) a norm's gradient is dz = (w - n mean(w n)) / rms(z), w that of n.
//   dx = dx' + (gradient of h's norm),  d(scale sigmoid(g) post_w n_y) = dx
// A thread keeps its columns' sums over the block's rows.
template <typename T, int NT, int VPT>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) block_norm_back_kernel(const __grid_constant__ BackArgs p, int parts)
{
    constexpr int kRows = NT == 32 ? 4 : 1;
    __shared__ float sh[2][32][3], sh1[2][32][1];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int part = blockIdx.x * kRows + (NT == 32 ? threadIdx.x >> 5 : 0);
    if (part >= parts) return;
    float2 sq[VPT][4], sp[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sq[i][j] = sp[i][j] = f2(0.f);
    const float inv_D = 1.f / p.D;
    const bool has_y = p.r.y, has_g = p.r.g, has_h = p.r.dh, has_dx1 = p.r.dx1;
    int turn = 0;
    for (int64_t row = part; row < p.M; row += parts, turn ^= 1) {
        V8<T> x[VPT], dh[VPT], dx1[VPT], y[VPT], g[VPT];
        float s[3] = {0.f, 0.f, 0.f};  // x^2, x dh pre_w, y^2
        float2 s0 = f2(0.f), s1 = s0, s2 = s0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (tid + i * NT);
            if (c >= p.D) continue;
            if (has_h) {
                load8(x[i], p.r.x_out, row * p.r.x_out_stride + c, c, p.D);
                load8(dh[i], p.r.dh, row * p.r.dh_stride + c, c, p.D);
            }
            if (has_dx1) load8(dx1[i], p.r.dx1, row * p.r.dx1_stride + c, c, p.D);
            if (has_y) load8(y[i], p.r.y, row * p.r.y_stride + c, c, p.D);
            if (has_g) load8(g[i], p.r.g, row * p.r.g_stride + c, c, p.D);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (tid + i * NT);
            if (c >= p.D) continue;
            W8 w;
            if (has_h) w.load(p.pre_w, c, p.D);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (has_h) {
                    s0 = f2_fma(x[i].get(j), x[i].get(j), s0);
                    s1 = f2_fma(f2_mul(dh[i].get(j), w.get(j)), x[i].get(j), s1);
                }
                if (has_y) s2 = f2_fma(y[i].get(j), y[i].get(j), s2);
            }
        }
        s[0] = s0.x + s0.y, s[1] = s1.x + s1.y, s[2] = s2.x + s2.y;
        row_sum<NT, 3>(s, sh[turn]);
        const float rx = rsqrtf(fmaf(s[0], inv_D, p.eps)), ry = rsqrtf(fmaf(s[2], inv_D, p.eps));
        const float mx = s[1] * rx * inv_D;  // mean(w n)
        float2 m = f2(0.f), d[VPT][4];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (tid + i * NT);
            if (c >= p.D) continue;
            W8 w, pw, sc;
            if (has_h) w.load(p.pre_w, c, p.D);
            if (has_y) pw.load(p.post_w, c, p.D), sc.load(p.scale, c, p.D);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[i][j] = has_dx1 ? dx1[i].get(j) : f2(0.f);
                if (has_h) {
                    const float2 n = f2_mul(x[i].get(j), f2(rx)), e = dh[i].get(j);
                    d[i][j] = f2_fma(f2(rx), f2_fma(n, f2(-mx), f2_mul(e, w.get(j))), d[i][j]);
                    sp[i][j] = f2_fma(e, n, sp[i][j]);
                }
                x[i].set(j, d[i][j]);
                if (has_y) {
                    const float2 n = f2_mul(y[i].get(j), f2(ry));
                    float2 k = d[i][j];
                    if (has_g) k = f2_mul(k, sigmoid2(g[i].get(j)));
                    sq[i][j] = f2_fma(k, n, sq[i][j]);
                    d[i][j] = f2_mul(k, f2_mul(sc.get(j), pw.get(j)));  // the gradient of n
                    m = f2_fma(d[i][j], n, m);
                }
            }
            store8(x[i], p.r.dx, row * p.r.dx_stride + c, c, p.D);
        }
        if (!has_y) continue;
        float t[1] = {m.x + m.y};
        row_sum<NT, 1>(t, sh1[turn]);
        const float my = t[0] * inv_D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (tid + i * NT);
            if (c >= p.D) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 n = f2_mul(y[i].get(j), f2(ry));
                if (has_g) {  // d sigmoid = s (1 - s); d[i][j] has a factor s
                    const float2 gg = g[i].get(j), o = sigmoid2(make_float2(-gg.x, -gg.y));
                    g[i].set(j, f2_mul(f2_mul(d[i][j], n), o));
                }
                y[i].set(j, f2_mul(f2(ry), f2_fma(n, f2(-my), d[i][j])));
            }
            store8(y[i], p.r.dy, row * p.r.dy_stride + c, c, p.D);
            if (has_g) store8(g[i], p.r.dg, row * p.r.dg_stride + c, c, p.D);
        }
    }
    float *out = p.part + (int64_t)part * 2 * p.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (tid + i * NT);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + 2 * j < p.D) {
                *reinterpret_cast<float2 *>(out + c + 2 * j) = sq[i][j];
                *reinterpret_cast<float2 *>(out + p.D + c + 2 * j) = sp[i][j];
            }
    }
}

__global__ void __launch_bounds__(kSumCols *kSumGroups)
block_norm_sums_kernel(const float *part, int parts, int D, const float *post_w, const float *scale, float *dpost_w, float *dscale, float *dpre_w)
{
    __shared__ float sh[kSumGroups][kSumCols];
    if (blockIdx.y == 0 ? !dpost_w && !dscale : !dpre_w) return;
    const float s = column_sum(part + (int64_t)blockIdx.y * D, parts, 2 * (int64_t)D, blockIdx.x * kSumCols, D, sh);
    const int c = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.y != 0 || c >= D) return;
    if (blockIdx.y == 1) {
        dpre_w[c] = s;
    } else {
        if (dpost_w) dpost_w[c] = s * scale[c];
        if (dscale) dscale[c] = s * post_w[c];
    }
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

bool cfg_ok(const kda_block_norm_config_t *c)
{
    if (!c) return fail(KDA_ERR_INVALID, "config is NULL"), false;
    if (c->io_dtype != KDA_F32 && c->io_dtype != KDA_BF16) return fail(KDA_ERR_INVALID, "io_dtype must be KDA_F32 or KDA_BF16"), false;
    const int unit = c->io_dtype == KDA_BF16 ? 8 : 4;
    if (c->dim < unit || c->dim % unit || c->dim > KDA_BLOCK_NORM_MAX_DIM)
        return fail(KDA_ERR_INVALID, "dim must be a positive multiple of %d up to %d (got %d)", unit, KDA_BLOCK_NORM_MAX_DIM, c->dim), false;
    if (!(c->eps > 0.f && c->eps < INFINITY)) return fail(KDA_ERR_INVALID, "eps must be finite and > 0"), false;
    return true;
}

// rows of esize bytes a channel, 16-byte aligned (8-byte for E4M3)
bool row_ok(const char *name, const void *ptr, int64_t stride, int64_t M, int32_t D, int esize)
{
    const int align = esize == 1 ? 8 : 16;
    if (!ptr) return fail(KDA_ERR_INVALID, "%s is NULL", name), false;
    if (M > 1 && stride < D) return fail(KDA_ERR_INVALID, "%s_stride must be >= %d (got %lld)", name, D, (long long)stride), false;
    if (stride < 0 || stride > ((int64_t)1 << 38) || (stride > 0 && M > ((int64_t)1 << 60) / stride))
        return fail(KDA_ERR_INVALID, "%s_stride out of range (%lld)", name, (long long)stride), false;
    if (reinterpret_cast<uintptr_t>(ptr) % align) return fail(KDA_ERR_INVALID, "%s must be %d-byte aligned", name, align), false;
    if ((stride * esize) % align)
        return fail(KDA_ERR_INVALID, "%s_stride must be a multiple of %d elements (got %lld)", name, align / esize, (long long)stride), false;
    return true;
}

bool f32_ok(const char *name, const void *ptr)
{
    if (!ptr || (reinterpret_cast<uintptr_t>(ptr) & 15u)) return fail(KDA_ERR_INVALID, "%s is NULL or not 16-byte aligned", name), false;
    return true;
}
bool f32_or_null_ok(const char *name, const void *ptr) { return !ptr || f32_ok(name, ptr); }

bool rows_ok(int64_t M)
{
    if (M < 0 || M > INT_MAX) return fail(KDA_ERR_INVALID, "M must be in 0 .. %d (got %lld)", INT_MAX, (long long)M), false;
    return true;
}

int64_t parts_of(int32_t D, int64_t M)
{
    const int64_t most = D <= 512 ? 1216 : 304;
    return M < most ? M : most;
}
size_t back_bytes(int32_t D, int64_t M) { return 256 + (size_t)parts_of(D, M) * 2 * D * sizeof(float); }

template <typename T, bool F8>
void launch(const Args &p, cudaStream_t s)
{
    const unsigned M = (unsigned)p.M, M4 = (unsigned)((p.M + 3) / 4);
    if (p.D <= 256) block_norm_kernel<T, 32, 1, F8><<<M4, 128, 0, s>>>(p);
    else if (p.D <= 512) block_norm_kernel<T, 32, 2, F8><<<M4, 128, 0, s>>>(p);
    else if (p.D <= 1024) block_norm_kernel<T, 128, 1, F8><<<M, 128, 0, s>>>(p);
    else if (p.D <= 2048) block_norm_kernel<T, 128, 2, F8><<<M, 128, 0, s>>>(p);
    else if (p.D <= 4096) block_norm_kernel<T, 256, 2, F8><<<M, 256, 0, s>>>(p);
    else if (p.D <= 8192) block_norm_kernel<T, 512, 2, F8><<<M, 512, 0, s>>>(p);
    else block_norm_kernel<T, 1024, 2, F8><<<M, 1024, 0, s>>>(p);
}

template <typename T>
void launch_back(const BackArgs &p, int parts, cudaStream_t s)
{
    const unsigned n = (unsigned)parts, n4 = (unsigned)((parts + 3) / 4);
    if (p.D <= 256) block_norm_back_kernel<T, 32, 1><<<n4, 128, 0, s>>>(p, parts);
    else if (p.D <= 512) block_norm_back_kernel<T, 32, 2><<<n4, 128, 0, s>>>(p, parts);
    else if (p.D <= 1024) block_norm_back_kernel<T, 128, 1><<<n, 128, 0, s>>>(p, parts);
    else if (p.D <= 2048) block_norm_back_kernel<T, 128, 2><<<n, 128, 0, s>>>(p, parts);
    else if (p.D <= 4096) block_norm_back_kernel<T, 256, 2><<<n, 256, 0, s>>>(p, parts);
    else if (p.D <= 8192) block_norm_back_kernel<T, 512, 2><<<n, 512, 0, s>>>(p, parts);
    else block_norm_back_kernel<T, 1024, 2><<<n, 1024, 0, s>>>(p, parts);
}

}  // namespace
}  // namespace bn
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_block_norm_config(kda_block_norm_config_t *cfg, int32_t dim, int32_t io_dtype)
{
    if (!cfg) return bn::fail(KDA_ERR_INVALID, "cfg is NULL");
    const kda_block_norm_config_t c = {dim, io_dtype, 1e-6f};
    if (!bn::cfg_ok(&c)) return KDA_ERR_INVALID;
    *cfg = c;
    return KDA_OK;
}

kda_status kda_block_norm(const kda_block_norm_config_t *cfg, const kda_block_norm_params *params, int64_t M, const kda_block_norm_rows *rows,
                          void *stream)
{
    if (!bn::cfg_ok(cfg) || !bn::rows_ok(M)) return KDA_ERR_INVALID;
    if (M == 0) return KDA_OK;
    if (!params || !rows) return bn::fail(KDA_ERR_INVALID, "params or rows is NULL");
    const kda_block_norm_rows &r = *rows;
    const int32_t D = cfg->dim;
    const int e = cfg->io_dtype == KDA_BF16 ? 2 : 4;
    if (!bn::row_ok("x", r.x, r.x_stride, M, D, e)) return KDA_ERR_INVALID;
    if (r.y && (!bn::row_ok("y", r.y, r.y_stride, M, D, e) || !bn::row_ok("x_out", r.x_out, r.x_out_stride, M, D, e) ||
                !bn::f32_ok("post_w", params->post_w) || !bn::f32_ok("scale", params->scale))) return KDA_ERR_INVALID;
    if (!r.y && (r.g || r.x_out)) return bn::fail(KDA_ERR_INVALID, "g and x_out must be NULL without y");
    if (r.g && !bn::row_ok("g", r.g, r.g_stride, M, D, e)) return KDA_ERR_INVALID;
    if (!r.h && (r.hs || !r.y)) return bn::fail(KDA_ERR_INVALID, r.hs ? "h is NULL" : "y and h are both NULL");
    if (r.h && (!bn::row_ok("h", r.h, r.h_stride, M, D, r.hs ? 1 : e) || !bn::f32_ok("pre_w", params->pre_w))) return KDA_ERR_INVALID;
    if (r.hs && D % 16) return bn::fail(KDA_ERR_INVALID, "dim must be a multiple of 16 for E4M3 rows (got %d)", D);
    if (r.hs && (reinterpret_cast<uintptr_t>(r.hs) & 3u)) return bn::fail(KDA_ERR_INVALID, "hs must be 4-byte aligned");
    const bn::Args p = {M, D, cfg->eps, params->post_w, params->scale, params->pre_w, r};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cfg->io_dtype == KDA_F32) {
        if (r.hs) bn::launch<float, true>(p, s);
        else bn::launch<float, false>(p, s);
    } else {
        if (r.hs) bn::launch<__nv_bfloat16, true>(p, s);
        else bn::launch<__nv_bfloat16, false>(p, s);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? KDA_OK : bn::fail(KDA_ERR_CUDA, "kda_block_norm: %s", cudaGetErrorString(err));
}

size_t kda_block_norm_workspace_bytes(const kda_block_norm_config_t *cfg, int64_t M)
{
    if (!bn::cfg_ok(cfg) || !bn::rows_ok(M)) return 0;
    return bn::back_bytes(cfg->dim, M);
}

kda_status kda_block_norm_backward(const kda_block_norm_config_t *cfg, const kda_block_norm_params *params, int64_t M,
                                   const kda_block_norm_grad_rows *rows, float *dpost_w, float *dscale, float *dpre_w, void *workspace,
                                   size_t workspace_bytes, void *stream)
{
    if (!bn::cfg_ok(cfg) || !bn::rows_ok(M)) return KDA_ERR_INVALID;
    if (!params || !rows) return bn::fail(KDA_ERR_INVALID, "params or rows is NULL");
    if (!bn::f32_or_null_ok("dpost_w", dpost_w) || !bn::f32_or_null_ok("dscale", dscale) || !bn::f32_or_null_ok("dpre_w", dpre_w)) return KDA_ERR_INVALID;
    const kda_block_norm_grad_rows &r = *rows;
    const int32_t D = cfg->dim;
    const int e = cfg->io_dtype == KDA_BF16 ? 2 : 4;
    if ((dpost_w || dscale) && (!bn::f32_ok("post_w", params->post_w) || !bn::f32_ok("scale", params->scale))) return KDA_ERR_INVALID;
    if (M > 0) {
        if (!r.y && !r.dh) return bn::fail(KDA_ERR_INVALID, "y and dh are both NULL");
        if (!bn::row_ok("dx", r.dx, r.dx_stride, M, D, e)) return KDA_ERR_INVALID;
        if (r.dh && (!bn::row_ok("x_out", r.x_out, r.x_out_stride, M, D, e) || !bn::row_ok("dh", r.dh, r.dh_stride, M, D, e) ||
                     !bn::f32_ok("pre_w", params->pre_w))) return KDA_ERR_INVALID;
        if (r.dx1 && !bn::row_ok("dx1", r.dx1, r.dx1_stride, M, D, e)) return KDA_ERR_INVALID;
        if (r.y && (!bn::row_ok("y", r.y, r.y_stride, M, D, e) || !bn::row_ok("dy", r.dy, r.dy_stride, M, D, e) ||
                    !bn::f32_ok("post_w", params->post_w) || !bn::f32_ok("scale", params->scale))) return KDA_ERR_INVALID;
        if (!r.y && (r.g || r.dg || r.dy)) return bn::fail(KDA_ERR_INVALID, "g, dg and dy must be NULL without y");
        if (!r.g != !r.dg) return bn::fail(KDA_ERR_INVALID, "g and dg must both be given or both be NULL");
        if (r.g && (!bn::row_ok("g", r.g, r.g_stride, M, D, e) || !bn::row_ok("dg", r.dg, r.dg_stride, M, D, e))) return KDA_ERR_INVALID;
        const size_t need = bn::back_bytes(D, M);
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need)
            return bn::fail(KDA_ERR_INVALID, "workspace is NULL, not 16-byte aligned, or holds %zu bytes of %zu needed", workspace_bytes, need);
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int parts = (int)bn::parts_of(D, M);
    cudaError_t err = cudaSuccess;
    if (M > 0) {
        const bn::BackArgs p = {M, D, cfg->eps, params->post_w, params->scale, params->pre_w, r, static_cast<float *>(workspace)};
        if (cfg->io_dtype == KDA_F32) bn::launch_back<float>(p, parts, s);
        else bn::launch_back<__nv_bfloat16>(p, parts, s);
        err = cudaGetLastError();
    }
    if (err == cudaSuccess && (dpost_w || dscale || dpre_w)) {  // without rows: zeros
        bn::block_norm_sums_kernel<<<dim3((D + kSumCols - 1) / kSumCols, 2), dim3(kSumCols, kSumGroups), 0, s>>>(
            static_cast<const float *>(workspace), parts, D, params->post_w, params->scale, dpost_w, dscale, dpre_w);
        err = cudaGetLastError();
    }
    return err == cudaSuccess ? KDA_OK : bn::fail(KDA_ERR_CUDA, "kda_block_norm_backward: %s", cudaGetErrorString(err));
}

}  // extern "C"
