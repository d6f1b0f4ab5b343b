// kda_block_norm.cu - the norms around a block of a stack, fused with its residual: from the stream x and the block's
// output y
//   x' = x + scale sigmoid(g) post_w y / rms(y),  h = pre_w x' / rms(x'),  rms(z) = sqrt(mean(z^2) + eps)
// h (the next block's input) in the rows' type or in E4M3 with a power-of-two scale for each 128 columns. And the
// gradients of that.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kda_cluster.cuh"
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
    __device__ __forceinline__ W8 times(const W8 &o) const
    {
        return W8{{make_float4(r[0].x * o.r[0].x, r[0].y * o.r[0].y, r[0].z * o.r[0].z, r[0].w * o.r[0].w),
                   make_float4(r[1].x * o.r[1].x, r[1].y * o.r[1].y, r[1].z * o.r[1].z, r[1].w * o.r[1].w)}};
    }
};

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
// sigmoid(g) and 1 - sigmoid(g) = exp(-g) sigmoid(g), without the difference; where sigmoid(g) is 0 the second is not used
__device__ __forceinline__ float2 both_sigmoids(float2 g, float2 &ns)
{
    constexpr float kHuge = 8.507059173023462e37f;  // 2^126
    const float2 E = make_float2(exp_ftz(-g.x), exp_ftz(-g.y)), s = make_float2(rcp_ftz(1.f + E.x), rcp_ftz(1.f + E.y));
    ns = make_float2(fminf(E.x, kHuge) * s.x, fminf(E.y, kHuge) * s.y);
    return s;
}
__device__ __forceinline__ float2 sigmoid2(float2 g) { return make_float2(sigmoid_ftz(g.x), sigmoid_ftz(g.y)); }

// 1 / sqrt(sum / D + eps), rounded as well as FP32 can: it is one number a row, and every element's
__device__ __forceinline__ float rstd(float sum, int D, float eps) { return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)D), eps)); }

// v to where `mine` (shared memory) is in the other block of a cluster of two
__device__ __forceinline__ void st_other(const float *mine, float v)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(cluster_rank() ^ 1u));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// A thread's columns, 8 at first + 8 NT i up to end. A backward row of more than 8192 channels has a cluster of
// two blocks (CL), half the columns each: the parameters' sums of all of them find no room in one SM's registers.
constexpr int kWide = 8192;
template <int CL>
struct Cols {
    int first, end;
    __device__ __forceinline__ Cols(int tid, int D) : first(8 * tid), end(D)
    {
        if (CL == 1) return;
        const int half = (D / 2 + 7) & ~7;
        if (cluster_rank() == 0) end = half;
        else first += half;
    }
};

// Sums over the NT threads (of each block of the cluster) that have a row; each thread gets them. A block of more than one warp
// has one row. Blocks of a cluster put their sums into both and meet: what follows finds all of them, and neither ends before
// the other has written.
template <int NT, int CL, int K>
__device__ __forceinline__ void row_sum(float (&s)[K], float (*sh)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = warp_sum(s[k]);
    if (NT == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = CL == 1 ? warp : (int)cluster_rank() * (NT / 32) + warp;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            sh[slot][k] = s[k];
            if (CL == 2) st_other(&sh[slot][k], s[k]);
        }
    if (CL == 1) {
        __syncthreads();
    } else {
        cluster_arrive();
        cluster_wait();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v = lane < CL * NT / 32 ? sh[lane][k] : 0.f;
#pragma unroll
        for (int o = CL * NT / 64; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        s[k] = __shfl_sync(0xFFFFFFFFu, v, 0);
    }
}

// What rows a call has: known to the compiler where it has all of them (kAll with a gate, kNoGate without), else asked (kAny).
enum { kAny, kNoGate, kAll };

// What is done to a row once its channels are in registers. W: pairs of the parameters of vector i: post_w times scale, and
// pre_w. sh: room for two sums a warp.
template <int HAS, typename T, int NT, int VPT, bool F8, typename PostW, typename PreW>
__device__ __forceinline__ void finish_row(const Args &p, int64_t row, const Cols<1> &cols, V8<T> (&x)[VPT], const V8<T> (&y)[VPT], const V8<T> (&g)[VPT],
                                           float (*sh0)[1], float (*sh1)[1], PostW post_w, PreW pre_w)
{
    const bool has_y = HAS != kAny || p.r.y, has_g = HAS == kAny ? p.r.g != nullptr : HAS == kAll, has_h = HAS != kAny || p.r.h;
    float s[1] = {0.f};
    float2 q = f2(0.f);
    if (has_y) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (cols.first + 8 * NT * i < cols.end)
#pragma unroll
                for (int j = 0; j < 4; ++j) q = f2_fma(y[i].get(j), y[i].get(j), q);
        s[0] = q.x + q.y;
        row_sum<NT, 1>(s, sh0);
    }
    const float ry = rstd(s[0], p.D, p.eps);
    float2 f[VPT][4];
    q = f2(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (c >= cols.end) continue;
        W8 w;
        if (has_y) w = post_w(i, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[i][j] = x[i].get(j);
            if (has_y) {
                float2 t = f2_mul(w.get(j), f2_mul(y[i].get(j), f2(ry)));
                if (has_g) t = f2_mul(t, sigmoid2(g[i].get(j)));
                f[i][j] = f2_add(f[i][j], t);
                x[i].set(j, f[i][j]);
            }
            q = f2_fma(f[i][j], f[i][j], q);
        }
        if (has_y) store8(x[i], p.r.x_out, row * p.r.x_out_stride + c, c, p.D);
    }
    if (!has_h) return;
    s[0] = q.x + q.y;
    row_sum<NT, 1>(s, sh1);
    const float rx = rstd(s[0], p.D, p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (!F8 && c >= cols.end) continue;
        W8 w;
        if (c < cols.end) w = pre_w(i, c);
        if (!F8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i].set(j, f2_mul(w.get(j), f2_mul(f[i][j], f2(rx))));
            store8(x[i], p.r.h, row * p.r.h_stride + c, c, p.D);
        } else {  // 16 lanes have 128 columns; every lane of the warp takes part
            Q8<float> v;
            v.zero();
            if (c < cols.end) {
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
            if (c < cols.end) {
                *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.r.h) + row * p.r.h_stride + c) = q8_codes(v, inv, odd);
                if ((threadIdx.x & 15) == 0) p.r.hs[row * ((p.D + kQb - 1) / kQb) + c / kQb] = sc;
            }
        }
    }
}

// One row a block (a warp of four for the shortest rows).
template <typename T, int NT, int VPT, bool F8>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) block_norm_kernel(const __grid_constant__ Args p)
{
    constexpr int kRows = NT == 32 ? 4 : 1;
    __shared__ float sh[2][32][1];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * kRows + (NT == 32 ? threadIdx.x >> 5 : 0);
    if (row >= p.M) return;  // a whole warp
    const Cols<1> cols(tid, p.D);
    V8<T> x[VPT], y[VPT], g[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (c < cols.end) {
            load8(x[i], p.r.x, row * p.r.x_stride + c, c, p.D);
            if (p.r.y) load8(y[i], p.r.y, row * p.r.y_stride + c, c, p.D);
            if (p.r.g) load8(g[i], p.r.g, row * p.r.g_stride + c, c, p.D);
        }
    }
    finish_row<kAny, T, NT, VPT, F8>(p, row, cols, x, y, g, sh[0], sh[1],
        [&](int, int c) {
            W8 w, sc;
            w.load(p.post_w, c, p.D), sc.load(p.scale, c, p.D);
            return w.times(sc);
        },
        [&](int, int c) {
            W8 w;
            w.load(p.pre_w, c, p.D);
            return w;
        });
}

// Many rows: blocks that stay, with the parameters in shared memory (from L2 they are as many bytes as the rows), and
// with the next row on its way into shared memory while one is worked on. A thread copies, and reads, its own columns.
template <typename T, int NT, int VPT>
struct Stage {
    float4 w[4][VPT][NT];                        // post_w scale, pre_w: four channels each
    V8<T> rows[3][VPT][NT];                      // x, y, g
};
template <typename T> __device__ __forceinline__ void copy8(V8<T> *to, const void *p, int64_t at, int c, int D)
{
    cp_async16(&to->r, static_cast<const T *>(p) + at, 16);
}
template <> __device__ __forceinline__ void copy8(V8<float> *to, const void *p, int64_t at, int c, int D)
{
    const float *from = static_cast<const float *>(p) + at;
    cp_async16(&to->r[0], from, 16);
    cp_async16(&to->r[1], c + 4 < D ? from + 4 : from, c + 4 < D ? 16 : 0);
}

template <typename T, int NT, int VPT, bool F8, int HAS>
__global__ void __launch_bounds__(NT, 512 / NT) block_norm_rows_kernel(const __grid_constant__ Args p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    Stage<T, NT, VPT> &st = *reinterpret_cast<Stage<T, NT, VPT> *>(smem);
    __shared__ float sh[2][2][32][1];
    const int tid = threadIdx.x;
    const Cols<1> cols(tid, p.D);
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = cols.first + 8 * NT * i;
            if (c >= cols.end) continue;
            copy8(&st.rows[0][i][tid], p.r.x, row * p.r.x_stride + c, c, p.D);
            copy8(&st.rows[1][i][tid], p.r.y, row * p.r.y_stride + c, c, p.D);
            if (HAS == kAll) copy8(&st.rows[2][i][tid], p.r.g, row * p.r.g_stride + c, c, p.D);
        }
    };
    fetch(blockIdx.x);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (c >= cols.end) continue;
        W8 w, sc;
        w.load(p.post_w, c, p.D), sc.load(p.scale, c, p.D);
        w = w.times(sc);
        st.w[0][i][tid] = w.r[0], st.w[1][i][tid] = w.r[1];
        w.load(p.pre_w, c, p.D);
        st.w[2][i][tid] = w.r[0], st.w[3][i][tid] = w.r[1];
    }
    int turn = 0;
#pragma unroll 1
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
        V8<T> x[VPT], y[VPT], g[VPT];
        cp_async_wait_all();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            x[i] = st.rows[0][i][tid];
            y[i] = st.rows[1][i][tid];
            if (HAS == kAll) g[i] = st.rows[2][i][tid];
        }
        if (row + gridDim.x < p.M) fetch(row + gridDim.x);
        finish_row<HAS, T, NT, VPT, F8>(p, row, cols, x, y, g, sh[turn][0], sh[turn][1],
            [&](int i, int) { return W8{{st.w[0][i][tid], st.w[1][i][tid]}}; }, [&](int i, int) { return W8{{st.w[2][i][tid], st.w[3][i][tid]}}; });
    }
}

// Gradients, a row at a time: with n = z / rms(z) a norm's gradient is dz = (w - n mean(w n)) / rms(z), w that of n.
//   dx = dx' + (gradient of h's norm),  d(scale sigmoid(g) post_w n_y) = dx
// A thread adds up its columns' sums over the block's rows, sq for post_w and scale, sp for pre_w.
template <int HAS, typename T, int NT, int VPT, int CL, typename PostW, typename PreW>
__device__ __forceinline__ void back_row(const BackArgs &p, int64_t row, const Cols<CL> &cols, V8<T> (&x)[VPT], const V8<T> (&dh)[VPT], const V8<T> (&dx1)[VPT],
                                         V8<T> (&y)[VPT], V8<T> (&g)[VPT], float2 (&sq)[VPT][4], float2 (&sp)[VPT][4], float (*sh)[3], float (*sh1)[1],
                                         PostW post_w, PreW pre_w)
{
    const float inv_D = 1.f / p.D;
    const bool has_y = HAS != kAny || p.r.y, has_g = HAS == kAny ? p.r.g != nullptr : HAS == kAll, has_h = HAS != kAny || p.r.dh, has_dx1 = HAS != kAny || p.r.dx1;
    float s[3] = {0.f, 0.f, 0.f};  // x^2, x dh pre_w, y^2
    float2 s0 = f2(0.f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (c >= cols.end) continue;
        W8 w;
        if (has_h) w = pre_w(i, c);
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
    row_sum<NT, CL>(s, sh);
    const float rx = rstd(s[0], p.D, p.eps), ry = rstd(s[2], p.D, p.eps);
    const float mx = s[1] * rx * inv_D;  // mean(w n)
    float2 m = f2(0.f), d[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (c >= cols.end) continue;
        W8 w, pw;
        if (has_h) w = pre_w(i, c);
        if (has_y) pw = post_w(i, c);
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
                float2 k = d[i][j], o;
                if (has_g) {
                    const float2 s = both_sigmoids(g[i].get(j), o);
                    k = f2_mul(k, s);
                }
                sq[i][j] = f2_fma(k, n, sq[i][j]);
                d[i][j] = f2_mul(k, pw.get(j));  // the gradient of n
                const float2 dn = f2_mul(d[i][j], n);
                m = f2_add(m, dn);
                if (has_g) g[i].set(j, f2_mul(dn, o));  // d sigmoid = s (1 - s); dn has a factor s
            }
        }
        store8(x[i], p.r.dx, row * p.r.dx_stride + c, c, p.D);
        if (has_g) store8(g[i], p.r.dg, row * p.r.dg_stride + c, c, p.D);
    }
    if (!has_y) return;
    float t[1] = {m.x + m.y};
    row_sum<NT, CL>(t, sh1);
    const float my = t[0] * inv_D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
        if (c >= cols.end) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 n = f2_mul(y[i].get(j), f2(ry));
            y[i].set(j, f2_mul(f2(ry), f2_fma(n, f2(-my), d[i][j])));
        }
        store8(y[i], p.r.dy, row * p.r.dy_stride + c, c, p.D);
    }
}

template <int NT, int VPT, int CL>
__device__ __forceinline__ void store_sums(const BackArgs &p, int part, const Cols<CL> &cols, const float2 (&sq)[VPT][4], const float2 (&sp)[VPT][4])
{
    float *out = p.part + (int64_t)part * 2 * p.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + 2 * j < cols.end) {
                *reinterpret_cast<float2 *>(out + c + 2 * j) = sq[i][j];
                *reinterpret_cast<float2 *>(out + p.D + c + 2 * j) = sp[i][j];
            }
    }
}

// Rows straight from global memory, in the forms that lack some: a warp each for the shortest ones.
template <typename T, int NT, int VPT, int CL>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) block_norm_back_kernel(const __grid_constant__ BackArgs p, int parts)
{
    constexpr int kRows = NT == 32 ? 4 : 1;
    __shared__ float sh[2][32][3], sh1[2][32][1];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int part = blockIdx.x / CL * kRows + (NT == 32 ? threadIdx.x >> 5 : 0);
    if (part >= parts) return;  // a whole warp
    const Cols<CL> cols(tid, p.D);
    if (CL == 2) {
        cluster_arrive();
        cluster_wait();
    }
    float2 sq[VPT][4], sp[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sq[i][j] = sp[i][j] = f2(0.f);
    int turn = 0;
    for (int64_t row = part; row < p.M; row += parts, turn ^= 1) {
        V8<T> x[VPT], dh[VPT], dx1[VPT], y[VPT], g[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = cols.first + 8 * NT * i;
            if (c >= cols.end) continue;
            if (p.r.dh) {
                load8(x[i], p.r.x_out, row * p.r.x_out_stride + c, c, p.D);
                load8(dh[i], p.r.dh, row * p.r.dh_stride + c, c, p.D);
            }
            if (p.r.dx1) load8(dx1[i], p.r.dx1, row * p.r.dx1_stride + c, c, p.D);
            if (p.r.y) load8(y[i], p.r.y, row * p.r.y_stride + c, c, p.D);
            if (p.r.g) load8(g[i], p.r.g, row * p.r.g_stride + c, c, p.D);
        }
        back_row<kAny, T, NT, VPT, CL>(p, row, cols, x, dh, dx1, y, g, sq, sp, sh[turn], sh1[turn],
            [&](int, int c) {
                W8 w, sc;
                w.load(p.post_w, c, p.D), sc.load(p.scale, c, p.D);
                return w.times(sc);
            },
            [&](int, int c) {
                W8 w;
                w.load(p.pre_w, c, p.D);
                return w;
            });
    }
    store_sums<NT, VPT>(p, part, cols, sq, sp);
}

// As block_norm_rows_kernel: the parameters and the next row in shared memory.
template <typename T, int NT, int VPT>
struct BackStage {
    float4 w[4][VPT][NT];    // post_w scale, pre_w: four channels each
    V8<T> rows[5][VPT][NT];  // x', dh, dx', y, g
};
template <typename T, int NT, int VPT, int CL, int HAS>
__global__ void __launch_bounds__(NT, 512 / NT) block_norm_back_rows_kernel(const __grid_constant__ BackArgs p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    BackStage<T, NT, VPT> &st = *reinterpret_cast<BackStage<T, NT, VPT> *>(smem);
    __shared__ float sh[2][32][3], sh1[2][32][1];
    const int tid = threadIdx.x, part = blockIdx.x / CL, parts = gridDim.x / CL;
    const Cols<CL> cols(tid, p.D);
    if (CL == 2) cluster_arrive();
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = cols.first + 8 * NT * i;
            if (c >= cols.end) continue;
            copy8(&st.rows[0][i][tid], p.r.x_out, row * p.r.x_out_stride + c, c, p.D);
            copy8(&st.rows[1][i][tid], p.r.dh, row * p.r.dh_stride + c, c, p.D);
            copy8(&st.rows[2][i][tid], p.r.dx1, row * p.r.dx1_stride + c, c, p.D);
            copy8(&st.rows[3][i][tid], p.r.y, row * p.r.y_stride + c, c, p.D);
            if (HAS == kAll) copy8(&st.rows[4][i][tid], p.r.g, row * p.r.g_stride + c, c, p.D);
        }
    };
    fetch(part);
    float2 sq[VPT][4], sp[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = cols.first + 8 * NT * i;
#pragma unroll
        for (int j = 0; j < 4; ++j) sq[i][j] = sp[i][j] = f2(0.f);
        if (c >= cols.end) continue;
        W8 w, sc;
        w.load(p.post_w, c, p.D), sc.load(p.scale, c, p.D);
        w = w.times(sc);
        st.w[0][i][tid] = w.r[0], st.w[1][i][tid] = w.r[1];
        w.load(p.pre_w, c, p.D);
        st.w[2][i][tid] = w.r[0], st.w[3][i][tid] = w.r[1];
    }
    if (CL == 2) cluster_wait();  // the other block runs, and has shared memory
    int turn = 0;
#pragma unroll 1
    for (int64_t row = part; row < p.M; row += parts, turn ^= 1) {
        V8<T> x[VPT], dh[VPT], dx1[VPT], y[VPT], g[VPT];
        cp_async_wait_all();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            x[i] = st.rows[0][i][tid], dh[i] = st.rows[1][i][tid];
            dx1[i] = st.rows[2][i][tid];
            y[i] = st.rows[3][i][tid];
            if (HAS == kAll) g[i] = st.rows[4][i][tid];
        }
        if (row + parts < p.M) fetch(row + parts);
        back_row<HAS, T, NT, VPT, CL>(p, row, cols, x, dh, dx1, y, g, sq, sp, sh[turn], sh1[turn],
            [&](int i, int) { return W8{{st.w[0][i][tid], st.w[1][i][tid]}}; }, [&](int i, int) { return W8{{st.w[2][i][tid], st.w[3][i][tid]}}; });
    }
    store_sums<NT, VPT>(p, part, cols, sq, sp);
}

__global__ void __launch_bounds__(kSumCols *kSumGroups)
block_norm_sums_kernel(const float *part, int parts, int D, const float *post_w, const float *scale, float *dpost_w, float *dscale, float *dpre_w)
{
    __shared__ float sh[kSumGroups][kSumCols];
    wait_for_previous();
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
    if (reinterpret_cast<uintptr_t>(ptr) % align) return fail(KDA_ERR_INVALID, "%s must be %d-byte aligned", name, align), false;
    if (M == 1) return true;  // the distance between rows is not used
    if (stride < D) return fail(KDA_ERR_INVALID, "%s_stride must be >= %d (got %lld)", name, D, (long long)stride), false;
    if (stride > ((int64_t)1 << 38) || M > ((int64_t)1 << 60) / stride)
        return fail(KDA_ERR_INVALID, "%s_stride out of range (%lld)", name, (long long)stride), false;
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

// Rows of partial sums. One more costs the sums' kernel what some M / 100 of a row fewer save a block, so the time is least
// near 10 sqrt(M) of them (BF16, 256 channels, M = 9600, in 608, 912, 1216, 1824: 15.4, 14.2, 13.8, 15.5 us; 1024 channels, M = 300, in
// 152, 300: 6.0, 7.0; M = 2400, in 304, 456, 608: 12.7, 12.0, 12.7): a whole number for each of the 152 SMs, up to what runs at once.
int64_t parts_of(int32_t D, int64_t M)
{
    const int64_t most = D <= 256 ? 2432 : D <= 512 ? 1216 : D <= 2048 ? 608 : 304, even = (int64_t)(10 * sqrt((double)M) / 152 + 0.5) * 152;
    const int64_t n = even < 152 ? 152 : even < most ? even : most;
    return M < n ? M : n;
}
size_t back_bytes(int32_t D, int64_t M) { return 256 + (size_t)parts_of(D, M) * 2 * D * sizeof(float); }

// Blocks of nt threads that stay on an SM: as many threads in all, as far as shared memory goes.
constexpr int blocks_per_sm(int threads, int nt, size_t smem)
{
    const int by_smem = (int)(233472 / (smem + 2048));
    return threads / nt < by_smem ? threads / nt : by_smem;
}

template <typename T, int NT, int VPT, bool F8, int HAS = kAny>
cudaError_t launch_rows(const Args &p, int dev, int sms, cudaStream_t s)
{
    if (HAS == kAny) return p.r.g ? launch_rows<T, NT, VPT, F8, kAll>(p, dev, sms, s) : launch_rows<T, NT, VPT, F8, kNoGate>(p, dev, sms, s);
    constexpr int kHas = HAS == kAny ? kAll : HAS;
    static std::atomic<uint64_t> raised;
    const int smem = (int)sizeof(Stage<T, NT, VPT>);
    const cudaError_t e = raise_smem_on(raised, dev, block_norm_rows_kernel<T, NT, VPT, F8, kHas>, smem);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)sms * blocks_per_sm(512, NT, sizeof(Stage<T, NT, VPT>));
    block_norm_rows_kernel<T, NT, VPT, F8, kHas><<<(unsigned)(p.M < most ? p.M : most), NT, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool F8>
cudaError_t launch(const Args &p, int dev, int sms, cudaStream_t s)
{
    const unsigned M = (unsigned)p.M, M4 = (unsigned)((p.M + 3) / 4);
    // Blocks that stay from about 2.4 million channels of rows on (BF16 without a gate, M = 600, 1200, 2400, 9600): D = 600 3.1, 3.7, 4.6,
    // 10.7 us for 3.1, 3.5, 5.4, 13.4 with a block each; 4096 6.2, 7.8, 11.7, 50.9 for 5.4, 9.7, 17.6, 64.7; 7168 7.6, 10.9, 23.8, 92.8
    // for 8.9, 16.8, 35.3, 129.8. FP32 turns at the same M. 16384 channels (M = 1200, 4800): 28.2, 109 for 44.9, 165 us; in FP32 the
    // parameters find no room there, and the rows alone gain 5% (77, 278 us with a block each). A cluster of two blocks a row takes 38.5, 127.
    constexpr bool kStageWide = sizeof(T) == 2;
    if (p.M >= 4 * sms && p.M * p.D >= 2400000 && p.D > 512 && (p.D <= kWide || kStageWide) && p.r.y && p.r.h) {
        if (p.D <= 1024) return launch_rows<T, 64, 2, F8>(p, dev, sms, s);
        if (p.D <= 2048) return launch_rows<T, 128, 2, F8>(p, dev, sms, s);
        if (p.D <= 4096) return launch_rows<T, 128, 4, F8>(p, dev, sms, s);
        if (p.D <= kWide) return launch_rows<T, 256, 4, F8>(p, dev, sms, s);
        if constexpr (kStageWide) return launch_rows<T, 512, 4, F8>(p, dev, sms, s);
    }
    if (p.D <= 256) block_norm_kernel<T, 32, 1, F8><<<M4, 128, 0, s>>>(p);
    else if (p.D <= 512) block_norm_kernel<T, 32, 2, F8><<<M4, 128, 0, s>>>(p);
    else if (p.D <= 1024) block_norm_kernel<T, 128, 1, F8><<<M, 128, 0, s>>>(p);
    else if (p.D <= 2048) block_norm_kernel<T, 128, 2, F8><<<M, 128, 0, s>>>(p);
    else if (p.D <= 4096) block_norm_kernel<T, 256, 2, F8><<<M, 256, 0, s>>>(p);
    else if (p.D <= 8192) block_norm_kernel<T, 512, 2, F8><<<M, 512, 0, s>>>(p);
    else block_norm_kernel<T, 1024, 2, F8><<<M, 1024, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int NT, int VPT, int CL = 1, int HAS = kAny>
cudaError_t launch_back_rows(const BackArgs &p, int *parts, int dev, int sms, cudaStream_t s)
{
    if (HAS == kAny) return p.r.g ? launch_back_rows<T, NT, VPT, CL, kAll>(p, parts, dev, sms, s) : launch_back_rows<T, NT, VPT, CL, kNoGate>(p, parts, dev, sms, s);
    constexpr int kHas = HAS == kAny ? kAll : HAS;
    static std::atomic<uint64_t> raised;
    const int smem = (int)sizeof(BackStage<T, NT, VPT>);
    const auto kernel = block_norm_back_rows_kernel<T, NT, VPT, CL, kHas>;
    const cudaError_t e = raise_smem_on(raised, dev, kernel, smem);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)sms * blocks_per_sm(512, NT, sizeof(BackStage<T, NT, VPT>)) / CL;
    *parts = (int)(most < *parts ? most : *parts);
    return launch_cluster(kernel, (unsigned)*parts * CL, CL, NT, smem, s, p);
}

// parts: rows of partial sums that the workspace has room for, and then those that are written
template <typename T>
cudaError_t launch_back(const BackArgs &p, int *parts, int dev, int sms, cudaStream_t s)
{
    const unsigned n = (unsigned)*parts, n4 = (unsigned)((*parts + 3) / 4);
    // Staged rows wherever a call has all of them (BF16, M = 20, 150, 9600): D = 512 4.5, 5.0, 18.1 us for 6.4, 6.8, 26.3 straight from
    // global memory; 7168 11.9, 14.0, 138 for 12.4, 14.3, 267; FP32 14.4, 17.2, 282 for 17.4, 19.2, 641.
    // Two blocks a row (BF16, M = 40, 300, 1200, 4800): D = 8200 12.8, 21.0, 60, 216 us; 16384 18.9, 28.5, 81, 259; FP32 24, 49, 135, 458.
    // One block, its sums in shared memory and the row read three times: 13.9, 20.6, 66, 308; 21.3, 40.8, 138, 506; 25, 49, 163, 603.
    if (p.r.y && p.r.dh && p.r.dx1) {
        if (p.D <= 256) return launch_back_rows<T, 32, 1>(p, parts, dev, sms, s);
        if (p.D <= 512) return launch_back_rows<T, 64, 1>(p, parts, dev, sms, s);
        if (p.D <= 1024) return launch_back_rows<T, 128, 1>(p, parts, dev, sms, s);
        if (p.D <= 2048) return launch_back_rows<T, 128, 2>(p, parts, dev, sms, s);
        if (p.D <= 4096) return launch_back_rows<T, 256, 2>(p, parts, dev, sms, s);
        if (p.D <= kWide) return launch_back_rows<T, 512, 2>(p, parts, dev, sms, s);
        return launch_back_rows<T, 512, 2, 2>(p, parts, dev, sms, s);
    }
    if (p.D <= 256) block_norm_back_kernel<T, 32, 1, 1><<<n4, 128, 0, s>>>(p, *parts);
    else if (p.D <= 512) block_norm_back_kernel<T, 32, 2, 1><<<n4, 128, 0, s>>>(p, *parts);
    else if (p.D <= 1024) block_norm_back_kernel<T, 128, 1, 1><<<n, 128, 0, s>>>(p, *parts);
    else if (p.D <= 2048) block_norm_back_kernel<T, 128, 2, 1><<<n, 128, 0, s>>>(p, *parts);
    else if (p.D <= 4096) block_norm_back_kernel<T, 256, 2, 1><<<n, 256, 0, s>>>(p, *parts);
    else if (p.D <= kWide) block_norm_back_kernel<T, 512, 2, 1><<<n, 512, 0, s>>>(p, *parts);
    else return launch_cluster(block_norm_back_kernel<T, 512, 2, 2>, 2 * n, 2, 512, 0, s, p, *parts);
    return cudaGetLastError();
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
    int dev = 0, sms = 0;
    cudaError_t err = current_sms(&dev, &sms);
    if (err == cudaSuccess) {
        if (cfg->io_dtype == KDA_F32) err = r.hs ? bn::launch<float, true>(p, dev, sms, s) : bn::launch<float, false>(p, dev, sms, s);
        else err = r.hs ? bn::launch<__nv_bfloat16, true>(p, dev, sms, s) : bn::launch<__nv_bfloat16, false>(p, dev, sms, s);
    }
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
    int parts = (int)bn::parts_of(D, M), dev = 0, sms = 0;
    cudaError_t err = cudaSuccess;
    if (M > 0) {
        const bn::BackArgs p = {M, D, cfg->eps, params->post_w, params->scale, params->pre_w, r, static_cast<float *>(workspace)};
        if ((err = current_sms(&dev, &sms)) == cudaSuccess)
            err = cfg->io_dtype == KDA_F32 ? bn::launch_back<float>(p, &parts, dev, sms, s) : bn::launch_back<__nv_bfloat16>(p, &parts, dev, sms, s);
    }
    if (err == cudaSuccess && (dpost_w || dscale || dpre_w)) {  // without rows: zeros
        const dim3 grid((D + kSumCols - 1) / kSumCols, 2);
        const float *part = static_cast<const float *>(workspace);
        // without rows no kernel of this call comes before it
        if (M > 0) err = launch_after(bn::block_norm_sums_kernel, grid, sum_block(parts), 0, s, part, parts, D, params->post_w, params->scale, dpost_w, dscale, dpre_w);
        else bn::block_norm_sums_kernel<<<grid, sum_block(0), 0, s>>>(part, 0, D, params->post_w, params->scale, dpost_w, dscale, dpre_w), err = cudaGetLastError();

    }
    return err == cudaSuccess ? KDA_OK : bn::fail(KDA_ERR_CUDA, "kda_block_norm_backward: %s", cudaGetErrorString(err));
}

}  // extern "C"
