// kda_glr_walk.cu - prefill of the gated linear recurrence over short sequences: a thread has two channels of a sequence, from
// its first token to its last. A scan's blocks cost some microseconds each, whatever their tokens, and here there are enough
// threads without one. Bound by the special function unit and the rows' way through HBM where there are many threads (4000
// sequences of up to 64 tokens, 4096 channels, BF16 with a gate: 1345 us, 390 channels a ns; the scan 2130), by 0.17 us a token
// where there are few.
#include "kda_glr_scan.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int kAhead = 4;  // tokens that a thread asks for at once

template <typename T, bool G>
__global__ void __launch_bounds__(128) glr_walk_kernel(const __grid_constant__ Args p)
{
    using Raw = typename Pair<T>::Raw;
    const int half = p.D / 2;
    const int64_t unit = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int row = (int)(unit / half), c = 2 * (int)(unit - (int64_t)row * half);
    if (row >= p.N) return;
    int src, dst, t0, t1;
    if (!bounds_ok(p.cu, row, p.N, p.total_T, t0, t1) || !slots_ok(p, row, src, dst)) {
        if (c == 0) set_err(p.err);
        return;
    }
    float2 h = src >= 0 ? *reinterpret_cast<const float2 *>(p.S + (size_t)src * p.D + c) : f2(0.f);
    const int n = t1 - t0;
    Chan ch;
    ch.load(p.A_log, p.a_bias, p.b_bias, c);
    const T *xp = static_cast<const T *>(p.rows.x) + (int64_t)t0 * p.rows.x_stride + c, *ap = static_cast<const T *>(p.rows.a) + (int64_t)t0 * p.rows.a_stride + c;
    const T *bp = static_cast<const T *>(p.rows.b) + (int64_t)t0 * p.rows.b_stride + c;
    const T *gp = G ? static_cast<const T *>(p.rows.g) + (int64_t)t0 * p.rows.g_stride + c : nullptr;
    T *op = static_cast<T *>(p.rows.out) + (int64_t)t0 * p.rows.out_stride + c;
    float *st = p.starts ? p.starts + first_chunk(t0, row) * p.D + c : nullptr;
#pragma unroll 1
    for (int t = 0; t < n; t += kAhead) {
        Raw x[kAhead], a[kAhead], b[kAhead], g[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t + i < n) {
                x[i] = ld_pair(xp + (t + i) * p.rows.x_stride);
                a[i] = ld_pair(ap + (t + i) * p.rows.a_stride);
                b[i] = ld_pair(bp + (t + i) * p.rows.b_stride);
                if (G) g[i] = ld_pair(gp + (t + i) * p.rows.g_stride);
            }
        if (st && t % kChunk == 0) *reinterpret_cast<float2 *>(st + (size_t)(t / kChunk) * p.D) = h;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t + i < n) {
                float2 e, u;
                gates(ch, Pair<T>::get(x[i]), Pair<T>::get(a[i]), Pair<T>::get(b[i]), e, u);
                h = step(h, e, u);
                st_pair(op + (t + i) * p.rows.out_stride, G ? f2_mul(h, silu2(Pair<T>::get(g[i]))) : h);
            }
    }
    *reinterpret_cast<float2 *>(p.S + (size_t)dst * p.D + c) = h;
}

}  // namespace

cudaError_t launch_walk(const Args &p, bool f32, cudaStream_t s)
{
    const unsigned grid = (unsigned)(((int64_t)p.N * (p.D / 2) + 127) / 128);
    if (p.rows.g) {
        if (f32) glr_walk_kernel<float, true><<<grid, 128, 0, s>>>(p);
        else glr_walk_kernel<__nv_bfloat16, true><<<grid, 128, 0, s>>>(p);
    } else {
        if (f32) glr_walk_kernel<float, false><<<grid, 128, 0, s>>>(p);
        else glr_walk_kernel<__nv_bfloat16, false><<<grid, 128, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace glr
}  // namespace kda
