// kda_gdr.cuh - shared pieces of the gated delta rule kernels (kda_gdr.cu: recurrent form and host
// side; kda_gdr_prefill.cu: chunked form).
//
// Per value head with state S[key][value], key head h / (H / Hk), and one decay per head:
//   alpha = exp(-exp(A_log) softplus(a + dt_bias)),  beta = sigmoid(b)
//   u = beta (v - alpha S^T k^),  S = alpha S + k^ u^T,  o = S^T q^
// with k^ = k / sqrt(|k|^2 + eps) and q^ = q_scale q / sqrt(|q|^2 + eps) (or k^ = k, q^ = q_scale q).
// It is the delta rule of the KDA mixer (kimi_k3.c header, "KDA per-head recurrence") with a scalar
// decay, without the convolution and the output norm.
#pragma once

#include "kda_internal.cuh"
#include "kda_ptx.cuh"

namespace kda {
namespace gdr {

// What every kernel of the operator is given.
struct Args {
    float *S;              // [max_slots][H][d][d]
    int32_t max_slots;
    const int32_t *src, *dst;
    int32_t *err;          // may be null
    const int32_t *cu;     // prefill: [N + 1]; decode: n tokens a row
    int32_t N, n;
    int64_t total_T;
    int32_t H, G;          // value heads, value heads per key head
    const float *A_log, *dt_bias;
    kda_gdr_rows rows;
    int32_t l2norm;
    float l2_eps, q_scale;
};

__device__ __forceinline__ void set_err(int32_t *err)
{
    if (err) atomicExch(err, kErrBadSlot);
}

// Slots of a row: false (and the error word set) when one is out of range. src may be -1: a zero state.
__device__ __forceinline__ bool slots_ok(const Args &p, int row, int &src, int &dst)
{
    src = __ldg(p.src + row);
    dst = __ldg(p.dst + row);
    return src >= -1 && src < p.max_slots && dst >= 0 && dst < p.max_slots;
}

// The decay's logarithm. Below -1e4 alpha is 0 in FP32 many times over; the bound keeps sums of
// logarithms over a chunk finite (a NaN passes through).
__device__ __forceinline__ float log_decay(float a, float dt_bias, float expA)
{
    const float x = a + dt_bias;
    const float sp = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    const float g = -expA * sp;
    return g < -1e4f ? -1e4f : g;
}

// ---------------------------------------------------------------- token by token
// A warp has 16 value columns of one (row, head) state; see kda_gdr.cu.

// 16 consecutive elements as FP32
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    uint4 r[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        r[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        r[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&f)[16]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
                f[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        }
    }
};
template <> struct Vec16<float> {
    float4 r[4];
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __ldg(reinterpret_cast<const float4 *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[16]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[4 * i] = r[i].x; f[4 * i + 1] = r[i].y; f[4 * i + 2] = r[i].z; f[4 * i + 3] = r[i].w;
        }
    }
};

template <typename T>
struct Token {
    Vec16<T> k, q;
    float v, a, b;
};

// Sums of p = S^T k and r = S^T q over the rows of all lanes, for the column 4 cg + (rg & 3) of this lane:
// halving exchanges over rg; lane bit 4 keeps p (0) or r (1), bits 3 and 2 pick the column.
__device__ __forceinline__ void column_sums(float2 p01, float2 p23, float2 r01, float2 r23, int lane, float &ps, float &rs)
{
    const bool hi = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float x0 = hi ? r01.x : p01.x, x1 = hi ? r01.y : p01.y, x2 = hi ? r23.x : p23.x, x3 = hi ? r23.y : p23.y;
    x0 += __shfl_xor_sync(0xFFFFFFFFu, hi ? p01.x : r01.x, 16);
    x1 += __shfl_xor_sync(0xFFFFFFFFu, hi ? p01.y : r01.y, 16);
    x2 += __shfl_xor_sync(0xFFFFFFFFu, hi ? p23.x : r23.x, 16);
    x3 += __shfl_xor_sync(0xFFFFFFFFu, hi ? p23.y : r23.y, 16);
    float y0 = b3 ? x2 : x0, y1 = b3 ? x3 : x1;
    y0 += __shfl_xor_sync(0xFFFFFFFFu, b3 ? x0 : x2, 8);
    y1 += __shfl_xor_sync(0xFFFFFFFFu, b3 ? x1 : x3, 8);
    float z = b2 ? y1 : y0;
    z += __shfl_xor_sync(0xFFFFFFFFu, b2 ? y0 : y1, 4);
    const float z2 = __shfl_xor_sync(0xFFFFFFFFu, z, 16);
    ps = hi ? z2 : z;
    rs = hi ? z : z2;
}
// this lane's 16 rows of its 4 columns: p += S^T k, r += S^T q
__device__ __forceinline__ void column_partials(const float4 (&s)[16], const float (&k)[16], const float (&q)[16], float2 &p01,
                                                float2 &p23, float2 &r01, float2 &r23)
{
    p01 = p23 = r01 = r23 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 k2 = make_float2(k[i], k[i]), q2 = make_float2(q[i], q[i]);
        const float2 s01 = make_float2(s[i].x, s[i].y), s23 = make_float2(s[i].z, s[i].w);
        p01 = f2_fma(k2, s01, p01);
        p23 = f2_fma(k2, s23, p23);
        r01 = f2_fma(q2, s01, r01);
        r23 = f2_fma(q2, s23, r23);
    }
}
// S = alpha S + k w^T; w is of column c = rg & 3 of every lane's own cg
__device__ __forceinline__ void column_update(float4 (&s)[16], const float (&k)[16], float alpha, float w, int cg)
{
    const float w0 = __shfl_sync(0xFFFFFFFFu, w, cg), w1 = __shfl_sync(0xFFFFFFFFu, w, cg + 4);
    const float w2 = __shfl_sync(0xFFFFFFFFu, w, cg + 8), w3 = __shfl_sync(0xFFFFFFFFu, w, cg + 12);
    const float2 w01 = make_float2(w0, w1), w23 = make_float2(w2, w3), al = make_float2(alpha, alpha);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 k2 = make_float2(k[i], k[i]);
        const float2 s01 = f2_fma(k2, w01, f2_mul(al, make_float2(s[i].x, s[i].y)));
        const float2 s23 = f2_fma(k2, w23, f2_mul(al, make_float2(s[i].z, s[i].w)));
        s[i] = make_float4(s01.x, s01.y, s23.x, s23.y);
    }
}
__device__ __forceinline__ void load_state(float4 (&s)[16], const Args &p, int src, int h, size_t at)
{
    const float *S = p.S + ((size_t)max(src, 0) * p.H + h) * kD * kD + at;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        s[i] = src >= 0 ? ld_stream(reinterpret_cast<const float4 *>(S + i * kD)) : make_float4(0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ void store_state(const float4 (&s)[16], const Args &p, int dst, int h, size_t at)
{
    float *S = p.S + ((size_t)dst * p.H + h) * kD * kD + at;
#pragma unroll
    for (int i = 0; i < 16; ++i) st_stream(reinterpret_cast<float4 *>(S + i * kD), s[i]);
}

// One warp: columns 16 cb .. of head h through n tokens from row t0 on, from slot src (-1: zeros) to slot dst; the next
// token's row is fetched while one is computed.
template <typename T>
__device__ __forceinline__ void walk_tokens(const Args &p, int src, int dst, int h, int cb, int64_t t0, int n)
{
    const int lane = threadIdx.x & 31, rg = lane >> 2, cg = lane & 3, c = rg & 3;
    const size_t at = (size_t)(16 * rg) * kD + 16 * cb + 4 * cg;
    float4 s[16];
    load_state(s, p, src, h, at);
    const int hk = h / p.G, col = 16 * cb + 4 * cg + c;
    const float expA = expf(__ldg(p.A_log + h)), dt_bias = __ldg(p.dt_bias + h);
    const T *kp = static_cast<const T *>(p.rows.k) + (size_t)hk * kD + 16 * rg;
    const T *qp = static_cast<const T *>(p.rows.q) + (size_t)hk * kD + 16 * rg;
    const T *vp = static_cast<const T *>(p.rows.v) + (size_t)h * kD + col;
    const T *ap = static_cast<const T *>(p.rows.a) + h;
    const T *bp = static_cast<const T *>(p.rows.b) + h;
    T *op = static_cast<T *>(p.rows.out) + (size_t)h * kD + col;
    auto load = [&](int64_t t, Token<T> &x) {
        x.k.load(kp + t * p.rows.k_stride);
        x.q.load(qp + t * p.rows.q_stride);
        x.v = IO<T>::ld(vp + t * p.rows.v_stride);
        x.a = IO<T>::ld(ap + t * p.rows.a_stride);
        x.b = IO<T>::ld(bp + t * p.rows.b_stride);
    };
    Token<T> next;
    load(t0, next);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int64_t t = t0 + i;
        float k[16], q[16];
        next.k.get(k);
        next.q.get(q);
        const float v = next.v;
        const float alpha = expf(log_decay(next.a, dt_bias, expA)), beta = sigmoidf_(next.b);
        if (i + 1 < n) load(t + 1, next);
        // |k|^2, |q|^2, k.q: the 16 rows of this lane, then over rg (lane bits 2..4)
        float2 kk2 = make_float2(0.f, 0.f), qq2 = kk2, kq2 = kk2;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float2 k2 = make_float2(k[i], k[i + 1]), q2 = make_float2(q[i], q[i + 1]);
            kk2 = f2_fma(k2, k2, kk2);
            qq2 = f2_fma(q2, q2, qq2);
            kq2 = f2_fma(k2, q2, kq2);
        }
        float kk = kk2.x + kk2.y, qq = qq2.x + qq2.y, kq = kq2.x + kq2.y;
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
            kk += __shfl_xor_sync(0xFFFFFFFFu, kk, o);
            qq += __shfl_xor_sync(0xFFFFFFFFu, qq, o);
            kq += __shfl_xor_sync(0xFFFFFFFFu, kq, o);
        }
        const float rk = p.l2norm ? rsqrtf(kk + p.l2_eps) : 1.f;
        const float rq = p.l2norm ? p.q_scale * rsqrtf(qq + p.l2_eps) : p.q_scale;
        float2 p01, p23, r01, r23;
        column_partials(s, k, q, p01, p23, r01, r23);
        float ps, rs;
        column_sums(p01, p23, r01, r23, lane, ps, rs);
        const float u = beta * fmaf(-alpha * rk, ps, v);
        const float o = rq * fmaf(rk * kq, u, alpha * rs);
        if (!(lane & 16)) IO<T>::st(op + t * p.rows.out_stride, o);
        column_update(s, k, alpha, rk * u, cg);
    }
    store_state(s, p, dst, h, at);
}

cudaError_t launch_decode_rows(const Args &p, bool f32, cudaStream_t stream);  // N rows of n tokens
cudaError_t launch_sequences(const Args &p, cudaStream_t stream);               // FP32 rows, N sequences

size_t chunked_workspace_bytes(int64_t n_chunks, int32_t H);
cudaError_t launch_chunked(const Args &p, int64_t n_chunks, int64_t longest, void *ws, int dev, int sms, cudaStream_t stream);

}  // namespace gdr
}  // namespace kda
