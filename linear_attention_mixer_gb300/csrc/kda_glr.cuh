// kda_glr.cuh - what the kernels of the gated linear recurrence share: the arguments, and one token's gates.
//
// Per channel, with the state h in FP32:
//   gk = -exp(A_log) sigmoid(a + a_bias),  alpha = exp(gk),  beta = sigmoid(b + b_bias)
//   h = alpha h + m beta x,  m = sqrt(1 - alpha^2),  out = h  or  h silu(g)
//
// A lane has two neighbouring channels, as FP32 pairs. The decay is held as e = alpha - 1 and a step taken as
// h + (e h + u): near alpha = 1, where a state remembers 1 / (1 - alpha) tokens, alpha itself in FP32 would be
// wrong by 2^-25 at each of them (the steady state of 1 - alpha = 1e-4 by 3e-4), e is not. m^2 = -e (2 + e) has
// no cancellation either. (The scan keeps its products of alphas in a like way.) What it costs: where alpha is far below 1, h's part of the sum is off by 2^-24 |h|.
#pragma once

#include "kda_internal.cuh"
#include "kda_ptx.cuh"

namespace kda {
namespace glr {

constexpr int kChunk = 16;   // tokens between the states that a forward keeps for its backward
constexpr int kSlab = 64;    // channels of a warp

// A long sequence of few channels in parts that different clusters take at once. A part's first state is folded from the
// pairs (A, H) of the `sub` tokens each before it, which another kernel works out before.
struct Split {
    int32_t parts;   // of a sequence; 1: not split
    int32_t plen;    // tokens of a part, a multiple of sub; the last part has what is left
    int32_t sub, subs;
    float4 *pairs;   // [N][subs][D / 2]
    float *S0;       // [N][D]: the states at the start, since the call writes to the slots
};

struct Args {
    float *S;  // [max_slots][D]
    int32_t max_slots;
    const int32_t *src, *dst;
    int32_t *err;       // may be null
    const int32_t *cu;  // prefill: [N + 1]; decode: n tokens a row
    int32_t N, n;
    int64_t total_T;
    int32_t D;
    const float *A_log, *a_bias, *b_bias;
    kda_glr_rows rows;
    float *starts;  // may be null
    Split split;
};

struct BackArgs {
    int32_t *err;
    const int32_t *cu;
    int32_t N;
    int64_t total_T;
    int32_t D;
    const float *A_log, *a_bias, *b_bias;
    const float *starts;
    kda_glr_grad_rows rows;
    const float *dS_last;  // may be null: zeros
    float *dS_first;       // may be null
    float *part;           // sums over tokens: [groups x blocks a cluster][3][D]
    int32_t groups;        // parts of sequences in work at once
    Split split;
};

__device__ __forceinline__ void set_err(int32_t *err, int32_t what = kErrBadSlot)
{
    if (err) atomicExch(err, what);
}

// Slots of a row: false when one is out of range. src may be -1: a zero state.
__device__ __forceinline__ bool slots_ok(const Args &p, int row, int &src, int &dst)
{
    src = __ldg(p.src + row);
    dst = __ldg(p.dst + row);
    return src >= -1 && src < p.max_slots && dst >= 0 && dst < p.max_slots;
}

// The bounds of sequence s: false unless they rise within [0, T], from 0 for the first, to T for the last. When this
// holds for every sequence, none overlaps another.
__device__ __forceinline__ bool bounds_ok(const int32_t *cu, int s, int N, int64_t T, int &t0, int &t1)
{
    t0 = __ldg(cu + s);
    t1 = __ldg(cu + s + 1);
    return t0 >= 0 && t1 >= t0 && t1 <= T && (s > 0 || t0 == 0) && (s < N - 1 || t1 == T);
}

// The first of sequence s's chunks among those of all sequences: of 16 tokens each, numbered so that a sequence needs
// only its own bounds (the numbers between one sequence's chunks and the next one's are not used).
__device__ __forceinline__ int64_t first_chunk(int t0, int s) { return (int64_t)(t0 / kChunk) + s; }

// ---------------------------------------------------------------- two channels of a row
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    typedef uint32_t Raw;
    static __device__ __forceinline__ float2 get(Raw r) { return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u)); }
    static __device__ __forceinline__ Raw put(float2 f)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <> struct Pair<float> {
    typedef float2 Raw;
    static __device__ __forceinline__ float2 get(Raw r) { return r; }
    static __device__ __forceinline__ Raw put(float2 f) { return f; }
};
template <typename T> __device__ __forceinline__ typename Pair<T>::Raw ld_pair(const T *p)
{
    return __ldg(reinterpret_cast<const typename Pair<T>::Raw *>(p));
}
template <typename T> __device__ __forceinline__ void st_pair(T *p, float2 f)
{
    *reinterpret_cast<typename Pair<T>::Raw *>(p) = Pair<T>::put(f);
}

// four channels of a row
template <typename T> struct Quad;
template <> struct Quad<__nv_bfloat16> {
    typedef uint2 Raw;
    static __device__ __forceinline__ float2 get(const Raw &r, int i) { return Pair<__nv_bfloat16>::get(i ? r.y : r.x); }
    static __device__ __forceinline__ Raw put(float2 a, float2 b) { return make_uint2(Pair<__nv_bfloat16>::put(a), Pair<__nv_bfloat16>::put(b)); }
};
template <> struct Quad<float> {
    typedef float4 Raw;
    static __device__ __forceinline__ float2 get(const Raw &r, int i) { return i ? make_float2(r.z, r.w) : make_float2(r.x, r.y); }
    static __device__ __forceinline__ Raw put(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
};
template <typename T> __device__ __forceinline__ typename Quad<T>::Raw ld_quad(const T *p)
{
    return __ldg(reinterpret_cast<const typename Quad<T>::Raw *>(p));
}

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float ex2_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b)  // NaN if either is
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// exp(x) - 1 for x <= 0. Above -1/4 it is x q(x), q of degree 4 (Chebyshev interpolation of (exp(x) - 1) / x on [-1/4, 0]; its
// error is 2.6e-9), to a few 2^-24 however near to 0. Below, the difference loses no more than two bits of the exponential: alpha is
// off by 2.1 x 2^-24 at most and 0.6 x 2^-24 in the root mean square (measured over x from -20 to -0.2), and is there remembered for no
// more than four tokens. NaN stays. (Reducing x to k ln 2 + r and a q of degree 5 on |r| <= ln 2 / 2, without the exponential, takes four instructions
// more for each channel: 65536 tokens of 4096 channels 535 us for 516.)
__device__ __forceinline__ float2 expm1_neg(float2 x)
{
    float2 q = f2_fma(f2(0.007513605989515781f), x, f2(0.04149065539240837f));
    q = f2_fma(q, x, f2(0.16665108501911163f));
    q = f2_fma(q, x, f2(0.4999995231628418f));
    q = f2_fma(q, x, f2(1.f));
    q = f2_mul(q, x);
    const float2 t = f2_mul(x, f2(kLog2e));
    const float2 far = f2_add(make_float2(ex2_ftz(t.x), ex2_ftz(t.y)), f2(-1.f));
    return make_float2(x.x > -0.25f ? q.x : far.x, x.y > -0.25f ? q.y : far.y);
}

// The parameters of two channels.
struct Chan {
    float2 nA, ca, cb;  // -exp(A_log), -log2(e) times the biases
    __device__ __forceinline__ void load(const float *A_log, const float *a_bias, const float *b_bias, int c)
    {
        const float2 l = *reinterpret_cast<const float2 *>(A_log + c), x = *reinterpret_cast<const float2 *>(a_bias + c);
        const float2 y = *reinterpret_cast<const float2 *>(b_bias + c);
        nA = make_float2(-expf(l.x), -expf(l.y));
        ca = f2_mul(f2(-kLog2e), x);
        cb = f2_mul(f2(-kLog2e), y);
    }
};

// exp(-(v + bias)) of two channels: 1 / (1 + that) is the sigmoid
__device__ __forceinline__ float2 neg_exp(float2 v, float2 c)
{
    const float2 t = f2_fma(v, f2(-kLog2e), c);
    return make_float2(ex2_ftz(t.x), ex2_ftz(t.y));
}
__device__ __forceinline__ float2 rcp2(float2 v) { return make_float2(rcp_ftz(v.x), rcp_ftz(v.y)); }

// z = 1 - alpha^2 from e, and 1 / sqrt(z), which is large and finite at z = 0
__device__ __forceinline__ float2 one_less_square(float2 e) { return f2_mul(e, f2_fma(e, f2(-1.f), f2(-2.f))); }
__device__ __forceinline__ float2 rsqrt2(float2 z)
{
    const float2 t = f2_add(z, f2(1e-36f));
    return make_float2(rsqrt_ftz(t.x), rsqrt_ftz(t.y));
}
// e = alpha - 1 and u = m beta x of one token.
__device__ __forceinline__ void gates(const Chan &p, float2 x, float2 a, float2 b, float2 &e, float2 &u)
{
    const float2 sa = rcp2(f2_add(neg_exp(a, p.ca), f2(1.f))), beta = rcp2(f2_add(neg_exp(b, p.cb), f2(1.f)));
    e = expm1_neg(f2_mul(p.nA, sa));
    const float2 z = one_less_square(e);
    u = f2_mul(f2_mul(f2_mul(z, rsqrt2(z)), beta), x);
}
__device__ __forceinline__ float2 step(float2 h, float2 e, float2 u) { return f2_add(h, f2_fma(e, h, u)); }
__device__ __forceinline__ float2 silu2(float2 g)
{
    return f2_mul(g, rcp2(f2_add(neg_exp(g, f2(0.f)), f2(1.f))));
}

constexpr float kHuge = 8.507059173023462e37f;  // 2^126: its reciprocal is still a normal number

// A sigmoid s and 1 - s from E = exp(-its argument), without the difference: 1 / (1 + E) and E / (1 + E). Where the reciprocal is 0
// the second is not used: what it multiplies has s as a factor.
__device__ __forceinline__ void both_sigmoids(float2 E, float2 &s, float2 &ns)
{
    s = rcp2(f2_add(E, f2(1.f)));
    ns = make_float2(min_nan(E.x, kHuge) * s.x, min_nan(E.y, kHuge) * s.y);
}

// One token's part in the gradients, with c the gradient of the state after it from the tokens behind:
//   lam = dh + c,  dx = lam m beta,  db = dx x (1 - beta),  c = alpha lam
//   d gk = lam alpha (h - beta x alpha / m), h the state before it,  d A_log = d gk gk,  da = d gk gk (1 - sigmoid(a + a_bias))
struct Back {
    float2 m, rm, beta, nb, gk, na;  // rm = 1 / m, nb = 1 - beta, na = 1 - sigmoid(a + a_bias)
    __device__ __forceinline__ void gates(const Chan &p, float2 e, float2 a, float2 b)
    {
        float2 sa;
        both_sigmoids(neg_exp(a, p.ca), sa, na);
        both_sigmoids(neg_exp(b, p.cb), beta, nb);
        gk = f2_mul(p.nA, sa);
        const float2 z = one_less_square(e);
        rm = rsqrt2(z);
        m = f2_mul(z, rm);
    }
    // Returns the next c.
    __device__ __forceinline__ float2 token(float2 e, float2 lam, float2 x, float2 h, float2 &dx, float2 &da, float2 &db, float2 &dA) const
    {
        const float2 alpha = f2_add(e, f2(1.f));
        dx = f2_mul(f2_mul(lam, m), beta);
        db = f2_mul(f2_mul(dx, x), nb);
        // gk / m goes to 0 with gk: taken first, so that 1 / m stays harmless
        const float2 w = f2_mul(f2_mul(f2_mul(beta, x), alpha), f2_mul(gk, rm));
        dA = f2_mul(f2_mul(lam, alpha), f2_fma(h, gk, make_float2(-w.x, -w.y)));
        da = f2_mul(dA, na);
        return f2_fma(e, lam, lam);
    }
};

}  // namespace glr
}  // namespace kda
