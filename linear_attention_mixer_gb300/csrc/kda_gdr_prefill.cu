// kda_gdr_prefill.cu - the gated delta rule over packed sequences of BF16 rows, in chunks of
// C = 64 tokens.
//
// With G the cumulative log decay inside a chunk (a scalar per token) and S0 the state before it,
//   A[t][i] = beta_t (k^_t . k^_i) exp(G_t - G_i)  (i < t),   T = (I + A)^-1 Diag(beta)
//   U = T (V - Diag(exp G) K^ S0)
//   O = Diag(exp G) Q^ S0 + P U,   P[t][i] = (q^_t . k^_i) exp(G_t - G_i)  (i <= t)
//   S = exp(G_last) S0 + (Diag(exp(G_last - G)) K^)^T U
// which is the token recurrence exactly in real arithmetic. Every exponent is <= 0.
//
// Two kernels:
//   gdr_prep_kernel   per (chunk, key head): the products K K^T and Q K^T once, then for each of its
//                     value heads the decays, A, its inverse by forward substitution, and one block of
//                     T, P and three scalars a token for the second kernel
//   gdr_state_kernel  per (sequence, head, VB value columns): the serial pass over the chunks
//
// The raw BF16 rows of K, Q and V are the matrix operands as they are, so those operands are exact;
// the norms and the decays are FP32 scalars a token, applied to FP32 accumulators. What carries the
// state is kept to about 16 bits: S, V - .., T and U go into the products as a BF16 high part and a
// BF16 low part (x - high), products of two such factors as hi hi + lo hi + hi lo, and sums are FP32.
// With single BF16 operands the state would be off by 2^-9 a chunk. The output, which is rounded to
// BF16 itself, takes the high parts of S and U and P in one BF16.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_gdr.cuh"

namespace kda {
namespace gdr {
namespace {

// One block per (chunk, value head): BF16 tiles of 64 rows t of 64 columns i (128 bytes), 16-byte
// piece c of row t at c ^ (t & 7), then FP32 scalars.
constexpr int kBlkTl = 8192, kBlkP = 16384;  // T high at 0, T low, P
constexpr int kBlkX = 24576;                 // rk exp G | rq exp G | rk exp(G_last - G) | exp G_last
constexpr int kBlkBytes = 25600;

__device__ __forceinline__ uint32_t swz(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm2t(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// c (16 x 8, FP32) += a (16 x 16, BF16) b (16 x 8, BF16). Lane (g, q) = (lane / 4, lane % 4): c = rows
// g, g + 8 at columns 2q, 2q + 1; a = those rows at k 2q, 2q + 1 (+ 8); b = k 2q, 2q + 1 (+ 8) of column g.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// x = high + low, each BF16
__device__ __forceinline__ void split2(float x, float y, uint32_t &h, uint32_t &l)
{
    h = pack2(x, y);
    l = pack2(x - lo_f(h), y - hi_f(h));
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One warp reads cu_seqlens once: checks it against what the host sized the call for and finds either
// the sequence of chunk `want` (seq < 0 on entry) or the first chunk of sequence seq. Every lane gets
// the result; false on a mismatch.
struct Place { int seq, t0, len; int64_t first; };
__device__ __forceinline__ bool find_place(const int32_t *cu, int N, int64_t total_T, int64_t n_chunks, int64_t want,
                                           int seq, Place &out)
{
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    bool ok = true, found = false;
    for (int s0 = 0; s0 < N; s0 += 32) {
        const int s = s0 + lane;
        int b = 0, e = 0;
        if (s < N) {
            b = __ldg(cu + s);
            e = __ldg(cu + s + 1);
            ok = ok && b >= 0 && e >= b && (s > 0 || b == 0) && (s < N - 1 || e == total_T);
        }
        int nc = e >= b ? (e - b + kC - 1) / kC : 0;
        const int mine = nc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, nc, o);
            if (lane >= o) nc += x;
        }
        const int64_t before = base + nc - mine;
        const bool hit = s < N && (seq >= 0 ? s == seq : (want >= before && want < before + mine));
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, hit);
        if (m && !found) {
            const int l = __ffs(m) - 1;
            out.seq = s0 + l;
            out.t0 = __shfl_sync(0xFFFFFFFFu, b, l);
            out.len = __shfl_sync(0xFFFFFFFFu, e, l) - out.t0;
            out.first = __shfl_sync(0xFFFFFFFFu, before, l);
            found = true;
        }
        base += __shfl_sync(0xFFFFFFFFu, nc, 31);
    }
    return __all_sync(0xFFFFFFFFu, ok) && base == n_chunks && found;
}

// ---------------------------------------------------------------- prep
// 128 threads. Shared memory: K and Q rows (swizzled 128-byte halves), later two FP32 T matrices in
// their place; two FP32 A^T matrices; per-token scalars of the two value heads in work.
constexpr int kPrepThreads = 128;
constexpr int kAp = kC + 4;                    // row pitch of A^T (16-byte rows, a step of 4 banks)
constexpr int kPsK = 0, kPsQ = 16384, kPsA = 32768;
constexpr int kPsS = kPsA + 2 * kC * kAp * 4;  // [2 heads][Gh, Gl, beta][64]
constexpr int kPsN = kPsS + 2 * 3 * kC * 4;    // rk[64], rq[64]
constexpr int kPrepSmem = kPsN + 2 * kC * 4 + 64;

__global__ void __launch_bounds__(kPrepThreads)
gdr_prep_kernel(const __grid_constant__ Args p, unsigned char *__restrict__ blocks, int64_t n_chunks, int Hk)
{
    extern __shared__ __align__(128) unsigned char sm[];
    Place *place = reinterpret_cast<Place *>(sm + kPsN + 2 * kC * 4);
    int *ok = reinterpret_cast<int *>(place + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t chunk = blockIdx.x / Hk;
    const int hk = (int)(blockIdx.x - chunk * Hk);
    if (warp == 0) {
        Place pl;
        const bool good = find_place(p.cu, p.N, p.total_T, n_chunks, chunk, -1, pl);
        if (lane == 0) {
            *place = pl;
            *ok = good;
            if (!good) set_err(p.err);
        }
    }
    __syncthreads();
    if (!*ok) return;
    const int pos = (int)(chunk - place->first) * kC;
    const int64_t t0 = (int64_t)place->t0 + pos;
    const int n = min(kC, place->len - pos);
    const uint32_t sK = smem_u32(sm + kPsK), sQ = smem_u32(sm + kPsQ);
    float *sA = reinterpret_cast<float *>(sm + kPsA);
    float *sS = reinterpret_cast<float *>(sm + kPsS);
    float *sRk = reinterpret_cast<float *>(sm + kPsN), *sRq = sRk + kC;

    // rows n .. 63 read as zeros
    const __nv_bfloat16 *kg = static_cast<const __nv_bfloat16 *>(p.rows.k) + t0 * p.rows.k_stride + (size_t)hk * kD;
    const __nv_bfloat16 *qg = static_cast<const __nv_bfloat16 *>(p.rows.q) + t0 * p.rows.q_stride + (size_t)hk * kD;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int x = tid + i * kPrepThreads, r = x >> 4, c = x & 15;  // 16 pieces of 16 bytes a row
        const uint32_t off = (uint32_t)(c >> 3) * 8192 + swz(r, c & 7);
        const int rr = r < n ? r : 0;
        cp_async16(sm + kPsK + off, kg + rr * p.rows.k_stride + 8 * c, r < n ? 16 : 0);
        cp_async16(sm + kPsQ + off, qg + rr * p.rows.q_stride + 8 * c, r < n ? 16 : 0);
    }
    cp_async_wait_all();
    __syncthreads();
    {  // norms: two threads a row of K and of Q
        const int r = tid >> 1, half = tid & 1;
        float kk = 0.f, qq = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t off = (uint32_t)half * 8192 + swz(r, c);
            const uint4 a = *reinterpret_cast<const uint4 *>(sm + kPsK + off);
            const uint4 b = *reinterpret_cast<const uint4 *>(sm + kPsQ + off);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                kk = fmaf(lo_f(aw[e]), lo_f(aw[e]), fmaf(hi_f(aw[e]), hi_f(aw[e]), kk));
                qq = fmaf(lo_f(bw[e]), lo_f(bw[e]), fmaf(hi_f(bw[e]), hi_f(bw[e]), qq));
            }
        }
        kk += __shfl_xor_sync(0xFFFFFFFFu, kk, 1);
        qq += __shfl_xor_sync(0xFFFFFFFFu, qq, 1);
        if (half == 0) {
            sRk[r] = p.l2norm ? rsqrtf(kk + p.l2_eps) : 1.f;
            sRq[r] = p.l2norm ? p.q_scale * rsqrtf(qq + p.l2_eps) : p.q_scale;
        }
    }
    // K K^T and Q K^T: warp w has rows t = 16 w .. 16 w + 15, columns i <= 16 w + 15
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[j][e] = qk[j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint32_t half = (uint32_t)(ks >> 2) * 8192;
        uint32_t ak[4], aq[4];
        const uint32_t oa = half + swz(16 * warp + (lane & 15), 2 * (ks & 3) + (lane >> 4));
        ldsm4(ak, sK + oa);
        ldsm4(aq, sQ + oa);
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {
            if (jp > warp) break;
            uint32_t b[4];
            ldsm4(b, sK + half + swz(16 * jp + (lane & 7) + ((lane >> 4) << 3), 2 * (ks & 3) + ((lane >> 3) & 1)));
            mma(kk[2 * jp], ak, b[0], b[1]);
            mma(kk[2 * jp + 1], ak, b[2], b[3]);
            mma(qk[2 * jp], aq, b[0], b[1]);
            mma(qk[2 * jp + 1], aq, b[2], b[3]);
        }
    }
    float *sT = reinterpret_cast<float *>(sm);  // [2][64][64], in the place of K and Q
    for (int j0 = 0; j0 < p.G; j0 += 2) {
        const int nh = min(2, p.G - j0);
        __syncthreads();  // K, Q (first time), A, T and the scalars are free
        if (warp < nh) {  // decays of value head j0 + warp: two tokens a lane
            const int h = hk * p.G + j0 + warp;
            const float expA = expf(__ldg(p.A_log + h)), dtb = __ldg(p.dt_bias + h);
            const __nv_bfloat16 *ag = static_cast<const __nv_bfloat16 *>(p.rows.a) + t0 * p.rows.a_stride + h;
            const __nv_bfloat16 *bg = static_cast<const __nv_bfloat16 *>(p.rows.b) + t0 * p.rows.b_stride + h;
            float *s = sS + warp * 3 * kC;
            unsigned char *blk = blocks + ((size_t)chunk * p.H + h) * kBlkBytes;
            double g[2];
            float be[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                g[e] = 0.0;
                be[e] = 0.f;
                if (t < n) {
                    g[e] = (double)log_decay(__bfloat162float(ag[t * p.rows.a_stride]), dtb, expA) * 1.4426950408889634;
                    be[e] = sigmoidf_(__bfloat162float(bg[t * p.rows.b_stride]));
                }
            }
            // sums in 64 bits, kept as two FP32: differences of tokens far down a strongly decaying chunk stay exact
            double c = g[0] + g[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double x = __shfl_up_sync(0xFFFFFFFFu, c, o);
                if (lane >= o) c += x;
            }
            const double last = __shfl_sync(0xFFFFFFFFu, c, 31);
            float *bx = reinterpret_cast<float *>(blk + kBlkX);
            const double Gs[2] = {c - g[1], c};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const float h0 = (float)Gs[e];
                s[t] = h0;
                s[kC + t] = (float)(Gs[e] - (double)h0);
                s[2 * kC + t] = be[e];
                const float eg = ex2((float)Gs[e]);
                bx[t] = t < n ? sRk[t] * eg : 0.f;
                bx[kC + t] = t < n ? sRq[t] * eg : 0.f;
                bx[2 * kC + t] = t < n ? sRk[t] * ex2((float)(last - Gs[e])) : 0.f;
            }
            if (lane == 0) bx[3 * kC] = ex2((float)last);
        }
        __syncthreads();
        for (int j = 0; j < nh; ++j) {  // A^T to shared memory, P to the block
            const float *s = sS + j * 3 * kC;
            float *A = sA + j * kC * kAp;
            unsigned char *P = blocks + ((size_t)chunk * p.H + hk * p.G + j0 + j) * kBlkBytes + kBlkP;
            const int ta = 16 * warp + (lane >> 2);
            float Gh[2], Gl[2], fb[2], fq[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = ta + 8 * e;
                Gh[e] = s[t];
                Gl[e] = s[kC + t];
                fb[e] = s[2 * kC + t] * sRk[t];
                fq[e] = sRq[t];
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                float pv[2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int t = ta + 8 * e, i = 8 * nt + 2 * (lane & 3) + f;
                        float av = 0.f, x = 0.f;
                        if (i <= t) {
                            const float d = ex2((Gh[e] - s[i]) + (Gl[e] - s[kC + i])) * sRk[i];
                            x = fq[e] * d * qk[nt][2 * e + f];
                            if (i < t) av = fb[e] * d * kk[nt][2 * e + f];
                        }
                        A[i * kAp + t] = av;
                        pv[e][f] = x;
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<uint32_t *>(P + swz(ta + 8 * e, nt) + 4 * (lane & 3)) = pack2(pv[e][0], pv[e][1]);
            }
        }
        __syncthreads();
        if ((warp >> 1) < nh) {  // column jc of (I + A)^-1 by forward substitution, 16 rows at a time
            const float *A = sA + (warp >> 1) * kC * kAp;
            float *Tm = sT + (warp >> 1) * kC * kC;
            const int half = warp & 1, jc = 32 * half + lane;
            if (half)
#pragma unroll
                for (int t = 0; t < 32; ++t) Tm[t * kC + jc] = 0.f;
#pragma unroll 1
            for (int b = 2 * half; b < 4; ++b) {
                float acc[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] = 16 * b + r == jc ? 1.f : 0.f;
#pragma unroll 4
                for (int i = 32 * half; i < 16 * b; ++i) {
                    const float x = Tm[i * kC + jc];
                    const float4 *a4 = reinterpret_cast<const float4 *>(A + i * kAp + 16 * b);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 a = a4[r];
                        acc[4 * r] = fmaf(-a.x, x, acc[4 * r]);
                        acc[4 * r + 1] = fmaf(-a.y, x, acc[4 * r + 1]);
                        acc[4 * r + 2] = fmaf(-a.z, x, acc[4 * r + 2]);
                        acc[4 * r + 3] = fmaf(-a.w, x, acc[4 * r + 3]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float x = acc[r];
                    Tm[(16 * b + r) * kC + jc] = x;
#pragma unroll
                    for (int r2 = r + 1; r2 < 16; ++r2) acc[r2] = fmaf(-A[(16 * b + r) * kAp + 16 * b + r2], x, acc[r2]);
                }
            }
        }
        __syncthreads();
        for (int x = tid; x < nh * 512; x += kPrepThreads) {  // T Diag(beta), high and low
            const int j = x >> 9, t = (x >> 3) & 63, c = x & 7;
            const float4 *T4 = reinterpret_cast<const float4 *>(sT + j * kC * kC + t * kC + 8 * c);
            const float4 *b4 = reinterpret_cast<const float4 *>(sS + j * 3 * kC + 2 * kC + 8 * c);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 a = T4[e], b = b4[e];
                split2(a.x * b.x, a.y * b.y, hi[2 * e], lo[2 * e]);
                split2(a.z * b.z, a.w * b.w, hi[2 * e + 1], lo[2 * e + 1]);
            }
            unsigned char *blk = blocks + ((size_t)chunk * p.H + hk * p.G + j0 + j) * kBlkBytes + swz(t, c);
            *reinterpret_cast<uint4 *>(blk) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(blk + kBlkTl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// ---------------------------------------------------------------- state
// Everything is held transposed, with the 16 value columns of a unit as the 16 rows of the MMA: the
// FP32 accumulators of S^T, X^T = S0^T K^T, U^T and O^T then have the register layout of the next
// product's A operand, and the operands in shared memory are only read. Two warps share a unit: warp kw
// has the key rows 64 kw .. 64 kw + 63 of S (its partial sums of X and O go to the other through shared
// memory) and half of the token tiles of U and O. The tiles are dealt so that both halves of the
// triangular products are equal: tokens 0..15 and 48..63 to warp 0, 16..47 to warp 1.
// A further warp copies: a ring of stages, each K | Q | block | V of one chunk.
template <int VB> struct St {
    static constexpr int kUnits = VB / 16, kWarps = 2 * kUnits, kThreads = 32 * (kWarps + 1);
    static constexpr int kStages = VB == 32 ? 3 : 2;
    static constexpr int kQ = 16384, kBlk = 32768, kV = kBlk + kBlkBytes, kStage = kV + kC * VB * 2;
    static constexpr int kXBytes = 2 * 8 * 512, kOBytes = 2 * 4 * 512, kUBytes = 2 * 4 * 512;  // per unit
    static constexpr int kX = kStages * kStage, kUnit = kXBytes + kOBytes + kUBytes;
    static constexpr int kBar = kX + kUnits * kUnit;
    static constexpr int kSmem = kBar + 2 * kStages * 8 + 64 + 1024;
};
static_assert(St<32>::kSmem <= 232448 && St<64>::kSmem <= 232448, "state kernel shared memory");
static_assert(St<32>::kStage % 1024 == 0 && St<64>::kStage % 1024 == 0, "swizzled boxes");
constexpr uint32_t kStSpin = 1u << 26;

// byte offset of 16-byte piece c of row r of the V tile (rows of 64 or 128 bytes, TMA's swizzle)
template <int VB> __device__ __forceinline__ uint32_t v_off(int r, int c)
{
    return VB == 64 ? swz(r, c) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

struct StateMaps { CUtensorMap k, q, v; };

// The chunks of one sequence for one warp of a unit.
template <int VB, int KW>
__device__ __forceinline__ bool state_pass(const Args &p, unsigned char *sm, uint64_t *full, uint64_t *empty, int u,
                                           const Place &pl, int h, int v0, float (&S)[8][4])
{
    using L = St<VB>;
    const int lane = threadIdx.x & 31, q2 = 2 * (lane & 3);
    float4 *xb = reinterpret_cast<float4 *>(sm + L::kX + u * L::kUnit);  // [2][8][32]
    float4 *ob = xb + 2 * 8 * 32, *ub = ob + 2 * 4 * 32;                 // [2][4][32]
    const int nc = (pl.len + kC - 1) / kC;
    bool good = true;
    // row within an ldmatrix of B operands: tokens in rows (lane / 16 picks the second tile), or key rows transposed
    const int rowB = (lane & 7) + ((lane >> 4) << 3), pcB = (lane >> 3) & 1;
    const int rowT = (lane & 7) + (((lane >> 3) & 1) << 3), pcT = lane >> 4;
    constexpr int pr0 = KW == 0 ? 0 : 1, pr1 = KW == 0 ? 3 : 2;   // this warp's pairs of token tiles
    constexpr int or0 = KW == 0 ? 1 : 0, or1 = KW == 0 ? 2 : 3;   // the other's
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
        const int st = c % L::kStages;
        unsigned char *base = sm + st * L::kStage;
        const uint32_t sb = smem_u32(base);
        const int n = min(kC, pl.len - c * kC);
        // after a wait that gave up the warp goes on without waiting, so that every barrier is met
        if (good) good = mbar_wait_bounded(&full[st], (uint32_t)((c / L::kStages) & 1), kStSpin);
        if (n < kC) {  // the last chunk: what follows the sequence in K and V counts as zero
            const int t = threadIdx.x;
            for (int x = t; x < (kC - n) * 16; x += 32 * L::kWarps)
                *reinterpret_cast<uint4 *>(base + ((x >> 3) & 1) * 8192 + (n + (x >> 4)) * 128 + (x & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            for (int x = t; x < (kC - n) * (VB / 8); x += 32 * L::kWarps)
                *reinterpret_cast<uint4 *>(base + L::kV + n * VB * 2 + x * 16) = make_uint4(0, 0, 0, 0);
            named_bar_sync(1 + L::kUnits, 32 * L::kWarps);
        }
        const float *sx = reinterpret_cast<const float *>(base + L::kBlk + kBlkX);
        // X^T and Q S0, over this warp's 64 key rows
        float X[8][4], O[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[j][e] = O[j][e] = 0.f;
        {
            uint32_t ah[4][4], al[4][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    split2(S[2 * ks + e][0], S[2 * ks + e][1], ah[ks][2 * e], al[ks][2 * e]);
                    split2(S[2 * ks + e][2], S[2 * ks + e][3], ah[ks][2 * e + 1], al[ks][2 * e + 1]);
                }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) {
                    uint32_t b[4];
                    ldsm4(b, sb + KW * 8192 + swz(16 * jp + rowB, 2 * ks + pcB));
                    mma(X[2 * jp], ah[ks], b[0], b[1]);
                    mma(X[2 * jp + 1], ah[ks], b[2], b[3]);
                    mma(X[2 * jp], al[ks], b[0], b[1]);
                    mma(X[2 * jp + 1], al[ks], b[2], b[3]);
                }
#pragma unroll
            for (int j = 0; j < 8; ++j) xb[(KW * 8 + j) * 32 + lane] = make_float4(X[j][0], X[j][1], X[j][2], X[j][3]);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) {
                    uint32_t b[4];
                    ldsm4(b, sb + L::kQ + KW * 8192 + swz(16 * jp + rowB, 2 * ks + pcB));
                    mma(O[2 * jp], ah[ks], b[0], b[1]);
                    mma(O[2 * jp + 1], ah[ks], b[2], b[3]);
                }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ob[(KW * 4 + e) * 32 + lane] = make_float4(O[2 * or0 + e][0], O[2 * or0 + e][1], O[2 * or0 + e][2], O[2 * or0 + e][3]);
            ob[(KW * 4 + 2 + e) * 32 + lane] = make_float4(O[2 * or1 + e][0], O[2 * or1 + e][1], O[2 * or1 + e][2], O[2 * or1 + e][3]);
        }
        named_bar_sync(1 + u, 64);
        // right side V - x X, split; token tiles 2 ks, 2 ks + 1 are k step ks of the next product
        uint32_t rh[4][4], rl[4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t vv[4];  // V^T of tiles 2 ks, 2 ks + 1: value rows g (0, 2) and g + 8 (1, 3)
            ldsm4t(vv, sb + L::kV + v_off<VB>(16 * ks + rowB, 2 * u + pcB));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * ks + e;
                const float4 o = xb[((1 - KW) * 8 + j) * 32 + lane];
                const float2 cx = *reinterpret_cast<const float2 *>(sx + 8 * j + q2);
                const float r0 = fmaf(-cx.x, X[j][0] + o.x, lo_f(vv[2 * e])), r1 = fmaf(-cx.y, X[j][1] + o.y, hi_f(vv[2 * e]));
                const float r2 = fmaf(-cx.x, X[j][2] + o.z, lo_f(vv[2 * e + 1])), r3 = fmaf(-cx.y, X[j][3] + o.w, hi_f(vv[2 * e + 1]));
                split2(r0, r1, rh[ks][2 * e], rl[ks][2 * e]);
                split2(r2, r3, rh[ks][2 * e + 1], rl[ks][2 * e + 1]);
            }
        }
        // U^T of this warp's token tiles
        float U[8][4];
#pragma unroll
        for (int pi = 0; pi < 2; ++pi) {
            const int pr = pi ? pr1 : pr0;
#pragma unroll
            for (int e = 0; e < 4; ++e) U[2 * pr][e] = U[2 * pr + 1][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks <= pr; ++ks) {
                uint32_t bh[4], bl[4];
                const uint32_t off = swz(16 * pr + rowB, 2 * ks + pcB);
                ldsm4(bh, sb + L::kBlk + off);
                ldsm4(bl, sb + L::kBlk + kBlkTl + off);
                mma(U[2 * pr], rh[ks], bh[0], bh[1]);
                mma(U[2 * pr + 1], rh[ks], bh[2], bh[3]);
                mma(U[2 * pr], rl[ks], bh[0], bh[1]);
                mma(U[2 * pr + 1], rl[ks], bh[2], bh[3]);
                mma(U[2 * pr], rh[ks], bl[0], bl[1]);
                mma(U[2 * pr + 1], rh[ks], bl[2], bl[3]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                ub[(KW * 4 + 2 * pi + e) * 32 + lane] =
                    make_float4(U[2 * pr + e][0], U[2 * pr + e][1], U[2 * pr + e][2], U[2 * pr + e][3]);
        }
        named_bar_sync(1 + u, 64);
#pragma unroll
        for (int pi = 0; pi < 2; ++pi)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * (pi ? or1 : or0) + e;
                const float4 o = ub[((1 - KW) * 4 + 2 * pi + e) * 32 + lane];
                U[j][0] = o.x; U[j][1] = o.y; U[j][2] = o.z; U[j][3] = o.w;
            }
        // S^T = exp(G_last) S^T + (x U)^T K over this warp's key rows
        const float gl = sx[3 * kC];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[j][e] *= gl;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * ks + e;
                const float2 cu = *reinterpret_cast<const float2 *>(sx + 2 * kC + 8 * j + q2);
                split2(cu.x * U[j][0], cu.y * U[j][1], ah[2 * e], al[2 * e]);
                split2(cu.x * U[j][2], cu.y * U[j][3], ah[2 * e + 1], al[2 * e + 1]);
            }
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) {
                uint32_t b[4];
                ldsm4t(b, sb + KW * 8192 + swz(16 * ks + rowT, 2 * jp + pcT));
                mma(S[2 * jp], ah, b[0], b[1]);
                mma(S[2 * jp + 1], ah, b[2], b[3]);
                mma(S[2 * jp], al, b[0], b[1]);
                mma(S[2 * jp + 1], al, b[2], b[3]);
            }
        }
        // O^T of this warp's token tiles: x (Q S0) + P U
        uint32_t uh[4][4];
#pragma unroll
        for (int ks = 0; ks <= pr1; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uh[ks][2 * e] = pack2(U[2 * ks + e][0], U[2 * ks + e][1]);
                uh[ks][2 * e + 1] = pack2(U[2 * ks + e][2], U[2 * ks + e][3]);
            }
        uint32_t om[4][2];
#pragma unroll
        for (int pi = 0; pi < 2; ++pi) {
            const int pr = pi ? pr1 : pr0;
            float o[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * pr + e;
                const float4 w = ob[((1 - KW) * 4 + 2 * pi + e) * 32 + lane];
                const float2 co = *reinterpret_cast<const float2 *>(sx + kC + 8 * j + q2);
                o[e][0] = co.x * (O[j][0] + w.x);
                o[e][1] = co.y * (O[j][1] + w.y);
                o[e][2] = co.x * (O[j][2] + w.z);
                o[e][3] = co.y * (O[j][3] + w.w);
            }
#pragma unroll
            for (int ks = 0; ks <= pr; ++ks) {
                uint32_t b[4];
                ldsm4(b, sb + L::kBlk + kBlkP + swz(16 * pr + rowB, 2 * ks + pcB));
                mma(o[0], uh[ks], b[0], b[1]);
                mma(o[1], uh[ks], b[2], b[3]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                om[2 * pi + e][0] = pack2(o[e][0], o[e][1]);
                om[2 * pi + e][1] = pack2(o[e][2], o[e][3]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        // the 32 tokens x 16 values as rows of 32 bytes, staged in this warp's own part of xb: the other
        // warp read it before the second barrier
        unsigned char *stg = reinterpret_cast<unsigned char *>(xb + KW * 8 * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            stsm2t(smem_u32(stg) + (uint32_t)((8 * j + (lane & 7)) * 32 + ((((lane >> 3) & 1) ^ ((lane >> 2) & 1)) << 4)), om[j][0], om[j][1]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int x = lane + 32 * i, r = x >> 1, half = x & 1;  // row r of the staged 32
            const int t = r < 16 ? 16 * pr0 + r : 16 * pr1 + r - 16;
            const uint4 w = *reinterpret_cast<const uint4 *>(stg + r * 32 + ((half ^ ((r >> 2) & 1)) << 4));
            if (t < n) {
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.rows.out) +
                                   ((int64_t)pl.t0 + c * kC + t) * p.rows.out_stride + (size_t)h * kD + v0 + 16 * u + 8 * half;
                *reinterpret_cast<uint4 *>(o) = w;
            }
        }
        __syncwarp();
    }
    return good;
}

template <int VB>
__global__ void __launch_bounds__(St<VB>::kThreads, 1)
gdr_state_kernel(const __grid_constant__ StateMaps maps, const __grid_constant__ Args p,
                 const unsigned char *__restrict__ blocks, int64_t n_chunks, int box_rows)
{
    using L = St<VB>;
    extern __shared__ unsigned char sm_raw[];
    unsigned char *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::kBar), *empty = full + L::kStages;
    Place *place = reinterpret_cast<Place *>(empty + L::kStages);
    int *ok = reinterpret_cast<int *>(place + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kVBlocks = kD / VB;
    const int vb = blockIdx.x % kVBlocks;
    const int h = (blockIdx.x / kVBlocks) % p.H, seq = blockIdx.x / (kVBlocks * p.H);
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], L::kWarps);
        }
        fence_mbar_init();
    }
    if (warp == L::kWarps) {
        Place pl;
        const bool good = find_place(p.cu, p.N, p.total_T, n_chunks, 0, seq, pl);
        if (lane == 0) {
            *place = pl;
            *ok = good;
        }
    }
    __syncthreads();
    int src, dst;
    if (!slots_ok(p, seq, src, dst) || !*ok) {  // the same for every thread
        if (threadIdx.x == 0) set_err(p.err);
        return;
    }
    const Place pl = *place;
    const int nc = (pl.len + kC - 1) / kC;
    if (warp == L::kWarps) {
        if (lane == 0) {
            const int hk = h / p.G;
            bool good = true;
            for (int c = 0; c < nc; ++c) {
                const int st = c % L::kStages;
                if (c >= L::kStages && !mbar_wait_bounded(&empty[st], (uint32_t)(((c / L::kStages) - 1) & 1), kStSpin)) {
                    good = false;
                    break;
                }
                unsigned char *b = sm + st * L::kStage;
                const int t = pl.t0 + c * kC;
                mbar_arrive_expect_tx(&full[st], (uint32_t)(box_rows * (4 * 128 + VB * 2) + kBlkBytes));
                tma_load_2d(b, &maps.k, hk * kD, t, &full[st]);
                tma_load_2d(b + 8192, &maps.k, hk * kD + 64, t, &full[st]);
                bulk_g2s(b + L::kBlk, blocks + ((size_t)(pl.first + c) * p.H + h) * kBlkBytes, kBlkBytes, &full[st]);
                tma_load_2d(b + L::kV, &maps.v, h * kD + vb * VB, t, &full[st]);
                tma_load_2d(b + L::kQ, &maps.q, hk * kD, t, &full[st]);
                tma_load_2d(b + L::kQ + 8192, &maps.q, hk * kD + 64, t, &full[st]);
            }
            if (!good) {
                if (p.err) atomicExch(p.err, KDA_ERR_TIMEOUT);
                for (int s = 0; s < L::kStages; ++s) mbar_wait_bounded(&full[s], 0, 1u << 16);  // copies in flight land
            }
        }
        return;
    }
    // this warp's part of S^T: value rows g, g + 8 of unit u, key rows 64 kw ..
    const int u = warp >> 1, kw = warp & 1, g = lane >> 2, q2 = 2 * (lane & 3);
    const size_t at = (size_t)(64 * kw + q2) * kD + vb * VB + 16 * u + g;
    float S[8][4];
    if (src >= 0) {
        const float *s = p.S + ((size_t)src * p.H + h) * kD * kD + at;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[j][e] = s[(8 * j + (e & 1)) * kD + 8 * (e >> 1)];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[j][e] = 0.f;
    }
    const bool good = kw == 0 ? state_pass<VB, 0>(p, sm, full, empty, u, pl, h, vb * VB, S)
                              : state_pass<VB, 1>(p, sm, full, empty, u, pl, h, vb * VB, S);
    if (!good) {
        if (lane == 0 && p.err) atomicExch(p.err, KDA_ERR_TIMEOUT);
        return;
    }
    float *d = p.S + ((size_t)dst * p.H + h) * kD * kD + at;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[(8 * j + (e & 1)) * kD + 8 * (e >> 1)] = S[j][e];
}

cudaError_t rows_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t stride, int box_cols, int box_rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? stride : cols) * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int VB>
cudaError_t launch_state(const Args &p, const unsigned char *blocks, int64_t n_chunks, cudaStream_t stream)
{
    const int64_t T = p.total_T;
    const int box = T < kC ? (T > 0 ? (int)T : 1) : kC;
    StateMaps m = {};
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        const int64_t Dk = (int64_t)(p.H / p.G) * kD, Dv = (int64_t)p.H * kD;
        if ((e = rows_map(&m.k, p.rows.k, T, Dk, p.rows.k_stride, 64, box)) != cudaSuccess ||
            (e = rows_map(&m.q, p.rows.q, T, Dk, p.rows.q_stride, 64, box)) != cudaSuccess ||
            (e = rows_map(&m.v, p.rows.v, T, Dv, p.rows.v_stride, VB, box)) != cudaSuccess)
            return e;
    }
    e = cudaFuncSetAttribute(gdr_state_kernel<VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, St<VB>::kSmem);
    if (e != cudaSuccess) return e;
    gdr_state_kernel<VB><<<(unsigned)((int64_t)p.N * p.H * (kD / VB)), St<VB>::kThreads, St<VB>::kSmem, stream>>>(
        m, p, blocks, n_chunks, box);
    return cudaGetLastError();
}

}  // namespace

size_t chunked_workspace_bytes(int64_t n_chunks, int32_t H) { return 256 + (size_t)n_chunks * H * kBlkBytes; }

cudaError_t launch_chunked(const Args &p, int64_t n_chunks, void *ws, int sms, cudaStream_t stream)
{
    unsigned char *blocks = static_cast<unsigned char *>(ws) +
                            ((128 - (reinterpret_cast<uintptr_t>(ws) & 127)) & 127);
    cudaError_t e;
    if (n_chunks > 0) {
        const int Hk = p.H / p.G;
        e = cudaFuncSetAttribute(gdr_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrepSmem);
        if (e != cudaSuccess) return e;
        gdr_prep_kernel<<<(unsigned)(n_chunks * Hk), kPrepThreads, kPrepSmem, stream>>>(p, blocks, n_chunks, Hk);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return (int64_t)p.N * p.H * 4 <= 2 * (int64_t)sms ? launch_state<32>(p, blocks, n_chunks, stream)
                                                      : launch_state<64>(p, blocks, n_chunks, stream);
}

}  // namespace gdr
}  // namespace kda
