// kda_gdr_prefill.cu - the gated delta rule over packed sequences of BF16 rows, in chunks of
// C = 64 tokens.
//
// With G the cumulative log decay inside a chunk (a scalar per token) and S0 the state before it,
//   A[t][i] = beta_t (k^_t . k^_i) exp(G_t - G_i)  (i < t),   T = (I + A)^-1
//   U = T Diag(beta) (V - Diag(exp G) K^ S0)
//   O = Diag(exp G) Q^ S0 + P U,   P[t][i] = (q^_t . k^_i) exp(G_t - G_i)  (i <= t)
//   S = exp(G_last) S0 + (Diag(exp(G_last - G)) K^)^T U
// which is the token recurrence exactly in real arithmetic. Every exponent is <= 0.
//
// Two kernels:
//   gdr_prep_kernel   per (chunk, key head): the products K K^T and Q K^T once, then for each of its
//                     value heads the decays, A, T, and one block of T, P and four scalars a token for
//                     the second kernel
//   gdr_state_kernel  per (sequence, head, 32 value columns): the serial pass over the chunks
//
// The raw BF16 rows of K, Q and V are the matrix operands as they are, so those operands are exact;
// the norms and the decays are FP32 scalars a token, applied to FP32 accumulators. What carries the
// state is kept to about 16 bits: S, beta (V - ..), T and U go into the products as a BF16 high part and a
// BF16 low part (x - high), products of two such factors as hi hi + lo hi + hi lo, and sums are FP32.
// With single BF16 operands the state would be off by 2^-9 a chunk. The output, which is rounded to
// BF16 itself, takes the high part of S alone, and P and U in two parts: with P in one it was 1.4 times as far
// from the exact result as that rounding for keys that have nothing in common, and 3 to 8 times where they are
// all positive or nearly equal, since Q S0 and P U then cancel. So it is 1.0 times, and 1.4 at the most measured.
// Keeping P's low part costs 1 to 5% (8192 tokens, 32 heads: 287 -> 295 us).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_gdr.cuh"
#include "kda_launch.cuh"
#include "kda_tc.cuh"
#include "kda_wait.cuh"

namespace kda {
namespace gdr {
namespace {

// One block per (chunk, value head), in two parts that go to different rings of the second kernel.
// Tiles: BF16, 64 rows t of 64 columns i (128 bytes), 16-byte piece c of row t at c ^ (t & 7); only the
// 16 x 16 blocks on and below the diagonal are meaningful.
//   T high | T low | FP32 scalars: beta rk exp G [64], beta [64], rk exp(G_last - G) [64], exp G_last
//   P high | rq exp G [64]
// P's low part lies where the tiles are not used: that of a 16 x 16 block below the diagonal in the block's mirror
// image in P's tile (not itself mirrored); of the diagonal blocks the lower left 8 x 8 in the upper right one, and the
// two 8 x 8 on the diagonal in columns 16 .. 63 of T high's rows 0 .. 15 (pd_off), which go to P's ring as well.
constexpr int kTl = 8192, kTx = 16384, kPartT = kTx + 1024;
constexpr int kPx = 8192, kPartP = kPx + 256, kPd = 2048;
constexpr int kBlkBytes = kPartT + kPartP;

__device__ __forceinline__ uint32_t swz(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }
// Row r of P's low part in the j-th 8 x 8 on the diagonal, in T high's tile. (As swz(8 + r, j - 4) for the last two,
// nvcc 13.0.88 addressed piece 0 of every row.)
__device__ __forceinline__ uint32_t pd_off(int j, int r) { return (j < 6 ? 0 : 1024) + swz(r, j < 6 ? 2 + j : j - 4); }

// Shared memory read as matrix operands. Volatile keeps these behind the barrier that the data came with;
// what this thread's warp wrote itself is followed by __syncwarp.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void stsm2t(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// c (16 x 8, FP32) += a (16 x 16, BF16) b (16 x 8, BF16). Lane (g, q) = (lane / 4, lane % 4): c = rows
// g, g + 8 at columns 2q, 2q + 1; a = those rows at k 2q, 2q + 1 (+ 8); b = k 2q, 2q + 1 (+ 8) of column g.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
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

// A sequence: its rows t0 .. t0 + len - 1 and its first chunk.
struct Place { int seq, t0, len, first; };

// What threads first, first + step, .. of a block read of cu_seqlens: whether it is one of total_T tokens, the
// chunks before sequence seq and all chunks (which cannot wrap in one that is right: the host has checked that
// chunks x heads fit 28 bits). The sums are over the warp. Shared by all of a state block's warps, and in the
// prep only the first item's: 4096 sequences of 1 to 16 tokens and 8 heads 3.9 ms (25.5 ms with one warp's scan
// for each block and item), 256 of them 221 us (281).
struct Scan { int ok; uint32_t before, all; };
__device__ __forceinline__ Scan scan_cu(const Args &p, int first, int step, int seq)
{
    bool ok = true;
    uint32_t before = 0, all = 0;
#pragma unroll 4
    for (int s = first; s < p.N; s += step) {
        const int b = __ldg(p.cu + s), e = __ldg(p.cu + s + 1);
        ok = ok && b >= 0 && e >= b && e <= p.total_T && (s > 0 || b == 0) && (s < p.N - 1 || e == p.total_T);
        const uint32_t c = ((uint32_t)e - (uint32_t)b + kC - 1) / kC;
        all += c;
        before += s < seq ? c : 0u;
    }
    return {__all_sync(0xFFFFFFFFu, ok), __reduce_add_sync(0xFFFFFFFFu, before), __reduce_add_sync(0xFFFFFFFFu, all)};
}

// One warp: the sequence that has chunk `want`, from the place `out` of an earlier chunk on (or of sequence 0). For a
// cu_seqlens that is right; false when there is none.
__device__ __forceinline__ bool find_chunk(const Args &p, int want, Place &out)
{
    const int lane = threadIdx.x & 31;
    int base = out.first;
    for (int s0 = out.seq; s0 < p.N; s0 += 32) {
        const int s = s0 + lane;
        const int b = s < p.N ? __ldg(p.cu + s) : 0, e = s < p.N ? __ldg(p.cu + s + 1) : 0;
        const int mine = (e - b + kC - 1) / kC;
        int nc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, nc, o);
            if (lane >= o) nc += x;
        }
        const int before = base + nc - mine;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, want >= before && want < before + mine);
        if (m) {
            const int l = __ffs(m) - 1;
            out.seq = s0 + l;
            out.t0 = __shfl_sync(0xFFFFFFFFu, b, l);
            out.len = __shfl_sync(0xFFFFFFFFu, e, l) - out.t0;
            out.first = __shfl_sync(0xFFFFFFFFu, before, l);
            return true;
        }
        base += __shfl_sync(0xFFFFFFFFu, nc, 31);
    }
    return false;
}

// (h, l) += (x, y) for sums kept as two FP32, |l| far below |h| (the exact error of the addition by Knuth's
// two-sum)
__device__ __forceinline__ void add2(float &h, float &l, float x, float y)
{
    const float s = h + x, t = s - h;
    const float e = (h - (s - t)) + (x - t) + (l + y);
    h = s + e;
    l = e - (h - s);
}

// ---------------------------------------------------------------- prep
// 128 threads; warp w has the rows t = 16 w .. 16 w + 15. T by blocks of 16 rows: the diagonal blocks
// D_w = (I + A_ww)^-1 by forward substitution in FP32, a warp each, one column a lane; below them
//   T[w][:] = -D_w sum_{j < w} A[w][j] T[j][:]
// on the tensor cores with split factors, three barriers deep. 61 to 64 us for 4096 (chunk, value head) pairs of
// two value heads a key head (92 us with the whole inverse by forward substitution, a column a lane; P is written
// before the inverse is formed, as its registers would spill otherwise); bound by the latency of its phases, 12
// warps an SM, with DRAM at 22% and compute throughput at 34%.
// Shared memory: two buffers of K and Q rows (the next item's are loaded while one is computed; a block is
// built in the place of the rows that it came from), A's diagonal blocks, scalars of up to four value heads.
constexpr int kPrepThreads = 128, kPrepPerSm = 3;
constexpr int kPsQ = 16384, kPsBuf = 32768;
constexpr int kDp = 20;                               // row pitch of a diagonal block of A^T
constexpr int kScal = 5 * kC + 4;                     // per head: G high, G low, beta, exp G, exp(G_last - G); exp G_last
constexpr int kPsDiag = 2 * kPsBuf, kPsScal = kPsDiag + 4 * 16 * kDp * 4, kPsNorm = kPsScal + 4 * kScal * 4;
constexpr int kPrepSmem = kPsNorm + 2 * kC * 4;
static_assert(kBlkBytes <= kPsBuf && kPrepPerSm * (kPrepSmem + 1024) <= 228 * 1024, "prep shared memory");

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

__global__ void __launch_bounds__(kPrepThreads, kPrepPerSm)
gdr_prep_kernel(const __grid_constant__ Args p, unsigned char *__restrict__ blocks, int n_chunks, int Hk)
{
    extern __shared__ __align__(1024) unsigned char sm_all[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q2 = 2 * (lane & 3);
    float *sRk = reinterpret_cast<float *>(sm_all + kPsNorm), *sRq = sRk + kC;
    float *scal = reinterpret_cast<float *>(sm_all + kPsScal);
    float *diag = reinterpret_cast<float *>(sm_all + kPsDiag) + warp * 16 * kDp;
    const int n_items = n_chunks * Hk;  // (chunk, key head), key heads fastest
    struct Item { int chunk, hk, n; int64_t t0; };
    Place pl = {0, 0, 0, 0};  // of the last chunk that was located; items only go up
    auto locate = [&](int item, Item &x) {
        x.chunk = item / Hk;
        x.hk = item - x.chunk * Hk;
        if (!find_chunk(p, x.chunk, pl)) return false;
        const int pos = (x.chunk - pl.first) * kC;
        x.t0 = (int64_t)pl.t0 + pos;
        x.n = min(kC, pl.len - pos);
        return true;
    };
    // rows n .. 63 read as zeros
    auto load_rows = [&](const Item &x, unsigned char *sm) {
        const __nv_bfloat16 *kg = static_cast<const __nv_bfloat16 *>(p.rows.k) + x.t0 * p.rows.k_stride + (size_t)x.hk * kD;
        const __nv_bfloat16 *qg = static_cast<const __nv_bfloat16 *>(p.rows.q) + x.t0 * p.rows.q_stride + (size_t)x.hk * kD;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (tid >> 4) + 8 * i, c = tid & 15;  // 16 pieces of 16 bytes a row
            const uint32_t off = (uint32_t)(c >> 3) * 8192 + swz(r, c & 7);
            const int rr = r < x.n ? r : 0;
            cp_async16(sm + off, kg + rr * p.rows.k_stride + 8 * c, r < x.n ? 16 : 0);
            cp_async16(sm + kPsQ + off, qg + rr * p.rows.q_stride + 8 * c, r < x.n ? 16 : 0);
        }
    };
    // decay and beta logits of value head j + warp, two tokens a lane
    struct Logits { float a[2], b[2], A_log, dt_bias; };
    auto load_logits = [&](const Item &x, int j, Logits &l) {
        if (j + warp >= p.G) return;
        const int h = x.hk * p.G + j + warp;
        const __nv_bfloat16 *ag = static_cast<const __nv_bfloat16 *>(p.rows.a) + x.t0 * p.rows.a_stride + h;
        const __nv_bfloat16 *bg = static_cast<const __nv_bfloat16 *>(p.rows.b) + x.t0 * p.rows.b_stride + h;
        l.A_log = __ldg(p.A_log + h);
        l.dt_bias = __ldg(p.dt_bias + h);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = min(2 * lane + e, x.n - 1);
            l.a[e] = __bfloat162float(ag[t * p.rows.a_stride]);
            l.b[e] = __bfloat162float(bg[t * p.rows.b_stride]);
        }
    };
    // The sums are kept as two FP32, so that differences of tokens far down a strongly decaying chunk stay exact.
    auto decays = [&](const Item &x, int j, const Logits &l) {
        if (j + warp >= p.G) return;
        const float expA = expf(l.A_log);
        float *s = scal + warp * kScal;
        float ga[2], be[2];  // base-2 logarithms
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool in = 2 * lane + e < x.n;
            ga[e] = in ? log_decay(l.a[e], l.dt_bias, expA) * 1.4426950408889634f : 0.f;
            be[e] = in ? sigmoidf_(l.b[e]) : 0.f;
        }
        float ch = ga[0], cl = 0.f;
        add2(ch, cl, ga[1], 0.f);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float xh = __shfl_up_sync(0xFFFFFFFFu, ch, o), xl = __shfl_up_sync(0xFFFFFFFFu, cl, o);
            if (lane >= o) add2(ch, cl, xh, xl);
        }
        const float lh = __shfl_sync(0xFFFFFFFFu, ch, 31), ll = __shfl_sync(0xFFFFFFFFu, cl, 31);
        float h0 = ch, l0 = cl;  // of token 2 lane
        add2(h0, l0, -ga[1], 0.f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            const float Gh = e ? ch : h0, Gl = e ? cl : l0;
            s[t] = Gh;
            s[kC + t] = Gl;
            s[2 * kC + t] = be[e];
            s[3 * kC + t] = ex2(Gh);
            s[4 * kC + t] = ex2((lh - Gh) + (ll - Gl));
        }
        if (lane == 0) s[5 * kC] = ex2(lh);
    };

    launch_dependents();
    int item = blockIdx.x, buf = 0;
    Item cur, nxt;
    const Scan cu = scan_cu(p, lane, 32, 0);  // a warp each: the same for every thread
    if (!cu.ok || cu.all != (uint32_t)n_chunks || !locate(item, cur)) {
        if (tid == 0) set_err(p.err);
        return;
    }
    Logits lg;
    load_rows(cur, sm_all);
    load_logits(cur, 0, lg);
#pragma unroll 1
    for (; item < n_items; item += gridDim.x, buf ^= 1, cur = nxt) {
        unsigned char *sm = sm_all + buf * kPsBuf;
        const uint32_t sK = smem_u32(sm), sQ = sK + kPsQ;
        const int64_t chunk = cur.chunk;
        const int hk = cur.hk;
        const bool more = item + (int)gridDim.x < n_items;
        if (more) locate(item + gridDim.x, nxt);
        decays(cur, 0, lg);
        cp_async_wait_all();
        if (tid == 0) bulk_wait_read_all();  // the other buffer's block has been read
        __syncthreads();
        if (more) {
            load_rows(nxt, sm_all + (buf ^ 1) * kPsBuf);
            load_logits(nxt, 0, lg);
        }
        {  // norms: two threads a row of K and of Q
            const int r = tid >> 1, half = tid & 1;
            float kk = 0.f, qq = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t off = (uint32_t)half * 8192 + swz(r, c);
                const uint4 a = *reinterpret_cast<const uint4 *>(sm + off);
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
        // K K^T and Q K^T: rows t of this warp, columns i <= 16 w + 15
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
        const int rowT = (lane & 7) + (((lane >> 3) & 1) << 3), pcT = lane >> 4;  // ldmatrix.trans of B operands
#pragma unroll 1
        for (int j = 0; j < p.G; ++j) {
            unsigned char *blk = sm;
            const uint32_t sT = sK;
            if (j && (j & 3) == 0) {
                __syncthreads();  // every warp has read the last four heads' scalars
                Logits l;
                load_logits(cur, j, l);
                decays(cur, j, l);
            }
            if (j == 0 || (j & 3) == 0) __syncthreads();  // scalars and norms are written
            const float *s = scal + (j & 3) * kScal;
            if (j) {
                if (tid == 0) bulk_wait_read_all();  // the previous head's block has been read
                __syncthreads();
            }
            // A and P from the products: A's blocks left of the diagonal stay in registers as split A operands, P goes
            // to the block, which takes the place of K and Q (read before the first head's barrier above)
            uint32_t ah[3][4], al[3][4];
            {
                const int ta = 16 * warp + g;
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
                    if ((nt >> 1) > warp) break;
                    const int i = 8 * nt + q2;
                    const float2 gh = *reinterpret_cast<const float2 *>(s + i), gl = *reinterpret_cast<const float2 *>(s + kC + i);
                    const float2 rk = *reinterpret_cast<const float2 *>(sRk + i);
                    float av[2][2], pv[2][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const float x = (Gh[e] - (f ? gh.y : gh.x)) + (Gl[e] - (f ? gl.y : gl.x));
                            const float d = ex2(x) * (f ? rk.y : rk.x);
                            av[e][f] = i + f < ta + 8 * e ? fb[e] * d * kk[nt][2 * e + f] : 0.f;
                            pv[e][f] = i + f <= ta + 8 * e ? fq[e] * d * qk[nt][2 * e + f] : 0.f;
                        }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool diag8 = nt == 2 * warp + e;  // 8 x 8 on the diagonal
                        if (nt <= 2 * warp + e) {               // or below it
                            uint32_t ph, pl;
                            split2(pv[e][0], pv[e][1], ph, pl);
                            *reinterpret_cast<uint32_t *>(blk + kPartT + swz(16 * warp + g + 8 * e, nt) + 2 * q2) = ph;
                            unsigned char *low = diag8                ? blk + pd_off(nt, g)
                                                 : (nt >> 1) == warp ? blk + kPartT + swz(16 * warp + g, nt + 1)
                                                                     : blk + kPartT + swz(16 * (nt >> 1) + g + 8 * e, 2 * warp + (nt & 1));
                            *reinterpret_cast<uint32_t *>(low + 2 * q2) = pl;
                        }
                        if ((nt >> 1) < warp) {
                            if (nt < 6) split2(av[e][0], av[e][1], ah[(nt >> 1) % 3][2 * (nt & 1) + e], al[(nt >> 1) % 3][2 * (nt & 1) + e]);
                        } else {
#pragma unroll
                            for (int f = 0; f < 2; ++f) diag[(8 * (nt & 1) + q2 + f) * kDp + g + 8 * e] = av[e][f];
                        }
                    }
                }
            }
            __syncwarp();
            const int jc = lane & 15;  // the diagonal block's inverse: column lane & 15
            float acc[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[r] = r == jc ? 1.f : 0.f;
#pragma unroll
            for (int r = 0; r < 15; ++r) {
                float a[16];
#pragma unroll
                for (int e = (r + 1) / 4; e < 4; ++e)
                    *reinterpret_cast<float4 *>(a + 4 * e) = *reinterpret_cast<const float4 *>(diag + r * kDp + 4 * e);
#pragma unroll
                for (int r2 = r + 1; r2 < 16; ++r2) acc[r2] = fmaf(-a[r2], acc[r], acc[r2]);
            }
            {
                unsigned char *dst = blk + (lane & 16 ? kTl : 0) + 2 * (jc & 7);  // lanes 0..15 the high part, 16..31 the low
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const __nv_bfloat16 hi = __float2bfloat16_rn(acc[r]);
                    const __nv_bfloat16 lo = __float2bfloat16_rn(acc[r] - __bfloat162float(hi));
                    *reinterpret_cast<__nv_bfloat16 *>(dst + swz(16 * warp + r, 2 * warp + (jc >> 3))) = lane & 16 ? lo : hi;
                }
                if (tid < kC) {
                    float *x = reinterpret_cast<float *>(blk + kTx);
                    x[tid] = s[2 * kC + tid] * sRk[tid] * s[3 * kC + tid];
                    x[kC + tid] = s[2 * kC + tid];
                    x[2 * kC + tid] = sRk[tid] * s[4 * kC + tid];
                    if (tid == 0) x[3 * kC] = s[5 * kC];
                    reinterpret_cast<float *>(blk + kPartT + kPx)[tid] = sRq[tid] * s[3 * kC + tid];
                }
            }
            float Y[6][4];
#pragma unroll
            for (int i = 0; i < 6; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) Y[i][e] = 0.f;
#pragma unroll
            for (int jb = 0; jb < 3; ++jb) {
                __syncthreads();  // block row jb of T is complete
                if (warp <= jb) continue;
#pragma unroll
                for (int np = 0; np <= jb; ++np) {
                    uint32_t bh[4], bl[4];
                    const uint32_t off = swz(16 * jb + rowT, 2 * np + pcT);
                    ldsm4t(bh, sT + off);
                    ldsm4t(bl, sT + kTl + off);
                    mma(Y[2 * np], ah[jb], bh[0], bh[1]);
                    mma(Y[2 * np + 1], ah[jb], bh[2], bh[3]);
                    mma(Y[2 * np], al[jb], bh[0], bh[1]);
                    mma(Y[2 * np + 1], al[jb], bh[2], bh[3]);
                    mma(Y[2 * np], ah[jb], bl[0], bl[1]);
                    mma(Y[2 * np + 1], ah[jb], bl[2], bl[3]);
                }
                if (warp == jb + 1) {  // T[w][:] = -D Y: Y goes to its own place in T first, to be read as a B operand
                    uint32_t dh[4], dl[4];
                    const uint32_t od = swz(16 * warp + (lane & 15), 2 * warp + (lane >> 4));
                    ldsm4(dh, sT + od);
                    ldsm4(dl, sT + kTl + od);
#pragma unroll
                    for (int nt = 0; nt < 2 * jb + 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t h, l;
                            split2(-Y[nt][2 * e], -Y[nt][2 * e + 1], h, l);
                            unsigned char *dst = blk + swz(16 * warp + g + 8 * e, nt) + 2 * q2;
                            *reinterpret_cast<uint32_t *>(dst) = h;
                            *reinterpret_cast<uint32_t *>(dst + kTl) = l;
                        }
                    __syncwarp();
#pragma unroll
                    for (int np = 0; np <= jb; ++np) {
                        uint32_t bh[4], bl[4];
                        const uint32_t off = swz(16 * warp + rowT, 2 * np + pcT);
                        ldsm4t(bh, sT + off);
                        ldsm4t(bl, sT + kTl + off);
                        __syncwarp();
                        float z[2][4] = {};
                        mma(z[0], dh, bh[0], bh[1]);
                        mma(z[1], dh, bh[2], bh[3]);
                        mma(z[0], dl, bh[0], bh[1]);
                        mma(z[1], dl, bh[2], bh[3]);
                        mma(z[0], dh, bl[0], bl[1]);
                        mma(z[1], dh, bl[2], bl[3]);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t h, l;
                                split2(z[x][2 * e], z[x][2 * e + 1], h, l);
                                unsigned char *dst = blk + swz(16 * warp + g + 8 * e, 2 * np + x) + 2 * q2;
                                *reinterpret_cast<uint32_t *>(dst) = h;
                                *reinterpret_cast<uint32_t *>(dst + kTl) = l;
                            }
                    }
                }
            }
            tc::fence_smem_to_async();
            __syncthreads();
            if (tid == 0) {
                bulk_s2g(blocks + ((size_t)chunk * p.H + hk * p.G + j) * kBlkBytes, blk, kBlkBytes);
                bulk_commit_group();
            }
        }
    }
    if (tid == 0) bulk_wait_all();
}

// ---------------------------------------------------------------- state
// A block takes 32 MT value columns of one (sequence, head) through its chunks. Everything is held transposed,
// with the 16 MT value columns of a unit as MT times the 16 rows of the MMA: the FP32 accumulators of S^T, X^T
// = S0^T K^T and U^T then have the register layout of the next product's A operand, and the operands in shared
// memory are only read.
//   warps 0-3  the chain: warp 2 u + kw has unit u and the key rows 64 kw .. 64 kw + 63 of S. Its partial
//              sums of X, then half of the token tiles of U, go to the unit's other warp through shared
//              memory. Of each pair of 8-token tiles a warp has one, in turn the first and the second, so
//              that both halves of the triangular product are equal.
//   warps 4-7  the output, one chunk behind the chain at most: unit and token tiles as above, O^T from the
//              high part of S0 and from U, which the chain hands over
//   warp 8     (of a third warpgroup, which leaves its registers to the first) copies: a ring of K, T and V
//              for the chain, one of Q and P for the output
// With MT = 1 what bounds it is the chain of a chunk: 158 MMAs a warp (m16n8k16, 8 cycles each on its quarter
// of the SM) with the exchanges between them, and shared memory, which delivers operands for 16 rows at a
// time: 2370 wavefronts and 540 of arriving copies in the 3400 cycles of a chunk. With MT = 2 an operand
// fetched serves 32 rows. A chunk of it takes longer, two columns' worth of it less; see the rule at the launch.
// Tcgen05 would run the same products in tiles of 64 or 128 rows at four times the MMA rate, but the four
// dependent products of a chunk (64 x 128 x 32 and smaller) would each pay for the way through tensor memory
// and back into shared memory, which lengthens the chain of one sequence. That is no reason for a batch with more
// (sequence, head) pairs than SMs: there 128 columns of a chunk cost 6.5 to 7.2 us of an SM here, and the KDA state
// pass, on tcgen05, takes 2.75. Such a form has not been built.
// 229 us for 32 heads of 8192 tokens (1.8 us a chunk), the tensor pipe 51% busy on the 128 SMs that have a block.
constexpr int kStThreads = 384;
template <int MT> struct St {
    static constexpr int kVB = 32 * MT;
    static constexpr int kNa = MT == 1 ? 3 : 2, kNo = 2, kNh = MT == 1 ? 2 : 1;  // stages of the rings, hand-over buffers
    static constexpr int kT = 16384, kV = kT + kPartT, kSa = kV + kC * kVB * 2;
    static constexpr int kP = 16384, kDiag = kP + kPartP, kSo = 27648;
    static constexpr int kO = kNa * kSa, kX = kO + kNo * kSo;         // X: [2 units][2 kw][8 tiles][MT][32 lanes] float4
    static constexpr int kU = kX + 16384 * MT, kH = kU + 8192 * MT;   // U split: [2][2][4][MT][32] uint4
    static constexpr int kHu = 8192 * MT, kHand = 2 * kHu;            // S [2][8 k steps][MT][32], U split [2][8 tiles][MT][32] uint4
    static constexpr int kStg = kH + kNh * kHand, kBar = kStg + 4096 * MT;
    static constexpr int kSmem = kBar + 384 + 1024;
};
static_assert(St<1>::kSa % 1024 == 0 && St<2>::kSa % 1024 == 0 && St<1>::kSo % 1024 == 0 && St<1>::kV % 1024 == 0 &&
              St<1>::kDiag + kPd <= St<1>::kSo, "stages");
static_assert(St<1>::kSmem <= 232448 && St<2>::kSmem <= 232448, "state kernel shared memory");
// Polls before a wait gives up (a test builds this file with limits that run out). A warp that gave up goes on
// without waiting, so that every named barrier is met, but releases no stage of the rings and writes nothing to
// the output or the states: a stage is filled again only when all its readers have seen the last copies land.
#ifndef KDA_GDR_WAIT_LIMIT
#define KDA_GDR_WAIT_LIMIT (1u << 26)
#endif
constexpr uint32_t kLandSpin = 1u << 26;  // for copies that are on their way when a block ends

struct StateMaps { CUtensorMap k, q, v; };
// full and empty of the two rings; S0 handed over, U handed over, both read; the output is written
struct StBars { uint64_t fa[3], ea[3], fo[2], eo[2], fs[2], fh[2], eh[2], done; };

// byte offset of 16-byte piece c of row r of the V tile (rows of 64 or 128 bytes, TMA's swizzle of that width)
template <int MT> __device__ __forceinline__ uint32_t v_off(int r, int c)
{
    return MT == 2 ? swz(r, c) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
// and of piece c of row r of the staged output (rows of 32 or 64 bytes)
template <int MT> __device__ __forceinline__ uint32_t o_off(int r, int c)
{
    return MT == 2 ? (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) : (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

// Token tiles (8 tokens) of the unit's warp kw: one of each pair, 2 p + own(p).
__device__ __forceinline__ int own(int kw, int p) { return (p ^ kw) & 1; }

// Two barriers at once: even lanes wait for one, odd lanes for the other.
__device__ __forceinline__ bool wait_both(uint64_t *x, uint32_t px, uint64_t *y, uint32_t py)
{
    const bool odd = threadIdx.x & 1;
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(odd ? y : x, odd ? py : px, KDA_GDR_WAIT_LIMIT));
    __syncwarp();
    return ok;
}

// The two k halves of a fragment of 16 values rows by 16, from FP32 pairs, split
__device__ __forceinline__ void split_tile(float2 x, float2 y, uint32_t *h, uint32_t *l)
{
    split2(x.x, x.y, h[0], l[0]);
    split2(y.x, y.y, h[1], l[1]);
}

template <int MT>
__device__ __forceinline__ bool chain_pass(unsigned char *sm, StBars *bar, int u, int kw, int len, float2 (&S)[MT][8][2])
{
    using L = St<MT>;
    const int lane = threadIdx.x & 31, q2 = 2 * (lane & 3);
    float4 *xb = reinterpret_cast<float4 *>(sm + L::kX) + u * (512 * MT) + lane;
    uint4 *ub = reinterpret_cast<uint4 *>(sm + L::kU) + u * (256 * MT) + lane;
    const int nc = (len + kC - 1) / kC;
    bool good = true;  // the same in every lane
    // row and 16-byte piece within an ldmatrix of B operands: two tiles of tokens in rows, or tokens as k
    // (transposed; own tile first), or one tile of tokens with two k steps
    const int rowB = (lane & 7) + ((lane >> 4) << 3), pcB = (lane >> 3) & 1;
    uint32_t offT[4];  // T rows of this warp's tile of pair p, k steps 0 and 1 (steps 2 and 3: ^ 64)
#pragma unroll
    for (int pr = 0; pr < 4; ++pr) offT[pr] = swz(16 * pr + 8 * own(kw, pr) + (lane & 7), lane >> 3);
    int st = 0, pa = 0;
    uint32_t b[2][4][4];          // B operands of a k step, fetched a step ahead
    // Chunk c's stage has arrived and its hand-over buffer is free. peek asks both barriers once, without using
    // the answer yet; enter waits if it was no, and fetches the first B operands.
    auto peek = [&](int c) {
        const bool odd = lane & (c >= L::kNh);
        return mbar_try_wait(odd ? &bar->eh[c % L::kNh] : &bar->fa[st], odd ? (uint32_t)(((c / L::kNh) - 1) & 1) : (uint32_t)pa);
    };
    auto enter = [&](int c, bool ready) {
        unsigned char *base = sm + st * L::kSa;
        if (!__all_sync(0xFFFFFFFFu, ready) && good)
            good = c < L::kNh ? mbar_wait_warp(&bar->fa[st], (uint32_t)pa, KDA_GDR_WAIT_LIMIT)
                              : wait_both(&bar->fa[st], (uint32_t)pa, &bar->eh[c % L::kNh], (uint32_t)(((c / L::kNh) - 1) & 1));
        __syncwarp();
        const int n = len - c * kC;
        if (n < kC) {  // the last chunk: what follows the sequence in K and V counts as zero
            for (int x = threadIdx.x; x < (kC - n) * 16; x += 128)
                *reinterpret_cast<uint4 *>(base + ((x >> 3) & 1) * 8192 + (n + (x >> 4)) * 128 + (x & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            for (int x = threadIdx.x; x < (kC - n) * (L::kVB / 8); x += 128)
                *reinterpret_cast<uint4 *>(base + L::kV + n * L::kVB * 2 + x * 16) = make_uint4(0, 0, 0, 0);
            named_bar_sync(3, 128);
        }
        const uint32_t sk = smem_u32(base) + kw * 8192;
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) ldsm4(b[0][jp], sk + swz(16 * jp + rowB, pcB));
    };
    if (nc > 0) enter(0, false);
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
        const int hb = c % L::kNh, now = st;
        unsigned char *base = sm + st * L::kSa;
        const uint32_t sb = smem_u32(base), sk = sb + kw * 8192;
        uint4 *hs = reinterpret_cast<uint4 *>(sm + L::kH + hb * L::kHand) + (u * 8 + kw * 4) * (32 * MT) + lane;
        uint4 *hu = reinterpret_cast<uint4 *>(sm + L::kH + hb * L::kHand + L::kHu) + u * (256 * MT) + lane;
        const float *sx = reinterpret_cast<const float *>(base + L::kT + kTx);
        // X^T over this warp's 64 key rows
        float X[MT][8][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) X[m][j][e] = 0.f;
        {
            uint32_t ah[2][MT][4], al[2][MT][4];  // A operand of a k step, split a step ahead
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) split_tile(S[m][e][0], S[m][e][1], ah[0][m] + 2 * e, al[0][m] + 2 * e);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const int x = ks & 1, y = x ^ 1;
#pragma unroll
                for (int m = 0; m < MT; ++m) hs[(ks * MT + m) * 32] = make_uint4(ah[x][m][0], ah[x][m][1], ah[x][m][2], ah[x][m][3]);
                if (ks < 3) {
#pragma unroll
                    for (int jp = 0; jp < 4; ++jp) ldsm4(b[y][jp], sk + swz(16 * jp + rowB, 2 * (ks + 1) + pcB));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            split_tile(S[m][2 * ks + 2 + e][0], S[m][2 * ks + 2 + e][1], ah[y][m] + 2 * e, al[y][m] + 2 * e);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 8; ++j) mma(X[m][j], ah[x][m], b[x][j >> 1][2 * (j & 1)], b[x][j >> 1][2 * (j & 1) + 1]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 8; ++j) mma(X[m][j], al[x][m], b[x][j >> 1][2 * (j & 1)], b[x][j >> 1][2 * (j & 1) + 1]);
            }
        }
        // fetched while the products drain (as far as the registers go): V^T (value rows g and g + 8 of a tile),
        // the scalars, T
        uint32_t vv[MT][4][4], th[2][4][4], tl[2][4][4];
        float2 cx[8], be[8];
        auto fetch_right = [&](int ks) {
#pragma unroll
            for (int m = 0; m < MT; ++m) ldsm4t(vv[m][ks], sb + L::kV + v_off<MT>(16 * ks + rowB, 2 * (MT * u + m) + pcB));
#pragma unroll
            for (int j = 2 * ks; j < 2 * ks + 2; ++j) {
                cx[j] = *reinterpret_cast<const float2 *>(sx + 8 * j + q2);
                be[j] = *reinterpret_cast<const float2 *>(sx + kC + 8 * j + q2);
            }
        };
        auto fetch_T = [&](int kp) {
#pragma unroll
            for (int pr = 2 * kp; pr < 4; ++pr) {
                ldsm4(th[kp][pr], sb + L::kT + (offT[pr] ^ (kp * 64)));
                ldsm4(tl[kp][pr], sb + L::kT + kTl + (offT[pr] ^ (kp * 64)));
            }
        };
        if (MT == 1) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) fetch_right(ks);
            fetch_T(0);
        }
        const float gl = sx[3 * kC];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                xb[((kw * 8 + j) * MT + m) * 32] = make_float4(X[m][j][0], X[m][j][1], X[m][j][2], X[m][j][3]);
        named_bar_sync(1 + u, 64);
        if (lane == 0) mbar_arrive(&bar->fs[hb]);
        // right side beta V - x X, split; token tiles 2 ks, 2 ks + 1 are k step ks of the next product
        uint32_t rh[MT][4][4], rl[MT][4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (MT > 1) fetch_right(ks);
            float4 o[2][MT];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 0; m < MT; ++m) o[e][m] = xb[(((1 - kw) * 8 + 2 * ks + e) * MT + m) * 32];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int j = 2 * ks + e;
                    const float2 x = make_float2(-cx[j].x, -cx[j].y);
                    const uint32_t w0 = vv[m][ks][2 * e], w1 = vv[m][ks][2 * e + 1];
                    const float2 v0 = make_float2(lo_f(w0), hi_f(w0)), v1 = make_float2(lo_f(w1), hi_f(w1));
                    const float2 x0 = f2_add(make_float2(X[m][j][0], X[m][j][1]), make_float2(o[e][m].x, o[e][m].y));
                    const float2 x1 = f2_add(make_float2(X[m][j][2], X[m][j][3]), make_float2(o[e][m].z, o[e][m].w));
                    split_tile(f2_fma(x, x0, f2_mul(be[j], v0)), f2_fma(x, x1, f2_mul(be[j], v1)), rh[m][ks] + 2 * e, rl[m][ks] + 2 * e);
                }
        }
        // U^T of this warp's tiles; with MT = 1 the high products and the mixed ones apart (shorter chains of MMAs)
        float U[MT][4][4], W[4][4];
#pragma unroll
        for (int pr = 0; pr < 4; ++pr)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                W[pr][e] = 0.f;
#pragma unroll
                for (int m = 0; m < MT; ++m) U[m][pr][e] = 0.f;
            }
        if (MT > 1) fetch_T(0);
        if (MT == 1) fetch_T(1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const int kp = ks >> 1, k2 = 2 * (ks & 1);
            if (MT > 1 && ks == 2) fetch_T(1);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int pr = ks; pr < 4; ++pr) mma(U[m][pr], rh[m][ks], th[kp][pr][k2], th[kp][pr][k2 + 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int pr = ks; pr < 4; ++pr) mma(MT == 1 ? W[pr] : U[m][pr], rl[m][ks], th[kp][pr][k2], th[kp][pr][k2 + 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int pr = ks; pr < 4; ++pr) mma(MT == 1 ? W[pr] : U[m][pr], rh[m][ks], tl[kp][pr][k2], tl[kp][pr][k2 + 1]);
        }
        // while they run: the state's decay, K as the next B operand, the scalars of U
        const float2 gl2 = make_float2(gl, gl);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                S[m][j][0] = f2_mul(S[m][j][0], gl2);
                S[m][j][1] = f2_mul(S[m][j][1], gl2);
            }
        const uint32_t rowT[2] = {(uint32_t)((lane & 7) + ((((lane >> 3) & 1) ^ own(kw, 0)) << 3)),
                                  (uint32_t)((lane & 7) + ((((lane >> 3) & 1) ^ own(kw, 1)) << 3))};
        const int pcT = lane >> 4;
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) ldsm4t(b[0][jp], sk + swz(rowT[0], 2 * jp + pcT));
        uint32_t uh[MT][4][4], ul[MT][4][4];  // (x U)^T of a pair, own tile first
#pragma unroll
        for (int pr = 0; pr < 4; ++pr) {
            const float2 cu = *reinterpret_cast<const float2 *>(sx + 2 * kC + 16 * pr + 8 * own(kw, pr) + q2);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (MT == 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) U[m][pr][e] += W[pr][e];
                const float2 u0 = make_float2(U[m][pr][0], U[m][pr][1]), u1 = make_float2(U[m][pr][2], U[m][pr][3]);
                uint32_t h[2], l[2];
                split_tile(u0, u1, h, l);
                hu[((2 * pr + own(kw, pr)) * MT + m) * 32] = make_uint4(h[0], h[1], l[0], l[1]);
                split_tile(f2_mul(cu, u0), f2_mul(cu, u1), uh[m][pr], ul[m][pr]);
                ub[((kw * 4 + pr) * MT + m) * 32] = make_uint4(uh[m][pr][0], uh[m][pr][1], ul[m][pr][0], ul[m][pr][1]);
            }
        }
        named_bar_sync(1 + u, 64);
        if (lane == 0) mbar_arrive(&bar->fh[hb]);
        // S^T = exp(G_last) S^T + (x U)^T K over this warp's key rows
        bool ready = true;
        {
#pragma unroll
            for (int pr = 0; pr < 4; ++pr)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 o = ub[(((1 - kw) * 4 + pr) * MT + m) * 32];
                    uh[m][pr][2] = o.x; uh[m][pr][3] = o.y; ul[m][pr][2] = o.z; ul[m][pr][3] = o.w;
                }
            float acc[MT][8][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[m][j][0] = S[m][j][0].x; acc[m][j][1] = S[m][j][0].y;
                    acc[m][j][2] = S[m][j][1].x; acc[m][j][3] = S[m][j][1].y;
                }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const int x = ks & 1, y = x ^ 1;
                if (ks < 3) {
#pragma unroll
                    for (int jp = 0; jp < 4; ++jp) ldsm4t(b[y][jp], sk + swz(16 * (ks + 1) + rowT[y], 2 * jp + pcT));
                }
                if (ks == 2 && c + 1 < nc) {
                    if (++st == L::kNa) st = 0, pa ^= 1;
                    ready = peek(c + 1);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 8; ++j) mma(acc[m][j], uh[m][ks], b[x][j >> 1][2 * (j & 1)], b[x][j >> 1][2 * (j & 1) + 1]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 8; ++j) mma(acc[m][j], ul[m][ks], b[x][j >> 1][2 * (j & 1)], b[x][j >> 1][2 * (j & 1) + 1]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    S[m][j][0] = make_float2(acc[m][j][0], acc[m][j][1]);
                    S[m][j][1] = make_float2(acc[m][j][2], acc[m][j][3]);
                }
        }
        __syncwarp();
        if (lane == 0 && good) mbar_arrive(&bar->ea[now]);
        if (c + 1 < nc) enter(c + 1, ready);
    }
    return good;
}

template <int MT>
__device__ __forceinline__ bool output_pass(const Args &p, unsigned char *sm, StBars *bar, int u, int kw, const Place &pl, int h, int v0)
{
    using L = St<MT>;
    const int lane = threadIdx.x & 31, q2 = 2 * (lane & 3);
    unsigned char *stg = sm + L::kStg + (2 * u + kw) * (1024 * MT);
    const int nc = (pl.len + kC - 1) / kC;
    uint32_t off[4];  // rows of this warp's tile of pair p, pieces 0..3 (4..7: ^ 64)
#pragma unroll
    for (int pr = 0; pr < 4; ++pr) off[pr] = swz(16 * pr + 8 * own(kw, pr) + (lane & 7), lane >> 3);
    // P's low part, five fetches of four 8 x 8: of pair 0's and 2's diagonal; of pair 1 (k step 0, the diagonal); of
    // pair 2 (k steps 0, 1); of pair 3 (k steps 0, 1; 2 and the diagonal)
    uint32_t lo[5];
    {
        const int i = lane >> 3, r = lane & 7;
        auto diag = [&](int pr) {  // tile own 0: its triangle, twice (the second is not used); 1: the full 8 x 8, its triangle
            const int w = own(kw, pr);
            return w && !(i & 1) ? (uint32_t)L::kP + swz(16 * pr + r, 2 * pr + 1) : (uint32_t)L::kDiag + pd_off(2 * pr + w, r);
        };
        auto low = [&](int pr, int ks) { return (uint32_t)L::kP + swz(16 * ks + 8 * own(kw, pr) + r, 2 * pr + (i & 1)); };
        lo[0] = diag(i < 2 ? 0 : 2);
        lo[1] = i < 2 ? low(1, 0) : diag(1);
        lo[2] = low(2, i >> 1);
        lo[3] = low(3, i >> 1);
        lo[4] = i < 2 ? low(3, 2) : diag(3);
    }
    bool good = true;
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
        const int st = c & 1, hb = c % L::kNh;
        static_assert(L::kNo == 2, "two stages");
        const uint32_t sb = smem_u32(sm + L::kO + st * L::kSo), ph = (uint32_t)((c / L::kNh) & 1);
        const float *co = reinterpret_cast<const float *>(sm + L::kO + st * L::kSo + L::kP + kPx);
        const uint4 *hs = reinterpret_cast<const uint4 *>(sm + L::kH + hb * L::kHand) + u * (256 * MT) + lane;
        const uint4 *hu = reinterpret_cast<const uint4 *>(sm + L::kH + hb * L::kHand + L::kHu) + u * (256 * MT) + lane;
        // Q is read once the chain has handed over S0, while it makes little use of shared memory itself
        if (good) good = wait_both(&bar->fo[st], (uint32_t)((c >> 1) & 1), &bar->fs[hb], ph);
        uint32_t qb[4][4][4];
#pragma unroll
        for (int kp = 0; kp < 4; ++kp)
#pragma unroll
            for (int pr = 0; pr < 4; ++pr) ldsm4(qb[kp][pr], sb + (kp >> 1) * 8192 + (off[pr] ^ ((kp & 1) * 64)));
        float o[MT][4][4] = {};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 w = hs[(ks * MT + m) * 32];
                const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int pr = 0; pr < 4; ++pr) mma(o[m][pr], a, qb[ks >> 1][pr][2 * (ks & 1)], qb[ks >> 1][pr][2 * (ks & 1) + 1]);
            }
        uint32_t pb[2][4][4];
        float2 x[4];
#pragma unroll
        for (int pr = 0; pr < 4; ++pr) {
            ldsm4(pb[0][pr], sb + L::kP + off[pr]);
            if (pr >= 2) ldsm4(pb[1][pr], sb + L::kP + (off[pr] ^ 64));
            x[pr] = *reinterpret_cast<const float2 *>(co + 16 * pr + 8 * own(kw, pr) + q2);
        }
        uint32_t plo[4][4][2];  // P's low part: pair, k step
        {
            uint32_t d[4], e[4], f[4], w[4], y[4];
            ldsm4(d, sb + lo[0]);
            ldsm4(e, sb + lo[1]);
            ldsm4(f, sb + lo[2]);
            ldsm4(w, sb + lo[3]);
            ldsm4(y, sb + lo[4]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                plo[0][0][i] = d[i]; plo[2][2][i] = d[2 + i];
                plo[1][0][i] = e[i]; plo[1][1][i] = e[2 + i];
                plo[2][0][i] = f[i]; plo[2][1][i] = f[2 + i];
                plo[3][0][i] = w[i]; plo[3][1][i] = w[2 + i];
                plo[3][2][i] = y[i]; plo[3][3][i] = y[2 + i];
            }
#pragma unroll
            for (int pr = 0; pr < 4; ++pr)  // what lies above the diagonal: zeros
                if (!own(kw, pr)) plo[pr][pr][1] = pb[pr >> 1][pr][2 * (pr & 1) + 1] = 0;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int pr = 0; pr < 4; ++pr) {
                o[m][pr][0] *= x[pr].x;
                o[m][pr][1] *= x[pr].y;
                o[m][pr][2] *= x[pr].x;
                o[m][pr][3] *= x[pr].y;
            }
        if (good) good = mbar_wait_warp(&bar->fh[hb], ph, KDA_GDR_WAIT_LIMIT);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 w0 = hu[(2 * ks * MT + m) * 32], w1 = hu[((2 * ks + 1) * MT + m) * 32];
                const uint32_t a[4] = {w0.x, w0.y, w1.x, w1.y}, al[4] = {w0.z, w0.w, w1.z, w1.w};
#pragma unroll
                for (int pr = ks; pr < 4; ++pr) mma(o[m][pr], a, pb[ks >> 1][pr][2 * (ks & 1)], pb[ks >> 1][pr][2 * (ks & 1) + 1]);
#pragma unroll
                for (int pr = ks; pr < 4; ++pr) mma(o[m][pr], al, pb[ks >> 1][pr][2 * (ks & 1)], pb[ks >> 1][pr][2 * (ks & 1) + 1]);
#pragma unroll
                for (int pr = ks; pr < 4; ++pr) mma(o[m][pr], a, plo[pr][ks][0], plo[pr][ks][1]);
            }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar->eh[hb]);
            if (good) mbar_arrive(&bar->eo[st]);
        }
        // 32 tokens x 16 MT values, staged as rows
        const int n = min(kC, pl.len - c * kC);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                stsm2t(smem_u32(stg) + o_off<MT>(8 * j + (lane & 7), 2 * m + ((lane >> 3) & 1)), pack2(o[m][j][0], o[m][j][1]),
                       pack2(o[m][j][2], o[m][j][3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int e = 32 * i + lane, r = e / (2 * MT), pc = e % (2 * MT), pr = r >> 3, t = 16 * pr + 8 * own(kw, pr) + (r & 7);
            const uint4 w = *reinterpret_cast<const uint4 *>(stg + o_off<MT>(r, pc));
            if (t < n && good)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.rows.out) + ((int64_t)pl.t0 + c * kC + t) * p.rows.out_stride +
                                           (size_t)h * kD + v0 + 16 * MT * u + 8 * pc) = w;
        }
        __syncwarp();
    }
    return good;
}

template <int MT>
__global__ void __launch_bounds__(kStThreads, 1)
gdr_state_kernel(const __grid_constant__ StateMaps maps, const __grid_constant__ Args p,
                 const unsigned char *__restrict__ blocks, int64_t n_chunks, int box_rows)
{
    using L = St<MT>;
    extern __shared__ unsigned char sm_raw[];
    unsigned char *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
    StBars *bar = reinterpret_cast<StBars *>(sm + L::kBar);
    Scan *scans = reinterpret_cast<Scan *>(bar + 1);
    uint32_t *odd = reinterpret_cast<uint32_t *>(scans + kStThreads / 32);
    static_assert(sizeof(StBars) + kStThreads / 32 * sizeof(Scan) + 4 * sizeof(*odd) <= 384, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kVBlocks = kD / L::kVB;
    const int vb = blockIdx.x % kVBlocks;
    const int h = (blockIdx.x / kVBlocks) % p.H, seq = blockIdx.x / (kVBlocks * p.H);
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kNa; ++s) {
            mbar_init(&bar->fa[s], 1);
            mbar_init(&bar->ea[s], 4);
        }
        for (int s = 0; s < L::kNo; ++s) {
            mbar_init(&bar->fo[s], 1);
            mbar_init(&bar->eo[s], 4);
        }
        for (int s = 0; s < L::kNh; ++s) {
            mbar_init(&bar->fs[s], 4);
            mbar_init(&bar->fh[s], 4);
            mbar_init(&bar->eh[s], 4);
        }
        mbar_init(&bar->done, 4);
        fence_mbar_init();
    }
    const Scan part = scan_cu(p, threadIdx.x, kStThreads, seq);
    if (lane == 0) scans[warp] = part;
    __syncthreads();
    Scan cu = {1, 0, 0};
#pragma unroll
    for (int w = 0; w < kStThreads / 32; ++w) {
        cu.ok &= scans[w].ok;
        cu.before += scans[w].before;
        cu.all += scans[w].all;
    }
    int src, dst;
    if (!slots_ok(p, seq, src, dst) || !cu.ok || cu.all != (uint64_t)n_chunks) {  // the same for every thread
        if (threadIdx.x == 0) set_err(p.err);
        // Every block waits for the prep kernel, those without work too: were all of a call's rows skipped, what
        // follows in the stream could otherwise start (and take the workspace) while it still writes its blocks.
        wait_for_previous();
        return;
    }
    const int t0 = __ldg(p.cu + seq);
    const Place pl = {seq, t0, __ldg(p.cu + seq + 1) - t0, (int)cu.before};
    const int nc = (pl.len + kC - 1) / kC;
    // 384 threads x 168 registers at the launch: 128 x (232 + 152 + 56) after this
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8 && lane == 0) {
            const int hk = h / p.G;
            bool good = true;
            int na = 0, no = 0;   // copies into either ring
            wait_for_previous();  // the blocks; everything else that is read here is older than the prep kernel
            for (int c = 0; c < nc && good; ++c) {
                const int sa = c % L::kNa, so = c % L::kNo, t = pl.t0 + c * kC;
                const unsigned char *blk = blocks + ((size_t)(pl.first + c) * p.H + h) * kBlkBytes;
                if (c >= L::kNa) good = mbar_wait_bounded(&bar->ea[sa], (uint32_t)(((c / L::kNa) - 1) & 1), KDA_GDR_WAIT_LIMIT);
                if (!good) break;
                ++na;
                unsigned char *b = sm + sa * L::kSa;
                mbar_arrive_expect_tx(&bar->fa[sa], (uint32_t)(box_rows * (2 * 128 + L::kVB * 2) + kPartT));
                tma_load_2d(b, &maps.k, hk * kD, t, &bar->fa[sa]);
                tma_load_2d(b + 8192, &maps.k, hk * kD + 64, t, &bar->fa[sa]);
                bulk_g2s(b + L::kT, blk, kPartT, &bar->fa[sa]);
                tma_load_2d(b + L::kV, &maps.v, h * kD + vb * L::kVB, t, &bar->fa[sa]);
                if (c >= L::kNo) good = mbar_wait_bounded(&bar->eo[so], (uint32_t)(((c / L::kNo) - 1) & 1), KDA_GDR_WAIT_LIMIT);
                if (!good) break;
                ++no;
                b = sm + L::kO + so * L::kSo;
                mbar_arrive_expect_tx(&bar->fo[so], (uint32_t)(box_rows * 2 * 128 + kPartP + kPd));
                tma_load_2d(b, &maps.q, hk * kD, t, &bar->fo[so]);
                tma_load_2d(b + 8192, &maps.q, hk * kD + 64, t, &bar->fo[so]);
                bulk_g2s(b + L::kP, blk + kPartT, kPartP, &bar->fo[so]);
                bulk_g2s(b + L::kDiag, blk, kPd, &bar->fo[so]);
            }
            // The last copies into every stage land before the block ends and its shared memory is another's,
            // whether the other warps have waited for them or gave up.
            for (int c = max(na - L::kNa, 0); c < na; ++c)
                if (!mbar_wait_bounded(&bar->fa[c % L::kNa], (uint32_t)((c / L::kNa) & 1), kLandSpin)) good = false;
            for (int c = max(no - L::kNo, 0); c < no; ++c)
                if (!mbar_wait_bounded(&bar->fo[c % L::kNo], (uint32_t)((c / L::kNo) & 1), kLandSpin)) good = false;
            if (!good && p.err) atomicExch(p.err, KDA_ERR_TIMEOUT);
        }
        return;
    }
    const int u = (warp >> 1) & 1, kw = warp & 1;
    bool good;
    if (warp >= 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 152;");
        good = output_pass<MT>(p, sm, bar, u, kw, pl, h, vb * L::kVB);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->done);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        // this warp's part of S^T: value rows g, g + 8 of the unit's tiles, key rows 64 kw ..
        const size_t at = (size_t)(64 * kw + 2 * (lane & 3)) * kD + vb * L::kVB + 16 * MT * u + (lane >> 2);
        float2 S[MT][8][2];
        const float *s = p.S + ((size_t)max(src, 0) * p.H + h) * kD * kD + at;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 8 * j * kD + 16 * m + 8 * e;
                    S[m][j][e] = src >= 0 ? make_float2(s[i], s[i + kD]) : make_float2(0.f, 0.f);
                }
        good = chain_pass<MT>(sm, bar, u, kw, pl.len, S);
        // A value that is not finite spreads inside its chunk through the zeros above the diagonals of T and P, to
        // tokens before its own. It always stays in its column of S as well (S is only ever scaled and added to), so
        // that columns whose S is finite are right; 16 columns with one that is not are taken token by token.
        uint32_t again = 0;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float2 z[4] = {};  // 0 as long as all is finite
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) z[2 * (j & 1) + e] = f2_fma(S[m][j][e], make_float2(0.f, 0.f), z[2 * (j & 1) + e]);
            const float2 y = f2_add(f2_add(z[0], z[1]), f2_add(z[2], z[3]));
            if (__any_sync(0xFFFFFFFFu, y.x + y.y != 0.f)) again |= 1u << (MT * u + m);
        }
        if (nc == 0) again = 0;
        volatile uint32_t *flags = odd;
        if (lane == 0) flags[warp] = again;
        named_bar_sync(1 + u, 64);
        again |= flags[warp ^ 1];  // the other half of these columns' key rows
        float *d = p.S + ((size_t)dst * p.H + h) * kD * kD + at;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (good && !(again >> (MT * u + m) & 1u))
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = 8 * j * kD + 16 * m + 8 * e;
                        d[i] = S[m][j][e].x;
                        d[i + kD] = S[m][j][e].y;
                    }
        named_bar_sync(3, 128);
        again = flags[0] | flags[1] | flags[2] | flags[3];
        if (again && !mbar_wait_warp(&bar->done, 0, kLandSpin)) good = false;
        if (good && again >> warp & 1u) walk_tokens<__nv_bfloat16>(p, src, dst, h, vb * (L::kVB / 16) + warp, pl.t0, pl.len);
    }
    if (!good && lane == 0 && p.err) atomicExch(p.err, KDA_ERR_TIMEOUT);
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

template <int MT>
cudaError_t launch_state(const Args &p, const unsigned char *blocks, int64_t n_chunks, int dev, cudaStream_t stream)
{
    const int64_t T = p.total_T;
    const int box = T < kC ? (T > 0 ? (int)T : 1) : kC;
    StateMaps m = {};
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        const int64_t Dk = (int64_t)(p.H / p.G) * kD, Dv = (int64_t)p.H * kD;
        if ((e = rows_map(&m.k, p.rows.k, T, Dk, p.rows.k_stride, 64, box)) != cudaSuccess ||
            (e = rows_map(&m.q, p.rows.q, T, Dk, p.rows.q_stride, 64, box)) != cudaSuccess ||
            (e = rows_map(&m.v, p.rows.v, T, Dv, p.rows.v_stride, St<MT>::kVB, box)) != cudaSuccess)
            return e;
    }
    static std::atomic<uint64_t> done;
    e = raise_smem_on(done, dev, gdr_state_kernel<MT>, St<MT>::kSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((int64_t)p.N * p.H * (kD / St<MT>::kVB));
    if (n_chunks > 0) return launch_after(gdr_state_kernel<MT>, dim3(grid), dim3(kStThreads), St<MT>::kSmem, stream, m, p, blocks, n_chunks, box);
    // no prep kernel before it: whatever the stream holds may still be writing the states
    gdr_state_kernel<MT><<<grid, kStThreads, St<MT>::kSmem, stream>>>(m, p, blocks, n_chunks, box);
    return cudaGetLastError();
}

}  // namespace

size_t chunked_workspace_bytes(int64_t n_chunks, int32_t H) { return 256 + (size_t)n_chunks * H * kBlkBytes; }

cudaError_t launch_chunked(const Args &p, int64_t n_chunks, int64_t longest, void *ws, int dev, int sms, cudaStream_t stream)
{
    unsigned char *blocks = static_cast<unsigned char *>(ws) +
                            ((128 - (reinterpret_cast<uintptr_t>(ws) & 127)) & 127);
    cudaError_t e;
    if (n_chunks > 0) {
        const int Hk = p.H / p.G;
        static std::atomic<uint64_t> done;
        e = raise_smem_on(done, dev, gdr_prep_kernel, kPrepSmem);
        if (e != cudaSuccess) return e;
        const int64_t items = n_chunks * Hk;
        const unsigned grid = (unsigned)(items < (int64_t)kPrepPerSm * sms ? items : (int64_t)kPrepPerSm * sms);
        gdr_prep_kernel<<<grid, kPrepThreads, kPrepSmem, stream>>>(p, blocks, (int)n_chunks, Hk);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    // 32 or 64 value columns a block, by the time that either is estimated to take: the longest sequence, or all
    // of the work over the SMs, at 1.65 us a chunk of 32 columns, 3.2 us a chunk of 64 and 3.5 us to start a
    // block. One sequence of 8192 tokens and 32 heads: 299 us with 32 columns, 482 us with 64; ten sequences of
    // up to 322 tokens and 64 heads: 212 and 187 us. It took the faster form in ten of twelve shapes; in the others
    // whole waves of blocks, which it does not count, decide (8192 tokens, 64 heads: 570 us for 543; 4071 + 3798
    // tokens, 40 heads: 463 for 406).
    auto estimate = [&](int mt, double chunk) {
        const double work = (n_chunks * chunk + p.N * 3.5) * p.H * (4 / mt) / sms, chain = longest * chunk + 3.5;
        return work > chain ? work : chain;
    };
    return estimate(1, 1.65) <= estimate(2, 3.2) ? launch_state<1>(p, blocks, n_chunks, dev, stream)
                                                 : launch_state<2>(p, blocks, n_chunks, dev, stream);
}

}  // namespace gdr
}  // namespace kda
