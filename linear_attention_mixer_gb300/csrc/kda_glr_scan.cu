// kda_glr_scan.cu - the gated linear recurrence over packed sequences: prefill and backward, by a scan along the tokens.
//
// A step h -> (1 + e) h + u is linear, so 16 of them are h -> A h + H with A the product of the (1 + e) and H what becomes
// of h = 0, and such pairs join as (A2 A1, A2 H1 + H2), with A or A - 1 held, whichever is the smaller. A warp has 16 tokens of 64 channels (two channels a lane), a block
// of W warps 16 W tokens, a cluster of nc blocks a window of 16 W nc tokens, and it goes through its sequence window by
// window. For each: every warp works out its tokens' e and u, once, and its pair; the warps' pairs are joined through
// shared memory, the blocks' through distributed shared memory, in the tokens' order (so results do not depend on timing);
// then each warp walks its tokens from the state that it now knows, with e and u still in registers. The rows are read
// once. No block waits for one of another cluster.
//
// 65536 tokens of 4096 channels in BF16: 529 us, 4.0 TB/s (506 with A alone, which is wrong for states that are kept long). Instructions,
// special functions and the FP32 pipe and the latency of a window's exchange share it, on 3.4 of the 4 blocks that an SM has room
// for. Eight sequences of 0 to 2048 tokens, 7168 channels in FP32: 97 us, 5.6 TB/s. With 8 tokens a warp (and 24 warps an SM)
// the first took 670 us where 16 took 566.
#include "kda_glr_scan.cuh"

namespace kda {
namespace glr {
namespace {

// ---------------------------------------------------------------- clusters
// The float4 at `mine` (shared memory) in block `rank` of the cluster, counted by its barrier at `bar`.
__device__ __forceinline__ void st_remote(const float4 *mine, const uint64_t *bar, uint32_t rank, float4 v)
{
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w), "r"(b) : "memory");
}
// Polls before a wait gives up (a test builds this file with a limit that runs out).
#ifndef KDA_GLR_WAIT_LIMIT
#define KDA_GLR_WAIT_LIMIT (1u << 24)
#endif
// Until what other blocks of the cluster sent has arrived; false when the limit ran out, or another warp of the cluster's
// did (`stop`): what is missing may then never be sent.
__device__ __forceinline__ bool wait_cluster(const uint64_t *bar, uint32_t parity, const volatile int32_t *stop)
{
    uint32_t ok = 0;
    for (uint32_t i = 0; i < KDA_GLR_WAIT_LIMIT && !ok; ++i) {
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
        if (!ok && *stop) break;
    }
    return __all_sync(0xFFFFFFFFu, ok != 0);
}

// ---------------------------------------------------------------- pairs
// h -> A h + H. What is held of A is v: A - 1 (below 0) where A >= 1/2, else A. Near 1, where a state is kept over many pairs,
// A itself in FP32 would be wrong by 2^-25 at each with a sign that a steady decay repeats (65536 tokens of 1 - alpha = 1e-6 to
// 1e-7: states off by 1e-3; held so, by 6e-7); near 0 a difference from 1 would leave 2^-24 of a state that has gone.
constexpr float kKept = -0x1p-100f;  // v where A is 1: it changes no h, and is below 0
constexpr float kForm = -0x1p110f;
__device__ __forceinline__ float2 form(float2 v) { return make_float2(__saturatef(v.x * kForm), __saturatef(v.y * kForm)); }  // 1 for A - 1, 0 for A
struct Lin {
    float2 v, H;
    __device__ __forceinline__ float2 at(float2 h) const { return f2_fma(form(v), h, f2_fma(v, h, H)); }
    __device__ __forceinline__ void then(const Lin &n)  // first this, then n
    {
        H = n.at(H);
        v = f2_fma(form(n.v), v, f2_fma(v, n.v, f2_mul(form(v), n.v)));  // the product in either's form, A - 1 only if both are
        v = make_float2(v.x < -0.5f ? v.x + 1.f : v.x, v.y < -0.5f ? v.y + 1.f : v.y);
    }
};
__device__ __forceinline__ Lin lin_identity() { return Lin{f2(kKept), f2(0.f)}; }
// The product A of up to 16 decays 1 + e, and E = A - 1 without the difference.
struct Decays {
    float2 A, E;
    __device__ __forceinline__ Decays() : A(f2(1.f)), E(f2(0.f)) {}
    __device__ __forceinline__ void add(float2 e)
    {
        E = f2_fma(A, e, E);
        A = f2_fma(A, e, A);
    }
    __device__ __forceinline__ float2 v() const { return make_float2(A.x >= 0.5f ? fminf(E.x, kKept) : A.x, A.y >= 0.5f ? fminf(E.y, kKept) : A.y); }
};
__device__ __forceinline__ Lin ld_lin(const float4 *p)
{
    const float4 v = *p;
    return Lin{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ float4 as_float4(const Lin &l) { return make_float4(l.v.x, l.v.y, l.H.x, l.H.y); }

// The places through which pairs are joined, for two windows in turn: a block sends for a window when it has joined the
// one before, to which every block sends when all its warps have read the one before that.
template <int W, int MAX>
struct Exchange {
    float4 warp[2][W][32];
    float4 block[2][MAX][32];
    uint64_t bar[2];
    int32_t stop;  // set in every block of the cluster by a warp that gave up
    __device__ __forceinline__ void open()  // one thread
    {
        stop = 0;
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        fence_mbar_init();
    }
};

// Joining the pairs of a window's warps, in two parts, so that a warp has something to do while they travel.
// post: this warp's own pair goes to the others of the block and, in a cluster, the block's pair to all its blocks: by one warp, in turn,
// since joining pairs takes three times the instructions of a state's way through them.
// meet: the state before the warp's tokens (BACK: behind them), from `carry`, that at the window's start, which becomes that at its end.
// `turn`: windows so far; good: no wait has given up (then nothing more is sent or waited for). All threads of the cluster
// take part.
template <bool BACK, int W, int MAX>
__device__ __forceinline__ void post(Exchange<W, MAX> &ex, const Lin &own, int turn, int nc, int rank, bool good)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, par = turn & 1;
    ex.warp[par][warp][lane] = as_float4(own);
    if (nc > 1 && threadIdx.x == 0 && good) mbar_arrive_expect_tx(&ex.bar[par], (uint32_t)nc * 32 * sizeof(float4));
    __syncthreads();
    if (nc == 1) return;
    if (turn == 0) cluster_wait();  // every block of the cluster runs and has its barriers: theirs is the arrival at the start
    if (warp != (turn + (int)blockIdx.x) % W || !good) return;
    static_assert(W == 1 || W % 4 == 0, "one warp, or whole groups of four");
    Lin all = ld_lin(&ex.warp[par][0][lane]);
#pragma unroll
    for (int i = 0; i + 4 <= W; i += 4) {  // four at a time in pairs: one after the other spilled registers with an output gate
        Lin l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) l[j] = ld_lin(&ex.warp[par][BACK ? W - 1 - i - j : i + j][lane]);
        l[0].then(l[1]);
        l[2].then(l[3]);
        l[0].then(l[2]);
        if (i == 0) all = l[0];
        else all.then(l[0]);
    }
    for (int r = 0; r < nc; ++r) st_remote(&ex.block[par][rank][lane], &ex.bar[par], r, as_float4(all));
}
template <bool BACK, int W, int MAX>
__device__ __forceinline__ float2 meet(Exchange<W, MAX> &ex, float2 &carry, int turn, int nc, int rank, bool &good)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, par = turn & 1;
    float2 h = carry, mine = carry;
    if (nc > 1) {
        if (good) {
            good = wait_cluster(&ex.bar[par], (uint32_t)(turn >> 1) & 1, &ex.stop);
            if (!good && lane < nc) {
                uint32_t a;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(&ex.stop)), "r"(lane));
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(1) : "memory");
            }
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < MAX; j += 4) {
            if (j >= nc) break;
            Lin l[4];  // loaded before they are needed one after the other
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = j + i < nc ? ld_lin(&ex.block[par][BACK ? nc - 1 - j - i : j + i][lane]) : lin_identity();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if ((BACK ? nc - 1 - j - i : j + i) == rank) mine = h;
                h = l[i].at(h);
            }
        }
        carry = h;
        h = mine;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {  // from the block's first token to this warp's, without a cluster to the window's end
        const int w = BACK ? W - 1 - i : i;
        if (w == warp) mine = h;
        if (nc == 1 || (BACK ? w > warp : w < warp)) h = ld_lin(&ex.warp[par][w][lane]).at(h);
    }
    if (nc == 1) carry = h;
    return mine;
}
// What the pairs q0 .. q1 - 1 of a split sequence make of `carry` (BACK: from the last of them on). Each warp folds its share of them;
// all threads of the block take part, before its first window.
template <bool BACK, int W, int MAX>
__device__ __forceinline__ float2 fold(Exchange<W, MAX> &ex, const Split &split, int row, int D, int c, bool live, int q0, int q1, float2 carry)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = q1 - q0;
    const int a = q0 + n * warp / W, b = q0 + n * (warp + 1) / W;
    Lin own = lin_identity();
    if (live) {
        const float4 *pair = split.pairs + (size_t)row * split.subs * (D / 2) + c / 2;
#pragma unroll 8
        for (int i = 0; i < b - a; ++i) own.then(ld_lin(pair + (size_t)(BACK ? b - 1 - i : a + i) * (D / 2)));
    }
    __syncthreads();  // a backward's part before this one has read what is written here
    ex.warp[1][warp][lane] = as_float4(own);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) carry = ld_lin(&ex.warp[1][BACK ? W - 1 - i : i][lane]).at(carry);
    __syncthreads();  // and the windows write it again
    return carry;
}
// Before a block of a cluster ends: none sends to it any more. What was sent to it has arrived, as it has waited for that;
// where a wait gave up, it gets some time to.
__device__ __forceinline__ void leave(int nc, bool joined, bool good)
{
    if (nc == 1) return;
    if (!joined) cluster_wait();  // the arrival at the start
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (!good)
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// ---------------------------------------------------------------- rows in shared memory
// p += n, not turned into a multiple of n that is kept in registers for every row
template <typename T> __device__ __forceinline__ void advance(T *&p, int64_t n)
{
    p += n;
    asm volatile("" : "+l"(p));
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Copies of 16 rows of 64 channels, asked for by 16-byte units; what lies past the sequence or past the row's end is 0.
template <typename T>
struct Tile {
    static constexpr int kUnits = kSlab * (int)sizeof(T) / 16;  // of a row
    static constexpr int kRowsAt = 32 / kUnits;                 // rows that a warp asks for at once
    static constexpr int kBytes = kChunk * kSlab * (int)sizeof(T);

    // row0: the first row's place in the slab, of nv rows that exist
    static __device__ __forceinline__ void fetch(unsigned char *to, const T *row0, int64_t stride, int nv, bool col_ok)
    {
        const int lane = threadIdx.x & 31, r0 = lane / kUnits;
        const T *at = row0 + r0 * stride + (16 / (int)sizeof(T)) * (lane % kUnits);
        if (nv >= kChunk && col_ok) {  // all of this lane's rows
#pragma unroll
            for (int i = 0; i < kChunk / kRowsAt; ++i, advance(at, kRowsAt * stride)) cp_async16(to + (size_t)(lane + 32 * i) * 16, at);
            return;
        }
#pragma unroll
        for (int i = 0; i < kChunk / kRowsAt; ++i, advance(at, kRowsAt * stride)) {
            const bool ok = col_ok && r0 + i * kRowsAt < nv;
            kda::cp_async16(to + (size_t)(lane + 32 * i) * 16, ok ? at : row0, ok ? 16 : 0);
        }
    }
    static __device__ __forceinline__ float2 get(const unsigned char *tile, int r)
    {
        return Pair<T>::get(reinterpret_cast<const typename Pair<T>::Raw *>(tile)[r * (kSlab / 2) + (threadIdx.x & 31)]);
    }
};
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// e and u of a warp's 16 tokens. (A reciprocal each for the two sigmoids: one for their product costs five multiplications
// and a test of its range, which is more than the special function unit's time for another; 574 us for 535.)
template <typename T>
__device__ __forceinline__ void all_gates(const Chan &ch, const unsigned char *x, const unsigned char *a, const unsigned char *b,
                                          float2 (&e)[kChunk], float2 (&u)[kChunk])
{
#pragma unroll
    for (int t = 0; t < kChunk; ++t) gates(ch, Tile<T>::get(x, t), Tile<T>::get(a, t), Tile<T>::get(b, t), e[t], u[t]);
    __syncwarp();
}

// ---------------------------------------------------------------- pairs of a split sequence
// The pair of `sub` tokens of 64 channels: each of eight warps takes an eighth of them, 16 at a time with the next 16 on their way.
// BACK: from the gradient of the state behind the tokens to that before them, else from the state before to that behind.
constexpr int kPairWarps = 8;
template <typename T, bool BACK, bool G>
__global__ void __launch_bounds__(32 * kPairWarps) glr_pairs_kernel(const __grid_constant__ Args p, const void *dout, int64_t dout_stride)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float4 sh[kPairWarps][32];
    using Tl = Tile<T>;
    constexpr int kTiles = BACK ? (G ? 3 : 2) : 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slabs = (p.D + kSlab - 1) / kSlab, q = blockIdx.x % p.split.subs, u = blockIdx.x / p.split.subs;
    const int row = u / slabs, c0 = (u - row * slabs) * kSlab, c = c0 + 2 * lane;
    int src = -1, dst, s0, s1;
    if (!bounds_ok(p.cu, row, p.N, p.total_T, s0, s1) || (!BACK && !slots_ok(p, row, src, dst))) return;  // the kernel behind this one says so
    const bool live = c < p.D;
    if (!BACK && q == 0 && warp == 0 && live)
        *reinterpret_cast<float2 *>(p.split.S0 + (size_t)row * p.D + c) = src >= 0 ? *reinterpret_cast<const float2 *>(p.S + (size_t)src * p.D + c) : f2(0.f);
    const int len = s1 - s0, off = q * p.split.sub;
    if (off >= len) return;
    Chan ch = {f2(0.f), f2(0.f), f2(0.f)};
    if (live) ch.load(p.A_log, p.a_bias, p.b_bias, c);
    const int each = p.split.sub / kPairWarps;  // a multiple of 16
    const int t0 = off + warp * each;
    // the last pair of a backward has all that is left
    const int t1 = BACK && q == p.split.subs - 1 && warp == kPairWarps - 1 ? len : min(len, t0 + each);
    unsigned char *tile = smem + (size_t)warp * 2 * kTiles * Tl::kBytes;
    const bool col_ok = c0 + (16 / (int)sizeof(T)) * (lane % Tl::kUnits) < p.D;
    auto fetch = [&](int t, int stage) {
        const int nv = t1 - t;
        unsigned char *to = tile + stage * kTiles * Tl::kBytes;
        const int64_t r = (int64_t)s0 + t;
        if (nv > 0) {
            Tl::fetch(to, static_cast<const T *>(p.rows.a) + r * p.rows.a_stride + c0, p.rows.a_stride, nv, col_ok);
            if (BACK) {
                Tl::fetch(to + Tl::kBytes, static_cast<const T *>(dout) + r * dout_stride + c0, dout_stride, nv, col_ok);
                if (G) Tl::fetch(to + 2 * Tl::kBytes, static_cast<const T *>(p.rows.g) + r * p.rows.g_stride + c0, p.rows.g_stride, nv, col_ok);
            } else {
                Tl::fetch(to + Tl::kBytes, static_cast<const T *>(p.rows.x) + r * p.rows.x_stride + c0, p.rows.x_stride, nv, col_ok);
                Tl::fetch(to + 2 * Tl::kBytes, static_cast<const T *>(p.rows.b) + r * p.rows.b_stride + c0, p.rows.b_stride, nv, col_ok);
            }
        }
        commit();
    };
    Lin own = lin_identity();
    fetch(t0, 0);
    int stage = 0;
#pragma unroll 1
    for (int t = t0; t < t1; t += kChunk, stage ^= 1) {
        fetch(t + kChunk, stage ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const unsigned char *a = tile + stage * kTiles * Tl::kBytes;
        const int nv = min(kChunk, t1 - t);
        Decays d;
        Lin some = lin_identity();
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (i < nv) {
                if (BACK) {
                    const float2 e = expm1_neg(f2_mul(ch.nA, rcp2(f2_add(neg_exp(Tl::get(a, i), ch.ca), f2(1.f)))));
                    float2 dh = Tl::get(a + Tl::kBytes, i);
                    if (G) dh = f2_mul(dh, silu2(Tl::get(a + 2 * Tl::kBytes, i)));
                    d.add(e);
                    some.H = f2_fma(d.A, dh, some.H);
                } else {
                    float2 e, u2;
                    gates(ch, Tl::get(a + Tl::kBytes, i), Tl::get(a, i), Tl::get(a + 2 * Tl::kBytes, i), e, u2);
                    some.H = step(some.H, e, u2);
                    d.add(e);
                }
            }
        some.v = d.v();
        if (BACK) {  // what lies behind comes first
            some.then(own);
            own = some;
        } else {
            own.then(some);
        }
        __syncwarp();
    }
    cp_async_wait_all();
    sh[warp][lane] = as_float4(own);
    __syncthreads();
    if (warp != 0 || !live) return;
    Lin run = lin_identity();
#pragma unroll
    for (int i = 0; i < kPairWarps; ++i) run.then(ld_lin(&sh[BACK ? kPairWarps - 1 - i : i][lane]));
    p.split.pairs[((size_t)row * p.split.subs + q) * (p.D / 2) + c / 2] = as_float4(run);
}

template <typename T, bool BACK, bool G>
cudaError_t launch_pairs(const Args &p, const void *dout, int64_t dout_stride, int dev, cudaStream_t s)
{
    static std::atomic<uint64_t> raised;
    const int smem = kPairWarps * 2 * (BACK ? (G ? 3 : 2) : 3) * Tile<T>::kBytes;
    const cudaError_t e = raise_smem_on(raised, dev, glr_pairs_kernel<T, BACK, G>, smem);
    if (e != cudaSuccess) return e;
    const int64_t slabs = (p.D + kSlab - 1) / kSlab;
    glr_pairs_kernel<T, BACK, G><<<(unsigned)(p.N * slabs * p.split.subs), 32 * kPairWarps, smem, s>>>(p, dout, dout_stride);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- prefill
template <typename T, bool G, int W>
__global__ void __launch_bounds__(32 * W, kScanPerSm / W) glr_scan_kernel(const __grid_constant__ Args p, int nc)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Exchange<W, max_cluster<T>()> ex;
    constexpr int kTiles = G ? 4 : 3;
    using Tl = Tile<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slabs = (p.D + kSlab - 1) / kSlab, cid = blockIdx.x / nc, rank = nc > 1 ? (int)cluster_rank() : 0;
    const int unit = cid / slabs, c0 = (cid - unit * slabs) * kSlab, c = c0 + 2 * lane;
    const int row = unit / p.split.parts, part = unit - row * p.split.parts;
    int src, dst, s0, s1;
    if (!bounds_ok(p.cu, row, p.N, p.total_T, s0, s1) || !slots_ok(p, row, src, dst)) {  // the same for the whole cluster
        if (threadIdx.x == 0 && rank == 0) set_err(p.err);
        return;
    }
    const bool live = c < p.D;
    const int off = part * p.split.plen;  // this part's first token
    if (part > 0 && off >= s1 - s0) return;
    const bool to_end = part == p.split.parts - 1 || s1 - s0 - off <= p.split.plen;
    const int len = to_end ? s1 - s0 - off : p.split.plen;
    float2 carry = f2(0.f);
    if (p.split.parts == 1) {
        if (live && src >= 0) carry = *reinterpret_cast<const float2 *>(p.S + (size_t)src * p.D + c);
    } else {
        if (live) carry = *reinterpret_cast<const float2 *>(p.split.S0 + (size_t)row * p.D + c);
        carry = fold<false>(ex, p.split, row, p.D, c, live, 0, off / p.split.sub, carry);
    }
    s0 += off;
    if (len > 0) {
        if (nc > 1) {
            if (threadIdx.x == 0) ex.open();
            __syncwarp();
            cluster_arrive();
        }
        bool good = true;
        Chan ch = {f2(0.f), f2(0.f), f2(0.f)};
        if (live) ch.load(p.A_log, p.a_bias, p.b_bias, c);
        unsigned char *tx = smem + (size_t)warp * kTiles * Tl::kBytes, *ta = tx + Tl::kBytes, *tb = ta + Tl::kBytes, *tg = tb + Tl::kBytes;
        const bool col_ok = c0 + (16 / (int)sizeof(T)) * (lane % Tl::kUnits) < p.D;
        const int window = kChunk * W * nc;
        int t = kChunk * (rank * W + warp);  // this warp's first token of the window
        const T *xp = static_cast<const T *>(p.rows.x) + (int64_t)s0 * p.rows.x_stride + c0, *ap = static_cast<const T *>(p.rows.a) + (int64_t)s0 * p.rows.a_stride + c0;
        const T *bp = static_cast<const T *>(p.rows.b) + (int64_t)s0 * p.rows.b_stride + c0, *gp = G ? static_cast<const T *>(p.rows.g) + (int64_t)s0 * p.rows.g_stride + c0 : nullptr;
        T *op = static_cast<T *>(p.rows.out) + (int64_t)s0 * p.rows.out_stride + c;
        float *st = p.starts ? p.starts + (first_chunk(s0 - off, row) + off / kChunk) * p.D + c : nullptr;
        auto fetch = [&](int at) {
            const int nv = len - at;
            if (nv > 0) {
                Tl::fetch(tx, xp + at * p.rows.x_stride, p.rows.x_stride, nv, col_ok);
                Tl::fetch(ta, ap + at * p.rows.a_stride, p.rows.a_stride, nv, col_ok);
                Tl::fetch(tb, bp + at * p.rows.b_stride, p.rows.b_stride, nv, col_ok);
            }
            commit();
        };
        auto fetch_g = [&](int at) {
            if (G && len - at > 0) Tl::fetch(tg, gp + at * p.rows.g_stride, p.rows.g_stride, len - at, col_ok);
            commit();
        };
        fetch(t);
        fetch_g(t);
        const int windows = (len + window - 1) / window;
#pragma unroll 1
        for (int k = 0; k < windows; ++k, t += window) {
            const int nv = min(kChunk, len - t);  // <= 0 behind the sequence's end
            float2 e[kChunk], u[kChunk];
            cp_async_wait_all();
            __syncwarp();
            Lin own = lin_identity();
            if (nv > 0) {
                Decays d;
                all_gates<T>(ch, tx, ta, tb, e, u);
                if (nv < kChunk)
#pragma unroll
                    for (int i = 0; i < kChunk; ++i)
                        if (i >= nv) e[i] = u[i] = f2(0.f);
                fetch(t + window);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    own.H = step(own.H, e[i], u[i]);
                    d.add(e[i]);
                }
                own.v = d.v();
            }
            post<false>(ex, own, k, nc, rank, good);
            float2 h = meet<false>(ex, carry, k, nc, rank, good);
            if (nv > 0) {
                if (live) {
                    if (st) *reinterpret_cast<float2 *>(st + (size_t)(t / kChunk) * p.D) = h;
                    T *o = op + t * p.rows.out_stride;
                    if (nv == kChunk) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i, advance(o, p.rows.out_stride)) {
                            h = step(h, e[i], u[i]);
                            st_pair(o, G ? f2_mul(h, silu2(Tl::get(tg, i))) : h);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i, advance(o, p.rows.out_stride)) {
                            h = step(h, e[i], u[i]);
                            if (i < nv) st_pair(o, G ? f2_mul(h, silu2(Tl::get(tg, i))) : h);
                        }
                    }
                }
                __syncwarp();
                fetch_g(t + window);
            }
        }
        leave(nc, true, good);
        if (!good && lane == 0) set_err(p.err, KDA_ERR_TIMEOUT);
    }
    if (to_end && rank == 0 && warp == 0 && live) *reinterpret_cast<float2 *>(p.S + (size_t)dst * p.D + c) = carry;
}

template <typename T, bool G>
cudaError_t launch_scan_t(const Args &p, const int32_t *cu, int dev, int sms, cudaStream_t s)
{
    constexpr int W = scan_warps<T>();
    static std::atomic<uint64_t> raised;
    static ClusterRoom room;
    const int smem = W * (G ? 4 : 3) * Tile<T>::kBytes;
    const cudaError_t e = raise_smem_on(raised, dev, glr_scan_kernel<T, G, W>, smem);
    if (e != cudaSuccess) return e;
    const int64_t slabs = (p.D + kSlab - 1) / kSlab;
    Args q = p;
    const int nc = choose_parts(cu, p.N, p.N, slabs, kChunk * W, max_cluster<T>(), sms, false, q.split,
                                [&](int n) { return room.of(glr_scan_kernel<T, G, W>, n, 32 * W, smem, dev); });
    if (q.split.parts > 1) {
        const cudaError_t first = launch_pairs<T, false, false>(q, nullptr, 0, dev, s);
        if (first != cudaSuccess) return first;
    }
    return launch_cluster(glr_scan_kernel<T, G, W>, (unsigned)(p.N * q.split.parts * slabs * nc), nc, 32 * W, smem, s, q, nc);
}

// ---------------------------------------------------------------- backward
// The same from the last window to the first, with c the gradient of the state behind a token: c -> alpha (dh + c) is linear
// too. What a token's gradients need beside it is the state before it, which a warp walks again from the one that the
// forward kept for its 16 tokens. A cluster has the sequences (or their parts) group, group + groups, .. and adds up its tokens' shares of
// the parameters' gradients in registers: one row of partial sums a block. 8192 tokens of 4096 channels in BF16 with an output gate:
// 199 us (569 MB, 2.9 TB/s; 190 with A alone), by latency and instructions (half of them issued) of 12 warps an SM.
template <typename T, bool G, int W>
__global__ void __launch_bounds__(32 * W, kBackPerSm / W) glr_back_kernel(const __grid_constant__ BackArgs p, int nc)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Exchange<W, W == 1 ? 1 : max_cluster<T>()> ex;
    constexpr int kTiles = G ? 5 : 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slabs = (p.D + kSlab - 1) / kSlab, cid = blockIdx.x / nc, rank = nc > 1 ? (int)cluster_rank() : 0;
    const int group = cid / slabs, c0 = (cid - group * slabs) * kSlab, c = c0 + 2 * lane;
    const bool live = c < p.D;
    Chan ch = {f2(0.f), f2(0.f), f2(0.f)};
    if (live) ch.load(p.A_log, p.a_bias, p.b_bias, c);
    unsigned char *tx = smem + (size_t)warp * kTiles * Tile<T>::kBytes, *ta = tx + Tile<T>::kBytes, *tb = ta + Tile<T>::kBytes;
    unsigned char *td = tb + Tile<T>::kBytes, *tg = td + Tile<T>::kBytes;
    const bool col_ok = c0 + (16 / (int)sizeof(T)) * (lane % Tile<T>::kUnits) < p.D;
    const int window = kChunk * W * nc, own_t = kChunk * (rank * W + warp);
    float2 sA = f2(0.f), sa = sA, sb = sA;
    int turn = 0;
    bool good = true;
    if (nc > 1) {
        if (threadIdx.x == 0) ex.open();
        __syncwarp();
        cluster_arrive();
    }
#pragma unroll 1
    for (int unit = group; unit < p.N * p.split.parts; unit += p.groups) {
        const int row = unit / p.split.parts, part = unit - row * p.split.parts;
        int s0, s1;
        if (!bounds_ok(p.cu, row, p.N, p.total_T, s0, s1)) {  // the same for the whole cluster
            if (threadIdx.x == 0 && rank == 0) set_err(p.err);
            continue;
        }
        const int off = part * p.split.plen;  // this part's first token
        if (part > 0 && off >= s1 - s0) continue;
        const bool to_end = part == p.split.parts - 1 || s1 - s0 - off <= p.split.plen;
        const int len = to_end ? s1 - s0 - off : p.split.plen;
        float2 carry = live && p.dS_last ? *reinterpret_cast<const float2 *>(p.dS_last + (size_t)row * p.D + c) : f2(0.f);
        if (len == 0) {  // no window, and no row that could be asked for
            if (rank == 0 && warp == 0 && live && p.dS_first) *reinterpret_cast<float2 *>(p.dS_first + (size_t)row * p.D + c) = carry;
            continue;
        }
        if (!to_end)
            carry = fold<true>(ex, p.split, row, p.D, c, live, (off + len) / p.split.sub, min((s1 - s0 + p.split.sub - 1) / p.split.sub, p.split.subs), carry);
        const float *st = p.starts + (first_chunk(s0, row) + off / kChunk) * p.D + c;
        s0 += off;
        auto fetch = [&](int at) {
            const int nv = len - at;
            const int64_t r = (int64_t)s0 + at;
            if (nv > 0) {
                Tile<T>::fetch(tx, static_cast<const T *>(p.rows.x) + r * p.rows.x_stride + c0, p.rows.x_stride, nv, col_ok);
                Tile<T>::fetch(ta, static_cast<const T *>(p.rows.a) + r * p.rows.a_stride + c0, p.rows.a_stride, nv, col_ok);
                Tile<T>::fetch(tb, static_cast<const T *>(p.rows.b) + r * p.rows.b_stride + c0, p.rows.b_stride, nv, col_ok);
                Tile<T>::fetch(td, static_cast<const T *>(p.rows.dout) + r * p.rows.dout_stride + c0, p.rows.dout_stride, nv, col_ok);
                if (G) Tile<T>::fetch(tg, static_cast<const T *>(p.rows.g) + r * p.rows.g_stride + c0, p.rows.g_stride, nv, col_ok);
            }
            commit();
        };
        int t = (len + window - 1) / window * window - window + own_t;
        fetch(t);
#pragma unroll 1
        for (; t >= own_t; t -= window, ++turn) {
            const int nv = min(kChunk, len - t);  // <= 0 behind the sequence's end
            float2 e[kChunk], u[kChunk], h = f2(0.f);
            if (nv > 0 && live) h = __ldg(reinterpret_cast<const float2 *>(st + (size_t)(t / kChunk) * p.D));
            cp_async_wait_all();
            __syncwarp();
            Lin own = lin_identity();
            if (nv > 0) {
                Decays d;
                all_gates<T>(ch, tx, ta, tb, e, u);
                if (nv < kChunk)
#pragma unroll
                    for (int i = 0; i < kChunk; ++i)
                        if (i >= nv) e[i] = u[i] = f2(0.f);
#pragma unroll
                for (int i = kChunk - 1; i >= 0; --i) {  // the rows of dout past the end are 0
                    float2 dh = Tile<T>::get(td, i);
                    if (G) dh = f2_mul(dh, silu2(Tile<T>::get(tg, i)));
                    own.H = f2_add(own.H, dh);
                    own.H = f2_fma(e[i], own.H, own.H);
                    d.add(e[i]);
                }
                own.v = d.v();
            }
            post<true>(ex, own, turn, nc, rank, good);
            if (nv > 0) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {  // u: the state before the token
                    const float2 before = h;
                    h = step(h, e[i], u[i]);
                    u[i] = before;
                }
            }
            float2 lc = meet<true>(ex, carry, turn, nc, rank, good);
            if (nv > 0) {
                const int64_t r = (int64_t)s0 + t + nv - 1;
                T *dxp = static_cast<T *>(p.rows.dx) + r * p.rows.dx_stride + c, *dap = static_cast<T *>(p.rows.da) + r * p.rows.da_stride + c;
                T *dbp = static_cast<T *>(p.rows.db) + r * p.rows.db_stride + c, *dgp = G ? static_cast<T *>(p.rows.dg) + r * p.rows.dg_stride + c : nullptr;
                float2 wA = f2(0.f), wa = wA, wb = wA;  // of this window
#pragma unroll
                for (int i = kChunk - 1; i >= 0; --i) {
                    if (i < nv) {
                        const float2 x = Tile<T>::get(tx, i);
                        float2 dh = Tile<T>::get(td, i);
                        Back bk;
                        bk.gates(ch, e[i], Tile<T>::get(ta, i), Tile<T>::get(tb, i));
                        if (G) {
                            const float2 g = Tile<T>::get(tg, i);
                            float2 s, ns;
                            both_sigmoids(neg_exp(g, f2(0.f)), s, ns);
                            if (live) st_pair(dgp, f2_mul(f2_mul(dh, h), f2_mul(s, f2_fma(g, ns, f2(1.f)))));
                            advance(dgp, -p.rows.dg_stride);
                            dh = f2_mul(dh, f2_mul(g, s));
                        }
                        h = u[i];
                        float2 dx, da, db, dA;
                        lc = bk.token(e[i], f2_add(dh, lc), x, h, dx, da, db, dA);
                        if (live) {
                            st_pair(dxp, dx);
                            st_pair(dap, da);
                            st_pair(dbp, db);
                        }
                        advance(dxp, -p.rows.dx_stride);
                        advance(dap, -p.rows.da_stride);
                        advance(dbp, -p.rows.db_stride);
                        wA = f2_add(wA, dA);
                        wa = f2_add(wa, da);
                        wb = f2_add(wb, db);
                    }
                }
                sA = f2_add(sA, wA);
                sa = f2_add(sa, wa);
                sb = f2_add(sb, wb);
                __syncwarp();
            }
            if (t >= own_t + window) fetch(t - window);
        }
        if (part == 0 && rank == 0 && warp == 0 && live && p.dS_first) *reinterpret_cast<float2 *>(p.dS_first + (size_t)row * p.D + c) = carry;
    }
    leave(nc, turn > 0, good);
    if (!good && lane == 0) set_err(p.err, KDA_ERR_TIMEOUT);
    // the warps' sums, in their order
    __syncthreads();
    float2(*sh)[W][32] = reinterpret_cast<float2(*)[W][32]>(&ex);
    static_assert(sizeof(ex) >= 3 * W * 32 * sizeof(float2), "room for three sums a lane");
    sh[0][warp][lane] = sA;
    sh[1][warp][lane] = sa;
    sh[2][warp][lane] = sb;
    __syncthreads();
    for (int q = warp; q < 3; q += W) {
        float2 s = sh[q][0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) s = f2_add(s, sh[q][w][lane]);
        if (live) *reinterpret_cast<float2 *>(p.part + ((size_t)(group * nc + rank) * 3 + q) * p.D + c) = s;
    }
}

template <typename T, bool G, int W>
cudaError_t launch_back_t(const BackArgs &p, const int32_t *cu, int *parts, int dev, int sms, cudaStream_t s)
{
    static std::atomic<uint64_t> raised;
    static ClusterRoom room;
    const int smem = W * (G ? 5 : 4) * Tile<T>::kBytes;
    const cudaError_t e = raise_smem_on(raised, dev, glr_back_kernel<T, G, W>, smem);
    if (e != cudaSuccess) return e;
    const int64_t slabs = (p.D + kSlab - 1) / kSlab;
    BackArgs q = p;
    const int nc = choose_parts(cu, p.N, p.groups, slabs, kChunk * W, W == 1 ? 1 : max_cluster<T>(), sms, true, q.split,
                                [&](int n) { return room.of(glr_back_kernel<T, G, W>, n, 32 * W, smem, dev); });
    if (q.split.parts > 1) {
        Args f = {};
        f.cu = p.cu; f.N = p.N; f.total_T = p.total_T; f.D = p.D; f.A_log = p.A_log; f.a_bias = p.a_bias; f.b_bias = p.b_bias; f.split = q.split;
        f.rows.a = p.rows.a; f.rows.a_stride = p.rows.a_stride; f.rows.g = p.rows.g; f.rows.g_stride = p.rows.g_stride;
        const cudaError_t first = launch_pairs<T, true, G>(f, p.rows.dout, p.rows.dout_stride, dev, s);
        if (first != cudaSuccess) return first;
        q.groups = p.N * q.split.parts;
    }
    *parts = q.groups * nc;
    return launch_cluster(glr_back_kernel<T, G, W>, (unsigned)(q.groups * slabs * nc), nc, 32 * W, smem, s, q, nc);
}

}  // namespace

cudaError_t launch_scan(const Args &p, bool f32, const int32_t *cu, int dev, int sms, cudaStream_t s)
{
    if (short_sequences(cu, p.N, p.D, f32)) return launch_walk(p, f32, s);
    if (p.rows.g) return f32 ? launch_scan_t<float, true>(p, cu, dev, sms, s) : launch_scan_t<__nv_bfloat16, true>(p, cu, dev, sms, s);
    return f32 ? launch_scan_t<float, false>(p, cu, dev, sms, s) : launch_scan_t<__nv_bfloat16, false>(p, cu, dev, sms, s);
}

cudaError_t launch_scan_back(const BackArgs &p, bool f32, const int32_t *cu, int *parts, int dev, int sms, cudaStream_t s)
{
    const bool one = one_warp(cu, p.N, (p.D + kSlab - 1) / kSlab, sms);
    if (f32) {
        if (p.rows.g) return one ? launch_back_t<float, true, 1>(p, cu, parts, dev, sms, s) : launch_back_t<float, true, kBackWarps>(p, cu, parts, dev, sms, s);
        return one ? launch_back_t<float, false, 1>(p, cu, parts, dev, sms, s) : launch_back_t<float, false, kBackWarps>(p, cu, parts, dev, sms, s);
    }
    if (p.rows.g) return one ? launch_back_t<__nv_bfloat16, true, 1>(p, cu, parts, dev, sms, s) : launch_back_t<__nv_bfloat16, true, kBackWarps>(p, cu, parts, dev, sms, s);
    return one ? launch_back_t<__nv_bfloat16, false, 1>(p, cu, parts, dev, sms, s) : launch_back_t<__nv_bfloat16, false, kBackWarps>(p, cu, parts, dev, sms, s);
}

}  // namespace glr
}  // namespace kda
