// kda_glr_scan.cuh - the launches over whole sequences: the scan along the tokens (kda_glr_scan.cu), how many blocks share one,
// and the walk of short sequences (kda_glr_walk.cu).
#pragma once

#include "kda_glr.cuh"
#include "kda_cluster.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace glr {

constexpr int kBackWarps = 4;                        // warps of a block: 64 tokens
// Warps that an SM's registers hold (128 and 168 a thread). With BF16 rows that many run; FP32 rows fill shared memory before: 16 in a
// prefill without an output gate, 8 with one (131 KB of rows a block), 8 in a backward.
constexpr int kScanPerSm = 16, kBackPerSm = 12;
// Warps of a prefill's block: eight with FP32 rows, two blocks an SM without an output gate; BF16 rows are faster in four blocks of four
// (65536 tokens of 4096 channels 569 us where two of eight took 597).
template <typename T> constexpr int scan_warps() { return sizeof(T) == 4 ? 8 : 4; }
// Blocks of a cluster at most. FP32 rows leave no room in shared memory for the pairs of more than 8.
template <typename T> constexpr int max_cluster() { return sizeof(T) == 4 ? 8 : 16; }
// Blocks that work on clusters of more than one, over all channels and sequences, at most: what bounds the workspace.
constexpr int kMaxShared = 16384;

// How many clusters of n blocks of a kernel run at once, asked once for each device and n. Not n times fewer than single
// blocks: a cluster stays within a group of SMs, and what does not divide there stays idle.
struct ClusterRoom {
    std::atomic<int> known[8][17];
    template <typename Fn>
    int of(Fn *kernel, int n, int threads, size_t smem, int dev)
    {
        std::atomic<int> *slot = dev >= 0 && dev < 8 ? &known[dev][n] : nullptr;
        int got = slot ? slot->load(std::memory_order_relaxed) : 0;
        if (got) return got;
        cudaLaunchAttribute at = {};
        const cudaLaunchConfig_t cfg = cluster_config(&at, (unsigned)n, n, threads, smem, nullptr);
        cudaError_t e = cudaSuccess;
        if (n > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) {
            cudaLaunchAttribute one = at;
            cudaLaunchConfig_t c = cfg;
            c.attrs = &one;
            c.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&got, kernel, &c);
        }
        if (e != cudaSuccess || got < 1) {
            cudaGetLastError();  // such clusters cannot be launched
            got = -1;
        }
        if (slot) slot->store(got, std::memory_order_relaxed);
        return got;
    }
};

// Blocks that share a sequence's 64 channels, of `groups` sequences at once: as many as make the call shortest. A window
// takes a while however few blocks an SM has (about as long as 192 tokens of one block's work, less without a cluster)
// and the work of all of the SM's blocks; where all clusters of long sequences run at once the longest one's windows
// count, else the work of all. Any number, or, to look at many sequences quickly, powers of two.
template <typename Room>
inline int choose_cluster(const int32_t *cu, int32_t N, int32_t groups, int64_t slabs, int tile, int most, int sms, Room room, double &least)
{
    int best = 1;
    for (int nc = 1; nc <= most; nc += N > 64 ? nc : 1) {
        if (nc > 1 && groups * slabs * nc > kMaxShared) break;
        const int at_once = room(nc);
        if (at_once < 0) continue;
        const uint32_t span = (uint32_t)(tile * nc);
        const int shift = __builtin_ctz(span);
        uint32_t path = 0;
        int64_t all = 0;
        for (int32_t i = 0; i < N; ++i) {
            const uint32_t n = (uint32_t)(cu[i + 1] - cu[i]) + span - 1, w = N > 64 ? n >> shift : n / span;
            all += w;
            if (w > path) path = w;
        }
        int64_t heavy = 0;  // sequences that take long
        for (int32_t i = 0; i < N; ++i) {
            const uint32_t n = (uint32_t)(cu[i + 1] - cu[i]);
            heavy += 8 * (uint64_t)n >= (uint64_t)(path - 1) * span && n > 0;
        }
        const double still = nc == 1 ? 128.0 : 192.0;  // in tokens
        double cost = path * (still + tile * (double)(heavy * slabs * nc) / sms);
        // not all at once: the SMs are full, with `at_once` clusters on them, until the work is done
        if (groups < N || heavy * slabs > at_once)
            cost = (double)all * slabs / at_once * (still + tile * (double)at_once * nc / sms) + 0.25 * path * (still + tile);
        if (nc == 1 || cost < 0.97 * least) least = cost, best = nc;
        if (path <= 1) break;  // more blocks would stand idle
    }
    return best;
}

inline int32_t longest_of(const int32_t *cu, int32_t N)
{
    int32_t n = 0;
    for (int32_t i = 0; i < N; ++i) n = cu[i + 1] - cu[i] > n ? cu[i + 1] - cu[i] : n;
    return n;
}

// Sequences of up to so many times 64 channels may be split, into so many pairs of tokens' (A, H) at most.
constexpr int kSplitUnits = 152, kSplitPairs = 4864;
inline size_t split_pairs_bytes(int32_t N, int64_t slabs) { return N * slabs <= kSplitUnits ? (size_t)kSplitPairs * (kSlab / 2) * sizeof(float4) : 0; }
inline size_t split_bytes(int32_t N, int64_t slabs)
{
    return N * slabs <= kSplitUnits ? split_pairs_bytes(N, slabs) + (size_t)N * slabs * kSlab * sizeof(float) : 0;
}

// choose_cluster, and whether each sequence is split into parts that run at once: where that pays for reading the rows twice, by
// the same estimate. The pairs' kernel takes a start, its blocks' 16 tokens one after the other, and the fold.
//   65536 tokens in BF16: 64 channels 31 us, in one part 141   256: 74, 143   1024: 225, 223   8192 tokens: 64: 21, 22.6
//   (with the backward 65536: 72, 441   217, 467   8192: 41, 64); not taken: 8192 tokens of 256 channels, 24.6 for 22.6
template <typename Room>
inline int choose_parts(const int32_t *cu, int32_t N, int32_t groups, int64_t slabs, int tile, int most, int sms, bool back, Split &split, Room room)
{
    double least = 0;
    int best = choose_cluster(cu, N, groups, slabs, tile, most, sms, room, least);
    split.parts = 1;
    const int32_t longest = longest_of(cu, N);
    split.plen = longest;
    split.sub = 512;
    split.subs = 0;
    if (N * slabs > kSplitUnits || groups < N || longest < 4096 || longest > 1 << 24) return best;
    while (longest > 128 * split.sub) split.sub *= 2;
    const int sub = split.sub;
    least *= 0.9;
    for (int parts = 2; parts <= 32; parts *= 2) {
        const int plen = (longest / parts + sub - 1) / sub * sub, subs = (parts - 1 + back) * (plen / sub);
        if ((int64_t)plen * (parts - 1) >= longest || N * subs * slabs > kSplitPairs) break;
        int64_t clusters = 0, blocks = 0;  // that have tokens
        for (int32_t i = 0; i < N; ++i) {
            const int n = cu[i + 1] - cu[i], in = (n + plen - 1) / plen, of = (n + sub - 1) / sub;
            clusters += (8 * (int64_t)n < longest / parts ? 0 : in < parts ? in : parts) * slabs;
            blocks += (of < subs ? of : subs) * slabs;
        }
        const double pairs = 600 + sub / 128 * (110.0 + 64.0 * blocks / sms) + 3.0 * subs;
        for (int nc = 1; nc <= most; nc *= 2) {
            if (N * parts * slabs * nc > kMaxShared || clusters > room(nc)) continue;
            const int path = ((plen > longest - (parts - 1) * plen ? plen : longest - (parts - 1) * plen) + tile * nc - 1) / (tile * nc);
            const double cost = pairs + path * ((nc == 1 ? 128.0 : 192.0) + tile * (double)(clusters * nc) / sms);
            if (cost < least) {
                least = cost, best = nc;
                split.parts = parts, split.plen = plen, split.subs = subs;
            }
        }
    }
    return best;
}

// Sequences that are in work at once in a backward: as many as give every SM's blocks several turns. Each has its rows
// of partial sums, so that these stay few beside the tokens' rows.
inline int back_groups(int32_t N, int64_t slabs)
{
    const int64_t g = (2432 + slabs - 1) / slabs;
    return (int)(N < g ? N : g < 64 ? (N < 64 ? N : 64) : g);
}
// Rows of partial sums of a backward at most, whatever the device.
inline int64_t back_parts(int32_t N, int64_t slabs)
{
    const int64_t groups = back_groups(N, slabs), shared = kMaxShared / slabs;
    return groups > shared ? groups : shared;
}

// Whether a thread takes each sequence of a prefill from end to end (kda_glr_walk.cu), by estimates in microseconds that were
// fitted to both: 0.17 a token of the longest sequence, or 400 (FP32: 300) channels of a token a ns, against a block's start
// for every sequence's 64 channels and 500 (234) channels a ns. Both sides, sequences of 0 to n tokens in BF16 with a gate:
//   300 of 1024 channels  n = 16: 12 us, scan 33   64: 41, 49   (128: 77, 73)      30 of 256  n = 16: 6.3, 8.2   (64: 12, 8.2)
//   4000 of 4096 channels n = 2: 225 us, scan 1248   16: 477, 1710   64: 1378, 2240    FP32, 300 of 1024: 64: 50, 147
inline bool short_sequences(const int32_t *cu, int32_t N, int32_t D, bool f32)
{
    const double longest = longest_of(cu, N), work = (double)cu[N] * D * 1e-3;
    const double chain = 0.17 * longest, flow = work / (f32 ? 300 : 400);
    const double walk = 2 + (chain > flow ? chain + 0.5 * flow : flow + 0.5 * chain);
    const double units = (double)N * ((D + kSlab - 1) / kSlab);
    return walk < 5.5 + units * (f32 ? 0.0165 : 0.0036) + work / (f32 ? 234 : 500) + longest / 700;
}
cudaError_t launch_walk(const Args &p, bool f32, cudaStream_t s);

// Whether a block of a backward has one warp: where no sequence has more than a warp's 16 tokens, or where they are short and
// many enough to fill the GPU so (12 a SM). Sequences of 0 to n tokens, BF16 with a gate:
//   300 of 4096 channels n = 8: 82 us, four warps 193   32: 172, 286   64: 292, 357   (128: 578 with four)
//   30 of 1024 channels  n = 16: 12.3 us, four warps 12.4   (32: 16.4 with four; 64: 17.6)
inline bool one_warp(const int32_t *cu, int32_t N, int64_t slabs, int sms)
{
    const int32_t longest = longest_of(cu, N);
    return longest <= kChunk || (longest <= 4 * kChunk && N * slabs >= kBackPerSm * sms);
}

// cu: the host's cu_seqlens
cudaError_t launch_scan(const Args &p, bool f32, const int32_t *cu, int dev, int sms, cudaStream_t s);
cudaError_t launch_scan_back(const BackArgs &p, bool f32, const int32_t *cu, int *parts, int dev, int sms, cudaStream_t s);

}  // namespace glr
}  // namespace kda
