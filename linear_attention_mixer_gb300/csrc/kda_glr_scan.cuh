// kda_glr_scan.cuh - the launches of the scan along the tokens (kda_glr_scan.cu) and how many blocks share one.
#pragma once

#include "kda_glr.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace glr {

constexpr int kMaxCluster = 8;
constexpr int kScanWarps = 8;                      // of a block: 128 tokens
constexpr int kScanTile = kChunk * kScanWarps;
constexpr int kBackWarps = 4;
constexpr int kBackTile = kChunk * kBackWarps;

// A launch of clusters of nc blocks (nc 1: without).
template <typename... P, typename... A>
inline cudaError_t launch_cluster(void (*kernel)(P...), unsigned grid, int nc, int threads, size_t smem, cudaStream_t stream, A &&...args)
{
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)nc;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = nc > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Blocks that share a sequence's 64 channels: as many as make the call shortest, where the longest sequence takes
// ceil(its tiles / nc) turns and, if the blocks do not all run at once, the work of all of them counts.
inline int choose_cluster(const int32_t *cu, int32_t N, int64_t slabs, int tile, int most, int slots)
{
    int best = 1;
    double least = 0;
    for (int nc = 1; nc <= most; nc *= 2) {
        int64_t path = 0, all = 0;
        const int64_t span = (int64_t)tile * nc;
        for (int32_t i = 0; i < N; ++i) {
            const int64_t w = (cu[i + 1] - cu[i] + span - 1) / span;
            all += w;
            if (w > path) path = w;
        }
        const double cost = N * slabs * nc <= slots ? (double)path : (double)all * nc * slabs / slots + 0.5 * path;
        if (nc == 1 || cost < 0.95 * least) least = cost, best = nc;
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

cudaError_t launch_scan(const Args &p, bool f32, int nc, int dev, cudaStream_t s);
cudaError_t launch_scan_back(const BackArgs &p, bool f32, int nc, int dev, cudaStream_t s);

}  // namespace glr
}  // namespace kda
