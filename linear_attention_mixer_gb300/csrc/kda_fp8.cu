// kda_fp8.cu - the projections around the mixer in 8-bit floating point: the quantiser of their
// operands and y = x W^T (+ r) with one FP32 scale for each 1 x 128 group of x and each 128 x 128
// block of W (both E4M3).
//
//   y[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in block b} xq[m][k] wq[n][k]  (+ r[m][n])
//
// The inner sums run on the tensor cores (tcgen05, kind::f8f6f4, FP32 accumulators in tensor memory),
// one accumulator per block b; the epilogue warps take each finished one out, multiply it by its scale
// and add it to FP32 sums in registers, while the tensor cores fill the other of two buffers.
// A persistent kernel; a unit is (128 rows, BN columns, k split), units ordered rows fastest. Warps:
//   0 .. 4 BN/128 - 1  sums: warp w on lanes 32 (w % 4) .., columns 128 (w / 4) ..
//   then               TMA producer (one lane), MMA issuer (one lane)
// With a k split the FP32 partial sums go to the workspace and a second kernel adds them in split
// order, so the result does not depend on timing.
//
// 8192 x 12288 x 7168: 541 to 549 us alone (2.65 PFLOP/s, the tensor pipe 62% busy), 606 to 617 us called again and
// again, under the power cap (2.36 PFLOP/s). The epilogue is well hidden: with neither its reads of tensor memory nor
// its sums the kernel took 504 us where it took 527 (before it looked at the scales' product, which costs 1 to 2%).
// The rest is operands and MMAs: 48 KB a block of 128 of K and SM, 8.5 GB, are 15.5 TB/s out of L2, the likely bound.
// Forms in which two CTAs share a unit of 256 x 256 (cta_group::2, a third fewer bytes) were no faster (560 us, the epilogue's hand-over
// being their bound), nor were they with 16 epilogue warps of half the columns (734 us).
// 16 x 7168 x 12288: 25 us, 19 to 21 of it in this kernel, about 4.4 TB/s, and the rest in adding the splits.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <climits>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kda_internal.cuh"
#include "kda_launch.cuh"
#include "kda_ptx.cuh"
#include "kda_tc.cuh"
#include "kda_wait.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- quantiser
constexpr int kQb = 128;  // columns per scale
constexpr int kMaxK = INT_MAX - 127;  // so that K's blocks of 128 and their columns are counted in 32 bits

// The scale of a group whose largest finite magnitude has the bits u: 2^e, e the smallest integer with it <=
// 448 2^e (448 is E4M3's largest number), at least 2^-126; 1 for an empty or all-zero group. x / 2^e is
// exact (but for what is far below E4M3's smallest step), so q is x rounded once.
__device__ __forceinline__ void q8_scale(uint32_t u, float &s, float &inv)
{
    if (u == 0) {
        s = inv = 1.f;
        return;
    }
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // 448 = 1.75 x 2^8
    e = max(e, -126);
    s = __uint_as_float((uint32_t)(e + 127) << 23);
    inv = __uint_as_float((uint32_t)(127 - e) << 23);
}
// 8 values as they lie in memory
template <typename T> struct Q8;
template <> struct Q8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void bits(uint32_t (&u)[8]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) u[2 * i] = w[i] << 16, u[2 * i + 1] = w[i] & 0xFFFF0000u;
    }
};
template <> struct Q8<float> {
    uint4 r[2];
    __device__ __forceinline__ void load(const float *p)
    {
        r[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
        r[1] = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { r[0] = r[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void bits(uint32_t (&u)[8]) const
    {
        u[0] = r[0].x; u[1] = r[0].y; u[2] = r[0].z; u[3] = r[0].w;
        u[4] = r[1].x; u[5] = r[1].y; u[6] = r[1].z; u[7] = r[1].w;
    }
};

constexpr uint32_t kQInf = 0x7F800000u;  // magnitudes from here on are not finite

// The largest magnitude of 8 values, as bits (whose order is that of the magnitudes).
template <typename T> __device__ __forceinline__ uint32_t q8_max(const Q8<T> &x)
{
    uint32_t u[8], m = 0;
    x.bits(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
    return m;
}
// The same over what is finite.
template <typename T> __device__ __forceinline__ uint32_t q8_max_finite(const Q8<T> &x)
{
    uint32_t u[8], m = 0;
    x.bits(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = u[i] & 0x7FFFFFFFu;
        if (a < kQInf) m = max(m, a);
    }
    return m;
}
// E4M3 codes. `odd`: some value of the group is not finite; such values become NaN.
template <typename T> __device__ __forceinline__ uint2 q8_codes(const Q8<T> &x, float inv, bool odd)
{
    uint32_t u[8], c[4];
    x.bits(u);
    if (odd)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((u[i] & 0x7FFFFFFFu) >= kQInf) u[i] = 0x7FC00000u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(u[2 * i]) * inv, __uint_as_float(u[2 * i + 1]) * inv),
                                                  __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// One scale per row and 128 columns: 16 lanes a group, 8 values a lane, kG groups a lane so that as many
// loads are in flight. 8192 x 7168 BF16: 33 us, 5.4 TB/s of reads and writes (8 groups a lane: 36, and FP32 rows 52 us for 40; 2: as 4).
template <typename T, int kG>
__global__ void __launch_bounds__(256)
q8_rows_kernel(const T *__restrict__ x, int64_t stride, int groups, int K, int nkb, unsigned char *__restrict__ q,
               float *__restrict__ s)
{
    const int lane16 = threadIdx.x & 15;
    const int first = blockIdx.x * (16 * kG) + (threadIdx.x >> 4);  // groups first, first + 16, ..
    Q8<T> f[kG];
    int row[kG], col[kG];
#pragma unroll
    for (int i = 0; i < kG; ++i) {
        const int g = first + 16 * i;
        row[i] = (int)((unsigned)g / (unsigned)nkb);
        col[i] = (g - row[i] * nkb) * kQb + 8 * lane16;
        if (g < groups && col[i] < K) f[i].load(x + row[i] * stride + col[i]);
        else f[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kG; ++i) {
        uint32_t m = q8_max(f[i]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const bool odd = m >= kQInf;
        if (__any_sync(0xFFFFFFFFu, odd)) {  // both groups of the warp
            m = q8_max_finite(f[i]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        }
        float sc, inv;
        q8_scale(m, sc, inv);
        const int g = first + 16 * i;
        if (g < groups) {
            if (col[i] < K) __stcs(reinterpret_cast<uint2 *>(q + (int64_t)row[i] * K + col[i]), q8_codes(f[i], inv, odd));
            if (lane16 == 0) s[g] = sc;
        }
    }
}

// One scale per 128 x 128 block: a thread block each, 64 values a thread in registers. 7168 x 7168 BF16: 29 us.
template <typename T>
__global__ void __launch_bounds__(256)
q8_blocks_kernel(const T *__restrict__ x, int64_t stride, int M, int K, int nkb, unsigned char *__restrict__ q,
                 float *__restrict__ s)
{
    __shared__ uint32_t part[2][8];
    const int mb = blockIdx.x / nkb, kb = blockIdx.x - mb * nkb;
    const int col = kb * kQb + 8 * (threadIdx.x & 15), r0 = mb * 128 + (threadIdx.x >> 4);
    Q8<T> f[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + 16 * i < M && col < K) f[i].load(x + (r0 + 16 * i) * stride + col);
        else f[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, q8_max(f[i]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) part[0][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, part[0][w]);
    const bool odd = m >= kQInf;  // the same for every thread
    if (odd) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, q8_max_finite(f[i]));
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0) part[1][threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, part[1][w]);
    }
    float sc, inv;
    q8_scale(m, sc, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (r0 + 16 * i < M && col < K)
            __stcs(reinterpret_cast<uint2 *>(q + (int64_t)(r0 + 16 * i) * K + col), q8_codes(f[i], inv, odd));
    if (threadIdx.x == 0) s[blockIdx.x] = sc;
}

// ---------------------------------------------------------------- product
constexpr int kF8M = 128;          // rows a unit (MMA M)
constexpr int kF8K = 128;          // K per stage: one scale block, one 128-byte row
// Polls before a wait gives up (a test builds this file with limits that run out).
#ifndef KDA_F8_WAIT_LIMIT
#define KDA_F8_WAIT_LIMIT (1u << 26)
#endif
constexpr uint32_t kF8Land = 1u << 26;  // for copies and products that are on their way when a block ends
constexpr int kF8MaxSplit = 16;

template <int BN> struct F8 {
    static constexpr int kEpi = 4 * (BN / 128);  // epilogue warps
    // with 8 epilogue warps the other warps fill a warpgroup, which gives its registers to them: 256 x 224
    // + 128 x 40 of the 384 x 168 that the block is launched with
    static constexpr int kThreads = 32 * (kEpi + (BN == 256 ? 4 : 2));
    static constexpr int kA = kF8M * kF8K, kStage = kA + BN * kF8K;
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kStg = 32 * 128;        // a store box: 32 rows of 128 bytes
    static constexpr int kSmem = kStages * kStage + kEpi * kStg + 256 + 1024;
};
static_assert(F8<256>::kSmem <= 232448 && F8<128>::kSmem <= 232448, "kda_linear_fp8 shared memory");

// kind::f8f6f4 descriptor: E4M3 x E4M3 -> FP32, both K-major (format codes 0)
__host__ __device__ constexpr uint32_t f8_idesc(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void f8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void f8_store3(const void *tmap, int x, int y, int z, const void *src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ uint32_t f8_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

struct F8Shape {
    int M, N, nkb;           // nkb: blocks of 128 along K
    int n_mblk, n_nblk, split, kb_per_split, n_units;
    int ysplit;              // columns per output matrix
    int a_rows, b_rows;      // rows of the operand boxes
};

template <int BN>
__global__ void __launch_bounds__(F8<BN>::kThreads, 1)
f8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
          const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_p,
          const float *__restrict__ xs, const float *__restrict__ ws, const __nv_bfloat16 *__restrict__ res,
          const F8Shape sh, int32_t *err)
{
    using L = F8<BN>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *stg = smem + L::kStages * L::kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(stg + L::kEpi * L::kStg), *empty = full + L::kStages;
    uint64_t *accfull = empty + L::kStages, *accempty = accfull + 2, *fin = accempty + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(fin + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (sh.split > 1) launch_dependents();  // the kernel that adds the splits
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&accfull[a], 1);
            mbar_init(&accempty[a], L::kEpi);
        }
        mbar_init(fin, 1);
        fence_mbar_init();
    }
    if (warp == L::kEpi + 1) tc::tmem_alloc(tslot, 2 * BN);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;

    auto unit = [&](int u, int &mb, int &nb, int &k0, int &k1, int &ks) {
        mb = u % sh.n_mblk;
        const int r = u / sh.n_mblk;
        ks = r % sh.split;
        nb = r / sh.split;
        k0 = ks * sh.kb_per_split;
        k1 = min(sh.nkb, k0 + sh.kb_per_split);
    };

    if (warp >= L::kEpi) {
        if (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == L::kEpi && lane == 0) {  // producer
            bool ok = true;
            int step = 0;
            const uint32_t bytes = (uint32_t)(sh.a_rows + sh.b_rows) * kF8K;
            for (int u = blockIdx.x; u < sh.n_units && ok; u += gridDim.x) {
                int mb, nb, k0, k1, ks;
                unit(u, mb, nb, k0, k1, ks);
                for (int kb = k0; kb < k1; ++kb, ++step) {
                    const int s = step % L::kStages;
                    if (step >= L::kStages && !mbar_wait_bounded(&empty[s], ((step / L::kStages) - 1) & 1, KDA_F8_WAIT_LIMIT)) {
                        ok = false;
                        break;
                    }
                    unsigned char *st = smem + s * L::kStage;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    tma_load_2d(st, &tm_x, kb * kF8K, mb * kF8M, &full[s]);
                    tma_load_2d(st + L::kA, &tm_w, kb * kF8K, nb * BN, &full[s]);
                }
            }
            // the last copy into every stage lands before the block ends, whether its products run or not
            for (int i = max(step - L::kStages, 0); i < step; ++i)
                if (!mbar_wait_bounded(&full[i % L::kStages], (i / L::kStages) & 1, kF8Land)) ok = false;
            if (!ok) atomicExch(err, KDA_ERR_TIMEOUT);
        } else if (warp == L::kEpi + 1 && lane == 0) {  // MMA issuer
            bool ok = true;
            int step = 0;
            const uint32_t idesc = f8_idesc(kF8M, BN);
            for (int u = blockIdx.x; u < sh.n_units && ok; u += gridDim.x) {
                int mb, nb, k0, k1, ks;
                unit(u, mb, nb, k0, k1, ks);
                for (int kb = k0; kb < k1; ++kb, ++step) {
                    const int s = step % L::kStages, a = step & 1;
                    if ((step >= 2 && !mbar_wait_bounded(&accempty[a], ((step >> 1) - 1) & 1, KDA_F8_WAIT_LIMIT)) ||
                        !mbar_wait_bounded(&full[s], (step / L::kStages) & 1, KDA_F8_WAIT_LIMIT)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t sa = smem_u32(smem + s * L::kStage);
#pragma unroll
                    for (int kk = 0; kk < kF8K / 32; ++kk)
                        f8_mma(tmem + (uint32_t)(a * BN), tc::sw128_desc(sa + kk * 32), tc::sw128_desc(sa + L::kA + kk * 32),
                               idesc, kk > 0 ? 1u : 0u);
                    tc::mma_commit(&empty[s]);
                    tc::mma_commit(&accfull[a]);
                }
            }
            tc::mma_commit(fin);
            if (!mbar_wait_bounded(fin, 0, kF8Land)) ok = false;
            if (!ok) atomicExch(err, KDA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        if (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3, half = warp >> 2;
        bool ok = true;  // the same in every lane
        int step = 0;
        unsigned char *box = stg + warp * L::kStg;
        for (int u = blockIdx.x; u < sh.n_units && ok; u += gridDim.x) {
            int mb, nb, k0, k1, ks;
            unit(u, mb, nb, k0, k1, ks);
            const int rbase = mb * kF8M + 32 * q, row = rbase + lane;
            const int n0 = nb * BN + 128 * half;
            const bool work = rbase < sh.M && n0 < sh.N;  // warp-uniform
            const float *xp = xs + (size_t)min(row, sh.M - 1) * sh.nkb;
            const float *wp = ws + (size_t)(work ? n0 / 128 : 0) * sh.nkb;
            const uint32_t tb = tmem + (uint32_t)(128 * half) + ((uint32_t)(32 * q) << 16);
            float2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
            float sx = __ldg(xp + k0), sw = __ldg(wp + k0);
#pragma unroll 1
            for (int kb = k0; kb < k1; ++kb, ++step) {
                const int a = step & 1;
                // Where the product of the scales is no normal number its product with a block's sum may be one: the
                // sum (0, or 2^-18 .. 2^25 of magnitude) is then multiplied by the larger scale first, which cannot
                // overflow unless the result does. (Lanes are rows; each has its own scale.)
                const float s = sx * sw;
                const bool apart = !(fabsf(s) >= FLT_MIN && fabsf(s) <= FLT_MAX) && sx != 0.f && sw != 0.f;
                const bool larger = fabsf(sx) >= fabsf(sw), odd = __any_sync(0xFFFFFFFFu, apart);
                const float h = apart ? (larger ? sx : sw) : s, l = apart ? (larger ? sw : sx) : 1.f;
                const float2 sc = make_float2(s, s), hi = make_float2(h, h), lo = make_float2(l, l);
                if (kb + 1 < k1) {
                    sx = __ldg(xp + kb + 1);
                    sw = __ldg(wp + kb + 1);
                }
                if (!mbar_wait_warp(&accfull[a], (step >> 1) & 1, KDA_F8_WAIT_LIMIT)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                if (work && !odd) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tc::tmem_ld32_nowait(tb + (uint32_t)(a * BN + 32 * c), v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[16 * c + i] = f2_fma(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                                     sc, acc[16 * c + i]);
                    }
                } else if (work) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tc::tmem_ld32_nowait(tb + (uint32_t)(a * BN + 32 * c), v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[16 * c + i] = f2_fma(f2_mul(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), hi),
                                                     lo, acc[16 * c + i]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&accempty[a]);
            }
            if (!ok || !work) continue;
            if (sh.split == 1) {
                const int zi = n0 / sh.ysplit, x0 = n0 - zi * sh.ysplit;
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // 64 columns = one 128-byte store box
                    if (n0 + 64 * c >= sh.N) break;
                    if (res && row < sh.M) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (n0 + 64 * c + 8 * e >= sh.N) break;
                            const uint4 rv = __ldg(reinterpret_cast<const uint4 *>(res + (size_t)row * sh.N + n0 + 64 * c) + e);
                            const uint32_t w4[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float2 &t = acc[32 * c + 4 * e + i];
                                t.x += __uint_as_float(w4[i] << 16);
                                t.y += __uint_as_float(w4[i] & 0xFFFF0000u);
                            }
                        }
                    }
                    if (lane == 0) bulk_wait_read_all();  // the box's previous store has read it
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 *t = acc + 32 * c + 4 * e;
                        *reinterpret_cast<uint4 *>(box + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                            make_uint4(f8_pack(t[0].x, t[0].y), f8_pack(t[1].x, t[1].y), f8_pack(t[2].x, t[2].y),
                                       f8_pack(t[3].x, t[3].y));
                    }
                    tc::fence_smem_to_async();
                    __syncwarp();
                    if (lane == 0) {
                        f8_store3(&tm_y, x0 + 64 * c, rbase, zi, box);
                        bulk_commit_group();
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 32 FP32 columns = one 128-byte store box
                    if (n0 + 32 * c >= sh.N) break;
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 *t = acc + 16 * c + 2 * e;
                        *reinterpret_cast<float4 *>(box + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                            make_float4(t[0].x, t[0].y, t[1].x, t[1].y);
                    }
                    tc::fence_smem_to_async();
                    __syncwarp();
                    if (lane == 0) {
                        f8_store3(&tm_p, n0 + 32 * c, rbase, ks, box);
                        bulk_commit_group();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        if (!ok && lane == 0) atomicExch(err, KDA_ERR_TIMEOUT);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == L::kEpi + 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 2 * BN);
    }
}

// y = sum over the splits in split order (+ r), rounded to BF16; 8 columns per thread.
__global__ void __launch_bounds__(256)
f8_reduce_kernel(const float *__restrict__ part, const __nv_bfloat16 *__restrict__ res, __nv_bfloat16 *__restrict__ y,
                 int M, int N, int split, int ysplit)
{
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    const int64_t plane = (int64_t)M * N;
    wait_for_previous();  // the partial sums
    if (e >= plane) return;
    const int64_t m = e / N;
    const int n = (int)(e - m * N);
    float acc[8] = {};
    for (int s = 0; s < split; ++s) {
        const float4 *p = reinterpret_cast<const float4 *>(part + s * plane + e);
        const float4 a = p[0], b = p[1];
        acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
        acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
    }
    if (res) {
        const uint4 rv = *reinterpret_cast<const uint4 *>(res + e);
        const uint32_t w4[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[2 * j] += __uint_as_float(w4[j] << 16);
            acc[2 * j + 1] += __uint_as_float(w4[j] & 0xFFFF0000u);
        }
    }
    const int zi = n / ysplit, xc = n - zi * ysplit;
    *reinterpret_cast<uint4 *>(y + ((int64_t)zi * M + m) * ysplit + xc) =
        make_uint4(f8_pack(acc[0], acc[1]), f8_pack(acc[2], acc[3]), f8_pack(acc[4], acc[5]), f8_pack(acc[6], acc[7]));
}

// rank-3 map: dims {d0, d1, d2}, byte strides of dims 1 and 2, box {b0, b1, 1}, 128-byte swizzle
cudaError_t f8_map(CUtensorMap *m, CUtensorMapDataType dt, int rank, const void *base, uint64_t d0, uint64_t d1,
                   uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {s1, s2};
    const cuuint32_t box[3] = {b0, b1, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = encode(m, dt, rank, const_cast<void *>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

thread_local char g_f8_msg[256];

kda_status f8_fail(kda_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_f8_msg, sizeof(g_f8_msg), fmt, ap);
    va_end(ap);
    return record_error(s, g_f8_msg);
}

// Tile width and k split: the pair with the least modelled time, in SM cycles. A unit takes the larger of
// its MMAs (BN cycles a block of 128 x 128 K) and its share of the operands' bytes, and a fixed part for its
// start and its store; a split adds the partial sums' bytes and a second launch.
struct F8Plan { int bn, split; };
F8Plan f8_plan(int M, int N, int nkb, int sms)
{
    const double bw = 3400.0 / sms;  // bytes a cycle and SM (6.8 TB/s at 2 GHz)
    F8Plan best = {128, 1};
    double best_t = 1e300;
    for (int bn = 128; bn <= 256; bn += 128)
        for (int s = 1; s <= kF8MaxSplit && s <= nkb; ++s) {
            const int per = (nkb + s - 1) / s;
            if ((nkb + per - 1) / per != s) continue;
            const int64_t mb = (M + kF8M - 1) / kF8M, nb = (N + bn - 1) / bn;
            const int64_t waves = (mb * nb * s + sms - 1) / sms;
            const double rows = M < kF8M ? M : kF8M;
            const double bytes = (bn / (mb > 4 ? 4.0 : (double)mb) + rows / 4) * kF8K;  // a block of weights is read once per 4 row blocks or so
            const double block = bn * 2.0 > bytes / bw ? bn * 2.0 : bytes / bw;
            double t = waves * (per * block + 2000.0);
            if (s > 1) t += 6000.0 + (2.0 * s + 0.5) * M * N * 4 / (bw * sms);
            if (t < best_t * 0.999) {
                best_t = t;
                best = {bn, s};
            }
        }
    return best;
}

bool f8_shape_ok(int M, int N, int K)
{
    if (M < 0 || N <= 0 || K <= 0) return f8_fail(KDA_ERR_INVALID, "M must be >= 0 and N, K > 0 (got %d, %d, %d)", M, N, K), false;
    if (N % 8 != 0) return f8_fail(KDA_ERR_INVALID, "N must be a multiple of 8 (got %d)", N), false;
    if (K % 16 != 0) return f8_fail(KDA_ERR_INVALID, "K must be a multiple of 16 (got %d)", K), false;
    if (K > kMaxK) return f8_fail(KDA_ERR_INVALID, "K must be at most %d (got %d)", kMaxK, K), false;
    if ((int64_t)M * N > INT_MAX / 2) return f8_fail(KDA_ERR_INVALID, "M * N is too large"), false;
    return true;
}

size_t f8_workspace(int M, int N, const F8Plan &p) { return 256 + (p.split > 1 ? (size_t)p.split * M * N * 4 : 0); }

template <int BN>
cudaError_t f8_launch(const CUtensorMap &tx, const CUtensorMap &tw, const CUtensorMap &ty, const CUtensorMap &tp,
                      const float *xs, const float *ws, const __nv_bfloat16 *r, const F8Shape &sh, int32_t *err, int dev,
                      int sms, cudaStream_t s)
{
    static std::atomic<uint64_t> done;
    const cudaError_t e = raise_smem_on(done, dev, f8_kernel<BN>, F8<BN>::kSmem);
    if (e != cudaSuccess) return e;
    f8_kernel<BN><<<sh.n_units < sms ? sh.n_units : sms, F8<BN>::kThreads, F8<BN>::kSmem, s>>>(tx, tw, ty, tp, xs, ws, r, sh, err);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_quant_fp8(int64_t M, int32_t K, const void *x, int64_t x_stride, int32_t x_dtype,
                                    int32_t block_rows, void *q, float *s, void *stream)
{
    if (M < 0 || K <= 0) return f8_fail(KDA_ERR_INVALID, "M must be >= 0 and K > 0 (got %lld, %d)", (long long)M, K);
    if (K % 16 != 0) return f8_fail(KDA_ERR_INVALID, "K must be a multiple of 16 (got %d)", K);
    if (K > kMaxK) return f8_fail(KDA_ERR_INVALID, "K must be at most %d (got %d)", kMaxK, K);
    if (x_dtype != KDA_F32 && x_dtype != KDA_BF16) return f8_fail(KDA_ERR_INVALID, "x_dtype must be KDA_F32 or KDA_BF16");
    if (block_rows != 1 && block_rows != 128) return f8_fail(KDA_ERR_INVALID, "block_rows must be 1 or 128 (got %d)", block_rows);
    if (M == 0) return KDA_OK;
    if (!x || !q || !s) return f8_fail(KDA_ERR_INVALID, "x, q or s is NULL");
    const int es = x_dtype == KDA_BF16 ? 2 : 4;
    if (M > 1 && (x_stride < K || x_stride > ((int64_t)1 << 38)))
        return f8_fail(KDA_ERR_INVALID, "x_stride must be >= K and at most 2^38 (got %lld)", (long long)x_stride);
    if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) & 15u) || (reinterpret_cast<uintptr_t>(s) & 3u) ||
        (M > 1 && (x_stride * es) % 16))
        return f8_fail(KDA_ERR_INVALID, "x and q must be 16-byte aligned, x_stride a multiple of 16 bytes, s 4-byte aligned");
    const int nkb = (K + kQb - 1) / kQb;
    if (M > (INT_MAX - 128) / nkb) return f8_fail(KDA_ERR_INVALID, "M * K is too large");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char *qp = static_cast<unsigned char *>(q);
    if (block_rows == 1) {
        constexpr int kG = 4;
        const int groups = (int)(M * nkb);
        const unsigned grid = (unsigned)((groups + 16 * kG - 1) / (16 * kG));
        if (es == 2) q8_rows_kernel<__nv_bfloat16, kG><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16 *>(x), x_stride, groups, K, nkb, qp, s);
        else q8_rows_kernel<float, kG><<<grid, 256, 0, st>>>(static_cast<const float *>(x), x_stride, groups, K, nkb, qp, s);
    } else {
        const unsigned grid = (unsigned)((M + 127) / 128 * nkb);
        if (es == 2) q8_blocks_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16 *>(x), x_stride, (int)M, K, nkb, qp, s);
        else q8_blocks_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float *>(x), x_stride, (int)M, K, nkb, qp, s);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KDA_OK : f8_fail(KDA_ERR_CUDA, "kda_quant_fp8: %s", cudaGetErrorString(e));
}

extern "C" size_t kda_linear_fp8_workspace_bytes(int32_t M, int32_t N, int32_t K)
{
    if (!f8_shape_ok(M, N, K)) return 0;
    if (M == 0) return 256;
    int dev = 0, sms = 0;
    if (current_sms(&dev, &sms) != cudaSuccess) {
        cudaGetLastError();
        sms = 148;
    }
    return f8_workspace(M, N, f8_plan(M, N, (K + kF8K - 1) / kF8K, sms));
}

extern "C" kda_status kda_linear_fp8(int32_t M, int32_t N, int32_t K, const void *xq, const float *xs, const void *wq,
                                     const float *ws, const void *r, void *y, int32_t ysplit, void *workspace,
                                     size_t workspace_bytes, void *stream)
{
    if (!f8_shape_ok(M, N, K)) return KDA_ERR_INVALID;
    if (M == 0) return KDA_OK;
    if (ysplit == 0) ysplit = N;
    if (ysplit != N && (ysplit < 0 || ysplit % 128 != 0 || N % ysplit != 0))
        return f8_fail(KDA_ERR_INVALID, "ysplit must divide N and be a multiple of 128 (got %d)", ysplit);
    if (r && ysplit != N) return f8_fail(KDA_ERR_INVALID, "a residual needs an unsplit output (ysplit 0 or N)");
    if (!xq || !xs || !wq || !ws || !y || !workspace) return f8_fail(KDA_ERR_INVALID, "xq, xs, wq, ws, y or workspace is NULL");
    const uintptr_t al = reinterpret_cast<uintptr_t>(xq) | reinterpret_cast<uintptr_t>(wq) | reinterpret_cast<uintptr_t>(y) |
                         reinterpret_cast<uintptr_t>(r) | reinterpret_cast<uintptr_t>(workspace);
    const uintptr_t al4 = reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ws);
    if ((al & 15u) || (al4 & 3u))
        return f8_fail(KDA_ERR_INVALID, "xq, wq, r, y and workspace must be 16-byte aligned, xs and ws 4-byte aligned");
    int dev = 0, sms = 0;
    cudaError_t e = current_sms(&dev, &sms);
    if (e != cudaSuccess) return f8_fail(KDA_ERR_CUDA, "%s", cudaGetErrorString(e));
    F8Shape sh;
    sh.M = M; sh.N = N; sh.nkb = (K + kF8K - 1) / kF8K; sh.ysplit = ysplit;
    const F8Plan plan = f8_plan(M, N, sh.nkb, sms);
    const size_t need = f8_workspace(M, N, plan);
    if (workspace_bytes < need)
        return f8_fail(KDA_ERR_INVALID, "workspace holds %zu bytes, %zu needed", workspace_bytes, need);
    sh.split = plan.split;
    sh.kb_per_split = (sh.nkb + sh.split - 1) / sh.split;
    sh.n_mblk = (M + kF8M - 1) / kF8M;
    sh.n_nblk = (N + plan.bn - 1) / plan.bn;
    if ((int64_t)sh.n_mblk * sh.n_nblk * sh.split > INT_MAX) return f8_fail(KDA_ERR_INVALID, "M * N is too large");
    sh.n_units = sh.n_mblk * sh.n_nblk * sh.split;
    sh.a_rows = M < kF8M ? M : kF8M;  // a box is never taller than its matrix
    sh.b_rows = N < plan.bn ? N : plan.bn;
    const int st_rows = M < 32 ? M : 32;
    int32_t *err = static_cast<int32_t *>(workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
    CUtensorMap tx, tw, ty, tp;
    if ((e = f8_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, xq, K, M, 1, K, 0, kF8K, sh.a_rows)) != cudaSuccess ||
        (e = f8_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, wq, K, N, 1, K, 0, kF8K, sh.b_rows)) != cudaSuccess ||
        (e = f8_map(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, y, ysplit, M, N / ysplit, (uint64_t)ysplit * 2,
                    (uint64_t)ysplit * 2 * M, 64, st_rows)) != cudaSuccess)
        return f8_fail(KDA_ERR_INVALID, "tensor map encoding failed (%s)", cudaGetErrorString(e));
    if (sh.split > 1) {
        if ((e = f8_map(&tp, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, part, N, M, sh.split, (uint64_t)N * 4, (uint64_t)N * 4 * M,
                        32, st_rows)) != cudaSuccess)
            return f8_fail(KDA_ERR_INVALID, "tensor map encoding failed (%s)", cudaGetErrorString(e));
    } else {
        memcpy(&tp, &ty, sizeof(tp));
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const __nv_bfloat16 *rr = sh.split == 1 ? static_cast<const __nv_bfloat16 *>(r) : nullptr;
    e = plan.bn == 256 ? f8_launch<256>(tx, tw, ty, tp, xs, ws, rr, sh, err, dev, sms, s)
                       : f8_launch<128>(tx, tw, ty, tp, xs, ws, rr, sh, err, dev, sms, s);
    if (e != cudaSuccess) return f8_fail(KDA_ERR_CUDA, "kda_linear_fp8: %s", cudaGetErrorString(e));
    if (sh.split > 1) {
        const int64_t total8 = (int64_t)M * N / 8;
        e = launch_after(f8_reduce_kernel, dim3((unsigned)((total8 + 255) / 256)), dim3(256), 0, s, (const float *)part,
                         static_cast<const __nv_bfloat16 *>(r), static_cast<__nv_bfloat16 *>(y), M, N, sh.split, ysplit);
        if (e != cudaSuccess) return f8_fail(KDA_ERR_CUDA, "kda_linear_fp8: %s", cudaGetErrorString(e));
    }
    return KDA_OK;
}
