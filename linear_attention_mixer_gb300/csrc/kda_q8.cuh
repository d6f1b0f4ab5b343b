// kda_q8.cuh - groups of values in 8-bit floating point (E4M3) with one power-of-two scale.
#pragma once

#include <cuda_fp8.h>

#include "kda_internal.cuh"

namespace kda {

constexpr int kQb = 128;  // columns per scale

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

}  // namespace kda
