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

cudaError_t launch_decode_rows(const Args &p, bool f32, cudaStream_t stream);  // N rows of n tokens
cudaError_t launch_sequences(const Args &p, cudaStream_t stream);               // FP32 rows, N sequences

size_t chunked_workspace_bytes(int64_t n_chunks, int32_t H);
cudaError_t launch_chunked(const Args &p, int64_t n_chunks, int64_t longest, void *ws, int dev, int sms, cudaStream_t stream);

}  // namespace gdr
}  // namespace kda
