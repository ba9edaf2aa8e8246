// kda_mla.cuh -- shared declarations of the latent-attention operators
// (internal; the operators are described in kda.h).
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace mla {

constexpr int LATENT = 512, ROPE = 64, ROW = LATENT + ROPE;   // a cached token
constexpr int NOPE = 128, DQK = NOPE + ROPE, DV = 128;        // an expanded head

struct AppendArgs {
    const void *c, *k_r, *q_r;
    void *cache, *k_out, *q_out;
    const int32_t *slots, *positions;
    const float *rope;
    int64_t c_stride, k_r_stride, k_out_stride;                // elements
    int64_t q_token_stride, q_head_stride, qo_token_stride, qo_head_stride;
    int64_t T, n_slots;
    int32_t max_pos, interleaved, H, dtype;
};

struct PrefillArgs {
    const void *q, *kv, *k_r;
    const int32_t *cu_q, *cu_k;
    void *o;
    float *lse;
    void *ws;
    int64_t Tq, Tk;
    int32_t N, H, dtype, causal;
    float scale;
};

struct DecodeArgs {
    const void *q, *cache;
    const int32_t *table, *seq_lens;
    void *o;
    float *lse;
    void *ws;
    int32_t B, H, n_pages, page, max_pages, dtype;
    float scale;
};

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st);
cudaError_t launch_prefill_simt(const PrefillArgs &a, cudaStream_t st);
cudaError_t launch_decode_simt(const DecodeArgs &a, cudaStream_t st);
uint64_t prefill_simt_workspace_bytes(int32_t N, int64_t Tq, int32_t H);
uint64_t decode_simt_workspace_bytes(int32_t H);
cudaError_t launch_decode_tc(const DecodeArgs &a, cudaStream_t st);
uint64_t decode_tc_workspace_bytes(int32_t H);
cudaError_t launch_prefill_tc(const PrefillArgs &a, cudaStream_t st);
uint64_t prefill_tc_workspace_bytes(int32_t N, int64_t Tq);

// SMs of the current device.
inline cudaError_t sm_count(int *nsm) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, dev);
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}

// Queries [bos, eos) of sequence n and its keys, from clamped offsets.
struct SeqSpan { int64_t q0, k0; int nq, nk; };
__device__ __forceinline__ SeqSpan seq_span(const int32_t *cu_q, const int32_t *cu_k, int n,
                                            int64_t Tq, int64_t Tk) {
    int64_t a, b, c, d;
    seq_bounds(cu_q, n, Tq, a, b);
    seq_bounds(cu_k, n, Tk, c, d);
    return {a, c, (int)(b - a), (int)(d - c)};
}

}  // namespace mla
}  // namespace kda
