// kda_mla_tc.cuh -- pieces shared by the tensor-core latent-attention kernels:
// tensor maps, TMA loads, waits that end early once a CTA has failed.
#pragma once

#include "kda_mla_split.cuh"
#include "kda_tc.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

namespace kda {
namespace tcp {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // kda_prefill_tc.cu
}
namespace mla {

using namespace tc;

// 4D bf16 map with 128-byte swizzle (boxes of 64 values along the first axis).
inline bool map4(CUtensorMap *m, const void *base, const uint64_t (&dims)[4],
                 const uint64_t (&strides)[3], const uint32_t (&box)[4]) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tcp::tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t d[4], s[3];
    cuuint32_t b[4], e[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) { d[i] = dims[i]; b[i] = box[i]; }
    for (int i = 0; i < 3; ++i) s[i] = strides[i];
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), d, s, b, e,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2,
                                     int c3, uint64_t *mbar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];"
                 :: "r"(dst), "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(mbar))
                 : "memory");
}
// The same box to L2 only.
__device__ __forceinline__ void tma4_prefetch(const CUtensorMap *m, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];"
                 :: "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_addr(mbar)) : "memory");
}

// Bounded wait of a whole warp that also gives up once another warp of the CTA
// has; the answer is the same in all lanes.
__device__ __forceinline__ bool wait_or_fail(uint64_t *mbar, uint32_t parity, volatile int *fail) {
    bool ok = false;
    for (int i = 0; i < 64; ++i) {
        ok = mbar_wait(mbar, parity, 1u << 16);
        if (ok || *fail) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *fail = FAIL_TIMEOUT;
    return ok;
}
// The same where the phase has most often completed: test_wait says so in a few
// tens of cycles, the loop above in about 300 (and where it has not, the test
// delays the loop: the prefill's softmax, whose scores are never there yet, is
// 5% slower with it).
__device__ __forceinline__ bool test_or_fail(uint64_t *mbar, uint32_t parity, volatile int *fail) {
    const bool ok = mbar_test(mbar, parity);
    return __all_sync(0xffffffffu, ok) || wait_or_fail(mbar, parity, fail);
}
// The wait of the thread that issues MMAs.  Two or three MMAs at most are
// queued ahead of it, so what it does between two groups of them has to fit
// into about 150 cycles.  Hence one thread, a test before the wait, and an
// answer that is collected rather than branched on: with a vote, an election
// or an early exit around each of seven waits a step of 2570 cycles of MMAs
// took 3100 to 4600, in this form 2580.  After a wait that gave up, the MMAs
// of the step still run, on whatever shared and tensor memory hold.
__device__ __forceinline__ bool wait_one(uint64_t *mbar, uint32_t parity) {
    return mbar_test(mbar, parity) || mbar_wait(mbar, parity);
}
// Barrier of `nthreads` threads that tells all of them whether any passed true.
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t nthreads, bool x) {
    uint32_t y;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %3, 0;\n"
                 "barrier.cta.red.or.pred q, %1, %2, p;\nselp.b32 %0, 1, 0, q;\n}"
                 : "=r"(y) : "r"(id), "r"(nthreads), "r"((uint32_t)x) : "memory");
    return y != 0;
}

__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 32 lanes x 16 consecutive 32-bit columns from registers.
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                    "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
                    "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const float (&v)[16]) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
    tmem_st16(a, w);
}

}  // namespace mla
}  // namespace kda
