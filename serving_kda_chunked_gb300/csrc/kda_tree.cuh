// kda_tree.cuh -- shared declarations of the operators for drafted tokens
// (internal; the operators are described in kda.h).
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace tree {

constexpr int MAX_NODES = 64;                // nodes of a sequence's tree: one bit each in a mask

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *beta, *S;
    const int32_t *slots, *parents;
    void *o;
    int32_t P, B, T, H, d, dtype;
    bool scalar_gate;
};

struct CommitArgs {
    const void *k, *v;
    const float *g, *beta;
    float *S;
    const int32_t *slots, *path;
    int32_t P, B, T, H, d, dtype;
    bool scalar_gate;
};

struct VerifyArgs {
    const void *target, *draft;
    const int32_t *tokens, *parents;
    const float *uniform;
    int32_t *path, *count, *next;
    int64_t target_stride, draft_stride;     // elements between rows
    int32_t B, T, V, dtype;
};

cudaError_t launch_step(const StepArgs &a, cudaStream_t st);
cudaError_t launch_commit(const CommitArgs &a, cudaStream_t st);
cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st);

// The nodes that node i sees (itself and its ancestors) as bits, 0 where i is
// padding.  A parent is an earlier node, or -1 (the committed tokens); whatever
// else stands there makes the node and all behind it padding.
__device__ __forceinline__ uint64_t ancestors(const int32_t *parents, int i) {
    uint64_t mask = 0;
    for (;;) {
        mask |= 1ull << i;
        const int p = parents[i];
        if (p == -1) return mask;
        if (p < 0 || p >= i) return 0;
        i = p;                               // falls with every step
    }
}
// The same for all nodes by a whole warp: nodes `lane` (x) and `lane + 32` (y).  Every
// round doubles how far up the nodes have looked; told(round, a, b) hears which nodes are
// that far above the two before it (negative: none).  Returns the rounds.
template <typename Told>
__device__ __forceinline__ int all_ancestors(const int32_t *parents, int T, int lane, uint64_t &x, uint64_t &y, Told told) {
    int up0 = lane < T ? parents[lane] : -2, up1 = lane + 32 < T ? parents[lane + 32] : -2;
    if (up0 < -1 || up0 >= lane) up0 = -2;
    if (up1 < -1 || up1 >= lane + 32) up1 = -2;
    x = 1ull << lane;
    y = 1ull << (lane + 32);
    const bool wide = T > 32;                // the same in all lanes
    int round = 0;
#pragma unroll 1
    for (; __any_sync(0xffffffffu, up0 >= 0 || up1 >= 0); ++round) {
        told(round, up0, up1);
        const uint64_t a = __shfl_sync(0xffffffffu, x, up0 & 31);           // node up0 is below 32
        const int na = __shfl_sync(0xffffffffu, up0, up0 & 31);
        if (wide) {
            const uint64_t lo = __shfl_sync(0xffffffffu, x, up1 & 31), hi = __shfl_sync(0xffffffffu, y, up1 & 31);
            const int nl = __shfl_sync(0xffffffffu, up0, up1 & 31), nh = __shfl_sync(0xffffffffu, up1, up1 & 31);
            if (up1 >= 0) {
                y |= up1 < 32 ? lo : hi;
                up1 = up1 < 32 ? nl : nh;
            }
        }
        if (up0 >= 0) {
            x |= a;
            up0 = na;
        }
    }
    if (up0 == -2) x = 0;
    if (up1 == -2) y = 0;
    return round;
}
__device__ __forceinline__ void all_ancestors(const int32_t *parents, int T, int lane, uint64_t &x, uint64_t &y) {
    all_ancestors(parents, T, lane, x, y, [](int, int, int) {});
}

}  // namespace tree
}  // namespace kda
