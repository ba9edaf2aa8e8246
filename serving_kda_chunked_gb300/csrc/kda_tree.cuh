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

}  // namespace tree
}  // namespace kda
