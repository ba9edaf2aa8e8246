// kda_tree_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers (kda_tree_verify in kda.h).
//
// At node `cur`, with target row p and draft row q over V tokens, the children are
// tried in order.  After j of them were rejected the next token's distribution is
// R_j / S_j with R_j = max(p - c_j q, 0), S_j = sum R_j; from max(R_j / S_j - q, 0) =
// max(p - (c_j + S_j) q, 0) / S_j follows c_{j+1} = c_j + S_j (c_0 = 0, S_0 = 1), so
// that no row is ever rewritten.  A child x is accepted when u q(x) S_j < R_j(x).
// Without draft probabilities q is a point mass at each child's token: R_j is p without
// the rejected tokens and S_j = 1 - the sum of their p, no pass over V needed.
//
// A pass over V gives S_j: sum over p > c q of p, less c times that of q, both as
// exact sums of pairs of floats, joined in float64 (in float32 a sum of 131,072 values
// is off by more than the smallest tokens' probabilities, and the token that a random
// number falls on would depend on the order of the sum; float64 throughout would take
// four times HBM's time at this GPU's rate).  The last pass's sums over pieces of the
// row say in which piece the random number falls, and only that piece is read again.
//
// What bounds it: HBM, a row of p and one of q a sequence.  A cluster of CTAs takes a
// sequence; all of its CTAs walk the tree alike and share each pass.
#include "kda_tree.cuh"

#include <math_constants.h>

namespace kda {
namespace tree {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32, PIECES = 512, MAX_CLUSTER = 8;

// A sum of float32 values kept exact: hi + lo, the rounding of every addition to hi
// goes to lo.
struct Exact {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x), z = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, z)), __fsub_rn(x, z)));
        hi = s;
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// x to the same variable of another CTA of the cluster
__device__ __forceinline__ void store_to(double *p, uint32_t rank, double x) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("st.shared::cluster.f64 [%0], %1;" :: "r"(to), "d"(x) : "memory");
}

// Values e .. e + 3 of a row; those outside [0, V) are 0.  `wide`: in one load (the
// row's blocks of four are aligned).
template <typename Tp> __device__ __forceinline__ float4 values(const Tp *row, int64_t e, int V, bool wide) {
    if (wide && e >= 0 && e + 3 < V) return load4(row + e);
    float4 y;
    y.x = e >= 0 && e < V ? to_f32(row[e]) : 0.f;
    y.y = e + 1 >= 0 && e + 1 < V ? to_f32(row[e + 1]) : 0.f;
    y.z = e + 2 >= 0 && e + 2 < V ? to_f32(row[e + 2]) : 0.f;
    y.w = e + 3 >= 0 && e + 3 < V ? to_f32(row[e + 3]) : 0.f;
    return y;
}

struct State {                               // of the walk, alike in all CTAs of a cluster
    int cur, at, count, gone;                // node, next node to look at, path's length, tokens in `dead`
    double c, left, total;                   // c_j, S_j, the last pass's sum
    int last;                                // which of `totals` the last pass used
    bool summed;                             // the last pass was over this node's rows at c
    bool bare;                               // the residual was empty: the last token is drawn from p
    bool pass;                               // a pass is wanted now
};

template <typename Tp>
__global__ void __launch_bounds__(THREADS, 2) verify_kernel(const VerifyArgs p, int cluster, int piece) {
    __shared__ int32_t par[MAX_NODES], tok[MAX_NODES], path[MAX_NODES], dead[MAX_NODES];
    __shared__ float uni[MAX_NODES], px[MAX_NODES], qx[MAX_NODES];
    __shared__ double sums[PIECES];          // R over this CTA's pieces of the row
    __shared__ double totals[2][MAX_CLUSTER];
    __shared__ double part[WARPS];
    __shared__ State st;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
    const int64_t b = blockIdx.x / cluster;
    const int T = p.T, V = p.V;
    const Tp *target = (const Tp *)p.target, *draft = (const Tp *)p.draft;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid < T) {
        par[tid] = p.parents[b * T + tid];
        tok[tid] = p.tokens[b * T + tid];
        uni[tid] = p.uniform[b * T + tid];
        path[tid] = -1;
        const int up = par[tid], x = tok[tid];
        const bool on = tid > 0 && up >= 0 && up < tid && x >= 0 && x < V;
        px[tid] = on ? to_f32(target[(b * T + up) * p.target_stride + x]) : 0.f;
        qx[tid] = on ? (draft ? to_f32(draft[(b * T + up) * p.draft_stride + x]) : 1.f) : 0.f;
    }
    if (tid == 0) {
        st.cur = 0; st.at = 1; st.count = 1; st.gone = 0;
        st.c = 0.0; st.left = 1.0; st.total = 0.0;
        st.summed = st.bare = false;
        path[0] = 0;
    }
    __syncthreads();
    const bool live = par[0] == -1;                          // the same in the whole cluster
    if (!live) {
        if (rank == 0) {
            if (tid < T) p.path[b * T + tid] = -1;
            if (tid == 0) { p.count[b] = 0; p.next[b] = -1; }
        }
        return;
    }

    if (cluster > 1) cluster_sync();                         // all CTAs are there to be written to
    for (int round = 0;; ++round) {
        if (warp == 0) {                                     // the walk, up to a pass or its end
            int cur = st.cur, at = st.at, count = st.count, gone = st.gone;
            double c = st.c, left = st.left;
            bool summed = st.summed, bare = st.bare, pass = false;
            while (!bare && !pass) {
                const uint32_t lo = __ballot_sync(0xffffffffu, lane < T && lane >= at && par[lane] == cur);
                const uint32_t hi = __ballot_sync(0xffffffffu, lane + 32 < T && lane + 32 >= at && par[lane + 32] == cur);
                if (!(lo | hi)) break;
                const int i = lo ? __ffs((int)lo) - 1 : 31 + __ffs((int)hi);
                at = i + 1;
                if (tok[i] < 0 || tok[i] >= V) continue;     // no token: as if the node were not there
                const double P = px[i], q = qx[i];
                bool was = false;
                if (!draft) for (int j = 0; j < gone; ++j) was |= dead[j] == tok[i];
                const double r = draft ? fmax(P - c * q, 0.0) : (was ? 0.0 : P);
                if ((double)uni[i] * q * left < r) {
                    if (lane == 0) path[count] = i;
                    ++count;
                    cur = i;
                    c = 0.0; left = 1.0; gone = 0;
                    summed = false;
                } else if (draft) {
                    c += left;
                    pass = true;
                } else {
                    left -= r;
                    if (lane == 0) dead[gone] = tok[i];
                    ++gone;
                    __syncwarp();
                }
            }
            if (!pass && !summed) pass = true;               // for the last token
            if (!pass && !bare && !(st.total > 0.0) && (c > 0.0 || gone)) bare = pass = true;
            __syncwarp();
            if (lane == 0) {
                st.cur = cur; st.at = at; st.count = count; st.gone = gone;
                st.c = c; st.left = left;
                st.summed = summed; st.bare = bare; st.pass = pass;
            }
        }
        __syncthreads();
        if (!st.pass) break;
        const double c = st.bare ? 0.0 : st.c;
        const int gone = st.bare ? 0 : st.gone;
        const Tp *pr = target + (b * T + st.cur) * p.target_stride;
        const Tp *qr = draft && c > 0.0 ? draft + (b * T + st.cur) * p.draft_stride : nullptr;
        const int lead = (int)((uintptr_t)pr / sizeof(Tp) & 3);
        const bool wide = !qr || (int)((uintptr_t)qr / sizeof(Tp) & 3) == lead;
        const int pieces = (int)(((int64_t)V + lead + piece - 1) / piece), per = (pieces + cluster - 1) / cluster;
        const int first = min(pieces, (int)rank * per), mine = min(pieces, first + per) - first;
        const float cf = (float)c;
        for (int k = warp; k < mine; k += WARPS) {
            const int64_t e0 = (int64_t)(first + k) * piece - lead;
            Exact sp, sq;
            bool odd = false;                                // rejected tokens in this piece
            for (int j = 0; j < gone; ++j) odd |= dead[j] >= e0 && dead[j] < e0 + piece;
            for (int i = 0; i < piece; i += 512) {
                float4 y[4], z[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) y[x] = values(pr, e0 + i + 128 * x + 4 * lane, V, wide);
                if (qr) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) z[x] = values(qr, e0 + i + 128 * x + 4 * lane, V, wide);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float yv[4] = {y[x].x, y[x].y, y[x].z, y[x].w};
                    if (qr) {
                        const float zv[4] = {z[x].x, z[x].y, z[x].z, z[x].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // a value this rounding puts on the other side counts for nothing
                            const bool in = yv[j] > cf * zv[j];
                            sp.add(in ? yv[j] : 0.f);
                            sq.add(in ? zv[j] : 0.f);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float val = fmaxf(yv[j], 0.f);
                            if (odd) for (int d = 0; d < gone; ++d) if (dead[d] == e0 + i + 128 * x + 4 * lane + j) val = 0.f;
                            sp.add(val);
                        }
                    }
                }
            }
            double s = sp.value();
            if (qr) s -= c * sq.value();
            s = warp_sum(s);
            if (lane == 0) sums[k] = fmax(s, 0.0);
        }
        __syncthreads();
        double s = 0.0;
        for (int k = tid; k < mine; k += THREADS) s += sums[k];
        s = warp_sum(s);
        if (lane == 0) part[warp] = s;
        __syncthreads();
        if (tid < cluster) {                                 // this CTA's sum to all
            double all = 0.0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) all += part[w];
            if (cluster > 1) store_to(&totals[round & 1][rank], tid, all);
            else totals[round & 1][0] = all;
        }
        if (cluster > 1) cluster_sync(); else __syncthreads();
        double total = 0.0;
        for (int k = 0; k < cluster; ++k) total += totals[round & 1][k];
        if (tid == 0) {
            if (c > 0.0) st.left = total;
            st.total = total;
            st.summed = true;
            st.last = round & 1;
        }
        __syncthreads();
    }

    // the last token: the first at which the running sum of R exceeds u times all of it
    const int now = st.last;
    const double c = st.bare ? 0.0 : st.c;
    const int gone = st.bare ? 0 : st.gone;
    double before = 0.0;
    int owner = -1, some = -1;
    const double goal = (double)uni[0] * st.total;
    {
        double run = 0.0;
        for (int k = 0; k < cluster; ++k) {
            const double x = totals[now][k];
            if (x > 0.0) some = k;
            if (owner < 0 && x > 0.0 && run + x > goal) { owner = k; before = run; }
            run += x;
        }
    }
    const bool past = owner < 0;                             // u of 1 or more: the last token there is
    if (past) owner = some;
    if (rank == 0) {
        if (tid < T) p.path[b * T + tid] = path[tid];
        if (tid == 0) {
            p.count[b] = st.count;
            if (owner < 0) p.next[b] = -1;                   // a row of zeros
        }
    }
    if ((int)rank != owner || warp) return;
    const Tp *pr = target + (b * T + st.cur) * p.target_stride;
    const Tp *qr = draft && c > 0.0 ? draft + (b * T + st.cur) * p.draft_stride : nullptr;
    const int lead = (int)((uintptr_t)pr / sizeof(Tp) & 3);
    const bool wide = !qr || (int)((uintptr_t)qr / sizeof(Tp) & 3) == lead;
    const int pieces = (int)(((int64_t)V + lead + piece - 1) / piece), per = (pieces + cluster - 1) / cluster;
    const int first = min(pieces, (int)rank * per), mine = min(pieces, first + per) - first;
    int k = -1, any = -1;
    for (int k0 = 0; k0 < mine && k < 0; k0 += 32) {
        const double x = k0 + lane < mine ? sums[k0 + lane] : 0.0;
        double incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t there = __ballot_sync(0xffffffffu, x > 0.0);
        const uint32_t hit = past ? 0u : __ballot_sync(0xffffffffu, x > 0.0 && before + incl > goal);
        if (there) any = k0 + 31 - __clz((int)there);
        if (hit) {
            const int l = __ffs((int)hit) - 1;
            k = k0 + l;
            before += __shfl_sync(0xffffffffu, incl - x, l);
        } else {
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    const bool seek = k >= 0;                                // else the last token of the last piece
    if (!seek) k = any;
    const int64_t e0 = (int64_t)(first + k) * piece - lead;
    int64_t found = -1, tail = -1;
    for (int i = 0; i < piece && found < 0; i += 128) {
        const int64_t e = e0 + i + 4 * lane;
        const float4 y = values(pr, e, V, wide), z = qr ? values(qr, e, V, wide) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float yv[4] = {y.x, y.y, y.z, y.w}, zv[4] = {z.x, z.y, z.z, z.w};
        double r[4], incl = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = fmax((double)yv[j] - c * (double)zv[j], 0.0);
            for (int d = 0; d < gone; ++d) if (!draft && dead[d] == e + j) r[j] = 0.0;
            if (r[j] > 0.0) tail = e + j;
            incl += r[j];
        }
        const double own = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        int64_t hit = -1;
        double run = before + incl - own;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            run += r[j];
            if (hit < 0 && r[j] > 0.0 && run > goal) hit = e + j;
        }
        const uint32_t who = seek ? __ballot_sync(0xffffffffu, hit >= 0) : 0u;
        if (who) found = __shfl_sync(0xffffffffu, hit, __ffs((int)who) - 1);
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (found < 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int64_t x = __shfl_xor_sync(0xffffffffu, tail, o);
            tail = x > tail ? x : tail;
        }
        found = tail;
    }
    if (lane == 0) p.next[b] = (int32_t)found;
}

template <typename Tp> cudaError_t run(const VerifyArgs &a, cudaStream_t st) {
    // CTAs a sequence: enough for two an SM, and few enough values each to be worth one
    int cluster = 1;
    while (cluster < MAX_CLUSTER && (int64_t)a.B * cluster < 304 && (int64_t)cluster * 8192 < a.V) cluster *= 2;
    // values a piece: 512, or as many as PIECES pieces a CTA need
    const int64_t cap = (int64_t)PIECES * cluster;
    int64_t piece = 512;
    while ((((int64_t)a.V + 3 + piece - 1) / piece + cluster - 1) / cluster * cluster > cap) piece *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<Tp>, a, cluster, (int)piece);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st) {
    return a.dtype == 0 ? run<__nv_bfloat16>(a, st) : run<float>(a, st);
}

}  // namespace tree
}  // namespace kda
