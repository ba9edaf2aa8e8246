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
// A pass over V gives S_j: sum over p > c q of p, less c times that of q, every sum a pair of
// floats that keeps what its additions round off.  In float32 a sum of 131,072 values is
// off by more than the smallest tokens' probabilities, and the token that a random number
// falls on would depend on the order of the sum; a float64 operation of a warp takes 60
// cycles of an SM here (a walk, three scans and the last piece's sums in float64 took 20,000
// cycles beside a pass of 8,000).  Pairs hold 48 bits, for about ten float32 operations an
// addition.  The last pass's sums over the warps' pieces of the row say in which piece the
// random number falls, and only that one is read again.
//
// What bounds it: HBM, a row of p and one of q a sequence.  A cluster of CTAs takes a
// sequence; all of its CTAs walk the tree alike and share each pass.  Measured, 256
// sequences over 131,072 tokens: one rejection each 50 us (5.4 TB/s), trees of 16 nodes with
// 1.9 passes on average and up to seven 96 us (the sequences with many passes end last), without
// draft rows 61, no drafted token 40; one sequence over 50,021 tokens 8.3 us, a chain of passes with
// a cluster barrier each.  The next loads under way beside a block's sums: 2% off.
// bf16 rows, half the bytes: 52, 103, 62, 39 and 10.7 us, so that HBM bounds none of them (the
// pairs' arithmetic is the same for a value of two bytes; how far it or the chain does has not been measured).
#include "kda_tree.cuh"


namespace kda {
namespace tree {
namespace {

// With 512 threads and two CTAs an SM a batch of 256 trees over 131,072 tokens takes 100 us
// (here 96), with 128 and eight 92, but single sequences 11 (here 8).
constexpr int THREADS = 256, MIN_CTAS = 4, WARPS = THREADS / 32, MAX_CLUSTER = 8;
constexpr int PER_LANE = MAX_CLUSTER * WARPS / 32;          // pieces a lane adds up

// A number as the sum of two floats, lo below half a unit of hi's last place.
struct Pair { float hi, lo; };
struct bool2 { bool x, y; };

__device__ __forceinline__ Pair two_sum(float a, float b) {                  // a + b, exact
    const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ Pair normal(float hi, float lo) {                 // |hi| >= |lo|
    const float s = __fadd_rn(hi, lo);
    return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi);
    return normal(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
__device__ __forceinline__ Pair operator*(Pair a, float b) {
    const float p = __fmul_rn(a.hi, b);
    return normal(p, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -p)));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    const float p = __fmul_rn(a.hi, b.hi);
    return normal(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p))));
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Pair not_below_0(Pair a) { return a.hi > 0.f ? a : Pair{0.f, 0.f}; }

// Two such sums of float32 values side by side, lo not yet below hi's last place.
struct Sums {
    float2 hi = {0.f, 0.f}, lo = {0.f, 0.f};
    __device__ __forceinline__ void add(float2 x) {
        const float2 s = add2(hi, x), z = sub2(s, hi);
        lo = add2(lo, add2(sub2(hi, sub2(s, z)), sub2(x, z)));
        hi = s;
    }
    __device__ __forceinline__ Pair value() const { return normal(hi.x, lo.x) + normal(hi.y, lo.y); }
    static __device__ __forceinline__ float2 add2(float2 a, float2 b) {
        float2 d;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(d))
            : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
        return d;
    }
    static __device__ __forceinline__ float2 sub2(float2 a, float2 b) {
        float2 d;
        asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(d))
            : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
        return d;
    }
};

// Which of two values p exceed c q.  c's hi alone would drop a value whose p / q lies within half of its
// last place of c, and that may be all that is left of R after some 25 rejections.  p - hi q is rounded
// once, so its sign is right, and against lo q it errs for what lies within 2^-46 of c only.
__device__ __forceinline__ bool2 exceeds(float2 p, float2 q, Pair c) {
    const float2 hi = make_float2(-c.hi, -c.hi), lo = make_float2(c.lo, c.lo);
    float2 d, e;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<const uint64_t &>(hi)), "l"(reinterpret_cast<uint64_t &>(q)), "l"(reinterpret_cast<uint64_t &>(p)));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(e))
        : "l"(reinterpret_cast<const uint64_t &>(lo)), "l"(reinterpret_cast<uint64_t &>(q)));
    return {d.x > e.x, d.y > e.y};
}

__device__ __forceinline__ Pair shfl(Pair x, int from) {
    return {__shfl_sync(0xffffffffu, x.hi, from), __shfl_sync(0xffffffffu, x.lo, from)};
}
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = x + Pair{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
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
__device__ __forceinline__ void store_to(Pair *p, uint32_t rank, Pair x) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" :: "r"(to), "f"(x.hi), "f"(x.lo) : "memory");
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
    Pair c, left, total;                     // c_j, S_j, the last pass's sum
    bool summed;                             // the last pass was over this node's rows at c
    bool bare;                               // the residual was empty: the last token is drawn from p
    bool pass;                               // a pass is wanted now
};

// The rows of a pass.
template <typename Tp> struct Rows {
    const Tp *p, *q;                         // q NULL: R is p (without rejected tokens)
    int lead;                                // values between the alignment boundary before the row and the row
    bool wide;
    Pair c;
    int gone;
    __device__ __forceinline__ Rows(const VerifyArgs &a, const State &st, int64_t b) {
        const int64_t row = b * a.T + st.cur;
        c = st.bare ? Pair{0.f, 0.f} : st.c;
        gone = st.bare ? 0 : st.gone;
        p = (const Tp *)a.target + row * a.target_stride;
        q = a.draft && c.hi > 0.f ? (const Tp *)a.draft + row * a.draft_stride : nullptr;
        lead = (int)((uintptr_t)p / sizeof(Tp) & 3);
        wide = !q || (int)((uintptr_t)q / sizeof(Tp) & 3) == lead;
    }
};

// R of the four values from e on, from their p and q.
__device__ __forceinline__ Pair residual(float p, float q, Pair c) {
    const Pair t = c * q, d = two_sum(p, -t.hi);
    return not_below_0(normal(d.hi, __fsub_rn(d.lo, t.lo)));
}
template <typename Tp>
__device__ __forceinline__ void residual(const Rows<Tp> &w, int64_t e, int V, const int32_t *dead, Pair (&r)[4]) {
    const float4 y = values(w.p, e, V, w.wide), z = w.q ? values(w.q, e, V, w.wide) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float yv[4] = {y.x, y.y, y.z, y.w}, zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r[j] = w.q ? residual(yv[j], zv[j], w.c) : Pair{fmaxf(yv[j], 0.f), 0.f};
        for (int d = 0; d < w.gone; ++d) if (dead[d] == e + j) r[j] = {0.f, 0.f};
    }
}

// Inclusive sums over the lanes.
__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if (lane >= o) x = x + y;
    }
    return x;
}

// Where the running sum of a warp's values x (lane after lane) first exceeds goal - before:
// the lane, and `before` moved to it.  Where it does not: the last lane whose x is not
// 0 (-1: none), and `past` is set.
__device__ __forceinline__ int find_lane(Pair x, Pair goal, Pair &before, bool &past, int lane) {
    const Pair incl = warp_scan(x, lane);
    const uint32_t some = __ballot_sync(0xffffffffu, x.hi > 0.f), hit = __ballot_sync(0xffffffffu, x.hi > 0.f && before + incl > goal);
    past = !hit;
    const int k = hit ? __ffs((int)hit) - 1 : (some ? 31 - __clz((int)some) : -1);
    if (k >= 0) before = before + shfl(incl - x, k);
    return k;
}

// `piece`: values of the row a warp takes in a pass, a multiple of 128; warp w of CTA r
// has piece r * WARPS + w.
template <typename Tp>
__global__ void __launch_bounds__(THREADS, MIN_CTAS) verify_kernel(const VerifyArgs p, int cluster, int64_t piece) {
    __shared__ int32_t par[MAX_NODES], tok[MAX_NODES], path[MAX_NODES], dead[MAX_NODES];
    __shared__ float uni[MAX_NODES], px[MAX_NODES], qx[MAX_NODES];
    __shared__ Pair part[2][MAX_CLUSTER * WARPS];            // R over the pieces, of two passes in turn
    __shared__ Pair sub[WARPS], sbefore;
    __shared__ int spiece;
    __shared__ bool spast;
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
        st.c = st.total = {0.f, 0.f};
        st.left = {1.f, 0.f};
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
    int last = 0;                                            // which of `part` the last pass used
    for (int round = 0;; ++round) {
        if (warp == 0) {                                     // the walk, up to a pass or its end
            int cur = st.cur, at = st.at, count = st.count, gone = st.gone;
            Pair c = st.c, left = st.left;
            bool summed = st.summed, bare = st.bare, pass = false;
            while (!bare && !pass) {
                const uint32_t lo = __ballot_sync(0xffffffffu, lane < T && lane >= at && par[lane] == cur);
                const uint32_t hi = __ballot_sync(0xffffffffu, lane + 32 < T && lane + 32 >= at && par[lane + 32] == cur);
                if (!(lo | hi)) break;
                const int i = lo ? __ffs((int)lo) - 1 : 31 + __ffs((int)hi);
                at = i + 1;
                if (tok[i] < 0 || tok[i] >= V) continue;     // no token: as if the node were not there
                const float P = px[i], q = qx[i];
                bool was = false;
                if (!draft) for (int j = 0; j < gone; ++j) was |= dead[j] == tok[i];
                const Pair r = draft ? residual(P, q, c) : Pair{was ? 0.f : P, 0.f};
                if (r > Pair{q, 0.f} * uni[i] * left) {
                    if (lane == 0) path[count] = i;
                    ++count;
                    cur = i;
                    c = {0.f, 0.f}; left = {1.f, 0.f}; gone = 0;
                    summed = false;
                } else if (draft) {
                    c = c + left;
                    pass = true;
                } else {
                    left = left - r;
                    if (lane == 0) dead[gone] = tok[i];
                    ++gone;
                    __syncwarp();
                }
            }
            if (!pass && !summed) pass = true;               // for the last token
            if (!pass && !bare && !(st.total.hi > 0.f) && (c.hi > 0.f || gone)) bare = pass = true;
            __syncwarp();
            if (lane == 0) {
                st.cur = cur; st.at = at; st.count = count; st.gone = gone;
                st.c = c; st.left = left;
                st.summed = summed; st.bare = bare; st.pass = pass;
            }
        }
        __syncthreads();
        if (!st.pass) break;
        const Rows<Tp> w(p, st, b);
        const int64_t e0 = ((int64_t)rank * WARPS + warp) * piece - w.lead;
        const int64_t size = min(piece, (int64_t)V - e0);   // none or less where the row ends before
        Pair s = {0.f, 0.f};
        if (w.q) {
            Sums sp, sq;
            for (int64_t i = 0; i < size; i += 512) {
                float4 y[4], z[4];
                if (w.wide && i + 512 <= size && e0 + i >= 0) {   // all of it in the row: nothing between the loads
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        y[x] = load4(w.p + e0 + i + 128 * x + 4 * lane);
                        z[x] = load4(w.q + e0 + i + 128 * x + 4 * lane);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int64_t e = i + 128 * x < size ? e0 + i + 128 * x + 4 * lane : V;
                        y[x] = values(w.p, e, V, w.wide);
                        z[x] = values(w.q, e, V, w.wide);
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const bool2 a = exceeds(make_float2(y[x].x, y[x].y), make_float2(z[x].x, z[x].y), w.c);
                    const bool2 o = exceeds(make_float2(y[x].z, y[x].w), make_float2(z[x].z, z[x].w), w.c);
                    sp.add(make_float2(a.x ? y[x].x : 0.f, a.y ? y[x].y : 0.f));
                    sq.add(make_float2(a.x ? z[x].x : 0.f, a.y ? z[x].y : 0.f));
                    sp.add(make_float2(o.x ? y[x].z : 0.f, o.y ? y[x].w : 0.f));
                    sq.add(make_float2(o.x ? z[x].z : 0.f, o.y ? z[x].w : 0.f));
                }
            }
            s = sp.value() - w.c * sq.value();
        } else {
            bool odd = false;                                // rejected tokens in this piece
            for (int j = 0; j < w.gone; ++j) odd |= dead[j] >= e0 && dead[j] < e0 + size;
            Sums sp;
            for (int64_t i = 0; i < size; i += 1024) {
                float4 y[8];
                if (i + 1024 <= size && e0 + i >= 0) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) y[x] = load4(w.p + e0 + i + 128 * x + 4 * lane);
                } else
#pragma unroll
                    for (int x = 0; x < 8; ++x) y[x] = values(w.p, i + 128 * x < size ? e0 + i + 128 * x + 4 * lane : V, V, w.wide);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (odd)
                        for (int d = 0; d < w.gone; ++d) {
                            const int64_t at = dead[d] - (e0 + i + 128 * x + 4 * lane);
                            if (at == 0) y[x].x = 0.f;
                            if (at == 1) y[x].y = 0.f;
                            if (at == 2) y[x].z = 0.f;
                            if (at == 3) y[x].w = 0.f;
                        }
                    sp.add(make_float2(fmaxf(y[x].x, 0.f), fmaxf(y[x].y, 0.f)));
                    sp.add(make_float2(fmaxf(y[x].z, 0.f), fmaxf(y[x].w, 0.f)));
                }
            }
            s = sp.value();
        }
        s = not_below_0(warp_sum(s));
        if (cluster > 1) {                                   // this piece's sum to all CTAs
            if (lane < cluster) store_to(&part[round & 1][rank * WARPS + warp], lane, s);
            cluster_sync();
        } else {
            if (lane == 0) part[round & 1][warp] = s;
            __syncthreads();
        }
        if (warp == 0) {
            Pair total = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < PER_LANE; ++k)
                if (PER_LANE * lane + k < cluster * WARPS) total = total + part[round & 1][PER_LANE * lane + k];
            total = warp_sum(total);
            if (lane == 0) {
                if (w.q) st.left = total;
                st.total = total;
                st.summed = true;
            }
            __syncwarp();
        }
        last = round & 1;
    }

    // the last token: the first at which the running sum of R exceeds u times all of
    // it, by piece, by a share of that, by value
    if (rank == 0) {
        if (tid < T) p.path[b * T + tid] = path[tid];
        if (tid == 0) p.count[b] = st.count;
    }
    const Pair goal = st.total * uni[0];
    if (warp == 0) {
        Pair x[PER_LANE], sum = {0.f, 0.f}, before = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < PER_LANE; ++k) {
            x[k] = PER_LANE * lane + k < cluster * WARPS ? part[last][PER_LANE * lane + k] : Pair{0.f, 0.f};
            sum = sum + x[k];
        }
        bool past;
        const int l = find_lane(sum, goal, before, past, lane);
        if (lane == l) {
            int k = 0;
            Pair run = before;
            if (past) {                                      // the last one that is not 0
                for (int j = 0; j < PER_LANE; ++j) if (x[j].hi > 0.f) k = j;
            } else {
                bool hit = false;
#pragma unroll
                for (int j = 0; j < PER_LANE; ++j)
                    if (!hit && x[j].hi > 0.f) {
                        k = j;
                        before = run;
                        run = run + x[j];
                        hit = run > goal;
                    }
            }
            spiece = PER_LANE * lane + k;
            sbefore = before;
            spast = past;
        }
        if (l < 0 && lane == 0) spiece = -1;
    }
    __syncthreads();
    if (spiece < 0) {                                        // a row of zeros
        if (rank == 0 && tid == 0) p.next[b] = -1;
        return;
    }
    if (spiece / WARPS != (int)rank) return;
    const Rows<Tp> w(p, st, b);
    const int64_t share = (piece / WARPS + 127) / 128 * 128; // of the piece, a warp
    const int64_t e0 = (int64_t)spiece * piece - w.lead, end = min(e0 + piece, (int64_t)V);
    {
        Pair s = {0.f, 0.f};
        const int64_t from = e0 + warp * share, to = min(from + share, end);
        for (int64_t e = from + 4 * lane; e < to; e += 128) {
            Pair r[4];
            residual(w, e, V, dead, r);
            s = s + ((r[0] + r[1]) + (r[2] + r[3]));
        }
        s = warp_sum(s);
        if (lane == 0) sub[warp] = s;
    }
    __syncthreads();
    Pair before = sbefore;
    bool past;
    const int x = find_lane(lane < WARPS ? sub[lane] : Pair{0.f, 0.f}, goal, before, past, lane);
    if (warp != max(x, 0)) return;
    const bool seek = !(spast || past);                      // (past: sums that differ in their last bits)
    const int64_t from = e0 + warp * share, to = min(from + share, end);
    int64_t found = -1, tail = -1;
    for (int64_t e1 = from; e1 < to && found < 0; e1 += 128) {
        const int64_t e = e1 + 4 * lane;
        Pair r[4] = {}, incl = {0.f, 0.f};
        if (e < to) residual(w, e, V, dead, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (r[j].hi > 0.f) tail = e + j;
            incl = incl + r[j];
        }
        const Pair own = incl;
        incl = warp_scan(incl, lane);
        int64_t hit = -1;
        Pair run = before + (incl - own);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            run = run + r[j];
            if (hit < 0 && r[j].hi > 0.f && run > goal) hit = e + j;
        }
        const uint32_t who = seek ? __ballot_sync(0xffffffffu, hit >= 0) : 0u;
        if (who) found = __shfl_sync(0xffffffffu, hit, __ffs((int)who) - 1);
        before = before + shfl(incl, 31);
    }
    if (found < 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int64_t y = __shfl_xor_sync(0xffffffffu, tail, o);
            tail = y > tail ? y : tail;
        }
        found = tail;
    }
    if (lane == 0) p.next[b] = (int32_t)found;
}

template <typename Tp> cudaError_t run(const VerifyArgs &a, cudaStream_t st) {
    // CTAs a sequence: until there are four an SM, and no fewer than 2048 values each.  The
    // batch of 256 trees: 148, 109, 94 and 100 us with 1, 2, 4 and 8; one sequence over 50,021
    // tokens 19, 12.6, 10.2 and 8.2.
    int cluster = 1;
    while (cluster < MAX_CLUSTER && (int64_t)a.B * cluster < 608 && (int64_t)cluster * 4096 <= a.V) cluster *= 2;
    const int64_t pieces = (int64_t)cluster * WARPS;
    const int64_t piece = ((int64_t)a.V + 3 + pieces * 128 - 1) / (pieces * 128) * 128;
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
    return cudaLaunchKernelEx(&cfg, verify_kernel<Tp>, a, cluster, piece);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st) {
    return a.dtype == 0 ? run<__nv_bfloat16>(a, st) : run<float>(a, st);
}

}  // namespace tree
}  // namespace kda
