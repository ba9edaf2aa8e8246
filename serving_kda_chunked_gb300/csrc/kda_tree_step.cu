// kda_tree_step.cu -- a KDA or Gated DeltaNet layer's outputs for a tree of
// drafted tokens, the state left as it is (kda_tree_step in kda.h).
//
// The decode recurrence along the path from the state S to node r, unrolled.
// With gamma_r the sum of the gates on that path, and i < r over r's ancestors:
//   A_ri = beta_r sum_c k_rc k_ic e^(gamma_rc - gamma_ic)
//   P_ri =        sum_c q_rc k_ic e^(gamma_rc - gamma_ic)        (and i = r)
//   u_r  = beta_r (v_r - (k_r e^gamma_r) S) - sum_i A_ri u_i
//   o_r  = (q_r e^gamma_r) S + sum_i P_ri u_i
// so that S meets all 2 T rows k_r e^gamma_r and q_r e^gamma_r in one product, is
// read once and not written; siblings share what is above them.
//
// What bounds it: S is 64 KB a head (D = 128) and is read once: HBM.  One CTA per (sequence,
// head), all of whose products are m16n8k8 tf32 MMAs (bf16 inputs).  With T nodes those
// have 2 T rows at most, 16 for the usual eight nodes: an eighth of a 128-row tcgen05.mma,
// which would want S in shared memory first, where two CTAs an SM would fit in place of six.
//   1. gamma by doubling: every round adds up twice as far a stretch of the paths;
//   2. A and P as one product of the rows k e^gamma, q e^gamma with k e^-gamma.  Where gamma
//      falls below -100 (log2), pair by pair in float32 instead, no exponent above 0;
//   3. M with M (I + A) = P by tiles of 8 nodes, from the last to the first;
//   4. the 2 T rows times S; d_j = beta_j (v_j - (k_j e^gamma_j) S);  o = (q e^gamma) S + M d.
// Operands are rounded to tf32's 11 bits, as many as the prefill's fp16 operands have;
// gates, sums and the state are float32, and what a commit writes never passes through here.
//
// Measured, 32 heads, D = 128: 256 sequences with chains of 8 nodes 99 us, with one 88 (6.2 TB/s;
// the latency of phases and L1 stand beside HBM); with up to 8 in a pool 102; 32 sequences with
// 64 nodes 73 us in trees three wide, 76 in chains: two CTAs an SM take 1,024 in 3.4 rounds,
// of which loads and phases 1 and 2 up to the rows are 27 us, A and P 12, M 6, the state's product 18
// (its MMAs alone, at 8 cycles, 14) and the rest 10.
// On the way, with 8 and with 64 nodes: gates and A, P by FMAs and shuffles 127 and 137; the
// state's lines read by four lanes each of eight rows (L1 wavefronts at 67%) 118 and 110; M node
// by node along the paths 105 and 89, and 108 and 185 for chains (a third of all instructions);
// k e^gamma and q e^gamma in rows of their own, whose loads are not in the order of an MMA's registers,
// 103 and 76.
// Pair by pair, where one channel of one node of a head falls below the range: 256 sequences of 8 nodes
// 102 -> 114 us, of 16 127 -> 221, 64 of 32 71 -> 168, 32 of 64 79 -> 310 (a node's path four ancestors
// at a time, each four with sums over the lanes; all of the CTA's nodes, whichever of them is far).
// Gated DeltaNet reads fewer gates and gains nothing by it, the phases being what they are: 256 sequences of
// 8 nodes 102 us, of 16 129, 32 of 64 80; D = 64: 32, 65 and 48 us (KDA 33, 62 and 43).
// Tried: what a later CTA reads asked into L2, 64 nodes 87 to 89 (of 82); 1, 2 or 8 unrolled steps of 4
// with 4 to 9 CTAs an SM in phase 4, 8 nodes 106 to 112 (of 105); values loaded before phase 4 103 (of 102).
//
// float32 inputs: FMAs, A and P pair by pair, M node by node along the paths (the deltas one node after
// the other, each from its ancestors': 32 sequences with chains of 64 1350 us, here 637; in trees
// three wide 623 and 352).
#include "kda_tree.cuh"

#include <mutex>

namespace kda {
namespace tree {
namespace {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// To nearest, ties to even: one instruction, where ties away from 0 take four (64 nodes: 76 us, 82).
__device__ __forceinline__ float to_tf32(float x) {
    uint32_t y;
    asm("cvt.rn.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
    return __uint_as_float(y);
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)),
                   "r"(__float_as_uint(a3)), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

__device__ __forceinline__ float2 load2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }
__device__ __forceinline__ void prefetch_bulk(const void *p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(p), "r"(bytes) : "memory");
}

// A row of bf16 as a lane loads it.
template <int D> struct Raw { uint32_t x[D / 64]; };
template <int D> __device__ __forceinline__ Raw<D> load_raw(const __nv_bfloat16 *p, int lane) {
    Raw<D> r;
    if constexpr (D == 128) {
        const uint2 y = *reinterpret_cast<const uint2 *>(p + 4 * lane);
        r.x[0] = y.x; r.x[1] = y.y;
    } else {
        r.x[0] = *reinterpret_cast<const uint32_t *>(p + 2 * lane);
    }
    return r;
}

// Channels a lane holds of a row of D: consecutive ones.
template <int D> struct Row { float x[D / 32]; };
template <int D, typename Tin> __device__ __forceinline__ Row<D> load_row(const Tin *p, int lane) {
    Row<D> r;
    if constexpr (D == 128) {
        const float4 y = load4(p + 4 * lane);
        r.x[0] = y.x; r.x[1] = y.y; r.x[2] = y.z; r.x[3] = y.w;
    } else {
        r.x[0] = to_f32(p[2 * lane]);
        r.x[1] = to_f32(p[2 * lane + 1]);
    }
    return r;
}
template <int D> __device__ __forceinline__ void store_row(float *p, int lane, const Row<D> &r) {
    if constexpr (D == 128) store4(p + 4 * lane, make_float4(r.x[0], r.x[1], r.x[2], r.x[3]));
    else *reinterpret_cast<float2 *>(p + 2 * lane) = make_float2(r.x[0], r.x[1]);
}
template <int D> __device__ __forceinline__ Row<D> spread(float x) {
    Row<D> r;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) r.x[c] = x;
    return r;
}
template <int D> __device__ __forceinline__ Row<D> unpack(const Raw<D> &a) {
    Row<D> r;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&a.x[i]));
        r.x[2 * i] = y.x;
        r.x[2 * i + 1] = y.y;
    }
    return r;
}

constexpr float LOG2E = 1.4426950408889634f;

// Shared memory.  bf16: rows of (k e^gamma, q e^gamma) channel by channel, as an MMA wants
// them in a thread's registers (before them gamma, after the product the deltas d), and k e^-gamma;
// A and P, then M; masks, betas, who is above whom.  With 64 nodes A and P take
// the place of k e^-gamma, so that two CTAs fit an SM.  fp32: rows k e^gamma, after the product the
// deltas, and q e^gamma; A and P, then M; masks, betas; up to 16 nodes the inputs.
template <int D, int NT> struct Smem {       // NT: nodes, a multiple of 8
    static constexpr int LD = D + 8;         // four rows' reads of eight channels meet different banks
    static constexpr int LDK = 2 * D + 16;   // two rows' reads of eight channels of both do
    static constexpr int LDU = D + 4;        // the deltas' rows: every other of eight rows' reads of 32 columns do
    static constexpr int LDS = D + 16;       // fp32: two rows' reads of 16 channels do
    static constexpr int LDA = NT + 4, LDP = NT + 8;   // A and P of node r: pa[r * LDA + i], pp[r * LDP + i]
    static constexpr bool OVER = NT == 64, STAGED = NT <= 16;
    static constexpr uint32_t AP_BYTES = NT * (LDA + LDP) * 4;
    // bf16
    static constexpr uint32_t KI = NT * LDK * 4, KI_BYTES = NT * LD * 4, AP = OVER ? KI : KI + KI_BYTES,
                              MASK = AP + (OVER && AP_BYTES < KI_BYTES ? KI_BYTES : AP_BYTES), BETA = MASK + NT * 8, UPS = BETA + NT * 4, TC_BYTES = UPS + 6 * NT + 16;
    // fp32
    static constexpr uint32_t SQG = NT * LDS * 4, SAP = 2 * SQG, SMASK = SAP + AP_BYTES, SBETA = SMASK + NT * 8,
                              ROWS = SBETA + NT * 4, SIMT_BYTES = ROWS + (STAGED ? NT * D * 16 : 0);
};
// Warps a CTA: one for every 32 columns; from 32 nodes on (D = 64: 16) two, which share the nodes.
template <int D, int NT> struct Warps { static constexpr int COLS = D / 32, SPLIT = NT >= 32 || (D == 64 && NT == 16) ? 2 : 1, ALL = COLS * SPLIT; };

// A and P pair by pair, and the rows that meet the state, all in float32: a warp a node,
// up its path, nearest ancestor first, with the gates between them summed on the way
// (differences of sums from the root would cancel); what the sum is at the end fades the
// rows.  Four ancestors at a time, so that their loads are under way together and the sums
// over the lanes share exchanges.  in, gs: elements between nodes of k and q, of the gates.
// EACH: floats between a row's channels.
template <int D, int NT, int LD, int EACH, int WARPS, typename Tin>
__device__ __forceinline__ void pair_by_pair(const Tin *q, const Tin *k, const float *g, int64_t in, int64_t gs, bool scalar_gate,
                                             const uint64_t *mask, const float *beta, float *kg, float *qg, float *pa, float *pp) {
    constexpr int LDA = Smem<D, NT>::LDA, LDP = Smem<D, NT>::LDP, C = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int r = warp; r < NT; r += WARPS) {
        uint64_t m = mask[r];
        const bool on = m != 0;
        Row<D> kr = {}, qr = {}, run = {};
        if (on) {
            kr = load_row<D>(k + r * in, lane);
            qr = load_row<D>(q + r * in, lane);
        }
        for (int i = lane; i < NT; i += 32) pa[r * LDA + i] = pp[r * LDP + i] = 0.f;
        __syncwarp();
        while (m) {
            int at[4];
            Row<D> ki[4], gi[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                at[u] = m ? 63 - __clzll((long long)m) : -1;
                ki[u] = {}; gi[u] = {};
                if (m) {
                    m ^= 1ull << at[u];
                    ki[u] = load_row<D>(k + at[u] * in, lane);
                    if (scalar_gate) {
                        const float x = g[at[u] * gs];
#pragma unroll
                        for (int c = 0; c < C; ++c) gi[u].x[c] = x;
                    } else {
                        gi[u] = load_row<D>(g + at[u] * gs, lane);
                    }
                }
            }
            float sum[8] = {};                           // A, P of each
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float w = ki[u].x[c] * ex2(run.x[c]);
                    sum[2 * u] += kr.x[c] * w;
                    sum[2 * u + 1] += qr.x[c] * w;
                    run.x[c] += gi[u].x[c] * LOG2E;
                }
            // every exchange halves the sums a lane keeps
#pragma unroll
            for (int bit = 16, half = 4; bit >= 4; bit >>= 1, half >>= 1) {
                const bool up = lane & bit;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < half) {
                        const float give = up ? sum[e] : sum[e + half], have = up ? sum[e + half] : sum[e];
                        sum[e] = have + __shfl_xor_sync(0xffffffffu, give, bit);
                    }
            }
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
            const int u = lane >> 3, i = u == 0 ? at[0] : (u == 1 ? at[1] : (u == 2 ? at[2] : at[3]));
            if ((lane & 3) == 0 && i >= 0) {
                if (lane & 4) pp[r * LDP + i] = sum[0];
                else pa[r * LDA + i] = beta[r] * sum[0];
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float f = on ? ex2(run.x[c]) : 0.f;
            const float a = kr.x[c] * f, z = qr.x[c] * f;
            kg[r * LD + EACH * (C * lane + c)] = sizeof(Tin) == 2 ? to_tf32(a) : a;
            qg[r * LD + EACH * (C * lane + c)] = sizeof(Tin) == 2 ? to_tf32(z) : z;
        }
    }
}

// CTAs an SM that registers are shared out for (bf16).  One more or fewer, 32 heads, D = 128: 8
// nodes 99 us, 5 102, 8 102; 16 nodes 67, 4 72, 6 69; 32 nodes 71, 2 81.  D = 64: 8 nodes 32, 9 35,
// 20 34; 16 nodes 35, 4 41; 32 nodes 29, 4 30, 6 33; 64 nodes 40, 2 48.
template <int D, int NT> constexpr int resident() {
    return D == 128 ? (NT == 8 ? 6 : (NT == 16 ? 5 : (NT == 32 ? 3 : 2))) : (NT == 8 ? 16 : (NT == 16 ? 6 : (NT == 32 ? 5 : 3)));
}
// Beyond 2^-RANGE of decay from the root, e^-gamma and the products with it could leave float32.
constexpr float RANGE = 100.f;

template <int D, int NT>
__global__ void __launch_bounds__(32 * Warps<D, NT>::ALL, resident<D, NT>()) step_tc_kernel(const StepArgs p) {
    using L = Smem<D, NT>;
    using Tin = __nv_bfloat16;
    constexpr int LD = L::LD, LDK = L::LDK, LDU = L::LDU, LDA = L::LDA, LDP = L::LDP, C = D / 32;
    constexpr int SPLIT = Warps<D, NT>::SPLIT, WARPS = Warps<D, NT>::ALL, THREADS = 32 * WARPS;
    extern __shared__ __align__(16) uint8_t sm[];
    float *kq = reinterpret_cast<float *>(sm), *ki = reinterpret_cast<float *>(sm + L::KI);
    float *pa = reinterpret_cast<float *>(sm + L::AP), *pp = pa + NT * LDA;
    uint64_t *mask = reinterpret_cast<uint64_t *>(sm + L::MASK);
    float *beta = reinterpret_cast<float *>(sm + L::BETA);
    int8_t *ups = reinterpret_cast<int8_t *>(sm + L::UPS);  // [round][node]: the node 2^round above
    int *rounds = reinterpret_cast<int *>(sm + L::UPS + 6 * NT);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, T = p.T;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t step = (int64_t)p.H * D;                              // between a head's nodes
    const int64_t at0 = (int64_t)b * T * step + (int64_t)h * D;         // of node 0
    const int64_t bt0 = (int64_t)b * T * p.H + h;
    const Tin *q = (const Tin *)p.q + at0, *k = (const Tin *)p.k + at0, *v = (const Tin *)p.v + at0;
    const float *g = p.scalar_gate ? p.g + bt0 : p.g + at0;
    const int64_t gs = p.scalar_gate ? p.H : step;
    Tin *o = (Tin *)p.o + at0;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) {
            for (int e = tid; e < T * D; e += THREADS) o[e / D * step + e % D] = from_f32<Tin>(0.f);
            return;
        }
    }
    const float *S = p.S + (slot * p.H + h) * (D * D);
    // values start on their way to L2, this warp's rows of k and q to registers, gates to shared
    // memory; behind them the state to L2: in front of them it kept them waiting (batch of 256
    // sequences with 8 nodes: 118 us, here 106; without 115)
    constexpr int LINES = D * (int)sizeof(Tin) / 128;
    for (int i = tid; i < T * LINES; i += THREADS) prefetch_l2((const char *)(v + i / LINES * step) + i % LINES * 128);
    constexpr int MINE = NT / WARPS;                     // nodes warp, warp + WARPS, ...
    Raw<D> kr[MINE], qr[MINE];
#pragma unroll
    for (int n = 0; n < MINE; ++n) {
        const int r = warp + n * WARPS;
        kr[n] = {}; qr[n] = {};
        if (r < T) {
            kr[n] = load_raw<D>(k + r * step, lane);
            qr[n] = load_raw<D>(q + r * step, lane);
        }
    }
    if (p.scalar_gate) {
#pragma unroll
        for (int n = 0; n < MINE; ++n) {
            const int r = warp + n * WARPS;
            if (r < T) {
                const float x = g[r * gs];
                store_row<D>(kq + r * LD, lane, spread<D>(x));
            }
        }
    } else {
        for (int e = tid; e < T * (D / 4); e += THREADS)
            copy16(kq + e / (D / 4) * LD + e % (D / 4) * 4, g + e / (D / 4) * step + e % (D / 4) * 4);
    }
    if (warp == 0) {
        uint64_t x, y;
        const int n = all_ancestors(p.parents + (int64_t)b * T, T, lane, x, y, [&](int round, int up0, int up1) {
            if (lane < NT) ups[round * NT + lane] = (int8_t)up0;
            if (NT > 32) ups[round * NT + lane + 32] = (int8_t)up1;
        });
        if (lane < NT) mask[lane] = x;
        if (NT > 32) mask[lane + 32] = y;
        if (lane == 0) *rounds = n;
    }
    if (tid < T) beta[tid] = p.beta[bt0 + (int64_t)tid * p.H];
    if (tid == 0) prefetch_bulk(S, D * D * 4);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // gamma: every round adds up twice as far a stretch of the paths, from one buffer to
    // the other; a warp its rows.  A row that stood still for two rounds is in both.
    float *was = kq, *now = ki;
    const int n_rounds = *rounds;
    Row<D> gm[MINE];
    int above[MINE];
#pragma unroll
    for (int n = 0; n < MINE; ++n) {
        gm[n] = load_row<D>(kq + (warp + n * WARPS) * LD, lane);
        above[n] = 0;
    }
    for (int k = 0; k < n_rounds; ++k) {
        bool moved[MINE];
        Row<D> y[MINE];
#pragma unroll
        for (int n = 0; n < MINE; ++n) {
            moved[n] = above[n] >= 0;
            if (moved[n]) above[n] = ups[k * NT + warp + n * WARPS];
        }
#pragma unroll
        for (int n = 0; n < MINE; ++n)
            y[n] = above[n] >= 0 ? load_row<D>(was + above[n] * LD, lane) : Row<D>{};
#pragma unroll
        for (int n = 0; n < MINE; ++n) {
#pragma unroll
            for (int c = 0; c < C; ++c) gm[n].x[c] += y[n].x[c];
            if (moved[n] && k + 1 < n_rounds) store_row<D>(now + (warp + n * WARPS) * LD, lane, gm[n]);
        }
        if (k + 1 < n_rounds) __syncthreads();
        float *z = was;
        was = now;
        now = z;
    }
    bool far = false;
#pragma unroll
    for (int n = 0; n < MINE; ++n) {
        const int r = warp + n * WARPS;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            gm[n].x[c] = mask[r] ? gm[n].x[c] * LOG2E : 0.f; // in log2 units
            far |= !(fabsf(gm[n].x[c]) <= RANGE);       // (or a gate that is not a number)
        }
    }
    const int gq = lane >> 2, c4 = lane & 3, cols = 32 * (warp / SPLIT);
    // A warp's tiles of 8 nodes.  With one each, the two warps of a scheduler (w, w + 4) have
    // 9 of the 36 products of two tiles.
    constexpr int TILES = (NT / 8 + WARPS - 1) / WARPS;
    const auto tile_of = [&](int t) { return NT == 64 && WARPS == 8 && warp >= 4 ? 11 - warp : warp + t * WARPS; };
    float pr[TILES][NT / 8][4] = {};                     // A and P; then in 0 and 1 row gq, columns 8 j + 2 c4 and the next
    if (__syncthreads_or(far)) {
        pair_by_pair<D, NT, LDK, 2, WARPS>(q, k, g, step, gs, p.scalar_gate, mask, beta, kq, kq + 1, pa, pp);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int j = 0; j < NT / 8; ++j)
                if (tile_of(t) < NT / 8) {
                    const float2 x = load2(pp + (8 * tile_of(t) + gq) * LDP + 8 * j + 2 * c4);
                    pr[t][j][0] = x.x;
                    pr[t][j][1] = x.y;
                }
    } else {
#pragma unroll
        for (int n = 0; n < MINE; ++n) {
            const int r = warp + n * WARPS;
            if (!mask[r]) kr[n] = qr[n] = {};
            Row<D> a = unpack<D>(kr[n]), z = unpack<D>(qr[n]), i;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float f = ex2(gm[n].x[c]);
                i.x[c] = to_tf32(a.x[c] * ex2(-gm[n].x[c]));
                a.x[c] = to_tf32(a.x[c] * f);
                z.x[c] = to_tf32(z.x[c] * f);
            }
#pragma unroll
            for (int c = 0; c < C; c += 2)
                store4(kq + r * LDK + 2 * (C * lane + c), make_float4(a.x[c], z.x[c], a.x[c + 1], z.x[c + 1]));
            store_row<D>(ki + r * LD, lane, i);
        }
        __syncthreads();
        // A and P of 8 nodes a warp: e^(gamma_r - gamma_i) is the product of the two rows' factors.
        // Channels 8 s + 2 c4 and the next one are the MMA's c4 and c4 + 4, so that one load has both.
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int tile = tile_of(t);
            if (tile >= NT / 8) break;
#pragma unroll 4
            for (int s = 0; s < D / 8; ++s) {
                const float4 a = load4(kq + (8 * tile + gq) * LDK + 16 * s + 4 * c4);
#pragma unroll
                for (int j = 0; j < NT / 8; ++j)
                    if (j / 2 * 2 <= tile) {             // nodes see earlier ones only
                        const float2 x = load2(ki + (8 * j + gq) * LD + 8 * s + 2 * c4);
                        mma_tf32(pr[t][j], a.x, a.y, a.z, a.w, x.x, x.y);
                    }
            }
        }
        if constexpr (L::OVER) __syncthreads();
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int tile = tile_of(t);
            if (tile >= NT / 8) break;
            const int r = 8 * tile + gq;
            const uint64_t m = mask[r];
            const float br = m ? beta[r] : 0.f;
            const uint32_t lo = (uint32_t)m >> 2 * c4, hi = (uint32_t)(m >> 32) >> 2 * c4;
#pragma unroll
            for (int j = 0; j < NT / 8; ++j) {           // zeros where r does not see a node
                const int i = 8 * j + 2 * c4;
                const uint32_t sees = j < 4 ? lo : hi;
                const bool s0 = sees >> 8 * (j % 4) & 1, s1 = sees >> 8 * (j % 4) & 2;
                *reinterpret_cast<float2 *>(pa + r * LDA + i) = make_float2(s0 ? br * pr[t][j][0] : 0.f, s1 ? br * pr[t][j][1] : 0.f);
                pr[t][j][0] = s0 ? pr[t][j][2] : 0.f;
                pr[t][j][1] = s1 ? pr[t][j][3] : 0.f;
                pr[t][j][2] = pr[t][j][3] = 0.f;
            }
        }
    }

    // The nodes' rows times the state.  Column group j's MMA column gq is S's column 4 gq + j of
    // the warp's 32.  The MMA wants channel c4 of four, columns 4 gq .. in lane 4 gq + c4;
    // the lanes load them as 8 c4 + gq, so that eight lanes read a line of 128 bytes (four
    // lines by two sectors each take four times the wavefronts of the L1), and exchange.
    constexpr int MT = NT / 8 / SPLIT;
    const int part = warp % SPLIT;                       // this warp's tiles of 8 nodes: part, part + SPLIT, ...
    const int from = 8 * c4 + gq;
    const float *Sl = S + 2 * (lane >> 3) * D + cols + 4 * (lane & 7);
    constexpr bool PIPE = MT > 2;                        // enough products to load the next lines behind
    float4 y[4];
    if constexpr (PIPE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = load4(Sl + (j / 2 * 8 + j % 2) * D);
    }

    // o_r = (q_r e^gamma_r) S + sum_j M_rj d_j with d_j = beta_j (v_j - (k_j e^gamma_j) S) and
    // M (I + A) = P.  Within a tile of 8 nodes one column comes after the other: one tile alone is
    // solved so, of several the inverses of I + A (in place of A's), with which P's columns are
    // multiplied from the last tile to the first; M A's other tiles come off P on the way.  All
    // factors are taken as two tf32 numbers (P's and M's two fill the MMA's 16 rows), which keeps
    // what float32 has.
    __syncthreads();
    const auto solve = [&](int J, float &x0, float &x1) {        // row gq, columns 2 c4 and the next: X (I + A_JJ)^-1
        float2 a[8];
#pragma unroll
        for (int c = 1; c < 8; ++c) a[c] = load2(pa + (8 * J + c) * LDA + 8 * J + 2 * c4);
#pragma unroll
        for (int c = 7; c > 0; --c) {
            const float m = __shfl_sync(0xffffffffu, c & 1 ? x1 : x0, (lane & 28) + c / 2);
            if (2 * c4 < c) x0 -= m * a[c].x;
            if (2 * c4 + 1 < c) x1 -= m * a[c].y;
        }
    };
    const auto times = [&](float (&y)[4], float (&z)[4], float h0, float h1, float l0, float l1, int J, int j) {      // y + z += rows times A_Jj
        const float *b = pa + (8 * J + 2 * c4) * LDA + 8 * j + gq;
        const float b0 = b[0], b1 = b[LDA], y0 = to_tf32(b0), y1 = to_tf32(b1);
        mma_tf32(y, h0, l0, h1, l1, y0, y1);
        mma_tf32(z, h0, l0, h1, l1, to_tf32(b0 - y0), to_tf32(b1 - y1));
    };
    if constexpr (NT > 8) {
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int tile = tile_of(t);
            if (tile >= NT / 8) break;
            float x0 = gq == 2 * c4 ? 1.f : 0.f, x1 = gq == 2 * c4 + 1 ? 1.f : 0.f;
            solve(tile, x0, x1);
            __syncwarp();
            *reinterpret_cast<float2 *>(pa + (8 * tile + gq) * LDA + 8 * tile + 2 * c4) = make_float2(x0, x1);
        }
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        const int tile = tile_of(t);
        if (tile >= NT / 8) break;
        const int r = 8 * tile + gq;
        const bool on = mask[r] != 0;
#pragma unroll
        for (int J = NT / 8 - 1; J >= 0; --J) {
            if (J > tile) continue;
            float x0 = pr[t][J][0] + pr[t][J][2], x1 = pr[t][J][1] + pr[t][J][3];
            float h0, h1, l0, l1;
            if constexpr (NT == 8) {
                if (n_rounds) solve(J, x0, x1);          // a node has a parent
            } else {
                h0 = to_tf32(x0); h1 = to_tf32(x1); l0 = to_tf32(x0 - h0); l1 = to_tf32(x1 - h1);
                float y[4] = {}, z[4] = {};
                times(y, z, h0, h1, l0, l1, J, J);
                x0 = (y[0] + y[2]) + (z[0] + z[2]);
                x1 = (y[1] + y[3]) + (z[1] + z[3]);
            }
            h0 = on ? to_tf32(x0) : 0.f; h1 = on ? to_tf32(x1) : 0.f;
            *reinterpret_cast<float2 *>(pp + r * LDP + 8 * J + 2 * c4) = make_float2(h0, h1);
            l0 = to_tf32(x0 - h0); l1 = to_tf32(x1 - h1);
#pragma unroll
            for (int j = J - 1; j >= 0; --j) times(pr[t][j], pr[t][j], -h0, -h1, -l0, -l1, J, j);
        }
    }
    // row gq of a tile: columns 8 c4 + j (from registers 0 and 2 of group j) and 8 c4 + 4 + j
    const int n0 = cols + 8 * c4;
    const auto values_of = [&](int mt) -> float4 {
        const int r = 8 * (mt * SPLIT + part) + gq;
        return mask[r] ? *reinterpret_cast<const float4 *>(v + r * step + n0) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    static_assert(!PIPE || MT == 4, "y holds a row's values of every tile");
    float4 vr[PIPE ? 1 : MT];
    float acc[MT][4][4] = {};
#pragma unroll(MT > 2 ? 1 : 4)
    for (int s = 0; s < D / 16; ++s) {
        if constexpr (!PIPE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = load4(Sl + (16 * s + j / 2 * 8 + j % 2) * D);
        }
        float f[4][4];                                   // [channel 16 s + 8 (j / 2) + 2 c4 + j % 2][column]
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j][0] = to_tf32(__shfl_sync(0xffffffffu, y[j].x, from));
            f[j][1] = to_tf32(__shfl_sync(0xffffffffu, y[j].y, from));
            f[j][2] = to_tf32(__shfl_sync(0xffffffffu, y[j].z, from));
            f[j][3] = to_tf32(__shfl_sync(0xffffffffu, y[j].w, from));
        }
        if (PIPE && s + 1 == D / 16) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) y[mt] = values_of(mt);
        } else if (PIPE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = load4(Sl + (16 * (s + 1) + j / 2 * 8 + j % 2) * D);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float4 a = load4(kq + (8 * (mt * SPLIT + part) + gq) * LDK + 32 * s + 16 * t + 4 * c4);
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_tf32(acc[mt][j], a.x, a.y, a.z, a.w, f[2 * t][j], f[2 * t + 1][j]);
            }
        }
    }
    if constexpr (!PIPE) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) vr[mt] = values_of(mt);
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = 8 * (mt * SPLIT + part) + gq;
        const __nv_bfloat162 *vv = reinterpret_cast<const __nv_bfloat162 *>(PIPE ? &y[mt] : &vr[PIPE ? 0 : mt]);
        const float2 v0 = __bfloat1622float2(vv[0]), v1 = __bfloat1622float2(vv[1]), v2 = __bfloat1622float2(vv[2]), v3 = __bfloat1622float2(vv[3]);
        const float br = mask[r] ? beta[r] : 0.f;        // padding: values and products are 0
        const float4 d0 = make_float4(br * (v0.x - acc[mt][0][0]), br * (v0.y - acc[mt][1][0]), br * (v1.x - acc[mt][2][0]), br * (v1.y - acc[mt][3][0]));
        const float4 d1 = make_float4(br * (v2.x - acc[mt][0][1]), br * (v2.y - acc[mt][1][1]), br * (v3.x - acc[mt][2][1]), br * (v3.y - acc[mt][3][1]));
        store4(kq + r * LDU + n0, make_float4(to_tf32(d0.x), to_tf32(d0.y), to_tf32(d0.z), to_tf32(d0.w)));
        store4(kq + r * LDU + n0 + 4, make_float4(to_tf32(d1.x), to_tf32(d1.y), to_tf32(d1.z), to_tf32(d1.w)));
    }
    __syncthreads();
    // M d on top of the q rows' products (registers 2 and 3); the k rows' are done with
#pragma unroll
    for (int ks = 0; ks < NT / 8; ++ks) {
        const float4 x = load4(kq + (8 * ks + 2 * c4) * LDU + cols + 4 * gq), y = load4(kq + (8 * ks + 2 * c4 + 1) * LDU + cols + 4 * gq);
        const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int tile = mt * SPLIT + part;
            if (mt * SPLIT + SPLIT - 1 < ks || tile < ks) continue;      // nodes see earlier ones only
            const float2 a = load2(pp + (8 * tile + gq) * LDP + 8 * ks + 2 * c4);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_tf32(acc[mt][j], 0.f, a.x, 0.f, a.y, xv[j], yv[j]);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = 8 * (mt * SPLIT + part) + gq;
        if (r < T) {
            __nv_bfloat162 y[4] = {__floats2bfloat162_rn(acc[mt][0][2], acc[mt][1][2]), __floats2bfloat162_rn(acc[mt][2][2], acc[mt][3][2]),
                                   __floats2bfloat162_rn(acc[mt][0][3], acc[mt][1][3]), __floats2bfloat162_rn(acc[mt][2][3], acc[mt][3][3])};
            *reinterpret_cast<uint4 *>(o + r * step + n0) = *reinterpret_cast<const uint4 *>(y);
        }
    }
}

// fp32: groups of 4 nodes that meet the state in one pass over it, and CTAs an SM that registers are
// shared out for.  32 heads, D = 128, trees three wide, with twice or half as many groups in a pass and
// the CTAs that leaves room for: 256 sequences of 8 nodes 203 us, 251; 128 of 16 213, 220; 64 of 32
// 255, 351 and 289; 32 of 64 352, 436 and 393.
template <int D, int NT> constexpr int simt_pass() { return D == 64 && NT == 8 ? 1 : (NT == 64 && D == 64 ? 4 : (NT == 16 && D == 128 ? 4 : 2)); }
template <int D, int NT> constexpr int simt_resident() {
    return D == 128 ? (NT == 8 ? 4 : (NT == 16 ? 3 : 2)) : (NT == 8 ? 8 : (NT == 16 ? 4 : (NT == 32 ? 3 : 1)));
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * Warps<D, NT>::ALL, simt_resident<D, NT>()) step_simt_kernel(const StepArgs p) {
    using L = Smem<D, NT>;
    using Tin = float;
    constexpr int LD = L::LDS, LDA = L::LDA, LDP = L::LDP;
    constexpr int SPLIT = Warps<D, NT>::SPLIT, WARPS = Warps<D, NT>::ALL, THREADS = 32 * WARPS;
    extern __shared__ __align__(16) uint8_t sm[];
    float *kg = reinterpret_cast<float *>(sm), *qg = reinterpret_cast<float *>(sm + L::SQG);
    float *pa = reinterpret_cast<float *>(sm + L::SAP), *pp = pa + NT * LDA;
    uint64_t *mask = reinterpret_cast<uint64_t *>(sm + L::SMASK);
    float *beta = reinterpret_cast<float *>(sm + L::SBETA);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, T = p.T;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t step = (int64_t)p.H * D;                              // between a head's nodes
    const int64_t at0 = (int64_t)b * T * step + (int64_t)h * D;         // of node 0
    const int64_t bt0 = (int64_t)b * T * p.H + h;
    const float *q = (const float *)p.q + at0, *k = (const float *)p.k + at0, *v = (const float *)p.v + at0;
    const float *g = p.scalar_gate ? p.g + bt0 : p.g + at0;
    int64_t in = step, gs = p.scalar_gate ? p.H : step;                 // between nodes of the inputs, of the gates
    float *o = (float *)p.o + at0;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) {
            for (int e = tid; e < T * D; e += THREADS) o[e / D * step + e % D] = 0.f;
            return;
        }
    }
    if constexpr (L::STAGED) {                           // all inputs to shared memory at once
        float *rows = reinterpret_cast<float *>(sm + L::ROWS), *gates = rows + 3 * NT * D;
        for (int e = tid; e < T * (D / 4); e += THREADS) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            copy16(rows + r * D + c, q + r * step + c);
            copy16(rows + (NT + r) * D + c, k + r * step + c);
            copy16(rows + (2 * NT + r) * D + c, v + r * step + c);
            if (!p.scalar_gate) copy16(gates + r * D + c, g + r * step + c);
        }
        if (p.scalar_gate && tid < T) gates[tid] = g[tid * gs];
        q = rows; k = rows + NT * D; v = rows + 2 * NT * D; g = gates;
        in = D;
        gs = p.scalar_gate ? 1 : D;
    }
    const float *S = p.S + (slot * p.H + h) * (D * D);
    if (tid == 0) prefetch_bulk(S, D * D * 4);
    if (warp == 0) {
        uint64_t x, y;
        all_ancestors(p.parents + (int64_t)b * T, T, lane, x, y);
        if (lane < NT) mask[lane] = x;
        if (NT > 32) mask[lane + 32] = y;
    }
    if (tid < T) beta[tid] = p.beta[bt0 + (int64_t)tid * p.H];
    if constexpr (L::STAGED) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    pair_by_pair<D, NT, LD, 1, WARPS>(q, k, g, in, gs, p.scalar_gate, mask, beta, kg, qg, pa, pp);
    __syncthreads();
    // M with M (I + A) = P, node by node along each node's path, nearest first (a warp a node, eight
    // chains side by side; a lane the nodes `lane` and `lane + 32`).  M replaces P.
    constexpr int MINE = NT / WARPS, CHAINS = MINE < 8 ? MINE : 8;
#pragma unroll 1
    for (int r0 = warp; r0 < T; r0 += CHAINS * WARPS) {
        int at[CHAINS];
        float m0[CHAINS], m1[CHAINS];
        bool any = false;
#pragma unroll
        for (int n = 0; n < CHAINS; ++n) {
            const int r = r0 + n * WARPS;
            at[n] = mask[r] ? r : -1;
            any |= at[n] >= 0;
            m0[n] = lane < NT ? pp[r * LDP + lane] : 0.f;
            m1[n] = NT > 32 ? pp[r * LDP + lane + 32] : 0.f;
        }
        while (any) {
            any = false;
#pragma unroll
            for (int n = 0; n < CHAINS; ++n) {
                const int i = at[n] < 0 ? 0 : at[n];
                float x = __shfl_sync(0xffffffffu, NT > 32 && i >= 32 ? m1[n] : m0[n], i & 31);
                const uint64_t above = mask[i] & ~(1ull << i);
                if (at[n] < 0) x = 0.f;                  // at its end
                at[n] = at[n] < 0 || !above ? -1 : 63 - __clzll((long long)above);
                any |= at[n] >= 0;
                // A's row i is 0 but for i's ancestors, and i
                if (lane < NT) m0[n] -= lane == i ? 0.f : x * pa[i * LDA + lane];
                if (NT > 32) m1[n] -= lane + 32 == i ? 0.f : x * pa[i * LDA + lane + 32];
            }
        }
#pragma unroll
        for (int n = 0; n < CHAINS; ++n) {
            const int r = r0 + n * WARPS;
            if (lane < NT) pp[r * LDP + lane] = mask[r] ? m0[n] : 0.f;
            if (NT > 32) pp[r * LDP + lane + 32] = mask[r] ? m1[n] : 0.f;
        }
    }

    const int gq = lane >> 2, c4 = lane & 3, cols = 32 * (warp / SPLIT);
    const float *Sw = S + cols + 4 * gq;                 // this thread's 4 columns
    // PASS groups of 4 nodes in one pass over the state; the four lanes of a column hold every
    // fourth group of 4 channels
    constexpr int GROUPS = NT / 4 / SPLIT, PASS = GROUPS < simt_pass<D, NT>() ? GROUPS : simt_pass<D, NT>();
    float4 keep[GROUPS][2];                          // node 4 t + c4: products with k, with q
#pragma unroll
    for (int x0 = 0; x0 < GROUPS; x0 += PASS) {
        if (4 * (x0 * SPLIT + warp % SPLIT) >= T) break;
        float w[PASS][4][4] = {}, z[PASS][4][4] = {};
#pragma unroll(D == 64 || NT == 8 ? 4 : 2)
        for (int s = 0; s < D / 16; ++s) {
            float4 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = load4(Sw + (16 * s + 4 * c4 + j) * D);
#pragma unroll
            for (int x = 0; x < PASS; ++x) {
                const int t = (x0 + x) * SPLIT + warp % SPLIT;
                if (4 * t >= T) break;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float4 a = load4(kg + (4 * t + n) * LD + 16 * s + 4 * c4);
                    const float4 c = load4(qg + (4 * t + n) * LD + 16 * s + 4 * c4);
                    const float av[4] = {a.x, a.y, a.z, a.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[x][n][0] += av[j] * y[j].x; w[x][n][1] += av[j] * y[j].y; w[x][n][2] += av[j] * y[j].z; w[x][n][3] += av[j] * y[j].w;
                        z[x][n][0] += cv[j] * y[j].x; z[x][n][1] += cv[j] * y[j].y; z[x][n][2] += cv[j] * y[j].z; z[x][n][3] += cv[j] * y[j].w;
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < PASS; ++x)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[x][n][e] += __shfl_xor_sync(0xffffffffu, w[x][n][e], 1);
                    w[x][n][e] += __shfl_xor_sync(0xffffffffu, w[x][n][e], 2);
                    z[x][n][e] += __shfl_xor_sync(0xffffffffu, z[x][n][e], 1);
                    z[x][n][e] += __shfl_xor_sync(0xffffffffu, z[x][n][e], 2);
                }
                if (n == c4) {
                    keep[x0 + x][0] = make_float4(w[x][n][0], w[x][n][1], w[x][n][2], w[x][n][3]);
                    keep[x0 + x][1] = make_float4(z[x][n][0], z[x][n][1], z[x][n][2], z[x][n][3]);
                }
            }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < GROUPS; ++x) {
        const int t = x * SPLIT + warp % SPLIT, r = 4 * t + c4, n = cols + 4 * gq;
        if (4 * t >= T) break;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mask[r]) {
            const float4 vv = load4(v + r * in + n), w = keep[x][0];
            const float br = beta[r];
            y = make_float4(br * (vv.x - w.x), br * (vv.y - w.y), br * (vv.z - w.z), br * (vv.w - w.w));
        }
        store4(kg + r * LD + n, y);                      // the delta
    }
    __syncthreads();
    // o = (q e^gamma) S + M d, four earlier nodes at a time
#pragma unroll 1
    for (int j = 0; j < T; j += 4) {
        float4 d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = load4(kg + (j + i) * LD + cols + 4 * gq);
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) {
            const int t = x * SPLIT + warp % SPLIT;
            if (4 * t >= T || 4 * t < j) continue;
            const float4 a = load4(pp + (4 * t + c4) * LDP + j);
            const float av[4] = {a.x, a.y, a.z, a.w};
            float4 &z = keep[x][1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z.x += av[i] * d[i].x; z.y += av[i] * d[i].y; z.z += av[i] * d[i].z; z.w += av[i] * d[i].w;
            }
        }
    }
#pragma unroll
    for (int x = 0; x < GROUPS; ++x) {
        const int t = x * SPLIT + warp % SPLIT, r = 4 * t + c4;
        if (4 * t >= T) break;
        if (r < T) store4(o + r * step + cols + 4 * gq, mask[r] ? keep[x][1] : make_float4(0.f, 0.f, 0.f, 0.f));
    }
}

template <int D, int NT, bool TC>
cudaError_t run(const StepArgs &a, cudaStream_t st) {
    constexpr uint32_t bytes = TC ? Smem<D, NT>::TC_BYTES : Smem<D, NT>::SIMT_BYTES;
    void (*kernel)(StepArgs) = TC ? step_tc_kernel<D, NT> : step_simt_kernel<D, NT>;
    if (bytes > 48 * 1024) {
        static std::mutex mu;
        static bool ready[64] = {false};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.H));
    cfg.blockDim = dim3(32 * Warps<D, NT>::ALL);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, bool TC>
cudaError_t by_nodes(const StepArgs &a, cudaStream_t st) {
    if (a.T <= 8) return run<D, 8, TC>(a, st);
    if (a.T <= 16) return run<D, 16, TC>(a, st);
    if (a.T <= 32) return run<D, 32, TC>(a, st);
    return run<D, 64, TC>(a, st);
}

}  // namespace

cudaError_t launch_step(const StepArgs &a, cudaStream_t st) {
    if (a.d == 128) return a.dtype == 0 ? by_nodes<128, true>(a, st) : by_nodes<128, false>(a, st);
    return a.dtype == 0 ? by_nodes<64, true>(a, st) : by_nodes<64, false>(a, st);
}

}  // namespace tree
}  // namespace kda
