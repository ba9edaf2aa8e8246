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
// read once and not written; siblings share what is above them.  No exponent is
// above 0, however strong the gates are.
//
// What bounds it: S is 64 KB a head (D = 128) and is read once, HBM.  One CTA of
// D threads per (sequence, head); a warp owns 32 of S's columns.  bf16 inputs:
// the product runs as m16n8k8 tf32 MMAs whose 16 rows are 8 nodes' k and q rows
// (S and the rows are rounded to 11 bits there, as the prefill's fp16 operands are;
// sums are float32, and the committed state never passes through it).  The MMA's
// columns and K steps are permuted so that a thread's S fragments are 16-byte
// loads straight from global memory.  With T <= 16 that is 16 or 32 rows: too few
// for a 128-row tcgen05.mma, which would want S in shared memory first.  float32
// inputs: the same loads, FMAs.
#include "kda_tree.cuh"

namespace kda {
namespace tree {
namespace {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float to_tf32(float x) {
    uint32_t y;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
    return __uint_as_float(y);
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)),
                   "r"(__float_as_uint(a3)), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }

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

// Up to 16 nodes: their rows come to shared memory, all at once.  More: from global memory
// where they are used (two CTAs an SM would not fit beside them).
template <int NT> constexpr bool STAGED = NT <= 16;

// Shared memory: rows k e^gamma and q e^gamma, in their place after the product the
// deltas (and fp32's outputs); A and P; masks, betas, parents.
template <int D, int NT> struct Smem {       // NT: nodes, a multiple of 8
    static constexpr int LD = D + 16;        // two rows' quarter-warp reads meet different banks
    static constexpr int LDU = D + 8;        // the deltas' rows: four rows' reads do
    static constexpr int LDP = NT + 4;       // pairs of node r: ap[r * LDP + i]
    static constexpr uint32_t KG = 0, QG = NT * LD * 4, AP = 2 * QG, MASK = AP + NT * LDP * 8, BETA = MASK + NT * 8,
                              PAR = BETA + NT * 4, ROWS = PAR + NT * 4;
    // staged: q, k, v, then gates
    static constexpr uint32_t bytes(int e) { return ROWS + (STAGED<NT> ? NT * D * (3 * e + 4) : 0); }
};
// Warps a CTA: one for every 32 columns; from 32 nodes on two, which share the nodes.
template <int D, int NT> struct Warps { static constexpr int COLS = D / 32, SPLIT = NT >= 32 ? 2 : 1, ALL = COLS * SPLIT; };
// CTAs an SM that registers are shared out for (bf16, D = 128).
template <int D, int NT> constexpr int resident(bool tc) { return !tc || D != 128 ? 1 : (NT == 8 ? 6 : (NT == 16 ? 5 : (NT == 32 ? 3 : 2))); }

template <int D, int NT, typename Tin>
__global__ void
__launch_bounds__(32 * Warps<D, NT>::ALL, resident<D, NT>(sizeof(Tin) == 2)) step_kernel(const StepArgs p) {
    using L = Smem<D, NT>;
    constexpr int LD = L::LD, LDU = L::LDU, LDP = L::LDP, C = D / 32;
    constexpr int SPLIT = Warps<D, NT>::SPLIT, WARPS = Warps<D, NT>::ALL, THREADS = 32 * WARPS;
    constexpr bool TC = sizeof(Tin) == 2;
    extern __shared__ __align__(16) uint8_t sm[];
    float *kg = reinterpret_cast<float *>(sm + L::KG), *qg = reinterpret_cast<float *>(sm + L::QG);
    float2 *ap = reinterpret_cast<float2 *>(sm + L::AP);
    uint64_t *mask = reinterpret_cast<uint64_t *>(sm + L::MASK);
    float *beta = reinterpret_cast<float *>(sm + L::BETA);
    int32_t *par = reinterpret_cast<int32_t *>(sm + L::PAR);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, T = p.T;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t step = (int64_t)p.H * D;                              // between a head's nodes
    const int64_t at0 = (int64_t)b * T * step + (int64_t)h * D;         // of node 0
    const int64_t bt0 = (int64_t)b * T * p.H + h;
    const Tin *q = (const Tin *)p.q + at0, *k = (const Tin *)p.k + at0, *v = (const Tin *)p.v + at0;
    const float *g = p.scalar_gate ? p.g + bt0 : p.g + at0;
    int64_t in = step, gs = p.scalar_gate ? p.H : step;                 // between nodes of the inputs, of the gates
    Tin *o = (Tin *)p.o + at0;
    int64_t slot = b;
    if (tid < T) {
        par[tid] = p.parents[(int64_t)b * T + tid];
        beta[tid] = p.beta[bt0 + (int64_t)tid * p.H];
    }
    if constexpr (STAGED<NT>) {
        Tin *rows = reinterpret_cast<Tin *>(sm + L::ROWS);
        float *gates = reinterpret_cast<float *>(rows + 3 * NT * D);
        constexpr int EL = 16 / sizeof(Tin), CH = D / EL;               // values and pieces of 16 bytes
        for (int e = tid; e < T * CH; e += THREADS) {
            const int r = e / CH, c = e % CH * EL;
            copy16(rows + r * D + c, q + r * step + c);
            copy16(rows + (NT + r) * D + c, k + r * step + c);
            copy16(rows + (2 * NT + r) * D + c, v + r * step + c);
        }
        if (p.scalar_gate) {
            if (tid < T) gates[tid] = g[tid * gs];
            gs = 1;
        } else {
            for (int e = tid; e < T * (D / 4); e += THREADS) copy16(gates + 4 * e, g + e / (D / 4) * step + e % (D / 4) * 4);
            gs = D;
        }
        q = rows; k = rows + NT * D; v = rows + 2 * NT * D; g = gates;
        in = D;
    }
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) {
            for (int e = tid; e < T * D; e += THREADS) o[e / D * step + e % D] = from_f32<Tin>(0.f);
            if (STAGED<NT>) asm volatile("cp.async.wait_all;" ::: "memory");
            return;
        }
    }
    const float *S = p.S + (slot * p.H + h) * (D * D);
    // the state starts on its way to L2 while gates and pairs are worked out
    if (tid == 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(S), "r"(D * D * 4) : "memory");
    if constexpr (!STAGED<NT>) {                         // the values start on their way to L2
        constexpr int LINES = D * (int)sizeof(Tin) / 128;
        for (int i = tid; i < T * LINES; i += THREADS) prefetch_l2((const char *)(v + i / LINES * step) + i % LINES * 128);
    } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();
    if (tid < NT) mask[tid] = tid < T ? ancestors(par, tid) : 0;
    __syncthreads();
    // A warp a node: up its path, nearest ancestor first, with the gates between them
    // summed on the way (differences of sums from the root would cancel); what the sum
    // is at the end fades the rows that meet the state.  Four ancestors at a time, so that
    // their loads are under way together and the sums over the lanes share exchanges.
    for (int r = warp; r < NT; r += WARPS) {
        uint64_t m = mask[r];
        Row<D> kr = {}, qr = {}, run = {};
        if (m) {
            kr = load_row<D>(k + r * in, lane);
            qr = load_row<D>(q + r * in, lane);
        }
        const float br = m ? beta[r] : 0.f;
        const bool on = m != 0;
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
                    if (p.scalar_gate) {
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
                    run.x[c] += gi[u].x[c] * 1.4426950408889634f;
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
            if ((lane & 3) == 0 && i >= 0)
                reinterpret_cast<float *>(ap + r * LDP + i)[lane >> 2 & 1] = lane & 4 ? sum[0] : br * sum[0];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float f = on ? ex2(run.x[c]) : 0.f;
            const float a = kr.x[c] * f, z = qr.x[c] * f;
            kg[r * LD + C * lane + c] = TC ? to_tf32(a) : a;
            qg[r * LD + C * lane + c] = TC ? to_tf32(z) : z;
        }
    }
    __syncthreads();

    const int gq = lane >> 2, c4 = lane & 3, cols = 32 * (warp / SPLIT);
    const float *Sw = S + cols + 4 * gq;                 // this thread's 4 columns
    if constexpr (TC) {
        // o_r = (q_r e^gamma_r) S + sum_j M_rj d_j with d_j = beta_j (v_j - (k_j e^gamma_j) S) and
        // M (I + A) = P: along r's path M_rj = P_rj - sum_{i below j} M_ri A_ij, nearest first.
        // A warp a node, a lane the nodes `lane` and `lane + 32`.  M replaces P.
        for (int r = warp; r < NT; r += WARPS) {
            const uint64_t all = mask[r];
            float m0 = 0.f, m1 = 0.f;
            if (lane < NT && (all >> lane & 1)) m0 = ap[r * LDP + lane].y;
            if (NT > 32 && (all >> (lane + 32) & 1)) m1 = ap[r * LDP + lane + 32].y;
            uint64_t m = all;
            while (m) {
                const int i = 63 - __clzll((long long)m);
                m ^= 1ull << i;                          // what is left is above i on the path
                const float x = __shfl_sync(0xffffffffu, NT > 32 && i >= 32 ? m1 : m0, i & 31);
                if (lane < NT && (m >> lane & 1)) m0 -= x * ap[i * LDP + lane].x;
                if (NT > 32 && (m >> (lane + 32) & 1)) m1 -= x * ap[i * LDP + lane + 32].x;
            }
            if (lane < NT) ap[r * LDP + lane].y = to_tf32(m0);
            if (NT > 32) ap[r * LDP + lane + 32].y = to_tf32(m1);
        }
        // K step (s, t): MMA column c4 is channel 16 s + 4 c4 + 2 t, column c4 + 4 the next
        // one; column group j's MMA column gq is S's column 4 gq + j of the warp's 32.
        constexpr int MT = NT / 8 / SPLIT;
        const int part = warp % SPLIT;                   // this warp's tiles of 8 nodes: part, part + SPLIT, ...
        float acc[MT][4][4] = {};
#pragma unroll(MT > 2 ? 2 : 4)
        for (int s = 0; s < D / 16; ++s) {
            float4 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = load4(Sw + (16 * s + 4 * c4 + j) * D);
            float f[4][4];                               // [channel][column]
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j][0] = to_tf32(y[j].x); f[j][1] = to_tf32(y[j].y); f[j][2] = to_tf32(y[j].z); f[j][3] = to_tf32(y[j].w);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int row = 8 * (mt * SPLIT + part) + gq;
                const float4 a = load4(kg + row * LD + 16 * s + 4 * c4);
                const float4 c = load4(qg + row * LD + 16 * s + 4 * c4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_tf32(acc[mt][j], a.x, c.x, a.y, c.y, f[0][j], f[1][j]);
                    mma_tf32(acc[mt][j], a.z, c.z, a.w, c.w, f[2][j], f[3][j]);
                }
            }
        }
        // row gq of a tile: columns 8 c4 + j (from registers 0 and 2 of group j) and 8 c4 + 4 + j
        const int n0 = cols + 8 * c4;
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = 8 * (mt * SPLIT + part) + gq;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (mask[r]) {
                x = load4(v + r * in + n0);
                y = load4(v + r * in + n0 + 4);
                const float br = beta[r];
                x = make_float4(br * (x.x - acc[mt][0][0]), br * (x.y - acc[mt][1][0]), br * (x.z - acc[mt][2][0]), br * (x.w - acc[mt][3][0]));
                y = make_float4(br * (y.x - acc[mt][0][1]), br * (y.y - acc[mt][1][1]), br * (y.z - acc[mt][2][1]), br * (y.w - acc[mt][3][1]));
            }
            store4(kg + r * LDU + n0, make_float4(to_tf32(x.x), to_tf32(x.y), to_tf32(x.z), to_tf32(x.w)));
            store4(kg + r * LDU + n0 + 4, make_float4(to_tf32(y.x), to_tf32(y.y), to_tf32(y.z), to_tf32(y.w)));
        }
        __syncthreads();
        // M d on top of the q rows' products (registers 2 and 3); the k rows' are done with
#pragma unroll
        for (int ks = 0; ks < NT / 8; ++ks) {
            const float4 x = load4(kg + (8 * ks + c4) * LDU + cols + 4 * gq), y = load4(kg + (8 * ks + c4 + 4) * LDU + cols + 4 * gq);
            const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int tile = mt * SPLIT + part;
                if (mt * SPLIT + SPLIT - 1 < ks || tile < ks) continue;      // nodes see earlier ones only
                const float a1 = ap[(8 * tile + gq) * LDP + 8 * ks + c4].y, a3 = ap[(8 * tile + gq) * LDP + 8 * ks + c4 + 4].y;
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_tf32(acc[mt][j], 0.f, a1, 0.f, a3, xv[j], yv[j]);
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
    } else {
        // 4 nodes at a time; the four lanes of a column hold every fourth group of 4 channels
        constexpr int GROUPS = NT / 4 / SPLIT;
        float4 keep[GROUPS][2];                          // node 4 t + c4: products with k, with q
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) {
            const int t = x * SPLIT + warp % SPLIT;
            if (4 * t >= T) break;
            float w[4][4] = {}, z[4][4] = {};
#pragma unroll 2
            for (int s = 0; s < D / 16; ++s) {
                float4 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = load4(Sw + (16 * s + 4 * c4 + j) * D);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float4 a = load4(kg + (4 * t + n) * LD + 16 * s + 4 * c4);
                    const float4 c = load4(qg + (4 * t + n) * LD + 16 * s + 4 * c4);
                    const float av[4] = {a.x, a.y, a.z, a.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[n][0] += av[j] * y[j].x; w[n][1] += av[j] * y[j].y; w[n][2] += av[j] * y[j].z; w[n][3] += av[j] * y[j].w;
                        z[n][0] += cv[j] * y[j].x; z[n][1] += cv[j] * y[j].y; z[n][2] += cv[j] * y[j].z; z[n][3] += cv[j] * y[j].w;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[n][e] += __shfl_xor_sync(0xffffffffu, w[n][e], 1);
                    w[n][e] += __shfl_xor_sync(0xffffffffu, w[n][e], 2);
                    z[n][e] += __shfl_xor_sync(0xffffffffu, z[n][e], 1);
                    z[n][e] += __shfl_xor_sync(0xffffffffu, z[n][e], 2);
                }
                if (n == c4) {
                    keep[x][0] = make_float4(w[n][0], w[n][1], w[n][2], w[n][3]);
                    keep[x][1] = make_float4(z[n][0], z[n][1], z[n][2], z[n][3]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) {
            const int t = x * SPLIT + warp % SPLIT, r = 4 * t + c4, n = cols + 4 * gq;
            if (4 * t >= T) break;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
            if (mask[r]) {
                const float4 vv = load4(v + r * in + n), w = keep[x][0];
                const float br = beta[r];
                y = make_float4(br * (vv.x - w.x), br * (vv.y - w.y), br * (vv.z - w.z), br * (vv.w - w.w));
                z = keep[x][1];
            }
            store4(kg + r * LD + n, y);
            store4(qg + r * LD + n, z);
        }
        __syncthreads();
        // the deltas, parents first; thread = column
        if (tid < D)
            for (int r = 0; r < T; ++r) {
                uint64_t m = mask[r];
                float u = kg[r * LD + tid], z = qg[r * LD + tid];
                if (m) {
                    m &= ~(1ull << r);
                    while (m) {
                        const int i = __ffsll((long long)m) - 1;
                        m &= m - 1;
                        const float2 x = ap[r * LDP + i];
                        const float ui = kg[i * LD + tid];
                        u -= x.x * ui;
                        z += x.y * ui;
                    }
                    z += ap[r * LDP + r].y * u;
                    kg[r * LD + tid] = u;
                }
                o[r * step + tid] = from_f32<Tin>(z);
            }
    }
}

template <int D, int NT, typename Tin>
cudaError_t run(const StepArgs &a, cudaStream_t st) {
    constexpr uint32_t bytes = Smem<D, NT>::bytes(sizeof(Tin));
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(step_kernel<D, NT, Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, step_kernel<D, NT, Tin>, a);
}

template <int D, typename Tin>
cudaError_t by_nodes(const StepArgs &a, cudaStream_t st) {
    if (a.T <= 8) return run<D, 8, Tin>(a, st);
    if (a.T <= 16) return run<D, 16, Tin>(a, st);
    if (a.T <= 32) return run<D, 32, Tin>(a, st);
    return run<D, 64, Tin>(a, st);
}

}  // namespace

cudaError_t launch_step(const StepArgs &a, cudaStream_t st) {
    if (a.d == 128) return a.dtype == 0 ? by_nodes<128, __nv_bfloat16>(a, st) : by_nodes<128, float>(a, st);
    return a.dtype == 0 ? by_nodes<64, __nv_bfloat16>(a, st) : by_nodes<64, float>(a, st);
}

}  // namespace tree
}  // namespace kda
