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

// Shared memory: rows k e^gamma and q e^gamma, after the product u and o; A and P;
// masks, betas, parents.
template <int D, int NT> struct Smem {       // NT: nodes, a multiple of 8
    static constexpr int LD = D + 16;        // two rows' quarter-warp reads meet different banks
    static constexpr uint32_t KG = 0, QG = NT * LD * 4, AP = 2 * QG, MASK = AP + NT * NT * 8, BETA = MASK + NT * 8,
                              PAR = BETA + NT * 4, BYTES = PAR + NT * 4;
};

template <int D, int NT, typename Tin>
__global__ void __launch_bounds__(D) step_kernel(const StepArgs p) {
    using L = Smem<D, NT>;
    constexpr int LD = L::LD, WARPS = D / 32, C = D / 32;
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
    Tin *o = (Tin *)p.o + at0;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) {
            for (int r = 0; r < T; ++r) o[r * step + tid] = from_f32<Tin>(0.f);
            return;
        }
    }
    const float *S = p.S + (slot * p.H + h) * (D * D);
    // the state starts on its way to L2 while the gates and pairs are worked out
    for (int i = tid; i < D * D * 4 / 128; i += D) asm volatile("prefetch.global.L2 [%0];" :: "l"((const char *)S + 128 * i));

    if (tid < T) {
        par[tid] = p.parents[(int64_t)b * T + tid];
        beta[tid] = p.beta[bt0 + (int64_t)tid * p.H];
    }
    __syncthreads();
    if (tid < NT) mask[tid] = tid < T ? ancestors(par, tid) : 0;
    __syncthreads();
    // A warp a node: up its path, nearest ancestor first, with the gates between them
    // summed on the way (differences of sums from the root would cancel); what the sum
    // is at the end fades the rows that meet the state.
    for (int r = warp; r < NT; r += WARPS) {
        uint64_t m = mask[r];
        Row<D> kr = {}, qr = {}, run = {};
        if (m) {
            kr = load_row<D>(k + r * step, lane);
            qr = load_row<D>(q + r * step, lane);
        }
        const float br = m ? beta[r] : 0.f;
        const bool on = m != 0;
        while (m) {
            const int i = 63 - __clzll((long long)m);
            m ^= 1ull << i;
            const Row<D> ki = load_row<D>(k + i * step, lane);
            Row<D> gi;
            if (p.scalar_gate) {
                const float x = p.g[bt0 + (int64_t)i * p.H];
#pragma unroll
                for (int c = 0; c < C; ++c) gi.x[c] = x;
            } else {
                gi = load_row<D>(p.g + at0 + i * step, lane);
            }
            float a = 0.f, z = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float w = ki.x[c] * ex2(run.x[c]);
                a += kr.x[c] * w;
                z += qr.x[c] * w;
                run.x[c] += gi.x[c] * 1.4426950408889634f;
            }
            // the half-warps finish one sum each
            const float give = lane < 16 ? z : a, have = lane < 16 ? a : z;
            float sum = have + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            if ((lane & 15) == 0) reinterpret_cast<float *>(ap + r * NT + i)[lane >> 4] = lane < 16 ? br * sum : sum;
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

    const int gq = lane >> 2, c4 = lane & 3;
    const float *Sw = S + 32 * warp + 4 * gq;            // this thread's 4 columns
    // u and o of node r, 4 or 8 columns from n on; zeros for padding
    auto put = [&](int r, int n, const float *w, const float *z, int count) {
        const bool on = r < T && mask[r] != 0;
        for (int x = 0; x < count; x += 4) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on) {
                const float4 vv = load4(v + r * step + n + x);
                const float br = beta[r];
                y = make_float4(br * (vv.x - w[x]), br * (vv.y - w[x + 1]), br * (vv.z - w[x + 2]), br * (vv.w - w[x + 3]));
            }
            store4(kg + r * LD + n + x, y);
            store4(qg + r * LD + n + x, on ? make_float4(z[x], z[x + 1], z[x + 2], z[x + 3]) : make_float4(0.f, 0.f, 0.f, 0.f));
        }
    };
    if constexpr (TC) {
        // K step (s, t): MMA column c4 is channel 16 s + 4 c4 + 2 t, column c4 + 4 the next
        // one; column group j's MMA column gq is S's column 4 gq + j of the warp's 32.
        constexpr int MT = NT / 8;
        float acc[MT][4][4] = {};
#pragma unroll 2
        for (int s = 0; s < D / 16; ++s) {
            float4 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __ldcs(reinterpret_cast<const float4 *>(Sw + (16 * s + 4 * c4 + j) * D));
            float f[4][4];                               // [channel][column]
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j][0] = to_tf32(y[j].x); f[j][1] = to_tf32(y[j].y); f[j][2] = to_tf32(y[j].z); f[j][3] = to_tf32(y[j].w);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float4 a = load4(kg + (8 * mt + gq) * LD + 16 * s + 4 * c4);
                const float4 c = load4(qg + (8 * mt + gq) * LD + 16 * s + 4 * c4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_tf32(acc[mt][j], a.x, c.x, a.y, c.y, f[0][j], f[1][j]);
                    mma_tf32(acc[mt][j], a.z, c.z, a.w, c.w, f[2][j], f[3][j]);
                }
            }
        }
        __syncthreads();
        // row gq of a tile: columns 8 c4 + j (from register 0 of group j) and 8 c4 + 4 + j
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float w[8], z[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = acc[mt][j][0]; w[4 + j] = acc[mt][j][1];
                z[j] = acc[mt][j][2]; z[4 + j] = acc[mt][j][3];
            }
            put(8 * mt + gq, 32 * warp + 8 * c4, w, z, 8);
        }
    } else {
        // 4 nodes at a time; the four lanes of a column hold every fourth group of 4 channels
        float4 keep[NT / 4][2];                          // node 4 t + c4: w, z
#pragma unroll
        for (int t = 0; t < NT / 4; ++t) {
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
                for (int x = 0; x < 4; ++x) {
                    w[n][x] += __shfl_xor_sync(0xffffffffu, w[n][x], 1);
                    w[n][x] += __shfl_xor_sync(0xffffffffu, w[n][x], 2);
                    z[n][x] += __shfl_xor_sync(0xffffffffu, z[n][x], 1);
                    z[n][x] += __shfl_xor_sync(0xffffffffu, z[n][x], 2);
                }
                if (n == c4) {
                    keep[t][0] = make_float4(w[n][0], w[n][1], w[n][2], w[n][3]);
                    keep[t][1] = make_float4(z[n][0], z[n][1], z[n][2], z[n][3]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT / 4; ++t) {
            if (4 * t >= T) break;
            const float w[4] = {keep[t][0].x, keep[t][0].y, keep[t][0].z, keep[t][0].w};
            const float z[4] = {keep[t][1].x, keep[t][1].y, keep[t][1].z, keep[t][1].w};
            put(4 * t + c4, 32 * warp + 4 * gq, w, z, 4);
        }
    }
    __syncthreads();
    // the deltas, parents first; thread = column
    for (int r = 0; r < T; ++r) {
        uint64_t m = mask[r];
        float u = kg[r * LD + tid], z = qg[r * LD + tid];
        if (m) {
            m &= ~(1ull << r);
            while (m) {
                const int i = __ffsll((long long)m) - 1;
                m &= m - 1;
                const float2 x = ap[r * NT + i];
                const float ui = kg[i * LD + tid];
                u -= x.x * ui;
                z += x.y * ui;
            }
            z += ap[r * NT + r].y * u;
            kg[r * LD + tid] = u;
        }
        o[r * step + tid] = from_f32<Tin>(z);
    }
}

template <int D, int NT, typename Tin>
cudaError_t run(const StepArgs &a, cudaStream_t st) {
    constexpr uint32_t bytes = Smem<D, NT>::BYTES;
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(step_kernel<D, NT, Tin>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.H));
    cfg.blockDim = dim3(D);
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
