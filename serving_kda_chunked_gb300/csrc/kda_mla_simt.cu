// kda_mla_simt.cu -- latent attention of fp32 tensors on the CUDA cores: the
// expanded form in tiles with a running maximum and sum, and the absorbed form.
// (tf32 tensor-core products keep 11 of the 24 bits.)
#include "kda_mla_split.cuh"

namespace kda {
namespace mla {
namespace {

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---- expanded form -------------------------------------------------------------
// One block per (64 queries of a sequence, head); 256 threads, each a 4 x 4
// piece of the 64 x 64 scores and a 4 x 8 piece of the 64 x 128 output.
constexpr int BQ = 64, BK = 64, LDT = BQ + 4;
constexpr int PRE_FLOATS = 2 * DQK * LDT + BK * DV + BK * LDT;

template <typename T>
__global__ void __launch_bounds__(256) prefill_simt_kernel(const PrefillArgs p) {
    extern __shared__ float smf[];
    float *Qt = smf;                       // [192][LDT], query fastest
    float *Kt = Qt + DQK * LDT;            // [192][LDT], key fastest
    float *Vs = Kt + DQK * LDT;            // [64][128]
    float *Pt = Vs + BK * DV;              // [64 keys][LDT], query fastest
    const int tid = threadIdx.x, h = blockIdx.y, H = p.H;
    // tile -> (sequence, first query): every sequence has ceil(nq / 64) tiles
    int tile = blockIdx.x, n = 0;
    SeqSpan s{0, 0, 0, 0};
    for (; n < p.N; ++n) {
        s = seq_span(p.cu_q, p.cu_k, n, p.Tq, p.Tk);
        const int tiles = (s.nq + BQ - 1) / BQ;
        if (tile < tiles) break;
        tile -= tiles;
    }
    if (n == p.N) return;
    const int i0 = tile * BQ;
    const T *q = (const T *)p.q, *kv = (const T *)p.kv, *kr = (const T *)p.k_r;
    for (int e = tid; e < BQ * (DQK / 4); e += 256) {
        const int r = e / (DQK / 4), c = e % (DQK / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + r < s.nq) x = load4(q + ((s.q0 + i0 + r) * H + h) * DQK + c);
        Qt[(c + 0) * LDT + r] = x.x; Qt[(c + 1) * LDT + r] = x.y;
        Qt[(c + 2) * LDT + r] = x.z; Qt[(c + 3) * LDT + r] = x.w;
    }
    const int tr = tid / 16, tc = tid % 16;          // rows 4 tr .., score columns 4 tc ..
    float m[4], l[4], acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -CUDART_INF_F; l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    }
    const int last = min(i0 + BQ, s.nq) - 1;         // keys seen by the tile's last query
    int64_t hi = p.causal ? (int64_t)last + s.nk - s.nq + 1 : s.nk;
    hi = hi < 0 ? 0 : (hi > s.nk ? s.nk : hi);
    for (int64_t j0 = 0; j0 < hi; j0 += BK) {
        __syncthreads();
        for (int e = tid; e < BK * (DQK / 4); e += 256) {
            const int r = e / (DQK / 4), c = e % (DQK / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + r < hi) {
                const int64_t t = s.k0 + j0 + r;
                x = c < NOPE ? load4(kv + (t * H + h) * (NOPE + DV) + c)
                             : load4(kr + t * ROPE + c - NOPE);
            }
            Kt[(c + 0) * LDT + r] = x.x; Kt[(c + 1) * LDT + r] = x.y;
            Kt[(c + 2) * LDT + r] = x.z; Kt[(c + 3) * LDT + r] = x.w;
        }
        for (int e = tid; e < BK * (DV / 4); e += 256) {
            const int r = e / (DV / 4), c = e % (DV / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + r < hi) x = load4(kv + ((s.k0 + j0 + r) * H + h) * (NOPE + DV) + NOPE + c);
            store4(Vs + r * DV + c, x);
        }
        __syncthreads();
        float sc[4][4] = {};
#pragma unroll 4
        for (int c = 0; c < DQK; ++c) {
            const float4 a = load4(Qt + c * LDT + 4 * tr), b = load4(Kt + c * LDT + 4 * tc);
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[i][j] += av[i] * bv[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t qi = i0 + 4 * tr + i;
            const int64_t end = p.causal ? qi + s.nk - s.nq + 1 : s.nk;   // keys it sees
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t kj = j0 + 4 * tc + j;
                sc[i][j] = kj < end && kj < s.nk ? sc[i][j] * p.scale : -CUDART_INF_F;
                top = fmaxf(top, sc[i][j]);
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            const float f = expf(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sc[i][j] = expf(sc[i][j] - ref);
                sum += sc[i][j];
                Pt[(4 * tc + j) * LDT + 4 * tr + i] = sc[i][j];
            }
            l[i] = l[i] * f + sum;                   // this thread's four columns
            m[i] = top;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] *= f;
        }
        __syncthreads();
#pragma unroll 4
        for (int j = 0; j < BK; ++j) {
            const float4 a = load4(Pt + j * LDT + 4 * tr);
            const float4 v0 = load4(Vs + j * DV + 4 * tc), v1 = load4(Vs + j * DV + 64 + 4 * tc);
            const float av[4] = {a.x, a.y, a.z, a.w};
            const float bv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[i][k] += av[i] * bv[k];
        }
    }
    T *o = (T *)p.o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sum = l[i];
#pragma unroll
        for (int of = 1; of < 16; of <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, of);
        const int qi = i0 + 4 * tr + i;
        if (qi >= s.nq) continue;
        const float r = sum > 0.f ? 1.f / sum : 0.f;
        const int64_t at = (s.q0 + qi) * H + h;
        store4(o + at * DV + 4 * tc, make_float4(acc[i][0] * r, acc[i][1] * r, acc[i][2] * r, acc[i][3] * r));
        store4(o + at * DV + 64 + 4 * tc, make_float4(acc[i][4] * r, acc[i][5] * r, acc[i][6] * r, acc[i][7] * r));
        if (p.lse && tc == 0) p.lse[at] = sum > 0.f ? m[i] + logf(sum) : -CUDART_INF_F;
    }
}

// ---- absorbed form --------------------------------------------------------------
// Shares and joins as in kda_mla_split.cuh, two CTAs per SM, groups of 8 heads,
// tiles of 32 tokens.  A tile's rows go to shared memory (padded, so that 32
// lanes read 32 rows without conflicts); a warp computes the scores of its 72
// of the 576 channels (lane = token) for all heads, one warp per head takes the
// softmax, and a thread owns 2 of the 512 output channels of all 8 heads.
// Shared-memory reads bound it: 12 wavefronts for 32 FMAs in the scores.
constexpr int HG = 8, TT = 32, LDR = ROW + 4, DTHREADS = 256;
constexpr int DEC_FLOATS = HG * ROW + TT * LDR + 8 * TT * HG + TT * HG + HG;
constexpr int DEC_CTAS = 320;                   // per launch, up to two per SM

__device__ __forceinline__ void copy16_or_zero(float *dst, const float *src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(copy ? 16 : 0) : "memory");
}

__global__ void __launch_bounds__(DTHREADS, 2) decode_simt_kernel(const SplitParams p, const float *q,
                                                                  const float *cache) {
    extern __shared__ __align__(16) float smf[];
    float *qs = smf;                        // [8][576]
    float *rows = qs + HG * ROW;            // [32][LDR]
    float *red = rows + TT * LDR;           // [8 warps][8 heads][32 tokens]
    float *ps = red + 8 * TT * HG;          // [32 tokens][8 heads]
    float *fs = ps + TT * HG;               // rescale factor per head
    __shared__ ShareScratch<DTHREADS> scratch;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h0 = blockIdx.x % p.groups * HG, nh = min(HG, p.H - h0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Share share = find_share<TT, DTHREADS, HG, float>(p, scratch);
    if (tid == 0) p.status[blockIdx.x] = 0;
    if (!share.busy) return;
    Walk<TT> w;
    w.start(p, share);
    const int shift = 31 - __clz(p.page);
    do {
        const int32_t *tab = p.table + (int64_t)w.b * p.max_pages;
        __syncthreads();
        for (int e = tid; e < HG * ROW / 4; e += DTHREADS) {
            const int r = e / (ROW / 4), c = e % (ROW / 4) * 4;
            store4(qs + r * ROW + c, r < nh ? load4(q + ((int64_t)w.b * p.H + h0 + r) * ROW + c)
                                            : make_float4(0.f, 0.f, 0.f, 0.f));
        }
        float m = -CUDART_INF_F, l = 0.f;   // of head `warp`, this lane's tokens
        float acc[HG][2] = {};
        for (int64_t i = w.lo; i < w.hi; ++i) {
            const int64_t t = i * TT;
            // lane = token: its row of the cache, or none
            int at = -1;
            if (t + lane < w.len) {
                const int pg = tab[(t + lane) >> shift];
                if (pg >= 0 && pg < p.n_pages) at = (pg << shift) + ((int)(t + lane) & (p.page - 1));
            }
            __syncthreads();                // the previous tile has been read
#pragma unroll
            for (int r = 0; r < TT / 8; ++r) {              // a warp copies rows warp, warp + 8, ...
                const int row = warp + 8 * r;
                const int src = __shfl_sync(0xffffffffu, at, row);
                for (int c = 4 * lane; c < ROW; c += 128)
                    copy16_or_zero(rows + row * LDR + c, cache + (src < 0 ? 0 : (int64_t)src * ROW + c), src >= 0);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            float sc[HG] = {};
#pragma unroll 6
            for (int c = warp * (ROW / 8); c < (warp + 1) * (ROW / 8); c += 4) {
                const float4 x = load4(rows + lane * LDR + c);
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float4 y = load4(qs + h * ROW + c);
                    sc[h] += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
                }
            }
#pragma unroll
            for (int h = 0; h < HG; ++h) red[(warp * HG + h) * TT + lane] = sc[h];
            __syncthreads();
            {                               // head `warp`, token `lane`
                float x = 0.f;
#pragma unroll
                for (int v = 0; v < 8; ++v) x += red[(v * HG + warp) * TT + lane];
                x = at >= 0 ? x * p.scale_log2 : -CUDART_INF_F;
                const float top = fmaxf(m, warp_max(x));
                const float ref = top == -CUDART_INF_F ? 0.f : top;
                const float f = exp2f(m - ref), e = exp2f(x - ref);
                l = l * f + e;
                m = top;
                ps[lane * HG + warp] = e;
                if (lane == 0) fs[warp] = f;
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < HG; ++h) { acc[h][0] *= fs[h]; acc[h][1] *= fs[h]; }
#pragma unroll 8
            for (int r = 0; r < TT; ++r) {
                const float2 v = *reinterpret_cast<const float2 *>(rows + r * LDR + 2 * tid);
                const float4 a = load4(ps + r * HG), c = load4(ps + r * HG + 4);
                const float e[HG] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                for (int h = 0; h < HG; ++h) { acc[h][0] += e[h] * v.x; acc[h][1] += e[h] * v.y; }
            }
        }
        // the segment's end
        l = warp_sum(l);
        const bool whole = w.whole();
        const int64_t slot = w.slot();
        if (lane == 0 && warp < nh) {
            if (whole) {
                if (p.lse)
                    p.lse[(int64_t)w.b * p.H + h0 + warp] =
                        l > 0.f ? (m + log2f(l)) * CUDART_LN2_F : -CUDART_INF_F;
            } else {
                *reinterpret_cast<float2 *>(p.stat + (slot * HG + warp) * 2) = make_float2(m, l);
            }
        }
        __syncthreads();                    // fs has been read
        if (lane == 0) fs[warp] = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < HG; ++h)
            if (h < nh) {
                float *to = whole ? (float *)p.o + ((int64_t)w.b * p.H + h0 + h) * LATENT
                                  : p.part + (slot * HG + h) * LATENT;
                *reinterpret_cast<float2 *>(to + 2 * tid) = make_float2(acc[h][0] * fs[h], acc[h][1] * fs[h]);
            }
    } while (w.next(p, share));
}

template <typename T>
cudaError_t run_prefill(const PrefillArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(prefill_simt_kernel<T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PRE_FLOATS * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.Tq + BQ - 1) / BQ + a.N;      // at most
    prefill_simt_kernel<T><<<dim3((unsigned)tiles, a.H), 256, PRE_FLOATS * sizeof(float), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

uint64_t decode_simt_workspace_bytes(int32_t H) { return ws_bytes(split_plan(H, HG, DEC_CTAS)); }

cudaError_t launch_prefill_simt(const PrefillArgs &a, cudaStream_t st) {
    return run_prefill<float>(a, st);
}

cudaError_t launch_decode_simt(const DecodeArgs &a, cudaStream_t st) {
    int nsm = 1;
    cudaError_t e = sm_count(&nsm);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 DEC_FLOATS * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    const SplitPlan pl = split_plan(a.H, HG, 2 * nsm < DEC_CTAS ? 2 * nsm : DEC_CTAS);
    SplitParams p;
    split_params(p, a, pl);
    return launch_split<HG, float>(decode_simt_kernel, p, pl, DTHREADS, DEC_FLOATS * sizeof(float), a.ws, st,
                                   (const float *)a.q, (const float *)a.cache);
}

}  // namespace mla
}  // namespace kda
