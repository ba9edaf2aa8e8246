// kda_mla_simt.cu -- latent attention on the CUDA cores in fp32 arithmetic:
// the expanded form (flash-style tiles) and the absorbed form (tokens split
// over blocks, joined by a second kernel).
#include "kda_mla.cuh"

#include <math_constants.h>

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
// One block per (split of a sequence's tokens, group of 8 heads, sequence):
// tiles of 32 tokens in shared memory; a warp computes the scores of its 72 of
// the 576 channels (lane = token), one warp per head takes the softmax, and a
// thread owns 2 of the 512 output channels of all 8 heads.
constexpr int HG = 8, TT = 32, LDR = ROW + 4;
constexpr int DEC_FLOATS = HG * ROW + TT * LDR + 8 * TT * HG + TT * HG + 2 * HG;
constexpr int MAX_SPLITS = 64;

// [split][B][H]: unnormalised output (512), then maximum and sum
__host__ __device__ inline int64_t part_index(int split, int b, int h, int B, int H) {
    return ((int64_t)split * B + b) * H + h;
}

int decode_splits(int32_t B, int32_t H) {
    const int64_t units = (int64_t)B * ((H + HG - 1) / HG);
    const int64_t want = (4 * 152 + units - 1) / units;
    return (int)(want < 1 ? 1 : (want > MAX_SPLITS ? MAX_SPLITS : want));
}

template <typename T>
__global__ void __launch_bounds__(256) decode_simt_kernel(const DecodeArgs p, int splits,
                                                          float *part, float *stat) {
    extern __shared__ float smf[];
    float *qs = smf;                        // [8][576]
    float *rows = qs + HG * ROW;            // [32][LDR]
    float *red = rows + TT * LDR;           // [8 warps][8 heads][32 tokens]
    float *ps = red + 8 * TT * HG;          // [32 tokens][8 heads]
    float *fs = ps + TT * HG;               // rescale factor per head, then sums
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split = blockIdx.x, h0 = blockIdx.y * HG, b = blockIdx.z, H = p.H;
    const int nh = min(HG, H - h0);
    int64_t len = p.seq_lens[b];
    const int64_t cap = (int64_t)p.max_pages * p.page;
    len = len < 0 ? 0 : (len > cap ? cap : len);
    const int64_t tiles = (len + TT - 1) / TT;
    const int64_t t0 = tiles * split / splits * TT;
    const int64_t t1 = min(len, tiles * (split + 1) / splits * TT);
    const T *q = (const T *)p.q, *cache = (const T *)p.cache;
    for (int e = tid; e < HG * ROW / 4; e += 256) {
        const int r = e / (ROW / 4), c = e % (ROW / 4) * 4;
        store4(qs + r * ROW + c, r < nh ? load4(q + ((int64_t)b * H + h0 + r) * ROW + c)
                                        : make_float4(0.f, 0.f, 0.f, 0.f));
    }
    float m = -CUDART_INF_F, l = 0.f;       // of head `warp`
    float acc[HG][2] = {};
    for (int64_t t = t0; t < t1; t += TT) {
        __syncthreads();
        for (int e = tid; e < TT * (ROW / 4); e += 256) {
            const int r = e / (ROW / 4), c = e % (ROW / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t + r < t1) {
                const int pg = p.table[(int64_t)b * p.max_pages + (t + r) / p.page];
                if (pg >= 0 && pg < p.n_pages)
                    x = load4(cache + ((int64_t)pg * p.page + (t + r) % p.page) * ROW + c);
            }
            store4(rows + r * LDR + c, x);
        }
        __syncthreads();
        float sc[HG] = {};
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
        {                                   // head `warp`, token `lane`
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) x += red[(w * HG + warp) * TT + lane];
            bool seen = t + lane < t1;
            if (seen) {
                const int pg = p.table[(int64_t)b * p.max_pages + (t + lane) / p.page];
                seen = pg >= 0 && pg < p.n_pages;
            }
            x = seen ? x * p.scale : -CUDART_INF_F;
            const float top = fmaxf(m, warp_max(x));
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            const float f = expf(m - ref), e = expf(x - ref);
            l = l * f + e;                  // this lane's tokens
            m = top;
            ps[lane * HG + warp] = e;
            if (lane == 0) fs[warp] = f;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < HG; ++h) { acc[h][0] *= fs[h]; acc[h][1] *= fs[h]; }
#pragma unroll 4
        for (int r = 0; r < TT; ++r) {
            const float2 v = *reinterpret_cast<const float2 *>(rows + r * LDR + 2 * tid);
            const float4 a = load4(ps + r * HG), c = load4(ps + r * HG + 4);
            const float w[HG] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
            for (int h = 0; h < HG; ++h) { acc[h][0] += w[h] * v.x; acc[h][1] += w[h] * v.y; }
        }
    }
    l = warp_sum(l);
    if (lane == 0 && warp < nh) {
        const int64_t at = part_index(split, b, h0 + warp, p.B, H);
        stat[2 * at] = m;
        stat[2 * at + 1] = l;
    }
    for (int h = 0; h < nh; ++h)
        *reinterpret_cast<float2 *>(part + part_index(split, b, h0 + h, p.B, H) * LATENT + 2 * tid) =
            make_float2(acc[h][0], acc[h][1]);
}

// joins the splits of one (sequence, head); 128 threads, 4 channels each
template <typename T>
__global__ void __launch_bounds__(128) decode_join_kernel(const DecodeArgs p, int splits,
                                                          const float *part, const float *stat) {
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    float m = -CUDART_INF_F;
    for (int s = 0; s < splits; ++s) m = fmaxf(m, stat[2 * part_index(s, b, h, p.B, p.H)]);
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < splits; ++s) {
        const int64_t at = part_index(s, b, h, p.B, p.H);
        const float f = expf(stat[2 * at] - ref);
        const float4 x = load4(part + at * LATENT + 4 * tid);
        l += f * stat[2 * at + 1];
        acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
    }
    const float r = l > 0.f ? 1.f / l : 0.f;
    const int64_t at = (int64_t)b * p.H + h;
    store4((T *)p.o + at * LATENT + 4 * tid, make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r));
    if (p.lse && tid == 0) p.lse[at] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
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

template <typename T>
cudaError_t run_decode(const DecodeArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(decode_simt_kernel<T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         DEC_FLOATS * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    const int splits = decode_splits(a.B, a.H);
    float *part = reinterpret_cast<float *>((uint8_t *)a.ws + 256);
    float *stat = part + (int64_t)splits * a.B * a.H * LATENT;
    decode_simt_kernel<T><<<dim3(splits, (a.H + HG - 1) / HG, a.B), 256, DEC_FLOATS * sizeof(float), st>>>(
        a, splits, part, stat);
    decode_join_kernel<T><<<dim3(a.H, a.B), 128, 0, st>>>(a, splits, part, stat);
    return cudaGetLastError();
}

}  // namespace

uint64_t decode_simt_workspace_bytes(int32_t B, int32_t H) {
    return 256 + (uint64_t)decode_splits(B, H) * B * H * (LATENT + 2) * sizeof(float);
}

cudaError_t launch_prefill_simt(const PrefillArgs &a, cudaStream_t st) {
    return run_prefill<float>(a, st);
}

cudaError_t launch_decode_simt(const DecodeArgs &a, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(a.ws, 0, 256, st);
    if (e != cudaSuccess) return e;
    return run_decode<float>(a, st);
}

}  // namespace mla
}  // namespace kda
