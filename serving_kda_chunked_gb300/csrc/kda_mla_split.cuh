// kda_mla_split.cuh -- how the absorbed form shares out its tokens, and how
// partial results are joined; used by the tensor-core and the CUDA-core kernel.
//
// The tiles (of TOK tokens) of all sequences, laid end to end, are cut into
// equal contiguous shares, one per CTA, by arithmetic that every CTA repeats
// from the lengths.  A sequence that lies in one share is finished there; one
// that a boundary cuts leaves an unnormalised partial result per share, and
// join_kernel adds those up in order of the shares.  Heads come in groups of N;
// CTA x works for group x % groups on share x / groups, so that the CTAs that
// read the same tokens for different heads do so at about the same time.
#pragma once

#include "kda_mla.cuh"

#include <math_constants.h>

namespace kda {
namespace mla {

constexpr int FAIL_TIMEOUT = 4;      // status word of a wait that gave up

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What the CTA with share c of C starts in: sequence b, whose tiles are
// [t0, t1) of all T; b < 0 marks an idle CTA.
struct Meta { int64_t t0, t1, T; int32_t b, C; };

struct SplitParams {
    const int32_t *table, *seq_lens;
    void *o;
    float *lse;
    int32_t *status;           // one word per CTA
    Meta *meta;                // per CTA
    float *part, *stat;        // two slots per CTA: [N][512], and [N][2] (maximum in log2 units, sum)
    int32_t B, H, n_pages, page, max_pages, groups;
    float scale_log2;
};

__device__ __forceinline__ int64_t seq_len(const SplitParams &p, int b) {
    const int64_t cap = (int64_t)p.max_pages * p.page, n = p.seq_lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
}
template <int TOK> __device__ __forceinline__ int64_t tiles_of(int64_t len) { return (len + TOK - 1) / TOK; }
__device__ __forceinline__ int64_t share_start(int64_t T, int c, int C) { return T * c / C; }

// A CTA's share: tiles [g0, g1) of all, beginning in sequence b0 (whose first
// tile is t00).
struct Share { int64_t g0, g1, t00; int b0; bool busy; };
template <int THREADS> struct ShareScratch { int64_t sums[THREADS / 32], t0; int b; };

// Finds the share (all THREADS threads; ends with a barrier), records it for
// the join, and writes the outputs of sequences with nothing cached.
template <int TOK, int THREADS, int N, typename To>
__device__ __forceinline__ Share find_share(const SplitParams &p, ShareScratch<THREADS> &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x % p.groups, c = blockIdx.x / p.groups, C0 = gridDim.x / p.groups;
    const int h0 = group * N, nh = min(N, p.H - h0);
    const int per = (p.B + THREADS - 1) / THREADS;
    const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += tiles_of<TOK>(seq_len(p, b));
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh.sums[warp] = incl;
    if (tid == 0) sh.b = -1;
    __syncthreads();
    int64_t T = 0, excl = incl - mine;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) excl += sh.sums[w];
        T += sh.sums[w];
    }
    Share s;
    const int C = (int)(T < C0 ? T : C0);
    s.busy = c < C;
    s.g0 = s.busy ? share_start(T, c, C) : 0;
    s.g1 = s.busy ? share_start(T, c + 1, C) : 0;
    if (s.busy && excl <= s.g0 && s.g0 < excl + mine) {
        int64_t at = excl;
        int b = b_lo;
        for (; b < b_hi; ++b) {
            const int64_t n = tiles_of<TOK>(seq_len(p, b));
            if (s.g0 < at + n) {
                Meta m;
                m.t0 = at; m.t1 = at + n; m.T = T; m.b = b; m.C = C;
                p.meta[blockIdx.x] = m;
                sh.t0 = at;
                sh.b = b;
                break;
            }
            at += n;
        }
    }
    if (!s.busy && tid == 0) p.meta[blockIdx.x].b = -1;
    for (int b = c; b < p.B; b += C0) {
        if (seq_len(p, b) > 0) continue;
        const int64_t at = (int64_t)b * p.H + h0;
        for (int e = tid; e < nh * (LATENT / 4); e += THREADS)
            store4((To *)p.o + at * LATENT + 4 * e, make_float4(0.f, 0.f, 0.f, 0.f));
        if (p.lse && tid < nh) p.lse[at + tid] = -CUDART_INF_F;
    }
    __syncthreads();
    s.b0 = sh.b;
    s.t00 = sh.t0;
    s.busy = s.busy && s.b0 >= 0;              // false only if lengths changed under the kernel
    return s;
}

// The share as segments: sequence b, its tiles [lo, hi); `at` is the
// sequence's first tile of all.  Every warp walks them with the same arithmetic.
template <int TOK> struct Walk {
    int64_t at, len, lo, hi;
    int b;
    __device__ __forceinline__ void open(const SplitParams &p, const Share &s, int b_, int64_t at_, int64_t g) {
        len = seq_len(p, b_);
        b = b_; at = at_;
        lo = g - at;
        const int64_t n = tiles_of<TOK>(len);
        hi = s.g1 - at < n ? s.g1 - at : n;
    }
    __device__ __forceinline__ void start(const SplitParams &p, const Share &s) { open(p, s, s.b0, s.t00, s.g0); }
    __device__ __forceinline__ bool next(const SplitParams &p, const Share &s) {
        const int64_t to = at + tiles_of<TOK>(len);
        if (to >= s.g1) return false;
        int n = b + 1;
        while (n < p.B && seq_len(p, n) == 0) ++n;
        if (n >= p.B) return false;            // lengths changed under the kernel
        open(p, s, n, to, to);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == tiles_of<TOK>(len); }
    // partial-result slot of this segment: a sequence's first piece goes to its
    // share's second slot, every other piece to the first
    __device__ __forceinline__ int64_t slot() const { return 2 * (int64_t)blockIdx.x + (lo == 0 ? 1 : 0); }
};

// Adds up the partial results of the sequences that a share boundary cuts.
// Blocks (boundary, 0 .. N / 2 - 1) work for the sequence their boundary lies
// in; an item is 128 channels of a head.  Up to eight pieces: one warp an item,
// all pieces' rows loaded before the weights are known.  More (the sequence then
// has eight boundaries' blocks or more): one block an item, every eighth piece
// a warp.  Pieces are added in a fixed order.
template <int N, typename To>
__global__ void __launch_bounds__(256) join_kernel(const SplitParams p, int ctas, int32_t *header) {
    __shared__ float4 buf[8][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0) {              // the call's status, from the CTAs'
        int st = 0;
        for (int i = tid; i < ctas; i += 256) st |= p.status[i];
        st = __syncthreads_or(st);
        if (tid == 0) *header = st ? FAIL_TIMEOUT : 0;
    }
    const int cta = blockIdx.y + p.groups;                  // shares 1 .. of every group
    if (cta >= ctas) return;
    const int group = cta % p.groups, c = cta / p.groups;
    const Meta m = p.meta[cta];
    if (m.b < 0 || share_start(m.T, c, m.C) <= m.t0) return;
    const int first = (int)(((m.t0 + 1) * m.C + m.T - 1) / m.T);   // boundaries inside the sequence
    const int last = (int)((m.t1 * m.C + m.T - 1) / m.T) - 1;
    const int pieces = last - first + 2;                    // of shares first - 1 .. last
    const int nh = min(N, p.H - group * N);
    const int slot0 = 2 * ((first - 1) * p.groups + group); // of piece i: slot0 + 2 groups i, + 1 for the first
    auto slot_of = [&](int i) { return slot0 + 2 * p.groups * i + (i == 0); };
    const bool wide = pieces > 8;
    const int block = (c - first) * gridDim.x + blockIdx.x;
    const int item = wide ? block : (block * 8 + warp);
    const int h = item >> 2, ch = (item & 3) * 128 + 4 * lane;
    if (h >= nh) return;                                    // of a wide item: the whole block
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -CUDART_INF_F, sum = 0.f, ref;
    int bad = 0;                                            // a share that gave up: o stays as it is
    if (!wide) {
        float4 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < pieces) y[i] = load4(p.part + ((int64_t)slot_of(i) * N + h) * LATENT + ch);
        float2 s = make_float2(-CUDART_INF_F, 0.f);
        if (lane < pieces) {
            s = *reinterpret_cast<const float2 *>(p.stat + ((int64_t)slot_of(lane) * N + h) * 2);
            bad = p.status[slot_of(lane) >> 1];
        }
        top = s.x;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = __shfl_sync(0xffffffffu, top, 0);
        ref = top == -CUDART_INF_F ? 0.f : top;
        const float f = ex2(s.x - ref);
        sum = f * s.y;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum = __shfl_sync(0xffffffffu, sum, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < pieces) {
                const float g = __shfl_sync(0xffffffffu, f, i);
                acc.x += g * y[i].x; acc.y += g * y[i].y; acc.z += g * y[i].z; acc.w += g * y[i].w;
            }
    } else {
        for (int i = lane; i < pieces; i += 32) {
            top = fmaxf(top, p.stat[((int64_t)slot_of(i) * N + h) * 2]);
            bad |= p.status[slot_of(i) >> 1];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        ref = top == -CUDART_INF_F ? 0.f : top;
        for (int i = lane; i < pieces; i += 32) {
            const float2 s = *reinterpret_cast<const float2 *>(p.stat + ((int64_t)slot_of(i) * N + h) * 2);
            sum += ex2(s.x - ref) * s.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll 8
        for (int i = warp; i < pieces; i += 8) {
            const int64_t at = (int64_t)slot_of(i) * N + h;
            const float f = ex2(p.stat[at * 2] - ref);
            const float4 y = load4(p.part + at * LATENT + ch);
            acc.x += f * y.x; acc.y += f * y.y; acc.z += f * y.z; acc.w += f * y.w;
        }
        buf[warp][lane] = acc;
        __syncthreads();
        if (warp != 0) return;
        for (int i = 1; i < 8; ++i) {
            const float4 y = buf[i][lane];
            acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
        }
    }
    if (__any_sync(0xffffffffu, bad)) return;
    const float r = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t at = (int64_t)m.b * p.H + group * N + h;
    store4((To *)p.o + at * LATENT + ch, make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r));
    if (p.lse && (item & 3) == 0 && lane == 0)
        p.lse[at] = sum > 0.f ? (top + log2f(sum)) * CUDART_LN2_F : -CUDART_INF_F;
}

// workspace: header | status | meta | stat | part
struct SplitPlan { int N, groups, ctas; };
constexpr uint64_t WS_STATUS = 256;
inline uint64_t ws_meta(const SplitPlan &s) { return WS_STATUS + ((uint64_t)s.ctas * 4 + 255) / 256 * 256; }
inline uint64_t ws_stat(const SplitPlan &s) { return ws_meta(s) + ((uint64_t)s.ctas * sizeof(Meta) + 255) / 256 * 256; }
inline uint64_t ws_part(const SplitPlan &s) { return ws_stat(s) + (uint64_t)s.ctas * 2 * s.N * 8; }
inline uint64_t ws_bytes(const SplitPlan &s) { return ws_part(s) + (uint64_t)s.ctas * 2 * s.N * LATENT * 4; }

inline SplitPlan split_plan(int32_t H, int N, int ctas) {
    SplitPlan s;
    s.N = N;
    s.groups = (H + N - 1) / N;
    s.ctas = s.groups * (ctas / s.groups > 0 ? ctas / s.groups : 1);
    return s;
}

inline void split_params(SplitParams &p, const DecodeArgs &a, const SplitPlan &s) {
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.table = a.table; p.seq_lens = a.seq_lens;
    p.o = a.o; p.lse = a.lse;
    p.status = reinterpret_cast<int32_t *>(ws + WS_STATUS);
    p.meta = reinterpret_cast<Meta *>(ws + ws_meta(s));
    p.stat = reinterpret_cast<float *>(ws + ws_stat(s));
    p.part = reinterpret_cast<float *>(ws + ws_part(s));
    p.B = a.B; p.H = a.H; p.n_pages = a.n_pages; p.page = a.page; p.max_pages = a.max_pages;
    p.groups = s.groups;
    p.scale_log2 = a.scale * 1.4426950408889634f;
}

// Launches `kernel` with the call's shares, then the join, each as a programmatic
// dependent of what is before it on the stream.
template <int N, typename To, typename Params, typename... More>
cudaError_t launch_split(void (*kernel)(Params, More...), const Params &p, const SplitPlan &s, int threads,
                         uint32_t smem, void *ws, cudaStream_t st, More... more) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s.ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, more...);
    if (e != cudaSuccess) return e;
    const int joins = s.ctas - s.groups;
    cfg.gridDim = dim3(N / 2, (unsigned)(joins > 0 ? joins : 1));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<N, To>, (const SplitParams &)p, s.ctas,
                              static_cast<int32_t *>(ws));
}

}  // namespace mla
}  // namespace kda
