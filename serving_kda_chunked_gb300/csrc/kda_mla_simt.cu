// kda_mla_simt.cu -- latent attention of fp32 tensors on the CUDA cores: the
// expanded form in tiles with a running maximum and sum, and the absorbed form.
// (A tf32 tensor-core product keeps 11 of the 24 bits.  Three products of operands
// split in two would keep nearly all; that has not been built.)
#include "kda_mla_split.cuh"
#include "kda_tree.cuh"

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
// One block per (32 queries of a sequence, head, part of their keys), four warps.
// A 16-byte shared-memory read of a warp costs four wavefronts, shared addresses
// or not, so a thread needs large pieces: in the scores a warp takes 48 of the
// 192 channels of the whole 32 x 32 tile (8 x 4 a thread: 128 FMAs for 12 reads)
// and the warps' sums are added in shared memory; in the output a warp takes 8
// of the tile's 32 keys for the whole 32 x 128 (8 x 16 a thread: 128 FMAs for 6
// reads), and the warps' outputs are added once, at the end.  Keys arrive with
// asynchronous copies one tile ahead, values while the scores are computed; two
// blocks an SM fill each other's gaps.  (With 4 x 4 and 2 x 4 pieces, shared
// memory held three prompts up to 777 tokens with four heads at 95 and 92 us.)
// The output's FMAs go two an instruction: 74 us in place of 78.  In the scores
// that takes 32 more sums or 4 more reads: 80 and 78 us.
// With few (queries, head) blocks the keys are cut into up to SPLITS parts,
// whose unnormalised results a second kernel joins.
constexpr int BQ = 32, BK = 32, LDQ = DQK + 4, LDP = BQ + 4, SPLITS = 8, PTHREADS = 128;
constexpr int PRE_FLOATS = (BQ + 2 * BK) * LDQ + BK * DV + BK * LDP + BQ;
// partial scores of a warp: element (row, key)
__device__ __forceinline__ int red_at(int w, int row, int key) {
    return w * (BQ * 36 + 32) + row * 36 + (row >> 3) * 8 + key;
}
static_assert(4 * (BQ * 36 + 32) <= BK * LDQ && 4 * BQ * DV <= (BQ + 2 * BK) * LDQ, "reused buffers");

__device__ __forceinline__ void copy16_or_zero(float *dst, const float *src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(copy ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

struct PreSplit { float *part, *stat; int parts; };     // [parts][Tq][H]: output (128), then maximum and sum

// What a block works on: sequence span, first query, keys of its part.  A warp
// looks at 32 sequences at a time.
struct PreUnit { SeqSpan s; int i0, j0, j1, parts; };
__device__ __forceinline__ bool pre_unit(const PrefillArgs &p, int tile, int part, int parts, PreUnit &u) {
    const int lane = threadIdx.x & 31;
    bool found = false;
    for (int n0 = 0; n0 < p.N && !found; n0 += 32) {     // every sequence has ceil(nq / 32) tiles
        SeqSpan s{0, 0, 0, 0};
        if (n0 + lane < p.N) s = seq_span(p.cu_q, p.cu_k, n0 + lane, p.Tq, p.Tk);
        const int64_t mine = (s.nq + BQ - 1) / BQ;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, tile < incl);
        if (in) {
            const int l = __ffs(in) - 1;
            u.s.q0 = __shfl_sync(0xffffffffu, s.q0, l);
            u.s.k0 = __shfl_sync(0xffffffffu, s.k0, l);
            u.s.nq = __shfl_sync(0xffffffffu, s.nq, l);
            u.s.nk = __shfl_sync(0xffffffffu, s.nk, l);
            tile -= (int)__shfl_sync(0xffffffffu, incl - mine, l);
            found = true;
        } else {
            tile -= (int)__shfl_sync(0xffffffffu, incl, 31);
        }
    }
    if (!found) return false;
    u.i0 = tile * BQ;
    const int last = min(u.i0 + BQ, u.s.nq) - 1;         // keys seen by the tile's last query
    const int64_t seen = p.causal ? (int64_t)last + u.s.nk - u.s.nq + 1 : u.s.nk;
    const int hi = seen < 0 ? 0 : (seen > u.s.nk ? u.s.nk : (int)seen);
    int len = ((hi + parts - 1) / parts + BK - 1) / BK * BK;
    len = max(len, 4 * BK);              // a part is worth four tiles at least
    u.parts = max(1, (hi + len - 1) / len);
    u.j0 = part * len;
    u.j1 = min(hi, u.j0 + len);
    return part < u.parts;
}

__global__ void __launch_bounds__(PTHREADS, 2) prefill_simt_kernel(const PrefillArgs p, const PreSplit sp) {
    extern __shared__ __align__(16) float smf[];
    float *Qs = smf;                       // [32][LDQ]
    float *Ks = Qs + BQ * LDQ;             // [2][32][LDQ]
    float *Vs = Ks + 2 * BK * LDQ;         // [32][128]
    float *Pt = Vs + BK * DV;              // [32 keys][LDP], query fastest
    float *fs = Pt + BK * LDP;             // [32] factors per query
    const int tid = threadIdx.x, h = blockIdx.y, H = p.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.ws && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        *static_cast<int32_t *>(p.ws) = 0;  // no wait here can give up: the call's status is clear
    PreUnit u;                             // long blocks first: the last queries see the most keys
    if (!pre_unit(p, gridDim.x - 1 - blockIdx.x, blockIdx.z, sp.parts, u)) return;
    const SeqSpan s = u.s;
    const float *q = (const float *)p.q, *kv = (const float *)p.kv, *kr = (const float *)p.k_r;
    auto load_keys = [&](int j, int buf) {
        float *K = Ks + buf * BK * LDQ;
        for (int e = tid; e < BK * (DQK / 4); e += PTHREADS) {
            const int r = e / (DQK / 4), c = e % (DQK / 4) * 4;
            const bool in = j + r < u.j1;
            const int64_t t = s.k0 + (in ? j + r : u.j0);
            copy16_or_zero(K + r * LDQ + c, c < NOPE ? kv + (t * H + h) * (NOPE + DV) + c : kr + t * ROPE + c - NOPE, in);
        }
        copy_commit();
    };
    auto load_values = [&](int j) {
        for (int e = tid; e < BK * (DV / 4); e += PTHREADS) {
            const int r = e / (DV / 4), c = e % (DV / 4) * 4;
            const bool in = j + r < u.j1;
            const int64_t t = s.k0 + (in ? j + r : u.j0);
            copy16_or_zero(Vs + r * DV + c, kv + (t * H + h) * (NOPE + DV) + NOPE + c, in);
        }
        copy_commit();
    };
    if (u.j0 < u.j1) {
        for (int e = tid; e < BQ * (DQK / 4); e += PTHREADS) {
            const int r = e / (DQK / 4), c = e % (DQK / 4) * 4;
            const bool in = u.i0 + r < s.nq;
            copy16_or_zero(Qs + r * LDQ + c, q + ((s.q0 + (in ? u.i0 + r : 0)) * H + h) * DQK + c, in);
        }
        load_keys(u.j0, 0);
        load_values(u.j0);
    }
    const int lane = tid & 31, warp = tid >> 5;
    const int lr = lane / 8, lc = lane % 8;          // rows 8 lr .., keys lc + 8 k or channels 32 g + 4 lc ..
    const int row = tid / 4, part = tid % 4;         // softmax: keys 8 part .. of a row
    const float sl = p.scale * 1.4426950408889634f;
    const int64_t qi = u.i0 + row;
    const int64_t end = p.causal ? qi + s.nk - s.nq + 1 : s.nk;           // keys the row sees
    alignas(16) float acc[8][16];
    float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
    int buf = 0;
    for (int j0 = u.j0; j0 < u.j1; j0 += BK, buf ^= 1) {
        if (j0 + BK < u.j1) load_keys(j0 + BK, buf ^ 1); else copy_commit();
        copy_wait<2>();                              // these keys (and the queries)
        __syncthreads();
        float *K = Ks + buf * BK * LDQ;
        float sc[8][4] = {};
#pragma unroll 2
        for (int c = warp * 48; c < warp * 48 + 48; c += 4) {
            float4 a[8], b[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = load4(Qs + (8 * lr + i) * LDQ + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = load4(K + (lc + 8 * k) * LDQ + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sc[i][k] += a[i].x * b[k].x;
                    sc[i][k] += a[i].y * b[k].y;
                    sc[i][k] += a[i].z * b[k].z;
                    sc[i][k] += a[i].w * b[k].w;
                }
        }
        __syncthreads();                             // these keys have been read: their place takes the sums
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) K[red_at(warp, 8 * lr + i, lc + 8 * k)] = sc[i][k];
        __syncthreads();
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            float4 y = load4(K + red_at(0, row, 8 * part + e));
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const float4 z = load4(K + red_at(w, row, 8 * part + e));
                y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
            }
            x[e] = y.x; x[e + 1] = y.y; x[e + 2] = y.z; x[e + 3] = y.w;
        }
        float top = -CUDART_INF_F;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int kj = j0 + 8 * part + e;
            x[e] = kj < end && kj < u.j1 ? x[e] * sl : -CUDART_INF_F;
            top = fmaxf(top, x[e]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // raised only by more than 2^8, so that the outputs are rarely rescaled
        const bool raise = top > m + 8.f;
        const float to = raise ? top : m, ref = to == -CUDART_INF_F ? 0.f : to;
        const float f = raise ? exp2f(m - ref) : 1.f;
        m = to;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float w = exp2f(x[e] - ref);
            sum += w;
            Pt[(8 * part + e) * LDP + row] = w;
        }
        l = l * f + sum;                             // this thread's eight keys
        if (part == 0) fs[row] = f;
        copy_wait<1>();                              // these values
        if (__syncthreads_or(raise)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float g = fs[8 * lr + i];
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[i][k] *= g;
            }
        }
#pragma unroll 2
        for (int k = warp * 8; k < warp * 8 + 8; ++k) {
            const float4 a0 = load4(Pt + k * LDP + 8 * lr), a1 = load4(Pt + k * LDP + 8 * lr + 4);
            const float w[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            float4 v[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) v[g] = load4(Vs + k * DV + 32 * g + 4 * lc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 ww = make_float2(w[i], w[i]);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float2 &lo = *reinterpret_cast<float2 *>(&acc[i][4 * g]), &hi = *reinterpret_cast<float2 *>(&acc[i][4 * g + 2]);
                    lo = fma2(ww, make_float2(v[g].x, v[g].y), lo);
                    hi = fma2(ww, make_float2(v[g].z, v[g].w), hi);
                }
            }
        }
        __syncthreads();
        if (j0 + BK < u.j1) load_values(j0 + BK); else copy_commit();
    }
    copy_wait<0>();
    __syncthreads();
    // the four warps' outputs, over the queries and keys
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            store4(smf + (warp * BQ + 8 * lr + i) * DV + 32 * g + 4 * lc,
                   make_float4(acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]));
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const bool whole = u.parts == 1;
    const int64_t at = (s.q0 + qi) * H + h, to = whole ? at : (int64_t)blockIdx.z * p.Tq * H + at;
    if (part == 0 && qi < s.nq) {
        if (!whole) *reinterpret_cast<float2 *>(sp.stat + 2 * to) = make_float2(m, l);
        else if (p.lse) p.lse[at] = lse_of(m, l);
    }
    if (part == 0) fs[row] = whole ? inverse_of(l) : 1.f;
    __syncthreads();
    for (int e = tid; e < BQ * DV / 4; e += PTHREADS) {
        const int r = e / (DV / 4), c = e % (DV / 4) * 4;
        if (u.i0 + r >= s.nq) break;                 // rows ascend
        float4 y = load4(smf + r * DV + c);
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 z = load4(smf + (w * BQ + r) * DV + c);
            y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        }
        const float g = fs[r];
        const int64_t out = (whole ? 0 : (int64_t)blockIdx.z * p.Tq * H) + (s.q0 + u.i0 + r) * H + h;
        store4((whole ? (float *)p.o : sp.part) + out * DV + c, make_float4(y.x * g, y.y * g, y.z * g, y.w * g));
    }
}

// Joins the parts of (32 queries, head); a warp takes a query, a lane 4 channels.
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillArgs p, const PreSplit sp) {
    const int lane = threadIdx.x & 31, r = blockIdx.z * 8 + (threadIdx.x >> 5), h = blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    PreUnit u;
    if (!pre_unit(p, blockIdx.x, 0, sp.parts, u) || u.parts == 1 || u.i0 + r >= u.s.nq) return;
    const int64_t at = (u.s.q0 + u.i0 + r) * p.H + h, step = p.Tq * p.H;
    float2 st[SPLITS];
    float4 y[SPLITS];
    float top = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < SPLITS; ++k)
        if (k < u.parts) {
            st[k] = *reinterpret_cast<const float2 *>(sp.stat + 2 * (k * step + at));
            y[k] = load4(sp.part + (k * step + at) * DV + 4 * lane);
        }
#pragma unroll
    for (int k = 0; k < SPLITS; ++k)
        if (k < u.parts) top = fmaxf(top, st[k].x);
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < SPLITS; ++k)
        if (k < u.parts) {
            const float f = exp2f(st[k].x - ref);
            sum += f * st[k].y;
            acc.x += f * y[k].x; acc.y += f * y[k].y; acc.z += f * y[k].z; acc.w += f * y[k].w;
        }
    const float f = inverse_of(sum);
    store4((float *)p.o + at * DV + 4 * lane, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
    if (p.lse && lane == 0) p.lse[at] = lse_of(top, sum);
}

// Parts per (queries, head) block: enough for about eight blocks an SM.
int prefill_parts(int32_t N, int64_t Tq, int32_t H) {
    const int64_t blocks = (Tq / BQ + N) * H, want = (1216 + blocks - 1) / blocks;
    return (int)(want < 1 ? 1 : (want > SPLITS ? SPLITS : want));
}

// ---- absorbed form --------------------------------------------------------------
// Shares and joins as in kda_mla_split.cuh, two CTAs per SM, groups of 8 heads,
// tiles of 32 tokens.  A tile's rows go to shared memory (padded, so that the
// lanes' reads meet different banks); a warp computes the scores of its 72 of the
// 576 channels for all tokens and heads, one warp per head takes the softmax, and
// a thread owns 4 of the 512 output channels of all 8 heads, for half the tokens.
// Shared-memory reads bound it: 3840 wavefronts a tile, with copies and sums 5100,
// for 1700 cycles of FMAs (16 sequences of 8000 tokens, 8 heads: 89 us, 97 with
// one FMA an instruction in the output; HBM would take 44).
constexpr int HG = 8, TT = 32, LDR = ROW + 4, LDS = TT + 4, DTHREADS = 256;
constexpr int DEC_FLOATS = HG * LDR + TT * LDR + 8 * HG * LDS + TT * HG + HG;
constexpr int OVER = 1;                         // tiles' time to begin and end a sequence
constexpr int DEC_CTAS = 320;                   // per launch, up to two per SM

// TREE: see kda_mla_decode.cu.
template <bool TREE>
__global__ void __launch_bounds__(DTHREADS, 2) decode_simt_kernel(const SplitParams p, const float *q,
                                                                  const float *cache) {
    extern __shared__ __align__(16) float smf[];
    float *qs = smf;                        // [8][LDR]
    float *rows = qs + HG * LDR;            // [32][LDR]
    float *red = rows + TT * LDR;           // [8 warps][8 heads][LDS]
    float *ps = red + 8 * HG * LDS;         // [32 tokens][8 heads]
    float *fs = ps + TT * HG;               // rescale factor per head
    __shared__ ShareScratch<DTHREADS> scratch;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Share share = find_share<TT, OVER, DTHREADS, HG, float, TREE>(p, scratch, nullptr);
    if (tid == 0) p.status[blockIdx.x] = 0;
    if (!share.busy) return;
    Walk<TT, OVER, HG, TREE> w;
    w.start(p, share);
    const int shift = 31 - __clz(p.page);
    do {
        const Item it = share.item<TREE, HG>(w.b);
        const int h0 = it.h0, nh = min(HG, p.H - h0);
        const int32_t *tab = p.table + (int64_t)it.b * p.max_pages;
        __syncthreads();
        for (int e = tid; e < HG * ROW / 4; e += DTHREADS) {
            const int r = e / (ROW / 4), c = e % (ROW / 4) * 4;
            store4(qs + r * LDR + c, r < nh ? load4(q + ((int64_t)it.b * p.H + h0 + r) * ROW + c)
                                            : make_float4(0.f, 0.f, 0.f, 0.f));
        }
        float m = -CUDART_INF_F, l = 0.f;   // of head `warp`, this lane's tokens
        const int32_t *par = TREE ? p.parents + (int64_t)it.b * p.T : nullptr;
        const int64_t front = TREE ? seq_len(p, it.b) : 0;
        const int node = TREE ? (h0 + warp) / p.heads : 0;
        const uint64_t sees = TREE && node < p.T ? tree::ancestors(par, node) : 0;
        float2 acc[HG][2] = {};             // channels 4 (tid % 128) .., tokens of half tid / 128
        const int ch = 4 * (tid & 127), half = tid >> 7;
        for (int64_t i = w.lo; i < w.hi; ++i) {
            const int64_t t = i * TT;
            // lane = token: its row of the cache, or none
            int at = -1;
            if (t + lane < w.len) {
                const int pg = tab[(t + lane) >> shift];
                if (pg >= 0 && pg < p.n_pages) at = (pg << shift) + ((int)(t + lane) & (p.page - 1));
            }
            bool see = !TREE || sees;
            if constexpr (TREE) {
                const int64_t d = t + lane - front;
                if (d >= 0) {               // a row that no node has is left out, and zero
                    if (d >= p.T || !tree::ancestors(par, (int)d)) at = -1;
                    see = d < p.T && (sees >> d & 1);
                }
            }
            see = see && at >= 0;
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
            // A lane takes 4 tokens x 4 heads of half the warp's channels: 8 reads
            // of 16 bytes for 64 products (a token and 8 heads a lane: 9 for 32,
            // and shared memory bounds it: 16 sequences of up to 2000 tokens, 8
            // heads, 24 us in place of 23; of 8000 tokens, 109 and 105).
            const int tg = lane >> 2, hg = lane >> 1 & 1, cs = lane & 1;
            float sc[4][4] = {};
#pragma unroll 3
            for (int g = 0; g < ROW / 64; ++g) {
                const int c = ((warp * (ROW / 64) + g) * 2 + cs) * 4;
                float4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = load4(rows + (4 * tg + i) * LDR + c);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float4 y = load4(qs + (4 * hg + h) * LDR + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[i][h] += x[i].x * y.x + x[i].y * y.y + x[i].z * y.z + x[i].w * y.w;
                }
            }
            // the lanes of the two halves of the channels keep two heads each
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float give = cs ? sc[i][h] : sc[i][h + 2], have = cs ? sc[i][h + 2] : sc[i][h];
                    z[i] = have + __shfl_xor_sync(0xffffffffu, give, 1);
                }
                store4(red + (warp * HG + 4 * hg + 2 * cs + h) * LDS + 4 * tg, make_float4(z[0], z[1], z[2], z[3]));
            }
            __syncthreads();
            {                               // head `warp`, token `lane`
                float x = 0.f;
#pragma unroll
                for (int v = 0; v < 8; ++v) x += red[(v * HG + warp) * LDS + lane];
                x = see ? x * p.scale_log2 : -CUDART_INF_F;
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
            for (int h = 0; h < HG; ++h) {
                const float f = fs[h];
                acc[h][0].x *= f; acc[h][0].y *= f; acc[h][1].x *= f; acc[h][1].y *= f;
            }
#pragma unroll 4
            for (int r = half * (TT / 2); r < (half + 1) * (TT / 2); ++r) {
                const float4 v = load4(rows + r * LDR + ch);
                const float4 a = load4(ps + r * HG), c = load4(ps + r * HG + 4);
                const float e[HG] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float2 ee = make_float2(e[h], e[h]);
                    acc[h][0] = fma2(ee, make_float2(v.x, v.y), acc[h][0]);
                    acc[h][1] = fma2(ee, make_float2(v.z, v.w), acc[h][1]);
                }
            }
        }
        // the segment's end
        l = warp_sum(l);
        const bool whole = w.whole();
        const int64_t slot = w.slot();
        if (lane == 0 && warp < nh) {
            if (whole) {
                if (p.lse) p.lse[(int64_t)it.b * p.H + h0 + warp] = lse_of(m, l);
            } else {
                *reinterpret_cast<float2 *>(p.stat + (slot * HG + warp) * 2) = make_float2(m, l);
            }
        }
        __syncthreads();                    // fs and the rows have been read
        if (lane == 0) fs[warp] = whole ? inverse_of(l) : 1.f;
        // the halves of the tokens: each thread gives the other one four heads
#pragma unroll
        for (int h = 0; h < HG; ++h)
            if (h / 4 != half) store4(rows + h * LDR + ch, make_float4(acc[h][0].x, acc[h][0].y, acc[h][1].x, acc[h][1].y));
        __syncthreads();
#pragma unroll
        for (int h = 0; h < HG; ++h)
            if (h / 4 == half && h < nh) {
                float *to = whole ? (float *)p.o + ((int64_t)it.b * p.H + h0 + h) * LATENT
                                  : p.part + (slot * HG + h) * LATENT;
                const float4 x = load4(rows + h * LDR + ch);
                const float f = fs[h];
                store4(to + ch, make_float4((acc[h][0].x + x.x) * f, (acc[h][0].y + x.y) * f,
                                            (acc[h][1].x + x.z) * f, (acc[h][1].y + x.w) * f));
            }
    } while (w.next(p, share));
}

}  // namespace

uint64_t decode_simt_workspace_bytes(int32_t H, bool tree) { return ws_bytes(split_plan(H, HG, DEC_CTAS, tree)); }

uint64_t prefill_simt_workspace_bytes(int32_t N, int64_t Tq, int32_t H) {
    const int parts = prefill_parts(N, Tq, H);
    return parts == 1 ? 0 : 256 + (uint64_t)parts * Tq * H * (DV + 2) * sizeof(float);
}

cudaError_t launch_prefill_simt(const PrefillArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(prefill_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PRE_FLOATS * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    PreSplit sp;
    sp.parts = prefill_parts(a.N, a.Tq, a.H);
    sp.part = reinterpret_cast<float *>((uint8_t *)a.ws + 256);
    sp.stat = sp.part + (int64_t)sp.parts * a.Tq * a.H * DV;
    const unsigned tiles = (unsigned)(a.Tq / BQ + a.N);     // at most
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, a.H, sp.parts);
    cfg.blockDim = dim3(PTHREADS);
    cfg.dynamicSmemBytes = PRE_FLOATS * sizeof(float);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, prefill_simt_kernel, a, sp);
    if (e != cudaSuccess || sp.parts == 1) return e;
    cfg.gridDim = dim3(tiles, a.H, BQ / 8);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, prefill_join_kernel, a, sp);
}

cudaError_t launch_decode_simt(const DecodeArgs &a, cudaStream_t st) {
    int nsm = 1;
    cudaError_t e = sm_count(&nsm);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(a.parents ? decode_simt_kernel<true> : decode_simt_kernel<false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, DEC_FLOATS * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    const SplitPlan pl = split_plan(a.H, HG, 2 * nsm < DEC_CTAS ? 2 * nsm : DEC_CTAS, a.parents != nullptr);
    SplitParams p;
    split_params(p, a, pl);
    return launch_split<HG, float>(a.parents ? decode_simt_kernel<true> : decode_simt_kernel<false>, p, pl, DTHREADS, DEC_FLOATS * sizeof(float), a.ws, st,
                                   (const float *)a.q, (const float *)a.cache);
}

}  // namespace mla
}  // namespace kda
