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
//
// Drafted trees (TREE): nothing is computed for groups of rows that are padding.  Where there are
// none, all is as above: the groups stay in step, and read a tile from L2 at the same time.
// Else sequences differ in groups, and every (sequence, group) is an item of its own in one list, in
// that order; what is said of sequences holds for items then, and groups of padding alone are
// items of length 0.  An item's tokens come from HBM, though, where L2 cannot hold them until
// the next group wants them: sequences with the same number of groups then have CTAs of their own, in
// step (alike_order).  32 heads, each way in us:
//   64 trees of 8 nodes over up to 8192 tokens, full: in step 192, items 223;
//     ragged: in step 201, items 162 (812 MB from HBM of 360), alike 151
//   128 and 256 ragged trees of 8, 560,000 tokens in all: items 279 and 273, alike 255 and 259
//   64 ragged trees of 8, 120,000 tokens: items 91, alike 90; 90,000: 77, 80; 66,000: 61, 64
//   64 and 256 ragged trees of 16 (8 groups): items 233 and 544, alike 238 and 580
//   8 trees of 48 over up to 32,768, full: in step 533, items 597; ragged: 530 and 457
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

// What a softmax's sum and maximum (in log2 units) give: the factor of the output, and
// the lse.  A sum of 0 says that nothing was seen; one that is NaN (NaN was seen, or a
// score overflowed) stays NaN in both.
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float lse_of(float top, float sum) {
    return sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * CUDART_LN2_F;
}

// What the share of a CTA starts in: sequence (or item) b, which the starts of the shares
// first .. last cut; b < 0 marks an idle CTA.  order: Order's groups, base (a CTA's
// number, 0 but for groups of 64 rows) from bit 16 on, and whether a sequence's groups are items.
struct __align__(16) Meta { int32_t b, first, last, order; };
constexpr int32_t LISTED = 1 << 15;
constexpr int MAX_ROWS = 65535, MIN_N = 8;     // rows of H that the calls take, of a group (fp32)
static_assert((MAX_ROWS + MIN_N - 1) / MIN_N < LISTED, "a group's number lies below the mark");

struct SplitParams {
    const int32_t *table, *seq_lens;
    void *o;
    float *lse;
    int32_t *status;           // one word per CTA
    Meta *meta;                // per CTA
    float *part, *stat;        // two slots per CTA: [N][512], and [N][2] (maximum in log2 units, sum)
    int32_t B, H, n_pages, page, max_pages, groups;
    float scale_log2;
    const int32_t *parents;    // drafted trees: [sequences, T], the heads of a node
    int32_t T, heads;
};

// Tokens of a sequence; with a tree, in front of it.
__device__ __forceinline__ int64_t seq_len(const SplitParams &p, int b) {
    const int64_t cap = (int64_t)p.max_pages * p.page, n = p.seq_lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
}
// How the work is listed: CTA base + x works for group x % groups on share x / groups of
// `shares`; a sequence is `items` items.  alike: only sequences of that many groups.
struct Order { int groups, items, base, shares; bool alike; };
// Item i: which sequence, and its first row of H.
struct Item { int b, h0; };
template <bool TREE, int N> __device__ __forceinline__ Item item_of(Order o, int i) {
    if (!TREE) return {i, (int)blockIdx.x % o.groups * N};
    return {i / o.items, (i % o.items + ((int)blockIdx.x - o.base) % o.groups) * N};
}
// Nodes of a tree up to the last that may not be padding.
__device__ __forceinline__ int tree_nodes(const SplitParams &p, int b) {
    const int32_t *par = p.parents + (int64_t)b * p.T;
    int n = p.T;
    for (; n > 0; --n) {
        const int up = par[n - 1];
        if (up >= -1 && up < n - 1) break;
    }
    return n;
}
// Tokens that items read; what is known of the sequence of the last one is kept.
template <bool TREE, int N> struct Lengths {
    int b = -1, rows = 0;
    int64_t len = 0;
    __device__ __forceinline__ int64_t of(const SplitParams &p, Order o, int i) {
        if (!TREE) return seq_len(p, i);
        const Item it = item_of<TREE, N>(o, i);
        if (it.b != b) {
            const int64_t cap = (int64_t)p.max_pages * p.page;
            const int n = tree_nodes(p, it.b);
            b = it.b;
            rows = n * p.heads;
            len = seq_len(p, b) + n;
            len = len > cap ? cap : len;
        }
        return it.h0 < rows && (!o.alike || rows > (o.groups - 1) * N && rows <= o.groups * N) ? len : 0;
    }
};
template <int TOK> __device__ __forceinline__ int64_t tiles_of(int64_t len) { return (len + TOK - 1) / TOK; }
template <int TOK, int OVER> __device__ __forceinline__ int64_t units_of(int64_t len) {
    return len > 0 ? tiles_of<TOK>(len) + OVER : 0;
}
// a / b of numbers >= 0.  Both fit into 32 bits but for caches of more than 2^37
// tokens; the compiler's 64-bit division takes the kernels 40 registers more.
__device__ __forceinline__ int64_t quotient(uint64_t a, uint64_t b) {
    if (!((a | b) >> 32)) return (uint32_t)a / (uint32_t)b;
    uint64_t q = 0, rest = 0;
#pragma unroll 1
    for (int i = 63; i >= 0; --i) {
        rest = rest << 1 | (a >> i & 1);
        q <<= 1;
        if (rest >= b) { rest -= b; q |= 1; }
    }
    return (int64_t)q;
}
// T units in C >= 1 shares of T / C or one more.
struct Shares {
    int64_t q;
    int r;
    __device__ __forceinline__ Shares(int64_t T, int C) : q(quotient(T, C)), r((int)(T - q * C)) {}
    __device__ __forceinline__ int64_t start(int c) const { return q * c + (c < r ? c : r); }
    // the first share that starts after unit x (q >= 1)
    __device__ __forceinline__ int after(int64_t x) const {
        const int64_t big = (q + 1) * r;
        return x < big ? (int)quotient(x, q + 1) + 1 : (int)quotient(x - big, q) + r + 1;
    }
};

// A CTA's share: units [g0, g1) of all, beginning in sequence b0 (whose first
// tile is unit t00).  A sequence is OVER units, for what it costs to begin and to
// end one, and then a unit a tile: without them the CTA with the most sequences
// ended 9 us after the others (48 sequences of up to 9001, 128 heads: 93 us in
// all, with one, two and three units 88, 86 and 86).
struct Share {
    int64_t g0, g1, t00, len0;
    Order o;
    int b0, items, h0;                         // h0: of all sequences, without trees
    bool busy;
    template <bool TREE, int N> __device__ __forceinline__ Item item(int i) const {
        if (!TREE) return {i, h0};             // (the modulus taken at every sequence: a short one 8.93 us, here 8.83)
        return item_of<TREE, N>(o, i);
    }
};
template <int THREADS> struct ShareScratch { int64_t sums[THREADS / 32], t0, t1, len; int b; };

// Groups in step for trees with different numbers of groups (up to ALIKE), where the tokens exceed what
// L2 holds, so that items would bring them in once for every group: sequences with g groups get
// g k_g CTAs of their own, with k_g the fewest whose shares are w units at most.  w is
// the least of 32 up to a quarter above an even share for which there are CTAs enough, and
// where there is none, `o` (items) stays.  units: ALIKE words of shared memory, 0.
// Not inlined, or the main loop spills.
constexpr int ALIKE = 4;
constexpr int64_t PAST_L2 = 2048;              // tiles of 73,728 bytes
template <int TOK, int OVER, int THREADS, int N> __device__ __noinline__ Order alike_order(const SplitParams &p, int64_t *units, Order o) {
    const int tid = threadIdx.x, lane = tid & 31;
    const Order first = {1, 1, 0, 0, false};   // a sequence's first group
    Lengths<true, N> lens;
    for (int b = tid; b < p.B; b += THREADS) {
        const int64_t n = units_of<TOK, OVER>(lens.of(p, first, b));
        if (n) atomicAdd(reinterpret_cast<unsigned long long *>(units + (lens.rows - 1) / N), (unsigned long long)n);
    }
    __syncthreads();
    int64_t sum = 0, once = 0;
#pragma unroll
    for (int g = 1; g <= ALIKE; ++g) {
        sum += g * units[g - 1];
        once += units[g - 1];
    }
    if (once < PAST_L2) return o;
    int64_t w = quotient(sum + gridDim.x - 1, gridDim.x);
    w += w * lane / 128;                       // every lane tries another one
    int need = 0;
#pragma unroll 1
    for (int g = 1; g <= ALIKE; ++g) need += g * (int)quotient(units[g - 1] + w - 1, w);
    const uint32_t fits = __ballot_sync(0xffffffffu, need <= (int)gridDim.x);
    if (!fits) return o;
    w = __shfl_sync(0xffffffffu, w, __ffs(fits) - 1);
    o = {1, 1, 0, 0, true};                    // CTAs that are left over
    int base = 0;
#pragma unroll 1
    for (int g = 1; g <= ALIKE; ++g) {
        const int k = (int)quotient(units[g - 1] + w - 1, w);
        if ((int)blockIdx.x >= base && (int)blockIdx.x < base + g * k) o = {g, 1, base, k, true};
        base += g * k;
    }
    return o;
}
// The order of the work of trees with several groups (all THREADS threads).
template <int TOK, int OVER, int THREADS, int N> __device__ __forceinline__ Order tree_order(const SplitParams &p, int64_t *units) {
    const int tid = threadIdx.x;
    bool even = true;                          // or has some sequence only padding for a group?
    for (int b = tid; b < p.B; b += THREADS) {
        asm volatile("prefetch.global.L1 [%0];" :: "l"(p.seq_lens + b));
        even &= tree_nodes(p, b) * p.heads > (p.groups - 1) * N;
    }
    if (N == 64 && tid < ALIKE) units[tid] = 0;
    Order o = {p.groups, 1, 0, (int)gridDim.x / p.groups, false};
    if (!__syncthreads_and(even)) {
        o = {1, p.groups, 0, (int)gridDim.x, false};
        if (N == 64 && p.groups <= ALIKE && (int64_t)p.max_pages * p.page * p.B >= PAST_L2 * TOK)      // could be as many
            o = alike_order<TOK, OVER, THREADS, N>(p, units, o);
    }
    // one lane's numbers for all, so that the compiler knows them to be a warp's (or the main loop spills)
    return {__shfl_sync(0xffffffffu, o.groups, 0), __shfl_sync(0xffffffffu, o.items, 0), __shfl_sync(0xffffffffu, o.base, 0),
            __shfl_sync(0xffffffffu, o.shares, 0), __shfl_sync(0xffffffffu, (int)o.alike, 0) != 0};
}

// Finds the share (all THREADS threads; ends with a barrier), records it for
// the join, and writes the outputs of sequences with nothing cached.
template <int TOK, int OVER, int THREADS, int N, typename To, bool TREE>
__device__ __forceinline__ Share find_share(const SplitParams &p, ShareScratch<THREADS> &sh, int64_t *units) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Order o = {p.groups, 1, 0, (int)gridDim.x / p.groups, false};
    if (TREE && p.groups > 1) o = tree_order<TOK, OVER, THREADS, N>(p, units);
    const int c = ((int)blockIdx.x - o.base) / o.groups, C0 = o.shares, items = p.B * o.items;
    const int per = (items + THREADS - 1) / THREADS;
    const int b_lo = min(items, tid * per), b_hi = min(items, b_lo + per);
    int64_t mine = 0;
    bool empty = false;
    Lengths<TREE, N> lens;
    for (int b = b_lo; b < b_hi; ++b) {
        const int64_t n = units_of<TOK, OVER>(lens.of(p, o, b));
        mine += n;
        empty |= n == 0;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh.sums[warp] = incl;
    if (tid == 0) sh.b = -1;
    bool empties = true;
    if (TREE) empties = __syncthreads_or(empty);             // the loop below reads much for nothing
    else __syncthreads();
    int64_t T = 0, excl = incl - mine;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) excl += sh.sums[w];
        T += sh.sums[w];
    }
    Share s;
    s.o = o;
    s.items = items;
    s.h0 = (int)blockIdx.x % o.groups * N;
    // the shares of several groups of 64 have two units at least: with one the partial results of 64 rows each
    // cost more than the second tile (one tree of 16 nodes, 32 heads, over 700 tokens: 23.3 us,
    // here 18.3, with three units 17.9, four 19.4; four trees of 8 25.7, 20.3, 20.8, 21.8)
    const int64_t cap = TREE && N == 64 && p.groups > 1 ? (T + 1) / 2 : T;
    const int C = (int)(cap < C0 ? cap : C0);
    s.busy = c < C;
    const Shares cuts(T, C > 0 ? C : 1);
    s.g0 = s.busy ? cuts.start(c) : 0;
    s.g1 = s.busy ? cuts.start(c + 1) : 0;
    if (s.busy && excl <= s.g0 && s.g0 < excl + mine) {
        int64_t at = excl;
        int b = b_lo;
        for (; b < b_hi; ++b) {
            const int64_t len = lens.of(p, o, b), n = units_of<TOK, OVER>(len);
            if (s.g0 < at + n) {
                sh.len = len;
                sh.t0 = at + OVER;
                sh.t1 = at + n;
                sh.b = b;
                break;
            }
            at += n;
        }
    }
    const Order e = {1, p.groups, 0, (int)gridDim.x, false};     // with sequences of a kind, of all there are
    const bool alike = TREE && o.alike;
    const int ec = alike ? blockIdx.x : c, eC = alike ? gridDim.x : C0, many = alike ? p.B * p.groups : items;
    for (int b = ec; (empties || alike) && b < many && ec < eC; b += eC) {
        if (lens.of(p, alike ? e : o, b) > 0) continue;
        const Item it = item_of<TREE, N>(alike ? e : o, b);
        const int nh = min(N, p.H - it.h0);
        const int64_t at = (int64_t)it.b * p.H + it.h0;
        for (int e = tid; e < nh * (LATENT / 4); e += THREADS)
            store4((To *)p.o + at * LATENT + 4 * e, make_float4(0.f, 0.f, 0.f, 0.f));
        if (p.lse && tid < nh) p.lse[at + tid] = -CUDART_INF_F;
    }
    __syncthreads();
    s.b0 = sh.b;
    s.t00 = sh.t0;
    s.len0 = sh.len;
    if (tid == THREADS - 64) {                 // of a warp that has nothing to do yet
        Meta m = {-1, 0, 0, 0};
        if (s.busy && s.b0 >= 0)
            m = {s.b0, cuts.after(s.t00), cuts.after(sh.t1 - 1) - 1, o.groups | (o.items > 1 ? LISTED : 0) | o.base << 16};
        p.meta[blockIdx.x] = m;
    }
    // no tile: the share lies in a sequence's OVER (or lengths changed under the kernel)
    s.busy = s.busy && s.b0 >= 0 && s.t00 < s.g1;
    return s;
}

// The share as segments: sequence b, its tiles [lo, hi); `at` is the unit of
// the sequence's first tile.  Every warp walks them with the same arithmetic.
template <int TOK, int OVER, int N, bool TREE> struct Walk {
    int64_t at, len, lo, hi;
    int b;
    Lengths<TREE, N> lens;
    __device__ __forceinline__ void open(const Share &s, int b_, int64_t len_, int64_t at_, int64_t g) {
        len = len_;
        b = b_; at = at_;
        lo = g > at ? g - at : 0;
        const int64_t n = tiles_of<TOK>(len);
        hi = s.g1 - at < n ? s.g1 - at : n;
    }
    __device__ __forceinline__ void start(const SplitParams &p, const Share &s) { open(s, s.b0, s.len0, s.t00, s.g0); }
    __device__ __forceinline__ bool next(const SplitParams &p, const Share &s) {
        const int64_t to = at + tiles_of<TOK>(len);
        if (to + OVER >= s.g1) return false;
        int n = b + 1;
        int64_t more = 0;
        while (n < s.items && (more = lens.of(p, s.o, n)) == 0) ++n;
        if (n >= s.items) return false;            // lengths changed under the kernel
        open(s, n, more, to + OVER, to + OVER);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == tiles_of<TOK>(len); }
    // partial-result slot of this segment: a sequence's first piece goes to its
    // share's second slot, every other piece to the first
    __device__ __forceinline__ int64_t slot() const { return 2 * (int64_t)blockIdx.x + (lo == 0 ? 1 : 0); }
};

// Adds up the partial results of the sequences that a share boundary cuts.
// Blocks (0 .. gridDim.x - 1, boundary) work for the sequence their boundary lies
// in; an item is 128 channels of a head.  Up to eight pieces: one warp an item,
// all pieces' rows loaded before the weights are known.  More: one block an item,
// every eighth piece a warp.  Pieces are added in a fixed order.  What counts is
// how many blocks fit beside one another: with 102 registers a thread instead of
// 64 one sequence takes 1% less, 48 sequences 6% more.
template <int N, typename To, bool TREE>
__global__ void __launch_bounds__(256, 4) join_kernel(const SplitParams p, int ctas, int32_t *header) {
    static_assert(N >= MIN_N, "more groups than Meta's order holds");
    __shared__ float4 buf[8][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0) {              // the call's status, from the CTAs'
        int st = 0;
        for (int i = tid; i < ctas; i += 256) st |= p.status[i];
        st = __syncthreads_or(st);
        if (tid == 0) *header = st ? FAIL_TIMEOUT : 0;
    }
    const int cta = blockIdx.y + (TREE ? 1 : p.groups);     // shares 1 .. of every group
    if (cta >= ctas) return;
    const Meta m = p.meta[cta];
    if (TREE && m.b < 0) return;                            // before its order is made sense of
    const int groups = TREE ? m.order & (LISTED - 1) : p.groups, base = TREE ? m.order >> 16 : 0;
    const int group = (cta - base) % groups, c = (cta - base) / groups;
    if (m.b < 0 || c < m.first || c > m.last) return;
    const int pieces = m.last - m.first + 2;                // of shares first - 1 .. last
    const int items = TREE && m.order & LISTED ? p.groups : 1;
    const int seq = TREE ? m.b / items : m.b, h0 = ((TREE ? m.b % items : 0) + group) * N;
    const int nh = min(N, p.H - h0);
    const int slot0 = 2 * (base + (m.first - 1) * groups + group);     // of piece i: slot0 + 2 groups i, + 1 for the first
    auto slot_of = [&](int i) { return slot0 + 2 * groups * i + (i == 0); };
    const int block = (c - m.first) * gridDim.x + blockIdx.x, blocks = (pieces - 1) * gridDim.x;
    auto write = [&](int item, float4 acc, float top, float sum, int bad) {
        if (__any_sync(0xffffffffu, bad)) return;           // a share that gave up: o stays as it is
        const float r = inverse_of(sum);
        const int64_t at = (int64_t)seq * p.H + h0 + (item >> 2);
        store4((To *)p.o + at * LATENT + (item & 3) * 128 + 4 * lane,
               make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r));
        if (p.lse && (item & 3) == 0 && lane == 0) p.lse[at] = lse_of(top, sum);
    };
    if (pieces <= 8) {
        for (int item = block * 8 + warp; item < 4 * nh; item += 8 * blocks) {
            const int h = item >> 2, ch = (item & 3) * 128 + 4 * lane;
            float4 y[8], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < pieces) y[i] = load4(p.part + ((int64_t)slot_of(i) * N + h) * LATENT + ch);
            float2 s = make_float2(-CUDART_INF_F, 0.f);
            int bad = 0;
            if (lane < pieces) {
                s = *reinterpret_cast<const float2 *>(p.stat + ((int64_t)slot_of(lane) * N + h) * 2);
                bad = p.status[slot_of(lane) >> 1];
            }
            float top = s.x;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = __shfl_sync(0xffffffffu, top, 0);
            const float f = ex2(s.x - (top == -CUDART_INF_F ? 0.f : top));
            float sum = f * s.y;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < pieces) {
                    const float g = __shfl_sync(0xffffffffu, f, i);
                    acc.x += g * y[i].x; acc.y += g * y[i].y; acc.z += g * y[i].z; acc.w += g * y[i].w;
                }
            write(item, acc, top, sum, bad);
        }
        return;
    }
    for (int item = block; item < 4 * nh; item += blocks) {
        const int h = item >> 2, ch = (item & 3) * 128 + 4 * lane;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -CUDART_INF_F, sum = 0.f;
        int bad = 0;
        for (int i = lane; i < pieces; i += 32) {
            top = fmaxf(top, p.stat[((int64_t)slot_of(i) * N + h) * 2]);
            bad |= p.status[slot_of(i) >> 1];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        for (int i = lane; i < pieces; i += 32) {
            const float2 s = *reinterpret_cast<const float2 *>(p.stat + ((int64_t)slot_of(i) * N + h) * 2);
            sum += ex2(s.x - ref) * s.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        for (int i0 = warp; i0 < pieces; i0 += 32) {
            float4 y[4];
            float f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + 8 * u < pieces) {
                    const int64_t at = (int64_t)slot_of(i0 + 8 * u) * N + h;
                    f[u] = p.stat[at * 2];
                    y[u] = load4(p.part + at * LATENT + ch);
                }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + 8 * u < pieces) {
                    const float g = ex2(f[u] - ref);
                    acc.x += g * y[u].x; acc.y += g * y[u].y; acc.z += g * y[u].z; acc.w += g * y[u].w;
                }
        }
        __syncthreads();                                    // the item before has been read
        buf[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
            for (int i = 1; i < 8; ++i) {
                const float4 y = buf[i][lane];
                acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
            }
            write(item, acc, top, sum, bad);
        }
    }
}

// workspace: header | status | meta | stat | part
struct SplitPlan { int N, groups, ctas; };
constexpr uint64_t WS_STATUS = 256;
inline uint64_t ws_meta(const SplitPlan &s) { return WS_STATUS + ((uint64_t)s.ctas * 4 + 255) / 256 * 256; }
inline uint64_t ws_stat(const SplitPlan &s) { return ws_meta(s) + ((uint64_t)s.ctas * sizeof(Meta) + 255) / 256 * 256; }
inline uint64_t ws_part(const SplitPlan &s) { return ws_stat(s) + (uint64_t)s.ctas * 2 * s.N * 8; }
inline uint64_t ws_bytes(const SplitPlan &s) { return ws_part(s) + (uint64_t)s.ctas * 2 * s.N * LATENT * 4; }

inline SplitPlan split_plan(int32_t H, int N, int ctas, bool tree) {
    SplitPlan s;
    s.N = N;
    s.groups = (H + N - 1) / N;
    s.ctas = s.groups * (ctas / s.groups > 0 ? ctas / s.groups : 1);
    if (tree && s.ctas < ctas) s.ctas = ctas;   // as items, all work
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
    p.parents = a.parents; p.T = a.T; p.heads = a.heads;
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
    const int joins = s.ctas - (p.parents ? 1 : s.groups);
    // two items a warp where one boundary cuts a sequence: with one, twice the
    // blocks come in more waves (48 sequences of up to 9001, 128 heads: 86 us, 84)
    cfg.gridDim = dim3(N / 4, (unsigned)(joins > 0 ? joins : 1));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, p.parents ? join_kernel<N, To, true> : join_kernel<N, To, false>,
                              (const SplitParams &)p, s.ctas, static_cast<int32_t *>(ws));
}

}  // namespace mla
}  // namespace kda
