// kda_mla_prefill.cu -- expanded latent attention of packed prompts on the
// tensor cores, bf16 (kda_mla_prefill in kda.h).
//
// Per head, with queries q_i and keys k_j (192 values) and values v_j (128):
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
// in one pass over the keys with the running maximum m_i and sum.
//
// What bounds it: 640 operations per (query, key, head) against 256 query
// rows of reuse for every key read from L2: the tensor cores.  A CTA takes 256
// queries of one head as two tiles (A, B) of 128 rows, so that one tile's
// products run while the other tile's softmax does, and each key tile of 128
// tokens is read once for both.  Measured: a prompt of 8192 tokens, 32 heads, 421 us
// = 1.63 PFLOP/s of the pairs that are seen, 465 to 477 us under the power cap (tensor
// pipe 71% busy; softmax between).
//
// CTAs take (256 queries, head) pairs, those with the most keys first.  Where
// there are few pairs, the keys of those above an SM's share of all key tiles, or
// of those that do not fill a last round of SMs, are cut into parts; parts leave
// unnormalised results that a join kernel adds up in a fixed order.
//
// With two tiles, tensor memory (all 512 columns): scores of A and B (128 columns each), their
// outputs (128 each).  The weights P replace the scores they come from, as
// bf16 pairs, and are the A operand of the output product straight from
// tensor memory.  Shared memory: both query tiles (96 KB) and a ring of eight
// 16 KB blocks: a key tile is three blocks of 64 channels (two of the head's
// own, one of the shared position key, which is never copied out per head), a
// value tile two blocks of 64 tokens.
//
// Warps 0-7: softmax of tile A, warps 8-15: of tile B, two threads a row (with
// one, a tile's softmax took longer than the other tile's products);
// warp 16: MMA issue; warp 17: loads.  MMAs run in issue order:
//   S_A(j)  O_B(j-1)  S_B(j)  O_A(j)  S_A(j+1)  ...
// so the scores of step j are complete only after the tile's output product of
// step j - 1, and then its output may be rescaled and its P overwritten.
#include "kda_mla_tc.cuh"

#include <float.h>
#include <mutex>

namespace kda {
namespace mla {
namespace {

constexpr int BQ = 128;                                     // rows a tile
constexpr uint32_t QBLOCK = BQ * 128;                       // 64 channels of a query tile
constexpr int RING = 8, PER = 5;                            // blocks in the ring, blocks a key tile

// TILES = 2: as above.  TILES = 1: one query tile, key tiles of 64 whose scores
// take turns in two places (S(0) S(1) O(0) S(2) O(1) ...: the products of the
// next scores run during a tile's softmax), one softmax thread a row, two CTAs an
// SM.  It reads the keys twice as often and its score products are 128 x 64,
// bound by their operands in shared memory; but one CTA's start and end run beside
// the other's products.  With one place for the scores 195 prompts of 400 tokens
// took the same time, 8 of up to 2048 131 us (then 115).
template <int TILES> struct Cfg {
    static constexpr int ROWS = TILES * BQ, BK = 64 * TILES;
    static constexpr int SPLIT = TILES;                     // softmax threads a row; each has 64 of a key tile's columns
    static constexpr int W_MMA = 4 * SPLIT * TILES, W_LOAD = W_MMA + 1, THREADS = 32 * (W_LOAD + 1);
    static constexpr uint32_t BLOCK = BK * 128;             // 64 channels of a key tile, or BK / 2 tokens of a value tile
    static constexpr uint32_t SM_RING = TILES * 3 * QBLOCK, SM_MISC = SM_RING + RING * BLOCK,
                              SM_SWAP = SM_MISC + 256, SM_BYTES = SM_SWAP + (SPLIT == 2 ? 2 * TILES * BQ * 4 : 0);
    static constexpr uint32_t O_COL = BQ * TILES, TCOLS = 256 * TILES;   // scores of tile x at column 128 x
};
static_assert(Cfg<2>::SM_BYTES <= 232448 && 2 * (Cfg<1>::SM_BYTES + 1024) <= 233472, "shared memory");
constexpr float RESCALE = 8.f;

// Which value row of a key tile a softmax thread zeroes where it lies behind the
// sequence's end: (token, chunk of 64 channels).  The output product reads the value
// tile in two blocks of BK / 2 tokens, all channels.  With two halves it begins with
// block b once the warps of half b have arrived on p_full[2 x + b], so that half
// zeroes the whole of that block; with one, all warps arrive before either block.
struct ValueRow { int token, chunk; };
__host__ __device__ constexpr ValueRow unseen_row(int row, int half) { return {64 * half + (row & 63), row >> 6}; }
template <int TILES> constexpr bool zeroed_before_read() {
    using G = Cfg<TILES>;
    bool done[2][G::BK] = {};
    for (int half = 0; half < G::SPLIT; ++half)
        for (int row = 0; row < BQ; ++row) {
            const ValueRow r = unseen_row(row, half);
            if (G::SPLIT == 1 || r.token / (G::BK / 2) == half) done[r.chunk][r.token] = true;
        }
    for (int t = 0; t < G::BK; ++t)
        if (!done[0][t] || !done[1][t]) return false;
    return true;
}
static_assert(zeroed_before_read<1>() && zeroed_before_read<2>(), "a product would read values that are not zeroed yet");

constexpr int MAX_SMS = 160;
constexpr int SLOTS = 2 * MAX_SMS;           // parts with results of their own, over all heads
constexpr int CUTS = MAX_SMS;                // blocks that are cut, over all heads
constexpr int MAX_TAIL = 320;                // blocks of a call whose last round is looked at
constexpr int MIN_PART = 512;                // keys that are worth a part

// A block of up to ROWS queries of a sequence, or a part of its keys; one CTA per
// head.  Everything a CTA needs in one read.
struct __align__(16) Entry {
    int32_t row0, rows;                      // first query among all, queries
    int32_t key0, keys;                      // first key of the part among all, the sequence's keys from there
    int32_t off;                             // query row0 + r sees keys up to key0 + r + off
    int32_t nA, nB;                          // key tiles of the part that tile A and tile B need
    int32_t base, part, parts;               // slot of the block's first part, over all heads; -1 if whole
    int32_t pad[2];
};
// workspace: header | first block of each sequence | entries, most keys first |
// blocks that are cut (as their first part) | partial results per slot:
// [ROWS][2] (maximum in log2 units, sum) and [ROWS][128]
struct Header { int32_t status, entries, cut; };
struct Layout { uint64_t base, entries, cut, stat, part, bytes; };
__host__ __device__ inline Layout layout(int64_t N, int64_t Tq) {
    const uint64_t cap = (uint64_t)Tq / BQ + N;             // blocks of either size, at most
    Layout l;
    l.base = 256;
    l.entries = (l.base + 4 * ((uint64_t)N + 1) + 255) / 256 * 256;
    l.cut = l.entries + (cap + SLOTS) * sizeof(Entry);
    l.stat = l.cut + CUTS * sizeof(Entry);
    l.part = l.stat + (uint64_t)SLOTS * 2 * BQ * 8;
    l.bytes = l.part + (uint64_t)SLOTS * 2 * BQ * DV * 4;
    return l;
}

struct PreParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_r;
    const int32_t *cu_q, *cu_k;
    __nv_bfloat16 *o;
    float *lse;
    Header *head;
    int32_t *base;
    Entry *entries, *cut;
    float2 *stat;
    float *part;
    int64_t Tq, Tk;
    int32_t N, H, causal, negative;   // negative: the scale is; scale_log2 is its magnitude
    float scale_log2;
    int32_t force_timeout;
};

// Lists the blocks of queries and the parts of them, those with the most keys
// first (CTAs start in list order, so the longest do not end last), and clears
// the status.  At most `cap` blocks: offsets that overlap or run backwards lose
// the rest.
template <int TILES>
__global__ void __launch_bounds__(1024) plan_kernel(const PreParams p, int cap, int sms, int may_cut) {
    constexpr int ROWS = Cfg<TILES>::ROWS, BK = Cfg<TILES>::BK, NB = 1024;
    __shared__ int start[NB];
    __shared__ int64_t warp_tot[32];
    __shared__ unsigned long long work;
    __shared__ int blocks, slots, cuts, listed, longest, first_work;
    __shared__ int sizes[MAX_TAIL];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto block_scan = [&](int64_t x) -> int64_t {           // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) warp_tot[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int64_t t = warp_tot[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            warp_tot[lane] = t;
        }
        __syncthreads();
        return x + (warp > 0 ? warp_tot[warp - 1] : 0);
    };
    auto count = [&](int n) { return (seq_span(p.cu_q, p.cu_k, n, p.Tq, p.Tk).nq + ROWS - 1) / ROWS; };
    const int per = (p.N + 1023) / 1024;
    const int n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    int64_t mine = 0;
    for (int n = n0; n < n1; ++n) mine += count(n);
    int64_t at = block_scan(mine) - mine;
    for (int n = n0; n < n1; ++n) {
        p.base[n] = (int)(at < cap ? at : cap);
        at += count(n);
    }
    start[tid] = 0;
    if (tid == 1023) blocks = (int)(at < cap ? at : cap);
    if (tid == 0) { work = 0; slots = 0; cuts = 0; listed = 0; longest = 0; first_work = 0; }
    __syncthreads();
    const int E = blocks;
    auto entry = [&](int e) {
        int lo = 0, hi = p.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.base[mid] <= e) lo = mid; else hi = mid - 1;
        }
        const SeqSpan s = seq_span(p.cu_q, p.cu_k, lo, p.Tq, p.Tk);
        const int i0 = (e - p.base[lo]) * ROWS;
        Entry x;
        x.row0 = (int)s.q0 + i0;
        x.rows = min(ROWS, s.nq - i0);
        x.key0 = (int)s.k0;
        x.keys = s.nk;
        x.off = p.causal ? i0 + s.nk - s.nq : s.nk - 1;
        auto need = [&](int r0) {            // key tiles for the rows r0 .. r0 + 127
            const int64_t seen = (int64_t)min(r0 + BQ, x.rows) + x.off;
            return r0 >= x.rows || seen < 0 ? 0 : (int)(((seen < x.keys ? seen : x.keys) + BK - 1) / BK);
        };
        x.nA = need(0);
        x.nB = need(BQ);
        x.base = -1; x.part = 0; x.parts = 1;
        return x;
    };
    auto tiles_of = [](const Entry &x) { return max(x.nA, x.nB); };
    // a thread's first block, which is mostly its only one, is worked out once
    Entry own = {};
    if (tid < E) own = entry(tid);
    auto get = [&](int e) { return e == tid ? own : entry(e); };
    // key tiles of all blocks, for one head
    if (may_cut) {
        unsigned long long tiles = 0;
        int most = 0;
        for (int e = tid; e < E; e += 1024) {
            const int t = tiles_of(get(e));
            tiles += t;
            most = max(most, t);
            if (TILES == 2 && e < MAX_TAIL) sizes[e] = t;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0 && tiles) { atomicAdd(&work, tiles); atomicMax(&longest, most); }
        __syncthreads();
    }
    // Where the CTAs are few, a block with more key tiles than an SM's share is cut
    // into parts of at most that: over all heads fewer than `sms` blocks and
    // 2 sms parts.
    int64_t share = may_cut ? ((int64_t)work * p.H + sms - 1) / sms : 0;
    if (share < MIN_PART / BK) share = MIN_PART / BK;
    // Without such blocks the last round of CTAs can leave many SMs idle: those
    // blocks that do not fill a round, the ones with the fewest keys, are cut into
    // up to 4 parts if that ends sooner (4 prompts of up to 512 queries after up to
    // 7700 tokens, 224 CTAs: 191 us, 213 without; with lengths that differ more the
    // longest-first order fills the SMs by itself, and looking costs 1 us).
    const int rounds = TILES == 2 && may_cut && longest <= min(share, (int64_t)1 << 20) && E <= MAX_TAIL ? E * p.H / sms : 0;
    const int whole = rounds * sms / p.H;                   // blocks that stay whole
    const int full = whole * p.H - (rounds - 1) * sms;      // SMs that run `rounds` of them, not one fewer
    int rank = 0, cut_into = 1;
    const bool tail = whole > 0 && E > whole && full > 0;
    if (tail) {
        if (tid < E)
            for (int i = 0; i < E; ++i) rank += sizes[i] > sizes[tid] || (sizes[i] == sizes[tid] && i < tid);
        if (tid < E && rank < whole) atomicAdd(&first_work, sizes[tid]);
        __syncthreads();
        // a lane tries lane + 1 parts, all blocks as long as the mean of their kind
        const int parts = lane + 1, rest = (E - whole) * p.H;
        const int w = first_work / whole, t = (int)(work - first_work) / (E - whole);
        const int q = max((t + parts - 1) / parts, 1);
        int end = 1 << 30;
        if (parts == 1 || (parts <= 4 && q >= MIN_PART / BK && rest * parts <= SLOTS)) {
            int i = 0;
            while (full * i + (sms - full) * ((w + i * q) / q) < rest * parts) ++i;
            end = rounds * w + i * q + (parts > 1 ? 4 : 0); // the join costs about four key tiles' time
        }
        const int best = __reduce_min_sync(0xffffffffu, end);
        cut_into = __ffs(__ballot_sync(0xffffffffu, best == end));
    }
    auto parts_of = [&](int tiles) {
        if (tail) return rank < whole ? 1 : max(min(cut_into, tiles), 1);
        return may_cut && tiles > share ? (int)((tiles + share - 1) / share) : 1;
    };
    auto bin_of = [&](int tiles) { return NB - 1 - min(tiles, NB - 1); };
    for (int e = tid; e < E; e += 1024) {
        const int tiles = tiles_of(get(e)), parts = parts_of(tiles);
        for (int k = 0; k < parts; ++k)
            atomicAdd(&start[bin_of((int)((int64_t)tiles * (k + 1) / parts - (int64_t)tiles * k / parts))], 1);
    }
    __syncthreads();
    const int c = start[tid];
    const int incl = (int)block_scan(c);
    start[tid] = incl - c;
    if (tid == 1023) listed = incl;
    __syncthreads();
    for (int e = tid; e < E; e += 1024) {
        const Entry whole = get(e);
        const int tiles = tiles_of(whole), parts = parts_of(tiles);
        const int base = parts > 1 ? atomicAdd(&slots, parts) : -1;
        for (int k = 0; k < parts; ++k) {
            const int t0 = (int)((int64_t)tiles * k / parts), t1 = (int)((int64_t)tiles * (k + 1) / parts);
            Entry x = whole;
            x.key0 += t0 * BK;
            x.keys -= t0 * BK;
            x.off -= t0 * BK;
            x.nA = max(min(x.nA, t1) - t0, 0);
            x.nB = max(min(x.nB, t1) - t0, 0);
            x.base = base; x.part = k; x.parts = parts;
            p.entries[atomicAdd(&start[bin_of(t1 - t0)], 1)] = x;
            if (parts > 1 && k == 0) p.cut[atomicAdd(&cuts, 1)] = x;
        }
    }
    __syncthreads();
    if (tid == 0) { p.head->status = 0; p.head->entries = listed; p.head->cut = cuts; }
}

__device__ __forceinline__ void mma_f16_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                               uint32_t accumulate) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
                   "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
                   "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
                   "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
                   "=f"(v[30]), "=f"(v[31]) : "r"(a) : "memory");
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int TILES>
__global__ void __launch_bounds__(Cfg<TILES>::THREADS, 3 - TILES) prefill_kernel(const __grid_constant__ PreParams p) {
    using G = Cfg<TILES>;
    constexpr int BK = G::BK, ROWS = G::ROWS, SPLIT = G::SPLIT, W_MMA = G::W_MMA, W_LOAD = G::W_LOAD;
    constexpr uint32_t BLOCK = G::BLOCK, SM_Q = 0, SM_RING = G::SM_RING, O_COL = G::O_COL;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + G::SM_MISC);    // [8] ring block loaded
    uint64_t *empty = full + RING;                          // [8] ring block read
    uint64_t *q_full = full + 16;                           // [TILES] query tiles
    uint64_t *s_full = full + 18;                           // [2] scores
    uint64_t *p_full = full + 20;                           // [2][2] halves of P
    uint64_t *o_full = full + 24, *drain = full + 25;       // all outputs
    uint64_t *o_step = full + 17;                           // TILES == 1: the output products of a step
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(full + 26);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);

    float *swap = reinterpret_cast<float *>(sm + G::SM_SWAP);  // [2 tiles][2 halves][128 rows]

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    // the first CTAs set up while the plan is still being made; of the later ones,
    // those that the plan has no entry for end at once
    if (blockIdx.x >= MAX_SMS * (3 - TILES)) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if ((int)(blockIdx.x / p.H) >= p.head->entries) return;
    }
    if (tid == 0) {
        for (int i = 0; i < 26; ++i) mbar_init(&full[i], i >= 20 && i < 24 ? 4 : 1);
        mbar_fence_init();
        *fail = 0;
    }
    if (warp == W_MMA) tmem_alloc<G::TCOLS>(tmem_slot);
    if (warp == W_LOAD && lane == 0) {
        prefetch_map(&p.tm_q);
        if (p.Tk > 0) { prefetch_map(&p.tm_k); prefetch_map(&p.tm_v); prefetch_map(&p.tm_r); }   // else there are none
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = warp_uniform(*tmem_slot);
    const uint32_t smb = warp_uniform(smem_addr(sm));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int e = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const bool forced = p.force_timeout;
    if (forced) {          // test build only: a wait that nothing ends, before any copy or MMA
        if (tid == 0 && !mbar_wait(drain, 0, 64)) *fail = FAIL_TIMEOUT;
        __syncthreads();
    }
    const Entry ent = p.entries[e];          // read beside the count
    if (e < p.head->entries && !forced) {
        const int nA = ent.nA, nB = ent.nB, n = max(nA, nB);
        if (warp == W_LOAD) {
            bool ok = true;
            int q = 0;                                      // blocks asked for
            if (n > 0) {
                if (elect_one()) {
                    if (nA > 0) {
                        mbar_arrive_expect_tx(&q_full[0], 3 * QBLOCK);
                        tma4(smb + SM_Q, &p.tm_q, 0, ent.row0, 0, h, &q_full[0]);
                    }
                }
                __syncwarp();
                for (int j = 0; ok && j < n; ++j) {
                    const int t = ent.key0 + j * BK;
#pragma unroll
                    for (int b = 0; b < PER; ++b) {
                        const int slot = q % RING;
                        if (q >= RING) ok = wait_or_fail(&empty[slot], ((q / RING) & 1) ^ 1, fail);
                        if (!ok) break;
                        if (elect_one()) {
                            const uint32_t dst = smb + SM_RING + slot * BLOCK;
                            mbar_arrive_expect_tx(&full[slot], BLOCK);
                            if (b < 2) tma4(dst, &p.tm_k, 0, t, b, h, &full[slot]);
                            else if (b == 2) tma4(dst, &p.tm_r, 0, t, 0, 0, &full[slot]);
                            else tma4(dst, &p.tm_v, 0, t + (b - 3) * (BK / 2), 2, h, &full[slot]);
                            if (j == 0 && b == 2 && nB > 0) {       // not before what tile A begins with
                                mbar_arrive_expect_tx(&q_full[1], 3 * QBLOCK);
                                tma4(smb + SM_Q + 3 * QBLOCK, &p.tm_q, 0, ent.row0 + BQ, 0, h, &q_full[1]);
                            }
                        }
                        __syncwarp();
                        ++q;
                    }
                }
            }
            if (!ok) {         // let what is in flight land before the CTA ends
                for (int b = max(0, q - RING); b < q; ++b) mbar_wait(&full[b % RING], (b / RING) & 1);
                if (nA > 0) mbar_wait(&q_full[0], 0);
                if (nB > 0) mbar_wait(&q_full[1], 0);
            }
        } else if (warp == W_MMA) {
            if (elect_one()) {
                constexpr uint32_t id_s = idesc(128, BK, FMT_BF16, FMT_BF16, 0, 0);
                constexpr uint32_t id_o = idesc(128, 128, FMT_BF16, FMT_BF16, 0, 1);
                bool ok = true;
                auto landed = [&](uint32_t q) { ok &= wait_one(&full[q % RING], (q / RING) & 1); };  // ring block q
                // S of tile x, step j
                // TILES == 1: scores of even steps in columns 0 .., of odd ones in 64 ..
                auto scores = [&](uint32_t x, uint32_t j, bool first, bool last) {
                    const uint32_t at = TILES == 2 ? 128 * x : 64 * (j & 1);
                    const uint64_t dq = sdesc_k_sw128(smb + SM_Q + x * 3 * QBLOCK);
#pragma unroll
                    for (uint32_t b = 0; b < 3; ++b) {
                        const uint32_t q = PER * j + b;
                        if (first) landed(q);
                        const uint64_t dk = sdesc_k_sw128(smb + SM_RING + q % RING * BLOCK);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16(tmem + at, sdesc_add(dq, b * QBLOCK + k * 32),
                                    sdesc_add(dk, k * 32), id_s, b > 0 || k > 0);
                        if (last) mma_commit(&empty[q % RING]);
                    }
                    mma_commit(&s_full[TILES == 2 ? x : j & 1]);
                };
                // O of tile x, step j, as the halves of P arrive
                auto outputs = [&](uint32_t x, uint32_t j, bool first, bool last) {
                    const uint32_t at = TILES == 2 ? 128 * x : 64 * (j & 1);
#pragma unroll
                    for (uint32_t b = 0; b < 2; ++b) {
                        const uint32_t q = PER * j + 3 + b;
                        if (first) landed(q);
                        if (TILES == 2) ok &= wait_one(&p_full[2 * x + b], j & 1);
                        else if (b == 0) ok &= wait_one(&p_full[j & 1], j >> 1 & 1);
                        fence_after_sync();
                        // values [2 chunks of 64 channels][BK / 2 tokens][128 bytes]: MN-major B
                        const uint64_t dv = sdesc(smb + SM_RING + q % RING * BLOCK, BLOCK / 2, 1024, LAYOUT_SW128);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            mma_f16_tmem_a(tmem + O_COL + 128 * x, tmem + at + (b * (BK / 32) + k) * 8,
                                           sdesc_add(dv, k * 2048), id_o, j > 0 || b > 0 || k > 0);
                        if (last) mma_commit(&empty[q % RING]);
                    }
                };
                uint32_t both = 0;
                if (nA > 0) ok &= wait_one(&q_full[0], 0);
                if constexpr (TILES == 2) {
                    both = min(nA, nB);
                    for (uint32_t j = 0; ok && j < both; ++j) {     // S_A(j) O_B(j-1) S_B(j) O_A(j)
                        scores(0, j, true, false);
                        if (j > 0) outputs(1, j - 1, false, true);
                        else ok &= wait_one(&q_full[1], 0);
                        scores(1, j, false, true);
                        outputs(0, j, true, false);
                    }
                    if (ok && both > 0) outputs(1, both - 1, false, true);
                    if (both == 0 && nB > 0) ok &= wait_one(&q_full[1], 0);
                }
                if constexpr (TILES == 1) {                 // S(0) S(1) O(0) S(2) O(1) ...
                    if (ok && n > 0) scores(0, 0, true, true);
                    for (uint32_t j = 0; ok && j < n; ++j) {
                        if (j + 1 < n) scores(0, j + 1, true, true);
                        outputs(0, j, true, true);
                        mma_commit(o_step);
                    }
                }
                for (uint32_t j = both; TILES == 2 && ok && j < n; ++j) {   // steps that only one tile has
                    const uint32_t x = nB > nA;
                    scores(x, j, true, true);
                    outputs(x, j, true, true);
                }
                mma_commit(o_full);
                if (!ok) {     // MMAs in flight end before tensor memory is freed
                    *fail = FAIL_TIMEOUT;
                    mma_commit(drain);
                    mbar_wait(drain, 0);
                }
            }
            __syncwarp();
        } else {
            // ---- softmax: SPLIT threads a row, each 64 of a key tile's columns ----
            constexpr int OC = DV / SPLIT;                  // output columns a thread
            const int x = SPLIT == 2 ? warp >> 3 : 0;       // tile
            const int half = SPLIT == 2 ? warp >> 2 & 1 : 0;    // columns 64 half ..
            const int row = tid & 127;                      // row of the tile
            const int i = x * BQ + row;                     // query of the block
            const int nX = x ? nB : nA;
            const int end = i < ent.rows ? min(i + ent.off + 1, ent.keys) : ent.keys;   // keys it sees
            // keys that every row of this warp sees
            const int warp_end = __reduce_min_sync(0xffffffffu, end);
            const uint32_t t_s0 = tmem_at(tmem, warp, 128 * x);
            const uint32_t t_o = tmem_at(tmem, warp, O_COL + 128 * x + OC * half);
            const uint32_t pair = 1 + 4 * x + (warp & 3);   // named barrier of the rows' two warps
            // what the row's two threads tell one another (SPLIT == 2)
            float *mine = swap + (2 * x + half) * 128 + row, *theirs = swap + (2 * x + 1 - half) * 128 + row;
            const float sc = p.scale_log2;
            float m = -CUDART_INF_F;                        // unscaled
            float2 l2 = make_float2(0.f, 0.f);
            bool ok = true;
            for (int j = 0; j < nX; ++j) {
                const uint32_t t_s = TILES == 2 ? t_s0 : t_s0 + 64 * (j & 1);
                ok = TILES == 2 ? wait_or_fail(&s_full[x], j & 1, fail)
                                : wait_or_fail(&s_full[j & 1], j >> 1 & 1, fail);
                fence_after_sync();
                float v[64];
                tmem_ld32(t_s + 64 * half, v);
                tmem_ld32(t_s + 64 * half + 32, v + 32);
                tmem_wait_ld();
                reg_fence(v);
                if (p.negative) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) v[c] = -v[c];
                }
                if ((j + 1) * BK > warp_end) {
                    const int lim = end - j * BK - 64 * half;
#pragma unroll
                    for (int c = 0; c < 64; ++c) v[c] = c < lim ? v[c] : -CUDART_INF_F;
                }
                float t0 = v[0], t1 = v[1], t2 = v[2], t3 = v[3];
#pragma unroll
                for (int c = 4; c < 60; c += 8) {
                    t0 = max3(t0, v[c], v[c + 1]);
                    t1 = max3(t1, v[c + 2], v[c + 3]);
                    t2 = max3(t2, v[c + 4], v[c + 5]);
                    t3 = max3(t3, v[c + 6], v[c + 7]);
                }
                t0 = max3(t0, v[60], v[61]);
                t1 = max3(t1, v[62], v[63]);
                const float part = max3(t0, t1, fmaxf(t2, t3));
                // The other half's maximum.  It is read before the other thread's
                // next write: that follows the next scores, which follow this P.
                float top = part;
                bool stop;
                if constexpr (SPLIT == 2) {
                    *mine = part;
                    stop = bar_or(pair, 64, !ok);
                    top = fmaxf(part, *theirs);
                } else {
                    stop = !ok;                             // the same for the whole warp
                }
                if (stop) { ok = false; break; }
                const int valid = ent.keys - j * BK;            // keys of the sequence in this tile
                if (valid < BK) {
                    // values behind the sequence's end hold anything: zero them
                    // (each tile for its own product; the arrival below releases them)
                    const ValueRow v0 = unseen_row(row, half);
                    const int q = PER * j + 3 + v0.token / (BK / 2), slot = q % RING;
                    ok = wait_or_fail(&full[slot], (q / RING) & 1, fail);
                    if (v0.token >= valid) {
                        uint8_t *r = sm + SM_RING + slot * BLOCK + v0.chunk * (BLOCK / 2) + v0.token % (BK / 2) * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(r + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                // The reference is raised only when a score exceeds it by more
                // than 2^8 (weights stay below 2^8, which float32 sums and bf16
                // weights hold as well as ones below 1): the output in tensor
                // memory is then rarely rescaled.  Both halves decide alike.
                if (__any_sync(0xffffffffu, (top - m) * sc > RESCALE || (m == -CUDART_INF_F && top > m))) {
                    const float to = fmaxf(m, top);
                    const float f = to == -CUDART_INF_F ? 1.f : ex2((m - to) * sc);
                    m = to;
                    l2.x *= f; l2.y *= f;
                    if (TILES == 1 && j > 0) {              // the output is not being added to
                        ok = wait_or_fail(o_step, (j - 1) & 1, fail);
                        if (!ok) break;
                        fence_after_sync();
                    }
                    if (j > 0) {
                        for (int c = 0; c < OC; c += 16) {
                            float y[16];
                            tmem_ld16(t_o + c, y);
                            tmem_wait_ld();
                            reg_fence(y);
#pragma unroll
                            for (int k = 0; k < 16; ++k) y[k] *= f;
                            tmem_st16(t_o + c, y);
                        }
                    }
                }
                const float off = m == -CUDART_INF_F ? 0.f : -m * sc;
                const float2 sc2 = make_float2(sc, sc), off2 = make_float2(off, off);
                float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float2 y0 = fma2(make_float2(v[c + k], v[c + k + 1]), sc2, off2);
                        float2 y1 = fma2(make_float2(v[c + k + 2], v[c + k + 3]), sc2, off2);
                        y0.x = ex2(y0.x); y0.y = ex2(y0.y);
                        y1.x = ex2(y1.x); y1.y = ex2(y1.y);
                        a0 = add2(a0, y0);
                        a1 = add2(a1, y1);
                        w[k / 2] = pack_bf(y0.x, y0.y);
                        w[k / 2 + 1] = pack_bf(y1.x, y1.y);
                    }
                    tmem_st16(t_s + 32 * half + c / 2, w);
                }
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[TILES == 2 ? 2 * x + half : j & 1]);
                l2 = add2(l2, add2(a0, a1));
            }
            if (ok && nX > 0) ok = wait_or_fail(o_full, 0, fail);
            const float part = l2.x + l2.y;
            float l = part;
            if constexpr (SPLIT == 2) {
                *mine = part;
                ok = !bar_or(pair, 64, !ok);
                l += *theirs;
            }
            if (ok && x * BQ < ent.rows) {
                const bool whole = ent.base < 0;
                const float r = whole ? inverse_of(l) : 1.f;
                const int64_t at = (int64_t)(ent.row0 + i) * p.H + h;
                const int64_t pr = ((int64_t)(ent.base + ent.part) * p.H + h) * ROWS + i;
                fence_after_sync();
#pragma unroll
                for (int c = 0; c < OC; c += 16) {
                    float y[16];
                    if (nX > 0) {
                        tmem_ld16(t_o + c, y);
                        tmem_wait_ld();
                        reg_fence(y);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) y[k] = 0.f;
                    }
                    if (i < ent.rows && whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = pack_bf(y[2 * k] * r, y[2 * k + 1] * r);
                        uint4 *to = reinterpret_cast<uint4 *>(p.o + at * DV + OC * half + c);
                        to[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        to[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else if (i < ent.rows) {
                        float *to = p.part + pr * DV + OC * half + c;
#pragma unroll
                        for (int k = 0; k < 16; k += 4) store4(to + k, make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]));
                    }
                }
                if (half == 0 && i < ent.rows) {
                    if (!whole) p.stat[pr] = make_float2(m * sc, l);
                    else if (p.lse) p.lse[at] = lse_of(m * sc, l);
                }
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && *fail) atomicExch(&p.head->status, *fail);
    if (warp == W_MMA) tmem_dealloc<G::TCOLS>(tmem);
}

// Adds up the parts of the blocks that are cut: a warp takes a query of a head,
// a lane 4 channels.
template <int TILES>
__global__ void __launch_bounds__(256) prefill_join_kernel(const PreParams p) {
    constexpr int ROWS = Cfg<TILES>::ROWS;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cuts = p.head->cut, lane = threadIdx.x & 31;
    if (p.head->status) return;              // a CTA gave up: o stays as it is
    const int total = cuts * p.H * (ROWS / 8);      // cuts x H is at most MAX_SMS
    for (int job = blockIdx.x; job < total; job += gridDim.x) {
        const int h = job / (ROWS / 8) % p.H, r = job % (ROWS / 8) * 8 + (threadIdx.x >> 5);
        const Entry x = p.cut[job / (ROWS / 8) / p.H];
        if (r >= x.rows) continue;
        auto row_of = [&](int k) { return ((int64_t)(x.base + k) * p.H + h) * ROWS + r; };
        float top = -CUDART_INF_F;
        for (int k = lane; k < x.parts; k += 32) top = fmaxf(top, p.stat[row_of(k)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < x.parts; ++k) {
            const float2 st = p.stat[row_of(k)];
            const float4 y = load4(p.part + row_of(k) * DV + 4 * lane);
            const float f = ex2(st.x - ref);
            sum += f * st.y;
            acc.x += f * y.x; acc.y += f * y.y; acc.z += f * y.z; acc.w += f * y.w;
        }
        const float f = inverse_of(sum);
        const int64_t at = (int64_t)(x.row0 + r) * p.H + h;
        store4(p.o + at * DV + 4 * lane, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
        if (p.lse && lane == 0) p.lse[at] = lse_of(top, sum);
    }
}

template <int TILES> cudaError_t launch(const PrefillArgs &a, cudaStream_t st) {
    using G = Cfg<TILES>;
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(prefill_kernel<TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)G::SM_BYTES);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    PreParams p = {};
    const uint64_t H = (uint64_t)a.H, Tq = (uint64_t)a.Tq, Tk = (uint64_t)a.Tk;
    const uint64_t qd[4] = {64, Tq, 3, H}, qs[3] = {H * DQK * 2, 128, DQK * 2};
    const uint32_t qb[4] = {64, BQ, 3, 1};
    if (!map4(&p.tm_q, a.q, qd, qs, qb)) return cudaErrorInvalidValue;
    if (Tk > 0) {      // without keys no tile is loaded, and no map is looked at
        const uint64_t kd[4] = {64, Tk, 4, H}, ks[3] = {H * (NOPE + DV) * 2, 128, (NOPE + DV) * 2};
        const uint32_t kb[4] = {64, G::BK, 1, 1}, vb[4] = {64, G::BK / 2, 2, 1};
        const uint64_t rd[4] = {64, Tk, 1, 1}, rs[3] = {ROPE * 2, ROPE * 2, ROPE * 2};
        if (!map4(&p.tm_k, a.kv, kd, ks, kb) || !map4(&p.tm_v, a.kv, kd, ks, vb) ||
            !map4(&p.tm_r, a.k_r, rd, rs, kb))
            return cudaErrorInvalidValue;
    }
    p.cu_q = a.cu_q; p.cu_k = a.cu_k; p.o = (__nv_bfloat16 *)a.o; p.lse = a.lse;
    const Layout l = layout(a.N, a.Tq);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.head = reinterpret_cast<Header *>(ws);
    p.base = reinterpret_cast<int32_t *>(ws + l.base);
    p.entries = reinterpret_cast<Entry *>(ws + l.entries);
    p.cut = reinterpret_cast<Entry *>(ws + l.cut);
    p.stat = reinterpret_cast<float2 *>(ws + l.stat);
    p.part = reinterpret_cast<float *>(ws + l.part);
    p.Tq = a.Tq; p.Tk = a.Tk; p.N = a.N; p.H = a.H; p.causal = a.causal;
    // a negative scale flips the scores' sign; a zero one makes them (almost) equal
    const float s2 = a.scale * 1.4426950408889634f;
    p.negative = s2 < 0.f;
    p.scale_log2 = fmaxf(fabsf(s2), FLT_MIN);
    p.force_timeout = fault_force_timeout();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int sms = 1;
    e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    if (sms > MAX_SMS) sms = MAX_SMS;
    const int64_t cap = a.Tq / G::ROWS + a.N;                  // blocks of queries, at most
    // Cutting pays where (queries / 256) x heads leaves the SMs fewer than two
    // CTAs each: two sequences of up to 3000 queries over up to 8000 keys, one
    // head: 106 us whole, 47 us cut; one prompt of 4096 tokens, four heads: 60 and
    // 46 us.  Where nothing is cut after all it costs 3 to 5 us (a join kernel and
    // CTAs with nothing to do), and with more CTAs the longest-first order balances
    // by itself.
    const bool may_cut = a.Tq / G::ROWS * a.H < 2 * sms && a.H < 2 * sms && a.Tk > MIN_PART;
    e = cudaLaunchKernelEx(&cfg, plan_kernel<TILES>, p, (int)cap, sms, (int)may_cut);
    if (e != cudaSuccess) return e;
    // a CTA per block and head, and one for each further part
    cfg.gridDim = dim3((unsigned)(cap * a.H + (may_cut ? SLOTS : 0)));
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SM_BYTES;
    e = cudaLaunchKernelEx(&cfg, prefill_kernel<TILES>, p);
    if (e != cudaSuccess || !may_cut) return e;
    cfg.gridDim = dim3(8 * (unsigned)sms);                  // all resident: without a cut they end at once
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, prefill_join_kernel<TILES>, p);
}

}  // namespace

uint64_t prefill_tc_workspace_bytes(int32_t N, int64_t Tq) { return layout(N, Tq).bytes; }

cudaError_t launch_prefill_tc(const PrefillArgs &a, cudaStream_t st) {
    // One tile where a CTA's start and end are much of its time (few keys or few
    // queries a sequence) or where the SMs get few CTAs; two where the products
    // decide.  In us, one tile and two, 16 heads where not said otherwise, all
    // under the power cap:
    //   64 prompts of up to 300 tokens                 69 and 95
    //   195 of 400, 8 heads                           269 and 284
    //   38 of 64 after 4000                           204 and 227
    //   1 of 2048 (work 860)                           44 and 52
    //   8 of up to 2048, 32 heads (work 2450)         117 and 125
    //   11 of 900, 31 heads (work 3550)               185 and 172
    //   4 of 2560, 30 heads (work 10100)              236 and 227
    //   1 of 8192, 32 heads (work 27600)              512 and 465
    // 11 of 900 is on the wrong side of the rule, which loses 8 % there.  Between
    // work 2450 and 3550 nothing is measured, nor how far ragged lengths move the
    // point: the host knows the sums of the lengths only.
    int sms = 1;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const double q = (double)a.Tq / a.N, k = (double)a.Tk / a.N;
    // keys that a block of 256 queries meets, times blocks an SM
    const double work = (a.causal ? k - q / 2 : k) * a.Tq / 256 * a.H / sms;
    return q <= 128 || k <= 640 || work <= 4000 ? launch<1>(a, st) : launch<2>(a, st);
}

}  // namespace mla
}  // namespace kda
