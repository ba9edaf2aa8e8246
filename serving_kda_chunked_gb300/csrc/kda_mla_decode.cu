// kda_mla_decode.cu -- absorbed latent attention of single tokens over the
// paged bf16 cache, on the tensor cores (kda_mla_decode in kda.h).
//
// Per sequence, with the H queries q_h (576 values) and n cached rows c_j:
//   s_jh = scale q_h . c_j,  p_jh = exp(s_jh - m_h),  o_h = sum_j p_jh c_j[:512] / sum_j p_jh
//
// What bounds it: the cache is read once (1152 bytes a token) for 2176 H
// operations a token, 60 per byte at H = 32, a fifth of what the tensor cores
// do in that time: HBM.  So a tile of 64 tokens is brought to shared memory
// once and serves as the keys and as the values.  Measured: 256 sequences of up to
// 8192 tokens, 32 heads, 203 us = 6.3 TB/s; one of 1 Mi tokens 183 us = 6.6 TB/s, 99 % of
// what a copy reaches; 48 of up to 9001, 128 heads (two groups of 64 read each tile), 83 us.
//
// Both products are transposed: S^T [64 tokens x N heads] = C Q^T and
// O^T [512 x N heads] = C^T P, so that the tokens or latent channels are the
// M rows of an MMA and the N columns are just the heads there are (16, 32 or
// 64 a CTA).  With the heads as M rows, 32 heads would waste half or more of
// every MMA, and 64 x 512 outputs would leave no tensor memory for the scores.
//
// Shared memory: two stages of 64 tokens x 576 (73,728 bytes each), the
// queries, P.  A stage is laid out [8 groups of 8 tokens][9 chunks of 64
// channels][8 tokens][128 bytes], 128-byte swizzled: one TMA box brings a
// whole page piece, and both the K-major (scores) and the MN-major (output)
// descriptors see uniform strides.
//
// Work split and join: kda_mla_split.cuh, one share per SM.
//
// Trees of drafted tokens (TREE) are the same with more rows, in groups of 64, and a mask
// in the tiles that hold nodes.  Each group reads every tile for itself, and shared memory bounds
// that: the MMAs of a tile read 147 KB for the scores (rows and queries) and 96 KB for the
// output, and 74 KB come in, 2480 cycles at 128 bytes of the 2750 that a tile takes (the
// issuing thread waits for 600 of them, for data or weights).  More rows a tile, or 128
// tokens at a time, would read less, but 64 rows of queries and two stages fill shared memory.
// Tried: the halves of a stage loaded and released apart (198 us for the 64 trees below, 204),
// a tile brought in once for two and four groups (204, 216).  Measured, 32 heads: 64 ragged trees
// of up to 8 nodes over up to 8192 tokens 151 us, of which tiles are 101, beginnings and ends of
// sequences some 10 and the join 4 (the rest has not been found: the order's arithmetic in front of
// the first load, shares of up to a quarter more than even, or L2 misses of CTAs that fall out of
// step); 8 trees of 48 nodes over up to 32,768 tokens 738 us = 0.9 PFLOP/s.
//
// Warps 0-3 and 4-7: softmax and epilogue of half the heads each; warp 8: MMA
// issue; warp 9: loads.
#include "kda_mla_split.cuh"
#include "kda_mla_tc.cuh"
#include "kda_tree.cuh"

#include <mutex>

namespace kda {
namespace mla {
namespace {

constexpr int TOK = 64, CHUNKS = ROW / 64;                  // tokens a tile, 128-byte chunks a row
constexpr uint32_t GROUP = CHUNKS * 1024;                   // 8 tokens
constexpr uint32_t STAGE = 8 * GROUP;
constexpr int THREADS = 320, W_MMA = 8, W_LOAD = 9;
constexpr int MAX_CTAS = 160;                               // per launch, up to one wave
constexpr float RESCALE = 8.f;                              // see the softmax below

template <int N> struct Smem {
    static constexpr uint32_t Q = 2 * STAGE, P = Q + CHUNKS * N * 128, RED = P + N * 128,
                              COL = RED + 2 * 4 * N * 4, MISC = COL + 2 * N * 4, BYTES = MISC + 256;
};
static_assert(Smem<64>::BYTES <= 232448, "shared memory");

struct DecParams : SplitParams {
    CUtensorMap tm_c, tm_q;
    int32_t force_timeout;
};

// NW columns of the S^T accumulator (M = 64) of this warp's 16 tokens: register
// 4 i + 2 r + j is token lane / 4 + 8 r, head 8 i + 2 (lane % 4) + j.
template <int NW> __device__ __forceinline__ void ld_scores(uint32_t a, float (&v)[NW / 2]);
template <> __device__ __forceinline__ void ld_scores<8>(uint32_t a, float (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(a) : "memory");
}
template <> __device__ __forceinline__ void ld_scores<16>(uint32_t a, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7]) : "r"(a) : "memory");
}
template <> __device__ __forceinline__ void ld_scores<32>(uint32_t a, float (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
                   "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]) : "r"(a) : "memory");
}
// 32 lanes x 8 consecutive columns.
__device__ __forceinline__ void ld_cols(uint32_t a, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7]) : "r"(a) : "memory");
}
__device__ __forceinline__ void st_cols(uint32_t a, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),
                    "f"(v[6]), "f"(v[7]) : "memory");
}
__device__ __forceinline__ void ld_cols(uint32_t a, float (&v)[16]) { tmem_ld16(a, v); }
__device__ __forceinline__ void st_cols(uint32_t a, const float (&v)[16]) { tmem_st16(a, v); }

// TREE: the rows are the heads of a tree's nodes (kda_mla_tree_decode); a node's rows see
// the tokens in front of the tree, the node and its ancestors.
template <int N, bool TREE>
__global__ void __launch_bounds__(THREADS, 1) decode_kernel(const __grid_constant__ DecParams p) {
    using L = Smem<N>;
    // tiles' time to begin and end a sequence (64 trees of 8 nodes: 2 154 us, 3 152, 4 151, 6 150; one: 17.3, 15.9, 17.2, 17.2)
    constexpr int OVER = TREE && N == 64 ? 4 : 2;
    constexpr uint32_t TCOLS = N == 64 ? 512 : 256;
    constexpr uint32_t S_COL = 0, O_COL = 2 * N;            // S^T twice, O^T in 4 blocks of 128 channels
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::MISC);   // [2] stage loaded
    uint64_t *empty = full + 2;                             // [2] stage read
    uint64_t *s_full = full + 4;                            // [2] S^T ready
    uint64_t *p_full = full + 6, *o_full = full + 7;        // P written; its O^T product done
    uint64_t *q_full = full + 8, *q_empty = full + 9, *o_empty = full + 10, *drain = full + 11;
    uint64_t *vmask = full + 12;                            // [2] tokens of the stage that are seen
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(full + 16);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
    auto *scratch = reinterpret_cast<ShareScratch<THREADS> *>(full + 18);
    float *red = reinterpret_cast<float *>(sm + L::RED);    // [2][4 warps][N]
    float *col_a = reinterpret_cast<float *>(sm + L::COL);  // [N]
    float *col_b = col_a + N;                               // [N]

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < 12; ++i) mbar_init(&full[i], i == 6 || i == 10 ? 8 : 1);
        mbar_fence_init();
        *fail = 0;
    }
    if (warp == W_MMA) tmem_alloc<TCOLS>(tmem_slot);
    if (warp == W_LOAD && lane == 0) { prefetch_map(&p.tm_c); prefetch_map(&p.tm_q); }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    fence_before_sync();
    const Share share = find_share<TOK, OVER, THREADS, N, __nv_bfloat16, TREE>(p, *scratch, reinterpret_cast<int64_t *>(sm + L::RED));
    fence_after_sync();
    const uint32_t tmem = warp_uniform(*tmem_slot);
    const uint32_t smb = warp_uniform(smem_addr(sm));
    const bool forced = p.force_timeout && share.busy;
    if (forced) {      // test build only: a wait that nothing ends, before any copy or MMA
        if (tid == 0 && !mbar_wait(drain, 0, 64)) *fail = FAIL_TIMEOUT;
        __syncthreads();
    }

    if (share.busy && !forced) {
        Walk<TOK, OVER, N, TREE> w;
        w.start(p, share);
        if (warp == W_LOAD) {
            // ---- loads: the table is read 32 entries at a time; what a tile
            // needs is ready before its stage is ----
            const int sh = 31 - __clz(p.page);                             // page = 1 << sh
            const int psh = sh < 6 ? sh : 6, piece = 1 << psh;             // tokens a box
            const int per_tile = TOK >> psh, bsh = 5 - (6 - psh);          // boxes a tile; 1 << bsh tiles a table read
            const uint32_t box_bytes = (uint32_t)piece * ROW * 2;
            const int rows8 = (int)((int64_t)p.n_pages * p.page / 8);      // out of range: zeros arrive
            uint32_t k = 0;                                                // tiles asked for
            int seg = 0;                                                   // queries asked for
            bool ok = true;
            do {
                if (seg > 0) ok = wait_or_fail(q_empty, (seg - 1) & 1, fail);
                if (!ok) break;
                const Item it = share.item<TREE, N>(w.b);
                if (elect_one()) {
                    mbar_arrive_expect_tx(q_full, CHUNKS * N * 128);
                    tma4(smb + L::Q, &p.tm_q, 0, it.h0, 0, it.b, q_full);
                }
                __syncwarp();
                ++seg;
                const int32_t *tab = p.table + (int64_t)it.b * p.max_pages;
                uint64_t nodes = 0;                                        // that are not padding, once known
                bool known = false;
                const int64_t front = TREE ? seq_len(p, it.b) : 0;
                // first row / 8 of this lane's box of 32, and of the next 32
                auto boxes = [&](int64_t i) {
                    const int64_t t = i * TOK + ((int64_t)lane << psh);
                    const int pg = i < w.hi && t < w.len ? tab[t >> sh] : -1;
                    return pg < 0 || pg >= p.n_pages ? rows8 : ((pg << sh) + ((int)t & (p.page - 1))) >> 3;
                };
                int at8 = rows8, next8 = boxes(w.lo);
                for (int64_t i = w.lo; i < w.hi; ++i, ++k) {
                    const int r = (int)(i - w.lo) & ((1 << bsh) - 1);
                    if (r == 0) {
                        at8 = next8;
                        next8 = boxes(i + (1 << bsh));
                    }
                    const int st = k & 1;
                    uint64_t mask = 0;
                    int g8[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g8[j] = __shfl_sync(0xffffffffu, at8, (r * per_tile + j) & 31);
                        if (j < per_tile && g8[j] < rows8)
                            mask |= (piece == 64 ? ~0ull : (1ull << piece) - 1) << (j * piece);
                    }
                    const int64_t left = w.len - i * TOK;
                    if (left < TOK) mask &= (1ull << left) - 1;
                    if constexpr (TREE) {
                        const int64_t d = i * TOK - front;                 // node of the tile's first token
                        if (d > -64 && !known) {
                            uint64_t a, c;
                            tree::all_ancestors(p.parents + (int64_t)it.b * p.T, p.T, lane, a, c);
                            nodes = (uint64_t)__ballot_sync(0xffffffffu, c != 0) << 32 | __ballot_sync(0xffffffffu, a != 0);
                            known = true;
                        }
                        if (d >= 0) mask &= d < 64 ? nodes >> d : 0ull;
                        else if (d > -64) mask &= nodes << -d | ((1ull << -d) - 1);
                    }
                    if (k >= 2) ok = wait_or_fail(&empty[st], ((k >> 1) & 1) ^ 1, fail);
                    if (!ok) break;
                    if (elect_one()) {
                        vmask[st] = mask;
                        mbar_arrive_expect_tx(&full[st], STAGE);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < per_tile)
                                tma4(smb + st * STAGE + j * box_bytes, &p.tm_c, 0, 0, 0, g8[j], &full[st]);
                    }
                    __syncwarp();
                    // The next tile to L2, before there is a stage for it.  Without: 1 Mi
                    // tokens 194 us (183), 256 sequences of up to 8192 217 (208), 48 of
                    // up to 9001, 128 heads 100 (93).  Two tiles ahead 187, 212 and 92,
                    // three 204, 224 and 93.
                    const bool here = r + 1 < 1 << bsh;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int ahead = __shfl_sync(0xffffffffu, here ? at8 : next8, ((r + 1) * per_tile + j) & 31);
                        if (j < per_tile && i + 1 < w.hi && ahead < rows8 && elect_one())
                            tma4_prefetch(&p.tm_c, 0, 0, 0, ahead);
                    }
                    __syncwarp();
                }
            } while (ok && w.next(p, share));
            if (!ok) {           // let what is in flight land before the CTA ends
                for (uint32_t j = k >= 2 ? k - 2 : 0; j < k; ++j) mbar_wait(&full[j & 1], (j >> 1) & 1);
                if (seg > 0) mbar_wait(q_full, (seg - 1) & 1);
            }
        } else if (warp == W_MMA) {
            // ---- MMA issue ----
            // O^T of tile i - 1 goes before S^T of tile i when its P is ready
            // and tile i has not landed: waiting for tile i first would keep
            // tile i - 1's stage, and with it the load of tile i + 1, waiting.
            constexpr uint32_t id_s = idesc(64, N, FMT_BF16, FMT_BF16, 0, 0);
            constexpr uint32_t id_o = idesc(128, N, FMT_BF16, FMT_BF16, 1, 0);
            if (elect_one()) {
                const uint64_t dq = sdesc_k_sw128(smb + L::Q);
                const uint64_t dp = sdesc_k_sw128(smb + L::P);
                uint32_t k = 0;                             // tiles whose S^T has been issued
                int seg = 0;
                bool ok = true;
                auto out = [&](uint32_t j, bool first) {    // O^T of tile j
                    ok &= wait_one(p_full, j & 1);
                    if (first && seg > 0) ok &= wait_one(o_empty, (seg - 1) & 1);
                    fence_after_sync();
                    const uint64_t dv = sdesc(smb + (j & 1) * STAGE, 1024, GROUP, LAYOUT_SW128);
#pragma unroll
                    for (int mb = 0; mb < 4; ++mb)
#pragma unroll
                        for (int s = 0; s < TOK / 16; ++s)
                            mma_f16(tmem + O_COL + mb * N, sdesc_add(dv, mb * 2048 + s * 2 * GROUP),
                                    sdesc_add(dp, s * 32), id_o, !(first && s == 0));
                    mma_commit(&empty[j & 1]);
                    mma_commit(o_full);
                };
                do {
                    ok &= wait_one(q_full, seg & 1);
                    for (int64_t i = w.lo; ok && i < w.hi; ++i, ++k) {
                        const int st = k & 1;
                        bool owed = i > w.lo;               // O^T of tile k - 1
                        if (owed) {
                            bool landed = false, ready = false;
                            for (int n = 0; n < (1 << 20) && !(landed || ready); ++n) {
                                ready = mbar_test(p_full, (k - 1) & 1);
                                landed = mbar_test(&full[st], (k >> 1) & 1);
                            }
                            if (!landed) {
                                out(k - 1, i - 1 == w.lo);
                                owed = false;
                            }
                        }
                        ok &= wait_one(&full[st], (k >> 1) & 1);
                        fence_after_sync();
                        const uint64_t dc = sdesc(smb + st * STAGE, 16, GROUP, LAYOUT_SW128);
#pragma unroll
                        for (int s = 0; s < ROW / 16; ++s)
                            mma_f16(tmem + S_COL + st * N, sdesc_add(dc, (s >> 2) * 1024 + (s & 3) * 32),
                                    sdesc_add(dq, (s >> 2) * (N * 128) + (s & 3) * 32), id_s, s > 0);
                        mma_commit(&s_full[st]);
                        if (i == w.hi - 1) mma_commit(q_empty);
                        if (owed) out(k - 1, i - 1 == w.lo);
                    }
                    out(k - 1, w.hi - 1 == w.lo);
                    ++seg;
                } while (ok && w.next(p, share));
                if (!ok) {       // MMAs in flight end before tensor memory is freed
                    *fail = FAIL_TIMEOUT;
                    mma_commit(drain);
                    mbar_wait(drain, 0);
                }
            }
            __syncwarp();
        } else {
            // ---- softmax and epilogue of half the heads a warpgroup ----
            // A warp whose wait failed stays in step with the others (their barriers
            // count all 128 threads) until the next bar_or tells all of them.
            constexpr int NW = N / 2, V = NW / 4;           // heads a warpgroup, heads a thread looks at
            constexpr int EC = NW < 16 ? NW : 16;           // columns moved at a time in the epilogue
            const int wg = warp >> 2, wt = tid & 127, w4 = warp & 3;
            const int n0 = wg * NW;                         // its first head of the CTA's
            const uint32_t bar = 1 + wg;
            float *red_w = red + wg * 8 * NW;               // [2][4 warps][NW]
            float *ca = col_a + n0, *cb = col_b + n0;
            uint32_t k = 0;
            bool ok = true, stop = false;
            const int row = 16 * w4 + (lane >> 2);          // this thread's tokens: row, row + 8
            do {
                float m[V], l[V];                           // heads 8 (v / 2) + 2 (lane % 4) + v % 2
                // lane: what nodes lane and lane + 32 see; which of the warpgroup's rows are padding's
                uint64_t sees = 0, sees32 = 0;
                uint32_t pad = 0;
                int64_t front = 0;
                const Item it = share.item<TREE, N>(w.b);
                const int h0 = it.h0, nh = min(N, p.H - h0);
                if constexpr (TREE) {
                    const int32_t *par = p.parents + (int64_t)it.b * p.T;
                    front = seq_len(p, it.b);
                    tree::all_ancestors(par, p.T, lane, sees, sees32);
                    const uint32_t lo = __ballot_sync(0xffffffffu, sees != 0), hi = __ballot_sync(0xffffffffu, sees32 != 0);
                    const int t = min((h0 + n0 + lane) / p.heads, p.T - 1);
                    pad = __ballot_sync(0xffffffffu, !((t < 32 ? lo : hi) >> (t & 31) & 1));
                }
#pragma unroll
                for (int v = 0; v < V; ++v) { m[v] = -CUDART_INF_F; l[v] = 0.f; }
                for (int64_t i = w.lo; i < w.hi; ++i, ++k) {
                    const int st = k & 1;
                    ok = wait_or_fail(&s_full[st], (k >> 1) & 1, fail);
                    ok = ok && test_or_fail(&full[st], (k >> 1) & 1, fail);  // for vmask
                    fence_after_sync();
                    float x[NW / 2];
                    ld_scores<NW>(tmem_at(tmem, warp, S_COL + st * N + n0), x);
                    const uint64_t vm = vmask[st];
                    tmem_wait_ld();
                    reg_fence(x);
                    const bool see0 = vm >> row & 1, see1 = vm >> (row + 8) & 1;
#pragma unroll
                    for (int e = 0; e < NW / 2; ++e)
                        x[e] = (e & 2 ? see1 : see0) ? x[e] * p.scale_log2 : -CUDART_INF_F;
                    if constexpr (TREE) {
                        const int64_t d = i * TOK - front;
                        if (d > -TOK) {                     // the tile has nodes
                            const int d0 = (int)d + row, d1 = d0 + 8;
#pragma unroll
                            for (int v = 0; v < V; ++v) {
                                const int col = n0 + 8 * (v >> 1) + 2 * (lane & 3) + (v & 1);
                                const int t = min((h0 + col) / p.heads, p.T - 1);
                                const uint64_t a = __shfl_sync(0xffffffffu, sees, t & 31), c = __shfl_sync(0xffffffffu, sees32, t & 31);
                                const uint64_t mine = t < 32 ? a : c;
                                if (d0 >= 0 && !(d0 < 64 && (mine >> d0 & 1))) x[(v >> 1) * 4 + (v & 1)] = -CUDART_INF_F;
                                if (d1 >= 0 && !(d1 < 64 && (mine >> d1 & 1))) x[(v >> 1) * 4 + 2 + (v & 1)] = -CUDART_INF_F;
                            }
                        }
                    }
                    if (vm != ~0ull) {
                        // rows that are not seen hold anything: zero them as values
                        const int t = tid >> 2;
                        if (!(vm >> t & 1)) {
                            uint8_t *r = sm + st * STAGE + (t >> 3) * GROUP + (t & 7) * 128 + (tid & 3) * 2048;
#pragma unroll
                            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    *reinterpret_cast<uint4 *>(r + ch * 1024 + e * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    // The reference maximum is raised only when a score exceeds it by
                    // more than 2^8: until then weights stay below 2^8, which float32
                    // sums and bf16 weights hold as well as ones below 1, and neither
                    // need the warps tell each other their maxima nor the output in
                    // tensor memory be rescaled.
                    bool raise = i == w.lo;
                    if (!raise) {
                        bool over = !ok;
#pragma unroll
                        for (int e = 0; e < NW / 2; ++e) over |= x[e] > m[(e >> 2) * 2 + (e & 1)] + RESCALE;
                        raise = bar_or(bar, 128, over);
                    }
                    if (raise) {
                        // maximum over the warp's 16 tokens: each exchange halves the
                        // heads a lane keeps, lane bits 4, 3, 2 choosing bits of v
                        float t[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) t[v] = fmaxf(x[(v >> 1) * 4 + (v & 1)], x[(v >> 1) * 4 + 2 + (v & 1)]);
                        int keep = 0;
#pragma unroll
                        for (int bit = 16, half = V / 2; bit >= 4; bit >>= 1, half >>= 1) {
                            if (half >= 1) {
                                const bool up = lane & bit;
#pragma unroll
                                for (int v = 0; v < V / 2; ++v)
                                    if (v < half) {
                                        const float give = up ? t[v] : t[v + half], have = up ? t[v + half] : t[v];
                                        t[v] = fmaxf(have, __shfl_xor_sync(0xffffffffu, give, bit));
                                    }
                                keep += up ? half : 0;
                            } else {
                                t[0] = fmaxf(t[0], __shfl_xor_sync(0xffffffffu, t[0], bit));
                            }
                        }
                        float *rd = red_w + (k & 1) * 4 * NW;
                        rd[w4 * NW + (keep >> 1) * 8 + 2 * (lane & 3) + (keep & 1)] = t[0];
                        stop = bar_or(bar, 128, !ok);
                        if (stop) break;
#pragma unroll
                        for (int v = 0; v < V; v += 2) {
                            const int at = (v >> 1) * 8 + 2 * (lane & 3);
                            float2 y = *reinterpret_cast<const float2 *>(rd + at);
#pragma unroll
                            for (int q = 1; q < 4; ++q) {
                                const float2 z = *reinterpret_cast<const float2 *>(rd + q * NW + at);
                                y.x = fmaxf(y.x, z.x); y.y = fmaxf(y.y, z.y);
                            }
                            const float top[2] = {y.x, y.y};
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float to = fmaxf(m[v + j], top[j]);
                                const float f = to == -CUDART_INF_F ? 1.f : ex2(m[v + j] - to);
                                l[v + j] *= f;
                                m[v + j] = to;
                                if (w4 == 0 && lane < 4) ca[at + j] = f;
                            }
                        }
                        if (i > w.lo) {
                            ok = wait_or_fail(o_full, (k - 1) & 1, fail);
                            bar_sync(bar, 128);             // ca
                            fence_after_sync();
                            for (int mb = 0; mb < 4; ++mb)
#pragma unroll
                                for (int c = 0; c < NW; c += EC) {
                                    float y[EC];
                                    const uint32_t at = tmem_at(tmem, warp, O_COL + mb * N + n0 + c);
                                    ld_cols(at, y);
                                    tmem_wait_ld();
                                    reg_fence(y);
#pragma unroll
                                    for (int e = 0; e < EC; ++e) y[e] *= ca[c + e];
                                    st_cols(at, y);
                                }
                            tmem_wait_st();
                        }
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float ref = m[v] == -CUDART_INF_F ? 0.f : m[v];
                        float &a = x[(v >> 1) * 4 + (v & 1)], &d = x[(v >> 1) * 4 + 2 + (v & 1)];
                        a = ex2(a - ref);
                        d = ex2(d - ref);
                        l[v] += a + d;
                    }
                    // P [head][token] bf16, K-major: the previous product must have read it
                    if (k > 0) ok = ok && test_or_fail(o_full, (k - 1) & 1, fail);
                    if (NW == 8) {
                        const uint32_t dst = smb + L::P + sw128_off(n0 + (lane & 7), 2 * w4 + (lane >> 3 & 1));
                        asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};"
                                     :: "r"(dst), "r"(pack_bf(x[0], x[1])), "r"(pack_bf(x[2], x[3])) : "memory");
                    } else {
#pragma unroll
                        for (int e = 0; e + 1 < NW / 8; e += 2) {
                            const uint32_t head = n0 + 8 * (e + (lane >> 4)) + (lane & 7);
                            const uint32_t dst = smb + L::P + sw128_off(head, 2 * w4 + (lane >> 3 & 1));
                            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                                         :: "r"(dst), "r"(pack_bf(x[4 * e], x[4 * e + 1])),
                                            "r"(pack_bf(x[4 * e + 2], x[4 * e + 3])),
                                            "r"(pack_bf(x[4 * e + 4], x[4 * e + 5])),
                                            "r"(pack_bf(x[4 * e + 6], x[4 * e + 7])) : "memory");
                        }
                    }
                    fence_async_smem();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full);
                }
                if (stop) break;
                // the segment's end: sums over the tokens, outputs out of tensor memory
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[v] += __shfl_xor_sync(0xffffffffu, l[v], o);
                }
                float *rd = red_w + (k & 1) * 4 * NW;
                if (lane < 4) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int at = (v >> 1) * 8 + 2 * lane + (v & 1);
                        rd[w4 * NW + at] = l[v];
                        if (w4 == 0) cb[at] = m[v];
                    }
                }
                const bool whole = w.whole();
                const int64_t slot = w.slot();
                bar_sync(bar, 128);
                if (wt < NW) {
                    float sum = rd[wt] + rd[NW + wt] + rd[2 * NW + wt] + rd[3 * NW + wt];
                    float top = cb[wt];
                    if (TREE && (pad >> wt & 1)) { sum = 0.f; top = -CUDART_INF_F; }
                    ca[wt] = whole ? inverse_of(sum) : 1.f;
                    if (whole) {
                        if (p.lse && n0 + wt < nh)
                            p.lse[(int64_t)it.b * p.H + h0 + n0 + wt] = lse_of(top, sum);
                    } else {
                        float2 *to = reinterpret_cast<float2 *>(p.stat + slot * N * 2) + n0 + wt;
                        *to = make_float2(top, sum);
                    }
                }
                ok = ok && wait_or_fail(o_full, (k - 1) & 1, fail);
                stop = bar_or(bar, 128, !ok);
                if (stop) break;
                fence_after_sync();
                for (int mb = 0; mb < 4; ++mb)
#pragma unroll
                    for (int c = 0; c < NW; c += EC) {
                        const int ch = mb * 128 + wt, n = n0 + c;          // this thread's channel
                        if (n >= nh) continue;
                        float y[EC];
                        ld_cols(tmem_at(tmem, warp, O_COL + mb * N + n), y);
                        tmem_wait_ld();
                        reg_fence(y);
                        if constexpr (TREE) {               // a padding node's queries hold anything
#pragma unroll
                            for (int e = 0; e < EC; ++e)
                                if (pad >> (c + e) & 1) y[e] = 0.f;
                        }
                        if (whole) {
                            __nv_bfloat16 *to = (__nv_bfloat16 *)p.o + ((int64_t)it.b * p.H + h0 + n) * LATENT + ch;
#pragma unroll
                            for (int e = 0; e < EC; ++e)
                                if (n + e < nh) to[e * LATENT] = __float2bfloat16_rn(y[e] * ca[c + e]);
                        } else {
                            float *to = p.part + (slot * N + n) * LATENT + ch;
#pragma unroll
                            for (int e = 0; e < EC; ++e)
                                if (n + e < nh) to[e * LATENT] = y[e];
                        }
                    }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty);
                bar_sync(bar, 128);                         // ca, cb are free again
            } while (w.next(p, share));
        }
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0) p.status[blockIdx.x] = *fail;
    if (warp == W_MMA) tmem_dealloc<TCOLS>(tmem);
}

// Heads a CTA: the fewest that hold all H, else 64 a group.
SplitPlan plan_of(int32_t H, int nsm, bool tree) { return split_plan(H, H <= 16 ? 16 : (H <= 32 ? 32 : 64), nsm, tree); }

template <int N, bool TREE>
cudaError_t run(const DecodeArgs &a, const SplitPlan &pl, cudaStream_t st) {
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(decode_kernel<N, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)Smem<N>::BYTES);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    DecParams p;
    split_params(p, a, pl);
    const uint64_t rows = (uint64_t)a.n_pages * a.page;
    const uint64_t cd[4] = {64, 8, CHUNKS, rows / 8}, cs[3] = {ROW * 2, 128, GROUP};
    const uint32_t cb[4] = {64, 8, CHUNKS, (uint32_t)(a.page < TOK ? a.page : TOK) / 8};
    const uint64_t qd[4] = {64, (uint64_t)a.H, CHUNKS, (uint64_t)a.B};
    const uint64_t qs[3] = {ROW * 2, 128, (uint64_t)a.H * ROW * 2};
    const uint32_t qb[4] = {64, N, CHUNKS, 1};
    if (!map4(&p.tm_c, a.cache, cd, cs, cb) || !map4(&p.tm_q, a.q, qd, qs, qb))
        return cudaErrorInvalidValue;
    p.force_timeout = fault_force_timeout();
    return launch_split<N, __nv_bfloat16>(decode_kernel<N, TREE>, p, pl, THREADS, Smem<N>::BYTES, a.ws, st);
}

}  // namespace

uint64_t decode_tc_workspace_bytes(int32_t H, bool tree) {
    return ws_bytes(plan_of(H, MAX_CTAS, tree));     // the most any device takes
}

cudaError_t launch_decode_tc(const DecodeArgs &a, cudaStream_t st) {
    int nsm = 1;
    const cudaError_t e = sm_count(&nsm);
    if (e != cudaSuccess) return e;
    if (nsm > MAX_CTAS) nsm = MAX_CTAS;
    const SplitPlan pl = plan_of(a.H, nsm, a.parents != nullptr);
    if (a.parents) switch (pl.N) {
    case 16: return run<16, true>(a, pl, st);
    case 32: return run<32, true>(a, pl, st);
    default: return run<64, true>(a, pl, st);
    }
    switch (pl.N) {
    case 16: return run<16, false>(a, pl, st);
    case 32: return run<32, false>(a, pl, st);
    default: return run<64, false>(a, pl, st);
    }
}

}  // namespace mla
}  // namespace kda
