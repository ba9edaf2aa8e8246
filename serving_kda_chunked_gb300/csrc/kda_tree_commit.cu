// kda_tree_commit.cu -- a KDA or Gated DeltaNet state advanced along the
// accepted path of a tree of drafted tokens (kda_tree_commit in kda.h).
//
// Per token of the path the decode step's state update:
//   S = Diag(e^g) S,  u = beta (v - S^T k),  S = S + k u^T
// The columns of S are independent.  What bounds it: S is read and written once,
// whatever the length of the path (the decode step would do so for every token):
// HBM.  A CTA owns 64 columns of a head, 16 rows x 4 columns a thread in registers; two
// warps share 32 columns and exchange one partial sum of S^T k a token.  All that a token
// needs comes to shared memory eight tokens at a time, so that no load stands in the chain
// from token to token.  Measured, 256 sequences, 32 heads, D = 128: 158 us for one token a
// sequence, 167 for two, 193 for four, 248 for eight (6.8, 6.5, 5.7, 4.5 TB/s; a decode
// step 157 each); with every token's loads a token ahead of it 161, 181, 258, 390.
#include "kda_tree.cuh"

namespace kda {
namespace tree {
namespace {

constexpr int THREADS = 128;                 // 64 columns
constexpr int AHEAD = 304;                   // CTAs
constexpr int BLOCK = 8;                     // tokens whose inputs are in shared memory at a time
static_assert(THREADS == 16 * BLOCK, "a thread brings in four of a token's 64 values");

template <int D, typename Tin>
__global__ void __launch_bounds__(THREADS, 4) commit_kernel(const CommitArgs p) {
    constexpr int ROWS = D / 8, PARTS = D / 64;             // rows a thread, CTAs a head
    __shared__ __align__(16) float sk[BLOCK][D], sa[BLOCK][D], sv[BLOCK][64];
    __shared__ float4 red[2][2][2][8];                      // [32 columns][token's parity][half]
    __shared__ float sb[BLOCK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x / PARTS, b = bh / p.H, h = bh % p.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the path, up to its first value that is no node; all warps alike
    const int32_t *path = p.path + (int64_t)b * p.T;
    const int n0 = lane < p.T ? path[lane] : -1, n1 = lane + 32 < p.T ? path[lane + 32] : -1;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) return;
    }
    const uint32_t end0 = __ballot_sync(0xffffffffu, n0 < 0 || n0 >= p.T), end1 = __ballot_sync(0xffffffffu, n1 < 0 || n1 >= p.T);
    const int n = end0 ? __ffs((int)end0) - 1 : (end1 ? 31 + __ffs((int)end1) : 64);
    if (n == 0) return;                                     // nothing accepted: the state stays as it is

    // a state that half a round of CTAs later will want, to L2: the memory goes on while
    // these here compute (batch of 256 166 us, here 159; a round ahead 158, two 164)
    if (tid == 0 && blockIdx.x % PARTS == 0) {
        const int64_t later = (int64_t)bh + AHEAD / PARTS;
        if (later < (int64_t)p.B * p.H) {
            const int b2 = (int)(later / p.H), h2 = (int)(later % p.H);
            const int64_t slot2 = p.slots ? p.slots[b2] : b2;
            const int next = p.path[(int64_t)b2 * p.T];
            if (next >= 0 && next < p.T && slot2 >= 0 && slot2 < p.P)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(p.S + (slot2 * p.H + h2) * (D * D)), "r"(D * D * 4) : "memory");
        }
    }
    // two warps share 32 columns, half the rows each
    const int half = warp & 1, rg = lane >> 3, cl = lane & 7;
    const int col = blockIdx.x % PARTS * 64 + 32 * (warp >> 1) + 4 * cl, row0 = half * (D / 2) + 4 * rg;
    float *S = p.S + (slot * p.H + h) * (D * D) + col;
    float4 s[ROWS];                                         // rows row0 + 16 i + j
#pragma unroll
    for (int i = 0; i < ROWS / 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[4 * i + j] = __ldcs(reinterpret_cast<const float4 *>(S + (row0 + 16 * i + j) * D));

    const int64_t step = (int64_t)p.H * D, at0 = (int64_t)b * p.T * step + (int64_t)h * D;
    const int64_t bt0 = (int64_t)b * p.T * p.H + h;
    const int col0 = blockIdx.x % PARTS * 64;
    auto node = [&](int t) -> int64_t {                     // t alike in all lanes, or any
        const int a = __shfl_sync(0xffffffffu, n0, t & 31), c = __shfl_sync(0xffffffffu, n1, t & 31);
        return t < 32 ? a : c;
    };
    for (int t0 = 0; t0 < n; t0 += BLOCK) {
        const int m = min(BLOCK, n - t0);
        if (t0) __syncthreads();
        // four channels a thread, all loads of the block under way together
        constexpr int EACH = BLOCK * D / 4 / THREADS;
        float4 kx[EACH], ax[EACH], vx;
        float bx = 0.f;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int t = (tid + e * THREADS) / (D / 4), c = (tid + e * THREADS) % (D / 4) * 4;
            const int64_t x = node(t0 + min(t, m - 1));
            kx[e] = load4((const Tin *)p.k + at0 + x * step + c);
            if (p.scalar_gate) ax[e].x = p.g[bt0 + x * p.H];
            else ax[e] = load4(p.g + at0 + x * step + c);
        }
        {
            const int64_t x = node(t0 + min(tid / 16, m - 1));
            vx = load4((const Tin *)p.v + at0 + x * step + col0 + tid % 16 * 4);
            if (tid % 16 == 0) bx = p.beta[bt0 + x * p.H];
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int t = (tid + e * THREADS) / (D / 4), c = (tid + e * THREADS) % (D / 4) * 4;
            store4(&sk[t][c], kx[e]);
            const float a = expf(ax[e].x);
            store4(&sa[t][c], p.scalar_gate ? make_float4(a, a, a, a) : make_float4(a, expf(ax[e].y), expf(ax[e].z), expf(ax[e].w)));
        }
        store4(&sv[tid / 16][tid % 16 * 4], vx);
        if (tid % 16 == 0) sb[tid / 16] = bx;
        __syncthreads();
        for (int t = 0; t < m; ++t) {
            const float4 now = load4(&sv[t][col - col0]);
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < ROWS / 4; ++i) {
                const float4 a = load4(&sa[t][row0 + 16 * i]), k = load4(&sk[t][row0 + 16 * i]);
                const float av[4] = {a.x, a.y, a.z, a.w}, kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 &x = s[4 * i + j];
                    x.x *= av[j]; x.y *= av[j]; x.z *= av[j]; x.w *= av[j];
                    w.x += x.x * kv[j]; w.y += x.y * kv[j]; w.z += x.z * kv[j]; w.w += x.w * kv[j];
                }
            }
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
                w.x += __shfl_xor_sync(0xffffffffu, w.x, o);
                w.y += __shfl_xor_sync(0xffffffffu, w.y, o);
                w.z += __shfl_xor_sync(0xffffffffu, w.z, o);
                w.w += __shfl_xor_sync(0xffffffffu, w.w, o);
            }
            // the other half of the rows
            float4 (*ex)[8] = red[warp >> 1][t & 1];
            if (rg == 0) ex[half][cl] = w;
            asm volatile("bar.sync %0, 64;" :: "r"(1 + (warp >> 1)) : "memory");
            const float4 w2 = ex[half ^ 1][cl];
            w.x += w2.x; w.y += w2.y; w.z += w2.z; w.w += w2.w;
            const float be = sb[t];
            const float4 u = make_float4(be * (now.x - w.x), be * (now.y - w.y), be * (now.z - w.z), be * (now.w - w.w));
#pragma unroll
            for (int i = 0; i < ROWS / 4; ++i) {
                const float4 k = load4(&sk[t][row0 + 16 * i]);
                const float kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 &x = s[4 * i + j];
                    x.x += kv[j] * u.x; x.y += kv[j] * u.y; x.z += kv[j] * u.z; x.w += kv[j] * u.w;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS / 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) __stcs(reinterpret_cast<float4 *>(S + (row0 + 16 * i + j) * D), s[4 * i + j]);
}

template <int D, typename Tin>
cudaError_t run(const CommitArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.H * (D / 64)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, commit_kernel<D, Tin>, a);
}

}  // namespace

cudaError_t launch_commit(const CommitArgs &a, cudaStream_t st) {
    if (a.d == 128) return a.dtype == 0 ? run<128, __nv_bfloat16>(a, st) : run<128, float>(a, st);
    return a.dtype == 0 ? run<64, __nv_bfloat16>(a, st) : run<64, float>(a, st);
}

}  // namespace tree
}  // namespace kda
