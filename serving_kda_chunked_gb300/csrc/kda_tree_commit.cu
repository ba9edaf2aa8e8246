// kda_tree_commit.cu -- a KDA or Gated DeltaNet state advanced along the
// accepted path of a tree of drafted tokens (kda_tree_commit in kda.h).
//
// Per token of the path the decode step's state update:
//   S = Diag(e^g) S,  u = beta (v - S^T k),  S = S + k u^T
// The columns of S are independent.  What bounds it: S is read and written once,
// whatever the length of the path (the decode step would do so for every token):
// HBM.  A warp owns 16 columns of one head, 16 rows x 4 columns a thread in
// registers, so that S^T k is a sum over 8 lanes and no two warps wait for one
// another but where the keys and gates of the next 16 tokens are brought in.
#include "kda_tree.cuh"

namespace kda {
namespace tree {
namespace {

constexpr int BLOCK = 16;                    // tokens whose keys and gates are in shared memory at a time

template <int D, typename Tin>
__global__ void __launch_bounds__(2 * D) commit_kernel(const CommitArgs p) {
    constexpr int ROWS = D / 8, THREADS = 2 * D;            // rows a thread, threads of D / 16 warps
    __shared__ __align__(16) float sk[BLOCK][D], sa[BLOCK][D];
    __shared__ float sb[MAX_NODES];
    __shared__ int node[MAX_NODES];
    __shared__ int n_path;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t *path = p.path + (int64_t)b * p.T;
    int64_t slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) return;
    }
    const int first = path[0];
    if (first < 0 || first >= p.T) return;                  // nothing accepted: the state stays as it is

    const int rg = lane >> 2, col = 16 * warp + 4 * (lane & 3);
    float *S = p.S + (slot * p.H + h) * (D * D) + col;
    float4 s[ROWS];                                         // rows 32 i + 4 rg + j
#pragma unroll
    for (int i = 0; i < ROWS / 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[4 * i + j] = __ldcs(reinterpret_cast<const float4 *>(S + (32 * i + 4 * rg + j) * D));

    const int64_t step = (int64_t)p.H * D, at0 = (int64_t)b * p.T * step + (int64_t)h * D;
    const int64_t bt0 = (int64_t)b * p.T * p.H + h;
    if (tid < MAX_NODES) {
        const int x = tid < p.T ? path[tid] : -1;
        node[tid] = x >= 0 && x < p.T ? x : -1;
        sb[tid] = node[tid] >= 0 ? p.beta[bt0 + (int64_t)x * p.H] : 0.f;
    }
    __syncthreads();
    if (tid == 0) {
        int n = 0;
        while (n < p.T && node[n] >= 0) ++n;
        n_path = n;
    }
    __syncthreads();
    const int n = n_path;
    for (int t0 = 0; t0 < n; t0 += BLOCK) {
        const int m = min(BLOCK, n - t0);
        if (t0) __syncthreads();
        for (int e = tid; e < m * D; e += THREADS) {
            const int t = e / D, c = e % D, x = node[t0 + t];
            sk[t][c] = to_f32(((const Tin *)p.k)[at0 + x * step + c]);
            sa[t][c] = expf(p.scalar_gate ? p.g[bt0 + (int64_t)x * p.H] : p.g[at0 + x * step + c]);
        }
        __syncthreads();
        float4 v = load4((const Tin *)p.v + at0 + node[t0] * step + col);
        for (int t = 0; t < m; ++t) {
            const float4 now = v;
            if (t + 1 < m) v = load4((const Tin *)p.v + at0 + node[t0 + t + 1] * step + col);
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < ROWS / 4; ++i) {
                const float4 a = load4(&sa[t][32 * i + 4 * rg]), k = load4(&sk[t][32 * i + 4 * rg]);
                const float av[4] = {a.x, a.y, a.z, a.w}, kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 &x = s[4 * i + j];
                    x.x *= av[j]; x.y *= av[j]; x.z *= av[j]; x.w *= av[j];
                    w.x += x.x * kv[j]; w.y += x.y * kv[j]; w.z += x.z * kv[j]; w.w += x.w * kv[j];
                }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                w.x += __shfl_xor_sync(0xffffffffu, w.x, o);
                w.y += __shfl_xor_sync(0xffffffffu, w.y, o);
                w.z += __shfl_xor_sync(0xffffffffu, w.z, o);
                w.w += __shfl_xor_sync(0xffffffffu, w.w, o);
            }
            const float be = sb[t0 + t];
            const float4 u = make_float4(be * (now.x - w.x), be * (now.y - w.y), be * (now.z - w.z), be * (now.w - w.w));
#pragma unroll
            for (int i = 0; i < ROWS / 4; ++i) {
                const float4 k = load4(&sk[t][32 * i + 4 * rg]);
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
        for (int j = 0; j < 4; ++j) __stcs(reinterpret_cast<float4 *>(S + (32 * i + 4 * rg + j) * D), s[4 * i + j]);
}

template <int D, typename Tin>
cudaError_t run(const CommitArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.H));
    cfg.blockDim = dim3(2 * D);
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
