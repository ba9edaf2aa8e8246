// kda_mla_append.cu -- tokens into the paged latent cache, with the position
// rotation of their keys and queries on the way (kda_mla_append in kda.h).
//
// Nothing is reused, so HBM bandwidth bounds it: per token the latent, the
// position key and H query parts are read once and written once (10.9 KB at
// H = 32 in bf16).  One block per token; a thread moves 32 bytes at a time:
// two 16-byte pieces that hold whole rotation pairs, so that every piece is
// loaded before it is stored by the same thread, which makes in-place
// rotation safe.
#include "kda_mla.cuh"

namespace kda {
namespace mla {
namespace {

// 16 bytes of elements as floats, and back
template <typename T> struct Piece;
template <> struct Piece<float> {
    static constexpr int E = 4;
    float v[E];
    __device__ __forceinline__ void load(const float *p) {
        const float4 x = load4(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    __device__ __forceinline__ void store(float *p) const {
        store4(p, make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int E = 8;
    float v[E];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint4 raw = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
            v[2 * i] = f.x; v[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Rotation unit u of a 64-value vector: 2E values whose pairs have the angles
// E u .. E u + E - 1.  Half-split pairs: piece a at E u, piece b 32 further on;
// interleaved: one run of 2E values.
template <typename T>
__device__ __forceinline__ void rotate_unit(const T *src, T *dst, T *dst2, int u,
                                            const float *cs, bool interleaved) {
    constexpr int E = Piece<T>::E;
    const int ia = interleaved ? 2 * E * u : E * u;
    const int ib = interleaved ? ia + E : ia + ROPE / 2;
    Piece<T> a, b;
    a.load(src + ia);
    b.load(src + ib);
    if (cs) {
        float c[E], s[E];
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 x = load4(cs + E * u + i), y = load4(cs + ROPE / 2 + E * u + i);
            c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
            s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
        }
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float x0 = a.v[2 * i], y0 = a.v[2 * i + 1];
                a.v[2 * i] = x0 * c[i] - y0 * s[i];
                a.v[2 * i + 1] = x0 * s[i] + y0 * c[i];
                const float x1 = b.v[2 * i], y1 = b.v[2 * i + 1];
                b.v[2 * i] = x1 * c[i + E / 2] - y1 * s[i + E / 2];
                b.v[2 * i + 1] = x1 * s[i + E / 2] + y1 * c[i + E / 2];
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = a.v[i], y = b.v[i];
                a.v[i] = x * c[i] - y * s[i];
                b.v[i] = x * s[i] + y * c[i];
            }
        }
    }
    if (dst) { a.store(dst + ia); b.store(dst + ib); }
    if (dst2) { a.store(dst2 + ia); b.store(dst2 + ib); }
}

template <typename T>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs p) {
    constexpr int E = Piece<T>::E;
    constexpr int UV = ROPE / (2 * E);              // rotation units of a vector
    constexpr int LU = LATENT / (2 * E);            // 32-byte units of the latent
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int64_t slot = p.slots[t];
    const bool put = slot >= 0 && slot < p.n_slots;
    const float *cs = nullptr;
    if (p.rope) {
        int pos = p.positions[t];
        pos = pos < 0 ? 0 : (pos >= p.max_pos ? p.max_pos - 1 : pos);
        cs = p.rope + (int64_t)pos * ROPE;
    }
    T *row = put ? (T *)p.cache + slot * ROW : nullptr;
    const int nq = p.q_r ? p.H * UV : 0;
    for (int i = threadIdx.x; i < LU + UV + nq; i += blockDim.x) {
        if (i < LU) {
            if (put) {
                const uint4 *src = (const uint4 *)((const T *)p.c + t * p.c_stride) + 2 * i;
                const uint4 a = src[0], b = src[1];
                uint4 *dst = (uint4 *)row + 2 * i;
                dst[0] = a;
                dst[1] = b;
            }
        } else if (i < LU + UV) {
            T *ko = p.k_out ? (T *)p.k_out + t * p.k_out_stride : nullptr;
            rotate_unit<T>((const T *)p.k_r + t * p.k_r_stride, put ? row + LATENT : nullptr, ko,
                           i - LU, cs, p.interleaved);
        } else {
            const int j = i - LU - UV, h = j / UV, u = j % UV;
            rotate_unit<T>((const T *)p.q_r + t * p.q_token_stride + h * p.q_head_stride,
                           (T *)p.q_out + t * p.qo_token_stride + h * p.qo_head_stride, (T *)nullptr,
                           u, cs, p.interleaved);
        }
    }
}

template <typename T>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
    constexpr int UNITS = (LATENT + ROPE) / (2 * Piece<T>::E);
    const int64_t items = UNITS + (a.q_r ? (int64_t)a.H * (ROPE / (2 * Piece<T>::E)) : 0);
    const int threads = items >= 256 ? 256 : (int)((items + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel<T>, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
    return a.dtype == 0 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace mla
}  // namespace kda
