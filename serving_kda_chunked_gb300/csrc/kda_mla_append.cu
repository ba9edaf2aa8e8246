// kda_mla_append.cu -- tokens into the paged latent cache, with the position
// rotation of their keys and queries on the way (kda_mla_append in kda.h).
//
// Nothing is reused, so HBM bandwidth bounds it: per token the latent, the
// position key and H query parts are read once and written once (10.9 KB at
// H = 32 in bf16).  A thread moves 32 bytes at a time: two 16-byte pieces that
// hold whole rotation pairs, loaded before either is stored by the same thread,
// which makes in-place rotation safe.  The queries' parts are 128-byte pieces
// of longer rows on both sides, so the memory sees no long runs: 65,536 tokens
// take 156 us = 4.57 TB/s (138 us = 5.2 TB/s where both sides are dense).
// Measured and rejected: two or four tokens or heads a thread at a time (168 to
// 300 us and 162 to 174 us), 16-byte units with the pair's other half fetched
// from a neighbouring lane (177 us), registers cut to 40 (216 us).
#include "kda_mla.cuh"

namespace kda {
namespace mla {
namespace {

// 16 bytes of elements as floats, and back
template <typename T> struct Piece;
template <> struct Piece<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&v)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
            v[2 * i] = f.x; v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Rotates the E pairs of two 16-byte pieces: half-split pairs (a[i], b[i]), or
// neighbours of one run a ‖ b.
template <typename T>
__device__ __forceinline__ void rotate(uint4 &ra, uint4 &rb, const float *cs, bool interleaved) {
    constexpr int E = Piece<T>::E;
    float a[E], b[E], c[E], s[E];
    Piece<T>::unpack(ra, a);
    Piece<T>::unpack(rb, b);
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        const float4 x = load4(cs + i), y = load4(cs + ROPE / 2 + i);
        c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
        s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
    }
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float x0 = a[2 * i], y0 = a[2 * i + 1], x1 = b[2 * i], y1 = b[2 * i + 1];
            a[2 * i] = x0 * c[i] - y0 * s[i];
            a[2 * i + 1] = x0 * s[i] + y0 * c[i];
            b[2 * i] = x1 * c[i + E / 2] - y1 * s[i + E / 2];
            b[2 * i + 1] = x1 * s[i + E / 2] + y1 * c[i + E / 2];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * c[i] - y * s[i];
            b[i] = x * s[i] + y * c[i];
        }
    }
    ra = Piece<T>::pack(a);
    rb = Piece<T>::pack(b);
}

// A thread moves one unit (32 bytes of the latent, of the position key or of
// one query) of every gridDim.x th token; the loads of its next token are under
// way while it rotates and stores this one.
template <typename T>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs p) {
    constexpr int E = Piece<T>::E;
    constexpr int UV = ROPE / (2 * E);              // rotation units of a vector
    constexpr int LU = LATENT / (2 * E);            // units of the latent
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int i = blockIdx.y * blockDim.x + threadIdx.x;
    if (i >= LU + UV + (p.q_r ? p.H * UV : 0)) return;
    // source and destination of the unit for token 0, and their token strides
    const T *src;
    T *dst = nullptr;
    int64_t step, dstep = 0;
    int u = 0, ia = 0, ib = E, row = -1;            // row: offset in the cache row
    if (i < LU) {
        src = (const T *)p.c + 2 * E * i;
        step = p.c_stride;
        row = 2 * E * i;
    } else {
        const bool key = i < LU + UV;
        const int j = i - LU - (key ? 0 : UV), h = j / UV;
        u = j % UV;
        ia = p.interleaved ? 2 * E * u : E * u;
        ib = p.interleaved ? ia + E : ia + ROPE / 2;
        if (key) {
            src = (const T *)p.k_r;
            step = p.k_r_stride;
            row = LATENT;
            if (p.k_out) { dst = (T *)p.k_out; dstep = p.k_out_stride; }
        } else {
            src = (const T *)p.q_r + h * p.q_head_stride;
            step = p.q_token_stride;
            dst = (T *)p.q_out + h * p.qo_head_stride;
            dstep = p.qo_token_stride;
        }
    }
    const bool turn = p.rope && i >= LU;
    struct Unit { uint4 a, b; int slot, pos; };
    auto fetch = [&](Unit &x, int64_t t) {
        if (t >= p.T) return;
        const T *s = src + t * step;
        x.a = __ldcs(reinterpret_cast<const uint4 *>(s + ia));
        x.b = __ldcs(reinterpret_cast<const uint4 *>(s + ib));
        if (row >= 0) x.slot = p.slots[t];
        if (turn) x.pos = p.positions[t];
    };
    Unit x, y;
    int64_t t = blockIdx.x;
    fetch(x, t);
    for (; t < p.T; t += gridDim.x, x = y) {
        fetch(y, t + gridDim.x);
        if (turn) {
            const int pos = x.pos < 0 ? 0 : (x.pos >= p.max_pos ? p.max_pos - 1 : x.pos);
            rotate<T>(x.a, x.b, p.rope + (int64_t)pos * ROPE + E * u, p.interleaved);
        }
        if (row >= 0 && x.slot >= 0 && x.slot < p.n_slots) {
            T *to = (T *)p.cache + (int64_t)x.slot * ROW + row;
            *reinterpret_cast<uint4 *>(to + ia) = x.a;
            *reinterpret_cast<uint4 *>(to + ib) = x.b;
        }
        if (dst) {
            T *to = dst + t * dstep;
            *reinterpret_cast<uint4 *>(to + ia) = x.a;
            *reinterpret_cast<uint4 *>(to + ib) = x.b;
        }
    }
}

template <typename T>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
    int nsm = 1;
    const cudaError_t e = sm_count(&nsm);
    if (e != cudaSuccess) return e;
    constexpr int UNITS = (LATENT + ROPE) / (2 * Piece<T>::E);
    const int64_t items = UNITS + (a.q_r ? (int64_t)a.H * (ROPE / (2 * Piece<T>::E)) : 0);
    const int64_t chunks = (items + 255) / 256;
    if (chunks > 65535) return cudaErrorInvalidValue;
    const int threads = (int)((items + chunks - 1) / chunks + 31) / 32 * 32;
    // up to 6144 threads an SM, about five times what is resident: 65,536 tokens
    // of 32 heads take 166 us with a grid of 1536 threads an SM, 156 us with
    // this one, 171 us with a block per token
    int64_t blocks = (int64_t)nsm * 6144 / (threads * chunks);
    blocks = blocks < 1 ? 1 : (blocks < a.T ? blocks : a.T);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)chunks);
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
