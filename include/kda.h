/*
 * kda.h -- C ABI of the KDA (Kimi Delta Attention) kernels for GB300 (sm_103a).
 *
 * KDA is a gated delta-rule linear attention with a per-channel gate.  Per
 * head it keeps a fixed-size state S (dk x dv, fp32) and, for every token t:
 *
 *     S   = Diag(exp(g_t)) S                decay first, one rate per channel
 *     S   = S + beta_t k_t (v_t - S^T k_t)^T   write the delta along k_t
 *     o_t = S^T q_t                          read out with the new state
 *
 * Sources: the delta rule and the decay-then-write order are in the lineage
 * essay "Baseten 엔지니어가 분석한 7년간의 어텐션 메커니즘 진화: GPT-2부터
 * Kimi K3까지", sections "DeltaNet: 이제 메모리를 편집할 수 있습니다" and
 * "Gated DeltaNet: 이제는 '망각'할 수 있습니다"; the per-channel gate in its
 * section "KDA: Kimi의 비법" and in "KV 캐시를 75% 줄였는데 성능은 더
 * 좋아졌다", section "KDA: 지우고 다시 쓰는 메모, 채널마다 다른 망각률".
 * The chunked form of prefill follows the essay's section "병렬화 트릭"
 * (chunks of C = 64 tokens, masked attention inside a chunk, the state
 * carried between chunks, a Householder/UT reparameterisation resolving all
 * deltas of a chunk at once).
 *
 * Conventions for every entry point
 *   - All tensors are dense, row-major, contiguous, in DEVICE memory owned by
 *     the caller.  Base pointers must be 16-byte aligned.  The library never
 *     allocates, frees or retains caller memory and keeps no per-call state.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL means
 *     the legacy default stream).  Outputs are valid once the stream reaches
 *     that point.
 *   - Arguments are validated on the host before any launch, without reading
 *     device memory.  A rejected call launches nothing and returns
 *     KDA_ERR_INVALID_ARG (malformed) or KDA_ERR_UNSUPPORTED (well formed but
 *     outside the compiled shapes).  A failed launch returns KDA_ERR_CUDA; the
 *     CUDA error is cleared with cudaGetLastError so that it does not leak
 *     into the caller's later checks.  No C++ exception or abort crosses the
 *     ABI.
 *   - Work runs on the CURRENT device (cudaGetDevice); `stream` must belong to
 *     it.  Every non-NULL tensor pointer of a device entry point is checked
 *     with cudaPointerGetAttributes: memory of another device, host memory
 *     (page-locked or not) and pointers the runtime does not know are
 *     rejected with KDA_ERR_INVALID_ARG; managed memory is accepted.  With no
 *     usable device the call returns KDA_ERR_CUDA.
 *   - The library caches per-device state for the life of the process
 *     (kernel attributes, the address of the no-allocation scratch, the
 *     host-buffer entry point's streams).  Do not use it across a
 *     cudaDeviceReset of a device it has run on.
 *   - Gates g are the log of the per-channel forgetting rate alpha in (0, 1]:
 *     finite values <= 0.  beta is the write strength in [0, 1].
 */
#ifndef KDA_H
#define KDA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,  /* null pointer, misalignment, bad size       */
    KDA_ERR_UNSUPPORTED = 2,  /* head size / chunk / dtype not compiled in   */
    KDA_ERR_CUDA = 3,         /* a CUDA launch or attribute call failed      */
    KDA_ERR_TIMEOUT = 4,      /* a bounded device wait gave up (see check) */
    KDA_ERR_TOO_LARGE = 5     /* beyond the fixed scratch of the no-allocation
                                 entry point                                  */
} kda_status;

typedef enum kda_dtype {
    KDA_BF16 = 0,             /* q, k, v and o are bfloat16                  */
    KDA_FP32 = 1              /* q, k, v and o are float32                   */
} kda_dtype;

/*
 * kda_prefill_chunked -- chunked prefill over a packed batch of N sequences.
 *
 *   q, k       [T_total, H, dk]   dtype        queries, keys
 *   v          [T_total, H, dv]   dtype        values
 *   g          [T_total, H, dk]   float32      log-gate, finite, <= 0
 *   beta       [T_total, H]       float32      write strength
 *   S0         [N, H, dk, dv]     float32      initial states, or NULL (zeros)
 *   cu_seqlens [N + 1]            int32        sequence offsets: cu[0] = 0,
 *                                              non-decreasing, cu[N] = T_total
 *   o          [T_total, H, dv]   dtype        outputs (written)
 *   S_T        [N, H, dk, dv]     float32      final states (written); may be
 *                                              the same buffer as S0
 *   dk, dv     64 or 128, dk == dv
 *   chunk      64 (tokens per chunk); chunks never cross sequences and a
 *              partial last chunk is handled as if padded with no-op tokens
 *   dtype      KDA_BF16 or KDA_FP32
 *   workspace  device scratch of at least kda_prefill_workspace_size(...)
 *              bytes, 16-byte aligned, owned by the caller; may be NULL when
 *              that size is 0.  Its contents on entry do not matter; calls
 *              that share one workspace must not overlap on the GPU.
 *
 * With bf16 inputs and dk = dv = 128 the work runs on the tensor cores in two
 * kernels per window of up to 2048 chunks: one resolves every (chunk, head)
 * independently and writes its operands to the workspace, the next walks
 * each sequence's chunks in order carrying the fp32 state.  Every other case
 * (fp32 inputs, or dk = dv = 64) runs a CUDA-core kernel in fp32 arithmetic
 * that needs no workspace.
 *
 * Sequence n covers tokens [cu[n], cu[n+1]).  A sequence of length 0 copies
 * its S0 (or zeros) to S_T.  cu_seqlens lives in device memory and is not
 * read on the host; the kernels clamp every offset into [0, T_total], so
 * inconsistent offsets can only shorten sequences, never cause an
 * out-of-bounds access.  N = 0 with T_total = 0 is a valid no-op.
 */
kda_status kda_prefill_chunked(const void *q, const void *k, const void *v,
                               const float *g, const float *beta,
                               const float *S0, const int32_t *cu_seqlens,
                               int32_t N, int64_t T_total, int32_t H,
                               int32_t dk, int32_t dv, int32_t dtype,
                               int32_t chunk, void *o, float *S_T,
                               void *workspace, uint64_t workspace_bytes,
                               void *stream);

/*
 * Bytes of workspace kda_prefill_chunked needs for these sizes (0 for fp32
 * inputs).  Pure host arithmetic: no device access.  Returns 0 as well for
 * arguments that kda_prefill_chunked would reject.
 */
uint64_t kda_prefill_workspace_size(int32_t N, int64_t T_total, int32_t H,
                                    int32_t dk, int32_t dv, int32_t dtype,
                                    int32_t chunk);

/*
 * Synchronise `stream` and report the device-side status of the last
 * kda_prefill_chunked call that used `workspace`: KDA_ERR_TIMEOUT if one of
 * its kernels gave up on a bounded wait (its outputs are then incomplete: a
 * state-chain kernel that finds the per-chunk kernel of its window failed
 * writes nothing), KDA_ERR_CUDA if the stream reports an error, else KDA_OK.
 */
kda_status kda_prefill_check(const void *workspace, void *stream);

/*
 * kda_prefill_chunked_noalloc -- kda_prefill_chunked for callers that cannot
 * allocate device memory: same arguments, outputs and results, no workspace.
 * (This entry point has no counterpart in the method's description; it exists
 * for integration.)
 *
 * Some callers cannot call cudaMalloc or any allocating library routine: code
 * running while a CUDA graph is being built by someone else's allocator, a
 * host process whose device memory is owned by a framework, or plain-C
 * callers that hold only the tensors they were handed.  This variant keeps
 * its scratch in one fixed device array of kda_noalloc_scratch_bytes() bytes
 * (64 MiB) inside the library, held by every GPU that loads the library
 * until the process exits.  Long inputs are processed in as many windows of
 * chunks as that array needs; the call is rejected with KDA_ERR_TOO_LARGE
 * only when not even one chunk of all H heads (74,240 bytes each) plus a
 * header of 8 N + 268 bytes (the chunk table and the chain plan) fits.
 *
 * - The first call on a device looks up the array's device address with
 *   cudaGetSymbolAddress while that device is current; make that first call
 *   outside any stream capture.
 * - Every call on a device shares the array and leaves its contents behind;
 *   each call rewrites what it reads, so no clearing is needed, but calls that
 *   overlap on the GPU (other streams, other host threads) race on it.
 * - It calls no allocator: no cudaMalloc, cudaFree or allocating library
 *   routine.  fp32 and d = 64 inputs need no scratch at all.
 * - Its device-side status (a bounded wait that gave up) is kept in the first
 *   word of the array; kda_prefill_noalloc_check reads it.
 */
kda_status kda_prefill_chunked_noalloc(const void *q, const void *k, const void *v,
                                       const float *g, const float *beta,
                                       const float *S0, const int32_t *cu_seqlens,
                                       int32_t N, int64_t T_total, int32_t H,
                                       int32_t dk, int32_t dv, int32_t dtype,
                                       int32_t chunk, void *o, float *S_T,
                                       void *stream);

/* Size in bytes of the fixed scratch array behind the no-allocation entry. */
uint64_t kda_noalloc_scratch_bytes(void);

/*
 * kda_prefill_noalloc_check -- kda_prefill_check for the no-allocation entry
 * point: synchronise `stream`, then read the status word that the last
 * kda_prefill_chunked_noalloc call on the current device left in the fixed
 * scratch array.  KDA_ERR_TIMEOUT if one of its kernels gave up on a bounded
 * wait (its outputs were then left incomplete or untouched), KDA_ERR_CUDA if
 * the stream reports an error, else KDA_OK (also before any such call).  The
 * word is shared like the rest of the array: a no-allocation call enqueued on
 * another stream of the same device between that call and this check
 * overwrites it.  (No counterpart in the method's description.)
 */
kda_status kda_prefill_noalloc_check(void *stream);

/*
 * kda_prefill_chunked_host -- kda_prefill_chunked with the tensors in HOST
 * memory: the call copies the inputs in and the outputs out itself, and
 * overlaps those copies with the kernels.  (No counterpart in the method's
 * description; it serves callers whose activations live on the host.)
 *
 *   q, k, v, g, beta, S0, o, S_T   as kda_prefill_chunked, in host memory;
 *              page-locked memory (cudaHostAlloc, cudaHostRegister) lets the
 *              copies run asynchronously, pageable memory works but the
 *              runtime then stages each copy through the host
 *   cu_seqlens [N + 1] int32 in host memory, read by this call on the host:
 *              cu[0] = 0, non-decreasing, cu[N] = T_total, else
 *              KDA_ERR_INVALID_ARG (so T_total < 2^31)
 *   workspace  DEVICE scratch of at least kda_prefill_host_workspace_size(...)
 *              bytes, 16-byte aligned; calls sharing it must not overlap
 *
 * The token range is cut into pieces of about T_total / 6 tokens (at least
 * 512, at most 16,384) that halve toward the end of the call (down to 256
 * tokens), every cut on a 64-token chunk boundary of the sequence it falls
 * in.  Each piece is copied into one of two device staging slots,
 * runs as a packed prefill over the sequences it overlaps (their states
 * carried in a device state buffer in the workspace, exactly as the state
 * crosses windows inside one kda_prefill_chunked call), and its outputs are
 * copied back while the next piece is copied in and computed.  The results
 * equal those of kda_prefill_chunked on the same values.
 *
 * The copies run on two internal streams per device (created, with their
 * events, on the first call on that device and kept until the process ends);
 * the call is ordered after earlier work on `stream`, and `stream` reaches
 * its end only after the last copy into o and S_T.  Host buffers must stay
 * valid and unchanged (outputs: unread) until then.  Calls from several host
 * threads on one device are serialised while they enqueue; calls on different
 * devices are not.  With pageable (not page-locked) buffers each copy runs
 * synchronously with respect to the host, so the pieces no longer overlap
 * their copies with the kernels and the call takes about as long as its
 * copies plus its kernels in series.  kda_prefill_check(workspace,
 * stream) reports the device-side status of every piece.  Pointers that the
 * runtime identifies as device memory in place of a host buffer (or host
 * memory, or another device's memory, as the workspace) are rejected with
 * KDA_ERR_INVALID_ARG.  The call runs on the current device.
 */
kda_status kda_prefill_chunked_host(const void *q, const void *k, const void *v,
                                    const float *g, const float *beta,
                                    const float *S0, const int32_t *cu_seqlens,
                                    int32_t N, int64_t T_total, int32_t H,
                                    int32_t dk, int32_t dv, int32_t dtype,
                                    int32_t chunk, void *o, float *S_T,
                                    void *workspace, uint64_t workspace_bytes,
                                    void *stream);

/*
 * Bytes of device workspace kda_prefill_chunked_host needs for these sizes
 * (staging for two pieces, the prefill scratch of one piece, the N states and
 * the offsets).  Pure host arithmetic; 0 for arguments the call would reject
 * on their sizes alone (and for N = 0, which needs none).
 */
uint64_t kda_prefill_host_workspace_size(int32_t N, int64_t T_total, int32_t H,
                                         int32_t dk, int32_t dv, int32_t dtype,
                                         int32_t chunk);

/*
 * kda_decode_step -- one token for each of B independent sequences; the
 * states are updated in place.
 *
 *   q, k       [B, H, dk]         dtype
 *   v          [B, H, dv]         dtype
 *   g          [B, H, dk]         float32      log-gate, finite, <= 0
 *   beta       [B, H]             float32
 *   S          [B, H, dk, dv]     float32      read, then overwritten with S'
 *   o          [B, H, dv]         dtype        outputs (written)
 *   dk, dv     64 or 128, dk == dv
 *
 * The essay's section "KV 캐시: 재계산하지 말고 저장하라" notes that decode
 * is bound by memory bandwidth, not arithmetic: this kernel streams each
 * state from HBM once and writes it back once.  B = 0 is a valid no-op.
 * S must not overlap any input or output.
 */
kda_status kda_decode_step(const void *q, const void *k, const void *v,
                           const float *g, const float *beta, float *S,
                           int32_t B, int32_t H, int32_t dk, int32_t dv,
                           int32_t dtype, void *o, void *stream);

/*
 * kda_decode_step_pooled -- one decode token for each of B sequences whose
 * states live in a shared pool of P slots; slot slots[b] holds the state of
 * sequence b and is updated in place.
 *
 *   q, k       [B, H, dk]         dtype
 *   v          [B, H, dv]         dtype
 *   g          [B, H, dk]         float32      log-gate, finite, <= 0
 *   beta       [B, H]             float32
 *   S_pool     [P, H, dk, dv]     float32      slots named in `slots` are
 *                                              read and overwritten
 *   slots      [B]                int32        device memory; a value outside
 *                                              [0, P) skips that sequence:
 *                                              its o row is zeroed and no
 *                                              state is touched
 *   o          [B, H, dv]         dtype
 *
 * This is the serving form of decode: a KDA state has a fixed size however
 * long the context (the essay's section "선형 어텐션 (Linear Attention):
 * 고정된 크기의 메모리"), so concurrent sessions can each own one slot of a
 * preallocated pool instead of a growing KV cache (the explainer's section
 * "한국 개발자에게 주는 시사점": the number of concurrent requests is set
 * by how much cache memory is left).  The slots of the non-skipped sequences
 * must be distinct (two sequences in one slot race).  Slot values are not
 * read on the host.  B = 0 is a valid no-op.
 */
kda_status kda_decode_step_pooled(const void *q, const void *k, const void *v,
                                  const float *g, const float *beta, float *S_pool,
                                  const int32_t *slots, int32_t P, int32_t B, int32_t H,
                                  int32_t dk, int32_t dv, int32_t dtype, void *o,
                                  void *stream);

/*
 * kda_gdn_prefill_chunked, kda_gdn_decode_step -- the same two operations for
 * Gated DeltaNet, whose gate is one scalar per head and token instead of one
 * rate per channel.  The lineage essay's section "Gated DeltaNet: 이제는
 * '망각'할 수 있습니다" gives its update (decay the old memory by alpha, then
 * write the delta along k); its section "KDA: Kimi의 비법" states that KDA
 * differs from it only in turning that scalar alpha into a per-channel
 * vector.  So a Gated DeltaNet head is a KDA head whose dk gates are all equal,
 * and these entry points run the KDA kernels reading one gate per head:
 *
 *   g   [T_total, H]   (prefill)   or   [B, H]   (decode)   float32, log of
 *       alpha, finite, <= 0; 4-byte alignment suffices.
 *
 * Every other argument, the workspace (kda_prefill_workspace_size gives its
 * size here too), the outputs, the status codes and kda_prefill_check are as
 * for kda_prefill_chunked and kda_decode_step.
 */
kda_status kda_gdn_prefill_chunked(const void *q, const void *k, const void *v,
                                   const float *g, const float *beta,
                                   const float *S0, const int32_t *cu_seqlens,
                                   int32_t N, int64_t T_total, int32_t H,
                                   int32_t dk, int32_t dv, int32_t dtype,
                                   int32_t chunk, void *o, float *S_T,
                                   void *workspace, uint64_t workspace_bytes,
                                   void *stream);

kda_status kda_gdn_decode_step(const void *q, const void *k, const void *v,
                               const float *g, const float *beta, float *S,
                               int32_t B, int32_t H, int32_t dk, int32_t dv,
                               int32_t dtype, void *o, void *stream);

/* Gated DeltaNet decode over a state-slot pool: kda_decode_step_pooled with
 * one log-gate per head, g [B, H] float32 (4-byte alignment suffices). */
kda_status kda_gdn_decode_step_pooled(const void *q, const void *k, const void *v,
                                      const float *g, const float *beta, float *S_pool,
                                      const int32_t *slots, int32_t P, int32_t B, int32_t H,
                                      int32_t dk, int32_t dv, int32_t dtype, void *o,
                                      void *stream);

/*
 * Latent attention: the full-attention layers that hybrid models interleave
 * with KDA layers (the lineage essay's and the explainer's 3 : 1 hybrid).
 * Keys and values of all H heads come from one latent vector per token (512
 * values) and one position key per token (64 values) that the heads share.
 * Per head h, with c_j the latent and r_j the position key of token j:
 *
 *     k_jh = [ c_j W_K,h (128 values) ; r_j (64) ],   v_jh = c_j W_V,h (128)
 *     s_ij = scale q_ih . k_jh,   o_ih = sum_j softmax_j(s_ij) v_jh
 *
 * Three operators, for the two forms that give the same result:
 *   - kda_mla_append puts each token's [c ; r] into a paged cache and applies
 *     the position rotation to r (and to the queries' position parts) on the
 *     way;
 *   - kda_mla_prefill is the expanded form, for prompts: k and v of every head
 *     have been multiplied out;
 *   - kda_mla_decode is the absorbed form, for single tokens: W_K has been
 *     multiplied into the query (q W_K^T, 512 values) and W_V is applied to the
 *     output afterwards, so that the kernel reads only the latent cache:
 *         s_j = scale q . [c_j ; r_j],   o = sum_j softmax_j(s_j) c_j.
 * The products with W_K and W_V are the caller's (plain matrix products).
 *
 * Conventions in addition to those at the top of this file
 *   - dtype is that of every tensor that is not stated to be float32 or int32.
 *   - The cache is [n_pages, page, 576]: a row is the latent (512) followed by
 *     the position key (64); page is 16, 32, 64 or 128 tokens.  Cache slot s
 *     is row s % page of page s / page.
 *   - Scores, softmax statistics and sums are float32.  bf16 weights of the
 *     softmax are rounded to bf16 where they meet the bf16 values; the
 *     normalisation uses the float32 sum.
 *   - lse is the natural logarithm of the sum of exp(s), float32; it lets a
 *     caller merge results over parts of the keys.  A query that sees no key
 *     gets o = 0 and lse = -inf.
 *   - Inputs that a query can see are finite.  Where it sees a NaN, or one of its
 *     scores is +infinity in float32, its o and lse are NaN.  What it cannot see by length
 *     or by sequence (cache rows behind a length, other sequences' tokens)
 *     may hold anything, infinities and NaN included.
 */

/*
 * kda_mla_append -- write T tokens to the paged latent cache, rotating their
 * position keys and (optionally) their queries' position parts.
 *
 *   c          [T, 512]      latents; row stride c_stride elements
 *   k_r        [T, 64]       position keys; row stride k_r_stride
 *   slots      [T]           int32, cache slot of each token; a value outside
 *                            [0, n_pages * page) leaves the cache untouched
 *                            (padding tokens); the others must be distinct
 *   positions  [T]           int32, row of `rope` per token, clamped into
 *                            [0, max_pos); NULL when rope is
 *   rope       [max_pos, 64] float32: cosines of the 32 pairs' angles, then
 *                            their sines; NULL: no rotation (layers without
 *                            position rotation)
 *   interleaved  pairs are (2i, 2i + 1) if nonzero, else (i, i + 32)
 *   cache      [n_pages, page, 576]  written at `slots`
 *   k_out      [T, 64]       rotated position keys, row stride k_out_stride,
 *                            or NULL; may be k_r itself
 *   q_r        [T, H, 64]    the queries' position parts, or NULL; element
 *                            strides q_token_stride and q_head_stride
 *   q_out      [T, H, 64]    rotated, with its own strides; NULL exactly when
 *                            q_r is; may be q_r itself (same strides)
 *
 * (a, b) -> (a cos - b sin, a sin + b cos) in float32, rounded once.  Strides
 * are multiples of 16 bytes (so that views of a projection's output can be
 * passed as they are); those of k_out and q_out keep the rows of 64 apart
 * (strides that make them overlap are rejected).  T = 0 is a valid no-op.
 * Outputs must not overlap inputs otherwise.
 */
kda_status kda_mla_append(const void *c, int64_t c_stride, const void *k_r,
                          int64_t k_r_stride, const int32_t *slots,
                          const int32_t *positions, const float *rope,
                          int32_t max_pos, int32_t interleaved, int64_t T,
                          void *cache, int32_t n_pages, int32_t page,
                          int32_t latent, int32_t rope_dim, int32_t dtype,
                          void *k_out, int64_t k_out_stride, const void *q_r,
                          int64_t q_token_stride, int64_t q_head_stride,
                          int32_t H, void *q_out, int64_t qo_token_stride,
                          int64_t qo_head_stride, void *stream);

/*
 * kda_mla_prefill -- the expanded form over a packed batch of N sequences.
 *
 *   q          [Tq, H, 192]  queries: 128 values that meet the latent's key,
 *                            then the 64 that meet the position key (rotated)
 *   kv         [Tk, H, 256]  the latents multiplied out: key (128), value (128)
 *   k_r        [Tk, 64]      position keys (rotated), shared by the heads
 *   cu_q, cu_k [N + 1]       int32 device offsets of the sequences' queries
 *                            and keys, as cu_seqlens of kda_prefill_chunked
 *                            (clamped into [0, Tq] and [0, Tk])
 *   scale      finite factor of the scores
 *   causal     if nonzero, the queries are the last of the keys' tokens: query
 *              i of nq sees key j of nk when j <= i + nk - nq (none when that
 *              is negative); else every query sees all nk keys
 *   o          [Tq, H, 128]  outputs (written)
 *   lse        [Tq, H]       float32 (written), or NULL
 *   workspace  device scratch of kda_mla_prefill_workspace_size(N, Tq, H,
 *              dtype) bytes, 16-byte aligned; may be NULL when that is 0.  One
 *              that is passed all the same takes the call's status (its first
 *              4 bytes, if it has them) and is otherwise left alone
 *
 * bf16 runs on the tensor cores, fp32 on the CUDA cores.  Calls that share a
 * workspace must not overlap on the GPU.  Tokens outside every [cu_q[n],
 * cu_q[n + 1]) are not written.
 */
kda_status kda_mla_prefill(const void *q, const void *kv, const void *k_r,
                           const int32_t *cu_q, const int32_t *cu_k, int32_t N,
                           int64_t Tq, int64_t Tk, int32_t H, int32_t nope,
                           int32_t rope_dim, int32_t dv, int32_t dtype,
                           float scale, int32_t causal, void *o, float *lse,
                           void *workspace, uint64_t workspace_bytes,
                           void *stream);

/* Bytes of workspace kda_mla_prefill needs (0: none).  Host arithmetic. */
uint64_t kda_mla_prefill_workspace_size(int32_t N, int64_t Tq, int32_t H,
                                        int32_t dtype);

/*
 * kda_mla_decode -- the absorbed form: one query token for each of B
 * sequences over the paged latent cache.
 *
 *   q          [B, H, 576]   queries: 512 values that meet the latent (W_K
 *                            multiplied in), then the 64 position values
 *   cache      [n_pages, page, 576]
 *   table      [B, max_pages] int32: page of tokens page*i .. page*i + page-1
 *                            of sequence b; a value outside [0, n_pages) hides
 *                            those tokens
 *   seq_lens   [B]           int32, tokens cached per sequence (the new one
 *                            included), clamped into [0, max_pages * page]
 *   scale      finite factor of the scores (that of the expanded form)
 *   o          [B, H, 512]   outputs over the latents (written)
 *   lse        [B, H]        float32 (written), or NULL
 *   workspace  device scratch of kda_mla_decode_workspace_size(B, H, dtype)
 *              bytes, 16-byte aligned; its contents on entry do not matter
 *
 * Neither the table nor the lengths are read on the host.  The tokens of all
 * sequences are shared out evenly over the SMs, whatever the lengths; a
 * sequence that several SMs worked on is joined by a second kernel.  Results
 * do not depend on timing: equal inputs give equal bits.  B = 0 is a valid
 * no-op.  Calls that share a workspace must not overlap on the GPU.
 */
kda_status kda_mla_decode(const void *q, const void *cache, const int32_t *table,
                          const int32_t *seq_lens, int32_t B, int32_t H,
                          int32_t n_pages, int32_t page, int32_t max_pages,
                          int32_t latent, int32_t rope_dim, int32_t dtype,
                          float scale, void *o, float *lse, void *workspace,
                          uint64_t workspace_bytes, void *stream);

/* Bytes of workspace kda_mla_decode needs.  Host arithmetic. */
uint64_t kda_mla_decode_workspace_size(int32_t B, int32_t H, int32_t dtype);

/*
 * kda_prefill_check for kda_mla_prefill and kda_mla_decode: synchronise
 * `stream` and report the device-side status of the last call that used
 * `workspace` (KDA_ERR_TIMEOUT: a bounded wait gave up and outputs are
 * incomplete).  Every call that launches something and was passed a workspace of
 * 4 bytes or more writes its status there, whether or not it needs the
 * workspace; the no-ops (Tq = 0, B = 0) leave it as it was.  A NULL workspace
 * (a call that needed none) reports the stream's status only.
 */
kda_status kda_mla_check(const void *workspace, void *stream);

/* Human-readable name of a status code (static storage; never NULL). */
const char *kda_status_string(int32_t status);

/* ABI version of this library: (major << 16) | minor. */
int32_t kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
