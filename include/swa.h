/*
 * swa.h - C ABI of libswa.so: sliding-window attention (SWA) with grouped-query
 * attention (GQA) over a rolling-buffer KV cache, on NVIDIA B200 (sm_100a).
 *
 * The operations follow Mistral 7B, section 2 "Architectural details":
 *   - Sliding Window Attention (paragraph, Figure 1): query position i attends
 *     to key positions j with i - W < j <= i (at most W of them).
 *   - Rolling Buffer Cache (paragraph, Figure 2): a cache of W slots per
 *     sequence and kv head; the key/value of position i live in slot i mod W.
 *   - Pre-fill and Chunking (paragraph, Figure 3): a prompt is fed in chunks of
 *     at most W tokens; each chunk attends to the cache and, causally, to itself.
 *   - Grouped-query attention (section 1): Hq / Hkv query heads share one kv
 *     head; query head h reads kv head h / (Hq / Hkv).
 *
 * Conventions for every entry point
 *   - Every tensor pointer is a DEVICE pointer owned by the caller.  The library
 *     allocates no device memory and keeps no pointer after the call returns.
 *   - Tensors are dense, row-major (last index fastest), with no padding
 *     between rows; the layouts below give the index order.  bf16 means IEEE
 *     bfloat16 (torch.bfloat16).  Base pointers must be 16-byte aligned.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *     enqueued asynchronously on it; no call synchronises the host.  Calls on
 *     one stream run in issue order.
 *   - Return value: SWA_OK, or an error code below with a message available
 *     from swa_last_error() (thread-local).  Argument errors are detected on
 *     the host before anything is launched, and then nothing is enqueued.
 *   - Integer per-sequence arguments (start_pos, n_tokens, pos) live in device
 *     memory so that calls can be captured in CUDA graphs; values the kernels
 *     find invalid there (negative positions, n_tokens > max_tokens) make the
 *     kernels skip that sequence and raise SWA_ERR_DEVICE_ARG in the device
 *     status word (swa_device_status).
 *   - Cache slots never written must hold finite values (allocate the caches
 *     zeroed): kernels read whole tiles and mask, and a NaN in a masked slot
 *     would still reach the output through 0 * NaN.
 */
#ifndef SWA_H_
#define SWA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SWA_API __attribute__((visibility("default")))
#else
#define SWA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define SWA_OK                      0
#define SWA_ERR_INVALID_ARG         1  /* null pointer, bad size, misalignment   */
#define SWA_ERR_UNSUPPORTED         2  /* head_dim not in {16,64,128}, Hq % Hkv  */
#define SWA_ERR_WORKSPACE_TOO_SMALL 3  /* swa_decode workspace below the minimum  */
#define SWA_ERR_CUDA                4  /* CUDA launch / driver error              */
#define SWA_ERR_TIMEOUT             5  /* a bounded device wait ran out           */
#define SWA_ERR_DEVICE_ARG          6  /* device-side argument out of range       */

/* Output element types. */
#define SWA_DTYPE_BF16 0
#define SWA_DTYPE_F32  1

/* Shape of one attention layer. */
typedef struct swa_dims {
    int32_t batch;       /* B: sequences                                        */
    int32_t n_q_heads;   /* Hq: query heads                                     */
    int32_t n_kv_heads;  /* Hkv: key/value heads, Hq % Hkv == 0 (G = Hq / Hkv)  */
    int32_t head_dim;    /* d: 16, 64 or 128                                    */
    int32_t window;      /* W >= 1: window length = cache slots per (seq, kv head) */
    float   scale;       /* multiplier on q.k before the softmax (e.g. 1/sqrt(d)) */
    int32_t out_dtype;   /* SWA_DTYPE_BF16 or SWA_DTYPE_F32                     */
} swa_dims;

/*
 * swa_cache_append - write a chunk's keys and values into the rolling cache.
 * Rolling Buffer Cache paragraph and Figure 2: position p goes to slot p mod W,
 * overwriting the position p - W that was there.
 *
 *   k_cache, v_cache  [B][Hkv][W][d] bf16, updated in place
 *   k, v              [B][max_tokens][Hkv][d] bf16: row t of sequence b is the
 *                     token at position start_pos[b] + t
 *   max_tokens        row capacity of k / v, 1 <= max_tokens <= W, and
 *                     max_tokens * Hkv * d / 8 < 2^31 (else SWA_ERR_UNSUPPORTED)
 *   start_pos         device int32[B], >= 0
 *   n_tokens          device int32[B], 0 <= n_tokens[b] <= max_tokens: rows
 *                     [0, n_tokens[b]) are written, the rest ignored
 * Because max_tokens <= W, no two rows of one call share a slot.
 * Must be issued after swa_prefill_chunk of the same chunk (which reads the
 * cache as it was before the chunk).
 */
SWA_API int swa_cache_append(const swa_dims* dims, void* k_cache, void* v_cache,
                     const void* k, const void* v, int32_t max_tokens,
                     const int32_t* start_pos, const int32_t* n_tokens, void* stream);

/*
 * swa_prefill_workspace_size - bytes of device scratch swa_prefill_chunk may
 * use for these dims and this max_tokens: per-row partial results of query
 * tiles whose key range is split across CTAs, and the work and merge counters.
 * Depends only on its arguments.  Returns 0 for invalid arguments.
 */
SWA_API size_t swa_prefill_workspace_size(const swa_dims* dims, int32_t max_tokens);

/*
 * swa_prefill_chunk - attention of one prefill chunk (Pre-fill and Chunking
 * paragraph, Figure 3).  Query row t of sequence b sits at position
 * i = start_pos[b] + t and attends to
 *   - the cache as it was before this chunk: the positions in
 *     [max(0, i - W + 1), start_pos[b]) it holds, and
 *   - the chunk itself, causally: rows u <= t.
 *
 *   out               [B][max_tokens][Hq][d], bf16 or f32 per dims->out_dtype;
 *                     rows t >= n_tokens[b] are not written
 *   q                 [B][max_tokens][Hq][d] bf16
 *   k, v              [B][max_tokens][Hkv][d] bf16 (the chunk's own keys/values);
 *                     rows [n_tokens[b], max_tokens) must hold finite values
 *                     (they are loaded with their tile and masked, and a NaN
 *                     there would reach the output through 0 * NaN)
 *   max_tokens        1 <= max_tokens <= W
 *   k_cache, v_cache  [B][Hkv][W][d] bf16, read only; slots must hold the
 *                     positions earlier appends put there.  A sequence whose
 *                     start_pos is 0 reads nothing from them.
 *   start_pos, n_tokens  device int32[B], as in swa_cache_append
 *   workspace         NULL (with workspace_bytes 0), or device scratch of at
 *                     least swa_prefill_workspace_size(dims, max_tokens) bytes,
 *                     16-byte aligned, ZERO-FILLED before its first use (every
 *                     call leaves it zero-filled again, so this is needed once).
 *                     With a workspace the kernel runs one CTA per SM that
 *                     takes query tiles from a shared counter and splits the
 *                     key ranges of the last tiles across CTAs (their partial
 *                     softmax results are merged by log-sum-exp); without one
 *                     it launches one CTA per query tile and head pair.  The
 *                     results agree within rounding.  Calls that may overlap
 *                     on the GPU need separate workspaces.
 * The softmax is computed in fp32 from bf16 q.k products accumulated in fp32;
 * the probabilities are rounded to bf16 for the P.V product.
 */
SWA_API int swa_prefill_chunk(const swa_dims* dims, void* out, const void* q, const void* k,
                      const void* v, int32_t max_tokens, const void* k_cache,
                      const void* v_cache, const int32_t* start_pos,
                      const int32_t* n_tokens, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * swa_decode_workspace_size - bytes of device scratch swa_decode may use for
 * these dims (fp32 partial results of a split cache sweep).  Depends only on
 * dims.  Some dims use none of it (one split per sequence and kv head, or
 * splits merged inside a thread-block cluster); the size is still reported so
 * that it stays a function of the dims.  Returns 0 for invalid dims.
 */
SWA_API size_t swa_decode_workspace_size(const swa_dims* dims);

/*
 * swa_decode_launch_info - how swa_decode runs for these dims, for callers
 * that count kernels (CUDA graphs, profilers).  Host only; enqueues nothing.
 *   n_splits    receives the number of parts the W slots of one (sequence,
 *               kv head) are split into (one CTA each)
 *   n_launches  receives the number of kernels one swa_decode call launches:
 *               1, or 2 when a combine kernel merges per-split partials
 * Either pointer may be NULL.  Returns SWA_OK, or the same codes as
 * swa_decode for invalid dims.
 */
SWA_API int swa_decode_launch_info(const swa_dims* dims, int32_t* n_splits, int32_t* n_launches);

/*
 * swa_decode - one generated token per sequence (token-by-token generation,
 * Rolling Buffer Cache paragraph).  The new key/value of position pos[b] is
 * written to slot pos[b] mod W, then the query attends over the cache: the
 * min(pos[b] + 1, W) positions (pos[b] - W, pos[b]].
 *
 *   out               [B][Hq][d], bf16 or f32 per dims->out_dtype
 *   q                 [B][Hq][d] bf16
 *   k_new, v_new      [B][Hkv][d] bf16
 *   k_cache, v_cache  [B][Hkv][W][d] bf16, slot pos[b] mod W updated in place
 *   pos               device int32[B], >= 0; the cache must hold positions
 *                     [max(0, pos[b] - W + 1), pos[b]) from earlier calls
 *   workspace         device scratch of at least swa_decode_workspace_size(dims)
 *                     bytes, 16-byte aligned; contents need no initialisation
 *                     and are garbage afterwards.  Calls that may overlap on
 *                     the GPU need separate workspaces.
 */
SWA_API int swa_decode(const swa_dims* dims, void* out, const void* q, const void* k_new,
               const void* v_new, void* k_cache, void* v_cache, const int32_t* pos,
               void* workspace, size_t workspace_bytes, void* stream);

/*
 * swa_decode_static - swa_decode for callers that cannot allocate device
 * memory.  The paper has no counterpart to this call; it exists for the
 * library's users.  Some callers cannot allocate: an engine that plans all GPU
 * memory up front and hands out only fixed buffers, or host code that gets
 * tensor pointers from a framework that owns every allocation.  Such a caller
 * passes the same inputs and outputs as to swa_decode (same meaning, layout
 * and ownership) but no workspace.
 *   - The decode scratch comes from one array built into the library,
 *     4 MiB (4194304 bytes) per device, held by every GPU that loads the
 *     library until the process exits.  A launch whose splits merge through
 *     memory needs B * Hq * n_splits * (d + 2) * 4 bytes of it (n_splits from
 *     swa_decode_launch_info; none when that reports one launch).  Dims that
 *     need more than 4 MiB are rejected with SWA_ERR_WORKSPACE_TOO_SMALL and
 *     nothing is enqueued.
 *   - The call allocates nothing.  Its first call on each device looks up the
 *     array's device address, with that device current; make that first call
 *     before any stream capture begins.
 *   - All calls on a device share the array, which keeps the previous call's
 *     contents.  Nothing in it needs clearing, because each call writes every
 *     scratch value it reads.  Calls that may overlap on the GPU (other
 *     streams, unordered host threads) race on it: order them on one stream,
 *     or use swa_decode with separate workspaces.
 */
SWA_API int swa_decode_static(const swa_dims* dims, void* out, const void* q, const void* k_new,
                      const void* v_new, void* k_cache, void* v_cache, const int32_t* pos,
                      void* stream);

/*
 * The 8-bit rolling cache.  swa_q8_append, swa_q8_prefill_chunk and
 * swa_q8_decode do what swa_cache_append, swa_prefill_chunk and swa_decode do,
 * over a cache that holds keys and values in 8 bits (half the bytes that a
 * decode step has to read).
 *
 * The W slots are divided into blocks of SWA_Q8_BLOCK (slots [64 j, 64 j + 64);
 * the last block of a ring whose W is not a multiple of 64 is shorter).  The
 * rows of a block are held as 8-bit numbers with one scale for the keys and one
 * for the values of each kv head: the smallest power of two (at least 2^-100)
 * that brings the block's largest magnitude into the format's range (448 for
 * e4m3, 127 for int8), or 1 for a block of zeros.  A row is held as
 * round-to-nearest-even(x / scale).
 * While a block is being filled, its new rows are in the tail, in bf16; they
 * are rounded once, together, by the call that brings the block's last row, and
 * until then the block still holds the rows of the ring's previous lap.  So what
 * the cache holds depends on the tokens alone, not on how they were cut into
 * calls, and the value that a row stands for (8-bit number times scale) is
 * exact in bf16: prefill and decode attend to the same numbers.
 *
 * Before the first token of a sequence no contents matter (the calls read no
 * row, scale or tail row that was not written before), but for the prefill
 * workspace.  A sequence's tokens are taken in in order: start_pos / pos is the
 * number of tokens that it has taken in so far (any number, for a sequence
 * begun anew, if start_pos is 0).
 * Keys and values must be finite; what an infinity or a NaN leaves in its block
 * is not defined, and harms no other block, head or sequence.
 *
 * Precision.  Scores, softmax sums and outputs are in fp32.  A decode step and a
 * chunk of few rows, which go straight over the bytes, hold a softmax weight to 11
 * bits, or to 2^-40 of the largest product of a weight and its block's value scale;
 * rows still in bf16 (the tail's, the new row, the chunk's) go through f16 with
 * 2^-39 of the largest of the 16 that are taken together (a chunk takes rows of very
 * different sizes one by one).  Their scores (scale q . k) must not exceed 2^23 in
 * size, or 2^12 over blocks whose value scale is not a power of two: where a row's
 * largest is above 2^23.5 its output is not defined and SWA_ERR_DEVICE_ARG is raised
 * in the device status word.  A longer chunk is written out in bf16 for the kernel of
 * swa_prefill_chunk, which rounds the weights to bf16 (8 bits).  Which way a chunk
 * goes is a function of dims and max_tokens: the same tokens cut into other chunks
 * give outputs that differ by these roundings.
 */
#define SWA_Q8_BLOCK 64
#define SWA_Q8_E4M3 0 /* 8-bit floating point: 4 exponent bits, 3 mantissa bits, no infinities */
#define SWA_Q8_INT8 1 /* whole numbers -127 .. 127 */

typedef struct swa_q8_cache {
    void*   k;       /* [B][Hkv][W][d], one byte an element                         */
    void*   v;
    float*  k_scale; /* [B][Hkv][ceil(W / 64)] powers of two; a block that was not   */
                     /* written by these calls may have any normal scale > 0         */
    float*  v_scale;
    void*   k_tail;  /* [B][Hkv][64][d] bf16: row i is slot 64 j + i of the block j  */
    void*   v_tail;  /* that the sequence's next token falls into, if i is before it */
    int32_t format;  /* SWA_Q8_E4M3 or SWA_Q8_INT8                                   */
} swa_q8_cache;

/*
 * swa_q8_append - swa_cache_append for the 8-bit cache (same k, v, max_tokens,
 * start_pos and n_tokens).  Blocks that the chunk fills up are rounded into the
 * cache; the rows of the block that it leaves unfilled go to the tail.  Issue it
 * after swa_q8_prefill_chunk of the same chunk.
 */
SWA_API int swa_q8_append(const swa_dims* dims, const swa_q8_cache* cache, const void* k, const void* v,
                  int32_t max_tokens, const int32_t* start_pos, const int32_t* n_tokens,
                  void* stream);

/*
 * swa_q8_prefill_workspace_size - bytes of device scratch swa_q8_prefill_chunk
 * needs: that of swa_prefill_chunk, and room for this layer's ring in bf16
 * (4 B Hkv W d bytes; one workspace serves all layers of a model in turn).  It is
 * the same for every max_tokens, also for chunks of few rows, which do not use it.
 * Depends only on its arguments.  Returns 0 for invalid arguments.
 */
SWA_API size_t swa_q8_prefill_workspace_size(const swa_dims* dims, int32_t max_tokens);

/*
 * swa_q8_prefill_chunk - swa_prefill_chunk over the 8-bit cache (which it does
 * not change).  The chunk's own keys and values are attended to as they are
 * given, in bf16.
 *   workspace   at least swa_q8_prefill_workspace_size(dims, max_tokens) bytes,
 *               16-byte aligned, ZERO-FILLED before its first use and again
 *               before it serves other dims.  Calls that may overlap on the GPU
 *               need separate workspaces.
 */
SWA_API int swa_q8_prefill_chunk(const swa_dims* dims, void* out, const void* q, const void* k,
                         const void* v, int32_t max_tokens, const swa_q8_cache* cache,
                         const int32_t* start_pos, const int32_t* n_tokens, void* workspace,
                         size_t workspace_bytes, void* stream);

/* swa_q8_decode_workspace_size - as swa_decode_workspace_size, for swa_q8_decode. */
SWA_API size_t swa_q8_decode_workspace_size(const swa_dims* dims);

/*
 * swa_q8_decode - swa_decode over the 8-bit cache: the new key and value of
 * position pos[b] are taken in (into the tail, or with the tail into the cache
 * if they fill a block up), and the query attends over the min(pos[b] + 1, W)
 * positions (pos[b] - W, pos[b]], the block being filled in bf16.
 * Other arguments as in swa_decode.
 */
SWA_API int swa_q8_decode(const swa_dims* dims, void* out, const void* q, const void* k_new,
                  const void* v_new, const swa_q8_cache* cache, const int32_t* pos,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rotary positions.  The first rotary_dim elements of each head's row are
 * taken as pairs, pair i being elements (i, i + rotary_dim / 2), or with
 * `interleaved` elements (2 i, 2 i + 1); the pair (a, b) of the row at position
 * p becomes factor * (a cos t - b sin t, b cos t + a sin t), t = p * inv_freq[i].
 * The other elements are passed through.  Scaled forms for long contexts are
 * other tables (and, for some, a factor).
 */
typedef struct swa_rope_spec {
    const float* inv_freq;    /* device float32[rotary_dim / 2]                     */
    int32_t      rotary_dim;  /* a multiple of 16, 16 <= rotary_dim <= head_dim     */
    int32_t      interleaved; /* 0: pairs (i, i + rotary_dim / 2); 1: (2 i, 2 i + 1) */
    float        factor;      /* multiplier of the rotated elements, finite and > 0 */
} swa_rope_spec;

/*
 * swa_rope - turn a chunk's q and k to their positions, before
 * swa_prefill_chunk / swa_cache_append (with max_tokens = 1, before swa_decode).
 *
 *   q_out, k_out  [B][max_tokens][Hq][d] and [B][max_tokens][Hkv][d] bf16; rows
 *                 t >= n_tokens[b] are not written
 *   q, k          the same shapes, bf16, with q_stride / k_stride elements from
 *                 a token's row to the next one's (max_tokens * stride from a
 *                 sequence to the next): Hq * d / Hkv * d for dense tensors, more
 *                 for heads inside a packed projection; multiples of 8
 *   in place      q_out may be q and k_out may be k if they are dense; other
 *                 overlaps of an output with any input are not allowed
 *   k, k_out      both may be NULL: q alone is turned
 *   max_tokens    >= 1, B * max_tokens < 2^31
 *   start_pos     device int32[B], >= 0: row t is at position start_pos[b] + t
 *   n_tokens      device int32[B], 0 <= n_tokens[b] <= max_tokens, or NULL: all
 *   transpose     0, or 1 for the transposed map (angles -t, same factor): the
 *                 gradient with respect to q and k from that of q_out and k_out
 * dims->window, scale and out_dtype are not used but must be valid.  The angle is
 * the product of position and inv_freq in 64 bits, so far positions keep it.
 */
SWA_API int swa_rope(const swa_dims* dims, const swa_rope_spec* spec, void* q_out, void* k_out,
             const void* q, const void* k, int64_t q_stride, int64_t k_stride,
             int32_t max_tokens, const int32_t* start_pos, const int32_t* n_tokens,
             int32_t transpose, void* stream);

/*
 * swa_device_status - synchronise `stream`, then read and clear the library's
 * device status word on the current device: SWA_OK, SWA_ERR_TIMEOUT (a
 * bounded wait inside a kernel ran out; that kernel's outputs are invalid) or
 * SWA_ERR_DEVICE_ARG.  Returns SWA_ERR_CUDA if the synchronisation fails.
 */
SWA_API int swa_device_status(void* stream);

/* Message of the last non-OK return on this thread ("" if none). */
SWA_API const char* swa_last_error(void);

/* ABI version (major * 100 + minor). */
SWA_API int swa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SWA_H_ */
