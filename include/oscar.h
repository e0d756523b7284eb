/*
 * oscar.h - C ABI of the GB300 (sm_103a) OScaR INT2 KV-cache library.
 *
 * The method ("OScaR: The Occam's Razor for Extreme KV Cache Quantization in
 * LLMs and Beyond", arXiv 2605.19660, Abstract; ai-papers.net summary,
 * section "OScaRの提案手法"): every key vector k is rotated by the normalised
 * Walsh-Hadamard matrix H_d ("Canalized Rotation"), its L2 norm n is stored and
 * the rotated key divided by it ("Omni-Token Scaling"), and the result is
 * quantised to INT2 per channel.  Values are quantised to INT2 per token (the
 * KIVI convention cited in the qiita.com NOVA-KV article, section
 * "KV キャッシュを「読む」時間が、計算そのものより長い").  Decoding reads the
 * packed cache directly (the pages compare against BF16 FlashDecoding-v2,
 * ai-papers.net section "実験結果").
 *
 * Fixed configuration of this library:
 *   d  = 128  head dimension
 *   G  = 128  tokens per key quantisation group; groups cover absolute
 *             positions [128 g, 128 g + 128)
 *   Gv = 32   channels per value quantisation group
 *   H_d[i][j] = (-1)^popcount(i & j) / sqrt(128)  (Sylvester order)
 *   s = (max - min) / 3, z = min (float32); code = clamp(rne((x - z) / s), 0, 3);
 *   s == 0 gives code 0.  Dequantised value: code * s + z.
 *   The L mod 128 most recent tokens of a sequence stay in bf16 (the
 *   residual window) until their group fills; then the whole group is
 *   quantised from the bf16 originals.
 *
 * Conventions
 *   - Ownership: the caller owns every device buffer (arena, inputs, outputs,
 *     workspace).  The library never allocates device memory; the opaque
 *     oscar_cache object is a small host allocation.
 *   - Asynchrony: compute calls enqueue kernels on `stream` (a cudaStream_t,
 *     NULL = legacy default stream) and return without synchronising.  The
 *     per-sequence lengths live on the host, so launch shapes are computed
 *     without device read-back.  All calls on one cache must use one stream
 *     (or be ordered by the caller).
 *   - Errors: every call returns an oscar_status.  Arguments are validated
 *     on the host before anything is enqueued; on error nothing is enqueued
 *     and the cache is unchanged.  oscar_last_error() returns a
 *     thread-local message for the last failing call.  No C++ exception or
 *     abort crosses this boundary.
 *   - GQA: query head h reads KV head h / (num_q_heads / num_kv_heads).
 *   - dtypes: k, v, q and out are bf16 (uint16 storage), row-major.
 */
#ifndef OSCAR_H
#define OSCAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct oscar_cache oscar_cache;

typedef enum oscar_status {
  OSCAR_OK = 0,
  OSCAR_ERR_INVALID_ARG = 1,   /* null pointer, bad size, bad sequence id    */
  OSCAR_ERR_CAPACITY = 2,      /* would exceed max_seq_len / arena / plan    */
  OSCAR_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed       */
  OSCAR_ERR_UNSUPPORTED = 4,   /* head_dim != 128, G != 128, Gv != 32, ...   */
  OSCAR_ERR_DEVICE_TIMEOUT = 5 /* a kernel's bounded wait gave up (see
                                  oscar_cache_check)                          */
} oscar_status;

typedef struct oscar_cache_config {
  int32_t max_batch;     /* number of sequence slots, >= 1                   */
  int32_t num_kv_heads;  /* Hkv, >= 1                                        */
  int32_t head_dim;      /* must be 128                                      */
  int32_t max_seq_len;   /* capacity in tokens per slot, >= 1                */
  int32_t group_size;    /* must be 128 (G)                                  */
  int32_t value_group;   /* must be 32 (Gv)                                  */
  int32_t device;        /* CUDA device ordinal of the arena                 */
  int32_t meta_bits;     /* 32 (default; 0 also means 32): float32 scales,   */
                         /* zeros and norms, 13,824-byte blocks; 16: float16 */
                         /* (rounded to nearest even; codes decided against  */
                         /* the rounded values), 11,008-byte blocks          */
} oscar_cache_config;

/* Kinds for oscar_cache_bytes. */
enum {
  OSCAR_BYTES_USED = 0,            /* packed groups + bf16 window in use     */
  OSCAR_BYTES_BF16_EQUIVALENT = 1, /* bytes of a plain bf16 K+V cache       */
  OSCAR_BYTES_ARENA = 2            /* arena size the configuration needs    */
};

/*
 * Device arena layout (all offsets in bytes from the arena base; the arena
 * must be 256-byte aligned):
 *
 *   [0, 256)                       status words; word 0 = device error flags
 *   [256, 256 + 4 S H)             per (slot, kv head): float32 bit pattern of
 *                                  the largest finite value scale s_v
 *                                  quantised so far (4 bytes each;
 *                                  S = max_batch, H = Hkv)
 *   [256 + 4 S H, M)               per (slot, kv head): float32 bit pattern of
 *                                  the largest finite |value zero| z_v
 *                                  quantised so far, M = 256-aligned end
 *   blocks  (base = M)             one block of B bytes per
 *                                  (slot, kv head, group g):
 *                                  base + ((slot*Hkv + head)*max_groups + g)*B,
 *                                  max_groups = ceil(max_seq_len / 128),
 *                                  B = 13,824 (meta_bits 32) or 11,008 (16)
 *   windows (after the blocks,     65,536 bytes per (slot, kv head): 128 bf16
 *            256-aligned)          key rows (slot p mod 128) then 128 bf16
 *                                  value rows, 256 bytes per row
 *
 * One group block (the unit the decode kernel streams), meta_bits 32:
 *   +0      K codes, 4,096 B, "fragment order" of the 128x128 matrix
 *           X[row = token][col = channel]
 *   +4096   K scale s_c, float32 [128] (per channel)
 *   +4608   K zero  z_c, float32 [128]
 *   +5120   K norm  n_t, float32 [128] (per token, position order)
 *   +5632   V codes, 4,096 B, fragment words of X[row = channel][col = token]
 *           in "V order"
 *   +9728   V scale s[t][0..3], float32 [128][4] (per token, one per
 *           32-channel group), token t in row t ^ ((t >> 3) & 1)
 *           (neighbouring tokens swap rows where bit 3 of t is set)
 *   +11776  V zero  z[t][0..3], float32 [128][4], rows as the V scale
 * meta_bits 16: the same sections with float16 metadata:
 *   +0 K codes, +4096 K scale, +4352 K zero, +4608 K norm (float16 [128]
 *   each), +4864 V codes, +8960 V scale, +9984 V zero (float16 [128][4]
 *   each); 11,008 bytes, 86 per token and head.
 *
 * Fragment words of a 128x128 matrix of 2-bit codes X[row][col]: the 32-bit
 * word F(mt, lane, j, r) holds the 16 codes with
 *   row = 16*mt + (lane >> 2) + 8*r,
 *   col = 16*(4*j + kk) + 8*hf + 2*(lane & 3) + e,   kk in 0..3, hf, e in {0,1},
 * code at bits [b, b+1] with b = 16*e + 4*kk + 2*hf
 * (mt in 0..7, lane in 0..31, r, j in {0,1}; words are little-endian).
 * "Fragment order" (K codes) stores F(mt, lane, j, r) as word
 *   w = (mt*32 + lane)*4 + 2*j + r,
 * "V order" (V codes) as word
 *   w = ((mt*2 + j)*32 + lane)*2 + r.
 */

/* Arena bytes needed by `cfg`.  Pure host arithmetic. */
oscar_status oscar_cache_required_bytes(const oscar_cache_config* cfg, size_t* out_bytes);

/* Create a cache over a caller-owned device arena of `arena_bytes` (at least
 * oscar_cache_required_bytes) on cfg->device.  Zeroes the status and
 * metadata region (a blocking cudaMemset of a few KB); all sequence lengths
 * start at 0.  *out receives a host object to pass to the other calls. */
oscar_status oscar_cache_create(const oscar_cache_config* cfg, void* device_arena,
                                size_t arena_bytes, oscar_cache** out);

/* Free the host object (never the arena). NULL is accepted. */
oscar_status oscar_cache_destroy(oscar_cache* cache);

/* Set the length of slot `seq` to 0 (or every slot if seq == -1) and clear its
 * value-scale maxima, enqueued on `stream`. */
oscar_status oscar_cache_reset(oscar_cache* cache, int32_t seq, void* stream);

/* Current length (tokens) of slot `seq`. */
oscar_status oscar_cache_length(const oscar_cache* cache, int32_t seq, int32_t* out_len);

/* The configuration the cache was created with (meta_bits 32 or 16, never 0). */
oscar_status oscar_cache_get_config(const oscar_cache* cache, oscar_cache_config* out);

/*
 * Append new tokens to `n_seqs` sequences (prefill chunks or single decode
 * tokens; the method's compression step, OScaR abstract / ai-papers.net
 * "OScaRの提案手法").
 *   seq_ids  host int32 [n_seqs], distinct slot ids in [0, max_batch)
 *   cu_new   host int32 [n_seqs + 1], cu_new[0] = 0, non-decreasing;
 *            sequence i appends rows cu_new[i] .. cu_new[i+1]-1
 *   k, v     device bf16 [cu_new[n_seqs], Hkv, 128] (rows of the raw, i.e.
 *            unrotated, keys and values; 16-byte aligned, and read with
 *            32-byte loads, which are faster, when both are 32-byte
 *            aligned); host memory fails with OSCAR_ERR_INVALID_ARG
 * Every 128-token group that fills is rotated, norm-scaled and quantised
 * (keys) and quantised (values) from its bf16 tokens (earlier ones from the
 * window, new ones from k/v) into its block; the remaining tokens go to the
 * window.  Fails with OSCAR_ERR_CAPACITY if a length would exceed
 * max_seq_len.  Lengths are updated on the host when the call returns.
 */
oscar_status oscar_quantize_append(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                   const int32_t* cu_new, const void* k, const void* v,
                                   void* stream);

/* Workspace bytes oscar_decode_attention needs for up to `n_seqs` sequences
 * and `num_q_heads` query heads (an upper bound independent of lengths). */
oscar_status oscar_decode_workspace_bytes(const oscar_cache* cache, int32_t n_seqs,
                                          int32_t num_q_heads, size_t* out_bytes);

/*
 * Single-query decode attention over the packed cache (split-K flash
 * decoding, GQA, ragged batch).
 *   seq_ids      host int32 [n_seqs]; every slot must have length >= 1
 *   q            bf16 [n_seqs, num_q_heads, 128] (unrotated queries), 16-byte
 *                aligned, in device memory or page-locked host memory
 *   num_q_heads  any multiple of Hkv; the kernels serve up to 8 query heads
 *                of a KV head per pass over the cache, so num_q_heads / Hkv
 *                = 9..16 takes two passes, 17..24 three, and so on
 *   softmax_scale  0 means 1 / sqrt(128)
 *   out          bf16 [n_seqs, num_q_heads, 128], 16-byte aligned, in device
 *                memory or page-locked host memory
 *   workspace    device scratch of >= oscar_decode_workspace_bytes bytes,
 *                16-byte aligned; contents need not be initialised
 * For a quantised token t with norm n_t the score is
 *   s_t = n_t * (H_d q) . (code_t * s + z) * softmax_scale,
 * for a window token s_t = q . k_t * softmax_scale; out = softmax(s) . v_hat.
 * Attends to exactly the tokens in the cache (append the current token first).
 * Host buffers: q and out may be page-locked host memory (cudaHostAlloc,
 * cudaHostRegister, torch pin_memory); the kernels then read q and write out
 * in place through the device mapping (over NVLink-C2C on Grace systems), so
 * a decode step from host inputs to host outputs needs no staging copies.
 * Pageable host memory and device memory of another device fail with
 * OSCAR_ERR_INVALID_ARG before anything is enqueued.
 * Stream order: the main kernel is launched as a programmatic dependent of
 * the kernel before it in `stream`.  Before it waits for that kernel it only
 * copies cache blocks of groups closed before the previous decode call on
 * this cache, when that call used the same stream (the library tracks its
 * appends and decodes); q, the workspace and all other inputs are read after
 * the wait, so a preceding kernel may produce q.  The arena must be written
 * through this library only.
 */
oscar_status oscar_decode_attention(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                    const void* q, int32_t num_q_heads, float softmax_scale,
                                    void* out, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * oscar_decode_attention with float32 outputs: the merged attention output
 * before any bf16 rounding, for callers that keep attention outputs in
 * float32 (and for checking the decode at float32 precision).
 *   out  float32 [n_seqs, num_q_heads, 128], 16-byte aligned, device or
 *        page-locked host memory
 * Every other argument, the result before the output rounding, and the
 * errors are those of oscar_decode_attention.
 */
oscar_status oscar_decode_attention_f32(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                        const void* q, int32_t num_q_heads, float softmax_scale,
                                        void* out, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * One decode step fused: append one token to each of `n_seqs` sequences,
 * then decode, with the same result as oscar_quantize_append (one row per
 * sequence) followed by oscar_decode_attention.  The ai-papers.net OScaR
 * summary, section "まとめと今後の展望", notes that the quantisation
 * overhead weighs relatively more at short context; this call removes one
 * launch from most decode steps.
 *   k_new, v_new  device bf16 [n_seqs, Hkv, 128], the new token of each
 *                 sequence (16-byte aligned)
 *   other arguments as for oscar_decode_attention (q and out may be host
 *   buffers in the same way).
 * When no sequence's new length is a multiple of 128 (127 steps in 128),
 * the step is one decode launch: the combine kernel attends the new token as
 * the last window row straight from k_new / v_new and stores it into the
 * window.  When a group closes, the quantiser runs first (two launches), so
 * the group is attended quantised.  All arguments are validated before
 * anything is enqueued; on error nothing changes.
 */
oscar_status oscar_append_decode(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                 const void* k_new, const void* v_new, const void* q,
                                 int32_t num_q_heads, float softmax_scale, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Chunked-prefill attention over the cache: each of the n_q queries of a new
 * chunk of sequence `seq` attends to every token already in its cache
 * (quantised groups and window; no mask, the cache precedes the chunk), with
 * the decode path's scores and values (OScaR abstract; ai-papers.net
 * "OScaRの提案手法").  Call it before appending the chunk; the chunk's own
 * causal attention is merged in by the caller with lse.
 *   q            bf16 [n_q, num_q_heads, 128], 16-byte aligned
 *   out          bf16 [n_q, num_q_heads, 128], 16-byte aligned
 *   lse          fp32 [n_q, num_q_heads] or NULL: ln sum_t exp(s_t) per row
 *                (natural log, scores times softmax_scale)
 *   q, out and lse may be device or page-locked host memory (see
 *   oscar_decode_attention); other memory fails with OSCAR_ERR_INVALID_ARG.
 *   softmax_scale  0 means 1 / sqrt(128)
 *   workspace    NULL, or device memory (16-byte aligned) of workspace_bytes
 *                for partial results: the history's groups are then split
 *                into parts processed by separate CTAs and merged by a
 *                second kernel, so that the CTAs fill whole waves of SMs.
 *                As many parts are used as fit, up to the number that
 *                oscar_prefill_workspace_bytes sizes; NULL (or too small for
 *                two parts) runs unsplit.  Results agree within rounding.
 * Any GQA ratio.  The sequence must be non-empty.
 */
oscar_status oscar_prefill_attention(oscar_cache* cache, int32_t seq, int32_t n_q, const void* q,
                                     int32_t num_q_heads, float softmax_scale, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes that let oscar_prefill_attention split the history of
 * sequence `seq` (at its current length) for n_q queries of num_q_heads
 * heads: parts x Hkv x n_q x (num_q_heads / Hkv) x 528 bytes, 0 when no
 * split pays off (short histories, or rows that already fill the SMs).
 */
oscar_status oscar_prefill_workspace_bytes(const oscar_cache* cache, int32_t seq, int32_t n_q,
                                           int32_t num_q_heads, size_t* out_bytes);

/*
 * Decode that allocates nothing and takes no workspace.  The OScaR pages have
 * no counterpart to this call; it exists for callers that cannot allocate
 * device memory where they decode (code inside a memory pool or arena it does
 * not own, plugins whose host framework forbids allocation on the serving
 * path, callers that must keep a fixed device footprint).
 *   Same arguments and results as oscar_decode_attention, without workspace.
 *   The split-K partials go to a file-scope device array of 4 MiB that every
 *   GPU loading this library holds until the process exits.  Calls needing
 *   more than that (sequences x KV heads plus two rows per SM of partials)
 *   fail with OSCAR_ERR_CAPACITY and a message; use oscar_decode_attention.
 *   The first call on a device looks up the array's device address (with
 *   the cache's device current); make that first call before any CUDA stream
 *   capture.  No device memory is allocated or freed, and nothing in the
 *   array needs to start at zero (each call writes every partial it reads).
 *   Every call shares the one array: calls whose kernels overlap on the GPU
 *   (different streams, or different threads without ordering) race on it
 *   and give wrong results.
 */
oscar_status oscar_decode_attention_noalloc(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                            const void* q, int32_t num_q_heads, float softmax_scale,
                                            void* out, void* stream);

/*
 * The calls below prepare, choose, attend and read back parts of the cache.
 * Element types of their float buffers:
 */
enum {
  OSCAR_BF16 = 0,
  OSCAR_F32 = 1
};

/* How rotary frequencies are scaled for contexts longer than the model was
 * trained for (oscar_rotary_config.scaling). */
enum {
  OSCAR_ROTARY_NONE = 0,
  OSCAR_ROTARY_LINEAR = 1, /* every frequency divided by `factor`            */
  OSCAR_ROTARY_BANDED = 2, /* by wavelength: with t = original_length f /
                              (2 pi) turns over the original context, f / factor
                              below `low` turns, f above `high`, between them
                              (1 - r) f / factor + r f, r = (t - low) / (high - low) */
  OSCAR_ROTARY_YARN = 3    /* by pair index: with c(t) = rotary_dim ln(
                              original_length / (2 pi t)) / (2 ln base), l =
                              max(floor(c(high)), 0), h = min(ceil(c(low)),
                              rotary_dim - 1) (h = l + 0.001 when equal), r =
                              clamp((i - l) / (h - l), 0, 1): f / factor r +
                              f (1 - r)                                       */
};

typedef struct oscar_rotary_config {
  int32_t head_dim;        /* must be 128                                     */
  int32_t rotary_dim;      /* rotated channels, the first of the head: a
                              multiple of 16 up to 128                        */
  int32_t interleaved;     /* 0: pair i is channels (i, i + rotary_dim / 2);
                              1: channels (2 i, 2 i + 1)                      */
  int32_t scaling;         /* OSCAR_ROTARY_*                                  */
  double base;             /* frequency of pair i: base^(-2 i / rotary_dim);
                              > 1                                             */
  double factor;           /* >= 1 (scaling other than NONE)                  */
  double original_length;  /* tokens of the original context (BANDED, YARN)   */
  double low, high;        /* BANDED: turns, 0 and 0 mean 1 and 4; YARN: slow
                              and fast turns, 0 and 0 mean 1 and 32           */
  double attention_factor; /* multiplies the rotated channels; 0 means 1, for
                              YARN 0.1 ln(factor) + 1                         */
} oscar_rotary_config;

/* Frequencies (radians per position, rotary_dim / 2 of them) and the factor
 * on the rotated channels that `cfg` stands for.  Pure host arithmetic. */
oscar_status oscar_rotary_frequencies(const oscar_rotary_config* cfg, double* frequencies,
                                      double* attention_factor);

/* A configuration made ready for oscar_rotary, by oscar_rotary_prepare (which
 * checks it): keep it beside the model and pass it to every call. */
typedef struct oscar_rotary_table {
  int32_t rotary_dim;
  int32_t interleaved;
  float factor;            /* on the rotated channels                         */
  int32_t reserved;
  uint64_t phase[64];      /* turns per position of pair i, 2^64 to the turn  */
} oscar_rotary_table;

oscar_status oscar_rotary_prepare(const oscar_rotary_config* cfg, oscar_rotary_table* table);

/* Rows of one tensor [n_tokens, heads, 128]: strides in elements, channels
 * contiguous.  `out` may be `in` with the same strides (in place); otherwise
 * the rows written must not overlap any rows read. */
typedef struct oscar_rotary_rows {
  const void* in;
  void* out;
  int64_t in_token_stride, in_head_stride;
  int64_t out_token_stride, out_head_stride;
  int32_t heads;
} oscar_rotary_rows;

/*
 * Rotary positions of queries and keys, before the keys are appended and the
 * queries attend: with t = positions[token] * frequency (a phase within 2^-31
 * of a turn at any int32 position, whose distance from the nearest quarter turn
 * is then rounded to float32: 2^-28 of a turn at most) and m the attention factor,
 *   (y_a, y_b) = m (x_a cos t - x_b sin t, x_a sin t + x_b cos t)
 * for every pair (a, b); channels from rotary_dim on are copied.
 *   positions  int32 [n_tokens], device or page-locked host memory, may be
 *              negative
 *   type       OSCAR_BF16 or OSCAR_F32 (q and k, in and out)
 *   q, k       rows on the current device; k may be NULL; 16-byte aligned
 *              pointers, strides of 16-byte multiples (those of a single
 *              token or head are not looked at); inputs may have any
 *              strides (0 broadcasts), output rows must be distinct: either
 *              the heads of a token or the tokens of a head side by side.
 *              Zero heads or zero tokens: nothing is done.
 *   transpose  0, or 1 for the transposed rotation (t -> -t, the same m): the
 *              gradient, and with m = 1 the inverse
 * float32 arithmetic, one rounding to the output type.
 */
oscar_status oscar_rotary(const oscar_rotary_table* table, int64_t n_tokens, const int32_t* positions,
                          int32_t type, const oscar_rotary_rows* q, const oscar_rotary_rows* k,
                          int32_t transpose, void* stream);

/*
 * Read tokens back: for each i, tokens start[i] .. end[i] - 1 of slot
 * seq_ids[i], packed one range after the other.
 *   seq_ids, start, end  host int32 [n_seqs]; 0 <= start <= end <= length; a
 *                        slot may appear more than once
 *   type                 OSCAR_BF16 or OSCAR_F32
 *   k_out, v_out         [sum(end - start), Hkv, 128], 16-byte aligned device
 *                        memory (float32 values are written in 32-byte pieces
 *                        when both are 32-byte aligned); either may be NULL
 * A quantised key is H_d (n (code s + z)) (back in the basis in which it was
 * appended), a quantised value code s + z, both in float32 and rounded once to
 * the output type; window tokens are their stored bf16 rows.
 */
oscar_status oscar_cache_read(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                              const int32_t* start, const int32_t* end, int32_t type, void* k_out,
                              void* v_out, void* stream);

/*
 * Move a sequence's packed state out of the cache and back in (swapping a
 * sequence to host memory, sending it to another cache of the same head count
 * and meta_bits).  With L tokens, g = L / 128 and w = L % 128:
 *   blocks  Hkv x g x B bytes: the group blocks, KV head by KV head (B = 13,824
 *           or 11,008)
 *   window  bf16 [Hkv, 2, 128, 128]: key rows, then value rows; the first w
 *           rows of each are read or written, the others left as they are
 *   maxima  float32 [2, Hkv]: the largest finite value scale and |value zero|
 * Device or page-locked host memory of any alignment; blocks may be NULL when
 * g = 0 and window when w = 0.  Plain copies on `stream`: until they have run
 * the buffers must stay allocated, those of an import unchanged.
 * oscar_cache_import replaces what the slot holds by `length` tokens.  It takes
 * the maxima as they are: they set the range of the float16 factors of every
 * decode and prefill over the slot.  Below the blocks' own scales or |zeros|
 * these overflow (infinite or NaN outputs), far above them they lose bits.
 */
oscar_status oscar_cache_export(oscar_cache* cache, int32_t seq, void* blocks, void* window,
                                float* maxima, void* stream);
oscar_status oscar_cache_import(oscar_cache* cache, int32_t seq, int32_t length, const void* blocks,
                                const void* window, const float* maxima, void* stream);

/*
 * Choosing the groups worth attending.  An index holds an 8-bit summary of
 * every quantised group, 264 bytes per (slot, KV head, group):
 *   +0            int8 [slot][Hkv][max_groups][32][2][4]: for channels 4 l .. 4 l + 3
 *                 the lowest values lo8 (4), then the highest hi8 (4) of the
 *                 group's unit keys, in steps of 2^e
 *   +256 S H max_groups   float32 [slot][Hkv][max_groups][2]: w_max, w_min, the
 *                 largest and the smallest token norm times 2^e
 * with lo = z, hi = fl32(z + 3 s), lo8 = rne(lo / 2^e), hi8 = rne(hi / 2^e), e
 * the smallest exponent >= -100 with |lo|, |hi| <= 127 2^e over the channels
 * (e = -100 for an all-zero group); values that are not finite count as 0.
 * The caller owns the index buffer (256-byte aligned device memory), attaches
 * it once, and brings it up to date after groups have closed.  Which groups
 * are in it is recorded on the host when oscar_index_update returns (as the
 * lengths are): a graph that captured the call must be replayed before the
 * record holds.
 */
oscar_status oscar_index_required_bytes(const oscar_cache* cache, size_t* out_bytes);

/* Attach an index buffer of at least oscar_index_required_bytes (nothing in
 * it is valid yet); NULL detaches. */
oscar_status oscar_index_attach(oscar_cache* cache, void* index, size_t index_bytes);

/* Summarise the groups of each slot that are not in the index yet (rebuild =
 * 0) or all of them (rebuild = 1).  Enqueues nothing when there are none.
 * At most 1,024 sequences per call. */
oscar_status oscar_index_update(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                int32_t rebuild, void* stream);

/*
 * For each (sequence, KV head), the n_select groups with the largest scores
 * for its query heads, in ascending order; -1 behind them when there are fewer
 * groups.  With E the smallest exponent >= -100 such that |q| < 2^E for the
 * query heads of the KV head (elements that are not finite count as 0),
 *   a = rne(q 2^(22 - E)),  b = Hu a (Hu = sqrt(128) H_d; whole numbers),
 *   q8 = floor(b / 2^B + 1/2), B >= 0 the smallest with |b| <= 127 2^B (no 1/2
 *        for B = 0),
 *   S = max over the heads of sum_c max(q8_c lo8_c, q8_c hi8_c),
 *   score = S w_max if S >= 0, else S w_min, exactly;
 * up to its 8-bit steps, the largest score any key within the group's box
 * could reach.  Equal scores: the lower group first.
 *   seq_ids     host int32 [n_seqs], distinct, at most 1,024; every group of
 *               each must be in the index (OSCAR_ERR_INVALID_ARG otherwise)
 *   q           bf16 [n_seqs, num_q_heads, 128], 16-byte aligned, device or
 *               page-locked host memory; num_q_heads a multiple of Hkv, at most
 *               64 per KV head
 *   n_select    1 .. 2^24
 *   keep_first, keep_last  that many first and last groups of each sequence are
 *               always chosen (attention sinks, recent tokens); >= 0, together
 *               <= n_select
 *   groups      int32 [n_seqs, Hkv, n_select], device memory
 * Sequences without a group get -1s.  A sequence of more than 12,000 groups
 * (1,536,000 tokens) and more than n_select fails with OSCAR_ERR_UNSUPPORTED.
 */
oscar_status oscar_select_groups(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids, const void* q,
                                 int32_t num_q_heads, int32_t n_select, int32_t keep_first,
                                 int32_t keep_last, int32_t* groups, void* stream);

/*
 * Single-query decode attention over listed groups: oscar_decode_attention
 * restricted, for each (sequence, KV head), to the groups listed for it and
 * the sequence's window.
 *   groups    int32 [n_seqs, Hkv, n_select] in device memory, read on
 *             `stream` (oscar_select_groups may produce it); an entry outside
 *             [0, length / 128) is empty, a group listed twice counts twice
 *   n_select  1 .. 2^24
 *   type      OSCAR_BF16 or OSCAR_F32: type of out.  With OSCAR_BF16 the value
 *             factors (softmax weight times value scale) are held in float16,
 *             with OSCAR_F32, and in oscar_decode_attention, in two float16
 *             terms.  Of n attended tokens, the largest value scale among them
 *             A and in the whole sequence S, bf16 outputs are off by 3 (2^-11 A
 *             + n 2^-31 S) at most through that, beside their own rounding: RMS
 *             errors up to 1.8e-3 of the output, at most 8 % above those of
 *             32-bit factors rounded once, in what was measured.  float32
 *             outputs lose 3 n 2^-30 S at most, which counts only where S is far
 *             above A
 *   lse       float32 [n_seqs, num_q_heads] or NULL: ln sum exp(score) over the
 *             attended tokens (natural log, scores times softmax_scale)
 * A row with nothing to attend (no valid entry, empty window) gets zeros and
 * an lse of -infinity; a query head that is not finite and has a token to
 * attend gets NaN outputs and lse, the other heads are unaffected.  q, out and
 * lse may be device or page-locked host memory; every other argument, the
 * workspace and the stream order are those of oscar_decode_attention.
 */
oscar_status oscar_sparse_decode_attention(oscar_cache* cache, int32_t n_seqs, const int32_t* seq_ids,
                                           const void* q, int32_t num_q_heads, float softmax_scale,
                                           const int32_t* groups, int32_t n_select, int32_t type,
                                           void* out, float* lse, void* workspace,
                                           size_t workspace_bytes, void* stream);

/* Footprint: kind = OSCAR_BYTES_USED / _BF16_EQUIVALENT for slot `seq`
 * (or all slots if seq == -1), or OSCAR_BYTES_ARENA.  Host arithmetic:
 * a full group costs 13,824 B per KV head (108 B per token) versus 65,536 B
 * (512 B per token) in bf16; a window token costs 512 B. */
oscar_status oscar_cache_bytes(const oscar_cache* cache, int32_t seq, int32_t kind,
                               size_t* out_bytes);

/* Arena offsets of the block of (seq, kv_head, group) and of the window of
 * (seq, kv_head), for inspection and tests. */
oscar_status oscar_cache_block_offset(const oscar_cache* cache, int32_t seq, int32_t kv_head,
                                      int32_t group, size_t* out_offset);
oscar_status oscar_cache_window_offset(const oscar_cache* cache, int32_t seq, int32_t kv_head,
                                       size_t* out_offset);

/*
 * Test hook of the failure path: the next INT2 decode, read-back or selection
 * launch made on the calling thread (oscar_decode_attention, _f32,
 * oscar_append_decode, oscar_sparse_decode_attention, oscar_cache_read,
 * oscar_select_groups) has one bulk copy of its first CTA left unissued, and its bounded waits give up after 2^14 polls
 * instead of 2^24.  (A listed decode of sequences without a group: the window
 * copies of its combine, where it has any.)  The consumer waiting for that copy then
 * gives up, the kernel sets the arena's error flag, skips its remaining work
 * and returns (no fault, no hang; the results of that call are undefined),
 * and oscar_cache_check reports OSCAR_ERR_DEVICE_TIMEOUT.  Later calls are
 * unaffected.  Not for production use.
 */
oscar_status oscar_test_arm_wait_timeout(void);

/* Test hook: for each of the n_seqs slots in seq_ids, the number of leading
 * groups whose blocks the next decode on `stream` would copy before its grid
 * dependency wait (INT32_MAX: all of them), from the host's record of the
 * appends, resets and decodes enqueued on this cache.  out: host int32
 * [n_seqs].  Enqueues nothing. */
oscar_status oscar_test_settled_groups(const oscar_cache* cache, int32_t n_seqs,
                                       const int32_t* seq_ids, void* stream, int32_t* out);

/* Synchronise `stream`, then read the device error flags of the arena.
 * Returns OSCAR_ERR_DEVICE_TIMEOUT if a kernel's bounded wait gave up since
 * the last check (and clears the flags), OSCAR_OK otherwise. */
oscar_status oscar_cache_check(oscar_cache* cache, void* stream);

/*
 * BF16 reference decode (the speed-ratio baseline standing in for the
 * pages' BF16 FlashDecoding-v2 comparator, ai-papers.net "実験結果"): the same
 * split-K structure over a plain bf16 cache.
 *   k_cache, v_cache  device bf16 [n_seqs_cap, Hkv, max_seq_len, 128]
 *   seq_ids / seq_lens host int32 [n_seqs]: slot and length (>= 1) of each
 *   q, out            bf16 [n_seqs, num_q_heads, 128], device or page-locked
 *                     host memory (the caches and the workspace: device only)
 * Scores are q . k_t * softmax_scale in float32, softmax and P.V in float32.
 */
oscar_status oscar_bf16_decode_workspace_bytes(int32_t n_seqs, int32_t num_kv_heads,
                                               int32_t num_q_heads, size_t* out_bytes);
oscar_status oscar_bf16_decode_attention(int32_t n_seqs, const int32_t* seq_ids,
                                         const int32_t* seq_lens, const void* k_cache,
                                         const void* v_cache, int32_t num_kv_heads,
                                         int32_t max_seq_len, const void* q,
                                         int32_t num_q_heads, float softmax_scale, void* out,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* Profiling hook: when both are non-NULL, the following decode calls on this
 * thread record `start_event` / `stop_event` (cudaEvent_t) around their main
 * split-K kernel.  Pass NULLs to turn it off. */
oscar_status oscar_set_timing_events(void* start_event, void* stop_event);

/* Thread-local message of the last failing call ("" if none). */
const char* oscar_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* OSCAR_H */
