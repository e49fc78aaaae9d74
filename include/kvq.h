/*
 * kvq.h -- C ABI of the quantized KV-cache decode-attention library.
 *
 * The library implements the decode hot path of a transformer whose KV cache
 * is stored as group-wise asymmetric INT4/INT8 codes:
 *
 *   kvq_append       quantize new K/V vectors into the cache
 *                    ("What actually happens when you quantize a KV cache",
 *                    section 3 steps 2-5 and section 4: per group s =
 *                    (max-min)/(2^b-1), z = round(-min/s), q = clamp(round(x/s)
 *                    + z, 0, 2^b-1); two INT4 codes per byte, even channel in
 *                    the low nibble; fp16 scale and zero kept in their own
 *                    contiguous arrays);
 *   kvq_decode_attn  one decode row per query head over every cached token of
 *                    its sequence, the token just appended included
 *                    ("Quantization & inference optimisation", "Prefill, then
 *                    decode": append, then attend without a mask; "Serving
 *                    many users at once", batched decode_step with per-user
 *                    lengths and grouped-query heads), reading the codes and
 *                    dequantizing x_hat = (q - z) * s in registers
 *                    ("What actually happens ...", section 6).
 *
 * Conventions shared by every entry point:
 *   - Pointers marked "device" are CUDA device memory owned by the caller; the
 *     library never allocates, frees or retains them.  Arrays must be
 *     16-byte aligned.  fp16 data is passed as uint16_t (IEEE binary16 bits).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is enqueued asynchronously; nothing synchronizes.
 *   - Errors that the host can see (bad sizes, null pointers, unsupported
 *     shapes, too small a workspace) are returned synchronously and nothing
 *     is launched.  A failed launch returns KVQ_ERR_CUDA (with KVQ_VERBOSE
 *     set in the environment, the CUDA error's name also goes to stderr).
 *   - Errors that only the data reveals (a length beyond the cache, a bad
 *     block-table entry, a group the format cannot store) are OR-ed as
 *     KVQ_FLAG_* bits into *dev_status (a device uint32_t, may be NULL) and
 *     the offending unit is skipped as documented per call; read the word
 *     after the stream has synchronized.  No kernel traps, and waits
 *     between the warps of one thread block end after two seconds.
 *
 * Cache layouts (one instance for K, one for V; the same shapes for both):
 *   row_bytes = head_dim * bits / 8;  groups = head_dim / group_size
 *   codes: INT8 one per byte; INT4 two per byte, even channel in the low
 *   nibble; INT2 four per byte, channel 4m + k in bits 2k and 2k + 1.
 *   DENSE  codes  [batch][num_kv_heads][capacity][row_bytes]       uint8
 *          scale  [batch][num_kv_heads][capacity][groups]          fp16
 *          zero   same shape as scale
 *          token p of sequence b lives in slot p (0 <= p < capacity).
 *   PAGED  codes  [num_pages][num_kv_heads][page_size][row_bytes]   uint8
 *          scale, zero  [num_pages][num_kv_heads][page_size][groups]
 *          block_table [batch][max_blocks_per_seq] int32 (device);
 *          token p of sequence b lives in page block_table[b][p / page_size]
 *          at offset p % page_size.  Pages may be shared by sequences.
 *   bits == 16 stores the fp16 vectors themselves in the codes arrays
 *   (row_bytes = 2 * head_dim) and uses no scale/zero arrays.
 *   symmetric == 1 and nf4 == 1 use no zero arrays (k_zero, v_zero ignored).
 *
 * Axis-aware caches (k_per_channel == 1; "What actually happens when you
 * quantize a KV cache", section 3 step 7 and section 7: K grouped per
 * channel, V per token, the first tokens and the newest ones kept in fp16).
 * With S = sink_tokens, g = group_size, and L tokens cached:
 *   positions [0, min(S, L))          fp16 sinks, window slot p;
 *   block j covers [S + j g, S + (j+1) g), quantized once all g of its
 *     tokens have arrived: K codes in row p of k_codes with one scale and
 *     zero per channel for the block, V codes in row p of v_codes with
 *     per-token groups of g channels as in the default layout;
 *   the newest L - S - floor((L - S) / g) g tokens (fewer than g) form the
 *     fp16 residual window, slot S + (p - S) mod g.
 *   DENSE: capacity must be a multiple of g and larger than S.
 *          k_codes, v_codes  [batch][num_kv_heads][capacity][row_bytes]
 *          k_scale, k_zero   [batch][num_kv_heads][capacity / g][head_dim]
 *          v_scale, v_zero   [batch][num_kv_heads][capacity][head_dim / g]
 *          k_window, v_window [batch][num_kv_heads][S + g][head_dim] fp16
 *   PAGED: only the positions after the sinks are paged, by u = p - S:
 *     position p >= S lives in page block_table[b][u / capacity] at row
 *     u mod capacity, and block j's K headers in that page's row
 *     j mod (capacity / g).  capacity (tokens per page) must be a multiple
 *     of g, so that no block straddles two pages.  A sequence holds at most
 *     S + capacity * max_blocks_per_seq positions.  The window stays per
 *     sequence.
 *          k_codes, v_codes  [num_pages][num_kv_heads][capacity][row_bytes]
 *          k_scale, k_zero   [num_pages][num_kv_heads][capacity / g][head_dim]
 *          v_scale, v_zero   [num_pages][num_kv_heads][capacity][head_dim / g]
 *          k_window, v_window [batch][num_kv_heads][S + g][head_dim] fp16
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

/* Every entry point below is exported from the shared library; the library
 * is built with hidden default visibility, so nothing else is. */
#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned array      */
  KVQ_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. head_dim 512) */
  KVQ_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required    */
  KVQ_ERR_CUDA = 4          /* a CUDA runtime call or launch failed          */
} kvq_status;

/* Largest batch of one decode call (and of one append on an axis-aware
 * cache): the kernels take the sequence from a grid dimension. */
#define KVQ_MAX_BATCH 65535

/* Bits OR-ed into the caller's device status word. */
#define KVQ_FLAG_SEQ_LEN      0x1u /* position/length outside the cache        */
#define KVQ_FLAG_BLOCK_TABLE  0x2u /* block-table entry outside [0,num_pages)  */
#define KVQ_FLAG_ZERO_CLAMPED 0x4u /* zero-point outside +-2048, clamped       */
#define KVQ_FLAG_NONFINITE    0x8u /* group held inf/NaN, stored as zeros      */
#define KVQ_FLAG_OOB          0x10u /* debug builds: an access outside its array
                                       was skipped (see kvq_debug_checks)      */
#define KVQ_FLAG_POOL_EMPTY   0x20u /* too few free pages: nothing was reserved */
#define KVQ_FLAG_PAGE_LIST    0x40u /* a copy list names a page twice as target,
                                       or one page as source and target       */
#define KVQ_FLAG_TIMEOUT      0x80u /* a kernel's internal wait ran out (2 s):
                                       the call's output is unusable (only this
                                       word tells; see kvq_extend_attn)       */

typedef enum { KVQ_DENSE = 0, KVQ_PAGED = 1 } kvq_layout;

typedef struct {
  int32_t bits;               /* 2, 4 or 8 (quantized), 16 (fp16 cache)       */
  int32_t group_size;         /* channels per group, multiple of 8, divides
                                 head_dim; ignored when bits == 16            */
  int32_t num_kv_heads;       /* >= 1                                          */
  int32_t head_dim;           /* 64, 128 or 256                                */
  int32_t layout;             /* kvq_layout                                    */
  int32_t capacity;           /* DENSE: token slots per sequence;
                                 PAGED: tokens per page (multiple of 8)        */
  int32_t num_pages;          /* PAGED only: pages in the pool                 */
  int32_t max_blocks_per_seq; /* PAGED only: row length of block_table         */
  int32_t symmetric;          /* 0: asymmetric, fp16 scale + zero per group;
                                 1: symmetric, fp16 scale only, codes offset
                                 by 2^(bits-1); must be 0 when bits == 16     */
  int32_t k_per_channel;      /* 1: axis-aware cache (bits 4/8,
                                 asymmetric): K grouped per channel over
                                 group_size consecutive tokens, V per token,
                                 fp16 sinks and residual window (see below)   */
  int32_t sink_tokens;        /* k_per_channel only: leading tokens kept fp16 */
  int32_t nf4;                /* 1: bits 4 coded as 16 normal-quantile levels
                                 with one fp16 absmax scale per group and no
                                 zero arrays (see kvq_append)                 */
} kvq_cache_desc;

typedef struct {              /* all device pointers, caller-owned             */
  void* k_codes;
  void* v_codes;
  uint16_t* k_scale;
  uint16_t* k_zero;
  uint16_t* v_scale;
  uint16_t* v_zero;
  const int32_t* block_table; /* PAGED only                                    */
  uint16_t* k_window;         /* k_per_channel only: fp16 sinks + residual     */
  uint16_t* v_window;
} kvq_cache;

/*
 * Bytes of K+V cache that `tokens` positions of ONE sequence occupy in one
 * layer: 2 * num_kv_heads * tokens * (row_bytes + 4 * groups), i.e. codes
 * plus a 4-byte fp16 scale+zero header per group ("What actually happens
 * when you quantize a KV cache", section 5; a symmetric or NF4 cache keeps
 * only the 2-byte scale; for bits == 16 the header is absent and this is
 * 2 * kv_heads * head_dim * 2 bytes per token, the formula of
 * "Quantization & inference optimisation", "What the cache costs").  Host
 * arithmetic only.  Returns 0 for an invalid descriptor.
 */
KVQ_API size_t kvq_cache_bytes(const kvq_cache_desc* desc, int64_t tokens);

/*
 * Bytes of each of k_window and v_window for `batch` sequences of an
 * axis-aware cache (batch * num_kv_heads * (sink_tokens + group_size) *
 * head_dim * 2); 0 for other caches or an invalid descriptor.
 */
KVQ_API size_t kvq_cache_window_bytes(const kvq_cache_desc* desc, int32_t batch);

/*
 * Allocation sizes for one layer's cache: *codes_bytes for each of k_codes
 * and v_codes, *header_bytes for each of k_scale, k_zero, v_scale, v_zero
 * (0 when bits == 16; a symmetric cache needs no zero arrays).  DENSE sizes
 * cover `batch` sequences of `capacity` slots; PAGED sizes cover num_pages
 * pages (`batch` is ignored).
 */
KVQ_API kvq_status kvq_cache_array_bytes(const kvq_cache_desc* desc, int32_t batch,
                                 size_t* codes_bytes, size_t* header_bytes);

/*
 * Quantize num_new new K and V vectors per sequence into the cache.
 *
 *   k_new, v_new     device fp16 [batch][num_new][num_kv_heads][head_dim]
 *   seq_lens_before  device int32 [batch]: tokens already cached; token t of
 *                    sequence b is written at position seq_lens_before[b]+t.
 *   dev_status       device uint32 (may be NULL)
 *
 * Per group of group_size consecutive channels of one vector: min and max;
 * s = fp16 rounded up from (max-min)/(2^bits-1) computed in fp64; z =
 * round-half-even(-min/s) in fp32, stored as an fp16 integer; codes
 * clamp(round-half-even(x/s) + z, 0, 2^bits-1) in fp32.  A constant group
 * stores s = |min| (1 if min == 0) so that it decodes exactly.  A zero-point
 * beyond +-2048 is clamped and flags KVQ_FLAG_ZERO_CLAMPED; a group with
 * inf/NaN is stored as s = z = 0, codes 0, and flags KVQ_FLAG_NONFINITE.
 * A position outside the cache (or an unmapped page) flags SEQ_LEN /
 * BLOCK_TABLE and that vector is not written.  Lengths are not modified:
 * the caller passes seq_lens_before + num_new to kvq_decode_attn.
 *
 * Symmetric caches (the zero-centred grid that "What actually happens when
 * you quantize a KV cache", section 3, compares against; the absmax
 * quantizer of "Serving many users at once", "Quantization: rounding the
 * weights"): per group a = max |x|; s = fp16 rounded up from
 * a/(2^(bits-1)-1) (s = 1 when a == 0); q = clamp(round-half-even(x/s),
 * -2^(bits-1), 2^(bits-1)-1) in fp32, stored as the code q + 2^(bits-1);
 * x_hat = (code - 2^(bits-1)) * s.  inf/NaN: s = 0, code 2^(bits-1), flagged.
 *
 * NF4 caches ("Gör inference billig", the NF4 paragraph: sixteen levels at
 * the quantiles of a normal distribution, block scaling): level i is the
 * (i + 1/2)/16 quantile of N(0, 1) divided by the outermost one, as fp16;
 * per group s = max |x| (an fp16 value, exact); the code is the level
 * nearest x/s (fp32 quotient, ties to the lower code); x_hat = level * s.
 * A group of zeros stores s = 0 (no level is 0); inf/NaN: s = 0, flagged;
 * codes are 0 where s = 0.
 *
 * Axis-aware caches: a token at a sink position or in the residual window is
 * stored as fp16.  When a token completes block j, the block is quantized
 * from the window and the new tokens: each K channel over the block's g
 * tokens, and each V token per group of g channels, with the formulas
 * above.  The tokens that remain in the residual window are then written
 * to their slots.  One call is two kernel launches, in stream order.
 * Axis-aware caches take at most KVQ_MAX_BATCH sequences per call (larger:
 * KVQ_ERR_UNSUPPORTED before any launch).
 * The window of an axis-aware sequence holds the newest tokens appended and no
 * others.  So its length is what has been appended: all num_new rows of a
 * padded batch count, and sequences of different numbers of new tokens take a
 * call each (with the sequence's part of the arrays, batch 1).  Nor can a
 * sequence of L tokens be cut back to any length: only to one of at most S
 * tokens, to a block's border S + j g, or to one within its last, unfinished
 * block.  Other lengths ask for window rows that have been replaced, which
 * nothing can flag.
 */
KVQ_API kvq_status kvq_append(const kvq_cache_desc* desc, const kvq_cache* cache,
                      int32_t batch, int32_t num_new,
                      const uint16_t* k_new, const uint16_t* v_new,
                      const int32_t* seq_lens_before, uint32_t* dev_status,
                      void* stream);

/*
 * Number of context splits kvq_decode_attn uses.  num_splits > 0 is taken
 * as given (capped so that every split holds at least one token tile);
 * num_splits == 0 lets the library choose from the SM count of the current
 * device (needs a device; returns 0 if none is available).
 */
KVQ_API int32_t kvq_decode_num_splits(const kvq_cache_desc* desc, int32_t batch,
                              int32_t num_q_heads, int32_t max_seq_len,
                              int32_t num_splits);

/*
 * Workspace bytes kvq_decode_attn needs for these arguments (0 when the
 * work runs in one split).  Same num_splits convention as above.
 */
KVQ_API size_t kvq_decode_workspace_size(const kvq_cache_desc* desc, int32_t batch,
                                 int32_t num_q_heads, int32_t max_seq_len,
                                 int32_t num_splits);

/*
 * Decode attention for one new query per sequence and query head.
 *
 *   q            device fp16 [batch][num_q_heads][head_dim]
 *   seq_lens     device int32 [batch]: cached tokens to attend over, the one
 *                just appended included.  0 gives a zero output row.
 *   max_seq_len  host upper bound on every seq_lens[b]; sizes the splits.
 *   num_splits   0 = library choice, else the split count (see above).
 *   softmax_scale  0 -> 1/sqrt(head_dim).
 *   out          device fp16 [batch][num_q_heads][head_dim]
 *   workspace    device scratch of kvq_decode_workspace_size() bytes
 *                (may be NULL when that size is 0); contents need no init.
 *
 * num_q_heads must be a multiple of num_kv_heads; query head h reads KV head
 * h / (num_q_heads / num_kv_heads).  For each (b, h):
 *   out = softmax(scale * q . k_hat_j) weighted sum of v_hat_j, j < seq_lens[b]
 * with k_hat = (q_k - z) * s dequantized in registers, fp32 accumulation,
 * an online softmax over token tiles and, when split, a log-sum-exp merge of
 * the per-split partials.  A length below 0 or above min(max_seq_len,
 * cache capacity) flags KVQ_FLAG_SEQ_LEN and yields a zero row; a token whose
 * page is unmapped flags KVQ_FLAG_BLOCK_TABLE and is left out.  batch is at
 * most KVQ_MAX_BATCH (one grid row per sequence); a larger batch returns
 * KVQ_ERR_UNSUPPORTED before any launch.
 */
KVQ_API kvq_status kvq_decode_attn(const kvq_cache_desc* desc, const kvq_cache* cache,
                           int32_t batch, int32_t num_q_heads,
                           const uint16_t* q, const int32_t* seq_lens,
                           int32_t max_seq_len, int32_t num_splits,
                           float softmax_scale, uint16_t* out,
                           void* workspace, size_t workspace_bytes,
                           uint32_t* dev_status, void* stream);

/*
 * One decode step in one call: kvq_append of one token per sequence followed
 * by kvq_decode_attn over the lengths seq_lens_before + 1 ("What actually
 * happens when you quantize a KV cache", section 3: the new K/V vectors are
 * quantized on arrival and attention then reads the quantized cache, the new
 * token included).
 *
 *   k_new, v_new     device fp16 [batch][num_kv_heads][head_dim]
 *   seq_lens_before  device int32 [batch]: tokens cached before this step; the
 *                    new token is written at position seq_lens_before[b] and
 *                    seq_lens_before[b] + 1 tokens are attended.
 *   max_seq_len      host upper bound on every seq_lens_before[b] + 1.
 *   the rest         as for kvq_decode_attn (same workspace size for the same
 *                    batch, num_q_heads, max_seq_len and num_splits).
 *
 * Cache contents and status flags are those of kvq_append (num_new = 1)
 * followed by kvq_decode_attn: the codes, scales and zero-points written are
 * bit-identical.  out is the same attention; it can differ from the two-call
 * result in fp32 rounding.  For per-token caches that the tensor-core kernel
 * takes (bits 4 and 8 and NF4 at head_dim 64 / 128, bits 2 at head_dim 128,
 * at most 8 query heads per KV head) this is one kernel launch (plus the
 * merge when split): the thread block that owns the new position quantizes
 * the token, stores it, and adds its dequantized K/V to the attention
 * directly.  Axis-aware caches of those shapes (group_size a multiple of 32,
 * bits 4 or 8) are one launch too when the call runs with one split: each
 * thread block, which owns one (sequence, KV head), first quantizes the
 * block its token completes (when it completes one) or reads the token from
 * k_new / v_new where the window would hold it, and stores it to its fp16
 * slot after attending.  Other shapes, and axis-aware caches split over the
 * context, run the append kernels and the decode in sequence.  Lengths are
 * not modified.
 */
KVQ_API kvq_status kvq_append_decode_attn(const kvq_cache_desc* desc, const kvq_cache* cache,
                                  int32_t batch, int32_t num_q_heads,
                                  const uint16_t* k_new, const uint16_t* v_new,
                                  const uint16_t* q, const int32_t* seq_lens_before,
                                  int32_t max_seq_len, int32_t num_splits,
                                  float softmax_scale, uint16_t* out,
                                  void* workspace, size_t workspace_bytes,
                                  uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * Prompts: several new tokens per sequence.  The calls below take a padded
 * batch: num_new token rows per sequence, of which sequence b uses the first
 * new_lens[b] (device int32 [batch]; NULL = all num_new).  The rows behind
 * are neither read nor written.  A new_lens[b] outside [0, num_new] or a
 * negative length flags KVQ_FLAG_SEQ_LEN and the sequence is skipped.
 * ------------------------------------------------------------------------ */

/*
 * Rotary positions.  Channels [0, rotary_dim) of a head form rotary_dim / 2
 * pairs, (2i, 2i+1) when interleaved, else (i, i + rotary_dim/2); pair i of
 * the token at position p turns by p * w_i radians and is scaled by the
 * amplitude:  y0 = a (x0 cos - x1 sin),  y1 = a (x1 cos + x0 sin).
 * The other channels pass unchanged.  w_i = base^(-2i / rotary_dim), changed
 * for contexts beyond the trained one by
 *   LINEAR  w_i / factor (position interpolation);
 *   NTK     base * factor^(rotary_dim / (rotary_dim - 2)) in place of base;
 *   BANDS   by turns in the original context, n = original_context w_i / 2pi:
 *           w_i where n >= high_turns, w_i / factor where n <= low_turns, and
 *           between them the mix with weight (n - low) / (high - low) on w_i;
 *   YARN    by pair index: w_i below lo = max(floor(at(high_turns)), 0),
 *           w_i / factor above hi = min(ceil(at(low_turns)), rotary_dim - 1),
 *           a linear ramp between, at(n) = rotary_dim ln(original_context /
 *           (2 pi n)) / (2 ln base); the amplitude is 0.1 ln(factor) + 1.
 * (LINEAR, NTK, YARN: the published methods of those names.)
 */
typedef enum {
  KVQ_ROPE_NONE = 0,
  KVQ_ROPE_LINEAR = 1,
  KVQ_ROPE_NTK = 2,
  KVQ_ROPE_BANDS = 3,
  KVQ_ROPE_YARN = 4
} kvq_rope_scaling;

#define KVQ_ROPE_MAX_PAIRS 128

typedef struct {
  int32_t rotary_dim;       /* even, 2 .. 256                                  */
  int32_t interleaved;      /* 1: pairs (2i, 2i+1); 0: (i, i + rotary_dim/2)   */
  int32_t scaling;          /* kvq_rope_scaling                                */
  int32_t original_context; /* BANDS, YARN: positions the model was trained on */
  double base;              /* > 1                                             */
  double factor;            /* >= 1; 1 when scaling is NONE                    */
  double low_turns;         /* BANDS: default 1; YARN: default 1  (0 = default)*/
  double high_turns;        /* BANDS: default 4; YARN: default 32 (0 = default)*/
  double amplitude;         /* 0 = as above (1, or YARN's); in (0, 4)          */
} kvq_rope_desc;

/* A filled rotation (host memory, passed by value to the kernels): turns[i]
 * is w_i / 2pi rounded to units of 2^-64 turns, so that position * turns[i]
 * modulo 2^64 is the angle without any further rounding, at any position. */
typedef struct {
  int32_t rotary_dim;
  int32_t interleaved;
  uint64_t amplitude;       /* units of 2^-61                                  */
  uint64_t turns[KVQ_ROPE_MAX_PAIRS];
} kvq_rope;

/* Fills *rope from *desc.  Host arithmetic only. */
KVQ_API kvq_status kvq_rope_init(const kvq_rope_desc* desc, kvq_rope* rope);

/*
 * Rotates q and / or k.
 *   q, q_out   device fp16 [batch][num_new][num_q_heads][head_dim]
 *   k, k_out   device fp16 [batch][num_new][num_k_heads][head_dim]
 *              (num_q_heads or num_k_heads 0: that tensor is not touched)
 *   positions        device int32 [batch][num_new], any value; or NULL:
 *   seq_lens_before  device int32 [batch]: token t of sequence b is at
 *                    position seq_lens_before[b] + t.
 * head_dim is a multiple of 8, rotary_dim <= head_dim <= 256.  x_out is x
 * itself (in place) or does not overlap it.  The angle is that of turns[]
 * exactly; cos, sin and the products carry 2^-42, and y is rounded once, so
 * it is the nearest fp16 to the formula's value unless that lies within
 * 2^-42 (|x0| + |x1|) of a tie.  An infinity or NaN in x gives one in y.
 */
KVQ_API kvq_status kvq_rope_apply(const kvq_rope* rope, int32_t head_dim, int32_t batch,
                          int32_t num_new, int32_t num_q_heads, const uint16_t* q,
                          uint16_t* q_out, int32_t num_k_heads, const uint16_t* k,
                          uint16_t* k_out, const int32_t* positions,
                          const int32_t* seq_lens_before, const int32_t* new_lens,
                          uint32_t* dev_status, void* stream);

/*
 * kvq_append of rotated keys, and the rotation of q, in one launch: the cache
 * and q_out are bit for bit those of kvq_rope_apply on q and k_new followed
 * by kvq_append of the result and v_new (num_q_heads 0: no q).  Unlike
 * kvq_append it takes new_lens.  Axis-aware caches: KVQ_ERR_UNSUPPORTED (call
 * kvq_rope_apply, then kvq_append).
 */
KVQ_API kvq_status kvq_rope_append(const kvq_cache_desc* desc, const kvq_cache* cache,
                           const kvq_rope* rope, int32_t batch, int32_t num_new,
                           const uint16_t* k_new, const uint16_t* v_new,
                           int32_t num_q_heads, const uint16_t* q, uint16_t* q_out,
                           const int32_t* seq_lens_before, const int32_t* new_lens,
                           uint32_t* dev_status, void* stream);

/*
 * Rotary positions by several axes (images: rows and columns; video: time
 * too).  A token has one position per axis, and every pair turns by the
 * position of its axis.
 *   pairs[a]    pairs of axis a; together rotary_dim / 2
 *   cycled      0: the pairs of an axis follow one another, axis by axis;
 *               1: the axes take turns, pair by pair, while they have pairs left
 *   own_ladders 0: pair i turns by w_i, whatever its axis; 1: the j-th pair of
 *               axis a turns as pair j of a rotation of 2 pairs[a] channels
 * (scaling YARN with own_ladders: the amplitude is the same for every axis.)
 */
#define KVQ_ROPE_MAX_AXES 4

typedef struct {
  kvq_rope_desc rope;       /* rotary_dim = twice the pairs of all axes        */
  int32_t num_axes;         /* 1 .. KVQ_ROPE_MAX_AXES                          */
  int32_t pairs[KVQ_ROPE_MAX_AXES];  /* >= 1 for a < num_axes                  */
  int32_t cycled;
  int32_t own_ladders;
} kvq_rope_axes_desc;

typedef struct {
  kvq_rope rope;
  int32_t num_axes;
  uint8_t axis[KVQ_ROPE_MAX_PAIRS];  /* of each pair, below num_axes           */
} kvq_rope_axes;

/* Fills *axes from *desc.  Host arithmetic only. */
KVQ_API kvq_status kvq_rope_axes_init(const kvq_rope_axes_desc* desc, kvq_rope_axes* axes);

/*
 * kvq_rope_apply with a position per axis:
 *   positions  device int32 [batch][num_new][num_axes], any value
 * Angles, roundings and the rest as there.
 */
KVQ_API kvq_status kvq_rope_axes_apply(const kvq_rope_axes* axes, int32_t head_dim, int32_t batch,
                               int32_t num_new, int32_t num_q_heads, const uint16_t* q,
                               uint16_t* q_out, int32_t num_k_heads, const uint16_t* k,
                               uint16_t* k_out, const int32_t* positions,
                               const int32_t* new_lens, uint32_t* dev_status, void* stream);

/*
 * kvq_rope_append with a position per axis: the angles come from positions
 * (as above), the cache rows from seq_lens_before[b] + t.  Bit for bit
 * kvq_rope_axes_apply on q and k_new followed by the append of the result and
 * v_new.  Axis-aware caches: KVQ_ERR_UNSUPPORTED, as there.
 */
KVQ_API kvq_status kvq_rope_axes_append(const kvq_cache_desc* desc, const kvq_cache* cache,
                                const kvq_rope_axes* axes, int32_t batch, int32_t num_new,
                                const uint16_t* k_new, const uint16_t* v_new,
                                int32_t num_q_heads, const uint16_t* q, uint16_t* q_out,
                                const int32_t* positions, const int32_t* seq_lens_before,
                                const int32_t* new_lens, uint32_t* dev_status, void* stream);

/*
 * Reads cached rows back: row t of sequence b is position start[b] + t, for
 * the t < num_rows with start[b] + t < seq_lens[b]; rows behind are left as
 * they were.
 *   seq_lens      device int32 [batch]: tokens cached (axis-aware caches: all
 *                 that have been appended, see kvq_append)
 *   start         device int32 [batch]
 *   k_out, v_out  device fp16 [batch][num_rows][num_kv_heads][head_dim]
 *                 (either may be NULL)
 * The value is x_hat = (q - z) s (fp32), rounded to fp16 and held at the
 * largest finite fp16; fp16 rows are copied.  A negative start, a length
 * outside the cache or an unmapped page is flagged and its rows are left.
 */
KVQ_API kvq_status kvq_cache_read(const kvq_cache_desc* desc, const kvq_cache* cache,
                          int32_t batch, int32_t num_rows, const int32_t* seq_lens,
                          const int32_t* start, uint16_t* k_out, uint16_t* v_out,
                          uint32_t* dev_status, void* stream);

/* Splits and workspace of kvq_extend_attn; the conventions of
 * kvq_decode_num_splits and kvq_decode_workspace_size. */
KVQ_API int32_t kvq_extend_num_splits(const kvq_cache_desc* desc, int32_t batch, int32_t num_new,
                              int32_t num_q_heads, int32_t max_seq_len, int32_t num_splits);
KVQ_API size_t kvq_extend_workspace_size(const kvq_cache_desc* desc, int32_t batch,
                                 int32_t num_new, int32_t num_q_heads, int32_t max_seq_len,
                                 int32_t num_splits);

/*
 * Causal attention of several new tokens per sequence over the cache, their
 * own rows included (kvq_append or kvq_rope_append has written them): a
 * prompt, a chunk of one, the suffix behind shared pages, drafted tokens.
 *   q                device fp16 [batch][num_new][num_q_heads][head_dim]
 *   seq_lens_before  device int32 [batch]: tokens cached before the new ones;
 *                    token t attends to positions [0, seq_lens_before[b] + t].
 *   max_seq_len      host upper bound on seq_lens_before[b] + new_lens[b]
 *   out              device fp16 like q; may not overlap it
 * Axis-aware caches: seq_lens_before[b] + new_lens[b] is all that has been
 * appended to the sequence (see kvq_append).
 * num_splits, softmax_scale and workspace as for kvq_decode_attn, but any
 * number of query heads per KV head.  Scores and softmax in fp32; K and V
 * enter the products as x_hat = (q - z) s, held at fp16's largest and otherwise
 * exact (as the sum of two fp16 numbers; NF4 values to within 2^-25), the
 * probabilities as fp16 (11 bits down to 2^-21 of the row's largest).  An infinity or NaN in a token's V row makes
 * NaN or infinities of the rows that see the token, possibly in more channels
 * than its own; rows that do not see it are untouched.  A sequence whose
 * length exceeds min(max_seq_len, cache capacity) flags KVQ_FLAG_SEQ_LEN and
 * yields zero rows; a token whose page is unmapped flags KVQ_FLAG_BLOCK_TABLE
 * and is left out; a row with nothing to attend to is zero.
 * The kernel's warps hand tiles to one another; should such a wait last two
 * seconds, which no input causes, the thread block gives up and its rows of
 * `out` are not written (or joined from what the workspace held).  Only
 * KVQ_FLAG_TIMEOUT in *dev_status tells, so pass it where that matters.
 */
KVQ_API kvq_status kvq_extend_attn(const kvq_cache_desc* desc, const kvq_cache* cache,
                           int32_t batch, int32_t num_new, int32_t num_q_heads,
                           const uint16_t* q, const int32_t* seq_lens_before,
                           const int32_t* new_lens, int32_t max_seq_len, int32_t num_splits,
                           float softmax_scale, uint16_t* out, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * Page pool: which pages the sequences of a paged cache hold.  One pool
 * serves every layer (the layers' caches share the block table).  Its state
 * is the block table and a reference count per page; a page with count 0 is
 * free, and pages are always taken lowest first, so the same calls give the
 * same tables.  All of it runs on the device, in stream order.
 * For an axis-aware cache the pool's positions are those after the sinks, and
 * the fp16 windows, which are per sequence, are the caller's to copy; which
 * lengths a sequence can be trimmed to, kvq_append says.
 * ------------------------------------------------------------------------ */

/* Largest batch of a pool (kvq_pages_reserve holds the batch on chip). */
#define KVQ_MAX_POOL_BATCH 16384

typedef struct {
  int32_t num_pages;
  int32_t page_size;          /* tokens per page                               */
  int32_t batch;              /* rows of the block table                       */
  int32_t max_blocks_per_seq;
  int32_t* ref_count;         /* device [num_pages]: block-table entries on it */
  int32_t* block_table;       /* device [batch][max_blocks_per_seq]; -1: none  */
} kvq_page_pool;

/* Device scratch of kvq_pages_reserve and kvq_pages_compact. */
KVQ_API size_t kvq_pages_workspace_size(const kvq_page_pool* pool);

/*
 * Fork, trim, permute and free: every row of the table becomes the first
 * ceil(keep_lens[b] / page_size) entries of the row parent[b] had before the
 * call, -1 behind; reference counts follow, so pages nobody holds any more
 * are free.  parent[b] = b keeps a sequence, -1 frees it, a parent named by
 * several rows is forked (its pages are shared, no data moves).
 *   parent     device int32 [batch], -1 .. batch-1 (others flag
 *              KVQ_FLAG_BLOCK_TABLE and count as -1)
 *   keep_lens  device int32 [batch], or NULL for whole rows; outside
 *              [0, page_size * max_blocks_per_seq]: KVQ_FLAG_SEQ_LEN, as -1
 */
KVQ_API kvq_status kvq_pages_reorder(const kvq_page_pool* pool, const int32_t* parent,
                             const int32_t* keep_lens, uint32_t* dev_status, void* stream);

/*
 * Makes positions [seq_lens_before[b], seq_lens_before[b] + new_lens[b])
 * writable for every sequence: blocks without a page get one, and a page
 * shared with another sequence is replaced by a fresh one:
 *   - a page in which the sequence keeps tokens (the first block, when
 *     seq_lens_before[b] lies inside it) has to be copied first; where all
 *     holders of such a page ask for it in this way, the last of them keeps it;
 *   - a page that is written from its start (sequences forked without a trim,
 *     then rewound) is replaced without a copy for every holder that asks, the
 *     last one included.
 *   copy_src, copy_dst  device int32 [batch]: the pair of sequence b, or -1;
 *                       pass them to kvq_pages_copy for every layer, before
 *                       the new tokens are appended and before pages are
 *                       reserved again (a source may be free by now)
 *   granted             device int32 [batch] or NULL: new_lens[b] (num_new
 *                       when new_lens is NULL); 0 for a skipped sequence
 * With too few free pages nothing changes for any sequence: KVQ_FLAG_POOL_EMPTY,
 * no copies, granted 0 throughout (pass granted as new_lens to the calls that
 * write and nothing is written).  A call whose sequences could touch 2^31
 * blocks together: KVQ_ERR_UNSUPPORTED.
 */
KVQ_API kvq_status kvq_pages_reserve(const kvq_page_pool* pool, const int32_t* seq_lens_before,
                             const int32_t* new_lens, int32_t num_new, int32_t* copy_src,
                             int32_t* copy_dst, int32_t* granted, void* workspace,
                             size_t workspace_bytes, uint32_t* dev_status, void* stream);

/*
 * Compacts the pool: with n pages in use, the k-th page at or behind n moves
 * to the k-th free page before n; table and counts follow.
 *   move_src, move_dst  device int32 [num_pages / 2]: the moves, -1 behind;
 *                       pass them to kvq_pages_copy for every layer
 *   num_live            device int32 [1]: n
 * An entry of the table that names a page of count 0 becomes -1
 * (KVQ_FLAG_BLOCK_TABLE).
 */
KVQ_API kvq_status kvq_pages_compact(const kvq_page_pool* pool, int32_t* move_src,
                             int32_t* move_dst, int32_t* num_live, void* workspace,
                             size_t workspace_bytes, uint32_t* dev_status, void* stream);

/*
 * Copies pages in num_layers caches of one descriptor (caches: host array):
 * page copy_dst[i] takes the bytes of page copy_src[i], i < num_pairs (device
 * arrays; pairs with a -1 are skipped).  No page may be the target of two
 * pairs, or source and target; then KVQ_FLAG_PAGE_LIST is set and the
 * contents of the targets concerned are unspecified.  An index outside the
 * pool flags KVQ_FLAG_BLOCK_TABLE and its pair is skipped; skipped pairs do
 * not count in the list.
 */
KVQ_API kvq_status kvq_pages_copy(const kvq_cache_desc* desc, const kvq_cache* caches,
                          int32_t num_layers, const int32_t* copy_src, const int32_t* copy_dst,
                          int32_t num_pairs, uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * Shared prefixes: sequences whose first tokens are the same (a system prompt,
 * a document or video with many questions about it, parallel samples of one
 * prompt) attend to them together, and the prefix is read once for all of them.
 * A prefix is a sequence of one cache, and every sequence's own tokens, its
 * tail, are a sequence of another (or of the same pages through another block
 * table, which kvq_prefix_find makes).  The two caches may differ in format,
 * layout and size; num_kv_heads and head_dim are the same.
 * ------------------------------------------------------------------------ */

/* Most prefixes of a plan. */
#define KVQ_MAX_PREFIXES 65535

/* Bytes of a plan; 0 for sizes that cannot be. */
KVQ_API size_t kvq_prefix_plan_size(int32_t batch, int32_t num_prefixes);

/*
 * Which sequence is on which prefix, once for all layers of a step.
 *   prefix_of    device int32 [batch]: 0 .. num_prefixes - 1, or -1 (none)
 *   prefix_lens  device int32 [num_prefixes]: tokens of each prefix; 0: empty
 *   plan         device, kvq_prefix_plan_size() bytes, 16-byte aligned: read by
 *                kvq_prefix_attn, which needs neither array again
 *                (may not overlap either of them)
 * Another prefix_of flags KVQ_FLAG_BLOCK_TABLE and counts as none, a negative
 * length KVQ_FLAG_SEQ_LEN and as empty.
 */
KVQ_API kvq_status kvq_prefix_plan(int32_t batch, int32_t num_prefixes, const int32_t* prefix_of,
                           const int32_t* prefix_lens, void* plan, size_t plan_bytes,
                           uint32_t* dev_status, void* stream);

/* Device scratch of kvq_prefix_find. */
KVQ_API size_t kvq_prefix_find_workspace_size(const kvq_page_pool* pool);

/*
 * The prefixes that a page pool's sequences share, from its block table alone.
 * With S tokens a page, sequence b holds n_b = seq_lens_before[b] / S whole
 * pages; k = max(1, ceil(min_tokens / S)):
 *   - a sequence with n_b >= k and a page in block k - 1 belongs to the group
 *     of the sequences with the same page there; its leader is the lowest one;
 *   - its run is the number of leading blocks that hold the leader's pages, at
 *     most min(n_b, n_leader); with a run below k it belongs to no group;
 *   - a group's prefix is as many blocks as some member's run r for which
 *     (members with a run >= r, less one) * r, the blocks not read again, is
 *     largest (the longest of equal ones); with nothing saved it has none;
 *   - members with a run of at least that are on the prefix.
 * Prefixes are numbered by their leaders, ascending; of more than max_prefixes
 * the first are kept.  The shared pages are whole, so tokens appended behind
 * seq_lens_before change none of them.
 *   prefix_of      device int32 [batch], -1: none
 *   prefix_lens    device int32 [max_prefixes]; 0 behind the last
 *   prefix_table   device int32 [max_prefixes][max_blocks_per_seq]; -1 behind
 *   tail_table     device int32 [batch][max_blocks_per_seq]: each row of the
 *                  pool's table without the prefix's blocks; -1 behind
 *   tail_lens      device int32 [batch]: seq_lens_before less the prefix
 *   num_prefixes   device int32 [1] or NULL: prefixes found, those beyond
 *                  max_prefixes among them
 * No array that is written may overlap another of the call.
 * kvq_prefix_plan takes prefix_of and prefix_lens; kvq_prefix_attn the pool's
 * caches with the two tables and tail_lens.  Appending goes through the pool's
 * own table and lengths.  For per-token caches: an axis-aware sequence's sinks
 * and window are not in the table.  A length that cannot be flags
 * KVQ_FLAG_SEQ_LEN; that sequence has no prefix and keeps its length.  batch *
 * max_blocks_per_seq^2 of 2^62 and above: KVQ_ERR_UNSUPPORTED.
 */
KVQ_API kvq_status kvq_prefix_find(const kvq_page_pool* pool, const int32_t* seq_lens_before,
                           int32_t min_tokens, int32_t max_prefixes, int32_t* prefix_of,
                           int32_t* prefix_lens, int32_t* prefix_table, int32_t* tail_table,
                           int32_t* tail_lens, int32_t* num_prefixes, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, void* stream);

/* Device scratch of kvq_prefix_attn (the splits as there). */
KVQ_API size_t kvq_prefix_attn_workspace_size(const kvq_cache_desc* prefix_desc,
                                      const kvq_cache_desc* desc, int32_t num_prefixes,
                                      int32_t batch, int32_t num_new, int32_t num_q_heads,
                                      int32_t max_prefix_len, int32_t max_seq_len,
                                      int32_t prefix_splits, int32_t tail_splits);

/*
 * Attention of one or several new tokens per sequence over its prefix and its
 * tail, the new tokens' own rows included (already appended to the tail): for
 * num_new = 1 a decode step, else as kvq_extend_attn.
 *   prefix_desc, prefix_cache  num_prefixes sequences (num_prefixes 0: NULL)
 *   desc, cache                batch tails
 *   q                device fp16 [batch][num_new][num_q_heads][head_dim]
 *   seq_lens_before  device int32 [batch]: tokens of the tail before the new
 *                    ones; token t attends to the whole prefix and to the
 *                    tail's positions [0, seq_lens_before[b] + t]
 *   new_lens         device int32 [batch] or NULL, as above
 *   plan             of kvq_prefix_plan, for this batch and num_prefixes
 *   max_prefix_len   host upper bound on the prefixes' lengths
 *   max_seq_len      host upper bound on seq_lens_before[b] + new_lens[b]
 * Kernels and splits are chosen by the host from these numbers, as if the batch
 * were shared out evenly over min(num_prefixes, batch) prefixes of
 * max_prefix_len tokens, with tails of max_seq_len: the nearer the truth, the
 * better the choice, and slots that kvq_prefix_find left empty are far from it
 * (give it few max_prefixes, or read its num_prefixes where a search serves
 * many steps).  What the caches hold is bound enough for any length.
 *   prefix_splits, tail_splits  0: library choice, else as num_splits of
 *                    kvq_decode_attn, for each of the two
 *   out              device fp16 like q
 *   workspace        kvq_prefix_attn_workspace_size() bytes for the same sizes
 *                    and splits (may be NULL when that is 0); calls that can
 *                    overlap on the GPU need one each
 * Neither out nor the workspace may overlap the other, q, the lengths or the plan.
 * (A row of q without a new token may be read, to no effect; its row of out is
 * not written.)
 * Axis-aware caches: a prefix's length is all that has been appended to it.
 * (Where sharing does not pay: axis-aware caches with one new token a sequence,
 * which kvq_decode_attn reads faster, and new tokens by the hundred over codes,
 * which are bound by their products.)
 * Precision: over the prefix as in kvq_extend_attn; INT4, INT8 and NF4 caches
 * may, where rows are few, take codes, scales and zero-points apart: a weight
 * times V's scale is then rounded to fp16 once more (11 bits, down to 2^-25 of
 * the row's largest weight times the group's largest scale), and the sums of
 * codes and of zero-points in fp32 are subtracted.  Over the tail as in
 * kvq_decode_attn (one new token, shapes its tensor-core kernels take) or
 * kvq_extend_attn; the partial results are joined in fp32.  A tail whose length
 * exceeds min(max_seq_len, its cache's capacity) flags KVQ_FLAG_SEQ_LEN and
 * yields zero rows.  A prefix longer than min(max_prefix_len, its cache's
 * capacity) flags KVQ_FLAG_SEQ_LEN and is left out; so is a token whose page
 * is unmapped (KVQ_FLAG_BLOCK_TABLE).  KVQ_FLAG_TIMEOUT as there.
 */
KVQ_API kvq_status kvq_prefix_attn(const kvq_cache_desc* prefix_desc, const kvq_cache* prefix_cache,
                           int32_t num_prefixes, const kvq_cache_desc* desc,
                           const kvq_cache* cache, int32_t batch, int32_t num_new,
                           int32_t num_q_heads, const uint16_t* q,
                           const int32_t* seq_lens_before, const int32_t* new_lens,
                           const void* plan, size_t plan_bytes, int32_t max_prefix_len,
                           int32_t max_seq_len, int32_t prefix_splits, int32_t tail_splits,
                           float softmax_scale, uint16_t* out, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, void* stream);

/* Size of the library's own split scratch used by kvq_decode_attn_static_ws. */
#define KVQ_STATIC_WORKSPACE_BYTES ((size_t)8 << 20)

/*
 * kvq_decode_attn without a caller workspace: the split partials go to a
 * static device array of KVQ_STATIC_WORKSPACE_BYTES inside the library.
 * The pages have no counterpart to this call. It exists for callers that
 * cannot allocate device memory around a decode call, such as a plugin that
 * is handed only its input and output buffers, or code whose device
 * footprint must stay fixed after start-up.
 *
 * Arguments, results and status flags are those of kvq_decode_attn. The
 * workspace is the library's array.
 *
 *   - Set-up: the first call on each device, with that device current,
 *     looks up the array's device address (cudaGetSymbolAddress) and keeps
 *     it with the identifier of the device's current context. This may load
 *     the library's device code on that device. Make that first call before
 *     any stream capture. A later call in a different context (after
 *     cudaDeviceReset, say) looks the address up again, since the array then
 *     lives elsewhere; make that call before any capture as well.
 *   - Size limit: when kvq_decode_workspace_size() for the same arguments
 *     exceeds KVQ_STATIC_WORKSPACE_BYTES, the call returns KVQ_ERR_WORKSPACE
 *     before any launch. Pass a smaller num_splits, or use kvq_decode_attn.
 *   - Allocation: none. No cudaMalloc, no cudaFree, no allocating library
 *     routine.
 *   - Initial contents: nothing in the array has to start at zero. Each
 *     call writes every partial it reads.
 *   - Concurrency: one array serves every call on a device. Calls whose
 *     kernels can overlap on the GPU race on it and give wrong results. That
 *     covers calls on different streams without ordering between them, and
 *     calls from several host threads. Calls on one stream are safe.
 */
KVQ_API kvq_status kvq_decode_attn_static_ws(const kvq_cache_desc* desc, const kvq_cache* cache,
                                     int32_t batch, int32_t num_q_heads,
                                     const uint16_t* q, const int32_t* seq_lens,
                                     int32_t max_seq_len, int32_t num_splits,
                                     float softmax_scale, uint16_t* out,
                                     uint32_t* dev_status, void* stream);

/*
 * Debug builds.  build(debug=True) in quantized_kv_decode_gb300/build.py
 * compiles the same sources with KVQ_DEBUG defined into libkvq_debug.so,
 * which exports the same entry points.  There each launch carries the byte
 * extent of every caller array it may touch, derived on the host from the
 * descriptor and the call's sizes:
 *   cache arrays   kvq_cache_array_bytes(desc, batch) each (DENSE: the
 *                  call's batch of sequences; PAGED: num_pages), the
 *                  windows kvq_cache_window_bytes(desc, batch) each;
 *   block_table    batch * max_blocks_per_seq int32;
 *   q, out         batch * num_q_heads * head_dim fp16 each;
 *   k_new, v_new   batch * num_new * num_kv_heads * head_dim fp16 each;
 *   seq_lens / seq_lens_before   batch int32;
 *   workspace      workspace_bytes (the static array for the
 *                  _static_ws call).
 *   kvq_cache_read: k_out and v_out as k_new and v_new with num_rows tokens;
 *   kvq_extend_attn: q and out batch * num_new rows; kvq_prefix_attn: the same,
 *   its prefixes' cache with num_prefixes sequences; kvq_rope_append and
 *   kvq_rope_axes_append: k_new and v_new.  The other arrays of the prompt, pool
 *   and prefix calls (q of the rotations, positions, new_lens, start, the pool's,
 *   the copy lists, plans) are read and written at indexes the kernels have
 *   checked against the sizes given, in every build, and carry no extents.
 * Every global load and store of the arrays above first checks that its bytes
 * lie inside the extent of the array it addresses.  An access that does not is
 * skipped (a load yields zeros), and KVQ_FLAG_OOB is OR-ed into *dev_status
 * (when dev_status is not NULL).  The checks cost time; results are otherwise
 * those of the release library, which never sets KVQ_FLAG_OOB.
 */

/* 1 when the loaded library is a debug build (bounds checks compiled in). */
KVQ_API int32_t kvq_debug_checks(void);

/* The caller arrays a debug build checks, named for kvq_debug_shrink_extent. */
typedef enum {
  KVQ_ARRAY_K_CODES = 0,
  KVQ_ARRAY_V_CODES = 1,
  KVQ_ARRAY_K_SCALE = 2,
  KVQ_ARRAY_K_ZERO = 3,
  KVQ_ARRAY_V_SCALE = 4,
  KVQ_ARRAY_V_ZERO = 5,
  KVQ_ARRAY_K_WINDOW = 6,
  KVQ_ARRAY_V_WINDOW = 7,
  KVQ_ARRAY_BLOCK_TABLE = 8,
  KVQ_ARRAY_Q = 9,
  KVQ_ARRAY_K_NEW = 10,
  KVQ_ARRAY_V_NEW = 11,
  KVQ_ARRAY_SEQ_LENS = 12,   /* seq_lens or seq_lens_before */
  KVQ_ARRAY_OUT = 13,
  KVQ_ARRAY_WORKSPACE = 14,
  KVQ_ARRAY_COUNT = 15
} kvq_array;

/*
 * Tests the checks themselves (debug builds only; a release build returns
 * KVQ_ERR_UNSUPPORTED).  Every later launch checks array `array` (a
 * kvq_array) against an extent `bytes` shorter than the one the host derives
 * (bytes = 0 restores it).  Accesses to the array's last `bytes` bytes are
 * then skipped and flagged although they lie inside the caller's allocation.
 * Process-wide host state; not safe to call while another thread launches.
 * Returns KVQ_ERR_INVALID_ARG for an unknown array or bytes < 0.
 */
KVQ_API kvq_status kvq_debug_shrink_extent(int32_t array, int64_t bytes);

/* The waits of kvq_extend_attn's tensor-core kernel (head_dim 64 and 128,
 * per-token formats), by the warp that waits, named for kvq_debug_fail_wait. */
typedef enum {
  KVQ_WAIT_NONE = 0,
  KVQ_WAIT_SOFTMAX = 1,     /* a softmax warp for a key tile's scores           */
  KVQ_WAIT_K = 2,           /* a warp that turns K codes into fp16 (fp16 caches:
                               that copies rows)                                */
  KVQ_WAIT_V = 3,           /* the same for V (fp16 caches: never)              */
  KVQ_WAIT_LOAD_K = 4,      /* the warp that copies K codes (fp16 caches: that
                               passes stages on)                                */
  KVQ_WAIT_LOAD_V = 5,      /* the same for V (fp16 caches: never)              */
  KVQ_WAIT_SCORES = 6,      /* the first warp that issues products, for K       */
  KVQ_WAIT_SUM = 7,         /* the same, between the halves of a weighted sum   */
  KVQ_WAIT_COUNT = 8
} kvq_debug_wait;

/*
 * Tests what happens when a wait runs out (debug builds only; a release build
 * returns KVQ_ERR_UNSUPPORTED).  In every later launch of that kernel the wait
 * `wait` (a kvq_debug_wait) for key tile `tile` of a thread block's share
 * counts as run out at once: the block gives up, waits for its copies and
 * products in flight, writes no more output and sets KVQ_FLAG_TIMEOUT.
 * KVQ_WAIT_NONE ends that.  Process-wide host state, as above.  Returns
 * KVQ_ERR_INVALID_ARG for an unknown wait or tile < 0.
 */
KVQ_API kvq_status kvq_debug_fail_wait(int32_t wait, int32_t tile);

/* Static, human-readable name of a status code. */
KVQ_API const char* kvq_status_string(kvq_status status);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
