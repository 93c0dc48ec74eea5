/*
 * dsa.h -- C ABI of the GB300 (sm_103a) DeepSeek-V4 DSA indexer hot path.
 *
 * The library computes, on one GPU, the three stages of the DeepSeek-V4
 * sparse-attention indexer:
 *
 *   1. the indexer score  logits[t, j] = sum_h w[t, h] * relu(q[t, h, :] . k[j, :])
 *      (xkernels issue #27 "DSA indexer + attention: validate/provide gfx942
 *      forward path", comment 2 "What shipped"; H = index_n_heads = 64,
 *      D = index_head_dim = 128 per the same issue's "Context");
 *   2. a per-query top-k under a fixed tie rule (larger value first, then the
 *      smaller key index), the deterministic "canonical" top-k sort of README
 *      "DeepSeek V4 Flash on a single AMD MI300X" (overlay table);
 *   3. the paged mxfp4 gather of the selected positions to bf16 (xkernels
 *      issue #28 "DeepSeek-V4 serving support -- tracking", comment 2 "What it
 *      does").
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every pointer argument is caller-owned DEVICE memory unless stated
 *   otherwise.  No call allocates or frees memory, synchronises, or keeps a
 *   pointer after it returns.  Calls are asynchronous on `stream` (a
 *   cudaStream_t passed as void*; NULL = the legacy default stream) and run on
 *   the device current to the calling thread.
 * - Query rows: T = B * next_n.  Row t belongs to sequence b = t / next_n and is
 *   query i = t % next_n of it, at absolute position p = L_b - next_n + i, where
 *   L_b = context_lens[b].  With causal != 0 the row sees keys j <= p (and
 *   j < L_b); otherwise every j < L_b.  This is this library's reading of the
 *   "optional per-query causal window" of xkernels issue #27, comment 2.
 * - Host-detectable argument errors return DSA_ERR_INVALID_ARG (or
 *   DSA_ERR_UNSUPPORTED for valid but unimplemented shapes) BEFORE anything is
 *   launched; outputs are then untouched.  A failed launch returns DSA_ERR_CUDA.
 * - Bad indices found on the device (a block id outside [0, num_blocks), a
 *   block-table column outside [0, bt_stride)) never cause an out-of-range
 *   access: the affected key is treated as masked (not selected, logit -inf) or
 *   the gathered row is written as zeros, and a bit is set in the per-device
 *   error word read by dsa_device_error().  A device-side wait that exceeds its
 *   time limit abandons the call's work, sets DSA_DEVERR_TIMEOUT in the same
 *   word and returns without hanging; outputs of that call are then undefined.
 * - v1 supports H = 64 and D = 128 (DSA_ERR_UNSUPPORTED otherwise); they stay
 *   parameters so the ABI does not change when other shapes are added.
 */
#ifndef DSA_GB300_H_
#define DSA_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,   /* bad pointer / size / stride / alignment      */
  DSA_ERR_UNSUPPORTED = 2,   /* valid request this build does not implement  */
  DSA_ERR_CUDA = 3,          /* a CUDA runtime or launch error               */
  DSA_ERR_WORKSPACE = 4      /* ws is NULL or smaller than dsa_workspace_bytes */
} dsa_status;

/* Storage of the indexer's inputs.  DSA_BF16: bf16 q and keys.  DSA_E4M3: OCP E4M3 q
 * and keys with fp32 row scales.  DSA_E4M3_MXFP4K: OCP E4M3 q (with q_scale) scored
 * against keys read straight from the paged mxfp4 cache (the fp8-q x fp4-k MQA-logits
 * form that xkernels issue #27 "DSA indexer + attention: validate/provide gfx942
 * forward path", "Status", names; see dsa_keys.scale_e8m0). */
typedef enum { DSA_BF16 = 0, DSA_E4M3 = 1, DSA_E4M3_MXFP4K = 2 } dsa_dtype;

/* Storage of hidden rows and of a projection's result. */
typedef enum { DSA_REAL_BF16 = 0, DSA_REAL_F32 = 1 } dsa_real;

/* Which dims of a head turn together: (2i, 2i + 1), or (i, i + rope_dim / 2). */
typedef enum { DSA_ROPE_INTERLEAVED = 0, DSA_ROPE_HALF = 1 } dsa_rope_layout;

/* Frequencies of rotary positions; see dsa_rope_table. */
typedef enum { DSA_ROPE_PLAIN = 0, DSA_ROPE_LINEAR = 1, DSA_ROPE_YARN = 2 } dsa_rope_scaling;
typedef struct {
  double base;               /* > 1, e.g. 10000                                          */
  dsa_rope_scaling scaling;
  double factor;             /* LINEAR, YARN: >= 1, how much longer the context gets     */
  double original_max_pos;   /* YARN: the context the frequencies were trained for       */
  double beta_fast;          /* YARN: turns within it above which a pair is kept         */
  double beta_slow;          /* YARN: turns below which it is slowed by the factor       */
  double amplitude;          /* multiplies cos and sin (1 for none); within fp32's range  */
} dsa_rope_params;

/*
 * Paged bf16 cache of keys and values (DEVICE memory): head h of position j of sequence b is
 * the D elements at k (or v) + block * block_stride + (j % block_size) * row_stride +
 * h * head_stride with block = block_table[b * bt_stride + j / block_size], strides in
 * elements.  [num_blocks, block_size, heads, D] and [num_blocks, heads, block_size, D] are
 * both cases of it.  v may be k (keys that are their own values).
 */
typedef struct {
  void* k;
  void* v;
  int64_t num_blocks;
  int32_t block_size;
  int64_t block_stride;
  int64_t row_stride;
  int64_t head_stride;
} dsa_kv_cache;

typedef enum { DSA_OP_TOPK = 1, DSA_OP_LOGITS_TOPK = 2 } dsa_op;

/* Bits of the per-device error word (see dsa_device_error). */
#define DSA_DEVERR_INDEX    1u  /* a block id / block-table column was out of range    */
#define DSA_DEVERR_TIMEOUT  2u  /* a bounded device-side wait expired                  */
#define DSA_DEVERR_OVERFLOW 4u  /* an on-chip candidate buffer would have overflowed:
                                   the candidate was dropped (an internal error; bits
                                   8..15 then name the library's internal site)        */

/*
 * Key source of the indexer (the shared MQA key of xkernels issue #27,
 * comment 2).  Keys are rows of D elements, row-major, d fastest; each row
 * starts 16-byte aligned (D * element size is a multiple of 16).
 *  - Paged (block_table != NULL): `data` is a pool of num_rows rows (num_rows =
 *    number of physical blocks * block_size).  Logical key j of sequence b is
 *    pool row block_table[b * bt_stride + j / block_size] * block_size +
 *    j % block_size.  block_size must be a multiple of 8 that divides 128 or is
 *    a multiple of 128; bt_stride >= ceil(L_b / block_size) for every b.
 *  - Contiguous (block_table == NULL): only B == 1; key j is row j, num_rows >= L_0.
 * `scale` is the per-row fp32 scale of E4M3 keys (same row indexing as `data`,
 * non-negative), NULL for bf16.
 * With dtype DSA_E4M3_MXFP4K the keys are rows of the paged mxfp4 cache that
 * mxfp4_paged_gather reads: `data` holds D/2 nibble bytes per row (low nibble = even
 * element, E2M1), `scale_e8m0` D/32 E8M0 bytes per row (2^(b-127), 0xFF -> 0), both
 * 16-byte aligned; `scale` is unused; a contiguous key array needs num_rows % 4 == 0.
 * The key's value is E2M1 * 2^(b-127) exactly; the tensor cores take the codes and
 * scale bytes as stored (block-scaled MMA, one scale per 32 elements).  Scale bytes
 * >= 254 can overflow the fp32 scores and are outside this mode's domain.
 */
typedef struct {
  const void* data;
  const float* scale;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t block_size;
  int64_t num_rows;
  const uint8_t* scale_e8m0;
} dsa_keys;

/*
 * Query batch layout.  context_lens is DEVICE memory [B] (int32, 0 <= L_b <=
 * max_context_len); max_context_len is a host-side upper bound used to size
 * launches and the logits width.
 */
typedef struct {
  int32_t B;
  int32_t next_n;
  const int32_t* context_lens;
  int32_t max_context_len;
  int32_t causal;
} dsa_queries;

/*
 * dsa_indexer_logits -- indexer score (xkernels issue #27, comment 2 "What
 * shipped"): logits[t * ld_logits + j] = sum_h weights[t*H + h] *
 * relu(qv[t,h,:] . kv[j,:]) for every visible key j, -inf for every other j in
 * [0, max_context_len).  Columns >= max_context_len are not written.
 *  q        [T, H, D] bf16 (dtype DSA_BF16) or E4M3 codes (DSA_E4M3), row-major.
 *  q_scale  [T, H] fp32, non-negative (E4M3 only, else NULL): qv = q * q_scale[t,h].
 *  weights  [T, H] fp32.
 *  keys     see dsa_keys; kv = k (bf16) or k * scale[row] (E4M3).
 *  logits   [T, ld_logits] fp32, ld_logits >= max_context_len.
 * Arithmetic: bf16 or E4M3 products summed in fp32 by the tensor cores, then
 * ReLU, weight and head sum in fp32 in a fixed order (heads 0..63 in four
 * interleaved partial sums), then -0.0 is written as +0.0.  Given the same
 * inputs the scores are bit-identical to those dsa_indexer_logits_topk ranks.
 */
dsa_status dsa_indexer_logits(const void* q, const float* q_scale, dsa_dtype dtype,
                              const float* weights, int H, int D, dsa_keys keys,
                              dsa_queries qs, float* logits, int64_t ld_logits,
                              void* stream);

/*
 * dsa_indexer_topk -- per-row top-k of a logits matrix laid out as
 * dsa_indexer_logits writes it.  Only the visible keys of row t (per `qs`) are
 * candidates; -inf and NaN values are never selected.  out_idx[t * topk + s]
 * (int32) lists the selected key indices in rank order: larger value first,
 * ties to the smaller index, -0.0 equal to +0.0; rows with fewer than topk
 * candidates are padded with -1.  out_val (nullable) receives the matching
 * values (-inf in padded slots).  1 <= topk <= 2048.
 *  ws / ws_bytes: device scratch of at least dsa_workspace_bytes(DSA_OP_TOPK,
 *  DSA_BF16, qs, topk) bytes (may be 0, then ws may be NULL); its contents on
 *  entry do not matter.
 */
dsa_status dsa_indexer_topk(const float* logits, int64_t ld_logits, dsa_queries qs, int topk,
                            int32_t* out_idx, float* out_val, void* ws, size_t ws_bytes,
                            void* stream);

/*
 * dsa_indexer_logits_topk -- dsa_indexer_topk(dsa_indexer_logits(...)) in one
 * pass that never writes the T x max_context_len logits to memory: the scores
 * are ranked on chip as the tensor cores produce them.  Arguments as for the
 * two calls above; the result is bit-identical to running them in sequence.
 * ws: at least dsa_workspace_bytes(DSA_OP_LOGITS_TOPK, dtype, qs, topk) bytes, 8-byte
 * aligned (the work plan, 8 bytes per query group, and two partial top-k lists per
 * CTA of the current device; contents on entry do not matter).
 */
dsa_status dsa_indexer_logits_topk(const void* q, const float* q_scale, dsa_dtype dtype,
                                   const float* weights, int H, int D, dsa_keys keys,
                                   dsa_queries qs, int topk, int32_t* out_idx, float* out_val,
                                   void* ws, size_t ws_bytes, void* stream);

/*
 * mxfp4_paged_gather -- xkernels issue #28, comment 2 "What it does": for every
 * query row t and slot s, pos = sel_pos[t * topk + s];
 *   pos < 0  -> out row is 128 x bf16 +0.0 (a padded slot);
 *   else     -> cache row (blk, off) = (block_table[b * bt_stride + pos / block_size],
 *               pos % block_size) with b = t / next_n, dequantised to bf16:
 *               element e = E2M1(nibble e) * 2^(kv_scale[row][e / 32] - 127),
 *               scale byte 0xFF -> 0 (the sign of the zero follows the nibble),
 *               rounded to nearest-even bf16 (exact except overflow -> inf).
 *  kv_fp4   [num_blocks, block_size, D/2] bytes; byte i of a row holds element
 *           2i in its low nibble and 2i+1 in its high nibble (E2M1: sign bit 3,
 *           two exponent bits, one mantissa bit).
 *  kv_scale [num_blocks, block_size, D/32] E8M0 bytes.
 *  out      [T, topk, D] bf16 bit patterns, row-major.
 * A block id outside [0, num_blocks) or pos / block_size >= bt_stride gives a
 * zero row and sets DSA_DEVERR_INDEX.  D must be 128 (DSA_ERR_UNSUPPORTED
 * otherwise); block_size >= 1.
 */
dsa_status mxfp4_paged_gather(const uint8_t* kv_fp4, const uint8_t* kv_scale, int64_t num_blocks,
                              int block_size, int D, const int32_t* block_table, int64_t bt_stride,
                              const int32_t* sel_pos, int B, int next_n, int topk,
                              uint16_t* out, void* stream);

/*
 * dsa_indexer_q_rope_quant -- the indexer-query producer ahead of the score (vllm PR #1
 * "Sparse-MLA bring-up on MI300X", "Root cause story" item 3: a fused RoPE + FP8
 * quantisation of the indexer query whose bytes the fp8 MQA-logits reader consumes;
 * FP8_MAX = 448 on the OCP path).  For every (token t, head h) row of q:
 *   1. RoPE: for i < rope_dim / 2 the pair (x[2i], x[2i+1]) becomes
 *      (x0 c - x1 s, x0 s + x1 c) with c = cos_sin[p * rope_dim + i],
 *      s = cos_sin[p * rope_dim + rope_dim / 2 + i], p = positions[t]; dims >= rope_dim
 *      pass through (this library's reading: interleaved pairs, a caller-built table);
 *   2. q_scale[t, h] = max_d |y[d]| / 448 (1 for an all-zero row);
 *   3. q_fp8[t, h, d] = E4M3(y[d] / q_scale[t, h]), nearest even, saturating at +-448.
 * All arithmetic in fp32, each product and sum rounded on its own.  The output is the
 * (q, q_scale) pair dsa_indexer_logits* take with dtype DSA_E4M3.
 *  q        [T, H, D] bf16 bit patterns, 16-byte aligned.
 *  positions [T] int32; a position outside [0, max_pos) gives a zero row (codes 0,
 *           scale 0) and sets DSA_DEVERR_INDEX.
 *  cos_sin  [max_pos, rope_dim] fp32 (rope_dim / 2 cosines, then rope_dim / 2 sines per
 *           position), 8-byte aligned; may be NULL when rope_dim == 0.
 *  q_fp8    [T, H, D] E4M3 codes (8-byte aligned); q_scale [T, H] fp32.
 * D must be 128 (DSA_ERR_UNSUPPORTED otherwise); rope_dim a multiple of 4, <= D.
 */
dsa_status dsa_indexer_q_rope_quant(const uint16_t* q, const int32_t* positions, const float* cos_sin,
                                    int64_t max_pos, int rope_dim, int T, int H, int D, uint8_t* q_fp8,
                                    float* q_scale, void* stream);

/*
 * dsa_indexer_k_hadamard_mxfp4 -- the indexer-key compressor's write into the paged FP4
 * cache (ROCm/ATOM issue #707, "CSA": "CSA Indexer Compressor (head_dim=128, Hadamard,
 * FP4)").  For every key n with pool row r = slot_mapping[n] >= 0:
 *   y = H k[n] / sqrt(128), H the Sylvester-ordered Walsh-Hadamard matrix
 *       (H[i][j] = (-1)^popcount(i & j)), in fp32;
 *   per 32-element group g: kv_scale[r, g] = E8M0 byte floor(log2(amax_g)) - 2 + 127
 *       (clamped to >= 0; 0 for an all-zero group), and each element is the nearest E2M1
 *       code of y / 2^(byte - 127) (ties to the even code, saturating at 6; zero results
 *       are +0), packed two per byte of kv_fp4[r], low nibble = even element
 *       (the OCP MX v1.0 conversion, in the layout mxfp4_paged_gather reads).
 *  k            [N, D] bf16 bit patterns, 16-byte aligned.
 *  slot_mapping [N] int64 pool rows (block * block_size + offset); < 0: key skipped;
 *               >= num_rows: skipped and DSA_DEVERR_INDEX set.
 *  kv_fp4       [num_rows, D/2] bytes; kv_scale [num_rows, D/32] bytes (both 4-byte aligned).
 * D must be 128.  The transform is summed by butterflies in fp32: a code can differ
 * from the one of the exactly rounded rotation only where that value lies within a few
 * fp32 ulps of an E2M1 rounding boundary.
 */
dsa_status dsa_indexer_k_hadamard_mxfp4(const uint16_t* k, const int64_t* slot_mapping, int64_t N, int D,
                                        uint8_t* kv_fp4, uint8_t* kv_scale, int64_t num_rows, void* stream);

/*
 * dsa_sparse_attn_mxfp4 -- the sparse-attention consumer of the selection, reading the
 * paged mxfp4 cache directly (ROCm/ATOM issue #707, "CSA": "index-gather + online
 * softmax + attn_sink bias").  This library's reading: for query row t and head h, over
 * the selected positions of row t (sel_pos >= 0), the key and the value are the same
 * dequantised cache row x (the row mxfp4_paged_gather produces); s = softmax_scale *
 * q[t,h,:] . x; the head's sink logit joins the softmax denominator only:
 *   out[t,h,:] = sum_j e^(s_j - m) x_j / (sum_j e^(s_j - m) + e^(sink[h] - m)),
 * m any shift (the result does not depend on it).  A row with no selected position
 * gives zeros.
 *  q        [T, H, D] bf16 bit patterns, 16-byte aligned.  H must be 64 and D 128
 *           (DSA_ERR_UNSUPPORTED otherwise).
 *  sel_pos  [T, topk] int32 positions in row t's sequence b = t / next_n (< 0: padded);
 *           may be NULL when topk == 0.
 *  kv_fp4 [num_blocks, block_size, D/2] (16-byte aligned), kv_scale [num_blocks,
 *           block_size, D/32] (4-byte aligned), block_table [ceil(T / next_n), bt_stride]:
 *           the cache and table exactly as mxfp4_paged_gather reads them.
 *  sink     [H] fp32 logits (-inf: no sink).  softmax_scale finite.
 *  out      [T, H, D] fp32, 4-byte aligned; every element is written.
 * Arithmetic: the scores on the tensor cores from bf16 q and the exactly decoded bf16
 * rows with fp32 accumulation; the softmax in base 2; each weight rounded once to bf16
 * and the same weights summed for the denominator.  So the result is a weighted mean of
 * the selected rows whose weights are off by the bf16 rounding (2^-9 relative) and by
 * the fp32 score error: |out - exact| <= (2^-8 + 2 max_j |ds_j|) max_j |x_j[e]| to first
 * order, ds_j the fp32 error of score j.  Scores must be finite: a row whose scale
 * overflows bf16 (scale bytes 253, 254 with large codes) gives undefined output.
 * A block id outside [0, num_blocks) or a page at or past bt_stride drops that position
 * (as if padded) and sets DSA_DEVERR_INDEX.  topk above 16384 or a cache of 2^31 rows or
 * more (num_blocks * block_size) is DSA_ERR_UNSUPPORTED.  One CTA of 160 threads per
 * query row; two share an SM up to topk 2048.
 */
dsa_status dsa_sparse_attn_mxfp4(const uint16_t* q, int64_t T, int H, int D, const int32_t* sel_pos, int topk,
                                 const uint8_t* kv_fp4, const uint8_t* kv_scale, int64_t num_blocks,
                                 int block_size, const int32_t* block_table, int64_t bt_stride, int next_n,
                                 const float* sink, float softmax_scale, float* out, void* stream);

/*
 * The three calls that prepare a step's inputs.  (The pages start from finished queries,
 * keys, weights, slots and tables; these calls make them in the layouts the calls above
 * read.)  A layer's step uses them in this order: dsa_assign_slots gives every new token its
 * cache slot and position; dsa_add_rmsnorm_e4m3 turns the hidden rows into E4M3 codes with
 * one scale per 128 elements; dsa_gemm_e4m3 projects those to the queries
 * (dsa_indexer_q_rope_quant), the keys (dsa_indexer_k_hadamard_mxfp4) and the fp32 head
 * weights (the score calls).
 *
 * dsa_assign_slots -- block tables, slot mapping and positions from request lengths.
 * Request b holds cached_lens[b] tokens in have_b = ceil(cached_lens[b] / block_size) pages
 * and brings new_lens[b] >= 0 tokens, which need need_b = ceil((cached_lens[b] +
 * new_lens[b]) / block_size) - have_b more.  With first_b = sum of need over the requests
 * before b and start_b = sum of new_lens over them:
 *   block_table[b, have_b + i] = free_blocks[first_b + i] for i < need_b (other entries stay);
 *   new token t = start_b + i of the step, i < new_lens[b], has positions[t] =
 *   cached_lens[b] + i and slot_mapping[t] = its pool row, block_table[b, pos / block_size] *
 *   block_size + pos % block_size: the row dsa_indexer_k_hadamard_mxfp4 writes;
 *   context_lens[b] = cached_lens[b] + new_lens[b]; query_start[b] = start_b, query_start[B]
 *   = the step's tokens; blocks_used[0] = the free-list entries the step needs (the caller's
 *   next step starts behind them).
 * Entries [step's tokens, max_tokens) of slot_mapping are -1 (the key writer skips them) and
 * of positions 0, so a captured graph can serve any step of up to max_tokens tokens.
 *  cached_lens, new_lens [B] int32; free_blocks [n_free] int32 block ids of a pool of
 *           num_blocks blocks; block_table [B, bt_stride] int32, updated in place.
 *  context_lens [B], query_start [B + 1], blocks_used [1] int32; slot_mapping [max_tokens]
 *           int64; positions [max_tokens] int32.  No output may overlap an input or another
 *           output (the same address is refused).
 * Flagged with DSA_DEVERR_INDEX, never accessed out of range: a negative length or a sum
 * past INT32_MAX (the request brings nothing; a negative cached length counts as 0); a page
 * at or past bt_stride (slot -1, no entry); a free-list rank at or past n_free or a block id
 * outside [0, num_blocks) (slot -1; a new page's entry is -1); tokens at or past max_tokens
 * (neither slot nor page).  Counts past INT32_MAX are written as INT32_MAX.
 * block_size >= 1; B <= 65536.  One launch; the result does not depend on timing.
 */
dsa_status dsa_assign_slots(const int32_t* cached_lens, const int32_t* new_lens, int B, int block_size,
                            const int32_t* free_blocks, int n_free, int64_t num_blocks, int32_t* block_table,
                            int64_t bt_stride, int64_t max_tokens, int32_t* context_lens, int32_t* query_start,
                            int64_t* slot_mapping, int32_t* positions, int32_t* blocks_used, void* stream);

/*
 * dsa_add_rmsnorm_e4m3 -- residual addition, RMS norm and E4M3 quantisation.  For each of T
 * rows of D elements:
 *   r = x + residual, rounded once to `type` (r = x without a residual);
 *   y = r * gamma / sqrt(mean(r^2) + eps), in fp32;
 *   per group g of 128 elements (the last may be shorter): y_scale[t, g] = max|y| / 448 (at
 *   least 2^-126; 1 for an all-zero group), with pow2_scale != 0 rounded up to a power of
 *   two; y_fp8 = E4M3(y / y_scale), nearest even, saturating at +-448.  The division by 448
 *   is a product with the rounded 1 / 448.
 *  x        [T, D] of `type`, rows ldx elements apart; residual, residual_out [T, D] of
 *           `type`, rows ldr apart, both nullable (residual_out receives r; it may be
 *           residual itself, or x where ldr == ldx).
 *  gamma    [D] fp32.  eps > 0.
 *  y        [T, D] of `type`, nullable: y rounded to `type`; may be x where ldy == ldx.
 *  y_fp8    [T, D] E4M3 codes with y_scale [T, ceil(D / 128)] fp32 (row-major), both or
 *           neither NULL.  y and y_fp8 have rows ldy elements apart.  A ldy that is a
 *           multiple of 16 makes the codes an operand of dsa_gemm_e4m3.
 * At least one of residual_out, y and y_fp8 is given; no other overlap of outputs with inputs
 * or with one another.  1 <= D <= 32768.  Any element-aligned
 * pointers and strides >= D work; with D and the strides multiples of 8 and 16-byte aligned
 * pointers the rows move in 16-byte accesses.
 * Arithmetic in fp32: the sum of squares in an order that D, T, the type, the alignment, the
 * device's SM count and which of residual, residual_out and y are given fix (so a row's last bits
 * may differ in another batch), 1 / rms by the hardware's reciprocal root (2 ulps), each product
 * rounded on its own; y / y_scale is formed as (r gamma) (448 / max|r gamma|), without the row's
 * common factor (from y itself where pow2_scale is set, y_scale is 2^-126, or max|r gamma| is
 * outside [1e-30, 1e30]), so a code can differ from the exact quotient's only where that lies
 * within a few fp32 ulps of a rounding boundary.  For the same reason a power-of-two scale can
 * be the neighbouring power where max|y| / 448 lies within 2^-18 of one.
 * r * gamma and the row's fp32 sum of squares must be finite (|r| up to 1.8e19 / sqrt(D) always
 * is enough; past it y and the codes are 0, not the formula's), and squares below 2^-126 lose
 * precision, which shows only where eps is as small.  A row holding a NaN gives NaN codes; an
 * infinity gives a NaN code at its place and zeros elsewhere in the row.  Every scale of such a
 * row is 1.
 */
dsa_status dsa_add_rmsnorm_e4m3(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                                float eps, int64_t T, int D, dsa_real type, void* residual_out, void* y,
                                uint8_t* y_fp8, int64_t ldy, float* y_scale, int pow2_scale, void* stream);

/*
 * dsa_gemm_e4m3 -- product of E4M3 rows with E4M3 weights under block scales:
 *   out[m, n] = sum_k a[m,k] a_scale[m, k / 128] * w[n,k] w_scale[n / 128, k / 128].
 *  a        [M, K] E4M3 codes, rows lda bytes apart; a_scale [M, ceil(K / 128)] fp32 (the
 *           pair dsa_add_rmsnorm_e4m3 writes).
 *  w        [N, K] E4M3 codes, rows ldw bytes apart; w_scale [ceil(N / 128), ceil(K / 128)]
 *           fp32.  Scales are row-major and may be any fp32 values.
 *  out      [M, N] of `out_type`, rows ldo elements apart.
 * a and w are 16-byte aligned, lda and ldw multiples of 16 and at least K; K >= 1 (what lies
 * past K in a row is not part of the product), M and N any; any element-aligned out and ldo
 * >= N (16-byte aligned rows are stored in 16-byte accesses).  out may not overlap an input.
 * Arithmetic: exact products summed in fp32 by the tensor cores within a block of 128, the
 * block's sum times its two scales (their product rounded to fp32: it overflows, or loses
 * precision below 2^-126, as any fp32 product) added in fp32 in the order
 * of K; with few tiles K is cut into 2, 4 or 8 parts whose sums are added in order.  One
 * rounding to bf16 at the end.  The result depends on the sizes and the device's SM count (a
 * row's sums may be cut differently in another batch) but not on timing.  No workspace.  A
 * device-side wait that expires sets DSA_DEVERR_TIMEOUT.
 */
dsa_status dsa_gemm_e4m3(const uint8_t* a, int64_t lda, const float* a_scale, const uint8_t* w, int64_t ldw,
                         const float* w_scale, int64_t M, int N, int K, void* out, int64_t ldo, dsa_real out_type,
                         void* stream);

/*
 * The calls of a layer that attends to every cached key and keeps them in bf16 (a draft layer, a
 * layer without the selection).  (The pages have no counterpart.)  The table is made once;
 * dsa_qk_norm_rope turns the projected heads and writes keys and values to the slots of
 * dsa_assign_slots; dsa_paged_attn reads them through its block table, query_start and
 * context_lens; dsa_rope with inverse set takes the rotation of an output back.
 *
 * dsa_rope_table -- cos / sin table of the positions pos0 .. pos0 + n - 1, in the layout that
 * dsa_rope, dsa_qk_norm_rope and dsa_indexer_q_rope_quant read: for i < rope_dim / 2
 *   cos_sin[r, i] = amplitude cos((pos0 + r) f_i), cos_sin[r, rope_dim / 2 + i] the sine,
 *   PLAIN:  f_i = base^(-2i / rope_dim);  LINEAR: that / factor;
 *   YARN (Peng et al. 2023): f_i (1 - w_i) + f_i / factor w_i, w_i = clamp((i - lo) / (hi -
 *   lo), 0, 1), lo = max(floor(c(beta_fast)), 0), hi = min(ceil(c(beta_slow)), rope_dim - 1),
 *   c(b) = rope_dim ln(original_max_pos / (2 pi b)) / (2 ln base); hi - lo is at least 0.001.
 *   (The paper's factor on the attention's scale, 0.1 ln(factor) + 1 on queries and keys alike,
 *   is the caller's to give as the amplitude; nothing is multiplied by itself.)
 *  cos_sin  [n, rope_dim] fp32.  rope_dim even, 2 .. 256; pos0 >= 0, pos0 + n <= 2^31.
 * Each value is within 2^-22 amplitude of the exact one at any position: the angle is reduced
 * by whole turns in 64-bit integers.  params is read on the host.
 */
dsa_status dsa_rope_table(dsa_rope_params params, int rope_dim, int64_t pos0, int64_t n, float* cos_sin, void* stream);

/*
 * dsa_rope -- rotation of heads.  For every token t and head h, with c and s the cosine and
 * sine of pair i at positions[t] (s negated where inverse is set), the elements (x0, x1) =
 * (rope_off + 2i, rope_off + 2i + 1) (INTERLEAVED) or (rope_off + i, rope_off + rope_dim / 2
 * + i) (HALF), i < rope_dim / 2, become (x0 c - x1 s, x0 s + x1 c); the other dims are copied.
 * With the same table the inverse is the gradient of the call without it; it takes the rotation
 * back where the table's amplitude is 1 (otherwise the turned dims come back times its square).
 *  x, y     heads of D elements of `type`: token t, head h at t * ldx + h * hx (t * ldy +
 *           h * hy), in elements.  y may be x where the strides are the same; no other overlap
 *           of y with an input, and heads of y do not overlap one another.
 *  positions [T] int32; one outside [0, max_pos) gives zeros in the rotated dims and sets
 *           DSA_DEVERR_INDEX.  cos_sin [max_pos, rope_dim] fp32 as dsa_rope_table writes it.
 * D <= 256 (DSA_ERR_UNSUPPORTED above); rope_dim even, >= 2, rope_off + rope_dim <= D; hx and
 * hy >= D where H > 1, ldx and ldy >= D where T > 1 (heads may lie outside tokens).  Any
 * element-aligned pointers and such strides work; heads move in units of four elements where D
 * is a multiple of 8, rope_off of 4, rope_dim of 4 (HALF: 8), the strides of 4, and pointers are
 * aligned to four elements (the table and gains to 16 bytes).
 * fp32 arithmetic, one rounding to `type` at the end.
 */
dsa_status dsa_rope(const void* x, int64_t ldx, int64_t hx, const int32_t* positions, const float* cos_sin,
                    int64_t max_pos, int rope_dim, int rope_off, dsa_rope_layout layout, int inverse, int64_t T, int H,
                    int D, dsa_real type, void* y, int64_t ldy, int64_t hy, void* stream);

/*
 * dsa_qk_norm_rope -- per-head RMS norm and rotation of queries and keys, and the write of
 * keys and values into the paged cache, in one pass.  For every token t and query head h:
 *   y = q[t, h] * gamma_q / sqrt(mean(q[t, h]^2) + eps) (q itself without a gamma), then the
 *   rotation of dsa_rope, in fp32 with one rounding to `type` (the cache: to bf16) at the end;
 * the same for the key heads with gamma_k; value heads are copied.
 *  q        [T, H, D] of `type`, tokens ldq elements apart, heads D apart; q_out the same with
 *           ldqo, and may be q where ldqo == ldq.  Both may be NULL where H == 0.
 *  k, v     [T, Hkv, D], tokens ldk and ldv apart (one projection's output holds q, k and v
 *           side by side).  v may be NULL: no values are written.  k may be NULL where Hkv == 0.
 *  k_out    [T, Hkv, D] of `type`, nullable; may be k where ldko == ldk.
 *  gamma_q, gamma_k [D] fp32: both, or both NULL (no norm); one that has no heads may be NULL.
 *  positions, cos_sin, max_pos, rope_dim, rope_off, layout as for dsa_rope; rope_dim may be 0
 *           (no rotation; positions and cos_sin may then be NULL).
 *  kv       the cache; kv.k NULL: none (then v is not read).  slot_mapping [T] int64: token t's
 *           keys and values go to row slot % block_size of block slot / block_size; negative:
 *           none; past the pool: none, and DSA_DEVERR_INDEX.  Slots are distinct.
 * No other overlap of outputs with inputs or with one another.  D <= 256, T * (H + 2 Hkv) <
 * 2^31.  Any element-aligned pointers and strides work, faster under the conditions of
 * dsa_rope.  A head's squares must sum to a finite fp32 and its elements' products with the gain
 * be finite (past that y is 0, infinite or NaN); |y| is the formula's within a few fp32 ulps
 * before the last rounding.
 */
dsa_status dsa_qk_norm_rope(const void* q, int64_t ldq, int H, const void* k, int64_t ldk, int Hkv, const void* v,
                            int64_t ldv, int64_t T, int D, dsa_real type, const float* gamma_q, const float* gamma_k,
                            float eps, const int32_t* positions, const float* cos_sin, int64_t max_pos, int rope_dim,
                            int rope_off, dsa_rope_layout layout, void* q_out, int64_t ldqo, void* k_out, int64_t ldko,
                            dsa_kv_cache kv, const int64_t* slot_mapping, void* stream);

/*
 * dsa_paged_attn -- attention of new tokens over a paged cache.  Sequence b brings the rows
 * t = query_start[b] .. query_start[b + 1] - 1 of q (n_b of them: one for a decode step, any
 * number for a chunk of a prompt) and has L_b = context_lens[b] keys in the cache, the new
 * tokens' own among them: token i of the n_b sits at position p = L_b - n_b + i.  It sees the
 * keys j < L_b with j <= p (causal != 0) and j > p - window (window > 0).  For query head h,
 * with key head h / (H / Hkv):
 *   s_j = softmax_scale * q[t,h,:] . k_j,
 *   out[t,h,:] = sum_j e^(s_j - m) v_j / (sum_j e^(s_j - m) + e^(sink[h] - m)),
 *   lse[t,h] = ln(sum_j e^(s_j) + e^(sink[h])),
 * m any shift.  A row that sees nothing gives zeros, and lse the sink (-inf without one).
 *  q        [T, H, D] bf16 bit patterns, tokens ldq elements apart, heads D apart; out the same
 *           with ldo.  Rows that belong to no sequence (past query_start[B], or in a gap) count
 *           for nothing, and their rows of out and lse are left as they are.
 *  query_start [B + 1] int32, ascending, as dsa_assign_slots writes it; context_lens [B] int32.
 *  block_table [B, bt_stride] int32; kv the cache (see dsa_kv_cache); block_size any >= 1.
 *           Entries of pages that hold no visible key are not read (with a window the old
 *           pages of a sequence may be gone).
 *  sink     [H] fp32 logits that join the denominators, nullable; an entry of -infinity counts for
 *           nothing, one of +infinity makes its head's rows zeros.  lse [T, H] fp32, nullable.
 *  ws       dsa_paged_attn_workspace_bytes(T, B, H, Hkv, D) bytes, 16-byte aligned; its
 *           contents on entry do not matter.  Calls that may run at the same time need one each.
 *           The size for some T and B is accepted for every smaller T and B too, although it may
 *           be less than their own: rows then go 128 at a time instead of 256 (a prompt of 8192
 *           tokens 908 us instead of 734), and results may differ in their last bits.
 * Pointers of q, out and kv are 16-byte aligned, ldq, ldo and kv's strides multiples of 8,
 * num_blocks at least 1.  The pool is addressed as rows row_stride apart: block_stride is a
 * multiple of row_stride, head_stride smaller than it or a multiple of it, and the pool's rows
 * fewer than 2^31 (DSA_ERR_UNSUPPORTED otherwise).
 * D is 64 or 128 (DSA_ERR_UNSUPPORTED otherwise), Hkv divides H, B <= 65536, T * H < 2^31,
 * softmax_scale > 0, its product with log2(e) within fp32's range.  No output overlaps an input
 * or another output.
 * Arithmetic: bf16 products summed in fp32 by the tensor cores, softmax in base 2 with fp32
 * statistics; each weight is rounded once to bf16 for its product with v, the denominator sums
 * the unrounded ones: |out - exact| <= (2^-8 + 2 max_j |ds_j|) sum_j p_j |v_j| + 2^-8 |exact| to
 * first order, p_j the exact weights and ds_j the fp32 error of score j; lse is fp32 throughout.
 * What is below 2^-126 of a row's denominator counts as zero.
 * Long rows are cut where the work of all sequences divides evenly among the SMs, and the parts
 * added in order: results depend on the batch, the device's SM count and whether ws has the
 * call's own size, but not on timing.
 * Keys and values that a row does not see never touch it, whatever they hold.  An infinity or a
 * NaN that it sees gives what the formula gives (at a value: an infinity or NaN in its dim),
 * but a row all of whose scores are -infinity counts as one that sees nothing.
 * Flagged with DSA_DEVERR_INDEX, never accessed out of range: a block id outside [0,
 * num_blocks) or a page at or past bt_stride (its keys are seen by no row); a negative length
 * (0); rows of a sequence outside [0, T) (left out); overlapping sequences (rows are lost).
 * A device-side wait that expires sets DSA_DEVERR_TIMEOUT.
 */
size_t dsa_paged_attn_workspace_bytes(int64_t T, int B, int H, int Hkv, int D);
dsa_status dsa_paged_attn(const uint16_t* q, int64_t ldq, int64_t T, int H, int Hkv, int D, const int32_t* query_start,
                          const int32_t* context_lens, int B, const int32_t* block_table, int64_t bt_stride,
                          dsa_kv_cache kv, float softmax_scale, int causal, int window, const float* sink, uint16_t* out,
                          int64_t ldo, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_indexer_logits_topk_noalloc -- dsa_indexer_logits_topk for callers that cannot
 * allocate device memory: a process whose device memory is all reserved at start-up
 * and handed out by its own pool, or a latency-critical loop that cannot afford
 * cudaMalloc / cudaFree (cudaFree waits for the whole device).  (The pages have no
 * counterpart: this is a convenience of this library.)
 * Same arguments and results as dsa_indexer_logits_topk, without ws / ws_bytes: the
 * scratch lives in a fixed 16 MiB array in the library's device image, which every
 * GPU that loads the library holds until the process exits.
 *  - Its plan takes no wider candidate buffers than the batch needs (the regular call
 *    widens them where shared memory allows, which grows its workspace); results are the
 *    same.  A batch whose scratch under that plan exceeds 16 MiB is rejected with
 *    DSA_ERR_WORKSPACE before anything is launched; that scratch is never more than
 *    dsa_workspace_bytes(DSA_OP_LOGITS_TOPK, ...).
 *  - The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 *    and keeps it for the process; make that first call before any stream capture, and do
 *    not use this call across a device reset (cudaDeviceReset may move the array).
 *  - Which batches fit depends on the device's SM count (the plan keeps two partial top-k
 *    lists per SM): on a 152-SM GB300 the tiny, Flash decode, Pro decode MTP and 16K
 *    prefill batches fit; the FP8 chunked prefill (8192 rows, top-1024) does not.
 *  - All calls share the one array; the call itself rewrites every part it reads
 *    (its work plan and partial top-k lists), so stale contents never matter.
 *    Calls whose executions overlap on the GPU (other streams, other threads) race on
 *    the array: serialise them.
 *  - Allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 */
dsa_status dsa_indexer_logits_topk_noalloc(const void* q, const float* q_scale, dsa_dtype dtype,
                                           const float* weights, int H, int D, dsa_keys keys,
                                           dsa_queries qs, int topk, int32_t* out_idx, float* out_val,
                                           void* stream);

/* Workspace bytes the op needs for this batch shape on the current device (host only,
 * no device work; the fused call's plan has one slice per resident CTA, so the size
 * depends on the device's SM count). */
size_t dsa_workspace_bytes(dsa_op op, dsa_dtype dtype, dsa_queries qs, int topk);

/* Static text for a status code. */
const char* dsa_status_string(dsa_status status);

/* Synchronises `stream`, then returns and clears the current device's error
 * word (DSA_DEVERR_* bits; 0 = no device-side error since the last read).
 * Returns -1 if the synchronisation or the read fails. */
int dsa_device_error(void* stream);

/* Number of kernels this library has launched in this process (all threads,
 * all devices); lets a caller count the launches inside a timed region. */
uint64_t dsa_launch_count(void);

/* Sets the limit, in nanoseconds, of every bounded device-side wait launched
 * after this call on the current device (default 2 s; 0 restores the
 * default).  Returns DSA_ERR_CUDA if the device symbol cannot be written. */
dsa_status dsa_set_wait_limit_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_H_ */
