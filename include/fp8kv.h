/*
 * fp8kv.h -- C ABI of libfp8kv.so: calibrated-scale E4M3 FP8 paged KV-cache
 * insertion and exact paged decode / speculative-verifier attention on one
 * NVIDIA GB300 (sm_103a).
 *
 * Sources (the "b70-optimization-lab" pages):
 *  - "Laguna S 2.1 INT4 -- calibrated FP8 KV on Intel B70", section "Contract":
 *    target KV is explicit E4M3 FP8 with one calibrated scalar K scale and one V
 *    scale per layer; no runtime scale calculation.  Section "Initial
 *    optimization order": profile the FP8 cache update and exact q1/M12 paged
 *    attention separately; scaled E4M3 insertion at the Q/K norm + RoPE boundary.
 *  - "Laguna S 2.1 KV-cache precision decision", section "What the official
 *    checkpoint requests": kv_cache_scheme = static ("dynamic": false),
 *    symmetric, per-tensor ("strategy": "tensor"), minmax observer; section
 *    "BF16 versus FP8 in concrete terms": 8 KV heads x dim 128, 2048 B per token
 *    per layer in FP8 vs 4096 B in BF16, "quantize, store FP8" on write and
 *    "scale/dequantize" on read; 36 sliding-window-512 and 12 global layers.
 *  - "Laguna FP8 KV -- replicated embedding win, page-32 build, and host
 *    boundary", section "Page-32 attention experiment": page 32 and page 64,
 *    global and sliding attention, and the rule that a fallback path
 *    invalidates a result.
 *  - "Laguna S 2.1 B70 campaign transfer ledger", table "Result progression",
 *    row "Persistent attention metadata": fixed-address metadata refreshed in
 *    place (here: every buffer is caller-owned; the library allocates no
 *    memory).
 *
 * Conventions for every entry point:
 *  - Pointers marked (device) are device pointers owned by the caller; they
 *    must stay valid until the work queued on `stream` has finished.  Host
 *    integers are sizes.  `stream` is a cudaStream_t (NULL = legacy default
 *    stream); all work is queued asynchronously on it, nothing synchronises.
 *  - Arguments are validated on the host before any launch.  A rejected call
 *    returns a status below and launches nothing.  Shapes the kernels do not
 *    implement return FP8KV_ERR_UNSUPPORTED: there is no slower fallback path.
 *  - A failed launch returns FP8KV_ERR_CUDA (cudaGetLastError is consumed).
 *  - Contents that the host cannot see (slot ids, positions, page ids,
 *    sequence lengths) are checked on the device: an offending row is skipped
 *    (never read or written out of bounds) and a bit is set in the device
 *    status word, read with fp8kv_device_status().
 *  - bf16 is the IEEE-like bfloat16 bit layout; every tensor is dense,
 *    row-major, in the order of its dimension list, 16-byte aligned.
 */
#ifndef FP8KV_H
#define FP8KV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8KV_OK = 0,
    FP8KV_ERR_INVALID_ARG = 1,  /* null pointer, negative size, misaligned, bad enum */
    FP8KV_ERR_UNSUPPORTED = 2,  /* valid request outside the implemented shapes     */
    FP8KV_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required       */
    FP8KV_ERR_CUDA = 4          /* a CUDA runtime call or a launch failed           */
} fp8kv_status;

typedef enum {
    FP8KV_CACHE_E4M3 = 0,       /* 1 byte per element, E4M3FN codes, scaled          */
    FP8KV_CACHE_BF16 = 1,       /* 2 bytes per element, stored as is, scales unused  */
    FP8KV_CACHE_INT4 = 2        /* 4.5 bits per element: 4-bit codes in blocks of 16, one E4M3 scale a block */
} fp8kv_cache_dtype;

/*
 * The INT4 cache.  A row (one token of one KV head, 128 elements) is 8 blocks
 * of 16 elements.  With the calibrated tensor scale c (k_scale or v_scale, as
 * for E4M3; 2^-100 <= c <= 2^100) a block x is stored as the E4M3 scale s and
 * 16 integers n, every step rounded to fp32:
 *     r = amax|x| / (7 c)         s = max(e4m3_rne_satfinite(r), 2^-9)
 *     inv = 1 / (s c)             n = clamp(rint(x inv), -7, 7)   (ties to even)
 * and stands for n s c: off by at most half a step s c / 2 where s >= 7 * 2^-9,
 * unless it saturates at 7 * 448 c.  Smaller scales are subnormal, and rounding
 * one down (by up to 2^-10) clamps the block's largest elements: they are off by
 * up to 7 * 2^-10 c (3.5 steps at s = 2^-9).  (Both bounds and 2^-18 of a step,
 * for the fp32 roundings.)  A NaN in the block makes s NaN (0x7F) and
 * n = 0: the whole block reads as NaN.  Infinities saturate.
 * k_cache, v_cache: [num_pages][Hkv][page_size * 72] bytes; the bytes of one
 * (page, head) are page_size rows of 64 code bytes (byte i: element 2i in the
 * low nibble, element 2i + 1 in the high one, each as n + 8), then page_size
 * rows of 8 scale bytes.
 */
#define FP8KV_INT4_ROW_BYTES 72

/* Device status bits (fp8kv_device_status). */
#define FP8KV_DEV_BAD_SLOT      0x1u  /* slot_mapping entry >= num_pages*page_size   */
#define FP8KV_DEV_BAD_POSITION  0x2u  /* position outside [0, max_pos)              */
#define FP8KV_DEV_BAD_SEQ_LEN   0x4u  /* seq_len < M or beyond the block-table row  */
#define FP8KV_DEV_WAIT_TIMEOUT  0x8u  /* a bounded pipeline wait gave up            */
#define FP8KV_DEV_BAD_TREE      0x10u /* a tree's parent, token or path out of order */
#define FP8KV_DEV_BAD_PROBS     0x20u /* a row of probabilities without a finite sum */

/* Nodes of a tree of drafted tokens, at most (the bits of one mask word). */
#define FP8KV_TREE_MAX_NODES 64

/* Types of probabilities (fp8kv_verify_tree). */
typedef enum {
    FP8KV_PROBS_FP32 = 0,
    FP8KV_PROBS_BF16 = 1
} fp8kv_probs_dtype;

/*
 * fp8kv_cache_insert -- write T new tokens into the paged K and V caches.
 *
 * Operation ("KV-cache precision decision", property table row "Cache
 * write/read work": quantize, store FP8; scales per "Contract"): for every
 * token t with slot s = slot_mapping[t] >= 0, head h, element d:
 *     E4M3:  cache[s / page_size][h][s % page_size][d] =
 *                e4m3_rne_satfinite( fp32(x[t][h][d]) / scale )
 *     BF16:  cache[...] = x[t][h][d]  (bits copied, scales ignored, may be NULL)
 * with fp32 IEEE division, round to nearest even, saturation to +-448
 * (infinities included), NaN -> 0x7F with the input's sign, -0 -> 0x80.
 *     INT4:  the row's codes and block scales as described above.
 * Slots < 0 are skipped; slots not named are left untouched.  Duplicate
 * non-negative slots race: such a row may hold parts of each of its tokens, and
 * over an INT4 cache the codes of one under a block scale of another.
 *
 *   k, v          (device) bf16 [T][Hkv][D]
 *   slot_mapping  (device) int64 [T]
 *   k_scale, v_scale (device) one fp32 each, > 0 (E4M3 and INT4 only)
 *   k_cache, v_cache (device) [num_pages][Hkv][page_size][D] of the cache dtype
 *                ([num_pages][Hkv][page_size * 72] bytes for INT4)
 *   D must be 128; page_size 32 or 64; T may be 0 (no launch, FP8KV_OK, no
 *   pointer is read).
 * Device check: slot >= num_pages*page_size -> row skipped, FP8KV_DEV_BAD_SLOT.
 */
int fp8kv_cache_insert(const void* k, const void* v, const int64_t* slot_mapping, int T,
                       int Hkv, int D, const float* k_scale, const float* v_scale,
                       void* k_cache, void* v_cache, int num_pages, int page_size,
                       int cache_dtype, void* stream);

/*
 * fp8kv_cache_insert_per_head -- fp8kv_cache_insert on an E4M3 cache with one
 * scale per KV head: head h of K (V) is encoded with k_scale[h] (v_scale[h]).
 * An extension the pages do not use: their checkpoint asks for one static
 * symmetric scale per tensor ("KV-cache precision decision", "What the
 * official checkpoint requests", strategy "tensor"); a per-head scale keeps
 * the same encoding with a finer calibration grain.
 *
 *   k_scale, v_scale (device) fp32 [Hkv], each > 0
 *   every other argument, check and status as fp8kv_cache_insert with
 *   cache_dtype = FP8KV_CACHE_E4M3.
 */
int fp8kv_cache_insert_per_head(const void* k, const void* v, const int64_t* slot_mapping, int T,
                                int Hkv, int D, const float* k_scale, const float* v_scale,
                                void* k_cache, void* v_cache, int num_pages, int page_size,
                                void* stream);

/*
 * fp8kv_cache_gather -- read T stored tokens back as bf16: for every token t
 * with slot s = slot_mapping[t] >= 0, head h, element d:
 *     k_out[t][h][d] = bf16( fp32( value of the stored k ) )
 * where the stored value is decode(code) * k_scale (E4M3), the stored bf16
 * bits (BF16), or n s k_scale (INT4), the product rounded to fp32 and then to
 * bf16; V likewise.  Rows of tokens with a negative slot are left as they are.
 * For reusing or inspecting cached tokens outside the attention kernels (the
 * pages have no counterpart).  Caches with per-tensor scales only.
 *
 *   slot_mapping  (device) int64 [T]; slots may repeat
 *   k_scale, v_scale, k_cache, v_cache, page sizes, D: as fp8kv_cache_insert
 *   k_out, v_out  (device) bf16 [T][Hkv][D]
 *   T may be 0 (no launch, FP8KV_OK, no pointer is read).
 * Device check: slot >= num_pages*page_size -> row skipped, FP8KV_DEV_BAD_SLOT.
 */
int fp8kv_cache_gather(const int64_t* slot_mapping, int T, int Hkv, int D, const float* k_scale,
                       const float* v_scale, const void* k_cache, const void* v_cache, int num_pages,
                       int page_size, int cache_dtype, void* k_out, void* v_out, void* stream);

/*
 * fp8kv_qk_norm_rope_insert -- the Q/K RMSNorm + RoPE boundary fused with the
 * E4M3 insert ("calibrated FP8 KV on Intel B70", "Initial optimization order",
 * item 3; ledger table "Result progression", row "Exact fusion stack").
 *
 * For each token t at position pos = positions[t] and each Q head and K head
 * row x (D = 128), in fp32 with this fixed order (reproduced bit for bit):
 *     part_l  = sum of squares of x[4l..4l+3] accumulated as
 *               fma(x3,x3, fma(x2,x2, fma(x1,x1, x0*x0)))          l = 0..31
 *     ss      = parts added pairwise: l + (l+16), then +8, +4, +2, +1
 *     r       = 1 / sqrt(ss / 128 + eps)                (IEEE sqrt, divide)
 *     y_i     = bf16( bf16(x_i * r) * w_i )
 *     o_k     = bf16( fma(y_k,    c_k, -(y_k+64 * s_k)) )   k = 0..63
 *     o_k+64  = bf16( fma(y_k+64, c_k,   y_k    * s_k ) )
 * with c_k = cos_sin[pos][k], s_k = cos_sin[pos][64 + k].  Q rows go to q_out;
 * rotated K rows and the raw V rows are inserted as in fp8kv_cache_insert
 * (E4M3 cache only).
 *
 *   q (device) bf16 [T][Hq][D]; k, v (device) bf16 [T][Hkv][D]
 *   positions (device) int64 [T]; q_norm_w, k_norm_w (device) bf16 [D]
 *   cos_sin (device) fp32 [max_pos][D]: cos of the 64 frequencies, then sines
 *   q_out (device) bf16 [T][Hq][D] (must not alias q)
 *   other arguments as fp8kv_cache_insert.
 * Device checks: position outside [0, max_pos) -> token skipped entirely
 * (FP8KV_DEV_BAD_POSITION); bad slot -> K/V of that token skipped.
 * T = 0 launches nothing and returns FP8KV_OK without reading any pointer.
 */
int fp8kv_qk_norm_rope_insert(const void* q, const void* k, const void* v,
                              const int64_t* positions, const void* q_norm_w,
                              const void* k_norm_w, float eps, const float* cos_sin,
                              int max_pos, void* q_out, const int64_t* slot_mapping, int T,
                              int Hq, int Hkv, int D, const float* k_scale,
                              const float* v_scale, void* k_cache, void* v_cache,
                              int num_pages, int page_size, void* stream);

/*
 * fp8kv_prompt_attention -- causal attention of whole prompts over the rows the
 * projection produced (before, or beside, their cache insert): B sequences
 * packed one after another, with the masks and head grouping of
 * fp8kv_paged_attention.  (The pages have no counterpart: their prefill is the
 * serving engine's own.)
 *
 * Sequence b is the tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1; its token
 * at position p sees the keys j of the same sequence with j <= p and, when
 * window_left >= 0, j >= p - window_left; query head h reads KV head
 * h / (Hq/Hkv):
 *     out[t][h] = softmax_j( (q[t][h] . k[j][h']) * sm_scale ) . v[j][h']
 * computed on the tensor cores with fp32 accumulation, the softmax weights
 * rounded to bf16 for the second product, the result rounded to bf16.
 *
 *   q (device) bf16 [T][Hq][D], tokens q_stride elements apart; k, v bf16
 *     [T][Hkv][D], k_stride and v_stride apart (views of one projection's
 *     output are fine); strides >= heads * D and multiples of 8
 *   cu_seqlens (device) int32 [B + 1], non-decreasing, 0 <= ... <= T; equal
 *     neighbours are an empty sequence
 *   max_seq_len (host) >= every length
 *   sm_scale (host) > 0;  window_left (host) -1, or >= 0
 *   out (device) bf16 [T][Hq][D], dense; must not overlap the inputs.  Rows of
 *     no sequence (before the first, behind the last) are left as they are, and
 *     q, k, v there may hold anything.
 * Supported: D = 128, Hq/Hkv <= 128, T / (2 * floor(128 / (Hq/Hkv))) + B <= 65535;
 * no workspace.  B = 0 or T = 0 launches nothing and reads no pointer.
 * An infinity or NaN in a v row may reach, beyond the rows that see it, the
 * rows up to 2 * floor(128 / (Hq/Hkv)) positions around it (0 * infinity).
 * Device check: a sequence with bounds outside [0, T], out of order, or longer
 * than max_seq_len is skipped, its output rows left as they are
 * (FP8KV_DEV_BAD_SEQ_LEN); with bounds out of order other sequences may be
 * skipped too.
 */
int fp8kv_prompt_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int32_t* cu_seqlens, int B, int T, int max_seq_len,
                           int Hq, int Hkv, int D, float sm_scale, int window_left, void* out, void* stream);

/*
 * fp8kv_paged_attention_plan -- the split-KV partition fp8kv_paged_attention
 * will use for these host-visible sizes on the current device.
 *   split_tokens: 0 = choose automatically; otherwise a positive multiple of
 *   page_size.  Returns FP8KV_OK and writes *num_splits (>= 1, the largest
 *   number of partitions any sequence can have) and *split_tokens_out.
 * Over an INT4 cache a call with split_tokens = 0 may use fewer partitions than
 * these, or up to 8 that combine on chip; the workspace size below serves it.
 */
int fp8kv_paged_attention_plan(int B, int M, int Hq, int Hkv, int D, int page_size,
                               int max_seq_len, int window_left, int split_tokens,
                               int* num_splits, int* split_tokens_out);

/* Workspace bytes fp8kv_paged_attention needs for the same arguments: room
 * for the split-KV partials (fp32 output, max and sum per query row and
 * partition) when a sequence spans several partitions, counted even when the
 * call combines them on chip.  The size does not depend on the cache dtype.
 * 0 for one partition; (size_t)-1 on bad arguments. */
size_t fp8kv_paged_attention_workspace_size(int B, int M, int Hq, int Hkv, int D,
                                            int page_size, int max_seq_len, int window_left,
                                            int split_tokens);

/*
 * fp8kv_paged_attention -- exact paged attention over the cache for M new
 * query rows per sequence ("calibrated FP8 KV on Intel B70", "Initial
 * optimization order", items 2 and 4; M = 1 is decode, M = 12 the width-12
 * verifier of "Contract").
 *
 * Sequence b has L = seq_lens[b] tokens cached, the last M of them the new
 * rows; row m sits at position p = L - M + m and query head h reads KV head
 * h / (Hq/Hkv).  Key j is visible to row m iff j <= p and, when
 * window_left >= 0, j >= p - window_left (a window of W keys including the
 * row itself is window_left = W - 1).  Logical key j lives in physical page
 * block_table[b][j / page_size] at offset j % page_size.  With
 * Kd = decode(k_code) * k_scale, Vd = decode(v_code) * v_scale (BF16 cache:
 * the stored values, scales unused; INT4 cache: n s k_scale, n s v_scale):
 *     out[b][m][h] = softmax_j( (q . Kd_j) * sm_scale ) . Vd      (rounded to bf16)
 * computed with fp32 accumulation.  Long contexts are cut into partitions of
 * split_tokens keys whose partial (max, sum, unnormalised output) are combined
 * through their log-sum-exp: by a reduce kernel over workspace partials, or,
 * for one sequence (B = 1) of 17 to 128 rows per KV head (one row tile) on an
 * E4M3 cache in at most 8 partitions, on chip by the partitions of a KV head running as one
 * thread-block cluster (fp8kv_last_dispatch reports "cluster=N").  Over an
 * INT4 cache any call of one row tile (16 or 128 rows per KV head) in 2 to 8
 * partitions is combined on chip where all its clusters run at once.
 *
 *   q            (device) bf16 [B][M][Hq][D]
 *   k_cache, v_cache (device) [num_pages][Hkv][page_size][D] (cache_dtype)
 *   block_table  (device) int32 [B][max_pages_per_seq]; entries of pages with
 *                no visible key are never read (INT4: never used)
 *   seq_lens     (device) int32 [B]; max_seq_len (host) >= every seq_lens[b]
 *   k_scale, v_scale (device) fp32 scalars (E4M3 and INT4 only)
 *   sm_scale     (host) fp32 logit multiplier, e.g. 1/sqrt(D)
 *   window_left  (host) -1 for a global layer, else >= 0
 *   split_tokens (host) 0 = automatic, else a multiple of page_size
 *   workspace    (device) >= fp8kv_paged_attention_workspace_size(...) bytes,
 *                may be NULL when that size is 0; contents need no
 *                initialisation and are scratch after the call
 *   out          (device) bf16 [B][M][Hq][D]
 * Supported: D = 128, page_size 32 or 64, Hq % Hkv == 0, and either
 * 1 <= M <= 16 with M * (Hq/Hkv) <= 144 rows per KV head (any cache type), or
 * up to M = 16384 query rows per sequence on an E4M3 cache with partitions of
 * whole 128-key tiles (split_tokens 0 or a multiple of 128): a prefill chunk
 * at the end of the context, causal within the chunk, on the tcgen05 kernel
 * in 128-row tiles (Hkv * ceil(M * Hq/Hkv / 128) <= 65535); other shapes
 * return FP8KV_ERR_UNSUPPORTED, as do B > 65535 and Hkv > 65535.  B = 0 launches
 * nothing and returns FP8KV_OK without reading any pointer.
 * A NaN in a K row reaches the rows that see it.  A NaN (BF16 cache: or an
 * infinity) in a V row may reach, beyond those, the other rows of its KV head and
 * sequence (0 * NaN), and nothing else.
 * Device checks: seq_len < M, seq_len > max_seq_len or more pages than
 * max_pages_per_seq -> that sequence's output is left untouched
 * (FP8KV_DEV_BAD_SEQ_LEN); page ids outside [0, num_pages) read zeros.
 */
int fp8kv_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                          int cache_dtype, const int32_t* block_table, int max_pages_per_seq,
                          const int32_t* seq_lens, int max_seq_len, int B, int M, int Hq,
                          int Hkv, int D, int page_size, int num_pages, const float* k_scale,
                          const float* v_scale, float sm_scale, int window_left,
                          int split_tokens, void* workspace, size_t workspace_bytes, void* out,
                          void* stream);

/*
 * fp8kv_append_paged_attention -- one verifier step of a layer: the M new
 * tokens of every sequence are written to the cache, then attention runs
 * ("calibrated FP8 KV on Intel B70", "Contract": the insert at the new rows'
 * positions followed by the exact paged attention over the cache).
 *
 * Token m of sequence b (k_new, v_new: bf16 [B][M][Hkv][D], device) goes to
 * position p = seq_lens[b] - M + m, i.e. slot
 * block_table[b][p / page_size] * page_size + p % page_size, with the
 * fp8kv_cache_insert encoding; then fp8kv_paged_attention runs with the same
 * arguments.  Cache bytes and output are identical to fp8kv_cache_insert
 * with those slots followed by fp8kv_paged_attention.  On the tensor-memory
 * path with one 128-row tile per KV head the CTA whose partition holds a new
 * position writes it before loading that page (no separate insert launch);
 * over an INT4 cache this holds for the mma.sync kernel too (one tile of 16
 * rows per KV head); otherwise (several row tiles, or the mma.sync kernels over
 * the other caches) an append kernel runs first.  k_new and v_new must be 16-byte aligned; B = 0 is a no-op.
 * Device check: a block-table entry outside [0, num_pages) at a new
 * position -> that token is not written (FP8KV_DEV_BAD_SLOT).
 */
int fp8kv_append_paged_attention(const void* k_new, const void* v_new, const void* q, void* k_cache,
                                 void* v_cache, int cache_dtype, const int32_t* block_table,
                                 int max_pages_per_seq, const int32_t* seq_lens, int max_seq_len, int B,
                                 int M, int Hq, int Hkv, int D, int page_size, int num_pages,
                                 const float* k_scale, const float* v_scale, float sm_scale,
                                 int window_left, int split_tokens, void* workspace,
                                 size_t workspace_bytes, void* out, void* stream);

/*
 * fp8kv_paged_attention_per_head, fp8kv_append_paged_attention_per_head --
 * fp8kv_paged_attention and fp8kv_append_paged_attention on an E4M3 cache
 * written with per-head scales (fp8kv_cache_insert_per_head): KV head hk is
 * dequantized with k_scale[hk], v_scale[hk] (device fp32 [Hkv]), and the
 * append encodes head hk's new tokens with them:
 *     Kd = decode(k_code) * k_scale[hk],  Vd = decode(v_code) * v_scale[hk]
 * Every other argument, kernel choice, check and status as the per-tensor
 * entry points with cache_dtype = FP8KV_CACHE_E4M3 (the same workspace size).
 */
int fp8kv_paged_attention_per_head(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_table, int max_pages_per_seq,
                                   const int32_t* seq_lens, int max_seq_len, int B, int M, int Hq,
                                   int Hkv, int D, int page_size, int num_pages, const float* k_scale,
                                   const float* v_scale, float sm_scale, int window_left,
                                   int split_tokens, void* workspace, size_t workspace_bytes, void* out,
                                   void* stream);

int fp8kv_append_paged_attention_per_head(const void* k_new, const void* v_new, const void* q,
                                          void* k_cache, void* v_cache, const int32_t* block_table,
                                          int max_pages_per_seq, const int32_t* seq_lens, int max_seq_len,
                                          int B, int M, int Hq, int Hkv, int D, int page_size,
                                          int num_pages, const float* k_scale, const float* v_scale,
                                          float sm_scale, int window_left, int split_tokens,
                                          void* workspace, size_t workspace_bytes, void* out,
                                          void* stream);

/*
 * fp8kv_paged_attention_layers -- the verifier step of several layers in one
 * launch: for each layer in order, fp8kv_append_paged_attention (or, with
 * k_new = v_new = NULL, fp8kv_paged_attention) with the same results
 * ("Laguna S 2.1 B70 campaign transfer ledger", table "Result progression",
 * rows on graph coverage and persistent attention metadata; "Laguna S 2.1
 * INT4 -- calibrated FP8 KV on Intel B70", section "Contract": the width-12
 * verifier over the FP8 cache).
 *
 * One persistent, cooperative launch with one CTA per SM.  Layer order is
 * kept: a layer's queries and new tokens are read only after every output row
 * of the previous layer has been written, as if the previous layer's output
 * produced them.  The pages of the earlier context are loaded ahead, across
 * layer boundaries.  Partitions of a sequence's keys combine through the
 * workspace (normalised f16 partials in E4M3 code units and fp32 (max, sum),
 * as the cluster combine of fp8kv_paged_attention), so results equal those of
 * the per-layer calls within the attention tolerance, not bit for bit.
 *
 *   layers     (host) n_layers descriptors (1 .. 64), each naming one layer's
 *              tensors with the meaning, layout and dtype they have in
 *              fp8kv_append_paged_attention: q, k_new, v_new (device, bf16,
 *              k_new/v_new may both be NULL), k_cache, v_cache (device, E4M3),
 *              block_table, seq_lens (device, int32), k_scale, v_scale
 *              (device fp32), out (device bf16), and host sizes
 *              max_pages_per_seq, max_seq_len, num_pages, window_left,
 *              sm_scale.  Layers may share or have their own tensors.
 *   B, M, Hq, Hkv, D, page_size, cache_dtype: as fp8kv_paged_attention, the
 *              same for every layer.
 *   workspace  (device) >= fp8kv_paged_attention_layers_workspace_size bytes,
 *              16-byte aligned.  Its first bytes hold the launch's
 *              synchronisation counters: they must be zero before the first
 *              call on a workspace (cudaMemset once) and every call leaves
 *              them zero.  Calls sharing a workspace must not overlap on the
 *              GPU.
 * Supported: E4M3 cache, D = 128, page_size 32 or 64, 16 < M*Hq/Hkv <= 128
 * (one 128-row tile of verifier rows per KV head), any B (with more work
 * units than SMs, a CTA runs several units of a layer one after another);
 * other shapes return FP8KV_ERR_UNSUPPORTED.  Per-layer arguments are
 * validated as in fp8kv_paged_attention before anything is launched.
 * Device checks as fp8kv_paged_attention; a wait that runs out (2 s) sets
 * FP8KV_DEV_WAIT_TIMEOUT and the launch still ends.
 */
typedef struct {
    const void* q;
    const void* k_new;
    const void* v_new;
    void* k_cache;
    void* v_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const float* k_scale;
    const float* v_scale;
    void* out;
    int max_pages_per_seq;
    int max_seq_len;
    int num_pages;
    int window_left;
    float sm_scale;
} fp8kv_layer;

/* Workspace bytes of fp8kv_paged_attention_layers; (size_t)-1 on bad arguments. */
size_t fp8kv_paged_attention_layers_workspace_size(int n_layers, int B, int M, int Hq, int Hkv);

int fp8kv_paged_attention_layers(const fp8kv_layer* layers, int n_layers, int B, int M, int Hq, int Hkv,
                                 int D, int page_size, int cache_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * Trees of drafted tokens.  The next five entry points are one step of
 * speculative decoding over a tree (the pages verify a chain of 12 rows and leave
 * the draft and the acceptance to the serving engine; a chain is the tree whose
 * node m hangs from m - 1).  A tree has M nodes (M <= 64), the same M for every
 * sequence of a batch: node 0 is the last accepted token, node m > 0 a drafted one
 * behind node parents[m] < m.  A node whose parent is -1, or is padding itself, is
 * padding (a sequence with fewer nodes).  The nodes' K and V rows are the last M of
 * the cache: node m at index L - M + m of a sequence of L = seq_lens[b], whatever
 * its depth; its position (what rotates it, and what a window counts) is
 * L - M + depth.
 *
 * fp8kv_tree_metadata -- what the other calls of the step need from the parents:
 *     tree_mask[b][m]    = bits of m and its ancestors (0 for padding)
 *     positions[b][m]    = L - M + depth of m          (padding: L - M)
 *     slot_mapping[b][m] = the cache slot of index L - M + m (padding: -1)
 *
 *   parents       (device) int32 [B][M]; parents[b][0] is not used
 *   seq_lens      (device) int32 [B], the nodes included
 *   block_table   (device) int32 [B][max_pages_per_seq]
 *   max_seq_len   (host) >= every length
 *   tree_mask     (device) uint64 [B][M];  positions, slot_mapping (device) int64 [B][M];
 *                 none overlaps another or an input
 * B = 0 launches nothing and reads no pointer.
 * Device checks: a parent outside [-1, m) -> padding, FP8KV_DEV_BAD_TREE; a length
 * < M, > max_seq_len or beyond the block-table row -> mask 0, position 0, slot -1
 * for the whole sequence, FP8KV_DEV_BAD_SEQ_LEN; a page outside [0, num_pages) ->
 * slot -1, FP8KV_DEV_BAD_SLOT.
 */
int fp8kv_tree_metadata(const int32_t* parents, const int32_t* seq_lens, const int32_t* block_table,
                        int max_pages_per_seq, int max_seq_len, int B, int M, int num_pages, int page_size,
                        uint64_t* tree_mask, int64_t* positions, int64_t* slot_mapping, void* stream);

/*
 * fp8kv_rope_insert -- rotary positions on Q and K, then K and V into the cache:
 * fp8kv_qk_norm_rope_insert without the norms, for every cache type, both layouts
 * of the pairs and heads that rotate in part.  With pos = positions[t],
 * c_k = cos_sin[pos][k], s_k = cos_sin[pos][rot_dim / 2 + k], for each Q and K head
 * row x and k < rot_dim / 2, (i, j) = (k, k + rot_dim / 2), or (2 k, 2 k + 1) when
 * interleaved:
 *     o_i = bf16( fma(x_i, c_k, -(x_j * s_k)) )     o_j = bf16( fma(x_j, c_k, x_i * s_k) )
 * in fp32; o = x for the elements behind rot_dim.  Q rows go to q_out, the rotated
 * K rows and the V rows into the cache as in fp8kv_cache_insert.  Angles scaled for
 * long contexts, and a factor on cosines and sines, are the table's.
 *
 *   q (device) bf16 [T][Hq][D], tokens q_stride elements apart; k, v bf16
 *     [T][Hkv][D], k_stride and v_stride apart (views of one projection's output are
 *     fine); strides >= heads * D and multiples of 8
 *   positions (device) int64 [T];  cos_sin (device) fp32 [max_pos][rot_dim]
 *   rot_dim (host) a multiple of 8, 8 .. D;  interleaved (host) 0 or not
 *   q_out (device) bf16 [T][Hq][D], dense; must not overlap q, k or v
 *   other arguments as fp8kv_cache_insert.
 * Device checks: position outside [0, max_pos) -> token skipped entirely
 * (FP8KV_DEV_BAD_POSITION); slot >= num_pages*page_size -> K/V of that token skipped
 * (FP8KV_DEV_BAD_SLOT).  A negative slot skips the token's K/V, not its Q.
 * T = 0 launches nothing and returns FP8KV_OK without reading any pointer.
 */
int fp8kv_rope_insert(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int64_t* positions, const float* cos_sin, int max_pos, int rot_dim,
                      int interleaved, void* q_out, const int64_t* slot_mapping, int T, int Hq, int Hkv, int D,
                      const float* k_scale, const float* v_scale, void* k_cache, void* v_cache, int num_pages,
                      int page_size, int cache_dtype, void* stream);

/*
 * fp8kv_tree_attention -- fp8kv_paged_attention (k_new = v_new = NULL) or
 * fp8kv_append_paged_attention for the M nodes of a tree: row m sees the L - M
 * cached keys before the nodes and the nodes i whose bit is set in
 * tree_mask[b][m] (an ancestor set with m itself, as fp8kv_tree_metadata writes
 * it; bits >= M are ignored).  With window_left >= 0 row m, at position
 * p_m = L - M + (bits in tree_mask[b][m]) - 1 (mask 0: L - M), sees of those the
 * keys at positions >= p_m - window_left, node i being at position p_i.  A row without visible keys,
 * and a row whose mask is 0 (padding), is written as zeros.  The mask of a chain
 * gives fp8kv_paged_attention's result (up to roundings).  The K and V rows of a node
 * that is in no row's mask reach no output, whatever they hold (nobody writes those of
 * padding, slot -1); of the others' V rows, as of the context's: a NaN or an infinity
 * may reach rows that do not see it (fp8kv_paged_attention), a sibling's too.
 *
 *   tree_mask  (device) uint64 [B][M]
 *   split_tokens (host) 0, or a multiple of page_size; of 128 for more than 16 rows
 *              M * Hq/Hkv per KV head
 *   every other argument, the workspace and the device checks: as
 *   fp8kv_append_paged_attention (per-tensor scales); out must not overlap q, k_new,
 *   v_new or tree_mask.
 * Supported: D = 128, page_size 32 or 64, Hq % Hkv == 0, 1 <= M <= 64, every cache
 * type.  With k_new, the rows of padding nodes are written too.
 */
int fp8kv_tree_attention(const void* k_new, const void* v_new, const void* q, void* k_cache, void* v_cache,
                         int cache_dtype, const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens,
                         int max_seq_len, const uint64_t* tree_mask, int B, int M, int Hq, int Hkv, int D,
                         int page_size, int num_pages, const float* k_scale, const float* v_scale, float sm_scale,
                         int window_left, int split_tokens, void* workspace, size_t workspace_bytes, void* out,
                         void* stream);

/*
 * fp8kv_verify_tree -- which drafted tokens stand, and the token after them.
 * Row n of target_probs is the target's distribution p_n of the token behind node n,
 * row n of draft_probs the distribution q_n that n's children were drawn from,
 * independently (draft_probs = NULL: they were chosen, q_n is 1 at a child's
 * token).  From node n = 0, with w = p_n and S = 1, n's children are taken in the
 * order of their index; child m with token x stands when
 *     w(x) > 0  and  uniforms[m] * S * q_n(x) < w(x)
 * and the walk goes on at n = m; otherwise
 *     w <- max(w - S q_n, 0), S <- sum of w     (NULL: S <- S - w(x), w(x) <- 0).
 * When no child is left, the next token is the first v whose running sum of w
 * exceeds uniforms[0] times the sum of w (of p_n, should nothing be left of it).
 * With uniforms drawn from [0, 1) and rows that sum to 1 the tokens are distributed as
 * the target alone would draw them (S begins at 1, not at a row's sum: what a row's sum
 * lacks, some 2^-9 of a bf16 row, the distribution may be off by).  A greedy target is
 * one with rows of one 1.
 *
 *   target_probs, draft_probs (device) fp32 or bf16 (prob_dtype) [B][M][V], the rows
 *     of consecutive nodes target_stride and draft_stride elements apart (>= V);
 *     entries that are negative or NaN count as 0.  Rows of leaves of draft_probs
 *     are not read.
 *   tokens, parents (device) int32 [B][M] (tokens[b][0], parents[b][0] not used)
 *   uniforms   (device) fp32 [B][M] in [0, 1)
 *   out_tokens (device) int32 [B][M]: the tokens that stand, the next one, then -1
 *   num_tokens (device) int32 [B]: how many those are, 1 .. M; without a next token
 *     (FP8KV_DEV_BAD_PROBS) one less, 0 .. M - 1
 *   path       (device) int32 [B][M]: node 0 and the nodes that stand, then -1
 *     The outputs overlap neither one another nor an input, but out_tokens and path
 *     may each be one of the [B][M] inputs itself.
 * Pairs of fp32: a weight is off by at most 2^-45 of what it was before the fall, a
 * sum by (16 + V / (256 c)) 2^-44 of itself, c = 1 .. 16 CTAs a sequence (1 for more
 * than 256 sequences, 16 for up to 32 of 32768 tokens or more).  Any V up to 2^30; no
 * workspace.  B = 0 launches nothing and reads no pointer.
 * Device checks: a parent outside [-1, m), or a node's token outside [0, V) -> that
 * node is padding, FP8KV_DEV_BAD_TREE; a row p_n without a positive, finite sum
 * where the next token is drawn -> no next token (-1, not counted),
 * FP8KV_DEV_BAD_PROBS.
 */
int fp8kv_verify_tree(const void* target_probs, int64_t target_stride, const void* draft_probs, int64_t draft_stride,
                      int prob_dtype, const int32_t* tokens, const int32_t* parents, const float* uniforms, int B,
                      int M, int V, int32_t* out_tokens, int32_t* num_tokens, int32_t* path, void* stream);

/*
 * fp8kv_cache_keep_path -- after the verification: in the caches of n_layers layers
 * (one launch) the K and V rows of the nodes path[b][0 .. n) (the leading entries
 * >= 0) go to indices L - M .. L - M + n - 1, as if all were read before any is
 * written, and new_seq_lens[b] = L - M + n.  What was behind them stays.  The next
 * token is not in the cache: with the next tree it is node 0.
 *
 *   k_caches, v_caches (host) arrays of n_layers (1 .. 64) device pointers, each a
 *     cache of its own (none overlaps another), all of the same cache_dtype, num_pages and Hkv
 *   block_table, seq_lens (device) as fp8kv_paged_attention, the same for all layers
 *   path         (device) int32 [B][M], as fp8kv_verify_tree writes it
 *   new_seq_lens (device) int32 [B]; must not overlap the other arguments
 * B = 0 launches nothing and reads no pointer.
 * Device checks: a path that does not begin with 0, ascend below M and end in -1s ->
 * that sequence keeps its rows and its length, FP8KV_DEV_BAD_TREE; a bad length
 * likewise, FP8KV_DEV_BAD_SEQ_LEN; a page outside [0, num_pages) -> the rows from
 * and to it are not moved, FP8KV_DEV_BAD_SLOT.
 */
int fp8kv_cache_keep_path(void* const* k_caches, void* const* v_caches, int n_layers, int cache_dtype,
                          const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens, int max_seq_len,
                          const int32_t* path, int B, int M, int Hkv, int D, int num_pages, int page_size,
                          int32_t* new_seq_lens, void* stream);

/*
 * fp8kv_paged_attention_noalloc -- fp8kv_paged_attention without a
 * caller-provided workspace.  (The pages have no counterpart: this is an
 * integration convenience, not part of the method.)
 *
 * For callers that cannot allocate device memory where they run attention
 * (an allocator-free serving loop, a fully carved-up memory pool, host code
 * holding only a raw stream): the split-KV partials go to a buffer that is a
 * file-scope __device__ array of FP8KV_NOALLOC_WORKSPACE_BYTES (32 MiB) inside
 * the library.  Every GPU that loads the library holds that buffer until the
 * process exits.  The call allocates nothing (no cudaMalloc, no allocating
 * library routine).
 *
 * Arguments and results are those of fp8kv_paged_attention without
 * workspace / workspace_bytes; out must hold B*M*Hq*D bf16 values (the C
 * entry point cannot check its size).  Every argument is validated first,
 * with the statuses of fp8kv_paged_attention; then a request whose workspace
 * size (fp8kv_paged_attention_workspace_size) exceeds 32 MiB returns
 * FP8KV_ERR_WORKSPACE (a larger split_tokens needs less; otherwise use the
 * allocating entry point).  The first call on a device looks up the buffer's
 * device address (cudaGetSymbolAddress, with that device current) and keeps
 * it for the life of the process; make that first call before any stream
 * capture.  A cudaDeviceReset while the library is loaded is not supported
 * (the kept address, like the kernels' shared-memory opt-ins, would be
 * stale).  Every call shares the one buffer, which keeps
 * the last call's contents (no part of it needs to start at zero): calls
 * that overlap on the GPU -- on different streams, or from several threads --
 * race and must be serialised by the caller.
 */
int fp8kv_paged_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                  int cache_dtype, const int32_t* block_table,
                                  int max_pages_per_seq, const int32_t* seq_lens, int max_seq_len,
                                  int B, int M, int Hq, int Hkv, int D, int page_size,
                                  int num_pages, const float* k_scale, const float* v_scale,
                                  float sm_scale, int window_left, int split_tokens, void* out,
                                  void* stream);

/*
 * fp8kv_e4m3_encode_bits -- encode the fp32 bit patterns first .. first+n-1
 * with the same device routine the insert kernels use (for exhaustive checks
 * of the encoder).  out (device) uint8 [n].
 */
int fp8kv_e4m3_encode_bits(uint32_t first, size_t n, uint8_t* out, void* stream);

/*
 * fp8kv_selftest_bounded_wait -- exercise the device-side failure path of a
 * pipeline wait: one warp waits on a barrier that by construction gets no
 * arrival; after limit_us microseconds (1 .. 2000000) the wait gives up, sets
 * FP8KV_DEV_WAIT_TIMEOUT in the device status word and the kernel returns, so
 * the context stays usable.  Every barrier wait of the attention kernels takes
 * the same path after 2 s.  ("Laguna S 2.1 B70 campaign transfer ledger",
 * section "Harness, recovery, and evidence lessons": a stage that does not
 * finish is classified from a bounded wait and a recorded marker, never left
 * to hang.)  Returns FP8KV_OK when launched; read the bit with
 * fp8kv_device_status().
 */
int fp8kv_selftest_bounded_wait(unsigned int limit_us, void* stream);

/* Text of a status code (static storage). */
const char* fp8kv_status_string(int status);

/* Kernel variant and partition count chosen by the last fp8kv_paged_attention
 * call on this host thread, as text (truncated to n-1 bytes).  Returns the
 * full length. */
int fp8kv_last_dispatch(char* buf, size_t n);

/* Number of kernel launches this library has made in this process (all
 * threads, all devices), e.g. the launches one step captures into a graph. */
unsigned long long fp8kv_launch_count(void);

/* Read (and with clear != 0, reset) the device status word of the current
 * device.  Synchronises the device.  Returns FP8KV_OK or FP8KV_ERR_CUDA. */
int fp8kv_device_status(unsigned int* status, int clear);

#ifdef __cplusplus
}
#endif

#endif /* FP8KV_H */
