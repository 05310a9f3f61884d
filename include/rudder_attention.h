/*
 * rudder_attention.h -- what stands between the QKV and the O linear of a
 * block: a paged cache of keys and values in 8 bits, attention over it, and
 * cross attention to an encoder's states.
 *
 * The conventions of rudder.h hold: device pointers, asynchronous calls on
 * `stream`, host checks before any launch, no allocation, safe to capture in a
 * HIP graph.  The device current on the calling thread must be the device of
 * `stream`.
 *
 * Rows.  Query, key and value rows of B sequences are packed one behind the
 * other: sequence b has rows row_start[b] .. row_start[b + 1] - 1 (int32
 * [B + 1], ascending) of T.  A row is [heads][D] with D contiguous; ld* is the
 * distance between rows in elements (a multiple of 8), so that the three parts
 * of a QKV linear's output can be passed as they lie.  max_rows is an upper
 * bound on the rows of one sequence; rows of a sequence beyond it are not
 * processed.  Rows behind row_start[B] are left as they were.
 *
 * Device arrays are not trusted with addresses: row numbers are clamped to
 * [0, T], lengths to [0, max_kv] and the page table's width, and a page number
 * outside [0, num_pages) is a page that is not there (its tokens are not
 * written, and not visible).
 *
 * Cache.  A page holds RUDDER_CACHE_PAGE = 64 tokens of every head:
 *   codes   int8 [num_pages][Hkv][2][64 * D]: half 0 the keys as
 *           [token][channel], half 1 the values as [channel][token]
 *   scales  fp32 [num_pages][Hkv][2]: one step size per block (page, head, K|V)
 *   page_table  int32 [B][max_pages]: page_table[b][i] holds the sequence's
 *           tokens 64 i .. 64 i + 63
 * A value is fl32(code * scale).  Pages belong to the caller: sequences may
 * share pages that no append writes to.
 * Undefined results (not checked; no access leaves the buffers): non-finite
 * keys, values (an encoder's too) or scales, sequences of one append call that
 * write to the same page, or one that lists it twice, overlapping buffers.
 */
#ifndef RUDDER_ATTENTION_H
#define RUDDER_ATTENTION_H

#include "rudder.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RUDDER_CACHE_PAGE 64

/* Bytes of codes of one page (Hkv * 2 * 64 * D), 0 for invalid sizes. */
size_t rudder_cache_page_bytes(int Hkv, int D);

/*
 * Quantizes new keys and values into the cache: sequence b's rows become its
 * tokens pos[b], pos[b] + 1, ...  Per block that receives rows, with x the
 * block's new values and s the scale it had (0 where its token 0 is new):
 *   s'  = max(s, fl32(max |x| / 127))                     (formed in fp64)
 *   old codes in front of the new ones:
 *   c'  = rne(c * fl32(s / s'))   where s' > s            (formed in fp64)
 *   new codes:  c = rne(clamp(x * fl32(1 / s'), -127, 127))
 * Codes behind the new ones are left as they were.  Appending the same rows at
 * the same place again changes nothing.  One launch.
 *
 *   K, V    bf16 bits [T][Hkv][D] with row distances ldk, ldv
 *   pos     int32 [B], the number of tokens in front; a negative one skips
 *           the sequence
 *   B, T >= 0 (0 is a no-op), max_rows >= 0, max_pages, num_pages, Hkv > 0,
 *   D 64 or 128
 * Errors: INVALID_ARG for a null pointer, a negative or zero size, ldk or ldv
 * below Hkv * D or not a multiple of 8, K, V, codes or scales not 16-byte aligned;
 * UNSUPPORTED for D other than 64 or 128, B > 65535, Hkv > 4096, more than
 * 2^29 rows.
 */
rudder_status_t rudder_cache_append(const uint16_t* K, const uint16_t* V,
                                    const int32_t* row_start, const int32_t* pos,
                                    const int32_t* page_table, int B, int T, int max_rows,
                                    int max_pages, int num_pages, int Hkv, int D, int ldk,
                                    int ldv, int8_t* codes, float* scales, void* stream);

/*
 * Whole pages back as values: K_out, V_out fp32 [n][Hkv][64][D], both as
 * [token][channel], for the n page numbers in `pages` (int32; repeated ones
 * are allowed; one outside the pool gives zeros).
 * Errors: INVALID_ARG for a null pointer, n < 0, num_pages or Hkv <= 0, codes,
 * K_out or V_out not 16-byte aligned; UNSUPPORTED for D other than 64 or 128,
 * Hkv > 4096, n > 2^23.
 */
rudder_status_t rudder_cache_dequant(const int8_t* codes, const float* scales,
                                     const int32_t* pages, int n, int num_pages, int Hkv, int D,
                                     float* K_out, float* V_out, void* stream);

/*
 * Bytes of workspace the two attention calls need for these sizes (0 for
 * sizes they refuse, and for sizes that need none).  Calls that may run at the
 * same time -- on two streams, or in two graphs replayed side by side -- need
 * a workspace each.
 * Smaller sizes may need more: fewer rows give fewer workgroups, and then the
 * keys are split (B = 2, 16 heads of 128 channels, 16384 keys: none for 4096
 * rows, 34 MB for one).  A buffer for calls of several sizes is as large as
 * rudder_attention_workspace_bound says for the largest of each: no call of the
 * same heads and channels with B, T, max_rows and max_kv up to these needs more.
 */
size_t rudder_attention_workspace_bytes(int B, int T, int max_rows, int max_kv, int Hq, int Hkv,
                                        int D);
size_t rudder_attention_workspace_bound(int B, int T, int max_rows, int max_kv, int Hq, int Hkv,
                                        int D);

/*
 * Attention of new rows to the cache.  For row i of sequence b (n rows,
 * kv = kv_len[b] tokens in the cache, the new ones among them once appended),
 * head h of Hq and its cached head h / (Hq / Hkv):
 *   o = sum_j softmax_j(sm * q . k_j) v_j,  j < kv, and where causal is
 *       not 0 also j <= kv - n + i
 * A row whose mask leaves nothing (kv = 0, or i in front of the first token)
 * gives zeros whatever its query, any other query row that is not finite NaN.
 * q enters q . k with an absolute error of at most 2^-15 of its row's largest
 * power of two (2^-14 for an element of magnitude 255/128 times that power);
 * the products with the codes are exact, their sums rounded to fp32 (2^-24).
 * The softmax is in fp32, its weights rounded to fp16 for the product with the
 * codes of V, fp32 sums, one rounding to bf16.  V scales below 2^-80 count as
 * 2^-80.
 *
 *   Q, O     bf16 bits [T][Hq][D], row distances ldq, ldo
 *   kv_len   int32 [B]; max_kv an upper bound on them (larger ones are cut)
 *   sm       the softmax scale, e.g. 1 / sqrt(D); sm times a row's largest element
 *            stays below 2^127
 *   workspace, workspace_bytes  at least rudder_attention_workspace_bytes(...)
 *            bytes (NULL if 0)
 *   B, T, max_rows, max_kv >= 0 (B, T or max_rows 0 is a no-op), Hq a multiple
 *   of Hkv, D 64 or 128
 * At most two launches: where the rows give too few workgroups, the tokens
 * are split in pieces, joined in a fixed order.  Results do not depend on
 * anything but the arguments.
 * Errors: INVALID_ARG for a null required pointer, negative sizes, Hq or Hkv
 * <= 0, Hq % Hkv != 0, max_pages or num_pages <= 0, ldq or ldo below Hq * D or
 * not a multiple of 8, sm not finite or beyond 2^127 in magnitude, a workspace
 * that is too small, Q, codes, O
 * or workspace not 16-byte aligned;
 * UNSUPPORTED for D other than 64 or 128, Hkv > 4096, B * Hkv > 65535,
 * max_kv > 2^30, min(max_rows, T) * Hq > 2^26, or B * Hkv *
 * ceil(max_rows * Hq / Hkv / 128) > 2^21 (give max_rows as it is, not a far
 * larger bound).
 */
rudder_status_t rudder_cache_attention(const uint16_t* Q, const int32_t* row_start,
                                       const int32_t* kv_len, const int32_t* page_table,
                                       const int8_t* codes, const float* scales, int B, int T,
                                       int max_rows, int max_kv, int max_pages, int num_pages,
                                       int Hq, int Hkv, int D, int ldq, int ldo, float sm,
                                       int causal, void* workspace, size_t workspace_bytes,
                                       uint16_t* O, void* stream);

/*
 * Cross attention to states of another length: as above without a cache, all
 * of a sequence's keys visible to each of its rows.
 *
 *   K, V      bf16 bits [Tkv][Hkv][D], row distances ldk, ldv
 *   kv_start  int32 [B]: sequence b's first key row (a padded batch has
 *             b * length, a packed one the sums of the lengths)
 *   kv_len    int32 [B]: its keys; rows behind them are not read
 * Products in bf16 with fp32 sums, the softmax weights as the sum of two bf16
 * numbers (2^-16 relative).
 * Errors: as rudder_cache_attention, also for K, V, ldk, ldv, Tkv < 0.
 */
rudder_status_t rudder_cross_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                       const int32_t* row_start, const int32_t* kv_start,
                                       const int32_t* kv_len, int B, int T, int Tkv, int max_rows,
                                       int max_kv, int Hq, int Hkv, int D, int ldq, int ldk,
                                       int ldv, int ldo, float sm, void* workspace,
                                       size_t workspace_bytes, uint16_t* O, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RUDDER_ATTENTION_H */
