/*
 * rudder_block.h -- what a block's forward pass does around its linears and
 * their attention to a cache: the norms with the residual's addition in front
 * of the QKV and up linears, rotary positions on the queries and keys, and
 * causal attention of whole prompts.
 *
 * The conventions of rudder.h hold: device pointers, asynchronous calls on
 * `stream`, host checks before any launch, no allocation, safe to capture in a
 * HIP graph.  The device current on the calling thread must be the device of
 * `stream`.  Rows of sequences, their clamping to the buffers, row distances
 * (ld*, in elements) and rows behind the last sequence are as in
 * rudder_attention.h.
 */
#ifndef RUDDER_BLOCK_H
#define RUDDER_BLOCK_H

#include "rudder.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm of the residual stream with the residual's addition in
 * front of it, bf16 rows out:
 *   h[m][k] = bf16_rne(R[m][k] + X[m][k])           (h = X without R)
 *   r[m]    = fl32(1 / sqrt(sum_k h^2 / K + eps))   (formed in fp64)
 *   y[m][k] = bf16_rne(fl32(fl32(h * r) * gamma[k]))
 * One launch; results do not depend on the order of the sum.
 *
 *   X       bf16 bits [M][K], row distance ldx
 *   R, H    bf16 bits [M][K], row distances ldr, ldh: the residual stream and
 *           where h is written; both or neither (NULL).  H may be R or X (with
 *           the same row distance)
 *   gamma   fp32 [K]
 *   Y       out: bf16 bits [M][K], row distance ldy; may be X or R (with the
 *           same row distance) where H is another buffer or NULL
 *   M       >= 0 (0 is a no-op), K > 0 a multiple of 8, eps >= 0 finite
 * A row that is not finite gives what the formula gives, in that row only.
 * Errors: INVALID_ARG for a null X, gamma or Y, R without H or H without R,
 * M < 0, K <= 0 or not a multiple of 8, a row distance below K or not a
 * multiple of 8 (those of NULL are not looked at), eps negative or not finite,
 * X, R, H, gamma or Y not 16-byte aligned, Y the same buffer as H, H or Y in the
 * place of X or R at another row distance; UNSUPPORTED for K > RUDDER_MAX_K, M >
 * 2^25 or M * K > 2^35.
 */
rudder_status_t rudder_norm(const uint16_t* X, const uint16_t* R, const float* gamma, float eps,
                            int M, int K, int ldx, int ldr, int ldh, int ldy, uint16_t* H,
                            uint16_t* Y, void* stream);

/*
 * The same norm with the next linear's activation quantizer behind it: packed
 * codes and row scales for rudder_linear, the bf16 rows never reach HBM.  With
 * step sizes from the (layer, step) table the codes are exactly those of
 * rudder_norm followed by rudder_quant_act; without one every row has a step
 * size of its own:
 *   u          = y[m][k] * inv_smooth[k]
 *   D          = act_scale[stream_id[m]], or fl32(max_k |u| / Qa)  (fp64 divide),
 *                0 in place of 2^-128 and below, whose reciprocal passes 32 bits
 *   q[m][k]    = rne(clamp(u * fl32(1 / D), -Qa, Qa)),  row_scale[m] = D
 * One launch.
 *
 *   stream_id, act_scale  uint8 [M], each < S, and fp32 [S], as for
 *              rudder_quant_act; act_scale NULL: a step size a row (stream_id
 *              and S are not looked at)
 *   inv_smooth fp32 [K] from rudder_quantize_weights
 *   abits, codes  as for rudder_quant_act
 *   Xq, row_scale out: as for rudder_quant_act (padding rows are 0)
 *   K          a multiple of 32 (64 for RUDDER_CODES_E2M3)
 * A row that is not finite has undefined codes, in that row only; without a
 * table its row scale is NaN or infinite.
 * Errors: those of rudder_norm (Y apart), INVALID_ARG also for a null
 * inv_smooth, Xq or row_scale, act_scale without stream_id, K not a multiple
 * of 32 (of 64 for E2M3), S outside 1..8 with a table, abits not 4 or 8, an
 * unknown container, inv_smooth or Xq not 16-byte aligned; UNSUPPORTED also for
 * E2M3 with abits = 8 (8-bit E2M3 codes are not built for this path).
 */
rudder_status_t rudder_norm_quant(const uint16_t* X, const uint16_t* R, const uint8_t* stream_id,
                                  const float* gamma, const float* inv_smooth,
                                  const float* act_scale, float eps, int M, int K, int S,
                                  int abits, int codes, int ldx, int ldr, int ldh, uint16_t* H,
                                  void* Xq, float* row_scale, void* stream);

/*
 * Packed activation codes (either container) back as values:
 * out[m][k] = fl32(q[m][k] * row_scale[m]), fp32 [M][K] row-major.
 * Errors: INVALID_ARG for a null pointer, M < 0, K <= 0 or not a multiple of 32
 * (64 for E2M3), abits not 4 or 8, an unknown container, Xq or out not 16-byte
 * aligned; UNSUPPORTED for K > RUDDER_MAX_K, M > 2^25 or M * K > 2^35.
 */
rudder_status_t rudder_dequant_act(const void* Xq, const float* row_scale, int M, int K, int abits,
                                   int codes, float* out, void* stream);

/* Which channels of a head's rotated part (its first rotary_dim channels, n =
 * rotary_dim / 2 pairs) are a pair. */
typedef enum {
    RUDDER_ROTARY_HALF = 0,    /* i and i + n */
    RUDDER_ROTARY_PAIRS = 1    /* 2 i and 2 i + 1 */
} rudder_rotary_layout_t;

/* How the frequencies base^(-i / n) are changed for contexts longer than those
 * trained on, by `factor` >= 1. */
typedef enum {
    RUDDER_ROTARY_PLAIN = 0,   /* not */
    RUDDER_ROTARY_LINEAR = 1,  /* divided by factor */
    RUDDER_ROTARY_BASE = 2,    /* base times factor^(n / (n - 1)): the slowest pair is divided by
                                  factor, the fastest stays (n = 1: not changed) */
    RUDDER_ROTARY_PARTS = 3    /* by a pair's turns over the trained length ("NTK by parts"):
                                  divided by factor up to `low` turns, left from `high` on, between
                                  them in proportion */
} rudder_rotary_scaling_t;

/*
 * Frequencies of the n = rotary_dim / 2 pairs in radians a position, HOST
 * memory fp64 [n], for rudder_rotary (which takes them on the device):
 *   f[i] = base^(-i / n), then by `scaling`; for RUDDER_ROTARY_PARTS
 *   keep = clamp((trained * f / (2 pi) - low) / (high - low), 0, 1)
 *   f[i] = f / factor * (1 - keep) + f * keep
 * trained, low and high are looked at for RUDDER_ROTARY_PARTS only, factor not
 * for RUDDER_ROTARY_PLAIN.
 * Errors: INVALID_ARG for a null freq, rotary_dim <= 0 or odd, base not above 0
 * or not finite, an unknown scaling, factor below 1 or not finite, trained not
 * above 0 or not finite, low negative, high not above low or not finite, a
 * raised base or a frequency that is not finite; UNSUPPORTED for rotary_dim >
 * 2^16.
 */
rudder_status_t rudder_rotary_frequencies(int rotary_dim, double base, int scaling, double factor,
                                          double trained, double low, double high, double* freq);

/*
 * Rotary positions on the query and key heads of B sequences.  Row i of
 * sequence b has position pos[b] + i; with a = position * freq[j],
 *   (x, y) -> (x c - y s, y c + x s),  c = magnitude * cos(a), s = magnitude * sin(a)
 * for each pair j of the first rotary_dim channels of each head; the others are
 * copied.  a is right to 2^-25 turns for every position and frequencies of up to
 * 2^24 in magnitude, c and s and the sums are fp32, one rounding to bf16.  One
 * launch.
 *
 *   Q, K      bf16 bits [T][Hq][D], [T][Hkv][D], row distances ldq, ldk: e.g.
 *             two parts of a QKV linear's output
 *   Qo, Ko    out, row distances ldqo, ldko; may be Q and K (with the same row
 *             distances)
 *   pos       int32 [B], or NULL for zeros; a negative one skips the sequence
 *   freq      fp64 [rotary_dim / 2]
 *   magnitude a factor on all rotated channels (1, or what a stretched context
 *             asks for)
 *   B, T, max_rows >= 0 (0 is a no-op), Hq > 0, Hkv >= 0 (0: K and Ko may be
 *   NULL), D 64 or 128, rotary_dim a multiple of 16 up to D
 * Errors: INVALID_ARG for a null pointer, negative sizes, Hq <= 0, an unknown
 * layout, rotary_dim <= 0, above D or not a multiple of 16, a row distance
 * below its heads' channels or not a multiple of 8, magnitude not finite, Q, K,
 * Qo or Ko not 16-byte aligned, Qo or Ko in the place of Q or K at another row
 * distance; UNSUPPORTED for D other than 64 or 128, B > 65535, Hq or Hkv > 4096,
 * more than 2^25 rows.
 */
rudder_status_t rudder_rotary(const uint16_t* Q, const uint16_t* K, const int32_t* row_start,
                              const int32_t* pos, const double* freq, float magnitude, int B,
                              int T, int max_rows, int Hq, int Hkv, int D, int rotary_dim,
                              int layout, int ldq, int ldk, int ldqo, int ldko, uint16_t* Qo,
                              uint16_t* Ko, void* stream);

/*
 * Bytes of workspace rudder_prompt_attention needs for these sizes (0 for sizes
 * it refuses, and for sizes that need none).  Calls that may run at the same
 * time -- on two streams, or in two graphs replayed side by side -- need a
 * workspace each.  No smaller B, T or max_rows of the same heads and channels
 * needs more.
 */
size_t rudder_prompt_attention_workspace_bytes(int B, int T, int max_rows, int Hq, int Hkv, int D);

/*
 * Causal attention of whole prompts, packed one behind the other, to their own
 * keys and values.  For row i of sequence b, head h of Hq and its key head
 * h / (Hq / Hkv):
 *   o = sum_j softmax_j(sm * q . k_j) v_j,  j <= i
 * Products of q and k in bf16 with fp32 sums; the softmax is in fp32 and goes by
 * the differences of these sums, however far from zero they are, its weights
 * rounded to fp16 (2^-11; 2^-33 of the largest below 2^-22 of it); v enters with
 * an absolute error of at most 2^-32 of the largest magnitude of its head in its
 * tile (64 tokens, counted from the prompt's first), or, where the row sees only
 * part of that tile, of at most 2^-24 of the largest of its own token and head;
 * fp32 sums, one rounding to bf16.  A row sees nothing of the rows behind it,
 * whatever they hold.  A query row that is not finite gives NaN in its row and
 * head, a key or value that is not finite in the rows that see it and the heads
 * that read it (a score of -inf is a weight of 0).
 *
 *   Q, O     bf16 bits [T][Hq][D], row distances ldq, ldo
 *   K, V     bf16 bits [T][Hkv][D], row distances ldk, ldv
 *   sm       the softmax scale, e.g. 1 / sqrt(D); q . k and sm * q . k stay below
 *            2^126 in magnitude
 *   workspace, workspace_bytes  at least
 *            rudder_prompt_attention_workspace_bytes(...) bytes (NULL if 0)
 *   B, T, max_rows >= 0 (0 is a no-op), Hq a multiple of Hkv, D 64 or 128
 * At most two launches.  Results do not depend on anything but the arguments
 * (max_rows, which chooses the kernel, among them).  Sequences that overlap (a
 * row_start that does not ascend) have undefined outputs; no access leaves the
 * buffers.
 * Errors: INVALID_ARG for a null required pointer, negative sizes, Hq or Hkv
 * <= 0, Hq % Hkv != 0, a row distance below its heads' channels or not a
 * multiple of 8, sm not finite or beyond 2^127 in magnitude, a workspace that
 * is too small, Q, K, V, O or workspace not 16-byte aligned; UNSUPPORTED for D
 * other than 64 or 128, Hkv > 4096, B * Hkv > 65535, min(max_rows, T) * Hq >
 * 2^26, or B * Hkv * ceil(max_rows * Hq / Hkv / 128) > 2^21 (give max_rows as
 * it is, not a far larger bound).
 */
rudder_status_t rudder_prompt_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                        const int32_t* row_start, int B, int T, int max_rows,
                                        int Hq, int Hkv, int D, int ldq, int ldk, int ldv, int ldo,
                                        float sm, void* workspace, size_t workspace_bytes,
                                        uint16_t* O, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RUDDER_BLOCK_H */
