// C ABI of librudder: argument validation, error reporting and dispatch to
// the kernel launchers.  Nothing is launched unless every check passes.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <string>

#include "rudder_block_launch.h"
#include "rudder_internal.h"
#include "rudder_operators.h"

namespace {

thread_local std::string g_last_error;

rudder_status_t fail(rudder_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

rudder_status_t fail(rudder_status_t st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

bool misaligned(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u); }

rudder_status_t ok() {
    g_last_error.clear();
    return RUDDER_OK;
}

rudder_status_t from_hip(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(RUDDER_ERR_HIP, "%s: HIP launch failed: %s", what, hipGetErrorString(e));
}

}  // namespace

extern "C" {

size_t rudder_packed_weight_bytes(int K, int N, int codes) {
    if (K <= 0 || N <= 0 || K % 32 || N % 32) return 0;
    if (codes == RUDDER_CODES_INT) return (size_t)N * (size_t)K / 2;
    if (codes == RUDDER_CODES_E2M3 && K % 64 == 0) return (size_t)N * (size_t)K * 3 / 4;
    return 0;
}

size_t rudder_packed_act_bytes(int M, int K, int abits, int codes) {
    if (M < 0 || K <= 0 || K % 32 || (abits != 4 && abits != 8)) return 0;
    const size_t rows = (size_t)((M + 31) / 32) * 32;
    if (codes == RUDDER_CODES_INT) return rows * (size_t)K * (size_t)abits / 8;
    if (codes == RUDDER_CODES_E2M3 && K % 64 == 0)
        return rows * (size_t)K * 3 / 4 * (abits == 8 ? 2 : 1);
    return 0;
}

size_t rudder_quant_act_workspace_bytes(int S) {
    (void)S;
    return rudder::quant_act_workspace_bytes();
}

rudder_status_t rudder_quantize_weights(const uint16_t* W, const float* smooth, int K, int N,
                                        int codes, uint8_t* Wq, float* w_scale,
                                        float* inv_smooth, void* stream) {
    const char* f = "rudder_quantize_weights";
    if (!W || !smooth || !Wq || !w_scale || !inv_smooth)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (K <= 0 || N <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d and N=%d must be positive", f, K, N);
    if (K % 32 || N % 32)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d and N=%d must be multiples of 32", f, K, N);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    if (codes == RUDDER_CODES_E2M3 && K % 64)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 64 for E2M3 codes",
                    f, K);
    if (misaligned(Wq) || misaligned(smooth) || misaligned(w_scale) || misaligned(inv_smooth))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Wq, smooth, w_scale and inv_smooth must be "
                    "16-byte aligned", f);
    if (K > RUDDER_MAX_K)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d", f, K, RUDDER_MAX_K);
    return from_hip(rudder::launch_quantize_weights(W, smooth, K, N, codes, Wq, w_scale,
                                                    inv_smooth, static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_quant_act(const uint16_t* X, const uint8_t* stream_id,
                                 const float* inv_smooth, const float* act_scale,
                                 float* act_scale_out, void* workspace, int M, int K, int S,
                                 int abits, int codes, void* Xq, float* row_scale,
                                 void* stream) {
    const char* f = "rudder_quant_act";
    if (!X || !stream_id || !inv_smooth || !Xq || !row_scale)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (act_scale == nullptr && workspace == nullptr)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: dynamic mode (act_scale NULL) needs a workspace",
                    f);
    if (M < 0 || K <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0 and K=%d > 0", f, M, K);
    if (K % 32) return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 32", f, K);
    if (S < 1 || S > RUDDER_MAX_STREAMS)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: S=%d must be in 1..%d", f, S, RUDDER_MAX_STREAMS);
    if (abits != 4 && abits != 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: abits=%d must be 4 or 8", f, abits);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    if (codes == RUDDER_CODES_E2M3 && K % 64)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 64 for E2M3 codes",
                    f, K);
    if (misaligned(X) || misaligned(inv_smooth) || misaligned(Xq) || misaligned(workspace))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: X, inv_smooth, Xq and workspace must be "
                    "16-byte aligned", f);
    if (K > RUDDER_MAX_K)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d", f, K, RUDDER_MAX_K);
    if (M == 0) return ok();
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (act_scale != nullptr)
        return from_hip(rudder::launch_quant_act_static(X, stream_id, inv_smooth, act_scale, M, K,
                                                        S, abits, codes, Xq, row_scale, st),
                        f);
    return from_hip(rudder::launch_quant_act_dynamic(X, stream_id, inv_smooth, act_scale_out,
                                                     workspace, M, K, S, abits, codes, Xq,
                                                     row_scale, st),
                    f);
}

rudder_status_t rudder_quant_act_noalloc(const uint16_t* X, const uint8_t* stream_id,
                                         const float* inv_smooth, float* act_scale_out, int M,
                                         int K, int S, int abits, int codes, void* Xq,
                                         float* row_scale, void* stream) {
    const char* f = "rudder_quant_act_noalloc";
    if (!X || !stream_id || !inv_smooth || !Xq || !row_scale)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (M < 0 || K <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0 and K=%d > 0", f, M, K);
    if (K % 32) return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 32", f, K);
    if (S < 1 || S > RUDDER_MAX_STREAMS)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: S=%d must be in 1..%d", f, S, RUDDER_MAX_STREAMS);
    if (abits != 4 && abits != 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: abits=%d must be 4 or 8", f, abits);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    if (codes == RUDDER_CODES_E2M3 && K % 64)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 64 for E2M3 codes",
                    f, K);
    if (misaligned(X) || misaligned(inv_smooth) || misaligned(Xq))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: X, inv_smooth and Xq must be 16-byte aligned",
                    f);
    if (K > RUDDER_MAX_K)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d", f, K, RUDDER_MAX_K);
    // the scratch holds the fixed-size dynamic-mode workspace, whatever M and K
    if (rudder::quant_act_workspace_bytes() > rudder::quant_act_noalloc_scratch_bytes())
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: the workspace (%zu bytes) exceeds the scratch "
                    "(%zu bytes)", f, rudder::quant_act_workspace_bytes(),
                    rudder::quant_act_noalloc_scratch_bytes());
    if (M == 0) return ok();
    return from_hip(rudder::launch_quant_act_dynamic_noalloc(X, stream_id, inv_smooth,
                                                             act_scale_out, M, K, S, abits, codes,
                                                             Xq, row_scale,
                                                             static_cast<hipStream_t>(stream)),
                    f);
}

namespace {

// Checks shared by rudder_linear and rudder_linear_gelu_quant (the output
// pointers are checked by the callers).
rudder_status_t check_linear(const char* f, const void* Xq, const float* row_scale,
                             const uint8_t* stream_id, const uint8_t* Wq, const float* w_scale,
                             const float* comp_a, const float* comp_b, int M, int N, int K,
                             int S, int abits, int codes) {
    if (!Xq || !row_scale || !stream_id || !Wq || !w_scale || !comp_a || !comp_b)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (M < 0 || N <= 0 || K <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0, N=%d and K=%d > 0", f, M, N,
                    K);
    if (N % 32) return fail(RUDDER_ERR_INVALID_ARG, "%s: N=%d must be a multiple of 32", f, N);
    if (S < 1 || S > RUDDER_MAX_STREAMS)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: S=%d must be in 1..%d", f, S, RUDDER_MAX_STREAMS);
    if (abits != 4 && abits != 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: abits=%d must be 4 or 8", f, abits);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    if (misaligned(Xq) || misaligned(Wq) || misaligned(w_scale) || misaligned(comp_a) ||
        misaligned(comp_b))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Xq, Wq, w_scale, comp_a and comp_b must be "
                    "16-byte aligned", f);
    if (K % 128)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d is not a multiple of 128", f, K);
    if (K > RUDDER_MAX_K)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d", f, K, RUDDER_MAX_K);
    if (codes == RUDDER_CODES_E2M3 && abits == 8 && K > RUDDER_MAX_K_E2M3_A8)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d for 8-bit E2M3 codes", f, K,
                    RUDDER_MAX_K_E2M3_A8);
    return RUDDER_OK;
}

}  // namespace

rudder_status_t rudder_linear(const void* Xq, const float* row_scale, const uint8_t* stream_id,
                              const uint8_t* Wq, const float* w_scale, const float* comp_a,
                              const float* comp_b, int M, int N, int K, int S, int abits,
                              int codes, uint16_t* Y, int32_t* acc_out, void* stream) {
    const char* f = "rudder_linear";
    if (!Y) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (misaligned(Y) || misaligned(acc_out))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Y and acc_out must be 16-byte aligned", f);
    const rudder_status_t st = check_linear(f, Xq, row_scale, stream_id, Wq, w_scale, comp_a,
                                            comp_b, M, N, K, S, abits, codes);
    if (st != RUDDER_OK) return st;
    if (M == 0) return ok();
    return from_hip(rudder::launch_linear(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b,
                                          M, N, K, S, abits, codes, Y, acc_out,
                                          static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_linear_gelu_quant(const void* Xq, const float* row_scale,
                                         const uint8_t* stream_id, const uint8_t* Wq,
                                         const float* w_scale, const float* comp_a,
                                         const float* comp_b, int M, int N, int K, int S,
                                         int abits, int codes, const float* next_inv_smooth,
                                         const float* next_act_scale, int next_abits,
                                         int next_codes, void* next_Xq, float* next_row_scale,
                                         void* stream) {
    const char* f = "rudder_linear_gelu_quant";
    if (!next_inv_smooth || !next_act_scale || !next_Xq || !next_row_scale)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (next_abits != 4 && next_abits != 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: next_abits=%d must be 4 or 8", f, next_abits);
    if (next_codes != RUDDER_CODES_INT && next_codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, next_codes);
    if (next_codes == RUDDER_CODES_E2M3 && N % 64)
        return fail(RUDDER_ERR_INVALID_ARG,
                    "%s: E2M3 next codes need N a multiple of 64 (N=%d)", f, N);
    if (misaligned(next_inv_smooth) || misaligned(next_Xq))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: next_inv_smooth and next_Xq must be 16-byte "
                    "aligned", f);
    const rudder_status_t st = check_linear(f, Xq, row_scale, stream_id, Wq, w_scale, comp_a,
                                            comp_b, M, N, K, S, abits, codes);
    if (st != RUDDER_OK) return st;
    if ((codes == RUDDER_CODES_E2M3 && abits == 8) ||
        (next_codes == RUDDER_CODES_E2M3 && next_abits == 8))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: 8-bit E2M3 codes are not built for this path",
                    f);
    if (M == 0) return ok();
    const rudder::NextLayerQuant next{next_inv_smooth, next_act_scale,
                                      static_cast<uint8_t*>(next_Xq), next_row_scale, next_abits,
                                      next_codes};
    return from_hip(rudder::launch_linear_gelu_quant(Xq, row_scale, stream_id, Wq, w_scale,
                                                     comp_a, comp_b, M, N, K, S, abits, codes,
                                                     next, static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_gelu_bf16(const uint16_t* in, uint16_t* out, size_t n, void* stream) {
    const char* f = "rudder_gelu_bf16";
    if (n == 0) return ok();
    if (!in || !out) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    return from_hip(rudder::launch_gelu_bf16(in, out, n, static_cast<hipStream_t>(stream)), f);
}

rudder_status_t rudder_dequant_weights(const uint8_t* Wq, const float* w_scale, int K, int N,
                                       int codes, float* out, void* stream) {
    const char* f = "rudder_dequant_weights";
    if (!Wq || !w_scale || !out) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (K <= 0 || N <= 0 || K % 32 || N % 32)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d and N=%d must be positive multiples of 32",
                    f, K, N);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    if (codes == RUDDER_CODES_E2M3 && K % 64)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 64 for E2M3 codes", f,
                    K);
    return from_hip(rudder::launch_dequant_weights(Wq, w_scale, K, N, codes, out,
                                                   static_cast<hipStream_t>(stream)),
                    f);
}

size_t rudder_stream_sq_error_workspace_bytes(void) {
    return rudder::stream_sq_error_workspace_bytes();
}

rudder_status_t rudder_stream_sq_error(const uint16_t* Y, const float* Yref,
                                       const uint8_t* stream_id, int M, int N, int S,
                                       void* workspace, double* sse, void* stream) {
    const char* f = "rudder_stream_sq_error";
    if (!Y || !Yref || !stream_id || !workspace || !sse)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (M < 0 || N <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0 and N=%d > 0", f, M, N);
    if (S < 1 || S > RUDDER_MAX_STREAMS)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: S=%d must be in 1..%d", f, S, RUDDER_MAX_STREAMS);
    return from_hip(rudder::launch_stream_sq_error(Y, Yref, stream_id, M, N, S, workspace, sse,
                                                   static_cast<hipStream_t>(stream)),
                    f);
}

// ---------------------------------------------------------------------------
// Few-row products with group-scaled 4-bit weights.
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxGroupedN = 1 << 24;

rudder_status_t check_grouped(const char* f, int K, int N, int group) {
    if (K <= 0 || N <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d and N=%d must be positive", f, K, N);
    if (group != 32 && group != 64 && group != 128)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: group=%d must be 32, 64 or 128", f, group);
    if (K % group)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of group=%d", f, K,
                    group);
    if (K > RUDDER_MAX_K)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d", f, K, RUDDER_MAX_K);
    if (N > kMaxGroupedN)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: N=%d exceeds %d", f, N, kMaxGroupedN);
    return RUDDER_OK;
}

}  // namespace

size_t rudder_grouped_weight_bytes(int K, int N) {
    if (K <= 0 || N <= 0 || K > RUDDER_MAX_K || N > kMaxGroupedN) return 0;
    return ((size_t)K + 127) / 128 * 128 * (((size_t)N + 15) / 16 * 16) / 2;
}

size_t rudder_grouped_scale_count(int K, int N, int group) {
    if (K <= 0 || N <= 0 || K > RUDDER_MAX_K || N > kMaxGroupedN ||
        (group != 32 && group != 64 && group != 128) || K % group)
        return 0;
    return ((size_t)K + 127) / 128 * (size_t)(128 / group) * (((size_t)N + 15) / 16 * 16);
}

rudder_status_t rudder_quantize_weights_grouped(const uint16_t* W, int K, int N, int group,
                                                uint8_t* Wq, uint16_t* g_scale, void* stream) {
    const char* f = "rudder_quantize_weights_grouped";
    if (!W || !Wq || !g_scale) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    const rudder_status_t st = check_grouped(f, K, N, group);
    if (st != RUDDER_OK) return st;
    if (misaligned(Wq) || misaligned(g_scale))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Wq and g_scale must be 16-byte aligned", f);
    return from_hip(rudder::launch_quantize_weights_grouped(W, K, N, group, Wq, g_scale,
                                                            static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_matvec_w4(const uint16_t* X, const uint8_t* stream_id, const uint8_t* Wq,
                                 const uint16_t* g_scale, const float* comp_a,
                                 const float* comp_b, int M, int N, int K, int group, int S,
                                 uint16_t* Y, void* stream) {
    const char* f = "rudder_matvec_w4";
    if (!X || !Wq || !g_scale || !Y)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if ((comp_a == nullptr) != (comp_b == nullptr) || (comp_a && !stream_id))
        return fail(RUDDER_ERR_INVALID_ARG,
                    "%s: compensation takes comp_a, comp_b and stream_id together", f);
    if (M < 0) return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0", f, M);
    const rudder_status_t st = check_grouped(f, K, N, group);
    if (st != RUDDER_OK) return st;
    if (comp_a && (S < 1 || S > RUDDER_MAX_STREAMS))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: S=%d must be in 1..%d", f, S, RUDDER_MAX_STREAMS);
    if (misaligned(X) || misaligned(Wq) || misaligned(g_scale))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: X, Wq and g_scale must be 16-byte aligned", f);
    if (M > (1 << 19)) return fail(RUDDER_ERR_UNSUPPORTED, "%s: M=%d exceeds %d", f, M, 1 << 19);
    if (M == 0) return ok();
    return from_hip(rudder::launch_matvec_w4(X, stream_id, Wq, g_scale, comp_a, comp_b, M, N, K,
                                             group, Y, static_cast<hipStream_t>(stream)),
                    f);
}

// ---------------------------------------------------------------------------
// Cache and attention (include/rudder_attention.h).
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxSequences = 65535;
constexpr int kMaxCacheHeads = 4096;
constexpr int kMaxKeys = 1 << 30;          // key numbers and the tiles' ends stay below 2^31
constexpr int kMaxAppendRows = 1 << 29;
constexpr float kMaxSoftmaxScale = 0x1p127f;

rudder_status_t check_heads(const char* f, int Hkv, int D) {
    if (Hkv <= 0) return fail(RUDDER_ERR_INVALID_ARG, "%s: Hkv=%d must be positive", f, Hkv);
    if (D != 64 && D != 128)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: D=%d is neither 64 nor 128", f, D);
    if (Hkv > kMaxCacheHeads)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: Hkv=%d exceeds %d", f, Hkv, kMaxCacheHeads);
    return RUDDER_OK;
}

rudder_status_t check_ld(const char* f, const char* name, int ld, int heads, int D) {
    if (ld % 8 || (int64_t)ld < (int64_t)heads * D)
        return fail(RUDDER_ERR_INVALID_ARG,
                    "%s: %s=%d must be a multiple of 8 and at least %d * %d", f, name, ld, heads,
                    D);
    return RUDDER_OK;
}

rudder_status_t check_attention(const char* f, bool cache, bool causal, const void* Q, const void* O,
                                const void* workspace, size_t workspace_bytes, int B, int T,
                                int max_rows, int max_kv, int Hq, int Hkv, int D, int ldq,
                                int ldo, float sm) {
    if (B < 0 || T < 0 || max_rows < 0 || max_kv < 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: B=%d, T=%d, max_rows=%d and max_kv=%d must be "
                    ">= 0", f, B, T, max_rows, max_kv);
    rudder_status_t st = check_heads(f, Hkv, D);
    if (st != RUDDER_OK) return st;
    if (Hq <= 0 || Hq % Hkv)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Hq=%d must be a positive multiple of Hkv=%d", f,
                    Hq, Hkv);
    if ((st = check_ld(f, "ldq", ldq, Hq, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldo", ldo, Hq, D)) != RUDDER_OK) return st;
    // the kernels multiply it by log2(e)
    if (!(sm >= -kMaxSoftmaxScale && sm <= kMaxSoftmaxScale))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: sm must be finite and at most 2^127", f);
    if (misaligned(Q) || misaligned(O) || misaligned(workspace))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Q, O and workspace must be 16-byte aligned", f);
    if (B > kMaxSequences)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d exceeds %d", f, B, kMaxSequences);
    if ((int64_t)B * Hkv > kMaxSequences)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d with Hkv=%d exceeds %d", f, B, Hkv,
                    kMaxSequences);
    if ((int64_t)(max_rows < T ? max_rows : T) * Hq > (1 << 26))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: max_rows=%d with Hq=%d exceeds 2^26 rows", f,
                    max_rows, Hq);
    if (max_kv > kMaxKeys)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: max_kv=%d exceeds %d", f, max_kv, kMaxKeys);
    if (B == 0 || T == 0 || max_rows == 0) return RUDDER_OK;
    size_t need = 0;
    if (!rudder::attention_workspace(cache, causal, B, T, max_rows, max_kv, Hq, Hkv, D, need))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d sequences of max_rows=%d rows exceed a launch",
                    f, B, max_rows);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: these sizes need a workspace of %zu bytes, not "
                    "%zu", f, need, workspace ? workspace_bytes : (size_t)0);
    return RUDDER_OK;
}

}  // namespace

size_t rudder_cache_page_bytes(int Hkv, int D) {
    if (Hkv <= 0 || Hkv > kMaxCacheHeads || (D != 64 && D != 128)) return 0;
    return (size_t)Hkv * 2 * RUDDER_CACHE_PAGE * (size_t)D;
}

rudder_status_t rudder_cache_append(const uint16_t* K, const uint16_t* V,
                                    const int32_t* row_start, const int32_t* pos,
                                    const int32_t* page_table, int B, int T, int max_rows,
                                    int max_pages, int num_pages, int Hkv, int D, int ldk,
                                    int ldv, int8_t* codes, float* scales, void* stream) {
    const char* f = "rudder_cache_append";
    if (!K || !V || !row_start || !pos || !page_table || !codes || !scales)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (B < 0 || T < 0 || max_rows < 0 || max_pages <= 0 || num_pages <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: B=%d, T=%d, max_rows=%d must be >= 0, "
                    "max_pages=%d and num_pages=%d > 0", f, B, T, max_rows, max_pages, num_pages);
    rudder_status_t st = check_heads(f, Hkv, D);
    if (st != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldk", ldk, Hkv, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldv", ldv, Hkv, D)) != RUDDER_OK) return st;
    if (misaligned(K) || misaligned(V) || misaligned(codes) || misaligned(scales))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K, V, codes and scales must be 16-byte aligned",
                    f);
    if (B > kMaxSequences)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d exceeds %d", f, B, kMaxSequences);
    if (max_rows > kMaxAppendRows && T > kMaxAppendRows)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: max_rows=%d exceeds %d", f, max_rows,
                    kMaxAppendRows);
    if (B == 0 || T == 0 || max_rows == 0) return ok();
    return from_hip(rudder::launch_cache_append(K, V, row_start, pos, page_table, B, T,
                                                max_rows < T ? max_rows : T, max_pages, num_pages,
                                                Hkv, D, ldk, ldv, codes, scales,
                                                static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_cache_dequant(const int8_t* codes, const float* scales,
                                     const int32_t* pages, int n, int num_pages, int Hkv, int D,
                                     float* K_out, float* V_out, void* stream) {
    const char* f = "rudder_cache_dequant";
    if (!codes || !scales || !pages || !K_out || !V_out)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (n < 0 || num_pages <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: n=%d must be >= 0 and num_pages=%d > 0", f, n,
                    num_pages);
    const rudder_status_t st = check_heads(f, Hkv, D);
    if (st != RUDDER_OK) return st;
    if (misaligned(codes) || misaligned(K_out) || misaligned(V_out))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: codes, K_out and V_out must be 16-byte aligned",
                    f);
    if (n > (1 << 23))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: n=%d exceeds %d", f, n, 1 << 23);
    if (n == 0) return ok();
    return from_hip(rudder::launch_cache_dequant(codes, scales, pages, n, num_pages, Hkv, D,
                                                 K_out, V_out, static_cast<hipStream_t>(stream)),
                    f);
}

namespace {

bool attention_sizes(int B, int T, int max_rows, int max_kv, int Hq, int Hkv, int D) {
    return B > 0 && T > 0 && max_rows > 0 && max_kv >= 0 && Hkv > 0 && Hkv <= kMaxCacheHeads &&
           Hq > 0 && Hq % Hkv == 0 && (D == 64 || D == 128) && (int64_t)B * Hkv <= kMaxSequences &&
           (int64_t)(max_rows < T ? max_rows : T) * Hq <= (1 << 26) && max_kv <= kMaxKeys;
}

}  // namespace

size_t rudder_attention_workspace_bound(int B, int T, int max_rows, int max_kv, int Hq, int Hkv,
                                        int D) {
    if (!attention_sizes(B, T, max_rows, max_kv, Hq, Hkv, D)) return 0;
    return rudder::attention_workspace_bound(B, T, max_rows, max_kv, Hq, Hkv, D);
}

size_t rudder_attention_workspace_bytes(int B, int T, int max_rows, int max_kv, int Hq, int Hkv,
                                        int D) {
    if (!attention_sizes(B, T, max_rows, max_kv, Hq, Hkv, D)) return 0;
    // one size for both calls, causal or not
    size_t bytes = 0, most = 0;
    for (const int kind : {0, 1, 2})
        if (rudder::attention_workspace(kind > 0, kind > 1, B, T, max_rows, max_kv, Hq, Hkv, D,
                                        bytes))
            most = most > bytes ? most : bytes;
    return most;
}

rudder_status_t rudder_cache_attention(const uint16_t* Q, const int32_t* row_start,
                                       const int32_t* kv_len, const int32_t* page_table,
                                       const int8_t* codes, const float* scales, int B, int T,
                                       int max_rows, int max_kv, int max_pages, int num_pages,
                                       int Hq, int Hkv, int D, int ldq, int ldo, float sm,
                                       int causal, void* workspace, size_t workspace_bytes,
                                       uint16_t* O, void* stream) {
    const char* f = "rudder_cache_attention";
    if (!Q || !row_start || !kv_len || !page_table || !codes || !scales || !O)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (max_pages <= 0 || num_pages <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: max_pages=%d and num_pages=%d must be positive",
                    f, max_pages, num_pages);
    const rudder_status_t st = check_attention(f, true, causal != 0, Q, O, workspace, workspace_bytes, B, T,
                                               max_rows, max_kv, Hq, Hkv, D, ldq, ldo, sm);
    if (st != RUDDER_OK) return st;
    if (misaligned(codes))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned", f);
    if (B == 0 || T == 0 || max_rows == 0) return ok();
    return from_hip(rudder::launch_cache_attention(Q, row_start, kv_len, page_table, codes,
                                                   scales, B, T, max_rows, max_kv, max_pages,
                                                   num_pages, Hq, Hkv, D, ldq, ldo, sm, causal,
                                                   workspace, O,
                                                   static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_cross_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                       const int32_t* row_start, const int32_t* kv_start,
                                       const int32_t* kv_len, int B, int T, int Tkv, int max_rows,
                                       int max_kv, int Hq, int Hkv, int D, int ldq, int ldk,
                                       int ldv, int ldo, float sm, void* workspace,
                                       size_t workspace_bytes, uint16_t* O, void* stream) {
    const char* f = "rudder_cross_attention";
    if (!Q || !K || !V || !row_start || !kv_start || !kv_len || !O)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (Tkv < 0) return fail(RUDDER_ERR_INVALID_ARG, "%s: Tkv=%d must be >= 0", f, Tkv);
    rudder_status_t st = check_attention(f, false, false, Q, O, workspace, workspace_bytes, B, T, max_rows,
                                         max_kv, Hq, Hkv, D, ldq, ldo, sm);
    if (st != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldk", ldk, Hkv, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldv", ldv, Hkv, D)) != RUDDER_OK) return st;
    if (misaligned(K) || misaligned(V))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K and V must be 16-byte aligned", f);
    if (B == 0 || T == 0 || max_rows == 0) return ok();
    return from_hip(rudder::launch_cross_attention(Q, K, V, row_start, kv_start, kv_len, B, T,
                                                   Tkv, max_rows, max_kv, Hq, Hkv, D, ldq, ldk,
                                                   ldv, ldo, sm, workspace, O,
                                                   static_cast<hipStream_t>(stream)),
                    f);
}

// ---------------------------------------------------------------------------
// Norms, rotary positions and prompt attention (include/rudder_block.h).
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxBlockRows = 1 << 25;             // a launch's threads stay below 2^32
constexpr int64_t kMaxElements = (int64_t)1 << 35;

rudder_status_t check_rows(const char* f, int M, int K) {
    if (K > RUDDER_MAX_K)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: K=%d exceeds %d", f, K, RUDDER_MAX_K);
    if (M > kMaxBlockRows || (int64_t)M * K > kMaxElements)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: M=%d rows of K=%d exceed 2^25 rows or 2^35 "
                    "elements", f, M, K);
    return RUDDER_OK;
}

rudder_status_t check_codes(const char* f, int K, int abits, int codes) {
    if (K % 32) return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 32", f, K);
    if (abits != 4 && abits != 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: abits=%d must be 4 or 8", f, abits);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    if (codes == RUDDER_CODES_E2M3 && K % 64)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 64 for E2M3 codes", f,
                    K);
    return RUDDER_OK;
}

// Rows written in the place of rows read: at other distances a row would overwrite others.
rudder_status_t check_place(const char* f, const void* out, int ld_out, const char* name_out,
                            const void* in, int ld_in, const char* name_in) {
    if (!out || out != in || ld_out == ld_in) return RUDDER_OK;
    return fail(RUDDER_ERR_INVALID_ARG, "%s: %s is %s, with rows %d and %d elements apart", f,
                name_out, name_in, ld_out, ld_in);
}

rudder_status_t check_norm(const char* f, const void* X, const void* R, const void* gamma,
                           float eps, int M, int K, int ldx, int ldr, int ldh, const void* H) {
    if (!X || !gamma) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (!R != !H) return fail(RUDDER_ERR_INVALID_ARG, "%s: R and H come together", f);
    if (M < 0 || K <= 0 || K % 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0 and K=%d a positive multiple "
                    "of 8", f, M, K);
    rudder_status_t st = check_ld(f, "ldx", ldx, 1, K);
    if (st == RUDDER_OK && R) st = check_ld(f, "ldr", ldr, 1, K);
    if (st == RUDDER_OK && R) st = check_ld(f, "ldh", ldh, 1, K);
    if (st != RUDDER_OK) return st;
    if (!(eps >= 0.0f && eps <= 3.4028234663852886e38f))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", f);
    if (misaligned(X) || misaligned(R) || misaligned(H) || misaligned(gamma))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: X, R, H and gamma must be 16-byte aligned", f);
    return RUDDER_OK;
}

}  // namespace

rudder_status_t rudder_norm(const uint16_t* X, const uint16_t* R, const float* gamma, float eps,
                            int M, int K, int ldx, int ldr, int ldh, int ldy, uint16_t* H,
                            uint16_t* Y, void* stream) {
    const char* f = "rudder_norm";
    if (!Y) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    rudder_status_t st = check_norm(f, X, R, gamma, eps, M, K, ldx, ldr, ldh, H);
    if (st == RUDDER_OK) st = check_ld(f, "ldy", ldy, 1, K);
    if (st != RUDDER_OK) return st;
    if (misaligned(Y)) return fail(RUDDER_ERR_INVALID_ARG, "%s: Y must be 16-byte aligned", f);
    if (Y == H) return fail(RUDDER_ERR_INVALID_ARG, "%s: Y and H are one buffer", f);
    if ((st = check_rows(f, M, K)) != RUDDER_OK) return st;
    if (M == 0) return ok();
    if (M > 1) {
        st = check_place(f, H, ldh, "H", X, ldx, "X");
        if (st == RUDDER_OK) st = check_place(f, H, ldh, "H", R, ldr, "R");
        if (st == RUDDER_OK) st = check_place(f, Y, ldy, "Y", X, ldx, "X");
        if (st == RUDDER_OK) st = check_place(f, Y, ldy, "Y", R, ldr, "R");
        if (st != RUDDER_OK) return st;
    }
    return from_hip(rudder::launch_norm(X, R, nullptr, gamma, nullptr, nullptr, eps, M, K, ldx,
                                        ldr, ldh, ldy, 0, 0, H, Y, nullptr, nullptr,
                                        static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_norm_quant(const uint16_t* X, const uint16_t* R, const uint8_t* stream_id,
                                  const float* gamma, const float* inv_smooth,
                                  const float* act_scale, float eps, int M, int K, int S,
                                  int abits, int codes, int ldx, int ldr, int ldh, uint16_t* H,
                                  void* Xq, float* row_scale, void* stream) {
    const char* f = "rudder_norm_quant";
    if (!inv_smooth || !Xq || !row_scale)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (act_scale && !stream_id)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: act_scale needs stream_id", f);
    rudder_status_t st = check_norm(f, X, R, gamma, eps, M, K, ldx, ldr, ldh, H);
    if (st == RUDDER_OK) st = check_codes(f, K, abits, codes);
    if (st != RUDDER_OK) return st;
    if (act_scale && (S < 1 || S > RUDDER_MAX_STREAMS))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: S=%d must be in 1..%d", f, S, RUDDER_MAX_STREAMS);
    if (misaligned(inv_smooth) || misaligned(Xq))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: inv_smooth and Xq must be 16-byte aligned", f);
    if (codes == RUDDER_CODES_E2M3 && abits == 8)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: 8-bit E2M3 codes are not built for this path", f);
    if ((st = check_rows(f, M, K)) != RUDDER_OK) return st;
    if (M == 0) return ok();
    if (M > 1) {
        st = check_place(f, H, ldh, "H", X, ldx, "X");
        if (st == RUDDER_OK) st = check_place(f, H, ldh, "H", R, ldr, "R");
        if (st != RUDDER_OK) return st;
    }
    return from_hip(rudder::launch_norm(X, R, stream_id, gamma, inv_smooth, act_scale, eps, M, K,
                                        ldx, ldr, ldh, 0, abits, codes, H, nullptr, Xq, row_scale,
                                        static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_dequant_act(const void* Xq, const float* row_scale, int M, int K, int abits,
                                   int codes, float* out, void* stream) {
    const char* f = "rudder_dequant_act";
    if (!Xq || !row_scale || !out)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (M < 0 || K <= 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: M=%d must be >= 0 and K=%d > 0", f, M, K);
    rudder_status_t st = check_codes(f, K, abits, codes);
    if (st != RUDDER_OK) return st;
    if (misaligned(Xq) || misaligned(out))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Xq and out must be 16-byte aligned", f);
    if ((st = check_rows(f, M, K)) != RUDDER_OK) return st;
    if (M == 0) return ok();
    return from_hip(rudder::launch_dequant_act(static_cast<const uint8_t*>(Xq), row_scale, M, K,
                                               abits, codes, out,
                                               static_cast<hipStream_t>(stream)),
                    f);
}

rudder_status_t rudder_rotary_frequencies(int rotary_dim, double base, int scaling, double factor,
                                          double trained, double low, double high, double* freq) {
    const char* f = "rudder_rotary_frequencies";
    if (!freq) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (rotary_dim <= 0 || rotary_dim % 2)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: rotary_dim=%d must be positive and even", f,
                    rotary_dim);
    const double most = 1.7976931348623157e308;
    if (!(base > 0 && base <= most))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: base must be positive and finite", f);
    if (scaling < RUDDER_ROTARY_PLAIN || scaling > RUDDER_ROTARY_PARTS)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown scaling %d", f, scaling);
    if (scaling != RUDDER_ROTARY_PLAIN && !(factor >= 1 && factor <= most))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: factor must be finite and at least 1", f);
    const bool parts = scaling == RUDDER_ROTARY_PARTS;
    if (parts && !(trained > 0 && trained <= most && low >= 0 && high > low && high <= most))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: by parts, trained must be positive, low >= 0, "
                    "high above low, all finite", f);
    if (rotary_dim > (1 << 16))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: rotary_dim=%d exceeds %d", f, rotary_dim, 1 << 16);
    const int n = rotary_dim / 2;
    if (scaling == RUDDER_ROTARY_BASE && n > 1) base *= pow(factor, (double)n / (n - 1));
    // from the first pair, of 1, on they rise or fall: the last one's is the largest or the smallest
    if (!(base <= most && pow(base, -(double)(n - 1) / n) <= most))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: base, or what factor raises it to, is so far from 1 "
                    "that it or a frequency passes 64 bits", f);
    for (int i = 0; i < n; ++i) {
        double x = pow(base, -(double)i / n);
        if (scaling == RUDDER_ROTARY_LINEAR) x /= factor;
        if (parts) {
            const double turns = trained * x / 6.283185307179586;
            const double keep = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
            x = x / factor * (1 - keep) + x * keep;
        }
        freq[i] = x;
    }
    return ok();
}

rudder_status_t rudder_rotary(const uint16_t* Q, const uint16_t* K, const int32_t* row_start,
                              const int32_t* pos, const double* freq, float magnitude, int B,
                              int T, int max_rows, int Hq, int Hkv, int D, int rotary_dim,
                              int layout, int ldq, int ldk, int ldqo, int ldko, uint16_t* Qo,
                              uint16_t* Ko, void* stream) {
    const char* f = "rudder_rotary";
    if (!Q || !row_start || !freq || !Qo || (Hkv != 0 && (!K || !Ko)))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (B < 0 || T < 0 || max_rows < 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: B=%d, T=%d and max_rows=%d must be >= 0", f, B, T,
                    max_rows);
    if (Hq <= 0 || Hkv < 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Hq=%d must be positive and Hkv=%d >= 0", f, Hq,
                    Hkv);
    if (layout != RUDDER_ROTARY_HALF && layout != RUDDER_ROTARY_PAIRS)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown layout %d", f, layout);
    rudder_status_t st = check_heads(f, Hq, D);
    if (st == RUDDER_OK && Hkv) st = check_heads(f, Hkv, D);
    if (st != RUDDER_OK) return st;
    if (rotary_dim <= 0 || rotary_dim > D || rotary_dim % 16)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: rotary_dim=%d must be a positive multiple of 16 "
                    "up to D=%d", f, rotary_dim, D);
    if ((st = check_ld(f, "ldq", ldq, Hq, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldqo", ldqo, Hq, D)) != RUDDER_OK) return st;
    if (Hkv && (st = check_ld(f, "ldk", ldk, Hkv, D)) != RUDDER_OK) return st;
    if (Hkv && (st = check_ld(f, "ldko", ldko, Hkv, D)) != RUDDER_OK) return st;
    if (!(fabsf(magnitude) <= 3.4028234663852886e38f))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: magnitude must be finite", f);
    if (misaligned(Q) || misaligned(Qo) || (Hkv && (misaligned(K) || misaligned(Ko))))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Q, K, Qo and Ko must be 16-byte aligned", f);
    if (B > kMaxSequences)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d exceeds %d", f, B, kMaxSequences);
    if ((max_rows < T ? max_rows : T) > kMaxBlockRows)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: max_rows=%d exceeds %d", f, max_rows,
                    kMaxBlockRows);
    if (B == 0 || T == 0 || max_rows == 0) return ok();
    if (T > 1) {
        st = check_place(f, Qo, ldqo, "Qo", Q, ldq, "Q");
        if (st == RUDDER_OK && Hkv) st = check_place(f, Ko, ldko, "Ko", K, ldk, "K");
        if (st != RUDDER_OK) return st;
    }
    return from_hip(rudder::launch_rotary(Q, K, row_start, pos, freq, magnitude, B, T, max_rows,
                                          Hq, Hkv, D, rotary_dim, layout, ldq, ldk, ldqo, ldko, Qo,
                                          Ko, static_cast<hipStream_t>(stream)),
                    f);
}

size_t rudder_prompt_attention_workspace_bytes(int B, int T, int max_rows, int Hq, int Hkv,
                                               int D) {
    size_t bytes = 0;
    if (!attention_sizes(B, T, max_rows, 0, Hq, Hkv, D) ||
        !rudder::prompt_attention_workspace(B, T, max_rows, Hq, Hkv, D, bytes))
        return 0;
    return bytes;
}

rudder_status_t rudder_prompt_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                        const int32_t* row_start, int B, int T, int max_rows,
                                        int Hq, int Hkv, int D, int ldq, int ldk, int ldv, int ldo,
                                        float sm, void* workspace, size_t workspace_bytes,
                                        uint16_t* O, void* stream) {
    const char* f = "rudder_prompt_attention";
    if (!Q || !K || !V || !row_start || !O)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (B < 0 || T < 0 || max_rows < 0)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: B=%d, T=%d and max_rows=%d must be >= 0", f, B, T,
                    max_rows);
    rudder_status_t st = check_heads(f, Hkv, D);
    if (st != RUDDER_OK) return st;
    if (Hq <= 0 || Hq % Hkv)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Hq=%d must be a positive multiple of Hkv=%d", f,
                    Hq, Hkv);
    if ((st = check_ld(f, "ldq", ldq, Hq, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldk", ldk, Hkv, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldv", ldv, Hkv, D)) != RUDDER_OK) return st;
    if ((st = check_ld(f, "ldo", ldo, Hq, D)) != RUDDER_OK) return st;
    if (!(sm >= -kMaxSoftmaxScale && sm <= kMaxSoftmaxScale))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: sm must be finite and at most 2^127", f);
    if (misaligned(Q) || misaligned(K) || misaligned(V) || misaligned(O) || misaligned(workspace))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Q, K, V, O and workspace must be 16-byte aligned",
                    f);
    if ((int64_t)B * Hkv > kMaxSequences)
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d with Hkv=%d exceeds %d", f, B, Hkv,
                    kMaxSequences);
    if ((int64_t)(max_rows < T ? max_rows : T) * Hq > (1 << 26))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: max_rows=%d with Hq=%d exceeds 2^26 rows", f,
                    max_rows, Hq);
    if (B == 0 || T == 0 || max_rows == 0) return ok();
    size_t need = 0;
    if (!rudder::prompt_attention_workspace(B, T, max_rows, Hq, Hkv, D, need))
        return fail(RUDDER_ERR_UNSUPPORTED, "%s: B=%d sequences of max_rows=%d rows exceed a launch",
                    f, B, max_rows);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: these sizes need a workspace of %zu bytes, not "
                    "%zu", f, need, workspace ? workspace_bytes : (size_t)0);
    return from_hip(rudder::launch_prompt_attention(Q, K, V, row_start, B, T, max_rows, Hq, Hkv, D,
                                                    ldq, ldk, ldv, ldo, sm, workspace, O,
                                                    static_cast<hipStream_t>(stream)),
                    f);
}

size_t rudder_mfma_ceiling_sink_bytes(void) { return rudder::mfma_ceiling_sink_bytes(); }

double rudder_mfma_ceiling_ops(int iters, int codes) {
    return iters > 0 ? rudder::mfma_ceiling_ops(iters, codes) : 0.0;
}

rudder_status_t rudder_mfma_ceiling(const uint8_t* Xq, const uint8_t* Wq, int M, int N, int K,
                                    int abits, int codes, int iters, int32_t* sink,
                                    void* stream) {
    return rudder_mfma_ceiling_shape(Xq, Wq, M, N, K, abits, codes, iters, RUDDER_CEILING_OWN,
                                     sink, stream);
}

rudder_status_t rudder_mfma_ceiling_shape(const uint8_t* Xq, const uint8_t* Wq, int M, int N,
                                          int K, int abits, int codes, int iters, int shape,
                                          int32_t* sink, void* stream) {
    const char* f = "rudder_mfma_ceiling";
    if (shape != RUDDER_CEILING_OWN && shape != RUDDER_CEILING_I8_16X16X64)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown instruction shape %d", f, shape);
    if (shape == RUDDER_CEILING_I8_16X16X64 && codes != RUDDER_CODES_INT)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: the 16x16x64 int8 shape takes int codes", f);
    if (!Xq || !Wq || !sink) return fail(RUDDER_ERR_INVALID_ARG, "%s: null pointer argument", f);
    if (misaligned(Xq) || misaligned(Wq) || misaligned(sink))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: Xq, Wq and sink must be 16-byte aligned", f);
    if (abits != 4 && abits != 8)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: abits=%d must be 4 or 8", f, abits);
    if (codes != RUDDER_CODES_INT && codes != RUDDER_CODES_E2M3)
        return fail(RUDDER_ERR_INVALID_ARG, "%s: unknown code container %d", f, codes);
    const int kmul = codes == RUDDER_CODES_E2M3 ? 64 : 32;
    if (M <= 0 || N <= 0 || K <= 0 || N % 32 || K % kmul)
        return fail(RUDDER_ERR_INVALID_ARG,
                    "%s: M=%d, N=%d, K=%d: need M > 0, N a multiple of 32, K a multiple of %d", f,
                    M, N, K, kmul);
    if (iters <= 0 || iters > (1 << 24))
        return fail(RUDDER_ERR_INVALID_ARG, "%s: iters=%d must be in 1..2^24", f, iters);
    return from_hip(rudder::launch_mfma_ceiling(Xq, Wq, M, N, K, abits, codes, iters, sink,
                                                static_cast<hipStream_t>(stream), shape),
                    f);
}

const char* rudder_status_string(rudder_status_t status) {
    switch (status) {
        case RUDDER_OK: return "RUDDER_OK";
        case RUDDER_ERR_INVALID_ARG: return "RUDDER_ERR_INVALID_ARG";
        case RUDDER_ERR_UNSUPPORTED: return "RUDDER_ERR_UNSUPPORTED";
        case RUDDER_ERR_HIP: return "RUDDER_ERR_HIP";
    }
    return "RUDDER_ERR_UNKNOWN";
}

const char* rudder_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
