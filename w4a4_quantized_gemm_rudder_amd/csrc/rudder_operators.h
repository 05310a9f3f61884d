// Launchers of the few-row products, the cache and attention: what the C entry
// points call after their checks.
#pragma once

#include "rudder_attention.h"
#include "rudder_internal.h"

namespace rudder {

hipError_t launch_quantize_weights_grouped(const uint16_t* W, int K, int N, int group,
                                           uint8_t* Wq, uint16_t* g_scale, hipStream_t stream);
hipError_t launch_matvec_w4(const uint16_t* X, const uint8_t* sid, const uint8_t* Wq,
                            const uint16_t* g_scale, const float* comp_a, const float* comp_b,
                            int M, int N, int K, int group, uint16_t* Y, hipStream_t stream);

// Cache and attention (include/rudder_attention.h).
hipError_t launch_cache_append(const uint16_t* K, const uint16_t* V, const int32_t* row_start,
                               const int32_t* pos, const int32_t* page_table, int B, int T,
                               int max_rows, int max_pages, int num_pages, int Hkv, int D,
                               int ldk, int ldv, int8_t* codes, float* scales,
                               hipStream_t stream);
hipError_t launch_cache_dequant(const int8_t* codes, const float* scales, const int32_t* pages,
                                int n, int num_pages, int Hkv, int D, float* Kout, float* Vout,
                                hipStream_t stream);
// Workspace of a call over the cache or to bf16 states; false for more work than a launch takes.
bool attention_workspace(bool cache, bool causal, int B, int T, int max_rows, int max_kv, int Hq,
                         int Hkv, int D, size_t& bytes);
// At least the workspace of every call of these sizes or smaller ones.
size_t attention_workspace_bound(int B, int T, int max_rows, int max_kv, int Hq, int Hkv, int D);
hipError_t launch_cache_attention(const uint16_t* Q, const int32_t* row_start,
                                  const int32_t* kv_len, const int32_t* page_table,
                                  const int8_t* codes, const float* scales, int B, int T,
                                  int max_rows, int max_kv, int max_pages, int num_pages, int Hq,
                                  int Hkv, int D, int ldq, int ldo, float sm, int causal,
                                  void* workspace, uint16_t* O, hipStream_t stream);
hipError_t launch_cross_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                  const int32_t* row_start, const int32_t* kv_start,
                                  const int32_t* kv_len, int B, int T, int Tkv, int max_rows,
                                  int max_kv, int Hq, int Hkv, int D, int ldq, int ldk, int ldv,
                                  int ldo, float sm, void* workspace, uint16_t* O,
                                  hipStream_t stream);

}  // namespace rudder
