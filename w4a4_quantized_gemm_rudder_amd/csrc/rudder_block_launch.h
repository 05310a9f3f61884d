// Launchers of the norms, rotary positions and prompt attention: what the C
// entry points call after their checks.
#pragma once

#include "rudder_block.h"
#include "rudder_internal.h"

namespace rudder {

// Y: bf16 rows; without it codes.  R (with H) and table may be null.
hipError_t launch_norm(const uint16_t* X, const uint16_t* R, const uint8_t* sid,
                       const float* gamma, const float* inv_smooth, const float* table, float eps,
                       int M, int K, int ldx, int ldr, int ldh, int ldy, int abits, int codes,
                       uint16_t* H, uint16_t* Y, void* Xq, float* row_scale, hipStream_t stream);
hipError_t launch_dequant_act(const uint8_t* Xq, const float* row_scale, int M, int K, int abits,
                              int codes, float* out, hipStream_t stream);

hipError_t launch_rotary(const uint16_t* Q, const uint16_t* K, const int32_t* row_start,
                         const int32_t* pos, const double* freq, float magnitude, int B, int T,
                         int max_rows, int Hq, int Hkv, int D, int rotary_dim, int layout, int ldq,
                         int ldk, int ldqo, int ldko, uint16_t* Qo, uint16_t* Ko,
                         hipStream_t stream);

// False for more work than a launch takes.
bool prompt_attention_workspace(int B, int T, int max_rows, int Hq, int Hkv, int D, size_t& bytes);
hipError_t launch_prompt_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                   const int32_t* row_start, int B, int T, int max_rows, int Hq,
                                   int Hkv, int D, int ldq, int ldk, int ldv, int ldo, float sm,
                                   void* workspace, uint16_t* O, hipStream_t stream);

}  // namespace rudder
