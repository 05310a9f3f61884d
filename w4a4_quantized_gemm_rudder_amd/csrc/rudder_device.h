// Device helpers of the operators around and between the linears.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rudder {

// Two numbers in a word, each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    union { bf16x2_t v; uint32_t u; } r;
    r.v = (bf16x2_t){(__bf16)a, (__bf16)b};
    return r.u;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    union { f16x2_t v; uint32_t u; } r;
    r.v = (f16x2_t){(_Float16)a, (_Float16)b};
    return r.u;
}

// The two bf16 numbers of a word.
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a / b of wave-uniform values, back in a scalar register (the division runs on the vector units)
__device__ __forceinline__ int quotient(int a, int b) {
    return __builtin_amdgcn_readfirstlane(a / b);
}

// Orders a wave's LDS accesses of different lanes (the hardware keeps their order; this keeps the
// compiler's).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A store past the caches, for what is not read again soon.
__device__ __forceinline__ void stream16(void* to, uint4 x) {
    typedef unsigned v4u __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(v4u{x.x, x.y, x.z, x.w}, static_cast<v4u*>(to));
}

}  // namespace rudder
