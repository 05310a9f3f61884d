// The paged 8-bit cache of keys and values: the quantizer that appends the
// rows of a QKV projection to it, and its inverse.
//
// A page holds 64 tokens.  codes[page][head][K|V] is 64 * D bytes: K as
// [token][channel], V as [channel][token] -- each the order in which a lane of
// the attention's matrix products wants consecutive bytes -- and
// scales[page][head][K|V] is one fp32 step size.
//
// Appending keeps one scale per block: a = max |x| of the block's new rows,
// s' = max(s, fl32(a / 127)), and when that grows the block's older codes are
// rescaled, c' = rne(c * fl32(s / s')).  One workgroup owns one (page, head,
// K|V), so that maximum, rescaling and writing need no other synchronization.
// Both kernels move bytes and compute next to nothing.
#include "rudder_internal.h"

namespace rudder {
namespace {

constexpr int kPage = RUDDER_CACHE_PAGE;
constexpr int kThreads = 256;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    int c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = (int)__builtin_rintf((float)(int8_t)(w >> (8 * i)) * ratio);
    return byte_word(c);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
cache_append_kernel(const uint16_t* __restrict__ Kx, const uint16_t* __restrict__ Vx,
                    const int32_t* __restrict__ row_start, const int32_t* __restrict__ pos,
                    const int32_t* __restrict__ page_table, int T, int max_rows, int max_pages,
                    int num_pages, int Hkv, size_t ldk, size_t ldv, int8_t* __restrict__ codes,
                    float* __restrict__ scales) {
    constexpr int kChunks = D / 8;                 // threads a row: 8 values each
    constexpr int kRows = kThreads / kChunks;      // rows a pass
    constexpr int kPasses = kPage / kRows;
    constexpr int kStride = kPage + 16;            // bytes of a V row in LDS
    __shared__ __align__(16) uint8_t tile[D * kStride];
    __shared__ float red[kThreads / 64];

    const int b = blockIdx.z, h = blockIdx.y >> 1, is_v = blockIdx.y & 1, tid = threadIdx.x;
    const int r0 = min(max(row_start[b], 0), T);
    const int n = min(min(max(row_start[b + 1], r0), T) - r0, max_rows);
    const int p0 = pos[b];
    if (n <= 0 || p0 < 0) return;
    // signed 64-bit: p0 may lie near 2^31
    const int64_t no = p0 / kPage + (int64_t)blockIdx.x;
    if (no >= max_pages || no * kPage >= (int64_t)p0 + n) return;
    const int page = page_table[(size_t)b * max_pages + no];
    if (page < 0 || page >= num_pages) return;
    const int lo = (int)max((int64_t)p0 - no * kPage, (int64_t)0);           // first new slot
    const int hi = (int)min((int64_t)p0 + n - no * kPage, (int64_t)kPage);   // behind the last
    const int64_t first = no * kPage - p0;                                   // row of slot 0

    const uint16_t* src = (is_v ? Vx : Kx) + (size_t)h * D;
    const size_t ld = is_v ? ldv : ldk;
    const size_t block = ((size_t)page * Hkv + h) * 2 + is_v;
    uint8_t* dst = reinterpret_cast<uint8_t*>(codes) + block * (size_t)(kPage * D);
    const int chunk = tid % kChunks;

    uint4 x[kPasses];
    float amax = 0.0f;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int slot = p * kRows + tid / kChunks;
        x[p] = make_uint4(0, 0, 0, 0);
        if (slot >= lo && slot < hi)
            x[p] = *reinterpret_cast<const uint4*>(src + (size_t)(r0 + first + slot) * ld +
                                                   chunk * 8);
        const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)),
                                     fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
    }
    amax = wave_max(amax);
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) amax = fmaxf(amax, red[i]);
    const float had = lo > 0 ? scales[block] : 0.0f;
    const float s = fmaxf(had, (float)((double)amax / 127.0));
    const float inv = step_reciprocal(s);
    const bool grown = lo > 0 && s > had;
    const float ratio = grown ? (float)((double)had / (double)s) : 1.0f;
    __syncthreads();                               // every thread has read scales[block]
    if (tid == 0) scales[block] = s;

    const bool whole = lo == 0 && hi == kPage;
    if (!is_v) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int slot = p * kRows + tid / kChunks;
            uint2* out = reinterpret_cast<uint2*>(dst + (size_t)slot * D + chunk * 8);
            if (slot >= lo && slot < hi) {
                const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
                int c[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[2 * i] = quantize_clamped(__uint_as_float(w[i] << 16) * inv, 127.0f);
                    c[2 * i + 1] =
                        quantize_clamped(__uint_as_float(w[i] & 0xFFFF0000u) * inv, 127.0f);
                }
                *out = make_uint2(byte_word(c), byte_word(c + 4));
            } else if (slot < lo && grown) {
                const uint2 o = *out;
                *out = make_uint2(rescale4(o.x, ratio), rescale4(o.y, ratio));
            }
        }
        return;
    }
    // V: through LDS, transposed.  A partly new page is read, changed and written whole.
    constexpr int kUnits = D * kPage / 16;         // 16-byte pieces of the page's V half
    if (!whole) {
        for (int u = tid; u < kUnits; u += kThreads)
            *reinterpret_cast<uint4*>(tile + (u / 4) * kStride + (u % 4) * 16) =
                *reinterpret_cast<const uint4*>(dst + (size_t)u * 16);
        __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int slot = p * kRows + tid / kChunks;
        uint8_t* out = tile + (size_t)(chunk * 8) * kStride + slot;
        if (slot >= lo && slot < hi) {
            const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                out[(2 * i) * kStride] = (uint8_t)quantize_clamped(
                    __uint_as_float(w[i] << 16) * inv, 127.0f);
                out[(2 * i + 1) * kStride] = (uint8_t)quantize_clamped(
                    __uint_as_float(w[i] & 0xFFFF0000u) * inv, 127.0f);
            }
        } else if (slot < lo && grown) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                out[i * kStride] =
                    (uint8_t)(int)__builtin_rintf((float)(int8_t)out[i * kStride] * ratio);
        }
    }
    __syncthreads();
    for (int u = tid; u < kUnits; u += kThreads)
        *reinterpret_cast<uint4*>(dst + (size_t)u * 16) =
            *reinterpret_cast<const uint4*>(tile + (u / 4) * kStride + (u % 4) * 16);
}

// Values of whole pages: out[i][head][token][channel] = fl32(code * scale), and
// zeros for a page number outside the pool.
template <int D>
__global__ void __launch_bounds__(kThreads)
cache_dequant_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                     const int32_t* __restrict__ pages, int num_pages, int Hkv,
                     float* __restrict__ Kout, float* __restrict__ Vout) {
    constexpr int kStride = kPage + 4;
    __shared__ __align__(16) uint8_t tile[D * kStride];
    const int i = blockIdx.x, h = blockIdx.y >> 1, is_v = blockIdx.y & 1, tid = threadIdx.x;
    const int page = pages[i];
    const bool good = page >= 0 && page < num_pages;
    const size_t block = ((size_t)(good ? page : 0) * Hkv + h) * 2 + is_v;
    const uint32_t* src =
        reinterpret_cast<const uint32_t*>(codes + block * (size_t)(kPage * D));
    const float s = good ? scales[block] : 0.0f;
    float* out = (is_v ? Vout : Kout) + ((size_t)i * Hkv + h) * (size_t)(kPage * D);
    constexpr int kWords = kPage * D / 4;
    if (is_v) {
        for (int u = tid; u < kWords; u += kThreads)
            *reinterpret_cast<uint32_t*>(tile + (u / 16) * kStride + (u % 16) * 4) =
                good ? src[u] : 0u;
        __syncthreads();
    }
    for (int u = tid; u < kWords; u += kThreads) {
        uint32_t w;
        if (is_v) {
            const uint8_t* t = tile + (size_t)((u % (D / 4)) * 4) * kStride + u / (D / 4);
            w = t[0] | (uint32_t)t[kStride] << 8 | (uint32_t)t[2 * kStride] << 16 |
                (uint32_t)t[3 * kStride] << 24;
        } else {
            w = good ? src[u] : 0u;
        }
        float4 v;
        v.x = (float)(int8_t)w * s;
        v.y = (float)(int8_t)(w >> 8) * s;
        v.z = (float)(int8_t)(w >> 16) * s;
        v.w = (float)(int8_t)(w >> 24) * s;
        reinterpret_cast<float4*>(out)[u] = v;
    }
}

}  // namespace

hipError_t launch_cache_append(const uint16_t* K, const uint16_t* V, const int32_t* row_start,
                               const int32_t* pos, const int32_t* page_table, int B, int T,
                               int max_rows, int max_pages, int num_pages, int Hkv, int D,
                               int ldk, int ldv, int8_t* codes, float* scales,
                               hipStream_t stream) {
    // rows p0 .. p0 + max_rows - 1 touch at most this many pages, whatever p0
    const int pages = (int)(((int64_t)max_rows + 2 * kPage - 2) / kPage);
    const dim3 grid(pages, 2 * Hkv, B);
    if (D == 64)
        cache_append_kernel<64><<<grid, kThreads, 0, stream>>>(
            K, V, row_start, pos, page_table, T, max_rows, max_pages, num_pages, Hkv, ldk, ldv,
            codes, scales);
    else
        cache_append_kernel<128><<<grid, kThreads, 0, stream>>>(
            K, V, row_start, pos, page_table, T, max_rows, max_pages, num_pages, Hkv, ldk, ldv,
            codes, scales);
    return hipGetLastError();
}

hipError_t launch_cache_dequant(const int8_t* codes, const float* scales, const int32_t* pages,
                                int n, int num_pages, int Hkv, int D, float* Kout, float* Vout,
                                hipStream_t stream) {
    const dim3 grid(n, 2 * Hkv);
    if (D == 64)
        cache_dequant_kernel<64><<<grid, kThreads, 0, stream>>>(codes, scales, pages, num_pages,
                                                                Hkv, Kout, Vout);
    else
        cache_dequant_kernel<128><<<grid, kThreads, 0, stream>>>(codes, scales, pages, num_pages,
                                                                 Hkv, Kout, Vout);
    return hipGetLastError();
}

}  // namespace rudder
