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
#include "rudder_operators.h"

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

// Eight bf16 values to codes.
__device__ __forceinline__ void quantize8(uint4 x, float inv, int (&c)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[2 * i] = quantize_clamped(__uint_as_float(w[i] << 16) * inv, 127.0f);
        c[2 * i + 1] = quantize_clamped(__uint_as_float(w[i] & 0xFFFF0000u) * inv, 127.0f);
    }
}

// A thread holds eight channels of kSlots consecutive tokens.  K rows are written as they are.  V
// is transposed: of a whole page through LDS, kSlots codes at a time; a few new tokens that leave
// the scale as it was are written as single bytes; else the page is read, changed and written.
// Measured: 2 x 4192 tokens of 16 heads and 128 channels 31 us (69 MB read, 34 MB written: 3.3
// TB/s, two thirds of a large copy's rate, the waves waiting for memory half of the time); 48
// single tokens of 8 heads 5.4 us, and 18 where every V page was read and written.
template <int D>
__global__ void __launch_bounds__(kThreads)
cache_append_kernel(const uint16_t* __restrict__ Kx, const uint16_t* __restrict__ Vx,
                    const int32_t* __restrict__ row_start, const int32_t* __restrict__ pos,
                    const int32_t* __restrict__ page_table, int T, int max_rows, int max_pages,
                    int num_pages, int Hkv, size_t ldk, size_t ldv, int8_t* __restrict__ codes,
                    float* __restrict__ scales) {
    constexpr int kChunks = D / 8;                 // threads a row
    constexpr int kSlots = kPage * kChunks / kThreads;     // 4 (D = 128) or 2
    constexpr int kStride = kPage + 4;             // bytes of a V row in LDS
    constexpr int kFew = 8;                        // new tokens written byte by byte
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
    const int chunk = tid % kChunks, slot0 = tid / kChunks * kSlots;
    const float had = lo > 0 ? scales[block] : 0.0f;

    uint4 x[kSlots];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int slot = slot0 + i;
        x[i] = make_uint4(0, 0, 0, 0);
        if (slot >= lo && slot < hi)
            x[i] = *reinterpret_cast<const uint4*>(src + (size_t)(r0 + first + slot) * ld +
                                                   chunk * 8);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                     fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
    }
    amax = wave_max(amax);
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();                               // every thread has read scales[block], too
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) amax = fmaxf(amax, red[i]);
    const float s = fmaxf(had, (float)((double)amax / 127.0));
    const float inv = step_reciprocal(s);
    const bool grown = lo > 0 && s > had;
    const float ratio = grown ? (float)((double)had / (double)s) : 1.0f;
    if (tid == 0) scales[block] = s;

    if (!is_v) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int slot = slot0 + i;
            uint2* out = reinterpret_cast<uint2*>(dst + (size_t)slot * D + chunk * 8);
            if (slot >= lo && slot < hi) {
                int c[8];
                quantize8(x[i], inv, c);
                *out = make_uint2(byte_word(c), byte_word(c + 4));
            } else if (slot < lo && grown) {
                const uint2 o = *out;
                *out = make_uint2(rescale4(o.x, ratio), rescale4(o.y, ratio));
            }
        }
        return;
    }
    if (!grown && hi - lo <= kFew) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int slot = slot0 + i;
            if (slot < lo || slot >= hi) continue;
            int c[8];
            quantize8(x[i], inv, c);
            uint8_t* out = dst + chunk * 8 * kPage + slot;
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j * kPage] = (uint8_t)c[j];
        }
        return;
    }
    const bool whole = lo == 0 && hi == kPage;
    constexpr int kWords = D * kPage / 4;
    if (!whole) {
        for (int u = tid; u < kWords; u += kThreads)
            *reinterpret_cast<uint32_t*>(tile + (u / 16) * kStride + (u % 16) * 4) =
                reinterpret_cast<const uint32_t*>(dst)[u];
        __syncthreads();
    }
    {
        int c[kSlots][8];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) quantize8(x[i], inv, c[i]);
        uint8_t* out = tile + chunk * 8 * kStride + slot0;
        if (slot0 >= lo && slot0 + kSlots <= hi) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < kSlots; ++i) w |= ((uint32_t)c[i][j] & 0xFFu) << (8 * i);
                if constexpr (kSlots == 4)
                    *reinterpret_cast<uint32_t*>(out + j * kStride) = w;
                else
                    *reinterpret_cast<uint16_t*>(out + j * kStride) = (uint16_t)w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int slot = slot0 + i;
                if (slot >= lo && slot < hi) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) out[j * kStride + i] = (uint8_t)c[i][j];
                } else if (slot < lo && grown) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        out[j * kStride + i] = (uint8_t)(int)__builtin_rintf(
                            (float)(int8_t)out[j * kStride + i] * ratio);
                }
            }
        }
    }
    __syncthreads();
    for (int u = tid; u < kWords / 2; u += kThreads) {
        const uint32_t* t =
            reinterpret_cast<const uint32_t*>(tile + (u / 8) * kStride + (u % 8) * 8);
        reinterpret_cast<uint2*>(dst)[u] = make_uint2(t[0], t[1]);
    }
}

// Values of whole pages: out[i][head][token][channel] = fl32(code * scale), and
// zeros for a page number outside the pool.  Bound by the bytes written, four a code (2 x 67 pages
// of 16 heads and 128 channels 29 us: 35 MB read, 139 MB written, 6.0 TB/s).
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
    float4* out = reinterpret_cast<float4*>((is_v ? Vout : Kout) +
                                            ((size_t)i * Hkv + h) * (size_t)(kPage * D));
    constexpr int kWords = kPage * D / 4;
    auto put = [&](int u, uint32_t w) {
        out[u] = make_float4((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s,
                             (float)(int8_t)(w >> 16) * s, (float)(int8_t)(w >> 24) * s);
    };
    if (!is_v) {
#pragma unroll 4
        for (int u = tid; u < kWords; u += kThreads) put(u, good ? src[u] : 0u);
        return;
    }
#pragma unroll 4
    for (int u = tid; u < kWords; u += kThreads)
        *reinterpret_cast<uint32_t*>(tile + (u / 16) * kStride + (u % 16) * 4) =
            good ? src[u] : 0u;
    __syncthreads();
    // four channels x four tokens at a time, transposed in registers
    for (int u = tid; u < kWords / 4; u += kThreads) {
        const int g = u % (D / 4), quad = u / (D / 4);
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            w[c] = *reinterpret_cast<const uint32_t*>(tile + (4 * g + c) * kStride + quad * 4);
        const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);
        const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
        const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
        const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
        const int row = quad * 4 * (D / 4) + g;
        put(row, __builtin_amdgcn_perm(c, a, 0x05040100u));
        put(row + D / 4, __builtin_amdgcn_perm(c, a, 0x07060302u));
        put(row + 2 * (D / 4), __builtin_amdgcn_perm(d, b, 0x05040100u));
        put(row + 3 * (D / 4), __builtin_amdgcn_perm(d, b, 0x07060302u));
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
