// Root-mean-square norm of the residual stream, with the residual's addition in
// front of it and the next linear's activation quantizer behind it; and the
// values of packed activation codes.
//
//   h = bf16_rne(R + X)      r = fl32(1 / sqrt(sum h^2 / K + eps)), in 64 bits
//   y = bf16_rne(fl32(fl32(h r) gamma))       codes of y as rudder_quant_act's
//
// Squares of bf16 values are exact in 64 bits and so is, but for 2^-53, their
// sum: r, and with it every row, step size and code, does not depend on the
// order of the sum.  Rows are rounded to bf16 in front of the quantizer, so that
// the codes are those of the norm's rows through rudder_quant_act.
//
// One pass: a row's elements stay in registers, as bf16, between the sum and
// the outputs.  Bound by memory: 16576 x 4096 with the residual to bf16 rows 102 us
// (5.3 TB/s, what a plain copy moves), to E2M3 codes 95 to 100 (459 MB, 4.6 TB/s) and
// to the 4-bit int ones 95; 8384 x 2048 to bf16 rows 12 (5.6 TB/s), to 8 bits 16 (51
// MB, 3.2 TB/s) and to 4 bits 16, the launch of a wave for one row each, whose
// loads, sum, codes and stores follow one another beside no other row's; a single
// row 2.3, a launch and the way to memory and back.
#include "rudder_block_launch.h"
#include "rudder_device.h"

namespace rudder {
namespace {

enum { kRows16 = 0, kInt8 = 1, kInt4 = 2, kE2M3 = 3 };    // what is written

struct Norm {
    const uint16_t *X, *R;
    const uint8_t* sid;
    const float *gamma, *inv_smooth, *table;
    double eps;
    int M, K;
    size_t ldx, ldr, ldh, ldy;
    uint16_t *H, *Y;
    uint8_t* Xq;
    float* row_scale;
};

// Two bf16 values a word, added in 32 bits and rounded.
__device__ __forceinline__ uint32_t add_bf16(uint32_t a, uint32_t b) {
    return pack_bf16(low(a) + low(b), high(a) + high(b));
}
__device__ __forceinline__ void load8(const float* from, float (&to)[8]) {
    const float4 u = reinterpret_cast<const float4*>(from)[0];
    const float4 v = reinterpret_cast<const float4*>(from)[1];
    to[0] = u.x;
    to[1] = u.y;
    to[2] = u.z;
    to[3] = u.w;
    to[4] = v.x;
    to[5] = v.y;
    to[6] = v.z;
    to[7] = v.w;
}

// Stored past the caches: the residual stream, which the next norm wants, several linears later (16576 x
// 4096 rows, with their values read back, 150 us, through the caches 152), and values (152, 190).  Rows and
// codes go to the next call and stay.

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off);
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int off = 32; off; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off));
    return v;
}

// Bytes of the codes of eight channels, and of what is stored at once: the codes of 16 channels, of 32
// in the E2M3 container.
constexpr int code_bytes(int out) { return out == kInt8 ? 8 : out == kInt4 ? 4 : 6; }
constexpr int slot_pieces(int out) { return out == kE2M3 ? 4 : 2; }

// Rows a workgroup whose codes pass through LDS, and their distance there.
__host__ __device__ constexpr bool staged(int out, int rows) {
    return out != kRows16 && (rows > 1 || out == kE2M3);
}
__host__ __device__ constexpr int stage_stride(int out, int K) {
    return K / 8 * code_bytes(out) + (out == kInt8 ? 16 : 8);
}

// ROWS rows a workgroup, WAVES waves a row, N pieces of eight channels a lane.
template <int OUT, int WAVES, int ROWS, int N, bool ADD>
__global__ void __launch_bounds__(64 * WAVES * ROWS) norm_kernel(const Norm a) {
    constexpr bool kEarly = N <= 2;                // gamma and inv_smooth on their way beside the row
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ double sums[ROWS][WAVES];
    __shared__ uint32_t tops[ROWS][WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int in_group = wave / WAVES, part = wave % WAVES;
    const int row = blockIdx.x * ROWS + in_group;
    const bool live = row < a.M;
    const int pieces = a.K / 8;
    auto piece = [&](int i) { return (i * WAVES + part) * 64 + lane; };
    // pieces behind the row's last read that one again and are left out below
    auto place = [&](int i) { return (size_t)min(piece(i), pieces - 1) * 8; };

    uint32_t h[N][4] = {};
    float early[kEarly ? N : 1][2][8];
    if constexpr (kEarly) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            load8(a.gamma + place(i), early[i][0]);
            if constexpr (OUT != kRows16) load8(a.inv_smooth + place(i), early[i][1]);
        }
    }
    auto gammas = [&](int i, float (&g)[8]) {
        if constexpr (kEarly) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = early[i][0][j];
        } else {
            load8(a.gamma + piece(i) * 8, g);
        }
    };
    auto smooths = [&](int i, float (&g)[8]) {
        if constexpr (kEarly) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = early[i][1][j];
        } else {
            load8(a.inv_smooth + piece(i) * 8, g);
        }
    };
    double sum = 0.0;
    if (live) {
        const uint16_t* x = a.X + (size_t)row * a.ldx;
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const uint4*>(x + place(i));
        if constexpr (ADD) {
            const uint16_t* r = a.R + (size_t)row * a.ldr;
            uint4 w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint4*>(r + place(i));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i].x = add_bf16(w[i].x, v[i].x);
                v[i].y = add_bf16(w[i].y, v[i].y);
                v[i].z = add_bf16(w[i].z, v[i].z);
                v[i].w = add_bf16(w[i].w, v[i].w);
                if (piece(i) < pieces) stream16(a.H + (size_t)row * a.ldh + place(i), v[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            h[i][0] = v[i].x;
            h[i][1] = v[i].y;
            h[i][2] = v[i].z;
            h[i][3] = v[i].w;
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double e = low(h[i][j]), f = high(h[i][j]);
                s = __builtin_fma(e, e, s);
                s = __builtin_fma(f, f, s);
            }
            sum += piece(i) < pieces ? s : 0.0;
        }
    }
    sum = wave_sum(sum);
    if constexpr (WAVES > 1) {
        if (lane == 0) sums[in_group][part] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += sums[in_group][w];
    }
    const float r = (float)(1.0 / sqrt(sum / (double)a.K + a.eps));

    uint32_t top = 0;                              // of |y inv_smooth|, as bits: a NaN is the largest
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!live || piece(i) >= pieces) continue;
        float g[8];
        gammas(i, g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[i][j] = pack_bf16(low(h[i][j]) * r * g[2 * j], high(h[i][j]) * r * g[2 * j + 1]);
        if constexpr (OUT == kRows16) {
            *reinterpret_cast<uint4*>(a.Y + (size_t)row * a.ldy + piece(i) * 8) =
                make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
        } else if (!a.table) {
            float s[8];
            smooths(i, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                top = max(top, __float_as_uint(low(h[i][j]) * s[2 * j]) & 0x7FFFFFFFu);
                top = max(top, __float_as_uint(high(h[i][j]) * s[2 * j + 1]) & 0x7FFFFFFFu);
            }
        }
    }
    if constexpr (OUT != kRows16) {
        constexpr float kMost = OUT == kInt8 ? 127.0f : 7.0f;
        float step = 0.0f;
        if (a.table) {
            if (live) step = a.table[a.sid[row] & (RUDDER_MAX_STREAMS - 1)];
        } else {
            top = wave_max(top);
            if constexpr (WAVES > 1) {
                if (lane == 0) tops[in_group][part] = top;
                __syncthreads();
                top = 0;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) top = max(top, tops[in_group][w]);
            }
            step = (float)((double)__uint_as_float(top) / (double)kMost);
            // its reciprocal would pass 32 bits, and zeros times that are no numbers
            if (step <= 0x1p-128f) step = 0.0f;
        }
        const float inv = step_reciprocal(step);
        if (live && part == 0 && lane == 0) a.row_scale[row] = step;
        // codes as integer-valued floats; padding rows and pieces behind the last hold zeros
        auto codes = [&](int i, float (&c)[8]) {
            float s[8] = {};
            if (live && piece(i) < pieces) smooths(i, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[2 * j] = quantize_clamped_f(low(h[i][j]) * s[2 * j] * inv, kMost);
                c[2 * j + 1] = quantize_clamped_f(high(h[i][j]) * s[2 * j + 1] * inv, kMost);
            }
        };
        uint8_t* line = stage + in_group * stage_stride(OUT, a.K);
        if constexpr (OUT == kE2M3) {
            // the fields of 32 codes are a string of 192 bits: those of four pieces, 48 bits each,
            // whose place in the row's string is six bytes a piece
#pragma unroll
            for (int i0 = 0; i0 < N; i0 += 4) {
                float c[32] = {};
#pragma unroll
                for (int i = 0; i < 4 && i0 + i < N; ++i) {
                    float part8[8];
                    codes(i0 + i, part8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) c[8 * i + j] = part8[j];
                }
                uint32_t d[6];
                pack_e2m3x32(c, d);
#pragma unroll
                for (int i = 0; i < 4 && i0 + i < N; ++i) {
                    if (piece(i0 + i) >= pieces) continue;
                    uint16_t* to = reinterpret_cast<uint16_t*>(line + piece(i0 + i) * 6);
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        to[j] = (uint16_t)(d[(3 * i + j) / 2] >> ((3 * i + j) % 2 * 16));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (piece(i) >= pieces) continue;
                float c[8];
                codes(i, c);
                int q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = (int)c[j];
                const int k0 = piece(i) * 8;
                if constexpr (OUT == kInt8) {
                    const uint2 w = make_uint2(byte_word(q), byte_word(q + 4));
                    if constexpr (staged(OUT, ROWS))
                        *reinterpret_cast<uint2*>(line + k0) = w;
                    else
                        *reinterpret_cast<uint2*>(a.Xq + tiled_slot_offset<8>(row, k0, a.K) +
                                                  (k0 & 8)) = w;
                } else {
                    const uint32_t w = split_nibble_word(q);
                    if constexpr (staged(OUT, ROWS))
                        *reinterpret_cast<uint32_t*>(line + k0 / 2) = w;
                    else
                        *reinterpret_cast<uint32_t*>(a.Xq + tiled_slot_offset<4>(row, k0, a.K) +
                                                     (k0 & 8) / 2) = w;
                }
            }
        }
        if constexpr (staged(OUT, ROWS)) {
            // slot by slot, a workgroup's rows beside each other: 16 ROWS bytes in a row (8 ROWS for
            // four bits)
            __syncthreads();
            constexpr int kSlot = slot_pieces(OUT) * 8;
            for (int u = threadIdx.x; u < a.K / kSlot * ROWS; u += 64 * WAVES * ROWS) {
                const int in = u % ROWS, k0 = u / ROWS * kSlot, to = blockIdx.x * ROWS + in;
                const uint8_t* from = stage + in * stage_stride(OUT, a.K);
                if constexpr (OUT == kInt8) {
                    *reinterpret_cast<uint4*>(a.Xq + tiled_slot_offset<8>(to, k0, a.K)) =
                        *reinterpret_cast<const uint4*>(from + k0);
                } else if constexpr (OUT == kInt4) {
                    *reinterpret_cast<uint2*>(a.Xq + tiled_slot_offset<4>(to, k0, a.K)) =
                        *reinterpret_cast<const uint2*>(from + k0 / 2);
                } else {
                    const uint2* w = reinterpret_cast<const uint2*>(from + k0 / 4 * 3);
                    const uint2 x = w[0], y = w[1], z = w[2];
                    uint8_t* block = a.Xq + e2m3_block_offset(to, k0, a.K);
                    const int slot = e2m3_slot(to, k0);
                    *reinterpret_cast<uint4*>(block + slot * 16) = make_uint4(x.x, x.y, y.x, y.y);
                    *reinterpret_cast<uint2*>(block + 1024 + slot * 8) = z;
                }
            }
        }
    }
}

template <int OUT, int WAVES, int ROWS, int N>
hipError_t start(const Norm& a, hipStream_t stream) {
    // codes: padding rows up to a multiple of 32 as well
    const int64_t rows = OUT == kRows16 ? a.M : ((int64_t)a.M + 31) / 32 * 32;
    const unsigned grid = (unsigned)((rows + ROWS - 1) / ROWS);
    const size_t lds = staged(OUT, ROWS) ? (size_t)ROWS * stage_stride(OUT, a.K) : 0;
    if (a.R)
        norm_kernel<OUT, WAVES, ROWS, N, true><<<grid, 64 * WAVES * ROWS, lds, stream>>>(a);
    else
        norm_kernel<OUT, WAVES, ROWS, N, false><<<grid, 64 * WAVES * ROWS, lds, stream>>>(a);
    return hipGetLastError();
}

// Few rows take eight waves each, their gamma and smoothing factors on the way beside them; many rows a
// wave each, four a workgroup: codes then leave in pieces of 64 bytes, and two to four workgroups share
// a compute unit.  us, eight waves a row | one, residual added, 8-bit codes with a step size a row: 512
// rows of 2048 channels 5.4 | 6.1, 1024 7.4 | 6.6; 1024 of 4096 9.7 | 10.6 (bf16 rows 6.6 | 7.8, 1536
// E2M3 13.6 | 13.5); 1536 of 8192 21.4 | 27.4; 16576 of 4096, E2M3 137 | 103.  Eight rows a workgroup
// 107, 16576 of 4096 8-bit 114 against 106; two rows 110.
// Wider rows than 8192 channels are rare and take one shape for all widths, eight waves a row and up to
// sixteen pieces a lane, of which narrow ones leave most unused: 2048 x 65536 with the residual to bf16
// rows 212 us (5.1 TB/s), 8384 x 12288 252 (3.3 TB/s; 8384 x 8192 110 with 5.0) and to 8 bits 358.
template <int OUT>
hipError_t launch(const Norm& a, hipStream_t stream) {
    if (a.K > 8192) return start<OUT, 8, 1, 16>(a, stream);
    if (a.M <= (a.K <= 2048 ? 512 : a.K <= 4096 ? 1024 : 1536))
        return a.K <= 4096 ? start<OUT, 8, 1, 1>(a, stream) : start<OUT, 8, 1, 2>(a, stream);
    if (a.K <= 2048) return start<OUT, 1, 4, 4>(a, stream);
    if (a.K <= 4096) return start<OUT, 1, 4, 8>(a, stream);
    return start<OUT, 1, 4, 16>(a, stream);
}

// ---------------------------------------------------------------------------
// Values of packed codes: eight lanes take 32 channels of a row, a wave eight rows at once, so that its
// stores are whole lines; 32 rows x 32 channels a wave.
// ---------------------------------------------------------------------------
// The value of a 6-bit E2M3 field: its exponent and mantissa at the places of a 32-bit number's, whose
// bias is 126 more; numbers below the first binade are subnormal in both.
__device__ __forceinline__ float e2m3_value(uint32_t field) {
    return __uint_as_float((field & 31u) << 20 | (field & 32u) << 26) * 0x1p126f;
}

template <int BITS, int CODES>
__global__ void __launch_bounds__(256)
dequant_act_kernel(const uint8_t* __restrict__ Xq, const float* __restrict__ row_scale, int M,
                   int K, float* __restrict__ out) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int columns = K >> 5;
    const int64_t at = (int64_t)blockIdx.x * 4 + wave;
    if (at >= (int64_t)((M + 31) >> 5) * columns) return;
    const int rb = (int)(at / columns), k = (int)(at - (int64_t)rb * columns) * 32 + lane % 8 * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = rb * 32 + i * 8 + lane / 8;
        if (row >= M) continue;
        float c[4];
        if constexpr (CODES == RUDDER_CODES_E2M3) {
            // four fields of six bits are the bytes 3 t .. 3 t + 2 of the slot's string, of which
            // 16 lie in plane 0
            const int slot = e2m3_slot(row, k), t = (k & 31) / 4;
            constexpr int kPlanes = BITS == 8 ? 2 : 1;
            const uint8_t* block = Xq + kPlanes * e2m3_block_offset(row, k, K);
            float digit[kPlanes][4];
#pragma unroll
            for (int p = 0; p < kPlanes; ++p) {
                uint32_t w = 0;
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const int b = 3 * t + j;
                    w |= (uint32_t)block[p * 1536 + (b < 16 ? slot * 16 + b
                                                           : 1024 + slot * 8 + b - 16)]
                         << (8 * j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) digit[p][j] = e2m3_value(w >> (6 * j));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c[j] = BITS == 8 ? 32.0f * digit[0][j] + 2.0f * digit[kPlanes - 1][j]
                                 : digit[0][j];
        } else if constexpr (BITS == 8) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(
                Xq + tiled_slot_offset<8>(row, k, K) + (k & 15));
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = (float)(int8_t)(w >> (8 * j));
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(
                Xq + tiled_slot_offset<4>(row, k, K) + (k & 8) / 2);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c[j] = (float)((int)(w << (28 - 8 * j - (k & 4))) >> 28);
        }
        const float s = row_scale[row];
        stream16(out + (size_t)row * K + k,
                 make_uint4(__float_as_uint(c[0] * s), __float_as_uint(c[1] * s),
                            __float_as_uint(c[2] * s), __float_as_uint(c[3] * s)));
    }
}

}  // namespace

hipError_t launch_norm(const uint16_t* X, const uint16_t* R, const uint8_t* sid,
                       const float* gamma, const float* inv_smooth, const float* table, float eps,
                       int M, int K, int ldx, int ldr, int ldh, int ldy, int abits, int codes,
                       uint16_t* H, uint16_t* Y, void* Xq, float* row_scale, hipStream_t stream) {
    Norm a = {};
    a.X = X;
    a.R = R;
    a.sid = sid;
    a.gamma = gamma;
    a.inv_smooth = inv_smooth;
    a.table = table;
    a.eps = (double)eps;
    a.M = M;
    a.K = K;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.H = H;
    a.Y = Y;
    a.Xq = static_cast<uint8_t*>(Xq);
    a.row_scale = row_scale;
    if (Y) return launch<kRows16>(a, stream);
    if (codes == RUDDER_CODES_E2M3) return launch<kE2M3>(a, stream);
    return abits == 8 ? launch<kInt8>(a, stream) : launch<kInt4>(a, stream);
}

hipError_t launch_dequant_act(const uint8_t* Xq, const float* row_scale, int M, int K, int abits,
                              int codes, float* out, hipStream_t stream) {
    const int64_t blocks = (int64_t)((M + 31) / 32) * (K / 32);
    const unsigned grid = (unsigned)((blocks + 3) / 4);
    auto go = [&](auto kernel) { kernel<<<grid, 256, 0, stream>>>(Xq, row_scale, M, K, out); };
    if (codes == RUDDER_CODES_E2M3 && abits == 8)
        go(dequant_act_kernel<8, RUDDER_CODES_E2M3>);
    else if (codes == RUDDER_CODES_E2M3)
        go(dequant_act_kernel<4, RUDDER_CODES_E2M3>);
    else if (abits == 8)
        go(dequant_act_kernel<8, RUDDER_CODES_INT>);
    else
        go(dequant_act_kernel<4, RUDDER_CODES_INT>);
    return hipGetLastError();
}

}  // namespace rudder
