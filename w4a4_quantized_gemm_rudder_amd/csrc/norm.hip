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
// the outputs.
#include "rudder_block_launch.h"

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

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    union { bf16x2_t v; uint32_t u; } r;
    r.v = (bf16x2_t){(__bf16)a, (__bf16)b};
    return r.u;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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

// Channels of one piece of a row, a lane's share of a load and a store.
constexpr int piece_of(int out) { return out == kRows16 ? 8 : out == kE2M3 ? 32 : 16; }

// ROWS rows a workgroup, WAVES waves a row, N pieces a lane.
template <int OUT, int WAVES, int ROWS, int N, bool ADD>
__global__ void __launch_bounds__(64 * WAVES * ROWS) norm_kernel(const Norm a) {
    constexpr int kPiece = piece_of(OUT), kWords = kPiece / 2, kLoads = kPiece / 8;
    __shared__ double sums[ROWS][WAVES];
    __shared__ uint32_t tops[ROWS][WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int in_group = wave / WAVES, part = wave % WAVES;
    const int row = blockIdx.x * ROWS + in_group;
    const bool live = row < a.M;
    const int pieces = a.K / kPiece;
    auto piece = [&](int i) { return (i * WAVES + part) * 64 + lane; };

    uint32_t h[N][kWords] = {};
    double sum = 0.0;
    if (live) {
        const uint16_t* x = a.X + (size_t)row * a.ldx;
        // pieces behind the row's last read that one again and are left out below
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4* from =
                reinterpret_cast<const uint4*>(x + (size_t)min(piece(i), pieces - 1) * kPiece);
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const uint4 v = from[j];
                h[i][4 * j] = v.x;
                h[i][4 * j + 1] = v.y;
                h[i][4 * j + 2] = v.z;
                h[i][4 * j + 3] = v.w;
            }
        }
        if constexpr (ADD) {
            const uint16_t* r = a.R + (size_t)row * a.ldr;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const size_t at = (size_t)min(piece(i), pieces - 1) * kPiece;
                const uint4* from = reinterpret_cast<const uint4*>(r + at);
                uint32_t w[kWords];
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    const uint4 v = from[j];
                    w[4 * j] = v.x;
                    w[4 * j + 1] = v.y;
                    w[4 * j + 2] = v.z;
                    w[4 * j + 3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    h[i][j] = pack_bf16(low(w[j]) + low(h[i][j]), high(w[j]) + high(h[i][j]));
                if (piece(i) < pieces) {
                    uint4* to = reinterpret_cast<uint4*>(a.H + (size_t)row * a.ldh + at);
#pragma unroll
                    for (int j = 0; j < kLoads; ++j)
                        to[j] = make_uint4(h[i][4 * j], h[i][4 * j + 1], h[i][4 * j + 2],
                                           h[i][4 * j + 3]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const double u = low(h[i][j]), v = high(h[i][j]);
                s = __builtin_fma(u, u, s);
                s = __builtin_fma(v, v, s);
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
        const int k0 = piece(i) * kPiece;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const float2 g = *reinterpret_cast<const float2*>(a.gamma + k0 + 2 * j);
            h[i][j] = pack_bf16(low(h[i][j]) * r * g.x, high(h[i][j]) * r * g.y);
        }
        if constexpr (OUT == kRows16) {
            *reinterpret_cast<uint4*>(a.Y + (size_t)row * a.ldy + k0) =
                make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
        } else if (!a.table) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const float2 s = *reinterpret_cast<const float2*>(a.inv_smooth + k0 + 2 * j);
                top = max(top, __float_as_uint(low(h[i][j]) * s.x) & 0x7FFFFFFFu);
                top = max(top, __float_as_uint(high(h[i][j]) * s.y) & 0x7FFFFFFFu);
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
        }
        const float inv = step_reciprocal(step);
        if (live && part == 0 && lane == 0) a.row_scale[row] = step;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (piece(i) >= pieces) continue;
            const int k0 = piece(i) * kPiece;
            float c[kPiece];
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const float2 s = *reinterpret_cast<const float2*>(a.inv_smooth + k0 + 2 * j);
                c[2 * j] = quantize_clamped_f(low(h[i][j]) * s.x * inv, kMost);
                c[2 * j + 1] = quantize_clamped_f(high(h[i][j]) * s.y * inv, kMost);
                if (!live) c[2 * j] = c[2 * j + 1] = 0.0f;      // padding rows
            }
            if constexpr (OUT == kE2M3) {
                uint32_t d[6];
                pack_e2m3x32(c, d);
                uint8_t* block = a.Xq + e2m3_block_offset(row, k0, a.K);
                const int slot = e2m3_slot(row, k0);
                *reinterpret_cast<uint4*>(block + slot * 16) = make_uint4(d[0], d[1], d[2], d[3]);
                *reinterpret_cast<uint2*>(block + 1024 + slot * 8) = make_uint2(d[4], d[5]);
            } else {
                int q[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) q[j] = (int)c[j];
                if constexpr (OUT == kInt8)
                    *reinterpret_cast<uint4*>(a.Xq + tiled_slot_offset<8>(row, k0, a.K)) =
                        make_uint4(byte_word(q), byte_word(q + 4), byte_word(q + 8),
                                   byte_word(q + 12));
                else
                    *reinterpret_cast<uint2*>(a.Xq + tiled_slot_offset<4>(row, k0, a.K)) =
                        make_uint2(split_nibble_word(q), split_nibble_word(q + 8));
            }
        }
    }
}

template <int OUT, int WAVES, int ROWS, int N>
hipError_t start(const Norm& a, hipStream_t stream) {
    // codes: padding rows up to a multiple of 32 as well
    const int64_t rows = OUT == kRows16 ? a.M : ((int64_t)a.M + 31) / 32 * 32;
    const unsigned grid = (unsigned)((rows + ROWS - 1) / ROWS);
    if (a.R)
        norm_kernel<OUT, WAVES, ROWS, N, true><<<grid, 64 * WAVES * ROWS, 0, stream>>>(a);
    else
        norm_kernel<OUT, WAVES, ROWS, N, false><<<grid, 64 * WAVES * ROWS, 0, stream>>>(a);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch(const Norm& a, hipStream_t stream) {
    constexpr int kPiece = piece_of(OUT);
    if (a.K > 8192) return start<OUT, 8, 1, 128 / kPiece>(a, stream);
    if (a.M <= 512) return start<OUT, 8, 1, 32 / kPiece>(a, stream);
    if (a.K <= 2048) return start<OUT, 1, 8, 32 / kPiece>(a, stream);
    if (a.K <= 4096) return start<OUT, 1, 8, 64 / kPiece>(a, stream);
    return start<OUT, 1, 8, 128 / kPiece>(a, stream);
}

// ---------------------------------------------------------------------------
// Values of packed codes: eight lanes take 32 channels of a row, a wave eight
// rows at once, so that its stores are whole lines; 32 rows x 32 channels a wave.
// ---------------------------------------------------------------------------
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
                for (int j = 0; j < 4; ++j) {
                    // eighths: m below the first binade, (8 + m) 2^(e - 1) from there on
                    const int f = w >> (6 * j), e = f >> 3 & 3, m = f & 7;
                    const int eighths = e ? (8 + m) << (e - 1) : m;
                    digit[p][j] = 0.125f * (float)(f & 32 ? -eighths : eighths);
                }
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
        *reinterpret_cast<float4*>(out + (size_t)row * K + k) =
            make_float4(c[0] * s, c[1] * s, c[2] * s, c[3] * s);
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
