// Few-row products with 4-bit weights that carry one scale per group of input
// channels and output channel (activations stay bf16), and their offline
// weight preparation.
//
//   t[m][n] = sum_g s[g][n] * sum_{k in g} q[k][n] * x[m][k]
//   Y[m][n] = bf16(fma(a[sid[m]][n], t, b[sid[m]][n]))
//
// The product is bound by the bytes of the weight codes (K * N / 2): at 16
// rows a code is used 16 times, far below what the matrix cores could do.
// What has to stay small is therefore the work per code.  A code q in
// [-7, 7] is stored as the nibble q + 8, and (nibble << 3 | 0x4180) is the bf16
// value 16 + nibble = 24 + q: two codes become two matrix operands with one
// shift and one and-or.  The matrix core then sums (24 + q) * x, and a
// second product with ones gives sum x, so that
//   sum q * x = sum (24 + q) * x - 24 * sum x
// in fp32, once per group.  The difference cancels: each of the two sums is
// formed at magnitudes up to 31 * sum |x| over the group, so that a group's
// result is off by a few 2^-19 * sum |x|, whatever its own size.  A code is
// off by up to a half, which makes that a few 2^-18 of what the weights'
// rounding may cost; results far below sum |x| have it relative to that.
#include "rudder_operators.h"

namespace rudder {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTileN = 16;       // output channels per tile (MFMA rows)
constexpr int kTileK = 128;      // input channels per tile: 16 bytes a lane

// ---------------------------------------------------------------------------
// Offline preparation: one thread per (group, output channel).  Not hot.
// ---------------------------------------------------------------------------
__global__ void quantize_weights_grouped_kernel(const uint16_t* __restrict__ W, int K, int N,
                                                int group, uint8_t* __restrict__ Wq,
                                                uint16_t* __restrict__ g_scale) {
    const int n_pad = (N + kTileN - 1) / kTileN * kTileN;
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    const int g = blockIdx.y;
    if (n >= n_pad) return;
    const int k_tiles = (K + kTileK - 1) / kTileK;
    const int k0 = g * group;                      // k0 >= K: the padding of the last k tile
    float amax = 0.0f;
    if (n < N && k0 < K)
        for (int k = k0; k < k0 + group; ++k)
            amax = fmaxf(amax, fabsf(bf16_bits_to_float(W[(size_t)k * N + n])));
    const uint32_t sb = float_to_bf16_bits((float)((double)amax / 7.0));
    const float inv = step_reciprocal(bf16_bits_to_float(sb));
    const int groups = kTileK / group;             // of a tile
    const size_t of_tile = ((size_t)(n / kTileN) * k_tiles + g / groups) * kTileN * groups;
    g_scale[of_tile + (n % kTileN) / 4 * 4 * groups + (g % groups) * 4 + n % 4] = (uint16_t)sb;
    // a dword holds k = 32 * step + 8 * quarter + 0..7: code 2p in nibble p, 2p + 1 in p + 4
    for (int k = k0; k < k0 + group; k += 8) {
        uint32_t word = 0;
        for (int j = 0; j < 8; ++j) {
            int c = 0;
            if (n < N && k + j < K)
                c = quantize_clamped(bf16_bits_to_float(W[(size_t)(k + j) * N + n]) * inv, 7.0f);
            word |= (uint32_t)(c + 8) << (4 * (j / 2 + 4 * (j & 1)));
        }
        const size_t tile = (size_t)(n / kTileN) * k_tiles + k / kTileK;
        const int lane = (n % kTileN) + kTileN * ((k % 32) / 8);
        const size_t at = tile * 1024 + (size_t)lane * 16 + (size_t)((k % kTileK) / 32) * 4;
        *reinterpret_cast<uint32_t*>(Wq + at) = word;
    }
}

// ---------------------------------------------------------------------------
// The product.
// ---------------------------------------------------------------------------
// Orders a wave's LDS accesses of different lanes (the hardware keeps their order; this keeps the
// compiler's).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ bf16x8_t widen_codes(uint32_t w, uint32_t magic) {
    union { uint32_t u[4]; bf16x8_t v; } r;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        r.u[p] = ((p ? w >> (4 * p - 3) : w << 3) & 0x00780078u) | magic;
    return r.v;
}

// Workgroup: NT tiles of 16 output channels, their K tiles dealt to WAVES
// waves.  What a wave needs of the activations for a K tile comes in MQ loads of
// whole 256-byte pieces of four rows and is exchanged through LDS: loading the
// products' operands as they are (64 bytes of each of 16 rows) took four loads
// for any row count and was bound by them (K = 4096, N = 12288, M = 1: 8.8 us,
// now 6.6; K = 16384, N = 4096, M = 13, groups of 32: 18.3 us, now 11.4).
template <int GROUP, int WAVES, int NT, int MQ>
__global__ void __launch_bounds__(WAVES * 64)
matvec_w4_kernel(const uint16_t* __restrict__ X, const uint8_t* __restrict__ sid,
                 const uint8_t* __restrict__ Wq, const uint16_t* __restrict__ g_scale,
                 const float* __restrict__ comp_a, const float* __restrict__ comp_b, int M, int N,
                 int K, uint16_t* __restrict__ Y) {
    constexpr int kGroups = kTileK / GROUP;        // groups a tile
    constexpr int kScaleTile = kTileN * kGroups * 2;       // bytes of a tile's scales
    // a wave's activations of one tile: 4 * MQ rows of 256 bytes, 16-byte pieces exchanged by
    // row so that a column of them spreads over the banks; later the waves' partial sums
    union Shared {
        uint8_t x[WAVES][MQ * 4 * 256];
        f32x4_t part[NT][WAVES][64];
    };
    __shared__ __align__(16) Shared lds;
    // wave-uniform: tile addresses stay in scalar registers
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
    const int nt0 = blockIdx.x * NT, m0 = blockIdx.y * 16;
    const int k_tiles = (K + kTileK - 1) / kTileK;
    const int n_tiles = (N + kTileN - 1) / kTileN;
    const char* w = reinterpret_cast<const char*>(Wq);
    const char* x = reinterpret_cast<const char*>(X + (size_t)m0 * K);
    const char* gs = reinterpret_cast<const char*>(g_scale);
    const uint32_t w_lane = lane * 16, gs_lane = quarter * (8 * kGroups);
    // a load takes 256 bytes of four rows; rows past M repeat the last one, and what the
    // columns past M compute is not stored
    uint32_t x_lane[MQ], x_put[MQ];
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
        const int r = 4 * j + quarter;
        x_lane[j] = (uint32_t)min(r, M - 1 - m0) * (uint32_t)K * 2 + col * 16;
        x_put[j] = r * 256 + (col ^ r) * 16;
    }
    const int x_row = col & (4 * MQ - 1);
    uint8_t* xs = lds.x[wave];
    // one of the two constants in a vector register: and-or takes one scalar operand
    uint32_t magic = 0x41804180u;
    asm("" : "+v"(magic));
    bf16x8_t ones;
#pragma unroll
    for (int j = 0; j < 8; ++j) ones[j] = (__bf16)1.0f;

    f32x4_t acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kt = wave; kt < k_tiles; kt += WAVES) {
        uint4 c[NT], xr[MQ];
        uint32_t sc[NT][2 * kGroups];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const size_t tile = (size_t)min(nt0 + t, n_tiles - 1) * k_tiles + kt;
            c[t] = *reinterpret_cast<const uint4*>(w + tile * 1024 + w_lane);
            const char* ts = gs + tile * kScaleTile + gs_lane;
            if constexpr (kGroups == 1) {
                const uint2 v = *reinterpret_cast<const uint2*>(ts);
                sc[t][0] = v.x;
                sc[t][1] = v.y;
            } else {
#pragma unroll
                for (int g = 0; g < kGroups / 2; ++g) {
                    const uint4 v = *reinterpret_cast<const uint4*>(ts + g * 16);
                    sc[t][4 * g] = v.x;
                    sc[t][4 * g + 1] = v.y;
                    sc[t][4 * g + 2] = v.z;
                    sc[t][4 * g + 3] = v.w;
                }
            }
        }
        // past K (the last tile's padding) the row's last piece is read again, under scale 0
        const uint32_t back = (uint32_t)max(kt * kTileK + col * 8 - (K - 8), 0) * 2;
#pragma unroll
        for (int j = 0; j < MQ; ++j)
            xr[j] = *reinterpret_cast<const uint4*>(x + (size_t)kt * (kTileK * 2) +
                                                    (x_lane[j] - back));
#pragma unroll
        for (int j = 0; j < MQ; ++j) *reinterpret_cast<uint4*>(xs + x_put[j]) = xr[j];
        wave_sync();
        union { uint4 u; bf16x8_t v; } xv[4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
            xv[s].u = *reinterpret_cast<const uint4*>(xs + x_row * 256 +
                                                      ((4 * s + quarter) ^ x_row) * 16);
        wave_sync();
        // Codes are widened behind this line.  Left to itself the compiler began with their shifts,
        // between a tile's loads, and waited for the first before it had asked for the last (K =
        // 16384, N = 4096, M = 13, groups of 32: 13.1 us, 10.5 so; K = 8192, N = 12288, M = 16:
        // 21.3, 16.2).
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            f32x4_t d[NT], sx = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < NT; ++t) d[t] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4 / kGroups; ++i) {
                const int s = g * (4 / kGroups) + i;
                sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xv[s].v, sx, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t cw = s == 0 ? c[t].x : s == 1 ? c[t].y
                                      : s == 2 ? c[t].z : c[t].w;
                    d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(cw, magic),
                                                                   xv[s].v, d[t], 0, 0, 0);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t lo = sc[t][2 * g], hi = sc[t][2 * g + 1];
                const float f[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u),
                                    __uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t][i] = fmaf(f[i], fmaf(-24.0f, sx[i], d[t][i]), acc[t][i]);
            }
        }
    }
    __syncthreads();                               // the activations have been read
#pragma unroll
    for (int t = 0; t < NT; ++t) lds.part[t][wave][lane] = acc[t];
    __syncthreads();
    // one thread an output: 16 rows x 16 channels a tile
    for (int i = threadIdx.x; i < NT * 256; i += WAVES * 64) {
        const int t = i >> 8, r = (i >> 4) & 15, nn = i & 15;
        const int m = m0 + r, n = (nt0 + t) * kTileN + nn;
        if (m >= M || n >= N) continue;
        const int at = (nn >> 2) * 16 + r;
        float y = lds.part[t][0][at][nn & 3];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) y += lds.part[t][v][at][nn & 3];
        if (comp_a) {
            const size_t o = (size_t)sid[m] * N + n;
            y = fmaf(comp_a[o], y, comp_b[o]);
        }
        Y[(size_t)m * N + n] = (uint16_t)float_to_bf16_bits(y);
    }
}

// Waves and channel tiles a workgroup, measured over K 2048..16384, N 2048..24576 and M 1..16:
//   - up to 8 rows, 8 waves and one tile (K = 4096, N = 12288, M = 1: 6.7 us; 16 waves 7.2); from
//     K = 8192 on 16 waves, which divide the longer loop (K = 16384, N = 4096: 8.6 against 10.8
//     us); from 1536 tiles on two share the activations (K = 4096, N = 24576: 10.6 against 11.2
//     us);
//   - more rows make the activations the larger part of what a workgroup reads, so two tiles share
//     them from 384 tiles on (M = 16, K = 16384, N = 8192: 17.3 against 19.6 us) and four from 768
//     on (K = 8192, N = 12288: 13.9 against 15.3 us); below, the compute units would run short.
template <int GROUP>
hipError_t launch_group(const uint16_t* X, const uint8_t* sid, const uint8_t* Wq,
                        const uint16_t* g_scale, const float* a, const float* b, int M, int N,
                        int K, uint16_t* Y, hipStream_t stream) {
    const int n_tiles = (N + kTileN - 1) / kTileN;
    const int k_tiles = (K + kTileK - 1) / kTileK;
    auto go = [&](auto kernel, int waves, int nt) {
        const dim3 grid((n_tiles + nt - 1) / nt, (M + 15) / 16);
        kernel<<<grid, waves * 64, 0, stream>>>(X, sid, Wq, g_scale, a, b, M, N, K, Y);
        return hipGetLastError();
    };
    if (M <= 8) {
        if (n_tiles >= 1536)
            return M <= 4 ? go(matvec_w4_kernel<GROUP, 8, 2, 1>, 8, 2)
                          : go(matvec_w4_kernel<GROUP, 8, 2, 2>, 8, 2);
        if (k_tiles >= 64)
            return M <= 4 ? go(matvec_w4_kernel<GROUP, 16, 1, 1>, 16, 1)
                          : go(matvec_w4_kernel<GROUP, 16, 1, 2>, 16, 1);
        return M <= 4 ? go(matvec_w4_kernel<GROUP, 8, 1, 1>, 8, 1)
                      : go(matvec_w4_kernel<GROUP, 8, 1, 2>, 8, 1);
    }
    if (n_tiles >= 768) return go(matvec_w4_kernel<GROUP, 8, 4, 4>, 8, 4);
    if (n_tiles >= 384) return go(matvec_w4_kernel<GROUP, 16, 2, 4>, 16, 2);
    if (k_tiles >= 32) return go(matvec_w4_kernel<GROUP, 16, 1, 4>, 16, 1);
    return go(matvec_w4_kernel<GROUP, 8, 1, 4>, 8, 1);
}

}  // namespace

hipError_t launch_quantize_weights_grouped(const uint16_t* W, int K, int N, int group,
                                           uint8_t* Wq, uint16_t* g_scale, hipStream_t stream) {
    const int n_pad = (N + kTileN - 1) / kTileN * kTileN;
    const int k_pad = (K + kTileK - 1) / kTileK * kTileK;
    const dim3 grid((n_pad + 63) / 64, k_pad / group);
    quantize_weights_grouped_kernel<<<grid, 64, 0, stream>>>(W, K, N, group, Wq, g_scale);
    return hipGetLastError();
}

hipError_t launch_matvec_w4(const uint16_t* X, const uint8_t* sid, const uint8_t* Wq,
                            const uint16_t* g_scale, const float* a, const float* b, int M, int N,
                            int K, int group, uint16_t* Y, hipStream_t stream) {
    if (group == 32) return launch_group<32>(X, sid, Wq, g_scale, a, b, M, N, K, Y, stream);
    if (group == 64) return launch_group<64>(X, sid, Wq, g_scale, a, b, M, N, K, Y, stream);
    return launch_group<128>(X, sid, Wq, g_scale, a, b, M, N, K, Y, stream);
}

}  // namespace rudder
