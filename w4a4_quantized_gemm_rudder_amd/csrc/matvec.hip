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
// [-7, 7] is stored as the nibble q + 8, and (nibble | 0x4300) is the bf16
// value 128 + nibble = 136 + q: two codes become two matrix operands with one
// shift and one and-or.  The matrix core then sums (136 + q) * x, and a
// second product with ones gives sum x, so that
//   sum q * x = sum (136 + q) * x - 136 * sum x
// in fp32, once per group.  The difference cancels: each of the two sums is
// rounded in fp32 at a magnitude up to about 40 times that of the result, an
// error of a few 2^-19 relative, 2^-10 of the rounding of the bf16 output.
#include "rudder_internal.h"

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
    if (k0 < K) g_scale[(size_t)g * n_pad + n] = (uint16_t)sb;
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
__device__ __forceinline__ bf16x8_t widen_codes(uint32_t w) {
    union { uint32_t u[4]; bf16x8_t v; } r;
#pragma unroll
    for (int p = 0; p < 4; ++p) r.u[p] = ((w >> (4 * p)) & 0x000F000Fu) | 0x43004300u;
    return r.v;
}

template <int GROUP, int WAVES>
__global__ void __launch_bounds__(WAVES * 64)
matvec_w4_kernel(const uint16_t* __restrict__ X, const uint8_t* __restrict__ sid,
                 const uint8_t* __restrict__ Wq, const uint16_t* __restrict__ g_scale,
                 const float* __restrict__ comp_a, const float* __restrict__ comp_b, int M, int N,
                 int K, uint16_t* __restrict__ Y) {
    __shared__ f32x4_t part[WAVES][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int col = lane & 15, quarter = lane >> 4;
    const int nt = blockIdx.x, m = blockIdx.y * 16 + col;
    const int k_tiles = (K + kTileK - 1) / kTileK;
    const int n_pad = (N + kTileN - 1) / kTileN * kTileN;
    const int n0 = nt * kTileN + quarter * 4;      // the lane's four output channels
    const uint4* w = reinterpret_cast<const uint4*>(Wq) + (size_t)nt * k_tiles * 64 + lane;
    const uint16_t* x = X + (size_t)m * K + quarter * 8;
    bf16x8_t ones;
#pragma unroll
    for (int j = 0; j < 8; ++j) ones[j] = (__bf16)1.0f;

    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kt = wave; kt < k_tiles; kt += WAVES) {
        const uint4 c = w[(size_t)kt * 64];
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
        f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f}, sx = d;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = kt * kTileK + s * 32;
            union { uint4 u; bf16x8_t v; } xv;
            xv.u = make_uint4(0, 0, 0, 0);
            if (m < M && k < K) xv.u = *reinterpret_cast<const uint4*>(x + k);
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(cw[s]), xv.v, d, 0, 0, 0);
            sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xv.v, sx, 0, 0, 0);
            if ((s * 32 + 32) % GROUP == 0 && k < K) {
                const uint2 sc = *reinterpret_cast<const uint2*>(
                    g_scale + (size_t)(k / GROUP) * n_pad + n0);
                const float f[4] = {__uint_as_float(sc.x << 16),
                                    __uint_as_float(sc.x & 0xFFFF0000u),
                                    __uint_as_float(sc.y << 16),
                                    __uint_as_float(sc.y & 0xFFFF0000u)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] = fmaf(f[i], fmaf(-136.0f, sx[i], d[i]), acc[i]);
                d = {0.0f, 0.0f, 0.0f, 0.0f};
                sx = d;
            }
        }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0 || m >= M) return;
#pragma unroll
    for (int i = 1; i < WAVES; ++i) acc += part[i][lane];
    if (comp_a) {
        const size_t row = (size_t)sid[m] * N;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + i < N) acc[i] = fmaf(comp_a[row + n0 + i], acc[i], comp_b[row + n0 + i]);
    }
    uint16_t* y = Y + (size_t)m * N + n0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + i < N) y[i] = (uint16_t)float_to_bf16_bits(acc[i]);
}

template <int GROUP>
hipError_t launch_group(const uint16_t* X, const uint8_t* sid, const uint8_t* Wq,
                        const uint16_t* g_scale, const float* a, const float* b, int M, int N,
                        int K, uint16_t* Y, hipStream_t stream) {
    const dim3 grid((N + kTileN - 1) / kTileN, (M + 15) / 16);
    matvec_w4_kernel<GROUP, 8><<<grid, 512, 0, stream>>>(X, sid, Wq, g_scale, a, b, M, N, K, Y);
    return hipGetLastError();
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
