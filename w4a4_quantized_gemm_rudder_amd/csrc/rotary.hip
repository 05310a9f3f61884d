// Rotary positions: pairs of channels (x, y) of the query and key heads are
// turned by an angle that grows with the row's position,
//   x' = x c - y s,  y' = y c + x s,  c, s = magnitude * cos, sin(position * freq[i]).
//
// The angle is formed in turns, as the sum of two 64-bit numbers: the product
// position * freq and its rounding error, times 1 / (2 pi) in two parts.  What
// is left of it behind the whole turns is right to 2^-60 for every int32
// position, and is rounded to 32 bits only then (2^-26 turns).
#include "rudder_block_launch.h"

namespace rudder {
namespace {

struct Rotary {
    const uint16_t *Q, *K;
    const int32_t *row_start, *pos;
    const double* freq;
    float magnitude;
    int T, max_rows, Hq, Hkv, part;
    size_t ldq, ldk, ldqo, ldko;
    uint16_t *Qo, *Ko;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    union { bf16x2_t v; uint32_t u; } r;
    r.v = (bf16x2_t){(__bf16)a, (__bf16)b};
    return r.u;
}

// position * freq in turns, in [-1/2, 1/2]
__device__ __forceinline__ float turns(int64_t position, double freq) {
    constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;   // 1 / (2 pi)
    const double p = (double)position, a = p * freq, da = __builtin_fma(p, freq, -a);
    const double t = a * kHigh;
    const double dt = __builtin_fma(a, kHigh, -t) + (a * kLow + da * kHigh);
    return (float)((t - __builtin_rint(t)) + dt);
}

// A wave takes a row (or, with SPLIT, its four waves a quarter of the heads each); a lane 16
// channels of a head: 8 pairs, or 16 channels that are not rotated.
template <int D, bool PAIRS, bool SPLIT>
__global__ void __launch_bounds__(256) rotary_kernel(const Rotary a) {
    constexpr int kUnits = D / 16, kHeads = 64 / kUnits;   // lanes a head, heads a wave
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int b = blockIdx.y;
    const int r0 = min(max(a.row_start[b], 0), a.T);
    const int n = min(min(max(a.row_start[b + 1], r0), a.T) - r0, a.max_rows);
    const int i = SPLIT ? blockIdx.x : blockIdx.x * 4 + wave;
    const int first = a.pos ? a.pos[b] : 0;
    if (i >= n || first < 0) return;

    // lane f's cosine and sine, then those of this lane's eight pairs
    const int pairs = a.part / 2;
    float cos1 = 1.0f, sin1 = 0.0f;
    if (lane < pairs) {
        const float t = turns((int64_t)first + i, a.freq[lane]);
        sincospif(2.0f * t, &sin1, &cos1);
        cos1 *= a.magnitude;
        sin1 *= a.magnitude;
    }
    const int unit = lane % kUnits;
    const bool turned = unit < a.part / 16;
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int f = turned ? unit * 8 + j : 0;
        c[j] = __shfl(cos1, f);
        s[j] = __shfl(sin1, f);
    }
    // the two pieces of eight channels
    const int at0 = turned && !PAIRS ? unit * 8 : unit * 16;
    const int at1 = turned && !PAIRS ? pairs + unit * 8 : unit * 16 + 8;
    const int heads = a.Hq + a.Hkv;
    const size_t row = (size_t)r0 + i;
    for (int head = lane / kUnits + (SPLIT ? wave * kHeads : 0); head < heads;
         head += SPLIT ? 4 * kHeads : kHeads) {
        const bool key = head >= a.Hq;
        const size_t off = (size_t)(key ? head - a.Hq : head) * D;
        const uint16_t* from = key ? a.K + row * a.ldk + off : a.Q + row * a.ldq + off;
        uint16_t* to = key ? a.Ko + row * a.ldko + off : a.Qo + row * a.ldqo + off;
        if (!turned && from == to) continue;
        const uint4 u = *reinterpret_cast<const uint4*>(from + at0);
        const uint4 v = *reinterpret_cast<const uint4*>(from + at1);
        uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
        if (turned) {
            float p[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[2 * j] = __uint_as_float(x[j] << 16);
                p[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
                p[8 + 2 * j] = __uint_as_float(y[j] << 16);
                p[8 + 2 * j + 1] = __uint_as_float(y[j] & 0xFFFF0000u);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float& e = p[PAIRS ? 2 * j : j];
                float& f = p[PAIRS ? 2 * j + 1 : 8 + j];
                const float e1 = fmaf(e, c[j], -(f * s[j])), f1 = fmaf(f, c[j], e * s[j]);
                e = e1;
                f = f1;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
                y[j] = pack_bf16(p[8 + 2 * j], p[8 + 2 * j + 1]);
            }
        }
        *reinterpret_cast<uint4*>(to + at0) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4*>(to + at1) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

template <int D, bool PAIRS>
hipError_t launch(const Rotary& a, int B, hipStream_t stream) {
    // single tokens: a row's heads over four waves
    if (a.max_rows < 4)
        rotary_kernel<D, PAIRS, true><<<dim3(a.max_rows, B), 256, 0, stream>>>(a);
    else
        rotary_kernel<D, PAIRS, false><<<dim3((a.max_rows + 3) / 4, B), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const uint16_t* Q, const uint16_t* K, const int32_t* row_start,
                         const int32_t* pos, const double* freq, float magnitude, int B, int T,
                         int max_rows, int Hq, int Hkv, int D, int rotary_dim, int layout, int ldq,
                         int ldk, int ldqo, int ldko, uint16_t* Qo, uint16_t* Ko,
                         hipStream_t stream) {
    Rotary a = {};
    a.Q = Q;
    a.K = K;
    a.row_start = row_start;
    a.pos = pos;
    a.freq = freq;
    a.magnitude = magnitude;
    a.T = T;
    a.max_rows = max_rows < T ? max_rows : T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.part = rotary_dim;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldqo = ldqo;
    a.ldko = ldko;
    a.Qo = Qo;
    a.Ko = Ko;
    const bool pairs = layout == RUDDER_ROTARY_PAIRS;
    if (D == 64) return pairs ? launch<64, true>(a, B, stream) : launch<64, false>(a, B, stream);
    return pairs ? launch<128, true>(a, B, stream) : launch<128, false>(a, B, stream);
}

}  // namespace rudder
