// Rotary positions: pairs of channels (x, y) of the query and key heads are
// turned by an angle that grows with the row's position,
//   x' = x c - y s,  y' = y c + x s,  c, s = magnitude * cos, sin(position * freq[i]).
//
// The angle is formed in turns, as the sum of two 64-bit numbers: the product
// position * freq and its rounding error, times 1 / (2 pi) in two parts.  What
// is left of it behind the whole turns is at most 3/4 and right to 2^-50 for
// every int32 position and frequencies of up to 2^24, and is rounded to 32 bits
// only then (2^-25 turns).
#include "rudder_block_launch.h"
#include "rudder_device.h"

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

// A pair in one word, turned.
__device__ __forceinline__ uint32_t turn(uint32_t w, float c, float s) {
    const float x = low(w), y = high(w);
    return pack_bf16(fmaf(x, c, -(y * s)), fmaf(y, c, x * s));
}

// position * freq in turns, at most 3/4 in magnitude
__device__ __forceinline__ float turns(int64_t position, double freq) {
    constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;   // 1 / (2 pi)
    const double p = (double)position, a = p * freq, da = __builtin_fma(p, freq, -a);
    const double t = a * kHigh;
    const double dt = __builtin_fma(a, kHigh, -t) + (a * kLow + da * kHigh);
    return (float)((t - __builtin_rint(t)) + dt);
}

// A wave takes a row (or, with SPLIT, four waves a quarter of its heads each); a lane 16 channels of
// every fourth or eighth head.  A row's cosines and sines are formed once, one a lane.  Bound by memory:
// 8384 rows of 32 heads of 128 channels move 137 MB at 5.9 TB/s; 48 single tokens of 40 heads 3.3 us,
// a launch and the way from lengths to rows to outputs.
template <int D, bool PAIRS, bool SPLIT, bool TURNS>
__global__ void __launch_bounds__(256) rotary_kernel(const Rotary a) {
    constexpr int kUnits = D / 16, kHeads = 64 / kUnits;   // lanes a head, heads a wave
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int b = blockIdx.y;
    const int r0 = min(max(a.row_start[b], 0), a.T);
    const int n = min(min(max(a.row_start[b + 1], r0), a.T) - r0, a.max_rows);
    int i = SPLIT ? blockIdx.x : blockIdx.x * 4 + wave;
    const int first = a.pos ? a.pos[b] : 0;
    if (i >= n || first < 0) return;

    do {
        // lane f's cosine and sine, then those of this lane's eight pairs
        const int pairs = a.part / 2;
        float cos1 = 1.0f, sin1 = 0.0f;
        if (lane < pairs) {
            const float t = turns((int64_t)first + i, a.freq[lane]);
            sincospif(2.0f * t, &sin1, &cos1);
            cos1 *= a.magnitude;
            sin1 *= a.magnitude;
        }
        // two pieces of eight channels: with halves a pair's two in the rotated part, else one in each
        // half of the head, so that neighbours' pieces follow each other
        const int unit = lane % kUnits;
        const bool both = !PAIRS && unit < a.part / 16;
        const int at0 = !PAIRS && !both ? unit * 16 : unit * 8;
        const int at1 = both ? pairs + unit * 8 : PAIRS ? D / 2 + unit * 8 : unit * 16 + 8;
        const bool turned0 = PAIRS ? at0 < a.part : both, turned1 = PAIRS ? at1 < a.part : both;
        float c[8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // PAIRS: four of the first piece, four of the second; 0 where nothing is rotated
            const int f = PAIRS ? (j < 4 ? (turned0 ? at0 / 2 + j : 0) : (turned1 ? at1 / 2 + j - 4 : 0))
                                : (both ? unit * 8 + j : 0);
            c[j] = __shfl(cos1, f);
            s[j] = __shfl(sin1, f);
        }
        const int heads = a.Hq + a.Hkv;
        const size_t row = (size_t)r0 + i;
        for (int head = lane / kUnits + (SPLIT ? wave * kHeads : 0); head < heads;
             head += SPLIT ? 4 * kHeads : kHeads) {
            const bool key = head >= a.Hq;
            const size_t off = (size_t)(key ? head - a.Hq : head) * D;
            const uint16_t* from = key ? a.K + row * a.ldk + off : a.Q + row * a.ldq + off;
            uint16_t* to = key ? a.Ko + row * a.ldko + off : a.Qo + row * a.ldqo + off;
            if (!turned0 && !turned1 && from == to) continue;
            const uint4 u = *reinterpret_cast<const uint4*>(from + at0);
            const uint4 v = *reinterpret_cast<const uint4*>(from + at1);
            uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
            if constexpr (PAIRS) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t p = turn(x[j], c[j], s[j]), q = turn(y[j], c[4 + j], s[4 + j]);
                    x[j] = turned0 ? p : x[j];
                    y[j] = turned1 ? q : y[j];
                }
            } else if (both) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e0 = low(x[j]), e1 = high(x[j]), f0 = low(y[j]), f1 = high(y[j]);
                    const float c0 = c[2 * j], c1 = c[2 * j + 1], s0 = s[2 * j], s1 = s[2 * j + 1];
                    x[j] = pack_bf16(fmaf(e0, c0, -(f0 * s0)), fmaf(e1, c1, -(f1 * s1)));
                    y[j] = pack_bf16(fmaf(f0, c0, e0 * s0), fmaf(f1, c1, e1 * s1));
                }
            }
            // past the caches: into buffers of their own 8384 rows of 32 heads of 128 channels 23.7 us,
            // through the caches 31; in place, behind the linear that wrote them and in front of
            // attention or an append, the same
            stream16(to + at0, make_uint4(x[0], x[1], x[2], x[3]));
            stream16(to + at1, make_uint4(y[0], y[1], y[2], y[3]));
        }
        i += gridDim.x * 4;
    } while (TURNS && i < n);
}

// Workgroups of a launch.  Where the bound on the rows asks for more, they take several turns, so that a
// bound far above the sequences' lengths costs little; the loop around the rows costs 1% elsewhere (8384
// rows of 32 heads 23.7 us against 23.4).
constexpr int kMostGroups = 1 << 20;

template <int D, bool PAIRS>
hipError_t launch(const Rotary& a, int B, hipStream_t stream) {
    const int groups = (a.max_rows + 3) / 4, most = kMostGroups / B;
    if (a.max_rows < 4)                            // single tokens: a row's heads over four waves
        rotary_kernel<D, PAIRS, true, false><<<dim3(a.max_rows, B), 256, 0, stream>>>(a);
    else if (groups <= most)
        rotary_kernel<D, PAIRS, false, false><<<dim3(groups, B), 256, 0, stream>>>(a);
    else
        rotary_kernel<D, PAIRS, false, true><<<dim3(most, B), 256, 0, stream>>>(a);
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
