// Causal attention of whole prompts, packed one behind the other, to their own
// bf16 keys and values.
//
//   o[t][h] = sum_{j <= t} softmax_j(sm * q[t][h] . k[j][h']) * v[j][h'],  h' = h / (Hq / Hkv)
//
// One pass over the keys with the running maximum and sum l of the softmax, in
// base 2: weights are exp2(c * z_j - maximum), z_j = q . k_j, c = sm * log2(e).  Both products are formed
// transposed, so that a query is a column of every matrix and a lane keeps one
// query's numbers: the accumulators of Z^T = K Q^T, packed in pairs, are the
// operand of O^T = V^T P^T, provided that the keys of V^T are stored in their
// order.  With 32x32x16 products a lane of half h = lane / 32 holds keys
// 8 * (j / 4) + 4 * h + j % 4, j = 0..15, of a block of 32.
//
// Weights P are held in fp16 (2^-11 relative; times 2^9, so that weights down to
// 2^-22 of the largest keep all of their bits), values in fp16 as well: a
// tile's values, times a power of two that brings their largest magnitude into
// [2^7, 2^15), are exact in fp16 down to 2^-24 of that magnitude and off by at
// most 2^-32 of it below.  The power is a multiple of 8, so that tiles of like
// values share one; where one differs, a row's O is brought to it in 32 bits
// (see follow()), so that no tile's values or weights lose bits to another's.
// A tile that a row sees only part of, whose tokens are of very different sizes,
// takes a slow way (uneven_values()): nothing behind a row takes bits from it.
#include <cmath>
#include <type_traits>

#include "rudder_block_launch.h"
#include "rudder_device.h"

namespace rudder {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_acc __attribute__((ext_vector_type(16)));

// Lambdas that hold registers of the kernel around them: a call would put those into memory.
#define RUDDER_INLINE __attribute__((always_inline))

constexpr int kTile = 64;                          // keys
constexpr int kWaveRows = 32;                      // query rows a wave
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 9.0f;                    // P and its sums are held times 2^9
// The running maximum is raised only where a score passes it by more than 2^6: P stays below 2^15.
constexpr float kMostP = kPShift + 6.0f;
// Weights of at most 2^-26 are zeros in fp16, whatever the exponential's last bits.
constexpr float kNothing = -26.0f;
// Of a row that has seen no score above -inf: any one is above its maximum.
constexpr float kUnset = 3e38f;
// Maxima below this magnitude are kept as whole numbers in base 2, exact in 32 bits, others as the score
// itself.
constexpr float kFar = 4194304.0f;
// O is brought to a larger power of two up to this size: further sums are far from 32 bits' end.
constexpr int kRoom = 96;

struct Prompt {
    const uint16_t *Q, *K, *V;
    const int32_t* row_start;
    int T, max_rows, G, Hkv, tile_rows;
    int dies, die_pairs, group;                    // order of the work units, see place_unit()
    size_t ldq, ldk, ldv, ldo;
    float sm;
    uint16_t* O;
    // of the kernel for many rows: transposed values in fp16, [slot][head][image of a tile], and
    // what else it has to know of a tile, [head][slot]
    uint8_t* images;
    int32_t* notes;
    int slots;
};

__device__ __forceinline__ f32x16_acc mma_bf16(uint4 a, uint4 b, f32x16_acc c) {
    union { uint4 u; bf16x8_t v; } x, y;
    x.u = a;
    y.u = b;
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.v, y.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_acc mma_f16(uint4 a, uint4 b, f32x16_acc c) {
    union { uint4 u; f16x8_t v; } x, y;
    x.u = a;
    y.u = b;
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(x.v, y.v, c, 0, 0, 0);
}

// Unit number -> (key head, sequence) pair and row tile.  Workgroups go round robin to the eight
// dies: where the pairs divide by eight, the units of a pair, which read the same keys, are kept on
// one (dies = 8, else 1).  A die's pairs are taken `group` at a time, the units of a group longest
// first over all its pairs, whose order turns by one from length to length: workgroups go round robin
// to the parts of a die too, and without the turn the longest of four prompts has a quarter of it
// (twelve prompts up to 4801 tokens 1749 us, in turn 832).
struct Unit {
    int b, h, tile;
};
__device__ __forceinline__ Unit place_unit(const Prompt& p) {
    const int slot = quotient(blockIdx.x, p.dies), low = blockIdx.x - slot * p.dies;
    const int g = quotient(slot, p.group * p.tile_rows), i = slot - g * (p.group * p.tile_rows);
    const int size = min(p.group, p.die_pairs - g * p.group);      // the last group may be smaller
    const int up = quotient(i, size);
    const int of = i - up * size + up, r = of - quotient(of, size) * size;
    const int pair = low + p.dies * (g * p.group + r);
    const int b = quotient(pair, p.Hkv);
    return {b, pair - b * p.Hkv, p.tile_rows - 1 - up};
}

// Two fp16 numbers a word, times a power of two.
__device__ __forceinline__ uint4 times(uint4 x, float f) {
    union { uint32_t u[4]; f16x2_t h[4]; } r;
    r.u[0] = x.x;
    r.u[1] = x.y;
    r.u[2] = x.z;
    r.u[3] = x.w;
    const f16x2_t g = {(_Float16)f, (_Float16)f};
#pragma unroll
    for (int i = 0; i < 4; ++i) r.h[i] *= g;
    return make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
}

// Largest magnitude bits of eight bf16 values.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2_t top_of(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    union { uint32_t u; u16x2_t v; } a;
    u16x2_t top = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a.u = w[j] & 0x7FFF7FFFu;
        top = __builtin_elementwise_max(top, a.v);
    }
    return top;
}

// Which four keys (of 16 such) and eight channels of a tile's values a thread takes: a wave 64 bytes
// of every row, so that its transposed writes go to whole lines and to different banks.
__device__ __forceinline__ int value_keys(int tid) { return tid / 4 % 16; }
__device__ __forceinline__ int value_channels(int tid) { return tid % 4 + tid / 64 * 4; }

// N times four rows of eight bf16 values: those that are not finite made zero; `bad` becomes the first
// such row (of four) where it is below.  Returns the largest magnitude bits of the others, `tops` each
// row's.
template <int N>
__device__ __forceinline__ uint32_t finite_top(uint4 (&x)[N][4], int& bad, uint32_t (&tops)[4]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u16x2_t most = {0, 0};
#pragma unroll
        for (int n = 0; n < N; ++n) most = __builtin_elementwise_max(most, top_of(x[n][i]));
        tops[i] = max((uint32_t)most[0], (uint32_t)most[1]);
        top = max(top, tops[i]);
    }
    if (!__any(top >= 0x7F80u)) return top;
    top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) tops[i] = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4] = {x[n][i].x, x[n][i].y, x[n][i].z, x[n][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = w[j] & 0x7FFFu, b = w[j] >> 16 & 0x7FFFu;
                const bool low = a >= 0x7F80u, high = b >= 0x7F80u;
                if (low || high) bad = min(bad, i);
                w[j] &= (low ? 0u : 0xFFFFu) | (high ? 0u : 0xFFFF0000u);
                tops[i] = max(tops[i], max(low ? 0u : a, high ? 0u : b));
            }
            x[n][i] = make_uint4(w[0], w[1], w[2], w[3]);
            top = max(top, tops[i]);
        }
    return top;
}

// Whether a token's largest magnitude is less than 2^-8 of the tile's: a row that sees the one and not the
// other would lose more than 2^-24 of it to the tile's power of two, or, where it is 0, bits of what
// it has summed.
__device__ __forceinline__ bool uneven(uint32_t token, uint32_t tile) {
    return token + (8 << 7) < tile;
}
// The largest of four neighbouring lanes, which hold 32 channels of a token.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 15, 15, true));   // 1 0 3 2
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 15, 15, true));  // 2 3 0 1
}

// Chunks of 16 bytes of an LDS row are exchanged so that 16 lanes reading one chunk of 16 rows find
// 16 places of the 64 banks.
template <int CHUNKS>
__device__ __forceinline__ int place(int row, int chunk) {
    return (row * CHUNKS + (chunk ^ (CHUNKS == 16 ? row & 15 : row >> 1 & 7))) * 16;
}

// A tile's image: values as the second product's operand, [channel][key].  Four keys (rows of x) x
// eight channels, times f, to their places.
__device__ __forceinline__ void store_values(uint8_t* image, const uint4 (&x)[4], float f, int quad,
                                             int chunk) {
    // keys 4 quad .. + 3 are the accumulators' order with bits 0 and 1 of quad exchanged
    const int to = (quad & ~3) | (quad & 1) << 1 | (quad >> 1 & 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a[4], e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = j == 0 ? x[i].x : j == 1 ? x[i].y : j == 2 ? x[i].z : x[i].w;
            a[i] = __uint_as_float(w << 16) * f;
            e[i] = __uint_as_float(w & 0xFFFF0000u) * f;
        }
        const int ch = chunk * 8 + 2 * j;
        *reinterpret_cast<uint2*>(image + place<8>(ch, to >> 1) + (to & 1) * 8) =
            make_uint2(pack_f16(a[0], a[1]), pack_f16(a[2], a[3]));
        *reinterpret_cast<uint2*>(image + place<8>(ch + 1, to >> 1) + (to & 1) * 8) =
            make_uint2(pack_f16(e[0], e[1]), pack_f16(e[2], e[3]));
    }
}

// The multiple of 8 that brings a largest magnitude of these bits into [2^7, 2^15); at most 120, so
// that 2^s is a number.  A tile of zeros takes that: it must not lower the others'.
__device__ __forceinline__ int scale_of(uint32_t top) {
    const int e = (int)(top >> 7) - 127;
    return top ? min((14 - e) & ~7, 120) : 120;
}

// A row's O, held times 2^scale by the row's two lanes, for a tile whose values are times 2^s: returns
// the power of two by which this tile's weights have to be smaller.  That is 0 but for a row whose O would
// not stay below 2^kRoom times 2^s; there the weights' lost bits are beneath O's own.  A row to which the
// tile adds nothing (`counts` false) keeps its scale, however large the values.
template <int DT>
__device__ __forceinline__ int follow(f32x16_acc (&o)[DT], int& scale, int s, bool counts) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(o[i][j]));
    top = fmaxf(top, __shfl_xor(top, 32));
    const int room = top > 0.0f ? max(kRoom + 127 - (int)(__float_as_uint(top) >> 23), 0) : 1 << 20;
    const int by = counts ? min(s - scale, room) : 0;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = __builtin_amdgcn_ldexpf(o[i][j], max(by, -300));
    scale += by;
    return counts ? s - scale : 0;
}

// 32 values of a tile that a row sees only part of, and that are uneven: straight from memory, in bf16,
// with every row at the power of two of those that it weighs, so that nothing behind a row takes bits from
// it, nor what it sees and does not weigh.  The fp16 weights w (16 keys each) are sums of two bf16 numbers;
// a key's power of two goes from its values to its weights.  `v`: the first key's channels; `there`: how
// many of the keys there are.
// Rare, and slow (two-byte loads, twice the products): where every tile is such a one, 77 tokens 16.0 us
// against 9.4, 2 x 4192 207 against 175.
template <int D>
__device__ __forceinline__ void uneven_values(f32x16_acc (&o)[D / 32], int& scale,
                                              const uint16_t* v, size_t ldv, int there, uint4 w0,
                                              uint4 w1) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane), "+s"(ldv));      // keeps the addresses out of the loop around this
    const int half = lane >> 5;
    auto of_lane = [](int from, int x) { return __builtin_amdgcn_ds_bpermute(from * 4, x); };
    int top = 0;                                   // a key a lane: its largest magnitude
    if ((lane & 31) < there) {
        const uint4* row = reinterpret_cast<const uint4*>(v + (size_t)(lane & 31) * ldv + half * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint4 x = row[i];
            const uint32_t word[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int a = word[j] & 0x7FFFu, b = word[j] >> 16 & 0x7FFFu;
                top = max(top, max(a >= 0x7F80 ? 0 : a, b >= 0x7F80 ? 0 : b));
            }
        }
    }
    top = max(top, of_lane(lane ^ 32, top));
    // the lane's two keys of word j of weights x, and the largest that its row weighs
    auto key_of = [&](int x, int j) { return 16 * x + 8 * (j >> 1) + 4 * half + 2 * (j & 1); };
    int most = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 w = i < 4 ? w0 : w1;
        const uint32_t word = i % 4 == 0 ? w.x : i % 4 == 1 ? w.y : i % 4 == 2 ? w.z : w.w;
        const int t0 = of_lane(key_of(i / 4, i % 4), top), t1 = of_lane(key_of(i / 4, i % 4) + 1, top);
        most = max(most, max(word & 0xFFFFu ? t0 : -1, word >> 16 ? t1 : -1));
    }
    most = max(most, of_lane(lane ^ 32, most));
    follow(o, scale, scale_of(max(most, 0)), most >= 0);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const uint4 w = x ? w1 : w0;
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
        uint32_t upper[4], lower[4], y[D / 32][4];             // two keys a word
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            __builtin_amdgcn_sched_barrier(0);     // few loads at a time: registers are full
            const int key = key_of(x, j);
            const int power0 = min(max((of_lane(key, top) >> 7) - 127, -120), 120);
            const int power1 = min(max((of_lane(key + 1, top) >> 7) - 127, -120), 120);
            union { uint32_t u; f16x2_t h; } p;
            p.u = word[j];
            const float e0 = __builtin_amdgcn_ldexpf((float)p.h[0], scale + power0);
            const float e1 = __builtin_amdgcn_ldexpf((float)p.h[1], scale + power1);
            upper[j] = pack_bf16(e0, e1);
            lower[j] = pack_bf16(e0 - __uint_as_float(upper[j] << 16),
                                 e1 - __uint_as_float(upper[j] & 0xFFFF0000u));
            const uint16_t* from0 = v + (size_t)min(key, there - 1) * ldv + (lane & 31);
            const uint16_t* from1 = v + (size_t)min(key + 1, there - 1) * ldv + (lane & 31);
            const float f0 = __uint_as_float((uint32_t)(127 - power0) << 23);
            const float f1 = __uint_as_float((uint32_t)(127 - power1) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t b0 = from0[i * 32], b1 = from1[i * 32];
                const bool good0 = key < there && (b0 & 0x7FFFu) < 0x7F80u;
                const bool good1 = key + 1 < there && (b1 & 0x7FFFu) < 0x7F80u;
                y[i][j] = pack_bf16(good0 ? __uint_as_float(b0 << 16) * f0 : 0.0f,
                                    good1 ? __uint_as_float(b1 << 16) * f1 : 0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 z = make_uint4(y[i][0], y[i][1], y[i][2], y[i][3]);
            o[i] = mma_bf16(z, make_uint4(upper[0], upper[1], upper[2], upper[3]), o[i]);
            o[i] = mma_bf16(z, make_uint4(lower[0], lower[1], lower[2], lower[3]), o[i]);
        }
    }
}

// What a row's weights are relative to: P = exp2(c (z - a) + b).  Near zero a is 0 and b a whole number,
// so that a new maximum is a power of two on all that was summed; far from it, where c z and a number
// beside it have no bits left for b, a is the largest score and the difference is taken first.
struct Reference {
    float a, b;
    // log2 of P for a score
    __device__ __forceinline__ float exponent(float c, float z) const { return fmaf(c, z - a, b); }
    // log2 of what turns weights relative to this into weights relative to another
    __device__ __forceinline__ float to(float c, const Reference& other) const {
        return fmaf(c, a - other.a, other.b - b);
    }
};
// The reference for a largest score of z.
__device__ __forceinline__ Reference reference(float c, float z) {
    const float t = c * z;
    return fabsf(t) < kFar ? Reference{0.0f, kPShift - ceilf(t)} : Reference{z, kPShift};
}

// ---------------------------------------------------------------------------
// Few rows: 32 of them a workgroup, a tile of keys a wave.
// ---------------------------------------------------------------------------
// Short prompts are a matter of latency: no launch goes in front, keys come from memory straight to
// registers as the first product's operand, every wave turns the values of its own tiles to fp16 and
// transposes them through its own part of LDS, and the four waves meet once, at the end.  One workgroup
// a compute unit, two of 64 channels (2 x 256 rows of 24 heads 8.6 us, one 12.1; three spill): a wave's
// keys and values on their way take half of its registers.  16 heads of 128
// channels, one token 7.7 us, 77 8.8, 200 10.4; with 128 rows a workgroup and a tile after the other
// 7.1, 10.7 and 15.4.  The next tile's keys are asked for as soon as the products have read these, its
// values once the registers are free of the last ones (both at once: 600 tokens 20.0 us against 18.9).
// What is left is the way from lengths to rows (two trips to memory), code that is met cold, and a tile's
// 960 vector instructions: waves wait for 64% of their time at 77 tokens, for 70% at one.
template <int D>
__global__ void __launch_bounds__(256, D == 64 ? 2 : 1) prompt_few_kernel(const Prompt p) {
    constexpr int kKS = D / 16, kDT = D / 32, kIts = D / 32, kBytes = kTile * D * 2;
    constexpr int kWaves = 4, kStride = D + 4;     // of a row of partial outputs, in floats
    __shared__ __align__(16) uint8_t lds[kWaves * (kBytes > kWaveRows * kStride * 4
                                                       ? kBytes : kWaveRows * kStride * 4)];
    __shared__ Reference refs[kWaves][kWaveRows];  // what a row's weights are relative to, ...
    __shared__ float sums[kWaves][kWaveRows];      // ... their sum ...
    __shared__ int scales[kWaves][kWaveRows];      // ... and the power of two of its outputs
    __shared__ int first_bads[kWaves];

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Unit unit = place_unit(p);
    const int b = unit.b, h = unit.h, row0 = unit.tile * kWaveRows;
    const int r0 = min(max(p.row_start[b], 0), p.T);
    const int n = min(min(max(p.row_start[b + 1], r0), p.T) - r0, p.max_rows);
    const int rows = n * p.G;
    if (row0 >= rows) return;

    const int row = row0 + (lane & 31);
    const bool live = row < rows;
    const int t = live ? row / p.G : 0, head = h * p.G + (live ? row % p.G : 0);
    const int limit = live ? t + 1 : 0;            // keys this lane's row sees
    const int least = quotient(row0, p.G) + 1;     // every row sees these
    const int most = quotient(min(rows, row0 + kWaveRows) - 1, p.G) + 1;
    const int tiles = (most + kTile - 1) / kTile;

    uint4 k[2][kKS], x[kIts][4];
    // rows behind the prompt are its last one again: no row sees the keys, and the values are made
    // zero below
    auto load_keys = [&](int tile) RUDDER_INLINE {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const size_t r = (size_t)min(r0 + tile * kTile + kb * 32 + (lane & 31), r0 + n - 1);
            const uint16_t* from = p.K + r * p.ldk + (size_t)h * D + half * 8;
#pragma unroll
            for (int i = 0; i < kKS; ++i)
                k[kb][i] = *reinterpret_cast<const uint4*>(from + i * 16);
        }
    };
    auto load_values = [&](int tile) RUDDER_INLINE {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const size_t r = (size_t)min(r0 + tile * kTile + value_keys(lane) * 4 + i, r0 + n - 1);
#pragma unroll
            for (int it = 0; it < kIts; ++it)
                x[it][i] = *reinterpret_cast<const uint4*>(
                    p.V + r * p.ldv + (size_t)h * D + value_channels(lane + it * 64) * 8);
        }
    };
    uint4 q[kKS];
    {
        const uint16_t* from = p.Q + (size_t)(r0 + t) * p.ldq + (size_t)head * D + half * 8;
#pragma unroll
        for (int i = 0; i < kKS; ++i) q[i] = *reinterpret_cast<const uint4*>(from + i * 16);
    }
    if (wave < tiles) {
        load_keys(wave);
        load_values(wave);
    }
    float l = 0.0f, c = fabsf(p.sm) * kLog2e;
    {
        u16x2_t most = {0, 0};
#pragma unroll
        for (int i = 0; i < kKS; ++i) most = __builtin_elementwise_max(most, top_of(q[i]));
        const uint32_t top = max((uint32_t)most[0], (uint32_t)most[1]);
        if (__any(top >= 0x7F80u)) {               // not finite
            if (max(top, (uint32_t)__shfl_xor((int)top, 32)) >= 0x7F80u)
                l = __uint_as_float(0x7FC00000u);
        }
        if (p.sm < 0.0f) {
#pragma unroll
            for (int i = 0; i < kKS; ++i)
                q[i] = make_uint4(q[i].x ^ 0x80008000u, q[i].y ^ 0x80008000u, q[i].z ^ 0x80008000u,
                                  q[i].w ^ 0x80008000u);
        }
        if (c == 0.0f) {                           // all keys alike, however large the scores
#pragma unroll
            for (int i = 0; i < kKS; ++i) q[i] = make_uint4(0, 0, 0, 0);
            c = 1.0f;
        }
    }

    f32x16_acc o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    Reference ref = {0.0f, kUnset};
    bool far = false;                              // of a row of the wave
    int scale = 0, first_bad = 1 << 30;            // O of the lane's row is held times 2^scale
    uint8_t* values = lds + wave * kBytes;
    uint4 w[4];
    int uneven_at = -1;
    for (int tile = wave; tile < tiles; tile += kWaves) {
        const int at = tile * kTile;
        f32x16_acc z[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[kb][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < kKS; ++i) z[kb] = mma_bf16(k[kb][i], q[i], z[kb]);
        }
        if (tile + kWaves < tiles) load_keys(tile + kWaves);
        // the values
        if (at + kTile > n) {                      // the prompt ends in this tile
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t there = at + value_keys(lane) * 4 + i < n ? ~0u : 0u;
#pragma unroll
                for (int it = 0; it < kIts; ++it)
                    x[it][i] = make_uint4(x[it][i].x & there, x[it][i].y & there,
                                          x[it][i].z & there, x[it][i].w & there);
            }
        }
        int bad = 4;
        uint32_t tops[4], top = finite_top(x, bad, tops);
        bad = bad < 4 ? value_keys(lane) * 4 + bad : kTile;
#pragma unroll
        for (int off = 32; off; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
        if (__any(bad < kTile)) {
#pragma unroll
            for (int off = 32; off; off >>= 1) bad = min(bad, __shfl_xor(bad, off));
            first_bad = min(first_bad, at + bad);
        }
        const int s = __builtin_amdgcn_readfirstlane(scale_of(top));
        const bool part = at + kTile > least;      // some rows see only part of the tile
        bool apart = false;
        if (part) {                                // four lanes hold a token's channels
            bool any = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                any |= uneven(quad_max(tops[i]), top) && at + value_keys(lane) * 4 + i < n;
            apart = __any(any);
        }
        const float f = __uint_as_float((uint32_t)(127 + s) << 23);
#pragma unroll
        for (int it = 0; it < kIts; ++it)
            store_values(values, x[it], f, value_keys(lane), value_channels(lane + it * 64));
        // the weights
        if (part) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (at + 32 * kb + 8 * (j >> 2) + 4 * half + (j & 3) >= limit)
                        z[kb][j] = -INFINITY;
        }
        float best = z[0][0];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int j = 0; j < 16; ++j) best = fmaxf(best, z[kb][j]);
        best = fmaxf(best, __shfl_xor(best, 32));
        const bool raised = ref.exponent(c, best) > kPShift;
        if (__any(raised)) {
            const Reference now = raised ? reference(c, best) : ref;
            if (tile >= kWaves) {                  // O is more than nothing
                const float alpha = __builtin_amdgcn_exp2f(ref.to(c, now));
                l *= alpha;
#pragma unroll
                for (int i = 0; i < kDT; ++i) o[i] *= alpha;
            }
            ref = now;
            far = __any(ref.a != 0.0f);
        }
        int above = 0;
        if (tile < kWaves)
            scale = s;
        else if (!apart && __any(scale != s && at < limit))
            above = follow(o, scale, s, ref.exponent(c, best) > kNothing);
        if (far) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < 16; ++j) z[kb][j] -= ref.a;
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at_z = (ks & 1) * 8 + 2 * j;
                const float a = __builtin_amdgcn_exp2f(fmaf(c, z[ks >> 1][at_z], ref.b));
                const float e = __builtin_amdgcn_exp2f(fmaf(c, z[ks >> 1][at_z + 1], ref.b));
                l += a + e;
                y[j] = pack_f16(a, e);
            }
            w[ks] = make_uint4(y[0], y[1], y[2], y[3]);
        }
        if (__any(above)) {
            const float down = __builtin_amdgcn_ldexpf(1.0f, -above);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) w[ks] = times(w[ks], down);
        }
        if (apart) {                               // the wave's last tile: no row sees one four on
            uneven_at = at;
            break;
        }
        wave_sync();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int i = 0; i < kDT; ++i)
                o[i] = mma_f16(*reinterpret_cast<const uint4*>(
                                   values + place<8>(i * 32 + (lane & 31), 2 * ks + half)),
                               w[ks], o[i]);
        wave_sync();
        if (tile + kWaves < tiles) load_values(tile + kWaves);
    }
    if (uneven_at >= 0) {
#pragma unroll 1
        for (int key = uneven_at; key < min(uneven_at + kTile, n); key += 32) {
            uneven_values<D>(o, scale, p.V + (size_t)(r0 + key) * p.ldv + (size_t)h * D, p.ldv,
                             n - key, w[0], w[1]);
            w[0] = w[2];
            w[1] = w[3];
        }
    }
    // the waves' results side by side
    l += __shfl_xor(l, 32);
    __syncthreads();                               // the values have been read
    if (half == 0) {
        refs[wave][lane] = ref;
        sums[wave][lane] = l;
        scales[wave][lane] = scale;
    }
    if (lane == 0) first_bads[wave] = first_bad;
    float* part = reinterpret_cast<float*>(lds) + wave * kWaveRows * kStride;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<float4*>(part + (lane & 31) * kStride + i * 32 + g * 8 + half * 4) =
                make_float4(o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]);
    __syncthreads();
    // eight channels a thread
    constexpr int kChunks = D / 8;
    for (int i = tid; i < kWaveRows * kChunks; i += 256) {
        const int r = i / kChunks, d = i % kChunks * 8, rr = row0 + r;
        if (rr >= rows) continue;
        const int tt = rr / p.G, hd = h * p.G + rr % p.G;
        Reference best = refs[0][r];               // of the largest score
        float sum = 0.0f, f[kWaves];
        int first = first_bads[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            if (refs[w][r].to(c, best) > 0.0f) best = refs[w][r];
            first = min(first, first_bads[w]);
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            // 0 for a wave that has seen no key of this row, whose sum is 0 (or NaN)
            f[w] = __builtin_amdgcn_exp2f(refs[w][r].to(c, best));
            sum += sums[w][r] * f[w];
        }
        // every row sees itself: a sum of zero is one of scores of -inf alone
        float share = sum > 0.0f ? 1.0f / sum : __uint_as_float(0x7FC00000u);
        if (tt >= first) share = __uint_as_float(0x7FC00000u);     // sees a value that is not finite
        float y[8] = {};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w >= tiles && w > 0) break;        // the wave had no tile
            const float4* from = reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(lds) + (w * kWaveRows + r) * kStride + d);
            const float4 u = from[0], v = from[1];
            const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            const float g = f[w] * share;
            const int e = -scales[w][r];           // a part of its own power of two each
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += __builtin_amdgcn_ldexpf(x[j] * g, e);
        }
        *reinterpret_cast<uint4*>(p.O + (size_t)(r0 + tt) * p.ldo + (size_t)hd * D + d) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                       pack_bf16(y[6], y[7]));
    }
}

constexpr int kUneven = 1 << 15;                   // in a tile's note

// A prompt's tiles are kept at slots of their own: floor((r0 + n) / 64) + 1 >= floor(r0 / 64) +
// ceil(n / 64), so that those of sequence b end before those of b + 1 begin.
__device__ __forceinline__ int first_slot(int r0, int b) { return r0 / kTile + b; }

// ---------------------------------------------------------------------------
// Values for the kernel of many rows: transposed, in fp16, times a tile's power of two, laid out as
// that kernel keeps them in LDS.  One tile and head a workgroup.  Bound by memory: 8384 tokens of 16
// heads of 128 channels 14 us, 68 MB read and written at 4.9 TB/s.  Converting in the kernel itself would
// repeat it for every 128 rows; weights in bf16, which need no conversion, put as much error into the
// outputs as their own rounding does.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) prompt_values_kernel(const Prompt p) {
    constexpr int kChunks = D / 8, kVThreads = 16 * kChunks;
    __shared__ uint32_t tops[4], tokens[4][kTile];
    __shared__ int first_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.z, h = blockIdx.y, at = blockIdx.x * kTile;
    const int r0 = min(max(p.row_start[b], 0), p.T);
    const int n = min(min(max(p.row_start[b + 1], r0), p.T) - r0, p.max_rows);
    if (at >= n) return;
    if (tid == 0) first_bad = kTile;
    __syncthreads();
    const int quad = value_keys(tid), chunk = value_channels(tid);
    uint4 x[1][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = at + quad * 4 + i;
        x[0][i] = make_uint4(0, 0, 0, 0);
        if (tid < kVThreads && key < n)
            x[0][i] = *reinterpret_cast<const uint4*>(p.V + (size_t)(r0 + key) * p.ldv +
                                                      (size_t)h * D + chunk * 8);
    }
    int bad = 4;
    uint32_t shares[4], top = finite_top(x, bad, shares);
    if (bad < 4) atomicMin(&first_bad, quad * 4 + bad);
    uint32_t token = 0;                            // four lanes' tokens, one a lane
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t share = quad_max(shares[i]);
        token = (lane & 3) == i ? share : token;
    }
    tokens[wave][lane] = token;
#pragma unroll
    for (int off = 32; off; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const int s = scale_of(top);
    const int slot = first_slot(r0, b) + (int)blockIdx.x;
    if (wave == 0) {                               // a token a lane
        token = max(max(tokens[0][lane], tokens[1][lane]), max(tokens[2][lane], tokens[3][lane]));
        const int apart = __any(uneven(token, top) && at + lane < n) ? kUneven : 0;
        if (lane == 0)
            p.notes[(size_t)h * p.slots + slot] = s + 128 + (first_bad << 8) + apart;
    }
    if (tid >= kVThreads) return;
    const float f = __uint_as_float((uint32_t)(127 + s) << 23);
    store_values(p.images + ((size_t)slot * p.Hkv + h) * (kTile * D * 2), x[0], f, quad, chunk);
}

// All but the wave's last N loads have landed, its LDS reads are done; then the workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}
// ---------------------------------------------------------------------------
// Many rows: waves of 32 rows that share the tiles in LDS.
// ---------------------------------------------------------------------------
// A software pipeline over halves of tiles: while the weights of 32 keys are formed on the vector
// units, the matrix cores work on the scores of the next 32 and the values of the last 32.
// Tiles come straight to LDS, into rings of RING for keys and values each.  The one barrier of
// tile i stands between its halves: K of i and V of i - 1 have been read then, their places are
// asked for K of i + RING and V of i + RING - 1; K of i + 1 and V of i have landed.
// 32 rows meet 32 keys in D / 8 products of 32 cycles; beside them stand, a lane, 16 exponentials and
// about 60 vector instructions.  16576 tokens of 32 heads (eight key heads) of 128 channels 2025 to
// 2190 us card by card with the launch in front, 1028 to 1112 TFLOP/s, where a library product of 8192^3
// reaches 1208 to 1379: matrix cores busy 57% of the time, vector units 52%, LDS 29%, bank conflicts in
// 1% of its cycles; the card lowers its clock for it (on zeros 1555 us where it takes 2190).  2 x 4192 of
// 16 heads 169 to 181 (matrix cores 46%), twelve prompts up to 4801 of 32 heads 725 to 773 (51%), 3 x
// 1500 of 24 heads of 64 channels 35 (17%, vector units 35%: the longest unit's 24 tiles one after the
// other), 16576 of 32 heads of 64 channels 1215: as many exponentials for half the products, vector units
// busy 80% of the time and matrix cores 49%.  Two phases
// apart with a barrier each, as in the cache's kernel for very many rows, 2304 us; 64 rows a wave, whose
// operands from LDS serve two products, 2360 (one wave a vector unit hides nothing); hints to the
// scheduler 2128 against 2097; a wave's priority raised for its products the same.
template <int D, int WAVES, int RING>
__global__ void __launch_bounds__(WAVES * 64, D == 64 ? 3 : 2) prompt_wide_kernel(const Prompt p) {
    constexpr int kRows = WAVES * kWaveRows, kKS = D / 16, kDT = D / 32, kChunks = D / 8;
    constexpr int kBytes = kTile * D * 2, kLoads = kBytes / 1024 / WAVES;   // a tile's; a wave's of one
    constexpr int kStride = D * 2 + 16;                               // of an output row in LDS
    __shared__ __align__(16) uint8_t lds[2 * RING * kBytes];          // keys, values
    static_assert(WAVES * kWaveRows * kStride <= 2 * RING * kBytes, "outputs pass through the rings");

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Unit unit = place_unit(p);
    const int b = unit.b, h = unit.h, first = unit.tile * kRows;
    const int r0 = min(max(p.row_start[b], 0), p.T);
    const int n = min(min(max(p.row_start[b + 1], r0), p.T) - r0, p.max_rows);
    const int rows = n * p.G;
    if (first >= rows) return;

    const int row0 = first + wave * kWaveRows, row = row0 + (lane & 31);
    const bool live = row < rows;
    const int t = live ? row / p.G : 0, head = h * p.G + (live ? row % p.G : 0);
    const int limit = live ? t + 1 : 0;            // keys this lane's row sees
    const int least = row0 < rows ? quotient(row0, p.G) + 1 : 0;       // every row of the wave sees these
    const int most = row0 < rows ? quotient(min(rows, row0 + kWaveRows) - 1, p.G) + 1 : 0;
    const int last = quotient(min(rows, first + kRows) - 1, p.G) + 1;
    const int tiles = (last + kTile - 1) / kTile;

    // this wave's pieces of a tile; tiles behind the last are the last one again, never read; rows
    // behind the prompt are its last one again
    const int slot0 = first_slot(r0, b);
    const uint32_t base = lds_offset(lds);
    const uint8_t* kp = reinterpret_cast<const uint8_t*>(p.K + (size_t)r0 * p.ldk + (size_t)h * D);
    const uint8_t* vp = p.images + ((size_t)slot0 * p.Hkv + h) * kBytes;
    const int whole = n / kTile;                   // tiles that lie in the prompt
    uint32_t k_from[kLoads], k_end[kLoads];        // in a tile, in the one that ends the prompt
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int key = (wave * kLoads + j) * (64 / kChunks) + lane / kChunks;
        const uint32_t ck = (lane % kChunks ^ (kChunks == 16 ? key & 15 : key >> 1 & 7)) * 16;
        const uint32_t step = (uint32_t)p.ldk * 2;
        k_from[j] = key * step + ck;
        k_end[j] = min(key, max(n - whole * kTile - 1, 0)) * step + ck;
    }
    auto load_keys = [&](int i, int slot) RUDDER_INLINE {
        const int tile = min(i, tiles - 1);
        const uint8_t* from = kp + (size_t)tile * kTile * (p.ldk * 2);
        const bool ends = tile == whole;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load_lds16(from, ends ? k_end[j] : k_from[j],
                       base + slot * kBytes + (wave * kLoads + j) * 1024);
    };
    auto load_values = [&](int i, int slot) RUDDER_INLINE {
        const uint8_t* from = vp + (size_t)min(i, tiles - 1) * p.Hkv * kBytes;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load_lds16(from, (wave * kLoads + j) * 1024 + lane * 16,
                       base + (RING + slot) * kBytes + (wave * kLoads + j) * 1024);
    };

    uint4 q[kKS];
    float l = 0.0f, c = fabsf(p.sm) * kLog2e;
    {
        const uint16_t* from = p.Q + (size_t)(r0 + t) * p.ldq + (size_t)head * D + half * 8;
        const uint32_t flip = p.sm < 0.0f ? 0x80008000u : 0u;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kKS; ++i) {
            q[i] = *reinterpret_cast<const uint4*>(from + i * 16);
            uint32_t w[4] = {q[i].x ^ flip, q[i].y ^ flip, q[i].z ^ flip, q[i].w ^ flip};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, w[j] >> 16 & 0x7FFFu));
            q[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        if (top >= 0x7F80u) l = __uint_as_float(0x7FC00000u);      // not finite
        if (c == 0.0f) {                           // all keys alike, however large the scores
#pragma unroll
            for (int i = 0; i < kKS; ++i) q[i] = make_uint4(0, 0, 0, 0);
            c = 1.0f;
        }
    }
    // notes of 64 tiles, one a lane
    const int32_t* notes = p.notes + (size_t)h * p.slots + slot0;
    auto notes_from = [&](int i) { return notes[min(i + lane, tiles - 1)]; };
    int note = notes_from(0);

    load_keys(0, 0);
    load_values(0, RING - 1);                      // in front of the first tile: weights of 0 meet these
#pragma unroll
    for (int i = 1; i < RING; ++i) {
        load_keys(i, i);
        load_values(i - 1, i - 1);
    }

    f32x16_acc o[kDT], z;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    Reference ref = {0.0f, kUnset};
    bool far = false;                              // of a row of the wave
    int scale = 1 << 20;                           // the row's, of no tile yet
    int first_bad = 1 << 30;
    int k_at[kKS], v_at[4];                        // where the lane's operands lie in a tile
#pragma unroll
    for (int i = 0; i < kKS; ++i) k_at[i] = place<kChunks>(lane & 31, 2 * i + half);
#pragma unroll
    for (int i = 0; i < 4; ++i) v_at[i] = RING * kBytes + place<8>(lane & 31, 2 * i + half);

    auto scores = [&](int slot, int hf) RUDDER_INLINE {
        f32x16_acc x;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kKS; ++i)
            x = mma_bf16(*reinterpret_cast<const uint4*>(lds + k_at[i] + slot * kBytes +
                                                         hf * 32 * D * 2), q[i], x);
        return x;
    };
    uint4 pend0 = make_uint4(0, 0, 0, 0), pend1 = pend0;       // weights of the 32 keys before
    auto weigh = [&](int slot, int hf) RUDDER_INLINE {
#pragma unroll
        for (int x = 0; x < 2; ++x)                // product after product of another accumulator
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt)
                o[dt] = mma_f16(*reinterpret_cast<const uint4*>(
                                    lds + slot * kBytes + dt * 32 * kTile * 2 + v_at[2 * hf + x]),
                                x ? pend1 : pend0, o[dt]);
    };
    int s = 0;                                     // the tile's power of two
    bool apart = false;                            // whether its values are uneven
    // z, the scores of half hf of the tile at `at`, become weights, while the matrix cores work on
    // the scores of half hf2 in place slot2 and the values of half hf1 in place slot1
    auto step = [&](auto masked, int at, int hf, int slot2, int hf2, int slot1, int hf1) RUDDER_INLINE {
        if constexpr (decltype(masked)::value) {
            const int key0 = at + 32 * hf + 4 * half;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                z[j] = key0 + 8 * (j >> 2) + (j & 3) < limit ? z[j] : -INFINITY;
        }
        float best = z[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) best = fmaxf(best, z[j]);
        if (__any(ref.exponent(c, best) > kMostP)) {
            const float top = fmaxf(best, __shfl_xor(best, 32));
            const Reference now = ref.exponent(c, top) > kMostP ? reference(c, top) : ref;
            const float less = ref.to(c, now);
            const bool was = far;
            far = __any(now.a != 0.0f);
            // near zero a power of two, exact for the weights of the 32 keys before as well
            const float alpha = ref.a != 0.0f || now.a != 0.0f
                                    ? __builtin_amdgcn_exp2f(less)
                                    : __builtin_amdgcn_ldexpf(1.0f, (int)fmaxf(less, -252.0f));
            // these have a factor in fp16; below its range, or where it is not a power of two, they go
            // first (in front of a row's first key there are none)
            if (was || far || __any(less < -14.0f && less > -1e30f)) {
                weigh(slot1, hf1);
                pend0 = pend1 = make_uint4(0, 0, 0, 0);
            }
            pend0 = times(pend0, alpha);
            pend1 = times(pend1, alpha);
            l *= alpha;
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) o[dt] *= alpha;
            ref = now;
        }
        // O of a row is held times 2^scale, the power of the tile that it saw last
        float shift = ref.b, share = 1.0f;
        if (!apart && __any(scale != s && (!decltype(masked)::value || at < limit))) {
            // the weights of the 32 keys before go first: they are of the power of two before
            weigh(slot1, hf1);
            pend0 = pend1 = make_uint4(0, 0, 0, 0);
            const float top = fmaxf(best, __shfl_xor(best, 32));
            const int above = follow(o, scale, s, ref.exponent(c, top) > kNothing);
            if (__any(above)) {                    // the sum takes exponentials of its own
                float apart = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    apart += __builtin_amdgcn_exp2f(ref.exponent(c, z[j]));
                l += above ? apart : 0.0f;
                share = above ? 0.0f : 1.0f;
                shift -= (float)above;
            }
        }
        if (far) {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] -= ref.a;
        }
        const f32x16_acc zn = scores(slot2, hf2);
        weigh(slot1, hf1);
        float sum = 0.0f;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = __builtin_amdgcn_exp2f(fmaf(c, z[2 * j], shift));
            const float e = __builtin_amdgcn_exp2f(fmaf(c, z[2 * j + 1], shift));
            sum += a + e;
            w[j] = pack_f16(a, e);
        }
        l = fmaf(sum, share, l);
        pend0 = make_uint4(w[0], w[1], w[2], w[3]);
        pend1 = make_uint4(w[4], w[5], w[6], w[7]);
        if constexpr (decltype(masked)::value) {
            const int key = at + 32 * hf;
            if (apart && key < most) {             // not in a half in front of which all has been seen
                uneven_values<D>(o, scale, p.V + (size_t)(r0 + key) * p.ldv + (size_t)h * D, p.ldv,
                                 n - key, pend0, pend1);
                pend0 = pend1 = make_uint4(0, 0, 0, 0);
            }
        }
        z = zn;
    };
    // Tile i in place SLOT, known when compiled: LDS addresses are then a register and a constant.
    // A wave that has seen its last key takes one more half, masked, for the values of the half
    // before.
    auto turn = [&](auto masked, int i, auto slot_constant) RUDDER_INLINE {
        constexpr int SLOT = decltype(slot_constant)::value;
        constexpr int kNext = (SLOT + 1) % RING, kBefore = (SLOT + RING - 1) % RING;
        const int at = i * kTile;
        if (!decltype(masked)::value || at < most + kTile) {
            if (i > 0 && (i & 63) == 0) note = notes_from(i);
            const int word = __builtin_amdgcn_readlane(note, i & 63);
            s = (word & 255) - 128;
            apart = decltype(masked)::value && (word & kUneven);
            const int bad = word >> 8 & 127;
            if (bad < kTile) first_bad = min(first_bad, at + bad);
            step(masked, at, 0, SLOT, 1, kBefore, 1);
        }
        wait_barrier<(RING - 2) * 2 * kLoads>();
        load_keys(i + RING, SLOT);
        load_values(i + RING - 1, kBefore);
        if (!decltype(masked)::value || at < most) step(masked, at, 1, kNext, 0, SLOT, 0);
    };

    wait_barrier<(RING - 1) * 2 * kLoads>();
    z = scores(0, 0);
    int i = 0;
    for (; (i + RING) * kTile <= least; i += RING) {       // all of the wave's rows see these
        turn(std::false_type(), i, std::integral_constant<int, 0>());
        turn(std::false_type(), i + 1, std::integral_constant<int, 1>());
        if constexpr (RING > 2) turn(std::false_type(), i + 2, std::integral_constant<int, 2>());
    }
    int slot = 0;                                  // behind the last tile
    for (; i < tiles; i += RING) {
        turn(std::true_type(), i, std::integral_constant<int, 0>());
        slot = 1;
        if (i + 1 == tiles) break;
        turn(std::true_type(), i + 1, std::integral_constant<int, 1>());
        slot = 2;
        if constexpr (RING > 2) {
            if (i + 2 == tiles) break;
            turn(std::true_type(), i + 2, std::integral_constant<int, 2>());
            slot = 3;
        }
    }
    // the weights of the last 32 keys, or of 0 (slot 0: a wave whose rows all see every tile)
    weigh(slot == 0 ? RING - 1 : slot - 1, 1);
    wait_barrier<0>();                             // no load is on its way to LDS any more
    l += __shfl_xor(l, 32);
    // every row sees itself: a sum of zero is one of scores of -inf alone
    float f = l > 0.0f ? 1.0f / l : __uint_as_float(0x7FC00000u);
    if (t >= first_bad) f = __uint_as_float(0x7FC00000u);          // sees a value that is not finite
    // through LDS, so that global memory sees whole rows
    uint8_t* slab = lds + wave * kWaveRows * kStride;
#pragma unroll
    for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = __builtin_amdgcn_ldexpf(o[dt][4 * g + j] * f, -scale);
            *reinterpret_cast<uint2*>(slab + (lane & 31) * kStride + (dt * 32 + g * 8 + half * 4) * 2) =
                make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        }
    wave_sync();
    constexpr int kAtOnce = 64 / kChunks;
#pragma unroll
    for (int i = 0; i < kWaveRows / kAtOnce; ++i) {
        const int r = i * kAtOnce + lane / kChunks, rr = row0 + r;
        const uint4 x = *reinterpret_cast<const uint4*>(slab + r * kStride + lane % kChunks * 16);
        if (rr < rows) {
            const int tt = rr / p.G, hd = h * p.G + rr % p.G;
            *reinterpret_cast<uint4*>(p.O + (size_t)(r0 + tt) * p.ldo + (size_t)hd * D +
                                      lane % kChunks * 8) = x;
        }
    }
}

}  // namespace

namespace {

// Workgroups of the kernel for few rows that run at once.
int round_of(int D) { return D == 64 ? 512 : 256; }

// Work units of the kernel for few rows.
int64_t few_units(int B, int T, int max_rows, int G, int Hkv) {
    const int64_t rows = (int64_t)(max_rows < T ? max_rows : T) * G;
    return (rows + kWaveRows - 1) / kWaveRows * B * Hkv;
}

// The kernel for few rows where its workgroups make one round, or, of 128 channels, one and a quarter and
// the prompts are long: there the rest of a round beside the launch in front costs less.  us, few | many
// rows, 128 channels, 16 heads: 4 x 77 rows (192 units) 9.1 | 12.9, 2 x 256 (256) 11.2 | 15.3, 4 x 130
// (320, 3 tiles) 16.4 | 13.7, 1 x 520 (272, 9 tiles) 17.1 | 18.9, 1 x 600 (304) 18.5 | 21.0, 1 x 700
// (352) 22.1 | 21.4, 1 x 800 (416) 26.6 | 23.3, 1 x 1000 (512) 31.1 | 27.8, 2 x 400 (416) 21.5 | 17.8, 2
// x 600 (608) 33.4 | 22.9, 8 heads, 1 x 2000 (504, 32 tiles) 44.9 | 43.0 (with inputs out of the caches 1
// to 2 more on both sides); 64 channels, 24 heads of eight key heads: 2 x 256 (384) 8.7 | 11.8, 1 x 600
// (456) 12.8 | 16.4, 8 x 77 (512) 8.1 | 10.7, 2 x 400 (608) 13.8 | 13.8, 12 x 77 (768) 11.9 | 10.9, 1 x
// 1000 (752) 22.0 | 21.5; 8 heads of two, 1 x 2000 (500) 23.3 | 32.8.
bool few_rows(int64_t units, int max_rows, int D) {
    const int tiles = (max_rows + kTile - 1) / kTile;
    return units <= round_of(D) || (D == 128 && units <= 320 && tiles >= 9);
}

// Waves of the kernel for many rows, eight or four.  Four make rounds of workgroups that end more
// evenly, two of them a compute unit go through their barriers apart; eight read every tile half as
// often.  us, eight | four; 128 channels: 2 x 1500 rows of 16 heads 55.5 | 49.2, 1 x 5000 of 8
// (two key heads) 121.6 | 97.5, 2 x 6000 of 16 352 | 335, 1 x 12000 of 8 (376 units of 256 rows) 350
// | 321, of 16 616 | 612, 1 x 8192 of 16 (512) 293 | 313, 1 x 16576 of 16 1110 | 1127, of 32 (eight key
// heads) 2130 | 2175.  64 channels, whose registers leave room for a third (an earlier form of the
// kernel): 3 x 1500 of 24 43.4 | 39.4, 1 x 16576 of 32 1255 | 1177.
bool eight_waves(int pairs, int max_rows, int G, int D) {
    const int64_t units = ((int64_t)max_rows * G + 255) / 256 * pairs;
    return D == 128 && units >= 512 && max_rows >= 128 * kTile;
}

constexpr int kMostLdk = 1 << 24;                  // a tile's keys are reached with 32-bit offsets

int slots_of(int B, int T) { return T / kTile + B; }

}  // namespace

bool prompt_attention_workspace(int B, int T, int max_rows, int Hq, int Hkv, int D, size_t& bytes) {
    const int64_t units = few_units(B, T, max_rows, Hq / Hkv, Hkv);
    // from more than one round of the few rows' kernel on, which is all there is up to there, whichever
    // is taken then: no smaller call needs more
    bytes = units > round_of(D) ? (size_t)slots_of(B, T) * Hkv * (kTile * D * 2 + 4) : 0;
    return units <= (1 << 23);
}

hipError_t launch_prompt_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                   const int32_t* row_start, int B, int T, int max_rows, int Hq,
                                   int Hkv, int D, int ldq, int ldk, int ldv, int ldo, float sm,
                                   void* workspace, uint16_t* O, hipStream_t stream) {
    Prompt p = {};
    p.Q = Q;
    p.K = K;
    p.V = V;
    p.row_start = row_start;
    p.T = T;
    p.max_rows = max_rows < T ? max_rows : T;
    p.G = Hq / Hkv;
    p.Hkv = Hkv;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldo = ldo;
    p.sm = sm;
    p.O = O;
    const bool many = !few_rows(few_units(B, T, max_rows, p.G, Hkv), p.max_rows, D) &&
                      ldk <= kMostLdk;
    const int pairs = B * Hkv;
    const bool eight = many && eight_waves(pairs, p.max_rows, p.G, D);
    const int unit_rows = kWaveRows * (eight ? 8 : many ? 4 : 1);
    p.tile_rows = (p.max_rows * p.G + unit_rows - 1) / unit_rows;
    p.dies = pairs % 8 == 0 ? 8 : 1;
    p.die_pairs = pairs / p.dies;
    const int64_t fit = (2 << 20) / ((int64_t)p.max_rows * (4 * D)), least = fit > 4 ? fit : 4;
    p.group = (int)(least < p.die_pairs ? least : p.die_pairs);
    const unsigned grid = (unsigned)((int64_t)pairs * p.tile_rows);
    if (!many) {
        if (D == 64)
            prompt_few_kernel<64><<<grid, 256, 0, stream>>>(p);
        else
            prompt_few_kernel<128><<<grid, 256, 0, stream>>>(p);
        return hipGetLastError();
    }
    if (!workspace) return hipErrorInvalidValue;
    p.slots = slots_of(B, T);
    p.images = static_cast<uint8_t*>(workspace);
    p.notes = reinterpret_cast<int32_t*>(p.images + (size_t)p.slots * Hkv * (kTile * D * 2));
    const dim3 tiles((p.max_rows + kTile - 1) / kTile, Hkv, B);
    if (D == 64) {
        prompt_values_kernel<64><<<tiles, 256, 0, stream>>>(p);
        prompt_wide_kernel<64, 4, 2><<<grid, 256, 0, stream>>>(p);
    } else {
        prompt_values_kernel<128><<<tiles, 256, 0, stream>>>(p);
        if (eight)
            prompt_wide_kernel<128, 8, 3><<<grid, 512, 0, stream>>>(p);
        else
            prompt_wide_kernel<128, 4, 2><<<grid, 256, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace rudder
