// Causal attention of whole prompts, packed one behind the other, to their own
// bf16 keys and values.
//
//   o[t][h] = sum_{j <= t} softmax_j(sm * q[t][h] . k[j][h']) * v[j][h'],  h' = h / (Hq / Hkv)
//
// One pass over the keys with the running maximum m and sum l of the softmax, in
// base 2: z_j = c * (q . k_j), c = sm * log2(e).  Both products are formed
// transposed, so that a query is a column of every matrix and a lane keeps one
// query's numbers: the accumulators of Z^T = K Q^T, packed in pairs, are the
// operand of O^T = V^T P^T, provided that the keys of V^T are stored in their
// order.  With 32x32x16 products a lane of half h = lane / 32 holds keys
// 8 * (j / 4) + 4 * h + j % 4, j = 0..15, of a block of 32.
//
// Weights P are held in fp16 (2^-11 relative; times 2^8, so that weights down to
// 2^-22 of the largest keep all of their bits), values in fp16 as well: a
// tile's values, times a power of two that brings their largest magnitude into
// [2^7, 2^15), are exact in fp16 down to 2^-24 of that magnitude and off by at
// most 2^-32 of it below.  The power is a multiple of 8, so that tiles of like
// values share one; where one differs, O follows the smallest.
#include <cmath>

#include "rudder_block_launch.h"

namespace rudder {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_acc __attribute__((ext_vector_type(16)));

constexpr int kTile = 64;                          // keys
constexpr int kWaveRows = 32;                      // query rows a wave
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 8.0f;                    // P and its sums are held times 2^8
// The running maximum is raised only where a score passes it by more than 2^6: P stays below 2^14.
constexpr float kLazy = 6.0f;

struct Prompt {
    const uint16_t *Q, *K, *V;
    const int32_t* row_start;
    int T, max_rows, G, Hkv, pairs, tile_rows;
    size_t ldq, ldk, ldv, ldo;
    float sm;
    uint16_t* O;
    // of the kernel for many rows: transposed values in fp16, [slot][head][image of a tile], and
    // what else it has to know of a tile, [head][slot]
    uint8_t* images;
    int32_t* notes;
    int slots;
};

__device__ __forceinline__ int quotient(int a, int b) {
    return __builtin_amdgcn_readfirstlane(a / b);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    union { bf16x2_t v; uint32_t u; } r;
    r.v = (bf16x2_t){(__bf16)a, (__bf16)b};
    return r.u;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    union { f16x2_t v; uint32_t u; } r;
    r.v = (f16x2_t){(_Float16)a, (_Float16)b};
    return r.u;
}
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

// Largest finite magnitude bits of eight bf16 values, and those that are not finite made zero.
__device__ __forceinline__ uint32_t finite_top(uint32_t (&w)[4], bool& bad) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a = w[j] & 0x7FFFu, b = w[j] >> 16 & 0x7FFFu;
        if (a >= 0x7F80u) {
            bad = true;
            w[j] &= 0xFFFF0000u;
            a = 0;
        }
        if (b >= 0x7F80u) {
            bad = true;
            w[j] &= 0xFFFFu;
            b = 0;
        }
        top = max(top, max(a, b));
    }
    return top;
}

// The multiple of 8 that brings a largest magnitude of these bits into [2^7, 2^15); at most 120, so
// that 2^s is a number.  A tile of zeros takes that: it must not lower the others'.
__device__ __forceinline__ int scale_of(uint32_t top) {
    const int e = (int)(top >> 7) - 127;
    return top ? min((14 - e) & ~7, 120) : 120;
}

// Chunks of 16 bytes of an LDS row are exchanged so that 16 lanes reading one chunk of 16 rows find
// 16 places of the 64 banks.
template <int CHUNKS>
__device__ __forceinline__ int place(int row, int chunk) {
    return (row * CHUNKS + (chunk ^ (CHUNKS == 16 ? row & 15 : row >> 1 & 7))) * 16;
}

// 128 rows a workgroup, (token, query head of the group) pairs of one sequence and key head, so that
// grouped heads read their keys once; four waves share the tiles through LDS.
template <int D>
__global__ void __launch_bounds__(256) prompt_tile_kernel(const Prompt p) {
    constexpr int kRows = 4 * kWaveRows, kKS = D / 16, kDT = D / 32, kChunks = D / 8;
    __shared__ __align__(16) uint8_t keys[kTile * D * 2], values[kTile * D * 2];
    __shared__ uint32_t tops[4];
    __shared__ int first_bad;

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // longest rows first; the units of a pair, eight apart, on one die where pairs divide by eight
    const int up = quotient(blockIdx.x, p.pairs), pair = blockIdx.x - up * p.pairs;
    const int b = quotient(pair, p.Hkv), h = pair - b * p.Hkv;
    const int first = (p.tile_rows - 1 - up) * kRows;
    const int r0 = min(max(p.row_start[b], 0), p.T);
    const int n = min(min(max(p.row_start[b + 1], r0), p.T) - r0, p.max_rows);
    const int rows = n * p.G;
    if (first >= rows) return;

    const int row0 = first + wave * kWaveRows, row = row0 + (lane & 31);
    const bool live = row < rows;
    const int t = live ? row / p.G : 0, head = h * p.G + (live ? row % p.G : 0);
    const int limit = live ? t + 1 : 0;            // keys this lane's row sees
    const int least = quotient(row0, p.G) + 1;     // every row of the wave sees these
    const int most = row0 < rows ? quotient(min(rows, row0 + kWaveRows) - 1, p.G) + 1 : 0;
    const int last = quotient(min(rows, first + kRows) - 1, p.G) + 1;

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

    f32x16_acc o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -INFINITY;
    int scale = 1 << 20;                           // O is held times 2^scale
    if (tid == 0) first_bad = 1 << 30;

    for (int at = 0; at < last; at += kTile) {
        // keys as they are; values transposed, four keys x eight channels a thread.  Rows behind
        // the prompt are seen by none of its rows, but they have to lie in the buffer.
        __syncthreads();                           // the tile before has been read
        constexpr int kVThreads = 16 * kChunks;
        uint32_t v[4][4] = {};
        uint32_t top = 0;
        const int quad = tid / kChunks % 16, chunk = tid % kChunks;
#pragma unroll
        for (int i = 0; i < kTile * kChunks / 256; ++i) {
            const int u = tid + i * 256, key = u / kChunks, ck = u % kChunks;
            const size_t r = (size_t)min(r0 + at + key, r0 + n - 1);
            *reinterpret_cast<uint4*>(keys + place<kChunks>(key, ck)) =
                *reinterpret_cast<const uint4*>(p.K + r * p.ldk + (size_t)h * D + ck * 8);
        }
        if (tid < kVThreads) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = at + quad * 4 + i;
                if (key >= n) continue;
                const uint4 x = *reinterpret_cast<const uint4*>(
                    p.V + (size_t)(r0 + key) * p.ldv + (size_t)h * D + chunk * 8);
                v[i][0] = x.x;
                v[i][1] = x.y;
                v[i][2] = x.z;
                v[i][3] = x.w;
                bool bad = false;
                top = max(top, finite_top(v[i], bad));
                if (bad) atomicMin(&first_bad, key);
            }
        }
#pragma unroll
        for (int off = 32; off; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
        const int s = __builtin_amdgcn_readfirstlane(scale_of(top));
        if (tid < kVThreads) {
            const float f = __uint_as_float((uint32_t)(127 + s) << 23);
            // keys 4 quad .. + 3 are the accumulators' order with bits 0 and 1 of quad exchanged
            const int to = (quad & ~3) | (quad & 1) << 1 | (quad >> 1 & 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a[4], e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = __uint_as_float(v[i][j] << 16) * f;
                    e[i] = __uint_as_float(v[i][j] & 0xFFFF0000u) * f;
                }
                const int ch = chunk * 8 + 2 * j;
                *reinterpret_cast<uint2*>(values + place<8>(ch, to >> 1) + (to & 1) * 8) =
                    make_uint2(pack_f16(a[0], a[1]), pack_f16(a[2], a[3]));
                *reinterpret_cast<uint2*>(values + place<8>(ch + 1, to >> 1) + (to & 1) * 8) =
                    make_uint2(pack_f16(e[0], e[1]), pack_f16(e[2], e[3]));
            }
        }
        __syncthreads();
        if (at >= most) continue;                  // no row of this wave sees the tile

        f32x16_acc z[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[kb][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < kKS; ++i)
                z[kb] = mma_bf16(*reinterpret_cast<const uint4*>(
                                     keys + place<kChunks>(kb * 32 + (lane & 31), 2 * i + half)),
                                 q[i], z[kb]);
        }
        if (at + kTile > least) {
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
        best *= c;
        float alpha = 1.0f;
        if (__any(best > m + kLazy)) {
            const float raised = fmaxf(m, fmaxf(best, __shfl_xor(best, 32)));
            alpha = raised == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
            m = raised;
            l *= alpha;
        }
        float down = 1.0f;                         // of this tile's weights, for the values
        if (s < scale) {
            alpha = __builtin_amdgcn_ldexpf(alpha, max(s - scale, -252));
            scale = s;
        } else {
            down = __builtin_amdgcn_ldexpf(1.0f, scale - s);
        }
        if (__any(alpha != 1.0f))
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) o[i][j] *= alpha;
        const float shift = kPShift - (m == -INFINITY ? 0.0f : m);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at_z = (ks & 1) * 8 + 2 * j;
                const float a = __builtin_amdgcn_exp2f(fmaf(c, z[ks >> 1][at_z], shift));
                const float e = __builtin_amdgcn_exp2f(fmaf(c, z[ks >> 1][at_z + 1], shift));
                l += a + e;
                w[j] = pack_f16(a * down, e * down);
            }
#pragma unroll
            for (int i = 0; i < kDT; ++i)
                o[i] = mma_f16(*reinterpret_cast<const uint4*>(
                                   values + place<8>(i * 32 + (lane & 31), 2 * ks + half)),
                               make_uint4(w[0], w[1], w[2], w[3]), o[i]);
        }
    }
    l += __shfl_xor(l, 32);
    __syncthreads();
    // every row sees itself: a sum of zero is one of scores of -inf alone
    float f = l > 0.0f ? 1.0f / l : __uint_as_float(0x7FC00000u);
    if (t >= first_bad) f = __uint_as_float(0x7FC00000u);          // sees a value that is not finite
    if (!live) return;
    uint16_t* to = p.O + (size_t)(r0 + t) * p.ldo + (size_t)head * D + half * 4;
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = __builtin_amdgcn_ldexpf(o[i][4 * g + j] * f, -scale);
            *reinterpret_cast<uint2*>(to + i * 32 + g * 8) =
                make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        }
}

// A prompt's tiles are kept at slots of their own: floor((r0 + n) / 64) + 1 >= floor(r0 / 64) +
// ceil(n / 64), so that those of sequence b end before those of b + 1 begin.
__device__ __forceinline__ int first_slot(int r0, int b) { return r0 / kTile + b; }

// ---------------------------------------------------------------------------
// Values for the kernel of many rows: transposed, in fp16, times a tile's power of two, laid out as
// that kernel keeps them in LDS.  One tile and head a workgroup.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) prompt_values_kernel(const Prompt p) {
    constexpr int kChunks = D / 8, kVThreads = 16 * kChunks;
    __shared__ uint32_t tops[4];
    __shared__ int first_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.z, h = blockIdx.y, at = blockIdx.x * kTile;
    const int r0 = min(max(p.row_start[b], 0), p.T);
    const int n = min(min(max(p.row_start[b + 1], r0), p.T) - r0, p.max_rows);
    if (at >= n) return;
    if (tid == 0) first_bad = kTile;
    __syncthreads();
    const int quad = tid / kChunks % 16, chunk = tid % kChunks;
    uint32_t v[4][4] = {};
    uint32_t top = 0;
    if (tid < kVThreads) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = at + quad * 4 + i;
            if (key >= n) continue;
            const uint4 x = *reinterpret_cast<const uint4*>(
                p.V + (size_t)(r0 + key) * p.ldv + (size_t)h * D + chunk * 8);
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bool bad = false;
            top = max(top, finite_top(v[i], bad));
            if (bad) atomicMin(&first_bad, quad * 4 + i);
        }
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const int s = scale_of(top);
    const int slot = first_slot(r0, b) + (int)blockIdx.x;
    if (tid == 0) p.notes[(size_t)h * p.slots + slot] = s + 128 + (first_bad << 8);
    if (tid >= kVThreads) return;
    const float f = __uint_as_float((uint32_t)(127 + s) << 23);
    const int to = (quad & ~3) | (quad & 1) << 1 | (quad >> 1 & 1);
    uint8_t* image = p.images + ((size_t)slot * p.Hkv + h) * (kTile * D * 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a[4], e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __uint_as_float(v[i][j] << 16) * f;
            e[i] = __uint_as_float(v[i][j] & 0xFFFF0000u) * f;
        }
        const int ch = chunk * 8 + 2 * j;
        *reinterpret_cast<uint2*>(image + place<8>(ch, to >> 1) + (to & 1) * 8) =
            make_uint2(pack_f16(a[0], a[1]), pack_f16(a[2], a[3]));
        *reinterpret_cast<uint2*>(image + place<8>(ch + 1, to >> 1) + (to & 1) * 8) =
            make_uint2(pack_f16(e[0], e[1]), pack_f16(e[2], e[3]));
    }
}

// 16 bytes a lane from `from` straight to LDS, lane after lane from `lds` on.  In assembly, so that
// the compiler waits for none of them in front of LDS reads: wait_barrier() orders them.
__device__ __forceinline__ void load_lds(const void* from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(from), "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}
// All but the wave's last N loads have landed, its LDS reads are done; then the workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    typedef __attribute__((address_space(3))) const void* lds_ptr;
    return (uint32_t)(uintptr_t)(lds_ptr)p;
}

// ---------------------------------------------------------------------------
// Many rows: 256 of them a workgroup, two groups of four waves in opposite phases.
// ---------------------------------------------------------------------------
// A wave alternates between a phase of products (scores of tile i + 1, values of tile i) and one of
// vector work (weights of tile i + 1).  Waves w and w + 4 share a vector unit and a matrix core and
// are one phase apart: group A has its products of step i in phase 2 i, B in 2 i + 1.
// Tiles come straight to LDS, into rings of four for keys and values each: the vector phase behind
// step i asks for K of i + 4 and V of i + 3, which are first read in phase 2 i + 6; their places
// were last read in phase 2 i - 1.
template <int D>
__global__ void __launch_bounds__(512, 2) prompt_wide_kernel(const Prompt p) {
    constexpr int kRows = 8 * kWaveRows, kKS = D / 16, kDT = D / 32, kChunks = D / 8;
    constexpr int kBytes = kTile * D * 2, kLoads = kBytes / 8192;     // a tile's; a wave's of one
    constexpr int kStride = D * 2 + 16;                               // of an output row in LDS
    __shared__ __align__(16) uint8_t lds[8 * kBytes];                 // four of keys, four of values
    static_assert(8 * kWaveRows * kStride <= 8 * kBytes, "the outputs pass through the rings");

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int up = quotient(blockIdx.x, p.pairs), pair = blockIdx.x - up * p.pairs;
    const int b = quotient(pair, p.Hkv), h = pair - b * p.Hkv;
    const int first = (p.tile_rows - 1 - up) * kRows;
    const int r0 = min(max(p.row_start[b], 0), p.T);
    const int n = min(min(max(p.row_start[b + 1], r0), p.T) - r0, p.max_rows);
    const int rows = n * p.G;
    if (first >= rows) return;

    const int row0 = first + wave * kWaveRows, row = row0 + (lane & 31);
    const bool live = row < rows;
    const int t = live ? row / p.G : 0, head = h * p.G + (live ? row % p.G : 0);
    const int limit = live ? t + 1 : 0;            // keys this lane's row sees
    const int least = quotient(row0, p.G) + 1;     // every row of the wave sees these
    const int most = row0 < rows ? quotient(min(rows, row0 + kWaveRows) - 1, p.G) + 1 : 0;
    const int last = quotient(min(rows, first + kRows) - 1, p.G) + 1;
    const int tiles = (last + kTile - 1) / kTile;

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
    const int slot0 = first_slot(r0, b);
    const int32_t* notes = p.notes + (size_t)h * p.slots + slot0;
    auto notes_from = [&](int i) { return notes[min(i + lane, tiles - 1)]; };
    int note = notes_from(0);

    // this wave's pieces of a tile; tiles behind the last are the last one again, never read
    const uint32_t base = lds_offset(lds);
    const uint8_t* kp = reinterpret_cast<const uint8_t*>(p.K + (size_t)r0 * p.ldk + (size_t)h * D);
    const uint8_t* vp = p.images + ((size_t)slot0 * p.Hkv + h) * kBytes + lane * 16;
    auto load_keys = [&](int i) {
        const int tile = min(i, tiles - 1);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int piece = wave * kLoads + j, key = piece * (64 / kChunks) + lane / kChunks;
            const int ck = lane % kChunks ^ (kChunks == 16 ? key & 15 : key >> 1 & 7);
            load_lds(kp + (size_t)min(tile * kTile + key, n - 1) * (p.ldk * 2) + ck * 16,
                     base + (i & 3) * kBytes + piece * 1024);
        }
    };
    auto load_values = [&](int i) {
        const int tile = min(i, tiles - 1);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int piece = wave * kLoads + j;
            load_lds(vp + (size_t)tile * p.Hkv * kBytes + piece * 1024,
                     base + (4 + (i & 3)) * kBytes + piece * 1024);
        }
    };

    f32x16_acc o[kDT], z[2];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    uint4 pk[4];
    float m = -INFINITY;
    int scale = 1 << 20;                           // O is held times 2^scale
    int first_bad = 1 << 30;
    int k_at[kKS], v_at[4];                        // where the lane's operands lie in a tile
#pragma unroll
    for (int i = 0; i < kKS; ++i) k_at[i] = place<kChunks>(lane & 31, 2 * i + half);
#pragma unroll
    for (int i = 0; i < 4; ++i) v_at[i] = place<8>(lane & 31, 2 * i + half);

    load_keys(0);
    load_keys(1);
    load_values(0);
    load_keys(2);
    load_values(1);
    wait_barrier<4 * kLoads>();
    if (wave >= 4) wait_barrier<63>();             // group B: one phase behind
    bool now = false;                              // the wave sees the tile whose V is next
    for (int i = -1;; ++i) {
        const bool more = i + 1 < tiles;
        const int at = (i + 1) * kTile;
        const bool ahead = more && at < most;
        if (ahead) {
            const uint8_t* kt = lds + (i + 1 & 3) * kBytes;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < 16; ++j) z[kb][j] = 0.0f;
#pragma unroll
            for (int k = 0; k < kKS; ++k)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    z[kb] = mma_bf16(
                        *reinterpret_cast<const uint4*>(kt + k_at[k] + kb * 32 * D * 2), q[k],
                        z[kb]);
        }
        if (now) {
            const uint8_t* vt = lds + (4 + (i & 3)) * kBytes;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int dt = 0; dt < kDT; ++dt)
                    o[dt] = mma_f16(
                        *reinterpret_cast<const uint4*>(vt + v_at[ks] + dt * 32 * kTile * 2),
                        pk[ks], o[dt]);
        }
        if (wave < 4)
            wait_barrier<63>();
        else
            wait_barrier<2 * kLoads>();
        if (!more) break;
        load_keys(i + 4);
        load_values(i + 3);
        now = ahead;
        if (ahead) {
            if (i + 1 > 0 && (i + 1 & 63) == 0) note = notes_from(i + 1);
            const int word = __builtin_amdgcn_readlane(note, i + 1 & 63);
            const int s = (word & 255) - 128, bad = word >> 8;
            if (bad < kTile) first_bad = min(first_bad, at + bad);
            if (at + kTile > least) {
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
            best *= c;
            if (__any(best > m + kLazy) || s < scale) {
                const float raised = fmaxf(m, fmaxf(best, __shfl_xor(best, 32)));
                float alpha = raised == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
                m = raised;
                l *= alpha;
                if (s < scale) {
                    alpha = __builtin_amdgcn_ldexpf(alpha, max(s - scale, -252));
                    scale = s;
                }
#pragma unroll
                for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[dt][j] *= alpha;
            }
            const float shift = kPShift - (m == -INFINITY ? 0.0f : m);
            float sum = 0.0f;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    z[kb][j] = __builtin_amdgcn_exp2f(fmaf(c, z[kb][j], shift));
                    sum += z[kb][j];
                }
            l += sum;
            if (s > scale) {                       // small values beside large ones
                const float down = __builtin_amdgcn_ldexpf(1.0f, scale - s);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int j = 0; j < 16; ++j) z[kb][j] *= down;
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = pack_f16(z[ks >> 1][(ks & 1) * 8 + 2 * j],
                                    z[ks >> 1][(ks & 1) * 8 + 2 * j + 1]);
                pk[ks] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (wave < 4)
            wait_barrier<4 * kLoads>();
        else
            wait_barrier<63>();
    }
    if (wave < 4) wait_barrier<63>();              // group B's last phase of products
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
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

// Whether a call takes the kernel for many rows.
bool many_rows(int B, int T, int max_rows, int G, int Hkv, int D) {
    return (int64_t)(max_rows < T ? max_rows : T) * G > 256;
}

int slots_of(int B, int T) { return T / kTile + B; }

}  // namespace

bool prompt_attention_workspace(int B, int T, int max_rows, int Hq, int Hkv, int D, size_t& bytes) {
    const int64_t rows = (int64_t)(max_rows < T ? max_rows : T) * (Hq / Hkv);
    bytes = 0;
    if (many_rows(B, T, max_rows, Hq / Hkv, Hkv, D))
        bytes = (size_t)slots_of(B, T) * Hkv * (kTile * D * 2 + 4);
    return (rows + 127) / 128 * B * Hkv <= (1 << 21);
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
    p.pairs = B * Hkv;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldo = ldo;
    p.sm = sm;
    p.O = O;
    if (!many_rows(B, T, max_rows, p.G, Hkv, D)) {
        p.tile_rows = (p.max_rows * p.G + 127) / 128;
        const unsigned grid = (unsigned)((int64_t)p.pairs * p.tile_rows);
        if (D == 64)
            prompt_tile_kernel<64><<<grid, 256, 0, stream>>>(p);
        else
            prompt_tile_kernel<128><<<grid, 256, 0, stream>>>(p);
        return hipGetLastError();
    }
    p.slots = slots_of(B, T);
    p.images = static_cast<uint8_t*>(workspace);
    p.notes = reinterpret_cast<int32_t*>(p.images + (size_t)p.slots * Hkv * (kTile * D * 2));
    const dim3 tiles((p.max_rows + kTile - 1) / kTile, Hkv, B);
    p.tile_rows = (p.max_rows * p.G + 255) / 256;
    const unsigned grid = (unsigned)((int64_t)p.pairs * p.tile_rows);
    if (D == 64) {
        prompt_values_kernel<64><<<tiles, 256, 0, stream>>>(p);
        prompt_wide_kernel<64><<<grid, 512, 0, stream>>>(p);
    } else {
        prompt_values_kernel<128><<<tiles, 256, 0, stream>>>(p);
        prompt_wide_kernel<128><<<grid, 512, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace rudder
