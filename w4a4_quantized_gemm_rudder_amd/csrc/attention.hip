// Attention over the paged 8-bit cache and cross attention to bf16 states.
//
//   o[t][h] = sum_j softmax_j(sm * q[t][h] . k[j][h']) * v[j][h'],  h' = h / (Hq / Hkv)
//
// One pass over the keys with the running maximum m and sum l of the softmax,
// in base 2: z_j = c * (q . k_j), c = sm * log2(e).
//
// Both products are formed transposed, so that a query is a column of every
// matrix and a lane keeps one query's numbers: Z^T = K Q^T has keys as rows,
// and its accumulator layout is, key for key, the operand layout of the second
// product O^T = V^T P^T.  P therefore never leaves its registers and m, l and
// the rescaling of O are one number a lane.  With 32x32x16 products a lane of
// half h = lane / 32 holds accumulator rows 8 * g + 4 * h + i and feeds keys
// 16 * s + 8 * h + 0..7: the key kept at row r of a block of 32 is the one
// whose number has bits 2 and 3 of r exchanged, and nothing has to move.
//
// The rows of a workgroup are (token, query head of the group) pairs of one
// sequence and cached head, so grouped heads read their keys once.
//
// Cache codes become fp16 operands: 0x6400 | (code ^ 0x80) is the fp16 value
// 1152 + code, and one packed subtraction leaves the code, exactly.  q is
// scaled by a power of two to a largest magnitude in [1, 2) and is then
// exact in fp16, but for elements below 2^-7 of the largest, which keep an
// absolute error of 2^-25 of it.  The K scale multiplies c.  The V scale sv is
// folded into the exponent: with t_j = z_j + log2(sv) and m the running
// maximum of t, P_j = exp2(t_j - m) multiplies plain codes, and
// l = sum P_j / sv.  P is rounded to fp16 (2^-11 relative, absolute 2^-33 below
// 2^-22); the sum l is formed from the unrounded values.
#include <cmath>

#include "rudder_internal.h"

namespace rudder {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_acc __attribute__((ext_vector_type(16)));

constexpr int kPage = RUDDER_CACHE_PAGE;           // keys a tile
constexpr int kThreads = 256;
constexpr int kWaveRows = 32;
constexpr int kRows = 4 * kWaveRows;               // query rows a workgroup
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 8.0f;                    // cache: P and its sums are held times 2^8
// Smallest V scale the exponent takes: smaller ones (an all-zero block's 0) are read as this.
constexpr float kMinVScale = 8.271806125530277e-25f;   // 2^-80

struct Problem {
    const uint16_t* Q;
    const int32_t* row_start;
    const int32_t* kv_len;
    // cache
    const int32_t* page_table;
    const int8_t* codes;
    const float* scales;
    int max_pages, num_pages;
    // bf16 states
    const uint16_t* K;
    const uint16_t* V;
    const int32_t* kv_start;
    int Tkv;
    size_t ldk, ldv;
    // both
    int T, max_rows, max_kv, Hq, Hkv, causal;
    size_t ldq, ldo;
    float sm;
    uint16_t* O;
    // split of the key axis: `splits` pieces of `split_tiles` tiles; partial results when > 1
    int splits, split_tiles;
    float* part_o;      // [splits][T * Hq][D]
    float2* part_ml;    // [splits][T * Hq]
};

// Sequence b's query rows and keys, clamped to the buffers whatever the arrays hold.
struct Sequence {
    int r0, n, kv, kv0;
};

template <bool CACHE>
__device__ __forceinline__ Sequence sequence(const Problem& p, int b) {
    Sequence s;
    s.r0 = min(max(p.row_start[b], 0), p.T);
    s.n = min(max(p.row_start[b + 1], s.r0), p.T) - s.r0;
    s.kv = min(max(p.kv_len[b], 0), p.max_kv);
    s.kv0 = 0;
    if (CACHE) {
        s.kv = (int)min((int64_t)s.kv, (int64_t)p.max_pages * kPage);
    } else {
        s.kv0 = min(max(p.kv_start[b], 0), p.Tkv);
        s.kv = min(s.kv, p.Tkv - s.kv0);
    }
    return s;
}

__device__ __forceinline__ uint32_t sub_1152(uint32_t pair) {
    union { uint32_t u; f16x2_t h; } r;
    r.u = pair;
    r.h -= (f16x2_t){(_Float16)1152.0f, (_Float16)1152.0f};
    return r.u;
}

// Four int8 codes to four fp16 values, exactly.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    w ^= 0x80808080u;
    return make_uint2(sub_1152(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)),
                      sub_1152(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)));
}

// Bits 2 and 3 exchanged: key number <-> accumulator row (its own inverse).
__device__ __forceinline__ int swap23(int r) {
    return (r & ~12) | ((r & 4) << 1) | ((r & 8) >> 1);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    union { bf16x2_t v; uint32_t u; } r;
    r.v = (bf16x2_t){(__bf16)a, (__bf16)b};
    return r.u;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    union { f16x2_t v; uint32_t u; } r;
    r.v = (f16x2_t){(_Float16)a, (_Float16)b};
    return r.u;
}

// Largest magnitude of a lane's share of a query row.
template <int N>
__device__ __forceinline__ float abs_max(const uint4 (&q)[N]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                     fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
    }
    return amax;
}

// A query row of largest magnitude amax = f * 2^e, f in [1, 2), to fp16 times 2^-e; returns 2^e.
// A row of zeros or infinities keeps e = 0.
template <int N>
__device__ __forceinline__ float to_f16(uint4 (&q)[N], float amax) {
    const int field = (int)(__float_as_uint(amax) >> 23);
    const int e = (field == 0 || field == 255) ? 0 : min(max(field - 127, -120), 120);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = pack_f16(__uint_as_float(w[j] << 16) * down,
                            __uint_as_float(w[j] & 0xFFFF0000u) * down);
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// Largest magnitude bits of a lane's share of a query row (NaN patterns are the largest).
template <int N>
__device__ __forceinline__ uint32_t abs_max_bits(const uint4 (&q)[N]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    }
    return top;
}

// A query row whose largest magnitude has the bf16 bits `top` = f * 2^e, f in [1, 2), as integers
// q * 2^(14 - e) in [-32639, 32639] and these as two digits, 256 * high + low: N pairs of 16 bytes
// (16 channels) become one of each.  Returns 2^(e - 14), or NaN for a row that is not finite.
template <int N>
__device__ __forceinline__ float to_digits(const uint4 (&q)[2 * N], uint32_t top, uint4 (&high)[N],
                                           uint4 (&low)[N]) {
    const int field = (int)(top >> 7);
    const int e = min(max(field - 127, -110), 127);
    const float up = __uint_as_float((uint32_t)(127 + min(14 - e, 127)) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint4 src = q[2 * i + (d >> 1)];
            const uint32_t a = d & 1 ? src.z : src.x, b = d & 1 ? src.w : src.y;
            const float f[4] = {__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u),
                                __uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)};
            int h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int x = quantize_clamped(f[j] * up, 32639.0f);
                h[j] = (x + 128) >> 8;
                l[j] = x - 256 * h[j];
            }
            hw[d] = byte_word(h);
            lw[d] = byte_word(l);
        }
        high[i] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        low[i] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
    return field == 255 ? __uint_as_float(0x7FC00000u)
                        : __uint_as_float((uint32_t)(127 + max(e - 14, -126)) << 23);
}

// What turns a row's sum of P * code (or P * v) into its output: 0 where no key is visible.
__device__ __forceinline__ float row_factor(float l) {
    return l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
}

template <bool CACHE>
__device__ __forceinline__ f32x16_acc mma(uint4 a, uint4 b, f32x16_acc c) {
    if (CACHE) {
        union { uint4 u; f16x8_t v; } x, y;
        x.u = a;
        y.u = b;
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(x.v, y.v, c, 0, 0, 0);
    } else {
        union { uint4 u; bf16x8_t v; } x, y;
        x.u = a;
        y.u = b;
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.v, y.v, c, 0, 0, 0);
    }
}

// exp2(t - m) / sv loses what underflows before the division.  With z the largest exponent so far
// and a page's log2(sv) at most 60 below the largest, m <= z + max log2(sv), so that keys within
// 30 of z have t - m >= -90: nothing of weight is lost.  Further apart, the sum takes exponents of
// its own.
__device__ __forceinline__ bool scales_apart(float lsv, float top_lsv) {
    return __builtin_amdgcn_readfirstlane(lsv < top_lsv - 60.0f);
}

// One tile of 64 keys on its way from HBM to LDS.
template <int D, bool CACHE>
struct Stage {
    static constexpr int kKStride = D * 2 + 16;    // bytes of a key's row in LDS
    static constexpr int kVStride = kPage * 2 + 16;    // bytes of a channel's row in LDS
    static constexpr int kKBytes = kPage * kKStride;
    static constexpr int kVBytes = D * kVStride;
    static constexpr int kNK = CACHE ? D / 64 : D / 32;    // 16-byte pieces a thread
    static constexpr int kNV = CACHE ? D / 64 : 4;
    uint4 k[kNK], v[kNV];                          // states: v[i] is key i of the thread's four

    // page: the tile's page number (cache); key0, kv: first key and the sequence's keys (states)
    __device__ __forceinline__ void load(const Problem& p, const Sequence& s, int h, int page,
                                         int key0) {
        const int tid = threadIdx.x;
        if constexpr (CACHE) {
            const uint4* src = reinterpret_cast<const uint4*>(
                p.codes + ((size_t)page * p.Hkv + h) * (size_t)(2 * kPage * D));
#pragma unroll
            for (int i = 0; i < kNK; ++i) k[i] = src[tid + i * kThreads];
#pragma unroll
            for (int i = 0; i < kNV; ++i) v[i] = src[kPage * D / 16 + tid + i * kThreads];
        } else {
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * kThreads, key = key0 + u / (D / 8);
                k[i] = make_uint4(0, 0, 0, 0);
                if (key < s.kv)
                    k[i] = *reinterpret_cast<const uint4*>(
                        p.K + (size_t)(s.kv0 + key) * p.ldk + (size_t)h * D + u % (D / 8) * 8);
            }
            // V: four keys x eight channels a thread (all threads for D = 128, half for 64)
            if (tid < 2 * D) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = key0 + tid / (D / 8) * 4 + i;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (key < s.kv)
                        v[i] = *reinterpret_cast<const uint4*>(
                            p.V + (size_t)(s.kv0 + key) * p.ldv + (size_t)h * D +
                            tid % (D / 8) * 8);
                }
            }
        }
    }

    __device__ __forceinline__ void store(uint8_t* lk, uint8_t* lv) const {
        const int tid = threadIdx.x;
        if constexpr (CACHE) {
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * kThreads, row = swap23(u / (D / 16));
                uint8_t* d = lk + row * kKStride + u % (D / 16) * 32;
                put(d, k[i]);
            }
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                const int u = tid + i * kThreads;
                put(lv + u / 4 * kVStride + u % 4 * 32, v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * kThreads, row = swap23(u / (D / 8));
                *reinterpret_cast<uint4*>(lk + row * kKStride + u % (D / 8) * 16) = k[i];
            }
            if (tid < 2 * D) {
                uint8_t* d = lv + tid % (D / 8) * 8 * kVStride + tid / (D / 8) * 8;
                put4(d, v[0].x, v[1].x, v[2].x, v[3].x);
                put4(d + 2 * kVStride, v[0].y, v[1].y, v[2].y, v[3].y);
                put4(d + 4 * kVStride, v[0].z, v[1].z, v[2].z, v[3].z);
                put4(d + 6 * kVStride, v[0].w, v[1].w, v[2].w, v[3].w);
            }
        }
    }

    // Two channels of four keys, transposed.
    static __device__ __forceinline__ void put4(uint8_t* d, uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t e) {
        *reinterpret_cast<uint2*>(d) = make_uint2(__builtin_amdgcn_perm(b, a, 0x05040100u),
                                                  __builtin_amdgcn_perm(e, c, 0x05040100u));
        *reinterpret_cast<uint2*>(d + kVStride) =
            make_uint2(__builtin_amdgcn_perm(b, a, 0x07060302u),
                       __builtin_amdgcn_perm(e, c, 0x07060302u));
    }

    static __device__ __forceinline__ void put(uint8_t* d, uint4 c) {
        const uint2 a = widen4(c.x), b = widen4(c.y), e = widen4(c.z), f = widen4(c.w);
        *reinterpret_cast<uint4*>(d) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(d + 16) = make_uint4(e.x, e.y, f.x, f.y);
    }
};

template <int D, bool CACHE>
__global__ void __launch_bounds__(kThreads, 2)
attention_tile_kernel(const Problem p) {
    using St = Stage<D, CACHE>;
    constexpr int kKS = D / 16;                    // steps of the first product
    constexpr int kDT = D / 32;                    // channel tiles of the second
    __shared__ __align__(16) uint8_t lk[St::kKBytes];
    __shared__ __align__(16) uint8_t lv[St::kVBytes];

    const int split = blockIdx.x % p.splits, tile_row = blockIdx.x / p.splits;
    const int h = blockIdx.y, b = blockIdx.z;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5;
    const Sequence s = sequence<CACHE>(p, b);
    const int G = p.Hq / p.Hkv;
    const int rows = min(s.n, p.max_rows) * G;     // (token, head of the group) pairs
    if (tile_row * kRows >= rows) return;

    // this lane's query row
    const int row = tile_row * kRows + wave * kWaveRows + (lane & 31);
    const bool live = row < rows;
    const bool wave_live = tile_row * kRows + wave * kWaveRows < rows;
    const int t = live ? row / G : 0;
    const int head = h * G + (live ? row % G : 0);
    // keys visible to it, and the last row of the workgroup that has any
    const int limit = !live ? 0 : p.causal ? min(max(s.kv - s.n + t + 1, 0), s.kv) : s.kv;
    const int last_t = (min(rows, (tile_row + 1) * kRows) - 1) / G;
    const int most = p.causal ? min(max(s.kv - s.n + last_t + 1, 0), s.kv) : s.kv;
    const int tile0 = split * p.split_tiles;
    const int tile1 = min((most + kPage - 1) / kPage, tile0 + p.split_tiles);
    if (p.splits > 1 && tile0 * kPage >= s.kv) return;     // the join does not read this piece

    uint4 q[kKS];
    float c = p.sm * kLog2e;
    {
        const uint16_t* src = p.Q + (size_t)(s.r0 + t) * p.ldq + (size_t)head * D + half * 8;
#pragma unroll
        for (int i = 0; i < kKS; ++i) {
            q[i] = make_uint4(0, 0, 0, 0);
            if (live) q[i] = *reinterpret_cast<const uint4*>(src + i * 16);
        }
        if (CACHE) {
            const float amax = abs_max<kKS>(q);
            c *= to_f16<kKS>(q, fmaxf(amax, __shfl_xor(amax, 32)));
        }
    }

    f32x16_acc o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -INFINITY, l = 0.0f, top_lsv = -INFINITY;

    const int32_t* table = CACHE ? p.page_table + (size_t)b * p.max_pages : nullptr;
    // The next tile at or behind `i` whose page lies in the pool (others hold no keys).
    auto next = [&](int i, int& page) {
        page = 0;
        if (CACHE)
            for (; i < tile1; ++i) {
                page = __builtin_amdgcn_readfirstlane(table[i]);
                if (page >= 0 && page < p.num_pages) break;
            }
        return i;
    };

    St stage;
    int page;
    int tile = next(tile0, page);
    if (tile < tile1) stage.load(p, s, h, page, tile * kPage);
    while (tile < tile1) {
        const int at = tile * kPage;
        float cz = c, lsv = 0.0f, sv_inv = 1.0f;
        if (CACHE) {
            const float* sc = p.scales + ((size_t)page * p.Hkv + h) * 2;
            cz = c * sc[0];
            const float sv = fmaxf(sc[1], kMinVScale);
            lsv = __builtin_amdgcn_logf(sv);       // log2
            sv_inv = 1.0f / sv;
        }
        __syncthreads();                           // the last tile has been read
        stage.store(lk, lv);
        tile = next(tile + 1, page);
        if (tile < tile1) stage.load(p, s, h, page, tile * kPage);
        __syncthreads();
        if (!wave_live) continue;

        f32x16_acc z[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[tt][j] = 0.0f;
            const uint8_t* kr = lk + (tt * 32 + (lane & 31)) * St::kKStride + half * 16;
#pragma unroll
            for (int i = 0; i < kKS; ++i)
                z[tt] = mma<CACHE>(*reinterpret_cast<const uint4*>(kr + i * 32), q[i], z[tt]);
        }
        // t = c * z + log2(sv); key of register j: 32 tt + 16 (j / 8) + 8 half + j % 8
        float top = -INFINITY;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int key = at + 32 * tt + 16 * (j >> 3) + 8 * half + (j & 7);
                const float v = key < limit ? fmaf(cz, z[tt][j], lsv) : -INFINITY;
                z[tt][j] = v;
                top = fmaxf(top, v);
            }
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top);
        const float base = (m_new == -INFINITY ? 0.0f : m_new) - (CACHE ? kPShift : 0.0f);
        const float alpha = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
        float sum = 0.0f, own = 0.0f;
        top_lsv = fmaxf(top_lsv, lsv);
        const bool far = CACHE && scales_apart(lsv, top_lsv);
        if (far)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int j = 0; j < 16; ++j) own += __builtin_amdgcn_exp2f(z[tt][j] - lsv - base);
        uint4 pk[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = (ks & 1) * 8 + 2 * j;
                const float a = __builtin_amdgcn_exp2f(z[ks >> 1][r] - base);
                const float e = __builtin_amdgcn_exp2f(z[ks >> 1][r + 1] - base);
                sum += a + e;
                w[j] = CACHE ? pack_f16(a, e) : pack_bf16(a, e);
            }
            pk[ks] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        l = fmaf(l, alpha, far ? own : sum * sv_inv);
        m = m_new;
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[dt][j] *= alpha;
            const uint8_t* vr = lv + (dt * 32 + (lane & 31)) * St::kVStride + half * 16;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                o[dt] = mma<CACHE>(*reinterpret_cast<const uint4*>(vr + ks * 32), pk[ks], o[dt]);
        }
    }
    l += __shfl_xor(l, 32);
    if (!live) return;
    const size_t out_row = (size_t)(s.r0 + t);
    if (p.splits > 1) {
        const size_t at = (size_t)split * ((size_t)p.T * p.Hq) + out_row * p.Hq + head;
        if (half == 0) p.part_ml[at] = make_float2(m, l);
        float* d = p.part_o + at * D;
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<float4*>(d + dt * 32 + g * 8 + half * 4) = make_float4(
                    o[dt][4 * g], o[dt][4 * g + 1], o[dt][4 * g + 2], o[dt][4 * g + 3]);
        return;
    }
    const float f = row_factor(l);
    uint16_t* d = p.O + out_row * p.ldo + (size_t)head * D;
#pragma unroll
    for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint2*>(d + dt * 32 + g * 8 + half * 4) =
                make_uint2(pack_bf16(o[dt][4 * g] * f, o[dt][4 * g + 1] * f),
                           pack_bf16(o[dt][4 * g + 2] * f, o[dt][4 * g + 3] * f));
}

// ---------------------------------------------------------------------------
// Few rows over the cache: at most 16 (token, head of the group) rows.
// ---------------------------------------------------------------------------
// Bound by the bytes of the codes.  Every wave takes pages of its own, from HBM straight to
// registers -- nothing is shared, so nothing passes through LDS -- and the waves' results are
// joined at the end.  16x16x32 products: with page layouts as they are, the 16 bytes a lane loads
// of a K row are two product steps of 32 channels (lane quarter g: channels 64 c + 16 g + 8 e +
// 0..7), the 16 bytes of a V row two steps of 32 tokens (16 g + 8 e + 0..7), and the key at row
// r of score tile (e, a) is 16 (r / 4) + 8 e + 4 a + r % 4, so that the scores of tiles (e, 0)
// and (e, 1) are the operand of step e.
// The running maximum is raised only where a score passes it by more than 2^6 (P has room for
// it): most pages then need no exchange between lanes and no rescaling.
constexpr float kLazy = 6.0f;

typedef float f32x4_acc __attribute__((ext_vector_type(4)));
typedef int i32x4_acc __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_acc mma16_i8(uint4 a, uint4 b, i32x4_acc c) {
    union { uint4 u; i32x4_acc v; } x, y;
    x.u = a;
    y.u = b;
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(x.v, y.v, c, 0, 0, 0);
}

__device__ __forceinline__ f32x4_acc mma16(uint4 a, uint4 b, f32x4_acc c) {
    union { uint4 u; f16x8_t v; } x, y;
    x.u = a;
    y.u = b;
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x.v, y.v, c, 0, 0, 0);
}

__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b) {
    const uint2 x = widen4(a), y = widen4(b);
    return make_uint4(x.x, x.y, y.x, y.y);
}

// Largest of a column's four lanes (l, l ^ 16, l ^ 32, l ^ 48), in all of them.
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ uint32_t column_max(uint32_t v) {
    v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    return max(v, (uint32_t)__shfl_xor((int)v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// 16 bytes that no other workgroup reads (6.9 against 6.2 TB/s over 512 MiB).
__device__ __forceinline__ uint4 load_once(const int8_t* p) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

template <int D, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, 2)
attention_few_kernel(const Problem p) {
    constexpr int kC = D / 64;                     // 16-byte pieces of a K row a lane
    constexpr int kDT = D / 16;                    // channel tiles
    __shared__ float lo[WAVES][16][D + 4];
    __shared__ float lm[WAVES][16], ll[WAVES][16];

    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int tile0 = split * p.split_tiles;
    // the wave's tiles are tile0 + wave + i * WAVES; the page numbers of 64 of them, one a lane
    const int32_t* table = p.page_table + (size_t)b * p.max_pages;
    auto page_numbers = [&](int i) {
        const int64_t at = (int64_t)tile0 + wave + (int64_t)(i + lane) * WAVES;
        return at < p.max_pages ? table[at] : -1;
    };
    int numbers = page_numbers(0);                 // needs no length: on its way beside them
    const Sequence s = sequence<true>(p, b);
    const int G = p.Hq / p.Hkv;
    const int rows = min(s.n, p.max_rows) * G;     // at most 16
    if (rows <= 0) return;
    const bool live = col < rows;
    const int t = live ? col / G : 0;
    const int head = h * G + (live ? col % G : 0);
    const int limit = !live ? 0 : p.causal ? min(max(s.kv - s.n + t + 1, 0), s.kv) : s.kv;
    const int last_t = (rows - 1) / G;
    const int least = p.causal ? min(max(s.kv - s.n + 1, 0), s.kv) : s.kv;
    const int most = p.causal ? min(max(s.kv - s.n + last_t + 1, 0), s.kv) : s.kv;
    const int tile1 = min((most + kPage - 1) / kPage, tile0 + p.split_tiles);
    if (p.splits > 1 && tile0 * kPage >= s.kv) return;     // the join does not read this piece

    const size_t block = (size_t)(2 * kPage * D);
    const uint32_t k_lane = (uint32_t)((col >> 2) * 16 + (col & 3)) * D + g * 16;
    const uint32_t v_lane = (uint32_t)col * kPage + g * 16;
    int index = -1, tile = 0;
    // this wave's next page that lies in the pool, -1 behind the last
    auto next = [&]() {
        for (;;) {
            tile = tile0 + wave + ++index * WAVES;
            if (tile >= tile1) return -1;
            if (index > 0 && (index & 63) == 0) numbers = page_numbers(index);
            const int page = __builtin_amdgcn_readlane(numbers, index & 63);
            if (page >= 0 && page < p.num_pages) return page;
        }
    };

    int page = next();
    uint4 k[4][kC], v[kDT];
    float sk = 0.0f, sv = 0.0f;
#define LOAD_K(page)                                                                            \
    {                                                                                           \
        const int8_t* src = p.codes + ((size_t)(page) * p.Hkv + h) * block;                     \
        _Pragma("unroll") for (int i = 0; i < 4; ++i)                                           \
            _Pragma("unroll") for (int cc = 0; cc < kC; ++cc) k[i][cc] =                        \
                load_once(src + ((i >> 1) * 8 + (i & 1) * 4) * D + cc * 64 + k_lane);           \
    }
#define LOAD_V(page)                                                                            \
    {                                                                                           \
        const int8_t* src = p.codes + ((size_t)(page) * p.Hkv + h) * block + kPage * D;         \
        _Pragma("unroll") for (int i = 0; i < kDT; ++i) v[i] =                                  \
            load_once(src + i * (16 * kPage) + v_lane);                                         \
    }
    if (page >= 0) {
        LOAD_K(page);
        LOAD_V(page);
        sk = p.scales[((size_t)page * p.Hkv + h) * 2];
        sv = p.scales[((size_t)page * p.Hkv + h) * 2 + 1];
    }

    uint4 high[kC], low[kC];
    // the softmax scale's sign goes to the query, so that exponents grow with the products
    float c = fabsf(p.sm) * kLog2e;
    {
        uint4 q[2 * kC];
        const uint16_t* src = p.Q + (size_t)(s.r0 + t) * p.ldq + (size_t)head * D + g * 16;
        const uint32_t flip = p.sm < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < 2 * kC; ++i) {
            q[i] = make_uint4(0, 0, 0, 0);
            if (live) q[i] = *reinterpret_cast<const uint4*>(src + (i >> 1) * 64 + (i & 1) * 8);
            q[i] = make_uint4(q[i].x ^ flip, q[i].y ^ flip, q[i].z ^ flip, q[i].w ^ flip);
        }
        c *= to_digits<kC>(q, column_max(abs_max_bits<2 * kC>(q)), high, low);
    }

    f32x4_acc o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i) o[i] = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f, top_lsv = -INFINITY;

    while (page >= 0) {
        const int at = tile * kPage;
        const float cz = c * sk, svc = fmaxf(sv, kMinVScale);
        const float lsv = __builtin_amdgcn_logf(svc), sv_inv = 1.0f / svc;
        // 256 * (high digits . K) + (low digits . K): |sums| < 2^30 for D = 128
        i32x4_acc zi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            zi[i] = {0, 0, 0, 0};
#pragma unroll
            for (int cc = 0; cc < kC; ++cc) zi[i] = mma16_i8(k[i][cc], high[cc], zi[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) zi[i][j] <<= 8;
#pragma unroll
            for (int cc = 0; cc < kC; ++cc) zi[i] = mma16_i8(k[i][cc], low[cc], zi[i]);
        }
        page = next();
        if (page >= 0) {
            LOAD_K(page);
            sk = p.scales[((size_t)page * p.Hkv + h) * 2];
            sv = p.scales[((size_t)page * p.Hkv + h) * 2 + 1];
        }
        f32x4_acc z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i][j] = (float)zi[i][j];
        const bool edge = at + kPage > least;      // some row does not see all of the page
        auto hide = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + 16 * g + 4 * i + j >= limit) z[i][j] = -INFINITY;
        };
        if (edge) hide();
        float top = z[0][0];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, z[i][j]);
        top = top == -INFINITY ? top : fmaf(cz, top, lsv);     // -inf: nothing visible
        if (__any(top > m + kLazy)) {
            const float m_new = fmaxf(m, column_max(top));
            const float alpha = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
            m = m_new;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= alpha;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        const float shift = lsv - base + kPShift;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i][j] = fmaf(cz, z[i][j], shift);
        if (edge) hide();                          // again: cz may be 0 or NaN
        float sum = 0.0f;
        top_lsv = fmaxf(top_lsv, lsv);
        if (scales_apart(lsv, top_lsv)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) l += __builtin_amdgcn_exp2f(z[i][j] - lsv);
            sum = -INFINITY;                       // marks l as done
        }
        uint4 pk[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a0 = __builtin_amdgcn_exp2f(z[2 * e + (j >> 1)][2 * (j & 1)]);
                const float a1 = __builtin_amdgcn_exp2f(z[2 * e + (j >> 1)][2 * (j & 1) + 1]);
                sum += a0 + a1;
                w[j] = pack_f16(a0, a1);
            }
            pk[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (sum != -INFINITY) l = fmaf(sum, sv_inv, l);
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
            o[i] = mma16(widen8(v[i].x, v[i].y), pk[0], o[i]);
            o[i] = mma16(widen8(v[i].z, v[i].w), pk[1], o[i]);
        }
        if (page >= 0) LOAD_V(page);
    }
#undef LOAD_K
#undef LOAD_V
    l = column_sum(l);
    if (g == 0) {
        lm[wave][col] = m;
        ll[wave][col] = l;
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, lm[w][col]);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int i = 0; i < kDT; ++i)
        *reinterpret_cast<float4*>(&lo[wave][col][i * 16 + g * 4]) =
            make_float4(o[i][0] * f, o[i][1] * f, o[i][2] * f, o[i][3] * f);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += WAVES * 64) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float best = -INFINITY, total = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) best = fmaxf(best, lm[w][r]);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float wm = lm[w][r];
            if (wm != -INFINITY) total = fmaf(ll[w][r], __builtin_amdgcn_exp2f(wm - best), total);
            const float4 x = *reinterpret_cast<const float4*>(&lo[w][r][d]);
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
        }
        const size_t row = (size_t)(s.r0 + r / G);
        const int hd = h * G + r % G;
        if (p.splits > 1) {
            const size_t to = (size_t)split * ((size_t)p.T * p.Hq) + row * p.Hq + hd;
            if (d == 0) p.part_ml[to] = make_float2(best, total);
            *reinterpret_cast<float4*>(p.part_o + to * D + d) = a;
        } else {
            const float k = row_factor(total);
            *reinterpret_cast<uint2*>(p.O + row * p.ldo + (size_t)hd * D + d) =
                make_uint2(pack_bf16(a.x * k, a.y * k), pack_bf16(a.z * k, a.w * k));
        }
    }
}

// Joins the pieces of the key axis in their order: one wave a (token, head) row.
template <int D, bool CACHE>
__global__ void __launch_bounds__(256) attention_join_kernel(const Problem p) {
    const int b = blockIdx.y, lane = threadIdx.x & 63;
    const Sequence s = sequence<CACHE>(p, b);
    const int idx = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int t = idx / p.Hq, head = idx % p.Hq;
    if (t >= min(s.n, p.max_rows)) return;
    const size_t stride = (size_t)p.T * p.Hq;
    const size_t at = (size_t)(s.r0 + t) * p.Hq + head;
    const int used = min(p.splits, ((s.kv + kPage - 1) / kPage + p.split_tiles - 1) /
                                       p.split_tiles);
    // the pieces' maxima and sums, 64 at a time, one a lane
    float m = -INFINITY, l = 0.0f, o[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) o[j] = 0.0f;
    for (int i0 = 0; i0 < used; i0 += 64) {
        const int n = min(used - i0, 64);
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < n) ml = p.part_ml[(size_t)(i0 + lane) * stride + at];
        float top = fmaxf(m, ml.x);
#pragma unroll
        for (int k = 32; k; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
        const float base = top == -INFINITY ? 0.0f : top;
        const float w = __builtin_amdgcn_exp2f(ml.x - base);
        const float alpha = __builtin_amdgcn_exp2f(m - base);
        m = top;
        float sum = ml.y * w;
#pragma unroll
        for (int k = 32; k; k >>= 1) sum += __shfl_xor(sum, k);
        l = fmaf(l, alpha, sum);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) o[j] *= alpha;
        const float* po = p.part_o + ((size_t)i0 * stride + at) * D + lane * (D / 64);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float wi =
                __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), i));
#pragma unroll
            for (int j = 0; j < D / 64; ++j) o[j] = fmaf(po[(size_t)i * stride * D + j], wi, o[j]);
        }
    }
    const float f = row_factor(l);
    uint16_t* d = p.O + (size_t)(s.r0 + t) * p.ldo + (size_t)head * D + lane * (D / 64);
    if (D == 128)
        *reinterpret_cast<uint32_t*>(d) = pack_bf16(o[0] * f, o[D / 64 - 1] * f);
    else
        *d = (uint16_t)(pack_bf16(o[0] * f, 0.0f) & 0xFFFFu);
}

// Pieces of the key axis, `tiles` tiles each.
struct Split {
    int splits, tiles;
};
Split pieces(int64_t wanted, int tiles, int least) {
    const int most = (tiles + least - 1) / least;
    const int splits = (int)(wanted < most ? wanted : most);
    if (splits <= 1) return {1, tiles > 0 ? tiles : 1};
    const int each = (tiles + splits - 1) / splits;
    return {(tiles + each - 1) / each, each};
}

constexpr int kFewRows = 16;
constexpr int kFewWaves = 4;

bool few_rows(int max_rows, int Hq, int Hkv) {
    return (int64_t)max_rows * (Hq / Hkv) <= kFewRows;
}

// Enough workgroups for the 256 compute units where sequences, heads and query rows give fewer.
// Few rows, measured with 16 heads of 128 channels, one sequence (us, pieces a head in brackets):
// 512 tokens 8.9 [1]; 777 tokens 12.2 [1], 10.6 [4]; 4096 tokens 17.8 [4], 14.1 [16]; 16384 tokens 23.3
// [16], 26 [32]; 65536 tokens 56 [32], 65 [64].  A single unit draws about 50 GB/s, so that up to
// 4096 tiles one workgroup a unit is best and above two; from 256 (sequence, head) pairs on, ragged
// lengths want shorter pieces (48 sequences of up to 8192 tokens, 8 heads: 110 [3], 135 [2]).
Split plan(bool cache, int B, int max_rows, int max_kv, int Hq, int Hkv, int D) {
    const int tiles = (int)(((int64_t)max_kv + kPage - 1) / kPage);
    if (cache && few_rows(max_rows, Hq, Hkv)) {
        const int64_t groups = (int64_t)B * Hkv;
        const int64_t total = groups * tiles;
        if (tiles * D <= 8 * 128) return {1, tiles > 0 ? tiles : 1};
        const int64_t want = groups >= 256 ? 1024 : total <= 4096 ? 256 : 512;
        return pieces((want + groups - 1) / groups, tiles, kFewWaves);
    }
    const int64_t groups =
        ((int64_t)max_rows * (Hq / Hkv) + kRows - 1) / kRows * Hkv * (int64_t)B;
    if (groups >= 512) return {1, tiles > 0 ? tiles : 1};
    return pieces((512 + groups - 1) / (groups > 0 ? groups : 1), tiles, 4);
}

template <int D, bool CACHE>
hipError_t launch(Problem p, int B, void* workspace, hipStream_t stream) {
    const Split sp = plan(CACHE, B, p.max_rows, p.max_kv, p.Hq, p.Hkv, D);
    p.splits = sp.splits;
    p.split_tiles = sp.tiles;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)sp.splits * p.T * p.Hq * D);
    bool few = false;
    if constexpr (CACHE) {
        few = few_rows(p.max_rows, p.Hq, p.Hkv);
        if (few && sp.splits == 1)
            attention_few_kernel<D, 8><<<dim3(1, p.Hkv, B), 512, 0, stream>>>(p);
        else if (few)
            attention_few_kernel<D, kFewWaves>
                <<<dim3(sp.splits, p.Hkv, B), kFewWaves * 64, 0, stream>>>(p);
    }
    if (!few) {
        const int64_t tiles = ((int64_t)p.max_rows * (p.Hq / p.Hkv) + kRows - 1) / kRows;
        attention_tile_kernel<D, CACHE>
            <<<dim3((unsigned)(tiles * sp.splits), p.Hkv, B), kThreads, 0, stream>>>(p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || sp.splits == 1) return e;
    attention_join_kernel<D, CACHE>
        <<<dim3((unsigned)(((int64_t)p.max_rows * p.Hq + 3) / 4), B), 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(int B, int T, int max_rows, int max_kv, int Hq, int Hkv, int D) {
    // one size for both calls
    int splits = 1;
    for (const bool cache : {false, true}) {
        const Split sp = plan(cache, B, max_rows < T ? max_rows : T, max_kv, Hq, Hkv, D);
        splits = splits > sp.splits ? splits : sp.splits;
    }
    if (splits == 1) return 0;
    return (size_t)splits * (size_t)T * (size_t)Hq * (size_t)(D + 2) * sizeof(float);
}

hipError_t launch_cache_attention(const uint16_t* Q, const int32_t* row_start,
                                  const int32_t* kv_len, const int32_t* page_table,
                                  const int8_t* codes, const float* scales, int B, int T,
                                  int max_rows, int max_kv, int max_pages, int num_pages, int Hq,
                                  int Hkv, int D, int ldq, int ldo, float sm, int causal,
                                  void* workspace, uint16_t* O, hipStream_t stream) {
    max_rows = max_rows < T ? max_rows : T;
    Problem p = {};
    p.Q = Q;
    p.row_start = row_start;
    p.kv_len = kv_len;
    p.page_table = page_table;
    p.codes = codes;
    p.scales = scales;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.T = T;
    p.max_rows = max_rows;
    p.max_kv = max_kv;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.causal = causal;
    p.ldq = ldq;
    p.ldo = ldo;
    p.sm = sm;
    p.O = O;
    return D == 64 ? launch<64, true>(p, B, workspace, stream)
                   : launch<128, true>(p, B, workspace, stream);
}

hipError_t launch_cross_attention(const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                                  const int32_t* row_start, const int32_t* kv_start,
                                  const int32_t* kv_len, int B, int T, int Tkv, int max_rows,
                                  int max_kv, int Hq, int Hkv, int D, int ldq, int ldk, int ldv,
                                  int ldo, float sm, void* workspace, uint16_t* O,
                                  hipStream_t stream) {
    max_rows = max_rows < T ? max_rows : T;
    Problem p = {};
    p.Q = Q;
    p.K = K;
    p.V = V;
    p.row_start = row_start;
    p.kv_start = kv_start;
    p.kv_len = kv_len;
    p.T = T;
    p.Tkv = Tkv;
    p.max_rows = max_rows;
    p.max_kv = max_kv;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldo = ldo;
    p.sm = sm;
    p.O = O;
    return D == 64 ? launch<64, false>(p, B, workspace, stream)
                   : launch<128, false>(p, B, workspace, stream);
}

}  // namespace rudder
