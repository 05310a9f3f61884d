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
// scaled by a power of two to a largest magnitude in [1, 2) and is then exact
// in fp16 down to 2^-17, and off by at most 2^-25 below.  The kernel for few
// rows multiplies the codes of K as they are, in integers, by q as two digits
// of 8 bits: its time is the codes' way from HBM, and what it spends beside
// that on widening them would show.  The K scale multiplies c.  The V scale sv is
// folded into the exponent: with t_j = z_j + log2(sv) and m the running
// maximum of t, P_j = exp2(t_j - m) multiplies plain codes, and
// l = sum P_j / sv.  P is rounded to fp16 (2^-11 relative, absolute 2^-33 below
// 2^-22), an eighth of what the output's rounding to bf16 adds; the sum l is formed from the
// unrounded values.  Products with bf16 states take P as the sum of two bf16 numbers.
#include <cmath>

#include "rudder_operators.h"

namespace rudder {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_acc __attribute__((ext_vector_type(16)));

constexpr int kPage = RUDDER_CACHE_PAGE;           // keys a tile
constexpr int kWaveRows = 32;                      // query rows a wave of the tile kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 8.0f;                    // cache: P and its sums are held times 2^8
// Smallest V scale the exponent takes: smaller ones (an all-zero block's 0) are read as this.
constexpr float kMinVScale = 8.271806125530277e-25f;   // 2^-80

// Smallest factor of a score over the cache: c or a K scale of 0 must leave masked scores at -inf.
// Codes times scaled queries stay below 2^30, so that the exponents it makes are zeros.
constexpr float kMinScale = 1e-30f;

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
    int B, T, max_rows, max_kv, Hq, Hkv, causal;
    size_t ldq, ldo;
    float sm;
    uint16_t* O;
    // Work units: `tile_rows` row tiles of each (head, sequence) pair.  The first `whole` of them
    // take all of their keys; the others are split into `pieces` of `piece_tiles` tiles whose
    // results are joined.
    int tile_rows, units, whole, pieces, piece_tiles, most_tiles;
    int dies, run, tile_major, descending;         // their order, see place()
    float* part_o;      // [pieces][units - whole][rows of a unit][D]
    float2* part_ml;    // [pieces][units - whole][rows of a unit]
};

// a / b of wave-uniform values, back in a scalar register (the division runs on the vector units)
__device__ __forceinline__ int quotient(int a, int b) {
    return __builtin_amdgcn_readfirstlane(a / b);
}

// Unit number -> row tile of a pair.  Workgroups go round robin to the eight dies: where the pairs
// divide by eight, the units of a pair, which read the same keys, are kept on one (dies = 8, else
// 1).  A pair's tiles follow each other, causal ones, whose lengths differ, longest first
// (descending = 1); where the keys of a die take at most half its L2 they go longest first over all
// its pairs (tile_major = 1), which ends more evenly: 4096 causal rows of 16 heads over 4096 tokens
// 126 us, pair by pair 162; over 16384 tokens, 2 x 4096 rows, 1077 against 918.  Chosen by
// arithmetic: a branch by p.causal made two kernels of one and cost 50 registers.
struct Place {
    int h, b, tile;
};
__device__ __forceinline__ Place place(const Problem& p, int unit) {
    const int slot = quotient(unit, p.dies), low = unit - slot * p.dies;
    const int q = quotient(slot, p.run), r = slot - q * p.run;
    const int pair = low + p.dies * (q + p.tile_major * (r - q));
    const int up = r + p.tile_major * (q - r);
    const int tile = up + p.descending * (p.tile_rows - 1 - 2 * up);
    const int b = quotient(pair, p.Hkv);
    return {pair - b * p.Hkv, b, tile};
}

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

// Weights as operands: for the cache in fp16.  For states in bf16, whose 8 bits alone would put as
// much into the outputs as their own rounding does (error 2.3e-3 against 1.7e-3 of their norm): a
// second operand holds what that rounding left, in bf16 again, so that a weight is off by 2^-16 of
// itself.  It costs half as many products again (2 x 4192 rows of 16 heads of 128 channels over 512
// keys 67 us, 56 without).
template <bool CACHE>
__device__ __forceinline__ uint32_t pack_weights(float a, float b, uint32_t& rest) {
    if (CACHE) return pack_f16(a, b);
    const uint32_t w = pack_bf16(a, b);
    rest = pack_bf16(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xFFFF0000u));
    return w;
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

// A query row whose largest magnitude has the bf16 bits `top` = f * 2^e, f in [1, 2), to fp16 times
// 2^-e.  Returns 2^e.  Between -120 and 120: rows below keep their last bit, 2^-133, above fp16's
// 2^-24, rows above stay below its largest number.
template <int N>
__device__ __forceinline__ float to_f16(uint4 (&q)[N], uint32_t top) {
    const int e = min(max((int)(top >> 7) - 127, -120), 120);
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

// Scores of bf16 queries may be of any size, and a factor c of 0 must still leave masked ones at
// -inf: there the query becomes 0 and the factor 1.
template <int N>
__device__ __forceinline__ float scale_of_zero(uint4 (&q)[N], float c) {
    if (c != 0.0f) return c;
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = make_uint4(0, 0, 0, 0);
    return 1.0f;
}

// A query row whose largest magnitude has the bf16 bits `top` = f * 2^e, f in [1, 2), as integers
// q * 2^(14 - e) in [-32639, 32639] and these as two digits, 256 * high + low: N pairs of 16 bytes
// (16 channels) become one of each.  Returns 2^(e - 14).  Subnormal rows count as e = -126, which
// leaves them exact.
template <int N>
__device__ __forceinline__ float to_digits(const uint4 (&q)[2 * N], uint32_t top, uint4 (&high)[N],
                                           uint4 (&low)[N]) {
    const int e = min(max((int)(top >> 7) - 127, -126), 127);
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
                const int x = quantize_clamped(__builtin_amdgcn_ldexpf(f[j], 14 - e), 32639.0f);
                h[j] = (x + 128) >> 8;
                l[j] = x - 256 * h[j];
            }
            hw[d] = byte_word(h);
            lw[d] = byte_word(l);
        }
        high[i] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        low[i] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
    return __builtin_amdgcn_ldexpf(1.0f, e - 14);
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

// One tile of 64 keys on its way from HBM to LDS, THREADS threads.  LDS holds the operands of the
// products: K rows at their accumulator rows, V as [channel][key], 16 bytes behind each row so that
// 16 rows start at 16 places of the 64 banks.
template <int D, bool CACHE, int THREADS>
struct Stage {
    static constexpr int kKStride = D * 2 + 16;            // bytes of a key's row
    static constexpr int kVStride = kPage * 2 + 16;        // bytes of a channel's row
    static constexpr int kKBytes = kPage * kKStride;
    static constexpr int kBytes = kKBytes + D * kVStride;
    static constexpr int kUnits = CACHE ? kPage * D / 16 : kPage * D / 8;  // 16-byte pieces of K
    static constexpr int kNK = (kUnits + THREADS - 1) / THREADS;
    // states: a thread takes kKeys keys x eight channels of V
    static constexpr int kKeys = kPage * D / 8 / THREADS > 2 ? 4 : 2;
    static constexpr int kVUnits = CACHE ? kUnits : kPage / kKeys * (D / 8);
    static constexpr int kNV = CACHE ? kNK : kKeys;
    uint4 k[kNK], v[kNV];

    static constexpr int kGroups = kPage / kKeys;          // of keys
    // a wave takes 64 bytes of 16 or 32 rows: whole sectors, and transposed writes whose lanes
    // differ in their keys
    static __device__ __forceinline__ int v_channel(int tid) {
        return (tid % 4 + tid / (4 * kGroups) * 4) * 8;
    }
    static __device__ __forceinline__ int v_key(int tid) { return tid / 4 % kGroups * kKeys; }

    // page: the tile's page number (cache); key0: its first key (states)
    __device__ __forceinline__ void load(const Problem& p, const Sequence& s, int h, int page,
                                         int key0) {
        const int tid = threadIdx.x;
        if constexpr (CACHE) {
            const int8_t* src = p.codes + ((size_t)page * p.Hkv + h) * (size_t)(2 * kPage * D);
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * THREADS;
                if (kUnits % THREADS == 0 || u < kUnits) {
                    k[i] = *reinterpret_cast<const uint4*>(src + u * 16);
                    v[i] = *reinterpret_cast<const uint4*>(src + kPage * D + u * 16);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * THREADS, key = key0 + u / (D / 8);
                k[i] = make_uint4(0, 0, 0, 0);
                if (key < s.kv)
                    k[i] = *reinterpret_cast<const uint4*>(
                        p.K + (size_t)(s.kv0 + key) * p.ldk + (size_t)h * D + u % (D / 8) * 8);
            }
            if (kVUnits % THREADS == 0 || tid < kVUnits) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    const int key = key0 + v_key(tid) + i;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (key < s.kv)
                        v[i] = *reinterpret_cast<const uint4*>(
                            p.V + (size_t)(s.kv0 + key) * p.ldv + (size_t)h * D + v_channel(tid));
                }
            }
        }
    }

    __device__ __forceinline__ void store(uint8_t* lds) const {
        const int tid = threadIdx.x;
        uint8_t* lv = lds + kKBytes;
        if constexpr (CACHE) {
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * THREADS;
                if (kUnits % THREADS == 0 || u < kUnits) {
                    uint8_t* d = lds + swap23(u / (D / 16)) * kKStride + u % (D / 16) * 32;
                    put(d, d + 16, k[i]);
                    d = lv + u / 4 * kVStride + u % 4 * 32;
                    put(d, d + 16, v[i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kNK; ++i) {
                const int u = tid + i * THREADS;
                *reinterpret_cast<uint4*>(lds + swap23(u / (D / 8)) * kKStride +
                                          u % (D / 8) * 16) = k[i];
            }
            if (kVUnits % THREADS == 0 || tid < kVUnits) {
                uint8_t* d = lv + v_channel(tid) * kVStride + v_key(tid) * 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[kKeys];
#pragma unroll
                    for (int i = 0; i < kKeys; ++i)
                        w[i] = j == 0 ? v[i].x : j == 1 ? v[i].y : j == 2 ? v[i].z : v[i].w;
                    put_keys(d + 2 * j * kVStride, w);
                }
            }
        }
    }

    // Two channels of kKeys keys, transposed.
    static __device__ __forceinline__ void put_keys(uint8_t* d, const uint32_t (&w)[kKeys]) {
        uint32_t lo[kKeys / 2], hi[kKeys / 2];
#pragma unroll
        for (int i = 0; i < kKeys / 2; ++i) {
            lo[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100u);
            hi[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302u);
        }
        if constexpr (kKeys == 4) {
            *reinterpret_cast<uint2*>(d) = make_uint2(lo[0], lo[1]);
            *reinterpret_cast<uint2*>(d + kVStride) = make_uint2(hi[0], hi[1]);
        } else {
            *reinterpret_cast<uint32_t*>(d) = lo[0];
            *reinterpret_cast<uint32_t*>(d + kVStride) = hi[0];
        }
    }

    static __device__ __forceinline__ void put(uint8_t* d0, uint8_t* d1, uint4 c) {
        const uint2 a = widen4(c.x), b = widen4(c.y), e = widen4(c.z), f = widen4(c.w);
        *reinterpret_cast<uint4*>(d0) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(d1) = make_uint4(e.x, e.y, f.x, f.y);
    }
};

// Order of a block of N products, their N LDS reads and the vector work beside them: reads four
// products ahead, four vector instructions a product.
template <int N>
__device__ __forceinline__ void interleave() {
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);     // LDS reads
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); // a product
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x400, 1, 0); // an exponential
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0); // vector instructions
    }
}

// The running maximum is raised only where a score passes it by more than 2^6 (P has room for it):
// most tiles then need no exchange between lanes and no rescaling of O.
constexpr float kLazy = 6.0f;

// Orders a wave's LDS accesses of different lanes (the hardware keeps their order; this keeps the
// compiler's).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The 32 query rows of a wave pass through LDS, so that global memory sees whole rows: a lane's
// share of its row is 16 bytes in 32 (loads) or 8 in 16 (stores).  2 x 4192 rows of 16 heads over
// 128 keys (with weights of one operand) 28.8 us, 33.9 without.
template <int D>
struct RowSlab {
    static constexpr int kStride = D * 2 + 16, kBytes = kWaveRows * kStride;
    static constexpr int kPartBytes = kWaveRows * (D * 4 + 16);    // of partial rows in 32 bits
    static constexpr int kPieces = D / 8, kRowsAtOnce = 64 / kPieces;

    // Lane l's row (token t, head) for l < 32, on its way to registers ...
    uint4 x[kWaveRows / kRowsAtOnce];
    __device__ __forceinline__ void fetch(const Problem& p, const Sequence& s, int t, int head) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < kWaveRows / kRowsAtOnce; ++i) {
            const int r = i * kRowsAtOnce + lane / kPieces;
            const int rt = __shfl(t, r), rh = __shfl(head, r);
            x[i] = *reinterpret_cast<const uint4*>(p.Q + (size_t)(s.r0 + rt) * p.ldq +
                                                   (size_t)rh * D + lane % kPieces * 8);
        }
    }
    // ... and as the lanes' operands of the first product.
    __device__ __forceinline__ void operands(uint8_t* slab, uint4 (&q)[D / 16]) const {
        const int lane = threadIdx.x & 63, piece = lane % kPieces;
#pragma unroll
        for (int i = 0; i < kWaveRows / kRowsAtOnce; ++i)
            *reinterpret_cast<uint4*>(slab + (i * kRowsAtOnce + lane / kPieces) * kStride +
                                      piece * 16) = x[i];
        wave_sync();
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            q[i] = *reinterpret_cast<const uint4*>(slab + (lane & 31) * kStride +
                                                   (lane >> 5) * 16 + i * 32);
    }

    // O times f of the rows that are live.
    static __device__ __forceinline__ void store(const Problem& p, const Sequence& s, uint8_t* slab,
                                                 int t, int head, bool live, float f,
                                                 const f32x16_acc (&o)[D / 32]) {
        const int lane = threadIdx.x & 63, piece = lane % kPieces;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<uint2*>(slab + (lane & 31) * kStride +
                                          (dt * 32 + g * 8 + (lane >> 5) * 4) * 2) =
                    make_uint2(pack_bf16(o[dt][4 * g] * f, o[dt][4 * g + 1] * f),
                               pack_bf16(o[dt][4 * g + 2] * f, o[dt][4 * g + 3] * f));
        wave_sync();
#pragma unroll
        for (int i = 0; i < kWaveRows / kRowsAtOnce; ++i) {
            const int r = i * kRowsAtOnce + lane / kPieces;
            const int rt = __shfl(t, r), rh = __shfl(head, r), there = __shfl((int)live, r);
            const uint4 x = *reinterpret_cast<const uint4*>(slab + r * kStride + piece * 16);
            if (there)
                *reinterpret_cast<uint4*>(p.O + (size_t)(s.r0 + rt) * p.ldo + (size_t)rh * D +
                                          piece * 8) = x;
        }
    }
};

// A wave's rows: their outputs, or for a piece of the keys their partial results.  Every lane comes
// here; `slab` is the wave's own.
template <int D>
__device__ __forceinline__ void write_rows(const Problem& p, const Sequence& s, uint8_t* slab,
                                           int split, int unit, int rest, int unit_rows,
                                           int unit_row, int t, int head, bool live, float m,
                                           float l, const f32x16_acc (&o)[D / 32]) {
    if (split < 0) {
        RowSlab<D>::store(p, s, slab, t, head, live, row_factor(l), o);
        return;
    }
    // through LDS as well, a wave's partial rows lie behind each other (1500 rows of 16 heads of
    // 128 channels over 2048 keys, in two pieces and with weights of one operand: 51.6 us, 54.2
    // without)
    constexpr int kStride = D * 4 + 16, kPieces = D / 4, kRowsAtOnce = 64 / kPieces;
    const int lane = threadIdx.x & 63;
    const size_t first = ((size_t)split * rest + (unit - p.whole)) * unit_rows + unit_row;
    if (live && lane < kWaveRows) p.part_ml[first] = make_float2(m, l);
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<float4*>(slab + (lane & 31) * kStride +
                                       (dt * 32 + g * 8 + (lane >> 5) * 4) * 4) =
                make_float4(o[dt][4 * g], o[dt][4 * g + 1], o[dt][4 * g + 2], o[dt][4 * g + 3]);
    wave_sync();
    // the wave's rows are consecutive, those that are not live the last ones
    const int rows = __popcll(__ballot(live && lane < kWaveRows));
    float* to = p.part_o + (first - (lane & 31)) * D + lane * 4;
#pragma unroll
    for (int i = 0; i < kWaveRows / kRowsAtOnce; ++i) {
        const int r = i * kRowsAtOnce + lane / kPieces;
        if (r < rows)
            *reinterpret_cast<float4*>(to + i * 256) =
                *reinterpret_cast<const float4*>(slab + r * kStride + lane % kPieces * 16);
    }
}

// ---------------------------------------------------------------------------
// Many rows: 128 of them a workgroup, four waves of 32 that share the tiles through LDS.
// ---------------------------------------------------------------------------
// A wave's 32 rows meet 32 keys in 2 D / 16 products of 32 cycles (states 3 D / 16); beside them
// stand, a lane, 16 exponentials of 16 cycles and about 80 vector instructions of 4 (scaling,
// maximum, sum, rounding, the codes' share of widening; states 120).  The pipeline over halves of
// tiles lets the two overlap within a wave, the second workgroup of the compute unit fills the
// barriers.  2 x 4192 rows of 16 heads of 128 channels over 512 states 68 us (430 TFLOP/s: eight
// tiles against one load and one store of the rows, 69 MB, and half as many products again as are
// counted here); 2 x 96 rows over 33536 cached tokens 103 us (515, and 685 counting the quarter of
// the rows that is empty).  Neither unit is half busy there (matrix cores 22 to 29%, vector units
// 44%): a wave's score products are two chains of D / 16 one behind the other, its tiles one
// ahead of its loads.
// 64 channels leave room for three workgroups a compute unit: the exponentials weigh twice as much
// there as with 128, and a third wave fills what two leave of the vector units, for four registers
// spilled outside of the loop (2 x 4096 causal rows of 24 heads over 4096 tokens 168 us, with two
// 215; 8 x 2000 over 2000 131 against 154).
template <int D, bool CACHE>
__global__ void __launch_bounds__(256, D == 64 ? 3 : 2)
attention_tile_kernel(const Problem p) {
    using St = Stage<D, CACHE, 256>;
    static_assert(4 * RowSlab<D>::kBytes <= St::kBytes, "a wave's rows fit beside a tile");
    static_assert(4 * RowSlab<D>::kPartBytes <= 2 * St::kBytes, "and its results in both");
    constexpr int kRows = 4 * kWaveRows;
    constexpr int kKS = D / 16;                    // steps of the first product
    constexpr int kDT = D / 32;                    // channel tiles of the second
    __shared__ __align__(16) uint8_t lds[2 * St::kBytes];

    const int rest = p.units - p.whole;            // split units
    const int split = (int)blockIdx.x < p.whole ? -1 : quotient(blockIdx.x - p.whole, rest);
    const int unit = split < 0 ? blockIdx.x : blockIdx.x - split * rest;
    const Place at_unit = place(p, unit);
    const int h = at_unit.h, b = at_unit.b, tile_row = at_unit.tile;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int tile0 = max(split, 0) * p.piece_tiles;
    // page numbers of 64 tiles, one a lane
    const int32_t* table = CACHE ? p.page_table + (size_t)b * p.max_pages : nullptr;
    auto page_numbers = [&](int i) {
        const int64_t at = (int64_t)tile0 + i + lane;
        return CACHE && at < p.max_pages ? table[at] : -1;
    };
    int numbers = page_numbers(0);
    const Sequence s = sequence<CACHE>(p, b);
    const int G = quotient(p.Hq, p.Hkv);
    const int rows = min(s.n, p.max_rows) * G;     // (token, head of the group) pairs
    if (tile_row * kRows >= rows) return;

    // this lane's query row and the keys it sees; the least and most any row of the wave sees
    const int row0 = tile_row * kRows + wave * kWaveRows, row = row0 + (lane & 31);
    const bool live = row < rows;
    const int t = live ? row / G : 0;
    const int head = h * G + (live ? row % G : 0);
    auto sees = [&](int tt) { return p.causal ? min(max(s.kv - s.n + tt + 1, 0), s.kv) : s.kv; };
    const int limit = live ? sees(t) : 0;
    const int least = sees(quotient(row0, G));
    const int wave_most = row0 < rows ? sees(quotient(min(rows, row0 + kWaveRows) - 1, G)) : 0;
    const int most = sees(quotient(min(rows, (tile_row + 1) * kRows) - 1, G));
    const int tile1 = min((most + kPage - 1) / kPage,
                          tile0 + (split < 0 ? p.most_tiles : p.piece_tiles));
    if (split >= 0 && tile0 * kPage >= s.kv) return;       // the join does not read this piece

    int index = -1;
    // the next tile's page that lies in the pool, -1 behind the last tile
    auto next = [&]() {
        for (;;) {
            if (tile0 + ++index >= tile1) return -1;
            if (!CACHE) return 0;
            if (index > 0 && (index & 63) == 0) numbers = page_numbers(index);
            const int page = __builtin_amdgcn_readlane(numbers, index & 63);
            if (page >= 0 && page < p.num_pages) return page;
        }
    };
    St stage;
    int page = -1, next_at = 0;
    float sk = 1.0f, sv = 1.0f;
    auto load = [&]() {                            // the next tile, on its way to registers
        page = next();
        if (page < 0) return;
        next_at = (tile0 + index) * kPage;
        stage.load(p, s, h, page, next_at);
        if (CACHE) {
            const float* sc = p.scales + ((size_t)page * p.Hkv + h) * 2;
            sk = sc[0];
            sv = sc[1];
        }
    };
    load();                                        // on its way beside the query rows

    uint4 q[kKS];
    float l = 0.0f;                                // the lane's share of the sum of weights
    // the softmax scale's sign goes to the query, so that exponents grow with the products
    float c = fabsf(p.sm) * kLog2e;
    {
        // the second tile's place is free until a barrier has passed
        RowSlab<D> rows_in;
        rows_in.fetch(p, s, t, head);
        rows_in.operands(lds + St::kBytes + wave * RowSlab<D>::kBytes, q);
        const uint32_t flip = p.sm < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < kKS; ++i) {
            q[i] = make_uint4(q[i].x ^ flip, q[i].y ^ flip, q[i].z ^ flip, q[i].w ^ flip);
        }
        uint32_t top = abs_max_bits<kKS>(q);
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        if (top >= 0x7F80u && limit > 0) l = __uint_as_float(0x7FC00000u);    // not finite
        if (CACHE)
            c *= to_f16<kKS>(q, top);
        else
            c = scale_of_zero<kKS>(q, c);
    }

    f32x16_acc o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -INFINITY, top_lsv = -INFINITY;

    // scores of 32 keys: register j holds key 16 (j / 8) + 8 half + j % 8
    const int k_lane = (lane & 31) * St::kKStride + half * 16;
    const int v_lane = St::kKBytes + (lane & 31) * St::kVStride + half * 16;
    auto scores = [&](const uint8_t* tile, int hf) {
        f32x16_acc z;
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kKS; ++i)
            z = mma<CACHE>(*reinterpret_cast<const uint4*>(tile + k_lane + hf * 32 * St::kKStride +
                                                           i * 32), q[i], z);
        return z;
    };
    // P of the 32 keys before, and its rest (states)
    uint4 pend0 = make_uint4(0, 0, 0, 0), pend1 = pend0, rest0 = pend0, rest1 = pend0;
    auto nothing_pending = [&]() { pend0 = pend1 = rest0 = rest1 = make_uint4(0, 0, 0, 0); };
    auto weigh = [&](const uint8_t* tile, int hf) {        // O += V P of these
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
            const uint8_t* v = tile + v_lane + dt * 32 * St::kVStride + hf * 64;
            const uint4 v0 = *reinterpret_cast<const uint4*>(v);
            const uint4 v1 = *reinterpret_cast<const uint4*>(v + 32);
            o[dt] = mma<CACHE>(v0, pend0, o[dt]);
            if (!CACHE) o[dt] = mma<CACHE>(v0, rest0, o[dt]);
            o[dt] = mma<CACHE>(v1, pend1, o[dt]);
            if (!CACHE) o[dt] = mma<CACHE>(v1, rest1, o[dt]);
        }
    };

    // Software pipeline over halves of tiles: while the weights of 32 keys are formed on the vector
    // units, the matrix cores work on the scores of the next 32 and the values of the last 32.
    if (page >= 0) {
        uint8_t* cur = lds;                        // holds the tile at hand
        uint8_t* old = lds;                        // the one before
        int slot = 0;
        stage.store(cur);
        int at = next_at;
        float cz = 0.0f, lsv = 0.0f, sv_inv = 1.0f;
        auto scales = [&]() {
            cz = CACHE ? fmaxf(c * sk, kMinScale) : c;
            const float svc = CACHE ? fmaxf(sv, kMinVScale) : 1.0f;
            lsv = CACHE ? __builtin_amdgcn_logf(svc) : 0.0f;       // log2
            sv_inv = CACHE ? 1.0f / svc : 1.0f;
        };
        scales();
        load();
        __syncthreads();
        f32x16_acc z;
        if (at < wave_most) z = scores(cur, 0);
        bool mine = at < wave_most;                // some row of this wave sees the tile at hand

        // z, the scores of half hf, become weights; `ahead` runs the products beside
        auto step = [&](int hf, auto ahead, const uint8_t* before, int before_hf) {
            const int key0 = at + 32 * hf;
            if (key0 + 32 > least) {               // some row does not see all of these keys
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (key0 + 16 * (j >> 3) + 8 * half + (j & 7) >= limit) z[j] = -INFINITY;
            }
            float top = z[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, z[j]);
            top = fmaf(cz, top, lsv);              // -inf: nothing visible
            if (__any(top > m + kLazy)) {
                weigh(before, before_hf);          // still under the old maximum
                nothing_pending();
                const float m_new = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
                const float alpha = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
                m = m_new;
                l *= alpha;
#pragma unroll
                for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[dt][j] *= alpha;
            }
            // P = exp2(c z + log2(sv) - m), for the cache times 2^8
            const float shift = lsv - (m == -INFINITY ? 0.0f : m) + (CACHE ? kPShift : 0.0f);
            bool apart = false;
            if (CACHE) {
                top_lsv = fmaxf(top_lsv, lsv);
                apart = scales_apart(lsv, top_lsv);
                if (apart)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        l += __builtin_amdgcn_exp2f(fmaf(cz, z[j], shift - lsv));
            }
            f32x16_acc zn = ahead();
            weigh(before, before_hf);
            float sum = 0.0f;
            uint32_t w[8], r[8] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = __builtin_amdgcn_exp2f(fmaf(cz, z[2 * j], shift));
                const float e = __builtin_amdgcn_exp2f(fmaf(cz, z[2 * j + 1], shift));
                sum += a + e;
                w[j] = pack_weights<CACHE>(a, e, r[j]);
            }
            interleave<(CACHE ? 2 : 4) * kDT + kKS>();
            l = fmaf(sum, apart ? 0.0f : sv_inv, l);
            pend0 = make_uint4(w[0], w[1], w[2], w[3]);
            pend1 = make_uint4(w[4], w[5], w[6], w[7]);
            rest0 = make_uint4(r[0], r[1], r[2], r[3]);
            rest1 = make_uint4(r[4], r[5], r[6], r[7]);
            z = zn;
        };
        for (;;) {
            if (mine) step(0, [&]() { return scores(cur, 1); }, old, 1);
            __syncthreads();                       // the tile before has been read
            const bool more = page >= 0;
            uint8_t* ahead = cur;
            const int ahead_at = next_at;
            const float sk1 = sk, sv1 = sv;
            if (more) {
                slot ^= 1;
                ahead = lds + slot * St::kBytes;
                stage.store(ahead);
                load();
            }
            __syncthreads();
            const bool mine_next = more && ahead_at < wave_most;
            if (mine_next)
                step(1, [&]() { return scores(ahead, 0); }, cur, 0);
            else if (mine) {
                step(1, [&]() { return z; }, cur, 0);
                weigh(cur, 1);                     // the wave's last keys
                nothing_pending();
            }
            if (!more) break;
            old = cur;
            cur = ahead;
            at = ahead_at;
            mine = mine_next;
            {
                const float sk2 = sk, sv2 = sv;
                sk = sk1;
                sv = sv1;
                scales();
                sk = sk2;
                sv = sv2;
            }
        }
    }
    l += __shfl_xor(l, 32);
    __syncthreads();                               // the tiles have been read
    write_rows<D>(p, s, lds + wave * RowSlab<D>::kPartBytes, split, unit, rest, kRows,
                  row - tile_row * kRows, t, head, live, m, l, o);
}

// ---------------------------------------------------------------------------
// Very many rows: 256 of them a workgroup, two groups of four waves in opposite phases.
// ---------------------------------------------------------------------------
// A wave alternates between a phase of products (scores of the next tile, values of this one) and a
// phase of vector work (weights of the next tile, staging of a later one).  Waves w and w + 4 share
// a vector unit and a matrix core and are one phase apart, kept so by a barrier a phase: one has
// the matrix core while the other has the vector unit.  Tile i lives in slot i % 4 of LDS: group
// A's phases of tile i are 2 i (products: K of i + 1, V of i) and 2 i + 1 (stores i + 3), B's one
// later, so that slot (i + 3) % 4 = (i - 1) % 4 was last read in phase 2 i - 1 and is first read in
// 2 i + 4.
// 2 x 4192 rows of 16 heads over 12576 cached tokens 920 to 980 us, card by card, 880 to 930 TFLOP/s
// (a library product of as many operations 715 to 750): the matrix cores are busy 39% of the time,
// the vector units half of it, LDS 28%; the longer of the two phases sets the pace.  States: 2 x
// 4700 rows over 8000 and 6280 834 us, 660 TFLOP/s, 990 with the products of the weights' second
// operand.  Raised wave priorities, hints to the scheduler and other pairs of waves measured the
// same or slower (1019, 1040 and 1112 against 1019 on one card).
template <int D, bool CACHE>
__global__ void __launch_bounds__(512, 2)
attention_wide_kernel(const Problem p) {
    using St = Stage<D, CACHE, 512>;
    static_assert(8 * RowSlab<D>::kBytes <= 2 * St::kBytes, "a wave's rows fit beside two tiles");
    static_assert(8 * RowSlab<D>::kPartBytes <= 4 * St::kBytes, "and its results in all four");
    constexpr int kRows = 8 * kWaveRows;
    constexpr int kKS = D / 16, kDT = D / 32;
    __shared__ __align__(16) uint8_t lds[4 * St::kBytes];
    __shared__ float2 lds_scale[4];
    __shared__ int lds_at[4];

    const int rest = p.units - p.whole;            // split units
    const int split = (int)blockIdx.x < p.whole ? -1 : quotient(blockIdx.x - p.whole, rest);
    const int unit = split < 0 ? blockIdx.x : blockIdx.x - split * rest;
    const Place at_unit = place(p, unit);
    const int h = at_unit.h, b = at_unit.b, tile_row = at_unit.tile;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int tile0 = max(split, 0) * p.piece_tiles;
    // page numbers of 64 tiles, one a lane
    const int32_t* table = CACHE ? p.page_table + (size_t)b * p.max_pages : nullptr;
    auto page_numbers = [&](int i) {
        const int64_t at = (int64_t)tile0 + i + lane;
        return CACHE && at < p.max_pages ? table[at] : -1;
    };
    int numbers = page_numbers(0);
    const Sequence s = sequence<CACHE>(p, b);
    const int G = quotient(p.Hq, p.Hkv);
    const int rows = min(s.n, p.max_rows) * G;     // (token, head of the group) pairs
    if (tile_row * kRows >= rows) return;

    // this lane's query row and the keys it sees; the least and most any row of the wave sees
    const int row0 = tile_row * kRows + wave * kWaveRows, row = row0 + (lane & 31);
    const bool live = row < rows;
    const int t = live ? row / G : 0;
    const int head = h * G + (live ? row % G : 0);
    auto sees = [&](int tt) { return p.causal ? min(max(s.kv - s.n + tt + 1, 0), s.kv) : s.kv; };
    const int limit = live ? sees(t) : 0;
    const int least = sees(quotient(row0, G));
    const int wave_most = row0 < rows ? sees(quotient(min(rows, row0 + kWaveRows) - 1, G)) : 0;
    const int most = sees(quotient(min(rows, (tile_row + 1) * kRows) - 1, G));
    const int tile1 = min((most + kPage - 1) / kPage,
                          tile0 + (split < 0 ? p.most_tiles : p.piece_tiles));
    if (split >= 0 && tile0 * kPage >= s.kv) return;       // the join does not read this piece

    int index = -1;
    // the next tile's page that lies in the pool, -1 behind the last tile
    auto next = [&]() {
        for (;;) {
            if (tile0 + ++index >= tile1) return -1;
            if (!CACHE) return 0;
            if (index > 0 && (index & 63) == 0) numbers = page_numbers(index);
            const int page = __builtin_amdgcn_readlane(numbers, index & 63);
            if (page >= 0 && page < p.num_pages) return page;
        }
    };
    St stage;
    int page = 0, stage_at = 0, stored = 0;        // page < 0: no tile is on its way
    float sk = 1.0f, sv = 1.0f;
    auto load = [&]() {                            // the next tile, on its way to registers
        page = page < 0 ? -1 : next();
        if (page < 0) return;
        stage_at = (tile0 + index) * kPage;
        stage.load(p, s, h, page, stage_at);
        if (CACHE) {
            const float* sc = p.scales + ((size_t)page * p.Hkv + h) * 2;
            sk = sc[0];
            sv = sc[1];
        }
    };
    auto store = [&]() {                           // the tile in registers, to its slot
        if (page < 0) return;
        const int slot = stored & 3;
        stage.store(lds + slot * St::kBytes);
        if (threadIdx.x == 0) {
            lds_scale[slot] = make_float2(sk, sv);
            lds_at[slot] = stage_at;
        }
        ++stored;
    };
    // the query rows in front of the first tile or behind it: the same within 1%; the tile kernel
    // prefers the latter (105 against 108 on 2 x 96 rows)
    RowSlab<D> rows_in;
    rows_in.fetch(p, s, t, head);
    load();

    uint4 q[kKS];
    float l = 0.0f;                                // the lane's share of the sum of weights
    // the softmax scale's sign goes to the query, so that exponents grow with the products
    float c = fabsf(p.sm) * kLog2e;
    {
        // the third and fourth tile's places are free until a barrier has passed
        rows_in.operands(lds + 2 * St::kBytes + wave * RowSlab<D>::kBytes, q);
        const uint32_t flip = p.sm < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < kKS; ++i) {
            q[i] = make_uint4(q[i].x ^ flip, q[i].y ^ flip, q[i].z ^ flip, q[i].w ^ flip);
        }
        uint32_t top = abs_max_bits<kKS>(q);
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        if (top >= 0x7F80u && limit > 0) l = __uint_as_float(0x7FC00000u);    // not finite
        if (CACHE)
            c *= to_f16<kKS>(q, top);
        else
            c = scale_of_zero<kKS>(q, c);
    }

    f32x16_acc o[kDT], z[2];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    uint4 pk[4], rest_k[4];                        // P, and its rest (states)
    float m = -INFINITY, top_lsv = -INFINITY;
    const int k_lane = (lane & 31) * St::kKStride + half * 16;
    const int v_lane = St::kKBytes + (lane & 31) * St::kVStride + half * 16;

    store();
    load();
    store();
    load();                                        // two tiles in LDS, the third on its way
    __syncthreads();
    if (wave >= 4) __syncthreads();                // group B: one phase behind
    bool now = false;                              // the wave sees the tile whose V is next
    for (int i = -1;; ++i) {
        // Phase of products.  Tile i + 1 is there if it has been stored: `stored` is the same in
        // both groups where it is compared with i + 1, the tiles up to i + 2 being decided.
        const bool more = i + 1 < stored;
        const uint8_t* kt = lds + ((i + 1) & 3) * St::kBytes;
        const uint8_t* vt = lds + (i & 3) * St::kBytes;
        const int at = more ? __builtin_amdgcn_readfirstlane(lds_at[(i + 1) & 3]) : 0;
        const bool ahead = more && at < wave_most;
        if (ahead) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                for (int j = 0; j < 16; ++j) z[tt][j] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kKS; ++k)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
                    z[tt] = mma<CACHE>(*reinterpret_cast<const uint4*>(
                                           kt + k_lane + tt * 32 * St::kKStride + k * 32),
                                       q[k], z[tt]);
        }
        if (now)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int dt = 0; dt < kDT; ++dt) {
                    const uint4 v = *reinterpret_cast<const uint4*>(
                        vt + v_lane + dt * 32 * St::kVStride + ks * 32);
                    o[dt] = mma<CACHE>(v, pk[ks], o[dt]);
                    if (!CACHE) o[dt] = mma<CACHE>(v, rest_k[ks], o[dt]);
                }
        __syncthreads();
        if (!more) break;
        // Phase of vector work: tile i + 3 to LDS, the one behind on its way, weights of i + 1.
        store();
        load();
        now = ahead;
        if (ahead) {
            const float2 sc = lds_scale[(i + 1) & 3];
            const float cz = CACHE ? fmaxf(c * sc.x, kMinScale) : c;
            const float svc = CACHE ? fmaxf(sc.y, kMinVScale) : 1.0f;
            const float lsv = CACHE ? __builtin_amdgcn_logf(svc) : 0.0f;       // log2
            if (at + kPage > least)                // some row does not see all of the tile
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (at + 32 * tt + 16 * (j >> 3) + 8 * half + (j & 7) >= limit)
                            z[tt][j] = -INFINITY;
            float top = z[0][0];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int j = 0; j < 16; ++j) top = fmaxf(top, z[tt][j]);
            top = fmaf(cz, top, lsv);              // -inf: nothing visible
            if (__any(top > m + kLazy)) {
                const float m_new = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
                const float alpha = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
                m = m_new;
                l *= alpha;
#pragma unroll
                for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[dt][j] *= alpha;
            }
            // P = exp2(c z + log2(sv) - m), for the cache times 2^8
            const float shift = lsv - (m == -INFINITY ? 0.0f : m) + (CACHE ? kPShift : 0.0f);
            bool apart = false;
            if (CACHE) {
                top_lsv = fmaxf(top_lsv, lsv);
                apart = scales_apart(lsv, top_lsv);
                if (apart)
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            l += __builtin_amdgcn_exp2f(fmaf(cz, z[tt][j], shift - lsv));
            }
            float sum = 0.0f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t w[4], left[4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = (ks & 1) * 8 + 2 * j;
                    const float a = __builtin_amdgcn_exp2f(fmaf(cz, z[ks >> 1][r], shift));
                    const float e = __builtin_amdgcn_exp2f(fmaf(cz, z[ks >> 1][r + 1], shift));
                    sum += a + e;
                    w[j] = pack_weights<CACHE>(a, e, left[j]);
                }
                pk[ks] = make_uint4(w[0], w[1], w[2], w[3]);
                rest_k[ks] = make_uint4(left[0], left[1], left[2], left[3]);
            }
            l = fmaf(sum, apart ? 0.0f : 1.0f / svc, l);
        }
        __syncthreads();
    }
    if (wave < 4) __syncthreads();                 // group B's last phase of products
    l += __shfl_xor(l, 32);
    write_rows<D>(p, s, lds + wave * RowSlab<D>::kPartBytes, split, unit, rest, kRows,
                  row - tile_row * kRows, t, head, live, m, l, o);
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
// and (e, 1) are the operand of step e.  48 rows over up to 8192 tokens, 8 heads of 128 channels:
// 104 us, 5.3 TB/s, where reads of such pieces of 16 KB in random order and nothing else reach 5.6
// to 5.9.  Scores from fp16 operands took 113 us, loads that stay in the caches 117, three waves a
// vector unit, which spill, 163.
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

constexpr int kFewRows = 16;
constexpr int kFewWaves = 4;           // of a workgroup where the keys are split, else eight

template <int D, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, 2)
attention_few_kernel(const Problem p) {
    constexpr int kC = D / 64;                     // 16-byte pieces of a K row a lane
    constexpr int kDT = D / 16;                    // channel tiles
    __shared__ float lo[WAVES][16][D + 4];
    __shared__ float lm[WAVES][16], ll[WAVES][16];

    // all pairs' first pieces, then the second ones: every die has its share of each, and short
    // sequences, which have no last pieces, end the launch early (768 pairs, up to 8192 tokens, two
    // pieces: 227 us pair by pair, 211)
    const int split = quotient(blockIdx.x, p.units), unit = blockIdx.x - split * p.units;
    const int b = quotient(unit, p.Hkv), h = unit - b * p.Hkv;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int tile0 = split * p.piece_tiles;
    // the wave's tiles are tile0 + wave + i * WAVES; the page numbers of 64 of them, one a lane
    const int32_t* table = p.page_table + (size_t)b * p.max_pages;
    auto page_numbers = [&](int i) {
        const int64_t at = (int64_t)tile0 + wave + (int64_t)(i + lane) * WAVES;
        return at < p.max_pages ? table[at] : -1;
    };
    int numbers = page_numbers(0);                 // needs no length: on its way beside them
    const Sequence s = sequence<true>(p, b);
    const int G = quotient(p.Hq, p.Hkv);
    const int rows = min(s.n, p.max_rows) * G;     // at most 16
    if (rows <= 0) return;
    const bool live = col < rows;
    const int t = live ? col / G : 0;
    const int head = h * G + (live ? col % G : 0);
    const int limit = !live ? 0 : p.causal ? min(max(s.kv - s.n + t + 1, 0), s.kv) : s.kv;
    const int last_t = (rows - 1) / G;
    const int least = p.causal ? min(max(s.kv - s.n + 1, 0), s.kv) : s.kv;
    const int most = p.causal ? min(max(s.kv - s.n + last_t + 1, 0), s.kv) : s.kv;
    const int tile1 = min((most + kPage - 1) / kPage, tile0 + p.piece_tiles);
    if (p.pieces > 1 && tile0 * kPage >= s.kv) return;     // the join does not read this piece

    const size_t block = (size_t)(2 * kPage * D);
    const uint32_t k_lane = (uint32_t)((col >> 2) * 16 + (col & 3)) * D + g * 16;
    const uint32_t v_lane = (uint32_t)col * kPage + g * 16;
    int index = -1, tile = 0;
    // this wave's next page that lies in the pool, -1 behind the last
    auto next = [&]() {
        for (;;) {
            tile = tile0 + wave + ++index * WAVES;
            if (tile >= tile1) return -1;
            // the numbers of the next 64.  Not with eight waves, which walk whole stretches: plan()
            // leaves at most 42 tiles whole
            if (WAVES == kFewWaves && index > 0 && (index & 63) == 0) numbers = page_numbers(index);
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
    float l = 0.0f;                                // the lane's share of the sum of weights
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
        const uint32_t top = column_max(abs_max_bits<2 * kC>(q));
        if (top >= 0x7F80u && limit > 0) l = __uint_as_float(0x7FC00000u);    // not finite
        c *= to_digits<kC>(q, top, high, low);
    }

    f32x4_acc o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i) o[i] = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, top_lsv = -INFINITY;

    while (page >= 0) {
        const int at = tile * kPage;
        const float cz = fmaxf(c * sk, kMinScale), svc = fmaxf(sv, kMinVScale);
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
        if (at + kPage > least) {                  // some row does not see all of the page
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + 16 * g + 4 * i + j >= limit) z[i][j] = -INFINITY;
        }
        float top = z[0][0];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, z[i][j]);
        top = fmaf(cz, top, lsv);                  // -inf: nothing visible
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
        top_lsv = fmaxf(top_lsv, lsv);
        const bool apart = scales_apart(lsv, top_lsv);
        if (apart)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    l += __builtin_amdgcn_exp2f(fmaf(cz, z[i][j], shift - lsv));
        float sum = 0.0f;
        uint4 pk[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4_acc& zt = z[2 * e + (j >> 1)];
                const float a0 = __builtin_amdgcn_exp2f(fmaf(cz, zt[2 * (j & 1)], shift));
                const float a1 = __builtin_amdgcn_exp2f(fmaf(cz, zt[2 * (j & 1) + 1], shift));
                sum += a0 + a1;
                w[j] = pack_f16(a0, a1);
            }
            pk[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        l = fmaf(sum, apart ? 0.0f : sv_inv, l);
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
            total = fmaf(ll[w][r], wm == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(wm - best),
                         total);
            const float4 x = *reinterpret_cast<const float4*>(&lo[w][r][d]);
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
        }
        const size_t row = (size_t)(s.r0 + r / G);
        const int hd = h * G + r % G;
        if (p.pieces > 1) {
            const size_t to = ((size_t)split * p.units + unit) * kFewRows + r;
            if (d == 0) p.part_ml[to] = make_float2(best, total);
            *reinterpret_cast<float4*>(p.part_o + to * D + d) = a;
        } else {
            const float k = row_factor(total);
            *reinterpret_cast<uint2*>(p.O + row * p.ldo + (size_t)hd * D + d) =
                make_uint2(pack_bf16(a.x * k, a.y * k), pack_bf16(a.z * k, a.w * k));
        }
    }
}

// Joins the pieces of the split units in their order, D / 4 lanes a row; unit_rows: rows of a
// unit.  A chain of dependent loads and little else: what the first pieces left is asked for beside
// the sequence's place and length, which say how many of them there are (a token over 777 tokens,
// both kernels: 10.4 us without, 9.4).
template <int D, bool CACHE>
__global__ void __launch_bounds__(256) attention_join_kernel(const Problem p, int unit_rows) {
    constexpr int kFirst = 8, kLanes = D / 4;      // pieces asked for at once; lanes a row
    const int lane = threadIdx.x % kLanes, rest = p.units - p.whole;
    const int r = (blockIdx.x * 256 + threadIdx.x) / kLanes;
    if (r >= unit_rows) return;
    const size_t stride = (size_t)rest * unit_rows, at = (size_t)blockIdx.y * unit_rows + r;
    const float* po = p.part_o + at * D + lane * 4;
    auto piece = [&](int i) {
        return *reinterpret_cast<const float4*>(po + (size_t)i * stride * D);
    };
    float4 first[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
        first[i] = i < p.pieces ? piece(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto stats = [&](int i) {
        return i < p.pieces ? p.part_ml[(size_t)i * stride + at] : make_float2(-INFINITY, 0.0f);
    };
    float2 ml = stats(lane);
    const Place u = place(p, p.whole + blockIdx.y);
    const Sequence s = sequence<CACHE>(p, u.b);
    const int G = p.Hq / p.Hkv;
    const int row = u.tile * unit_rows + r;
    if (row >= min(s.n, p.max_rows) * G) return;
    const int t = row / G, head = u.h * G + row % G;
    const int used = min(p.pieces, ((s.kv + kPage - 1) / kPage + p.piece_tiles - 1) /
                                       p.piece_tiles);
    // the pieces' maxima and sums, kLanes at a time, one a lane
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < used; i0 += kLanes) {
        const int n = min(used - i0, kLanes);
        if (i0) ml = stats(i0 + lane);
        if (lane >= n) ml = make_float2(-INFINITY, 0.0f);          // nobody wrote these
        float top = fmaxf(m, ml.x);
#pragma unroll
        for (int k = kLanes / 2; k; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
        const float base = top == -INFINITY ? 0.0f : top;
        const float w = __builtin_amdgcn_exp2f(ml.x - base);
        const float alpha = __builtin_amdgcn_exp2f(m - base);
        m = top;
        float sum = ml.y * w;
#pragma unroll
        for (int k = kLanes / 2; k; k >>= 1) sum += __shfl_xor(sum, k);
        l = fmaf(l, alpha, sum);
        o = make_float4(o.x * alpha, o.y * alpha, o.z * alpha, o.w * alpha);
        auto add = [&](float4 x, int i) {
            const float wi = __shfl(w, i, kLanes);
            o = make_float4(fmaf(x.x, wi, o.x), fmaf(x.y, wi, o.y), fmaf(x.z, wi, o.z),
                            fmaf(x.w, wi, o.w));
        };
        int i = 0;
        if (i0 == 0) {
#pragma unroll
            for (int f = 0; f < kFirst; ++f)
                if (f < n) add(first[f], f);
            i = kFirst;
        }
#pragma unroll 8
        for (; i < n; ++i) add(piece(i0 + i), i);
    }
    const float f = row_factor(l);
    *reinterpret_cast<uint2*>(p.O + (size_t)(s.r0 + t) * p.ldo + (size_t)head * D + lane * 4) =
        make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
}

// How a call's work is laid out (Problem's fields of the same names).
struct Plan {
    int waves;          // of a workgroup; 0: the kernel for few rows
    int unit_rows, tile_rows, units, whole, pieces, piece_tiles;
    size_t part_rows() const {
        return pieces > 1 ? (size_t)pieces * (units - whole) * unit_rows : 0;
    }
};

// Pieces of at least `least` tiles, `wanted` of them where the tiles suffice.
void split(Plan& p, int64_t wanted, int tiles, int least) {
    const int most = (tiles + least - 1) / least;
    const int n = (int)(wanted < most ? wanted : most);
    p.piece_tiles = tiles > 0 ? tiles : 1;
    p.pieces = 1;
    if (n <= 1) return;
    p.piece_tiles = (tiles + n - 1) / n;
    p.pieces = (tiles + p.piece_tiles - 1) / p.piece_tiles;
}

// Enough workgroups for the 256 compute units where sequences, heads and query rows give fewer.
// Few rows, 128 channels, in us with the pieces of a (sequence, head) pair in brackets; a compute
// unit draws about 50 GB/s, a join costs about 2 us:
//   - short stretches, and what is short for many pairs, stay whole: 16 pairs, 512 tokens 9.2 [1],
//     9.1 [8]; up to 777 tokens of 192 pairs 12.9 [1], 15.2 [2], up to 2048 of 256 23.8 [1], 30.0
//     [4], up to 1500 of 384 29.6 [1], 31.2 [2].  At the limits: 128 pairs, 20 tiles 15.0 [1],
//     15.3 [2], 24 tiles 16.6 [1], 15.6 [2]; 256 pairs, 42 tiles 28.4 [1], 33.3 [4], 48 tiles 31.6
//     [1], 34.9 [4]; 264 pairs, which no longer fit one round of workgroups, 24 tiles 22.3 [1],
//     24.6 [4], 32 tiles 31.5 [1], 29.6 [4]; 384 pairs, 24 tiles 30.1 [1], 30.2 [3], 28 tiles 33.1
//     [1], 32.8 [3];
//   - else one workgroup a unit up to 4096 tiles, above two, but pieces of two tiles and more, and
//     of four where that makes more than eight: 16 pairs, 777 tokens 10.2 [4], 9.5 [8]; 2048 tokens
//     9.9 [8], 12.0 [16]; 65536 tokens 56 [32], 65 [64];
//   - from 256 pairs on four a unit and three a pair at least, for ragged lengths: up to 8192
//     tokens of 384 pairs 129 [1], 109 [3], of 768 211 [2], 204 [3].
// False for more workgroups than a launch takes.
bool plan(bool cache, bool causal, int B, int max_rows, int max_kv, int Hq, int Hkv, int D,
          Plan& p) {
    const int tiles = (int)(((int64_t)max_kv + kPage - 1) / kPage);
    const int64_t rows = (int64_t)max_rows * (Hq / Hkv), pairs = (int64_t)B * Hkv;
    p.whole = 0;
    if (cache && rows <= kFewRows) {
        p.waves = 0;
        p.unit_rows = kFewRows;
        p.tile_rows = 1;
        p.units = (int)pairs;
        const bool whole = tiles * D <= 8 * 128 ||
                           (pairs >= 128 && tiles <= (pairs <= 256 ? pairs / 6 : 24));
        const int64_t want = pairs >= 256 ? (pairs > 341 ? 3 * pairs : 1024)
                                          : pairs * tiles <= 4096 ? 256 : 512;
        const int64_t most = tiles / 4 > 8 ? tiles / 4 : 8, each = (want + pairs - 1) / pairs;
        split(p, whole ? 1 : each < most ? each : most, tiles, 2);
        return pairs * p.pieces <= (1 << 22);
    }
    // 256 rows a workgroup where every row sees long stretches of keys (128 channels: 2 x 4096 rows
    // over 16384 tokens 1149 us, 1311 with 128; 4 x 1000 over 1000 50 against 55; causal 941
    // against 918, and with 64 channels 925 against 886)
    p.waves = D == 128 && !causal && rows > 128 && tiles >= 16 ? 8 : 4;
    p.unit_rows = kWaveRows * p.waves;
    const int64_t tile_rows = (rows + p.unit_rows - 1) / p.unit_rows, units = tile_rows * pairs;
    if (units > (1 << 21)) return false;
    p.tile_rows = (int)tile_rows;
    p.units = (int)units;
    // A round is what runs at once.  What is left over after whole rounds, or all where it is less
    // than one, is split over its keys where that repays the join (us, whole | split; 16 heads):
    //   - less than a round, the sooner the fewer: where pieces times tiles of keys reach `enough`.
    //     256 rows a workgroup, two pieces from 16 tiles (1500 rows over 1024 tokens 42.3 | 39.8,
    //     states 46.0 | 40.5; 128 rows a workgroup over 960 states 41.0 | 42.6).  128 channels, two
    //     from 20 (1500 causal rows over 1500 tokens 51.8 | 44.0; 1900 rows over 768 states 36.8 |
    //     42.4), four from 10 (900 rows over 768 tokens 30.2 | 27.4, states 33.6 | 29.2, over 512
    //     24.7 | 26.1), more from 4 (40 rows over 300 tokens 15.1 | 13.0, one over 300 states
    //     15.9 | 12.6).  64 channels, whose rounds are larger, two from 32 (2400 rows over 2048
    //     tokens 66.6 | 59.0, over 1024 states 38.3 | 39.3), more from 12 (1200 causal rows over
    //     1200 tokens 30.3 | 24.4, over 768 states 22.4 | 24.1; 600 rows over 768 states 22.1 |
    //     18.7), below only very many (600 rows over 512 states 16.6 | 18.4);
    //   - behind whole rounds, little of it: from 8 tiles (2 x 4192 rows over 512 tokens 71.8 |
    //     65.1, states 73.6 | 69.0, over 12576 tokens, 32 of 544 units, 1224 | 960); much: from 64
    //     (288 of 1056 units of 64 channels, 2048 states 105 | 114, 6000 390 | 366); never causal
    //     ones, whose last units are the shortest (3 x 2000 rows of 24 heads of 64 channels 77.8 |
    //     86.6).
    const int round = p.waves == 8 ? 256 : D == 64 ? 768 : 512, rest = p.units % round;
    const bool alone = p.units < round;
    const int enough = p.waves == 8 ? 32 : D == 128 ? 40 : tiles >= 12 ? 64 : 128;
    const bool worth =
        rest > 0 && rest <= round / 2 &&
        (alone ? tiles >= 4 && round / rest * tiles >= enough
               : !causal && tiles >= (rest * 8 > round ? 64 : 8));
    split(p, worth ? round / rest : 1, tiles, 2);
    p.whole = p.pieces > 1 ? p.units - rest : p.units;
    return true;
}

template <int D, bool CACHE>
hipError_t launch(Problem p, void* workspace, hipStream_t stream) {
    Plan sp;
    if (!plan(CACHE, p.causal, p.B, p.max_rows, p.max_kv, p.Hq, p.Hkv, D, sp))
        return hipErrorInvalidValue;
    p.tile_rows = sp.tile_rows;
    p.units = sp.units;
    p.whole = sp.whole;
    p.pieces = sp.pieces;
    p.piece_tiles = sp.piece_tiles;
    const int pairs = p.Hkv * p.B;
    p.dies = pairs % 8 == 0 ? 8 : 1;
    p.descending = p.causal ? 1 : 0;
    p.tile_major = p.causal && (int64_t)(pairs / p.dies) * p.max_kv * (2 * D) <= (2 << 20) ? 1 : 0;
    p.run = p.tile_major ? pairs / p.dies : p.tile_rows;
    p.most_tiles = (int)(((int64_t)p.max_kv + kPage - 1) / kPage);
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + sp.part_rows() * D);
    const unsigned grid = (unsigned)(p.whole + (p.units - p.whole) * p.pieces);
    if (sp.waves == 0) {
        if constexpr (CACHE) {
            if (p.pieces == 1)
                attention_few_kernel<D, 8><<<grid, 512, 0, stream>>>(p);
            else
                attention_few_kernel<D, kFewWaves><<<grid, kFewWaves * 64, 0, stream>>>(p);
        }
    } else if (sp.waves == 8) {
        if constexpr (D == 128) attention_wide_kernel<D, CACHE><<<grid, 512, 0, stream>>>(p);
    } else {
        attention_tile_kernel<D, CACHE><<<grid, 256, 0, stream>>>(p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.pieces == 1) return e;
    const int64_t rows = (int64_t)p.max_rows * (p.Hq / p.Hkv);
    const unsigned most = (unsigned)(rows < sp.unit_rows ? rows : sp.unit_rows);
    attention_join_kernel<D, CACHE>
        <<<dim3((most * (D / 4) + 255) / 256, p.units - p.whole), 256, 0, stream>>>(
            p, sp.unit_rows);
    return hipGetLastError();
}

}  // namespace

bool attention_workspace(bool cache, bool causal, int B, int T, int max_rows, int max_kv, int Hq,
                         int Hkv, int D, size_t& bytes) {
    Plan p;
    if (!plan(cache, causal, B, max_rows < T ? max_rows : T, max_kv, Hq, Hkv, D, p)) return false;
    bytes = p.part_rows() * (size_t)(D + 2) * sizeof(float);
    return true;
}

// From plan(): few rows, where a group has at most 16 of them, take at most 512 workgroups and one
// a pair below 256 pairs, 1024 and one a pair up to 341 and three a pair above; else pieces and
// split units make at most one round.  Pieces have two tiles at least.
size_t attention_workspace_bound(int B, int T, int max_rows, int max_kv, int Hq, int Hkv, int D) {
    const int64_t tiles = ((int64_t)max_kv + kPage - 1) / kPage, most = (tiles + 1) / 2;
    if (most <= 1) return 0;
    const int64_t pairs = (int64_t)B * Hkv, group = Hq / Hkv;
    const int64_t few = pairs < 256 ? 511 + pairs : 3 * pairs > 1364 ? 3 * pairs : 1364;
    int64_t rows = 0;
    if (group <= kFewRows) rows = kFewRows * (few < most * pairs ? few : most * pairs);
    const int64_t all = (max_rows < T ? max_rows : T) * group;
    for (const int waves : {4, 8}) {
        const int64_t unit = kWaveRows * waves, round = waves == 8 ? 256 : D == 64 ? 768 : 512;
        const int64_t units = most * ((all + unit - 1) / unit) * pairs;
        const int64_t parts = unit * (units < round ? units : round);
        rows = rows > parts ? rows : parts;
    }
    return (size_t)rows * (size_t)(D + 2) * sizeof(float);
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
    p.B = B;
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
    return D == 64 ? launch<64, true>(p, workspace, stream)
                   : launch<128, true>(p, workspace, stream);
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
    p.B = B;
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
    return D == 64 ? launch<64, false>(p, workspace, stream)
                   : launch<128, false>(p, workspace, stream);
}

}  // namespace rudder
