// kv_attend.h - softmax attention of new tokens over the paged cache of
// quantised keys and values.
//
//   s_j = scale * q . k_j     over the visible positions j of a row
//   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = ln sum_j exp(s_j)
//
// A wave takes 32 tokens of one head at a time, with tiles of 16 rows (query
// heads of the group times new tokens) as the columns of its matrix
// instructions, in one pass over the cache:
//
//   S^T = K Q^T  16 keys x 16 rows, a block of 32 dims an instruction: codes
//                as binary16 (exact), the query as hi + lo binary16 of the row
//                scaled by a power of two (22 bits; a binary16 query is exact
//                in hi alone), the block's scale on the float32 result
//   O^T = V^T P  16 dims x 16 rows, 32 keys an instruction: codes as binary16
//                (exact), the weights p * (scale of the value's block) as
//                binary16 where q and out are (a rounding of 2^-11, as the
//                output's own: 2.9e-4 from 64 bits where the output's alone is
//                2.1e-4), else as hi + lo (22 bits).  hi + lo there too takes 705
//                us for 501 (prompt chunk), 137 for 122 (own heads, 4 bits)
//
// so all sums are float32.  S^T leaves a lane with 4 keys of each half of its
// 32, of one row; the second product takes its k index in that order, so
// weights go from one to the other in place, and a lane's scales are those of
// 4 + 4 keys, two words a block pair, that mixed-precision multiply-adds take
// as they are.
//
// The softmax keeps a running reference r per row; sums and weights are of
// exp2(s - r).  What binary16 has to hold is a weight times its value's scale, so
// r goes by the largest such product: it is put 2^5 below that of the first step, and
// moves (everything so far is rescaled) only when a product may pass binary16's
// range, which few steps do: those leave the inner loop.  Products lose bits below
// 2^-14, by 2^-25 absolutely: 2^-30 of the largest so far, of which a code's step is 2^-8
// or 2^-4.  Weights alone do not tell: beside a first token that has nearly all of the
// weight but a small value the others make the output.  1200 tokens that share 2^-17 of
// the weight beside one without a value: 4e-7 off in float32, 4% with a reference that
// goes by the scores.  A reference that also falls where a step's scores are 2^8 (2^20)
// lower takes 1125 (716) us for 603, a prompt chunk whose scores spread (standard
// deviation 5).
//
// Few rows (kNarrow, kWide) are bound by the cache: every wave has its own steps,
// copied straight into LDS while the step before is worked on, and joins the
// others in LDS at the end.  One token of 32 query heads on 8, 131000 tokens, 8 bits
// (285 MB): 56 us, 5.1 TB/s, and 7 for the join; 64 ragged sequences up to 8100
// (539 MB) 120 + 5; 32 sequences of own heads, 4 bits (517 MB) 114 + 5; 16 windows of
// 1024, 48 rows 26 (latency: 9 steps of a workgroup, 128 workgroups).  Many rows
// (kTall) are bound by vector issue: 2048 rows of 4 over 6100 tokens before them 500 us,
// 480 TFLOP/s, the vector units busy 67% of the time, the matrix units 19%.  Per
// 32 keys and 16 rows a wave has 16 matrix instructions of 16 cycles and some 200 vector
// ones of 4: 32 scales on scores, 32 on weights, 40 of the softmax, the rest copies and
// codes, which 8 waves share.  Without either scale it would take 560 and 510 us (of
// then 604), without converting 520, without copying 527.  Keys scaled before
// the product, as hi + lo, take 725 us against then 611; 4 waves of 32 rows 630 against
// 605; 8 waves of 32 569 against 498.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv.h"

namespace mmq {
namespace kv {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;   // tokens of a wave's step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFloor = -3e38f;      // the reference of a row that has seen nothing
// log2 of products of weights and scales: what the reference puts the largest at,
// where a step is looked at, and how far a product may rise (65504 is binary16's largest).
constexpr float kLift = 5.0f, kLook = 15.8f, kTop = 15.9f;
constexpr float kNoScale = -64.0f;    // what counts as the exponent of a scale of 0 (the smallest other is 2^-24)
constexpr float kLarge = 0x1p23f;     // references from here on are coarser than a score's difference to them may be

struct Attend {
    KvCache c;
    KvPlan p;
    KvQuery q;
    int wgs;                // workgroups the work is split over (split form)
    float* part;            // [wgs * 2][16 * QT][dim] unnormalised sums
    float2* stat;           // [wgs * 2][16 * QT] (reference, sum)
    struct Join* join;      // [wgs]
};

// The rows that a workgroup began and others go on with, to be joined once all
// are done.
struct alignas(16) Join {
    int count;              // workgroups that have a part of them, from this one on; 0: no such rows
    int slot;               // of this workgroup's part (the others': 0)
    int token, rows;        // first row of the sequence, rows of the tile
    int head, row;          // of the cache; the tile's first row (token * group + query head of the group)
    int unused[2];
};

// What a sequence asks for: its rows, their positions, and the tokens any of them sees.
struct Sequence {
    int row0, rows;         // first row of the call, rows taken
    int pos0;               // position of the first row
    int first, last;        // tokens first .. last - 1; first is a multiple of 32
    int units;              // the workgroup's steps over them; 1 at least where there are rows
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Offsets and lengths may hold anything: rows stay within the call's, tokens
// within the table, and positions (below 2^31, as lengths are) above -2^30, so
// that a window of 2^30 back from them is an int.
template <int UNIT>
__device__ __forceinline__ Sequence sequence(const Attend& a, int s) {
    Sequence r;
    int64_t lo = s, hi = s + 1;
    if (a.p.offsets) {
        lo = a.p.offsets[s];
        hi = a.p.offsets[s + 1];
    }
    lo = lo < 0 ? 0 : lo;
    const int64_t pos0 = (int64_t)a.p.lengths[s] - (hi - lo);
    const int64_t top = (int64_t)a.p.width << a.c.shift;
    hi = hi > a.q.n ? a.q.n : hi;
    int64_t rows = hi - lo;
    rows = rows < 0 ? 0 : rows > a.q.most ? a.q.most : rows;
    r.row0 = (int)lo;
    r.rows = (int)rows;
    r.pos0 = rows > 0 && pos0 > -(1 << 30) ? (int)pos0 : -(1 << 30);
    int64_t last = (int64_t)r.pos0 + rows;
    last = last < 0 ? 0 : last > top ? top : last;
    int64_t first = a.q.window ? (int64_t)r.pos0 - a.q.window + 1 : 0;
    first = first < 0 ? 0 : first > last ? last : first;
    r.first = (int)first & ~(kTile - 1);
    r.last = (int)last;
    const int units = (r.last - r.first + UNIT - 1) / UNIT;
    r.units = rows > 0 ? (units > 0 ? units : 1) : 0;
    return r;
}

// The same, s being the workgroup's: in scalar registers.
template <int UNIT>
__device__ __forceinline__ Sequence sequence_of_all(const Attend& a, int s) {
    Sequence r = sequence<UNIT>(a, s);
    r.row0 = uniform(r.row0);
    r.rows = uniform(r.rows);
    r.pos0 = uniform(r.pos0);
    r.first = uniform(r.first);
    r.last = uniform(r.last);
    r.units = uniform(r.units);
    return r;
}

// Four outputs of query head hq of row tok: sums x over the weights' sum.
__device__ __forceinline__ void put_row(const KvQuery& q, int64_t tok, int hq, int heads, int dim, int d, v4f x,
                                        float m, float sum) {
    x *= sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = tok * q.out_stride + (int64_t)hq * dim + d;
    if (q.out_half) {
        _Float16* p = static_cast<_Float16*>(q.out) + at;
        const v4h y = {(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
        if (q.out_vec) {
            *reinterpret_cast<v4h*>(p) = y;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = y[i];
        }
    } else {
        float* p = static_cast<float*>(q.out) + at;
        if (q.out_vec) {
            *reinterpret_cast<v4f*>(p) = x;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = x[i];
        }
    }
    if (q.lse && d == 0) q.lse[tok * heads + hq] = (m + log2f(sum)) * kLn2;
}

// Four sums of a tile's row: out, or to partial `part`.
__device__ __forceinline__ void put(const Attend& a, const Sequence& sq, int h, int first, int row, int part, int tile_rows,
                                    int dim, int d, v4f x, float m, float sum) {
    if (part >= 0) {
        const int64_t at = (int64_t)part * tile_rows + row;
        *reinterpret_cast<v4f*>(a.part + at * dim + d) = x;
        if (d == 0) a.stat[at] = make_float2(m, sum);
    } else {
        const int ri = first + row, group = a.q.group;
        put_row(a.q, sq.row0 + ri / group, h * group + ri % group, a.c.heads * group, dim, d, x, m, sum);
    }
}

// 8 values of a query, or 0.
__device__ __forceinline__ void query8(const KvQuery& q, int64_t at, bool there, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (!there) return;
    if (q.q_half) {
        const _Float16* p = static_cast<const _Float16*>(q.q) + at;
        v8h x;
        if (q.q_vec) {
            x = *reinterpret_cast<const v8h*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
    } else {
        const float* p = static_cast<const float*>(q.q) + at;
        if (q.q_vec) {
            const v4f x = *reinterpret_cast<const v4f*>(p), y = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = x[i];
                v[4 + i] = y[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i];
        }
    }
}

// The largest power of two that divides n, at most 16: how runs of n bytes lie.
constexpr int alignment(int n) { return (n & -n) < 16 ? n & -n : 16; }

// (x & mask) | bits in one instruction (the compiler makes two).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(mask), "v"(bits));
    return r;
}

__device__ __forceinline__ uint32_t pk_add(uint32_t a, float b) {
    const v2h c = {(_Float16)b, (_Float16)b};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) + c);
}

// Nibbles 0 and 4 (low) or 1 and 5 of a word as codes: 1024 + n by its bits,
// less 1032; or 1024 + 16 n, a sixteenth of it less 72.  All exact.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, bool low) {
    if (low) return pk_add(and_or(w, 0x000F000Fu, 0x64006400u), -1032.0f);
    const v2h a = __builtin_bit_cast(v2h, and_or(w, 0x00F000F0u, 0x64006400u));
    const v2h f = {(_Float16)0.0625f, (_Float16)0.0625f}, c = {(_Float16)-72.0f, (_Float16)-72.0f};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(a, f, c));
}

// A step's 32 tokens of one head in LDS, copied there by the loads themselves,
// 16 bytes a lane in lane order (the order in LDS is free at that grain):
//   keys    [half of 16][16-byte piece of a token][token]
//   values  [half][i][g][16-byte piece], token 4 g + i: what the lanes of one read
//           need lies in their order
//   scales  of keys, then of values, [token][block]
template <bool Q4, int NB>
struct Step {
    static constexpr int kCode = (Q4 ? 16 : 32) * NB, kPieces = kCode / 16;   // of a token
    static constexpr int kKey = kCode / 4, kValue = kCode / 16;               // bytes of a lane
    static constexpr int kCopies = (32 * kPieces + 63) / 64;                  // copies of 64 pieces, keys or values
    static constexpr int kValues = kCopies * 1024, kScales = 2 * kCopies * 1024, kBytes = kScales + 128 * NB;
    static constexpr int kLoads = 2 * kCopies + 1;

    // Where copy j of the kLoads that a step takes has a lane's piece: half h of 16
    // tokens, bytes past that half's first code or scale.
    struct Piece {
        uint32_t at;
        bool h;
    };
    static __device__ __forceinline__ Piece piece_of(int j, int64_t half, int shift, int lane) {
        Piece p;
        if (j < 2 * kCopies) {
            const bool value = j >= kCopies;
            int n = 64 * (value ? j - kCopies : j) + lane;
            if (32 * kPieces % 64 != 0) n = n < 32 * kPieces ? n : 32 * kPieces - 1;   // (the last copy ends in its own area)
            const int row = n / kPieces;
            p.h = n >= 16 * kPieces;
            const int token = value ? 4 * (row & 3) + (row >> 2 & 3) : n & 15;
            const int c = value ? n - row * kPieces : (n - 16 * kPieces * p.h) >> 4;
            p.at = (value ? (uint32_t)half : 0) + token * kCode + 16 * c;
        } else {
            const int v = lane >= 4 * NB, n = lane - 4 * NB * v;
            p.h = n >= 2 * NB;
            p.at = (v ? (uint32_t)half : 0) + ((uint32_t)kCode << shift) + 16 * (n - 2 * NB * p.h);
        }
        return p;
    }

    // Copy j, of the tokens at slot0, slot1 of the records rec0, rec1.
    static __device__ __forceinline__ void load(int j, Piece p, uint32_t lds, const uint8_t* rec0, const uint8_t* rec1,
                                                int slot0, int slot1, int lane) {
        if (j < 2 * kCopies) {
            copy(lds + 1024 * j, (p.h ? rec1 + slot1 * kCode : rec0 + slot0 * kCode) + p.at);
        } else if (lane < 8 * NB) {
            copy(lds + kScales, (p.h ? rec1 + slot1 * 2 * NB : rec0 + slot0 * 2 * NB) + p.at);
        }
    }

    // A copy of 16 bytes a lane from `from` to lds + 16 lane.  Outside the
    // compiler's bookkeeping: landed() is what waits for it.  M0 is read by the
    // load one wait state after its write.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    static __device__ __forceinline__ void copy(uint32_t lds, const uint8_t* from) {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
    }
#pragma clang diagnostic pop

    // The operand of half h and block b: 8 dims of the lane's key.
    static __device__ __forceinline__ v8h key(const uint8_t* at, int h, int b, int lane) {
        const int col = lane & 15, g = lane >> 4;
        const int byte = g * kKey + b * (kKey / NB);
        const uint8_t* p = at + ((h * kPieces + (byte >> 4)) * 16 + col) * 16 + (byte & 15);
        v4u w;
        if constexpr (Q4) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(p), y = x >> 8;
            w[0] = q4_pair(x, true);
            w[1] = q4_pair(x, false);
            w[2] = q4_pair(y, true);
            w[3] = q4_pair(y, false);
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // 1152 + code by its bits, less 1152
                const uint32_t u = (i ? x.y : x.x) ^ 0x80808080u;
                w[2 * i] = pk_add(__builtin_amdgcn_perm(0x64646464u, u, 0x04010400u), -1152.0f);
                w[2 * i + 1] = pk_add(__builtin_amdgcn_perm(0x64646464u, u, 0x04030402u), -1152.0f);
            }
        }
        return __builtin_bit_cast(v8h, w);
    }

    // The lane's scales of half h, [4 keys][block], two to a word.
    static __device__ __forceinline__ void scales(const uint8_t* at, bool value, int h, int lane, uint32_t (&s)[2 * NB]) {
        scales_at(at + kScales, value, h, lane, s);
    }
    static __device__ __forceinline__ void scales_at(const uint8_t* at, bool value, int h, int lane, uint32_t (&s)[2 * NB]) {
        const uint8_t* p = at + 64 * NB * (int)value + 2 * NB * (16 * h + 4 * (lane >> 4));
        __builtin_memcpy(s, __builtin_assume_aligned(p, alignment(8 * NB)), 8 * NB);
    }

    // The values' scales spread over the lanes, words lane and lane + 64 of the 16 NB.
    static constexpr int kLevels = NB > 4 ? 2 : 1;
    static __device__ __forceinline__ int level_word(int i, int lane) {
        return 64 * i + lane < 16 * NB ? 64 * i + lane : 16 * NB - 1;
    }
    static __device__ __forceinline__ void levels(const uint8_t* at, int lane, uint32_t (&w)[kLevels]) {
        levels_at(at + kScales, lane, w);
    }
    static __device__ __forceinline__ void levels_at(const uint8_t* at, int lane, uint32_t (&w)[kLevels]) {
#pragma unroll
        for (int i = 0; i < kLevels; ++i)
            w[i] = *reinterpret_cast<const uint32_t*>(at + 64 * NB + 4 * level_word(i, lane));
    }

    // The lane's bytes of its 8 keys.
    struct Codes {
        uint32_t w[8][(kValue + 3) / 4];
    };
    static __device__ __forceinline__ void codes(const uint8_t* at, int lane, Codes& c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (kValue & 3) c.w[i][kValue / 4] = 0;
            __builtin_memcpy(c.w[i], __builtin_assume_aligned(at + kValues + i * 4 * kCode + lane * kValue, alignment(kValue)), kValue);
        }
    }

    // Values of all lanes as operands, [tile][lane][pair of keys], by shares of a
    // sixteenth of the lanes' keys and kChunk bytes of each: two lanes' bytes of a
    // word, which lie apart, come together in one lane.
    static constexpr int kChunk = alignment(kValue) < (Q4 ? 2 : 4) ? alignment(kValue) : (Q4 ? 2 : 4);
    static constexpr int kShares = 4 * (kValue / kChunk);
    static __device__ __forceinline__ void convert_values(const uint8_t* at, int share, int lane, uint32_t* to) {
        const int g = share & 3, c = share >> 2, col = lane & 15, pair = lane >> 4;
        const uint8_t* p = at + kValues + (2 * pair * 4 + g) * kCode + col * kValue + c * kChunk;
        uint32_t x = 0, y = 0;
        __builtin_memcpy(&x, __builtin_assume_aligned(p, kChunk), kChunk);
        __builtin_memcpy(&y, __builtin_assume_aligned(p + 4 * kCode, kChunk), kChunk);
        if (!Q4) x ^= 0x80808080u, y ^= 0x80808080u;
        to += ((Q4 ? 2 : 1) * c * kChunk * 64 + 16 * g + col) * 4 + pair;
#pragma unroll
        for (int b = 0; b < kChunk; ++b) {
            const uint32_t w = __builtin_amdgcn_perm(y, x, 0x0C000C00u | b | (4 + b) << 16);
            if constexpr (Q4) {
                to[2 * b * 256] = q4_pair(w, true);
                to[(2 * b + 1) * 256] = q4_pair(w, false);
            } else {
                to[b * 256] = pk_add(w | 0x64006400u, -1152.0f);
            }
        }
    }

    // Dims 16 t + lane of the lane's 8 keys.
    static __device__ __forceinline__ v8h value(const Codes& c, int t) {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Q4) {
                const int b = t >> 1;   // bytes b of two keys
                const uint32_t x = __builtin_amdgcn_perm(c.w[2 * i + 1][b >> 2], c.w[2 * i][b >> 2],
                                                         0x0C000C00u | (b & 3) | (4 + (b & 3)) << 16);
                w[i] = q4_pair(x, (t & 1) == 0);
            } else {
                const uint32_t x = c.w[2 * i][t >> 2], y = c.w[2 * i + 1][t >> 2];
                w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz((float)(int8_t)(x >> (8 * (t & 3))),
                                                                               (float)(int8_t)(y >> (8 * (t & 3)))));
            }
        }
        return __builtin_bit_cast(v8h, w);
    }
};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// The largest of a row's four lanes, which lie 16 apart.
__device__ __forceinline__ float row_most(float v) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const uint32_t p0 = p[0], p1 = p[1];   // (a cast of an element itself would take the first)
    const uint32_t b = __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1)));
    const auto q = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t q0 = q[0], q1 = q[1];
    return fmaxf(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
}

// Waits until at most N loads are under way (older ones have landed), and until
// what was read from LDS has arrived.
template <int N>
__device__ __forceinline__ void landed() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The scale of key i (0 .. 3 of the lane's half) and block b.
template <int N>
__device__ __forceinline__ _Float16 scale_of(const uint32_t (&s)[N], int i, int b) {
    const int at = i * (N / 2) + b;
    return __builtin_bit_cast(v2h, s[at >> 1])[at & 1];
}

// How the rows of a workgroup are laid out over its waves.
//   kNarrow  tiles of 16 rows, and
//   kWide    of 64 (32 above 128 dims): each of 4 waves has all of them, the waves
//            take steps of 32 tokens in turns
//   kWide8   the same with 8 waves, one workgroup a CU
//   kTall    tiles of 128 rows, 16 a wave; all 8 waves take the same steps, whose
//            codes they turn into operands together
enum Form { kNarrow, kWide, kWide8, kTall };
constexpr int row_tiles(Form f, int nb) { return f == kNarrow || f == kTall ? 1 : nb <= 4 ? 4 : 2; }   // of a wave
constexpr int waves_of(Form f) { return f == kNarrow || f == kWide ? 4 : 8; }
constexpr int tile_rows(Form f, int nb) { return 16 * row_tiles(f, nb) * (f == kTall ? waves_of(f) : 1); }

// Heads of 128 in 8 bits go from kNarrow to kTall (cut() in kv_attend.hip).
constexpr bool has_wide(bool q4, int nb) { return q4 || nb != 4; }

// Bytes of LDS of a workgroup, by how many steps there is room for:
// of each wave, as loaded; kTall: of operands, beside two as loaded.
constexpr int kLds = 160 * 1024;
constexpr int step_bytes(bool q4, int nb) { return 2 * ((32 * (q4 ? 1 : 2) * nb + 63) / 64) * 1024 + 128 * nb; }
constexpr int operand_bytes(int nb) { return 4096 * nb + 128 * nb; }
constexpr int lds_bytes(bool q4, int nb, Form f, bool full, int stages) {
    const int waves = waves_of(f), query = tile_rows(f, nb) * nb * 64 * (full ? 2 : 1);
    const int out = f == kTall ? 0 : waves * 16 * (32 * nb + 4) * 4;
    const int in = f == kTall ? 2 * step_bytes(q4, nb) + stages * operand_bytes(nb)
                              : query + waves * stages * step_bytes(q4, nb);
    const int rest = tile_rows(f, nb) * 4 * (f == kTall ? 1 : 1 + 2 * waves) + 256;
    return (in > out ? in : out) > query ? (in > out ? in : out) + rest : query + rest;
}
constexpr bool fits(bool q4, int nb, Form f, bool full) { return lds_bytes(q4, nb, f, full, 1) <= kLds; }
// Workgroups a CU by registers: waves with four tiles of sums, of heads above 128
// dims, and kTall's with queries of two parts from 96 dims on take more than half of
// what two of a SIMD share (600 rows of 4 over 3000 tokens, float32, 128 dims: two
// workgroups with spills 188 us, one 159, 32 rows of 32 sequences of 2048 140 and 108; 96
// dims, with fewer spills, 135 and 144; the binary16 chunk with one 714 us where two take
// 502).
constexpr int by_registers(int nb, Form f, bool full) {
    return 4 * (f == kNarrow ? 3 : f == kTall && nb <= (full ? 2 : 4) ? 4 : 2) / waves_of(f);
}
// Two steps where that leaves as many workgroups a CU (two count as many): with
// one, one sequence of 131000 tokens takes 73 us instead of 67, 32 of 4096, 4 bits, 130
// instead of 123; kTall with one is 1 to 3% faster up to 128 dims, 4% slower at 256.
constexpr int stages(bool q4, int nb, Form f, bool full) {
    const int want = by_registers(nb, f, full) < 2 || 2 * lds_bytes(q4, nb, f, full, 1) > kLds ? 1 : 2;
    return want * lds_bytes(q4, nb, f, full, 2) <= kLds ? 2 : 1;
}
constexpr int wgs_per_cu(bool q4, int nb, Form f, bool full) {
    const int by_lds = kLds / lds_bytes(q4, nb, f, full, stages(q4, nb, f, full)), regs = by_registers(nb, f, full);
    return by_lds < regs ? by_lds : regs;
}
// Tokens of a workgroup's step, the grain of the cuts.
constexpr int unit_of(Form f) { return kTile * (f == kWide8 ? 8 : 4); }

template <bool Q4, int NB, Form F, bool FULL>
struct Shared {
    static constexpr int kRows = tile_rows(F, NB), kPitch = 32 * NB + 4, kStages = stages(Q4, NB, F, FULL);
    static constexpr int kWaves = waves_of(F), kUnit = unit_of(F);
    struct Query {
        uint4 q[kRows / 16][NB][FULL ? 2 : 1][64];   // hi and lo of the queries, as operands
    };
    struct Own {
        Query query;
        uint8_t step[kWaves][kStages][step_bytes(Q4, NB)];
    };
    struct Common {
        uint8_t step[2][step_bytes(Q4, NB)];
        struct {
            uint4 key[2][NB][64], value[2 * NB][64];
            uint8_t scale[128 * NB];
        } operand[kStages];
    };
    union {
        typename std::conditional<F == kTall, Common, Own>::type in;
        Query query;                              // kTall: until the waves have theirs in registers
        float o[F == kTall ? 1 : kWaves][16][F == kTall ? 1 : kPitch];   // the waves' sums of 16 rows
    };
    float factor[kRows];                          // log2(e) * |scale| / the row's power of two
    float m[F == kTall ? 1 : kWaves][F == kTall ? 1 : kRows], l[F == kTall ? 1 : kWaves][F == kTall ? 1 : kRows];
    int64_t scan[kWaves], base;
    int found;
};

// The queries of a tile of `rows` rows as operands, into LDS: 16 lanes a row,
// chunk (b, g) of 8 dims each.
template <int NB, bool FULL, int W, class S>
__device__ __forceinline__ void stage_queries(const Attend& a, S& sh, uint4 (*q)[NB][FULL ? 2 : 1][64], const Sequence& sq,
                                              int h, int first, int live) {
    const int tid = threadIdx.x, group = a.q.group;
    const float size = fabsf(a.q.scale) * kLog2e, sign = a.q.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll 1
    for (int row = tid >> 4; row < S::kRows; row += 4 * W) {
        const int t = row >> 4, ri = first + row;
        float v[(NB + 3) / 4][8];
        float amax = 0.0f;
        const bool there = row < live;
        const int64_t at =
            there ? (int64_t)(sq.row0 + ri / group) * a.q.q_stride + (int64_t)(h * group + ri % group) * 32 * NB : 0;
#pragma unroll
        for (int c = 0; c < (NB + 3) / 4; ++c) {
            const int ch = 16 * c + (tid & 15);
            query8(a.q, at + 8 * ch, there && ch < 4 * NB, v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[c][i]));
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
        int e = amax > 0.0f && amax < INFINITY ? __builtin_amdgcn_frexp_expf(amax) : 14;
        if (a.q.q_half) e = e < 14 ? e : 14;   // binary16 has them as they are; scaled down, subnormals would lose bits
        if ((tid & 15) == 0) sh.factor[row] = fmaxf(ldexpf(size, e - 14), 0x1p-126f);   // not 0: hidden scores stay -inf
#pragma unroll
        for (int c = 0; c < (NB + 3) / 4; ++c) {
            const int ch = 16 * c + (tid & 15);
            if (ch >= 4 * NB) continue;
            v8h hi, lo;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = ldexpf(v[c][i] * sign, 14 - e);
                hi[i] = (_Float16)x;
                lo[i] = (_Float16)(x - (float)hi[i]);
            }
            const int at16 = (ch & 3) * 16 + (row & 15);
            q[t][ch >> 2][0][at16] = __builtin_bit_cast(uint4, hi);
            if (FULL) q[t][ch >> 2][1][at16] = __builtin_bit_cast(uint4, lo);
        }
    }
}

// A wave's rows: QT tiles of 16, a lane having row `col` of each (in four of
// its 64 lanes), and what they have seen so far.  Scores are raw: times the
// row's factor they are log2 of weights.
template <int NB, int QT, bool FULL>
struct Rows {
    float factor[QT], ref[QT], l[QT];
    int see_lo[QT], see_hi[QT];      // visible tokens
    v4f o[QT][2 * NB];               // sums of dims 16 d + 4 g + i, d the second index
    int exponent;                    // steps with scales of 2^exponent and more are looked at; so is every step
    bool always;                     // where a reference is large
    int all_lo, all_hi, any_lo, any_hi;   // tokens that every row sees, that some row sees

    // Rows first .. first + live - 1 (token * group + head of the group) of the sequence.
    __device__ __forceinline__ void begin(const Attend& a, const Sequence& sq, int first, int live, const float* factors) {
        const int col = threadIdx.x & 15, group = a.q.group, cap = sq.last - 1;
        const int t0 = sq.pos0 + first / group, t1 = sq.pos0 + (first + live - 1) / group;
        all_hi = uniform(t0);
        all_lo = uniform(a.q.window ? t1 - a.q.window + 1 : 0);
        any_lo = uniform(a.q.window ? t0 - a.q.window + 1 : 0);
        any_hi = uniform(t1 < cap ? t1 : cap);
        exponent = -24;
        always = false;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int row = 16 * t + col, pos = sq.pos0 + (first + (row < live ? row : 0)) / group;
            factor[t] = factors[row];
            see_hi[t] = row < live ? (pos < cap ? pos : cap) : -1;
            see_lo[t] = a.q.window ? pos - a.q.window + 1 : 0;
            ref[t] = kFloor;
            l[t] = 0.0f;
#pragma unroll
            for (int d = 0; d < 2 * NB; ++d) o[t][d] = v4f{0, 0, 0, 0};
        }
    }

    // Scores of a step's tokens: key(h, b), query(t, b, lo) are the operands,
    // ks the lane's scales.
    template <class Key, class Query>
    __device__ __forceinline__ void scores(const Key& key, const Query& query, const uint32_t (&ks)[2][2 * NB],
                                           float (&sc)[QT][8]) const {
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[t][i] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const v8h k_0 = key(0, b), k_1 = key(1, b);
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const v8h hi = query(t, b, 0);
                v4f x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
                x = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_0, hi, x, 0, 0, 0);
                y = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_1, hi, y, 0, 0, 0);
                if constexpr (FULL) {
                    const v8h lo = query(t, b, 1);
                    x = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_0, lo, x, 0, 0, 0);
                    y = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_1, lo, y, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[t][i] = __builtin_fmaf((float)scale_of(ks[0], i, b), x[i], sc[t][i]);
                    sc[t][4 + i] = __builtin_fmaf((float)scale_of(ks[1], i, b), y[i], sc[t][4 + i]);
                }
            }
        }
    }

    // Hidden tokens' scores become -inf; whether a reference has to move; and
    // whether the step has hidden tokens (beyond some row's position, before its
    // window, or without a page), where anything may lie.  levels: the values'
    // scales, spread over the lanes.
    template <int N>
    __device__ __forceinline__ bool look(float (&sc)[QT][8], float (&top)[QT], const uint32_t (&levels)[N], int at, int have,
                                         int end, bool& masked) const {
        masked = uniform((have != 3) | (at + kTile - 1 > all_hi) | (at < all_lo) | (at + kTile > end)) != 0;
        if (masked) {
            asm volatile("");   // a branch, not selects in every step
            const int g = threadIdx.x >> 4 & 3;
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = at + 16 * (i >> 2) + 4 * g + (i & 3);
                    const bool hidden = (j < see_lo[t]) | (j > see_hi[t]) | !(have >> (i >> 2) & 1);
                    sc[t][i] = hidden ? -INFINITY : sc[t][i];
                }
        }
        // The largest scale as bits: they order as the values do, and NaN and
        // infinity lie above.
        v2u16 lv = __builtin_bit_cast(v2u16, levels[0]);
        if constexpr (N > 1) lv = __builtin_elementwise_max(lv, __builtin_bit_cast(v2u16, levels[1]));
        const int bits = lv[0] > lv[1] ? lv[0] : lv[1];
        bool move = ((bits >> 10) - 14 > exponent) | (bits >= 0x7C00);
        const float rise = kLook - (float)exponent;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            top[t] = fmaxf(sc[t][0], sc[t][1]);
#pragma unroll
            for (int i = 2; i < 8; ++i) top[t] = fmaxf(top[t], sc[t][i]);
            move |= __builtin_fmaf(top[t], factor[t], -ref[t]) > rise;
        }
        return always | (uniform(__builtin_amdgcn_ballot_w64(move) != 0) != 0);
    }

    // Moves the references, once in a while, and with them what the sums hold.  What
    // is done to a row goes by the scores and scales of the tokens that it sees,
    // whatever brought the wave here: a token that only other rows see leaves a
    // row's bits alone.  top: the lane's largest scores; vs: its scales.
    __device__ __forceinline__ void shift(const float (&top)[QT], const float (&sc)[QT][8], const uint32_t (&vs)[2][2 * NB]) {
        float e[8], most = -14.0f;   // exponents of the tokens' largest scales; look() takes subnormals for 2^-14
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float largest = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float d = fabsf((float)scale_of(vs[i >> 2], i & 3, b));
                largest = d < INFINITY ? fmaxf(largest, d) : largest;
            }
            e[i] = largest > 0.0f ? (float)__builtin_amdgcn_frexp_expf(largest) : kNoScale;
            most = fmaxf(most, e[i]);
        }
        exponent = uniform((int)row_most(most));
        bool large = false;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            // The largest product.  That of far scores is rounded to their float32 steps, up
            // to 1/2: one that counts as kTop at most is 2^15.94 then (15.875 and half of 1/8).
            float y = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) y = fmaxf(y, __builtin_fmaf(sc[t][i], factor[t], e[i]));
            y = row_most(y);
            const float x = row_most(top[t]) * factor[t];
            const bool up = (y - ref[t] > kTop) | ((fabsf(ref[t]) >= kLarge) & (x > ref[t]));
            // a large reference is a score's own, so that differences to it are exact
            const float to = up ? (fabsf(x) >= kLarge ? x : y - kLift) : ref[t];
            const float f = __builtin_amdgcn_exp2f(ref[t] - to);
            ref[t] = to;
            l[t] *= f;
#pragma unroll
            for (int d = 0; d < 2 * NB; ++d) o[t][d] *= f;
            large |= (fabsf(to) >= kLarge) & (to != kFloor);
        }
        always = uniform(__builtin_amdgcn_ballot_w64(large) != 0) != 0;
    }

    // CAREFUL: where the reference is large, the score is rounded before the
    // difference, as the reference was, so that the largest one's is 0.  Elsewhere
    // either way gives the same bits: a row's are its own tokens' affair.
    template <bool CAREFUL>
    __device__ __forceinline__ void weights(float (&sc)[QT][8]) {
#pragma clang fp contract(off)
#pragma unroll
        for (int t = 0; t < QT; ++t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float d = __builtin_fmaf(sc[t][i], factor[t], -ref[t]);
                if (CAREFUL) d = fabsf(ref[t]) >= kLarge ? sc[t][i] * factor[t] - ref[t] : d;
                sc[t][i] = __builtin_amdgcn_exp2f(d);
                l[t] += sc[t][i];
            }
        }
    }

    // Weights p times the values, value(t) being their operand and vs the lane's
    // scales.  CAREFUL: a hidden token's scale may be no number; its weight, 0,
    // must stay 0.
    template <bool CAREFUL, class Value>
    __device__ __forceinline__ void add(const Value& value, const uint32_t (&vs)[2][2 * NB], const float (&p)[QT][8]) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const v8h v0 = value(2 * b), v1 = value(2 * b + 1);
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                v8h hi, lo;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float d = (float)scale_of(vs[i >> 2], i & 3, b);
                    if (CAREFUL) d = p[t][i] > 0.0f ? d : 0.0f;
                    hi[i] = (_Float16)__builtin_fmaf(p[t][i], d, 0.0f);
                    if (FULL) lo[i] = (_Float16)__builtin_fmaf(p[t][i], d, -(float)hi[i]);
                }
                o[t][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, hi, o[t][2 * b], 0, 0, 0);
                o[t][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, hi, o[t][2 * b + 1], 0, 0, 0);
                if (FULL) {
                    o[t][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, lo, o[t][2 * b], 0, 0, 0);
                    o[t][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, lo, o[t][2 * b + 1], 0, 0, 0);
                }
            }
        }
    }
};

// Page ids of a piece's steps, every `stride` tokens from k0 on, and where a
// step's halves lie.
struct Pages {
    const int32_t* table;
    const uint8_t* head;     // record of page 0
    int64_t per_page, pages;
    int shift, k0, k1, stride;
    uint32_t lo, hi;         // records of 32 steps' halves, one a lane
    uint64_t there;          // which of them have a page
    const uint8_t* rec[2];
    int slot[2];

    // Bit h of the result: half h of the step has a page (else any page is taken).
    __device__ __forceinline__ int find(int step) {
        if ((step & 31) == 0) {
            const int lane = threadIdx.x & 63, at = k0 + (step + (lane >> 1)) * stride + (lane & 1) * 16;
            int id = -1;
            if (at < k1) {
                id = table[at >> shift];
                if (id >= pages) id = -1;
            }
            const uint64_t address = (uint64_t)(uintptr_t)head + (id >= 0 ? id : 0) * per_page;
            lo = (uint32_t)address;
            hi = (uint32_t)(address >> 32);
            there = __builtin_amdgcn_ballot_w64(id >= 0);
        }
        const int at = k0 + step * stride, mask = (1 << shift) - 1, first = 2 * (step & 31);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t l = __builtin_amdgcn_readlane(lo, first + h), u = __builtin_amdgcn_readlane(hi, first + h);
            rec[h] = reinterpret_cast<const uint8_t*>((uintptr_t)((uint64_t)u << 32 | l));
            slot[h] = (at + 16 * h) & mask;
        }
        return (int)(there >> first) & 3;
    }
};

__device__ __forceinline__ Pages pages_of(const Attend& a, int s, int h, int k0, int k1, int stride) {
    const int64_t per_page = a.c.heads * a.c.record;
    return Pages{a.p.table + s * a.p.stride, a.c.data + h * a.c.record, per_page, a.c.pages, a.c.shift, k0, k1, stride, 0, 0, 0,
                 {nullptr, nullptr}, {0, 0}};
}

// Where a piece from token `from` on begins for rows from `first` on: not before
// their window.
__device__ __forceinline__ int begin_of(const Attend& a, const Sequence& sq, int first, int from) {
    if (!a.q.window) return from;
    const int lo = (sq.pos0 + first / a.q.group - a.q.window + 1) & ~(kTile - 1);
    return from > lo ? from : lo;
}

// The sums of one piece: rows tile `tile` of sequence s and head h over the
// workgroup's
// steps u0 .. u1 - 1.  part < 0: the piece is all there is, and
// the rows go out; else they go to partial `part`.  kNarrow and kWide.
template <bool Q4, int NB, Form F, bool FULL>
__device__ __forceinline__ void piece(const Attend& a, Shared<Q4, NB, F, FULL>& sh, int s, const Sequence& sq, int h, int tile,
                                      int u0, int u1, int part) {
    typedef Step<Q4, NB> S;
    constexpr int QT = row_tiles(F, NB), kRows = 16 * QT, D = 32 * NB, kStages = Shared<Q4, NB, F, FULL>::kStages;
    constexpr int kWaves = Shared<Q4, NB, F, FULL>::kWaves, kUnit = Shared<Q4, NB, F, FULL>::kUnit;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int group = a.q.group, first = tile * kRows;
    const int total = sq.rows * group - first;            // rows from this tile on
    const int live = total < kRows ? total : kRows;

    // Where the wave's steps lie, and the first one's loads on their way.
    const int pos_end = sq.pos0 + (first + live - 1) / group + 1;    // no row of the tile sees further
    const int end = pos_end < sq.last ? pos_end : sq.last;
    const int k0 = begin_of(a, sq, first, sq.first + u0 * kUnit) + wave * kTile;
    int k1 = sq.first + u1 * kUnit;
    k1 = k1 < end ? k1 : end;
    const int steps = k1 > k0 ? (k1 - k0 + kUnit - 1) / kUnit : 0;
    Pages pages = pages_of(a, s, h, k0, k1, kUnit);
    __syncthreads();   // the previous piece is done with LDS
    const auto fetch = [&](int step) {
        const int have = pages.find(step);
#pragma unroll
        for (int j = 0; j < S::kLoads; ++j)
            S::load(j, S::piece_of(j, a.c.record >> 1, a.c.shift, lane), lds_address(&sh.in.step[wave][step % kStages][0]),
                    pages.rec[0], pages.rec[1], pages.slot[0], pages.slot[1], lane);
        return have;
    };
    int have = steps > 0 ? fetch(0) : 0;
    stage_queries<NB, FULL, kWaves>(a, sh, sh.in.query.q, sq, h, first, live);
    __syncthreads();
    Rows<NB, QT, FULL> rows;
    rows.begin(a, sq, first, live, sh.factor);

    // With two steps in LDS the next one is asked for before this one is worked
    // on, with one after it.  A step that moves a reference, or needs care, leaves
    // the inner loop: with the rescaling inside it the sums would be copied every
    // step.
    for (int step = 0; step < steps; ++step) {
        float sc[QT][8], top[QT];
        const uint8_t* buf = nullptr;
        bool out;
        const auto add = [&](auto careful) {
            uint32_t vs[2][2 * NB];
            typename S::Codes codes;
            S::scales(buf, true, 0, lane, vs[0]);
            S::scales(buf, true, 1, lane, vs[1]);
            S::codes(buf, lane, codes);
            rows.template add<decltype(careful)::value>([&](int t) { return S::value(codes, t); }, vs, sc);
            reads_done();
            if (kStages == 1 && step + 1 < steps) have = fetch(step + 1);
        };
        do {
            const int at = k0 + step * kUnit;
            buf = &sh.in.step[wave][step % kStages][0];
            const int had = have;
            if (kStages > 1 && step + 1 < steps) {
                have = fetch(step + 1);
                landed<S::kLoads>();
            } else {
                landed<0>();
            }
            uint32_t ks[2][2 * NB], levels[S::kLevels];
            S::scales(buf, false, 0, lane, ks[0]);
            S::scales(buf, false, 1, lane, ks[1]);
            S::levels(buf, lane, levels);
            rows.scores([&](int hf, int b) { return S::key(buf, hf, b, lane); },
                        [&](int t, int b, int lo) { return __builtin_bit_cast(v8h, sh.in.query.q[t][b][lo][lane]); }, ks, sc);
            bool masked;
            out = rows.look(sc, top, levels, at, had, k1, masked);
            if (!out) {
                rows.template weights<false>(sc);
                add(std::false_type{});
                ++step;
            }
        } while (!out && step < steps);
        if (!out) break;
        uint32_t vs[2][2 * NB];
        S::scales(buf, true, 0, lane, vs[0]);
        S::scales(buf, true, 1, lane, vs[1]);
        rows.shift(top, sc, vs);
        rows.template weights<true>(sc);
        add(std::true_type{});
    }

    // Join the waves: a common reference, then their sums in order.
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float l = rows.l[t];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) {
            sh.m[wave][16 * t + col] = rows.ref[t];
            sh.l[wave][16 * t + col] = l;
        }
    }
    __syncthreads();   // and all waves are done with the queries
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if (16 * t >= live) break;
        float top = sh.m[0][16 * t + col];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sh.m[w][16 * t + col]);
        const float f = __builtin_amdgcn_exp2f(rows.ref[t] - top);
        if (t > 0) __syncthreads();
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d)
            *reinterpret_cast<v4f*>(&sh.o[wave][col][16 * d + 4 * g]) = rows.o[t][d] * f;
        __syncthreads();
        for (int i = tid; i < 16 * D / 4; i += 64 * kWaves) {
            const int r = i / (D / 4), d = 4 * (i - r * (D / 4)), row = 16 * t + r;
            if (row >= live) break;
            v4f x = *reinterpret_cast<const v4f*>(&sh.o[0][r][d]);
#pragma unroll
            for (int w = 1; w < kWaves; ++w) x += *reinterpret_cast<const v4f*>(&sh.o[w][r][d]);
            float mr = sh.m[0][row], sum = 0.0f;
#pragma unroll
            for (int w = 1; w < kWaves; ++w) mr = fmaxf(mr, sh.m[w][row]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) sum += sh.l[w][row] * __builtin_amdgcn_exp2f(sh.m[w][row] - mr);
            put(a, sq, h, first, row, part, kRows, D, d, x, mr, sum);
        }
    }
}

// The same for kTall.  Step i + 1 becomes operands while all waves work on step
// i (with room for one step of operands: step i before they do), and step i + 2
// is under way meanwhile; one barrier a step, two with one step of operands.
template <bool Q4, int NB, Form F, bool FULL>
__device__ __forceinline__ void tall_piece(const Attend& a, Shared<Q4, NB, F, FULL>& sh, int s, const Sequence& sq, int h,
                                           int tile, int u0, int u1, int part) {
    typedef Step<Q4, NB> S;
    constexpr int QT = row_tiles(F, NB), kRows = tile_rows(F, NB), D = 32 * NB, kStages = Shared<Q4, NB, F, FULL>::kStages;
    constexpr int W = Shared<Q4, NB, F, FULL>::kWaves, kUnit = Shared<Q4, NB, F, FULL>::kUnit;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int group = a.q.group, first = tile * kRows;
    const int total = sq.rows * group - first;
    const int live = total < kRows ? total : kRows;
    const int own = 16 * QT * wave, mine = live - own < 0 ? 0 : live - own < 16 * QT ? live - own : 16 * QT;   // this wave's

    const int pos_end = sq.pos0 + (first + live - 1) / group + 1;
    const int end = pos_end < sq.last ? pos_end : sq.last;
    const int k0 = begin_of(a, sq, first, sq.first + u0 * kUnit);
    int k1 = sq.first + u1 * kUnit;
    k1 = k1 < end ? k1 : end;
    const int steps = k1 > k0 ? (k1 - k0 + kTile - 1) / kTile : 0;
    Pages pages = pages_of(a, s, h, k0, k1, kTile);
    // A wave's share of a step's copies, and of its operands.
    constexpr int kOwn = (S::kLoads + W - 1) / W;
    typename S::Piece pieces[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) pieces[i] = S::piece_of(i * W + wave, a.c.record >> 1, a.c.shift, lane);
    const auto fetch = [&](int step) {
        const int have = pages.find(step);
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (i * W + wave < S::kLoads)
                S::load(i * W + wave, pieces[i], lds_address(&sh.in.step[step & 1][0]), pages.rec[0], pages.rec[1],
                        pages.slot[0], pages.slot[1], lane);
        return have;
    };
    const auto convert = [&](int step) {
        const uint8_t* from = &sh.in.step[step & 1][0];
        auto& to = sh.in.operand[step % kStages];
#pragma unroll
        for (int i = 0; i < (2 * NB + S::kShares + W - 1) / W; ++i) {
            const int f = W * i + wave, v = f - 2 * NB;   // operand (half, block) of keys, then share of the values
            if (f < 2 * NB)
                to.key[f & 1][f >> 1][lane] = __builtin_bit_cast(uint4, S::key(from, f & 1, f >> 1, lane));
            else if (v < S::kShares)
                S::convert_values(from, v, lane, reinterpret_cast<uint32_t*>(&to.value[0][0]));
        }
        const int c = tid - 64 * (W - 1);   // not the wave that has a copy more
        if (c >= 0 && c < 8 * NB) reinterpret_cast<uint4*>(to.scale)[c] = reinterpret_cast<const uint4*>(from + S::kScales)[c];
    };

    __syncthreads();   // the previous piece is done with LDS
    stage_queries<NB, FULL, W>(a, sh, sh.query.q, sq, h, first, live);
    __syncthreads();
    v8h q[QT][NB][FULL ? 2 : 1];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < (FULL ? 2 : 1); ++i) q[t][b][i] = __builtin_bit_cast(v8h, sh.query.q[QT * wave + t][b][i][lane]);
    Rows<NB, QT, FULL> rows;
    rows.begin(a, sq, first + own, mine > 0 ? mine : 1, sh.factor + own);
    if (mine == 0) rows.any_hi = -1;
    reads_done();
    __syncthreads();

    int have = 0, next = 0, after = 0;
    if (steps > 0) have = fetch(0);
    if (kStages == 2 && steps > 0) {
        landed<0>();
        __syncthreads();
        if (steps > 1) next = fetch(1);
        convert(0);
    }
    for (int step = 0; step < steps; ++step) {
        float sc[QT][8], top[QT];
        bool out = false;
        const auto* op = &sh.in.operand[0];
        const auto add = [&](auto careful) {
            uint32_t vs[2][2 * NB];
            S::scales_at(op->scale, true, 0, lane, vs[0]);
            S::scales_at(op->scale, true, 1, lane, vs[1]);
            rows.template add<decltype(careful)::value>([&](int t) { return __builtin_bit_cast(v8h, op->value[t][lane]); }, vs,
                                                        sc);
        };
        do {
            const int at = k0 + step * kTile;
            landed<0>();
            __syncthreads();   // the copies of all waves have landed, and step - 1 is done with
            if (kStages == 2) {
                if (step + 1 < steps) convert(step + 1);
                if (step + 2 < steps) after = fetch(step + 2);
            } else {
                if (step + 1 < steps) next = fetch(step + 1);
                convert(step);
                __syncthreads();
            }
            op = &sh.in.operand[step % kStages];
            const int had = have;
            have = next;
            next = after;
            // a step past what this wave's rows see, or before it, is the others'
            if (at <= rows.any_hi && at + kTile > rows.any_lo) {
                uint32_t ks[2][2 * NB], levels[S::kLevels];
                S::scales_at(op->scale, false, 0, lane, ks[0]);
                S::scales_at(op->scale, false, 1, lane, ks[1]);
                S::levels_at(op->scale, lane, levels);
                // ahead of waves that still copy and convert: else those that work on the
                // matrix units wait for their issue slots, and the barrier for them
                __builtin_amdgcn_s_setprio(1);
                rows.scores([&](int hf, int b) { return __builtin_bit_cast(v8h, op->key[hf][b][lane]); },
                            [&](int t, int b, int lo) { return q[t][b][lo]; }, ks, sc);
                bool masked;
                out = rows.look(sc, top, levels, at, had, k1, masked);
                if (!out) {
                    rows.template weights<false>(sc);
                    add(std::false_type{});
                }
            }
            __builtin_amdgcn_s_setprio(0);
            if (!out) ++step;
        } while (!out && step < steps);
        if (!out) break;
        uint32_t vs[2][2 * NB];
        S::scales_at(op->scale, true, 0, lane, vs[0]);
        S::scales_at(op->scale, true, 1, lane, vs[1]);
        rows.shift(top, sc, vs);
        rows.template weights<true>(sc);
        add(std::true_type{});
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int row = 16 * t + col;
        float l = rows.l[t];
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (row >= mine) continue;
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d)
            put(a, sq, h, first, own + row, part, kRows, D, 16 * d + 4 * g, rows.o[t][d], rows.ref[t], l);
    }
}

// Where this workgroup's run begins (s, base: the sequence and its first step;
// u .. end - 1: the run): each thread adds up its share of the sequences, and
// the one whose share holds the run's first step finds it.
template <int W, class S>
__device__ __forceinline__ void find_run(const Attend& a, S& sh, int rows, int& s, int64_t& base, int64_t& u,
                                         int64_t& end, int64_t& total, int64_t& wgs) {
    const int tid = threadIdx.x;
    const int per_thread = (a.p.seqs + 64 * W - 1) / (64 * W);
    const int s0 = tid * per_thread, s1 = s0 + per_thread < a.p.seqs ? s0 + per_thread : a.p.seqs;
    const auto cost = [&](int i) {
        const Sequence sq = sequence<S::kUnit>(a, i);
        return (int64_t)a.c.heads * ((sq.rows * a.q.group + rows - 1) / rows) * sq.units;
    };
    int64_t mine = 0;
    for (int i = s0; i < s1; ++i) mine += cost(i);
    int64_t upto = mine;   // inclusive, within the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t v = __shfl_up(upto, o);
        if ((tid & 63) >= o) upto += v;
    }
    if ((tid & 63) == 63) sh.scan[tid >> 6] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < tid >> 6) upto += sh.scan[w];
        total += sh.scan[w];
    }
    wgs = a.wgs < total ? a.wgs : total;   // no run is empty
    const int64_t wg = blockIdx.x;
    if (wg >= wgs) return;
    u = total * wg / wgs;
    end = total * (wg + 1) / wgs;
    if (u >= upto - mine && u < upto) {
        int64_t at = upto - mine;
        int i = s0;
        for (;; ++i) {
            const int64_t c = cost(i);
            if (u < at + c) break;
            at += c;
        }
        sh.found = i;
        sh.base = at;
    }
    __syncthreads();
    s = uniform(sh.found);
    base = sh.base;
}

// wgs > 0: the steps of all sequences, heads and row tiles in one line, cut
// into wgs equal runs, one a workgroup; a piece that is not all of its rows'
// tokens leaves its sums for join_kernel.  At most two pieces of a run are such:
// its first (slot 0) and its last.  wgs == 0: a workgroup per row tile, head
// and sequence, the last rows, which see most, first.
template <bool Q4, int NB, Form F, bool FULL>
__global__ __launch_bounds__(64 * waves_of(F),
                             wgs_per_cu(Q4, NB, F, FULL) * waves_of(F) / 4) void attend_kernel(Attend a) {
    static_assert(sizeof(Shared<Q4, NB, F, FULL>) <= lds_bytes(Q4, NB, F, FULL, stages(Q4, NB, F, FULL)));
    __shared__ __attribute__((aligned(16))) Shared<Q4, NB, F, FULL> sh;
    constexpr int kRows = tile_rows(F, NB), kWaves = Shared<Q4, NB, F, FULL>::kWaves, kUnit = Shared<Q4, NB, F, FULL>::kUnit;
    const int heads = a.c.heads, group = a.q.group;
    int s = 0, slot = 0;
    int64_t base = 0, u = 0, end = 0, total = 0, wgs = 0;
    Join join = {};
    if (a.wgs == 0) {
        s = blockIdx.z;
        const Sequence sq = sequence_of_all<kUnit>(a, s);
        const int tiles = (sq.rows * group + kRows - 1) / kRows, tile = (int)gridDim.x - 1 - (int)blockIdx.x;
        if (tile < tiles) {
            u = (int64_t)((int)blockIdx.y * tiles + tile) * sq.units;
            end = u + sq.units;
        }
    } else {
        find_run<kWaves>(a, sh, kRows, s, base, u, end, total, wgs);
    }
    while (u < end) {
        const Sequence sq = sequence_of_all<kUnit>(a, s);
        const int tiles = (sq.rows * group + kRows - 1) / kRows;
        const int64_t here = u - base, all = (int64_t)heads * tiles * sq.units;
        if (here >= all) {
            base += all;
            ++s;
            continue;
        }
        const int e = uniform((int)((uint32_t)here / (uint32_t)sq.units)), off = uniform((int)here - e * sq.units);
        const int most = sq.units - off, count = uniform(end - u < most ? (int)(end - u) : most);
        const bool whole = count == sq.units;
        const int tile = e % tiles;
        const int part = whole ? -1 : 2 * (int)blockIdx.x + slot;
        if constexpr (F == kTall)
            tall_piece<Q4, NB, F, FULL>(a, sh, s, sq, e / tiles, tile, off, off + count, part);
        else
            piece<Q4, NB, F, FULL>(a, sh, s, sq, e / tiles, tile, off, off + count, part);
        if (!whole && off == 0)   // begun here: these rows are this workgroup's to join
            join = {(int)(((base + (int64_t)(e + 1) * sq.units) * wgs - 1) / total) - (int)blockIdx.x + 1, slot,
                    sq.row0, sq.rows * group - tile * kRows, e / tiles, tile * kRows, {0, 0}};
        u += count;
        slot = 1;
    }
    if (a.wgs > 0 && threadIdx.x == 0) a.join[blockIdx.x] = join;
}

template <bool Q4, int NB, Form F>
hipError_t launch_form(const Attend& a, dim3 grid, hipStream_t stream) {
    if (a.q.q_half && a.q.out_half) {   // else the query or the output has more bits than binary16
        hipLaunchKernelGGL((attend_kernel<Q4, NB, F, false>), grid, dim3(64 * waves_of(F)), 0, stream, a);
    } else if constexpr (fits(Q4, NB, F, true)) {
        hipLaunchKernelGGL((attend_kernel<Q4, NB, F, true>), grid, dim3(64 * waves_of(F)), 0, stream, a);
    } else {
        return hipErrorInvalidConfiguration;   // not built
    }
    return hipGetLastError();
}

template <bool Q4, int LO, int HI>
hipError_t launch_dims(const Attend& a, Form f, dim3 grid, hipStream_t stream) {
    // cut() takes these without a look at fits()
    static_assert(fits(Q4, LO, kNarrow, true) && fits(Q4, LO, kTall, true) && (!has_wide(Q4, LO) || fits(Q4, LO, kWide, true)));
    if constexpr (LO < HI) {
        if (a.c.dim > 32 * LO) return launch_dims<Q4, LO + 1, HI>(a, f, grid, stream);
    }
    if (f == kNarrow) return launch_form<Q4, LO, kNarrow>(a, grid, stream);
    if (f == kTall) return launch_form<Q4, LO, kTall>(a, grid, stream);
    if constexpr (has_wide(Q4, LO)) {
        if (f == kWide) return launch_form<Q4, LO, kWide>(a, grid, stream);
        if (f == kWide8) return launch_form<Q4, LO, kWide8>(a, grid, stream);
    }
    return hipErrorInvalidConfiguration;   // not built
}

// Head sizes up to 128, and above: each in a file of its own, to build side by side.
hipError_t launch_q8_narrow(const Attend& a, Form f, dim3 grid, hipStream_t stream);
hipError_t launch_q8_broad(const Attend& a, Form f, dim3 grid, hipStream_t stream);
hipError_t launch_q4_narrow(const Attend& a, Form f, dim3 grid, hipStream_t stream);
hipError_t launch_q4_broad(const Attend& a, Form f, dim3 grid, hipStream_t stream);

}  // namespace kv
}  // namespace mmq
