// mmq_group_few.hip - streaming few-token products on 16x16x32 int8 MFMA: the
// matmuls grouped by expert for experts of few slots, and q6_K with an
// epilogue where there are few tiles of tokens and rows.
//
// Method as in the other kernels: exact integer dots of a chunk (k = 32; in
// q6_K of its two scale groups, k = 16), then the fold.
//
//   * A is 16 tokens, B 16 weight rows: lane l supplies k = 8 (l / 16) .. +7 of
//     the chunk for token / row l % 16, and holds the results of row l % 16
//     with tokens 4 (l / 16) .. +3, so the weight scales are per-lane values.
//     Unused tokens of a tile are padding: the stream of weights leaves the
//     vector unit time for them.
//   * q4_K: the MFMA starts from the bits of 1.5 * 2^23, so its result D read
//     as float32 is 1.5 * 2^23 + D exactly; fma(sc, that, -1.5 * 2^23 * sc) is
//     sc * D, exact as |sc * D| < 2^22; then acc_b += da * it, da taken as
//     binary16 by the mixed-precision multiply-add.  Per super-block out += d *
//     acc_b, and the min term on v_mfma_f32_16x16x4_f32.
//   * q6_K: the two groups' dots come from two MFMAs on the same tokens, the
//     weights of the other group's lanes set to 0 (lanes 0-31 hold the first
//     group's k); sc0*D0 + sc1*D1 is exact in 24-bit integer operations.
//   * A workgroup of W waves goes over its units, a unit being 16 W/KS rows of
//     one item: W/KS row tiles of 16, KS waves on each that take its
//     super-blocks in turn.  KS > 1 adds the waves' sums through LDS, in wave
//     order.  The kernel counts the items and chooses KS itself (split()).
//   * A wave's step is one super-block and one tile of 16 tokens.  It reads
//     its copy of the step (weights, codes, scale words) from its LDS area into
//     registers, and at once sends the next step's copies into the same area
//     (buffer loads that write LDS directly, in inline asm outside the
//     compiler's wait bookkeeping); they are in flight during the arithmetic,
//     also from one unit to the next.  One area per wave leaves room for 16
//     waves per CU: with 8 waves and two areas a SIMD's two waves issued
//     vector instructions at less than half its rate (8 experts of 14336 x
//     4096, 8 slots each: 99 us, 87 of them without any copies; this form 71).
//   * T = 1 takes items of up to 16 tokens.  T = 4 takes up to 64, the weights
//     decoded once for all their tiles; its copy addresses are computed anew,
//     which leaves the loop its registers.
//
// Measured (graph of calls): q4_K, 14336 x 4096, 2 / 8 experts of 2 slots 18 /
// 66-72 us (weights alone at the copy rate 13 / 52), 8 of 16 82, of 32 121; 64
// experts of 1536 x 4096 at 4 / 16 / 32 slots 58 / 73 / 105 us (45 / 46 / 48);
// q6_K, 64 of 4096 x 1536 at 1 / 16 / 32 / 64 slots 85-90 / 104 / 157 / 261 us (64
// / 68 / 71 / 79).  Up to 16 slots the weights stream at 3 to 4.3 TB/s (with the
// codes of 4 tokens only and two steps in flight no faster, so not for want of
// copies in flight); above, vector issue bounds it (per 16 x 16 outputs and
// chunk 8 operations in q4_K, 16 in q6_K, and the decode): at 32 slots in q4_K
// the vector unit is busy 72% of the time and the matrix core 15%, at 64 in q6_K
// 80% and 16%.
#include <algorithm>
#include <type_traits>

#include "f16_operand.h"
#include "group.h"
#include "internal.h"
#include "kquant_device.h"
#include "q6k_device.h"
#include "q6k_stage.h"

namespace mmq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kFlush = 256;      // super-blocks of a wave between accumulator moves (BIG)

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
constexpr int kMagicBits = 0x4B400000;

// By value: a bit cast of a vector's element reads its first element.
__device__ __forceinline__ float as_float(int x) { return __builtin_bit_cast(float, x); }

typedef __attribute__((address_space(3))) uint8_t* Lds;
template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
    return *(__attribute__((address_space(3))) const V*)(uintptr_t)at;
}
template <class V>
__device__ __forceinline__ void lds_write(uint32_t at, V v) {
    *(__attribute__((address_space(3))) V*)(uintptr_t)at = v;
}

// Barrier of the workgroup for LDS only: copies stay in flight over it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A plain call: `tokens` tokens, the rows of q.
struct OneGroup {
    int tokens;
};

// The sum of v over this lane and those below it: DPP moves within rows of 16
// lanes (row_shr 1, 2, 4, 8), then from lane 15 of a row to the next row and
// from lane 31 to the upper half (row_bcast 15, 31).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// The items of a launch: their number and item i (wave-collective).  Up to 64
// experts are held in registers, lane e the slots of expert e, so that only
// the kernel's start loads the offsets.
template <int TB, class Grp>
struct Finder {
    const Groups& g;
    int first, slots, incl;   // first slot, slots, items up to this expert
    int total;
    __device__ __forceinline__ explicit Finder(const Groups& grp) : g(grp), total(0) {
        int high = 0;
        for (int base = 0; base < g.experts; base += 64) {
            const Span s = expert_slots(g, base, high);
            first = s.first;
            slots = s.slots;
            incl = wave_scan(slots >= g.lo && slots <= g.hi ? (slots + TB - 1) / TB : 0);
            total += __builtin_amdgcn_readlane(incl, 63);
        }
    }
    __device__ __forceinline__ int count() const { return total; }
    __device__ __forceinline__ Item operator()(int i) const {
        if (g.experts > 64) return find_item<TB>(g, i);
        const uint64_t past = __ballot(incl > i);
        if (!past) return Item{0, 0, 0, false};
        const int l = __builtin_ctzll(past);
        const int before = l ? __builtin_amdgcn_readlane(incl, l - 1) : 0;
        const int skip = (i - before) * TB, n = __builtin_amdgcn_readlane(slots, l);
        return Item{l, __builtin_amdgcn_readlane(first, l) + skip, min(TB, n - skip), true};
    }
};
template <int TB>
struct Finder<TB, OneGroup> {
    const int tokens;
    __device__ __forceinline__ explicit Finder(const OneGroup& g) : tokens(g.tokens) {}
    __device__ __forceinline__ int count() const { return (tokens + TB - 1) / TB; }
    __device__ __forceinline__ Item operator()(int i) const {
        return Item{0, i * TB, min(TB, tokens - i * TB), i < count()};
    }
};

// ------------------------------------------------------------------- q4_K
struct Q4k {
    static constexpr int kBlock = kBlockBytes;
    // 16 rows of 144 bytes (9 pieces, an odd number, so 16 rows' reads of one
    // piece meet different banks): two copies and a quarter of one.
    static constexpr int kRow = kBlockBytes, kBytes = 16 * kRow, kCopies = 3, kLast = 16;
    // Byte offset in the tile, for super-block 0, of copy c's piece (slot i =
    // 64c + lane: piece i % 9 of row i / 9; rows past the tile lie past the
    // resource: zeros, not used).
    __device__ static uint32_t piece(int c, int lane, int S) {
        const int i = 64 * c + lane;
        return (uint32_t)(i / 9) * (uint32_t)(S * kBlock) + 16u * (uint32_t)(i % 9);
    }
    __device__ static uint32_t offset(uint32_t piece, int sb) { return piece + (uint32_t)(sb * kBlock); }

    // A super-block's bytes of row r, k = 8kg.. of each chunk, as they are.
    struct Raw {
        v4u hdr;
        v2u qs[4];
        __device__ __forceinline__ void read(uint32_t area, int r, int kg, int, int) {
            const uint32_t p = area + kRow * r;
            hdr = lds_read<v4u>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) qs[i] = lds_read<v2u>(p + 16 + 32 * i + 8 * kg);
        }
    };
    __device__ static void patch(uint32_t, uint64_t, int, int, int, int) {}

    int64_t b[8];
    uint32_t sc[2];   // eight scale bytes
    float d, bneg[2];
    __device__ __forceinline__ float scale(int c) const { return (float)((sc[c >> 2] >> (8 * (c & 3))) & 0xFFu); }
    __device__ __forceinline__ void decode(const Raw& x, int kg) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const v2u y = x.qs[p];
            b[2 * p] = (int64_t)(((uint64_t)(y[1] & 0x0F0F0F0Fu) << 32) | (y[0] & 0x0F0F0F0Fu));
            b[2 * p + 1] = (int64_t)(((uint64_t)((y[1] >> 4) & 0x0F0F0F0Fu) << 32) | ((y[0] >> 4) & 0x0F0F0F0Fu));
        }
        // the 6-bit fields as bytes (packing: kquant_device.h), scales 0-3 and
        // 4-7, mins alike
        const v4u h = x.hdr;
        sc[0] = h[1] & 0x3F3F3F3Fu;
        sc[1] = (h[3] & 0x0F0F0F0Fu) | ((h[1] >> 2) & 0x30303030u);
        const uint32_t m0 = h[2] & 0x3F3F3F3Fu, m1 = ((h[3] >> 4) & 0x0F0F0F0Fu) | ((h[2] >> 2) & 0x30303030u);
        d = half_lo(h[0]);
        const float dmin = -half_lo(h[0] >> 16);
        bneg[0] = dmin * (float)((m0 >> (8 * kg)) & 0xFFu);
        bneg[1] = dmin * (float)((m1 >> (8 * kg)) & 0xFFu);
    }
    // out's part of the super-block: a = the lane's token operands, da(i, c) =
    // da of token 4 kg + i, own = the words of token r, chunks kg and kg + 4.
    template <class D>
    __device__ __forceinline__ v4f fold(const int64_t (&a)[8], const D& da, const uint32_t (&own)[2], int) const {
        v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f}, part = s;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            part = __builtin_amdgcn_mfma_f32_16x16x4f32(half_lo(own[j]) * (float)(int16_t)(uint16_t)(own[j] >> 16),
                                                        bneg[j], part, 0, 0, 0);
        const v4i magic = v4i{kMagicBits, kMagicBits, kMagicBits, kMagicBits};
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // four dots before their folds, which then find them done
            v4i D4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                D4[c] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[4 * h + c], b[4 * h + c], magic, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float f = scale(4 * h + c), kf = -kMagic * f;   // exact: 6 bits times 2
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = fmaf(da(i, 4 * h + c), fmaf(f, as_float(D4[c][i]), kf), s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) part[i] = fmaf(d, s[i], part[i]);
        return part;
    }
};

// ------------------------------------------------------------------- q6_K
struct Q6k {
    static constexpr int kBlock = kQ6kBlockBytes;
    // Rows of 14 pieces from the 16-byte boundary at or below the block, and a
    // padding slot (q6k_stage.h): three copies and three quarters of one.
    static constexpr int kRow = Seg<1>::kBytes, kBytes = 16 * kRow, kCopies = 4, kLast = 48;
    static_assert(kBytes == 3 * 1024 + 16 * kLast, "the last copy's lanes");
    __device__ static uint32_t piece(int c, int lane, int S) {
        const int i = 64 * c + lane;
        // the row's bytes and the piece number (its low 4 bits free: rows are
        // a multiple of 16 bytes only with the block's offset added)
        return (uint32_t)min(i / Seg<1>::kSlots, 15) * (uint32_t)(S * kBlock) |
               ((uint32_t)min(i % Seg<1>::kSlots, Seg<1>::kChunks - 1) << 28);
    }
    __device__ static uint32_t offset(uint32_t piece, int sb) {
        return (((piece & 0x0FFFFFFFu) + (uint32_t)(sb * kBlock)) & ~15u) + ((piece >> 28) << 4);
    }

    struct Raw {
        uint32_t l0[2][3], l1[2][3], h[2][3], sc[5], d;
        uint32_t sh;
        __device__ __forceinline__ void read(uint32_t area, int r, int kg, int S, int sb) {
            const uint32_t off = ((uint32_t)(r * S + sb) * (uint32_t)kBlock) & 15u;
            sh = off & 3u;
            const uint32_t row = area + kRow * r + (off & ~3u), p = row + 8 * kg;
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    l0[g][i] = lds_read<uint32_t>(p + 64 * g + 4 * i);
                    l1[g][i] = lds_read<uint32_t>(p + 64 * g + 32 + 4 * i);
                    h[g][i] = lds_read<uint32_t>(p + 128 + 32 * g + 4 * i);
                }
#pragma unroll
            for (int i = 0; i < 5; ++i) sc[i] = lds_read<uint32_t>(row + 192 + 4 * i);
            d = lds_read<uint32_t>(row + 208);
        }
    };
    // The tile's last bytes, where they end inside a 16-byte piece.
    __device__ static void patch(uint32_t area, uint64_t base, int rows, int S, int sb, int lane) {
        const int end = rows * S * kBlock, end16 = end & ~15;
        if (end16 == end) return;
        const int ch = (end16 - ((((rows - 1) * S + sb) * kBlock) & ~15)) >> 4;
        if (lane == 0 && ch >= 0 && ch < Seg<1>::kChunks) {
            const uint4 v = load_piece(reinterpret_cast<const uint8_t*>(base), end16, end);
            lds_write<v4u>(area + (uint32_t)((rows - 1) * kRow + 16 * ch), v4u{v.x, v.y, v.z, v.w});
        }
    }

    int64_t b[8];
    uint32_t sc[4];   // sixteen scale bytes
    float d;
    __device__ __forceinline__ void decode(const Raw& x, int) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t l0[2], l1[2], h[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l0[i] = __builtin_amdgcn_alignbyte(x.l0[g][i + 1], x.l0[g][i], x.sh);
                l1[i] = __builtin_amdgcn_alignbyte(x.l1[g][i + 1], x.l1[g][i], x.sh);
                h[i] = __builtin_amdgcn_alignbyte(x.h[g][i + 1], x.h[g][i], x.sh);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    c[i] = q6k::signed_codes(((j & 1) ? l1[i] : l0[i]) >> (4 * (j >> 1)), h[i] >> (2 * j));
                b[4 * g + j] = (int64_t)(((uint64_t)c[1] << 32) | c[0]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = __builtin_amdgcn_alignbyte(x.sc[i + 1], x.sc[i], x.sh);
        d = half_lo(x.d >> (8 * x.sh));
    }
    template <class D>
    __device__ __forceinline__ v4f fold(const int64_t (&a)[8], const D& da, const uint32_t (&)[2], int kg) const {
        v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        const v4i zero = v4i{0, 0, 0, 0};
        const int64_t lo = kg < 2 ? -1 : 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {   // two chunks' dots before their folds
            v4i d0[2], d1[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                d0[c] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[2 * h + c], b[2 * h + c] & lo, zero, 0, 0, 0);
                d1[c] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[2 * h + c], b[2 * h + c] & ~lo, zero, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int sc0 = (int8_t)(sc[h] >> (16 * c)), sc1 = (int8_t)(sc[h] >> (16 * c + 8));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[i] = fmaf(da(i, 2 * h + c), (float)(__mul24(sc0, d0[c][i]) + __mul24(sc1, d1[c][i])), s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] *= d;
        return s;
    }
};

// The waves on a row tile, as the logarithm of their number: the least time by
// a model of the work on the busiest CU, its units times a unit's steps and
// 4/3 of a step for its ends, a quarter more where a CU has one workgroup of 8
// waves.  (q4_K, k = 4096, KS = 1 / 2 / 4 / 8: 1792 tiles 21.7 / 20.2 / 21.5 /
// 21.8 us, 2688 tiles 31.1 / 24.6 / - / 28.5 us, 7168 tiles 82.5 / - / - / 71.8 us.)
// With 2^16 tiles or more (32 units per CU) a wave each; below that the model's
// numbers fit 32 bits, as S <= 2^16.
template <int W>
__device__ __forceinline__ int split(int items, int tiles, int S) {
    if ((uint64_t)(uint32_t)items * (uint32_t)tiles >= 1u << 16) return 0;
    int best = 0;
    uint32_t least = ~0u;
#pragma unroll
    for (int l = 0; 1 << l <= W; ++l) {
        const uint32_t units = (uint32_t)items * ((uint32_t)((tiles << l) + W - 1) / W);
        const uint32_t cost = ((units + 255) >> 8) * (uint32_t)(3 * ((S + (1 << l) - 1) >> l) + 4) *
                              (W < 16 && units <= 256 ? 5u : 4u);
        if ((1 << l) <= S && cost < least) {
            least = cost;
            best = l;
        }
    }
    return best;
}

// BIG: rows of more than kFlush super-blocks, whose sums move into a second
// accumulator every kFlush.
// W waves per workgroup, 16 / W workgroups per CU.
template <class F, int T, bool BIG, class Grp, int W>
__global__ __launch_bounds__(64 * W, 4) void mmq_group_few_kernel(const uint8_t* __restrict__ w,
                                                                       const int8_t* __restrict__ q,
                                                                       const uint32_t* __restrict__ ds, int M, int K,
                                                                       OutEpi out, Grp grp) {
    // a wave's area: weights; codes, slot 16t + s holding piece s ^ t of token t;
    // 8 scale words per token
    // (T > 1: then the row of q of each token of the item)
    constexpr int kCodes = F::kBytes, kWords = kCodes + 16 * 256, kRows = kWords + 16 * 32;
    constexpr int kArea = kRows + (T > 1 ? (64 * T + 255) / 256 * 256 : 0);
    static_assert(kCodes % 256 == 0 && kArea % 256 == 0, "the codes start on a 256-byte boundary");
    __shared__ __attribute__((aligned(256))) uint8_t areas[W * kArea];
    __shared__ v4f red[W][64];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // wave-uniform
    const int r = lane & 15, kg = lane >> 4;
    const int S = K >> 8;
    const int tiles = (M + 15) >> 4;
    const uint32_t area = (uint32_t)(uintptr_t)(Lds)areas + (uint32_t)(wv * kArea);

    const Finder<16 * T, Grp> find(grp);
    const int items = find.count();
    // KS = 1 << ksl waves on a row tile, a unit's row tiles, its place among an
    // item's (units are numbered item by item)
    const int ksl = split<W>(items, tiles, S), KS = 1 << ksl;
    const int per_unit = W >> ksl, unit_tiles = (int)((uint32_t)((tiles << ksl) + W - 1) / W);
    const int rt = wv >> ksl, ks = wv & (KS - 1);

    // A wave's place in its stream: tile tt of 16 tokens, super-block sb of a
    // row tile (its rows from base) of a unit; off, woff (T = 1): this lane's
    // copy offsets of the item's tokens' codes and words at super-block 0.
    struct Pos {
        int unit, tile0, sb, tt;   // tile0: the unit's first row tile
        Item it;
        uint64_t base;
        int rows;
        uint32_t off[4], woff;
    };
    const auto enter = [&](Pos& x, int unit) {
        x.unit = unit;
        x.sb = ks;
        x.tt = 0;
        const int item = (int)((uint32_t)unit / (uint32_t)unit_tiles);
        x.tile0 = (unit - item * unit_tiles) * per_unit;
        x.it = find(item);
        if (!x.it.valid) return;
        // past the last tile: its rows again, not stored
        const int row0 = min(x.tile0 + rt, tiles - 1) * 16;
        const uint64_t base = reinterpret_cast<uint64_t>(w) + ((uint64_t)x.it.expert * M + row0) * S * F::kBlock;
        x.base = base;
        x.rows = min(16, M - row0);
        const auto row_of = [&](int i) {
            if constexpr (std::is_same<Grp, Groups>::value)
                return TokenRows<Groups>(grp, x.it, 0).row(i);
            else
                return (uint32_t)(x.it.start + min(i, x.it.count - 1));
        };
        if constexpr (T == 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c) x.off[c] = row_of(4 * c + kg) * (uint32_t)K + 16u * (uint32_t)(r ^ (4 * c + kg));
            x.woff = row_of(lane >> 1) * (uint32_t)(K >> 3) + 16u * (uint32_t)(lane & 1);
        } else if (lane < 16 * T) {
            lds_write<uint32_t>(area + kRows + 4 * lane, row_of(lane));
        }
    };
    const auto advance = [&](Pos& x) {
        if (T > 1 && 16 * ++x.tt < x.it.count) return;
        x.tt = 0;
        x.sb += KS;
        if (x.sb >= S) enter(x, x.unit + gridDim.x);
    };

    const uint32_t q_bytes = (uint32_t)grp.tokens * (uint32_t)K;
    const uint64_t qa = reinterpret_cast<uint64_t>(q), da_ = reinterpret_cast<uint64_t>(ds);
    const u32x4 qrs = {(uint32_t)qa, (uint32_t)(qa >> 32) & 0xFFFFu, q_bytes, (uint32_t)kBufferFlags};
    const u32x4 drs = {(uint32_t)da_, (uint32_t)(da_ >> 32) & 0xFFFFu, q_bytes / 8, (uint32_t)kBufferFlags};
    uint32_t at[F::kCopies];
    const auto pieces = [&](int ln) {
#pragma unroll
        for (int c = 0; c < F::kCopies; ++c) at[c] = F::piece(c, ln, S);
    };
    if constexpr (T == 1) pieces(lane);
    // The copies of one step.  Those of four tokens past the item's last are
    // left out: what the area holds then is computed with and not stored.
    const auto issue = [&](const Pos& ps) {
        const u32x4 rs = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)ps.base),
                          (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(ps.base >> 32) & 0xFFFFu),
                          (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(ps.rows * S * F::kBlock) & ~15u),
                          (uint32_t)kBufferFlags};
        const uint32_t tok = (uint32_t)ps.sb * 256u;
        if (T == 1 || ps.tt == 0) {
            if constexpr (T > 1) pieces(opaque(lane));   // no registers between the copies
#pragma unroll
            for (int c = 0; c < F::kCopies - 1; ++c) lds_copy16(rs, area + 1024 * c, (int)F::offset(at[c], ps.sb));
            if (lane < F::kLast)
                lds_copy16(rs, area + 1024 * (F::kCopies - 1), (int)F::offset(at[F::kCopies - 1], ps.sb));
        }
        uint32_t off[4], woff;
        if constexpr (T == 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c) off[c] = ps.off[c];
            woff = ps.woff;
        } else {
            const uint32_t row = area + kRows + 64 * ps.tt;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                off[c] = lds_read<uint32_t>(row + 16 * c + 4 * kg) * (uint32_t)K + 16u * (uint32_t)(r ^ (4 * c + kg));
            woff = lds_read<uint32_t>(row + 4 * ((lane >> 1) & 15)) * (uint32_t)(K >> 3) + 16u * (uint32_t)(lane & 1);
        }
        if (lane < 32) lds_copy16(drs, area + kWords, (int)(woff + (tok >> 3)));
        lds_copy16(qrs, area + kCodes, (int)(off[0] + tok));
#pragma unroll
        for (int c = 1; c < 4; ++c)
            if (16 * ps.tt + 4 * c < ps.it.count) lds_copy16(qrs, area + kCodes + 1024 * c, (int)(off[c] + tok));
    };

    // Where this lane reads: token r's bytes 32c + 8kg of the super-block are
    // piece 2c + (kg >> 1), in slot 16 r + (piece ^ r): bits 5-7 of the address
    // are c ^ (r >> 1).
    const uint32_t arow = area + kCodes + 256 * r + 32 * (r >> 1) + 16 * ((kg >> 1) ^ (r & 1)) + 8 * (kg & 1);
    const uint32_t drow = area + kWords + 128 * kg;

    v4f acc[T], acc2[T];
#pragma unroll
    for (int j = 0; j < T; ++j) acc[j] = acc2[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    F x;
    Pos cur, nxt;
    enter(cur, blockIdx.x);
    if (!cur.it.valid) return;   // the same for every wave
    issue(cur);
    nxt = cur;
    advance(nxt);
    for (int done = 0;;) {
        __builtin_amdgcn_s_waitcnt(kWaitVmcnt(0));
        asm volatile("" ::: "memory");
        // the step out of the area
        int64_t a[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) a[c] = lds_read<int64_t>(arow ^ (uint32_t)(32 * c));
        uint32_t da[4][4], own[2];   // of token 4 kg + i, chunks 2j and 2j + 1: binary16 da
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4u t = lds_read<v4u>(drow + 32 * i + 16 * h);
                da[i][2 * h] = __builtin_amdgcn_perm(t[1], t[0], 0x05040100u);
                da[i][2 * h + 1] = __builtin_amdgcn_perm(t[3], t[2], 0x05040100u);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) own[h] = lds_read<uint32_t>(area + kWords + 32 * r + 4 * kg + 16 * h);
        typename F::Raw raw;
        if (T == 1 || cur.tt == 0) {
            F::patch(area, cur.base, cur.rows, S, cur.sb, lane);
            raw.read(area, r, kg, S, cur.sb);
            if constexpr (T > 1) x.decode(raw, kg);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (nxt.it.valid) issue(nxt);   // the next step into it
        __builtin_amdgcn_sched_barrier(0);
        if (T == 1 || cur.tt == 0) {
            if constexpr (T == 1) x.decode(raw, kg);
            if (BIG && done++ == kFlush) {
                done = 1;
#pragma unroll
                for (int j = 0; j < T; ++j) {
                    acc2[j] += acc[j];
                    acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
        }
        const v4f part = x.fold(
            a,
            [&](int i, int c) {
                const uint32_t dd = da[i][c >> 1];
                return half_lo((c & 1) ? dd >> 16 : dd);
            },
            own, kg);
#pragma unroll
        for (int j = 0; j < T; ++j)
            if (T == 1 || cur.tt == j) acc[j] += part;
        if (!nxt.it.valid || nxt.unit != cur.unit) {
            // The unit's end: the KS waves of a row tile are added.
            OutEpi o = out;
            o.advance(cur.it.start);
            if (o.bias) o.bias += (int64_t)cur.it.expert * M;
#pragma unroll 1
            for (int tt = 0; tt < (T == 1 ? 1 : cur.tt + 1); ++tt) {
                v4f sum;
#pragma unroll
                for (int j = 0; j < T; ++j)
                    if (T == 1 || tt == j) sum = BIG ? acc2[j] + acc[j] : acc[j];
                if (KS > 1) {
                    red[wv][lane] = sum;
                    lds_barrier();
                }
                // Output i of each lane of a row tile at a time: with KS > 1
                // spread over the waves.  One store in a loop: unrolled, the
                // epilogue's constants fill the registers of the main loop.
#pragma unroll 1
                for (int u = KS > 1 ? wv : 0; u < (KS > 1 ? 4 * per_unit : 4); u += KS > 1 ? W : 1) {
                    const int i = u & 3, tl = KS > 1 ? u >> 2 : rt;
                    float v = i == 0 ? sum[0] : i == 1 ? sum[1] : i == 2 ? sum[2] : sum[3];
                    if (KS > 1) {
                        v = red[tl * KS][lane][i];
#pragma unroll 1
                        for (int p = 1; p < KS; ++p) v += red[tl * KS + p][lane][i];
                    }
                    const int row = 16 * (cur.tile0 + tl) + r, tok = 16 * tt + 4 * kg + i;
                    if (row < M && tok < cur.it.count) o.put(tok, row, v);
                }
                if (KS > 1) lds_barrier();
            }
#pragma unroll
            for (int j = 0; j < T; ++j) acc[j] = acc2[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            done = 0;
        }
        if (!nxt.it.valid) break;
        cur = nxt;
        advance(nxt);
    }
}

template <class F, int T, int W, class Grp>
hipError_t launch(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, const Grp& g, int64_t items,
                  const OutEpi& out, hipStream_t stream) {
    const int64_t units = items * ((m + 15) / 16);
    const dim3 grid((unsigned)std::min<int64_t>(units, 256 * (16 / W))), block(64 * W);
    const void* f = (k >> 8) > kFlush ? (const void*)mmq_group_few_kernel<F, T, true, Grp, W>
                                      : (const void*)mmq_group_few_kernel<F, T, false, Grp, W>;
    void* args[] = {(void*)&w, (void*)&q, (void*)&ds, (void*)&m, (void*)&k, (void*)&out, (void*)&g};
    return hipLaunchKernel(f, grid, block, args, 0, stream);
}

// Workgroups of 8 waves: with 16, 8 experts of 14336 x 4096 at 2 slots take 73
// us for 66.  A plain matrix has few units, and 16 waves to share one's k
// (8192 x 4096 in q6_K, 64 tokens: 28 us for 31).
template <class F>
hipError_t grouped(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, const Groups& g,
                   const OutEpi& out, hipStream_t stream) {
    const auto items = [&](int64_t tb) { return most_items(g.experts, g.slots, g.lo, g.hi, tb); };
    return g.hi <= kGroupFewMaxTile ? launch<F, 1, 8>(w, m, k, q, ds, g, items(16), out, stream)
                                    : launch<F, 4, 8>(w, m, k, q, ds, g, items(64), out, stream);
}

}  // namespace

hipError_t launch_few_grouped(bool q6k, const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds,
                              const Groups& g, const OutEpi& out, hipStream_t stream) {
    return q6k ? grouped<Q6k>(w, m, k, q, ds, g, out, stream) : grouped<Q4k>(w, m, k, q, ds, g, out, stream);
}

hipError_t launch_q6k_stream(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, int n,
                             const OutEpi& out, hipStream_t stream) {
    const OneGroup g{n};
    return n <= 16 ? launch<Q6k, 1, 16>(w, m, k, q, ds, g, 1, out, stream)
                   : launch<Q6k, 4, 16>(w, m, k, q, ds, g, (n + 63) / 64, out, stream);
}

}  // namespace mmq
