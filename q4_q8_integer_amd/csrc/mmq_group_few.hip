// mmq_group_few.hip - q4_K x q8 products grouped by expert, for experts of up
// to 64 slots: 16x16x32 int8 MFMA, the active experts' weights streamed once.
//
// Method as in the other kernels: exact integer dots of a chunk (k = 32), then
// the two-term fold.
//
//   * A is 16 tokens, B 16 weight rows: lane l supplies k = 8 (l / 16) .. +7 of
//     the chunk for token / row l % 16, and holds the results of row l % 16
//     with tokens 4 (l / 16) .. +3, so the weight scales are per-lane values.
//     Unused tokens of a tile are padding: the stream of weights leaves the
//     vector unit time for them.
//   * The MFMA starts from the bits of 1.5 * 2^23, so its result D read as
//     float32 is 1.5 * 2^23 + D exactly; fma(sc, that, -1.5 * 2^23 * sc) is
//     sc * D, exact as |sc * D| < 2^22; then acc_b += da * it, da taken as
//     binary16 by the mixed-precision multiply-add.  Per super-block out += d *
//     acc_b, and the min term on v_mfma_f32_16x16x4_f32.
//   * A workgroup of 8 waves goes over its units, a unit being 128/KS rows of
//     one item: 8/KS row tiles of 16, KS waves on each that take its
//     super-blocks in turn.  KS (1, 2, 4 or 8) is the least that gives the
//     CUs' 4096 waves a tile each, from the number of items, which the kernel
//     counts itself.  KS > 1 adds the waves' sums through LDS, in wave order.
//   * A wave's step is one super-block and one tile of 16 tokens.  It reads
//     its copy of the step (weights, codes, scale words) from its LDS area
//     into registers, and at once sends the next step's copies into the same
//     area (buffer loads that write LDS directly, in inline asm outside the
//     compiler's wait bookkeeping); they are in flight during the arithmetic,
//     also from one unit to the next.  One area per wave leaves room for 16
//     waves per CU: with 8 (and two areas) a SIMD's two waves issued vector
//     instructions at less than half its rate (8 experts of 14336 x 4096, 8
//     slots each: 99 us, 87 without any copies).
#include <algorithm>

#include "f16_operand.h"
#include "group.h"
#include "internal.h"
#include "kquant_device.h"

namespace mmq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8, kHeld = 2;   // waves per workgroup, workgroups per CU
constexpr int kTokens = 16;            // per item
constexpr int kNT = 64 * kWaves;
constexpr int kFlush = 256;      // super-blocks of a wave between accumulator moves (BIG)

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
constexpr int kMagicBits = 0x4B400000;

// By value: a bit cast of a vector's element reads its first element.
__device__ __forceinline__ float as_float(int x) { return __builtin_bit_cast(float, x); }

// A wave's area, by byte offset.  Weights: 16 rows of 144 bytes (9 pieces, an
// odd number, so 16 rows' reads of one piece meet different banks).  Codes:
// slot 16t + s holds piece s ^ t of token t.  Words: 8 per token.
constexpr int kCodes = 16 * kBlockBytes, kWords = kCodes + 16 * 256, kArea = kWords + 16 * 32;
static_assert(kCodes % 256 == 0 && kArea % 256 == 0, "the codes start on a 256-byte boundary");

typedef __attribute__((address_space(3))) uint8_t* Lds;
template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
    return *(__attribute__((address_space(3))) const V*)(uintptr_t)at;
}

// Barrier of the workgroup for LDS only: copies stay in flight over it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The number of items of a launch (wave-collective).
template <int TB>
__device__ __forceinline__ int count_items(const Groups& g) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int base = 0; base < g.experts; base += 64) {
        const int e = base + lane;
        int c = 0;
        if (e < g.experts) {
            const int a = min(max(g.offsets[e], 0), g.slots);
            c = min(max(g.offsets[e + 1], a), g.slots) - a;
        }
        n += c >= g.lo && c <= g.hi ? (c + TB - 1) / TB : 0;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
    return __builtin_amdgcn_readfirstlane(n);
}

// The weights of one super-block as a lane's operands.
struct Weights {
    int64_t b[8];
    uint32_t sc[2];   // eight scale bytes
    float d, bneg[2];
    __device__ __forceinline__ float scale(int c) const { return (float)((sc[c >> 2] >> (8 * (c & 3))) & 0xFFu); }
    __device__ __forceinline__ void decode(const v4u& hdr, const v2u (&x)[4], int kg) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            b[2 * p] = (int64_t)(((uint64_t)(x[p][1] & 0x0F0F0F0Fu) << 32) | (x[p][0] & 0x0F0F0F0Fu));
            b[2 * p + 1] = (int64_t)(((uint64_t)((x[p][1] >> 4) & 0x0F0F0F0Fu) << 32) | ((x[p][0] >> 4) & 0x0F0F0F0Fu));
        }
        // the 6-bit fields as bytes (packing: kquant_device.h), scales 0-3 and
        // 4-7, mins alike
        const uint32_t s0 = hdr[1] & 0x3F3F3F3Fu, s1 = (hdr[3] & 0x0F0F0F0Fu) | ((hdr[1] >> 2) & 0x30303030u);
        const uint32_t m0 = hdr[2] & 0x3F3F3F3Fu, m1 = ((hdr[3] >> 4) & 0x0F0F0F0Fu) | ((hdr[2] >> 2) & 0x30303030u);
        sc[0] = s0;
        sc[1] = s1;
        d = half_lo(hdr[0]);
        const float dmin = -half_lo(hdr[0] >> 16);
        bneg[0] = dmin * (float)((m0 >> (8 * kg)) & 0xFFu);
        bneg[1] = dmin * (float)((m1 >> (8 * kg)) & 0xFFu);
    }
};

// BIG: rows of more than kFlush super-blocks, whose sums move into a second
// accumulator every kFlush.
template <bool BIG>
__global__ __launch_bounds__(kNT, 2 * kHeld) void mmq_group_few_kernel(const uint8_t* __restrict__ w,
                                                                       const int8_t* __restrict__ q,
                                                                       const uint32_t* __restrict__ ds, int M, int K,
                                                                       OutEpi out, Groups grp) {
    __shared__ __attribute__((aligned(256))) uint8_t areas[kWaves * kArea];
    __shared__ v4f red[kWaves][64];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // wave-uniform
    const int r = lane & 15, kg = lane >> 4;
    const int S = K >> 8;
    const int tiles = (M + 15) >> 4;
    const uint32_t area = (uint32_t)(uintptr_t)(Lds)areas + (uint32_t)(wv * kArea);

    // KS waves on a row tile
    const int items = count_items<kTokens>(grp);
    int KS = 1;
    while (KS < kWaves && 2 * KS <= S && (int64_t)items * tiles * KS < 256 * kHeld * kWaves) KS *= 2;
    const int per_unit = kWaves / KS, unit_tiles = (tiles + per_unit - 1) / per_unit;
    const int rt = wv / KS, ks = wv - rt * KS;

    // A wave's place in its stream: super-block sb of a row tile of a unit; the
    // tile's weights as a buffer resource (base, bytes); off, woff: this lane's
    // copy offsets of the item's tokens' codes and words at super-block 0.
    struct Pos {
        int unit, sb;
        Item it;
        uint32_t lo, hi, bytes;
        uint32_t off[4], woff;
    };
    const auto enter = [&](Pos& x, int unit) {
        x.unit = unit;
        x.sb = ks;
        const int item = unit / unit_tiles, ut = unit - item * unit_tiles;
        x.it = find_item<kTokens>(grp, item);
        if (!x.it.valid) return;
        // past the last tile: its rows again, not stored
        const int row0 = min(ut * per_unit + rt, tiles - 1) * 16;
        const uint64_t base = reinterpret_cast<uint64_t>(w) + ((uint64_t)x.it.expert * M + row0) * S * kBlockBytes;
        x.lo = (uint32_t)base;
        x.hi = (uint32_t)(base >> 32) & 0xFFFFu;
        x.bytes = (uint32_t)(min(16, M - row0) * S * kBlockBytes);
        const TokenRows<Groups> src(grp, x.it, 0);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            x.off[c] = src.row(4 * c + kg) * (uint32_t)K + 16u * (uint32_t)(r ^ (4 * c + kg));
        x.woff = src.row(lane >> 1) * (uint32_t)(K >> 3) + 16u * (uint32_t)(lane & 1);
    };
    const auto advance = [&](Pos& x) {
        x.sb += KS;
        if (x.sb >= S) enter(x, x.unit + gridDim.x);
    };

    const uint32_t q_bytes = (uint32_t)grp.tokens * (uint32_t)K;
    const uint64_t qa = reinterpret_cast<uint64_t>(q), da_ = reinterpret_cast<uint64_t>(ds);
    const u32x4 qrs = {(uint32_t)qa, (uint32_t)(qa >> 32) & 0xFFFFu, q_bytes, (uint32_t)kBufferFlags};
    const u32x4 drs = {(uint32_t)da_, (uint32_t)(da_ >> 32) & 0xFFFFu, q_bytes / 8, (uint32_t)kBufferFlags};
    // Copy c of a step's weights: slot i = 64c + lane holds piece i % 9 of row
    // i / 9 (rows past the tile lie past the resource: zeros, not used).
    uint32_t at[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const int i = 64 * c + lane;
        at[c] = (uint32_t)(i / 9) * (uint32_t)(S * kBlockBytes) + 16u * (uint32_t)(i % 9);
    }
    // The copies of one step.  Those of four tokens past the item's last are
    // left out: what the area holds then is computed with and not stored.
    const auto issue = [&](const Pos& ps) {
        const u32x4 rs = {(uint32_t)__builtin_amdgcn_readfirstlane(ps.lo), (uint32_t)__builtin_amdgcn_readfirstlane(ps.hi),
                          (uint32_t)__builtin_amdgcn_readfirstlane(ps.bytes), (uint32_t)kBufferFlags};
        const uint32_t add = (uint32_t)(ps.sb * kBlockBytes), tok = (uint32_t)ps.sb * 256u;
        lds_copy16(rs, area, (int)(at[0] + add));
        lds_copy16(rs, area + 1024, (int)(at[1] + add));
        if (lane < 16) lds_copy16(rs, area + 2048, (int)(at[2] + add));
        if (lane < 32) lds_copy16(drs, area + kWords, (int)(ps.woff + (tok >> 3)));
        lds_copy16(qrs, area + kCodes, (int)(ps.off[0] + tok));
#pragma unroll
        for (int c = 1; c < 4; ++c)
            if (4 * c < ps.it.count) lds_copy16(qrs, area + kCodes + 1024 * c, (int)(ps.off[c] + tok));
    };

    // Where this lane reads: token r's bytes 32c + 8kg of the super-block are
    // piece 2c + (kg >> 1), in slot 16 r + (piece ^ r): bits 5-7 of the address
    // are c ^ (r >> 1).
    const uint32_t arow = area + kCodes + 256 * r + 32 * (r >> 1) + 16 * ((kg >> 1) ^ (r & 1)) + 8 * (kg & 1);
    const uint32_t wrow = area + kBlockBytes * r, drow = area + kWords + 128 * kg;

    v4f acc = v4f{0.0f, 0.0f, 0.0f, 0.0f}, acc2 = acc;
    Pos cur, nxt;
    enter(cur, blockIdx.x);
    if (!cur.it.valid) return;   // the same for every wave
    issue(cur);
    nxt = cur;
    advance(nxt);
    for (int done = 1;; ++done) {
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
        const v4u hdr = lds_read<v4u>(wrow);
        v2u qs[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) qs[p] = lds_read<v2u>(wrow + 16 + 32 * p + 8 * kg);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (nxt.it.valid) issue(nxt);   // the next step into it
        __builtin_amdgcn_sched_barrier(0);
        Weights x;
        x.decode(hdr, qs, kg);
        // out's part of the super-block
        v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f}, part = s;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            part = __builtin_amdgcn_mfma_f32_16x16x4f32(half_lo(own[j]) * (float)(int16_t)(uint16_t)(own[j] >> 16),
                                                        x.bneg[j], part, 0, 0, 0);
        const v4i magic = v4i{kMagicBits, kMagicBits, kMagicBits, kMagicBits};
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // four dots before their folds, which then find them done
            v4i D[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                D[c] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[4 * h + c], x.b[4 * h + c], magic, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float sc = x.scale(4 * h + c), ksc = -kMagic * sc;   // exact: 6 bits times 2
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t dd = da[i][2 * h + (c >> 1)];
                    s[i] = fmaf(half_lo((c & 1) ? dd >> 16 : dd), fmaf(sc, as_float(D[c][i]), ksc), s[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += fmaf(x.d, s[i], part[i]);
        if (BIG && done % kFlush == 0) {
            acc2 += acc;
            acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if (!nxt.it.valid || nxt.unit != cur.unit) {
            // The unit's end: the KS waves of a row tile are added.
            v4f sum = BIG ? acc2 + acc : acc;
            int tile = cur.unit % unit_tiles * per_unit + rt;
            bool mine = true;
            if (KS > 1) {
                red[wv][lane] = sum;
                lds_barrier();
                // wave v < per_unit stores row tile v of the unit
                mine = wv < per_unit;
                tile += wv - rt;
                if (mine) {
                    sum = red[wv * KS][lane];
#pragma unroll 1
                    for (int v = 1; v < KS; ++v) sum += red[wv * KS + v][lane];
                }
                lds_barrier();
            }
            const int row = 16 * tile + r;
            if (mine && row < M) {
                OutEpi o = out;
                o.advance(cur.it.start);
                if (o.bias) o.bias += (int64_t)cur.it.expert * M;
                // one store in a loop: four of them fill the registers of the
                // main loop with the epilogue's constants
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int tok = 4 * kg + i;
                    if (tok < cur.it.count)
                        o.put(tok, row, i == 0 ? sum[0] : i == 1 ? sum[1] : i == 2 ? sum[2] : sum[3]);
                }
            }
            acc = acc2 = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            done = 0;
        }
        if (!nxt.it.valid) break;
        cur = nxt;
        advance(nxt);
    }
}

}  // namespace

hipError_t launch_few_grouped(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, const Groups& g,
                              const OutEpi& out, hipStream_t stream) {
    const int64_t units = most_items(g.experts, g.slots, g.lo, g.hi, kTokens) * ((m + 15) / 16);
    const dim3 grid((unsigned)std::min<int64_t>(units, 256 * kHeld)), block(kNT);
    if ((k >> 8) > kFlush)
        hipLaunchKernelGGL((mmq_group_few_kernel<true>), grid, block, 0, stream, w, q, ds, m, k, out, g);
    else
        hipLaunchKernelGGL((mmq_group_few_kernel<false>), grid, block, 0, stream, w, q, ds, m, k, out, g);
    return hipGetLastError();
}

}  // namespace mmq
