// mmq_q6k_few.hip - q6_K x q8 matmul for few tokens (up to 64), on int8 MFMA:
// the epilogue entry point between the dot4 kernel (8 tokens) and the
// binary16-MFMA kernel (128-token tiles).
//
// Method as in the other q6_K kernels: per 16-weight group an exact integer
// dot D = sum (q - 32) * q8, then out[t][o] = sum_g d*sc[g] * da[t, g/2] * D.
//
//   * A workgroup is 16 rows and 8 waves that take the super-blocks in turn,
//     so even 4096 rows give every CU a workgroup (the 128-row tiles of the
//     binary16 kernel gave 32), and the weights are read once.
//   * One v_mfma_i32_16x16x32_i8 is a chunk (k = 32: two scale groups) of 16
//     tokens (A) x 16 rows (B).  The two groups' dots come from two MFMAs on
//     the same tokens, the weights of the lanes of the other group set to 0
//     (lane l holds row l % 16 and k = 8 (l / 16) .. +7: lanes 0-31 are the
//     first group).  Half the matrix work is zeros; the matrix core is the
//     least busy unit all the same.
//   * The output column of a lane is its own weight row, so the scales are
//     per-lane integers: I = sc0*D0 + sc1*D1 is exact (two 24-bit
//     multiply-adds, |I| <= 2^24), then acc_b += da * float(I): 4 vector
//     operations per output and chunk.  Per super-block out += d * acc_b,
//     and every kFlush super-blocks of a wave that sum moves into a second
//     one, so that no float32 sum grows long.
//   * A step is one super-block and one tile of 16 tokens.  The wave copies
//     the next step's tokens (and the next super-block's 16 weight rows) into
//     LDS areas of its own with buffer loads that write LDS directly, while a
//     step computes; the weights are decoded once per super-block for all
//     token tiles.  The copies are inline asm, outside the compiler's wait
//     bookkeeping; one wait for everything opens each step.
//   * The 8 partial sums are added in LDS in a fixed order.
//
// 4096 x 11008 at 16 / 33 / 64 tokens 14.9 / 27 / 33 us (weights at the copy rate
// 7.2; the binary16 kernel 203).  Nothing is full: at 33 / 64 tokens the vector
// unit is busy 49 / 54% of the time (16 operations per chunk and 16 x 16 outputs,
// and 24 per chunk for the decode, shared by the token tiles), the matrix core
// 11 / 13%, and HBM gives 1.5 TB/s; the two waves of a SIMD do not cover each
// other's waits.
#include "f16_operand.h"
#include "internal.h"
#include "kquant_device.h"
#include "q6k_device.h"
#include "q6k_stage.h"

namespace mmq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kNT = 64 * kWaves;
constexpr int kFlush = 32;     // super-blocks of a wave between accumulator moves
constexpr int kWBytes = 4096;  // a step's 16 weight rows: 240 slots and padding, 4 copy instructions
constexpr int kTBytes = 4096;  // a 16-token tile of a super-block, 4 copy instructions

static_assert(16 * Seg<1>::kSlots <= 256 && Seg<1>::kLoads == 4, "a step's rows fill 4 copy instructions");

struct alignas(16) WaveLds {
    uint8_t w[2][kWBytes];
    uint8_t tok[2][kTBytes];
    float da[8][16];           // of the step's tile, [chunk][token]
};
template <int T>
union Lds {
    WaveLds wave[kWaves];
    v4f red[kWaves][T][64];
};

// Four copies of one KiB: 16 bytes per lane from byte off[c] of rs to
// 1024 c + 16 lane of dst.
__device__ __forceinline__ void copy4(u32x4 rs, const uint32_t (&off)[4], const uint8_t* dst) {
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)dst;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        lds_copy16(rs, __builtin_amdgcn_readfirstlane(base + 1024 * c), (int)off[c]);
}

__device__ __forceinline__ u32x4 resource(const void* p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, (uint32_t)kBufferFlags};
}

// The weights of one super-block as a lane's operands: row r's codes at k =
// 32c + 8kg .. +7 of each chunk c, once for each group of the chunk (zero in
// the lanes of the other), and its scales.
struct Weights {
    int64_t lo[8], hi[8];
    int sc0[8], sc1[8];
    float d;
};

__device__ __forceinline__ void decode(Weights& x, const uint8_t* row, int off, int kg) {
    const uint32_t sh = (uint32_t)off & 3u;
    const uint8_t* p = row + (off & ~3) + 8 * kg;
    const auto run8 = [&](int at, uint32_t (&v)[2]) {   // 8 bytes at field offset `at`
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + at);
        const uint32_t a = q[0], b = q[1], c = q[2];
        v[0] = __builtin_amdgcn_alignbyte(b, a, sh);
        v[1] = __builtin_amdgcn_alignbyte(c, b, sh);
    };
    const uint32_t mlo = kg < 2 ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t l0[2], l1[2], hb[2];
        run8(64 * h, l0);
        run8(64 * h + 32, l1);
        run8(128 + 32 * h, hb);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                c[i] = q6k::signed_codes(((g & 1) ? l1[i] : l0[i]) >> (4 * (g >> 1)), hb[i] >> (2 * g));
            x.lo[4 * h + g] = (int64_t)(((uint64_t)(c[1] & mlo) << 32) | (c[0] & mlo));
            x.hi[4 * h + g] = (int64_t)(((uint64_t)(c[1] & ~mlo) << 32) | (c[0] & ~mlo));
        }
    }
    uint32_t sc[5];
    lds_run(row, off + 192, sc);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t word = q6k::run_word(sc, c >> 1, sh);
        x.sc0[c] = (int)(int8_t)(word >> (16 * (c & 1)));
        x.sc1[c] = (int)(int8_t)(word >> (16 * (c & 1) + 8));
    }
    x.d = half_lo(*reinterpret_cast<const uint32_t*>(row + ((off + 208) & ~3)) >> (8 * sh));
}

// N <= 16 T.
template <int T>
__global__ __launch_bounds__(kNT) void mmq_q6k_few_kernel(const uint8_t* __restrict__ w, const int8_t* __restrict__ q,
                                                          const uint32_t* __restrict__ ds, int M, int N, int K,
                                                          OutEpi out) {
    __shared__ Lds<T> L;
    const int row0 = blockIdx.x * 16;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // wave-uniform
    const int r = lane & 15, kg = lane >> 4;
    const int S = K >> 8, C = K >> 5;
    const int tiles = (N + 15) >> 4;
    WaveLds& my = L.wave[wv];

    Tile tl;
    tl.rows = min(16, M - row0);
    tl.end = tl.rows * S * kQ6kBlockBytes;
    tl.base = w + (int64_t)row0 * S * kQ6kBlockBytes;
    const u32x4 wrs = resource(tl.base, (uint32_t)tl.end & ~15u);
    const u32x4 qrs = resource(q, (uint32_t)N * (uint32_t)K);

    // Copy sources.  Weights: slot i = 64c + lane holds piece i % kSlots of
    // row i / kSlots (the padding slot and those past the 16 rows repeat a
    // piece), from the 16-byte boundary below the row's block.  Tokens: slot
    // 16t + s of a tile holds piece s ^ t of token t.
    int wrow[4], wpiece[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int i = 64 * c + lane;
        wrow[c] = min(i / Seg<1>::kSlots, 15) * S;
        wpiece[c] = 16 * min(i % Seg<1>::kSlots, Seg<1>::kChunks - 1);
    }
    const auto issue_weights = [&](int buf, int sb) {
        uint32_t off[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) off[c] = (((uint32_t)(wrow[c] + sb) * kQ6kBlockBytes) & ~15u) + wpiece[c];
        copy4(wrs, off, my.w[buf]);
    };
    uint32_t word[2];   // the next step's scale words: token r of its tile, chunks kg and kg + 4
    const auto issue_tokens = [&](int buf, int tt, int sb) {
        uint32_t off[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int tk = 4 * c + kg;   // tokens past N - 1 repeat it
            off[c] = (uint32_t)min(16 * tt + tk, N - 1) * (uint32_t)K + (uint32_t)sb * 256u + 16u * (uint32_t)(r ^ tk);
        }
        const uint32_t* dp = ds + (int64_t)min(16 * tt + r, N - 1) * C + sb * 8 + kg;
#pragma unroll
        for (int h = 0; h < 2; ++h) word[h] = dp[4 * h];
        copy4(qrs, off, my.tok[buf]);
    };

    v4f acc[T], acc2[T];
#pragma unroll
    for (int tt = 0; tt < T; ++tt) acc[tt] = acc2[tt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    int wb = 0, tb = 0;
    if (wv < S) {
        issue_tokens(0, 0, wv);
        issue_weights(0, wv);
    }
    Weights x;
    for (int sb = wv, done = 1; sb < S; sb += kWaves, ++done) {
        const int next = sb + kWaves;
        for (int tt = 0; tt < tiles; ++tt) {
            __builtin_amdgcn_s_waitcnt(kWaitVmcnt(0));
            asm volatile("" ::"v"(word[0]), "v"(word[1]));   // the compiler's own wait for them, if any, is here
            __builtin_amdgcn_sched_barrier(0);
            // da of this step's tile; LDS accesses of one wave complete in order
#pragma unroll
            for (int h = 0; h < 2; ++h) my.da[kg + 4 * h][r] = half_lo(word[h]);
            if (tt + 1 < tiles)
                issue_tokens(tb ^ 1, tt + 1, sb);
            else if (next < S)
                issue_tokens(tb ^ 1, 0, next);
            if (tt == 0) {
                if (next < S) issue_weights(wb ^ 1, next);
                stage_patch<1>(tl, S, sb, lane, my.w[wb]);
                decode(x, my.w[wb] + r * Seg<1>::kBytes,
                       (int)((((uint32_t)(row0 + r) * (uint32_t)S + sb) * kQ6kBlockBytes) & 15u), kg);
            }
            __builtin_amdgcn_sched_barrier(0);
            const uint8_t* arow = my.tok[tb] + 256 * r + 8 * (kg & 1);
            v4f b = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                // token r's bytes 32c + 8kg: piece 2c + (kg >> 1), swizzled
                const int64_t a = *reinterpret_cast<const int64_t*>(arow + 16 * ((2 * c + (kg >> 1)) ^ r));
                const v4f da = *reinterpret_cast<const v4f*>(&my.da[c][4 * kg]);
                const v4i zero = v4i{0, 0, 0, 0};
                const v4i d0 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, x.lo[c], zero, 0, 0, 0);
                const v4i d1 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, x.hi[c], zero, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = __mul24(x.sc0[c], d0[i]) + __mul24(x.sc1[c], d1[i]);
                    b[i] = fmaf(da[i], (float)s, b[i]);
                }
            }
            // a loop over the tiles with a branch per accumulator: unrolled, the
            // steps' operands take all 256 registers and spill
#pragma unroll
            for (int j = 0; j < T; ++j)
                if (tt == j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(x.d, b[i], acc[j][i]);
            tb ^= 1;
        }
        wb ^= 1;
        if (done % kFlush == 0)
#pragma unroll
            for (int tt = 0; tt < T; ++tt) {
                acc2[tt] += acc[tt];
                acc[tt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            }
    }

    __syncthreads();  // every wave is done with the areas the sums reuse
#pragma unroll
    for (int tt = 0; tt < T; ++tt) L.red[wv][tt][lane] = acc2[tt] + acc[tt];
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * tiles; e += kNT) {
        const int l = e & 63, tt = e >> 6;
        v4f sum = L.red[0][tt][l];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) sum += L.red[v][tt][l];
        const int row = row0 + (l & 15);
        if (row >= M) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 16 * tt + 4 * (l >> 4) + i;
            if (tok < N) out.put(tok, row, sum[i]);
        }
    }
}

template <int T>
hipError_t launch_t(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, int n, const OutEpi& out,
                    hipStream_t stream) {
    hipLaunchKernelGGL((mmq_q6k_few_kernel<T>), dim3((unsigned)((m + 15) / 16)), dim3(kNT), 0, stream,
                       w, q, ds, m, n, k, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_q6k_few(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, int n, const OutEpi& out,
                          hipStream_t stream) {
    return n <= 16 ? launch_t<1>(w, m, k, q, ds, n, out, stream) : launch_t<4>(w, m, k, q, ds, n, out, stream);
}

}  // namespace mmq
