// internal.h - launchers shared between the kernel translation units and the
// C-ABI entry points.  Arguments are validated by the caller (mmq_api.hip);
// each launcher only enqueues work and returns the hipError_t of the launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "out.h"

namespace mmq {

// Bytes of one q4_K super-block (256 weights).
constexpr int kBlockBytes = 144;
// Bytes of one record (16 rows x one super-block) of the repacked q4_K layout.
constexpr int kRepackRecordBytes = 2368;

hipError_t launch_q8_quantize(const float* x, int64_t nblocks, int8_t* q, uint32_t* ds,
                              hipStream_t stream);

// q8 quantize with the codes written as binary16 operand tiles (token tiles
// of 128, k stages of 128, 32 KiB per tile and stage; k % 256 == 0).
hipError_t launch_q8_quantize_tiled(const float* x, int n, int k, uint16_t* qt, uint32_t* ds,
                                    hipStream_t stream);

// The same, with the codes written as operand tiles.
hipError_t launch_q8_quantize_silu_mul_tiled(const float* g, const float* u, int n, int k, uint16_t* qt,
                                             uint32_t* ds, hipStream_t stream);

// q8 quantize of h = float32(g*u / (1 + exp(-g))) (float64 evaluation).
hipError_t launch_q8_quantize_silu_mul(const float* g, const float* u, int64_t nblocks, int8_t* q,
                                       uint32_t* ds, hipStream_t stream);

// The fused norm (norm_quantize.hip): the pointers and strides of
// include/mmq.h's q8_norm, checked.
struct NormArgs {
    const float* x;
    int64_t x_stride;
    float x_scale;            // residual scale
    const void* y;            // null: no block output, r = x
    int64_t y_stride;
    int y_f16;
    const float* y_weight;    // null: no norm of y
    const float* gate;        // null: none
    int64_t gate_stride;      // 0: one gate row for all tokens
    const float* weight;
    float eps;
    float* r;
    int64_t r_stride;
    float* h;                 // null: h is not written
};
// Codes to q (rows), to qt (operand tiles, k % 256 == 0), or nowhere.
hipError_t launch_norm(const NormArgs& a, int n, int k, int8_t* q, uint16_t* qt, uint32_t* ds, hipStream_t stream);

// Router and combination of the matmuls grouped by expert (moe.hip).
constexpr int kRouteMaxExperts = 1024, kRouteMaxTop = 64;
constexpr int kTopkWaves = 4;   // tokens per workgroup of the choosing kernel, a wave each
hipError_t launch_route(const float* logits, int64_t stride, int n, int experts, int top, bool normalize, float scale,
                        int32_t* ids, float* weights, int32_t* slot, int32_t* rows, int32_t* offsets,
                        hipStream_t stream);
// Workgroups of 256 threads on a token's m columns: 16 bytes of y per thread
// where m is a multiple of that many values, else one value.
inline int64_t combine_cols(bool y_f16, int64_t m) {
    const int64_t vec = y_f16 ? 8 : 4, per = 256 * (m % vec == 0 ? vec : 1);
    return (m + per - 1) / per;
}
hipError_t launch_combine(const void* y, bool y_f16, int64_t slots, int m, const int32_t* slot, const float* weights,
                          int n, int top, const float* residual, float* out, hipStream_t stream);

// Exact int32 block dots, dots[t][o][c].
hipError_t launch_mmq_dots(const uint8_t* w, int m, int k, const int8_t* q, int n,
                           int32_t* dots, hipStream_t stream);

// The low 16 bits of h as a binary16 value, widened to float32 (exact).
__device__ __forceinline__ float half_lo(uint32_t h) {
    return (float)__builtin_bit_cast(_Float16, (unsigned short)(h & 0xFFFFu));
}

// Two-term fold, out[t][o] (float32 or binary16), int8 MFMA + three-operation epilogue.
hipError_t launch_mmq_fp32(const uint8_t* w, int m, int k, const int8_t* q,
                           const uint32_t* ds, int n, const Out& out, hipStream_t stream);

// Two-term fold, out[t][o], binary16 MFMA on exact sc*q4 and q8 operands +
// float32 MFMA for the min term (above 64 tokens).
hipError_t launch_mmq_fp32_f16(const uint8_t* w, int m, int k, const int8_t* q,
                               const uint32_t* ds, int n, const Out& out,
                               hipStream_t stream);

// The binary16-MFMA kernel on q4k_repack records (same arithmetic and order
// as launch_mmq_fp32_f16, so the same float32 result bit for bit).
hipError_t launch_mmq_fp32_f16_repacked(const uint8_t* wr, int m, int k, const int8_t* q,
                                        const uint32_t* ds, int n, const Out& out, hipStream_t stream);

// The binary16-MFMA kernel with the activations as q8 operand tiles (from
// launch_q8_quantize_tiled), on q4_K rows or q4k_repack records; the same
// float32 result bit for bit as the int8-activation kernel.
hipError_t launch_mmq_fp32_f16_tiles(const uint8_t* w, bool repacked, int m, int k, const uint16_t* qt,
                                     const uint32_t* ds, int n, const Out& out, hipStream_t stream);

// Two-term fold, out[t][o], for n <= 64 tokens: weight-streaming int8-MFMA
// kernel (8 waves per 16 rows, each over a slice of k).
hipError_t launch_mmq_fp32_small(const uint8_t* w, int m, int k, const int8_t* q,
                                 const uint32_t* ds, int n, const Out& out,
                                 hipStream_t stream);

// Two-term fold, out[t][o], for 1 <= n <= kGemvMaxN tokens: 4-way int8 dot
// products on the vector ALU, no token padding.
hipError_t launch_mmq_fp32_gemv(const uint8_t* w, int m, int k, const int8_t* q,
                                const uint32_t* ds, int n, const Out& out,
                                hipStream_t stream);
constexpr int kGemvMaxN = 8;

// Load-time repack of q4_K into 16-row records (repack.hip), and the dot4
// kernel on that layout (1 <= n <= kGemvMaxN; w is the repacked buffer).
hipError_t launch_q4k_repack(const uint8_t* w, int m, int k, uint8_t* wr, hipStream_t stream);
hipError_t launch_mmq_fp32_gemv_repacked(const uint8_t* wr, int m, int k, const int8_t* q,
                                         const uint32_t* ds, int n, const Out& out,
                                         hipStream_t stream);

// Largest token count the few-token kernel takes.
constexpr int kSmallMaxN = 64;

// Two-term fold, out[t][o], for 1 <= n <= kNarrowMaxN tokens: 4x4x4 int8
// MFMA on weights and tokens staged through LDS, one (row, super-block,
// chunk half) per lane (mmq_narrow.hip).
hipError_t launch_mmq_fp32_narrow(const uint8_t* w, int m, int k, const int8_t* q,
                                  const uint32_t* ds, int n, const Out& out,
                                  hipStream_t stream);
constexpr int kNarrowMaxN = 16;

// The narrow kernel's layout for an m x k weight: 32-row tiles where they
// fill the 256 CUs (at least 256 tiles) with at least 8 super-blocks per
// wave, run by 4 waves per workgroup from 512 tiles on (two workgroups per
// CU) and by 8 below; the return value is that wave count, or 0 for 16-row
// tiles.
inline int narrow_waves32(int64_t m, int64_t k) {
    const int64_t tiles = (m + 31) / 32, w = tiles >= 512 ? 4 : 8;
    return tiles >= 256 && (k >> 8) >= 8 * w ? (int)w : 0;
}

// q6_K weights (210-byte super-blocks, one int8 scale per 16 weights).
// Exact int32 group dots, dots[t][o][g] (g = k/16 groups).
hipError_t launch_q6k_dots(const uint8_t* w, int m, int k, const int8_t* q, int n,
                           int32_t* dots, hipStream_t stream);

// out[t][o] (float32 or binary16) for any n: int8 MFMA per scale group.
hipError_t launch_q6k_i8(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds,
                         int n, const Out& out, hipStream_t stream);

// out[t][o] for any n: binary16 MFMA on the split exact operands sc*nibble/64
// and sc*(hi2 - 2)/4 (one FMA per output and chunk).
hipError_t launch_q6k_f16(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, int n,
                          const Out& out, hipStream_t stream);

// launch_q6k_f16 with the activations as q8 operand tiles (float32 output).
hipError_t launch_q6k_f16_tiles(const uint8_t* w, int m, int k, const uint16_t* qt, const uint32_t* ds,
                                int n, const Out& out, hipStream_t stream);

// out[t][o] for 1 <= n <= kQ6kGemvMaxN: 4-way int8 dots on the vector ALU.
hipError_t launch_q6k_gemv(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds,
                           int n, const Out& out, hipStream_t stream);
constexpr int kQ6kGemvMaxN = 8;

// out[t][o] with an epilogue for n <= kQ6kFewMaxN: int8 MFMA on 16-row tiles,
// the waves of a workgroup split over k (mmq_q6k_few.hip); and on the
// streaming kernel (mmq_group_few.hip).  Where every CU has one tile at most
// the first is faster (4096 x 11008, 16 / 33 / 64 tokens: 14.6 / 26.6 / 32.1
// us against 15.0 / 29.0 / 36.2), above that the second, which has 16 waves per
// CU (8192 x 4096: 13.5 / 22.2 / 26.6 against 11.2 / 21.8 / 27.8; 14336 x 4096:
// 24.0 / 39.3 / 47.8 against 15.7 / 34.7 / 43.8).
hipError_t launch_q6k_few(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, int n,
                          const OutEpi& out, hipStream_t stream);
hipError_t launch_q6k_stream(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, int n,
                             const OutEpi& out, hipStream_t stream);
constexpr int kQ6kFewMaxN = 64, kQ6kFewMaxM = 4096;

// The matmuls grouped by expert (group.h), over the items of the experts with
// g.lo .. g.hi slots.  tokens_per_item: 64 or 128, the slots of one item.
struct Groups;
hipError_t launch_f16_grouped(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds, const Groups& g,
                              const OutEpi& out, int tokens_per_item, hipStream_t stream);
// Slots of an expert up to which the streaming kernel (mmq_group_few.hip) takes
// it, in its form with one tile of 16 tokens and in the other one.  Against the
// binary16 kernel, 64 experts of 1536 x 4096 in q4_K: 32 slots 105 us (117),
// 33 slots 129 (116); of 4096 x 1536 in q6_K: 64 slots 261 us (312), 65 slots
// 490 (315).
constexpr int kGroupFewMaxTile = 16, kGroupFewMaxQ4k = 32, kGroupFewMaxQ6k = 64;
hipError_t launch_few_grouped(bool q6k, const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds,
                              const Groups& g, const OutEpi& out, hipStream_t stream);
hipError_t launch_q6k_f16_grouped(const uint8_t* w, int m, int k, const int8_t* q, const uint32_t* ds,
                                  const Groups& g, const OutEpi& out, hipStream_t stream);

}  // namespace mmq
