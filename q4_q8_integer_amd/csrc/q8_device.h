// q8_device.h - the q8 quantization of one 32-value block by a DPP quad (4
// lanes, 8 values each), shared by the quantizers (quantize.hip) and the
// fused norm (norm_quantize.hip).
//
// Numerics: x/da is the IEEE fp32 division (hipcc's default correctly
// rounded divide; never built with fast-math), roundf rounds ties away from
// zero, and v_cvt_f16_f32 rounds to nearest even keeping subnormals.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmq {

// quad_perm controls: lane i of each quad reads lane i^1, or lane i^2.
constexpr int kQuadXor1 = 0xB1;  // [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;  // [2,3,0,1]

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(
                                                __builtin_bit_cast(int, v), kQuadXor1, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(
                                                __builtin_bit_cast(int, v), kQuadXor2, 0xF, 0xF, false)));
    return v;
}

__device__ __forceinline__ int quad_sum(int v) {
    v += __builtin_amdgcn_mov_dpp(v, kQuadXor1, 0xF, 0xF, false);
    v += __builtin_amdgcn_mov_dpp(v, kQuadXor2, 0xF, 0xF, false);
    return v;
}

// Codes and scale word of the quad's block, v = this lane's 8 values.  Every
// lane of the quad must call it; all four get the same word.
__device__ __forceinline__ uint32_t q8_block(const float (&v)[8], uint32_t (&packed)[2]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = quad_max(amax);

    packed[0] = packed[1] = 0u;
    int sum = 0;
    uint32_t word = 0u;
    if (amax > 0.0f) {
        const float da = amax / 127.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float r = roundf(v[i] / da);
            r = fminf(fmaxf(r, -127.0f), 127.0f);
            const int qi = (int)r;
            sum += qi;
            packed[i >> 2] |= (uint32_t)(qi & 0xFF) << (8 * (i & 3));
        }
        word = (uint32_t)__builtin_bit_cast(unsigned short, (_Float16)da);
    }
    sum = quad_sum(sum);
    return word | (uint32_t)(uint16_t)(int16_t)sum << 16;
}

// The codes of lane `part` of block c of token tok as its operand-tile slot
// (16 bytes at qt + 8 * q8_slot): slot ((cl * 2 + h) * 2 + g) * 128 + tt of
// block (tile, stage), part = 2 g + h, C = blocks per row.
__device__ __forceinline__ int64_t q8_slot(int tok, int c, int part, int C) {
    const int cl = c & 3, g = part >> 1, h = part & 1;
    const int64_t stage = c >> 2, stages = C >> 2;
    return (((int64_t)(tok >> 7) * stages + stage) * 16 + (cl * 2 + h) * 2 + g) * 128 + (tok & 127);
}

// Eight codes as binary16, in the operands' pair order.
__device__ __forceinline__ uint4 q8_slot_value(const uint32_t (&packed)[2]) {
    uint32_t hv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int qi = (int8_t)(uint8_t)(packed[i >> 2] >> (8 * (i & 3)));
        hv[i] = __builtin_bit_cast(unsigned short, (_Float16)(float)qi);   // exact
    }
    return make_uint4(hv[0] | (hv[2] << 16), hv[1] | (hv[3] << 16), hv[4] | (hv[6] << 16),
                      hv[5] | (hv[7] << 16));
}

}  // namespace mmq
