// norm_quantize.hip - the norms before and after a transformer block, with
// the block's gate and the residual scale, fused with the q8 quantizer that
// feeds the next projections.
//
//   z = y                                        without a post-norm
//   z = y * yw / sqrt(mean(y^2) + eps)           with one
//   r = float32(a * x + gate * z)                the new residual stream
//   h = float32(r * w / sqrt(mean(r^2) + eps))
//   q, ds = q8(h)
//
// Everything between the roundings is float64.  The sums therefore do not
// depend on their order in any bit that reaches h (but for about one value in
// 10^8), so a code next to a rounding border is the definition's, whatever
// the split; the float64 rate covers it: per value about 12 float64
// operations, against 13 to 26 bytes of HBM traffic that take longer.
//
// A workgroup owns a row.  Lane t of it holds the 8-value pieces t, t + T, ..
// of the row in registers (T threads, V pieces each), so x and y are read
// once and r, h, q are written once; a DPP quad holds a whole 32-value block,
// as the quantizer wants it.  Rows beyond 32768 values do not fit the
// registers: there the workgroup goes over the row in pieces and reads r
// (or x) again, from cache, for the second norm.
//
// Measured: 8192 rows of 4096, y in binary16 with its norm, a gate per channel
// and h out, 99 us (470 MB: 91 us at the copy rate; HBM bound); y in float32, no
// operands, with codes as rows 83 us (440 MB: 86), as operand tiles 108 (474 MB:
// 92).  One row of 4096 with codes 4 us in a graph, a launch and two reductions
// across 8 waves; 22 us a call from Python, three allocations among them.
//
// With operand tiles a lane's codes are one 16-byte slot, and the slots of
// consecutive tokens are adjacent: eight consecutive rows go to the same XCD
// (workgroups are dealt to the 8 XCDs in turn), so that its L2 joins their
// stores into whole lines.
#include "internal.h"
#include "q8_device.h"

namespace mmq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

enum { kNoY = 0, kY32 = 1, kY16 = 2 };
enum { kNoCodes = 0, kRows = 1, kTiles = 2 };

constexpr uint32_t kNanScale = 0x7E00u;   // a scale word: binary16 NaN, sum of codes 0

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const v4f a = *reinterpret_cast<const v4f*>(p), b = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
}

template <int YT>
__device__ __forceinline__ void load_y(const NormArgs& a, int64_t row, int col, float (&v)[8]) {
    if (YT == kY16) {
        const v8h y = *reinterpret_cast<const v8h*>(static_cast<const _Float16*>(a.y) + row * a.y_stride + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)y[i];
    } else {
        load8(static_cast<const float*>(a.y) + row * a.y_stride + col, v);
    }
}

// The sum of v over the workgroup, in every lane: waves in index order.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = red[0];
    for (int i = 1; i < waves; ++i) s += red[i];
    return s;
}

__device__ __forceinline__ double sum_sq(const float (&v)[8], double s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma((double)v[i], (double)v[i], s);
    return s;
}

// r of one piece, from y's values (yinv = 1 / its root mean square, or
// unused); written to a.r.
template <int YT>
__device__ __forceinline__ void residual(const NormArgs& a, int64_t row, int col, const float (&y)[8], double yinv,
                                         float (&r)[8]) {
    load8(a.x + row * a.x_stride + col, r);
    if (YT == kNoY) return;
    float yw[8], g[8];
    if (a.y_weight) load8(a.y_weight + col, yw);
    if (a.gate) load8(a.gate + row * a.gate_stride + col, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        double z = (double)y[i];
        if (a.y_weight) z = z * (double)yw[i] * yinv;
        if (a.gate) z *= (double)g[i];
        r[i] = (float)fma((double)a.x_scale, (double)r[i], z);
    }
    store8(a.r + row * a.r_stride + col, r);
}

// h of one piece, and what is written of it.
template <int OUT>
__device__ __forceinline__ void emit(const NormArgs& a, int row, int col, int k, const float (&r)[8], double inv,
                                     int8_t* q, uint16_t* qt, uint32_t* ds) {
    float w[8], h[8];
    load8(a.weight + col, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (float)((double)r[i] * (double)w[i] * inv);
    if (a.h) store8(a.h + (int64_t)row * k + col, h);
    if (OUT == kNoCodes) return;
    uint32_t packed[2];
    uint32_t word = q8_block(h, packed);
    // The quantizer's maximum passes over a NaN.  Here one NaN or infinity in a
    // token makes all its h NaN or 0, which would be a scale of 0 and a product
    // of 0, so a block with a NaN gets a NaN scale.
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; i += 2) nan |= __builtin_isunordered(h[i], h[i + 1]);
    if ((__ballot(nan) >> (threadIdx.x & 60)) & 15) word = kNanScale;   // of the quad's 32 values
    const int c = col >> 5, part = (col >> 3) & 3, C = k >> 5;
    if (OUT == kTiles)
        *reinterpret_cast<uint4*>(qt + q8_slot(row, c, part, C) * 8) = q8_slot_value(packed);
    else
        *reinterpret_cast<uint2*>(q + (int64_t)row * k + col) = make_uint2(packed[0], packed[1]);
    if (part == 0) ds[(int64_t)row * C + c] = word;
}

// V: pieces per lane held in registers; 0 = any row length, in passes.
template <int YT, int OUT, int V>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a, int n, int k, int8_t* q, uint16_t* qt, uint32_t* ds) {
    __shared__ double red[2][16];
    int row = blockIdx.x;
    if (OUT == kTiles) {   // grid: whole tiles of 128 tokens; 64 workgroups cover 64 rows, 8 per XCD
        row = (row & ~63) | ((row & 7) << 3) | ((row >> 3) & 7);
        if (row >= n) {
            for (int col = threadIdx.x * 8; col < k; col += blockDim.x * 8)
                *reinterpret_cast<uint4*>(qt + q8_slot(row, col >> 5, (col >> 3) & 3, k >> 5) * 8) = make_uint4(0, 0, 0, 0);
            return;
        }
    }
    const int step = blockDim.x * 8, col0 = threadIdx.x * 8;
    const double rk = 1.0 / (double)k;

    if constexpr (V > 0) {
        float y[V][8], r[V][8];
        double yinv = 0.0;
        if (YT != kNoY) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (col0 + i * step < k) load_y<YT>(a, row, col0 + i * step, y[i]);
            if (a.y_weight) {
                double s = 0.0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (col0 + i * step < k) s = sum_sq(y[i], s);
                yinv = 1.0 / sqrt(block_sum(s, red[0]) * rk + (double)a.eps);
            }
        }
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col0 + i * step < k) {
                residual<YT>(a, row, col0 + i * step, y[i], yinv, r[i]);
                s = sum_sq(r[i], s);
            }
        const double inv = 1.0 / sqrt(block_sum(s, red[1]) * rk + (double)a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col0 + i * step < k) emit<OUT>(a, row, col0 + i * step, k, r[i], inv, q, qt, ds);
    } else {
        double yinv = 0.0, s = 0.0;
        float y[8], r[8];
        if (YT != kNoY && a.y_weight) {
            for (int col = col0; col < k; col += step) {
                load_y<YT>(a, row, col, y);
                s = sum_sq(y, s);
            }
            yinv = 1.0 / sqrt(block_sum(s, red[0]) * rk + (double)a.eps);
            s = 0.0;
        }
        for (int col = col0; col < k; col += step) {
            if (YT != kNoY) load_y<YT>(a, row, col, y);
            residual<YT>(a, row, col, y, yinv, r);
            s = sum_sq(r, s);
        }
        const double inv = 1.0 / sqrt(block_sum(s, red[1]) * rk + (double)a.eps);
        for (int col = col0; col < k; col += step) {   // each lane reads what it wrote itself
            load8(YT != kNoY ? a.r + row * a.r_stride + col : a.x + row * a.x_stride + col, r);
            emit<OUT>(a, row, col, k, r, inv, q, qt, ds);
        }
    }
}

template <int YT, int OUT>
hipError_t launch(const NormArgs& a, int n, int k, int8_t* q, uint16_t* qt, uint32_t* ds, hipStream_t stream) {
    const int pieces = k / 8;
    const int v = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : pieces <= 4096 ? 4 : 0;
    const int lanes = v ? (pieces + v - 1) / v : 1024;
    const dim3 block((lanes + 63) / 64 * 64);
    const dim3 grid(OUT == kTiles ? (unsigned)((n + 127) / 128 * 128) : (unsigned)n);
    switch (v) {
        case 1: hipLaunchKernelGGL((norm_kernel<YT, OUT, 1>), grid, block, 0, stream, a, n, k, q, qt, ds); break;
        case 2: hipLaunchKernelGGL((norm_kernel<YT, OUT, 2>), grid, block, 0, stream, a, n, k, q, qt, ds); break;
        case 4: hipLaunchKernelGGL((norm_kernel<YT, OUT, 4>), grid, block, 0, stream, a, n, k, q, qt, ds); break;
        default: hipLaunchKernelGGL((norm_kernel<YT, OUT, 0>), grid, block, 0, stream, a, n, k, q, qt, ds); break;
    }
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_y(const NormArgs& a, int n, int k, int8_t* q, uint16_t* qt, uint32_t* ds, hipStream_t stream) {
    if (!a.y) return launch<kNoY, OUT>(a, n, k, q, qt, ds, stream);
    return a.y_f16 ? launch<kY16, OUT>(a, n, k, q, qt, ds, stream) : launch<kY32, OUT>(a, n, k, q, qt, ds, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int n, int k, int8_t* q, uint16_t* qt, uint32_t* ds, hipStream_t stream) {
    return qt  ? launch_y<kTiles>(a, n, k, q, qt, ds, stream)
           : q ? launch_y<kRows>(a, n, k, q, qt, ds, stream)
               : launch_y<kNoCodes>(a, n, k, q, qt, ds, stream);
}

}  // namespace mmq
