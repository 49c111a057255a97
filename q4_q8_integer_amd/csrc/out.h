// out.h - where the float32 results of a fold kernel go: the kernels take one
// of three output types as a template parameter and hand it each result with
// its token and row.
//
//   OutF32  float32 [n][m]
//   OutF16  binary16 [n][m], rounded to nearest-even from the float32 value
//   OutEpi  act(v + bias[row]) + residual[token][row], float32 or binary16,
//           rows of the output and the residual at strides of their own
//
// The epilogue is float32 throughout and rounds once, at a binary16 store.
// Its choices (activation, types, which operands there are) are uniform
// run-time values: per output they cost a few scalar branches in kernels
// that spend k / 32 vector operations on it, where a template per choice
// would multiply every kernel by 40.  Measured: 4096 x 4096, 2630 tokens, fold
// 161-177 us, with bias and float32 residual 180 (the residual's 43 MB are 8 us
// at the copy rate), with bias and SiLU 177 (173 with the hardware's
// exponential alone, 184 with a full division too), GELU 182 (the consumer
// waves' last step); 28672 x 8192, 7 tokens, 29-31 us with any of them, as the
// fold.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmq {

typedef float out4f __attribute__((ext_vector_type(4)));
typedef _Float16 out4h __attribute__((ext_vector_type(4)));

struct OutF32 {
    float* p;
    int64_t stride;   // m
    __device__ __forceinline__ bool vec() const { return (stride & 3) == 0; }
    __device__ __forceinline__ void put(int64_t tok, int row, float v) const { p[tok * stride + row] = v; }
    // Rows row .. row + 3 (row % 4 == 0, vec()).
    __device__ __forceinline__ void put4(int64_t tok, int row, float a, float b, float c, float d) const {
        *reinterpret_cast<float4*>(p + tok * stride + row) = make_float4(a, b, c, d);
    }
};

struct OutF16 {
    _Float16* p;
    int64_t stride;   // m
    __device__ __forceinline__ bool vec() const { return (stride & 3) == 0; }
    __device__ __forceinline__ void put(int64_t tok, int row, float v) const { p[tok * stride + row] = (_Float16)v; }
    __device__ __forceinline__ void put4(int64_t tok, int row, float a, float b, float c, float d) const {
        *reinterpret_cast<out4h*>(p + tok * stride + row) =
            out4h{(_Float16)a, (_Float16)b, (_Float16)c, (_Float16)d};
    }
};

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// v * sigmoid(x) = v / (1 + exp(-x)), the exponential and the hardware's
// reciprocal to an ulp each.  (The hardware's exponential on x * log2(e)
// rounded once takes 2 to 3% off a prefill call, but is off by up to |x| half
// steps in the lower tail.)  Below x = -87 the reciprocal leaves float32's normal
// range and the result may be -0 for an exact value below 1.1e-36.
__device__ __forceinline__ float times_sigmoid(float v, float x) {
    return v * __builtin_amdgcn_rcpf(1.0f + expf(-x));
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case kActRelu: return v < 0.0f ? 0.0f : v;   // NaN stays
        case kActSilu: return times_sigmoid(v, v);
        // v * Phi(v); erfc keeps its relative accuracy where 1 + erf cancels
        case kActGelu: return 0.5f * v * erfcf(-0.70710678118654752f * v);
        // 0.5 v (1 + tanh u) = v * sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
        case kActGeluTanh: return times_sigmoid(v, 1.59576912160573076f * fmaf(0.044715f * v * v, v, v));
        default: return v;
    }
}

// bias and residual may be null.  The residual may be the output itself
// (same type and stride): a value is read by the thread that writes it.
struct OutEpi {
    void* p;
    const float* bias;
    const void* res;
    int64_t stride, res_stride;
    int act;
    int half, res_half;   // binary16 output, binary16 residual
    int vec4;             // every row of 4-value groups is aligned for put4

    __device__ __forceinline__ bool vec() const { return vec4 != 0; }
    __device__ __forceinline__ void put(int64_t tok, int row, float v) const {
        if (bias) v += bias[row];
        v = activate(v, act);
        if (res) {
            const int64_t i = tok * res_stride + row;
            v += res_half ? (float)static_cast<const _Float16*>(res)[i] : static_cast<const float*>(res)[i];
        }
        if (half)
            static_cast<_Float16*>(p)[tok * stride + row] = (_Float16)v;
        else
            static_cast<float*>(p)[tok * stride + row] = v;
    }
    __device__ __forceinline__ void put4(int64_t tok, int row, float a, float b, float c, float d) const {
        out4f v = out4f{a, b, c, d};
        if (bias) v += *reinterpret_cast<const out4f*>(bias + row);
        if (act != kActNone)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = activate(v[i], act);
        if (res) {
            const int64_t i = tok * res_stride + row;
            if (res_half) {
                const out4h r = *reinterpret_cast<const out4h*>(static_cast<const _Float16*>(res) + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += (float)r[j];
            } else {
                v += *reinterpret_cast<const out4f*>(static_cast<const float*>(res) + i);
            }
        }
        if (half)
            *reinterpret_cast<out4h*>(static_cast<_Float16*>(p) + tok * stride + row) =
                out4h{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        else
            *reinterpret_cast<out4f*>(static_cast<float*>(p) + tok * stride + row) = v;
    }
    // The output from token `toks` on.
    __host__ __device__ __forceinline__ void advance(int64_t toks) {
        p = static_cast<char*>(p) + toks * stride * (half ? 2 : 4);
        if (res) res = static_cast<const char*>(res) + toks * res_stride * (res_half ? 2 : 4);
    }
};

// The output of a launch: which of the three, and its values (for OutF32 and
// OutF16 only p and stride).
enum OutKind { kOutF32, kOutF16, kOutEpi };
struct Out {
    OutKind kind;
    OutEpi epi;
    static Out plain(void* p, int64_t m, bool half) {
        Out o{};
        o.kind = half ? kOutF16 : kOutF32;
        o.epi.p = p;
        o.epi.stride = m;
        o.epi.half = half;
        return o;
    }
};

// f(output) with the launch's output type.
template <class F>
hipError_t with_out(const Out& o, F f) {
    switch (o.kind) {
        case kOutF32: return f(OutF32{static_cast<float*>(o.epi.p), o.epi.stride});
        case kOutF16: return f(OutF16{static_cast<_Float16*>(o.epi.p), o.epi.stride});
        default: return f(o.epi);
    }
}

// The same for the entry points that have no plain binary16 form.
template <class F>
hipError_t with_out_f32(const Out& o, F f) {
    return o.kind == kOutEpi ? f(o.epi) : f(OutF32{static_cast<float*>(o.epi.p), o.epi.stride});
}

}  // namespace mmq
