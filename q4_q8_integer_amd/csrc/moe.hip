// moe.hip - the router in front of the matmuls grouped by expert, and the
// combination of the experts' outputs behind them.
//
// Routing, two launches:
//   * route_topk_kernel, a wave per token: the scores sit in registers
//     (expert 64 j + lane), and each choice is a maximum over the wave and a
//     ballot for the lowest index that has it.  The softmax needs no second
//     pass: the first choice is its maximum.
//   * route_sort_kernel, a workgroup per expert: a stable counting sort that
//     needs neither atomics nor a workspace.  Expert e's workgroup reads all
//     n * top ids (they come from L2), counts those below e (its first slot)
//     and, per thread over a contiguous run, those equal to e (a prefix sum
//     gives each thread its first slot), then goes over the run again and
//     writes slots and rows.  Slots of an expert are in token order.
//
// Combining: out[t] = residual[t] + sum_j weights[t][j] * y[slot[t][j]], a
// thread per 16 bytes of y columns; slots and weights of a token are the
// same for a whole workgroup.  Bound by HBM.
#include <cfloat>

#include "internal.h"

namespace mmq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kTopkWaves = 4;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// J: experts per lane.  A score of NaN counts as -inf and one of +inf as the
// largest float32; an expert at -inf is not chosen.
template <int J>
__global__ __launch_bounds__(64 * kTopkWaves) void route_topk_kernel(const float* __restrict__ logits, int64_t stride,
                                                                     int n, int experts, int top, int normalize,
                                                                     float scale, int32_t* __restrict__ ids,
                                                                     float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTopkWaves + (threadIdx.x >> 6);
    if (t >= n) return;   // whole waves
    const float kNone = -__builtin_inff();
    float v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = 64 * j + lane;
        const float x = e < experts ? logits[t * stride + e] : kNone;
        v[j] = x != x ? kNone : fminf(x, FLT_MAX);
    }
    float best = kNone;
#pragma unroll
    for (int j = 0; j < J; ++j) best = fmaxf(best, v[j]);
    const float top1 = wave_max(best);
    float total = 0.0f;
    if (!normalize) {
#pragma unroll
        for (int j = 0; j < J; ++j) total += v[j] > kNone ? expf(v[j] - top1) : 0.0f;
        total = wave_sum(total);
    }
    // lane c keeps choice c
    int my_id = -1;
    float my_v = kNone;
    for (int c = 0; c < top; ++c) {
        best = kNone;
#pragma unroll
        for (int j = 0; j < J; ++j) best = fmaxf(best, v[j]);
        const float m = wave_max(best);
        if (m == kNone) break;
        bool found = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint64_t has = __ballot(v[j] == m);
            if (!found && has) {
                found = true;
                const int l = __builtin_ctzll(has);
                if (lane == l) v[j] = kNone;
                if (lane == c) {
                    my_id = 64 * j + l;
                    my_v = m;
                }
            }
        }
    }
    const float p = my_id >= 0 ? expf(my_v - top1) : 0.0f;
    if (normalize) total = wave_sum(p);
    if (lane < top) {
        ids[(int64_t)t * top + lane] = my_id;
        weights[(int64_t)t * top + lane] = my_id >= 0 ? p / total * scale : 0.0f;
    }
}

constexpr int kSortThreads = 1024;

// Workgroup e: the slots of expert e.  count = n * top.
__global__ __launch_bounds__(kSortThreads) void route_sort_kernel(const int32_t* __restrict__ ids, int count, int top,
                                                                  int experts, int32_t* __restrict__ slot,
                                                                  int32_t* __restrict__ rows,
                                                                  int32_t* __restrict__ offsets) {
    __shared__ int sums[2][kSortThreads / 64];
    const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int waves = blockDim.x >> 6;
    // contiguous runs of whole 16-byte groups
    const int run = ((count + (int)blockDim.x - 1) / (int)blockDim.x + 3) & ~3;
    const int i0 = min((int64_t)tid * run, (int64_t)count), i1 = min(i0 + run, count);
    int below = 0, equal = 0, none = 0;
    const bool last = e == experts - 1;
    auto tally = [&](int x) {
        below += x >= 0 && x < e;
        equal += x == e;
        none += x < 0;
    };
    int i = i0;
    for (; i + 4 <= i1; i += 4) {
        const int4 x = *reinterpret_cast<const int4*>(ids + i);
        tally(x.x); tally(x.y); tally(x.z); tally(x.w);
    }
    for (; i < i1; ++i) tally(ids[i]);

    // this thread's place among the equal ones, and all threads' counts below
    int place = equal;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(place, o);
        if (lane >= o) place += up;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) below += __shfl_xor(below, o);
    if (lane == 63) sums[0][wave] = place;
    if (lane == 0) sums[1][wave] = below;
    __syncthreads();
    int first = 0, before = 0, all = 0;
    for (int w = 0; w < waves; ++w) {
        first += sums[1][w];
        before += w < wave ? sums[0][w] : 0;
        all += sums[0][w];
    }
    int s = first + before + place - equal;
    if (equal)
        for (i = i0; i < i1; ++i)
            if (ids[i] == e) {
                slot[i] = s;
                rows[s] = i / top;
                ++s;
            }
    if (tid == 0) offsets[e] = first;
    if (last) {   // what no expert takes
        if (tid == 0) offsets[experts] = first + all;
        if (none)
            for (i = i0; i < i1; ++i)
                if (ids[i] < 0) slot[i] = -1;
        for (i = first + all + tid; i < count; i += blockDim.x) rows[i] = -1;
    }
}

template <bool H>
struct YVec;
template <>
struct YVec<false> {
    typedef float T;
    static constexpr int kN = 4;
    __device__ static void load(const float* p, float (&v)[4]) {
        const v4f a = *reinterpret_cast<const v4f*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i];
    }
};
template <>
struct YVec<true> {
    typedef _Float16 T;
    static constexpr int kN = 8;
    __device__ static void load(const _Float16* p, float (&v)[8]) {
        const v8h a = *reinterpret_cast<const v8h*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
    }
};

// VEC: 16 bytes of y per thread (m a multiple of that many values); otherwise
// one value.
template <bool H, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ y, int64_t slots, int m,
                                                      const int32_t* __restrict__ slot,
                                                      const float* __restrict__ weights, int top, int cols,
                                                      const float* residual, float* out) {
    typedef YVec<H> Y;
    constexpr int kN = VEC ? Y::kN : 1;
    const int64_t t = blockIdx.x / cols;
    const int64_t col = ((int64_t)(blockIdx.x % cols) * 256 + threadIdx.x) * kN;
    if (col >= m) return;
    const typename Y::T* yp = static_cast<const typename Y::T*>(y) + col;
    float acc[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
    for (int j = 0; j < top; ++j) {
        const int64_t s = slot[t * top + j];
        if (s < 0 || s >= slots) continue;
        const float w = weights[t * top + j];
        float v[kN];
        if constexpr (VEC)
            Y::load(yp + s * m, v);
        else
            v[0] = (float)yp[s * m];
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
    const int64_t o = t * m + col;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
            v4f r = v4f{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
            if (residual) r += *reinterpret_cast<const v4f*>(residual + o + i);
            *reinterpret_cast<v4f*>(out + o + i) = r;
        }
    } else {
        out[o] = residual ? residual[o] + acc[0] : acc[0];
    }
}

template <bool H>
hipError_t launch_combine_t(const void* y, int64_t slots, int m, const int32_t* slot, const float* weights, int n,
                            int top, const float* residual, float* out, hipStream_t stream) {
    const bool vec = m % YVec<H>::kN == 0;
    const int per = 256 * (vec ? YVec<H>::kN : 1), cols = (m + per - 1) / per;
    const dim3 grid((unsigned)((int64_t)n * cols));
    if (vec)
        hipLaunchKernelGGL((combine_kernel<H, true>), grid, dim3(256), 0, stream, y, slots, m, slot, weights, top, cols,
                           residual, out);
    else
        hipLaunchKernelGGL((combine_kernel<H, false>), grid, dim3(256), 0, stream, y, slots, m, slot, weights, top,
                           cols, residual, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const float* logits, int64_t stride, int n, int experts, int top, bool normalize, float scale,
                        int32_t* ids, float* weights, int32_t* slot, int32_t* rows, int32_t* offsets,
                        hipStream_t stream) {
    const dim3 grid((unsigned)((n + kTopkWaves - 1) / kTopkWaves)), block(64 * kTopkWaves);
    const int per = (experts + 63) / 64;
    switch (per) {
#define MMQ_TOPK(J)                                                                                                 \
    hipLaunchKernelGGL((route_topk_kernel<J>), grid, block, 0, stream, logits, stride, n, experts, top, (int)normalize, \
                       scale, ids, weights)
        case 1: MMQ_TOPK(1); break;
        case 2: MMQ_TOPK(2); break;
        case 3:
        case 4: MMQ_TOPK(4); break;
        case 5:
        case 6:
        case 7:
        case 8: MMQ_TOPK(8); break;
        default: MMQ_TOPK(16); break;
#undef MMQ_TOPK
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int count = n * top;
    const int threads = count <= 1024 ? 256 : kSortThreads;
    hipLaunchKernelGGL(route_sort_kernel, dim3((unsigned)experts), dim3(threads), 0, stream, ids, count, top, experts,
                       slot, rows, offsets);
    return hipGetLastError();
}

hipError_t launch_combine(const void* y, bool y_f16, int64_t slots, int m, const int32_t* slot, const float* weights,
                          int n, int top, const float* residual, float* out, hipStream_t stream) {
    return y_f16 ? launch_combine_t<true>(y, slots, m, slot, weights, n, top, residual, out, stream)
                 : launch_combine_t<false>(y, slots, m, slot, weights, n, top, residual, out, stream);
}

}  // namespace mmq
