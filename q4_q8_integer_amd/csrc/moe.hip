// moe.hip - the router in front of the matmuls grouped by expert, and the
// combination of the experts' outputs behind them.
//
// Routing:
//   * choose_experts, a wave per token: the scores sit in registers (expert
//     64 j + lane), and each choice is a maximum over the wave (DPP moves, no
//     LDS) and a ballot for the lowest index that has it.  The softmax needs
//     no second pass: the first choice is its maximum.
//   * route_sort_kernel, a workgroup per expert: a stable counting sort that
//     needs neither atomics nor a workspace.  Expert e's workgroup reads all
//     n * top ids (they come from L2), counts those below e (its first slot)
//     and, per wave over a contiguous run, those equal to e, then goes over
//     the run again, 256 ids at a time, and writes slots and rows where there
//     are any.  Slots of an expert are in token order.
//   * A decode step's few ids (at most kSmallIds, times the rounds in which the
//     16 waves take the tokens) are chosen and sorted by one workgroup in one
//     launch, the ids in LDS: each id's slot is the number of ids below it and
//     of equal ones before it, counted by four lanes.
// Measured in a graph, one launch against two, 64 / 1024 experts: 1 token of 8
// experts 3.6 / 8.0 us against 5.8 / 12.2, 16 of 4 4.8 / 9.0 against 5.6 / 10.7,
// 16 of 8 (128 ids) 6.8 / 14.0 against 6.2 / 12.8, where a call from Python is
// 13.6 against 16.5 us; 32 of 2 5.4 / 10.4 against 5.5 / 9.4; beyond the rule 16
// of 16 11 / 26 against 7.1 / 17, 32 of 8 12 / 27 against 6.1 / 12.8.
// 8192 tokens, 8 of 128 experts 22 us: 8 us choosing, 14 sorting, where the 5 MB
// moved take 1 us: every expert's workgroup reads all ids, once or twice.
//
// Combining: out[t] = residual[t] + sum_j weights[t][j] * y[slot[t][j]], a
// thread per 16 bytes of y columns; slots and weights of a token are the
// same for a whole workgroup.  Bound by HBM: 8192 tokens of 4 experts, 4096
// binary16 values each, with a residual 106 us (523 MB: 102 us at the copy rate).
#include <cfloat>

#include "internal.h"
#include "q8_device.h"

namespace mmq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// One step of a wave reduction: v of the lane that CTRL names, or `other` in
// lanes that have none.
template <int CTRL>
__device__ __forceinline__ float dpp(float other, float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, other),
                                                                 __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// The maximum over the wave, in every lane: within rows of 16 lanes
// (row_shr 1, 2, 4, 8), then over rows (row_bcast 15, 31), from lane 63.
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<0x111>(v, v));
    v = fmaxf(v, dpp<0x112>(v, v));
    v = fmaxf(v, dpp<0x114>(v, v));
    v = fmaxf(v, dpp<0x118>(v, v));
    v = fmaxf(v, dpp<0x142>(v, v));
    v = fmaxf(v, dpp<0x143>(v, v));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// The choices of one token: lane c < top returns choice c and its weight.
// J: experts per lane.  A score of NaN counts as -inf and one of +inf as the
// largest float32; an expert at -inf is not chosen.
struct Choice {
    int id;
    float weight;
};
template <int J>
__device__ __forceinline__ Choice choose_experts(const float* __restrict__ logits, int experts, int top, int normalize,
                                                 float scale) {
    const int lane = threadIdx.x & 63;
    const float kNone = -__builtin_inff();
    float v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = 64 * j + lane;
        const float x = e < experts ? logits[e] : kNone;
        v[j] = x != x ? kNone : fminf(x, FLT_MAX);
    }
    float best = kNone;
#pragma unroll
    for (int j = 0; j < J; ++j) best = fmaxf(best, v[j]);
    float m = wave_max(best);
    const float top1 = m;
    float total = 0.0f;
    if (!normalize) {
#pragma unroll
        for (int j = 0; j < J; ++j) total += v[j] > kNone ? expf(v[j] - top1) : 0.0f;
        total = wave_sum(total);
    }
    Choice mine{-1, 0.0f};
    float my_v = kNone;
    for (int c = 0; c < top && m > kNone; ++c) {
        bool found = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint64_t has = __ballot(v[j] == m);
            if (!found && has) {
                found = true;
                const int l = __builtin_ctzll(has);
                if (lane == l) v[j] = kNone;
                if (lane == c) {
                    mine.id = 64 * j + l;
                    my_v = m;
                }
            }
        }
        best = kNone;
#pragma unroll
        for (int j = 0; j < J; ++j) best = fmaxf(best, v[j]);
        m = wave_max(best);
    }
    const float p = mine.id >= 0 ? expf(my_v - top1) : 0.0f;
    if (normalize) total = wave_sum(p);
    if (mine.id >= 0) mine.weight = p / total * scale;
    return mine;
}

template <int J>
__global__ __launch_bounds__(64 * kTopkWaves) void route_topk_kernel(const float* __restrict__ logits, int64_t stride,
                                                                     int n, int experts, int top, int normalize,
                                                                     float scale, int32_t* __restrict__ ids,
                                                                     float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTopkWaves + (threadIdx.x >> 6);
    if (t >= n) return;   // whole waves
    const Choice c = choose_experts<J>(logits + t * stride, experts, top, normalize, scale);
    if (lane < top) {
        ids[(int64_t)t * top + lane] = c.id;
        weights[(int64_t)t * top + lane] = c.weight;
    }
}

// The whole routing of up to kSmallIds ids, in one workgroup.
constexpr int kSmallIds = 128, kSmallThreads = 1024;
template <int J>
__global__ __launch_bounds__(kSmallThreads) void route_small_kernel(const float* __restrict__ logits, int64_t stride,
                                                                    int n, int experts, int top, int normalize,
                                                                    float scale, int32_t* __restrict__ ids,
                                                                    float* __restrict__ weights,
                                                                    int32_t* __restrict__ slot,
                                                                    int32_t* __restrict__ rows,
                                                                    int32_t* __restrict__ offsets) {
    __shared__ __attribute__((aligned(16))) int chosen[kSmallIds];
    const int tid = threadIdx.x, lane = tid & 63;
    const int count = n * top, padded = (count + 3) & ~3;
    if (tid < padded) chosen[tid] = -1;
    __syncthreads();
    for (int t = tid >> 6; t < n; t += kSmallThreads / 64) {
        const Choice c = choose_experts<J>(logits + t * stride, experts, top, normalize, scale);
        if (lane < top) {
            chosen[t * top + lane] = c.id;
            ids[t * top + lane] = c.id;
            weights[t * top + lane] = c.weight;
        }
    }
    __syncthreads();
    // Four lanes count for id p, then for expert e, each over a quarter of the
    // ids (16-byte groups part, part + 4, ..).  -1 is above every id.
    const int part = tid & 3, entry = tid >> 2;
    if (entry < ((count + 15) & ~15)) {   // whole waves
        const unsigned id = entry < count ? (unsigned)chosen[entry] : 0xFFFFFFFFu;
        int at = 0, used = 0;   // equal ids before it and all below it; ids that name an expert
        for (int i = 4 * part; i < padded; i += 16) {
            const int4 x = *reinterpret_cast<const int4*>(chosen + i);
            const unsigned v[4] = {(unsigned)x.x, (unsigned)x.y, (unsigned)x.z, (unsigned)x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                at += v[j] < id || (v[j] == id && i + j < entry);
                used += v[j] != 0xFFFFFFFFu;
            }
        }
        at = quad_sum(at);
        used = quad_sum(used);
        if (part == 0 && entry < count) {
            const bool none = id == 0xFFFFFFFFu;
            slot[entry] = none ? -1 : at;
            if (!none) rows[at] = entry / top;
            if (entry >= used) rows[entry] = -1;
        }
    }
    for (int e = entry; e < ((experts + 16) & ~15); e += kSmallThreads / 4) {   // 0 .. experts, whole waves
        int first = 0;
        for (int i = 4 * part; i < padded; i += 16) {
            const int4 x = *reinterpret_cast<const int4*>(chosen + i);
            first += ((unsigned)x.x < (unsigned)e) + ((unsigned)x.y < (unsigned)e) + ((unsigned)x.z < (unsigned)e) +
                     ((unsigned)x.w < (unsigned)e);
        }
        first = quad_sum(first);
        if (part == 0 && e <= experts) offsets[e] = first;
    }
}

constexpr int kSortThreads = 1024;

// i / top for 0 <= i < 2^30, inv = floor(2^32 / top) (2^32 - 1 for top = 1):
// the product's high half is at most one too small.
__device__ __forceinline__ int divide(int i, int top, uint32_t inv) {
    const int q = (int)__umulhi((uint32_t)i, inv);
    return i - q * top >= top ? q + 1 : q;
}

// Workgroup e: the slots of expert e.  count = n * top.
__global__ __launch_bounds__(kSortThreads) void route_sort_kernel(const int32_t* __restrict__ ids, int count, int top,
                                                                  uint32_t inv, int experts, int32_t* __restrict__ slot,
                                                                  int32_t* __restrict__ rows,
                                                                  int32_t* __restrict__ offsets) {
    constexpr int kWaves = kSortThreads / 64;
    __shared__ int sums[2][kWaves];
    const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // wave w takes a contiguous run of ids in steps of 256, four neighbours
    // per lane
    const int run = ((count + kWaves - 1) / kWaves + 255) & ~255;
    const int i0 = (int)min((int64_t)wave * run, (int64_t)count), i1 = min(i0 + run, count);
    const auto load = [&](int i) {   // ids i .. i + 3, -1 past the run
        int4 x = make_int4(-1, -1, -1, -1);
        if (i + 4 <= i1) return *reinterpret_cast<const int4*>(ids + i);
        if (i < i1) x.x = ids[i];
        if (i + 1 < i1) x.y = ids[i + 1];
        if (i + 2 < i1) x.z = ids[i + 2];
        return x;
    };
    int below = 0, equal = 0;
#pragma unroll 4
    for (int i = i0 + 4 * lane; i < i1; i += 256) {
        const int4 x = load(i);
        // -1 is not below: as unsigned it is above every id
        below += ((unsigned)x.x < (unsigned)e) + ((unsigned)x.y < (unsigned)e) + ((unsigned)x.z < (unsigned)e) +
                 ((unsigned)x.w < (unsigned)e);
        equal += (x.x == e) + (x.y == e) + (x.z == e) + (x.w == e);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        below += __shfl_xor(below, o);
        equal += __shfl_xor(equal, o);
    }
    if (lane == 0) {
        sums[0][wave] = equal;
        sums[1][wave] = below;
    }
    __syncthreads();
    int first = 0, s = 0, all = 0;
    for (int w = 0; w < kWaves; ++w) {
        first += sums[1][w];
        s += w < wave ? sums[0][w] : 0;
        all += sums[0][w];
    }
    s += first;
    const bool last = e == experts - 1;
    if (equal || last) {
        int4 next = load(i0 + 4 * lane);
        for (int i = i0; i < i1; i += 256) {
            const int p = i + 4 * lane;
            const int v[4] = {next.x, next.y, next.z, next.w};
            next = load(p + 256);
            uint64_t has[4];
            int at = s;   // and the equal ids in lower lanes
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                has[j] = __ballot(v[j] == e);
                at = __builtin_amdgcn_mbcnt_hi((uint32_t)(has[j] >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)has[j], at));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (has[j]) {
                    if (v[j] == e) {
                        slot[p + j] = at;
                        rows[at] = divide(p + j, top, inv);
                        ++at;
                    }
                    s += __builtin_popcountll(has[j]);
                }
            if (last) {   // ids that name no expert
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (p + j < i1 && v[j] < 0) slot[p + j] = -1;
            }
        }
    }
    if (tid == 0) offsets[e] = first;
    if (last) {
        if (tid == 0) offsets[experts] = first + all;
        for (int i = first + all + tid; i < count; i += kSortThreads) rows[i] = -1;
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
    const int cols = (int)combine_cols(H, m);
    const dim3 grid((unsigned)((int64_t)n * cols));
    if (vec)
        hipLaunchKernelGGL((combine_kernel<H, true>), grid, dim3(256), 0, stream, y, slots, m, slot, weights, top, cols,
                           residual, out);
    else
        hipLaunchKernelGGL((combine_kernel<H, false>), grid, dim3(256), 0, stream, y, slots, m, slot, weights, top,
                           cols, residual, out);
    return hipGetLastError();
}

template <int J>
hipError_t launch_route_t(const float* logits, int64_t stride, int n, int experts, int top, bool normalize, float scale,
                          int32_t* ids, float* weights, int32_t* slot, int32_t* rows, int32_t* offsets,
                          hipStream_t stream) {
    const int count = n * top;
    const int rounds = (n + kSmallThreads / 64 - 1) / (kSmallThreads / 64);   // of the small kernel's waves
    if ((int64_t)count * rounds <= kSmallIds) {
        hipLaunchKernelGGL((route_small_kernel<J>), dim3(1), dim3(kSmallThreads), 0, stream, logits, stride, n, experts,
                           top, (int)normalize, scale, ids, weights, slot, rows, offsets);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((route_topk_kernel<J>), dim3((unsigned)((n + kTopkWaves - 1) / kTopkWaves)),
                       dim3(64 * kTopkWaves), 0, stream, logits, stride, n, experts, top, (int)normalize, scale, ids,
                       weights);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t inv = top == 1 ? 0xFFFFFFFFu : (uint32_t)((1ULL << 32) / (unsigned)top);
    hipLaunchKernelGGL(route_sort_kernel, dim3((unsigned)experts), dim3(kSortThreads), 0, stream, ids, count, top, inv,
                       experts, slot, rows, offsets);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const float* logits, int64_t stride, int n, int experts, int top, bool normalize, float scale,
                        int32_t* ids, float* weights, int32_t* slot, int32_t* rows, int32_t* offsets,
                        hipStream_t stream) {
    const auto f = experts <= 64    ? launch_route_t<1>
                   : experts <= 128 ? launch_route_t<2>
                   : experts <= 256 ? launch_route_t<4>
                   : experts <= 512 ? launch_route_t<8>
                                    : launch_route_t<16>;
    return f(logits, stride, n, experts, top, normalize, scale, ids, weights, slot, rows, offsets, stream);
}

hipError_t launch_combine(const void* y, bool y_f16, int64_t slots, int m, const int32_t* slot, const float* weights,
                          int n, int top, const float* residual, float* out, hipStream_t stream) {
    return y_f16 ? launch_combine_t<true>(y, slots, m, slot, weights, n, top, residual, out, stream)
                 : launch_combine_t<false>(y, slots, m, slot, weights, n, top, residual, out, stream);
}

}  // namespace mmq
