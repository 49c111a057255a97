// rope.hip - rotary positions with several axes on rows of heads.
//
//   pair j of a head: (a, b) -> scale * (a cos t - b sin t, a sin t + b cos t),
//   t = positions[row][axis[j]] * freq[j]; values past the pairs are copied
//
// The rows are read and written once and bound it: 8192 rows of 32 binary16 heads
// of 128 with three axes, 134 MB, take 32 us, 4.2 TB/s.  A workgroup takes a row:
// its first lanes put the pairs' cosines and sines into LDS, once for all
// heads, then each lane turns 8 pairs (halves) or 4 (adjacent) at a time with
// 16-byte accesses; sizes or strides that do not allow those go value by value.
#include "internal.h"
#include "rope.h"

namespace mmq {
namespace {

constexpr int kMaxPairs = 512;

// Rows, and so runs of 8, lie on 16-byte boundaries, float32 too: what is promised
// to the compiler is no more.
template <typename T, int N>
struct alignas(16) Vec {
    T v[N];
};

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void rope_kernel(Rope rope, HeadRows x, HeadRows out, int heads, int dim) {
    __shared__ double2 cs[kMaxPairs];
    const int64_t row = blockIdx.x;
    for (int j = threadIdx.x; j < rope.pairs; j += blockDim.x) cs[j] = rope_angle(rope, row, j);
    __syncthreads();
    const T* src = static_cast<const T*>(x.p) + row * x.stride;
    T* dst = static_cast<T*>(out.p) + row * out.stride;
    const int pairs = rope.pairs, rest = dim - 2 * pairs;
    if constexpr (VEC) {
        // Pieces of 8 values: first halves (with their partners) or whole
        // pairs, then what is not rotated.
        typedef Vec<T, 8> V;
        static_assert(alignof(V) == 16 && sizeof(V) == 8 * sizeof(T));
        const int turned = (rope.adjacent ? 2 * pairs : pairs) >> 3, per = turned + (rest >> 3);
        for (int i = threadIdx.x; i < heads * per; i += blockDim.x) {
            const int h = i / per, c = i - h * per;
            if (c >= turned) {
                const int at = h * dim + 2 * pairs + 8 * (c - turned);
                *reinterpret_cast<V*>(dst + at) = *reinterpret_cast<const V*>(src + at);
            } else if (rope.adjacent) {
                const int at = h * dim + 8 * c;
                V a = *reinterpret_cast<const V*>(src + at);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float u, w;
                    rope_turn(cs[4 * c + j], (float)a.v[2 * j], (float)a.v[2 * j + 1], u, w);
                    a.v[2 * j] = (T)u;
                    a.v[2 * j + 1] = (T)w;
                }
                *reinterpret_cast<V*>(dst + at) = a;
            } else {
                const int at = h * dim + 8 * c;
                V a = *reinterpret_cast<const V*>(src + at), b = *reinterpret_cast<const V*>(src + at + pairs);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float u, w;
                    rope_turn(cs[8 * c + j], (float)a.v[j], (float)b.v[j], u, w);
                    a.v[j] = (T)u;
                    b.v[j] = (T)w;
                }
                *reinterpret_cast<V*>(dst + at) = a;
                *reinterpret_cast<V*>(dst + at + pairs) = b;
            }
        }
    } else {
        const int per = pairs + rest;
        for (int i = threadIdx.x; i < heads * per; i += blockDim.x) {
            const int h = i / per, c = i - h * per;
            if (c >= pairs) {
                const int at = h * dim + pairs + c;
                dst[at] = src[at];
                continue;
            }
            const int a = h * dim + (rope.adjacent ? 2 * c : c), b = a + (rope.adjacent ? 1 : pairs);
            float u, w;
            rope_turn(cs[c], (float)src[a], (float)src[b], u, w);
            dst[a] = (T)u;
            dst[b] = (T)w;
        }
    }
}

template <typename T>
hipError_t launch(const Rope& rope, const HeadRows& x, const HeadRows& out, int n, int heads, int dim,
                  hipStream_t stream) {
    const int unit = 16 / (int)sizeof(T);   // rows and runs start on 16-byte boundaries
    const bool vec = (rope.pairs & (rope.adjacent ? 3 : 7)) == 0 && (dim & 7) == 0 && x.stride % unit == 0 &&
                     out.stride % unit == 0;
    if (vec)
        hipLaunchKernelGGL((rope_kernel<T, true>), dim3(n), dim3(256), 0, stream, rope, x, out, heads, dim);
    else
        hipLaunchKernelGGL((rope_kernel<T, false>), dim3(n), dim3(256), 0, stream, rope, x, out, heads, dim);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const Rope& rope, const HeadRows& x, const HeadRows& out, int n, int heads, int dim,
                       hipStream_t stream) {
    return x.half ? launch<_Float16>(rope, x, out, n, heads, dim, stream)
                  : launch<float>(rope, x, out, n, heads, dim, stream);
}

}  // namespace mmq
