// group.h - the token groups of the matmuls grouped by expert.
//
// Expert e has the slots offsets[e] .. offsets[e + 1] - 1; the offsets are
// device data, so the host launches a grid for the most work there can be
// and every workgroup finds its own: an item is up to TB consecutive slots
// of one expert, items are numbered expert by expert, and a wave finds item
// i with one load of 64 offsets, a prefix sum and a ballot per 64 experts
// (about a microsecond, most of it the load).  Workgroups take items in
// strides of the grid until there are no more, so a launch whose experts
// are all outside [lo, hi] costs one lookup per workgroup.
//
// Offsets and rows outside their ranges are clamped: a wrong one gives wrong
// values, never an access outside the buffers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmq {

// The tokens of a plain call: token i is row i of q, ds and the output.
struct NoGroups {
    static constexpr bool kOn = false;
};

struct Groups {
    static constexpr bool kOn = true;
    const int32_t* offsets;   // [experts + 1]
    const int32_t* rows;      // [slots] the row of q of each slot; null: the slot itself
    int experts, slots;
    int tokens;               // rows of q
    int lo, hi;               // this launch takes the experts with lo .. hi slots (lo >= 1)
};

struct Item {
    int expert, start, count;   // slots start .. start + count - 1
    bool valid;
};

// Item i of the launch.  Wave-collective, every lane active; the result is
// wave-uniform.
template <int TB>
__device__ __forceinline__ Item find_item(const Groups& g, int i) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base < g.experts; base += 64) {
        const int e = base + lane;
        int a = 0, c = 0;
        if (e < g.experts) {
            a = min(max(g.offsets[e], 0), g.slots);
            c = min(max(g.offsets[e + 1], a), g.slots) - a;
        }
        const int items = c >= g.lo && c <= g.hi ? (c + TB - 1) / TB : 0;
        int incl = items;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(incl, o);
            if (lane >= o) incl += up;
        }
        const uint64_t past = __ballot(before + incl > i);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int skip = (i - before - __builtin_amdgcn_readlane(incl - items, l)) * TB;
            const int cl = __builtin_amdgcn_readlane(c, l);
            return Item{base + l, __builtin_amdgcn_readlane(a, l) + skip, min(TB, cl - skip), true};
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return Item{0, 0, 0, false};
}

// x, as a value the compiler knows nothing of: addresses computed from it in
// a loop over items are not kept in registers from one item to the next.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The most items a launch can have.
inline int64_t most_items(int64_t experts, int64_t slots, int64_t lo, int64_t hi, int64_t tb) {
    const int64_t full = slots / lo < experts ? slots / lo : experts;   // experts with lo slots or more
    const int64_t per = (hi + tb - 1) / tb;
    const int64_t a = slots / tb + full;
    return per < 1 ? 0 : full <= a / per ? full * per : a;
}

// Where a kernel finds its tokens' codes and scale words: row i of the item
// starts at byte row(i) * K of q.
template <class Grp>
struct TokenRows;

template <>
struct TokenRows<NoGroups> {
    int count;
    __device__ TokenRows(const NoGroups&, const Item&, int n) : count(n) {}
    __device__ __forceinline__ uint32_t row(int i) const { return (uint32_t)min(i, count - 1); }
};

template <>
struct TokenRows<Groups> {
    const int32_t* rows;
    int count, tokens, start;
    __device__ TokenRows(const Groups& g, const Item& it, int)
        : rows(g.rows ? g.rows + it.start : nullptr), count(it.count), tokens(g.tokens), start(it.start) {}
    __device__ __forceinline__ uint32_t row(int i) const {
        const int j = min(i, count - 1);
        return (uint32_t)(rows ? min(max(rows[j], 0), tokens - 1) : start + j);
    }
};

}  // namespace mmq
