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
// Offsets and rows outside their ranges are clamped, and an offset below an
// earlier one counts as the largest before it: a wrong one gives wrong values,
// never an access outside the buffers.  So the groups never overlap, and a
// launch has no more items than the slots make (most_items).
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

// The largest v of this lane and those below it: DPP moves within rows of 16
// lanes (row_shr 1, 2, 4, 8), then from lane 15 of a row to the next row and
// from lane 31 to the upper half (row_bcast 15, 31); a lane without a source
// keeps its own.
__device__ __forceinline__ int wave_max_scan(int v) {
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x111, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x112, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x114, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x118, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x142, 0xA, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x143, 0xC, 0xF, false));
    return v;
}

// The slots of expert base + lane.  high: the largest offset before this
// chunk of 64 experts, and then before the next (0 for the first); offsets
// that do not decrease need no scan for it.  Wave-collective, every lane
// active.
struct Span {
    int first, slots;
};
__device__ __forceinline__ Span expert_slots(const Groups& g, int base, int& high) {
    const int e = base + (int)(threadIdx.x & 63);
    int a = high, b = high;
    if (e < g.experts) {
        a = min(max(g.offsets[e], 0), g.slots);
        b = min(max(g.offsets[e + 1], 0), g.slots);
    }
    if (__ballot(b < a || a < high)) {
        a = max(wave_max_scan(a), high);
        b = max(a, b);
    }
    high = __builtin_amdgcn_readlane(b, 63);
    return Span{a, b - a};
}

// Item i of the launch.  Wave-collective, every lane active; the result is
// wave-uniform.
template <int TB>
__device__ __forceinline__ Item find_item(const Groups& g, int i) {
    const int lane = threadIdx.x & 63;
    int before = 0, high = 0;
    for (int base = 0; base < g.experts; base += 64) {
        const Span s = expert_slots(g, base, high);
        const int items = s.slots >= g.lo && s.slots <= g.hi ? (s.slots - 1) / TB + 1 : 0;   // lo >= 1
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
            const int n = __builtin_amdgcn_readlane(s.slots, l);
            return Item{base + l, __builtin_amdgcn_readlane(s.first, l) + skip, min(TB, n - skip), true};
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
