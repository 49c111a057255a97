// q6k_stage.h - a wave's LDS copy of q6_K weight rows (shared by the few-token
// q6_K kernels).
#pragma once
#include "internal.h"
#include "kquant_device.h"
#include "q6k_device.h"

namespace mmq {
namespace {

// One wave step: SW super-blocks of 16 rows.  The rows' bytes are copied
// into the wave's LDS area by buffer loads that write LDS directly (no
// registers hold the copy): row r's run of SW blocks, from the 16-byte
// boundary below its first byte, in aligned 16-byte pieces.  Slot i of the
// area (16 bytes at 16*i) holds piece i % kSlots of row i / kSlots; the last
// slot of a row is padding, which spreads the 16 rows' reads over the banks.
// The 2-byte-aligned block fields are then read from LDS as aligned dwords
// and shifted into place (see q6k_device.h).
template <int SW>
struct Seg {
    static constexpr int kChunks = (SW * kQ6kBlockBytes + 14 + 15) / 16;  // pieces per row
    static constexpr int kSlots = kChunks + 1;
    static constexpr int kBytes = 16 * kSlots;                           // row stride in LDS
    static constexpr int kArea = 16 * kBytes;
    static constexpr int kLoads = (16 * kSlots + 63) / 64;               // load instructions per step
};

// A 16-byte piece at byte offset a (a % 16 == 0) of the weights, reading
// nothing at or past byte `total` (its bytes past the end read as 0).
__device__ __forceinline__ uint4 load_piece(const uint8_t* __restrict__ w, int64_t a, int64_t total) {
    uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (a + 2 * i + 2 <= total)
            d[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(w + a + 2 * i) << (16 * (i & 1));
    return make_uint4(d[0], d[1], d[2], d[3]);
}

// The five LDS dwords covering 16 bytes at LDS byte address `a` (2-aligned).
__device__ __forceinline__ void lds_run(const uint8_t* base, int a, uint32_t (&v)[5]) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(base + (a & ~3));
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = p[i];
}

// The weights of a workgroup's tile of rows: a buffer resource over its
// whole 16-byte pieces, and the partial piece at its end (the tile's bytes
// need not end on a 16-byte boundary), which a buffer load would read as
// zeros and stage_patch copies in with 2-byte loads.
struct Tile {
    __amdgpu_buffer_rsrc_t rs;
    const uint8_t* base;
    int end;     // the tile's bytes
    int rows;    // rows in the tile
};

// After the copy of step s has landed: the tile's partial last piece, if
// this step's run of the tile's last row covers it.
template <int SW>
__device__ __forceinline__ void stage_patch(const Tile& tl, int S, int s, int lane, uint8_t* area) {
    typedef Seg<SW> G;
    const int end16 = tl.end & ~15;
    if (end16 == tl.end) return;
    const int rr = tl.rows - 1;
    const int ch = (end16 - (((rr * S + s) * kQ6kBlockBytes) & ~15)) >> 4;
    if (lane == 0 && ch >= 0 && ch < G::kChunks)
        *reinterpret_cast<uint4*>(area + rr * G::kBytes + 16 * ch) = load_piece(tl.base, end16, tl.end);
}

}  // namespace
}  // namespace mmq
