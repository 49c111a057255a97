// kv_attend.hip - how the attention over the cache is spread over the chip, and
// the join of its pieces (kv_attend.h has the kernel).
#include "internal.h"
#include "kv_attend.h"

namespace mmq {
namespace kv {
namespace {

constexpr int kCus = 256, kJoinWaves = 8, kMaxRuns = 3 * kCus;

// The x-th workgroup that began rows for others to go on with, -1 if there are
// not that many.
__device__ __forceinline__ int began(const Attend& a, int x) {
    const int lane = threadIdx.x & 63;
    uint64_t some[kMaxRuns / 64];
#pragma unroll
    for (int i = 0; i < kMaxRuns / 64; ++i) {
        const int at = 64 * i + lane;
        some[i] = __builtin_amdgcn_ballot_w64(at < a.wgs && a.join[at < a.wgs ? at : 0].count > 0);
    }
#pragma unroll
    for (int i = 0; i < kMaxRuns / 64; ++i) {
        const int n = __popcll(some[i]);
        if (x < n) {
            uint64_t left = some[i];
            for (; x > 0; --x) left &= left - 1;
            return 64 * i + __builtin_ctzll(left);
        }
        x -= n;
    }
    return -1;
}

// All of a row's parts, in order.  dim / 4 lanes take a row, 4 dims each, as
// many rows as fit a wave; where there are many parts (SHARED) a workgroup takes
// one such set of rows, its waves a share of the parts each, and joins in LDS.
template <bool SHARED>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(Attend a, int tile_rows) {
    __shared__ v4f sums[kJoinWaves][64];
    __shared__ float2 stats[SHARED ? kMaxRuns : 1][SHARED ? 8 : 1];   // (reference, sum) of a part's row
    const int wg = (int)gridDim.x == a.wgs ? (int)blockIdx.x : began(a, blockIdx.x), lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int group = a.q.group, dim = a.c.dim, lanes = dim >> 2, per_wave = 64 / lanes;   // 1 .. 8 rows
    const int sub = lane / lanes, d = 4 * (lane - sub * lanes);
    const int row = (SHARED ? blockIdx.y : blockIdx.y * kJoinWaves + wave) * per_wave + sub;
    if (wg < 0) return;
    const Join j = a.join[wg];
    if (j.count <= 0) return;
    const bool live = sub < per_wave && row < j.rows && row < tile_rows;
    const auto at = [&](int i) { return (int64_t)(2 * (wg + i) + (i == 0 ? j.slot : 0)) * tile_rows + (live ? row : 0); };
    float top = kFloor, sum = 0.0f;
    v4f x = {0, 0, 0, 0};
    if (SHARED) {
        for (int i = threadIdx.x / per_wave; i < j.count; i += blockDim.x / per_wave) {
            const int r = threadIdx.x % per_wave, at_row = blockIdx.y * per_wave + r < tile_rows ? blockIdx.y * per_wave + r : 0;
            if (threadIdx.x / per_wave < blockDim.x / per_wave)
                stats[i][r] = a.stat[(int64_t)(2 * (wg + i) + (i == 0 ? j.slot : 0)) * tile_rows + at_row];
        }
        __syncthreads();
    }
    const auto stat = [&](int i) { return SHARED ? stats[i][sub < per_wave ? sub : 0] : a.stat[at(i)]; };
#pragma unroll 8
    for (int i = 0; i < j.count; ++i) top = fmaxf(top, stat(i).x);
#pragma unroll 8
    for (int i = SHARED ? wave : 0; i < j.count; i += SHARED ? kJoinWaves : 1)
        x += *reinterpret_cast<const v4f*>(a.part + at(i) * dim + d) * __builtin_amdgcn_exp2f(stat(i).x - top);
#pragma unroll 8
    for (int i = 0; i < j.count; ++i) {
        const float2 st = stat(i);
        sum += st.y * __builtin_amdgcn_exp2f(st.x - top);
    }
    if (SHARED) {
        sums[wave][lane] = x;
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (int w = 1; w < kJoinWaves; ++w) x += sums[w][lane];
    }
    const int ri = j.row + row;
    if (live)
        put_row(a.q, j.token + ri / group, j.head * group + ri % group, a.c.heads * group, dim, d, x, top, sum);
}

// How a call is cut.
struct Cut {
    Form form;
    int rows;          // of a tile
    int most;          // of them, used
    int tiles;         // per sequence and head, at most
    int wgs;           // 0: a workgroup per tile, head and sequence
    bool joined;       // some piece may need joining
    bool many;         // of many parts
    int joins;         // workgroups of join_kernel: of every run, or of the tiles in pieces alone
    int join_rows;     // and of their rows
};

Cut cut(const KvCache& c, const KvPlan& p, const KvQuery& q) {
    Cut r;
    const int64_t rows = (int64_t)q.most * q.group;
    const int nb = c.dim / 32;
    const bool full = !(q.q_half && q.out_half);
    const auto form = [&](Form f) {
        r.form = f;
        r.rows = tile_rows(f, nb);
        r.most = rows < r.rows ? (int)rows : r.rows;
        r.tiles = (int)((rows + r.rows - 1) / r.rows);
        return (int64_t)r.tiles * c.heads * p.seqs;
    };
    // Tiles of 16 rows up to there.  From 128 rows on (65 above 128 dims, where
    // kWide's tiles are of 32) kTall, whose waves share the codes' way to operands;
    // below, it has idle waves, but of 96 and 128 dims codes are most of the work: of
    // 128 in 8 bits always, else while tiles are few (kTall / kWide, us, 8 heads, 2048
    // tokens: 128 dims, 8 bits, 32 rows of 32 sequences 72 / 82, in float32 106 / 103, 96
    // rows 107 / 121 and 135 / 163; 4 bits, 32 rows of 2 sequences 26 / 27, of 8 42 / 45, in
    // float32 29 / 30 and 42 / 53, of 32 69 / 66 and 102 / 90; 96 dims, 8 bits, of 2 24 /
    // 24, of 8 37 / 35, in float32 27 / 26 and 39 / 42; 64 dims, of 32 50 / 40, 124 rows 72
    // / 56, 128 71 / 56 but of 2 27 / 34; 256 dims, 64 rows 151 / 136, 65 175 / 198).  Of
    // kWide's workgroups those of 8 waves where there are no more tiles than CUs, else
    // of 4, whose beginnings and ends overlap (8 / 4 waves, us, 8 heads of 128, 4 bits, 32
    // rows: 16 sequences of 2048 tokens 49 / 52, 32 61 / 66, 64 108 / 97; of 64, 48 rows: 16
    // windows of 1024 26 / 30, 64 sequences of 1024 49 / 37).
    const bool codes = !has_wide(c.q4, nb) || ((nb == 3 || nb == 4) && c.heads * (int64_t)p.seqs <= kCus / 4);
    int64_t all = form(rows <= 16 ? kNarrow : rows < (nb > 4 ? 65 : codes ? 17 : 128) ? kWide : kTall);
    if (r.form == kWide && all <= kCus && fits(c.q4, nb, kWide8, full)) all = form(kWide8);
    const int runs = kCus * wgs_per_cu(c.q4, nb, r.form, full);   // what the chip holds
    // Splitting takes steps off the longest sequence's and spreads them over idle
    // CUs; the second launch and the parts' way through memory cost what 2 to 5 of
    // a workgroup's steps do.  Not split, us, against split, caches from HBM, 8 heads
    // of 128 with 4 query heads each: 1 sequence of 512 tokens 11.7 / 12.4, of 768 15.0
    // / 13.2, of 1024 17.4 / 12.9; 16 of 1024 18.8 / 22.1, of 2048 29.0 / 28.4; 64 of
    // 1024 33.1 / 36.6; with 32 rows 1 of 256 20.2 / 22.4, of 768 39.9 / 24.0, 16 of 768
    // 42.6 / 41.1, of 2048 90 / 53; 600 rows of 4 over 1024 60 / 77, over 2048 106 / 98;
    // 8 heads of 256, 4 rows: 1 of 256 13.4 / 15.5, of 512 19.9 / 16.4.  Not past 1280
    // tokens, as the host does not know how ragged the lengths are; but also where
    // one sequence is all there is and its tiles fill the chip, as its last ones see
    // most and go first (1500 rows of 4, 376 tiles, over 2048 129 / 164, over 4096 249 /
    // 251; 2048, 512 tiles, over 2048 143 / 148, over 8192 505 / 509; 4096 over 4096 438 /
    // 517).  Of more sequences equal ones would be level (4 of 512 rows over 2048 145 / 152,
    // over 8192 508 / 512; 16 of 130 over 4096 472 / 363), but a long history among
    // them would be one workgroup's a tile (63 decoding sequences of 4000 tokens and a chunk of
    // 512 2617 us, 323 cut).
    int64_t span = (int64_t)p.width << c.shift;
    if (q.window && q.window < span - q.most - kTile) span = q.window + (int64_t)q.most + kTile;
    const int unit = unit_of(r.form);
    const int64_t units = (span + unit - 1) / unit, idle = all < kCus ? kCus - all : 0;
    const int worth = r.form == kWide8 ? (c.dim > 64 ? 2 : 3) : c.dim > 128 ? 3 : 5;
    const bool direct = (span <= 1280 && units * idle <= worth * kCus) || (p.seqs == 1 && r.tiles > 1 && all >= 2 * kCus);
    r.wgs = direct ? 0 : runs;
    r.many = runs > 16 * all;
    r.joined = !direct;
    const int per_join = 256 / c.dim * (r.many ? 1 : kJoinWaves);   // rows of a workgroup
    r.join_rows = (r.most + per_join - 1) / per_join;
    // Workgroups that find nothing to join take their time too; a look at all runs
    // for those that have is 1 to 2 us (1 sequence of 4096 tokens, 8 heads of 128, 96
    // rows: 39 us with it, 54 without).
    r.joins = all < runs && (int64_t)runs * r.join_rows > 2048 ? (int)all : runs;
    return r;
}

}  // namespace
}  // namespace kv

int64_t kv_attend_workspace(const KvCache& c, const KvPlan& p, const KvQuery& q) {
    const kv::Cut t = kv::cut(c, p, q);
    return (int64_t)t.wgs * (2LL * t.rows * (4LL * c.dim + 8) + (int64_t)sizeof(kv::Join));
}

hipError_t launch_kv_attend(const KvCache& c, const KvPlan& p, const KvQuery& q, void* workspace, hipStream_t stream) {
    const kv::Cut t = kv::cut(c, p, q);
    kv::Attend a{c, p, q, t.wgs, nullptr, nullptr, nullptr};
    const int64_t slots = 2LL * t.wgs * t.rows;
    a.part = static_cast<float*>(workspace);
    a.stat = reinterpret_cast<float2*>(a.part + slots * c.dim);
    a.join = reinterpret_cast<kv::Join*>(a.stat + slots);
    const dim3 grid = t.wgs ? dim3(t.wgs) : dim3(t.tiles, c.heads, p.seqs);
    const bool broad = c.dim > 128;
    hipError_t rc = c.q4 ? (broad ? kv::launch_q4_broad(a, t.form, grid, stream) : kv::launch_q4_narrow(a, t.form, grid, stream))
                         : (broad ? kv::launch_q8_broad(a, t.form, grid, stream) : kv::launch_q8_narrow(a, t.form, grid, stream));
    if (rc != hipSuccess || !t.joined) return rc;
    const dim3 join(t.joins, t.join_rows), block(64 * kv::kJoinWaves);
    if (t.many)
        hipLaunchKernelGGL(kv::join_kernel<true>, join, block, 0, stream, a, t.rows);
    else
        hipLaunchKernelGGL(kv::join_kernel<false>, join, block, 0, stream, a, t.rows);
    return hipGetLastError();
}

}  // namespace mmq
