// mmq_api.hip - the C ABI declared in include/mmq.h.
//
// Every argument is checked on the host before any HIP call; only then is
// the current device checked (once per device: gfx950 or MMQ_ERR_DEVICE) and
// the kernel enqueued on the caller's stream.  Nothing here allocates.
#include <atomic>
#include <cstring>

#include "../../include/mmq.h"
#include "group.h"
#include "internal.h"
#include "stream.h"
#include "q6k_device.h"

namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;      // n, m
constexpr int64_t kMaxK = 1LL << 24;
constexpr int64_t kMaxExperts = 4096;
constexpr int64_t kMaxRouteIds = 1LL << 30;    // n*top
constexpr int64_t kMaxElems = 1LL << 40;       // n*k, m*k/256*144, n*m, n*m*k/32

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 0 = not yet checked, 1 = gfx950, 2 = something else.
std::atomic<int> g_device_ok[64];

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return MMQ_ERR_DEVICE;
    }
    if (dev < 64) {
        const int known = g_device_ok[dev].load(std::memory_order_relaxed);
        if (known == 1) return MMQ_OK;
        if (known == 2) return MMQ_ERR_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
        (void)hipGetLastError();
        return MMQ_ERR_DEVICE;
    }
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) g_device_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? MMQ_OK : MMQ_ERR_DEVICE;
}

// Shared checks of the MMQ calls (before any HIP call); block_bytes is the
// weight format's super-block size (144 for q4_K, 210 for q6_K).
int check_mmq(const void* w, int64_t m, int64_t k, const int8_t* q, int64_t n, const void* out,
              bool* empty, int64_t block_bytes = 144) {
    if (n < 0 || m < 0 || k <= 0 || (k & 255) != 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim || m > kMaxDim || k > kMaxK) return MMQ_ERR_OVERFLOW;
    if (n * k >= kMaxElems || m * (k / 256) * block_bytes >= kMaxElems || n * m >= kMaxElems)
        return MMQ_ERR_OVERFLOW;
    *empty = (n == 0 || m == 0);
    if (*empty) return MMQ_OK;
    if (!w || !q || !out) return MMQ_ERR_NULL;
    if (!aligned16(w) || !aligned16(q) || !aligned16(out)) return MMQ_ERR_ALIGN;
    return MMQ_OK;
}

using FoldLaunch = hipError_t (*)(const uint8_t*, int, int, const int8_t*, const uint32_t*, int, const mmq::Out&,
                                  hipStream_t);

// HIP takes at most 2^32 - 1 work-items per grid dimension.
bool threads_ok(int64_t blocks, int64_t per_block) { return blocks * per_block < (1LL << 32); }

// Kernel behind the q4_K fold entry points for MMQ_KERNEL_AUTO, by token
// count and shape.  Set from timing sweeps of every kernel at 1-64 tokens
// over 22 matrices from 1024 x 4096 to 32768 x 4096, 28672 x 8192 and
// 8192 x 28672 (weights streamed from HBM; 478 cases): against the fastest
// named kernel per case the choice loses 0.18% in the geometric mean, 8.4% at
// most.
//   dot4 (1-2 tokens, and 5 unless the narrow kernel has long rows): its
//     workgroups of 16 rows fill the chip from about 10240 rows (8192 with
//     rows of >= 64 super-blocks), and its waves split a row's super-blocks
//     in 4-block steps, so it needs a multiple of 16 super-blocks: on
//     4096-row matrices the narrow kernel is 2-86% faster, on 13824 x 5120
//     (20 super-blocks) 23-51%;
//   stream (3-4 and 6-16 tokens): where it fits (at least 7 x 256 tiles of 8
//     rows, k <= 8192) and k is whole token phases (it computes every step
//     of the last one: 16 super-blocks up to 8 tokens, 8 above; 24576 x 6144
//     at 3-8 tokens is 8-18% slower than the narrow kernel); up to 8 tokens
//     with 7 or 8 waves per workgroup (5-6 waves, from 9-12 tiles per
//     workgroup, leave SIMDs idle: 20480 x 4096 5-13% behind), above 8
//     where k > 4096 or a workgroup holds at least 14 tiles (one phase is
//     paid back only over many rows: 14336 x 4096 at 9-16 tokens 8-24%
//     behind the few-token kernel); and at 9-12 tokens on rows of at least
//     64 super-blocks whatever the row count (6144 x 16384, 6144 x 28672 and
//     8160 x 28672: 24.2 / 39.6 / 39.1 us against 27.3 / 44.3 / 45.2 us for
//     the few-token kernel; at 13-16 tokens, or on rows of 32 super-blocks,
//     the few-token kernel leads):
//     28672 x 8192 at 4 / 7 / 12 / 16 tokens 25.9 / 30.9 / 39.3 / 45.1 us
//     against 28.3 / 34.5 / 45.1 / 47.9 us for the next kernel;
//   narrow (elsewhere up to 8 tokens; 9-16 where its 32-row tiles give each
//     wave at least 11 super-blocks, or on at most 4096 rows; 8192 x 22528,
//     11 per wave, at 12 tokens 28.9 us against 32.1 us for the stream kernel): 8192 x 28672
//     at 4 / 12 tokens 26.1 / 37.6 us against 28.7 / 45.8 us; 4096 x 14336
//     at 1 / 12 tokens 8.2 / 13.6 us against 11.4 / 20.4 us;
//   few-token int8-MFMA kernels (9-64 tokens otherwise): 11008 x 4096 at 12
//     tokens 10.1 us against 12.5 us for the stream kernel;
//   binary16-MFMA kernel: at 17-32 tokens where its 64-token tiles fill
//     224-255 CUs in one round (28672 rows: 67.1-68.4 us against 70.2-78.5
//     us; 24576 rows, 192 tiles, 8-10% behind; with 256 or more row tiles it
//     takes 128-token tiles and loses), at
//     33-64 tokens from 160 tiles (90.4 against 68.4 us at 33 tokens on
//     28672 x 8192), and above 64 tokens.
int q4k_auto_kernel(int64_t m, int64_t k, int64_t n) {
    const int64_t S = k >> 8;
    const int64_t f16_tiles = ((m + 127) / 128) * ((n + 127) / 128);
    const int w32 = mmq::narrow_waves32(m, k);
    const bool narrow_long = w32 > 0 && S / w32 >= 11;
    // the stream kernel's tiles per workgroup and its waves (two tiles each above 8)
    const int64_t tg = std::min<int64_t>(16, ((m + 7) / 8 + 255) / 256), tq = tg > 8 ? (tg + 1) / 2 : tg;
    const bool stream = mmq::stream_fits(m, k) && S % 16 == 0 && tq >= 7;               // up to 8 tokens
    const bool stream16 = mmq::stream_fits(m, k) && S % 8 == 0 && (S > 16 || tg >= 14);  // 9-16 tokens
    const bool stream12 = stream16 || (S % 8 == 0 && S >= 64);                           // 9-12 tokens
    const bool dot4 = S % 16 == 0 && (m >= 10240 || (m >= 8192 && S >= 64));
    if (n <= 2) return dot4 ? MMQ_KERNEL_DOT4 : MMQ_KERNEL_NARROW;
    if (n <= 4) return stream ? MMQ_KERNEL_STREAM : MMQ_KERNEL_NARROW;
    if (n <= 5) return dot4 && !narrow_long ? MMQ_KERNEL_DOT4 : MMQ_KERNEL_NARROW;
    if (n <= 8) return stream ? MMQ_KERNEL_STREAM : MMQ_KERNEL_NARROW;
    if (n <= mmq::kNarrowMaxN)
        return narrow_long || m <= 4096                  ? MMQ_KERNEL_NARROW
               : stream16 || (n <= 12 && stream12)       ? MMQ_KERNEL_STREAM
                                                         : MMQ_KERNEL_FEW;
    if (n <= 32) return f16_tiles >= 224 && f16_tiles < 256 ? MMQ_KERNEL_F16 : MMQ_KERNEL_FEW;
    if (n <= mmq::kSmallMaxN) return f16_tiles >= 160 ? MMQ_KERNEL_F16 : MMQ_KERNEL_FEW;
    return MMQ_KERNEL_F16;
}

// The repacked-weight entry: above 16 tokens the binary16-MFMA kernel on the
// records, where it has tiles enough for the CUs (>= 160 of 128 x 128) or the
// slices would be many (> 40 tokens); otherwise the dot4 kernel, in slices of
// 8 tokens.  Measured per call: 28672 x 8192 (224 tiles) at 9 / 16 / 24
// tokens 60 / 76 / 121 us in slices against 75 us; 8192 x 28672 (64 tiles)
// at 33 / 48 tokens 197 / 273 us in slices against 221 us.
int q4kr_auto_kernel(int64_t m, int64_t n) {
    const int64_t f16_tiles = ((m + 127) / 128) * ((n + 127) / 128);
    return n > 16 && (f16_tiles >= 160 || n > 40) ? MMQ_KERNEL_F16 : MMQ_KERNEL_DOT4;
}

// The launcher of a q4_K fold kernel choice, and whether its grid fits.
int q4k_fold_launcher(int kernel, int64_t m, int64_t k, int64_t n, FoldLaunch* f) {
    if (kernel == MMQ_KERNEL_AUTO) kernel = q4k_auto_kernel(m, k, n);
    switch (kernel) {
        case MMQ_KERNEL_DOT4:
            if (n > mmq::kGemvMaxN) return MMQ_ERR_KERNEL;
            *f = mmq::launch_mmq_fp32_gemv;
            return threads_ok((m + 15) / 16, 256) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_FEW:
            if (n > mmq::kSmallMaxN) return MMQ_ERR_KERNEL;
            *f = mmq::launch_mmq_fp32_small;
            return threads_ok((m + 15) / 16, 512) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_F16:
            *f = mmq::launch_mmq_fp32_f16;
            return threads_ok((m + 127) / 128 * ((n + 63) / 64), 1024) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_I8:
            *f = mmq::launch_mmq_fp32;
            return threads_ok((m + 127) / 128 * ((n + 127) / 128), 256) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_NARROW:
            if (n > mmq::kNarrowMaxN) return MMQ_ERR_KERNEL;
            *f = mmq::launch_mmq_fp32_narrow;
            return threads_ok((m + 15) / 16, 512) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_STREAM:
            if (n > mmq::kStreamMaxN) return MMQ_ERR_KERNEL;
            *f = mmq::launch_mmq_fp32_stream;
            return threads_ok((m + 7) / 8, 512) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        default:
            return MMQ_ERR_KERNEL;
    }
}

int hip_status(hipError_t e) {
    if (e == hipSuccess) return MMQ_OK;
    (void)hipGetLastError();
    return MMQ_ERR_HIP;
}

// The q4_K fold entry points: same checks, same kernels, float32 or binary16
// stores of the same float32 result, or its epilogue.
int fold_entry(const void* w, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds, int64_t n,
               const mmq::Out& out, int kernel, hipStream_t stream) {
    bool empty = false;
    int rc = check_mmq(w, m, k, q, n, out.epi.p, &empty);
    if (rc != MMQ_OK || empty) return rc;
    if (!ds) return MMQ_ERR_NULL;
    if (!aligned16(ds)) return MMQ_ERR_ALIGN;
    FoldLaunch launch = nullptr;
    rc = q4k_fold_launcher(kernel, m, k, n, &launch);
    if (rc != MMQ_OK) return rc;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    return hip_status(launch(static_cast<const uint8_t*>(w), (int)m, (int)k, q, ds, (int)n, out, stream));
}

// The fold entry points on q8 operand tiles: always the binary16-MFMA kernel
// (the tiles are its operand layout), on q4_K rows or repacked records.
int tiles_fold_entry(const void* w, bool repacked, int64_t m, int64_t k, const uint16_t* qt,
                     const uint32_t* ds, int64_t n, const mmq::Out& out, hipStream_t stream) {
    bool empty = false;
    int rc = check_mmq(w, m, k, reinterpret_cast<const int8_t*>(qt), n, out.epi.p, &empty);
    if (rc != MMQ_OK || empty) return rc;
    if (n > kMaxDim - 127 || (n + 127) / 128 * 128 * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (repacked && (m + 15) / 16 * (k / 256) * mmq::kRepackRecordBytes >= kMaxElems)
        return MMQ_ERR_OVERFLOW;
    if (!threads_ok((m + 127) / 128 * ((n + 63) / 64), 1024)) return MMQ_ERR_OVERFLOW;
    if (!ds) return MMQ_ERR_NULL;
    if (!aligned16(ds)) return MMQ_ERR_ALIGN;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    return hip_status(mmq::launch_mmq_fp32_f16_tiles(static_cast<const uint8_t*>(w), repacked, (int)m,
                                                     (int)k, qt, ds, (int)n, out, stream));
}

// Kernel behind the q6_K fold entry points for MMQ_KERNEL_AUTO: the
// vector-ALU dot4 kernel for n <= 8, the binary16-MFMA kernel above.
int q6k_auto_kernel(int64_t n) { return n <= mmq::kQ6kGemvMaxN ? MMQ_KERNEL_DOT4 : MMQ_KERNEL_F16; }

int q6k_fold_launcher(int kernel, int64_t m, int64_t n, FoldLaunch* f) {
    if (kernel == MMQ_KERNEL_AUTO) kernel = q6k_auto_kernel(n);
    switch (kernel) {
        case MMQ_KERNEL_DOT4:
            if (n > mmq::kQ6kGemvMaxN) return MMQ_ERR_KERNEL;
            *f = mmq::launch_q6k_gemv;
            return threads_ok((m + 15) / 16, 256) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_F16:
            *f = mmq::launch_q6k_f16;
            return threads_ok((m + 127) / 128 * ((n + 127) / 128), 1024) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        case MMQ_KERNEL_I8:
            *f = mmq::launch_q6k_i8;
            return threads_ok((m + 127) / 128 * ((n + 127) / 128), 256) ? MMQ_OK : MMQ_ERR_OVERFLOW;
        default:
            return MMQ_ERR_KERNEL;
    }
}

// Where a q6_K call with an epilogue runs kernels of its own (launch_q6k_few,
// launch_q6k_stream): from 9 tokens, while there are few tiles of 16 rows x 64
// tokens for the binary16 kernel's 128 x 128 ones to fill the chip.  Streaming
// against binary16, us: 4096 x 11008 at 128 / 256 / 512 tokens (512 / 1024 /
// 2048 tiles) 62 / 113 / 204 and 235 / 228 / 223; 4096 x 4096 at 128 / 384 / 512
// (512 / 1536 / 2048) 28 / 78 / 84 and 81 / 78 / 78; 8192 x 4096 at 128 / 192 /
// 320 (1024 / 1536 / 2560) 46 / 78 / 120 and 81 / 79 / 79.
// Their offsets into q are 32 bits.
bool q6k_epilogue_own(int64_t m, int64_t k, int64_t n) {
    return n > mmq::kQ6kGemvMaxN &&
           (n <= mmq::kQ6kFewMaxN || ((m + 15) / 16 * ((n + 63) / 64) <= 1536 && n * k < (1LL << 32)));
}

int q6k_fold_entry(const void* w, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds,
                   int64_t n, const mmq::Out& out, int kernel, hipStream_t stream) {
    bool empty = false;
    int rc = check_mmq(w, m, k, q, n, out.epi.p, &empty, mmq::kQ6kBlockBytes);
    if (rc != MMQ_OK || empty) return rc;
    if (!ds) return MMQ_ERR_NULL;
    if (!aligned16(ds)) return MMQ_ERR_ALIGN;
    if (out.kind == mmq::kOutEpi && q6k_epilogue_own(m, k, n)) {
        if (!threads_ok((m + 15) / 16, 512)) return MMQ_ERR_OVERFLOW;
        rc = check_device();
        if (rc != MMQ_OK) return rc;
        const auto own = m <= mmq::kQ6kFewMaxM && n <= mmq::kQ6kFewMaxN ? mmq::launch_q6k_few : mmq::launch_q6k_stream;
        return hip_status(own(static_cast<const uint8_t*>(w), (int)m, (int)k, q, ds, (int)n, out.epi, stream));
    }
    FoldLaunch launch = nullptr;
    rc = q6k_fold_launcher(kernel, m, n, &launch);
    if (rc != MMQ_OK) return rc;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    return hip_status(launch(static_cast<const uint8_t*>(w), (int)m, (int)k, q, ds, (int)n, out, stream));
}

// The fold entry points on repacked records.
int repacked_fold_entry(const void* wr, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds, int64_t n,
                        const mmq::Out& out, hipStream_t stream) {
    bool empty = false;
    int rc = check_mmq(wr, m, k, q, n, out.epi.p, &empty);
    if (rc != MMQ_OK || empty) return rc;
    if ((m + 15) / 16 * (k / 256) * mmq::kRepackRecordBytes >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!ds) return MMQ_ERR_NULL;
    if (!aligned16(ds)) return MMQ_ERR_ALIGN;
    const bool f16 = q4kr_auto_kernel(m, n) == MMQ_KERNEL_F16;
    if (f16 ? !threads_ok((m + 127) / 128 * ((n + 63) / 64), 1024) : !threads_ok((m + 15) / 16, 256))
        return MMQ_ERR_OVERFLOW;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    if (f16)
        return hip_status(mmq::launch_mmq_fp32_f16_repacked(static_cast<const uint8_t*>(wr), (int)m, (int)k,
                                                            q, ds, (int)n, out, stream));
    // Up to 8 tokens per launch; more tokens run as slices of 8 (each reads
    // the weights again: this layout serves the few-token path).  Slice
    // starts stay 16-byte aligned: 8 rows of q, ds and out are 8k, k/4 and
    // 32m bytes.
    mmq::Out part = out;
    for (int64_t t0 = 0; t0 < n; t0 += mmq::kGemvMaxN) {
        const int nn = (int)(n - t0 < mmq::kGemvMaxN ? n - t0 : mmq::kGemvMaxN);
        rc = hip_status(mmq::launch_mmq_fp32_gemv_repacked(
            static_cast<const uint8_t*>(wr), (int)m, (int)k, q + t0 * k, ds + t0 * (k / 32), nn,
            part, stream));
        if (rc != MMQ_OK) return rc;
        part.epi.advance(mmq::kGemvMaxN);
    }
    return MMQ_OK;
}

// The q6_K fold entry points on q8 operand tiles.
int q6k_tiles_fold_entry(const void* w, int64_t m, int64_t k, const uint16_t* qt,
                         const uint32_t* ds, int64_t n, const mmq::Out& out, hipStream_t stream) {
    bool empty = false;
    int rc = check_mmq(w, m, k, reinterpret_cast<const int8_t*>(qt), n, out.epi.p, &empty, mmq::kQ6kBlockBytes);
    if (rc != MMQ_OK || empty) return rc;
    if (n > kMaxDim - 127 || (n + 127) / 128 * 128 * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((m + 127) / 128 * ((n + 127) / 128), 1024)) return MMQ_ERR_OVERFLOW;
    if (!ds) return MMQ_ERR_NULL;
    if (!aligned16(ds)) return MMQ_ERR_ALIGN;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    return hip_status(mmq::launch_q6k_f16_tiles(static_cast<const uint8_t*>(w), (int)m, (int)k, qt, ds,
                                                (int)n, out, stream));
}

// ------------------------------------------------------------- epilogue
bool opt_aligned16(const void* p) { return !p || aligned16(p); }

// A row stride: 0 stands for m, less than m is an error.
int row_stride(int64_t given, int64_t m, int64_t rows, int64_t* stride) {
    *stride = given == 0 ? m : given;
    if (*stride < m) return MMQ_ERR_SHAPE;
    return *stride > kMaxElems || rows > kMaxElems / (*stride > 0 ? *stride : 1) ? MMQ_ERR_OVERFLOW : MMQ_OK;
}

// The output of an epilogue call; experts: how many bias rows.
int make_epilogue(const mmq_epilogue* e, void* out, int64_t m, int64_t rows, int64_t experts, mmq::Out* o) {
    if (!e) return MMQ_ERR_NULL;
    if (e->activation < MMQ_ACT_NONE || e->activation > MMQ_ACT_GELU_TANH) return MMQ_ERR_KERNEL;
    *o = mmq::Out{};
    o->kind = mmq::kOutEpi;
    o->epi.p = out;
    o->epi.bias = e->bias;
    o->epi.res = e->residual;
    o->epi.act = e->activation;
    o->epi.half = e->out_f16 != 0;
    o->epi.res_half = e->residual_f16 != 0;
    int rc = row_stride(e->out_stride, m, rows, &o->epi.stride);
    if (rc == MMQ_OK) rc = row_stride(e->residual ? e->residual_stride : 0, m, rows, &o->epi.res_stride);
    if (rc != MMQ_OK) return rc;
    if (!opt_aligned16(e->bias) || !opt_aligned16(e->residual)) return MMQ_ERR_ALIGN;
    o->epi.vec4 = (o->epi.stride & 3) == 0 && (!e->residual || (o->epi.res_stride & 3) == 0) &&
                  (!e->bias || experts == 1 || (m & 3) == 0);
    return MMQ_OK;
}

// -------------------------------------------------------------- grouped
// Experts run on the kernels that suit their slot counts, which only the
// device knows: each kernel is launched over the experts within its range,
// unless there are too few slots for any.
int grouped_entry(int format, const void* w, int64_t experts, int64_t m, int64_t k, const int8_t* q,
                  const uint32_t* ds, int64_t tokens, const int32_t* rows, const int32_t* offsets, int64_t slots,
                  const mmq_epilogue* epilogue, void* out, hipStream_t stream) {
    if (format != MMQ_FORMAT_Q4K && format != MMQ_FORMAT_Q6K) return MMQ_ERR_KERNEL;
    const bool q6k = format == MMQ_FORMAT_Q6K;
    const int64_t block = q6k ? mmq::kQ6kBlockBytes : mmq::kBlockBytes;
    if (experts <= 0 || tokens < 0 || slots < 0 || m < 0 || k <= 0 || (k & 255) != 0) return MMQ_ERR_SHAPE;
    if (experts > kMaxExperts || tokens > kMaxDim || slots > kMaxDim || m > kMaxDim || k > kMaxK)
        return MMQ_ERR_OVERFLOW;
    if (slots > 0 && (tokens == 0 || (!rows && tokens < slots))) return MMQ_ERR_SHAPE;
    if (tokens * k > 0xFFFFFFFFLL || m * (k / 256) * block >= kMaxElems / experts || slots * m >= kMaxElems)
        return MMQ_ERR_OVERFLOW;
    mmq::Out o;
    int rc = make_epilogue(epilogue, out, m, slots, experts, &o);
    if (rc != MMQ_OK) return rc;
    if (slots == 0 || m == 0) return MMQ_OK;
    if (!w || !q || !ds || !offsets || !out) return MMQ_ERR_NULL;
    if (!aligned16(w) || !aligned16(q) || !aligned16(ds) || !aligned16(offsets) || !opt_aligned16(rows) ||
        !aligned16(out))
        return MMQ_ERR_ALIGN;
    if (experts > 1 && (m * (k / 256) * block) % 16 != 0) return MMQ_ERR_ALIGN;   // every expert's first row
    // The kernels number their tiles (items times tiles of rows) in 32 bits, which
    // hold the most that the limits above leave.  An item of the four-tile few-token
    // form takes 64 slots, all but the last of an expert, and 16 rows: at most
    // slots*m / 2^10 + experts*m / 2^4 tiles, below 2^30 + 2^36 / 144 (a row has 144
    // bytes or more), and an item's last, partial tile of rows.  The one-tile form
    // runs for a mean below 16 slots only, with fewer than 2*experts items; the
    // binary16 kernels' tiles are 128 rows of 64 slots.
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    const uint8_t* wb = static_cast<const uint8_t*>(w);
    const int64_t mean = slots / experts;
    mmq::Groups g{offsets, rows, (int)experts, (int)slots, (int)tokens, 0, 0};
    // The launches, each over the experts with up to `most` slots that the one
    // before has not taken, until there can be none left.
    const auto take = [&](int64_t most) {
        g.lo = g.hi + 1;
        g.hi = (int)most;
        return g.lo <= slots;
    };
    // The few-token kernel's one-tile form is 2 to 18% faster than its other one
    // at 1 or 2 slots per expert and even at 16, where its launch is left out.
    if (mean < mmq::kGroupFewMaxTile && take(mmq::kGroupFewMaxTile))
        rc = hip_status(mmq::launch_few_grouped(q6k, wb, (int)m, (int)k, q, ds, g, o.epi, stream));
    if (rc == MMQ_OK && take(q6k ? mmq::kGroupFewMaxQ6k : mmq::kGroupFewMaxQ4k))
        rc = hip_status(mmq::launch_few_grouped(q6k, wb, (int)m, (int)k, q, ds, g, o.epi, stream));
    // q4_K's binary16 tiles of 64 tokens where the mean is below 96 slots, of 128
    // above (tiles of 64 / 128, us): 8 experts of 14336 x 4096 with 64 slots each
    // 159 / 254, 96: 266 / 263, 128: 281 / 274, 256: 518 / 469; 64 experts of 1536
    // x 4096 with ragged loads of 64 on average 175 / 252, of 96 267 / 271.
    if (rc == MMQ_OK && take(slots)) {
        if (q6k)
            rc = hip_status(mmq::launch_q6k_f16_grouped(wb, (int)m, (int)k, q, ds, g, o.epi, stream));
        else
            rc = hip_status(mmq::launch_f16_grouped(wb, (int)m, (int)k, q, ds, g, o.epi, mean < 96 ? 64 : 128, stream));
    }
    return rc;
}

// ----------------------------------------------------------------- norm
int norm_entry(const q8_norm* a, int64_t n, int64_t k, int8_t* q, uint16_t* qt, uint32_t* ds, bool codes, bool tiles,
               hipStream_t stream) {
    if (n < 0 || k <= 0 || (k & (tiles ? 255 : 31)) != 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim - 127 || k > kMaxK || (n + 127) / 128 * 128 * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((n + 127) / 128 * 128, 1024)) return MMQ_ERR_OVERFLOW;   // a workgroup per row
    if (n == 0) return MMQ_OK;
    if (!a || !a->x || !a->weight) return MMQ_ERR_NULL;
    if (codes && ((tiles ? (const void*)qt : (const void*)q) == nullptr || !ds)) return MMQ_ERR_NULL;
    if (!codes && !a->h) return MMQ_ERR_NULL;
    // the stream needs a place where it changes; without y it does not
    if (a->y ? !a->r : (a->r || a->y_weight || a->gate || a->residual_scale != 1.0f)) return MMQ_ERR_NULL;
    mmq::NormArgs v{};
    int rc = row_stride(a->x_stride, k, n, &v.x_stride);
    if (rc == MMQ_OK && a->y) rc = row_stride(a->y_stride, k, n, &v.y_stride);
    if (rc == MMQ_OK && a->y) rc = row_stride(a->r_stride, k, n, &v.r_stride);
    if (rc != MMQ_OK) return rc;
    if (a->gate && a->gate_stride != 0) {
        rc = row_stride(a->gate_stride, k, n, &v.gate_stride);
        if (rc != MMQ_OK) return rc;
    }
    if (!aligned16(a->x) || !opt_aligned16(a->y) || !opt_aligned16(a->y_weight) || !opt_aligned16(a->gate) ||
        !aligned16(a->weight) || !opt_aligned16(a->r) || !opt_aligned16(a->h) || !opt_aligned16(q) ||
        !opt_aligned16(qt) || !opt_aligned16(ds))
        return MMQ_ERR_ALIGN;
    // rows start on 16-byte boundaries
    if ((v.x_stride & 3) || (v.y_stride & (a->y_f16 ? 7 : 3)) || (v.r_stride & 3) || (v.gate_stride & 3))
        return MMQ_ERR_ALIGN;
    v.x = a->x;
    v.x_scale = a->residual_scale;
    v.y = a->y;
    v.y_f16 = a->y_f16 != 0;
    v.y_weight = a->y_weight;
    v.gate = a->gate;
    v.weight = a->weight;
    v.eps = a->eps;
    v.r = a->r;
    v.h = a->h;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_norm(v, (int)n, (int)k, q, qt, ds, stream));
}

}  // namespace

extern "C" {

int q8_quantize_rows(const float* x, int64_t n, int64_t k, int8_t* q, uint32_t* ds,
                     hipStream_t stream) {
    if (n < 0 || k <= 0 || (k & 31) != 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim || k > kMaxK || n * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!threads_ok(n * (k / 32) * 4, 1)) return MMQ_ERR_OVERFLOW;   // 4 lanes per 32-block
    if (n == 0) return MMQ_OK;
    if (!x || !q || !ds) return MMQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(ds)) return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_q8_quantize(x, n * (k / 32), q, ds, stream));
}

int q8_quantize_rows_tiled(const float* x, int64_t n, int64_t k, uint16_t* qt, uint32_t* ds,
                           hipStream_t stream) {
    if (n < 0 || k <= 0 || (k & 255) != 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim - 127 || k > kMaxK || (n + 127) / 128 * 128 * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((n + 127) / 128 * 128 * (k / 32) * 4, 1)) return MMQ_ERR_OVERFLOW;   // 4 lanes per 32-block
    if (n == 0) return MMQ_OK;
    if (!x || !qt || !ds) return MMQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(qt) || !aligned16(ds)) return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_q8_quantize_tiled(x, (int)n, (int)k, qt, ds, stream));
}

int q8_quantize_silu_mul(const float* gate, const float* up, int64_t n, int64_t k, int8_t* q,
                         uint32_t* ds, hipStream_t stream) {
    if (n < 0 || k <= 0 || (k & 31) != 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim || k > kMaxK || n * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!threads_ok(n * (k / 32) * 4, 1)) return MMQ_ERR_OVERFLOW;
    if (n == 0) return MMQ_OK;
    if (!gate || !up || !q || !ds) return MMQ_ERR_NULL;
    if (!aligned16(gate) || !aligned16(up) || !aligned16(q) || !aligned16(ds)) return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_q8_quantize_silu_mul(gate, up, n * (k / 32), q, ds, stream));
}

int q8_quantize_silu_mul_tiled(const float* gate, const float* up, int64_t n, int64_t k, uint16_t* qt,
                               uint32_t* ds, hipStream_t stream) {
    if (n < 0 || k <= 0 || (k & 255) != 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim - 127 || k > kMaxK || (n + 127) / 128 * 128 * k >= kMaxElems) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((n + 127) / 128 * 128 * (k / 32) * 4, 1)) return MMQ_ERR_OVERFLOW;   // 4 lanes per 32-block
    if (n == 0) return MMQ_OK;
    if (!gate || !up || !qt || !ds) return MMQ_ERR_NULL;
    if (!aligned16(gate) || !aligned16(up) || !aligned16(qt) || !aligned16(ds)) return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_q8_quantize_silu_mul_tiled(gate, up, (int)n, (int)k, qt, ds, stream));
}

int mmq_q4k_q8(const void* w, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds,
               int64_t n, int32_t* dots, hipStream_t stream) {
    (void)ds;  // not read: the block dots do not depend on the scales
    bool empty = false;
    int rc = check_mmq(w, m, k, q, n, dots, &empty);
    if (rc != MMQ_OK || empty) return rc;
    if (n * m >= kMaxElems / (k / 32)) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((m + 127) / 128 * ((n + 127) / 128), 256)) return MMQ_ERR_OVERFLOW;
    if (ds && !aligned16(ds)) return MMQ_ERR_ALIGN;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    return hip_status(mmq::launch_mmq_dots(static_cast<const uint8_t*>(w), (int)m, (int)k, q,
                                           (int)n, dots, stream));
}

int mmq_q4k_q8_fp32out(const void* w, int64_t m, int64_t k, const int8_t* q,
                       const uint32_t* ds, int64_t n, float* out, hipStream_t stream) {
    return fold_entry(w, m, k, q, ds, n, mmq::Out::plain(out, m, false), MMQ_KERNEL_AUTO, stream);
}

int mmq_q4k_q8_f16out(const void* w, int64_t m, int64_t k, const int8_t* q,
                      const uint32_t* ds, int64_t n, uint16_t* out, hipStream_t stream) {
    return fold_entry(w, m, k, q, ds, n, mmq::Out::plain(out, m, true), MMQ_KERNEL_AUTO, stream);
}

int mmq_q4k_q8_fold(const void* w, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds, int64_t n,
                    void* out, int out_f16, int kernel, hipStream_t stream) {
    return fold_entry(w, m, k, q, ds, n, mmq::Out::plain(out, m, out_f16 != 0), kernel, stream);
}

int mmq_q6k_q8(const void* w, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds,
               int64_t n, int32_t* dots, hipStream_t stream) {
    (void)ds;  // not read: the group dots do not depend on the scales
    bool empty = false;
    int rc = check_mmq(w, m, k, q, n, dots, &empty, mmq::kQ6kBlockBytes);
    if (rc != MMQ_OK || empty) return rc;
    if (n * m >= kMaxElems / (k / 16)) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((m + 127) / 128 * ((n + 127) / 128), 256)) return MMQ_ERR_OVERFLOW;
    if (ds && !aligned16(ds)) return MMQ_ERR_ALIGN;
    rc = check_device();
    if (rc != MMQ_OK) return rc;
    return hip_status(mmq::launch_q6k_dots(static_cast<const uint8_t*>(w), (int)m, (int)k, q,
                                           (int)n, dots, stream));
}

int mmq_q6k_q8_fp32out(const void* w, int64_t m, int64_t k, const int8_t* q,
                       const uint32_t* ds, int64_t n, float* out, hipStream_t stream) {
    return q6k_fold_entry(w, m, k, q, ds, n, mmq::Out::plain(out, m, false), MMQ_KERNEL_AUTO, stream);
}

int mmq_q6k_q8_f16out(const void* w, int64_t m, int64_t k, const int8_t* q,
                      const uint32_t* ds, int64_t n, uint16_t* out, hipStream_t stream) {
    return q6k_fold_entry(w, m, k, q, ds, n, mmq::Out::plain(out, m, true), MMQ_KERNEL_AUTO, stream);
}

int mmq_q6k_q8_fold(const void* w, int64_t m, int64_t k, const int8_t* q, const uint32_t* ds, int64_t n,
                    void* out, int out_f16, int kernel, hipStream_t stream) {
    return q6k_fold_entry(w, m, k, q, ds, n, mmq::Out::plain(out, m, out_f16 != 0), kernel, stream);
}

int mmq_kernel_choice(int format, int64_t m, int64_t k, int64_t n) {
    if (n < 0 || m < 0 || k <= 0 || (k & 255) != 0) return MMQ_ERR_SHAPE;
    switch (format) {
        case MMQ_FORMAT_Q4K: return q4k_auto_kernel(m, k, n);
        case MMQ_FORMAT_Q4K_REPACKED: return q4kr_auto_kernel(m, n);
        case MMQ_FORMAT_Q6K: return q6k_auto_kernel(n);
        case MMQ_FORMAT_Q4K_TILES:
        case MMQ_FORMAT_Q4K_REPACKED_TILES:
        case MMQ_FORMAT_Q6K_TILES: return MMQ_KERNEL_F16;
        default: return MMQ_ERR_KERNEL;
    }
}

int q4k_repack(const void* w, int64_t m, int64_t k, void* wr, hipStream_t stream) {
    if (m < 0 || k <= 0 || (k & 255) != 0) return MMQ_ERR_SHAPE;
    if (m > kMaxDim || k > kMaxK) return MMQ_ERR_OVERFLOW;
    if (m * (k / 256) * 144 >= kMaxElems || (m + 15) / 16 * (k / 256) * mmq::kRepackRecordBytes >= kMaxElems)
        return MMQ_ERR_OVERFLOW;
    if (!threads_ok((m + 15) / 16 * (k / 256), 64)) return MMQ_ERR_OVERFLOW;   // 64 lanes per record
    if (m == 0) return MMQ_OK;
    if (!w || !wr) return MMQ_ERR_NULL;
    if (!aligned16(w) || !aligned16(wr)) return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_q4k_repack(static_cast<const uint8_t*>(w), (int)m, (int)k,
                                             static_cast<uint8_t*>(wr), stream));
}

int mmq_q4kr_q8_fp32out(const void* wr, int64_t m, int64_t k, const int8_t* q,
                        const uint32_t* ds, int64_t n, float* out, hipStream_t stream) {
    return repacked_fold_entry(wr, m, k, q, ds, n, mmq::Out::plain(out, m, false), stream);
}

int mmq_q4k_q8t_fp32out(const void* w, int64_t m, int64_t k, const uint16_t* qt,
                        const uint32_t* ds, int64_t n, float* out, hipStream_t stream) {
    return tiles_fold_entry(w, false, m, k, qt, ds, n, mmq::Out::plain(out, m, false), stream);
}

int mmq_q4kr_q8t_fp32out(const void* wr, int64_t m, int64_t k, const uint16_t* qt,
                         const uint32_t* ds, int64_t n, float* out, hipStream_t stream) {
    return tiles_fold_entry(wr, true, m, k, qt, ds, n, mmq::Out::plain(out, m, false), stream);
}

int mmq_q6k_q8t_fp32out(const void* w, int64_t m, int64_t k, const uint16_t* qt,
                        const uint32_t* ds, int64_t n, float* out, hipStream_t stream) {
    return q6k_tiles_fold_entry(w, m, k, qt, ds, n, mmq::Out::plain(out, m, false), stream);
}

int q8_quantize_norm(const q8_norm* a, int64_t n, int64_t k, int8_t* q, uint32_t* ds, hipStream_t stream) {
    return norm_entry(a, n, k, q, nullptr, ds, true, false, stream);
}

int q8_quantize_norm_tiled(const q8_norm* a, int64_t n, int64_t k, uint16_t* qt, uint32_t* ds, hipStream_t stream) {
    return norm_entry(a, n, k, nullptr, qt, ds, true, true, stream);
}

int residual_norm(const q8_norm* a, int64_t n, int64_t k, hipStream_t stream) {
    return norm_entry(a, n, k, nullptr, nullptr, nullptr, false, false, stream);
}

int mmq_fold_epilogue(int format, const void* w, int64_t m, int64_t k, const void* q, const uint32_t* ds, int64_t n,
                      const mmq_epilogue* epilogue, void* out, hipStream_t stream) {
    if (n < 0 || m < 0) return MMQ_ERR_SHAPE;
    if (n > kMaxDim || m > kMaxDim) return MMQ_ERR_OVERFLOW;
    mmq::Out o;
    const int rc = make_epilogue(epilogue, out, m, n, 1, &o);
    if (rc != MMQ_OK) return rc;
    const int8_t* codes = static_cast<const int8_t*>(q);
    const uint16_t* tiles = static_cast<const uint16_t*>(q);
    switch (format) {
        case MMQ_FORMAT_Q4K: return fold_entry(w, m, k, codes, ds, n, o, MMQ_KERNEL_AUTO, stream);
        case MMQ_FORMAT_Q4K_REPACKED: return repacked_fold_entry(w, m, k, codes, ds, n, o, stream);
        case MMQ_FORMAT_Q6K: return q6k_fold_entry(w, m, k, codes, ds, n, o, MMQ_KERNEL_AUTO, stream);
        case MMQ_FORMAT_Q4K_TILES: return tiles_fold_entry(w, false, m, k, tiles, ds, n, o, stream);
        case MMQ_FORMAT_Q4K_REPACKED_TILES: return tiles_fold_entry(w, true, m, k, tiles, ds, n, o, stream);
        case MMQ_FORMAT_Q6K_TILES: return q6k_tiles_fold_entry(w, m, k, tiles, ds, n, o, stream);
        default: return MMQ_ERR_KERNEL;
    }
}

int mmq_fold_grouped(int format, const void* w, int64_t experts, int64_t m, int64_t k, const int8_t* q,
                     const uint32_t* ds, int64_t tokens, const int32_t* rows, const int32_t* offsets, int64_t slots,
                     const mmq_epilogue* epilogue, void* out, hipStream_t stream) {
    return grouped_entry(format, w, experts, m, k, q, ds, tokens, rows, offsets, slots, epilogue, out, stream);
}

int moe_route(const float* logits, int64_t n, int64_t experts, int64_t stride, int top, int normalize, float scale,
              int32_t* ids, float* weights, int32_t* slot, int32_t* rows, int32_t* offsets, hipStream_t stream) {
    if (n < 0 || experts <= 0 || top <= 0 || top > experts) return MMQ_ERR_SHAPE;
    if (experts > mmq::kRouteMaxExperts || top > mmq::kRouteMaxTop) return MMQ_ERR_OVERFLOW;
    int64_t s = 0;
    const int rc = row_stride(stride, experts, n, &s);
    if (rc != MMQ_OK) return rc;
    if (n > kMaxDim || n * top > kMaxRouteIds) return MMQ_ERR_OVERFLOW;
    if (!threads_ok((n + mmq::kTopkWaves - 1) / mmq::kTopkWaves, 64 * mmq::kTopkWaves)) return MMQ_ERR_OVERFLOW;
    if (n == 0) return MMQ_OK;
    if (!logits || !ids || !weights || !slot || !rows || !offsets) return MMQ_ERR_NULL;
    if (!aligned16(logits) || !aligned16(ids) || !aligned16(weights) || !aligned16(slot) || !aligned16(rows) ||
        !aligned16(offsets))
        return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_route(logits, s, (int)n, (int)experts, top, normalize != 0, scale, ids, weights, slot,
                                        rows, offsets, stream));
}

int moe_combine(const void* y, int y_f16, int64_t slots, int64_t m, const int32_t* slot, const float* weights,
                int64_t n, int top, const float* residual, float* out, hipStream_t stream) {
    if (slots < 0 || n < 0 || m < 0 || top <= 0) return MMQ_ERR_SHAPE;
    if (slots > kMaxDim || n > kMaxDim || m > kMaxDim || top > mmq::kRouteMaxTop) return MMQ_ERR_OVERFLOW;
    if (slots * m >= kMaxElems || n * m >= kMaxElems || n * top > kMaxRouteIds) return MMQ_ERR_OVERFLOW;
    if (!threads_ok(n * mmq::combine_cols(y_f16 != 0, m), 256)) return MMQ_ERR_OVERFLOW;
    if (n == 0 || m == 0) return MMQ_OK;
    if ((slots > 0 && !y) || !slot || !weights || !out) return MMQ_ERR_NULL;
    if (!opt_aligned16(y) || !aligned16(slot) || !aligned16(weights) || !opt_aligned16(residual) || !aligned16(out))
        return MMQ_ERR_ALIGN;
    const int dev = check_device();
    if (dev != MMQ_OK) return dev;
    return hip_status(mmq::launch_combine(y, y_f16 != 0, slots, (int)m, slot, weights, (int)n, top, residual, out,
                                          stream));
}

const char* mmq_status_string(int status) {
    switch (status) {
        case MMQ_OK: return "MMQ_OK";
        case MMQ_ERR_NULL: return "MMQ_ERR_NULL: a required pointer is NULL";
        case MMQ_ERR_SHAPE: return "MMQ_ERR_SHAPE: invalid size (negative, k == 0, or k not a multiple of 32/256)";
        case MMQ_ERR_ALIGN: return "MMQ_ERR_ALIGN: a pointer is not 16-byte aligned";
        case MMQ_ERR_OVERFLOW: return "MMQ_ERR_OVERFLOW: size beyond the kernels' index range";
        case MMQ_ERR_DEVICE: return "MMQ_ERR_DEVICE: no HIP device, or the current device is not gfx950";
        case MMQ_ERR_HIP: return "MMQ_ERR_HIP: the HIP runtime reported a launch error";
        case MMQ_ERR_KERNEL: return "MMQ_ERR_KERNEL: unknown kernel, format or activation, or a kernel outside its token range";
        default: return "unknown mmq status";
    }
}

}  // extern "C"
