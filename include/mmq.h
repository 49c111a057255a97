/*
 * mmq.h - C ABI of the q4_K x q8 quantized matrix multiply (MMQ) for MI355X.
 *
 * The operation (the yusiwen.cn "minfer" pages: r31 "q-major sda scale-read
 * repack", sections 1 and 2, and r22 "qa8 XOR swizzle"): LLM prefill
 * multiplies a weight matrix W[m x k], stored as 4-bit k-quant (q4_K)
 * super-blocks, by activations X[n x k] that are quantized per token and per
 * 32-element block to int8 with a per-block scale word.  Each 32-element
 * chunk is an exact integer dot product, rescaled by the two-term rank-1 fold
 *
 *   out[t][o] = sum_c (d*sc)[o,c]*da[t,c]*D[t][o][c] - (dmin*m)[o,c]*da[t,c]*ssum[t,c]
 *   D[t][o][c] = sum_{i<32} q4[o][32c+i] * q8[t][32c+i]
 *
 * Data formats
 *   q4_K weights: m rows, each row k/256 super-blocks of 144 bytes, rows
 *     contiguous (row o's super-block b at byte (o*(k/256) + b)*144).  Block:
 *     d (binary16) at 0, dmin (binary16) at 2, twelve bytes of 6-bit (sc, m)
 *     pairs at 4 (GGUF k-quant packing), 128 bytes of nibbles at 16: weight
 *     64p+i is the low nibble of byte 32p+i, weight 64p+32+i its high nibble.
 *   q8 activations: q int8 [n][k] row-major and one 32-bit scale word per
 *     (token, 32-element block), ds uint32 [n][k/32]: binary16 da in the low
 *     16 bits, ssum = sum of the block's 32 q values as a two's-complement
 *     16-bit integer in the high 16 bits (r31 page, section 3.2).
 *
 * Conventions for every call
 *   - All array pointers are DEVICE pointers, allocated and owned by the
 *     caller; the library allocates nothing, keeps no pointer after
 *     returning, and keeps no global state other than a per-device
 *     "is this a gfx950" check.  Calls are reentrant.
 *   - Work is enqueued asynchronously on `stream` (NULL = the default
 *     stream); the caller keeps every buffer alive until the stream has
 *     finished.  Output buffers must not overlap inputs.
 *   - Every pointer must be 16-byte aligned.
 *   - n or m equal to 0 is an empty call: it returns MMQ_OK and touches
 *     nothing (pointers may then be NULL).  Negative sizes are MMQ_ERR_SHAPE.
 *   - Argument errors are detected on the host before any HIP call and
 *     before anything is enqueued.  No call throws or aborts.
 *   - Inputs must be finite.
 */
#ifndef Q4Q8_MMQ_H
#define Q4Q8_MMQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t *hipStream_t;

enum mmq_status {
    MMQ_OK = 0,
    MMQ_ERR_NULL = -1,      /* a required pointer is NULL */
    MMQ_ERR_SHAPE = -2,     /* negative size, k not a multiple of 32 (quantize) or 256 (MMQ), k == 0 */
    MMQ_ERR_ALIGN = -3,     /* a pointer is not 16-byte aligned */
    MMQ_ERR_OVERFLOW = -4,  /* a size beyond the kernels' index range (see limits below) */
    MMQ_ERR_DEVICE = -5,    /* no HIP device, or the current device is not gfx950 */
    MMQ_ERR_HIP = -6,       /* the HIP runtime reported an error at launch */
    MMQ_ERR_KERNEL = -7     /* unknown kernel, format or activation id, or a kernel outside its token range */
};

/* Size limits (MMQ_ERR_OVERFLOW beyond them): n, m <= 2^31 - 1; k <= 2^24;
 * n*k and m*k/256*144 below 2^40; for mmq_q4k_q8 also n*m*(k/32) < 2^40;
 * and every launch the call makes below 2^32 work-items (HIP's grid limit):
 * for the quantizers n*k/8 (tiled: ceil(n/128)*128*k/8), for the matmuls
 * 1024 per tile of 128 rows x 64 tokens, 512 per 16 rows (few tokens). */

/*
 * q8_quantize_rows - per-token, per-32-element q8 quantization of activations.
 * (Workload definition of the q8 activations: da = max|x|/127, q = round(x/da),
 * ssum = sum q; packed scale word as in the r31 page, section 3.2.)
 *
 *   x   : float [n][k], row-major, k % 32 == 0.
 *   q   : int8 [n][k] (out).   q = round(x / da), fp32 division, ties away from
 *         zero, in [-127, 127]; da = fp32(max|x| / 127) of the block.
 *   ds  : uint32 [n][k/32] (out).  binary16(da) (round to nearest even,
 *         subnormals kept) | (uint16)ssum << 16.  An all-zero block gives
 *         q = 0 and ds = 0.
 */
int q8_quantize_rows(const float *x, int64_t n, int64_t k, int8_t *q, uint32_t *ds,
                     hipStream_t stream);

/*
 * q8_quantize_silu_mul - the q8 quantization of an FFN down projection's
 * input h = SiLU(gate) * up, without writing h.  (The pages' later
 * "quantize-transpose prepass", named on the r22 page, moved activation
 * quantization into a pass of its own; fusing the gate product into that
 * pass is this library's reading.)
 *
 *   gate, up : float [n][k] each, row-major, k % 32 == 0 (the gate and up
 *              projections' outputs).
 *   q, ds    : as for q8_quantize_rows, of
 *              h = float32( g*u / (1 + exp(-g)) ) evaluated in float64
 *              (g*u exact, IEEE add and divide, one rounding to float32).
 * The result equals q8_quantize_rows applied to that h.  Errors and empty
 * calls as for q8_quantize_rows.
 */
int q8_quantize_silu_mul(const float *gate, const float *up, int64_t n, int64_t k, int8_t *q,
                         uint32_t *ds, hipStream_t stream);

/*
 * mmq_q4k_q8 - exact per-block integer dot products (the int32 result of the
 * 32-deep integer contraction, before the two-term rescale; r31 page, section 1).
 *
 *   w    : q4_K super-blocks of W [m][k] (m*(k/256)*144 bytes), k % 256 == 0.
 *   q    : int8 [n][k] q8 activations.
 *   ds   : the activations' scale words; accepted for a signature uniform with
 *          mmq_q4k_q8_fp32out and not read (may be NULL).
 *   dots : int32 [n][m][k/32] (out), dots[t][o][c] = D[t][o][c], exact.
 * A parity/inspection entry: its output is 4*n*m*k/32 bytes.
 */
int mmq_q4k_q8(const void *w, int64_t m, int64_t k, const int8_t *q, const uint32_t *ds,
               int64_t n, int32_t *dots, hipStream_t stream);

/*
 * mmq_q4k_q8_fp32out - the quantized matmul with the two-term rank-1 fold
 * applied per 32-element chunk (r31 page, sections 1-2), float32 result.
 *
 *   w   : q4_K super-blocks of W [m][k], k % 256 == 0.
 *   q   : int8 [n][k];  ds : uint32 [n][k/32] (as written by q8_quantize_rows).
 *   out : float [n][m] (out), token-major: out[t][o].  The summation order is
 *         the kernel's; results agree with the exact value to float32
 *         rounding of the accumulation: relative L2 error <= 1e-5, and every
 *         element within 1e-3 of its token row's largest |value|, for every
 *         k accepted (no float32 sum runs over more than 256 super-blocks).
 */
int mmq_q4k_q8_fp32out(const void *w, int64_t m, int64_t k, const int8_t *q,
                       const uint32_t *ds, int64_t n, float *out, hipStream_t stream);

/*
 * mmq_q4k_q8_f16out - the same quantized matmul and fold as
 * mmq_q4k_q8_fp32out, stored as IEEE binary16: out[t][o] is the float32
 * result rounded to nearest-even (overflow to +-inf), halving the output
 * bytes.  The pages only name a binary16 step after the output store (the
 * r22 page's round index, "r23 - f16 wall decomposition"); a binary16 output
 * is this library's reading of it.
 *
 *   w, q, ds : as for mmq_q4k_q8_fp32out.
 *   out      : binary16 bit patterns [n][m] (out), token-major, 16-byte
 *              aligned.  For the same inputs and binary, out[t][o] equals the
 *              binary16 rounding of mmq_q4k_q8_fp32out's out[t][o] bit for bit.
 * Errors and empty calls as for mmq_q4k_q8_fp32out.
 */
int mmq_q4k_q8_f16out(const void *w, int64_t m, int64_t k, const int8_t *q,
                      const uint32_t *ds, int64_t n, uint16_t *out, hipStream_t stream);

/*
 * Kernels behind the fold entry points.  Every one computes the same exact
 * integer dots and the same fold; they differ in how the work maps onto the
 * chip, and each meets the same accuracy bar on every shape it accepts.
 */
enum mmq_kernel {
    MMQ_KERNEL_AUTO = 0,  /* the entry point's own choice, by m, k and n (mmq_kernel_choice) */
    MMQ_KERNEL_DOT4 = 1,  /* vector-ALU 4-way int8 dots, weights streamed once; n <= 8 */
    MMQ_KERNEL_FEW = 2,   /* int8 MFMA on 16-token tiles, weights streamed once; n <= 64 (q4_K) */
    MMQ_KERNEL_F16 = 3,   /* binary16 MFMA on exact sc*q4 and q8 operands, 128-row tiles; any n */
    MMQ_KERNEL_I8 = 4,    /* int8 MFMA on 128 x 128 tiles with a three-operation fold; any n */
    MMQ_KERNEL_NARROW = 5, /* int8 4x4x4 MFMA, weights staged through LDS, streamed once; n <= 16 */
    MMQ_KERNEL_STREAM = 6  /* the narrow kernel's arithmetic, tokens held in LDS per workgroup of many
                              row tiles, weights streamed in 576-byte runs; n <= 16 */
};

/*
 * mmq_q4k_q8_fold - mmq_q4k_q8_fp32out (out_f16 == 0) or mmq_q4k_q8_f16out
 * (out_f16 != 0) on a kernel the caller names, for comparisons, benchmarks
 * and validation of every kernel on any shape.  With MMQ_KERNEL_AUTO it is
 * exactly that entry point.  A kernel outside its token range (DOT4 above 8
 * tokens, NARROW and STREAM above 16, FEW above 64) or an unknown id returns MMQ_ERR_KERNEL before any
 * HIP call; other arguments, errors and empty calls as for
 * mmq_q4k_q8_fp32out.
 */
int mmq_q4k_q8_fold(const void *w, int64_t m, int64_t k, const int8_t *q, const uint32_t *ds,
                    int64_t n, void *out, int out_f16, int kernel, hipStream_t stream);

/*
 * q6_K weights: the second k-quant format, named in the r31 page's closing
 * notes (its "q6_K line" of rounds); the pages print no layout, and the
 * GGUF k-quant super-block is taken: 256 weights in 210 bytes, rows
 * contiguous (row o's super-block b at byte (o*(k/256) + b)*210, so blocks
 * are only 2-byte aligned).  Block: ql[128] at 0 (low nibbles), qh[64] at 128
 * (2-bit high parts), sixteen int8 scales at 192 (one per 16 weights),
 * binary16 d at 208.  Weight 128h + 32g + l (h < 2, g < 4, l < 32) has the
 * code q = (nibble g/2 of ql[64h + 32(g%2) + l]) | (bits 2g..2g+1 of
 * qh[32h + l]) << 4 and the value d*sc[(128h + 32g + l)/16]*(q - 32).  The
 * same q8 activations as above.  There is no min term: with G = k/16 groups,
 *
 *   out[t][o] = sum_g d[o]*sc[o,g]*da[t,g/2]*D[t][o][g]
 *   D[t][o][g] = sum_{i<16} (q[o][16g+i] - 32) * q8[t][16g+i]
 *
 * Limits, errors, alignment (of w itself) and empty calls as above, with
 * m*(k/256)*210 below 2^40 and, for mmq_q6k_q8, n*m*(k/16) below 2^40.
 */

/*
 * mmq_q6k_q8 - exact per-group integer dot products of q6_K weights.
 *
 *   w    : q6_K super-blocks of W [m][k] (m*(k/256)*210 bytes), k % 256 == 0.
 *   q    : int8 [n][k] q8 activations.
 *   ds   : accepted for a uniform signature, not read (may be NULL).
 *   dots : int32 [n][m][k/16] (out), dots[t][o][g] = D[t][o][g], exact.
 */
int mmq_q6k_q8(const void *w, int64_t m, int64_t k, const int8_t *q, const uint32_t *ds,
               int64_t n, int32_t *dots, hipStream_t stream);

/*
 * mmq_q6k_q8_fp32out - the q6_K quantized matmul, float32 result.
 *
 *   w   : q6_K super-blocks of W [m][k], k % 256 == 0.
 *   q   : int8 [n][k];  ds : uint32 [n][k/32] (as written by q8_quantize_rows;
 *         only the binary16 da is read).
 *   out : float [n][m] (out), token-major.  The summation order is the
 *         kernel's; the same accuracy bar as mmq_q4k_q8_fp32out.
 */
int mmq_q6k_q8_fp32out(const void *w, int64_t m, int64_t k, const int8_t *q,
                       const uint32_t *ds, int64_t n, float *out, hipStream_t stream);

/*
 * mmq_q6k_q8_f16out - mmq_q6k_q8_fp32out's float32 result stored as binary16
 * (nearest-even, bit for bit the rounding of the float32 result of the same
 * inputs and binary), as mmq_q4k_q8_f16out is for q4_K.
 */
int mmq_q6k_q8_f16out(const void *w, int64_t m, int64_t k, const int8_t *q,
                      const uint32_t *ds, int64_t n, uint16_t *out, hipStream_t stream);

/*
 * mmq_q6k_q8_fold - mmq_q4k_q8_fold for q6_K weights: MMQ_KERNEL_AUTO,
 * MMQ_KERNEL_DOT4 (n <= 8), MMQ_KERNEL_F16 or MMQ_KERNEL_I8 (MMQ_KERNEL_FEW,
 * MMQ_KERNEL_NARROW and MMQ_KERNEL_STREAM return MMQ_ERR_KERNEL).
 */
int mmq_q6k_q8_fold(const void *w, int64_t m, int64_t k, const int8_t *q, const uint32_t *ds,
                    int64_t n, void *out, int out_f16, int kernel, hipStream_t stream);

/*
 * q4k_repack - load-time re-layout of q4_K weights (read by the few-token
 * dot4 kernel and the binary16-MFMA prefill kernel).
 * (The pages name a "load-time B pre-expansion" round and a scale
 * "predecode" round, r18 and r35 in the r17 and r31 pages' notes; the
 * layout is this library's.)
 *
 *   w  : q4_K super-blocks of W [m][k] (as for mmq_q4k_q8), k % 256 == 0.
 *   wr : ceil(m/16) * (k/256) * 2368 bytes (out), 16-byte aligned.  Rows in
 *        tiles of 16, one 2368-byte record per (tile, super-block), records
 *        tile-major.  Record: [0, 64) dword r = d | dmin << 16 of row r;
 *        [64, 320) dword 16p + r = sc[2p] | sc[2p+1] << 8 | m[2p] << 16 |
 *        m[2p+1] << 24 (the 6-bit fields as bytes); [320, 2368) the 16 bytes
 *        at 320 + 512p + 256h + 16r are qs bytes 32p + 16h .. +15 of row r
 *        (p < 4, h < 2, r < 16).  Rows past m are zero.
 * Pure byte work: the same values, 148 bytes per row and super-block
 * against 144.  Errors as for mmq_q4k_q8 (m == 0 is an empty call).
 */
int q4k_repack(const void *w, int64_t m, int64_t k, void *wr, hipStream_t stream);

/*
 * mmq_q4kr_q8_fp32out - mmq_q4k_q8_fp32out on repacked weights (wr from
 * q4k_repack of the same m, k).  For n <= 8 it runs the vector-ALU dot4
 * kernel with the same arithmetic, in the same order, as
 * mmq_q4k_q8_fp32out's kernel for that n, so the two results are equal bit
 * for bit.  Above 16 tokens, where the tiles fill the CUs (at least 160
 * tiles of 128 rows x 128 tokens) or n > 40, it runs the binary16-MFMA
 * kernel on the records, again with mmq_q4k_q8_fp32out's arithmetic and
 * order for that kernel (equal bit for bit where mmq_q4k_q8_fp32out takes it,
 * n > 64).  Other token counts run as slices of 8 tokens, each reading the
 * weights again.  Other arguments, errors and empty calls as for
 * mmq_q4k_q8_fp32out.
 */
int mmq_q4kr_q8_fp32out(const void *wr, int64_t m, int64_t k, const int8_t *q,
                        const uint32_t *ds, int64_t n, float *out, hipStream_t stream);

/*
 * q8_quantize_rows_tiled - q8_quantize_rows with the codes written as the
 * binary16 matrix-core operands of the prefill matmul, in its tile order (a
 * quantize-transpose pass ahead of the matmul: the r22 page, section 5,
 * names a later "quantize-transpose prepass" that changed the activation
 * side's layout at its root; this layout is the library's).  The codes and
 * scale words are q8_quantize_rows' bit for bit.
 *
 *   x  : float32 [n][k], k % 256 == 0.
 *   qt : ceil(n/128) * 128 * k binary16 values (out, 2 bytes each): tokens in
 *        tiles of 128, k in stages of 128, one block of 16 x 128 slots of 8
 *        values (32768 bytes) per (tile T, stage s), blocks tile-major.  Slot
 *        ((c*2 + h)*2 + g)*128 + tt of block (T, s) holds the codes of token
 *        128T + tt at k = 128s + 32c + 16g + 8h + e for e = 0,2,1,3,4,6,5,7
 *        (c < 4, h < 2, g < 2, tt < 128).  Tokens past n hold zeros.
 *   ds : uint32 [n][k/32] (out), as for q8_quantize_rows.
 * Errors as for q8_quantize_rows, except that k must be a multiple of 256
 * (MMQ_ERR_SHAPE) and n at most 2^31 - 128.
 */
int q8_quantize_rows_tiled(const float *x, int64_t n, int64_t k, uint16_t *qt, uint32_t *ds,
                           hipStream_t stream);

/*
 * q8_quantize_silu_mul_tiled - q8_quantize_silu_mul (h = SiLU(gate) * up,
 * never written) with the codes written as operand tiles, as
 * q8_quantize_rows_tiled does; codes and words bit for bit those of
 * q8_quantize_silu_mul.  Errors as for q8_quantize_rows_tiled, with `up`
 * checked beside `gate`.
 */
int q8_quantize_silu_mul_tiled(const float *gate, const float *up, int64_t n, int64_t k,
                               uint16_t *qt, uint32_t *ds, hipStream_t stream);

/*
 * mmq_q4k_q8t_fp32out / mmq_q4kr_q8t_fp32out - mmq_q4k_q8_fp32out (q4_K
 * rows) and mmq_q4kr_q8_fp32out (q4k_repack records) with the activations
 * as operand tiles (qt and ds from q8_quantize_rows_tiled of the same n and
 * k).  Every n runs the binary16-MFMA kernel, whose producers copy the tiles
 * straight into LDS instead of converting q8; the arithmetic and its order
 * are that kernel's, so the result equals mmq_q4k_q8_fp32out's bit for bit
 * wherever that takes the binary16 kernel (n > 64, and n > 32 where m
 * gives at least 160 tiles of 128 x 128).  Meant for prefill.
 * With few tokens it is faster than mmq_q4k_q8_fp32out only where m gives
 * many 128-row tiles (m = 28672 at n = 33); with few row tiles (m = 8192)
 * or n <= 8 the int8-code entry point is faster.  Other arguments, errors and
 * empty calls as for mmq_q4k_q8_fp32out / mmq_q4kr_q8_fp32out, and n at most
 * 2^31 - 128.
 */
int mmq_q4k_q8t_fp32out(const void *w, int64_t m, int64_t k, const uint16_t *qt,
                        const uint32_t *ds, int64_t n, float *out, hipStream_t stream);
int mmq_q4kr_q8t_fp32out(const void *wr, int64_t m, int64_t k, const uint16_t *qt,
                         const uint32_t *ds, int64_t n, float *out, hipStream_t stream);

/*
 * mmq_q6k_q8t_fp32out - mmq_q6k_q8_fp32out with the activations as operand
 * tiles (from q8_quantize_rows_tiled; one tiled quantization serves q4_K and
 * q6_K layers alike).  Every n runs the q6_K binary16-MFMA kernel, whose
 * producers copy the tiles straight into LDS; same arithmetic in the same
 * order, so the result equals mmq_q6k_q8_fp32out's bit for bit wherever that
 * takes the binary16 kernel (n > 8).  Other arguments, errors and empty
 * calls as for mmq_q6k_q8_fp32out, and n at most 2^31 - 128.
 */
int mmq_q6k_q8t_fp32out(const void *w, int64_t m, int64_t k, const uint16_t *qt,
                        const uint32_t *ds, int64_t n, float *out, hipStream_t stream);

/* Weight and activation formats of the fold entry points. */
enum mmq_format {
    MMQ_FORMAT_Q4K = 0,                /* mmq_q4k_q8_fp32out / _f16out */
    MMQ_FORMAT_Q4K_REPACKED = 1,       /* mmq_q4kr_q8_fp32out */
    MMQ_FORMAT_Q6K = 2,                /* mmq_q6k_q8_fp32out / _f16out */
    MMQ_FORMAT_Q4K_TILES = 3,          /* mmq_q4k_q8t_fp32out */
    MMQ_FORMAT_Q4K_REPACKED_TILES = 4, /* mmq_q4kr_q8t_fp32out */
    MMQ_FORMAT_Q6K_TILES = 5           /* mmq_q6k_q8t_fp32out */
};

/*
 * mmq_kernel_choice - the kernel (enum mmq_kernel, never MMQ_KERNEL_AUTO)
 * that the fold entry point of `format` runs for an m x k weight and n
 * tokens; host logic only, no HIP call.  (mmq_fold_epilogue runs the same but
 * for MMQ_FORMAT_Q6K, see there; its kernels and those of mmq_fold_grouped have
 * no id.)  MMQ_ERR_SHAPE for negative sizes or k not a positive multiple of 256,
 * MMQ_ERR_KERNEL for an unknown format.
 */
int mmq_kernel_choice(int format, int64_t m, int64_t k, int64_t n);

/*
 * mmq_fold_epilogue - a fold entry point with an epilogue: what follows the
 * matmul elementwise is done as its results are stored, in float32 (exp and the
 * sigmoid's reciprocal to an ulp), with one rounding at a binary16 store.
 *
 *   out[t][o] = act( fold[t][o] + bias[o] ) + residual[t][o]
 *
 * where fold is the float32 result of the entry point of `format` for the
 * same arguments, bit for bit (with every operand absent and MMQ_ACT_NONE the
 * call is that entry point), except MMQ_FORMAT_Q6K at 9 to 64 tokens, and above
 * while ceil(m/16)*ceil(n/64) <= 1536 (and n*k < 2^32), which runs kernels of
 * its own with the same accuracy.  Outputs and residuals may be rows of larger
 * arrays (strides), and the residual may be the output itself (same type and
 * stride: x += W h); otherwise they must not overlap.
 *
 *   w, q, ds : as for the entry point of `format` (q: its int8 codes or its
 *              operand tiles); m, k, n and their limits too.
 *   out      : float32 or binary16 [n][out_stride], columns 0 .. m - 1 written.
 * Errors as for that entry point; MMQ_ERR_NULL for a NULL epilogue,
 * MMQ_ERR_KERNEL for an unknown format or activation, MMQ_ERR_SHAPE for a
 * stride below m, MMQ_ERR_ALIGN for a bias or residual not 16-byte aligned.
 */
enum mmq_activation {
    MMQ_ACT_NONE = 0,
    MMQ_ACT_RELU = 1,      /* max(v, 0) */
    MMQ_ACT_SILU = 2,      /* v / (1 + exp(-v)) */
    MMQ_ACT_GELU = 3,      /* v * Phi(v) = v * erfc(-v / sqrt(2)) / 2 */
    MMQ_ACT_GELU_TANH = 4  /* v * (1 + tanh(sqrt(2/pi) * (v + 0.044715 v^3))) / 2 */
};

typedef struct mmq_epilogue {
    const float *bias;        /* [m], or NULL (mmq_fold_grouped: [experts][m]) */
    const void *residual;     /* [n][residual_stride], or NULL */
    int64_t residual_stride;  /* elements between rows; 0 = m */
    int64_t out_stride;       /* elements between output rows; 0 = m */
    int activation;           /* enum mmq_activation */
    int residual_f16;         /* residual is binary16 (else float32) */
    int out_f16;              /* out is binary16 (else float32) */
} mmq_epilogue;

int mmq_fold_epilogue(int format, const void *w, int64_t m, int64_t k, const void *q, const uint32_t *ds,
                      int64_t n, const mmq_epilogue *epilogue, void *out, hipStream_t stream);

/*
 * mmq_fold_grouped - matrix products grouped by expert, with ragged sizes that
 * only the device knows: slots s with offsets[e] <= s < offsets[e+1] belong
 * to expert e and are multiplied by its matrix,
 *
 *   out[s][o] = act( fold(W[e], row r(s) of q)[o] + bias[e][o] ) + residual[s][o]
 *
 * with r(s) = rows[s], or s without rows.  Any expert may have no slots, and
 * any row may be taken any number of times.  Slots outside
 * [offsets[0], offsets[experts]) are left as they were.  The call reads
 * nothing back and has no launch that depends on the offsets' values, so it
 * can be captured into a graph and replayed over new ones.
 *
 *   format  : MMQ_FORMAT_Q4K or MMQ_FORMAT_Q6K (others: MMQ_ERR_KERNEL).
 *   w       : [experts] matrices of [m][k], one behind the other; with more
 *             than one expert the bytes of a matrix must be a multiple of 16
 *             (MMQ_ERR_ALIGN; always so in q4_K, in q6_K where m*(k/256) is a
 *             multiple of 8).
 *   q, ds   : [tokens] rows, as for the fold entry points.
 *   rows    : int32 [slots], 0 <= rows[s] < tokens, or NULL (then tokens must
 *             be at least slots, MMQ_ERR_SHAPE).  Not read outside the groups.
 *   offsets : int32 [experts + 1], not decreasing, within 0 .. slots.
 *   slots   : rows of out (and of the residual): the most there can be.
 *   epilogue, out : as for mmq_fold_epilogue; bias is [experts][m].
 * A value of rows or offsets outside its range is clamped into it, and an
 * offset below an earlier one counts as the largest before it (the result is
 * then meaningless, but nothing outside the arrays is touched).  The float32
 * arithmetic is that of the fold entry points on the kernel that the group's
 * size takes, with the same accuracy; equal calls give equal bits, but the
 * order of a sum, and so a result's last bits, may depend on the sizes of all
 * groups.  Limits: experts <= 4096, tokens*k < 2^32, slots*m and
 * experts*m*(k/256)*(block bytes) below 2^40.
 * slots or m of 0 is an empty call.
 */
int mmq_fold_grouped(int format, const void *w, int64_t experts, int64_t m, int64_t k, const int8_t *q,
                     const uint32_t *ds, int64_t tokens, const int32_t *rows, const int32_t *offsets,
                     int64_t slots, const mmq_epilogue *epilogue, void *out, hipStream_t stream);

/*
 * moe_route - the router of mmq_fold_grouped: the `top` experts of each token
 * by score, their softmax weights, and the slots of the grouped products.
 *
 *   logits  : float [n][stride] (0 = experts), experts <= 1024.  -inf and NaN
 *             mask an expert out; +inf counts as the largest float.
 *   top     : 1 .. min(experts, 64).
 *   ids     : int32 [n][top] (out), the chosen experts, best first, equal
 *             scores by lowest index; -1 where fewer experts are left (a
 *             token whose scores are all masked has only -1).
 *   weights : float [n][top] (out), scale * exp(l - max) / sum, the sum over
 *             the chosen (normalize != 0) or over all unmasked experts; 0
 *             beside -1.
 *   slot    : int32 [n][top] (out), the slot of each choice, or -1.  Slots
 *             are grouped by expert and in token order within one.
 *   rows    : int32 [n*top] (out), the token of each slot; -1 behind the last.
 *   offsets : int32 [experts + 1] (out), as mmq_fold_grouped takes them.
 * Deterministic, no workspace.  n == 0 is an empty call (offsets too stay as
 * they are).  MMQ_ERR_SHAPE for top outside 1 .. experts or a stride below
 * experts; MMQ_ERR_OVERFLOW for experts above 1024, top above 64, n above
 * 2^26 - 4 (a wave per token), or n*top above 2^30.
 */
int moe_route(const float *logits, int64_t n, int64_t experts, int64_t stride, int top, int normalize, float scale,
              int32_t *ids, float *weights, int32_t *slot, int32_t *rows, int32_t *offsets, hipStream_t stream);

/*
 * moe_combine - the experts' outputs back in token order:
 *
 *   out[t][o] = residual[t][o] + sum_j weights[t][j] * y[slot[t][j]][o]
 *
 * in float32, over the j whose slot lies in 0 .. slots - 1 (a token without
 * any gets its residual, or 0).
 *
 *   y        : float (y_f16 == 0) or binary16 [slots][m].
 *   slot, weights : [n][top] from moe_route, top <= 64.
 *   residual : float [n][m] or NULL; may be out itself.
 *   out      : float [n][m] (out).
 * n or m of 0 is an empty call.  Limits: slots*m and n*m below 2^40, n*top at
 * most 2^30, and n*c below 2^24 for c workgroups on a token's columns, c =
 * ceil(m/2048) for binary16 y and m a multiple of 8, ceil(m/1024) for float y and
 * m a multiple of 4, else ceil(m/256).
 */
int moe_combine(const void *y, int y_f16, int64_t slots, int64_t m, const int32_t *slot, const float *weights,
                int64_t n, int top, const float *residual, float *out, hipStream_t stream);

/*
 * q8_quantize_norm - the norms before and after a transformer block with the
 * block's gate and the residual scale, fused with the q8 quantization of the
 * next projections' input:
 *
 *   z  = y                                           without y_weight
 *      = y * y_weight / sqrt(mean(y^2) + eps)        with it (the norm after the block)
 *   r  = float32( residual_scale * x + gate * z )    the new residual stream (no gate: 1)
 *   h  = float32( r * weight / sqrt(mean(r^2) + eps) )   (the norm before the next)
 *   q, ds = q8_quantize_rows(h)
 *
 * evaluated in float64 between the roundings named, means over the k values
 * of a token.  A NaN or an infinity in a token's x or y makes its h NaN or 0
 * throughout; a 32-value block whose h has a NaN gets a NaN da (and any codes),
 * so that every product of the token is NaN, not 0.  Without y the stream is
 * not changed: r = x, and y_weight, gate and r must be NULL and residual_scale
 * 1 (MMQ_ERR_NULL).
 *
 *   n, k     : k % 32 == 0; limits as for q8_quantize_rows, n at most 2^31 - 128
 *              and n*1024 below 2^32.
 *   q, ds    : as for q8_quantize_rows.
 * Strides are elements between rows, 0 = k (gate_stride 0: one gate row for
 * all tokens); below k they are MMQ_ERR_SHAPE, and rows must start on 16-byte
 * boundaries (MMQ_ERR_ALIGN).  r may be x itself (same stride); otherwise
 * outputs must not overlap inputs.
 */
typedef struct q8_norm {
    const float *x;          /* [n][x_stride] residual stream */
    const void *y;           /* [n][y_stride] block output, or NULL */
    const float *y_weight;   /* [k], or NULL: y is not normed */
    const float *gate;       /* [k] or [n][gate_stride], or NULL */
    const float *weight;     /* [k] */
    float *r;                /* [n][r_stride] (out), required with y */
    float *h;                /* [n][k] (out), or NULL: not written */
    int64_t x_stride, y_stride, gate_stride, r_stride;
    float residual_scale, eps;
    int y_f16;               /* y is binary16 (else float32) */
} q8_norm;

int q8_quantize_norm(const q8_norm *args, int64_t n, int64_t k, int8_t *q, uint32_t *ds, hipStream_t stream);

/*
 * q8_quantize_norm_tiled - q8_quantize_norm with the codes as operand tiles
 * (k % 256 == 0), as q8_quantize_rows_tiled writes them.
 */
int q8_quantize_norm_tiled(const q8_norm *args, int64_t n, int64_t k, uint16_t *qt, uint32_t *ds,
                           hipStream_t stream);

/*
 * residual_norm - q8_quantize_norm without the codes: r (with y) and h, which
 * must not be NULL.  For the readers that take float32: a router, an output
 * head.
 */
int residual_norm(const q8_norm *args, int64_t n, int64_t k, hipStream_t stream);

/*
 * Attention between the projections: rotary positions, a paged cache of
 * quantised keys and values, and softmax attention over it.
 *
 * rope_rows - rotary positions with several axes, on rows of heads.
 *
 *   pair j of every head, t = positions[row][axis[j]] * freq[j]:
 *     (a, b) -> scale * (a cos t - b sin t, a sin t + b cos t)
 *
 * evaluated in float64, rounded to float32 and then to the rows' type.  Pair j
 * is values (j, pairs + j) of a head, or (2 j, 2 j + 1) where `adjacent`; what
 * lies past the 2 * pairs rotated values is copied.  Text has one axis; images
 * and video have one each for time, height and width.
 *
 *   x, out   : float32 or binary16 (half) [n][stride], heads * head_dim values a
 *              row; strides are elements between rows, 0 = heads * head_dim.
 *              out may be x (same stride); otherwise they must not overlap.
 *   head_dim : 2 .. 1024, odd too; 1 <= pairs, 2 * pairs <= head_dim.
 * axis values outside 0 .. axes - 1 are clamped into it.  n or heads of 0 is an
 * empty call.  MMQ_ERR_OVERFLOW for n * 256 or more than 2^32 - 1 work-items.
 */
typedef struct rope_plan {
    const int32_t *positions;   /* [n][positions_stride], `axes` a row */
    const float *freq;          /* [pairs], radians per position */
    const int32_t *axis;        /* [pairs], the axis of each pair, or NULL: axis 0 */
    int64_t positions_stride;   /* elements between rows; 0 = axes */
    int axes, pairs;
    int adjacent;               /* pairs are neighbours (else halves) */
    float scale;                /* of cosine and sine; usually 1 */
} rope_plan;

int rope_rows(const rope_plan *rope, const void *x, int64_t x_stride, int half, int64_t n, int64_t heads,
              int64_t head_dim, void *out, int64_t out_stride, hipStream_t stream);

/*
 * The cache: pages of `page` tokens, each a record per head,
 *
 *   key codes [page][cb], key scales [page][head_dim/32] (binary16),
 *   value codes [page][cb], value scales [page][head_dim/32],
 *
 * cb = head_dim bytes (KV_Q8) or head_dim / 2 (KV_Q4); data holds
 * [pages][heads] records of kv_cache_bytes / (pages * heads) bytes.  A value is
 * code * scale of its 32-value block, with
 *   KV_Q8: da = max|x| * r in float32, r = float32(1/127); code = round(x / da),
 *          IEEE division, ties away from zero; int8, -127 .. 127;
 *          scale = binary16(da).  (A step by multiplication, as tensor libraries
 *          take it on a device: codes are compared with theirs.  q8_quantize_rows
 *          divides by 127 instead: a da a float32 step apart at most, so the code
 *          of a value within that of a tie may be its neighbour.)
 *   KV_Q4: the same with float32(1/7), code -7 .. 7, stored as code + 8.
 * A block with a NaN or an infinity gets a NaN scale, and one whose da is past
 * binary16 an infinite one.  Order of a token's codes (nb = head_dim / 32):
 *   keys:   value 32 b + 8 g + i is code 8 (g nb + b) + i (b < nb, g < 4, i < 8);
 *           in KV_Q4 nibbles j and j + 4 of those eight are values 2 j, 2 j + 1;
 *   values: value 16 t + r is code 2 nb r + t (t < 2 nb, r < 16);
 * nibble 2 i of KV_Q4 is the low one of byte i.  A token not written may hold
 * anything.
 *
 * The plan says which row of a call is which token: rows
 * offsets[s] <= r < offsets[s+1] are the last tokens of sequence s, row r at
 * position lengths[s] - (offsets[s+1] - r), on page table[s][position / page].
 * So lengths count the call's own tokens.  Without offsets row s is the last
 * token of sequence s (n must be seqs, MMQ_ERR_SHAPE).  A position below 0 or
 * past the table, or with a page id outside 0 .. pages - 1 (-1 for pages
 * dropped), has no place in the cache.  All of it is read on the device: calls
 * can be captured and replayed over new values.  Rows outside
 * [offsets[0], offsets[seqs]) are left as they were; offsets that decrease give
 * meaningless results, but nothing outside the arrays is touched.
 *
 * Limits: heads <= 1024, seqs <= 65535, width * page <= 2^30, n < 2^24, pages <
 * 2^31, a cache and n * stride below 2^40; head_dim a multiple of 32 up to 256,
 * page a power of two, 16 .. 1024 (MMQ_ERR_SHAPE); MMQ_ERR_KERNEL for an unknown
 * format.  n == 0 or seqs == 0 is an empty call.
 */
enum kv_format { KV_Q8 = 0, KV_Q4 = 1 };

typedef struct kv_cache {
    void *data;
    int64_t pages;
    int heads, head_dim;
    int page;                   /* tokens of a page */
    int format;                 /* enum kv_format */
} kv_cache;

typedef struct kv_plan {
    const int32_t *table;       /* [seqs][table_stride], page ids */
    const int32_t *lengths;     /* [seqs] */
    const int32_t *offsets;     /* [seqs + 1], or NULL */
    int64_t seqs, width;        /* width: page ids of a sequence */
    int64_t table_stride;       /* 0 = width */
} kv_plan;

/* Bytes of a cache (its data need not be set); host logic only. */
int kv_cache_bytes(const kv_cache *cache, int64_t *bytes);

/*
 * kv_write - the keys and values of new tokens into the cache, the keys rotated
 * first where `rope` is not NULL (to float32 as rope_rows evaluates them, and
 * quantised from that).  rope's positions are per row of k, its pairs at most
 * head_dim / 2.
 *
 *   k, v : float32 or binary16 (half) [n][stride], heads * head_dim a row.
 * Rows without a place are not written.  Two rows with one place (a page shared
 * by two sequences) leave a mixture there.
 */
int kv_write(const kv_cache *cache, const kv_plan *plan, const rope_plan *rope, const void *k, const void *v, int half,
             int64_t n, int64_t k_stride, int64_t v_stride, hipStream_t stream);

/*
 * kv_read - rows read back: code * scale, rounded once.  offsets that give a
 * sequence as many rows as it is long read all of it.  Rows without a place
 * become 0.
 */
int kv_read(const kv_cache *cache, const kv_plan *plan, void *k, void *v, int half, int64_t n, int64_t k_stride,
            int64_t v_stride, hipStream_t stream);

/*
 * kv_attend - causal softmax attention of new tokens over the cache, which
 * holds them already:
 *
 *   out[r][hq] = sum_j w_j v_j[h],  w = softmax over j of scale * q[r][hq] . k_j[h]
 *   h = hq / (heads / cache heads),  max(0, pos - window + 1) <= j <= pos
 *
 * over the positions j that have a place; pos is row r's, and without a window
 * (0) j starts at 0.  lse[r][hq] = ln sum_j exp(scale * q . k_j).  A row that
 * sees nothing gets out 0 and lse -inf.  What hidden positions hold (NaN scales
 * too) does not matter.  One new token per sequence, some tens, and chunks of a
 * prompt are all meant.
 *
 * Sums, scores and the softmax are float32; codes and binary16 queries enter the
 * products exactly, float32 queries with 22 bits, or to 2^-39 of the head's
 * largest value.  Weights times their scales are rounded to binary16 (relative
 * 2^-11) before they meet the values' codes where q and out are both binary16,
 * else to 22 bits (who keeps binary16 and wants these takes a float32 out and
 * rounds it); either way absolutely by 2^-29 of the largest product of a weight
 * and its token's largest value that the row has met.  Equal calls give equal
 * bits, but the order of a sum may depend on the lengths of all sequences.
 *
 *   most      : an upper bound of any sequence's rows in this call; rows past it
 *               are left as they were.  It chooses the kernel, for all sequences:
 *               the nearer it is, the faster the call.
 *   out       : must not overlap q or the cache.
 *   workspace : kv_attend_workspace's bytes, for this call alone until it has
 *               finished (calls on two streams need two).  MMQ_ERR_SHAPE if it is
 *               smaller.
 * A window of more than 2^30 is none.  MMQ_ERR_SHAPE for heads not a multiple of
 * the cache's, a negative window or most < 1; MMQ_ERR_OVERFLOW for most * heads /
 * cache heads >= 2^28, or 2^31 and more steps of 128 tokens of a sequence (and one
 * more) times tiles of 16 of its rows of a cache head times cache heads.
 */
typedef struct kv_query {
    const void *q;              /* [n][q_stride], heads * head_dim a row */
    void *out;                  /* [n][out_stride] */
    float *lse;                 /* [n][heads], or NULL */
    int64_t q_stride, out_stride;   /* 0 = heads * head_dim */
    int64_t n, most;
    int heads;                  /* query heads */
    int q_half, out_half;       /* binary16 (else float32) */
    int window;
    float scale;
} kv_query;

int kv_attend_workspace(const kv_cache *cache, const kv_plan *plan, const kv_query *query, int64_t *bytes);
int kv_attend(const kv_cache *cache, const kv_plan *plan, const kv_query *query, void *workspace,
              int64_t workspace_bytes, hipStream_t stream);

/* A static, human-readable name for a status code (never NULL). */
const char *mmq_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* Q4Q8_MMQ_H */
