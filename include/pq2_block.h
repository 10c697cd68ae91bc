/*
 * pq2_block.h -- C ABI of the operators around the packed matmul that a
 * decoder's feed-forward block needs: products with 4-bit weights, the gated
 * feed-forward product, and the norms between blocks with the INT8 quantiser.
 * Part of libpq2.so; the conventions, status codes, element types and limits
 * are those of pq2.h (device pointers on the current device, caller-owned
 * buffers, everything checked on the host before any HIP call, work enqueued
 * on `stream`, nothing allocated, nothing kept after the call).
 *
 * q and xs are the outputs of pq2_quantize_act_i8 (groups of 128) throughout,
 * unless an entry point takes `agroup`.  A row stride above 2^31 elements (or
 * bytes of codes) is PQ2_ESHAPE.
 */
#ifndef PQ2_BLOCK_H
#define PQ2_BLOCK_H

#include "pq2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the gated feed-forward product, on the fp32 gate output g:
 * SiLU g / (1 + exp(-g)); GELU 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))). */
enum { PQ2_ACT_SILU = 0, PQ2_ACT_GELU_TANH = 1 };

/* Largest m and n of the entry points below (n: what one launch can hold a
 * row of workgroups for, with the narrowest of the kernels' column blocks). */
#define PQ2_MAX_BLOCK_M (65535 * 16)
#define PQ2_MAX_BLOCK_N ((1 << 30) - 512)

/* ---- 4-bit weights.
 *
 *   w[n][k] = (c[n][k] - 8) * ws[n][k / wgroup]     c in 0..15, ws fp16, wgroup 128, 64 or 32
 *   y[m][n] = sum_g xs[m][g] * sum_{s in g} ws[n][s] * dot[m][n][s]
 *
 * with dot[m][n][s] the exact integer dot of weight group s, and g running
 * over the k/128 activation groups.  Each activation group adds one FP32 term.
 *
 * w4 tile layout: T = ceil(n/16) tiles of 16 rows, S8 = ceil(k/1024)
 * segments of 1024 weights, S = 128/wgroup.  Unit (t, sb) at
 * (t*S8 + sb) * (8192 + 256*S) holds
 *  - eight code blocks of 1024 bytes, block b = the 128 weights from
 *    kb0 = 1024*sb + 128*b: bytes 16*l .. 16*l + 15 with l = j + 16*kb
 *    (j = 0..15, kb = 0..3) hold four dwords u = 0..3 of row 16t + j; with
 *    k0 = kb0 + 64*(u/2) + 16*kb + 8*(u%2), byte v of dword u holds weight
 *    k0 + v in its low half and weight k0 + 4 + v in its high half, each as
 *    the four-bit two's complement of c - 8;
 *  - then the fp16 scales: row j's 8*S scales of the segment, in k order, at
 *    8192 + 16*S*j;
 *  - padding rows (>= n) and weights (>= k) hold weight 0, scale 0. */

/* Bytes of the w4 tile layout; -1 if n < 1, n > PQ2_MAX_BLOCK_N, k < 128,
 * k % 128, k > PQ2_MAX_K, or wgroup is not 128, 64 or 32. */
int64_t pq2_w4_tiles_bytes(int64_t n, int64_t k, int64_t wgroup);

/* Rows of 4-bit codes and fp16 scales -> w4 tile layout.  One-time weight
 * preparation.
 *   codes   device, n rows of codes_row_stride_bytes >= k/2 bytes, any
 *           alignment: byte i of a row holds weight 2i in its low half and
 *           weight 2i + 1 in its high half, as codes c = 0..15.
 *   scales  device fp16, n rows of scales_row_stride_elems >= k/wgroup
 *           elements; 2-byte aligned.
 *   tiles   device, pq2_w4_tiles_bytes(n, k, wgroup) bytes, 16-byte aligned,
 *           fully written (padding included); must not overlap the inputs.
 * Errors: EINVAL (null, wgroup, overlap), ESHAPE, EALIGN, ELAUNCH, EDEVICE. */
int pq2_prepare_w4_tiles(const uint8_t* codes, int64_t codes_row_stride_bytes, const void* scales,
                         int64_t scales_row_stride_elems, int64_t n, int64_t k, int64_t wgroup, void* tiles,
                         void* stream);

/* y = the definition above for any 1 <= m <= PQ2_MAX_BLOCK_M: the decode
 * engine for few columns, the prefill engine for many.  For m <= 16 a
 * column's bits do not depend on m or on the other columns.
 *   q       device int8 [m][k], 16-byte aligned.  xs  device float [m][k/128], 4-byte aligned.
 *   tiles   device w4 tile layout, 16-byte aligned.
 *   y       device float [m][n], 4-byte aligned; fully overwritten; must not
 *           overlap any input.
 * Errors: EINVAL (null, wgroup, overlap), ESHAPE (m, n or k out of range,
 *         k % 128), EALIGN, ELAUNCH, EDEVICE. */
int pq2_matmul_w4(const int8_t* q, const float* xs, const void* tiles, int64_t m, int64_t n, int64_t k,
                  int64_t wgroup, float* y, void* stream);

/* The complete call: y from bf16 / fp16 / fp32 activations, the bits of
 * pq2_quantize_act_i8 into q_work / xs_work followed by pq2_matmul_w4.  For
 * few columns (and 16-byte aligned rows of x) one launch does both and the
 * scratch is not written.  m * k above 2^34 is PQ2_ESHAPE, here and in the
 * gated complete calls.
 *   x       as pq2_quantize_act_i8.
 *   q_work  device int8 [m][k], 16-byte aligned; xs_work device float
 *           [m][k/128], 4-byte aligned: scratch owned by the caller.  Calls
 *           that share scratch must be ordered by the caller.
 * Errors: as pq2_quantize_act_i8 and pq2_matmul_w4, all checked before
 *         anything is enqueued. */
int pq2_linear_w4(const void* x, int dtype, int64_t x_row_stride_elems, const void* tiles, int64_t m, int64_t n,
                  int64_t k, int64_t wgroup, float* y, int8_t* q_work, float* xs_work, void* stream);

/* ---- Gated feed-forward product
 *
 *   h[m][n] = act(yg[m][n]) * yu[m][n]
 *
 * with yg and yu the fp32 products of the same activations with two weight
 * matrices of one shape, in one kernel: act and the product run on the fp32
 * sums, h is rounded once to h_dtype.
 *
 * _tiles: ternary weights in the tile layout of pq2_prepare_tiles; for
 * m <= 16, yg and yu have the bits of pq2_matmul_small_m_tiles.
 * _w4: 4-bit weights in the w4 tile layout (one wgroup for both); yg and yu
 * have the bits of pq2_matmul_w4 with the same m.
 *   gate, up  device tile layouts, 16-byte aligned (may be the same matrix).
 *   h         device [m][n] of h_dtype, element-aligned; fully overwritten;
 *             must not overlap any input.
 * Errors: EINVAL (null, act, dtype, wgroup, overlap), ESHAPE, EALIGN,
 *         ELAUNCH, EDEVICE. */
int pq2_gated_matmul_tiles(const int8_t* q, const float* xs, const void* gate, const void* up, int64_t m, int64_t n,
                           int64_t k, int act, void* h, int h_dtype, void* stream);
int pq2_gated_matmul_w4(const int8_t* q, const float* xs, const void* gate, const void* up, int64_t m, int64_t n,
                        int64_t k, int64_t wgroup, int act, void* h, int h_dtype, void* stream);

/* The complete calls: quantiser into the caller's scratch, then the product
 * (x, q_work, xs_work as pq2_linear_w4). */
int pq2_gated_linear_tiles(const void* x, int dtype, int64_t x_row_stride_elems, const void* gate, const void* up,
                           int64_t m, int64_t n, int64_t k, int act, void* h, int h_dtype, int8_t* q_work,
                           float* xs_work, void* stream);
int pq2_gated_linear_w4(const void* x, int dtype, int64_t x_row_stride_elems, const void* gate, const void* up,
                        int64_t m, int64_t n, int64_t k, int64_t wgroup, int act, void* h, int h_dtype,
                        int8_t* q_work, float* xs_work, void* stream);

/* ---- Norms around a block, with its gate, its residual scale and the
 * quantiser of the next product.  Per row, each line one FP32 operation per
 * element unless stated:
 *
 *   t  = block                                       (block given)
 *   t  = (t * rstd(t)) * post_w                      (post_w given)
 *   t  = t * gate                                    (gate given)
 *   t  = t * alpha
 *   r' = round(r + t) to r_dtype                     (r' = r without block)
 *   x  = round((r' * rstd(r')) * w) to x_dtype
 *   q, xs = INT8 codes and scales of x in groups of agroup elements, those
 *           of pq2_quantize_act_i8_g on x
 *   rstd(v) = float(1 / sqrt(sum(v^2) / k + eps)), the sum in FP64
 *
 * With unit_offset the norm weights are 1 + w and 1 + post_w (one FP32 add).
 * Any of the outputs r_out, x_out and (q, xs) may be absent (NULL); at least
 * one is given.  A row does not depend on the others, and r_out may be r
 * itself (same pointer, same stride): otherwise no output overlaps an input
 * or another output.  Rows of one stride in bytes may lie between each other
 * (columns of one buffer); with different strides the whole spans from first
 * to last element are kept apart. */
typedef struct pq2_block_norm_args {
    const void* r;            /* residual stream [m][r_stride]                              */
    int64_t r_stride;         /* row strides in elements, >= k                              */
    const void* block;        /* the block's output [m][block_stride]; NULL: none           */
    int64_t block_stride;
    const void* post_w;       /* weights of the norm after the block [k]; NULL: no norm     */
    const void* gate;         /* [k] (gate_stride 0) or [m][gate_stride]; NULL: none        */
    int64_t gate_stride;
    const void* w;            /* weights of the norm before the next block [k]              */
    void* r_out;              /* r' [m][r_out_stride] of r_dtype                            */
    int64_t r_out_stride;
    void* x_out;              /* x [m][x_out_stride] of x_dtype                             */
    int64_t x_out_stride;
    int8_t* q;                /* int8 [m][k], 8-byte aligned                                */
    float* xs;                /* float [m][k/agroup]                                        */
    int64_t m, k;             /* k as pq2_quantize_act_i8                                   */
    int64_t agroup;           /* 128, 64 or 32; read with q only                            */
    double eps;               /* >= 1e-70, finite                                           */
    float alpha;              /* residual scale                                             */
    int r_dtype, block_dtype; /* PQ2_BF16 / PQ2_F16 / PQ2_F32                               */
    int w_dtype;              /* of w, post_w and gate                                      */
    int x_dtype;              /* what x is rounded to                                       */
    int unit_offset;          /* 0 or 1                                                     */
} pq2_block_norm_args;

/* Errors: EINVAL (null args, r or w; no output; q without xs or xs without
 *         q; post_w or gate without block; dtype; agroup; eps; alpha not
 *         finite; unit_offset; overlap), ESHAPE (m < 1 or > PQ2_MAX_BLOCK_M, k, a
 *         stride below k), EALIGN (a pointer not aligned to its element, q
 *         not to 8 bytes), ELAUNCH, EDEVICE. */
int pq2_block_norm(const pq2_block_norm_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PQ2_BLOCK_H */
