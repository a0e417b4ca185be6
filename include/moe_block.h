/*
 * moe_block.h - C ABI of the MI355X (gfx950) operators that stand around and
 * beside the 4-bit expert layer of moe_w4.h:
 *   - the residual addition with its root-mean-square norm, whose output can
 *     also be written in 8 bits with a scale per token, and its gradient;
 *   - matrix products in 8-bit integers with a scale for each token and each
 *     output channel: dense, and grouped by expert over moe_route's tables
 *     (the expert layer with an 8-bit bank instead of a 4-bit one);
 *   - token rows sorted by expert and back, with the routing weights applied,
 *     and the gradients of both directions.
 *
 * Conventions are moe_w4.h's: array arguments are DEVICE pointers to memory
 * the caller allocated and owns, dense and row-major; the library never
 * allocates, frees or synchronises and keeps no state between calls; `stream`
 * is a hipStream_t passed as void*, on the current device, which has to own
 * the arrays; every argument is validated before anything is enqueued; the
 * return codes are moe_w4.h's MOE_* codes; no C++ exception crosses this
 * interface.  Calls launch kernels only (no memset, no allocation), so they
 * can be captured into a HIP graph; two calls may overlap as long as neither
 * writes what the other uses.  Unless an argument says otherwise, outputs may
 * not overlap inputs.  No kernel uses floating-point atomics: equal inputs
 * give equal bits.  A call without rows (T = 0, M = 0) enqueues nothing and
 * looks at no array, except that moe_add_rmsnorm_backward clears dweight.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "moe_w4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows (const void * arguments). */
#define MOE_ELEM_F32 0
#define MOE_ELEM_BF16 1
#define MOE_ELEM_F16 2

/*
 * Shape of a norm: T rows (0 <= T <= 2^24) of H elements (a positive multiple
 * of 8, at most 16384) of the element type `type`; eps >= 0, finite.
 */
typedef struct moe_norm_dims {
  int32_t T, H;
  int32_t type;
  float eps;
} moe_norm_dims;

/*
 * moe_add_rmsnorm - s = x + res, y = s / sqrt(mean(s^2) + eps) * weight, row
 * by row, and the 8-bit form of y.
 *   x       [T][H] rows (16-byte aligned)
 *   res     [T][H] residual rows of the same type (16-byte aligned), or NULL
 *           (then s = x)
 *   weight  [H] float32 (16-byte aligned)
 *   sum     [T][H] s rounded once to the row type (16-byte aligned), or NULL;
 *           may be x or res itself (updated in place)
 *   y       [T][H] rounded once to the row type (16-byte aligned), or NULL;
 *           may be x or res itself, but not sum
 *   yq, ys  [T][H] int8 (16-byte aligned) and [T] float32 (4-byte aligned):
 *           ys = max|y| / 127 and yq = y (127 / max|y|), in float32, rounded to
 *           the nearest integer (ties to even), from y before its rounding; both
 *           or neither NULL
 * At least one of y and yq.  The sum, the statistics and y are float32; the
 * norm reads s before its rounding.  Row sums of squares past float32's range
 * (elements above about 1e19) give rows of zeros, as float32 arithmetic does.
 * A row of zeros has y = 0, yq = 0 and ys = 0 (with eps = 0 it has no norm: y
 * is NaN).  A row whose y holds a NaN or an infinity has yq = 0 and ys = NaN,
 * so whatever is computed from it is NaN.
 */
int moe_add_rmsnorm(const moe_norm_dims *d, const void *x, const void *res, const float *weight,
                    void *sum, void *y, int8_t *yq, float *ys, void *stream);

/*
 * moe_add_rmsnorm_backward - gradients of moe_add_rmsnorm.  With
 * rho = 1 / sqrt(mean(s^2) + eps), xh = s rho and g = dy weight:
 *   dx = rho (g - xh mean(g xh)) + dsum        (the gradient of x and of res)
 *   dweight = sum over rows of dy xh
 *   sum     [T][H] s as moe_add_rmsnorm stored it (x itself where there was
 *           no residual); the row statistics are recomputed from it
 *   dy      [T][H] gradient of y
 *   dsum    [T][H] gradient that reaches s by the residual path, or NULL
 *   dx      [T][H] output in the row type; may be dy or dsum itself
 *   dweight [H] float32 (4-byte aligned), overwritten; or NULL.  T = 0 sets it
 *           to zeros.
 *   ws      scratch of at least moe_add_rmsnorm_backward_ws_bytes(d) bytes,
 *           16-byte aligned, overwritten (may be NULL when dweight is); calls
 *           that can overlap, captured ones among them, need one each
 * Rows are 16-byte aligned, float32 inside; dweight is summed in an order
 * fixed by T and H.
 */
size_t moe_add_rmsnorm_backward_ws_bytes(const moe_norm_dims *d); /* 0 for invalid dims */
int moe_add_rmsnorm_backward(const moe_norm_dims *d, const void *sum, const float *weight,
                             const void *dy, const void *dsum, void *dx, float *dweight, void *ws,
                             size_t ws_bytes, void *stream);

/*
 * moe_q8_quantize - the 8-bit form alone: T rows of H elements to int8 with a
 * scale per row, by moe_add_rmsnorm's rule (d->eps is not used).  It makes the
 * tokens of a product from rows that no norm produces, and the weights of a
 * bank from float rows (one row per output channel).
 *   x [T][H] (16-byte aligned);  xq [T][H] (16-byte aligned);  xs [T]
 */
int moe_q8_quantize(const moe_norm_dims *d, const void *x, int8_t *xq, float *xs, void *stream);

/*
 * Shape of a dense product: M rows (0 <= M <= 2^24), N output channels (a
 * positive multiple of 8, at most 2^20), K inputs (a positive multiple of 64,
 * at most 65536); `type` the output's element type.
 */
typedef struct moe_q8_dims {
  int32_t M, N, K;
  int32_t type;
} moe_q8_dims;

/*
 * moe_q8_matmul - out[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k].
 *   xq  [M][K] int8 tokens, xs [M] float32 their scales
 *   wq  [N][K] int8 weights, ws [N] float32 the channels' scales
 *   out [M][N] in d->type
 * xq, wq, ws and out are 16-byte aligned, xs 4-byte aligned.  The integer sum
 * is exact (any int8 values, -128 included, stay below 2^31); it is converted
 * to float32, multiplied by xs and then by ws, and rounded once to the output
 * type.  A row's bits do not depend on the other rows or on M.
 */
int moe_q8_matmul(const moe_q8_dims *d, const int8_t *xq, const float *xs, const int8_t *wq,
                  const float *ws, void *out, void *stream);

/*
 * An 8-bit bank of n experts, straight row-major (no repacking):
 *   gu   [n][2I][H] int8 (gate rows 0..I-1, up rows I..2I-1), gu_s [n][2I]
 *   dn   [n][H][I] int8, dn_s [n][H];  float32 scales, everything 16-byte
 *        aligned
 * moe_q8_gate_up reads only gu and gu_s, moe_q8_down only dn and dn_s.
 */
typedef struct moe_q8_bank {
  const int8_t *gu;
  const float *gu_s;
  const int8_t *dn;
  const float *dn_s;
} moe_q8_bank;

/*
 * moe_q8_gate_up - grouped gate/up product with SwiGLU, as moe_w4_gate_up with
 * 8-bit tokens and weights: for every row of the block map h = silu(g) u, g
 * and u as in moe_q8_matmul in float32, rounded once to bfloat16.
 *   xq [T][H] int8 tokens (16-byte aligned), xs [T] their scales
 *   r  tables from moe_route;  routed bank of E experts;  shared bank of 1
 *      expert, or NULL if n_shared = 0
 *   h  [Rows][I] bfloat16 (16-byte aligned)
 * Table entries out of range, blocks of more than d->tile_m_max rows among them,
 * set MOE_STATUS_BAD_INDEX and are skipped.  Entries of r->blocks behind the
 * first *r->n_blocks are not read.
 */
int moe_q8_gate_up(const moe_dims *d, const int8_t *xq, const float *xs, const moe_route_out *r,
                   const moe_q8_bank *routed, const moe_q8_bank *shared, uint16_t *h, void *stream);

/*
 * moe_q8_down - grouped down product, as moe_w4_down: y_slots[row] = W_down of
 * the row's expert times the row, rounded once to bfloat16 for moe_combine.
 *   hq [Rows][I] int8 rows (16-byte aligned), hs [Rows] their scales
 *      (moe_q8_quantize over h)
 *   y_slots [Rows][H] bfloat16 (16-byte aligned)
 */
int moe_q8_down(const moe_dims *d, const moe_route_out *r, const moe_q8_bank *routed,
                const moe_q8_bank *shared, const int8_t *hq, const float *hs, uint16_t *y_slots,
                void *stream);

/*
 * Token rows sorted by expert and back.  Rows are d->H elements of `type`
 * (MOE_ELEM_*), 16-byte aligned; `rows` arrays hold Rows = T*k + n_shared*T
 * rows in moe_route's order (the routed slots by expert, then one row per
 * token for the shared expert).  The calls read slot_pos, topk_w and status of
 * the tables only.  A slot position out of range sets MOE_STATUS_BAD_INDEX and
 * its slot is skipped (its dtopk_w is 0); slot_pos has to be a permutation, as
 * moe_route writes it.
 *
 * moe_dispatch_rows - rows[slot_pos[t*k+j]] = x[t] for every slot, and
 * rows[T*k+t] = x[t] when n_shared = 1 (bit copies).
 *   x [T][H];  rows [Rows][H] output
 */
int moe_dispatch_rows(const moe_dims *d, int32_t type, const void *x, const moe_route_out *r,
                      void *rows, void *stream);

/*
 * moe_dispatch_rows_backward - dx[t] = sum_j drows[slot_pos[t*k+j]]
 * (+ drows[T*k+t]), float32, j ascending, shared last, rounded once.
 */
int moe_dispatch_rows_backward(const moe_dims *d, int32_t type, const void *drows,
                               const moe_route_out *r, void *dx, void *stream);

/*
 * moe_combine_rows - moe_combine for any row type:
 * y[t] = sum_j topk_w[t][j] rows[slot_pos[t*k+j]] (+ rows[T*k+t]), float32
 * fused multiply-adds, j ascending, shared last, rounded once.  For bfloat16
 * it gives moe_combine's bits.
 */
int moe_combine_rows(const moe_dims *d, int32_t type, const void *rows, const moe_route_out *r,
                     void *y, void *stream);

/*
 * moe_combine_rows_backward - gradients of the combine:
 *   drows[slot_pos[t*k+j]] = topk_w[t][j] dy[t]  (rounded once),
 *   drows[T*k+t] = dy[t] when n_shared = 1,
 *   dtopk_w[t][j] = sum_h dy[t][h] rows[slot_pos[t*k+j]][h]  (float32, in an
 *   order fixed by H and the type)
 *   dy [T][H];  rows [Rows][H] as given to the combine;  drows [Rows][H]
 *   output, may be rows itself;  dtopk_w [T][k] float32 (4-byte aligned) or
 *   NULL (then rows is not read and may be NULL)
 */
int moe_combine_rows_backward(const moe_dims *d, int32_t type, const void *dy, const void *rows,
                              const moe_route_out *r, void *drows, float *dtopk_w, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
