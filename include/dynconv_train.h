/*
 * What a training step needs around the layers' own backward (sm_100a): the
 * load-balance loss of a router with its gradient, the norm of all gradients
 * with the factor that clips it, and an AdamW step over many tensors at once.
 *
 * The kernels and the router are learned (CondConv: Conditionally Parameterized
 * Convolutions for Efficient Inference, abstract; KernelWarehouse: Rethinking
 * the Design of Dynamic Convolution, abstract). The pages name no balance loss
 * and no optimizer; the formulas below are the usual ones.
 *
 * A step, in order: dynconv_route, dynconv_balance_forward, dynconv_forward;
 * dynconv_backward_weight, dynconv_balance_backward (adds to dalpha),
 * dynconv_route_backward, dynconv_backward_data; the sum over ranks;
 * dynconv_grad_norm, dynconv_adamw.
 * Warehouse cells are forward only (dynconv_cells.h): the balance loss and counts of
 * dynconv_route_cells' attentions are there to watch, and its gradient for a backward
 * of the caller's own; no call of this library takes it further.
 *
 * Conventions are those of dynconv.h: device pointers owned by the caller, work
 * enqueued on `stream` of the current device, nothing allocated, arguments
 * checked before anything is launched, negative status codes, deterministic
 * results (no floating-point atomics). The calls may be captured into CUDA
 * graphs; two calls in flight at once need two workspaces.
 */
#ifndef DYNCONV_TRAIN_H
#define DYNCONV_TRAIN_H

#include "dynconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- load-balance loss ---------------------------------------------------
 * For a router's attentions a[b][j][i] (row b, group j, expert i; one group for
 * dynconv_route, `cells` groups for dynconv_route_cells) over the M rows that
 * `row_mask` keeps:
 *
 *   p[b][j][i]   = a                                    (SOFTMAX: rows sum to 1)
 *                  a / S, S = sum_i a[b][j][i]; 0 if S = 0          (SIGMOID)
 *   counts[j][i] = kept rows in which a[b][j][i] is among the top_k largest of
 *                  its group (equal values: the lower index first; NaN last)
 *   mean[j][i]   = sum over kept b of p[b][j][i] / M
 *   loss         = coef * n / (top_k * groups) * sum_ji counts[j][i]/M * mean[j][i]
 *
 * so that perfectly even routing gives coef. M = 0 gives loss 0 and mean 0.
 * The gradient takes the counts as constants:
 *
 *   c[j][i]         = dloss * coef * n / (top_k * groups) * counts[j][i] / M^2
 *   dalpha[b][j][i] = c                                              (SOFTMAX)
 *                     (c[j][i] - sum_l c[j][l] p[b][j][l]) / S; 0 if S = 0  (SIGMOID)
 *
 * and 0 on the rows that the mask drops, or with M = 0.
 *
 * rows >= 0; 1 <= n <= 1024; 1 <= groups <= 65535 with groups * n <= 65536;
 * 1 <= top_k <= min(n, 32), or top_k = n; mode a dynconv_mode; row_stride >=
 * groups * n: floats from one row of alpha to the next (a row is contiguous).
 * Few rows (4096 attentions in the busiest of eight CTAs, n <= 256) take one
 * launch, others two. coef is fp32 like the tensors it scales: 0.01 is taken as the
 * nearest fp32 number, 2.2e-8 of it away, and the results follow that number. */
typedef struct {
  int rows, groups, n, top_k;
  int mode;
  long long row_stride;
} dynconv_balance_desc;

/* Bytes of device workspace of dynconv_balance_forward (0 on an invalid
 * descriptor). Pure host function. */
size_t dynconv_balance_workspace_size(const dynconv_balance_desc* desc);

/* Counts, mean probabilities and loss.
 *   alpha      fp32, [rows][groups][n] with row_stride
 *   row_mask   one byte per row, nonzero = kept, or NULL (all kept). Rows that
 *              it drops are not read into any result, whatever they hold.
 *   counts     int32 [groups][n]   (out)
 *   mean       fp32  [groups][n]   (out)
 *   rows_kept  int32 [1]: M        (out)
 *   loss       fp32  [1]           (out)
 *   workspace  at least dynconv_balance_workspace_size bytes, 16-byte aligned;
 *              contents need not be preserved.
 * The sums over rows keep fp64's precision (fp32 pairs with their rounding
 * errors, joined in fp64) and have a fixed order.
 * Errors: INVALID_ARG, UNSUPPORTED (a size above those limits), MISALIGNED (a
 * pointer not aligned to its element; the workspace), WORKSPACE, CUDA. */
int dynconv_balance_forward(const dynconv_balance_desc* desc, const float* alpha,
                            const unsigned char* row_mask, float coef, int* counts, float* mean,
                            int* rows_kept, float* loss, void* workspace, size_t workspace_bytes,
                            void* stream);

/* The gradient with respect to alpha.
 *   counts, rows_kept  from dynconv_balance_forward
 *   dloss      fp32 [1] on the device, or NULL for 1
 *   dalpha     fp32, [rows][groups][n] with dalpha_stride >= groups * n floats
 *              between rows; accumulate = 1: added to (rows that the mask drops
 *              are left as they were), 0: overwritten (zero on those rows).
 *              Must not overlap alpha.
 * alpha is read in SIGMOID mode only (it may be NULL in SOFTMAX mode).
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, CUDA. */
int dynconv_balance_backward(const dynconv_balance_desc* desc, const float* alpha,
                             const unsigned char* row_mask, float coef, const int* counts,
                             const int* rows_kept, const float* dloss, float* dalpha,
                             long long dalpha_stride, int accumulate, void* stream);

/* ---- a list of tensors -------------------------------------------------------
 * One parameter tensor with its gradient and optimizer state, all contiguous,
 * numel elements each. dynconv_grad_norm reads grad, grad_dtype and numel only.
 *   param       dtype (DYNCONV_F32 or DYNCONV_BF16), updated in place
 *   master      fp32 copy of a BF16 param, updated in place (param is then
 *               written, not read: the master rounded to nearest), or NULL. A
 *               BF16 param without one is updated in fp32 and rounded up or
 *               down at random (below), so that small steps are not lost.
 *   grad        grad_dtype
 *   m, v        state_bits 32: fp32 first and second moments;
 *               state_bits 8: e4m3 codes of m and of sqrt(v), one byte each
 *   m_scale, v_scale  state_bits 8: fp32 [ceil(numel / 256)], the factor of each
 *               block of 256 consecutive codes; else ignored. Zeroed codes and
 *               scales are the state before the first step.
 *   lr_scale    factor on the learning rate for this tensor
 *   weight_decay  decoupled: param is multiplied by 1 - lr * lr_scale * weight_decay
 * Pointers are aligned to their elements (16-byte aligned ones are faster). No
 * buffer may overlap another buffer that the call writes; a param given twice
 * in the list is refused. */
typedef struct {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long numel;
  int dtype;
  int grad_dtype;
  int state_bits;
  float lr_scale;
  float weight_decay;
} dynconv_train_tensor;

/* ---- norm of the gradients ---------------------------------------------------- */

/* Bytes of device workspace of dynconv_grad_norm for a list of `count` tensors.
 * Pure host function. */
size_t dynconv_grad_norm_workspace_size(int count);

/* stats[0] = sqrt(sum over all tensors of grad^2) (fp64 squares and sums, rounded
 * once), stats[1] = min(1, max_norm / (stats[0] + 1e-6)), the factor that
 * dynconv_adamw takes as grad_scale. A norm that is not finite gives stats[1] =
 * NaN, with which dynconv_adamw leaves everything as it was.
 *   stats  device fp32 [2]  (out)
 *   step   device int64 [1] or NULL: the number of the step, increased by one
 *          unless the norm is not finite
 *   workspace  at least dynconv_grad_norm_workspace_size(count) bytes, 16-byte
 *          aligned; contents need not be preserved.
 * count = 0 gives norm 0. max_norm > 0 (infinity: no clipping).
 * Errors: INVALID_ARG, MISALIGNED, WORKSPACE, CUDA. */
int dynconv_grad_norm(const dynconv_train_tensor* tensors, int count, double max_norm,
                      float* stats, long long* step, void* workspace, size_t workspace_bytes,
                      void* stream);

/* ---- AdamW ----------------------------------------------------------------------
 * For every element, in fp32 (t = the step's number, from 1):
 *
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr lr_scale weight_decay)
 *           - lr lr_scale / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * An 8-bit state is widened, advanced as above and stored again: per block of
 * 256 the scale is its largest magnitude / 448 (0 below 2^-100), and every value
 * x / scale goes to one of its two e4m3 neighbours, the nearer the likelier
 * (dithered rounding: no change is too small to count on average, which a
 * rounding to nearest would lose at beta2 near 1). sqrt(v) > 0 never becomes 0.
 * The update itself uses m and v before they are stored. A gradient that is not
 * finite spoils its block of 256 (grad_norm's factor skips such a step).
 *
 * The dither is a function of (seed, t, place in the list, element), 16 bits
 * u / 2^16 of a neighbour's distance: with F(x) = { x ^= x >> 16; x *= 0x9E3779B9;
 * x ^= x >> 15; x *= 0x6A09E667; x ^= x >> 16 } on 32-bit words (modulo 2^32),
 * K = F(F(F(seed) ^ t) ^ place), h = F(K ^ (element / 2)) gives the low half of
 * its bits to an even element and the high half to an odd one (from element 2^33
 * on, K ^= F(element >> 33) first). The same inputs give the same bits.
 *
 * lr >= 0, 0 <= beta < 1, 2^-126 <= eps <= 1e30, step >= 1. */
typedef struct {
  double lr, beta1, beta2, eps;
  long long step;
  unsigned int seed;
} dynconv_adamw_hyper;

/* One step over `count` tensors, in place.
 *   grad_scale  device fp32 [1] or NULL (1); not finite: nothing is changed
 *   lr          device fp32 [1] or NULL: the learning rate instead of hyper->lr
 *   step        device int64 [1] or NULL: t instead of hyper->step (read only)
 * With the three device pointers a captured step follows its schedule when it
 * is replayed.
 * Errors: INVALID_ARG (NULL pointers, bad sizes, enums or hyper-parameters, a
 * param twice), UNSUPPORTED (state_bits other than 8 and 32, numel >= 2^40),
 * MISALIGNED (a pointer not aligned to its element), CUDA. */
int dynconv_adamw(const dynconv_train_tensor* tensors, int count,
                  const dynconv_adamw_hyper* hyper, const float* grad_scale, const float* lr,
                  const long long* step, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DYNCONV_TRAIN_H */
