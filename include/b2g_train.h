/*
 * b2g_train.h -- C ABI of the operators that a language model's training and
 * scoring steps run around their matrix products: layer norm, embedding
 * lookup, softmax cross entropy of a linear layer, and clipping by the global
 * gradient norm.  Part of the library behind b2g_sgemm.h, with its rules:
 * DEVICE pointers owned by the caller, row-major operands with leading
 * dimensions in elements, calls that are asynchronous on `stream` (a
 * cudaStream_t, NULL = the legacy default stream), thread-safe, and a 0 or a
 * negative B2G_ERR_* code as the result.
 *
 * Element types: every tensor of a call has the type `dtype` names, B2G_F32
 * (IEEE binary32) or B2G_BF16 (bfloat16), unless its pointer type says
 * otherwise.  Sums, means, norms, softmax statistics and gradients' partial
 * sums are held in FP32 and each result is rounded once to its type.
 *
 * Workspaces: a call that needs one takes it from the caller (16-byte aligned
 * device memory; its size comes from the ..._workspace_size query next to it,
 * which launches nothing) and never allocates, so every call may be captured
 * into a CUDA graph.  The contents need not be initialised and are not kept.  A
 * workspace that is NULL or too small is B2G_ERR_WORKSPACE.  The caller orders
 * its reuse across streams.
 *
 * Results are the same bits run to run for given arguments: every sum has a
 * fixed order, and no floating-point atomics are used.
 *
 * Sizes: row lengths, vocab and the cross entropy's tokens are at most 2^31 - 2^16,
 * layer norm's rows 2^31 - 1 and the embedding's tokens 2^30, else B2G_ERR_INVALID_DIM.
 *
 * Alignment: any multiple of the element's size.  Operands whose base is 16-byte aligned and whose leading
 * dimensions (and width) are multiples of 16 bytes run with 16-byte accesses.
 */
#ifndef B2G_TRAIN_H
#define B2G_TRAIN_H

#include <stddef.h>

#include "b2g_sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define B2G_F32 0
#define B2G_BF16 1

#define B2G_ERR_INVALID_TYPE (-12) /* dtype is neither B2G_F32 nor B2G_BF16 */
#define B2G_ERR_WORKSPACE (-13)    /* the workspace is NULL, misaligned or too small */
#define B2G_ERR_INDEX (-14)        /* b2g_status(): an id or target was out of range */

/*
 * Layer norm of each row of x (rows x cols):
 *     mean = sum_j x_j / cols,  var = sum_j (x_j - mean)^2 / cols,
 *     rstd = 1 / sqrt(var + eps),  y_j = (x_j - mean) * rstd * weight_j + bias_j.
 *   weight, bias  cols values each; NULL weight: ones; NULL bias: zeros.
 *   mean, rstd    rows FP32 values each, for the backward pass; either may be NULL.
 *   eps           >= 0 (else B2G_ERR_INVALID_DIM).
 * y may be x itself (same leading dimension) and must not overlap it otherwise.
 * rows == 0 or cols == 0: nothing is launched, and nothing written.
 */
int b2g_layernorm(int dtype, long long rows, int cols, const void* x, long long ldx,
                  const void* weight, const void* bias, float eps, void* y, long long ldy,
                  float* mean, float* rstd, void* stream);

/*
 * Gradients of b2g_layernorm.  With xhat = (x - mean) * rstd and g = dy * weight:
 *     dx      = rstd * (g - mean_j(g) - xhat * mean_j(g * xhat)),
 *     dweight = sum over the rows of dy * xhat,   dbias = sum over the rows of dy.
 *   mean, rstd        what b2g_layernorm stored for x.
 *   dweight, dbias    cols values each; either may be NULL.  rows == 0 writes zeros.
 * dx may be dy itself (same leading dimension); no other overlap.
 */
int b2g_layernorm_backward(int dtype, long long rows, int cols, const void* dy, long long lddy,
                           const void* x, long long ldx, const void* weight, const float* mean,
                           const float* rstd, void* dx, long long lddx, void* dweight, void* dbias,
                           void* workspace, size_t workspace_bytes, void* stream);
int b2g_layernorm_backward_workspace_size(int dtype, long long rows, int cols, size_t* bytes);

/*
 * Embedding lookup: out_i = scale * table[ids_i], one row per token.
 *   ids    `tokens` row numbers, 64-bit (id_bytes == 8) or 32-bit (id_bytes == 4)
 *          signed; any other id_bytes is B2G_ERR_INVALID_TYPE.
 *   table  vocab x width, ldt >= max(1, width).   out  tokens x width, ldo.
 * An id outside [0, vocab) reads nothing: its row is filled with NaN and the
 * status word's bit 16 is set, which b2g_status() reports as B2G_ERR_INDEX.
 */
int b2g_embedding(int dtype, long long tokens, int vocab, int width, const void* ids, int id_bytes,
                  const void* table, long long ldt, float scale, void* out, long long ldo,
                  void* stream);

/*
 * The table's gradient: dtable_v = scale * (sum of dout_i over the tokens with
 * ids_i == v), plus dtable_v's previous value when accumulate != 0 (otherwise
 * dtable is write-only and rows without a token become zero).  A row's tokens
 * are added in a fixed order in FP32, wherever they stand in ids.
 *   padding   the tokens with this id are left out (a negative number: none).
 * An id outside [0, vocab) is left out and sets the status word's bit 16.
 * tokens is at most 2^30, else B2G_ERR_INVALID_DIM.
 */
int b2g_embedding_backward(int dtype, long long tokens, int vocab, int width, const void* ids,
                           int id_bytes, const void* dout, long long ldd, float scale,
                           long long padding, int accumulate, void* dtable, long long ldt,
                           void* workspace, size_t workspace_bytes, void* stream);
int b2g_embedding_backward_workspace_size(int dtype, long long tokens, int vocab, int width,
                                          size_t* bytes);

/*
 * Softmax cross entropy of a linear layer, without storing its logits.  With
 * z = h * w^T (tokens x vocab, FP32):
 *     lse_i = log(sum_j exp(z_ij)),   loss_i = lse_i - z_{i, target_i}.
 *   h       tokens x width, ldh.   w  vocab x width, ldw (the head, one row per class).
 *   target  `tokens` class numbers, id_bytes 8 or 4 as for b2g_embedding.
 *           ignore_index rows get loss 0; any other target outside [0, vocab)
 *           gets loss NaN and sets the status word's bit 16.
 *   loss    `tokens` FP32 values, or NULL.   lse  `tokens` FP32 values.
 * tokens == 0 launches nothing; vocab and width are at least 1, else
 * B2G_ERR_INVALID_DIM.
 * BF16 operands are multiplied exactly and summed in FP32; FP32 operands are
 * split into three BF16 pieces each, whose six leading products carry 24 bits: they
 * must be finite (an infinity's pieces make its row's results NaN).
 */
int b2g_linear_xent(int dtype, int tokens, int vocab, int width, const void* h, long long ldh,
                    const void* w, long long ldw, const void* target, int id_bytes,
                    long long ignore_index, float* loss, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * Gradients of sum_i grad_loss_i * loss_i.  With
 *     dz_ij = grad_loss_i * (exp(z_ij - lse_i) - [j == target_i])
 * (zero in rows whose target is ignore_index or out of range, whatever lse_i and
 * grad_loss_i are),
 *     dh = dz * w,   dw = dz^T * h  (plus dw's previous value when accumulate != 0).
 * z is computed again, a piece of the vocabulary at a time; dz exists for one
 * piece at a time, rounded to BF16 (BF16 operands) or held in three BF16 pieces
 * (FP32 operands) for the two products.
 * A row without a gradient still enters dw as 0 * h_i, so its h must be finite.
 *   lse        what b2g_linear_xent stored.   grad_loss  `tokens` FP32 values.
 *   dh         tokens x width, lddh, or NULL.   dw  vocab x width, lddw, or NULL.
 */
int b2g_linear_xent_backward(int dtype, int tokens, int vocab, int width, const void* h,
                             long long ldh, const void* w, long long ldw, const void* target,
                             int id_bytes, long long ignore_index, const float* lse,
                             const float* grad_loss, void* dh, long long lddh, int accumulate,
                             void* dw, long long lddw, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Workspace bytes of b2g_linear_xent (backward == 0) or
 * b2g_linear_xent_backward (backward != 0) for these arguments.  h and w are
 * inspected for their alignment only: BF16 operands that are not on 16-byte
 * boundaries (base or leading dimension) are copied into the workspace first,
 * FP32 operands always (as BF16 pieces), except that up to 64 tokens read a w on
 * 16-byte boundaries where it is.  The backward pass also holds one piece of dz
 * there, at most about 512 MB.
 */
int b2g_linear_xent_workspace_size(int dtype, int tokens, int vocab, int width, const void* h,
                                   long long ldh, const void* w, long long ldw, int backward,
                                   size_t* bytes);

/*
 * The 2-norm of all elements of `count` tensors together, sqrt(sum x^2), in
 * *norm (device, FP32).  tensors and numels are HOST arrays of device pointers
 * and of element counts (>= 0; a NULL pointer is allowed where the count is 0);
 * they may be freed when the call returns.  Each tensor is contiguous.
 */
int b2g_grad_norm(int dtype, int count, const void* const* tensors, const long long* numels,
                  float* norm, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Clipping by that norm: out = x * min(1, max_norm / (norm + 1e-6)) for every
 * tensor.  outs is a HOST array like tensors; outs[i] may be tensors[i] (in
 * place) and must not overlap any tensor otherwise.  max_norm >= 0, else
 * B2G_ERR_INVALID_DIM.  A norm of infinity multiplies by 0, a NaN norm by NaN.
 */
int b2g_clip_grad_norm(int dtype, int count, const void* const* tensors, const long long* numels,
                       float max_norm, void* const* outs, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream);
int b2g_grad_norm_workspace_size(int dtype, int count, const long long* numels, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* B2G_TRAIN_H */
