/*
 * gq_train.h -- C ABI of libgq's training operators: what stands between and
 * behind the message-passing layers of gq.h in a training step.  The
 * conventions of gq.h (device pointers, workspaces, streams, errors, thread
 * safety) hold here too.
 */
#ifndef GQ_TRAIN_H
#define GQ_TRAIN_H

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a matrix whose parameter is `const void*` / `void*`. */
typedef enum { GQ_F32 = 0, GQ_BF16 = 1, GQ_F16 = 2 } gq_type;

/* ------------------------------------------------------------------------
 * gq_dropout -- dropout of a matrix from the counter hash; the mask is never
 * stored.  No counterpart on the pages, whose training loops use it between
 * layers.
 *   Y[r,j] = X[r,j] * s  if h(seed, r, j) >= ceil(p * 2^23), else 0
 * with h the 23-bit noise code of gq_quantize_pack (u = h * 2^-23) and
 * s = (float)(1 / (1 - p)); the product is one fp32 operation, rounded once
 * to the type.  Dropped elements are +0 whatever X holds there (NaN and
 * infinity included).  The backward pass is the same call on dY with the
 * same p and seed.  Attention values are dropped the same way, as an
 * E x heads matrix (by a caller of the edge operators; gq_gat_layer_fwd and
 * _bwd drop none).  Bit-for-bit reproducible; independent of the leading
 * dimensions.  A call whose seed also drives a quantizer on the same rows
 * passes seed ^ GQ_DROPOUT_SEED_TAG, so that the two draw different noise.
 *   type   gq_type of X and Y (n x d, ldx, ldy >= d, any alignment of the
 *          type; 16-byte aligned rows take the vector path)
 *   p      in [0, 1]; 1 drops everything
 *   Y      may be X (ldy == ldx)
 * Errors: GQ_ERR_INVALID_ARG (bad type, p, n < 0, n >= 2^32, d < 1, short
 * leading dimension, null or misaligned pointers); GQ_ERR_UNSUPPORTED for
 * d > 2^31 - 4096; n == 0 is a no-op.
 * ---------------------------------------------------------------------- */
#define GQ_DROPOUT_SEED_TAG 0xD6E8FEB86659FD93ULL
GQ_API int gq_dropout(const void* X, int type, int64_t n, int d, int64_t ldx, double p, uint64_t seed, void* Y,
                      int64_t ldy, gq_stream stream);

/* ------------------------------------------------------------------------
 * Layer normalization of node rows, with the ReLU and the dropout that
 * follow it in a layer stack.  No counterpart on the pages.
 *
 * gq_layer_norm_fwd:
 *   mean[r] = (1/d) sum_j X[r,j]
 *   rstd[r] = 1 / sqrt((1/d) sum_j (X[r,j] - mean)^2 + eps)
 *   z = (X - mean) rstd gamma + beta;  Y = drop(act(z))
 *   drop is gq_dropout's with p and seed (p = 0: none).  mean, rstd
 *   (n fp32 each) and relu_bits (as in gq_gcn_layer_fwd: bit c % 32 of word
 *   relu_bits[r * ldrb + c / 32] = [z > 0], act = RELU only) are nullable;
 *   the backward pass needs them.  gamma, beta: d fp32; NULL: 1 and 0.
 *   Y may be X (ldy == ldx).  RELU keeps z where z > 0 and gives 0 elsewhere,
 *   for a NaN too (its bit is clear), as the layers' own ReLU does; without
 *   it a NaN in X fills its row of Y.
 * gq_layer_norm_bwd:
 *   dz = drop'(dY), with dz[r,c] = 0 where act = RELU and the bit is clear
 *   dgamma[j] = sum_r dz[r,j] xhat[r,j];  dbeta[j] = sum_r dz[r,j]
 *   g = dz gamma;  dX = rstd (g - mean_j(g) - xhat mean_j(g xhat))
 *   dgamma, dbeta (d fp32): nullable; zero when n == 0.  dx_type is `type`,
 *   or GQ_BF16 with GQ_F32 inputs: dX is then the dZ_in that
 *   gq_gcn_layer_bwd takes.  dX may be dY or X where type and leading
 *   dimension agree.  ws: gq_layer_norm_bwd_workspace_bytes(n, d) bytes
 *   (4-byte aligned; depends on the current device's SM count; not needed
 *   when dgamma and dbeta are NULL).
 * All sums run in fp32 in a fixed order; results are rounded once.
 * Matrices: n x d of `type` (gq_type), any alignment of the type; 16-byte
 * aligned rows take the vector path.
 * Errors: GQ_ERR_INVALID_ARG (bad type, act, p, eps < 0 or not finite,
 * n < 0, n >= 2^32, d < 1, short leading dimensions, null or misaligned
 * pointers, relu_bits without act = RELU, act = RELU backward without
 * relu_bits); GQ_ERR_UNSUPPORTED for d > 16384; GQ_ERR_WORKSPACE.
 * ---------------------------------------------------------------------- */
GQ_API int gq_layer_norm_fwd(const void* X, int type, int64_t n, int d, int64_t ldx, const float* gamma,
                             const float* beta, float eps, int act, double p, uint64_t seed, void* Y, int64_t ldy,
                             float* mean, float* rstd, uint32_t* relu_bits, int64_t ldrb, gq_stream stream);
GQ_API size_t gq_layer_norm_bwd_workspace_bytes(int64_t n, int d);
GQ_API int gq_layer_norm_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, int type, int64_t n, int d,
                             const float* mean, const float* rstd, const float* gamma, int act, double p,
                             uint64_t seed, const uint32_t* relu_bits, int64_t ldrb, void* dX, int dx_type,
                             int64_t lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                             gq_stream stream);

/* ------------------------------------------------------------------------
 * gq_linear_xent -- softmax cross entropy of a linear class head, with its
 * gradients; the logits are never kept.  No counterpart on the pages.
 *   Z = X W^T                       (n x C, fp32 sums of bf16 products)
 *   for a row with 0 <= labels[r] < C:
 *     lse[r]  = log sum_c exp(Z[r,c]);  loss[r] = lse[r] - Z[r, labels[r]]
 *       (one Z: a certain row's loss is 0 to within 2^-20, whatever the size of
 *       its logits, up to 1e38)
 *     G[r,c]  = weight[r] * (exp(Z[r,c] - lse[r]) - [c = labels[r]])
 *   for any other row (an unlabelled node, padding): loss = lse = 0, its
 *     row of dX is zero, and what X holds there enters nothing
 *   dX = scale G W,  dW = scale G^T X    (G in bf16, fp32 sums and scaling,
 *     rounded to bf16)
 * so dX and dW are the gradients of scale * sum_r weight[r] loss[r].
 *   X       n x k bf16 (ldx), W  C x k bf16 (ldw), one class per row
 *   labels  n int32;  weight: n fp32 or NULL (1);  scale: host value
 *   loss, lse: n fp32, nullable;  dX (n x k bf16), dW (C x k bf16):
 *           nullable; without both only the losses are computed
 *   bf16 matrices: 16-byte aligned, leading dimension a multiple of 8;
 *           columns past k are neither read as values nor written
 *   ws      gq_linear_xent_workspace_bytes(n, k, C, need_grad) bytes,
 *           256-byte aligned, need_grad != 0 when dX or dW is given.  With n
 *           and k rounded up to multiples of 256 and 8: 2 n k + 16 n bytes;
 *           for t = ceil(C / 256) > 1 another 4 n + 16 n ceil(t / run), where
 *           run = n t / (1024 SMs), at least 1 and at most 16; with gradients
 *           two pieces of G (2 n c bytes each, c classes a piece: at most
 *           1 GB, but no fewer than C or 256 classes; one if it holds every
 *           class), 16 n for t > 1 and, where sums are split or carried from
 *           piece to piece, 4 n k bytes for each split of dX's, 4 c k of dW's
 *           (k a multiple of 128).  It depends on the current device's SM
 *           count.  Calls sharing one workspace must not overlap.
 *   dev_err nullable device int, as for the GEMMs (codes 21 .. 26).  Without it
 *           a bounded wait that gave up, and left results half made, is not
 *           reported
 * Results are the same from run to run.  dX and dW must not overlap X or W.
 * Errors: GQ_ERR_INVALID_ARG (null X, W or labels, n < 0, k < 1, C < 1, bad
 * leading dimensions or alignment); GQ_ERR_UNSUPPORTED for k > 16384,
 * n > 2^28, C > 2^30 or ceil(n / 256) * ceil(C / 64) >= 2^29;
 * GQ_ERR_WORKSPACE.  n == 0 writes dW = 0.
 * ---------------------------------------------------------------------- */
GQ_API size_t gq_linear_xent_workspace_bytes(int64_t n, int k, int C, int need_grad);
GQ_API int gq_linear_xent(const uint16_t* X, int64_t n, int k, int64_t ldx, const uint16_t* W, int C, int64_t ldw,
                          const int32_t* labels, const float* weight, float scale, float* loss, float* lse,
                          uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, void* ws, size_t ws_bytes,
                          int* dev_err, gq_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* GQ_TRAIN_H */
