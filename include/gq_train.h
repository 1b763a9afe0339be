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

/* ------------------------------------------------------------------------
 * Products of 8-bit integers with a scale for each row of both operands
 * (Tango Sec. 3.2: the update's products on quantized operands), with the
 * quantizers and the linear layer made of them.
 *
 * gq_quantize_i8: for every row i of X (n x d of `type`), or with transpose
 * for every column i, whose codes are then row i of Q (d rows of n):
 *   scale[i] = max |x| / 127 (fp32);  Q[i,.] = x / scale[i] rounded to the nearest
 *   integer, ties to even, decided exactly;  |Q| <= 127
 *   A row whose largest magnitude is below 2^-100 has scale and codes 0.  One
 *   that holds a NaN or an infinity has scale NaN and codes 0.
 *   Q is 16-byte aligned, ldq a multiple of 16 and at least the row's length;
 *   bytes behind a row's last code, up to the next multiple of 4, may be written.  ws (transpose only):
 *   gq_quantize_i8_workspace_bytes bytes, 16-byte aligned.
 * gq_gemm_i8: C = act(diag(scale_a) A B^T diag(scale_b) + bias)
 *   A m x k, B n x k, any int8 values (16-byte aligned, lda and ldb multiples
 *   of 16; the bytes of a row up to the next multiple of 16 are read, and count
 *   for nothing); C m x n of `type` (gq_type), any alignment; bias n fp32 or NULL.
 *   The sum over k is exact; (float)sum times one scale, times the other plus
 *   bias, is rounded at each step and once more to the type.  act = RELU gives 0 for
 *   a NaN.  ws: gq_gemm_i8_workspace_bytes(m, n, k), 256-byte aligned (operands
 *   as fp16, the sums of a split contraction; 0 for few rows; depends on the
 *   device's SM count).  dev_err as for the GEMMs (codes 31 .. 48).
 * gq_linear_i8: Y = act(X W^T + bias) with X's rows (n x k) quantized in the call
 *   and W (out x k) as gq_quantize_i8 left it.
 * gq_linear_i8_bwd, W (out x k) and X in full precision, each product of
 *   quantized operands with a scale for each row or column that is not summed over:
 *   dX = dY W (dY by rows, W by columns);  dW = dY^T X (both by columns);
 *   dbias[j] = sum_r dY[r,j] (fp32 in a fixed order, its parts joined without loss).
 *   dX, dW, dbias: nullable, dbias only with dW; W is not read without dX, X not without dW.
 *   n == 0 gives dW = 0, dbias = 0.
 * ws of both: the ..._workspace_bytes bytes, 256-byte aligned.  Calls sharing a
 * workspace must not overlap.  Outputs must not overlap inputs.  Results are
 * the same from run to run.
 * Errors: GQ_ERR_INVALID_ARG (bad types, act, negative or zero sizes, short or
 * unaligned leading dimensions, null or misaligned pointers);
 * GQ_ERR_UNSUPPORTED for sizes beyond 2^30, or 2,097,120 columns of a matrix
 * to be quantized; GQ_ERR_WORKSPACE.  n == 0 (m == 0) is a no-op.
 * ---------------------------------------------------------------------- */
GQ_API size_t gq_quantize_i8_workspace_bytes(int64_t n, int d, int transpose);
GQ_API int gq_quantize_i8(const void* X, int type, int64_t n, int d, int64_t ldx, int transpose, int8_t* Q,
                          int64_t ldq, float* scale, void* ws, size_t ws_bytes, gq_stream stream);
GQ_API size_t gq_gemm_i8_workspace_bytes(int64_t m, int64_t n, int64_t k);
GQ_API int gq_gemm_i8(const int8_t* A, int64_t m, int64_t lda, const float* scale_a, const int8_t* B, int64_t n,
                      int64_t ldb, const float* scale_b, int64_t k, const float* bias, int act, void* C, int type,
                      int64_t ldc, void* ws, size_t ws_bytes, int* dev_err, gq_stream stream);
GQ_API size_t gq_linear_i8_workspace_bytes(int64_t n, int k, int out);
GQ_API int gq_linear_i8(const void* X, int type, int64_t n, int k, int64_t ldx, const int8_t* W, int out,
                        int64_t ldw, const float* scale_w, const float* bias, int act, void* Y, int y_type,
                        int64_t ldy, void* ws, size_t ws_bytes, int* dev_err, gq_stream stream);
GQ_API size_t gq_linear_i8_bwd_workspace_bytes(int64_t n, int k, int out, int need_dx, int need_dw);
GQ_API int gq_linear_i8_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, int type, int64_t n, int k,
                            int out, const void* W, int w_type, int64_t ldw, void* dX, int dx_type, int64_t lddx,
                            void* dW, int dw_type, int64_t lddw, float* dbias, void* ws, size_t ws_bytes,
                            int* dev_err, gq_stream stream);

/* ------------------------------------------------------------------------
 * Group normalization of segments of rows, with the activation that follows
 * it: the nodes of each graph of a batch are consecutive rows, channels last.  No
 * counterpart on the pages.
 *   segment j: rows ptr[j] .. ptr[j+1] - 1 (ptr: segments + 1 device int64, rising;
 *   NULL with segments = 1: all rows).  Groups of d / groups consecutive
 *   channels.  Over a segment's rows and a group's channels (N cells):
 *     mean = sum x / N;  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
 *     z = (x - mean) rstd gamma + beta;  Y = act(z)
 *   act: GQ_ACT_NONE, GQ_ACT_RELU (0 for a NaN) or GQ_ACT_SILU, z / (1 + exp(-z)).
 *   mean, rstd: segments x groups fp32, which the backward pass takes; an empty
 *   segment's are 0 and 1 / sqrt(eps).  groups = 1 is layer normalization over
 *   a whole graph, groups = d normalizes each channel (instance norm).
 * gq_group_norm_bwd: dz = dY act'(z), z recomputed; h = dz gamma;
 *     dX = rstd (h - mean(h) - xhat mean(h xhat));  dgamma[c] = sum dz xhat;
 *     dbeta[c] = sum dz, over all segments (nullable)
 *   Rows outside every segment are neither read nor written.  Offsets outside
 *   [0, n] are taken as the nearest inside.  max_rows: the longest segment's rows,
 *   or 0 if the caller does not know; it chooses between kernels, a wrong value
 *   costs time only.  gamma, beta: d fp32; NULL: 1 and 0.  Y may be X, dX may be
 *   dY or X (same leading dimension).  Matrices: n x d of `type`, any alignment of
 *   the type; rows of a multiple of 4 values that start aligned for 4 take the
 *   vector path.  Sums run in fp32 in a fixed order; results are rounded once.
 *   Sums of a segment's rows, and squares of x - mean, that leave fp32's range
 *   (|x| rows > 3.4e38, |x - mean| > 1.8e19) make the statistics infinite or NaN.
 *   ReLU's derivative is 1 exactly where forward's z, rounded as there, is above 0.
 *   ws: gq_group_norm_workspace_bytes(n, d, groups, type, segments, max_rows,
 *   backward), 256-byte aligned; it depends on the device's SM count.
 * Errors: GQ_ERR_INVALID_ARG (bad type, act, sizes, eps; d not a multiple of
 * groups; short leading dimensions; null or misaligned pointers; ptr NULL with
 * segments != 1); GQ_ERR_UNSUPPORTED for d > 16384, n >= 2^31, segments > 2^30
 * or segments * groups >= 2^31; GQ_ERR_WORKSPACE.
 * ---------------------------------------------------------------------- */
#define GQ_ACT_SILU 2 /* group normalization only */
GQ_API size_t gq_group_norm_workspace_bytes(int64_t n, int d, int groups, int type, int64_t segments,
                                            int64_t max_rows, int backward);
GQ_API int gq_group_norm_fwd(const void* X, int type, int64_t n, int d, int64_t ldx, int groups, const int64_t* ptr,
                             int64_t segments, int64_t max_rows, const float* gamma, const float* beta, float eps,
                             int act, void* Y, int64_t ldy, float* mean, float* rstd, void* ws, size_t ws_bytes,
                             gq_stream stream);
GQ_API int gq_group_norm_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, int type, int64_t n, int d,
                             int groups, const int64_t* ptr, int64_t segments, int64_t max_rows, const float* mean,
                             const float* rstd, const float* gamma, const float* beta, int act, void* dX,
                             int64_t lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                             gq_stream stream);

/* ------------------------------------------------------------------------
 * gq_adamw_step -- one AdamW step over many tensors at once.  No counterpart on
 * the pages.  With t the step's number (1 for the first) and g the gradient
 * times *grad_scale:
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32, p rounded once to its type.
 *   tensors  `count` of them (host memory, read by the call); each n values:
 *            p (p_type), g (g_type), and the moments m and v (dense)
 *     cols   0: p and g are dense.  Otherwise rows of `cols` values with
 *            leading dimensions ldp and ldg (n a multiple of cols); what lies
 *            between the rows is neither read nor written
 *     m, v   state_bits 32: n fp32 each.  state_bits 8: n codes each, and in
 *            m_exp, v_exp an exponent byte for each 256 values (the last block
 *            may be short).  A first moment is sign, 4 exponent bits, 3 of
 *            mantissa, a second 4 and 4; with x the exponent bits, f the others
 *            and b of them: (1 + f / 2^b) 2^(x - 7), or f 2^(-6 - b) where x = 0,
 *            times 2^(e - 134) (first) or 2^(e - 135) (second).  All zeros is 0.
 *            New codes are rounded down or up at random by the counter hash
 *            of (seed + t 0x9E3779B97F4A7C15, block0 + block, place in the block):
 *            its upper 20 bits for m, its lower 19 for v; a v > 0 is never
 *            rounded to 0.  e lies in [16, 254], which keeps 2^-111 to 2^127, and
 *            is that of the block's largest finite value: of values 2^17 times
 *            smaller a first moment is rounded to 0 but for one draw in many, a
 *            second (2^19) to its least code.  No code is above 31/16 of the power of
 *            two below a block's largest second moment, which is therefore not rounded
 *            up beyond it: it grows into the next octave only in a step that adds a
 *            32nd of it, and with beta2 = 0.999 stays behind its 32-bit value (half of
 *            it on average, a quarter at worst).  A moment that is not finite takes
 *            the greatest code and leaves its block's others alone; p is NaN where
 *            m is not finite, and only decays where the square of |g| > 1.8e19
 *            makes v infinite (32-bit moments stay so)
 *     block0 the number of the tensor's first block in the noise; tensors with
 *            ranges of their own draw different noise
 *   args->grad_scale  device fp32 or NULL (1).  Where it is not finite the
 *            step is left out: nothing is written
 *   args->dev  NULL, or gq_adamw_dev_bytes() of device memory (8-byte aligned)
 *            that begin with an int64 step number and a double lr: the call
 *            takes lr from there and, with args->advance, counts the step
 *            number up first (unless the step is left out), so that a captured
 *            call counts at every replay.  args->lr and args->step are not
 *            used then.  Calls of one step on several lists of tensors advance
 *            in the first one
 * No tensor may appear twice or overlap another.  Results are the same from
 * run to run.
 * Errors: GQ_ERR_INVALID_ARG (null or misaligned pointers, bad types or bits,
 * betas outside [0, 1), eps < 0, values that are not finite, step < 1, n or
 * cols < 0, n not a multiple of cols, short leading dimensions, block0 outside
 * 32 bits); GQ_ERR_UNSUPPORTED for n > 2^40.  n = 0 is skipped.
 *
 * gq_adam_moment: the values (fp32, bf16 or fp16, dense) of n 8-bit codes of a
 * first (second = 0) or second moment.
 * ---------------------------------------------------------------------- */
typedef struct {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* m_exp;
  uint8_t* v_exp;
  int64_t n, cols, ldp, ldg, block0;
} gq_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  uint64_t seed;
  const float* grad_scale;
  void* dev;
  int32_t advance;
} gq_adamw_args;

GQ_API size_t gq_adamw_dev_bytes(void);
GQ_API int gq_adamw_step(const gq_adamw_tensor* tensors, int count, int p_type, int g_type, int state_bits,
                         const gq_adamw_args* args, gq_stream stream);
GQ_API int gq_adam_moment(const uint8_t* codes, const uint8_t* exps, int64_t n, int second, void* out, int type,
                          gq_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* GQ_TRAIN_H */
