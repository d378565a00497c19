/*
 * mmaops.h -- C ABI of the native training operators in libmmaemu.so.
 *
 * The emulated GEMM of mmaemu.h settles the bits of a matrix product as
 * another GPU computed it.  These operators are what a program that replays
 * a training or serving step on an MI355X runs around it, in the card's own
 * arithmetic (FP32 sums, one rounding of each output): the layer norm
 * before a product, the product with its epilogue, the 8-bit checkpoints
 * that a forward pass leaves, and the backward passes that use them.  The
 * same call on the same inputs gives the same bits, and an output's bits do
 * not depend on which others are asked for, so a forward pass and its
 * recomputation can be compared word for word (AEGIS, "Redundancy already
 * exists in the training computation").  The order of a product's sums, and
 * so the last bits, goes with the sizes (M too: a row's result beside other
 * rows is not that of the row alone), the weight's layout, and with whether
 * the operands' rows start on 16 bytes and how far apart they are.
 *
 * OPERATORS
 *   mma_layer_norm            for each row: mu = mean(x),
 *                             r = 1 / sqrt(mean((x - mu)^2) + eps),
 *                             y = (x - mu) r w + b; mu and r are written too
 *   mma_layer_norm_backward   xh = (x - mu) r, h = dy w,
 *                             dx = r (h - mean(h) - xh mean(h xh)),
 *                             dw = sum over rows of dy xh, db = of dy
 *   mma_linear                z = X W + b, Y = act(z) + residual
 *   mma_linear_backward       dz = dY act'(z), db = sum over rows of dz,
 *                             dX = dz W^T, dW = X^T dz
 *   mma_checkpoint, mma_restore   x to 8 bits and back
 *   mma_gated_linear          g = X Wg + bg, u = X Wu + bu, Y = act(g) u
 *   mma_gated_linear_backward dg = dY u act'(g), du = dY act(g), their sums
 *                             over the rows, dX = dg Wg^T + du Wu^T,
 *                             dWg = X^T dg, dWu = X^T du
 *   mma_dropout               y = m x / (1 - p) + residual, m 0 with
 *                             probability p, else 1; its backward pass is
 *                             the same of dY
 *   mma_residual_norm         v = post(branch), R = scale X + gate drop(v),
 *                             H = pre(R): the sum of a block's output into
 *                             the residual stream, with the norm after that
 *                             block and the one before the next, each a layer
 *                             norm, an rms norm (a layer norm with mu = 0) or
 *                             none; H is made from R before its rounding
 *   mma_residual_norm_backward   t = dR + pre'(dH), dX = scale t,
 *                             dbranch = post'(gate drop(t)), and the gradients
 *                             of the five vectors, sums over the rows
 *
 * DROPOUT
 *   A mask is never stored: it is a function of an element's place and the
 *   call's seed and offset, and the backward pass, or a replay, makes it again.
 *   Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
 *   numbers: as easy as 1, 2, 3", 2011) of the counter (row * 2^24 + column /
 *   8, offset), both of 64 bits with the lower word first, under the key seed
 *   (the lower word first) gives four words for eight columns; column c has
 *   half c mod 2 (the lower one first) of word (c mod 8) / 2.  An element is kept where
 *   these 16 bits are at least T = round(65536 p), and 1 / (1 - p) is 65536 /
 *   (65536 - T) (0 where T = 65536): p is met to within 2^-17, the mean
 *   exactly.  What is dropped is 0 whatever it was.  state: NULL, or device
 *   memory with (seed, offset) that the call reads when it runs, in the place
 *   of its two arguments: a captured graph draws anew when they change.
 *
 * CHECKPOINTS
 *   codes   rows x cols E4M3 codes (OCP "FN"), contiguous
 *   scales  rows x ceil(cols / 32) bytes: e + 127 for each block of 32
 *           consecutive elements of a row, where 2^e is the smallest power
 *           of two, -117 <= e <= 120, with max |x| <= 448 * 2^e over the
 *           block's finite elements (e = -117 for a block without any)
 *   A code is x / 2^e rounded to nearest, ties to even; a code restores to
 *   code * 2^e, which the type that was saved holds exactly (a
 *   pre-activation that mma_linear saves as FP16 comes from FP32 sums: below
 *   FP16's 2^-24 its restored matrix is rounded, what mma_linear_backward
 *   reads of it is not).  Magnitudes above 61440 (FP16) or 1.875 * 2^127 are
 *   saved as that bound, so that no code restores to an infinity.  NaN and
 *   infinities are saved as the code 0xFF, NaN (E4M3 has no infinity), and
 *   do not enter the block's maximum.  Where an operator reads a checkpoint,
 *   codes and scales stand in the place of the matrix, which is then NULL.
 *   codes are read and written in whole words where they and the row length
 *   allow it; no alignment is asked.
 *
 * MEMORY
 *   Every pointer is a DEVICE pointer on the current HIP device, owned by
 *   the caller and aligned to its elements.  Matrices are row-major with a
 *   leading dimension in elements (ld >= the row length); sizes may be odd
 *   and zero (an empty output is a no-op; sums over no rows are +0; with
 *   K = 0 a product is 0).  cols of a layer norm is at least 1; row lengths
 *   and the sizes of a product are at most 2^27.  Outputs
 *   may not overlap any input or each other, except dX over dY of a layer
 *   norm (exactly, with the same leading dimension).
 *   WORKSPACE.  The library allocates nothing here: a call that needs
 *   scratch memory takes it from the caller (device memory, 256-byte
 *   aligned, contents undefined, free again once the stream has run the
 *   call), of at least the size that its ..._workspace function returns
 *   for the same sizes, or for a product the same arguments (an operand
 *   whose rows do not start on 16 bytes, or lie too far apart, is copied
 *   to the workspace for some shapes).  A smaller one is MMAEMU_ERR_SCRATCH.  Calls can
 *   so be captured into a graph, and need no synchronisation.
 *
 * TYPES
 *   dtype is MMAEMU_DTYPE_FP16, MMAEMU_DTYPE_BF16 or (not for products)
 *   MMAOPS_DTYPE_FP32.  Weights, biases and outputs that may also be FP32
 *   have a type of their own, which is dtype or FP32.
 *
 * ERRORS are mmaemu.h's codes, reported before anything is enqueued;
 * mma_ops_strerror gives their text.  Calls are enqueued on hip_stream
 * (NULL = null stream) and return after enqueue.
 */
#ifndef MMAOPS_H
#define MMAOPS_H

#include "mmaemu.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MMAOPS_DTYPE_FP32 = 3 };

/* activations: none, max(z, 0), z Phi(z), its tanh form
 * z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2, z / (1 + exp(-z)) */
enum {
  MMAOPS_ACT_NONE = 0,
  MMAOPS_ACT_RELU = 1,
  MMAOPS_ACT_GELU = 2,
  MMAOPS_ACT_GELU_TANH = 3,
  MMAOPS_ACT_SILU = 4
};

/* Layer norm of the rows of X (rows x cols).  weight and bias: cols values
 * of param_dtype, or NULL (1 and 0).  mean and rstd: rows floats each, or
 * both NULL.  codes and scales: both NULL, or the checkpoint of X, written
 * in the same pass over X. */
int mma_layer_norm(int dtype, int param_dtype, const void *X, int64_t ldx,
                   const void *weight, const void *bias, void *Y, int64_t ldy,
                   float *mean, float *rstd, uint8_t *codes, uint8_t *scales,
                   int64_t rows, int64_t cols, float eps, void *hip_stream);

/* Its backward pass.  X, or codes and scales, hold the forward pass's
 * input.  dX, dweight, dbias: any of them NULL to leave it out; dweight
 * and dbias are of param_dtype. */
int mma_layer_norm_backward(int dtype, int param_dtype, const void *dY, int64_t lddy,
                            const void *X, int64_t ldx, const uint8_t *codes,
                            const uint8_t *scales, const void *weight, const float *mean,
                            const float *rstd, void *dX, int64_t lddx, void *dweight,
                            void *dbias, int64_t rows, int64_t cols, void *workspace,
                            int64_t workspace_bytes, void *hip_stream);
int64_t mma_layer_norm_backward_workspace(int64_t rows, int64_t cols);

/* The checkpoint of X (rows x cols), and its values as a matrix of dtype. */
int mma_checkpoint(int dtype, const void *X, int64_t ldx, uint8_t *codes, uint8_t *scales,
                   int64_t rows, int64_t cols, void *hip_stream);
int mma_restore(int dtype, const uint8_t *codes, const uint8_t *scales, void *Y, int64_t ldy,
                int64_t rows, int64_t cols, void *hip_stream);

/* Y = act(X W + bias) + residual.  X is M x K, W is K x N, stored row-major
 * (w_transposed = 0, ldw >= N) or as its transpose, N x K row-major
 * (w_transposed = 1, ldw >= K). */
typedef struct {
  int32_t dtype;        /* of X and W: FP16 or BF16 */
  int32_t out_dtype;    /* of Y and residual: dtype or FP32 */
  int32_t bias_dtype;   /* dtype or FP32 */
  int32_t activation;   /* MMAOPS_ACT_... */
  int32_t w_transposed; /* 0 or 1 */
  int32_t reserved;     /* 0 */
  int64_t M, N, K;
  const void *X;
  int64_t ldx;
  const void *W;
  int64_t ldw;
  const void *bias;     /* N values, or NULL */
  const void *residual; /* M x N, or NULL */
  int64_t ldr;
  void *Y;
  int64_t ldy;
  void *Z;              /* NULL, or M x N of dtype: X W + bias */
  int64_t ldz;
  uint8_t *codes;       /* both NULL, or the checkpoint of X W + bias */
  uint8_t *scales;
} mma_linear_args;

int mma_linear(const mma_linear_args *args, void *workspace, int64_t workspace_bytes,
               void *hip_stream);
int64_t mma_linear_workspace(const mma_linear_args *args);

/* The backward pass of mma_linear (the gradient of residual is dY itself).
 * X and Z: matrices or checkpoints; neither Z nor its checkpoint is read
 * where activation is NONE.  dX, dW, dbias: any of them NULL to leave it
 * out.  dz enters the two products rounded to dtype; dbias sums it before
 * that rounding.  Where a kept Z is infinite (past the range of its 16 bits)
 * act' is its limit, 0 or 1. */
typedef struct {
  int32_t dtype;        /* of dY, X, W, Z and dX */
  int32_t dw_dtype;     /* of dW: dtype or FP32 */
  int32_t bias_dtype;   /* of dbias: dtype or FP32 */
  int32_t activation;
  int32_t w_transposed; /* of W and dW */
  int32_t reserved;     /* 0 */
  int64_t M, N, K;
  const void *dY;       /* M x N */
  int64_t lddy;
  const void *X;        /* M x K, or NULL with x_codes and x_scales */
  int64_t ldx;
  const uint8_t *x_codes;
  const uint8_t *x_scales;
  const void *W;
  int64_t ldw;
  const void *Z;        /* M x N, or NULL with z_codes and z_scales */
  int64_t ldz;
  const uint8_t *z_codes;
  const uint8_t *z_scales;
  void *dX;             /* M x K */
  int64_t lddx;
  void *dW;             /* stored as W is */
  int64_t lddw;
  void *dbias;          /* N values */
} mma_linear_backward_args;

int mma_linear_backward(const mma_linear_backward_args *args, void *workspace,
                        int64_t workspace_bytes, void *hip_stream);
int64_t mma_linear_backward_workspace(const mma_linear_backward_args *args);

/* Y = act(X Wg + bias_g) (X Wu + bias_u), the weights stored alike as in
 * mma_linear, with leading dimensions of their own. */
typedef struct {
  int32_t dtype;        /* of X and the weights: FP16 or BF16 */
  int32_t out_dtype;    /* of Y: dtype or FP32 */
  int32_t bias_dtype;   /* dtype or FP32 */
  int32_t activation;   /* MMAOPS_ACT_... */
  int32_t w_transposed; /* 0 or 1 */
  int32_t reserved;     /* 0 */
  int64_t M, N, K;
  const void *X;
  int64_t ldx;
  const void *Wg;
  int64_t ldwg;
  const void *Wu;
  int64_t ldwu;
  const void *bias_g;   /* N values, or NULL */
  const void *bias_u;
  void *Y;
  int64_t ldy;
  void *G;              /* both NULL, or M x N of dtype each: g and u */
  int64_t ldg;
  void *U;
  int64_t ldu;
  uint8_t *g_codes;     /* all four NULL, or the checkpoints of g and u */
  uint8_t *g_scales;
  uint8_t *u_codes;
  uint8_t *u_scales;
} mma_gated_linear_args;

int mma_gated_linear(const mma_gated_linear_args *args, void *workspace, int64_t workspace_bytes,
                     void *hip_stream);
int64_t mma_gated_linear_workspace(const mma_gated_linear_args *args);

/* Its backward pass.  X, and g and u together: matrices or checkpoints; both
 * g and u are read whatever the activation.  dX, dWg and dWu, dbias_g, dbias_u:
 * any of them NULL to leave it out (dWg and dWu both or neither).  dg and du
 * enter the products rounded to dtype (in FP16 an infinity past its range);
 * the biases' gradients sum them before that.  An infinity in G or U, past
 * the range of its 16 bits, stands for a large number. */
typedef struct {
  int32_t dtype;        /* of dY, X, the weights, G, U and dX */
  int32_t dw_dtype;     /* of dWg and dWu: dtype or FP32 */
  int32_t bias_dtype;   /* of dbias_g and dbias_u: dtype or FP32 */
  int32_t activation;
  int32_t w_transposed; /* of the weights and their gradients */
  int32_t reserved;     /* 0 */
  int64_t M, N, K;
  const void *dY;       /* M x N */
  int64_t lddy;
  const void *X;        /* M x K, or NULL with x_codes and x_scales */
  int64_t ldx;
  const uint8_t *x_codes;
  const uint8_t *x_scales;
  const void *Wg;
  int64_t ldwg;
  const void *Wu;
  int64_t ldwu;
  const void *G;        /* M x N each, or NULL with the four below */
  int64_t ldg;
  const void *U;
  int64_t ldu;
  const uint8_t *g_codes;
  const uint8_t *g_scales;
  const uint8_t *u_codes;
  const uint8_t *u_scales;
  void *dX;             /* M x K */
  int64_t lddx;
  void *dWg;            /* stored as the weights are */
  int64_t lddwg;
  void *dWu;
  int64_t lddwu;
  void *dbias_g;        /* N values each */
  void *dbias_u;
} mma_gated_linear_backward_args;

int mma_gated_linear_backward(const mma_gated_linear_backward_args *args, void *workspace,
                              int64_t workspace_bytes, void *hip_stream);
int64_t mma_gated_linear_backward_workspace(const mma_gated_linear_backward_args *args);

/* Y = drop(X) + residual (rows x cols of dtype; residual may be NULL); p in
 * [0, 1].  With dY as X and no residual, the gradient of X. */
int mma_dropout(int dtype, const void *X, int64_t ldx, const void *residual, int64_t ldr, void *Y,
                int64_t ldy, int64_t rows, int64_t cols, double p, uint64_t seed, uint64_t offset,
                const uint64_t *state, void *hip_stream);

enum { MMAOPS_NORM_NONE = 0, MMAOPS_NORM_LAYER = 1, MMAOPS_NORM_RMS = 2 };

/* R = scale X + gate drop(post(branch)), H = pre(R), for matrices rows x cols
 * of dtype, cols at least 1.  The weight, bias, statistics and output of a norm
 * that is not there may be any pointers: they are neither used nor checked. */
typedef struct {
  int32_t dtype;
  int32_t param_dtype;     /* of the five vectors: dtype or FP32 */
  int32_t post, pre;       /* MMAOPS_NORM_... */
  float scale;
  float eps;               /* of both norms */
  double p;                /* of dropout, in [0, 1] */
  uint64_t seed, offset;
  const uint64_t *state;   /* NULL, or (seed, offset) on the device */
  int64_t rows, cols;
  const void *X;
  int64_t ldx;
  const void *branch;
  int64_t ldb;
  const void *gate;        /* cols values, or NULL (1) */
  const void *post_weight; /* or NULL (1) */
  const void *post_bias;   /* or NULL (0) */
  const void *pre_weight;
  const void *pre_bias;
  void *R;
  int64_t ldr;
  void *H;                 /* not written without a pre norm */
  int64_t ldh;
  float *post_mean;        /* rows floats each, or NULL; a mean is written by */
  float *post_rstd;        /* a layer norm only */
  float *mean;
  float *rstd;
} mma_residual_norm_args;

int mma_residual_norm(const mma_residual_norm_args *args, void *hip_stream);

/* Its backward pass, with the forward pass's settings and statistics (a
 * mean for a layer norm only).  dR may be NULL (0) where there is a pre norm; dH and R
 * are read with one only.  branch is read with a post norm or for dgate.  What is not
 * read may be any pointer.  dX, dbranch and the vectors' gradients (of param_dtype): any
 * of them NULL to leave it out. */
typedef struct {
  int32_t dtype, param_dtype, post, pre;
  float scale;
  int32_t reserved;        /* 0 */
  double p;
  uint64_t seed, offset;
  const uint64_t *state;
  int64_t rows, cols;
  const void *dR;
  int64_t lddr;
  const void *dH;
  int64_t lddh;
  const void *R;
  int64_t ldr;
  const void *branch;
  int64_t ldb;
  const void *gate;
  const void *post_weight;
  const void *post_bias;
  const void *pre_weight;
  const float *post_mean;
  const float *post_rstd;
  const float *mean;
  const float *rstd;
  void *dX;
  int64_t lddx;
  void *dbranch;
  int64_t lddb;
  void *dgate;
  void *dpost_weight;
  void *dpost_bias;
  void *dpre_weight;
  void *dpre_bias;
} mma_residual_norm_backward_args;

int mma_residual_norm_backward(const mma_residual_norm_backward_args *args, void *workspace,
                               int64_t workspace_bytes, void *hip_stream);
int64_t mma_residual_norm_backward_workspace(const mma_residual_norm_backward_args *args);

/* Text for a return code of these functions (thread-local for
 * MMAEMU_ERR_HIP).  Never NULL. */
const char *mma_ops_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif
