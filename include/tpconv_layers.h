/*
 * tpconv_layers.h — node layers around the streaming convolution of tpconv.h,
 * on AMD MI355X (gfx950): layer norm over irreps, a linear layer with one
 * weight matrix per group of nodes, and the orthogonalised (Muon) update of
 * banks of weight matrices.
 *
 * With the convolution they make one training step of an interaction block:
 *
 *     y = norm(x);  z = conv(pos, y, W);  out = linear(z, group)   (and their gradients)
 *     W, linear weights <- muon step(their gradients)
 *
 * Node features are [N][F] as in tpconv.h: per node the blocks [2l+1][mul] of
 * the irreps string in order (one multiplicity: exactly [N][rows][C]).  A
 * string of scalars such as "1024x0e" makes these the usual layers on rows of
 * 1024 values.  The rules of tpconv.h hold here too: device memory is the
 * caller's and contiguous, outputs are overwritten, calls are asynchronous and
 * ordered on the given HIP stream, arguments are checked before any launch, a
 * handle is immutable and may be used from several streams while concurrent
 * calls must not share a workspace, nothing allocates, no exception crosses
 * the ABI.  Inputs and outputs must not overlap unless a call allows it.
 * All results are deterministic: every sum has a fixed order, nothing is added
 * with atomics.  Pointers need the alignment of their element type, workspaces
 * one of 16 bytes (TPCONV_ERROR_WORKSPACE otherwise).
 * All sums and statistics are fp32 whatever the input types.
 */
#ifndef TPCONV_LAYERS_H_
#define TPCONV_LAYERS_H_

#include "tpconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- layer norm ---------------------------------------------------------
 * Per node and irrep (block v of 2l+1 rows and mul channels):
 *   0e:     mu = mean(v), z = (v - mu) / sqrt(mean((v - mu)^2) + eps), y = w_c z + b_c
 *   others: z = v / sqrt(mean(v^2) + eps), y = w_c z
 * (means over the block's (2l+1) mul values; a mean or a bias on a block that
 * rotates or changes sign would break its equivariance).  w has one value per
 * channel of every irrep, b one per channel of every 0e irrep, in order.
 * A block of zeros gives b (0 without bias) and gradients scaled by 1/sqrt(eps).
 * A block whose sum of squares passes 3.4e38 is out of range (z is zero or NaN).
 * First derivatives only: neither the norm nor the linear layer has an entry
 * point for the second. */
typedef struct tpconv_norm_s* tpconv_norm;

typedef struct {
  const char* irreps; /* l <= 3, at most 16 blocks */
  float eps;          /* > 0 */
  int32_t x_dtype;    /* tpconv_dtype of x */
  int32_t y_dtype;    /* tpconv_dtype of y (bf16: rounded once, to nearest even) */
} tpconv_norm_desc;

tpconv_status tpconv_norm_create(tpconv_norm* out, const tpconv_norm_desc* desc);
tpconv_status tpconv_norm_destroy(tpconv_norm norm); /* NULL is accepted */

/* features per node, irreps, values of weight and of bias; any pointer may be NULL. */
tpconv_status tpconv_norm_info(tpconv_norm norm, int64_t* features, int32_t* num_irreps, int64_t* num_weights,
                               int64_t* num_biases);

/* Bytes of workspace tpconv_norm_backward needs for a weight or bias gradient. */
tpconv_status tpconv_norm_workspace_size(tpconv_norm norm, int64_t num_nodes, size_t* bytes);

/* y = norm(x).  weight, bias: fp32 (NULL: ones, zeros).  stats: NULL, or fp32
 * [N][num_irreps][2] that receives (mu, 1 / sqrt(...)) of every block (mu = 0
 * for blocks without a mean) for a later backward. */
tpconv_status tpconv_norm_forward(tpconv_norm norm, int64_t num_nodes, const void* x, const float* weight,
                                  const float* bias, void* y, float* stats, void* stream);

/* Gradients of <grad_y, y>, all fp32: grad_x [N][F], grad_weight, grad_bias
 * (each may be NULL, at least one must be given; grad_bias of a norm without
 * 0e irreps is not written).  stats: from tpconv_norm_forward on the same x,
 * or NULL to recompute them.  workspace: needed for grad_weight or grad_bias. */
tpconv_status tpconv_norm_backward(tpconv_norm norm, int64_t num_nodes, const void* x, const float* weight,
                                   const float* grad_y, const float* stats, float* grad_x, float* grad_weight,
                                   float* grad_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ---- linear layer, one weight per group of nodes ---------------------------
 * Every node belongs to one of num_groups groups (chemical element, expert):
 *   y[v, o, m, c'] = sum_{i ~ o} sum_c x[v, i, m, c] W[group(v)][(i, o)][c, c']
 * over the input irreps i of the same degree and parity as the output irrep o
 * (an output irrep without such an input is zero).  W is [num_groups][w_numel],
 * per group the blocks [mul_i][mul_o] in the order of i, then o (at most 64
 * blocks and 2^31 - 1 weights per group, or UNSUPPORTED).
 * A product of fp32 operands is within 2^-21 of its value, towards zero: each
 * operand is exactly the sum of three bf16 values, of whose nine products the six
 * largest are added in fp32 (fp32 x bf16: all three; bf16 x bf16: exact).  A value
 * that is not finite makes the results that it takes part in not finite. */
typedef struct tpconv_linear_s* tpconv_linear;

typedef struct {
  const char* irreps_in;  /* l <= 3, at most 16 blocks */
  const char* irreps_out; /* the same rules */
  int32_t num_groups;     /* 1..4096 */
  int32_t x_dtype;        /* tpconv_dtype of x */
  int32_t w_dtype;        /* tpconv_dtype of W */
  int32_t y_dtype;        /* tpconv_dtype of y */
} tpconv_linear_desc;

tpconv_status tpconv_linear_create(tpconv_linear* out, const tpconv_linear_desc* desc);
tpconv_status tpconv_linear_destroy(tpconv_linear linear);

/* features per node of x and y, weights per group, weight blocks; any pointer may be NULL. */
tpconv_status tpconv_linear_info(tpconv_linear linear, int64_t* feat_in, int64_t* feat_out, int64_t* w_numel,
                                 int32_t* num_blocks);

/* Weight block `block`: irrep_idx[2] = (input irrep, output irrep), shape[2] =
 * (mul_i, mul_o), offset within a group's weights; any pointer may be NULL. */
tpconv_status tpconv_linear_block(tpconv_linear linear, int32_t block, int32_t* irrep_idx, int32_t* shape,
                                  int64_t* offset);

/* The grouping of N nodes, built once per set of nodes: order [N] = the nodes
 * sorted by group (stable: increasing node ids within a group), offsets
 * [num_groups + 1] = the group boundaries in it.  group: device int32 [N].  With
 * validate != 0 group ids outside 0..num_groups-1 are reported as
 * TPCONV_ERROR_GRAPH without writing the outputs (synchronises the stream);
 * without it such nodes are left out of order (their outputs are not written). */
tpconv_status tpconv_linear_groups_workspace_size(tpconv_linear linear, int64_t num_nodes, size_t* bytes);
tpconv_status tpconv_linear_groups(tpconv_linear linear, int64_t num_nodes, const int32_t* group, int32_t* offsets,
                                   int32_t* order, int32_t validate, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Bytes of workspace of TPCONV_OP_FORWARD (may be 0) and TPCONV_OP_BACKWARD;
 * independent of how the nodes spread over the groups. */
tpconv_status tpconv_linear_workspace_size(tpconv_linear linear, int32_t op, int64_t num_nodes, size_t* bytes);

/* offsets, order: from tpconv_linear_groups; both NULL for num_groups = 1
 * (every node in the one group).  The split over groups is read on the device,
 * so nothing waits for it. */
tpconv_status tpconv_linear_forward(tpconv_linear linear, int64_t num_nodes, const int32_t* offsets,
                                    const int32_t* order, const void* x, const void* W, void* y, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Gradients of <grad_y, y>, all fp32: grad_x [N][F_in], grad_W
 * [num_groups][w_numel] (zero for groups without nodes); each may be NULL, at
 * least one must be given. */
tpconv_status tpconv_linear_backward(tpconv_linear linear, int64_t num_nodes, const int32_t* offsets,
                                     const int32_t* order, const void* x, const void* W, const float* grad_y,
                                     float* grad_x, float* grad_W, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* ---- orthogonalised (Muon) update of weight matrices --------------------------
 * For every matrix U of the banks:
 *   X = U / max(|U|_F, eps);  per step  A = X X^T,  X <- a X + (b A + c A A) X
 * (X^T X form for matrices with more rows than columns, the same result), which
 * takes the singular values s of X to a s + b s^3 + c s^5 and leaves the
 * singular vectors alone.  U may hold any finite values (its norm is scaled by
 * a power of two where the squares would leave fp32); a matrix with a value that
 * is not finite comes out as NaN. */
typedef struct tpconv_muon_s* tpconv_muon;

/* `count` row-major matrices of rows x cols at element offset + i * stride. */
typedef struct {
  int32_t rows, cols;
  int64_t count, offset, stride; /* stride >= rows * cols */
} tpconv_matrix_block;

typedef struct {
  int32_t num_blocks; /* 1..64; the blocks must not overlap */
  const tpconv_matrix_block* blocks;
  int32_t num_steps;         /* 1..16 */
  const float* coefficients; /* [num_steps][3] = (a, b, c) of every step */
  float eps;                 /* > 0: lower bound of the Frobenius norm */
} tpconv_muon_desc;

tpconv_status tpconv_muon_create(tpconv_muon* out, const tpconv_muon_desc* desc);
tpconv_status tpconv_muon_destroy(tpconv_muon muon);
tpconv_status tpconv_muon_workspace_size(tpconv_muon muon, size_t* bytes);

/* The weight blocks of a plan's W (fully connected plans: one block per path,
 * or a single one for uniform multiplicities; rows = C_in, cols = C_out) and of
 * a linear layer's W.  *count receives the number of blocks; blocks may be NULL
 * to ask for it, and capacity must not be smaller otherwise.  Channel-wise plans
 * have no matrices (UNSUPPORTED). */
tpconv_status tpconv_plan_weight_blocks(tpconv_plan plan, tpconv_matrix_block* blocks, int32_t capacity,
                                        int32_t* count);
tpconv_status tpconv_linear_weight_blocks(tpconv_linear linear, tpconv_matrix_block* blocks, int32_t capacity,
                                          int32_t* count);

/* out = the matrices of u orthogonalised (fp32; the elements between the
 * blocks are not written).  out may be u. */
tpconv_status tpconv_muon_orthogonalize(tpconv_muon muon, const float* u, float* out, void* workspace,
                                        size_t workspace_bytes, void* stream);

typedef struct {
  float lr;
  float beta;           /* momentum */
  int32_t nesterov;     /* 1: u = (1 - beta) grad + beta m';  0: u = m' */
  float weight_decay;
} tpconv_muon_step_args;

/* m' = beta m + (1 - beta) grad;  W' = (1 - lr weight_decay) W - lr s X(u),
 * s = sqrt(max(1, cols / rows)): rows are the inputs of W, cols its outputs.
 * All tensors are fp32, the operands of the products within X(u) sums of two
 * fp16 values (22 bits).  W_out may be W and momentum_out may be momentum (in place).
 * W_bf16: NULL, or the new weights rounded to bf16 as well, in the same layout
 * (what a forward with bf16 weights reads). */
tpconv_status tpconv_muon_step(tpconv_muon muon, const tpconv_muon_step_args* args, const float* W,
                               const float* grad, const float* momentum, float* W_out, float* momentum_out,
                               void* W_bf16, void* workspace, size_t workspace_bytes, void* stream);

/* Kernel classes of these layers for tpconv_kernel_timing_read. */
typedef enum {
  TPCONV_KERNEL_NORM = 17,
  TPCONV_KERNEL_LINEAR = 18,
  TPCONV_KERNEL_MUON = 19
} tpconv_layer_kernel;

#ifdef __cplusplus
}
#endif

#endif /* TPCONV_LAYERS_H_ */
