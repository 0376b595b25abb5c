/*
 * tpconv_attention.h — attention among the nodes of each graph of a batch and
 * what stands around it, on AMD MI355X (gfx950): attention with a distance
 * bias and capped scores, the embedding of node types, and dropout from a
 * counter-based generator.
 *
 * With the layers of tpconv_layers.h they make one attention block:
 *
 *     x = embed(type);  y = norm(x);  q, k, v = linear(y)
 *     x = x + dropout(linear(attention(q, k, v, positions)))   (and the gradients)
 *
 * Node features are [N][F] as in tpconv.h: per node the blocks [2l+1][mul] of
 * the irreps string in order.  The rules of tpconv_layers.h hold here too:
 * device memory is the caller's, outputs are overwritten, calls are
 * asynchronous and ordered on the given HIP stream, arguments are checked
 * before any launch, a handle is immutable and may be used from several
 * streams while concurrent calls must not share a workspace, nothing
 * allocates, no exception crosses the ABI, inputs and outputs must not overlap
 * unless a call allows it.  All results are deterministic: every sum has a
 * fixed order, nothing is added with atomics.  Pointers need the alignment of
 * their element type, workspaces one of 16 bytes.  All sums and statistics are
 * fp32 whatever the input types, and so are all gradients.  First derivatives
 * only.  All calls can be captured into a graph.
 */
#ifndef TPCONV_ATTENTION_H_
#define TPCONV_ATTENTION_H_

#include "tpconv_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- attention among the nodes of each graph -------------------------------
 * Head h of H takes the channels [h mul / H, (h + 1) mul / H) of every row of
 * every irrep, of q and k (irreps_qk) and of v and out (irreps_v).  For query i
 * and key j of the same graph
 *   s_ij = scale <q_i, k_j>_h;   s_ij <- cap tanh(s_ij / cap)  (cap > 0)
 *   s_ij <- s_ij - slope_h |r_i - r_j|                          (with slopes)
 *   out_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij)
 * The inner product runs over all rows of the irreps, so that scores do not
 * change under rotations and outputs rotate as the values do.  A query whose
 * graph has no keys gets zeros.  Products of fp32 operands are within 2^-25 of
 * their values, and sums over more than 4096 rows of a graph are made in runs of
 * so many; inputs must stay below 3.38e38, scores within fp32 range and distances below
 * 1.8e19.  A value that is not finite shows in results of its own graph and head alone. */
typedef struct tpconv_attention_s* tpconv_attention;

typedef struct {
  const char* irreps_qk; /* l <= 3, at most 16 blocks, all multiplicities divisible by num_heads */
  const char* irreps_v;  /* the same rules */
  int32_t num_heads;     /* 1..256; at most 256 values per head on either side (UNSUPPORTED) */
  float scale;           /* -2^100..2^100; usually one over the square root of the values per head */
  float score_cap;       /* 0: scores are not capped; or 2^-100..2^100, and scale / score_cap finite */
  int32_t x_dtype;       /* tpconv_dtype of q, k and v */
  int32_t y_dtype;       /* tpconv_dtype of out (bf16: rounded once, to nearest even) */
} tpconv_attention_desc;

tpconv_status tpconv_attention_create(tpconv_attention* out, const tpconv_attention_desc* desc);
tpconv_status tpconv_attention_destroy(tpconv_attention attention); /* NULL is accepted */

/* features per node of q and k, of v and out, and values per head; any pointer may be NULL. */
tpconv_status tpconv_attention_info(tpconv_attention attention, int64_t* feat_qk, int64_t* feat_v,
                                    int32_t* head_qk, int32_t* head_v);

/* Which rows belong together.  Graph g's queries are the rows offsets[g] ..
 * offsets[g + 1] - 1; rows outside of all graphs are left as they were in
 * every output (a caller that goes on with whole tensors, as a layer over padded
 * batches does, clears them once).  offsets NULL: one graph of all rows (num_graphs = 1).
 * key_offsets NULL: the keys are the queries' own nodes (self form; num_keys
 * and key_pos are not read); otherwise graph g's keys are the rows
 * key_offsets[g] .. of k and v, and there may be none.  Offsets must not
 * decrease; they are clamped to the rows there are, so that no call reads or
 * writes outside of its tensors.  Row strides in elements let q, k and v (and
 * their gradients) be column ranges of one wider tensor; 0: contiguous. */
typedef struct {
  int64_t num_graphs;
  int64_t num_queries;
  const int32_t* offsets;     /* device [num_graphs + 1], or NULL */
  const float* pos;           /* device [num_queries][3], or NULL without slopes */
  int64_t num_keys;
  const int32_t* key_offsets; /* device [num_graphs + 1], or NULL (self form) */
  const float* key_pos;       /* device [num_keys][3] */
} tpconv_attention_batch;

typedef struct {
  const void* q; /* [num_queries] rows of feat_qk values */
  const void* k; /* [num_keys] rows of feat_qk values */
  const void* v; /* [num_keys] rows of feat_v values */
  int64_t q_stride, k_stride, v_stride; /* elements from row to row */
  const float* slope; /* device [num_heads], or NULL: no distance bias */
} tpconv_attention_inputs;

/* fp32 values that tpconv_attention_forward saves for the backward:
 * [2][num_heads][num_queries], a reference m of every row and 1 / l, so that its
 * weights are 2^(s_ij log2(e) - m) / l (no keys: minus infinity and 0), and, for a
 * bf16 output, [num_queries][feat_v], the output before its rounding. */
tpconv_status tpconv_attention_saved_size(tpconv_attention attention, int64_t num_queries, int64_t* values);

/* Bytes of workspace of TPCONV_OP_FORWARD (may be 0; with `saved` it may need
 * less) and TPCONV_OP_BACKWARD for a batch of these counts (its pointers are only
 * compared with NULL).  At most 64 fp32 copies of the results: where there are few
 * rows, which are then worked on in parts of the other side, and up to eight where
 * the mean graph has more than 4096 rows. */
tpconv_status tpconv_attention_workspace_size(tpconv_attention attention, int32_t op,
                                              const tpconv_attention_batch* batch, size_t* bytes);

/* out [num_queries][feat_v].  saved: NULL, or see above. */
tpconv_status tpconv_attention_forward(tpconv_attention attention, const tpconv_attention_batch* batch,
                                       const tpconv_attention_inputs* in, void* out, float* saved, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* Where the gradients go (each may be NULL, at least one must be given), all
 * fp32.  grad_pos: of the queries' positions, in the self form of the nodes'
 * (both ends of a pair); grad_key_pos: of the keys' positions, cross form only.
 * A pair of nodes in the same place (closer than 1e-19) has no direction and adds nothing. */
typedef struct {
  float* grad_q;
  float* grad_k;
  float* grad_v;
  int64_t q_stride, k_stride, v_stride; /* elements from row to row; 0: contiguous */
  float* grad_slope;   /* [num_heads] */
  float* grad_pos;     /* [num_queries][3] */
  float* grad_key_pos; /* [num_keys][3] */
} tpconv_attention_grads;

/* Gradients of <grad_out, out>; out and saved are those of a forward on the same inputs. */
tpconv_status tpconv_attention_backward(tpconv_attention attention, const tpconv_attention_batch* batch,
                                        const tpconv_attention_inputs* in, const void* out, const float* saved,
                                        const float* grad_out, const tpconv_attention_grads* grads,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* ---- embedding of node types ----------------------------------------------------
 * y[v] = scale W[index[v]],  W [num_rows][features]; a node whose index lies
 * outside 0..num_rows-1 (a padding node) gets zeros and no gradient. */
typedef struct tpconv_embed_s* tpconv_embed;

typedef struct {
  int32_t num_rows;  /* 1..2^24 */
  int32_t features;  /* 1..65536 */
  float scale;       /* finite */
  int32_t w_dtype;   /* tpconv_dtype of W */
  int32_t y_dtype;   /* tpconv_dtype of y */
} tpconv_embed_desc;

tpconv_status tpconv_embed_create(tpconv_embed* out, const tpconv_embed_desc* desc);
tpconv_status tpconv_embed_destroy(tpconv_embed embed);
tpconv_status tpconv_embed_workspace_size(tpconv_embed embed, int64_t num_nodes, size_t* bytes);
/* index: device int32 [num_nodes] */
tpconv_status tpconv_embed_forward(tpconv_embed embed, int64_t num_nodes, const int32_t* index, const void* W, void* y,
                                   void* stream);
/* grad_W [num_rows][features] fp32, every row written: scale times the sum of
 * grad_y (fp32) over the nodes of a type, in the order of a stable sort of the
 * nodes by type (made within the call). */
tpconv_status tpconv_embed_backward(tpconv_embed embed, int64_t num_nodes, const int32_t* index, const float* grad_y,
                                    float* grad_W, void* workspace, size_t workspace_bytes, void* stream);

/* ---- dropout ----------------------------------------------------------------------
 * y = residual + x * keep / (1 - p'), where keep is drawn once per node and
 * channel of every irrep and shared by its 2l+1 rows (a mask that changed from
 * row to row would break the equivariance).  It is never stored: channel c of
 * irrep i of node v takes 16-bit word c % 8 of Philox4x32-10 (J. Salmon et al.,
 * 2011) with counter (b, offset), b = v U + u_i + c / 8 and offset as two 32-bit
 * words each, low word first, and key seed (low word first): word w is the low
 * (w even) or high half of output w / 2.  u_i counts the groups of eight
 * channels of the irreps before i, U those of all.  The channel is kept if the
 * word is at least t = round(65536 p); p' = t / 65536.  t = 65536 keeps none.
 * The mask depends on seed, offset and irreps alone: every call that shall draw for
 * itself (each layer of each step) needs an offset of its own. */
typedef struct tpconv_dropout_s* tpconv_dropout;

typedef struct {
  const char* irreps; /* l <= 3, at most 16 blocks */
  float p;            /* 0..1 */
  int32_t x_dtype;    /* tpconv_dtype of x */
  int32_t y_dtype;    /* tpconv_dtype of y and residual */
} tpconv_dropout_desc;

tpconv_status tpconv_dropout_create(tpconv_dropout* out, const tpconv_dropout_desc* desc);
tpconv_status tpconv_dropout_destroy(tpconv_dropout dropout);
/* features per node and the probability that is used (p'); any pointer may be NULL */
tpconv_status tpconv_dropout_info(tpconv_dropout dropout, int64_t* features, float* p);

/* rng: device int64 [2] = (seed, offset), read when the kernel runs, so that a
 * captured graph draws anew when the caller changes the offset; the backward
 * needs the values that its forward had.  residual may be NULL or y; y may be x
 * if their types agree.  A dropped value that is not finite becomes zero. */
tpconv_status tpconv_dropout_forward(tpconv_dropout dropout, int64_t num_nodes, const void* x, const int64_t* rng,
                                     const void* residual, void* y, void* stream);
/* grad_x = grad_y * keep / (1 - p'), fp32; grad_x may be grad_y.  (The residual's gradient is grad_y.) */
tpconv_status tpconv_dropout_backward(tpconv_dropout dropout, int64_t num_nodes, const float* grad_y,
                                      const int64_t* rng, float* grad_x, void* stream);

/* Kernel classes of these layers for tpconv_kernel_timing_read. */
typedef enum {
  TPCONV_KERNEL_ATTENTION = 20,
  TPCONV_KERNEL_EMBED = 21,
  TPCONV_KERNEL_DROPOUT = 22
} tpconv_attention_kernel;

#ifdef __cplusplus
}
#endif

#endif /* TPCONV_ATTENTION_H_ */
