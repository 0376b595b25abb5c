// Argument blocks and host launchers of include/tpconv_attention.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tpconv_attention.h"
#include "plan.h"

namespace tpconv {

// ---- attention ------------------------------------------------------------------

// One irrep of a side as a head sees it: head element first + r * cph + c is
// channel h * cph + c of row r, at feature off + r * mul + h * cph + c.
struct AttnIrrep {
  int32_t off, mul, cph, first;
};
struct AttnSide {
  int32_t nirr, D, F;  // irreps, values per head, features per node
  int32_t vec;         // every cph is a multiple of 4: quads of head elements are contiguous
  AttnIrrep ir[kMaxGroups];
};

struct AttnArgs {
  int32_t H, G, self;
  int32_t x_bf16, y_bf16;
  int32_t nsplit;           // parts the long axis is cut into, joined by a second kernel
  int32_t heads_inner;      // order of the work: the heads of a tile together, or the tiles of a head
  int64_t tiles;            // row tiles of the launch
  float scale, cap;
  int64_t Nq, Nk;
  const int32_t *qo, *ko;   // NULL: one graph of all rows
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const float *slope, *qpos, *kpos;  // all NULL without the distance bias
  // forward
  void* out;
  float* stat;              // [2][H][Nq]: the references of the rows' weights and 1 / their sums; NULL: not saved
  float* out32;             // fp32 output of a bf16 forward that saves, or NULL
  float *sums, *part_ml;    // [nsplit][Nq][F_v], [nsplit][H][Nq][2]; sums: with one part the fp32 result, or room for runs
  int32_t put_f32, put_bf16;  // whether the kernel's last sums go to `sums`, and rounded to out
  // backward
  const float* go;
  const float* o;           // fp32 output
  float* delta;             // [H][Nq]: <grad_out, out> per head
  float *gq, *gk, *gv;      // the gradients, or their parts [nsplit][rows][F]
  int64_t ldgq, ldgk, ldgv;
  float* part_pos;          // [nsplit][H][rows][3], or NULL
  float* part_slope;        // [nsplit][H][Nq][3]: a row's sums of dS d, of dS, of P d; or NULL
  AttnSide sqk, sv;
};

// Joins what the kernels left in parts.
struct AttnJoinArgs {
  int32_t H, G, nsplit_q, nsplit_k;
  int64_t Nq, Nk;
  const int32_t *qo, *ko;
  const float *part_gq, *part_gk, *part_gv;  // NULL: already in place
  float *gq, *gk, *gv;
  int64_t ldgq, ldgk, ldgv;
  int32_t Fqk, Fv;
  const float *part_qpos, *part_kpos;  // [nsplit][H][rows][3]
  float *gpos, *gkpos;                 // gkpos NULL in the self form: both ends are added to gpos
  const float* part_slope;             // [nsplit][H][Nq][3]
  float* gslope;
};

constexpr int kAttnMaxHead = 256;
constexpr int64_t kAttnRun = 4096;  // rows in one accumulator; a multiple of the 64 that a block takes at a time

// Rows per block where the graphs are small: 32, but blocks of wide heads need LDS for
// several waves' worth of registers (a CU's LDS holds two of 160 values, one of 256).
constexpr int attn_small_cols(int DC) { return DC <= 96 ? 32 : DC <= 160 ? 64 : 128; }

struct AttnShape {
  int cls;       // index of the width class
  int cols;      // rows per block: 128 or attn_small_cols
  int nsplit;
  int64_t tiles;
};
// The shape of a launch whose rows are `rows` and whose long axis is `other`; exact: its results are fp32.
AttnShape attn_shape(int D, int64_t rows, int64_t other, int64_t graphs, int heads, bool exact);

hipError_t launch_attn_forward(AttnArgs& a, const AttnShape& s, hipStream_t st);
hipError_t launch_attn_combine(AttnArgs& a, const AttnShape& s, hipStream_t st);
hipError_t launch_attn_grad_q(AttnArgs& a, const AttnShape& s, hipStream_t st);
hipError_t launch_attn_grad_kv(AttnArgs& a, const AttnShape& s, hipStream_t st);
hipError_t launch_attn_join(const AttnJoinArgs& a, hipStream_t st);

// ---- embedding --------------------------------------------------------------------

struct EmbedArgs {
  int32_t rows, features, w_bf16, y_bf16;
  float scale;
  int64_t N;
  const int32_t* index;
  const void* W;
  void* y;
  const float* gy;
  float* gW;
};
size_t embed_workspace(int32_t rows, int32_t features, int64_t N);
hipError_t launch_embed_forward(const EmbedArgs& a, hipStream_t s);
hipError_t launch_embed_backward(const EmbedArgs& a, void* ws, hipStream_t s);

// ---- dropout ------------------------------------------------------------------------

struct DropIrrep {
  int32_t mul, n, off, first;  // channels, rows, feature offset, first group of eight channels
};
struct DropArgs {
  int32_t nirr, groups;  // irreps, groups of eight channels per node
  int32_t x_bf16, y_bf16, has_res;
  int32_t limit;         // kept if word >= limit
  float factor;
  int64_t N, F;
  const void* x;
  const int64_t* rng;
  const void* res;
  void* y;
  DropIrrep ir[kMaxGroups];
};
hipError_t launch_dropout(const DropArgs& a, hipStream_t s);

}  // namespace tpconv
