// Argument blocks and host launchers of the node layers (include/tpconv_layers.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tpconv_layers.h"
#include "plan.h"

namespace tpconv {

// ---- layer norm ---------------------------------------------------------------

struct NormIrrep {
  int32_t mul, n;        // channels, rows (2l+1)
  int32_t scalar;        // 1: 0e (mean and bias)
  int32_t off;           // feature offset of the block within a node
  int32_t w_off, b_off;  // offsets in weight and bias
  int32_t lanes;         // lanes per (node, irrep) of narrow blocks
  int32_t first_block, blocks;  // the irrep's blocks of the launch
  int64_t part_off;      // backward: the irrep's partial sums, [blocks][mul] (scalar irreps: [blocks][2][mul])
};

struct NormArgs {
  int32_t nirreps;
  int32_t x_bf16, y_bf16;
  float eps;
  int64_t N, F;
  const void* x;
  const float* w;
  const float* b;
  void* y;
  float* stats;        // forward: written or NULL; backward: read or NULL
  const float* gy;
  float* gx;
  float* gw;
  float* gb;
  float* part;         // backward: NULL when no parameter gradient is wanted
  NormIrrep ir[kMaxGroups];
};

// Blocks of the backward launch per irrep (they bound the partial sums);
// fills first_block / blocks / part_off and returns the floats of partials.
int64_t norm_backward_blocks(NormArgs& a);
hipError_t launch_norm_forward(NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(NormArgs& a, hipStream_t s);

// ---- grouped linear layer -------------------------------------------------------

constexpr int kMaxLinBlocks = 64;

// One weight block: input irrep (mul_i) x output irrep (mul_o).
struct LinBlock {
  int32_t i, o;        // irrep indices
  int32_t mi, mo;
  int32_t n;           // rows per node (2l+1)
  int32_t xoff, yoff;  // feature offsets of the two irreps
  int64_t woff;        // offset within a group's weights
};

// Rows kernel (forward, input gradient): out[(v, m), c'] = sum over segments
// sum_c in[(v, m), c] B(c, c').
// (32-bit throughout: the argument blocks are copied at every launch, at about
// a microsecond per KiB; a group's weights and a launch's tiles stay below 2^31.)
struct LinSeg {
  int32_t off;   // feature offset of the input block
  int32_t len;   // reduction length
  int32_t woff;  // weight block within the group's weights
};
struct LinJob {
  int32_t n;           // rows per node
  int32_t off, cols;   // feature offset and channels of the output block
  int32_t seg0, nseg;
  int32_t tiles_n;     // column tiles
  int32_t by_row;      // row tiles numbered by their first row (fewer rows than groups)
  int32_t first_tile;  // first block of the job in the launch
};
struct LinRowsArgs {
  int32_t njobs, G;
  int32_t in_bf16, w_bf16, out_bf16, wt;  // wt: B(c, c') = W[c'][c] (input gradient)
  int64_t N, F_in, F_out, w_per_group, tiles;
  const int32_t* offsets;  // NULL: one group
  const int32_t* order;
  const void* in;
  const void* W;
  void* out;
  LinJob job[kMaxGroups];
  LinSeg seg[kMaxLinBlocks];
};

// Weight-gradient kernel: W_g[c][c'] = sum over the rows (v, m) of group g in[(v, m), c] gy[(v, m), c'].
struct LinGwJob {
  int32_t n, mi, mo, xoff, yoff;
  int32_t woff;         // weight block within a group's weights: also its first element of the reduction launch
  int32_t by_row;       // slots numbered by their first row (fewer rows than groups)
  int32_t first_tile;   // first block of the job
  int64_t part_off;     // [places][mi][mo] partial sums of the groups of several slots
};
struct LinGwArgs {
  int32_t njobs, G, x_bf16;
  int32_t width;   // tile width
  int32_t rshift;  // rows per slot = 1 << rshift
  int64_t N, F_in, F_out, w_per_group, tiles;
  const int32_t* offsets;
  const int32_t* order;
  const void* x;
  const float* gy;
  float* gW;
  float* part;
  LinGwJob job[kMaxLinBlocks];
};

// Both gradients: njobs = 0 leaves one out.
struct LinBackwardArgs {
  LinRowsArgs rows;    // gy -> gx
  LinGwArgs gw;
  int64_t rows_first;  // first block of the input gradient
};

hipError_t launch_lin_rows(LinRowsArgs& a, hipStream_t s);
// Fills the slots of the jobs and returns the floats of partial sums.
int64_t lin_gw_plan(LinGwArgs& a);
hipError_t launch_lin_backward(LinBackwardArgs& a, hipStream_t s);
size_t lin_groups_workspace(int64_t N, int G);
hipError_t launch_lin_groups_validate(const int32_t* group, int64_t N, int G, int32_t* flag, hipStream_t s);
hipError_t launch_lin_groups(const int32_t* group, int64_t N, int G, int32_t* offsets, int32_t* order, void* ws,
                             hipStream_t s);

// ---- orthogonalised update --------------------------------------------------------

constexpr int kMaxMuonBlocks = 64;
constexpr int kMaxMuonSteps = 16;

struct MuonStep {
  float a, b, c;
  int32_t ex, ea, eb;  // powers of two that put X, A = X X^T and B = b A + c A A into the fp16 range
};

struct MuonBlock {
  int32_t rows, cols;
  int64_t count, offset, stride;
};

struct MuonUpdate {
  const float* u;      // orthogonalize: the matrices (grad, momentum, W unused)
  const float* W;
  const float* grad;
  const float* mom;
  float* out;          // orthogonalize: X; step: W'
  float* mom_out;
  uint16_t* w_bf16;
  float lr, beta, decay;
  int32_t nesterov;
};

struct MuonPlan {
  int32_t nsteps = 0;
  float eps = 0.f;
  MuonStep step[kMaxMuonSteps + 1];  // [nsteps]: the exponents of the result
  int32_t nblocks = 0;
  MuonBlock block[kMaxMuonBlocks];
};

size_t muon_workspace(const MuonPlan& p);
hipError_t launch_muon(const MuonPlan& p, const MuonUpdate& u, void* ws, hipStream_t s);

}  // namespace tpconv
