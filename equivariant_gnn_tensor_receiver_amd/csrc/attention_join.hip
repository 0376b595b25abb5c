// Attention: the choice of launch shapes, and the kernels that join what was
// cut along the long axis (forward: partial softmax sums; backward: partial
// gradients) or left per head (gradients of positions and slopes).
#include <algorithm>

#include "attention_kernels.h"
#include "timing.h"

namespace tpconv {

hipError_t launch_attn_class_32(int kind, const AttnArgs& a, int cols, hipStream_t st);
hipError_t launch_attn_class_64(int kind, const AttnArgs& a, int cols, hipStream_t st);
hipError_t launch_attn_class_96(int kind, const AttnArgs& a, int cols, hipStream_t st);
hipError_t launch_attn_class_128(int kind, const AttnArgs& a, int cols, hipStream_t st);
hipError_t launch_attn_class_160(int kind, const AttnArgs& a, int cols, hipStream_t st);
hipError_t launch_attn_class_256(int kind, const AttnArgs& a, int cols, hipStream_t st);

namespace {

using namespace attn;

typedef hipError_t (*ClassLauncher)(int, const AttnArgs&, int, hipStream_t);
constexpr int kClasses = 6;
constexpr int kWidth[kClasses] = {32, 64, 96, 128, 160, 256};
const ClassLauncher kLaunch[kClasses] = {launch_attn_class_32,  launch_attn_class_64,  launch_attn_class_96,
                                         launch_attn_class_128, launch_attn_class_160, launch_attn_class_256};

// Head of feature f of a side.
__device__ __forceinline__ int head_of(const AttnSide& s, int f) {
  int i = 0;
  while (i + 1 < s.nirr && f >= s.ir[i + 1].off) ++i;
  return (f - s.ir[i].off) % s.ir[i].mul / s.ir[i].cph;
}

// out = sum over the parts of w o / sum of w l, w = 2^(m - largest m).  One block per 32 rows.
__global__ __launch_bounds__(256) void combine_kernel(const AttnArgs a) {
  Tile t;
  if (!find_tile(a.qo, a.G, a.Nq, 5, blockIdx.x, t)) return;
  const int F = a.sv.F;
  for (int i = threadIdx.x; i < t.rows * F; i += 256) {
    const int row = i / F, f = i - row * F;
    const int64_t query = t.row0 + row;
    const int h = head_of(a.sv, f);
    float top = -INFINITY;
    for (int p = 0; p < a.nsplit; ++p) top = fmaxf(top, a.part_ml[2 * (((int64_t)p * a.H + h) * a.Nq + query)]);
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f, o = 0.f;
    for (int p = 0; p < a.nsplit; ++p) {
      const float* ml = a.part_ml + 2 * (((int64_t)p * a.H + h) * a.Nq + query);
      if (ml[0] == -INFINITY && ml[1] == 0.f) continue;  // a part without keys
      const float w = exp2_fast(ml[0] - ref);
      l = fmaf(w, ml[1], l);
      o = fmaf(w, a.part_o[((int64_t)p * a.Nq + query) * F + f], o);
    }
    o *= l > 0.f || l != l ? 1.f / l : 0.f;
    if (a.out32) a.out32[query * F + f] = o;
    if (a.y_bf16)
      static_cast<uint16_t*>(a.out)[query * F + f] = __builtin_bit_cast(uint16_t, (__bf16)o);
    else
      static_cast<float*>(a.out)[query * F + f] = o;
  }
  if (!a.stat) return;
  for (int i = threadIdx.x; i < t.rows * a.H; i += 256) {
    const int h = i / t.rows;
    const int64_t query = t.row0 + (i - h * t.rows);
    float top = -INFINITY, l = 0.f;
    for (int p = 0; p < a.nsplit; ++p) top = fmaxf(top, a.part_ml[2 * (((int64_t)p * a.H + h) * a.Nq + query)]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int p = 0; p < a.nsplit; ++p) {
      const float* ml = a.part_ml + 2 * (((int64_t)p * a.H + h) * a.Nq + query);
      if (ml[0] == -INFINITY && ml[1] == 0.f) continue;
      l = fmaf(exp2_fast(ml[0] - ref), ml[1], l);
    }
    a.stat[(int64_t)h * a.Nq + query] = top;
    a.stat[(int64_t)(a.H + h) * a.Nq + query] = l > 0.f || l != l ? 1.f / l : 0.f;
  }
}

__device__ __forceinline__ bool covered(const int32_t* off, int G, int64_t N, int64_t row) {
  return !off || (row >= clamp_row(off[0], N) && row < clamp_row(off[G], N));
}

// Sums of parts [n][rows][F] into rows of stride ld, in order.
__device__ __forceinline__ void sum_rows(const float* part, int n, int64_t rows, int F, float* out, int64_t ld,
                                         const int32_t* off, int G, int64_t first, int64_t step) {
  for (int64_t i = first; i < rows * F; i += step) {
    const int64_t row = i / F;
    if (!covered(off, G, rows, row)) continue;
    float v = 0.f;
    for (int p = 0; p < n; ++p) v += part[p * rows * F + i];
    out[row * ld + (i - row * F)] = v;
  }
}

// The first `slope_blocks` blocks add the heads' slope gradients, the others everything else.
__global__ __launch_bounds__(256) void join_kernel(const AttnJoinArgs a, int slope_blocks) {
  if ((int)blockIdx.x < slope_blocks) {
    // per row: sum dS d - sum dS * sum P d over its parts
    __shared__ float red[256];
    const int h = blockIdx.x;
    float v = 0.f;
    if (a.part_slope)
      for (int64_t i = threadIdx.x; i < a.Nq; i += 256) {
        if (!covered(a.qo, a.G, a.Nq, i)) continue;
        float sd = 0.f, s = 0.f, pd = 0.f;
        for (int p = 0; p < a.nsplit_q; ++p) {
          const float* o = a.part_slope + (((int64_t)p * a.H + h) * a.Nq + i) * 3;
          sd += o[0];
          s += o[1];
          pd += o[2];
        }
        v += fmaf(-s, pd, sd);
      }
    red[threadIdx.x] = v;
    __syncthreads();
    for (int s = 128; s > 0; s >>= 1) {
      if ((int)threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
      __syncthreads();
    }
    if (threadIdx.x == 0) a.gslope[h] = -red[0];
    return;
  }
  const int64_t first = (int64_t)(blockIdx.x - slope_blocks) * 256 + threadIdx.x;
  const int64_t step = (int64_t)(gridDim.x - slope_blocks) * 256;
  if (a.part_gq) sum_rows(a.part_gq, a.nsplit_q, a.Nq, a.Fqk, a.gq, a.ldgq, a.qo, a.G, first, step);
  if (a.part_gk) sum_rows(a.part_gk, a.nsplit_k, a.Nk, a.Fqk, a.gk, a.ldgk, a.ko, a.G, first, step);
  if (a.part_gv) sum_rows(a.part_gv, a.nsplit_k, a.Nk, a.Fv, a.gv, a.ldgv, a.ko, a.G, first, step);
  if (a.gpos)
    for (int64_t i = first; i < a.Nq * 3; i += step) {
      if (!covered(a.qo, a.G, a.Nq, i / 3)) continue;
      float v = 0.f;
      if (a.part_qpos)
        for (int p = 0; p < a.nsplit_q * a.H; ++p) v += a.part_qpos[p * a.Nq * 3 + i];
      if (!a.gkpos && a.part_kpos)  // self form: the nodes' other ends
        for (int p = 0; p < a.nsplit_k * a.H; ++p) v += a.part_kpos[p * a.Nk * 3 + i];
      a.gpos[i] = v;
    }
  if (a.gkpos)
    for (int64_t i = first; i < a.Nk * 3; i += step) {
      if (!covered(a.ko, a.G, a.Nk, i / 3)) continue;
      float v = 0.f;
      for (int p = 0; p < a.nsplit_k * a.H; ++p) v += a.part_kpos[p * a.Nk * 3 + i];
      a.gkpos[i] = v;
    }
}

hipError_t launch_class(int kind, AttnArgs& a, const AttnShape& s, hipStream_t st) {
  TimingScope ts(kcAttention, st);
  a.tiles = s.tiles;
  a.nsplit = s.nsplit;
  return kLaunch[s.cls](kind, a, s.cols, st);
}

}  // namespace

AttnShape attn_shape(int D, int64_t rows, int64_t other, int64_t graphs, int heads) {
  AttnShape s;
  s.cls = 0;
  while (kWidth[s.cls] < D) ++s.cls;
  const int64_t g = std::max<int64_t>(1, graphs);
  s.cols = rows / g >= 96 ? 128 : attn_small_cols(kWidth[s.cls]);
  const int64_t m = s.cols;
  s.tiles = rows / m + g;
  // too few blocks for the 256 CUs: cut the long axis, 64 rows of it at least per part
  const int64_t blocks = std::max<int64_t>((rows + m - 1) / m, std::min(rows, g)) * heads;
  const int64_t most = std::max<int64_t>(1, other / g / 64), enough = s.cols < 128 ? 2048 : 512;
  s.nsplit = (int)std::min<int64_t>(std::min<int64_t>(64, most), std::max<int64_t>(1, enough / std::max<int64_t>(1, blocks)));
  return s;
}

hipError_t launch_attn_forward(AttnArgs& a, const AttnShape& s, hipStream_t st) { return launch_class(0, a, s, st); }
hipError_t launch_attn_grad_q(AttnArgs& a, const AttnShape& s, hipStream_t st) { return launch_class(1, a, s, st); }
hipError_t launch_attn_grad_kv(AttnArgs& a, const AttnShape& s, hipStream_t st) { return launch_class(2, a, s, st); }

hipError_t launch_attn_combine(AttnArgs& a, const AttnShape& s, hipStream_t st) {
  TimingScope ts(kcAttention, st);
  const int64_t tiles = a.Nq / 32 + std::max(1, a.G);
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)tiles), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_attn_join(const AttnJoinArgs& a, hipStream_t st) {
  TimingScope ts(kcAttention, st);
  int64_t most = std::max(a.Nq, a.Nk) * 3;
  if (a.part_gq) most = std::max(most, a.Nq * a.Fqk);
  if (a.part_gk) most = std::max(most, a.Nk * a.Fqk);
  if (a.part_gv) most = std::max(most, a.Nk * a.Fv);
  const int64_t blocks = std::min<int64_t>(2048, (most + 255) / 256);
  const int slope = a.gslope ? a.H : 0;
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)std::max<int64_t>(1, blocks) + slope), dim3(256), 0, st, a, slope);
  return hipGetLastError();
}

}  // namespace tpconv
