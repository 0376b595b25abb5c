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

__device__ __forceinline__ bool covered(const int32_t* off, int G, int64_t N, int64_t row) {
  return !off || (row >= clamp_row(off[0], N) && row < clamp_row(off[G], N));
}

// Head of feature f of a side.
__device__ __forceinline__ int head_of(const AttnSide& s, int f) {
  int i = 0;
  while (i + 1 < s.nirr && f >= s.ir[i + 1].off) ++i;
  return (f - s.ir[i].off) % s.ir[i].mul / s.ir[i].cph;
}

// out = sum over the parts of w o / sum of w l, w = 2^(m - largest m).  A block takes one
// query at a time: its threads first turn the parts' (m, l) into factors w / sum of w l
// per part and head, then add the parts of a feature each.
constexpr int kMaxParts = 64, kCombineHeads = 64;  // heads per step
__global__ __launch_bounds__(256) void combine_kernel(const AttnArgs a) {
  __shared__ float f[kCombineHeads * kMaxParts];
  const int F = a.sv.F, S = a.nsplit;
  for (int64_t query = blockIdx.x; query < a.Nq; query += gridDim.x) {
    if (!covered(a.qo, a.G, a.Nq, query)) continue;
    for (int h0 = 0; h0 < a.H; h0 += kCombineHeads) {
      const int heads = min(kCombineHeads, a.H - h0);
      // a wave per head: lane p holds part p
      for (int hh = threadIdx.x >> 6; hh < heads; hh += 4) {
        const int p = lane_id(), h = h0 + hh;
        float m = -INFINITY, l = 0.f;
        if (p < S) {
          const float* ml = a.part_ml + 2 * (((int64_t)p * a.H + h) * a.Nq + query);
          m = ml[0];
          l = ml[1];
        }
        float top = m;
#pragma unroll
        for (int i = 32; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor(top, i));
        const bool none = m == -INFINITY && l == 0.f;  // a part without keys
        const float w = none ? 0.f : exp2_fast(m - (top == -INFINITY ? 0.f : top));
        float sum = w * l;
#pragma unroll
        for (int i = 32; i > 0; i >>= 1) sum += __shfl_xor(sum, i);
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        f[hh * kMaxParts + p] = none ? 0.f : w * inv;
        if (a.stat && p == 0) {
          a.stat[(int64_t)h * a.Nq + query] = top;
          a.stat[(int64_t)(a.H + h) * a.Nq + query] = inv;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < F; i += 256) {
        const int h = head_of(a.sv, i);
        if (h < h0 || h >= h0 + heads) continue;
        const float* w = f + (h - h0) * kMaxParts;
        float o = 0.f;
#pragma unroll 8
        for (int p = 0; p < S; ++p) {
          const float v = a.sums[((int64_t)p * a.Nq + query) * F + i];
          o = fmaf(w[p], v, o);  // (also under a factor of zero: a NaN shows as in a launch without parts)
        }
        if (a.out32) a.out32[query * F + i] = o;
        if (a.y_bf16)
          static_cast<uint16_t*>(a.out)[query * F + i] = __builtin_bit_cast(uint16_t, (__bf16)o);
        else
          static_cast<float*>(a.out)[query * F + i] = o;
      }
      __syncthreads();
    }
  }
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
  // the other side of a graph, all heads: in an XCD's L2 (4 MiB) beside what else passes through it
  const int64_t rows = (kind == 2 ? a.Nq : a.Nk) / std::max(1, a.G);
  a.heads_inner = rows * (a.sqk.F + a.sv.F) * 4 <= int64_t(2) << 20;
  return kLaunch[s.cls](kind, a, s.cols, st);
}

}  // namespace

AttnShape attn_shape(int D, int64_t rows, int64_t other, int64_t graphs, int heads, bool exact) {
  AttnShape s;
  s.cls = 0;
  while (kWidth[s.cls] < D) ++s.cls;
  const int64_t g = std::max<int64_t>(1, graphs);
  s.cols = rows / g >= 96 ? 128 : attn_small_cols(kWidth[s.cls]);
  const int64_t m = s.cols;
  s.tiles = rows / m + g;
  // too few blocks for the 256 CUs: cut the long axis, 64 rows of it at least per part, into 768 blocks, of
  // 128 columns into 512, whatever a CU holds of the kernel.  us at 256, 512, 768 and 1024 blocks: 16 queries in
  // 16 graphs over 32768 keys, fp32, 32 values per head 71, 47, 36, 30; 72 values 88, 56, 48, 56; bf16, 32 values
  // 77, 47, 36, 30; 128 values 51, 32, 30, 26; fp32, 256 values (128 columns) 68, 76, 83, 90; training of
  // 1024 nodes in one graph, 4 heads of 64 (128 columns), fp32 74, 95, 94, 94; bf16 67, 81, 81, 81
  const int64_t blocks = std::max<int64_t>((rows + m - 1) / m, std::min(rows, g)) * heads;
  const int64_t most = std::max<int64_t>(1, other / g / 64), enough = s.cols < 128 ? 768 : 512;
  s.nsplit = (int)std::min<int64_t>(std::min<int64_t>(kMaxParts, most), std::max<int64_t>(1, enough / std::max<int64_t>(1, blocks)));
  // more than 4096 rows: at least a part for each of them, up to eight, so that blocks which do not come out
  // even on the CUs are short (16384 nodes in one graph, fp32, 4 heads of 64, training: 12.1 ms in one
  // part, 7.8 in four; 8 heads of 144 38.6 and 38.7).  Not for bf16 results, which fp32 parts would be several times the size of.
  if (exact) s.nsplit = (int)std::max<int64_t>(s.nsplit, std::min<int64_t>(8, (other / g + 4095) / 4096));
  return s;
}

hipError_t launch_attn_forward(AttnArgs& a, const AttnShape& s, hipStream_t st) { return launch_class(0, a, s, st); }
hipError_t launch_attn_grad_q(AttnArgs& a, const AttnShape& s, hipStream_t st) { return launch_class(1, a, s, st); }
hipError_t launch_attn_grad_kv(AttnArgs& a, const AttnShape& s, hipStream_t st) { return launch_class(2, a, s, st); }

hipError_t launch_attn_combine(AttnArgs& a, const AttnShape& s, hipStream_t st) {
  TimingScope ts(kcAttention, st);
  a.nsplit = s.nsplit;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)std::min<int64_t>(a.Nq, 1 << 16)), dim3(256), 0, st, a);
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
