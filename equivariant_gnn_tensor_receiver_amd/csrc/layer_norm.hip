// Layer norm over irreps: forward, backward and the reduction of the weight
// and bias gradients.
//
//   0e blocks:    mu = mean(v), r = 1 / sqrt(mean((v - mu)^2) + eps), z = (v - mu) r, y = w z + b
//   other blocks: r = 1 / sqrt(mean(v^2) + eps), z = v r, y = w z
//   backward with h = w g:  gx = r (h - z mean(h z) - [0e] mean(h)),
//   gw_c = sum over nodes and rows of g z,  gb_c = sum over nodes of g
//
// The mean is taken first and the squares are summed around it (two passes
// over the block), so a large mean costs no digits of the variance.
//
// Bound by HBM: the forward reads x and writes y, the backward reads x and g
// and writes gx; the parameter gradients are summed per block of threads over
// the nodes it takes, and the blocks' sums are added in a fixed order.
#include "device_common.h"
#include "layers.h"
#include "timing.h"

namespace tpconv {

namespace {

constexpr int kThreads = 256;

template <int CTRL>
__device__ __forceinline__ float dpp_step(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Sum over aligned groups of `lanes` lanes (a power of two, uniform), the
// result in every lane.  All lanes of the wave take part.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes >= 2) v = dpp_step<0xB1>(v);    // quad_perm [1,0,3,2]
  if (lanes >= 4) v = dpp_step<0x4E>(v);    // quad_perm [2,3,0,1]
  if (lanes >= 8) v = dpp_step<0x141>(v);   // row_half_mirror
  if (lanes >= 16) v = dpp_step<0x140>(v);  // row_mirror
  if (lanes >= 32) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (lanes >= 64) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sum over the block's 256 threads, the result in every thread.
__device__ __forceinline__ float block_sum(float v, float* tmp) {
  v = group_sum(v, 64);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
  __syncthreads();
  return v;
}

template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return load_feat(static_cast<const T*>(p), i);
}
__device__ __forceinline__ void store1(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store1(uint16_t* p, int64_t i, float v) {
  p[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

__device__ __forceinline__ const NormIrrep& find_irrep(const NormArgs& a, int block) {
  int i = 0;
  while (i + 1 < a.nirreps && block >= a.ir[i + 1].first_block) ++i;
  return a.ir[i];
}

// Mean and 1 / deviation of one block of values, one thread block per (node, irrep).
template <typename TX>
__device__ __forceinline__ void block_stats(const void* x, int64_t at, const NormIrrep& ir, float eps, float* tmp,
                                            float& mu, float& r) {
  const int len = ir.mul * ir.n;
  mu = 0.f;
  if (ir.scalar) {
    float s = 0.f;
    for (int i = threadIdx.x; i < len; i += kThreads) s += load1<TX>(x, at + i);
    mu = block_sum(s, tmp) / (float)len;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < len; i += kThreads) {
    const float d = load1<TX>(x, at + i) - mu;
    q = __builtin_fmaf(d, d, q);
  }
  r = 1.f / sqrtf(block_sum(q, tmp) / (float)len + eps);
}

template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_forward_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float tmp[4];
  const NormIrrep& ir = find_irrep(a, blockIdx.x);
  const int len = ir.mul * ir.n;
  for (int64_t v = blockIdx.x - ir.first_block; v < a.N; v += ir.blocks) {
    const int64_t at = v * a.F + ir.off;
    float mu, r;
    block_stats<TX>(a.x, at, ir, a.eps, tmp, mu, r);
    for (int i = threadIdx.x; i < len; i += kThreads) {
      const int c = i % ir.mul;
      float y = (load1<TX>(a.x, at + i) - mu) * r;
      if (a.w) y *= a.w[ir.w_off + c];
      if (ir.scalar && a.b) y += a.b[ir.b_off + c];
      store1(static_cast<TY*>(a.y), at + i, y);
    }
    if (a.stats && threadIdx.x == 0) {
      float* st = a.stats + (v * a.nirreps + (&ir - a.ir)) * 2;
      st[0] = mu;
      st[1] = r;
    }
  }
}

template <typename TX>
__global__ __launch_bounds__(kThreads) void norm_backward_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float tmp[4];
  const NormIrrep& ir = find_irrep(a, blockIdx.x);
  const int len = ir.mul * ir.n;
  const int rank = blockIdx.x - ir.first_block;
  float* part = a.part ? a.part + ir.part_off + (int64_t)rank * ir.mul * (1 + ir.scalar) : nullptr;
  if (part)
    for (int c = threadIdx.x; c < ir.mul * (1 + ir.scalar); c += kThreads) part[c] = 0.f;
  for (int64_t v = rank; v < a.N; v += ir.blocks) {
    const int64_t at = v * a.F + ir.off;
    float mu, r;
    if (a.stats) {
      const float* st = a.stats + (v * a.nirreps + (&ir - a.ir)) * 2;
      mu = st[0];
      r = st[1];
    } else {
      block_stats<TX>(a.x, at, ir, a.eps, tmp, mu, r);
    }
    float sh = 0.f, shz = 0.f;
    for (int i = threadIdx.x; i < len; i += kThreads) {
      const float h = a.gy[at + i] * (a.w ? a.w[ir.w_off + i % ir.mul] : 1.f);
      const float z = (load1<TX>(a.x, at + i) - mu) * r;
      sh += h;
      shz = __builtin_fmaf(h, z, shz);
    }
    const float mz = block_sum(shz, tmp) / (float)len;
    const float mh = ir.scalar ? block_sum(sh, tmp) / (float)len : 0.f;
    // a thread keeps its channels over the rows m, so the sums need no atomics
    for (int c = threadIdx.x; c < ir.mul; c += kThreads) {
      const float w = a.w ? a.w[ir.w_off + c] : 1.f;
      float sw = 0.f, sb = 0.f;
      for (int m = 0; m < ir.n; ++m) {
        const int64_t i = at + (int64_t)m * ir.mul + c;
        const float g = a.gy[i], z = (load1<TX>(a.x, i) - mu) * r;
        if (a.gx) a.gx[i] = r * (g * w - z * mz - mh);
        sw = __builtin_fmaf(g, z, sw);
        sb += g;
      }
      if (part) {
        part[c] += sw;
        if (ir.scalar) part[ir.mul + c] += sb;
      }
    }
  }
}

// One thread per parameter of an irrep: the blocks' sums in order.
__global__ __launch_bounds__(kThreads) void norm_reduce_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const NormIrrep& ir = a.ir[blockIdx.y];
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int len = ir.mul * (1 + ir.scalar);
  if (c >= len) return;
  const float* p = a.part + ir.part_off + c;
  float s = 0.f;
  for (int k = 0; k < ir.blocks; ++k) s += p[(int64_t)k * len];
  if (c < ir.mul) {
    if (a.gw) a.gw[ir.w_off + c] = s;
  } else if (a.gb) {
    a.gb[ir.b_off + c - ir.mul] = s;
  }
}

}  // namespace

int64_t norm_backward_blocks(NormArgs& a) {
  int32_t first = 0;
  int64_t part = 0;
  for (int i = 0; i < a.nirreps; ++i) {
    NormIrrep& ir = a.ir[i];
    ir.first_block = first;
    ir.blocks = (int32_t)(a.N < 512 ? (a.N > 0 ? a.N : 1) : 512);
    first += ir.blocks;
    ir.part_off = part;
    part += (int64_t)ir.blocks * ir.mul * (1 + ir.scalar);
  }
  return part;
}

hipError_t launch_norm_forward(NormArgs& a, hipStream_t s) {
  TimingScope ts(kcNorm, s);
  int32_t first = 0;
  for (int i = 0; i < a.nirreps; ++i) {
    a.ir[i].first_block = first;
    a.ir[i].blocks = (int32_t)(a.N < 65536 ? a.N : 65536);
    first += a.ir[i].blocks;
  }
  const dim3 g((unsigned)first), b(kThreads);
  if (a.x_bf16 && a.y_bf16)
    hipLaunchKernelGGL((norm_forward_kernel<uint16_t, uint16_t>), g, b, 0, s, a);
  else if (a.x_bf16)
    hipLaunchKernelGGL((norm_forward_kernel<uint16_t, float>), g, b, 0, s, a);
  else if (a.y_bf16)
    hipLaunchKernelGGL((norm_forward_kernel<float, uint16_t>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((norm_forward_kernel<float, float>), g, b, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(NormArgs& a, hipStream_t s) {
  TimingScope ts(kcNorm, s);
  norm_backward_blocks(a);
  const NormIrrep& last = a.ir[a.nirreps - 1];
  const dim3 g((unsigned)(last.first_block + last.blocks)), b(kThreads);
  if (a.x_bf16)
    hipLaunchKernelGGL((norm_backward_kernel<uint16_t>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((norm_backward_kernel<float>), g, b, 0, s, a);
  if (a.part) {
    int most = 0;
    for (int i = 0; i < a.nirreps; ++i) most = a.ir[i].mul * (1 + a.ir[i].scalar) > most ? a.ir[i].mul * (1 + a.ir[i].scalar) : most;
    hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((most + kThreads - 1) / kThreads), (unsigned)a.nirreps), b,
                       0, s, a);
  }
  return hipGetLastError();
}

}  // namespace tpconv
