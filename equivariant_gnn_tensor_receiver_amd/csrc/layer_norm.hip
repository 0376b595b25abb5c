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
//
// Measured (kernel times; a plain copy of the sizes runs at 5.4 to 8.5 TB/s on
// this chip): 32768 nodes of 288 fp32 values forward 14.2 us (5.3 TB/s),
// backward 20.5 (5.5) and 4.1 for the sums of the parameters; 8192 rows of 4096
// bf16 values forward 25 us (5.4 TB/s; 28.7 with other inputs in between),
// backward 65.1 (fp32 gradients, 5.2) and 5.0; 64 nodes of 32 values 3.1 us (a
// launch).
//
// Range: sums are plain fp32 sums, so a block whose sum of squares passes 3.4e38
// has r = 0 (or NaN, once its plain sum does).
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

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));  // at any element's address

// Wide accesses need no more than an element's alignment.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// The four neighbouring channels a thread holds of one row: one wide access,
// or one by one where the row ends among them (TAIL; rows of a multiple of four
// channels have no such quad, and the wide kernels are built for them apart:
// 8192 x 4096 bf16 forward 28.6 us against 38.2, backward 64 against 82);
// channels past the row read as zero.
template <bool TAIL>
struct Quad {
  int c0, mul;
  __device__ __forceinline__ bool has(int q) const { return TAIL ? c0 + q < mul : c0 < mul; }
  __device__ __forceinline__ bool whole() const { return TAIL ? c0 + 4 <= mul : c0 < mul; }
  // (zero first, then the load: an else branch that zeroes would wait for the loads in flight)
  __device__ __forceinline__ void load(const float* p, bool ok, float (&v)[4]) const {
    floatx4_any x = {0.f, 0.f, 0.f, 0.f};
    if (ok && whole()) x = *reinterpret_cast<const floatx4_any*>(p + c0);
    if (TAIL && ok && !whole())
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (has(q)) x[q] = p[c0 + q];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = x[q];
  }
  __device__ __forceinline__ void load(const uint16_t* p, bool ok, float (&v)[4]) const {
    u32x2_any x = {0, 0};
    if (ok && whole()) x = *reinterpret_cast<const u32x2_any*>(p + c0);
    if (TAIL && ok && !whole()) {
      if (has(0)) x[0] = p[c0];
      if (has(1)) x[0] |= (uint32_t)p[c0 + 1] << 16;
      if (has(2)) x[1] = p[c0 + 2];
    }
    v[0] = __uint_as_float(x[0] << 16);
    v[1] = __uint_as_float(x[0] & 0xffff0000u);
    v[2] = __uint_as_float(x[1] << 16);
    v[3] = __uint_as_float(x[1] & 0xffff0000u);
  }
  __device__ __forceinline__ void store(float* p, const float (&v)[4]) const {
    if (whole()) {
      *reinterpret_cast<floatx4_any*>(p + c0) = (floatx4_any){v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (TAIL && has(q)) p[c0 + q] = v[q];
    }
  }
  __device__ __forceinline__ void store(uint16_t* p, const float (&v)[4]) const {
    if (whole()) {
      const bf16x2 lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};
      *reinterpret_cast<u32x2_any*>(p + c0) =
          (u32x2_any){__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (TAIL && has(q)) store1(p, c0 + q, v[q]);
    }
  }
  // weight and bias: `none` where there are none
  __device__ __forceinline__ void load_param(const float* p, float none, float (&v)[4]) const {
    if (p) {
      load(p, true, v);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = none;
    }
  }
};

// ---- narrow blocks (at most 256 channels) -------------------------------------------
// A group of `lanes` lanes (a power of two, four channels per lane) takes one
// (node, irrep) and keeps its N rows in registers: one read, statistics by lane
// swaps, one write.  (A block of threads per node and irrep with the values read
// again for each sum, the general path below, takes 437 us for the 32768 x 288
// training step against 39.)

template <int N, typename TX, typename TY>
__device__ __forceinline__ void forward_narrow(const NormArgs& a, const NormIrrep& ir) {
  const int lanes = ir.lanes, t = threadIdx.x & (lanes - 1), per = kThreads / lanes, slot = threadIdx.x / lanes;
  const Quad<true> qd{4 * t, ir.mul};
  const float len = (float)(ir.mul * N);
  float w[4], b[4];
  qd.load_param(a.w ? a.w + ir.w_off : nullptr, 1.f, w);
  qd.load_param(ir.scalar && a.b ? a.b + ir.b_off : nullptr, 0.f, b);
  for (int64_t v0 = (int64_t)(blockIdx.x - ir.first_block) * per; v0 < a.N; v0 += (int64_t)ir.blocks * per) {
    const int64_t v = v0 + slot;
    const bool ok = v < a.N;
    const int64_t at = v * a.F + ir.off;
    float x[N][4];
#pragma unroll
    for (int m = 0; m < N; ++m) qd.load(static_cast<const TX*>(a.x) + at + m * ir.mul, ok, x[m]);
    float mu = 0.f;
    if (N == 1 && ir.scalar) {
      mu = group_sum((x[0][0] + x[0][1]) + (x[0][2] + x[0][3]), lanes) / len;
#pragma unroll
      for (int q = 0; q < 4; ++q) x[0][q] = qd.has(q) ? x[0][q] - mu : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) s = __builtin_fmaf(x[m][q], x[m][q], s);
    const float r = 1.f / sqrtf(group_sum(s, lanes) / len + a.eps);
    if (!ok) continue;
#pragma unroll
    for (int m = 0; m < N; ++m) {
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(x[m][q] * r, w[q], b[q]);
      qd.store(static_cast<TY*>(a.y) + at + m * ir.mul, y);
    }
    if (a.stats && t == 0) {
      float* st = a.stats + (v * a.nirreps + (&ir - a.ir)) * 2;
      st[0] = mu;
      st[1] = r;
    }
  }
}

template <int N, typename TX>
__device__ __forceinline__ void backward_narrow(const NormArgs& a, const NormIrrep& ir, float (*red)[512]) {
  const int lanes = ir.lanes, t = threadIdx.x & (lanes - 1), per = kThreads / lanes, slot = threadIdx.x / lanes;
  const int rank = blockIdx.x - ir.first_block;
  const Quad<true> qd{4 * t, ir.mul};
  const float len = (float)(ir.mul * N);
  float w[4], sw[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
  qd.load_param(a.w ? a.w + ir.w_off : nullptr, 1.f, w);
  for (int64_t v0 = (int64_t)rank * per; v0 < a.N; v0 += (int64_t)ir.blocks * per) {
    const int64_t v = v0 + slot;
    const bool ok = v < a.N;
    const int64_t at = v * a.F + ir.off;
    float x[N][4], g[N][4];
#pragma unroll
    for (int m = 0; m < N; ++m) {
      qd.load(static_cast<const TX*>(a.x) + at + m * ir.mul, ok, x[m]);
      qd.load(a.gy + at + m * ir.mul, ok, g[m]);
    }
    float mu = 0.f, r = 0.f;
    if (a.stats) {
      if (ok) {
        const float* st = a.stats + (v * a.nirreps + (&ir - a.ir)) * 2;
        mu = st[0];
        r = st[1];
      }
    } else if (N == 1 && ir.scalar) {
      mu = group_sum((x[0][0] + x[0][1]) + (x[0][2] + x[0][3]), lanes) / len;
    }
    if (N == 1 && ir.scalar)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[0][q] = qd.has(q) ? x[0][q] - mu : 0.f;
    if (!a.stats) {
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < N; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q) s = __builtin_fmaf(x[m][q], x[m][q], s);
      r = 1.f / sqrtf(group_sum(s, lanes) / len + a.eps);
    }
    float sh = 0.f, shz = 0.f;
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[m][q] *= r;  // z
        sw[q] = ok ? __builtin_fmaf(g[m][q], x[m][q], sw[q]) : sw[q];
        sb[q] += g[m][q];
        g[m][q] *= w[q];  // h
        sh += g[m][q];
        shz = __builtin_fmaf(g[m][q], x[m][q], shz);
      }
    const float mz = group_sum(shz, lanes) / len;
    const float mh = N == 1 && ir.scalar ? group_sum(sh, lanes) / len : 0.f;
    if (!a.gx || !ok) continue;
#pragma unroll
    for (int m = 0; m < N; ++m) {
      float d[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = r * (g[m][q] - x[m][q] * mz - mh);
      qd.store(a.gx + at + m * ir.mul, d);
    }
  }
  if (!a.part) return;
  // the block's sums: over the groups of a wave by lane swaps, over the waves in order
#pragma unroll
  for (int q = 0; q < 4; ++q)
    for (int d = lanes; d < 64; d <<= 1) {
      sw[q] += __shfl_xor(sw[q], d);
      sb[q] += __shfl_xor(sb[q], d);
    }
  const int wave = threadIdx.x >> 6;
  if ((int)(threadIdx.x & 63) < lanes)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (qd.has(q)) {
        red[wave][qd.c0 + q] = sw[q];
        red[wave][256 + qd.c0 + q] = sb[q];
      }
  __syncthreads();
  float* part = a.part + ir.part_off + (int64_t)rank * ir.mul * (1 + ir.scalar);
  const int c = threadIdx.x;
  if (c >= ir.mul) return;
  part[c] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
  if (ir.scalar) part[ir.mul + c] = (red[0][256 + c] + red[1][256 + c]) + (red[2][256 + c] + red[3][256 + c]);
}

template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_forward_narrow_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const NormIrrep& ir = find_irrep(a, blockIdx.x);
  switch (ir.n) {
    case 1: forward_narrow<1, TX, TY>(a, ir); break;
    case 3: forward_narrow<3, TX, TY>(a, ir); break;
    case 5: forward_narrow<5, TX, TY>(a, ir); break;
    default: forward_narrow<7, TX, TY>(a, ir); break;
  }
}

template <typename TX>
__global__ __launch_bounds__(kThreads) void norm_backward_narrow_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float red[4][512];
  const NormIrrep& ir = find_irrep(a, blockIdx.x);
  switch (ir.n) {
    case 1: backward_narrow<1, TX>(a, ir, red); break;
    case 3: backward_narrow<3, TX>(a, ir, red); break;
    case 5: backward_narrow<5, TX>(a, ir, red); break;
    default: backward_narrow<7, TX>(a, ir, red); break;
  }
}

// ---- wide scalar rows (one row of 257 to 8192 channels) ------------------------------
// A block of threads per node; a thread keeps its 4 V channels of the row, of
// the weights and of the parameter gradients in registers over all its nodes.
// (8192 x 4096 bf16 training step: 699 us on the general path, 142 with a row's
// values in registers, 99 with the weights kept and the next row prefetched.)

__device__ __forceinline__ void block_sum2(float& u, float& v, float2* tmp) {
  u = group_sum(u, 64);
  v = group_sum(v, 64);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = {u, v};
  __syncthreads();
  u = (tmp[0].x + tmp[1].x) + (tmp[2].x + tmp[3].x);
  v = (tmp[0].y + tmp[1].y) + (tmp[2].y + tmp[3].y);
  __syncthreads();
}

// Runs of 1024 channels per j.
template <bool TAIL>
__device__ __forceinline__ Quad<TAIL> wide_quad(const NormIrrep& ir, int j) {
  return {4 * ((int)threadIdx.x + j * kThreads), ir.mul};
}

template <int V, bool TAIL, typename TX, typename TY>
__device__ __forceinline__ void forward_wide(const NormArgs& a, const NormIrrep& ir, float* tmp) {
  const float len = (float)ir.mul;
  const TX* in = static_cast<const TX*>(a.x) + ir.off;
  float w[V][4], b[V][4], x[V][4], next[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const Quad<TAIL> qd = wide_quad<TAIL>(ir, j);
    qd.load_param(a.w ? a.w + ir.w_off : nullptr, 1.f, w[j]);
    qd.load_param(ir.scalar && a.b ? a.b + ir.b_off : nullptr, 0.f, b[j]);
  }
  int64_t v = blockIdx.x - ir.first_block;
#pragma unroll
  for (int j = 0; j < V; ++j) wide_quad<TAIL>(ir, j).load(in + min(v, a.N - 1) * a.F, true, next[j]);
  for (; v < a.N; v += ir.blocks) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[j][q] = next[j][q];
    // the next row (or the last one again) is on its way during the sums
#pragma unroll
    for (int j = 0; j < V; ++j) wide_quad<TAIL>(ir, j).load(in + min(v + ir.blocks, a.N - 1) * a.F, true, next[j]);
    float mu = 0.f, s = 0.f;
    if (ir.scalar) {
#pragma unroll
      for (int j = 0; j < V; ++j) s += (x[j][0] + x[j][1]) + (x[j][2] + x[j][3]);
      mu = block_sum(s, tmp) / len;
      s = 0.f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[j][q] = wide_quad<TAIL>(ir, j).has(q) ? x[j][q] - mu : 0.f;
        s = __builtin_fmaf(x[j][q], x[j][q], s);
      }
    const float r = 1.f / sqrtf(block_sum(s, tmp) / len + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(x[j][q] * r, w[j][q], b[j][q]);
      wide_quad<TAIL>(ir, j).store(static_cast<TY*>(a.y) + v * a.F + ir.off, y);
    }
    if (a.stats && threadIdx.x == 0) {
      float* st = a.stats + (v * a.nirreps + (&ir - a.ir)) * 2;
      st[0] = mu;
      st[1] = r;
    }
  }
}

template <int V, bool TAIL, typename TX>
__device__ __forceinline__ void backward_wide(const NormArgs& a, const NormIrrep& ir, float2* tmp) {
  const float len = (float)ir.mul;
  const int rank = blockIdx.x - ir.first_block;
  float w[V][4], sw[V][4], sb[V][4], x[V][4], g[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    wide_quad<TAIL>(ir, j).load_param(a.w ? a.w + ir.w_off : nullptr, 1.f, w[j]);
#pragma unroll
    for (int q = 0; q < 4; ++q) sw[j][q] = sb[j][q] = 0.f;
  }
  for (int64_t v = rank; v < a.N; v += ir.blocks) {
    const int64_t at = v * a.F + ir.off;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      wide_quad<TAIL>(ir, j).load(static_cast<const TX*>(a.x) + at, true, x[j]);
      wide_quad<TAIL>(ir, j).load(a.gy + at, true, g[j]);
    }
    float mu = 0.f, r, none = 0.f;
    if (a.stats) {
      const float* st = a.stats + (v * a.nirreps + (&ir - a.ir)) * 2;
      mu = st[0];
      r = st[1];
    } else {
      if (ir.scalar) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) s += (x[j][0] + x[j][1]) + (x[j][2] + x[j][3]);
        block_sum2(s, none, tmp);
        mu = s / len;
      }
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float d = wide_quad<TAIL>(ir, j).has(q) ? x[j][q] - mu : 0.f;
          s = __builtin_fmaf(d, d, s);
        }
      block_sum2(s, none, tmp);
      r = 1.f / sqrtf(s / len + a.eps);
    }
    float sh = 0.f, shz = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // (past the row z is not zero, but its g is)
        x[j][q] = (x[j][q] - mu) * r;
        const float h = g[j][q] * w[j][q];
        sw[j][q] = __builtin_fmaf(g[j][q], x[j][q], sw[j][q]);
        sb[j][q] += g[j][q];
        sh += h;
        shz = __builtin_fmaf(h, x[j][q], shz);
      }
    block_sum2(sh, shz, tmp);
    const float mz = shz / len, mh = ir.scalar ? sh / len : 0.f;
    if (!a.gx) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = r * (g[j][q] * w[j][q] - x[j][q] * mz - mh);
      wide_quad<TAIL>(ir, j).store(a.gx + at, d);
    }
  }
  if (!a.part) return;
  float* part = a.part + ir.part_off + (int64_t)rank * ir.mul * (1 + ir.scalar);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const Quad<TAIL> qd = wide_quad<TAIL>(ir, j);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (qd.has(q)) {
        part[qd.c0 + q] = sw[j][q];
        if (ir.scalar) part[ir.mul + qd.c0 + q] = sb[j][q];
      }
  }
}

template <int V, typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_forward_wide_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float tmp[4];
  const NormIrrep& ir = find_irrep(a, blockIdx.x);
  if (ir.mul % 4 == 0)
    forward_wide<V, false, TX, TY>(a, ir, tmp);
  else
    forward_wide<V, true, TX, TY>(a, ir, tmp);
}

template <int V, typename TX>
__global__ __launch_bounds__(kThreads) void norm_backward_wide_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float2 tmp[4];
  const NormIrrep& ir = find_irrep(a, blockIdx.x);
  if (ir.mul % 4 == 0)
    backward_wide<V, false, TX>(a, ir, tmp);
  else
    backward_wide<V, true, TX>(a, ir, tmp);
}

// ---- everything else (several rows of more than 256 channels, longer rows) -----------
// A block of threads per (node, irrep) that reads the block again for each sum
// (4096 x 8193 fp32: forward 85 us, backward 511, where 8192 channels take 42 and
// 93; 16384 nodes of 300x1o: 33 and 160).

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

// The blocks' sums of 32 parameters of an irrep: 32 threads per parameter take
// every 32nd block each, and their sums are added in order.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const NormArgs /*args*/) {
  const NormArgs& a = *(const NormArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float red[32][33];
  const NormIrrep& ir = a.ir[blockIdx.y];
  const int len = ir.mul * (1 + ir.scalar), col = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  if ((int)blockIdx.x * 32 >= len) return;
  float s = 0.f;
  if (c < len) {
    const float* p = a.part + ir.part_off + c;
#pragma unroll 8
    for (int k = row; k < ir.blocks; k += 32) s += p[(int64_t)k * len];
  }
  red[row][col] = s;
  __syncthreads();
  for (int h = 16; h > 0; h >>= 1) {
    if (row < h) red[row][col] += red[row + h][col];
    __syncthreads();
  }
  if (row != 0 || c >= len) return;
  s = red[0][col];
  if (c < ir.mul) {
    if (a.gw) a.gw[ir.w_off + c] = s;
  } else if (a.gb) {
    a.gb[ir.b_off + c - ir.mul] = s;
  }
}

enum Kind { kNarrow = 0, kWide1, kWide2, kWide4, kWide8, kLong, kKinds };

// How an irrep's blocks are computed.
int irrep_kind(const NormIrrep& ir) {
  if (ir.mul <= 256) return kNarrow;
  if (ir.n > 1 || ir.mul > 8192) return kLong;
  return ir.mul <= 1024 ? kWide1 : ir.mul <= 2048 ? kWide2 : ir.mul <= 4096 ? kWide4 : kWide8;
}

// Lanes per (node, irrep) of narrow blocks: four channels per lane.
void set_lanes(NormArgs& a) {
  for (int i = 0; i < a.nirreps; ++i) {
    NormIrrep& ir = a.ir[i];
    ir.lanes = 1;
    while (ir.lanes < 64 && ir.lanes * 4 < ir.mul) ir.lanes *= 2;
  }
}

// The irreps of one kind as a launch of their own.
int64_t kind_args(const NormArgs& a, int kind, NormArgs& k) {
  k = a;
  int64_t blocks = 0;
  for (int i = 0; i < a.nirreps; ++i) {
    NormIrrep& ir = k.ir[i];
    if (irrep_kind(ir) != kind) ir.blocks = 0;
    ir.first_block = (int32_t)blocks;
    blocks += ir.blocks;
  }
  return blocks;
}

#define TP_NORM_XY(KERNEL, ...)                                                                          \
  (a.x_bf16 ? (a.y_bf16 ? (const void*)KERNEL<__VA_ARGS__ uint16_t, uint16_t>                            \
                        : (const void*)KERNEL<__VA_ARGS__ uint16_t, float>)                              \
            : (a.y_bf16 ? (const void*)KERNEL<__VA_ARGS__ float, uint16_t> : (const void*)KERNEL<__VA_ARGS__ float, float>))
#define TP_NORM_X(KERNEL, ...) \
  (a.x_bf16 ? (const void*)KERNEL<__VA_ARGS__ uint16_t> : (const void*)KERNEL<__VA_ARGS__ float>)
#define TP_COMMA ,

hipError_t launch(const void* kernel, NormArgs& k, int64_t blocks, hipStream_t s) {
  void* args[] = {&k};
  return hipLaunchKernel(kernel, dim3((unsigned)blocks), dim3(kThreads), args, 0, s);
}

}  // namespace

int64_t norm_backward_blocks(NormArgs& a) {
  // about 2048 blocks of narrow irreps, shared by their sizes; 512 per wider irrep, whose rows of
  // partial sums are as long as the irrep (8 KiB per block at 1024 scalar channels)
  int64_t total = 0, part = 0;
  for (int i = 0; i < a.nirreps; ++i) total += irrep_kind(a.ir[i]) == kNarrow ? (int64_t)a.ir[i].mul * a.ir[i].n : 0;
  set_lanes(a);
  for (int i = 0; i < a.nirreps; ++i) {
    NormIrrep& ir = a.ir[i];
    int64_t most = a.N, want = 512;
    if (irrep_kind(ir) == kNarrow) {
      const int per = kThreads / ir.lanes;
      most = (a.N + per - 1) / per;
      want = 2048 * (int64_t)ir.mul * ir.n / total + 1;
    }
    ir.blocks = (int32_t)(want < most ? want : most > 0 ? most : 1);
    ir.part_off = part;
    part += (int64_t)ir.blocks * ir.mul * (1 + ir.scalar);
  }
  return part;
}

hipError_t launch_norm_forward(NormArgs& a, hipStream_t s) {
  TimingScope ts(kcNorm, s);
  set_lanes(a);
  for (int i = 0; i < a.nirreps; ++i) {
    NormIrrep& ir = a.ir[i];
    const int per = irrep_kind(ir) == kNarrow ? kThreads / ir.lanes : 1;
    const int kind = irrep_kind(ir);
    // wide rows: 1024 blocks that keep the weights in registers over their rows (8192 x 4096
    // bf16: 28.6 us, 29.8 with 2048 blocks, 31.9 with 4096; 76 us a block per row)
    const int64_t n = (a.N + per - 1) / per, most = kind == kNarrow || kind == kLong ? 65536 : 1024;
    ir.blocks = (int32_t)(n < most ? n : most);
  }
  for (int kind = 0; kind < kKinds; ++kind) {
    NormArgs k;
    const int64_t blocks = kind_args(a, kind, k);
    if (blocks == 0) continue;
    const void* f = kind == kNarrow  ? TP_NORM_XY(norm_forward_narrow_kernel, )
                    : kind == kWide1 ? TP_NORM_XY(norm_forward_wide_kernel, 1 TP_COMMA)
                    : kind == kWide2 ? TP_NORM_XY(norm_forward_wide_kernel, 2 TP_COMMA)
                    : kind == kWide4 ? TP_NORM_XY(norm_forward_wide_kernel, 4 TP_COMMA)
                    : kind == kWide8 ? TP_NORM_XY(norm_forward_wide_kernel, 8 TP_COMMA)
                                     : TP_NORM_XY(norm_forward_kernel, );
    const hipError_t e = launch(f, k, blocks, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_norm_backward(NormArgs& a, hipStream_t s) {
  TimingScope ts(kcNorm, s);
  norm_backward_blocks(a);
  for (int kind = 0; kind < kKinds; ++kind) {
    NormArgs k;
    const int64_t blocks = kind_args(a, kind, k);
    if (blocks == 0) continue;
    const void* f = kind == kNarrow  ? TP_NORM_X(norm_backward_narrow_kernel, )
                    : kind == kWide1 ? TP_NORM_X(norm_backward_wide_kernel, 1 TP_COMMA)
                    : kind == kWide2 ? TP_NORM_X(norm_backward_wide_kernel, 2 TP_COMMA)
                    : kind == kWide4 ? TP_NORM_X(norm_backward_wide_kernel, 4 TP_COMMA)
                    : kind == kWide8 ? TP_NORM_X(norm_backward_wide_kernel, 8 TP_COMMA)
                                     : TP_NORM_X(norm_backward_kernel, );
    const hipError_t e = launch(f, k, blocks, s);
    if (e != hipSuccess) return e;
  }
  if (!a.part) return hipSuccess;
  int most = 0;
  for (int i = 0; i < a.nirreps; ++i) {
    const int len = a.ir[i].mul * (1 + a.ir[i].scalar);
    most = len > most ? len : most;
  }
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((most + 31) / 32), (unsigned)a.nirreps), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace tpconv
