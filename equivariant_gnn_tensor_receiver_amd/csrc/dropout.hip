// Dropout of irreps features with a mask from a counter-based generator
// (include/tpconv_attention.h): y = residual + x * keep / (1 - p').
//
// The mask is drawn again wherever it is needed and never stored.  One call of
// Philox4x32-10 gives eight 16-bit words, the draws of eight channels; a thread
// makes one call and applies it to the 2l+1 rows of its eight channels, 16 or
// 32 bytes at a time.  The draws cost ten rounds of two 32 x 32 bit products
// per eight channels, about 15 operations per scalar channel and less for the
// other degrees, which a pass over fp32 features hides behind its memory
// accesses.
#include "attention.h"
#include "device_common.h"
#include "timing.h"

#include <algorithm>

namespace tpconv {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Philox4x32-10 (J. Salmon et al., Parallel random numbers: as easy as 1, 2, 3, 2011).
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
    const uint32_t n0 = (uint32_t)(q >> 32) ^ c1 ^ k0, n2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)q;
    c3 = (uint32_t)p;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return (u32x4){c0, c1, c2, c3};
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const floatx4 x = *reinterpret_cast<const floatx4_any*>(p + 4 * j);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * j + e] = x[e];
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 x = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(x[j] << 16);
    v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<floatx4_any*>(p + 4 * j) = (floatx4){v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  u32x4 x;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = bf16_bits(v[2 * j]) | (bf16_bits(v[2 * j + 1]) << 16);
  *reinterpret_cast<u32x4_any*>(p) = x;
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)bf16_bits(v); }

constexpr int kThreads = 256;

// x, res and y may be the same memory: every value is read and written by one thread.
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const DropArgs a, int nodes) {
  const uint64_t seed = (uint64_t)a.rng[0], offset = (uint64_t)a.rng[1];
  const TX* x = static_cast<const TX*>(a.x);
  const TY* res = static_cast<const TY*>(a.res);
  TY* y = static_cast<TY*>(a.y);
  const uint32_t limit = (uint32_t)a.limit;
  // `nodes` nodes per block and step
  for (int64_t base = (int64_t)blockIdx.x * nodes; base < a.N; base += (int64_t)gridDim.x * nodes) {
    const int here = (int)(a.N - base < nodes ? a.N - base : nodes), items = here * a.groups;
    for (int idx = threadIdx.x; idx < items; idx += kThreads) {
      const int nd = idx / a.groups, g = idx - nd * a.groups;
      int i = 0;
      while (i + 1 < a.nirr && g >= a.ir[i + 1].first) ++i;
      const int c = (g - a.ir[i].first) * 8, mul = a.ir[i].mul, n = a.ir[i].n;
      const uint64_t b = (uint64_t)(base + nd) * (uint64_t)a.groups + (uint64_t)g;
      int64_t at = (base + nd) * a.F + a.ir[i].off + c;
      const bool whole = c + 8 <= mul;
      // the first row is on its way while the mask is drawn, the next one while a row is written
      float v[8], q[8];
      auto load = [&](int64_t p) {
        load8(x + p, v);
        if (a.has_res) load8(res + p, q);
      };
      if (whole) load(at);
      const u32x4 w = philox((uint32_t)b, (uint32_t)(b >> 32), (uint32_t)offset, (uint32_t)(offset >> 32),
                             (uint32_t)seed, (uint32_t)(seed >> 32));
      bool keep[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) keep[e] = ((w[e >> 1] >> (16 * (e & 1))) & 0xffffu) >= limit;
      if (whole) {
        for (int r = 0; r < n; ++r, at += mul) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            o[e] = keep[e] ? v[e] * a.factor : 0.f;
            if (a.has_res) o[e] += q[e];
          }
          if (r + 1 < n) load(at + mul);
          store8(y + at, o);
        }
      } else {
        for (int r = 0; r < n; ++r, at += mul)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < mul) {
              float o = keep[e] ? load_feat(x, at + e) * a.factor : 0.f;
              if (a.has_res) o += load_feat(res, at + e);
              store1(y + at + e, o);
            }
      }
    }
  }
}

}  // namespace

hipError_t launch_dropout(const DropArgs& a, hipStream_t s) {
  TimingScope ts(kcDropout, s);
  const int nodes = std::max(1, 512 / a.groups);
  const int64_t blocks = std::min<int64_t>((a.N + nodes - 1) / nodes, 1 << 20);
  const dim3 grid((unsigned)blocks), block(kThreads);
  if (a.x_bf16 && a.y_bf16)
    hipLaunchKernelGGL((dropout_kernel<uint16_t, uint16_t>), grid, block, 0, s, a, nodes);
  else if (a.x_bf16)
    hipLaunchKernelGGL((dropout_kernel<uint16_t, float>), grid, block, 0, s, a, nodes);
  else if (a.y_bf16)
    hipLaunchKernelGGL((dropout_kernel<float, uint16_t>), grid, block, 0, s, a, nodes);
  else
    hipLaunchKernelGGL((dropout_kernel<float, float>), grid, block, 0, s, a, nodes);
  return hipGetLastError();
}

}  // namespace tpconv
