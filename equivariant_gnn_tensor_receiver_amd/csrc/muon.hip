// Orthogonalised (Muon) update of banks of weight matrices.
//
//   X = U / max(|U|_F, eps), then per step  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// with X laid so that it has r rows and c >= r columns (a matrix with more rows
// than columns is transposed on the way in and out; the iteration commutes with
// the transposition).  Each step costs 4 r^2 c + 2 r^3 operations per matrix.
//
// Products run on v_mfma_f32_32x32x16_f16 at fp32 accuracy: every operand is
// hi + lo, two fp16 values of 11 bits each, and a product is hi hi' + hi lo' +
// lo hi' (the dropped lo lo' and the rounding of lo are below 2^-22 of the
// operands' magnitudes, and what X, A and B can reach is known: |X|_2 <= s_t
// with s_0 = 1 and s_{t+1} the largest |a s + b s^3 + c s^5| on [0, s_t]; so
// powers of two fixed by the host per step keep them inside the fp16 range
// with their lo parts normal).  X lives in these two planes between the steps.
#include "device_common.h"
#include "layers.h"
#include "timing.h"

#include <algorithm>
#include <utility>

namespace tpconv {

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTile = 64;            // rows and columns of a block's tile
constexpr int kKC = 64;              // reductions per chunk
constexpr int kLD = kKC + 8;
constexpr int kNormChunk = 8192;     // elements per block of the norm

// What one launch works on: a bank of `count` matrices.
struct Bank {
  MuonUpdate u;
  MuonBlock m;
  int32_t r, c, rp, cp;    // X is r x c (r <= c); padded to multiples of kTile
  int32_t transposed;      // rows > cols: X = U^T
  int32_t chunks;          // blocks per matrix of the norm
  float eps, scale;        // scale: sqrt(max(1, cols / rows))
  int32_t update;          // 0: orthogonalize, 1: optimiser step
  float* norm;             // [count][chunks] sums of squares
  _Float16 *xh, *xl;       // [count][rp][cp]
  _Float16 *th, *tl;       // [count][cp][rp]: X^T
  _Float16 *nh, *nl;       // X^T of the next step (a launch reads one and writes the other)
  _Float16 *ah, *al, *bh, *bl;  // [count][rp][rp]
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ void split2(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// U at element e of the caller's layout; m' (the new momentum) is in place already.
__device__ __forceinline__ float u_at(const Bank& b, int64_t e) {
  if (!b.update) return b.u.u[e];
  const float m = b.u.mom_out[e];
  return b.u.nesterov ? (1.f - b.u.beta) * b.u.grad[e] + b.u.beta * m : m;
}

__global__ __launch_bounds__(kThreads) void muon_norm_kernel(const Bank /*args*/) {
  const Bank& b = *(const Bank*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float tmp[kThreads];
  const int64_t n = (int64_t)b.m.rows * b.m.cols;
  const int64_t base = b.m.offset + (int64_t)blockIdx.y * b.m.stride;
  const int64_t lo = (int64_t)blockIdx.x * kNormChunk, hi = min(n, lo + kNormChunk);
  float q = 0.f;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int64_t e = base + i;
    if (b.update) b.u.mom_out[e] = b.u.beta * b.u.mom[e] + (1.f - b.u.beta) * b.u.grad[e];
    const float v = u_at(b, e);
    q = __builtin_fmaf(v, v, q);
  }
  tmp[threadIdx.x] = q;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if ((int)threadIdx.x < s) tmp[threadIdx.x] += tmp[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) b.norm[(int64_t)blockIdx.y * b.chunks + blockIdx.x] = tmp[0];
}

// X = U / max(|U|, eps) into the planes of X and X^T (zero in the padding).
__global__ __launch_bounds__(kThreads) void muon_init_kernel(const Bank /*args*/, int ex) {
  const Bank& b = *(const Bank*)__builtin_amdgcn_kernarg_segment_ptr();
  float q = 0.f;
  for (int i = 0; i < b.chunks; ++i) q += b.norm[(int64_t)blockIdx.y * b.chunks + i];
  const float inv = 1.f / fmaxf(sqrtf(q), b.eps);
  const int64_t pad = (int64_t)b.rp * b.cp;
  const int64_t base = b.m.offset + (int64_t)blockIdx.y * b.m.stride;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < pad; e += (int64_t)gridDim.x * kThreads) {
    const int i = (int)(e / b.cp), j = (int)(e - (int64_t)i * b.cp);
    float v = 0.f;
    if (i < b.r && j < b.c) {
      const int64_t at = b.transposed ? (int64_t)j * b.m.cols + i : (int64_t)i * b.m.cols + j;
      v = u_at(b, base + at) * inv * pow2(ex);
    }
    _Float16 h, l;
    split2(v, h, l);
    const int64_t x = blockIdx.y * pad + e, t = blockIdx.y * pad + (int64_t)j * b.rp + i;
    b.xh[x] = h;
    b.xl[x] = l;
    b.th[t] = h;
    b.tl[t] = l;
  }
}

enum Phase { kGram, kPoly, kApply, kLast };

// C[i][j] = sum_k P[i][k] Q[j][k] over one 64 x 64 tile, then the phase's epilogue:
//   kGram:  P = Q = X:           A = C
//   kPoly:  P = Q = A (A = A^T): B = b A + c C
//   kApply: P = B, Q = X^T:      X = a X + C, in both layouts
//   kLast:  the same, written out as X or as the updated weights
template <int PHASE>
__global__ __launch_bounds__(kThreads) void muon_gemm_kernel(const Bank /*args*/, MuonStep st, int ex_next) {
  const Bank& b = *(const Bank*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ __align__(16) _Float16 sp[2][kTile][kLD];
  __shared__ __align__(16) _Float16 sq[2][kTile][kLD];
  const int64_t xsize = (int64_t)b.rp * b.cp, asize = (int64_t)b.rp * b.rp, bz = blockIdx.z;
  const int K = PHASE == kGram ? b.cp : b.rp;
  const _Float16* p[2];
  const _Float16* q[2];
  if constexpr (PHASE == kGram) {
    p[0] = q[0] = b.xh + bz * xsize;
    p[1] = q[1] = b.xl + bz * xsize;
  } else if constexpr (PHASE == kPoly) {
    p[0] = q[0] = b.ah + bz * asize;
    p[1] = q[1] = b.al + bz * asize;
  } else {
    p[0] = b.bh + bz * asize;
    p[1] = b.bl + bz * asize;
    q[0] = b.th + bz * xsize;
    q[1] = b.tl + bz * xsize;
  }
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 31, lh = lane >> 5;
  const int mw = (wave >> 1) * 32, nw = (wave & 1) * 32;
  floatx16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kKC) {
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      const int row = pass * 32 + (tid >> 3), kk = (tid & 7) * 8;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        *reinterpret_cast<half8*>(&sp[z][row][kk]) =
            *reinterpret_cast<const half8*>(p[z] + (int64_t)(i0 + row) * K + k0 + kk);
        *reinterpret_cast<half8*>(&sq[z][row][kk]) =
            *reinterpret_cast<const half8*>(q[z] + (int64_t)(j0 + row) * K + k0 + kk);
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kKC / 16; ++s) {
      const int k = 16 * s + 8 * lh;
      const half8 ph = *reinterpret_cast<const half8*>(&sp[0][mw + li][k]);
      const half8 pl = *reinterpret_cast<const half8*>(&sp[1][mw + li][k]);
      const half8 qh = *reinterpret_cast<const half8*>(&sq[0][nw + li][k]);
      const half8 ql = *reinterpret_cast<const half8*>(&sq[1][nw + li][k]);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, ql, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl, qh, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, qh, acc, 0, 0, 0);
    }
    __syncthreads();
  }
  const int j = j0 + nw + li;
#pragma unroll
  for (int rq = 0; rq < 4; ++rq) {
    const int i = i0 + mw + 8 * rq + 4 * lh;  // four consecutive rows of one column
    half4 h4, l4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = acc[4 * rq + e];
      if constexpr (PHASE == kGram || PHASE == kPoly) {
        const int64_t at = bz * asize + (int64_t)(i + e) * b.rp + j;
        _Float16 h, l;
        if constexpr (PHASE == kGram) {
          split2(v * pow2(st.ea - 2 * st.ex), h, l);
          b.ah[at] = h;
          b.al[at] = l;
        } else {
          const float av = ((float)b.ah[at] + (float)b.al[at]) * pow2(-st.ea);
          split2((st.b * av + st.c * (v * pow2(-2 * st.ea))) * pow2(st.eb), h, l);
          b.bh[at] = h;
          b.bl[at] = l;
        }
      } else {
        const int64_t at = bz * xsize + (int64_t)(i + e) * b.cp + j;
        const float x = ((float)b.xh[at] + (float)b.xl[at]) * pow2(-st.ex);
        const float y = st.a * x + v * pow2(-st.ex - st.eb);
        if constexpr (PHASE == kApply) {
          _Float16 h, l;
          split2(y * pow2(ex_next), h, l);
          b.xh[at] = h;
          b.xl[at] = l;
          h4[e] = h;
          l4[e] = l;
        } else if (i + e < b.r && j < b.c) {
          const int64_t o = b.m.offset + bz * b.m.stride +
                            (b.transposed ? (int64_t)j * b.m.cols + i + e : (int64_t)(i + e) * b.m.cols + j);
          if (b.update) {
            const float w = (1.f - b.u.lr * b.u.decay) * b.u.W[o] - b.u.lr * b.scale * y;
            b.u.out[o] = w;
            if (b.u.w_bf16) b.u.w_bf16[o] = __builtin_bit_cast(uint16_t, (__bf16)w);
          } else {
            b.u.out[o] = y;
          }
        }
      }
    }
    if constexpr (PHASE == kApply) {
      const int64_t t = bz * xsize + (int64_t)j * b.rp + i;
      *reinterpret_cast<half4*>(b.nh + t) = h4;
      *reinterpret_cast<half4*>(b.nl + t) = l4;
    }
  }
}

// ---- small matrices: all steps of one matrix in one block of threads ---------------
// Padded shapes RP x CP that fit the registers and the 160 KB of LDS of one CU.
// X stays in fp32 accumulator registers over all steps; LDS holds its planes
// (row-major for X X^T, then transposed for B X) and those of A, later B.  The
// only global traffic is the update's own.

struct SmallBlock {
  int32_t rows, cols;
  int64_t offset, stride;
  int64_t first;  // first matrix of the block in the launch
};

struct SmallArgs {
  MuonUpdate u;
  int32_t update, nsteps, nblocks;
  float eps;
  MuonStep step[kMaxMuonSteps + 1];
  SmallBlock block[kMaxMuonBlocks];
};

template <int RP_, int CP_, int NW_, int TPW_>
struct Small {
  static constexpr int RP = RP_, CP = CP_, NW = NW_, TPW = TPW_;
  static constexpr int RT = RP / 32, CT = CP / 32;
  static constexpr int APW = RT == 4 ? 2 : 1;               // tiles of A per wave
  static constexpr int AW = RT * RT / APW;                  // waves that hold tiles of A
  static constexpr int KS = NW / AW;                        // waves that share the reduction of X X^T
  static constexpr int LX = CP + 8, LT = RP + 8;            // LDS rows, padded by 16 bytes
  static constexpr int kX = RP * LX > CP * LT ? RP * LX : CP * LT;
  static constexpr int kBytes = 2 * (2 * kX + 2 * RP * LT) + (KS - 1) * AW * APW * 1024 * 4;
  static_assert(RT * CT == NW * TPW && AW * KS == NW, "tiles per wave");
  static_assert(kBytes <= 160 * 1024, "LDS");
};

template <int TILES>
__device__ __forceinline__ void mul_tiles(const _Float16* p, int lp, int plane_p, const _Float16* q, int lq, int plane_q,
                                          int k0, int steps, floatx16 (&acc)[TILES]) {
  // p: rows of TILES stacked 32-row tiles, q: rows of one 32-column tile
  const int lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
#pragma unroll 2
  for (int s = 0; s < steps; ++s) {
    const int k = k0 + 16 * s + 8 * h;
    const half8 qh = *reinterpret_cast<const half8*>(q + i * lq + k);
    const half8 ql = *reinterpret_cast<const half8*>(q + plane_q + i * lq + k);
    half8 ph[TILES], pl[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      ph[t] = *reinterpret_cast<const half8*>(p + (32 * t + i) * lp + k);
      pl[t] = *reinterpret_cast<const half8*>(p + plane_p + (32 * t + i) * lp + k);
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[t], ql, acc[t], 0, 0, 0);
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[t], qh, acc[t], 0, 0, 0);
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[t], qh, acc[t], 0, 0, 0);
  }
}

// The tile (rows i0.., columns j0..) of v * 2^e into planes whose rows are the
// tile's columns: four consecutive rows of a column are one 8-byte write.
__device__ __forceinline__ void put_columns(_Float16* s, int ld, int plane, int i0, int j0, const floatx16& v, float f) {
  const int lane = threadIdx.x & 63, j = j0 + (lane & 31), h = lane >> 5;
#pragma unroll
  for (int rq = 0; rq < 4; ++rq) {
    half4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      _Float16 a, b;
      split2(v[4 * rq + e] * f, a, b);
      hi[e] = a;
      lo[e] = b;
    }
    _Float16* at = s + j * ld + i0 + 8 * rq + 4 * h;
    *reinterpret_cast<half4*>(at) = hi;
    *reinterpret_cast<half4*>(at + plane) = lo;
  }
}

// The same into planes whose rows are the tile's rows.
__device__ __forceinline__ void put_rows(_Float16* s, int ld, int plane, int i0, int j0, const floatx16& v, float f) {
  const int lane = threadIdx.x & 63, j = j0 + (lane & 31), h = lane >> 5;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    _Float16 a, b;
    split2(v[r] * f, a, b);
    _Float16* at = s + (i0 + 8 * (r >> 2) + 4 * h + (r & 3)) * ld + j;
    at[0] = a;
    at[plane] = b;
  }
}

template <typename S>
__global__ __launch_bounds__(64 * S::NW) void muon_small_kernel(const SmallArgs /*args*/) {
  const SmallArgs& a = *(const SmallArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ __align__(16) char smem[S::kBytes];
  __shared__ float s_norm[S::NW];
  constexpr int RP = S::RP, RT = S::RT, TPW = S::TPW, APW = S::APW, AW = S::AW, KS = S::KS, LX = S::LX, LT = S::LT;
  constexpr int kXPlane = S::kX, kAPlane = RP * LT;
  _Float16* sx = reinterpret_cast<_Float16*>(smem);
  _Float16* sq = sx + 2 * kXPlane;
  float* sr = reinterpret_cast<float*>(sq + 2 * kAPlane);
  int bi = 0;
  while (bi + 1 < a.nblocks && (int64_t)blockIdx.x >= a.block[bi + 1].first) ++bi;
  const SmallBlock& m = a.block[bi];
  const int64_t base = m.offset + (blockIdx.x - m.first) * m.stride;
  const bool transposed = m.rows > m.cols;
  const int nr = transposed ? m.cols : m.rows, nc = transposed ? m.rows : m.cols;
  const int si = transposed ? 1 : m.cols, sj = transposed ? m.cols : 1;  // X[i][j] is U at i * si + j * sj
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, lj = lane & 31, lh = lane >> 5;

  // X in registers: tile t of the wave covers rows 32 (tile % RT), columns 32 (tile / RT)
  floatx16 x[TPW];
  float q = 0.f;
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tile = wave * TPW + t, i0 = 32 * (tile % RT) + 4 * lh, j = 32 * (tile / RT) + lj;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = i0 + 8 * (r >> 2) + (r & 3);
      float v = 0.f;
      if (i < nr && j < nc) {
        const int64_t e = base + (int64_t)i * si + (int64_t)j * sj;
        if (a.update) {
          const float g = (1.f - a.u.beta) * a.u.grad[e], mo = a.u.beta * a.u.mom[e] + g;
          a.u.mom_out[e] = mo;
          v = a.u.nesterov ? g + a.u.beta * mo : mo;
        } else {
          v = a.u.u[e];
        }
      }
      x[t][r] = v;
      q = __builtin_fmaf(v, v, q);
    }
  }
  for (int d = 32; d > 0; d >>= 1) q += __shfl_xor(q, d);
  if (lane == 0) s_norm[wave] = q;
  __syncthreads();
  q = 0.f;
  for (int w = 0; w < S::NW; ++w) q += s_norm[w];
  const float inv = 1.f / fmaxf(sqrtf(q), a.eps);
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) x[t][r] *= inv;

  for (int k = 0; k < a.nsteps; ++k) {
    const MuonStep st = a.step[k];
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      const int tile = wave * TPW + t;
      put_rows(sx, LX, kXPlane, 32 * (tile % RT), 32 * (tile / RT), x[t], pow2(st.ex));
    }
    __syncthreads();
    // A = X X^T: KS waves per tile group take a part of the columns each
    const int aw = wave % AW, ks = wave / AW;
    const int ai = 32 * ((aw * APW) % RT), aj = 32 * ((aw * APW) / RT);
    floatx16 acc[APW];
#pragma unroll
    for (int t = 0; t < APW; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
    mul_tiles<APW>(sx + ai * LX, LX, kXPlane, sx + aj * LX, LX, kXPlane, ks * (S::CP / KS), S::CP / (16 * KS), acc);
    if constexpr (KS > 1) {
      if (ks > 0)
#pragma unroll
        for (int r = 0; r < 16; ++r) sr[((ks - 1) * AW + aw) * 1024 + r * 64 + lane] = acc[0][r];
    }
    __syncthreads();
    const float fa = pow2(-2 * st.ex);
    if (ks == 0) {
#pragma unroll
      for (int t = 0; t < APW; ++t) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if constexpr (KS > 1)
            for (int w = 0; w < KS - 1; ++w) acc[t][r] += sr[(w * AW + aw) * 1024 + r * 64 + lane];
          acc[t][r] *= fa;
        }
        put_columns(sq, LT, kAPlane, ai + 32 * t, aj, acc[t], pow2(st.ea));  // A is symmetric
      }
    }
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      const int tile = wave * TPW + t;
      put_columns(sx, LT, kXPlane, 32 * (tile % RT), 32 * (tile / RT), x[t], pow2(st.ex));  // X^T
    }
    __syncthreads();
    // B = b A + c A A, over A
    floatx16 sqr[APW];
    if (ks == 0) {
#pragma unroll
      for (int t = 0; t < APW; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) sqr[t][r] = 0.f;
      mul_tiles<APW>(sq + ai * LT, LT, kAPlane, sq + aj * LT, LT, kAPlane, 0, RP / 16, sqr);
    }
    __syncthreads();
    if (ks == 0) {
      const float fc = st.c * pow2(-2 * st.ea);
#pragma unroll
      for (int t = 0; t < APW; ++t) {
#pragma unroll
        for (int r = 0; r < 16; ++r) sqr[t][r] = st.b * acc[t][r] + fc * sqr[t][r];
        put_columns(sq, LT, kAPlane, ai + 32 * t, aj, sqr[t], pow2(st.eb));
      }
    }
    __syncthreads();
    // X <- a X + B X, the wave's own tiles (all in one column of tiles, or single)
    const float fx = pow2(-st.ex - st.eb);
    if constexpr (RT > 1 || TPW == 1) {
      floatx16 bx[TPW];
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) bx[t][r] = 0.f;
      const int tile = wave * TPW;
      mul_tiles<TPW>(sq + 32 * (tile % RT) * LT, LT, kAPlane, sx + 32 * (tile / RT) * LT, LT, kXPlane, 0, RP / 16, bx);
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[t][r] = st.a * x[t][r] + fx * bx[t][r];
    } else {
#pragma unroll
      for (int t = 0; t < TPW; ++t) {
        floatx16 bx[1];
#pragma unroll
        for (int r = 0; r < 16; ++r) bx[0][r] = 0.f;
        mul_tiles<1>(sq, LT, kAPlane, sx + 32 * (wave * TPW + t) * LT, LT, kXPlane, 0, RP / 16, bx);
#pragma unroll
        for (int r = 0; r < 16; ++r) x[t][r] = st.a * x[t][r] + fx * bx[0][r];
      }
    }
    __syncthreads();
  }

  const float keep = 1.f - a.u.lr * a.u.decay;
  const float rate = a.u.lr * (m.cols > m.rows ? sqrtf((float)m.cols / (float)m.rows) : 1.f);
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tile = wave * TPW + t, i0 = 32 * (tile % RT) + 4 * lh, j = 32 * (tile / RT) + lj;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = i0 + 8 * (r >> 2) + (r & 3);
      if (i >= nr || j >= nc) continue;
      const int64_t e = base + (int64_t)i * si + (int64_t)j * sj;
      float v = x[t][r];
      if (a.update) {
        v = keep * a.u.W[e] - rate * v;
        if (a.u.w_bf16) a.u.w_bf16[e] = __builtin_bit_cast(uint16_t, (__bf16)v);
      }
      a.u.out[e] = v;
    }
  }
}

// The padded shapes, by rows then columns.
enum SmallKind { kS32x32, kS32x64, kS32x128, kS32x256, kS32x512, kS64x64, kS64x128, kS64x256, kS128x128, kSmallKinds };

// The smallest padded shape of an r x c matrix (r <= c); -1: none, the matrix takes the tiled path.
int small_kind(int r, int c) {
  if (r <= 32) return c <= 32 ? kS32x32 : c <= 64 ? kS32x64 : c <= 128 ? kS32x128 : c <= 256 ? kS32x256 : c <= 512 ? kS32x512 : -1;
  if (r <= 64) return c <= 64 ? kS64x64 : c <= 128 ? kS64x128 : c <= 256 ? kS64x256 : -1;
  return r <= 128 && c <= 128 ? kS128x128 : -1;
}
int small_kind(const MuonBlock& b) {
  return b.rows < b.cols ? small_kind(b.rows, b.cols) : small_kind(b.cols, b.rows);
}

template <typename S>
hipError_t launch_small(const SmallArgs& k, int64_t matrices, hipStream_t s) {
  hipLaunchKernelGGL((muon_small_kernel<S>), dim3((unsigned)matrices), dim3(64 * S::NW), 0, s, k);
  return hipGetLastError();
}

hipError_t launch_small_kinds(const MuonPlan& p, const MuonUpdate& u, hipStream_t s) {
  for (int kind = 0; kind < kSmallKinds; ++kind) {
    SmallArgs k{};
    int64_t n = 0;
    for (int i = 0; i < p.nblocks; ++i) {
      const MuonBlock& b = p.block[i];
      if (b.count == 0 || small_kind(b) != kind) continue;
      k.block[k.nblocks++] = {b.rows, b.cols, b.offset, b.stride, n};
      n += b.count;
    }
    if (n == 0) continue;
    k.u = u;
    k.update = u.W != nullptr;
    k.nsteps = p.nsteps;
    k.eps = p.eps;
    std::copy(p.step, p.step + kMaxMuonSteps + 1, k.step);
    hipError_t e = hipSuccess;
    switch (kind) {
      case kS32x32: e = launch_small<Small<32, 32, 1, 1>>(k, n, s); break;
      case kS32x64: e = launch_small<Small<32, 64, 2, 1>>(k, n, s); break;
      case kS32x128: e = launch_small<Small<32, 128, 4, 1>>(k, n, s); break;
      case kS32x256: e = launch_small<Small<32, 256, 8, 1>>(k, n, s); break;
      case kS32x512: e = launch_small<Small<32, 512, 8, 2>>(k, n, s); break;
      case kS64x64: e = launch_small<Small<64, 64, 4, 1>>(k, n, s); break;
      case kS64x128: e = launch_small<Small<64, 128, 8, 1>>(k, n, s); break;
      case kS64x256: e = launch_small<Small<64, 256, 8, 2>>(k, n, s); break;
      default: e = launch_small<Small<128, 128, 8, 2>>(k, n, s); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t align_up(size_t b) { return (b + 255) / 256 * 256; }

void set_bank(const MuonPlan& p, int i, Bank& b) {
  b.m = p.block[i];
  b.transposed = b.m.rows > b.m.cols;
  b.r = b.transposed ? b.m.cols : b.m.rows;
  b.c = b.transposed ? b.m.rows : b.m.cols;
  b.rp = (b.r + kTile - 1) / kTile * kTile;
  b.cp = (b.c + kTile - 1) / kTile * kTile;
  b.chunks = (int32_t)(((int64_t)b.m.rows * b.m.cols + kNormChunk - 1) / kNormChunk);
  b.eps = p.eps;
  b.scale = b.m.cols > b.m.rows ? sqrtf((float)b.m.cols / (float)b.m.rows) : 1.f;
}

// X in two planes, X^T in two buffers of two planes, A and B.
size_t bank_bytes(const Bank& b) {
  const size_t x = (size_t)b.m.count * b.rp * b.cp * 2, a = (size_t)b.m.count * b.rp * b.rp * 2;
  return align_up((size_t)b.m.count * b.chunks * 4) + align_up(6 * x) + align_up(4 * a);
}

}  // namespace

size_t muon_workspace(const MuonPlan& p) {
  size_t most = 0;
  for (int i = 0; i < p.nblocks; ++i) {
    Bank b{};
    set_bank(p, i, b);
    const size_t n = b.m.count > 0 && small_kind(b.m) < 0 ? bank_bytes(b) : 0;
    most = n > most ? n : most;
  }
  return most;  // the blocks run one after the other in the same workspace
}

hipError_t launch_muon(const MuonPlan& p, const MuonUpdate& u, void* ws, hipStream_t s) {
  TimingScope ts(kcMuon, s);
  const hipError_t e = launch_small_kinds(p, u, s);
  if (e != hipSuccess) return e;
  for (int i = 0; i < p.nblocks; ++i) {
    Bank b{};
    set_bank(p, i, b);
    if (b.m.count == 0 || small_kind(b.m) >= 0) continue;
    b.u = u;
    b.update = u.W != nullptr;
    const size_t x = (size_t)b.m.count * b.rp * b.cp, a = (size_t)b.m.count * b.rp * b.rp;
    b.norm = static_cast<float*>(ws);
    _Float16* h = reinterpret_cast<_Float16*>(static_cast<char*>(ws) + align_up((size_t)b.m.count * b.chunks * 4));
    b.xh = h;
    b.xl = h + x;
    b.th = h + 2 * x;
    b.tl = h + 3 * x;
    b.nh = h + 4 * x;
    b.nl = h + 5 * x;
    b.ah = reinterpret_cast<_Float16*>(reinterpret_cast<char*>(h) + align_up(12 * x));
    b.al = b.ah + a;
    b.bh = b.ah + 2 * a;
    b.bl = b.ah + 3 * a;
    const unsigned n = (unsigned)b.m.count, R = b.rp / kTile, C = b.cp / kTile;
    hipLaunchKernelGGL(muon_norm_kernel, dim3(b.chunks, n), dim3(kThreads), 0, s, b);
    const int64_t pad = (int64_t)b.rp * b.cp;
    hipLaunchKernelGGL(muon_init_kernel, dim3((unsigned)((pad + 4 * kThreads - 1) / (4 * kThreads)), n), dim3(kThreads),
                       0, s, b, p.step[0].ex);
    for (int k = 0; k < p.nsteps; ++k) {
      const MuonStep& st = p.step[k];
      hipLaunchKernelGGL((muon_gemm_kernel<kGram>), dim3(R, R, n), dim3(kThreads), 0, s, b, st, 0);
      hipLaunchKernelGGL((muon_gemm_kernel<kPoly>), dim3(R, R, n), dim3(kThreads), 0, s, b, st, 0);
      if (k + 1 < p.nsteps)
        hipLaunchKernelGGL((muon_gemm_kernel<kApply>), dim3(C, R, n), dim3(kThreads), 0, s, b, st, p.step[k + 1].ex);
      else
        hipLaunchKernelGGL((muon_gemm_kernel<kLast>), dim3(C, R, n), dim3(kThreads), 0, s, b, st, 0);
      std::swap(b.th, b.nh);
      std::swap(b.tl, b.nl);
    }
  }
  return hipGetLastError();
}

}  // namespace tpconv
