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
// with their lo parts normal).
//
// Matrices up to 128 x 128 (or 64 x 256, 32 x 512) run all their steps in one
// block of threads; larger ones run one launch per product (norm, init, then
// three per step), with X, X^T, A and B as hi and lo planes in the workspace.
//
// Measured (traced kernels, five steps, one set of inputs): 88 matrices of 32 x
// 32 9.0 us, 184 of 64 x 64 17.5 and 176 of 128 x 128 46 to 49 (40 a call in a
// row of calls): one block per CU, each a chain of 15 dependent products through
// LDS, bound by that latency and, at 64 and 128, by four LDS reads for three
// products; the matrix cores see 11 GFLOP x 3 = 0.7 PFLOP/s at 128.  Two of 1024 x
// 2048: X X^T 34 us (half of it: 13.7 GFLOP of fp16 products), A A 22, B X 36 (25.8
// GFLOP, 0.72 PFLOP/s), the last B X with the update 44, init 18, norm 11.
// There 272 blocks share 256 CUs in the r x r products: the doubled-up CUs set
// the time (256 blocks of the same size take 60% of it); cutting the reduction
// into equal parts instead gave 25 + 8 us (the join) and 18 + 8 where X X^T took
// 39 and A A 25, no gain.
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
constexpr int kKC = 64;              // reductions per chunk of the tiled products
constexpr int kLD = kKC + 8;         // LDS rows padded by 16 bytes
// Rows of the planes in memory are 128 bytes longer than the padded matrix: at
// a power-of-two row length one chunk of all rows of a tile lies in the same
// L2 channels.
constexpr int kSkew = 64;
constexpr int kNormChunk = 4096;     // elements per block of the norm

// What one launch works on: a bank of `count` matrices.
struct Bank {
  MuonUpdate u;
  MuonBlock m;
  int32_t r, c, rp, cp;    // X is r x c (r <= c); padded to multiples of the larger tile
  int32_t rl, cl;          // row lengths of the planes (rp and cp, and kSkew)
  int32_t square_tile, apply_tile;  // tile widths of the r x r products and of B X
  int32_t transposed;      // rows > cols: X = U^T
  int32_t chunks;          // blocks per matrix of the norm
  float eps, scale;        // scale: sqrt(max(1, cols / rows))
  int32_t update;          // 0: orthogonalize, 1: optimiser step
  float2* norm;            // [count][chunks] sums of squares (Squares)
  int64_t xsize, tsize, asize;  // halfs per matrix of the planes of X, X^T, and A or B
  _Float16 *xh, *xl;       // [count][rp][cl]
  _Float16 *th, *tl;       // [count][cp][rl]: X^T
  _Float16 *nh, *nl;       // X^T of the next step (a launch reads one and writes the other)
  _Float16 *ah, *al, *bh, *bl;  // [count][rp][rl]
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

// |U|^2 as s 4^e.  e is 0 where the plain sum is in range (`plain_sum`); else the values are taken
// times 2^-e, with e the exponent of the largest of them, so that any finite matrix has its norm:
// X = (U 2^-e) / max(sqrt(s), eps 2^-e).
constexpr int kLeastExponent = -100;  // of the smallest value, 2^-149, the square still has room at 2^(2 (100 - 149))
struct Squares {
  float s;
  int e;
};
__device__ __forceinline__ Squares add(const Squares& a, const Squares& b) {
  const int e = max(a.e, b.e);
  return {ldexpf(a.s, 2 * (a.e - e)) + ldexpf(b.s, 2 * (b.e - e)), e};
}
// Neither overflown (of up to 2^18 such sums either) nor made of squares that underflow, unless eps decides anyway.
__device__ __forceinline__ bool plain_sum(float s, float eps) {
  return s <= 0x1p100f && (s >= 0x1p-90f || eps >= 0x1p-44f);
}
__device__ __forceinline__ int scale_exponent(float largest) {
  return largest > 0.f ? max(__builtin_amdgcn_frexp_expf(largest) - 1, kLeastExponent) : kLeastExponent;
}

__global__ __launch_bounds__(kThreads) void muon_norm_kernel(const Bank /*args*/) {
  const Bank& b = *(const Bank*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float tmp[kThreads];
  const int64_t n = (int64_t)b.m.rows * b.m.cols;
  const int64_t base = b.m.offset + (int64_t)blockIdx.y * b.m.stride;
  const int64_t lo = (int64_t)blockIdx.x * kNormChunk, hi = min(n, lo + kNormChunk);
  float q = 0.f;
  for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += 4 * kThreads) {
    float g[4], m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // every load of the round is in flight at once; past the end the last element again
      const int64_t e = base + min(i0 + k * kThreads, hi - 1);
      g[k] = b.update ? b.u.grad[e] : b.u.u[e];
      m[k] = b.update ? b.u.mom[e] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + k * kThreads;
      if (i >= hi) break;
      float v = g[k];
      if (b.update) {
        const float mo = b.u.beta * m[k] + (1.f - b.u.beta) * g[k];
        b.u.mom_out[base + i] = mo;
        v = b.u.nesterov ? (1.f - b.u.beta) * g[k] + b.u.beta * mo : mo;
      }
      q = __builtin_fmaf(v, v, q);
    }
  }
  auto reduce = [&](float v, auto join) {  // over the block, the result in every thread
    tmp[threadIdx.x] = v;
    __syncthreads();
    for (int s = kThreads / 2; s > 0; s >>= 1) {
      if ((int)threadIdx.x < s) tmp[threadIdx.x] = join(tmp[threadIdx.x], tmp[threadIdx.x + s]);
      __syncthreads();
    }
    v = tmp[0];
    __syncthreads();
    return v;
  };
  auto sum = [](float x, float y) { return x + y; };
  Squares all = {reduce(q, sum), 0};
  if (!plain_sum(all.s, b.eps)) {  // (uniform over the block; every thread reads the elements that it wrote)
    float largest = 0.f;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) largest = fmaxf(largest, fabsf(u_at(b, base + i)));
    all.e = scale_exponent(reduce(largest, [](float x, float y) { return fmaxf(x, y); }));
    q = 0.f;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const float v = ldexpf(u_at(b, base + i), -all.e);
      q = __builtin_fmaf(v, v, q);
    }
    all.s = reduce(q, sum);
  }
  if (threadIdx.x == 0) b.norm[(int64_t)blockIdx.y * b.chunks + blockIdx.x] = {all.s, __int_as_float(all.e)};
}

// X = U / max(|U|, eps) into the planes of X and X^T (zero in the padding), by
// 64 x 64 tiles turned through LDS so that reads and writes run along rows.
__global__ __launch_bounds__(kThreads) void muon_init_kernel(const Bank /*args*/, int ex) {
  const Bank& b = *(const Bank*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ float tile[64][65];
  __shared__ Squares tmp[kThreads];
  const int64_t bz = blockIdx.z;
  Squares q = {0.f, kLeastExponent};
  for (int i = threadIdx.x; i < b.chunks; i += kThreads) {
    const float2 n = b.norm[bz * b.chunks + i];
    q = add(q, {n.x, __float_as_int(n.y)});
  }
  tmp[threadIdx.x] = q;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if ((int)threadIdx.x < s) tmp[threadIdx.x] = add(tmp[threadIdx.x], tmp[threadIdx.x + s]);
    __syncthreads();
  }
  q = tmp[0];
  const float f = pow2(ex) / fmaxf(sqrtf(q.s), ldexpf(b.eps, -q.e));
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t base = b.m.offset + bz * b.m.stride;
  // rows of U: rows of X, or its columns when X = U^T
  const int u0 = b.transposed ? j0 : i0, v0 = b.transposed ? i0 : j0;
  for (int k = w; k < 64; k += 4) {
    float v = 0.f;
    if (u0 + k < b.m.rows && v0 + lane < b.m.cols)
      v = ldexpf(u_at(b, base + (int64_t)(u0 + k) * b.m.cols + v0 + lane), -q.e) * f;
    tile[k][lane] = v;
  }
  __syncthreads();
  for (int k = w; k < 64; k += 4) {
    _Float16 h, l;
    split2(b.transposed ? tile[lane][k] : tile[k][lane], h, l);
    const int64_t x = bz * b.xsize + (int64_t)(i0 + k) * b.cl + j0 + lane;
    b.xh[x] = h;
    b.xl[x] = l;
    split2(b.transposed ? tile[k][lane] : tile[lane][k], h, l);
    const int64_t t = bz * b.tsize + (int64_t)(j0 + k) * b.rl + i0 + lane;
    b.th[t] = h;
    b.tl[t] = l;
  }
}

enum Phase { kGram, kPoly, kApply, kLast };

constexpr int kGemmThreads = 512;

// C[i][j] = sum_k P[i][k] Q[j][k] over one T x T tile, then the phase's epilogue:
//   kGram:  P = Q = X:           A = C
//   kPoly:  P = Q = A (A = A^T): B = b A + c C
//   kApply: P = B, Q = X^T:      X = a X + C, in both layouts
//   kLast:  the same, written out as X or as the updated weights
// A and B are symmetric: only tiles on and below the diagonal are computed, and
// the others written as their mirror images.  Eight waves: T = 128 gives each
// 64 x 32 (six LDS reads for six products); T = 64 one of four 32 x 32 tiles
// and half of every chunk of the reduction (few blocks, so more waves per block).
// Chunks go through two LDS buffers, with the loads of the next two in flight.
// The results pass through LDS as well, so that every plane is read and written
// in 16-byte pieces of its rows.
template <int PHASE, int T>
__global__ __launch_bounds__(kGemmThreads) void muon_gemm_kernel(const Bank /*args*/, MuonStep st, int ex_next, int tiles) {
  const Bank& b = *(const Bank*)__builtin_amdgcn_kernarg_segment_ptr();
  constexpr int MT = T == 128 ? 2 : 1, KS = T == 128 ? 1 : 2;
  constexpr int kPlane = T * kLD, kOp = 2 * kPlane, kBuf = 2 * kOp;  // halfs
  constexpr int kUnits = T * (kKC / 8) / kGemmThreads;               // 16-byte units per thread, plane and operand
  __shared__ __align__(16) _Float16 smem[2 * kBuf];
  const int K = PHASE == kGram ? b.cp : b.rp, ldk = PHASE == kGram ? b.cl : b.rl;
  // consecutive tiles run on one XCD and share the operands' rows in its L2
  const int64_t item = xcd_item(blockIdx.x, gridDim.x);
  if (item >= tiles * b.m.count) return;
  const int64_t bz = item / tiles;
  const int tile = (int)(item - bz * tiles);
  int i0, j0;
  if constexpr (PHASE == kGram || PHASE == kPoly) {
    int t = tile, ti = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    while (ti * (ti + 1) / 2 > t) --ti;
    i0 = ti * T;
    j0 = (t - ti * (ti + 1) / 2) * T;
  } else {
    const int rt = b.rp / T;
    j0 = tile / rt * T;
    i0 = tile % rt * T;
  }
  const _Float16* src[4];  // P hi, P lo, Q hi, Q lo
  if constexpr (PHASE == kGram) {
    src[0] = src[2] = b.xh + bz * b.xsize;
    src[1] = src[3] = b.xl + bz * b.xsize;
  } else if constexpr (PHASE == kPoly) {
    src[0] = src[2] = b.ah + bz * b.asize;
    src[1] = src[3] = b.al + bz * b.asize;
  } else {
    src[0] = b.bh + bz * b.asize;
    src[1] = b.bl + bz * b.asize;
    src[2] = b.th + bz * b.tsize;
    src[3] = b.tl + bz * b.tsize;
  }
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 31, lh = lane >> 5;
  const int srow = tid >> 3, sk = (tid & 7) * 8;  // this thread's 16 bytes of a row
#pragma unroll
  for (int z = 0; z < 4; ++z) src[z] += (int64_t)((z < 2 ? i0 : j0) + srow) * ldk + sk;
  constexpr int kAhead = 2;
  half8 raw[kAhead][4][kUnits];
  auto load = [&](int d, int k0) {
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        raw[d][z][u] = *reinterpret_cast<const half8*>(src[z] + (int64_t)u * (kGemmThreads / 8) * ldk + k0);
  };
  auto put = [&](int d, int buf) {
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        *reinterpret_cast<half8*>(smem + buf * kBuf + z * kPlane + (srow + u * (kGemmThreads / 8)) * kLD + sk) =
            raw[d][z][u];
  };
  const int mw = T == 128 ? (wave >> 2) * 64 : ((wave >> 1) & 1) * 32;
  const int nw = T == 128 ? (wave & 3) * 32 : (wave & 1) * 32;
  const int kw = KS == 2 ? (wave >> 2) * (kKC / 2) : 0;
  floatx16 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
  const int chunks = K / kKC;
  load(0, 0);
  put(0, 0);
#pragma unroll
  for (int d = 1; d <= kAhead; ++d) load(d % kAhead, min(d, chunks - 1) * kKC);
  __syncthreads();
  for (int c0 = 0; c0 < chunks; c0 += 2) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int c = c0 + d;
      if (c >= chunks) break;
      const int buf = d, slot = (d + 1) % kAhead;
      const _Float16* p = smem + buf * kBuf + (mw + li) * kLD + kw + 8 * lh;
      const _Float16* q = smem + buf * kBuf + kOp + (nw + li) * kLD + kw + 8 * lh;
#pragma unroll
      for (int s = 0; s < kKC / (16 * KS); ++s) {
        half8 ph[MT], pl[MT];
        const half8 qh = *reinterpret_cast<const half8*>(q + 16 * s);
        const half8 ql = *reinterpret_cast<const half8*>(q + kPlane + 16 * s);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          ph[t] = *reinterpret_cast<const half8*>(p + 32 * t * kLD + 16 * s);
          pl[t] = *reinterpret_cast<const half8*>(p + kPlane + 32 * t * kLD + 16 * s);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[t], ql, acc[t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[t], qh, acc[t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[t], qh, acc[t], 0, 0, 0);
      }
      put(slot, buf ^ 1);
      __builtin_amdgcn_sched_barrier(0);
      load(slot, min(c + 1 + kAhead, chunks - 1) * kKC);  // (past the end: the last chunk again, not used)
      __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the next products
      __syncthreads();
    }
  }
  // KS = 2: the waves of one tile exchange halves of their sums, so each
  // finishes eight of the sixteen rows of registers
  if constexpr (KS == 2) {
    float* part = reinterpret_cast<float*>(smem) + (wave & 3) * 1024 + lane;
    const int mine = (wave >> 2) * 8;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float other = mine ? acc[0][r] : acc[0][8 + r];
      part[64 * (8 - mine + r)] = other;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 8; ++r) acc[0][r] = (mine ? acc[0][8 + r] : acc[0][r]) + part[64 * (mine + r)];
    __syncthreads();
  }
  // Two LDS tiles of two planes: `cols` holds the tile by columns (rows of X^T,
  // or of the symmetric A and B), `rows` by rows.
  constexpr int kOut = T + 8, kTilePlane = T * kOut, kPieces = T * T / 8 / kGemmThreads;
  _Float16* cols = smem;
  _Float16* rows = smem + 2 * kTilePlane;
  const int64_t col_at = bz * (PHASE == kGram || PHASE == kPoly ? b.asize : b.tsize) + (int64_t)j0 * b.rl + i0;
  auto piece = [&](int u, int& row, int& k) {
    const int n = tid + u * kGemmThreads;
    row = n / (T / 8);
    k = (n % (T / 8)) * 8;
  };
  if constexpr (PHASE != kGram) {  // the old tile: A of kPoly, X of the others
    const _Float16* from[2] = {(PHASE == kPoly ? b.ah : b.th) + col_at, (PHASE == kPoly ? b.al : b.tl) + col_at};
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        int row, k;
        piece(u, row, k);
        *reinterpret_cast<half8*>(cols + z * kTilePlane + row * kOut + k) =
            *reinterpret_cast<const half8*>(from[z] + (int64_t)row * b.rl + k);
      }
    __syncthreads();
  }
  const int lj = nw + li, first = KS == 2 ? (wave >> 2) * 2 : 0;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int rq = 0; rq < 4 / KS; ++rq) {
      const int i = mw + 32 * t + 8 * (rq + first) + 4 * lh;  // four consecutive rows of one column of the tile
      _Float16* at = cols + lj * kOut + i;
      half4 oh = {0, 0, 0, 0}, ol = {0, 0, 0, 0}, h4, l4;
      if constexpr (PHASE != kGram) {
        oh = *reinterpret_cast<const half4*>(at);
        ol = *reinterpret_cast<const half4*>(at + kTilePlane);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float old = (float)oh[e] + (float)ol[e], c = acc[t][4 * rq + e];
        float v;
        if constexpr (PHASE == kGram)
          v = c * pow2(st.ea - 2 * st.ex);
        else if constexpr (PHASE == kPoly)
          v = (st.b * (old * pow2(-st.ea)) + st.c * (c * pow2(-2 * st.ea))) * pow2(st.eb);
        else
          v = st.a * (old * pow2(-st.ex)) + c * pow2(-st.ex - st.eb);
        if constexpr (PHASE == kLast) {
          const int gi = i0 + i + e, gj = j0 + lj;
          if (gi < b.r && gj < b.c) {
            const int64_t o = b.m.offset + bz * b.m.stride +
                              (b.transposed ? (int64_t)gj * b.m.cols + gi : (int64_t)gi * b.m.cols + gj);
            if (b.update) {
              v = (1.f - b.u.lr * b.u.decay) * b.u.W[o] - b.u.lr * b.scale * v;
              if (b.u.w_bf16) b.u.w_bf16[o] = __builtin_bit_cast(uint16_t, (__bf16)v);
            }
            b.u.out[o] = v;
          }
        } else {
          _Float16 h, l;
          split2(PHASE == kApply ? v * pow2(ex_next) : v, h, l);
          h4[e] = h;
          l4[e] = l;
          rows[(i + e) * kOut + lj] = h;
          rows[kTilePlane + (i + e) * kOut + lj] = l;
        }
      }
      if constexpr (PHASE != kLast) {
        *reinterpret_cast<half4*>(at) = h4;
        *reinterpret_cast<half4*>(at + kTilePlane) = l4;
      }
    }
  if constexpr (PHASE != kLast) {
    __syncthreads();
    _Float16* to[2] = {(PHASE == kGram ? b.ah : PHASE == kPoly ? b.bh : b.nh) + col_at,
                       (PHASE == kGram ? b.al : PHASE == kPoly ? b.bl : b.nl) + col_at};
    const int ld = PHASE == kApply ? b.cl : b.rl;
    const int64_t row_at = bz * (PHASE == kApply ? b.xsize : b.asize) + (int64_t)i0 * ld + j0;
    _Float16* mirror[2] = {(PHASE == kGram ? b.ah : PHASE == kPoly ? b.bh : b.xh) + row_at,
                           (PHASE == kGram ? b.al : PHASE == kPoly ? b.bl : b.xl) + row_at};
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        int row, k;
        piece(u, row, k);
        *reinterpret_cast<half8*>(to[z] + (int64_t)row * b.rl + k) =
            *reinterpret_cast<const half8*>(cols + z * kTilePlane + row * kOut + k);
        if (PHASE == kApply || i0 != j0)
          *reinterpret_cast<half8*>(mirror[z] + (int64_t)row * ld + k) =
              *reinterpret_cast<const half8*>(rows + z * kTilePlane + row * kOut + k);
      }
  }
}

// ---- small matrices: all steps of one matrix in one block of threads ---------------
// Padded shapes RP x CP that fit the registers and the 160 KB of LDS of one CU.
// X stays in fp32 accumulator registers over all steps; LDS holds the planes of
// X^T (read along rows for B X, turned on the way for X X^T) and those of A,
// later B.  The only global traffic is the update's own.

struct SmallBlock {
  int32_t rows, cols;
  int64_t offset, stride;
  int64_t first;  // first matrix of the block in the launch
};

struct SmallArgs {
  MuonUpdate u;
  int32_t update, nsteps, nblocks;
  float eps;
  MuonStep step[kMaxMuonSteps];
  SmallBlock block[kMaxMuonBlocks];
};

// Tiles of T x T: 32 (v_mfma_f32_32x32x16_f16), or 16 (16x16x32) where a matrix
// has so few tiles that more, smaller ones are needed to keep the SIMDs busy.
template <int RP_, int CP_, int T_, int NW_, int TPW_>
struct Small {
  static constexpr int RP = RP_, CP = CP_, T = T_, NW = NW_, TPW = TPW_;
  static constexpr int RT = RP / T, CT = CP / T;
  static constexpr int APW = RT * RT > NW ? RT * RT / NW : 1;  // tiles of A per wave
  static constexpr int AW = RT * RT / APW;                     // waves that hold tiles of A
  static constexpr int KS = NW / AW;                           // waves that share the reduction of X X^T
  static constexpr int kStep = T == 32 ? 16 : 32;              // reductions of one product
  // LDS rows of X^T and of A: paddings that keep both the 16-byte reads of 16
  // rows and the transposing reads of 4 rows x 32 bytes free of bank conflicts
  static constexpr int LT = RP == 128 ? 152 : RP == 64 ? 72 : 56;
  static constexpr int LA = RP + 8;
  static constexpr int kX = CP * LT, kA = RP * LA;
  static constexpr int kBytes = 2 * 2 * (kX + kA) + (KS - 1) * AW * APW * T * T * 4;
  static_assert(RT * CT == NW * TPW && AW * KS == NW && CP % (KS * kStep) == 0, "tiles per wave");
  static_assert(kBytes <= 160 * 1024, "LDS");
};

template <int T>
struct Acc;
template <>
struct Acc<32> {
  typedef floatx16 type;
  static constexpr int regs = 16;
  static __device__ __forceinline__ floatx16 mul(half8 a, half8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Acc<16> {
  typedef float type __attribute__((ext_vector_type(4)));
  static constexpr int regs = 4;
  static __device__ __forceinline__ type mul(half8 a, half8 b, type c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
// Row of accumulator register r within a tile (columns run along the lanes).
template <int T>
__device__ __forceinline__ int tile_row(int r) {
  const int lane = threadIdx.x & 63;
  return T == 32 ? 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3) : 4 * (lane >> 4) + r;
}

// An operand's run of eight reductions from rows of the reduction: row i of the tile at s.
template <int T>
__device__ __forceinline__ half8 run_of_rows(const _Float16* s, int ld, int k) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const half8*>(s + (lane & (T - 1)) * ld + k + 8 * (lane / T));
}
// The same from the transposed matrix (its rows are the reductions), by LDS
// reads that turn 4 x 16 blocks: in each group of 16 lanes, lane l supplies the
// address of four values of row l / 4 and receives column l of the four rows.
template <int T>
__device__ __forceinline__ half8 run_of_columns(const _Float16* s, int ld, int i0, int k) {
  typedef __fp16 fp16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) fp16x4* lds_ptr;
  const int lane = threadIdx.x & 63, l = lane & 15;
  const int row = k + 8 * (lane / T) + (l >> 2), col = i0 + (T == 32 ? 16 * ((lane >> 4) & 1) : 0) + 4 * (l & 3);
  const _Float16* p = s + row * ld + col;
  const fp16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_ptr)p);
  const fp16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_ptr)(p + 4 * ld));
  const half4 x = __builtin_bit_cast(half4, a), y = __builtin_bit_cast(half4, b);
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

// acc[t] += P Q^T for TILES stacked tiles of P's rows from row i0 and one tile
// of Q's rows from row j0, over `steps` products from reduction k0.
// COLS: the planes hold the transposed operands.
template <int T, int TILES, bool COLS>
__device__ __forceinline__ void mul_tiles(const _Float16* p, int lp, int plane_p, int i0, const _Float16* q, int lq,
                                          int plane_q, int j0, int k0, int steps, typename Acc<T>::type (&acc)[TILES]) {
  constexpr int kStep = T == 32 ? 16 : 32;
  auto get = [&](const _Float16* s, int ld, int row, int k) {
    if constexpr (COLS)
      return run_of_columns<T>(s, ld, row, k);
    else
      return run_of_rows<T>(s + row * ld, ld, k);
  };
#pragma unroll  // (176 x 128 x 128: 51.8 us by two, 47.7 in full)
  for (int s = 0; s < steps; ++s) {
    const int k = k0 + kStep * s;
    const half8 qh = get(q, lq, j0, k), ql = get(q + plane_q, lq, j0, k);
    half8 ph[TILES], pl[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      ph[t] = get(p, lp, i0 + T * t, k);
      pl[t] = get(p + plane_p, lp, i0 + T * t, k);
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = Acc<T>::mul(ph[t], ql, acc[t]);
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = Acc<T>::mul(pl[t], qh, acc[t]);
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = Acc<T>::mul(ph[t], qh, acc[t]);
  }
}

// The tile (rows i0.., columns j0..) of v f into planes whose rows are the
// tile's columns: four consecutive rows of a column are one 8-byte write.
template <int T>
__device__ __forceinline__ void put_columns(_Float16* s, int ld, int plane, int i0, int j0,
                                            const typename Acc<T>::type& v, float f) {
  typedef float floatx4 __attribute__((ext_vector_type(4)));
  const int j = j0 + (threadIdx.x & (T - 1));
#pragma unroll
  for (int q = 0; q < Acc<T>::regs / 4; ++q) {
    const floatx4 x = {v[4 * q] * f, v[4 * q + 1] * f, v[4 * q + 2] * f, v[4 * q + 3] * f};
    const half4 hi = __builtin_convertvector(x, half4);
    const half4 lo = __builtin_convertvector(x - __builtin_convertvector(hi, floatx4), half4);
    _Float16* at = s + j * ld + i0 + tile_row<T>(4 * q);
    *reinterpret_cast<half4*>(at) = hi;
    *reinterpret_cast<half4*>(at + plane) = lo;
  }
}

template <typename S>
__global__ __launch_bounds__(64 * S::NW) void muon_small_kernel(const SmallArgs /*args*/) {
  const SmallArgs& a = *(const SmallArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ __align__(16) char smem[S::kBytes];
  __shared__ float s_norm[S::NW];
  constexpr int RP = S::RP, RT = S::RT, T = S::T, TPW = S::TPW, APW = S::APW, AW = S::AW, KS = S::KS, LT = S::LT, LA = S::LA;
  constexpr int R = Acc<T>::regs;
  typedef typename Acc<T>::type acc_t;
  _Float16* sx = reinterpret_cast<_Float16*>(smem);
  _Float16* sq = sx + 2 * S::kX;
  float* sr = reinterpret_cast<float*>(sq + 2 * S::kA);
  int bi = 0;
  while (bi + 1 < a.nblocks && (int64_t)blockIdx.x >= a.block[bi + 1].first) ++bi;
  const SmallBlock& m = a.block[bi];
  const int64_t base = m.offset + (blockIdx.x - m.first) * m.stride;
  const bool transposed = m.rows > m.cols;
  const int nr = transposed ? m.cols : m.rows, nc = transposed ? m.rows : m.cols;
  const int si = transposed ? 1 : m.cols, sj = transposed ? m.cols : 1;  // X[i][j] is U at i * si + j * sj
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, lj = lane & (T - 1);

  // X in registers: tile t of the wave covers rows T (tile % RT), columns T (tile / RT)
  acc_t x[TPW];
  float q = 0.f;
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tile = wave * TPW + t, j = T * (tile / RT) + lj;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = T * (tile % RT) + tile_row<T>(r);
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
  auto reduce = [&](float v, auto join) {  // over the block, the result in every thread
    for (int d = 32; d > 0; d >>= 1) v = join(v, __shfl_xor(v, d));
    if (lane == 0) s_norm[wave] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < S::NW; ++w) v = join(v, s_norm[w]);
    return v;
  };
  auto sum = [](float u, float v) { return u + v; };
  q = reduce(q, sum);
  float least = a.eps;
  if (!plain_sum(q, a.eps)) {  // uniform over the block
    float largest = 0.f;
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) largest = fmaxf(largest, fabsf(x[t][r]));
    __syncthreads();
    const int e = scale_exponent(reduce(largest, [](float u, float v) { return fmaxf(u, v); }));
    q = 0.f;
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[t][r] = ldexpf(x[t][r], -e);
        q = __builtin_fmaf(x[t][r], x[t][r], q);
      }
    __syncthreads();
    q = reduce(q, sum);
    least = ldexpf(a.eps, -e);
  }
  const float inv = 1.f / fmaxf(sqrtf(q), least);
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int r = 0; r < R; ++r) x[t][r] *= inv;

  for (int k = 0; k < a.nsteps; ++k) {
    const MuonStep st = a.step[k];
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
      const int tile = wave * TPW + t;
      put_columns<T>(sx, LT, S::kX, T * (tile % RT), T * (tile / RT), x[t], pow2(st.ex));  // X^T
    }
    __syncthreads();
    // A = X X^T: KS waves per tile take a part of the columns each
    const int aw = wave % AW, ks = wave / AW;
    const int ai = T * ((aw * APW) % RT), aj = T * ((aw * APW) / RT);
    acc_t acc[APW];
#pragma unroll
    for (int t = 0; t < APW; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[t][r] = 0.f;
    mul_tiles<T, APW, true>(sx, LT, S::kX, ai, sx, LT, S::kX, aj, ks * (S::CP / KS), S::CP / (S::kStep * KS), acc);
    if constexpr (KS > 1) {
      if (ks > 0)
#pragma unroll
        for (int r = 0; r < R; ++r) sr[((ks - 1) * AW + aw) * T * T + r * 64 + lane] = acc[0][r];
      __syncthreads();
    }
    const float fa = pow2(-2 * st.ex);
    if (ks == 0) {
#pragma unroll
      for (int t = 0; t < APW; ++t) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if constexpr (KS > 1)
            for (int w = 0; w < KS - 1; ++w) acc[t][r] += sr[(w * AW + aw) * T * T + r * 64 + lane];
          acc[t][r] *= fa;
        }
        put_columns<T>(sq, LA, S::kA, ai + T * t, aj, acc[t], pow2(st.ea));  // A is symmetric
      }
    }
    __syncthreads();
    // B = b A + c A A, over A
    acc_t sqr[APW];
    if (ks == 0) {
#pragma unroll
      for (int t = 0; t < APW; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) sqr[t][r] = 0.f;
      mul_tiles<T, APW, false>(sq, LA, S::kA, ai, sq, LA, S::kA, aj, 0, RP / S::kStep, sqr);
    }
    __syncthreads();
    if (ks == 0) {
      const float fc = st.c * pow2(-2 * st.ea);
#pragma unroll
      for (int t = 0; t < APW; ++t) {
#pragma unroll
        for (int r = 0; r < R; ++r) sqr[t][r] = st.b * acc[t][r] + fc * sqr[t][r];
        put_columns<T>(sq, LA, S::kA, ai + T * t, aj, sqr[t], pow2(st.eb));
      }
    }
    __syncthreads();
    // X <- a X + B X, the wave's own tiles
    const float fx = pow2(-st.ex - st.eb);
    acc_t bx[TPW];
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) bx[t][r] = 0.f;
    if constexpr (RT % TPW == 0) {  // (all in one column of tiles)
      const int tile = wave * TPW;
      mul_tiles<T, TPW, false>(sq, LA, S::kA, T * (tile % RT), sx, LT, S::kX, T * (tile / RT), 0, RP / S::kStep, bx);
    } else {
#pragma unroll
      for (int t = 0; t < TPW; ++t) {
        const int tile = wave * TPW + t;
        acc_t one[1] = {bx[t]};
        mul_tiles<T, 1, false>(sq, LA, S::kA, T * (tile % RT), sx, LT, S::kX, T * (tile / RT), 0, RP / S::kStep, one);
        bx[t] = one[0];
      }
    }
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) x[t][r] = st.a * x[t][r] + fx * bx[t][r];
    __syncthreads();
  }

  const float keep = 1.f - a.u.lr * a.u.decay;
  const float rate = a.u.lr * (m.cols > m.rows ? sqrtf((float)m.cols / (float)m.rows) : 1.f);
#pragma unroll
  for (int t = 0; t < TPW; ++t) {
    const int tile = wave * TPW + t, j = T * (tile / RT) + lj;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = T * (tile % RT) + tile_row<T>(r);
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
  uint32_t kinds = 0;
  for (int i = 0; i < p.nblocks; ++i)
    if (p.block[i].count > 0 && small_kind(p.block[i]) >= 0) kinds |= 1u << small_kind(p.block[i]);
  if (kinds == 0) return hipSuccess;
  SmallArgs k;
  k.u = u;
  k.update = u.W != nullptr;
  k.nsteps = p.nsteps;
  k.eps = p.eps;
  std::copy(p.step, p.step + p.nsteps, k.step);
  for (int kind = 0; kind < kSmallKinds; ++kind) {
    if (!(kinds >> kind & 1)) continue;
    int64_t n = 0;
    k.nblocks = 0;
    for (int i = 0; i < p.nblocks; ++i) {
      const MuonBlock& b = p.block[i];
      if (b.count == 0 || small_kind(b) != kind) continue;
      k.block[k.nblocks++] = {b.rows, b.cols, b.offset, b.stride, n};
      n += b.count;
    }
    hipError_t e = hipSuccess;
    switch (kind) {
      case kS32x32: e = launch_small<Small<32, 32, 16, 4, 1>>(k, n, s); break;
      case kS32x64: e = launch_small<Small<32, 64, 16, 8, 1>>(k, n, s); break;
      case kS32x128: e = launch_small<Small<32, 128, 16, 16, 1>>(k, n, s); break;
      case kS32x256: e = launch_small<Small<32, 256, 32, 8, 1>>(k, n, s); break;
      case kS32x512: e = launch_small<Small<32, 512, 32, 8, 2>>(k, n, s); break;
      case kS64x64: e = launch_small<Small<64, 64, 16, 16, 1>>(k, n, s); break;
      case kS64x128: e = launch_small<Small<64, 128, 32, 8, 1>>(k, n, s); break;
      case kS64x256: e = launch_small<Small<64, 256, 32, 8, 2>>(k, n, s); break;
      default: e = launch_small<Small<128, 128, 32, 16, 1>>(k, n, s); break;
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
  // 128-wide tiles, which read LDS six times for six products instead of four for
  // three, where there are enough of them: r x r products of 144 such tiles
  // (4 x 1024 x 1024, whole call) 502 us against 522 at 64, of 160 (16 x 512 x
  // 512) 335 against 355, of 72 to 96 slower (32 x 256 x 256: 224 against 205);
  // B X in 256 tiles (16 x 512 x 512) 355 against 385
  const int64_t R = (b.r + 127) / 128, C = (b.c + 127) / 128;
  b.square_tile = R * (R + 1) / 2 * b.m.count >= 128 ? 128 : 64;
  b.apply_tile = R * C * b.m.count >= 192 ? 128 : 64;
  const int pad = b.square_tile > b.apply_tile ? b.square_tile : b.apply_tile;
  b.rp = (b.r + pad - 1) / pad * pad;
  b.cp = (b.c + pad - 1) / pad * pad;
  b.rl = b.rp + kSkew;
  b.cl = b.cp + kSkew;
  b.xsize = (int64_t)b.rp * b.cl;
  b.tsize = (int64_t)b.cp * b.rl;
  b.asize = (int64_t)b.rp * b.rl;
  b.chunks = (int32_t)(((int64_t)b.m.rows * b.m.cols + kNormChunk - 1) / kNormChunk);
  b.eps = p.eps;
  b.scale = b.m.cols > b.m.rows ? sqrtf((float)b.m.cols / (float)b.m.rows) : 1.f;
}

template <int PHASE>
hipError_t launch_phase(const Bank& b, int tile, const MuonStep& st, int ex_next, hipStream_t s) {
  const int R = b.rp / tile, C = b.cp / tile, tiles = PHASE == kGram || PHASE == kPoly ? R * (R + 1) / 2 : R * C;
  if (tiles * b.m.count >= INT32_MAX - 8) return hipErrorInvalidValue;
  const dim3 g((unsigned)((tiles * b.m.count + 7) / 8 * 8));
  if (tile == 128)
    hipLaunchKernelGGL((muon_gemm_kernel<PHASE, 128>), g, dim3(kGemmThreads), 0, s, b, st, ex_next, tiles);
  else
    hipLaunchKernelGGL((muon_gemm_kernel<PHASE, 64>), g, dim3(kGemmThreads), 0, s, b, st, ex_next, tiles);
  return hipGetLastError();
}

// X in two planes, X^T in two buffers of two planes, A and B.
size_t bank_bytes(const Bank& b) {
  const size_t n = (size_t)b.m.count * 2;
  return align_up((size_t)b.m.count * b.chunks * sizeof(float2)) + n * (2 * b.xsize + 4 * b.tsize + 4 * b.asize);
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
    b.norm = static_cast<float2*>(ws);
    _Float16* at =
        reinterpret_cast<_Float16*>(static_cast<char*>(ws) + align_up((size_t)b.m.count * b.chunks * sizeof(float2)));
    auto take = [&](int64_t size) {
      _Float16* p = at;
      at += b.m.count * size;
      return p;
    };
    b.xh = take(b.xsize);
    b.xl = take(b.xsize);
    b.th = take(b.tsize);
    b.tl = take(b.tsize);
    b.nh = take(b.tsize);
    b.nl = take(b.tsize);
    b.ah = take(b.asize);
    b.al = take(b.asize);
    b.bh = take(b.asize);
    b.bl = take(b.asize);
    const unsigned n = (unsigned)b.m.count;
    hipLaunchKernelGGL(muon_norm_kernel, dim3(b.chunks, n), dim3(kThreads), 0, s, b);
    hipLaunchKernelGGL(muon_init_kernel, dim3(b.cp / 64, b.rp / 64, n), dim3(kThreads), 0, s, b, p.step[0].ex);
    for (int k = 0; k < p.nsteps; ++k) {
      const int ex_next = p.step[k + 1].ex;
      hipError_t e = launch_phase<kGram>(b, b.square_tile, p.step[k], ex_next, s);
      if (e == hipSuccess) e = launch_phase<kPoly>(b, b.square_tile, p.step[k], ex_next, s);
      if (e == hipSuccess)
        e = k + 1 < p.nsteps ? launch_phase<kApply>(b, b.apply_tile, p.step[k], ex_next, s)
                             : launch_phase<kLast>(b, b.apply_tile, p.step[k], ex_next, s);
      if (e != hipSuccess) return e;
      std::swap(b.th, b.nh);
      std::swap(b.tl, b.nl);
    }
  }
  return hipGetLastError();
}

}  // namespace tpconv
