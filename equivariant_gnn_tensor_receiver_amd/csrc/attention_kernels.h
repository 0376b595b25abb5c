// Attention among the nodes of each graph (include/tpconv_attention.h).
//
// A wave takes CT = 32 or 16 columns of a head (queries in the forward and in the
// gradient of the queries, keys in the gradients of keys and values) and runs
// over the rows of the other side, 32 at a time:
//
//   forward:   S^T = K Q^T, P = exp(S - m), O^T += V^T P^T
//   grad_q:    S^T = K Q^T, dP^T = V dO^T, dS = P (dP - D), dQ^T += K^T dS^T
//   grad_k/v:  S = Q K^T,  dP = dO V^T,   dV^T += dO^T P,  dK^T += Q^T dS
//
// Every score tile has its own column in the lane and its other index along the
// accumulator registers, so that softmax statistics are sums over a lane's
// registers and one swap of the two half waves, and the tile is, as it stands,
// the right operand of the product that follows: a matrix instruction wants
// eight reductions per lane, and which eight they are does not matter as long
// as the left operand's are the same (the transposing LDS reads take the two
// quads of rows that the accumulators of a lane's group hold).
//
// bf16 takes 32 columns and v_mfma_f32_32x32x16_bf16, four waves per block: bound by
// the vector unit (exponentials, distances, splitting), with two to four waves per
// SIMD.  fp32, and bf16 heads wider than 96, take 16 columns and v_mfma_f32_16x16x32_bf16, eight waves per block:
// its three pieces per operand would leave room for one wave of 32 columns per SIMD
// only, whose products and vector work then follow one another (8192 nodes of
// 128x0e+128x1o+128x2e, 8 heads: forward 369 us, gradients 725 and 1130; this way 270, 334 and 593).
//
// Precision: an fp32 operand is the sum of three bf16 pieces, each the rounded
// rest of those before (|p1| <= 2^-9 |x|, |p2| <= 2^-18 |x|, 2^-27 |x| is left out),
// and the products of the pieces whose ranks add up to at most two are added in
// fp32, smallest first: 2^-25 of a term is left out, of either sign.  bf16
// operands are one piece.  P and dS are fp32 and split like inputs.
//
// The forward saves the reference m that a row's weights were taken against and
// 1 / l, not log(l) + m: the rounding of that sum would leave the weights of a
// row off by a common factor, which sums of dS with something large (distances,
// keys with a common part) do not forgive (gradient of the slopes of 8192 nodes in
// 16 graphs: 1.1e-5 off in place of 1e-6).
//
// Sums over more than kAttnRun rows of the other side are made in runs of that many: the
// matrix instructions' roundings of one accumulator add up along a run (16384 nodes in one
// graph, fp32, 4 heads of 64: gradients off by 4e-6 in one run, 8e-7 in four).  A run's
// sums are added to what the block left of those before in its own rows of the result,
// which costs a read and a write of them per run (forward of 16384 nodes in bf16, 8 heads
// of 64, in four runs: 1654 us in one, 1749).
//
// The rows of the other side go through LDS as planes of pieces, [row][value],
// padded so that 16-byte reads of rows and the transposing reads of columns
// both touch every bank once.
#pragma once

#include "attention.h"
#include "device_common.h"

#include <cfloat>
#include <type_traits>

namespace tpconv {
namespace attn {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
// wide accesses at any element's address (the hardware needs no more alignment)
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

template <typename T>
constexpr int pieces() {
  return sizeof(T) == 4 ? 3 : 1;
}

// LDS row length in values (see the header of this file; checked for 64 banks).
constexpr int row_len(int D) { return D + (D % 64 == 32 || D % 128 == 0 ? 16 : 8); }

// Columns per wave (see the header of this file).
template <typename T, int DC>
constexpr int col_tile() {
  return sizeof(T) == 4 || DC > 96 ? 16 : 32;
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// ---- pieces ---------------------------------------------------------------------

// Three pieces of inputs.  Each value on its own, so that one that is not finite stays alone.
__device__ __forceinline__ void split_inputs(const float (&v)[8], bf16x8 (&p)[3]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    p[0][t] = (__bf16)v[t];
    const float r = v[t] - (float)p[0][t];
    p[1][t] = (__bf16)r;
    p[2][t] = (__bf16)(r - (float)p[1][t]);
  }
}

// Pieces of weights, made beside every tile of scores: the rest v - p comes from a
// dot product of the pair with (-1, 0) or (0, -1), one instruction in place of two.
template <int P>
__device__ __forceinline__ void split_weights(const float (&v)[8], bf16x8 (&p)[P], const SplitConsts& k) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float x = v[2 * t], y = v[2 * t + 1];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bf16x2 h = {(__bf16)x, (__bf16)y};
      p[i][2 * t] = h[0];
      p[i][2 * t + 1] = h[1];
      if (i + 1 < P) {
        x = __builtin_amdgcn_fdot2_f32_bf16(h, k.neg_x, x, false);
        y = __builtin_amdgcn_fdot2_f32_bf16(h, k.neg_y, y, false);
      }
    }
  }
}

__device__ __forceinline__ floatx16 mfma(bf16x8 a, bf16x8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma(bf16x8 a, bf16x8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// acc += sum of the products of pieces of ranks up to 2, smallest first.
template <int PA, int PB, typename ACC>
__device__ __forceinline__ void mul(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], ACC& acc) {
#pragma unroll
  for (int rank = 2; rank >= 0; --rank)
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j)
        if (i + j == rank) acc = mfma(a[i], b[j], acc);
}

// ---- tiles ------------------------------------------------------------------------

// CT columns: lane = group * CT + column.  A tile of 32 rows of scores is a lane's
// registers 4 q + e, row first_row(q) + e; right operands hold 512 / CT reductions
// per step, 8 per lane, from 8 * group on.
template <int CT>
struct Geo;
template <>
struct Geo<32> {
  using Acc = floatx16;                   // one matrix instruction's result
  static constexpr int kRows = 32;        // its rows
  static constexpr int kStep = 16;        // its reductions
  static constexpr int kQuads = 4;        // quads of rows per lane in 32 rows
  static __device__ __forceinline__ int col() { return lane_id() & 31; }
  static __device__ __forceinline__ int group() { return lane_id() >> 5; }
  static __device__ __forceinline__ int first_row(int q) { return 8 * q + 4 * group(); }
};
template <>
struct Geo<16> {
  using Acc = floatx4;
  static constexpr int kRows = 16;
  static constexpr int kStep = 32;
  static constexpr int kQuads = 2;
  static __device__ __forceinline__ int col() { return lane_id() & 15; }
  static __device__ __forceinline__ int group() { return lane_id() >> 4; }
  static __device__ __forceinline__ int first_row(int q) { return 16 * q + 4 * group(); }
};

// 32 rows x CT columns of scores.
template <int CT>
struct Tile32 {
  using G = Geo<CT>;
  static constexpr int kTiles = 32 / G::kRows, kRegs = 4 * G::kQuads, kPer = kRegs / kTiles;
  typename G::Acc a[kTiles];
  __device__ __forceinline__ float get(int r) const { return a[r / kPer][r % kPer]; }
  __device__ __forceinline__ void set(int r, float v) { a[r / kPer][r % kPer] = v; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < kRegs; ++r) set(r, 0.f);
  }
};

// Sums and maxima over the groups of lanes that share a column.
template <int CT, typename F>
__device__ __forceinline__ float join_groups(float v, F f) {
  if constexpr (CT == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <int CT>
__device__ __forceinline__ float col_sum(float v) {
  return join_groups<CT>(v, [](float a, float b) { return a + b; });
}
template <int CT>
__device__ __forceinline__ float col_max(float v) {
  return join_groups<CT>(v, [](float a, float b) { return fmaxf(a, b); });
}

// ---- loads ----------------------------------------------------------------------

// Eight values of a head, e0.., of the row at p; zero from D on.  VEC: channels
// come in whole quads, which are contiguous.
template <typename T>
struct Octet;
template <>
struct Octet<float> {
  float v[8];
  template <bool VEC>
  __device__ __forceinline__ void load(const float* p, const int* at, int e0, int D) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        floatx4 x = {0.f, 0.f, 0.f, 0.f};
        if (e0 + 4 * j < D) x = *reinterpret_cast<const floatx4_any*>(p + at[e0 + 4 * j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * j + e] = x[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e0 + e < D ? p[at[e0 + e]] : 0.f;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
  }
  __device__ __forceinline__ void planes(bf16x8 (&p)[3]) const { split_inputs(v, p); }
};
template <>
struct Octet<uint16_t> {
  u32x4 v;
  template <bool VEC>
  __device__ __forceinline__ void load(const uint16_t* p, const int* at, int e0, int D) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x2 x = {0, 0};
        if (e0 + 4 * j < D) x = *reinterpret_cast<const u32x2_any*>(p + at[e0 + 4 * j]);
        v[2 * j] = x[0];
        v[2 * j + 1] = x[1];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = e0 + 2 * j < D ? p[at[e0 + 2 * j]] : 0;
        const uint32_t hi = e0 + 2 * j + 1 < D ? p[at[e0 + 2 * j + 1]] : 0;
        v[j] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ void clear() { v = (u32x4){0, 0, 0, 0}; }
  __device__ __forceinline__ void planes(bf16x8 (&p)[1]) const { p[0] = __builtin_bit_cast(bf16x8, v); }
};

// Feature offsets of the head's elements (0 from D on, never used).
template <int DC>
__device__ __forceinline__ void fill_table(int* at, const AttnSide& s, int h) {
  for (int e = threadIdx.x; e < DC; e += blockDim.x) {
    int f = 0;
    if (e < s.D) {
      int i = 0;
      while (i + 1 < s.nirr && e >= s.ir[i + 1].first) ++i;
      const int d = e - s.ir[i].first, cph = s.ir[i].cph;
      const int r = d / cph;
      f = s.ir[i].off + r * s.ir[i].mul + h * cph + (d - r * cph);
    }
    at[e] = f;
  }
}

// R rows of the other side from row0 on, `valid` of them there: into registers, and
// from there as planes into LDS, each row multiplied by its factor (fp32 rows
// alone) where there are any.
template <typename T, int DC, int R, int THREADS, bool VEC>
struct Stage {
  static constexpr int P = pieces<T>(), LD = row_len(DC), plane = R * LD, per = DC / 8, total = R * per;
  static constexpr int passes = (total + THREADS - 1) / THREADS;
  // Without whole quads the loads are many: each is stored before the next, to keep the code short.
  static constexpr bool held = VEC || passes == 1;
  Octet<T> o[held ? passes : 1];
  const T* base;
  const float* factor;
  int64_t ld;
  const int* at;
  int D;
  __device__ __forceinline__ Stage(const void* b, int64_t l, const int* t, int d, const float* f = nullptr)
      : base(static_cast<const T*>(b)), factor(f), ld(l), at(t), D(d) {}
  static __device__ __forceinline__ void place(int pass, int& row, int& e0) {
    const int idx = pass * THREADS + (int)threadIdx.x;
    row = idx / per;
    e0 = (idx - row * per) * 8;
  }
  __device__ __forceinline__ void get(int pass, Octet<T>& x, int64_t row0, int valid) const {
    int row, e0;
    place(pass, row, e0);
    x.clear();
    if (row < valid) {
      x.template load<VEC>(base + (row0 + row) * ld, at, e0, D);
      if constexpr (sizeof(T) == 4)
        if (factor) x.scale(factor[row0 + row]);
    }
  }
  static __device__ __forceinline__ void set(int pass, const Octet<T>& x, uint16_t* s) {
    int row, e0;
    place(pass, row, e0);
    if (total % THREADS == 0 || row < R) {
      bf16x8 pl[P];
      x.planes(pl);
#pragma unroll
      for (int i = 0; i < P; ++i) *reinterpret_cast<bf16x8*>(s + i * plane + row * LD + e0) = pl[i];
    }
  }
  __device__ __forceinline__ void load(int64_t row0, int valid) {
    if constexpr (held)
#pragma unroll
      for (int p = 0; p < passes; ++p) get(p, o[p], row0, valid);
  }
  __device__ __forceinline__ void put(uint16_t* s, int64_t row0, int valid) {
    if constexpr (held) {
#pragma unroll
      for (int p = 0; p < passes; ++p) set(p, o[p], s);
    } else {
#pragma unroll 1
      for (int p = 0; p < passes; ++p) {
        get(p, o[0], row0, valid);
        set(p, o[0], s);
      }
    }
  }
};

// Left operand whose rows are rows of LDS: lane (row, group) reads values k + 8 group.. of row `row` + its own.
template <int CT, int P, int DC, int R>
__device__ __forceinline__ void rows_frag(const uint16_t* s, int row, int k, bf16x8 (&f)[P]) {
  constexpr int LD = row_len(DC), plane = R * LD;
#pragma unroll
  for (int i = 0; i < P; ++i)
    f[i] = *reinterpret_cast<const bf16x8*>(s + i * plane + (row + Geo<CT>::col()) * LD + k + 8 * Geo<CT>::group());
}

// Left operand whose rows are columns d.. of LDS and whose reductions are the LDS
// rows of the registers 8 step .. 8 step + 7 of a lane's scores: two quads of rows.
// Each group of 16 lanes turns 4 rows x 16 columns: lane l supplies the address of
// four columns of row l / 4 and receives column l of the four rows.
template <int CT, int P, int DC, int R>
__device__ __forceinline__ void cols_frag(const uint16_t* s, int row, int step, int d, bf16x8 (&f)[P]) {
  constexpr int LD = row_len(DC), plane = R * LD;
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  const int l = lane_id() & 15;
  const uint16_t* p = s + (row + Geo<CT>::first_row(2 * step) + (l >> 2)) * LD + d + (lane_id() & (CT - 16)) + 4 * (l & 3);
  constexpr int next = (CT == 32 ? 8 : 16) * LD;  // the other quad
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + i * plane));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + i * plane + next));
    f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// s += left rows (LDS) x right operand, 32 rows from `row` on, the c-th reduction step.
template <int CT, int PA, int PB, int DC, int R>
__device__ __forceinline__ void add_scores(const uint16_t* lds, int row, int c, const bf16x8 (&b)[PB], Tile32<CT>& s) {
  using G = Geo<CT>;
#pragma unroll
  for (int t = 0; t < Tile32<CT>::kTiles; ++t) {
    bf16x8 f[PA];
    rows_frag<CT, PA, DC, R>(lds, row + G::kRows * t, G::kStep * c, f);
    mul<PA, PB>(f, b, s.a[t]);
  }
}

// A transposed result: rows are head elements, columns the wave's own.
template <int CT, int DC>
struct Result {
  using G = Geo<CT>;
  static constexpr int kTiles = DC / G::kRows, kQuads = CT == 32 ? 4 : 1;
  typename G::Acc a[kTiles];
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4 * kQuads; ++r) a[t][r] *= f;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4 * kQuads; ++r) a[t][r] = 0.f;
  }
  // += columns of LDS (rows row..) x right operand of the step
  template <int PA, int PB, int R>
  __device__ __forceinline__ void add(const uint16_t* lds, int row, int step, const bf16x8 (&b)[PB]) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      bf16x8 f[PA];
      cols_frag<CT, PA, DC, R>(lds, row, step, G::kRows * t, f);
      mul<PA, PB>(f, b, a[t]);
    }
  }
  // Adds f times a lane's row of features to its column.
  template <bool VEC>
  __device__ __forceinline__ void fold(float f, const int* at, int D, const float* row) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int e0 = G::kRows * t + (CT == 32 ? 8 * q : 0) + 4 * G::group();
        if constexpr (VEC) {
          if (e0 < D) {
            const floatx4 x = *reinterpret_cast<const floatx4_any*>(row + at[e0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[t][4 * q + e] = fmaf(f, x[e], a[t][4 * q + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e0 + e < D) a[t][4 * q + e] = fmaf(f, row[at[e0 + e]], a[t][4 * q + e]);
        }
      }
  }
  // Writes a lane's column, times f, to its row of features.
  template <bool VEC, typename O>
  __device__ __forceinline__ void put(float f, const int* at, int D, O* row) const {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int e0 = G::kRows * t + (CT == 32 ? 8 * q : 0) + 4 * G::group();
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[t][4 * q + e] * f;
        if constexpr (VEC) {
          if (e0 < D) put4(row + at[e0], v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e0 + e < D) put1(row + at[e0 + e], v[e]);
        }
      }
  }
  static __device__ __forceinline__ uint32_t bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
  static __device__ __forceinline__ void put1(float* p, float v) { *p = v; }
  static __device__ __forceinline__ void put1(uint16_t* p, float v) { *p = (uint16_t)bits(v); }
  static __device__ __forceinline__ void put4(float* p, const float (&v)[4]) {
    *reinterpret_cast<floatx4_any*>(p) = (floatx4){v[0], v[1], v[2], v[3]};
  }
  static __device__ __forceinline__ void put4(uint16_t* p, const float (&v)[4]) {
    *reinterpret_cast<u32x2_any*>(p) = (u32x2){bits(v[0]) | (bits(v[1]) << 16), bits(v[2]) | (bits(v[3]) << 16)};
  }
};

// ---- rows of graphs ---------------------------------------------------------------

// The rows of tile `t` of M = 1 << shift rows.  Graph g's first tile is
// floor(first row / M) + g, which leaves every graph enough tile numbers, so that
// floor(N / M) + G tiles cover any split of the rows and nothing waits for the
// host.  The graph is found by a search with 64 probes per step.
struct Tile {
  int g;
  int64_t row0;        // first row
  int rows;            // rows of the tile that are in the graph
  int64_t begin, end;  // the graph's rows
};
__device__ __forceinline__ int64_t clamp_row(int32_t v, int64_t N) { return v < 0 ? 0 : v > N ? N : v; }
__device__ __forceinline__ bool find_tile(const int32_t* off, int G, int64_t N, int shift, int64_t t, Tile& o) {
  const int64_t M = int64_t(1) << shift;
  o.g = 0;
  o.begin = 0;
  o.end = N;
  int64_t first = 0;
  if (off) {
    const int lane = lane_id();
    int lo = 0, n = G;  // the last graph of [lo, lo + n) that starts at or before t
    while (true) {
      const int step = (n + 63) >> 6;
      const int i = lane * step;
      const int g = lo + (i < n ? i : 0);
      const int32_t v = off[g];
      const uint64_t m = __ballot(i < n && (clamp_row(v, N) >> shift) + g <= t);
      const int c = __popcll(m);
      if (c == 0) return false;  // before the first graph
      lo += (c - 1) * step;
      const int left = n - (c - 1) * step;
      if (step == 1) {
        // one lane per graph: its rows begin at lane c - 1's value and end at the next one's
        o.begin = clamp_row(__builtin_amdgcn_readlane(v, c - 1), N);
        o.end = clamp_row(c < n && c < 64 ? __builtin_amdgcn_readlane(v, c < 64 ? c : 63) : off[lo + 1], N);
        break;
      }
      n = min(step, left);
    }
    o.g = __builtin_amdgcn_readfirstlane(lo);
    first = (o.begin >> shift) + o.g;
    if (t < first) return false;  // (offsets that decrease)
  }
  o.row0 = o.begin + ((t - first) << shift);
  if (o.row0 >= o.end) return false;
  o.rows = (int)(o.end - o.row0 < M ? o.end - o.row0 : M);
  return true;
}

// Rows [b, e) of graph g's other side, cut to part `part` of `nsplit` (whole tiles of R rows each).
template <int R>
__device__ __forceinline__ void other_rows(const int32_t* off, const Tile& t, bool self, int64_t N, int part, int nsplit,
                                           int64_t& b, int64_t& e) {
  b = self ? t.begin : 0;
  e = self ? t.end : N;
  if (off && !self) {
    b = clamp_row(off[t.g], N);
    e = clamp_row(off[t.g + 1], N);
  }
  if (nsplit > 1) {
    const int64_t len = e > b ? e - b : 0;
    const int64_t per = ((len + nsplit - 1) / nsplit + R - 1) / R * R;
    const int64_t pb = b + per * part;
    e = pb + per < e ? pb + per : e;
    b = pb;
  }
}

// A value that is the same in all lanes, kept in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Which part, head and tile a block works on.  Consecutive items run on one XCD and
// share its L2.  Large graphs: the tiles of a head together, whose other side the L2
// then holds.  Small graphs: the heads of a tile together, since a line of memory holds
// several heads' channels, and eight XCDs that each read every line, and write parts of
// it, cost more than the work (128 graphs of 32 nodes, 8 heads of 36 values, fp32, biased:
// forward and the two gradient kernels 33, 43 and 42 us, this way 24, 29 and 31).
struct Work {
  int part, h;
  uint32_t tile;
};
__device__ __forceinline__ bool find_work(const AttnArgs& a, Work& w) {
  const uint32_t tiles = (uint32_t)a.tiles, H = (uint32_t)a.H, items = tiles * H * (uint32_t)a.nsplit;
  const uint32_t per = gridDim.x >> 3, item = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (item >= items) return false;
  uint32_t rest;
  if (a.heads_inner) {
    rest = item / H;
    w.h = (int)(item - rest * H);
    w.part = (int)(rest / tiles);
    w.tile = rest - (uint32_t)w.part * tiles;
  } else {
    rest = item / tiles;
    w.tile = item - rest * tiles;
    w.part = (int)(rest / H);
    w.h = (int)(rest - (uint32_t)w.part * H);
  }
  return true;
}

// Per-row positions of the other side in LDS, one plane per coordinate, loaded ahead like the rows.
template <int R, int THREADS>
struct StagePos {
  static constexpr int passes = (3 * R + THREADS - 1) / THREADS;
  float v[passes];
  __device__ __forceinline__ void load(const float* pos, int64_t row0, int valid) {
#pragma unroll
    for (int p = 0; p < passes; ++p) {
      const int i = p * THREADS + (int)threadIdx.x;
      v[p] = i < 3 * valid ? pos[row0 * 3 + i] : 0.f;
    }
  }
  __device__ __forceinline__ void put(float* s) const {
#pragma unroll
    for (int p = 0; p < passes; ++p) {
      const int i = p * THREADS + (int)threadIdx.x;
      if (i < 3 * R) s[(i % 3) * R + i / 3] = v[p];
    }
  }
};

// The reference that the forward's weights are taken against moves only when a score
// passes it by more than 2^kSlack, so that the sums are rarely scaled again; weights
// stay below 2^kSlack, which fp32 sums and bf16 pieces hold as well as below 1.
constexpr float kSlack = 8.f;

// A weight made again from its score in the backward: the products come in another order
// there, and scores of 1e9 and more differ by so much that the weight would be infinite
// (one instruction, which keeps NaN).
__device__ __forceinline__ float weight_again(float v) {
  return exp2_fast(__builtin_elementwise_minimum(v, kSlack + 1.f));
}

// A column's (lane's) side of the distance bias.
struct Place {
  float x, y, z, slope2;  // position, slope in units of log2
};
__device__ __forceinline__ Place place_of(const AttnArgs& a, bool bias, const float* pos, int64_t row, int h) {
  Place p = {0.f, 0.f, 0.f, 0.f};
  if (bias) {
    p.x = pos[row * 3];
    p.y = pos[row * 3 + 1];
    p.z = pos[row * 3 + 2];
    p.slope2 = uniform(a.slope[h] * kLog2e);
  }
  return p;
}

// A column's sums for the gradients of slopes and positions.
struct BiasSums {
  float sd = 0.f, s = 0.f, pd = 0.f;  // of dS d, of dS, of P d
  float x = 0.f, y = 0.f, z = 0.f;    // of dS (r - r') / d
};

// How scores are capped: not at all; all of a tile below a quarter of the cap, where
// the odd series of tanh does (the next term is below 2^-26 there); any.
enum CapKind { kNoCap, kSmall, kAnyCap };

// cap tanh(scale s / cap) log2(e), accurate relative to its value.  The series is in
// x = scale s / cap: its coefficients times powers of scale / cap instead would save a
// product per score, but leave fp32's range for caps below about 2e-4 scale, and their
// products with a score of zero are NaN.
struct Cap {
  float in, out, unout;  // scale / cap, cap log2(e), 1 / out
  float k[6];            // of the series in x^2, times x
  __device__ __forceinline__ Cap(const AttnArgs& a) {
    in = uniform(a.cap > 0.f ? a.scale / a.cap : 0.f);
    out = uniform(a.cap * kLog2e);
    unout = uniform(a.cap > 0.f ? 1.f / out : 0.f);
    const float c[6] = {1.f, -1.f / 3.f, 2.f / 15.f, -17.f / 315.f, 62.f / 2835.f, -1382.f / 155925.f};
#pragma unroll
    for (int i = 0; i < 6; ++i) k[i] = uniform(c[i] * out);
  }
  __device__ __forceinline__ float series(float x) const {
    const float t = x * x;
    float v = k[5];
#pragma unroll
    for (int i = 4; i >= 0; --i) v = fmaf(v, t, k[i]);
    return v * x;
  }
  __device__ __forceinline__ float small(float s) const { return series(s * in); }
  __device__ __forceinline__ float any(float s) const {
    const float x = s * in, e = exp2_fast(-2.f * kLog2e * fabsf(x));
    const float big = copysignf((1.f - e) * __builtin_amdgcn_rcpf(1.f + e) * out, x);
    return fabsf(x) < 0.25f ? series(x) : big;
  }
};

// What scores get, known to the compiler: the two kinds of branches around every
// tile would keep copies of it in registers (forward of 16384 nodes x 512 in bf16, when it was split: 1944 -> 1722 us).
// kRuntime leaves both to the run: heads whose channels are not whole quads.
enum ScoreKind { kRuntime = -1, kPlain = 0, kBiased = 1, kCapped = 2, kCappedBiased = 3 };
template <int KIND>
__device__ __forceinline__ bool has_bias(const AttnArgs& a) {
  return KIND == kRuntime ? a.slope != nullptr : (KIND & kBiased) != 0;
}
template <int KIND>
__device__ __forceinline__ bool has_cap(const AttnArgs& a) {
  return KIND == kRuntime ? a.cap > 0.f : (KIND & kCapped) != 0;
}

// f(cap kind, bias) with the two as compile-time constants.
template <int KIND, int CT, typename F>
__device__ __forceinline__ void with_kind(const AttnArgs& a, const Cap& cap, const Tile32<CT>& s, F f) {
  auto go = [&](auto kind) {
    if (has_bias<KIND>(a))
      f(kind, std::true_type{});
    else
      f(kind, std::false_type{});
  };
  if (!has_cap<KIND>(a)) {
    go(std::integral_constant<int, kNoCap>{});
    return;
  }
  float top = fabsf(s.get(0));
#pragma unroll
  for (int r = 1; r < Tile32<CT>::kRegs; ++r) top = fmaxf(top, fabsf(s.get(r)));
  if (__any(!(top * fabsf(cap.in) < 0.25f)))
    go(std::integral_constant<int, kAnyCap>{});
  else
    go(std::integral_constant<int, kSmall>{});
}

// Scores of a tile.  CAP or BIAS: in units of log2; otherwise as they are, to be
// multiplied by scale log2(e).
template <int CAP, bool BIAS, int R, int CT>
__device__ __forceinline__ void score_tile(const Cap& cap, float c, Tile32<CT>& s, const float* spos, int row,
                                           const Place& p) {
  using G = Geo<CT>;
#pragma unroll
  for (int q = 0; q < G::kQuads; ++q) {
    floatx4 x, y, z;
    if constexpr (BIAS) {
      const int at = row + G::first_row(q);
      x = *reinterpret_cast<const floatx4*>(spos + at);
      y = *reinterpret_cast<const floatx4*>(spos + R + at);
      z = *reinterpret_cast<const floatx4*>(spos + 2 * R + at);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = s.get(4 * q + e);
      if constexpr (CAP == kSmall) v = cap.small(v);
      if constexpr (CAP == kAnyCap) v = cap.any(v);
      if constexpr (BIAS) {
        const float dx = p.x - x[e], dy = p.y - y[e], dz = p.z - z[e];
        const float dist = __builtin_amdgcn_sqrtf(fmaf(dx, dx, fmaf(dy, dy, dz * dz)));
        v = CAP != kNoCap ? fmaf(-p.slope2, dist, v) : fmaf(v, c, -p.slope2 * dist);
      }
      s.set(4 * q + e, v);
    }
  }
}

// The tile of the backward: s (scores as products) -> weights against the rows'
// references ref(q), ds (dP) -> dS = P (dP - delta(q)), in the end with the cap's
// factor; adds to the column's sums where there is a bias.
template <int CAP, bool BIAS, int R, int CT, typename REF, typename DELTA>
__device__ __forceinline__ void grad_tile(const Cap& cap, float c, Tile32<CT>& s, Tile32<CT>& ds, const float* spos,
                                          int row, const Place& p, BiasSums& b, REF ref, DELTA delta) {
  using G = Geo<CT>;
#pragma unroll
  for (int q = 0; q < G::kQuads; ++q) {
    const int at = row + G::first_row(q);
    floatx4 x, y, z;
    if constexpr (BIAS) {
      x = *reinterpret_cast<const floatx4*>(spos + at);
      y = *reinterpret_cast<const floatx4*>(spos + R + at);
      z = *reinterpret_cast<const floatx4*>(spos + 2 * R + at);
    }
    const floatx4 m4 = ref(q), d4 = delta(q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * q + e;
      float u = s.get(r);
      if constexpr (CAP == kSmall) u = cap.small(u);
      if constexpr (CAP == kAnyCap) u = cap.any(u);
      float v = CAP != kNoCap ? u - m4[e] : fmaf(u, c, -m4[e]);
      float g;
      if constexpr (BIAS) {
        const float dx = p.x - x[e], dy = p.y - y[e], dz = p.z - z[e];
        const float d2 = fmaf(dx, dx, fmaf(dy, dy, dz * dz));
        const float over = d2 >= FLT_MIN ? __builtin_amdgcn_rsqf(d2) : 0.f;  // (of a subnormal: infinity)
        const float dist = d2 * over;
        v = weight_again(fmaf(-p.slope2, dist, v));
        g = v * (ds.get(r) - d4[e]);
        b.sd = fmaf(g, dist, b.sd);
        b.s += g;
        b.pd = fmaf(v, dist, b.pd);
        const float w = g * over;
        b.x = fmaf(w, dx, b.x);
        b.y = fmaf(w, dy, b.y);
        b.z = fmaf(w, dz, b.z);
      } else {
        v = weight_again(v);
        g = v * (ds.get(r) - d4[e]);
      }
      if constexpr (CAP != kNoCap) {
        const float th = u * cap.unout;
        g *= fmaf(-th, th, 1.f);
      }
      ds.set(r, g);
      s.set(r, v);
    }
  }
}

// Eight registers of a tile as a right operand's pieces.
template <int P, int CT>
__device__ __forceinline__ void weights_frag(const Tile32<CT>& s, int step, bf16x8 (&p)[P], const SplitConsts& k) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = s.get(8 * step + e);
  split_weights<P>(v, p, k);
}

// A block takes 128 columns of a head, or attn_small_cols where the graphs are small.  (64 for
// wide fp32 heads, which lets a CU hold two blocks, splits the other side's rows
// twice as often: 8192 nodes of 128x0e+128x1o+128x2e, 8 heads: 269, 434, 434 and 274 us where 128 take 259, 332, 332 and 255.)
template <typename T, int DC, int COLS>
struct Block {
  static constexpr int CT = col_tile<T, DC>(), kWaves = COLS / CT, kThreads = 64 * kWaves;
  static constexpr int kShift = COLS == 128 ? 7 : COLS == 64 ? 6 : 5;
  static_assert(COLS == 128 || COLS == attn_small_cols(DC), "rows per block");
  // whether none of the wave's columns is there: it helps with the rows and skips the products
  static __device__ __forceinline__ bool idle(int rows) {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) * CT >= rows;
  }
  // the block's column of this lane
  static __device__ __forceinline__ int col() { return (int)(threadIdx.x >> 6) * CT + Geo<CT>::col(); }
  // the same where the compiler cannot tell: what a run's end needs of it is made there and takes no
  // registers in the loop before
  static __device__ __forceinline__ int col_again() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return (t >> 6) * CT + (t & (CT - 1));
  }
};

// A column's right operand: values of the row at p.
template <typename T, int DC, bool VEC, int CT, int P>
__device__ __forceinline__ void own_row(const T* p, const int* at, int D, bf16x8 (&f)[DC / Geo<CT>::kStep][P]) {
#pragma unroll
  for (int c = 0; c < DC / Geo<CT>::kStep; ++c) {
    Octet<T> o;
    o.template load<VEC>(p, at, Geo<CT>::kStep * c + 8 * Geo<CT>::group(), D);
    o.planes(f[c]);
  }
}

// Waves per SIMD that the registers are held to, from an estimate of what a wave
// holds: a block's waves meet at every step, and others hide the latency.  Two at
// least, which also keeps every kernel out of the accumulation registers: with these
// in use and values spilled at once, ROCm 7.2's compiler ended in its pass over MFMA
// operands in accumulation registers or made kernels with wrong results (the build
// refuses such a kernel).
constexpr int waves_for(int regs) { return regs <= 110 ? 4 : regs <= 150 ? 3 : 2; }
// registers of: right operands of n pieces in all, results, scores, and the rest
template <typename T, int DC>
constexpr int regs_for(int right, int results, int rest) {
  return DC * col_tile<T, DC>() / 128 * right + results * DC * col_tile<T, DC>() / 64 + rest;
}

// Whether a kernel holds the other side's next rows in registers while it works on
// the present ones: not where wide heads leave none for it, nor in the backward of
// small graphs, which take one or two steps.  (The first rows are on their way before
// the own row is wherever heads are not wide.)
template <typename T, int DC, int COLS>
constexpr bool rows_ahead(bool forward) {
  return forward ? DC <= (COLS == 128 ? 160 : 96) : COLS == 128 && DC <= 96;
}

// ---- forward ----------------------------------------------------------------------

template <typename T, int DC, int COLS, bool VEC, int KIND>
__global__ __launch_bounds__((Block<T, DC, COLS>::kThreads), (waves_for(regs_for<T, DC>(pieces<T>(), 1, (KIND & kCapped) != 0 ? 80 : 60)))) void forward_kernel(
    const AttnArgs a) {
  using B = Block<T, DC, COLS>;
  constexpr int CT = B::CT, P = pieces<T>(), R = 32, LD = row_len(DC);
  using G = Geo<CT>;
  constexpr int NC = DC / G::kStep, kRegs = Tile32<CT>::kRegs;
  __shared__ __align__(16) uint16_t sk[P * R * LD], sv[P * R * LD];
  __shared__ int at_qk[DC], at_v[DC];
  __shared__ __align__(16) float spos[3 * R];
  __shared__ float runs[2][B::kThreads];  // what the sums of the runs so far are taken against, and of their weights
  Work w;
  Tile t;
  if (!find_work(a, w) || !find_tile(a.qo, a.G, a.Nq, B::kShift, w.tile, t)) return;
  fill_table<DC>(at_qk, a.sqk, w.h);
  fill_table<DC>(at_v, a.sv, w.h);
  __syncthreads();
  const bool idle = B::idle(t.rows);
  const int64_t query = t.row0 + min(B::col(), t.rows - 1);
  const int Dqk = a.sqk.D, Dv = a.sv.D;
  const bool bias = has_bias<KIND>(a);
  int64_t kb, ke;
  other_rows<R>(a.ko, t, a.self, a.Nk, w.part, a.nsplit, kb, ke);
  Stage<T, DC, R, B::kThreads, VEC> rk(a.k, a.ldk, at_qk, Dqk), rv(a.v, a.ldv, at_v, Dv);
  StagePos<R, B::kThreads> rp;
  auto load = [&](int64_t k0) {
    const int valid = (int)(ke - k0 < R ? ke - k0 : R);
    rk.load(k0, valid);
    rv.load(k0, valid);
    if (bias) rp.load(a.kpos, k0, valid);
  };
  constexpr bool kAhead = rows_ahead<T, DC, COLS>(true), kFirst = kAhead || DC <= 96;
  if (kFirst && kb < ke) load(kb);
  bf16x8 q[NC][P];
  own_row<T, DC, VEC, CT>(static_cast<const T*>(a.q) + query * a.ldq, at_qk, Dqk, q);
  const Place place = place_of(a, bias, a.qpos, query, w.h);
  const Cap cap(a);
  const SplitConsts consts;
  // scores are multiplied by this on their way into the exponent
  const float c2 = uniform(a.scale * kLog2e);
  const bool raw = !bias && !has_cap<KIND>(a);
  // unless they are (next to) zero then: rows that are not there would not stay at minus infinity
  const bool flat = raw && fabsf(c2) < FLT_MIN;
  const float unit = uniform(raw && !flat ? c2 : 1.f);
  Result<CT, DC> acc;
  acc.clear();
  float m = -INFINITY, l = 0.f;
  for (int64_t k0 = kb;;) {
    const int64_t begin = k0, stop = ke - k0 < kAttnRun ? ke : k0 + kAttnRun;
    for (; k0 < stop; k0 += R) {
      const int valid = (int)(ke - k0 < R ? ke - k0 : R);
      if (!kAhead && (!kFirst || k0 > kb)) load(k0);
      __syncthreads();
      rk.put(sk, k0, valid);
      rv.put(sv, k0, valid);
      if (bias) rp.put(spos);
      __syncthreads();
      if (kAhead && k0 + R < ke) {
        load(k0 + R);
        __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
      }
      for (int sub = idle ? valid : 0; sub < valid; sub += 32) {
        Tile32<CT> s;
        s.clear();
#pragma unroll
        for (int c = 0; c < NC; ++c) add_scores<CT, P, P, DC, R>(sk, sub, c, q[c], s);
        if (!raw)
          with_kind<KIND>(a, cap, s, [&](auto kind, auto bs) {
            score_tile<decltype(kind)::value, decltype(bs)::value, R>(cap, c2, s, spos, sub, place);
          });
        if (flat)
#pragma unroll
          for (int r = 0; r < kRegs; ++r) s.set(r, s.get(r) * c2);
        if (valid - sub < 32)
#pragma unroll
          for (int r = 0; r < kRegs; ++r)
            if (sub + G::first_row(r / 4) + r % 4 >= valid) s.set(r, unit < 0.f ? INFINITY : -INFINITY);
        float top = s.get(0);
        if (unit < 0.f) {
#pragma unroll
          for (int r = 1; r < kRegs; ++r) top = fminf(top, s.get(r));
        } else {
#pragma unroll
          for (int r = 1; r < kRegs; ++r) top = fmaxf(top, s.get(r));
        }
        top = col_max<CT>(top * unit);
        if (__any(top > m + kSlack)) {
          const float next = fmaxf(m, top);
          const float f = m == -INFINITY ? 0.f : exp2_fast(m - next);
          l *= f;
          acc.scale(f);
          m = next;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float here = 0.f;  // (a tile's weights before the running sum: fewer roundings at its size)
#pragma unroll
        for (int r = 0; r < kRegs; ++r) {
          const float p = exp2_fast(fmaf(s.get(r), unit, -ref));
          s.set(r, p);
          here += p;
        }
        l += here;
#pragma unroll
        for (int st = 0; st < kRegs / 8; ++st) {
          bf16x8 p[3];
          weights_frag<3>(s, st, p, consts);
          acc.template add<P, 3, R>(sv, sub, st, p);
        }
      }
    }
    // the end of a run
    const int col = B::col_again();
    const bool mine = col < t.rows, last = k0 >= ke;
    const int64_t query = t.row0 + min(col, t.rows - 1);
    const int F = a.sv.F;
    float* const row = a.sums + ((int64_t)w.part * a.Nq + query) * F;
    if (begin > kb) {
      const float then = runs[0][threadIdx.x], f = then == -INFINITY ? 0.f : exp2_fast(then - m);
      l = fmaf(runs[1][threadIdx.x], f, l);
      if (mine) acc.template fold<VEC>(f, at_v, Dv, row);
    }
    if (last) break;
    runs[0][threadIdx.x] = m;
    runs[1][threadIdx.x] = l;
    if (mine) acc.template put<VEC>(1.f, at_v, Dv, row);
    acc.clear();
    l = 0.f;
  }
  l = col_sum<CT>(l);
  const int col = B::col_again();
  if (col >= t.rows) return;
  const int64_t own = t.row0 + col;
  const int F = a.sv.F;
  float f = 1.f;
  if (a.nsplit > 1) {
    const int64_t at = ((int64_t)w.part * a.H + w.h) * a.Nq + own;
    if (G::group() == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
  } else {
    f = l > 0.f || l != l ? 1.f / l : 0.f;
    if (a.stat && G::group() == 0) {
      a.stat[(int64_t)w.h * a.Nq + own] = m;
      a.stat[(int64_t)(a.H + w.h) * a.Nq + own] = f;
    }
  }
  if (a.put_f32) acc.template put<VEC>(f, at_v, Dv, a.sums + ((int64_t)w.part * a.Nq + own) * F);
  if (a.put_bf16) acc.template put<VEC>(f, at_v, Dv, static_cast<uint16_t*>(a.out) + own * F);
}

// A value of a run after the first joins what is there of those before.
__device__ __forceinline__ void put_sum(float* o, bool first, float v) { *o = first ? v : *o + v; }

// A column's share of its position's gradient, per part and head.
template <int CT>
__device__ __forceinline__ void put_pos(const AttnArgs& a, bool bias, const Work& w, int64_t rows, int64_t row, bool mine,
                                        bool first, BiasSums& b, float f) {
  if (!bias || !a.part_pos) return;
  b.x = col_sum<CT>(b.x);
  b.y = col_sum<CT>(b.y);
  b.z = col_sum<CT>(b.z);
  if (!mine || Geo<CT>::group() != 0) return;
  float* o = a.part_pos + (((int64_t)w.part * a.H + w.h) * rows + row) * 3;
  f *= -a.slope[w.h];
  put_sum(o, first, f * b.x);
  put_sum(o + 1, first, f * b.y);
  put_sum(o + 2, first, f * b.z);
}

// ---- gradient of the queries ----------------------------------------------------------

template <typename T, int DC, int COLS, bool VEC, int KIND>
__global__ __launch_bounds__((Block<T, DC, COLS>::kThreads),
                             (waves_for(regs_for<T, DC>(pieces<T>() + 3, 1, 110)))) void grad_q_kernel(const AttnArgs a) {
  using B = Block<T, DC, COLS>;
  constexpr int CT = B::CT, P = pieces<T>(), R = COLS > 32 && DC <= 64 ? 64 : 32, LD = row_len(DC);
  using G = Geo<CT>;
  constexpr int NC = DC / G::kStep, kRegs = Tile32<CT>::kRegs;
  __shared__ __align__(16) uint16_t sk[P * R * LD], sv[P * R * LD];
  __shared__ int at_qk[DC], at_v[DC];
  __shared__ __align__(16) float spos[3 * R];
  Work w;
  Tile t;
  if (!find_work(a, w) || !find_tile(a.qo, a.G, a.Nq, B::kShift, w.tile, t)) return;
  fill_table<DC>(at_qk, a.sqk, w.h);
  fill_table<DC>(at_v, a.sv, w.h);
  __syncthreads();
  const bool idle = B::idle(t.rows);
  const int64_t query = t.row0 + min(B::col(), t.rows - 1);
  const int Dqk = a.sqk.D, Dv = a.sv.D;
  const bool bias = has_bias<KIND>(a);
  int64_t kb, ke;
  other_rows<R>(a.ko, t, a.self, a.Nk, w.part, a.nsplit, kb, ke);
  Stage<T, DC, R, B::kThreads, VEC> rk(a.k, a.ldk, at_qk, Dqk), rv(a.v, a.ldv, at_v, Dv);
  StagePos<R, B::kThreads> rp;
  auto load = [&](int64_t k0) {
    const int valid = (int)(ke - k0 < R ? ke - k0 : R);
    rk.load(k0, valid);
    rv.load(k0, valid);
    if (bias) rp.load(a.kpos, k0, valid);
  };
  constexpr bool kAhead = rows_ahead<T, DC, COLS>(false), kFirst = kAhead || DC <= 96;
  if (kFirst && kb < ke) load(kb);
  bf16x8 q[NC][P], g[NC][3];
  own_row<T, DC, VEC, CT>(static_cast<const T*>(a.q) + query * a.ldq, at_qk, Dqk, q);
  float delta = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    Octet<float> go, y;
    go.template load<VEC>(a.go + query * a.sv.F, at_v, G::kStep * c + 8 * G::group(), Dv);
    y.template load<VEC>(a.o + query * a.sv.F, at_v, G::kStep * c + 8 * G::group(), Dv);
    go.planes(g[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) delta = fmaf(go.v[e], y.v[e], delta);
  }
  delta = col_sum<CT>(delta);
  if (B::col() < t.rows && G::group() == 0 && w.part == 0) a.delta[(int64_t)w.h * a.Nq + query] = delta;
  const float m = a.stat[(int64_t)w.h * a.Nq + query], inv = a.stat[(int64_t)(a.H + w.h) * a.Nq + query];
  const Place place = place_of(a, bias, a.qpos, query, w.h);
  const floatx4 delta4 = {delta, delta, delta, delta};
  const Cap cap(a);
  const SplitConsts consts;
  const float c2 = uniform(a.scale * kLog2e);
  BiasSums sums;
  Result<CT, DC> acc;
  acc.clear();
  for (int64_t k0 = kb;;) {
    const int64_t begin = k0, stop = ke - k0 < kAttnRun ? ke : k0 + kAttnRun;
    for (; k0 < stop; k0 += R) {
      const int valid = (int)(ke - k0 < R ? ke - k0 : R);
      if (!kAhead && (!kFirst || k0 > kb)) load(k0);
      __syncthreads();
      rk.put(sk, k0, valid);
      rv.put(sv, k0, valid);
      if (bias) rp.put(spos);
      __syncthreads();
      if (kAhead && k0 + R < ke) {
        load(k0 + R);
        __builtin_amdgcn_sched_barrier(0);
      }
      for (int sub = idle ? valid : 0; sub < valid; sub += 32) {
        Tile32<CT> s, ds;
        s.clear();
        ds.clear();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          add_scores<CT, P, P, DC, R>(sk, sub, c, q[c], s);
          add_scores<CT, P, 3, DC, R>(sv, sub, c, g[c], ds);
        }
        with_kind<KIND>(a, cap, s, [&](auto kind, auto bs) {
          grad_tile<decltype(kind)::value, decltype(bs)::value, R>(
              cap, c2, s, ds, spos, sub, place, sums,
              [&](int q4) {  // keys that are not there: a weight of zero
                floatx4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = sub + G::first_row(q4) + e < valid ? m : INFINITY;
                return v;
              },
              [&](int) { return delta4; });
        });
#pragma unroll
        for (int st = 0; st < kRegs / 8; ++st) {
          bf16x8 p[3];
          weights_frag<3>(ds, st, p, consts);
          acc.template add<P, 3, R>(sk, sub, st, p);
        }
      }
    }
    const int col = B::col_again();
    const bool mine = col < t.rows, first = begin == kb, last = k0 >= ke;
    const int64_t query = t.row0 + min(col, t.rows - 1);
    put_pos<CT>(a, bias, w, a.Nq, query, mine, first, sums, inv);
    if (bias && a.part_slope) {
      // sum dS d = sum dS (d - mean d) as far as the sum of dS is zero, which it is but for
      // rounding: the join takes sum dS d - sum dS * sum P d, which does not see that rounding
      sums.sd = col_sum<CT>(sums.sd);
      sums.s = col_sum<CT>(sums.s);
      sums.pd = col_sum<CT>(sums.pd);
      if (mine && G::group() == 0) {
        float* o = a.part_slope + (((int64_t)w.part * a.H + w.h) * a.Nq + query) * 3;
        put_sum(o, first, sums.sd * inv);
        put_sum(o + 1, first, sums.s * inv);
        put_sum(o + 2, first, sums.pd * inv);
      }
    }
    if (a.gq && mine) {
      float* const row = a.gq + ((int64_t)w.part * a.Nq + query) * a.ldgq;
      if (!first) acc.template fold<VEC>(1.f, at_qk, Dqk, row);
      acc.template put<VEC>(last ? a.scale * inv : 1.f, at_qk, Dqk, row);
    }
    if (last) break;
    acc.clear();
    sums = BiasSums();
  }
}

// ---- gradients of keys and values --------------------------------------------------------

// Wide heads take the two gradients in two launches: the operands and sums of
// both are 200 registers of the 256 that two waves per SIMD leave each, and what
// went to scratch memory cost more than doing the scores twice (8192 nodes of
// 128x0e+128x1o+128x2e, 8 heads, when they were split: 952 us in one launch, 710 in two; the two now take 593).
enum KvPart { kBoth, kValues, kKeys };
template <typename T, int DC>
constexpr bool kv_in_two() {
  return DC > (sizeof(T) == 4 ? 96 : 160);
}

template <typename T, int DC, int COLS, bool VEC, int KIND, int PART>
__global__ __launch_bounds__((Block<T, DC, COLS>::kThreads),
                             (waves_for(regs_for<T, DC>((PART == kValues ? 1 : 2) * pieces<T>(), PART == kBoth ? 2 : 1, 110)))) void grad_kv_kernel(const AttnArgs a) {
  using B = Block<T, DC, COLS>;
  constexpr int CT = B::CT, P = pieces<T>(), R = COLS > 32 && DC <= 64 && P == 1 ? 64 : 32, LD = row_len(DC);
  using G = Geo<CT>;
  constexpr int NC = DC / G::kStep, kRegs = Tile32<CT>::kRegs;
  __shared__ __align__(16) uint16_t sq[P * R * LD], sg[3 * R * LD];
  __shared__ int at_qk[DC], at_v[DC];
  __shared__ __align__(16) float spos[3 * R], sl[R], sd[R];
  Work w;
  Tile t;
  if (!find_work(a, w) || !find_tile(a.ko, a.G, a.Nk, B::kShift, w.tile, t)) return;
  fill_table<DC>(at_qk, a.sqk, w.h);
  fill_table<DC>(at_v, a.sv, w.h);
  __syncthreads();
  const bool idle = B::idle(t.rows);
  const int64_t key = t.row0 + min(B::col(), t.rows - 1);
  const int Dqk = a.sqk.D, Dv = a.sv.D;
  const bool bias = has_bias<KIND>(a);
  int64_t qb, qe;
  other_rows<R>(a.qo, t, a.self, a.Nq, w.part, a.nsplit, qb, qe);
  // rows of grad_out are taken times 1 / l, so that the weights need no factor of their own
  const float *ref = a.stat + (int64_t)w.h * a.Nq, *inv = ref + (int64_t)a.H * a.Nq, *delta = a.delta + (int64_t)w.h * a.Nq;
  Stage<T, DC, R, B::kThreads, VEC> rq(a.q, a.ldq, at_qk, Dqk);
  Stage<float, DC, R, B::kThreads, VEC> rg(a.go, a.sv.F, at_v, Dv, inv);
  StagePos<R, B::kThreads> rp;
  float row_m = INFINITY, row_d = 0.f;
  auto load = [&](int64_t q0) {
    const int valid = (int)(qe - q0 < R ? qe - q0 : R);
    rq.load(q0, valid);
    rg.load(q0, valid);
    if (bias) rp.load(a.qpos, q0, valid);
    row_m = INFINITY;  // a weight of zero
    row_d = 0.f;
    if ((int)threadIdx.x < valid) {
      row_m = ref[q0 + threadIdx.x];
      row_d = delta[q0 + threadIdx.x] * inv[q0 + threadIdx.x];
    }
  };
  constexpr bool kAhead = rows_ahead<T, DC, COLS>(false), kFirst = kAhead || DC <= 96;
  if (kFirst && qb < qe) load(qb);
  bf16x8 k[NC][P], v[NC][P];
  own_row<T, DC, VEC, CT>(static_cast<const T*>(a.k) + key * a.ldk, at_qk, Dqk, k);
  if constexpr (PART != kValues) own_row<T, DC, VEC, CT>(static_cast<const T*>(a.v) + key * a.ldv, at_v, Dv, v);
  const Place place = place_of(a, bias, a.kpos, key, w.h);
  const Cap cap(a);
  const SplitConsts consts;
  const float c2 = uniform(a.scale * kLog2e);
  BiasSums sums;
  Result<CT, DC> gv, gk;
  gv.clear();
  gk.clear();
  for (int64_t q0 = qb;;) {
    const int64_t begin = q0, stop = qe - q0 < kAttnRun ? qe : q0 + kAttnRun;
    for (; q0 < stop; q0 += R) {
      const int valid = (int)(qe - q0 < R ? qe - q0 : R);
      if (!kAhead && (!kFirst || q0 > qb)) load(q0);
      __syncthreads();
      rq.put(sq, q0, valid);
      rg.put(sg, q0, valid);
      if (bias) rp.put(spos);
      if ((int)threadIdx.x < R) {
        sl[threadIdx.x] = row_m;
        sd[threadIdx.x] = row_d;
      }
      __syncthreads();
      if (kAhead && q0 + R < qe) {
        load(q0 + R);
        __builtin_amdgcn_sched_barrier(0);
      }
      for (int sub = idle ? valid : 0; sub < valid; sub += 32) {
        Tile32<CT> s, ds;
        s.clear();
        ds.clear();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          add_scores<CT, P, P, DC, R>(sq, sub, c, k[c], s);
          if constexpr (PART != kValues) add_scores<CT, 3, P, DC, R>(sg, sub, c, v[c], ds);
        }
        with_kind<KIND>(a, cap, s, [&](auto kind, auto bs) {
          if constexpr (PART == kValues) {
            score_tile<decltype(kind)::value, decltype(bs)::value, R>(cap, c2, s, spos, sub, place);
            const float unit = decltype(kind)::value == kNoCap && !decltype(bs)::value ? c2 : 1.f;
#pragma unroll
            for (int q4 = 0; q4 < G::kQuads; ++q4) {
              const floatx4 m4 = *reinterpret_cast<const floatx4*>(sl + sub + G::first_row(q4));
#pragma unroll
              for (int e = 0; e < 4; ++e) s.set(4 * q4 + e, weight_again(fmaf(s.get(4 * q4 + e), unit, -m4[e])));
            }
            return;
          }
          grad_tile<decltype(kind)::value, decltype(bs)::value, R>(
              cap, c2, s, ds, spos, sub, place, sums,
              [&](int q4) { return *reinterpret_cast<const floatx4*>(sl + sub + G::first_row(q4)); },
              [&](int q4) { return *reinterpret_cast<const floatx4*>(sd + sub + G::first_row(q4)); });
        });
#pragma unroll
        for (int st = 0; st < kRegs / 8; ++st) {
          bf16x8 p[3];
          if constexpr (PART != kKeys) {
            weights_frag<3>(s, st, p, consts);
            gv.template add<3, 3, R>(sg, sub, st, p);
          }
          if constexpr (PART != kValues) {
            weights_frag<3>(ds, st, p, consts);
            gk.template add<P, 3, R>(sq, sub, st, p);
          }
        }
      }
    }
    const int col = B::col_again();
    const bool mine = col < t.rows, first = begin == qb, last = q0 >= qe;
    const int64_t key = t.row0 + min(col, t.rows - 1);
    if constexpr (PART != kValues) {
      put_pos<CT>(a, bias, w, a.Nk, key, mine, first, sums, 1.f);
      if (a.gk && mine) {
        float* const row_k = a.gk + ((int64_t)w.part * a.Nk + key) * a.ldgk;
        if (!first) gk.template fold<VEC>(1.f, at_qk, Dqk, row_k);
        gk.template put<VEC>(last ? a.scale : 1.f, at_qk, Dqk, row_k);
      }
    }
    if constexpr (PART != kKeys)
      if (a.gv && mine) {
        float* const row_v = a.gv + ((int64_t)w.part * a.Nk + key) * a.ldgv;
        if (!first) gv.template fold<VEC>(1.f, at_v, Dv, row_v);
        gv.template put<VEC>(1.f, at_v, Dv, row_v);
      }
    if (last) break;
    gk.clear();
    gv.clear();
    sums = BiasSums();
  }
}

}  // namespace attn
}  // namespace tpconv
