// Attention among the nodes of each graph (include/tpconv_attention.h).
//
// A wave takes 32 columns of a head (queries in the forward and in the
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
// the right operand of the product that follows: v_mfma_f32_32x32x16_bf16 wants
// eight reductions per lane, and which eight they are does not matter as long
// as the left operand's are the same (the transposing LDS reads take keys
// 4h..4h+3 and 8+4h..8+4h+3 for half wave h, which is how the accumulators lie).
//
// Precision: an fp32 operand is the sum of three bf16 pieces, each the rounded
// rest of those before (|p1| <= 2^-9 |x|, |p2| <= 2^-18 |x|, 2^-27 |x| is left out),
// and the products of the pieces whose ranks add up to at most two are added in
// fp32, smallest first: 2^-25 of a term is left out, of either sign.  bf16
// operands are one piece.  P and dS are fp32 and split like inputs, except in a
// bf16 forward that saves nothing, where P is two pieces (2^-18).
//
// The forward saves the reference m that a row's weights were taken against and
// 1 / l, not log(l) + m: the rounding of that sum would leave the weights of a
// row off by a common factor, which sums of dS with something large (distances,
// keys with a common part) do not forgive (gradient of the slopes of 8192 nodes in
// 16 graphs: 1.1e-5 off in place of 1e-6).
//
// The rows of the other side go through LDS as planes of pieces, [row][value],
// padded so that 16-byte reads of rows and the transposing reads of columns
// both touch every bank once.
#pragma once

#include "attention.h"
#include "device_common.h"

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

// ---- pieces ---------------------------------------------------------------------

template <int P>
__device__ __forceinline__ void split(const float (&v)[8], bf16x8 (&p)[P]) {
  if constexpr (P == 3) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      p[0][t] = (__bf16)v[t];
      const float r = v[t] - (float)p[0][t];
      p[1][t] = (__bf16)r;
      p[2][t] = (__bf16)(r - (float)p[1][t]);
    }
  } else {
    static_assert(P == 2, "fp32 values are three or two pieces");
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      p[0][t] = (__bf16)v[t];
      p[1][t] = (__bf16)(v[t] - (float)p[0][t]);
    }
  }
}

// acc += sum of the products of pieces of ranks up to 2, smallest first.
template <int PA, int PB>
__device__ __forceinline__ void mul(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], floatx16& acc) {
#pragma unroll
  for (int rank = 2; rank >= 0; --rank)
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j)
        if (i + j == rank) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc, 0, 0, 0);
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
  __device__ __forceinline__ void planes(bf16x8 (&p)[3]) const { split<3>(v, p); }
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
// alone) where there are any.  Blocks of four waves share the rows; a block of one
// wave (R = 32) loads them as the left operand of the products wants them, lane
// (i, h) values 16 c + 8 h.. of row i, and uses them from the registers too.
template <typename T, int DC, int R, int W, bool VEC>
struct Stage {
  static constexpr int P = pieces<T>(), LD = row_len(DC), plane = R * LD, per = DC / 8, total = R * per;
  static constexpr int passes = (total + 64 * W - 1) / (64 * W);
  static_assert(W == 4 || R == 32, "one wave takes 32 rows");
  // Without whole quads the loads are many: each is stored before the next, to keep the code short.
  static constexpr bool held = VEC || W == 1;
  Octet<T> o[held ? passes : 1];
  const T* base;
  const float* factor;
  int64_t ld;
  const int* at;
  int D;
  __device__ __forceinline__ Stage(const void* b, int64_t l, const int* t, int d, const float* f = nullptr)
      : base(static_cast<const T*>(b)), factor(f), ld(l), at(t), D(d) {}
  static __device__ __forceinline__ void place(int pass, int& row, int& e0) {
    if constexpr (W == 1) {
      row = threadIdx.x & 31;
      e0 = 16 * pass + 8 * ((threadIdx.x >> 5) & 1);
    } else {
      const int idx = pass * 64 * W + (int)threadIdx.x;
      row = idx / per;
      e0 = (idx - row * per) * 8;
    }
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
    if (row < R) {
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

// Left operand whose rows are rows of LDS: lane (i, h) reads values k + 8h.. of row `row` + i.
template <int P, int DC, int R>
__device__ __forceinline__ void rows_frag(const uint16_t* s, int row, int k, bf16x8 (&f)[P]) {
  constexpr int LD = row_len(DC), plane = R * LD;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < P; ++i)
    f[i] = *reinterpret_cast<const bf16x8*>(s + i * plane + (row + (lane & 31)) * LD + k + 8 * (lane >> 5));
}

// The same, of rows that a block of one wave holds in its registers.
template <typename T, int DC, int R, int W, bool VEC>
__device__ __forceinline__ void left_rows(const Stage<T, DC, R, W, VEC>& st, const uint16_t* s, int row, int c,
                                          bf16x8 (&f)[pieces<T>()]) {
  if constexpr (W == 1)
    st.o[c].planes(f);
  else
    rows_frag<pieces<T>(), DC, R>(s, row, 16 * c, f);
}

// Left operand whose rows are columns d + 0..31 of LDS and whose reductions are
// LDS rows row + 4h + 0..3 and row + 8 + 4h + 0..3.  Each group of 16 lanes turns
// 4 rows x 16 columns: lane l supplies the address of four columns of row l / 4
// and receives column l of the four rows.
template <int P, int DC, int R>
__device__ __forceinline__ void cols_frag(const uint16_t* s, int row, int d, bf16x8 (&f)[P]) {
  constexpr int LD = row_len(DC), plane = R * LD;
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  const int lane = threadIdx.x & 63, l = lane & 15;
  const uint16_t* p = s + (row + 4 * (lane >> 5) + (l >> 2)) * LD + d + 16 * ((lane >> 4) & 1) + 4 * (l & 3);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + i * plane));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + i * plane + 8 * LD));
    f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// ---- rows of graphs ---------------------------------------------------------------

// The rows of tile `t` of M = 1 << shift rows.  Graph g's first tile is
// floor(first row / M) + g, which leaves every graph enough tile numbers, so that
// floor(N / M) + G tiles cover any split of the rows and nothing waits for the
// host.  The graph is found by a search with 64 probes per step.
struct Tile {
  int g;
  int64_t row0;  // first row
  int rows;      // rows of the tile that are in the graph
};
__device__ __forceinline__ int64_t clamp_row(int32_t v, int64_t N) { return v < 0 ? 0 : v > N ? N : v; }
__device__ __forceinline__ bool find_tile(const int32_t* off, int G, int64_t N, int shift, int64_t t, Tile& o) {
  const int64_t M = int64_t(1) << shift;
  int64_t b = 0, e = N, first = 0;
  o.g = 0;
  if (off) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = G;  // the last graph of [lo, lo + n) that starts at or before t
    while (true) {
      const int step = (n + 63) >> 6;
      const int i = lane * step;
      const int g = lo + (i < n ? i : 0);
      const uint64_t m = __ballot(i < n && (clamp_row(off[g], N) >> shift) + g <= t);
      const int c = __popcll(m);
      if (c == 0) return false;  // before the first graph
      lo += (c - 1) * step;
      n = min(step, n - (c - 1) * step);
      if (step == 1) break;
    }
    o.g = __builtin_amdgcn_readfirstlane(lo);
    b = clamp_row(off[o.g], N);
    e = clamp_row(off[o.g + 1], N);
    first = (b >> shift) + o.g;
    if (t < first) return false;  // (offsets that decrease)
  }
  o.row0 = b + ((t - first) << shift);
  if (o.row0 >= e) return false;
  o.rows = (int)(e - o.row0 < M ? e - o.row0 : M);
  return true;
}

// Rows [b, e) of graph g's other side, cut to part `part` of `nsplit` (whole tiles of R rows each).
template <int R>
__device__ __forceinline__ void other_rows(const int32_t* off, int g, int64_t N, int part, int nsplit, int64_t& b,
                                           int64_t& e) {
  b = 0;
  e = N;
  if (off) {
    b = clamp_row(off[g], N);
    e = clamp_row(off[g + 1], N);
  }
  if (nsplit > 1) {
    const int64_t len = e > b ? e - b : 0;
    const int64_t per = ((len + nsplit - 1) / nsplit + R - 1) / R * R;
    const int64_t pb = b + per * part;
    e = pb + per < e ? pb + per : e;
    b = pb;
  }
}

// Row of accumulator register r: columns run along the lanes.
__device__ __forceinline__ int acc_row(int r) { return 8 * (r >> 2) + 4 * ((threadIdx.x >> 5) & 1) + (r & 3); }

// The other half wave's value of the same column.
__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  // r[0]: lower half's values in both halves, r[1]: the upper half's
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}
__device__ __forceinline__ float half_sum(float v) { return v + other_half(v); }

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// tanh, accurate relative to its value: the odd series below 1/4 (the next term
// is below 2^-26 there), (1 - e) / (1 + e) with e = exp(-2 |x|) above.
__device__ __forceinline__ float tanh_acc(float x) {
  const float a = fabsf(x), t = x * x;
  const float e = exp2_fast(-2.f * kLog2e * a);
  const float big = copysignf((1.f - e) * __builtin_amdgcn_rcpf(1.f + e), x);
  const float small =
      x + x * t * (-1.f / 3.f + t * (2.f / 15.f + t * (-17.f / 315.f + t * (62.f / 2835.f - t * (1382.f / 155925.f)))));
  return a < 0.25f ? small : big;
}

// Per-row fp32 values of the other side in LDS (positions: one plane per
// coordinate), loaded ahead like the rows.
template <int R, int W>
struct StagePos {
  static constexpr int passes = (3 * R + 64 * W - 1) / (64 * W);
  float v[passes];
  __device__ __forceinline__ void load(const float* pos, int64_t row0, int valid) {
#pragma unroll
    for (int p = 0; p < passes; ++p) {
      const int i = p * 64 * W + (int)threadIdx.x;
      v[p] = i < 3 * valid ? pos[row0 * 3 + i] : 0.f;
    }
  }
  __device__ __forceinline__ void put(float* s) const {
#pragma unroll
    for (int p = 0; p < passes; ++p) {
      const int i = p * 64 * W + (int)threadIdx.x;
      if (i < 3 * R) s[(i % 3) * R + i / 3] = v[p];
    }
  }
};

// A column's (lane's) side of the distance bias.
struct Place {
  float x, y, z, slope2;  // position, slope in units of log2
};
__device__ __forceinline__ Place place_of(const AttnArgs& a, const float* pos, int64_t row, int h) {
  Place p = {0.f, 0.f, 0.f, 0.f};
  if (a.slope) {
    p.x = pos[row * 3];
    p.y = pos[row * 3 + 1];
    p.z = pos[row * 3 + 2];
    p.slope2 = a.slope[h] * kLog2e;
  }
  return p;
}

// A column's sums for the gradients of slopes and positions.
struct BiasSums {
  float sd = 0.f, s = 0.f, pd = 0.f;  // of dS d, of dS, of P d
  float x = 0.f, y = 0.f, z = 0.f;    // of dS (r - r') / d
};

// Scores of a 32 x 32 tile.  CAP or BIAS: in units of log2; otherwise as they
// are, to be multiplied by scale log2(e).
template <bool CAP, bool BIAS, int R>
__device__ __forceinline__ void score_tile(const AttnArgs& a, floatx16& s, const float* spos, int row, const Place& p) {
  const float in = CAP ? a.scale / a.cap : 0.f, out = a.cap * kLog2e, c = a.scale * kLog2e;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    floatx4 x, y, z;
    if constexpr (BIAS) {
      const int at = row + 8 * q + 4 * ((threadIdx.x >> 5) & 1);
      x = *reinterpret_cast<const floatx4*>(spos + at);
      y = *reinterpret_cast<const floatx4*>(spos + R + at);
      z = *reinterpret_cast<const floatx4*>(spos + 2 * R + at);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = s[4 * q + e];
      if constexpr (CAP) v = tanh_acc(v * in) * out;
      if constexpr (BIAS) {
        const float dx = p.x - x[e], dy = p.y - y[e], dz = p.z - z[e];
        const float dist = __builtin_amdgcn_sqrtf(fmaf(dx, dx, fmaf(dy, dy, dz * dz)));
        v = CAP ? fmaf(-p.slope2, dist, v) : fmaf(v, c, -p.slope2 * dist);
      }
      s[4 * q + e] = v;
    }
  }
}

// The tile of the backward: s (scores as products) -> weights against the
// rows' references `ref(r)`, ds (dP) -> dS = P (dP - delta(r)), in the end with the
// cap's factor; adds to the column's sums where there is a bias.
template <bool CAP, bool BIAS, int R, typename REF, typename DELTA>
__device__ __forceinline__ void grad_tile(const AttnArgs& a, floatx16& s, floatx16& ds, const float* spos, int row,
                                          const Place& p, BiasSums& b, REF ref, DELTA delta) {
  const float in = CAP ? a.scale / a.cap : 0.f, out = a.cap * kLog2e, c = a.scale * kLog2e;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = row + 8 * q + 4 * ((threadIdx.x >> 5) & 1);
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
      float th = 0.f, v;
      if constexpr (CAP) th = tanh_acc(s[r] * in);
      float dx, dy, dz, d2, over;
      if constexpr (BIAS) {
        dx = p.x - x[e], dy = p.y - y[e], dz = p.z - z[e];
        d2 = fmaf(dx, dx, fmaf(dy, dy, dz * dz));
        over = d2 > 0.f ? __builtin_amdgcn_rsqf(d2) : 0.f;
        const float dist = d2 * over;
        v = CAP ? fmaf(th, out, -m4[e]) : fmaf(s[r], c, -m4[e]);
        v = exp2_fast(fmaf(-p.slope2, dist, v));
        const float g = v * (ds[r] - d4[e]);
        b.sd = fmaf(g, dist, b.sd);
        b.s += g;
        b.pd = fmaf(v, dist, b.pd);
        const float w = g * over;
        b.x = fmaf(w, dx, b.x);
        b.y = fmaf(w, dy, b.y);
        b.z = fmaf(w, dz, b.z);
        ds[r] = g;
      } else {
        v = exp2_fast(CAP ? fmaf(th, out, -m4[e]) : fmaf(s[r], c, -m4[e]));
        ds[r] = v * (ds[r] - d4[e]);
      }
      if constexpr (CAP) ds[r] *= fmaf(-th, th, 1.f);
      s[r] = v;
    }
  }
}

// f(cap, bias) with the two as compile-time constants.
template <typename F>
__device__ __forceinline__ void with_kind(const AttnArgs& a, F f) {
  if (a.cap > 0.f) {
    if (a.slope)
      f(std::true_type{}, std::true_type{});
    else
      f(std::true_type{}, std::false_type{});
  } else {
    if (a.slope)
      f(std::false_type{}, std::true_type{});
    else
      f(std::false_type{}, std::false_type{});
  }
}

// Writes a lane's column of a transposed result (rows: head elements) to its row of features.
template <int DC, bool VEC>
__device__ __forceinline__ void put_column(const floatx16 (&acc)[DC / 32], float f, const int* at, int D, float* row) {
#pragma unroll
  for (int t = 0; t < DC / 32; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e0 = 32 * t + 8 * q + 4 * ((threadIdx.x >> 5) & 1);
      if constexpr (VEC) {
        if (e0 < D) {
          floatx4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[t][4 * q + e] * f;
          *reinterpret_cast<floatx4_any*>(row + at[e0]) = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e0 + e < D) row[at[e0 + e]] = acc[t][4 * q + e] * f;
      }
    }
}
template <int DC, bool VEC>
__device__ __forceinline__ void put_column(const floatx16 (&acc)[DC / 32], float f, const int* at, int D,
                                           uint16_t* row) {
#pragma unroll
  for (int t = 0; t < DC / 32; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e0 = 32 * t + 8 * q + 4 * ((threadIdx.x >> 5) & 1);
      uint16_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = __builtin_bit_cast(uint16_t, (__bf16)(acc[t][4 * q + e] * f));
      if constexpr (VEC) {
        if (e0 < D)
          *reinterpret_cast<u32x2_any*>(row + at[e0]) =
              (u32x2){b[0] | ((uint32_t)b[1] << 16), b[2] | ((uint32_t)b[3] << 16)};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e0 + e < D) row[at[e0 + e]] = b[e];
      }
    }
}

template <int N>
__device__ __forceinline__ void zero(floatx16 (&acc)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
}

// Which part, head and tile a block works on: the tiles of a head run together
// on an XCD, whose L2 then holds that head's other side.
struct Work {
  int part, h;
  int64_t tile, item;
};
__device__ __forceinline__ bool find_work(const AttnArgs& a, Work& w) {
  const int64_t items = a.tiles * a.H * a.nsplit;
  w.item = xcd_item(blockIdx.x, gridDim.x);
  if (w.item >= items) return false;
  const int64_t ph = w.item / a.tiles;
  w.tile = w.item - ph * a.tiles;
  w.part = (int)(ph / a.H);
  w.h = (int)(ph - (int64_t)w.part * a.H);
  return true;
}

// Waves per SIMD that the registers are held to: two where a wave's operands and
// sums leave room (one hides the latency of the other), else one.
constexpr int waves_for(int regs) { return regs <= 200 ? 2 : 1; }

// ---- forward ----------------------------------------------------------------------

// The reference that the weights are taken against moves only when a score passes
// it by more than 2^kSlack, so that the sums are rarely scaled again; weights
// stay below 2^kSlack, which fp32 sums and bf16 pieces hold as well as below 1.
constexpr float kSlack = 8.f;

template <typename T, int DC, int W, int PP, bool VEC>
__global__ __launch_bounds__(64 * W, waves_for(DC / 4 * pieces<T>() + DC / 2 + 60)) void forward_kernel(const AttnArgs a) {
  constexpr int P = pieces<T>(), R = W == 4 && DC <= 64 ? 64 : 32, LD = row_len(DC), NT = DC / 32, NC = DC / 16;
  constexpr int kShift = W == 4 ? 7 : 5;
  __shared__ __align__(16) uint16_t sk[W == 1 ? 8 : P * R * LD], sv[P * R * LD];
  __shared__ int at_qk[DC], at_v[DC];
  __shared__ __align__(16) float spos[3 * R];
  Work w;
  Tile t;
  if (!find_work(a, w) || !find_tile(a.qo, a.G, a.Nq, kShift, w.tile, t)) return;
  fill_table<DC>(at_qk, a.sqk, w.h);
  fill_table<DC>(at_v, a.sv, w.h);
  __syncthreads();
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int col = (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool mine = col < t.rows;
  const int64_t query = t.row0 + min(col, t.rows - 1);
  const int Dqk = a.sqk.D, Dv = a.sv.D;
  const bool bias = a.slope != nullptr;
  int64_t kb, ke;
  other_rows<R>(a.ko, t.g, a.Nk, w.part, a.nsplit, kb, ke);
  Stage<T, DC, R, W, VEC> rk(a.k, a.ldk, at_qk, Dqk), rv(a.v, a.ldv, at_v, Dv);
  StagePos<R, W> rp;
  auto load = [&](int64_t k0) {
    const int valid = (int)(ke - k0 < R ? ke - k0 : R);
    rk.load(k0, valid);
    rv.load(k0, valid);
    if (bias) rp.load(a.kpos, k0, valid);
  };
  if (kb < ke) load(kb);
  bf16x8 q[NC][P];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    Octet<T> o;
    o.template load<VEC>(static_cast<const T*>(a.q) + query * a.ldq, at_qk, 16 * c + 8 * half, Dqk);
    o.planes(q[c]);
  }
  const Place place = place_of(a, a.qpos, query, w.h);
  // scores are multiplied by this on their way into the exponent
  const bool raw = !bias && !(a.cap > 0.f);
  const float unit = raw ? a.scale * kLog2e : 1.f;
  floatx16 acc[NT];
  zero(acc);
  float m = -INFINITY, l = 0.f;
  for (int64_t k0 = kb; k0 < ke; k0 += R) {
    const int valid = (int)(ke - k0 < R ? ke - k0 : R);
    __syncthreads();
    if constexpr (W == 4) rk.put(sk, k0, valid);
    rv.put(sv, k0, valid);
    if (bias) rp.put(spos);
    __syncthreads();
    if (W == 4 && k0 + R < ke) {
      load(k0 + R);
      __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
    }
    for (int sub = 0; sub < (W == 1 ? 1 : valid); sub += 32) {
      floatx16 s;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        bf16x8 f[P];
        left_rows(rk, sk, sub, c, f);
        mul<P, P>(f, q[c], s);
      }
      if (W == 1 && k0 + R < ke) load(k0 + R);
      if (!raw) with_kind(a, [&](auto cap, auto bs) {
        score_tile<decltype(cap)::value, decltype(bs)::value, R>(a, s, spos, sub, place);
      });
      if (valid - sub < 32)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (sub + acc_row(r) >= valid) s[r] = unit < 0.f ? INFINITY : -INFINITY;
      float top = s[0];
      if (unit < 0.f) {
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fminf(top, s[r]);
      } else {
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
      }
      top *= unit;
      top = fmaxf(top, other_half(top));
      if (__any(top > m + kSlack)) {
        const float next = fmaxf(m, top);
        const float f = m == -INFINITY ? 0.f : exp2_fast(m - next);
        l *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[n][r] *= f;
        m = next;
      }
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[r] = exp2_fast(fmaf(s[r], unit, -ref));
        l += s[r];
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        float pv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pv[e] = s[8 * kk + e];
        bf16x8 p[PP];
        split<PP>(pv, p);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf16x8 f[P];
          cols_frag<P, DC, R>(sv, sub + 16 * kk, 32 * n, f);
          mul<P, PP>(f, p, acc[n]);
        }
      }
    }
  }
  l = half_sum(l);
  if (!mine) return;
  if (a.nsplit > 1) {
    const int64_t at = ((int64_t)w.part * a.H + w.h) * a.Nq + query;
    if (half == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
    put_column<DC, VEC>(acc, 1.f, at_v, Dv, a.part_o + ((int64_t)w.part * a.Nq + query) * a.sv.F);
    return;
  }
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
  if (a.stat && half == 0) {
    a.stat[(int64_t)w.h * a.Nq + query] = m;
    a.stat[(int64_t)(a.H + w.h) * a.Nq + query] = f;
  }
  if (a.out32) put_column<DC, VEC>(acc, f, at_v, Dv, a.out32 + query * a.sv.F);
  if (a.y_bf16)
    put_column<DC, VEC>(acc, f, at_v, Dv, static_cast<uint16_t*>(a.out) + query * a.sv.F);
  else
    put_column<DC, VEC>(acc, f, at_v, Dv, static_cast<float*>(a.out) + query * a.sv.F);
}

// A column's share of its position's gradient, per part and head.
__device__ __forceinline__ void put_pos(const AttnArgs& a, const Work& w, int64_t rows, int64_t row, bool mine,
                                        BiasSums& b, float f) {
  if (!a.part_pos) return;
  b.x = half_sum(b.x);
  b.y = half_sum(b.y);
  b.z = half_sum(b.z);
  if (!mine || (threadIdx.x & 32)) return;
  float* o = a.part_pos + (((int64_t)w.part * a.H + w.h) * rows + row) * 3;
  f *= -a.slope[w.h];
  o[0] = f * b.x;
  o[1] = f * b.y;
  o[2] = f * b.z;
}

// ---- gradient of the queries ----------------------------------------------------------

template <typename T, int DC, int W, bool VEC>
__global__ __launch_bounds__(64 * W, waves_for(DC / 4 * (pieces<T>() + 3) + DC / 2 + 80)) void grad_q_kernel(
    const AttnArgs a) {
  constexpr int P = pieces<T>(), R = W == 4 && DC <= 64 ? 64 : 32, LD = row_len(DC), NT = DC / 32, NC = DC / 16;
  constexpr int kShift = W == 4 ? 7 : 5;
  __shared__ __align__(16) uint16_t sk[P * R * LD], sv[W == 1 ? 8 : P * R * LD];
  __shared__ int at_qk[DC], at_v[DC];
  __shared__ __align__(16) float spos[3 * R];
  Work w;
  Tile t;
  if (!find_work(a, w) || !find_tile(a.qo, a.G, a.Nq, kShift, w.tile, t)) return;
  fill_table<DC>(at_qk, a.sqk, w.h);
  fill_table<DC>(at_v, a.sv, w.h);
  __syncthreads();
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int col = (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool mine = col < t.rows;
  const int64_t query = t.row0 + min(col, t.rows - 1);
  const int Dqk = a.sqk.D, Dv = a.sv.D;
  const bool bias = a.slope != nullptr;
  int64_t kb, ke;
  other_rows<R>(a.ko, t.g, a.Nk, w.part, a.nsplit, kb, ke);
  Stage<T, DC, R, W, VEC> rk(a.k, a.ldk, at_qk, Dqk), rv(a.v, a.ldv, at_v, Dv);
  StagePos<R, W> rp;
  auto load = [&](int64_t k0) {
    const int valid = (int)(ke - k0 < R ? ke - k0 : R);
    rk.load(k0, valid);
    rv.load(k0, valid);
    if (bias) rp.load(a.kpos, k0, valid);
  };
  if (kb < ke) load(kb);
  bf16x8 q[NC][P], g[NC][3];
  float delta = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    Octet<T> o;
    o.template load<VEC>(static_cast<const T*>(a.q) + query * a.ldq, at_qk, 16 * c + 8 * half, Dqk);
    o.planes(q[c]);
    Octet<float> go, y;
    go.template load<VEC>(a.go + query * a.sv.F, at_v, 16 * c + 8 * half, Dv);
    y.template load<VEC>(a.o + query * a.sv.F, at_v, 16 * c + 8 * half, Dv);
    go.planes(g[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) delta = fmaf(go.v[e], y.v[e], delta);
  }
  delta = half_sum(delta);
  if (mine && half == 0 && w.part == 0) a.delta[(int64_t)w.h * a.Nq + query] = delta;
  const float m = a.stat[(int64_t)w.h * a.Nq + query], inv = a.stat[(int64_t)(a.H + w.h) * a.Nq + query];
  const Place place = place_of(a, a.qpos, query, w.h);
  const floatx4 m4 = {m, m, m, m}, delta4 = {delta, delta, delta, delta};
  BiasSums sums;
  floatx16 acc[NT];
  zero(acc);
  for (int64_t k0 = kb; k0 < ke; k0 += R) {
    const int valid = (int)(ke - k0 < R ? ke - k0 : R);
    __syncthreads();
    rk.put(sk, k0, valid);
    if constexpr (W == 4) rv.put(sv, k0, valid);
    if (bias) rp.put(spos);
    __syncthreads();
    if (W == 4 && k0 + R < ke) {
      load(k0 + R);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int sub = 0; sub < (W == 1 ? 1 : valid); sub += 32) {
      floatx16 s, ds;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = ds[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        bf16x8 f[P];
        left_rows(rk, sk, sub, c, f);
        mul<P, P>(f, q[c], s);
        left_rows(rv, sv, sub, c, f);
        mul<P, 3>(f, g[c], ds);
      }
      if (W == 1 && k0 + R < ke) load(k0 + R);
      if (valid - sub < 32) {
        // keys that are not there: a weight of zero
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (sub + acc_row(r) >= valid) s[r] = ds[r] = 0.f;
        with_kind(a, [&](auto cap, auto bs) {
          grad_tile<decltype(cap)::value, decltype(bs)::value, R>(
              a, s, ds, spos, sub, place, sums,
              [&](int q4) {
                floatx4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = sub + acc_row(4 * q4 + e) < valid ? m : INFINITY;
                return v;
              },
              [&](int) { return delta4; });
        });
      } else {
        with_kind(a, [&](auto cap, auto bs) {
          grad_tile<decltype(cap)::value, decltype(bs)::value, R>(
              a, s, ds, spos, sub, place, sums, [&](int) { return m4; }, [&](int) { return delta4; });
        });
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        float pv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pv[e] = ds[8 * kk + e];
        bf16x8 p[3];
        split<3>(pv, p);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf16x8 f[P];
          cols_frag<P, DC, R>(sk, sub + 16 * kk, 32 * n, f);
          mul<P, 3>(f, p, acc[n]);
        }
      }
    }
  }
  put_pos(a, w, a.Nq, query, mine, sums, inv);
  if (a.part_slope) {
    // sum dS d = sum dS (d - mean d) as far as the sum of dS is zero, which it is but for
    // rounding: the join takes sum dS d - sum dS * sum P d, which does not see that rounding
    sums.sd = half_sum(sums.sd);
    sums.s = half_sum(sums.s);
    sums.pd = half_sum(sums.pd);
    if (mine && half == 0) {
      float* o = a.part_slope + (((int64_t)w.part * a.H + w.h) * a.Nq + query) * 3;
      o[0] = sums.sd * inv;
      o[1] = sums.s * inv;
      o[2] = sums.pd * inv;
    }
  }
  if (a.gq && mine) put_column<DC, VEC>(acc, a.scale * inv, at_qk, Dqk, a.gq + ((int64_t)w.part * a.Nq + query) * a.ldgq);
}

// ---- gradients of keys and values --------------------------------------------------------

// fp32 operands of more than 128 values leave no registers to hold the next rows in.
template <typename T, int DC>
constexpr bool kv_ahead() {
  return sizeof(T) == 2 || DC <= 128;
}

template <typename T, int DC, int W, bool VEC>
__global__ __launch_bounds__(64 * W, waves_for(DC / 4 * 2 * pieces<T>() + DC + 80)) void grad_kv_kernel(const AttnArgs a) {
  constexpr int P = pieces<T>(), R = W == 4 && DC <= 64 && P == 1 ? 64 : 32, LD = row_len(DC), NT = DC / 32, NC = DC / 16;
  constexpr int kShift = W == 4 ? 7 : 5;
  constexpr bool kAhead = W == 4 && kv_ahead<T, DC>();
  __shared__ __align__(16) uint16_t sq[P * R * LD], sg[3 * R * LD];
  __shared__ int at_qk[DC], at_v[DC];
  __shared__ __align__(16) float spos[3 * R], sl[R], sd[R];
  Work w;
  Tile t;
  if (!find_work(a, w) || !find_tile(a.ko, a.G, a.Nk, kShift, w.tile, t)) return;
  fill_table<DC>(at_qk, a.sqk, w.h);
  fill_table<DC>(at_v, a.sv, w.h);
  __syncthreads();
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int col = (threadIdx.x >> 6) * 32 + (lane & 31);
  const bool mine = col < t.rows;
  const int64_t key = t.row0 + min(col, t.rows - 1);
  const int Dqk = a.sqk.D, Dv = a.sv.D;
  const bool bias = a.slope != nullptr;
  int64_t qb, qe;
  other_rows<R>(a.qo, t.g, a.Nq, w.part, a.nsplit, qb, qe);
  // rows of grad_out are taken times 1 / l, so that the weights need no factor of their own
  const float *ref = a.stat + (int64_t)w.h * a.Nq, *inv = ref + (int64_t)a.H * a.Nq, *delta = a.delta + (int64_t)w.h * a.Nq;
  Stage<T, DC, R, W, VEC> rq(a.q, a.ldq, at_qk, Dqk);
  Stage<float, DC, R, W, VEC> rg(a.go, a.sv.F, at_v, Dv, inv);
  StagePos<R, W> rp;
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
  if (kAhead && qb < qe) load(qb);
  bf16x8 k[NC][P], v[NC][P];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    Octet<T> o;
    o.template load<VEC>(static_cast<const T*>(a.k) + key * a.ldk, at_qk, 16 * c + 8 * half, Dqk);
    o.planes(k[c]);
    o.template load<VEC>(static_cast<const T*>(a.v) + key * a.ldv, at_v, 16 * c + 8 * half, Dv);
    o.planes(v[c]);
  }
  const Place place = place_of(a, a.kpos, key, w.h);
  BiasSums sums;
  floatx16 gv[NT], gk[NT];
  zero(gv);
  zero(gk);
  for (int64_t q0 = qb; q0 < qe; q0 += R) {
    const int valid = (int)(qe - q0 < R ? qe - q0 : R);
    __syncthreads();
    if constexpr (!kAhead) load(q0);
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
    for (int sub = 0; sub < (W == 1 ? 1 : valid); sub += 32) {
      floatx16 s, ds;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = ds[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        bf16x8 f[P], f3[3];
        left_rows(rq, sq, sub, c, f);
        mul<P, P>(f, k[c], s);
        left_rows(rg, sg, sub, c, f3);
        mul<3, P>(f3, v[c], ds);
      }
      with_kind(a, [&](auto cap, auto bs) {
        grad_tile<decltype(cap)::value, decltype(bs)::value, R>(
            a, s, ds, spos, sub, place, sums,
            [&](int q4) { return *reinterpret_cast<const floatx4*>(sl + sub + 8 * q4 + 4 * half); },
            [&](int q4) { return *reinterpret_cast<const floatx4*>(sd + sub + 8 * q4 + 4 * half); });
      });
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        float pv[8], dv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          pv[e] = s[8 * kk + e];
          dv[e] = ds[8 * kk + e];
        }
        bf16x8 p[3], dp[3];
        split<3>(pv, p);
        split<3>(dv, dp);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf16x8 f3[3], f[P];
          cols_frag<3, DC, R>(sg, sub + 16 * kk, 32 * n, f3);
          mul<3, 3>(f3, p, gv[n]);
          cols_frag<P, DC, R>(sq, sub + 16 * kk, 32 * n, f);
          mul<P, 3>(f, dp, gk[n]);
        }
      }
    }
  }
  put_pos(a, w, a.Nk, key, mine, sums, 1.f);
  if (!mine) return;
  if (a.gk) put_column<DC, VEC>(gk, a.scale, at_qk, Dqk, a.gk + ((int64_t)w.part * a.Nk + key) * a.ldgk);
  if (a.gv) put_column<DC, VEC>(gv, 1.f, at_v, Dv, a.gv + ((int64_t)w.part * a.Nk + key) * a.ldgv);
}

}  // namespace attn
}  // namespace tpconv
