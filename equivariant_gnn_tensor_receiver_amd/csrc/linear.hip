// Linear layer on node features with one weight matrix per group of nodes.
//
//   forward:          y[(v, m), c']  = sum_c x[(v, m), c] W_g[c][c']
//   input gradient:   gx[(v, m), c]  = sum_c' gy[(v, m), c'] W_g[c][c']
//   weight gradient:  gW_g[c][c']    = sum over the rows (v, m) of group g of x[(v, m), c] gy[(v, m), c']
//
// per pair of irreps of equal degree and parity; g is the group of node v.
// The nodes of a group are found through a stable sort of the nodes by group
// (lin_groups): a row tile belongs to one group and gathers its nodes' rows.
//
// Tiles without a count of the groups' tiles on the host: with M rows per tile
// (M a power of two), group g's first tile is floor(rows before g / M) + g.
// That leaves every group at least ceil(rows of g / M) tile numbers, so a
// launch of floor(rows / M) + G row tiles covers every split of the nodes, and
// a block finds its group by one comparison per group; the few tile numbers
// past a group's last row return at once.
//
// Products run on v_mfma_f32_32x32x16_bf16.  An fp32 operand is the exact sum
// of three bf16 values (8 + 8 + 8 bits, by truncation), and the products of
// the pieces whose ranks add up to at most 2 are added in fp32, smallest
// first.  What is left out, p1 q2 + p2 q1 + p2 q2 with |p1| < 2^-7 and |p2| <
// 2^-15 of the operand's leading power of two, is below 2^-21 of a term and has
// its sign (pieces by truncation, which keep the largest fp32 values finite).
// bf16 operands are one piece, so bf16 x bf16 takes one product, mixed types
// three, both exact; fp32 takes six.
//
// Measured (kernel times): 8192 nodes of 128x0e+128x1o+128x2e in fp32, 16
// groups: forward 37 us (2.4 GFLOP x 6 products: 390 TFLOP/s of the matrix
// cores, 2.1 TB/s), both gradients 49, their join 9.  The wave slots start
// together, so address setup, loads, splitting, products and stores follow one
// another over the whole chip, and no single one of them is the limit (leaving
// any one out saves 6 to 8 us).  8192 nodes of 1024x0e in bf16 to 2048x0e, 8
// groups, on one set of inputs: forward 65 us (34 GFLOP, 525 TFLOP/s; one LDS
// buffer and two barriers per chunk), both gradients 254 (69 GFLOP x 3
// products, 810 TFLOP/s; three waves per SIMD), bound by the splitting of the
// fp32 gradients into pieces beside the products.
#include "device_common.h"
#include "layers.h"
#include "timing.h"

#include <algorithm>
#include <type_traits>

namespace tpconv {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kCUs = 256;

// N fp32 values as three planes of packed bf16 (exact: truncation leaves 8 bits
// per piece); bf16 values are one plane already.
template <int N, typename V>
__device__ __forceinline__ void split3(const float (&v)[N], V (&p)[3]) {
#pragma unroll
  for (int t = 0; t < N / 2; ++t) {
    const uint32_t x0 = __float_as_uint(v[2 * t]), x1 = __float_as_uint(v[2 * t + 1]);
    const float r0 = v[2 * t] - __uint_as_float(x0 & 0xffff0000u);
    const float r1 = v[2 * t + 1] - __uint_as_float(x1 & 0xffff0000u);
    const float q0 = r0 - __uint_as_float(__float_as_uint(r0) & 0xffff0000u);
    const float q1 = r1 - __uint_as_float(__float_as_uint(r1) & 0xffff0000u);
    p[0][t] = __builtin_amdgcn_perm(x1, x0, 0x07060302);
    p[1][t] = __builtin_amdgcn_perm(__float_as_uint(r1), __float_as_uint(r0), 0x07060302);
    p[2][t] = __builtin_amdgcn_perm(__float_as_uint(q1), __float_as_uint(q0), 0x07060302);
  }
}

// The row tile (or row slot) `t` of M = 1 << shift rows, n rows per node: its
// group, the group's first position in `order`, its rows, and the tile's first
// row within the group.  Uniform over the wave; false past the group's rows.
struct Slot {
  int g;
  int64_t node0, rows, row0;
};
__device__ __forceinline__ bool find_slot(const int32_t* offsets, int G, int64_t N, int n, int shift, bool by_row,
                                          int64_t t, Slot& s) {
  if (!offsets) {
    s = {0, 0, N * n, t << shift};
    return s.row0 < s.rows;
  }
  const int lane = threadIdx.x & 63;
  // lane l looks at group base + l; the last group that starts at or before t
  // is the tile's (group 0 starts at tile 0), its ends are in two lanes
  int64_t o0 = 0, o1 = 0;
  int32_t before_last = 0;
  for (int base = 0; base <= G; base += 64) {
    const int g = base + lane;
    const int32_t off = offsets[g <= G ? g : G];
    const int64_t start = (int64_t)off * n;
    const uint64_t mask = __ballot(g < G && (by_row ? start : (start >> shift) + g) <= t);
    const int count = __popcll(mask);
    if (count < 64) {
      s.g = base + count - 1;
      o0 = count > 0 ? __builtin_amdgcn_readlane(off, count - 1) : before_last;
      o1 = __builtin_amdgcn_readlane(off, count);
      break;
    }
    before_last = __builtin_amdgcn_readlane(off, 63);
  }
  s.node0 = o0;
  s.rows = (o1 - o0) * n;
  if (by_row) {
    s.row0 = t - o0 * n;
    return s.row0 < s.rows && (s.row0 & ((int64_t(1) << shift) - 1)) == 0;
  }
  s.row0 = (t - (((o0 * n) >> shift) + s.g)) << shift;
  return s.row0 < s.rows;
}

// The weight gradient's partial sums of a group that starts at `row0` of `rows`.  Only groups of several
// slots have any, that is of r > M = 1 << shift rows: ceil(r / M) of them, and floor(2 r / M) is at least as
// many, so with fewer whole slots than groups floor(2 row0 / M) is a free place to start; else the slot's
// own number is.  (1024 x 2048 weights of 64 groups: 8 MiB for 100 nodes; a place for every slot took 0.5 GiB.)
__host__ __device__ inline int64_t first_part(int64_t rows, int64_t row0, int g, int G, int shift) {
  const bool half = (rows >> shift) < G;
  return (row0 << half >> shift) + (half ? 0 : g);
}

// The job of a block: the last one whose first tile is at or before it, one lane per job.
template <typename J>
__device__ __forceinline__ int find_job(const J* job, int njobs, int64_t tile) {
  static_assert(kMaxLinBlocks <= 64 && kMaxGroups <= 64, "one lane per job");
  const int lane = threadIdx.x & 63;
  return __popcll(__ballot(lane < njobs && job[lane < njobs ? lane : 0].first_tile <= tile)) - 1;
}

__device__ __forceinline__ int64_t div_rows(int64_t r, int n) {
  return n == 1 ? r : n == 3 ? r / 3 : n == 5 ? r / 5 : r / 7;
}

// Wide accesses at any element's address (the hardware needs no more alignment).
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight values along the reduction of one row: p[k..k+8), as loaded.  Runs past
// `len` read on into the memory behind the row (a run wholly past it reads the
// row's start) and mask_run8 zeroes what they got before use, so every load is
// wide, issued unconditionally, and can stay in flight while the previous chunk
// is multiplied.  Blocks that could read past the tensor's `end` that way (not
// WIDE) take the elements of such a run one by one.  WIDE is a compile-time
// copy of the main loop: with the choice made at every load the compiler waits
// for the loads in flight where the two ways meet (force-sized forward 41 -> 52 us).
template <bool WIDE>
__device__ __forceinline__ void load_run8(const float* p, int k, int len, const float* end, float (&v)[8]) {
  const float* q = p + (k < len ? k : 0);
  if (WIDE || q + 8 <= end) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const floatx4 x = *reinterpret_cast<const floatx4_any*>(q + 4 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = x[e];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[min(k + j, len - 1)];
  }
}
template <bool WIDE>
__device__ __forceinline__ void load_run8(const uint16_t* p, int k, int len, const uint16_t* end, u32x4& v) {
  const uint16_t* q = p + (k < len ? k : 0);
  if (WIDE || q + 8 <= end) {
    v = *reinterpret_cast<const u32x4_any*>(q);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = (uint32_t)p[min(k + 2 * j, len - 1)] | ((uint32_t)p[min(k + 2 * j + 1, len - 1)] << 16);
  }
}
// Zeroes the values j >= left.
__device__ __forceinline__ void mask_run8(float (&v)[8], int left) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? v[j] : 0.f;
}
__device__ __forceinline__ void mask_run8(u32x4& v, int left) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = 2 * j + 1 < left ? v[j] : 2 * j < left ? v[j] & 0xffffu : 0u;
}

template <typename T>
struct Planes;
template <>
struct Planes<float> {
  static constexpr int count = 3;
};
template <>
struct Planes<uint16_t> {
  static constexpr int count = 1;
};

// Operands in LDS, one plane after the other, in the layout they come in:
//   by rows:    [row][reduction], for operands whose reduction is contiguous in
//               memory; rows padded by 16 bytes, so that 16-byte reads of 16
//               rows touch every bank once;
//   by columns: [reduction][row], for operands whose rows are contiguous; they
//               are turned by the LDS reads (run_of_columns), and padded so
//               that the four rows of 32 bytes of such a read do not meet.
template <bool COLS, int ROWS, int KC>
struct Layout {
  static constexpr int LD = !COLS ? KC + 8 : ROWS == 128 ? 144 : ROWS == 64 ? 72 : 48;
  static constexpr int plane = (COLS ? KC : ROWS) * LD;
};

// The values one thread loads of an operand for one chunk.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float v[8];
};
template <>
struct Raw8<uint16_t> {
  u32x4 v;
};

// RunPart: operands by rows; eight reductions of a row at a time.
template <typename T, int ROWS, int KC>
struct RunPart {
  using L = Layout<false, ROWS, KC>;
  static constexpr bool kCols = false;
  static constexpr int kPer = KC / 8;                        // threads per row
  static constexpr int kPasses = (ROWS * kPer + kThreads - 1) / kThreads;
  static constexpr bool kWhole = ROWS * kPer >= kThreads;    // else the first threads alone
  Raw8<T> raw[kPasses];
  static __device__ __forceinline__ bool mine() { return kWhole || (int)threadIdx.x < ROWS * kPer; }
  static __device__ __forceinline__ int row(int p) { return p * (kThreads / kPer) + (int)threadIdx.x / kPer; }
  static __device__ __forceinline__ int k() { return ((int)threadIdx.x % kPer) * 8; }
  __device__ __forceinline__ void put(uint16_t* s, int left) {
    if (!mine()) return;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      if (left < KC) mask_run8(raw[p].v, left - k());  // `left` is uniform
      uint16_t* at = s + row(p) * L::LD + k();
      if constexpr (sizeof(T) == 4) {
        u32x4 pl[3];
        split3(raw[p].v, pl);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x4*>(at + i * L::plane) = pl[i];
      } else {
        *reinterpret_cast<u32x4*>(at) = raw[p].v;
      }
    }
  }
};

// ColPart: operands by columns; 16 bytes of neighbouring columns of one reduction at a time.
template <typename T, int ROWS, int KC>
struct ColPart {
  using L = Layout<true, ROWS, KC>;
  static constexpr bool kCols = true;
  static constexpr int kUnit = 16 / sizeof(T);
  static constexpr int kPer = ROWS / kUnit;          // threads per reduction
  static constexpr int kStep = kThreads / kPer;      // reductions per pass
  static constexpr bool kWhole = KC >= kStep;        // else the first threads alone
  static constexpr int kPasses = kWhole ? KC / kStep : 1;
  static_assert(!kWhole || KC % kStep == 0, "whole passes");
  u32x4 raw[kPasses];
  static __device__ __forceinline__ bool mine() { return kWhole || (int)threadIdx.x < KC * kPer; }
  static __device__ __forceinline__ int col() { return ((int)threadIdx.x % kPer) * kUnit; }
  static __device__ __forceinline__ int k(int p) { return p * kStep + (int)threadIdx.x / kPer; }
  // The columns c.. of the row at p of `cols` columns: those past it are never
  // stored and take what follows in memory (or the row's start).
  template <bool WIDE>
  __device__ __forceinline__ void load(int pass, const T* p, int c, int cols, const T* end) {
    const T* q = p + (c < cols ? c : 0);
    if (WIDE || q + kUnit <= end) {
      raw[pass] = *reinterpret_cast<const u32x4_any*>(q);
    } else {
      u32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < kUnit; ++e) {
        const T x = p[min(c + e, cols - 1)];
        if constexpr (sizeof(T) == 4)
          v[e] = __builtin_bit_cast(uint32_t, x);
        else
          v[e >> 1] |= (uint32_t)x << (16 * (e & 1));
      }
      raw[pass] = v;
    }
  }
  __device__ __forceinline__ void put(uint16_t* s, int left) {
    if (!mine()) return;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      u32x4 v = raw[p];
      if (left < KC && k(p) >= left) v = (u32x4){0, 0, 0, 0};
      uint16_t* at = s + k(p) * L::LD + col();
      if constexpr (sizeof(T) == 4) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
        u32x2 pl[3];
        split3(f, pl);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x2*>(at + i * L::plane) = pl[i];
      } else {
        *reinterpret_cast<u32x4*>(at) = v;
      }
    }
  }
};

// A lane's eight reductions k.. of its row of the 32-row tile at `row`.
template <typename L, bool COLS>
__device__ __forceinline__ bf16x8 fragment(const uint16_t* s, int row, int k) {
  const int lane = threadIdx.x & 63, h = lane >> 5;
  if constexpr (!COLS) {
    return *reinterpret_cast<const bf16x8*>(s + (row + (lane & 31)) * L::LD + k + 8 * h);
  } else {
    // each group of 16 lanes turns 4 reductions x 16 rows: lane l supplies the address of four
    // rows of reduction l / 4 and receives row l of the four
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int l = lane & 15;
    const uint16_t* p = s + (k + 8 * h + (l >> 2)) * L::LD + row + 16 * ((lane >> 4) & 1) + 4 * (l & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * L::LD));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// acc += A B over the k16 steps of this wave from the staged planes.
template <int PA, int PB, int MT, int NT, typename A, typename B>
__device__ __forceinline__ void multiply(const uint16_t* sa, const uint16_t* sb, int m0, int n0, int k0, int steps,
                                         floatx16 (&acc)[MT][NT]) {
  for (int st = 0; st < steps; ++st) {
    const int k = k0 + 16 * st;
    bf16x8 fa[PA][MT], fb[PB][NT];
#pragma unroll
    for (int p = 0; p < PA; ++p)
#pragma unroll
      for (int t = 0; t < MT; ++t) fa[p][t] = fragment<typename A::L, A::kCols>(sa + p * A::L::plane, m0 + 32 * t, k);
#pragma unroll
    for (int p = 0; p < PB; ++p)
#pragma unroll
      for (int t = 0; t < NT; ++t) fb[p][t] = fragment<typename B::L, B::kCols>(sb + p * B::L::plane, n0 + 32 * t, k);
#pragma unroll
    for (int rank = 2; rank >= 0; --rank)
#pragma unroll
      for (int p = 0; p < PA; ++p)
#pragma unroll
        for (int q = 0; q < PB; ++q)
          if (p + q == rank)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
              for (int b = 0; b < NT; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[p][a], fb[q][b], acc[a][b], 0, 0, 0);
  }
}

// Row of accumulator register r (32x32 tiles): columns run along the lanes.
__device__ __forceinline__ int acc_row(int r) { return 8 * (r >> 2) + 4 * ((threadIdx.x >> 5) & 1) + (r & 3); }

__device__ __forceinline__ void store_out(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_out(uint16_t* p, int64_t i, float v) {
  p[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Tile shapes.  A block of four waves computes BM x BN; with KS = 1 its waves
// take WM x WN each, with KS = 4 every wave takes a quarter of the reduction of
// the whole tile and the sums are added in order through LDS.
// AHEAD chunks of loads are in flight: one in the wide shapes (two or three
// changed nothing for fp32 and slowed the bf16 experts), more where few blocks
// wait for memory: four bf16 rows over 64 matrices of 1024 x 2048 took 16.3 us
// with one and take 10.0 with the chunks of the shape for few rows.
template <int BM_, int BN_, int WM_, int WN_, int KS_, int KC_, int AHEAD_ = 1>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KS = KS_, KC = KC_, kAhead = AHEAD_;
  static constexpr int MT = WM / 32, NT = WN / 32;
  static_assert((BM / WM) * (BN / WN) * KS == kThreads / 64, "four waves");
};

constexpr int max_int(int a, int b) { return a > b ? a : b; }

// LDS bytes: the operands' planes (later the partial sums of KS > 1) and the
// tables of row addresses.
template <typename S, int PA, int PB, typename A, typename B>
constexpr int plane_bytes() {
  return max_int((PA * A::L::plane + PB * B::L::plane) * 2, (S::KS - 1) * S::BM * S::BN * 4);
}
constexpr int kRowTable = 256;  // weight gradient: rows of a slot whose addresses are in LDS at a time
// The operands' parts: x or gy by rows, W by rows or columns; both by columns in the weight gradient.
template <typename S, typename TI, typename TW, bool WT>
struct RowsParts {
  using A = RunPart<TI, S::BM, S::KC>;
  using B = std::conditional_t<WT, RunPart<TW, S::BN, S::KC>, ColPart<TW, S::BN, S::KC>>;
  static constexpr int planes = plane_bytes<S, Planes<TI>::count, Planes<TW>::count, A, B>();
  static constexpr int lds = planes + 2 * S::BM * 4;
};
template <typename S, typename TX>
struct GwParts {
  using A = ColPart<TX, S::BM, S::KC>;
  using B = ColPart<float, S::BN, S::KC>;
  static constexpr int planes = plane_bytes<S, Planes<TX>::count, 3, A, B>();
  static constexpr int lds = planes + 2 * kRowTable * 8;
};

// Adds the waves' sums of KS > 1 in order; the result is wave 0's.
template <typename S>
__device__ __forceinline__ void join_waves(floatx16 (&acc)[S::MT][S::NT], char* smem) {
  if constexpr (S::KS > 1) {
    static_assert(S::MT == 1 && S::NT == 1, "one tile per wave");
    float(*part)[S::BM * S::BN] = reinterpret_cast<float(*)[S::BM * S::BN]>(smem);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (wave > 0)
#pragma unroll
      for (int r = 0; r < 16; ++r) part[wave - 1][r * 64 + lane] = acc[0][0][r];
    __syncthreads();
    if (wave == 0)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        for (int w = 0; w < S::KS - 1; ++w) acc[0][0][r] += part[w][r * 64 + lane];
  }
}

template <typename S, typename TI, typename TW, typename TO, bool WT>
__device__ __forceinline__ void lin_rows(const LinRowsArgs& a, int64_t block, char* smem) {
  using Parts = RowsParts<S, TI, TW, WT>;
  using PartA = typename Parts::A;
  using PartB = typename Parts::B;
  constexpr int PA = Planes<TI>::count, PB = Planes<TW>::count, BM = S::BM, BN = S::BN, KC = S::KC;
  int32_t* s_node = reinterpret_cast<int32_t*>(smem + Parts::planes);
  int32_t* s_m = s_node + BM;
  uint16_t* sa = reinterpret_cast<uint16_t*>(smem);
  uint16_t* sb = sa + PA * PartA::L::plane;
  // consecutive tiles (the column tiles of one row tile, then its group's next
  // rows) run on one XCD and share its L2
  const int64_t tile = xcd_item(block, (a.tiles + 7) / 8 * 8);
  if (tile >= a.tiles) return;
  const LinJob& J = a.job[find_job(a.job, a.njobs, tile)];
  const int64_t lt = tile - J.first_tile;
  const int64_t tm = lt / J.tiles_n;
  const int n0 = (int)(lt - tm * J.tiles_n) * BN;
  Slot s;
  constexpr int kShift = BM == 128 ? 7 : BM == 64 ? 6 : 5;
  static_assert(BM == 1 << kShift, "row tile");
  if (!find_slot(a.offsets, a.G, a.N, J.n, kShift, J.by_row, tm, s)) return;
  const int tid = threadIdx.x, wave = tid >> 6;
  if (tid < BM) {
    const int64_t r = s.row0 + tid;
    const int64_t rr = min(r, s.rows - 1);  // rows past the end repeat the last one and are not stored
    const int64_t p = div_rows(rr, J.n);
    const int32_t node = a.order ? a.order[s.node0 + p] : (int32_t)p;
    s_node[tid] = node;
    s_m[tid] = r < s.rows ? (int32_t)(rr - p * J.n) : -1 - (int32_t)(rr - p * J.n);
  }
  __syncthreads();
  floatx16 acc[S::MT][S::NT];
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const TI* in = static_cast<const TI*>(a.in);
  const TW* Wg = static_cast<const TW*>(a.W) + s.g * a.w_per_group;
  const TI* in_end = in + a.N * a.F_in;
  const TW* w_end = static_cast<const TW*>(a.W) + a.G * a.w_per_group;

  constexpr int kAhead = S::kAhead;
  const TI* row_ptr[PartA::kPasses];
  int row_m[PartA::kPasses];
  // reads past a row could leave the tensor: rows at its end whose length is not a multiple of a run
  bool near_end = false, odd = false;
  for (int i = 0; i < J.nseg; ++i) {
    const LinSeg& G = a.seg[J.seg0 + i];
    const bool tail = G.len % 8 != 0;
    odd = odd || tail;
    if constexpr (WT)
      near_end = near_end || (tail && Wg + G.woff + (int64_t)min(n0 + BN, J.cols) * G.len + 8 > w_end);
    else
      near_end = near_end || (J.cols % 8 != 0 && n0 + BN > J.cols - 8 && Wg + G.woff + (int64_t)G.len * J.cols + 8 > w_end);
  }
#pragma unroll
  for (int p = 0; p < PartA::kPasses; ++p) {
    const int m = s_m[PartA::row(p) % BM];
    row_m[p] = m < 0 ? -1 - m : m;
    row_ptr[p] = in + (int64_t)s_node[PartA::row(p) % BM] * a.F_in;
    near_end = near_end || (odd && row_ptr[p] + a.F_in + 8 > in_end);
  }
  auto main_loop = [&](auto wide) {
    constexpr bool WIDE = decltype(wide)::value;
    PartA pa[kAhead];
    PartB pb[kAhead];
    // the next chunk to load and the one to multiply: segment and first reduction
    int lsi = 0, lk = 0, si = 0, k0 = 0;
    auto load = [&](int d) {
      if (lsi >= J.nseg) return;
      const LinSeg& G = a.seg[J.seg0 + lsi];
      const int k0 = lk;
      lk += KC;
      if (lk >= G.len) {
        lk = 0;
        ++lsi;
      }
#pragma unroll
      for (int p = 0; p < PartA::kPasses; ++p)
        if (PartA::mine())
          load_run8<WIDE>(row_ptr[p] + G.off + row_m[p] * G.len, k0 + PartA::k(), G.len, in_end, pa[d].raw[p].v);
      if constexpr (WT) {  // B(k, c') = W[c'][k]
        if (PartB::mine())
#pragma unroll
          for (int p = 0; p < PartB::kPasses; ++p)
            load_run8<WIDE>(Wg + G.woff + (int64_t)min(n0 + PartB::row(p), J.cols - 1) * G.len, k0 + PartB::k(), G.len,
                            w_end, pb[d].raw[p].v);
      } else {  // B(k, c') = W[k][c']
        if (PartB::mine())
#pragma unroll
          for (int p = 0; p < PartB::kPasses; ++p)
            pb[d].template load<WIDE>(p, Wg + G.woff + (int64_t)min(k0 + PartB::k(p), G.len - 1) * J.cols,
                                    n0 + PartB::col(), J.cols, w_end);
      }
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(d);
    while (si < J.nseg) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (si >= J.nseg) break;
        const int left = a.seg[J.seg0 + si].len - k0;
        pa[d].put(sa, left);
        pb[d].put(sb, left);
        __syncthreads();
        k0 += KC;
        if (left <= KC) {
          k0 = 0;
          ++si;
        }
        load(d);
        __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
        if constexpr (S::KS > 1) {
          const int kw = wave * (KC / S::KS);  // a wave without reductions left skips its products
          if (kw < left) multiply<PA, PB, S::MT, S::NT, PartA, PartB>(sa, sb, 0, 0, kw, KC / (16 * S::KS), acc);
        } else {
          constexpr int kCols = BN / S::WN;
          multiply<PA, PB, S::MT, S::NT, PartA, PartB>(sa, sb, (wave / kCols) * S::WM, (wave % kCols) * S::WN, 0, KC / 16,
                                                       acc);
        }
        __syncthreads();
      }
    }
  };
  if (__syncthreads_or(near_end))
    main_loop(std::false_type{});
  else
    main_loop(std::true_type{});
  join_waves<S>(acc, smem);
  if (S::KS > 1 && wave > 0) return;
  constexpr int kCols = S::KS > 1 ? 1 : BN / S::WN;
  const int mw = (wave / kCols) * S::WM, nw = (wave % kCols) * S::WN;
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = mw + 32 * i + acc_row(r), m = s_m[row];
      TO* out = static_cast<TO*>(a.out) + (int64_t)s_node[row] * a.F_out + J.off + (int64_t)m * J.cols;
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        const int col = n0 + nw + 32 * j + (tid & 31);
        if (m >= 0 && col < J.cols) store_out(out, col, acc[i][j][r]);
      }
    }
}

// Weight gradient: one BM x BN tile of gW_g over the rows of one slot.  A group
// with a single slot is written at once, others through partial sums that
// lin_gw_reduce_kernel adds in order.
template <typename S, typename TX>
__device__ __forceinline__ void lin_gw(const LinGwArgs& a, int64_t tile, char* smem) {
  using Parts = GwParts<S, TX>;
  using PartA = typename Parts::A;
  using PartB = typename Parts::B;
  constexpr int PA = Planes<TX>::count, PB = 3, BM = S::BM, BN = S::BN, KC = S::KC;
  int64_t* s_x = reinterpret_cast<int64_t*>(smem + Parts::planes);
  int64_t* s_y = s_x + kRowTable;
  uint16_t* sa = reinterpret_cast<uint16_t*>(smem);
  uint16_t* sb = sa + PA * PartA::L::plane;
  // every slot's tiles are shared out evenly over the XCDs (groups differ in
  // size, so whole slots per XCD would leave most of them waiting), each
  // XCD taking a run of them: the tiles of one or two column tiles of gy
  const LinGwJob& J = a.job[find_job(a.job, a.njobs, tile)];
  const int64_t lt = tile - J.first_tile;
  const int tiles_i = (J.mi + BM - 1) / BM, tiles = tiles_i * ((J.mo + BN - 1) / BN);
  const int64_t slot = lt / tiles;
  int ti = (int)(lt - slot * tiles);
  if (tiles % 8 == 0) ti = (ti & 7) * (tiles >> 3) + (ti >> 3);
  const int i0 = (ti % tiles_i) * BM, o0 = (ti / tiles_i) * BN;
  Slot s;
  if (!find_slot(a.offsets, a.G, a.N, J.n, a.rshift, J.by_row, slot, s)) return;
  const int rows = (int)min(s.rows - s.row0, int64_t(1) << a.rshift);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  floatx16 acc[S::MT][S::NT];
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const TX* x = static_cast<const TX*>(a.x) + J.xoff;
  const float* gy = a.gy + J.yoff;
  const TX* x_end = static_cast<const TX*>(a.x) + a.N * a.F_in;
  const float* y_end = a.gy + a.N * a.F_out;
  constexpr int kAhead = S::kAhead;
  // reads past a row could leave the tensors: multiplicities that are not a multiple of a unit and the
  // last nodes (a group's nodes ascend, so the slot's last row tells)
  bool near_end = false;
  if (J.mi % PartA::kUnit != 0 || J.mo % PartB::kUnit != 0) {
    const int64_t p = div_rows(s.row0 + rows - 1, J.n), left = a.N - 1 - (a.order ? a.order[s.node0 + p] : p);
    near_end = left * min(a.F_in, a.F_out) < 8;
  }
  auto main_loop = [&](auto wide) {
    constexpr bool WIDE = decltype(wide)::value;
    PartA pa[kAhead];
    PartB pb[kAhead];
    auto load = [&](int d, int r0) {
      if (r0 >= rows) return;
      if (r0 % kRowTable == 0) {  // the next rows' addresses (no thread reads the old ones any more)
        __syncthreads();
        for (int i = tid; i < kRowTable; i += kThreads) {
          const int64_t r = s.row0 + min(r0 + i, rows - 1);
          const int64_t p = div_rows(r, J.n);
          const int32_t m = (int32_t)(r - p * J.n);
          const int64_t node = a.order ? a.order[s.node0 + p] : p;
          s_x[i] = node * a.F_in + (int64_t)m * J.mi;
          s_y[i] = node * a.F_out + (int64_t)m * J.mo;
        }
        __syncthreads();
      }
      const int t0 = r0 % kRowTable;
      if (PartA::mine())
#pragma unroll
        for (int p = 0; p < PartA::kPasses; ++p)
          pa[d].template load<WIDE>(p, x + s_x[t0 + PartA::k(p)], i0 + PartA::col(), J.mi, x_end);
      if (PartB::mine())
#pragma unroll
        for (int p = 0; p < PartB::kPasses; ++p)
          pb[d].template load<WIDE>(p, gy + s_y[t0 + PartB::k(p)], o0 + PartB::col(), J.mo, y_end);
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(d, d * KC);
    for (int r = 0; r < rows; r += kAhead * KC) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        const int r0 = r + d * KC, left = rows - r0;
        if (left <= 0) break;
        pa[d].put(sa, left);
        pb[d].put(sb, left);
        __syncthreads();
        load(d, r0 + kAhead * KC);
        __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
        if constexpr (S::KS > 1) {
          const int kw = wave * (KC / S::KS);
          if (kw < left) multiply<PA, PB, S::MT, S::NT, PartA, PartB>(sa, sb, 0, 0, kw, KC / (16 * S::KS), acc);
        } else {
          constexpr int kCols = BN / S::WN;
          multiply<PA, PB, S::MT, S::NT, PartA, PartB>(sa, sb, (wave / kCols) * S::WM, (wave % kCols) * S::WN, 0, KC / 16,
                                                       acc);
        }
        __syncthreads();
      }
    }
  };
  if (near_end)
    main_loop(std::false_type{});
  else
    main_loop(std::true_type{});
  join_waves<S>(acc, smem);
  if (S::KS > 1 && wave > 0) return;
  constexpr int kCols = S::KS > 1 ? 1 : BN / S::WN;
  const int mw = (wave / kCols) * S::WM, nw = (wave % kCols) * S::WN;
  const bool whole = s.rows <= (int64_t(1) << a.rshift);
  float* dst = a.gW + s.g * a.w_per_group + J.woff;
  if (!whole)
    dst = a.part + J.part_off + (first_part(a.N * J.n, s.node0 * J.n, s.g, a.G, a.rshift) + (s.row0 >> a.rshift)) *
                                    ((int64_t)J.mi * J.mo);
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int ci = i0 + mw + 32 * i + acc_row(r);
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        const int co = o0 + nw + 32 * j + (lane & 31);
        if (ci < J.mi && co < J.mo) dst[(int64_t)ci * J.mo + co] = acc[i][j][r];
      }
    }
}

template <typename S, typename TI, typename TW, typename TO, bool WT>
__global__ __launch_bounds__(kThreads, 2) void lin_rows_kernel(const LinRowsArgs /*args*/) {
  __shared__ __align__(16) char smem[RowsParts<S, TI, TW, WT>::lds];
  lin_rows<S, TI, TW, TO, WT>(*(const LinRowsArgs*)__builtin_amdgcn_kernarg_segment_ptr(), blockIdx.x, smem);
}

// Both gradients in one launch: the weight gradient's tiles, then the input
// gradient's.  They read the same gy and wait for memory at different times
// (8192 nodes of 128x0e+128x1o+128x2e, fp32: 130 us of kernels for the training
// step with a launch each, 104 with one).  bf16 x and W: three waves per SIMD
// fit, two registers short of it without the bound (416 -> 358 us for the
// experts above).
template <typename S, typename SG, typename TX, typename TW>
__global__ __launch_bounds__(kThreads, Planes<TX>::count + Planes<TW>::count == 2 ? 3 : 2) void lin_backward_kernel(const LinBackwardArgs /*args*/) {
  const LinBackwardArgs& a = *(const LinBackwardArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ __align__(16) char smem[max_int(RowsParts<S, float, TW, true>::lds, GwParts<SG, TX>::lds)];
  if ((int64_t)blockIdx.x < a.rows_first) {
    if ((int64_t)blockIdx.x < a.gw.tiles) lin_gw<SG, TX>(a.gw, blockIdx.x, smem);
  } else {
    lin_rows<S, float, TW, float, true>(a.rows, blockIdx.x - a.rows_first, smem);
  }
}

// gW of the groups with several slots (their partial sums in slot order) or none (zero).
// `run` elements per thread: one, or eight where most threads would find nothing to do.
__global__ __launch_bounds__(kThreads) void lin_gw_reduce_kernel(const LinGwArgs /*args*/, int run) {
  const LinGwArgs& a = *(const LinGwArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const int g = blockIdx.y;
  const int64_t o0 = a.offsets ? a.offsets[g] : 0, o1 = a.offsets ? a.offsets[g + 1] : a.N;
  const int64_t first = (int64_t)blockIdx.x * (kThreads * run), last = min(a.w_per_group, first + kThreads * run);
  int ji = 0;
  while (ji + 1 < a.njobs && first >= a.job[ji + 1].woff) ++ji;
  for (; ji < a.njobs && a.job[ji].woff < last; ++ji) {  // the jobs this block's run of elements meets
    const LinGwJob& J = a.job[ji];
    const int64_t slots = ((o1 - o0) * J.n + (int64_t(1) << a.rshift) - 1) >> a.rshift;
    if (slots == 1) continue;
    const int64_t size = (int64_t)J.mi * J.mo;
    const float* p = a.part + J.part_off + first_part(a.N * J.n, o0 * J.n, g, a.G, a.rshift) * size;
    int64_t next = size;
    asm("" : "+s"(next));  // a value of its own: the compiler makes slower loads of a known product (8.8 us against 10.9)
    float* dst = a.gW + g * a.w_per_group + J.woff;
    const int64_t e1 = min(last - J.woff, size);
    for (int64_t e = max(first - J.woff, int64_t(0)) + threadIdx.x; e < e1; e += kThreads) {
      float v = 0.f;
#pragma unroll 8
      for (int64_t i = 0; i < slots; ++i) v += p[i * next + e];
      dst[e] = v;
    }
  }
}

// ---- grouping: a stable counting sort of the nodes by group ----------------------

constexpr int kGroupChunk = 256;  // nodes per wave

__global__ __launch_bounds__(64) void groups_validate_kernel(const int32_t* group, int64_t N, int G, int32_t* flag) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i < N && (group[i] < 0 || group[i] >= G)) *flag = 1;  // every writer writes the same value
}

__global__ void groups_zero_kernel(int32_t* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0;
}

// count[chunk][g] of each chunk of nodes.
__global__ __launch_bounds__(64) void groups_count_kernel(const int32_t* group, int64_t N, int G, int32_t* count) {
  extern __shared__ int32_t bins[];
  for (int g = threadIdx.x; g < G; g += 64) bins[g] = 0;
  __syncthreads();
  const int64_t b = (int64_t)blockIdx.x * kGroupChunk;
  for (int i = threadIdx.x; i < kGroupChunk && b + i < N; i += 64) {
    const int32_t g = group[b + i];
    if (g >= 0 && g < G) atomicAdd(&bins[g], 1);  // whole numbers: any order gives the same counts
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += 64) count[(int64_t)blockIdx.x * G + g] = bins[g];
}

// Turns the counts into every chunk's first position per group, and the
// totals into offsets [G + 1].  One block.
__global__ __launch_bounds__(1024) void groups_scan_kernel(int32_t* count, int64_t chunks, int G, int32_t* offsets) {
  __shared__ int32_t tot[1024];
  __shared__ int32_t carry;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int base = 0; base < G; base += 1024) {
    const int g = base + threadIdx.x;
    int32_t sum = 0;
    if (g < G)
      for (int64_t c = 0; c < chunks; ++c) sum += count[c * G + g];
    tot[threadIdx.x] = sum;
    __syncthreads();
    for (int off = 1; off < 1024; off <<= 1) {
      const int32_t v = (int)threadIdx.x >= off ? tot[threadIdx.x - off] : 0;
      __syncthreads();
      tot[threadIdx.x] += v;
      __syncthreads();
    }
    int32_t run = carry + tot[threadIdx.x] - sum;
    if (g < G) {
      offsets[g] = run;
      for (int64_t c = 0; c < chunks; ++c) {
        const int32_t n = count[c * G + g];
        count[c * G + g] = run;
        run += n;
      }
    }
    __syncthreads();
    if (threadIdx.x == 1023) carry += tot[1023];
    __syncthreads();
  }
  if (threadIdx.x == 0) offsets[G] = carry;
}

// One wave per chunk: a node's place is its chunk's first position in the
// group plus the nodes of the same group before it in the chunk.
__global__ __launch_bounds__(64) void groups_scatter_kernel(const int32_t* group, int64_t N, int G,
                                                            const int32_t* count, int32_t* order) {
  extern __shared__ int32_t next[];
  for (int g = threadIdx.x; g < G; g += 64) next[g] = count[(int64_t)blockIdx.x * G + g];
  __syncthreads();
  const int lane = threadIdx.x;
  const int64_t b = (int64_t)blockIdx.x * kGroupChunk;
  for (int i0 = 0; i0 < kGroupChunk; i0 += 64) {
    const int64_t v = b + i0 + lane;
    int32_t g = v < N ? group[v] : -1;
    if (g >= G) g = -1;
    int before = 0, after = 0;
#pragma unroll 8
    for (int j = 0; j < 64; ++j) {
      const bool same = __builtin_amdgcn_readlane(g, j) == g;
      before += same && j < lane;
      after += same && j > lane;
    }
    if (g >= 0) order[next[g] + before] = (int32_t)v;
    __syncthreads();
    if (g >= 0 && after == 0) next[g] += before + 1;  // the group's last node of these 64
    __syncthreads();
  }
}

inline unsigned blocks(int64_t n, int b) { return (unsigned)((n + b - 1) / b); }

}  // namespace

size_t lin_groups_workspace(int64_t N, int G) {
  const int64_t chunks = (N + kGroupChunk - 1) / kGroupChunk;
  return (size_t)(chunks > 0 ? chunks : 1) * G * sizeof(int32_t) + 256;
}

hipError_t launch_lin_groups_validate(const int32_t* group, int64_t N, int G, int32_t* flag, hipStream_t s) {
  hipLaunchKernelGGL(groups_zero_kernel, dim3(1), dim3(64), 0, s, flag, (int64_t)1);
  hipLaunchKernelGGL(groups_validate_kernel, dim3(blocks(N, 64)), dim3(64), 0, s, group, N, G, flag);
  return hipGetLastError();
}

hipError_t launch_lin_groups(const int32_t* group, int64_t N, int G, int32_t* offsets, int32_t* order, void* ws,
                             hipStream_t s) {
  TimingScope ts(kcGraph, s);
  if (N == 0) {
    hipLaunchKernelGGL(groups_zero_kernel, dim3(blocks(G + 1, 256)), dim3(256), 0, s, offsets, (int64_t)(G + 1));
    return hipGetLastError();
  }
  const int64_t chunks = (N + kGroupChunk - 1) / kGroupChunk;
  int32_t* count = static_cast<int32_t*>(ws);
  const size_t lds = (size_t)G * sizeof(int32_t);
  hipLaunchKernelGGL(groups_count_kernel, dim3((unsigned)chunks), dim3(64), lds, s, group, N, G, count);
  hipLaunchKernelGGL(groups_scan_kernel, dim3(1), dim3(1024), 0, s, count, chunks, G, offsets);
  hipLaunchKernelGGL(groups_scatter_kernel, dim3((unsigned)chunks), dim3(64), lds, s, group, N, G, count, order);
  return hipGetLastError();
}

namespace {

// The grid of `tiles` blocks in XCD order: a multiple of the eight XCDs.
unsigned xcd_grid(int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8); }

// Rows kernel shapes: 128 rows by 128, 64 or 32 columns, and 32 x 32 with the
// reduction split over the waves for launches of few rows.  One-piece operands
// take longer chunks (the same LDS holds more of the reduction).
template <int BN, bool ONE>
struct RowsShape {
  using type = Shape<128, BN, BN == 32 ? 32 : 64, BN == 128 ? 64 : 32, 1, ONE ? 64 : 32>;
};
template <bool ONE>
struct RowsShape<0, ONE> {
  using type = Shape<32, 32, 32, 32, 4, ONE ? 256 : 128, ONE ? 4 : 2>;
};

template <int BN, typename TI, typename TW, typename TO>
hipError_t launch_rows_typed(const LinRowsArgs& a, hipStream_t s) {
  using S = typename RowsShape<BN, Planes<TI>::count == 1 && Planes<TW>::count == 1>::type;
  hipLaunchKernelGGL((lin_rows_kernel<S, TI, TW, TO, false>), dim3(xcd_grid(a.tiles)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
template <int BN>
hipError_t launch_rows_types(const LinRowsArgs& a, hipStream_t s) {
  using H = uint16_t;
  switch ((a.in_bf16 ? 4 : 0) + (a.w_bf16 ? 2 : 0) + (a.out_bf16 ? 1 : 0)) {
    case 0: return launch_rows_typed<BN, float, float, float>(a, s);
    case 1: return launch_rows_typed<BN, float, float, H>(a, s);
    case 2: return launch_rows_typed<BN, float, H, float>(a, s);
    case 3: return launch_rows_typed<BN, float, H, H>(a, s);
    case 4: return launch_rows_typed<BN, H, float, float>(a, s);
    case 5: return launch_rows_typed<BN, H, float, H>(a, s);
    case 6: return launch_rows_typed<BN, H, H, float>(a, s);
    default: return launch_rows_typed<BN, H, H, H>(a, s);
  }
}

// Weight-gradient shapes of the same widths.
template <int BN>
struct GwShape {
  using type = Shape<128, 128, 64, 64, 1, 32>;
};
template <>
struct GwShape<64> {
  using type = Shape<64, 64, 32, 32, 1, 64>;
};
template <>
struct GwShape<32> {
  using type = Shape<32, 32, 32, 32, 4, 64>;
};

template <int BN, int BG, typename TX, typename TW>
hipError_t launch_backward_typed(LinBackwardArgs& a, hipStream_t s) {
  using S = typename RowsShape<BN, false>::type;
  a.rows_first = (a.gw.tiles + 7) / 8 * 8;
  const int64_t grid = a.rows_first + (a.rows.tiles + 7) / 8 * 8;
  if (grid >= INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((lin_backward_kernel<S, typename GwShape<BG>::type, TX, TW>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
template <int BN, int BG>
hipError_t launch_backward_types(LinBackwardArgs& a, hipStream_t s) {
  using H = uint16_t;
  if (a.gw.x_bf16)
    return a.rows.w_bf16 ? launch_backward_typed<BN, BG, H, H>(a, s) : launch_backward_typed<BN, BG, H, float>(a, s);
  return a.rows.w_bf16 ? launch_backward_typed<BN, BG, float, H>(a, s) : launch_backward_typed<BN, BG, float, float>(a, s);
}
template <int BN>
hipError_t launch_backward_shapes(int gw_width, LinBackwardArgs& a, hipStream_t s) {
  return gw_width == 128  ? launch_backward_types<BN, 128>(a, s)
         : gw_width == 64 ? launch_backward_types<BN, 64>(a, s)
                          : launch_backward_types<BN, 32>(a, s);
}

// Row tiles (or slots) of 1 << shift rows that cover every split of N n rows over G groups.
int64_t row_tiles(int64_t rows, int G, int shift, int32_t& by_row) {
  const int64_t tiles = (rows >> shift) + G;
  by_row = rows < tiles;
  return by_row ? rows : tiles;
}

// Tiles of the rows jobs of a launch, all of one shape (a launch per shape would
// run one after the other: the training step of 5003 nodes, 65x0e+33x1o+20x1o+
// 17x2e, 89 groups took 91 us in seven launches and takes 53 in three).  The
// width is the one of least padded work (narrow tiles count more per column
// because they re-read the rows and share less: 5/4 per halving), of which
// launches of fewer blocks than CUs reach only their share: 1024 rows x 1024 x
// 1024 in fp32 take 63 us in 64 blocks of 128 columns, 43.5 in 256 of 32; 2048
// rows 64.5 in 128 blocks, 57.5 in 256 of 64; 4000 x 256 x 256 21.5 against
// 13.9; 20000 nodes of 48x0e+48x1o 23.9 at 128, 14.9 at 64.  The groups' sizes
// are not known here and take no part: tiles of small groups are partly empty.
// 0: the 32 x 32 shape, its reduction split over the waves, below 64 blocks of
// 128 x 128: 512 rows of 1024 channels 33.2 us against 36.9, 256 rows 19.8
// against 36.9; at 1024 rows (64 blocks) it takes 47.4 against 43.5.
int plan_rows(LinRowsArgs& a) {
  int width = 128;
  double best = 0.0;
  int64_t wide = 0;
  for (int w : {128, 64, 32}) {
    double cost = 0.0;
    int64_t blocks = 0;
    for (int j = 0; j < a.njobs; ++j) {
      const int64_t tiles = (a.job[j].cols + w - 1) / w;
      cost += (double)a.N * a.job[j].n * tiles * w * (w == 128 ? 1.0 : w == 64 ? 1.25 : 1.5625);
      blocks += ((a.N * a.job[j].n + 127) / 128) * tiles;
    }
    if (w == 128) wide = blocks;
    if (blocks < kCUs) cost *= (double)kCUs / blocks;
    if (w == 128 || cost < best) {
      best = cost;
      width = w;
    }
  }
  if (wide < 64) width = 0;
  const int bn = width ? width : 32, shift = width ? 7 : 5;
  a.tiles = 0;
  for (int j = 0; j < a.njobs; ++j) {
    LinJob& J = a.job[j];
    J.tiles_n = (J.cols + bn - 1) / bn;
    J.first_tile = (int32_t)(a.tiles < INT32_MAX ? a.tiles : INT32_MAX);  // (the launch refuses more)
    a.tiles += row_tiles(a.N * J.n, a.offsets ? a.G : 1, shift, J.by_row) * J.tiles_n;
  }
  return width;
}

// The same for the weight gradient's tiles of W x W; smaller tiles read both
// operands more often (20000 nodes of 48x0e+48x1o, backward: 41.0 us at 128,
// 29.4 at 64; of 96x0e+96x1o: 47.2 at 128, 56.6 at 64).
int gw_width(const LinGwArgs& a) {
  int width = 128;
  double best = 0.0;
  for (int w : {128, 64, 32}) {
    double cost = 0.0;
    for (int j = 0; j < a.njobs; ++j) {
      const double ti = (a.job[j].mi + w - 1) / w, to = (a.job[j].mo + w - 1) / w;
      cost += (double)a.job[j].n * ti * to * w * w * (w == 128 ? 1.0 : w == 64 ? 1.5 : 3.0);
    }
    if (w == 128 || cost < best) {
      best = cost;
      width = w;
    }
  }
  return width;
}

}  // namespace

hipError_t launch_lin_rows(LinRowsArgs& a, hipStream_t s) {
  TimingScope ts(kcLinear, s);
  const int width = plan_rows(a);
  if (a.tiles >= INT32_MAX - 8) return hipErrorInvalidValue;
  return width == 128  ? launch_rows_types<128>(a, s)
         : width == 64 ? launch_rows_types<64>(a, s)
         : width == 32 ? launch_rows_types<32>(a, s)
                       : launch_rows_types<0>(a, s);
}

int64_t lin_gw_plan(LinGwArgs& a) {
  // rows per slot: about 512 blocks over all jobs, at least 128 rows each
  a.width = gw_width(a);
  auto tiles = [&](const LinGwJob& J) {
    return (int64_t)((J.mi + a.width - 1) / a.width) * ((J.mo + a.width - 1) / a.width);
  };
  int64_t work = 0;
  for (int j = 0; j < a.njobs; ++j) work += a.N * a.job[j].n * tiles(a.job[j]);
  int shift = 7;
  while (shift < 30 && (work >> shift) > 512) ++shift;
  a.rshift = shift;
  int64_t part = 0;
  a.tiles = 0;
  for (int j = 0; j < a.njobs; ++j) {
    LinGwJob& J = a.job[j];
    const int64_t slots = row_tiles(a.N * J.n, a.G, shift, J.by_row);
    J.first_tile = (int32_t)(a.tiles < INT32_MAX ? a.tiles : INT32_MAX);  // (the launch refuses more)
    a.tiles += slots * tiles(J);
    J.part_off = part;
    // (one place at least, so that a missing workspace is always noticed)
    part += std::max<int64_t>(1, first_part(a.N * J.n, a.N * J.n, a.G, a.G, shift)) * J.mi * J.mo;
  }
  return part;
}

hipError_t launch_lin_backward(LinBackwardArgs& a, hipStream_t s) {
  TimingScope ts(kcLinear, s);
  int width = 0;
  a.rows.tiles = a.gw.tiles = 0;
  if (a.rows.njobs > 0) width = plan_rows(a.rows);
  if (a.gw.njobs > 0) lin_gw_plan(a.gw);
  const hipError_t e = width == 128  ? launch_backward_shapes<128>(a.gw.width, a, s)
                       : width == 64 ? launch_backward_shapes<64>(a.gw.width, a, s)
                       : width == 32 ? launch_backward_shapes<32>(a.gw.width, a, s)
                                     : launch_backward_shapes<0>(a.gw.width, a, s);
  if (e != hipSuccess || a.gw.njobs == 0) return e;
  // How many groups have one slot, and so nothing to do here, is known on the device only; the number of
  // elements stands for it (49152 x 16 elements over two slots each: 10.6 us with one per thread, 22 with
  // eight; 2 M x 8 of groups with one slot: 25 us with one, 5.8 with eight; nothing between was measured)
  const int run = a.gw.w_per_group * a.gw.G < (int64_t(1) << 22) ? 1 : 8;
  hipLaunchKernelGGL(lin_gw_reduce_kernel, dim3(blocks(a.gw.w_per_group, kThreads * run), (unsigned)a.gw.G), dim3(kThreads), 0, s,
                     a.gw, run);
  return hipGetLastError();
}

}  // namespace tpconv
