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
// first: what is left out is below 2^-22 of a term.  bf16 operands are one
// piece, so bf16 x bf16 takes one product, mixed types three, fp32 six.
#include "device_common.h"
#include "layers.h"
#include "timing.h"

namespace tpconv {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// Eight fp32 values as three planes of packed bf16 (exact: truncation leaves
// 8 bits per piece); bf16 values are one plane already.
__device__ __forceinline__ void split3(const float (&v)[8], u32x4 (&p)[3]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
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
__device__ __forceinline__ bool find_slot(const int32_t* offsets, int G, int64_t N, int n, int shift, int64_t t,
                                          Slot& s) {
  if (!offsets) {
    s = {0, 0, N * n, t << shift};
    return s.row0 < s.rows;
  }
  const int lane = threadIdx.x & 63;
  int count = 0;
  for (int base = 0; base < G; base += 64) {
    const int g = base + lane;
    const bool before = g < G && (((int64_t)offsets[g < G ? g : 0] * n) >> shift) + g <= t;
    const uint64_t mask = __ballot(before);
    count += __popcll(mask);
    if (~mask) break;
  }
  s.g = count - 1;  // group 0 starts at tile 0, so count >= 1
  const int64_t o0 = offsets[s.g], o1 = offsets[s.g + 1];
  s.node0 = o0;
  s.rows = (o1 - o0) * n;
  s.row0 = (t - (((o0 * n) >> shift) + s.g)) << shift;
  return s.row0 < s.rows;
}

__device__ __forceinline__ int64_t div_rows(int64_t r, int n) {
  return n == 1 ? r : n == 3 ? r / 3 : n == 5 ? r / 5 : r / 7;
}

// Eight values along the reduction: p[0..8) where k + j < len, else zero.
__device__ __forceinline__ void load_run8(const float* p, int k, int len, bool vec, float (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      floatx4 x = {0.f, 0.f, 0.f, 0.f};
      if (k + 4 * j < len) x = *reinterpret_cast<const floatx4*>(p + 4 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = x[e];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k + j < len ? p[j] : 0.f;
  }
}
__device__ __forceinline__ void load_run8(const uint16_t* p, int k, int len, bool vec, u32x4& v) {
  if (vec) {
    v = (u32x4){0, 0, 0, 0};
    if (k < len) v = *reinterpret_cast<const u32x4*>(p);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = k + 2 * j < len ? p[2 * j] : 0, b = k + 2 * j + 1 < len ? p[2 * j + 1] : 0;
      v[j] = a | (b << 16);
    }
  }
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

// Eight values of one row to its place in every plane.
template <int LD, int ROWS>
__device__ __forceinline__ void put_run8(uint16_t (*s)[ROWS][LD], int row, int k, const float (&v)[8]) {
  u32x4 p[3];
  split3(v, p);
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x4*>(&s[i][row][k]) = p[i];
}
template <int LD, int ROWS>
__device__ __forceinline__ void put_run8(uint16_t (*s)[ROWS][LD], int row, int k, const u32x4& v) {
  *reinterpret_cast<u32x4*>(&s[0][row][k]) = v;
}

template <typename T>
struct Run8;
template <>
struct Run8<float> {
  float v[8];
  __device__ __forceinline__ void set(int j, float x) { v[j] = x; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
};
template <>
struct Run8<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void set(int j, uint16_t x) { v[j >> 1] |= (uint32_t)x << (16 * (j & 1)); }
  __device__ __forceinline__ void clear() { v = (u32x4){0, 0, 0, 0}; }
};

// acc += A B over the k16 steps of this wave from the staged planes.
template <int PA, int PB, int MT, int NT, int BM, int BN, int LD>
__device__ __forceinline__ void multiply(const uint16_t (*sa)[BM][LD], const uint16_t (*sb)[BN][LD], int m0, int n0,
                                         int k0, int steps, floatx16 (&acc)[MT][NT]) {
  const int lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
  for (int st = 0; st < steps; ++st) {
    const int k = k0 + 16 * st + 8 * h;
    bf16x8 fa[PA][MT], fb[PB][NT];
#pragma unroll
    for (int p = 0; p < PA; ++p)
#pragma unroll
      for (int t = 0; t < MT; ++t) fa[p][t] = *reinterpret_cast<const bf16x8*>(&sa[p][m0 + 32 * t + i][k]);
#pragma unroll
    for (int p = 0; p < PB; ++p)
#pragma unroll
      for (int t = 0; t < NT; ++t) fb[p][t] = *reinterpret_cast<const bf16x8*>(&sb[p][n0 + 32 * t + i][k]);
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

// 32 x 32 tiles; the block's four waves take a quarter of every 128-long chunk
// of the reduction each, and their sums are added in order through LDS.
constexpr int kBM = 32, kBN = 32, kKC = 128, kLD = kKC + 8;  // rows padded by 16 bytes: conflict-free 16-byte reads

template <typename TI, typename TW, typename TO>
__global__ __launch_bounds__(kThreads) void lin_rows_kernel(const LinRowsArgs /*args*/) {
  const LinRowsArgs& a = *(const LinRowsArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  constexpr int PA = Planes<TI>::count, PB = Planes<TW>::count;
  __shared__ __align__(16) uint16_t sa[PA][kBM][kLD];
  __shared__ __align__(16) uint16_t sb[PB][kBN][kLD];
  __shared__ float part[3][kBM * kBN];
  __shared__ int32_t s_node[kBM], s_m[kBM];
  int ji = 0;
  while (ji + 1 < a.njobs && (int64_t)blockIdx.x >= a.job[ji + 1].first_tile) ++ji;
  const LinJob& J = a.job[ji];
  const int64_t lt = blockIdx.x - J.first_tile;
  const int64_t tm = lt / J.tiles_n;
  const int n0 = (int)(lt - tm * J.tiles_n) * kBN;
  Slot s;
  if (!find_slot(a.offsets, a.G, a.N, J.n, 5, tm, s)) return;
  const int tid = threadIdx.x, wave = tid >> 6;
  if (tid < kBM) {
    const int64_t r = s.row0 + tid;
    int32_t node = -1, m = 0;
    if (r < s.rows) {
      const int64_t p = div_rows(r, J.n);
      m = (int32_t)(r - p * J.n);
      node = a.order ? a.order[s.node0 + p] : (int32_t)p;
    }
    s_node[tid] = node;
    s_m[tid] = m;
  }
  __syncthreads();
  floatx16 acc[1][1];
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.f;
  const TI* in = static_cast<const TI*>(a.in);
  const TW* Wg = static_cast<const TW*>(a.W) + s.g * a.w_per_group;
  for (int si = 0; si < J.nseg; ++si) {
    const LinSeg& S = a.seg[J.seg0 + si];
    for (int k0 = 0; k0 < S.len; k0 += kKC) {
      // A: 16 threads per row, eight reductions each
      for (int p = 0; p < kBM * (kKC / 8) / kThreads; ++p) {
        const int row = p * (kThreads / (kKC / 8)) + tid / (kKC / 8), kk = (tid % (kKC / 8)) * 8;
        Run8<TI> v;
        v.clear();
        const int32_t node = s_node[row];
        if (node >= 0 && k0 + kk < S.len)
          load_run8(in + (int64_t)node * a.F_in + S.off + (int64_t)s_m[row] * S.len + k0 + kk, k0 + kk, S.len, a.vec_x, v.v);
        put_run8<kLD, kBM>(sa, row, kk, v.v);
      }
      if (a.wt) {  // B(k, c') = W[c'][k]: contiguous along the reduction
        for (int p = 0; p < kBN * (kKC / 8) / kThreads; ++p) {
          const int col = p * (kThreads / (kKC / 8)) + tid / (kKC / 8), kk = (tid % (kKC / 8)) * 8;
          Run8<TW> v;
          v.clear();
          if (n0 + col < J.cols && k0 + kk < S.len)
            load_run8(Wg + S.woff + (int64_t)(n0 + col) * S.ldw + k0 + kk, k0 + kk, S.len, a.vec_w, v.v);
          put_run8<kLD, kBN>(sb, col, kk, v.v);
        }
      } else {  // B(k, c') = W[k][c']: a thread takes eight reductions of one column
        for (int p = 0; p < kBN * (kKC / 8) / kThreads; ++p) {
          const int col = tid % kBN, kk = (p * (kThreads / kBN) + tid / kBN) * 8;
          Run8<TW> v;
          v.clear();
          if (n0 + col < J.cols)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (k0 + kk + j < S.len) v.set(j, Wg[S.woff + (int64_t)(k0 + kk + j) * S.ldw + n0 + col]);
          put_run8<kLD, kBN>(sb, col, kk, v.v);
        }
      }
      __syncthreads();
      const int kw = wave * (kKC / 4);  // a wave without reductions left skips its products
      if (k0 + kw < S.len) multiply<PA, PB, 1, 1, kBM, kBN, kLD>(sa, sb, 0, 0, kw, kKC / 64, acc);
      __syncthreads();
    }
  }
  const int lane = tid & 63;
  if (wave > 0)
#pragma unroll
    for (int r = 0; r < 16; ++r) part[wave - 1][r * 64 + lane] = acc[0][0][r];
  __syncthreads();
  if (wave > 0) return;
  const int col = n0 + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float v = ((acc[0][0][r] + part[0][r * 64 + lane]) + part[1][r * 64 + lane]) + part[2][r * 64 + lane];
    const int row = acc_row(r);
    if (s_node[row] >= 0 && col < J.cols)
      store_out(static_cast<TO*>(a.out), (int64_t)s_node[row] * a.F_out + J.off + (int64_t)s_m[row] * J.cols + col, v);
  }
}

// Weight gradient: one 32 x 32 tile of gW_g over the rows of one slot.  A group
// with a single slot is written at once, others through partial sums that
// lin_gw_reduce_kernel adds in order.
template <typename TX>
__global__ __launch_bounds__(kThreads) void lin_gw_kernel(const LinGwArgs /*args*/) {
  const LinGwArgs& a = *(const LinGwArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  constexpr int PA = Planes<TX>::count, PB = 3;
  __shared__ __align__(16) uint16_t sa[PA][kBM][kLD];
  __shared__ __align__(16) uint16_t sb[PB][kBN][kLD];
  __shared__ float part[3][kBM * kBN];
  __shared__ int32_t s_node[kKC], s_m[kKC];
  int ji = 0;
  while (ji + 1 < a.njobs && (int64_t)blockIdx.x >= a.job[ji + 1].first_tile) ++ji;
  const LinGwJob& J = a.job[ji];
  const int64_t lt = blockIdx.x - J.first_tile;
  const int tiles = J.tiles_i * J.tiles_o;
  const int64_t slot = lt / tiles;
  const int ti = (int)(lt - slot * tiles);
  const int i0 = (ti / J.tiles_o) * kBM, o0 = (ti % J.tiles_o) * kBN;
  Slot s;
  if (!find_slot(a.offsets, a.G, a.N, J.n, J.rshift, slot, s)) return;
  const int64_t row_end = min(s.rows, s.row0 + (int64_t(1) << J.rshift));
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  floatx16 acc[1][1];
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.f;
  const TX* x = static_cast<const TX*>(a.x);
  for (int64_t r0 = s.row0; r0 < row_end; r0 += kKC) {
    if (tid < kKC) {
      const int64_t r = r0 + tid;
      int32_t node = -1, m = 0;
      if (r < row_end) {
        const int64_t p = div_rows(r, J.n);
        m = (int32_t)(r - p * J.n);
        node = a.order ? a.order[s.node0 + p] : (int32_t)p;
      }
      s_node[tid] = node;
      s_m[tid] = m;
    }
    __syncthreads();
    for (int p = 0; p < kBM * (kKC / 8) / kThreads; ++p) {
      const int c = tid % kBM, kk = (p * (kThreads / kBM) + tid / kBM) * 8;
      Run8<TX> v;
      Run8<float> w;
      v.clear();
      w.clear();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int32_t node = s_node[kk + j], m = s_m[kk + j];
        if (node < 0) continue;
        if (i0 + c < J.mi) v.set(j, x[(int64_t)node * a.F_in + J.xoff + (int64_t)m * J.mi + i0 + c]);
        if (o0 + c < J.mo) w.set(j, a.gy[(int64_t)node * a.F_out + J.yoff + (int64_t)m * J.mo + o0 + c]);
      }
      put_run8<kLD, kBM>(sa, c, kk, v.v);
      put_run8<kLD, kBN>(sb, c, kk, w.v);
    }
    __syncthreads();
    const int kw = wave * (kKC / 4);
    if (r0 + kw < row_end) multiply<PA, PB, 1, 1, kBM, kBN, kLD>(sa, sb, 0, 0, kw, kKC / 64, acc);
    __syncthreads();
  }
  if (wave > 0)
#pragma unroll
    for (int r = 0; r < 16; ++r) part[wave - 1][r * 64 + lane] = acc[0][0][r];
  __syncthreads();
  if (wave > 0) return;
  const bool whole = s.rows <= (int64_t(1) << J.rshift);
  float* dst = whole ? a.gW + s.g * a.w_per_group + J.woff : a.part + J.part_off + slot * ((int64_t)J.mi * J.mo);
  const int co = o0 + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float v = ((acc[0][0][r] + part[0][r * 64 + lane]) + part[1][r * 64 + lane]) + part[2][r * 64 + lane];
    const int ci = i0 + acc_row(r);
    if (ci < J.mi && co < J.mo) dst[(int64_t)ci * J.mo + co] = v;
  }
}

// gW of the groups with several slots (their partial sums in slot order) or none (zero).
__global__ __launch_bounds__(kThreads) void lin_gw_reduce_kernel(const LinGwArgs /*args*/) {
  const LinGwArgs& a = *(const LinGwArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int g = blockIdx.y;
  if (e >= a.elems) return;
  int ji = 0;
  while (ji + 1 < a.njobs && e >= a.job[ji + 1].first_elem) ++ji;
  const LinGwJob& J = a.job[ji];
  const int64_t o0 = a.offsets ? a.offsets[g] : 0, o1 = a.offsets ? a.offsets[g + 1] : a.N;
  const int64_t slots = ((o1 - o0) * J.n + (int64_t(1) << J.rshift) - 1) >> J.rshift;
  if (slots == 1) return;
  const int64_t size = (int64_t)J.mi * J.mo, le = e - J.first_elem;
  const float* p = a.part + J.part_off + (((o0 * J.n) >> J.rshift) + g) * size + le;
  float v = 0.f;
  for (int64_t i = 0; i < slots; ++i) v += p[i * size];
  a.gW[g * a.w_per_group + J.woff + le] = v;
}

// Weights no block covers do not exist, so the jobs cover w_per_group.

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

hipError_t launch_lin_rows(LinRowsArgs& a, hipStream_t s) {
  TimingScope ts(kcLinear, s);
  a.tiles = 0;
  for (int j = 0; j < a.njobs; ++j) {
    LinJob& J = a.job[j];
    J.tiles_n = (J.cols + kBN - 1) / kBN;
    J.first_tile = a.tiles;
    a.tiles += ((a.N * J.n) / kBM + a.G) * J.tiles_n;
  }
  if (a.tiles >= INT32_MAX) return hipErrorInvalidValue;
  const dim3 g((unsigned)a.tiles), b(kThreads);
#define TP_ROWS(TI, TW, TO) hipLaunchKernelGGL((lin_rows_kernel<TI, TW, TO>), g, b, 0, s, a)
  const int key = (a.in_bf16 ? 4 : 0) + (a.w_bf16 ? 2 : 0) + (a.out_bf16 ? 1 : 0);
  switch (key) {
    case 0: TP_ROWS(float, float, float); break;
    case 1: TP_ROWS(float, float, uint16_t); break;
    case 2: TP_ROWS(float, uint16_t, float); break;
    case 3: TP_ROWS(float, uint16_t, uint16_t); break;
    case 4: TP_ROWS(uint16_t, float, float); break;
    case 5: TP_ROWS(uint16_t, float, uint16_t); break;
    case 6: TP_ROWS(uint16_t, uint16_t, float); break;
    default: TP_ROWS(uint16_t, uint16_t, uint16_t); break;
  }
#undef TP_ROWS
  return hipGetLastError();
}

int64_t lin_gw_plan(LinGwArgs& a) {
  // rows per slot: about 2048 blocks over all jobs, at least 256 rows each
  int64_t work = 0;
  for (int j = 0; j < a.njobs; ++j) {
    LinGwJob& J = a.job[j];
    J.tiles_i = (J.mi + kBM - 1) / kBM;
    J.tiles_o = (J.mo + kBN - 1) / kBN;
    work += a.N * J.n * J.tiles_i * J.tiles_o;
  }
  int shift = 8;
  while (shift < 30 && (work >> shift) > 2048) ++shift;
  int64_t part = 0, elems = 0;
  a.tiles = 0;
  for (int j = 0; j < a.njobs; ++j) {
    LinGwJob& J = a.job[j];
    J.rshift = shift;
    J.slots = ((a.N * J.n) >> shift) + a.G;
    J.first_tile = a.tiles;
    a.tiles += J.slots * J.tiles_i * J.tiles_o;
    J.part_off = part;
    part += J.slots * J.mi * J.mo;
    J.first_elem = elems;
    elems += (int64_t)J.mi * J.mo;
  }
  a.elems = elems;
  return part;
}

hipError_t launch_lin_gw(LinGwArgs& a, hipStream_t s) {
  TimingScope ts(kcLinear, s);
  lin_gw_plan(a);
  if (a.tiles >= INT32_MAX || a.elems >= (int64_t)INT32_MAX * kThreads) return hipErrorInvalidValue;
  const dim3 b(kThreads);
  if (a.N > 0) {
    if (a.x_bf16)
      hipLaunchKernelGGL((lin_gw_kernel<uint16_t>), dim3((unsigned)a.tiles), b, 0, s, a);
    else
      hipLaunchKernelGGL((lin_gw_kernel<float>), dim3((unsigned)a.tiles), b, 0, s, a);
  }
  hipLaunchKernelGGL(lin_gw_reduce_kernel, dim3(blocks(a.elems, kThreads), (unsigned)a.G), b, 0, s, a);
  return hipGetLastError();
}

}  // namespace tpconv
