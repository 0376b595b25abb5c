// Embedding of node types (include/tpconv_attention.h): y[v] = scale W[index[v]],
// and the gradient of W, a sum over the nodes of every type.
//
// The backward sorts the nodes by type (stable, so that every sum has a fixed
// order), cuts the sorted list into chunks of equal length whatever the types'
// shares, and lets one wave add the rows of a chunk, 64 lanes side by side over
// the columns.  A run of equal types inside a chunk is written at once; the
// parts of a run that crosses chunks go to the workspace and are added in order
// by a second kernel.  Rows of types without nodes are cleared by blocks of their own
// beside the sums (16383 nodes over 32000 x 1024: clearing the whole table beside the
// sort wrote the rows of present types twice, 93 us for both directions where this takes 79).
//
// Up to kOneBlock nodes are sorted by one block in LDS (4096 nodes 9 us), more of
// them by 8-bit radix passes over many blocks: a count and a scatter per pass while a
// block can add up the counts before its own (32768 nodes of 89 types: 4 and 6 us),
// with a scan of the counts between them for longer lists.
#include "attention.h"
#include "device_common.h"
#include "timing.h"

#include <algorithm>
#include <type_traits>

namespace tpconv {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

constexpr int kOneBlock = 4096;  // nodes that one block sorts
constexpr int kSortThreads = 1024, kWaves = kSortThreads / 64;
// nodes per thread of a block of a radix pass: one while there are few blocks, else four
constexpr int kFewBlocks = 64, kManyK = 4;
constexpr int kFew = 128;         // nodes that every block of a single launch sorts for itself

// ---- forward --------------------------------------------------------------------

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const floatx4 x = *reinterpret_cast<const floatx4_any*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = x[e];
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
  const u32x2 x = *reinterpret_cast<const u32x2_any*>(p);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    v[2 * j] = __uint_as_float(x[j] << 16);
    v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<floatx4_any*>(p) = (floatx4){v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<u32x2_any*>(p) =
      (u32x2){bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)bf16_bits(v); }

// `nodes` nodes per block and step; a thread takes four columns of kInFlight nodes'
// quads at a time, so that the index and the row of several are on their way together.
constexpr int kInFlight = 4;
template <typename TW, typename TY>
__global__ __launch_bounds__(256) void embed_forward_kernel(const EmbedArgs a, int nodes) {
  const int F = a.features, quads = (F + 3) / 4;
  const TW* W = static_cast<const TW*>(a.W);
  TY* y = static_cast<TY*>(a.y);
  for (int64_t base = (int64_t)blockIdx.x * nodes; base < a.N; base += (int64_t)gridDim.x * nodes) {
    const int here = (int)(a.N - base < nodes ? a.N - base : nodes), items = here * quads;
    for (int idx0 = threadIdx.x; idx0 < items; idx0 += 256 * kInFlight) {
      int nd[kInFlight], c[kInFlight];
      int32_t t[kInFlight];
      float v[kInFlight][4];
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int idx = min(idx0 + 256 * k, items - 1);
        nd[k] = idx / quads;
        c[k] = (idx - nd[k] * quads) * 4;
        t[k] = a.index[base + nd[k]];
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const bool there = t[k] >= 0 && t[k] < a.rows;
        const TW* w = W + (int64_t)(there ? t[k] : 0) * F + c[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = 0.f;
        if (there) {
          if (c[k] + 4 <= F) {
            load4(w, v[k]);
          } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (c[k] + e < F) v[k][e] = load_feat(w, e);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        if (idx0 + 256 * k >= items) continue;
        TY* o = y + (base + nd[k]) * F + c[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] *= a.scale;
        if (c[k] + 4 <= F) {
          store4(o, v[k]);
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (c[k] + e < F) store1(o + e, v[k][e]);
        }
      }
    }
  }
}

// ---- sort -------------------------------------------------------------------------

// Types outside of the table sort behind all others.
__device__ __forceinline__ uint32_t sort_key(int32_t t, int32_t rows) {
  return t >= 0 && t < rows ? (uint32_t)t : (uint32_t)rows;
}

// Stable ranks by an 8-bit digit within a block of kSortThreads threads: item k
// of a thread is number (wave * K + k) * 64 + lane.  cnt[wave][digit] ends as the
// count of the digit in the waves before, total[digit] as the block's; the rank
// of an item among the block's items of its digit is cnt[wave][digit] + pre[k].
// Items k >= used (uniform) and those with !there[k] are not counted.
template <int K>
__device__ __forceinline__ void block_ranks(const uint32_t (&key)[K], const bool (&there)[K], int used, int shift,
                                            int32_t (&pre)[K], int32_t* cnt, int32_t* total) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kWaves * 256; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int32_t* mine = cnt + wave * 256;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    pre[k] = 0;
    if (k >= used) continue;
    const uint32_t d = (key[k] >> shift) & 255u;
    // the lanes whose digits agree in every bit
    const uint64_t all = __ballot(there[k]);
    uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t own = (uint32_t)((int32_t)(d << (31 - b)) >> 31);  // the bit in all places
      const uint64_t m = __ballot((d >> b) & 1u);
      lo &= ~((uint32_t)m ^ own);
      hi &= ~((uint32_t)(m >> 32) ^ own);
    }
    const uint64_t peers = lo | ((uint64_t)hi << 32);
    const int below = __popcll(peers & ((uint64_t(1) << lane) - 1));
    const int32_t old = mine[d];
    __builtin_amdgcn_wave_barrier();  // every lane of the wave has read before the first writes
    if (there[k] && below == 0) mine[d] = old + __popcll(peers);
    __builtin_amdgcn_wave_barrier();
    pre[k] = old + below;
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    int32_t s = 0;
    for (int w = 0; w < kWaves; ++w) {
      const int32_t c = cnt[w * 256 + threadIdx.x];
      cnt[w * 256 + threadIdx.x] = s;
      s += c;
    }
    total[threadIdx.x] = s;
  }
  __syncthreads();
}

// Exclusive scan of 256 values in LDS by the first 256 threads.
__device__ __forceinline__ void scan256(int32_t* v) {
  const int t = threadIdx.x;
  int32_t s = t < 256 ? v[t] : 0;
  const int32_t own = s;
  for (int o = 1; o < 256; o <<= 1) {
    __syncthreads();
    if (t < 256) v[t] = s;
    __syncthreads();
    if (t < 256 && t >= o) s += v[t - o];
  }
  __syncthreads();
  if (t < 256) v[t] = s - own;
  __syncthreads();
}

// One block sorts all nodes (at most kOneBlock) in LDS.
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(const EmbedArgs a, int bits, int32_t* skey,
                                                                 int32_t* order) {
  __shared__ uint32_t s_key[kOneBlock];
  __shared__ uint16_t s_idx[kOneBlock];
  __shared__ int32_t cnt[kWaves * 256], total[256];
  constexpr int K = kOneBlock / kSortThreads;
  const int n = (int)a.N, used = (n + kSortThreads - 1) / kSortThreads;
  const int first = (threadIdx.x >> 6) * used * 64 + (threadIdx.x & 63);
  uint32_t key[K];
  int32_t pre[K];
  uint16_t idx[K];
  bool there[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = first + 64 * k;
    there[k] = k < used && i < n;
    key[k] = there[k] ? sort_key(a.index[i], a.rows) : 0;
    idx[k] = (uint16_t)i;
  }
  for (int shift = 0; shift < bits; shift += 8) {
    block_ranks<K>(key, there, used, shift, pre, cnt, total);
    scan256(total);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (there[k]) {
        const uint32_t d = (key[k] >> shift) & 255u;
        const int at = total[d] + cnt[(threadIdx.x >> 6) * 256 + d] + pre[k];
        s_key[at] = key[k];
        s_idx[at] = idx[k];
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (there[k]) {
        key[k] = s_key[first + 64 * k];
        idx[k] = s_idx[first + 64 * k];
      }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (there[k]) {
      skey[first + 64 * k] = (int32_t)key[k];
      order[first + 64 * k] = idx[k];
    }
}

template <int K>
__device__ __forceinline__ void load_items(const EmbedArgs& a, const int32_t* in_key, int64_t base, uint32_t (&key)[K],
                                           bool (&there)[K]) {
  const int first = (threadIdx.x >> 6) * K * 64 + (threadIdx.x & 63);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = base + first + 64 * k;
    there[k] = i < a.N;
    key[k] = !there[k] ? 0 : in_key ? (uint32_t)in_key[i] : sort_key(a.index[i], a.rows);
  }
}

// Digit counts of every block: few blocks [block][digit], many [digit][block] (for the
// scan).
template <int K>
__global__ __launch_bounds__(kSortThreads) void count_kernel(const EmbedArgs a, const int32_t* in_key, int shift,
                                                              int nblocks, int32_t* counts) {
  __shared__ int32_t cnt[kWaves * 256], total[256];
  uint32_t key[K];
  int32_t pre[K];
  bool there[K];
  load_items<K>(a, in_key, (int64_t)blockIdx.x * kSortThreads * K, key, there);
  block_ranks<K>(key, there, K, shift, pre, cnt, total);
  if (threadIdx.x < 256)
    counts[K == 1 ? (int64_t)blockIdx.x * 256 + threadIdx.x : (int64_t)threadIdx.x * nblocks + blockIdx.x] =
        total[threadIdx.x];
}

// Exclusive scan of n counts in place, one block.
__global__ __launch_bounds__(1024) void scan_counts_kernel(int32_t* v, int64_t n) {
  __shared__ int32_t part[1024];
  const int t = threadIdx.x;
  int32_t carry = 0;
  for (int64_t base = 0; base < n; base += 4096) {
    int32_t x[4], s = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t i = base + 4 * t + e;
      x[e] = i < n ? v[i] : 0;
      s += x[e];
    }
    part[t] = s;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
      const int32_t u = t >= o ? part[t - o] : 0;
      __syncthreads();
      part[t] += u;
      __syncthreads();
    }
    int32_t at = carry + part[t] - s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t i = base + 4 * t + e;
      if (i < n) v[i] = at;
      at += x[e];
    }
    carry += part[1023];
    __syncthreads();
  }
}

// K = 1: `counts` are the blocks' counts, and every block adds up what lies before its
// own items; else they are scanned.
template <int K>
__global__ __launch_bounds__(kSortThreads) void scatter_kernel(const EmbedArgs a, const int32_t* in_key,
                                                                const int32_t* in_idx, int shift, int nblocks,
                                                                const int32_t* counts, int32_t* out_key,
                                                                int32_t* out_idx) {
  __shared__ int32_t cnt[kWaves * 256], total[256], base[256];
  uint32_t key[K];
  int32_t pre[K];
  bool there[K];
  const int64_t b0 = (int64_t)blockIdx.x * kSortThreads * K;
  load_items<K>(a, in_key, b0, key, there);
  int32_t before = 0, all = 0;
  if (threadIdx.x < 256) {
    if constexpr (K == 1) {
#pragma unroll 8
      for (int b = 0; b < nblocks; ++b) {
        const int32_t c = counts[(int64_t)b * 256 + threadIdx.x];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    } else {
      before = counts[(int64_t)threadIdx.x * nblocks + blockIdx.x];
    }
    base[threadIdx.x] = all;
  }
  if constexpr (K == 1) {
    __syncthreads();
    scan256(base);
  }
  if (threadIdx.x < 256) base[threadIdx.x] = (K == 1 ? base[threadIdx.x] : 0) + before;
  block_ranks<K>(key, there, K, shift, pre, cnt, total);
  const int first = (threadIdx.x >> 6) * K * 64 + (threadIdx.x & 63);
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (there[k]) {
      const uint32_t d = (key[k] >> shift) & 255u;
      const int64_t i = b0 + first + 64 * k;
      const int32_t at = base[d] + cnt[(threadIdx.x >> 6) * 256 + d] + pre[k];
      out_key[at] = (int32_t)key[k];
      out_idx[at] = in_idx ? in_idx[i] : (int32_t)i;
    }
}

// ---- sums ---------------------------------------------------------------------------

// A wave's columns: C per lane from c0 on.
template <int C>
struct Cols {
  float v[C];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ void load(const float* p, int left) {
    if constexpr (C == 4) {
      if (left >= 4) {
        load4(p, v);
        return;
      }
    }
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = e < left ? p[e] : 0.f;
  }
  __device__ __forceinline__ void add(const Cols& o) {
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] += o.v[e];
  }
  __device__ __forceinline__ void store(float* p, int left, float f) const {
    if constexpr (C == 4) {
      if (left >= 4) {
        const float w[4] = {v[0] * f, v[1] * f, v[2] * f, v[3] * f};
        store4(p, w);
        return;
      }
    }
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < left) p[e] = v[e] * f;
  }
};

struct SumArgs {
  int32_t rows, F, slices;  // slices of 64 C columns
  int32_t chunk;            // sorted nodes per wave
  int64_t N, chunks;
  int64_t sum_blocks;       // the blocks behind them clear `clear_rows` rows per wave
  int32_t clear_rows;
  float scale;
  const int32_t *skey, *order;
  const float* gy;
  float* gW;
  float* part;  // [chunks][2][F]: the run that began before the chunk, the run that goes on behind it
};

// Clears the rows of types without nodes among the `unit`-th clear_rows rows: a lane
// looks for each, and the wave writes those that are not there.
__device__ __forceinline__ void clear_absent(const SumArgs& a, int64_t unit) {
  const int lane = threadIdx.x & 63;
  const int64_t row0 = unit * a.clear_rows;
  const int64_t row = row0 + lane;
  bool absent = false;
  if (lane < a.clear_rows && row < a.rows) {
    int64_t lo = 0, hi = a.N;  // the first position whose type is not below the row
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (a.skey[mid] < row) lo = mid + 1; else hi = mid;
    }
    absent = lo == a.N || a.skey[lo] != row;
  }
  for (uint64_t m = __ballot(absent); m; m &= m - 1) {
    float* p = a.gW + (row0 + __ffsll((unsigned long long)m) - 1) * a.F;
    int c = lane * 4;
    for (; c + 4 <= a.F; c += 256) *reinterpret_cast<floatx4_any*>(p + c) = (floatx4){0.f, 0.f, 0.f, 0.f};
    for (; c < a.F; ++c) p[c] = 0.f;
  }
}

// One wave per (chunk, slice): its sorted nodes, added run by run.
template <int C>
__global__ __launch_bounds__(256) void sum_kernel(const SumArgs a) {
  const int lane = threadIdx.x & 63;
  if (blockIdx.x >= a.sum_blocks) {
    clear_absent(a, ((int64_t)blockIdx.x - a.sum_blocks) * 4 + (threadIdx.x >> 6));
    return;
  }
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t c = unit / a.slices;
  if (c >= a.chunks) return;
  const int c0 = (int)(unit - c * a.slices) * 64 * C + lane * C, left = a.F - c0;
  const int64_t p0 = c * a.chunk, p1 = p0 + a.chunk < a.N ? p0 + a.chunk : a.N;
  const int32_t before = p0 > 0 ? a.skey[p0 - 1] : -1, behind = p1 < a.N ? a.skey[p1] : -1;
  Cols<C> acc;
  acc.clear();
  int32_t run = a.skey[p0];
  bool opened = run == before;  // the run began in an earlier chunk
  auto finish = [&](bool goes_on) {
    if (run < a.rows && left > 0) {
      if (opened)
        acc.store(a.part + (2 * c) * a.F + c0, left, 1.f);
      else if (goes_on)
        acc.store(a.part + (2 * c + 1) * a.F + c0, left, 1.f);
      else
        acc.store(a.gW + (int64_t)run * a.F + c0, left, a.scale);
    }
  };
  constexpr int U = 8;  // rows in flight
  for (int64_t p = p0; p < p1; p += 64) {
    const int n = (int)(p1 - p < 64 ? p1 - p : 64);
    const int32_t my_key = a.skey[p + (lane < n ? lane : 0)], my_idx = a.order[p + (lane < n ? lane : 0)];
    for (int j = 0; j < n; j += U) {
      Cols<C> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u].clear();
        if (j + u < n && left > 0) {
          const int32_t node = __builtin_amdgcn_readlane(my_idx, (j + u) & 63);
          v[u].load(a.gy + (int64_t)node * a.F + c0, left);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j + u < n) {
          const int32_t key = __builtin_amdgcn_readlane(my_key, (j + u) & 63);
          if (key != run) {
            finish(false);
            acc.clear();
            run = key;
            opened = false;
          }
          acc.add(v[u]);
        }
    }
  }
  finish(run == behind);
}

// Runs that cross chunks: a block's waves add equal parts of the list of partial sums,
// then the waves' sums in order.  One block per (type, slice), or where there are more
// types than chunks per (chunk in which such a run begins, slice).
template <int C, int WAVES, bool BY_TYPE>
__global__ __launch_bounds__(64 * WAVES) void join_kernel(const SumArgs a) {
  __shared__ float red[WAVES][64 * C];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t item = blockIdx.x / a.slices;
  const int slice = (int)(blockIdx.x - item * a.slices);
  // searches with 64 probes per step: the first position whose type is not below `t`
  auto first_of = [&](int64_t from, int32_t t) {
    int64_t lo = from, n = a.N - from;  // in [lo, lo + n]
    while (n > 0) {
      const int64_t step = (n + 63) / 64, i = lane * step;
      const int count = __popcll(__ballot(i < n && a.skey[lo + (i < n ? i : 0)] < t));
      if (count == 0) break;
      lo += (count - 1) * step + 1;
      n = min(step - 1, n - (count - 1) * step - 1);
    }
    return lo;
  };
  int32_t run;
  int64_t begin, end;
  if (BY_TYPE) {
    run = (int32_t)item;
    begin = first_of(0, run);
    if (begin >= a.N || a.skey[begin] != run) return;
  } else {
    const int64_t next = (item + 1) * a.chunk;
    if (next >= a.N) return;
    run = a.skey[next - 1];
    if (run >= a.rows || a.skey[next] != run) return;
    if (item > 0 && a.skey[item * a.chunk - 1] == run) return;  // began earlier
    begin = next - 1;  // (any place of the run in its first chunk)
  }
  end = first_of(begin, run + 1);
  const int64_t c = begin / a.chunk, last = (end - 1) / a.chunk;  // chunks c .. last
  if (last == c) return;
  const int c0 = slice * 64 * C + lane * C, left = a.F - c0;
  Cols<C> acc;
  acc.clear();
  const int64_t total = last - c + 1, per = (total + WAVES - 1) / WAVES;
  const int64_t b = c + wave * per, e = b + per < c + total ? b + per : c + total;
  if (left > 0) {
    constexpr int U = 8;
    for (int64_t i = b; i < e; i += U) {
      Cols<C> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u].clear();
        if (i + u < e) v[u].load(a.part + (2 * (i + u) + (i + u == c)) * a.F + c0, left);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) acc.add(v[u]);
    }
  }
#pragma unroll
  for (int k = 0; k < C; ++k) red[wave][lane * C + k] = acc.v[k];
  __syncthreads();
  if (wave > 0 || left <= 0) return;
  for (int w = 1; w < WAVES; ++w)
#pragma unroll
    for (int k = 0; k < C; ++k) acc.v[k] += red[w][lane * C + k];
  acc.store(a.gW + (int64_t)run * a.F + c0, left, a.scale);
}

// Few nodes: one launch.  Every block orders them for itself (a node's place is
// the number of smaller types, and of equal types before it) and writes its part of the table.
__global__ __launch_bounds__(256) void few_kernel(const EmbedArgs a, int64_t per_block) {
  __shared__ uint32_t raw[kFew], s_key[kFew];
  __shared__ int32_t s_idx[kFew];
  const int n = (int)a.N;
  for (int i = threadIdx.x; i < n; i += 256) raw[i] = sort_key(a.index[i], a.rows);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    const uint32_t k = raw[i];
    int at = 0;
    for (int j = 0; j < n; ++j) at += raw[j] < k || (raw[j] == k && j < i);
    s_key[at] = k;
    s_idx[at] = i;
  }
  __syncthreads();
  const int64_t end = min((int64_t)a.rows * a.features, (blockIdx.x + 1) * per_block);
  for (int64_t i = blockIdx.x * per_block + threadIdx.x; i < end; i += 256) {
    const uint32_t row = (uint32_t)(i / a.features);
    const int col = (int)(i - (int64_t)row * a.features);
    int lo = 0, hi = n;  // the first node of type `row`
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_key[mid] < row) lo = mid + 1; else hi = mid;
    }
    float v = 0.f;
    for (; lo < n && s_key[lo] == row; ++lo) v += a.gy[(int64_t)s_idx[lo] * a.features + col];
    a.gW[i] = v * a.scale;
  }
}

struct EmbedPlan {
  int slices, cols;  // column slices of 64 * cols
  int chunk;
  int64_t chunks;
  int k, nblocks;    // nodes per thread and blocks of a radix pass
  size_t key, order, key2, order2, counts, part, bytes;
};

EmbedPlan make_plan(int32_t features, int64_t N) {
  EmbedPlan p{};
  p.cols = features <= 64 ? 1 : features <= 128 ? 2 : 4;
  p.slices = (features + 64 * p.cols - 1) / (64 * p.cols);
  // about 2048 waves or more, chunks of 8 to 256 nodes (longer where the launch would grow past 2^20 blocks)
  p.chunk = 8;
  while ((p.chunk < 256 && N / (2 * p.chunk) * p.slices >= 2048) || N / p.chunk * p.slices >= 1 << 20) p.chunk *= 2;
  p.chunks = (N + p.chunk - 1) / p.chunk;
  p.k = N <= (int64_t)kFewBlocks * kSortThreads ? 1 : kManyK;
  p.nblocks = (int)((N + (int64_t)kSortThreads * p.k - 1) / ((int64_t)kSortThreads * p.k));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  if (N <= kFew) return p;
  p.key = take((size_t)N * 4);
  p.order = take((size_t)N * 4);
  if (N > kOneBlock) {
    p.key2 = take((size_t)N * 4);
    p.order2 = take((size_t)N * 4);
    p.counts = take((size_t)p.nblocks * 256 * 4);
  }
  p.part = take((size_t)p.chunks * 2 * features * 4);
  p.bytes = at;
  return p;
}

}  // namespace

size_t embed_workspace(int32_t rows, int32_t features, int64_t N) { return make_plan(features, N).bytes; }

hipError_t launch_embed_forward(const EmbedArgs& a, hipStream_t s) {
  TimingScope ts(kcEmbed, s);
  const int quads = (a.features + 3) / 4, nodes = std::max(1, 256 * kInFlight / quads);
  const dim3 grid((unsigned)std::min<int64_t>((a.N + nodes - 1) / nodes, 1 << 20)), block(256);
  if (a.w_bf16 && a.y_bf16)
    hipLaunchKernelGGL((embed_forward_kernel<uint16_t, uint16_t>), grid, block, 0, s, a, nodes);
  else if (a.w_bf16)
    hipLaunchKernelGGL((embed_forward_kernel<uint16_t, float>), grid, block, 0, s, a, nodes);
  else if (a.y_bf16)
    hipLaunchKernelGGL((embed_forward_kernel<float, uint16_t>), grid, block, 0, s, a, nodes);
  else
    hipLaunchKernelGGL((embed_forward_kernel<float, float>), grid, block, 0, s, a, nodes);
  return hipGetLastError();
}

hipError_t launch_embed_backward(const EmbedArgs& a, void* ws, hipStream_t s) {
  TimingScope ts(kcEmbed, s);
  const int64_t table = (int64_t)a.rows * a.features;
  if (a.N <= kFew) {
    const int64_t per = std::max<int64_t>(1024, (table + (1 << 16) - 1) / (1 << 16));
    hipLaunchKernelGGL(few_kernel, dim3((unsigned)((table + per - 1) / per)), dim3(256), 0, s, a, per);
    return hipGetLastError();
  }
  const EmbedPlan p = make_plan(a.features, a.N);
  char* w = static_cast<char*>(ws);
  auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(w + at); };
  int32_t *key = ints(p.key), *order = ints(p.order);
  int bits = 1;
  while ((int64_t(1) << bits) <= a.rows) ++bits;  // keys 0 .. rows
  if (a.N <= kOneBlock) {
    hipLaunchKernelGGL(sort_one_kernel, dim3(1), dim3(kSortThreads), 0, s, a, bits, key, order);
  } else {
    const int passes = (bits + 7) / 8;
    int32_t *k2 = ints(p.key2), *o2 = ints(p.order2), *counts = ints(p.counts);
    // the last pass writes key and order
    const int32_t *in_k = nullptr, *in_o = nullptr;
    for (int i = 0; i < passes; ++i) {
      int32_t *out_k = (passes - 1 - i) % 2 == 0 ? key : k2, *out_o = (passes - 1 - i) % 2 == 0 ? order : o2;
      const dim3 grid(p.nblocks), threads(kSortThreads);
      if (p.k == 1) {
        hipLaunchKernelGGL(count_kernel<1>, grid, threads, 0, s, a, in_k, 8 * i, p.nblocks, counts);
        hipLaunchKernelGGL(scatter_kernel<1>, grid, threads, 0, s, a, in_k, in_o, 8 * i, p.nblocks, counts, out_k, out_o);
      } else {
        hipLaunchKernelGGL(count_kernel<kManyK>, grid, threads, 0, s, a, in_k, 8 * i, p.nblocks, counts);
        hipLaunchKernelGGL(scan_counts_kernel, dim3(1), dim3(1024), 0, s, counts, (int64_t)p.nblocks * 256);
        hipLaunchKernelGGL(scatter_kernel<kManyK>, grid, threads, 0, s, a, in_k, in_o, 8 * i, p.nblocks, counts, out_k,
                           out_o);
      }
      in_k = out_k;
      in_o = out_o;
    }
  }
  SumArgs m{};
  m.rows = a.rows;
  m.F = a.features;
  m.slices = p.slices;
  m.chunk = p.chunk;
  m.N = a.N;
  m.chunks = p.chunks;
  m.scale = a.scale;
  m.skey = key;
  m.order = order;
  m.gy = a.gy;
  m.gW = a.gW;
  m.part = reinterpret_cast<float*>(w + p.part);
  m.sum_blocks = (p.chunks * p.slices + 3) / 4;
  m.clear_rows = a.features >= 256 ? 16 : 64;  // rows that a wave clears: about as long as its search
  const dim3 sum_grid((unsigned)(m.sum_blocks + (a.rows + 4 * m.clear_rows - 1) / (4 * m.clear_rows)));
  const bool by_type = a.rows <= p.chunks;
  auto sums = [&](auto c) {
    constexpr int C = decltype(c)::value;
    hipLaunchKernelGGL(sum_kernel<C>, sum_grid, dim3(256), 0, s, m);
    if (p.chunks == 1) return;  // no run crosses chunks
    if (by_type)
      hipLaunchKernelGGL((join_kernel<C, 8, true>), dim3((unsigned)((int64_t)a.rows * p.slices)), dim3(512), 0, s, m);
    else
      hipLaunchKernelGGL((join_kernel<C, 4, false>), dim3((unsigned)(p.chunks * p.slices)), dim3(256), 0, s, m);
  };
  if (p.cols == 1)
    sums(std::integral_constant<int, 1>{});
  else if (p.cols == 2)
    sums(std::integral_constant<int, 2>{});
  else
    sums(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace tpconv
