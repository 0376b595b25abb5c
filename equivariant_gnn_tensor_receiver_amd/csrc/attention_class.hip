// The attention kernels of one width class (TP_DC values per head at most), one object per class.
#include "attention_kernels.h"

namespace tpconv {
namespace {

using namespace attn;

template <typename K>
hipError_t launch(K kernel, const AttnArgs& a, int threads, hipStream_t st) {
  const int64_t items = a.tiles * a.H * a.nsplit;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((items + 7) / 8 * 8)), dim3(threads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

#define TP_CAT2(a, b) a##b
#define TP_CAT(a, b) TP_CAT2(a, b)

// kind 0: forward, 1: gradient of the queries, 2: of keys and values
hipError_t TP_CAT(launch_attn_class_, TP_DC)(int kind, const AttnArgs& a, int cols, hipStream_t st) {
  auto go = [&](auto c, auto vec, auto score) -> hipError_t {
    constexpr int C = decltype(c)::value, S = decltype(score)::value;
    constexpr bool V = decltype(vec)::value;
    constexpr int f32 = Block<float, TP_DC, C>::kThreads, b16 = Block<uint16_t, TP_DC, C>::kThreads;
    if (kind == 0)
      return a.x_bf16 ? launch(forward_kernel<uint16_t, TP_DC, C, V, S>, a, b16, st)
                      : launch(forward_kernel<float, TP_DC, C, V, S>, a, f32, st);
    if (kind == 1)
      return a.x_bf16 ? launch(grad_q_kernel<uint16_t, TP_DC, C, V, S>, a, b16, st)
                      : launch(grad_q_kernel<float, TP_DC, C, V, S>, a, f32, st);
    auto kv = [&](auto t, int threads) -> hipError_t {
      using T = decltype(t);
      if constexpr (kv_in_two<T, TP_DC>()) {
        hipError_t e = hipSuccess;
        if (a.gv) e = launch(grad_kv_kernel<T, TP_DC, C, V, S, kValues>, a, threads, st);
        if (e == hipSuccess && (a.gk || a.part_pos)) e = launch(grad_kv_kernel<T, TP_DC, C, V, S, kKeys>, a, threads, st);
        return e;
      } else {
        return launch(grad_kv_kernel<T, TP_DC, C, V, S, kBoth>, a, threads, st);
      }
    };
    return a.x_bf16 ? kv(uint16_t{}, b16) : kv(float{}, f32);
  };
  auto sized = [&](auto vec, auto score) -> hipError_t {
    return cols == 128 ? go(std::integral_constant<int, 128>{}, vec, score)
                       : go(std::integral_constant<int, attn_small_cols(TP_DC)>{}, vec, score);
  };
  if (!a.sqk.vec || !a.sv.vec) return sized(std::false_type{}, std::integral_constant<int, kRuntime>{});
  const bool bias = a.slope != nullptr, cap = a.cap > 0.f;
  if (cap) return bias ? sized(std::true_type{}, std::integral_constant<int, kCappedBiased>{})
                       : sized(std::true_type{}, std::integral_constant<int, kCapped>{});
  return bias ? sized(std::true_type{}, std::integral_constant<int, kBiased>{})
              : sized(std::true_type{}, std::integral_constant<int, kPlain>{});
}

}  // namespace tpconv
