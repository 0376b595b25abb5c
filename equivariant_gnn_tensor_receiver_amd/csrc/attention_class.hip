// The attention kernels of one width class (TP_DC values per head at most), one object per class.
#include "attention_kernels.h"

namespace tpconv {
namespace {

using namespace attn;

template <typename K>
hipError_t launch(K kernel, const AttnArgs& a, int waves, hipStream_t st) {
  const int64_t items = a.tiles * a.H * a.nsplit;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((items + 7) / 8 * 8)), dim3(64 * waves), 0, st, a);
  return hipGetLastError();
}

}  // namespace

#define TP_CAT2(a, b) a##b
#define TP_CAT(a, b) TP_CAT2(a, b)

// kind 0: forward, 1: gradient of the queries, 2: of keys and values
hipError_t TP_CAT(launch_attn_class_, TP_DC)(int kind, const AttnArgs& a, int waves, hipStream_t st) {
  auto go = [&](auto w, auto vec) -> hipError_t {
    constexpr int W = decltype(w)::value;
    constexpr bool V = decltype(vec)::value;
    if (kind == 0) {
      if (!a.x_bf16) return launch(forward_kernel<float, TP_DC, W, 3, V>, a, W, st);
      if (a.y_bf16 && !a.stat) return launch(forward_kernel<uint16_t, TP_DC, W, 2, V>, a, W, st);
      return launch(forward_kernel<uint16_t, TP_DC, W, 3, V>, a, W, st);
    }
    if (kind == 1)
      return a.x_bf16 ? launch(grad_q_kernel<uint16_t, TP_DC, W, V>, a, W, st)
                      : launch(grad_q_kernel<float, TP_DC, W, V>, a, W, st);
    return a.x_bf16 ? launch(grad_kv_kernel<uint16_t, TP_DC, W, V>, a, W, st)
                    : launch(grad_kv_kernel<float, TP_DC, W, V>, a, W, st);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 4> four;
  if (a.sqk.vec && a.sv.vec) return waves == 1 ? go(one, std::true_type{}) : go(four, std::true_type{});
  return waves == 1 ? go(one, std::false_type{}) : go(four, std::false_type{});
}

}  // namespace tpconv
