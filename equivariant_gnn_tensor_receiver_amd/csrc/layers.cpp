// C ABI of the node layers (declared in include/tpconv_layers.h): handles,
// argument checks, workspace sizes, and the launches' argument blocks.
#include "layers.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <string>
#include <vector>

#include "kernels.h"

struct tpconv_norm_s {
  std::vector<tpconv::Irrep> irreps;
  std::vector<int32_t> off, w_off, b_off;
  int64_t F = 0;
  int32_t weights = 0, biases = 0;
  float eps = 0.f;
  int x_dtype = 0, y_dtype = 0;
};

struct tpconv_linear_s {
  std::vector<tpconv::Irrep> in, out;
  std::vector<int32_t> in_off, out_off;
  std::vector<tpconv::LinBlock> blocks;
  int64_t F_in = 0, F_out = 0, w_numel = 0;
  int32_t groups = 1;
  int x_dtype = 0, w_dtype = 0, y_dtype = 0;
};

struct tpconv_muon_s {
  tpconv::MuonPlan plan;
};

namespace tpconv {
namespace {

tpconv_status dev(hipError_t e) { return e == hipSuccess ? TPCONV_SUCCESS : TPCONV_ERROR_DEVICE; }
bool bad_dtype(int t) { return t != TPCONV_F32 && t != TPCONV_BF16; }
// Too small, or not aligned for the 16-byte accesses of the kernels.
bool bad_workspace(const void* ws, size_t bytes, size_t need) {
  return need > 0 && (!ws || bytes < need || reinterpret_cast<uintptr_t>(ws) % 16 != 0);
}
bool bad_count(int64_t n) { return n < 0 || n >= INT32_MAX; }

// Irreps of one side and their feature offsets.
tpconv_status parse_side(const char* text, std::vector<Irrep>& ir, std::vector<int32_t>& off, int64_t& F) {
  if (!text) return TPCONV_ERROR_INVALID_VALUE;
  if (!parse_irreps(text, ir)) return TPCONV_ERROR_IRREPS;
  if ((int)ir.size() > kMaxGroups) return TPCONV_ERROR_UNSUPPORTED;
  F = 0;
  for (const auto& i : ir) {
    if (i.l > kMaxL) return TPCONV_ERROR_UNSUPPORTED;
    off.push_back((int32_t)F);
    F += (int64_t)i.mul * (2 * i.l + 1);
  }
  return TPCONV_SUCCESS;
}

NormArgs norm_args(const tpconv_norm_s& h, int64_t N) {
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.nirreps = (int32_t)h.irreps.size();
  a.x_bf16 = h.x_dtype == TPCONV_BF16;
  a.y_bf16 = h.y_dtype == TPCONV_BF16;
  a.eps = h.eps;
  a.N = N;
  a.F = h.F;
  for (int i = 0; i < a.nirreps; ++i) {
    NormIrrep& r = a.ir[i];
    r.mul = h.irreps[i].mul;
    r.n = 2 * h.irreps[i].l + 1;
    r.scalar = h.irreps[i].l == 0 && h.irreps[i].parity > 0;
    r.off = h.off[i];
    r.w_off = h.w_off[i];
    r.b_off = h.b_off[i];
  }
  return a;
}

// Rows kernel arguments: the forward (x -> y) or the input gradient (gy -> gx).
void rows_args(const tpconv_linear_s& h, bool grad, int64_t N, const int32_t* offsets, const int32_t* order,
               const void* in, const void* W, void* out, LinRowsArgs& a) {
  std::memset(&a, 0, sizeof(a));
  const auto& to = grad ? h.in : h.out;
  const auto& to_off = grad ? h.in_off : h.out_off;
  a.G = h.groups;
  a.N = N;
  a.F_in = grad ? h.F_out : h.F_in;
  a.F_out = grad ? h.F_in : h.F_out;
  a.w_per_group = h.w_numel;
  a.in_bf16 = !grad && h.x_dtype == TPCONV_BF16;
  a.w_bf16 = h.w_dtype == TPCONV_BF16;
  a.out_bf16 = !grad && h.y_dtype == TPCONV_BF16;
  a.wt = grad;
  a.offsets = offsets;
  a.order = order;
  a.in = in;
  a.W = W;
  a.out = out;
  int ns = 0;
  for (size_t o = 0; o < to.size(); ++o) {
    LinJob& J = a.job[a.njobs++];
    J.n = 2 * to[o].l + 1;
    J.off = to_off[o];
    J.cols = to[o].mul;
    J.seg0 = ns;
    for (const auto& b : h.blocks) {
      if ((grad ? b.i : b.o) != (int32_t)o) continue;
      LinSeg& S = a.seg[ns++];
      S.off = grad ? b.yoff : b.xoff;
      S.len = grad ? b.mo : b.mi;
      S.woff = (int32_t)b.woff;
      J.nseg++;
    }
  }
}

void gw_args(const tpconv_linear_s& h, int64_t N, const int32_t* offsets, const int32_t* order, const void* x,
             const float* gy, float* gW, float* part, LinGwArgs& a) {
  std::memset(&a, 0, sizeof(a));
  a.G = h.groups;
  a.N = N;
  a.F_in = h.F_in;
  a.F_out = h.F_out;
  a.w_per_group = h.w_numel;
  a.x_bf16 = h.x_dtype == TPCONV_BF16;
  a.offsets = offsets;
  a.order = order;
  a.x = x;
  a.gy = gy;
  a.gW = gW;
  a.part = part;
  for (const auto& b : h.blocks) {
    LinGwJob& J = a.job[a.njobs++];
    J.n = b.n;
    J.mi = b.mi;
    J.mo = b.mo;
    J.xoff = b.xoff;
    J.yoff = b.yoff;
    J.woff = (int32_t)b.woff;
  }
}

size_t linear_workspace(const tpconv_linear_s& h, int op, int64_t N) {
  if (op == TPCONV_OP_FORWARD || h.blocks.empty()) return 0;
  LinGwArgs a;
  gw_args(h, N, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, a);
  return (size_t)lin_gw_plan(a) * sizeof(float);
}

tpconv_status linear_inputs(const tpconv_linear_s* h, int64_t N, const int32_t* offsets, const int32_t* order) {
  if (!h || bad_count(N)) return TPCONV_ERROR_INVALID_VALUE;
  if ((offsets == nullptr) != (order == nullptr) || (!offsets && h->groups != 1 && N > 0))
    return TPCONV_ERROR_INVALID_VALUE;
  return TPCONV_SUCCESS;
}

// Largest |a s + b s^3 + c s^5| and |b t + c t^2|, t = s^2, on [0, top]: at the
// ends or where the derivative vanishes.
void bounds(double a, double b, double c, double top, double& x, double& poly) {
  auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + c * s * s))); };
  auto g = [&](double t) { return std::fabs(t * (b + c * t)); };
  x = f(top);
  poly = g(top * top);
  if (c != 0.0) {
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0)
      for (double r : {(-3.0 * b + std::sqrt(d)) / (10.0 * c), (-3.0 * b - std::sqrt(d)) / (10.0 * c)})
        if (r > 0.0 && r < top * top) x = std::max(x, f(std::sqrt(r)));
    const double t = -b / (2.0 * c);
    if (t > 0.0 && t < top * top) poly = std::max(poly, g(t));
  } else if (b != 0.0) {
    const double r = -a / (3.0 * b);
    if (r > 0.0 && r < top * top) x = std::max(x, f(std::sqrt(r)));
  }
}

// The power of two that takes a bound to 2^13 (fp16 ends at 2^16: three bits of
// headroom for rounding; values down to 2^-15 of the bound keep a normal lo part).
bool exponent(double bound, int32_t& e) {
  if (!(bound > 1e-6)) bound = 1e-6;
  if (!(bound < 1e12)) return false;
  e = 13 - (int32_t)std::ceil(std::log2(bound));
  return true;
}

}  // namespace
}  // namespace tpconv

using namespace tpconv;

extern "C" {

// ---- layer norm -----------------------------------------------------------------

tpconv_status tpconv_norm_create(tpconv_norm* out, const tpconv_norm_desc* desc) {
  if (!out || !desc) return TPCONV_ERROR_INVALID_VALUE;
  *out = nullptr;
  if (!(desc->eps > 0.f) || std::isinf(desc->eps) || bad_dtype(desc->x_dtype) || bad_dtype(desc->y_dtype))
    return TPCONV_ERROR_INVALID_VALUE;
  try {
    auto h = std::make_unique<tpconv_norm_s>();
    const tpconv_status st = parse_side(desc->irreps, h->irreps, h->off, h->F);
    if (st != TPCONV_SUCCESS) return st;
    for (const auto& i : h->irreps) {
      const bool scalar = i.l == 0 && i.parity > 0;
      h->w_off.push_back(h->weights);
      h->b_off.push_back(h->biases);
      h->weights += i.mul;
      if (scalar) h->biases += i.mul;
    }
    h->eps = desc->eps;
    h->x_dtype = desc->x_dtype;
    h->y_dtype = desc->y_dtype;
    *out = h.release();
    return TPCONV_SUCCESS;
  } catch (...) {
    return TPCONV_ERROR_INVALID_VALUE;
  }
}

tpconv_status tpconv_norm_destroy(tpconv_norm norm) {
  delete norm;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_norm_info(tpconv_norm norm, int64_t* features, int32_t* num_irreps, int64_t* num_weights,
                               int64_t* num_biases) {
  if (!norm) return TPCONV_ERROR_INVALID_VALUE;
  if (features) *features = norm->F;
  if (num_irreps) *num_irreps = (int32_t)norm->irreps.size();
  if (num_weights) *num_weights = norm->weights;
  if (num_biases) *num_biases = norm->biases;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_norm_workspace_size(tpconv_norm norm, int64_t num_nodes, size_t* bytes) {
  if (!norm || !bytes || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  NormArgs a = norm_args(*norm, num_nodes);
  *bytes = (size_t)norm_backward_blocks(a) * sizeof(float);
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_norm_forward(tpconv_norm norm, int64_t num_nodes, const void* x, const float* weight,
                                  const float* bias, void* y, float* stats, void* stream) {
  if (!norm || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  if (num_nodes == 0) return TPCONV_SUCCESS;
  if (!x || !y) return TPCONV_ERROR_INVALID_VALUE;
  NormArgs a = norm_args(*norm, num_nodes);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.stats = stats;
  return dev(launch_norm_forward(a, static_cast<hipStream_t>(stream)));
}

tpconv_status tpconv_norm_backward(tpconv_norm norm, int64_t num_nodes, const void* x, const float* weight,
                                   const float* grad_y, const float* stats, float* grad_x, float* grad_weight,
                                   float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  if (!norm || bad_count(num_nodes) || (!grad_x && !grad_weight && !grad_bias)) return TPCONV_ERROR_INVALID_VALUE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (norm->biases == 0) grad_bias = nullptr;
  if (num_nodes == 0) {
    if (grad_weight) {
      const tpconv_status st = dev(launch_fill(grad_weight, norm->weights, 0.f, s));
      if (st != TPCONV_SUCCESS) return st;
    }
    return grad_bias ? dev(launch_fill(grad_bias, norm->biases, 0.f, s)) : TPCONV_SUCCESS;
  }
  if (!x || !grad_y) return TPCONV_ERROR_INVALID_VALUE;
  NormArgs a = norm_args(*norm, num_nodes);
  const size_t need = (size_t)norm_backward_blocks(a) * sizeof(float);
  const bool params = grad_weight || grad_bias;
  if (params && bad_workspace(workspace, workspace_bytes, need)) return TPCONV_ERROR_WORKSPACE;
  if (!params && !grad_x) return TPCONV_SUCCESS;
  a.x = x;
  a.w = weight;
  a.gy = grad_y;
  a.stats = const_cast<float*>(stats);
  a.gx = grad_x;
  a.gw = grad_weight;
  a.gb = grad_bias;
  a.part = params ? static_cast<float*>(workspace) : nullptr;
  return dev(launch_norm_backward(a, s));
}

// ---- grouped linear layer ----------------------------------------------------------

tpconv_status tpconv_linear_create(tpconv_linear* out, const tpconv_linear_desc* desc) {
  if (!out || !desc) return TPCONV_ERROR_INVALID_VALUE;
  *out = nullptr;
  if (desc->num_groups < 1 || desc->num_groups > 4096 || bad_dtype(desc->x_dtype) || bad_dtype(desc->w_dtype) ||
      bad_dtype(desc->y_dtype))
    return TPCONV_ERROR_INVALID_VALUE;
  try {
    auto h = std::make_unique<tpconv_linear_s>();
    tpconv_status st = parse_side(desc->irreps_in, h->in, h->in_off, h->F_in);
    if (st == TPCONV_SUCCESS) st = parse_side(desc->irreps_out, h->out, h->out_off, h->F_out);
    if (st == TPCONV_SUCCESS) {
      for (size_t i = 0; i < h->in.size(); ++i)
        for (size_t o = 0; o < h->out.size(); ++o) {
          if (h->in[i].l != h->out[o].l || h->in[i].parity != h->out[o].parity) continue;
          LinBlock b;
          b.i = (int32_t)i;
          b.o = (int32_t)o;
          b.mi = h->in[i].mul;
          b.mo = h->out[o].mul;
          b.n = 2 * h->in[i].l + 1;
          b.xoff = h->in_off[i];
          b.yoff = h->out_off[o];
          b.woff = h->w_numel;
          h->w_numel += (int64_t)b.mi * b.mo;
          h->blocks.push_back(b);
        }
      if ((int)h->blocks.size() > kMaxLinBlocks || h->w_numel > INT32_MAX) st = TPCONV_ERROR_UNSUPPORTED;
    }
    if (st != TPCONV_SUCCESS) return st;
    h->groups = desc->num_groups;
    h->x_dtype = desc->x_dtype;
    h->w_dtype = desc->w_dtype;
    h->y_dtype = desc->y_dtype;
    *out = h.release();
    return TPCONV_SUCCESS;
  } catch (...) {
    return TPCONV_ERROR_INVALID_VALUE;
  }
}

tpconv_status tpconv_linear_destroy(tpconv_linear linear) {
  delete linear;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_linear_info(tpconv_linear linear, int64_t* feat_in, int64_t* feat_out, int64_t* w_numel,
                                 int32_t* num_blocks) {
  if (!linear) return TPCONV_ERROR_INVALID_VALUE;
  if (feat_in) *feat_in = linear->F_in;
  if (feat_out) *feat_out = linear->F_out;
  if (w_numel) *w_numel = linear->w_numel;
  if (num_blocks) *num_blocks = (int32_t)linear->blocks.size();
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_linear_block(tpconv_linear linear, int32_t block, int32_t* irrep_idx, int32_t* shape,
                                  int64_t* offset) {
  if (!linear || block < 0 || block >= (int32_t)linear->blocks.size()) return TPCONV_ERROR_INVALID_VALUE;
  const LinBlock& b = linear->blocks[block];
  if (irrep_idx) {
    irrep_idx[0] = b.i;
    irrep_idx[1] = b.o;
  }
  if (shape) {
    shape[0] = b.mi;
    shape[1] = b.mo;
  }
  if (offset) *offset = b.woff;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_linear_groups_workspace_size(tpconv_linear linear, int64_t num_nodes, size_t* bytes) {
  if (!linear || !bytes || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  *bytes = lin_groups_workspace(num_nodes, linear->groups);
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_linear_groups(tpconv_linear linear, int64_t num_nodes, const int32_t* group, int32_t* offsets,
                                   int32_t* order, int32_t validate, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!linear || bad_count(num_nodes) || !offsets || (num_nodes > 0 && (!group || !order)))
    return TPCONV_ERROR_INVALID_VALUE;
  if (bad_workspace(workspace, workspace_bytes, lin_groups_workspace(num_nodes, linear->groups)))
    return TPCONV_ERROR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (validate && num_nodes > 0) {
    int32_t* flag = static_cast<int32_t*>(workspace);
    if (launch_lin_groups_validate(group, num_nodes, linear->groups, flag, s) != hipSuccess)
      return TPCONV_ERROR_DEVICE;
    int32_t bad = 0;
    if (hipMemcpyAsync(&bad, flag, sizeof(bad), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
      return TPCONV_ERROR_DEVICE;
    if (bad) return TPCONV_ERROR_GRAPH;
  }
  return dev(launch_lin_groups(group, num_nodes, linear->groups, offsets, order, workspace, s));
}

tpconv_status tpconv_linear_workspace_size(tpconv_linear linear, int32_t op, int64_t num_nodes, size_t* bytes) {
  if (!linear || !bytes || bad_count(num_nodes) || (op != TPCONV_OP_FORWARD && op != TPCONV_OP_BACKWARD))
    return TPCONV_ERROR_INVALID_VALUE;
  *bytes = linear_workspace(*linear, op, num_nodes);
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_linear_forward(tpconv_linear linear, int64_t num_nodes, const int32_t* offsets,
                                    const int32_t* order, const void* x, const void* W, void* y, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const tpconv_status st = linear_inputs(linear, num_nodes, offsets, order);
  if (st != TPCONV_SUCCESS) return st;
  if (num_nodes == 0) return TPCONV_SUCCESS;
  if (!x || !y || (!W && linear->w_numel > 0)) return TPCONV_ERROR_INVALID_VALUE;
  const size_t need = linear_workspace(*linear, TPCONV_OP_FORWARD, num_nodes);
  if (bad_workspace(workspace, workspace_bytes, need)) return TPCONV_ERROR_WORKSPACE;
  LinRowsArgs a;
  rows_args(*linear, false, num_nodes, offsets, order, x, W, y, a);
  return dev(launch_lin_rows(a, static_cast<hipStream_t>(stream)));
}

tpconv_status tpconv_linear_backward(tpconv_linear linear, int64_t num_nodes, const int32_t* offsets,
                                     const int32_t* order, const void* x, const void* W, const float* grad_y,
                                     float* grad_x, float* grad_W, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  const tpconv_status st = linear_inputs(linear, num_nodes, offsets, order);
  if (st != TPCONV_SUCCESS) return st;
  if (!grad_x && !grad_W) return TPCONV_ERROR_INVALID_VALUE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (num_nodes == 0)
    return grad_W ? dev(launch_fill(grad_W, linear->w_numel * linear->groups, 0.f, s)) : TPCONV_SUCCESS;
  if (!grad_y || (grad_x && !W && linear->w_numel > 0) || (grad_W && !x)) return TPCONV_ERROR_INVALID_VALUE;
  const size_t need = grad_W ? linear_workspace(*linear, TPCONV_OP_BACKWARD, num_nodes) : 0;
  if (bad_workspace(workspace, workspace_bytes, need)) return TPCONV_ERROR_WORKSPACE;
  LinBackwardArgs a;
  std::memset(&a, 0, sizeof(a));
  if (grad_x) rows_args(*linear, true, num_nodes, offsets, order, grad_y, W, grad_x, a.rows);
  if (grad_W && !linear->blocks.empty())
    gw_args(*linear, num_nodes, offsets, order, x, grad_y, grad_W, static_cast<float*>(workspace), a.gw);
  a.rows.w_bf16 = linear->w_dtype == TPCONV_BF16;
  a.gw.x_bf16 = linear->x_dtype == TPCONV_BF16;
  if (a.rows.njobs == 0 && a.gw.njobs == 0) return TPCONV_SUCCESS;
  return dev(launch_lin_backward(a, s));
}

// ---- orthogonalised update ----------------------------------------------------------

tpconv_status tpconv_muon_create(tpconv_muon* out, const tpconv_muon_desc* desc) {
  if (!out || !desc) return TPCONV_ERROR_INVALID_VALUE;
  *out = nullptr;
  if (desc->num_blocks < 1 || desc->num_blocks > kMaxMuonBlocks || !desc->blocks || desc->num_steps < 1 ||
      desc->num_steps > kMaxMuonSteps || !desc->coefficients || !(desc->eps > 0.f) || std::isinf(desc->eps))
    return TPCONV_ERROR_INVALID_VALUE;
  try {
    for (int i = 0; i < desc->num_blocks; ++i) {
      const tpconv_matrix_block& b = desc->blocks[i];
      if (b.rows < 1 || b.cols < 1 || b.rows > 32768 || b.cols > 32768 || b.count < 0 || b.count > 65535 ||
          b.offset < 0 || b.stride < (int64_t)b.rows * b.cols || b.stride > (int64_t(1) << 40) ||
          b.offset > (int64_t(1) << 56))
        return TPCONV_ERROR_INVALID_VALUE;
    }
    auto h = std::make_unique<tpconv_muon_s>();
    MuonPlan& p = h->plan;
    p.nsteps = desc->num_steps;
    p.eps = desc->eps;
    p.nblocks = desc->num_blocks;
    for (int i = 0; i < p.nblocks; ++i) {
      const tpconv_matrix_block& b = desc->blocks[i];
      p.block[i] = {b.rows, b.cols, b.count, b.offset, b.stride};
    }
    double top = 1.0;
    bool ok = true;
    for (int k = 0; k < p.nsteps && ok; ++k) {
      MuonStep& t = p.step[k];
      t.a = desc->coefficients[3 * k];
      t.b = desc->coefficients[3 * k + 1];
      t.c = desc->coefficients[3 * k + 2];
      double x = 0.0, poly = 0.0;
      bounds(t.a, t.b, t.c, top, x, poly);
      ok = std::isfinite(x) && std::isfinite(poly) && exponent(top, t.ex) && exponent(top * top, t.ea) &&
           exponent(poly, t.eb);
      top = x;
    }
    ok = ok && exponent(top, p.step[p.nsteps].ex);
    if (!ok) return TPCONV_ERROR_INVALID_VALUE;  // coefficients that are not finite or let X grow past any use
    *out = h.release();
    return TPCONV_SUCCESS;
  } catch (...) {
    return TPCONV_ERROR_INVALID_VALUE;
  }
}

tpconv_status tpconv_muon_destroy(tpconv_muon muon) {
  delete muon;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_muon_workspace_size(tpconv_muon muon, size_t* bytes) {
  if (!muon || !bytes) return TPCONV_ERROR_INVALID_VALUE;
  *bytes = muon_workspace(muon->plan);
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_plan_weight_blocks(tpconv_plan plan, tpconv_matrix_block* blocks, int32_t capacity,
                                        int32_t* count) {
  if (!plan || !count) return TPCONV_ERROR_INVALID_VALUE;
  const Plan& p = plan->plan;
  if (p.connection != TPCONV_FULLY_CONNECTED) return TPCONV_ERROR_UNSUPPORTED;
  *count = p.P == 0 ? 0 : p.ragged ? p.P : 1;
  if (!blocks) return TPCONV_SUCCESS;
  if (capacity < *count) return TPCONV_ERROR_INVALID_VALUE;
  for (int i = 0; i < *count; ++i) {
    tpconv_matrix_block& b = blocks[i];
    if (p.ragged)
      b = {p.rag.mul_in[p.paths[i].i1], p.rag.mul_out[p.paths[i].i3], p.K, p.rag.woff[i], p.rag.W_per_k};
    else
      b = {p.C_in, p.C_out, (int64_t)p.K * p.P, 0, (int64_t)p.C_in * p.C_out};
  }
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_linear_weight_blocks(tpconv_linear linear, tpconv_matrix_block* blocks, int32_t capacity,
                                          int32_t* count) {
  if (!linear || !count) return TPCONV_ERROR_INVALID_VALUE;
  *count = (int32_t)linear->blocks.size();
  if (!blocks) return TPCONV_SUCCESS;
  if (capacity < *count) return TPCONV_ERROR_INVALID_VALUE;
  for (int i = 0; i < *count; ++i) {
    const LinBlock& b = linear->blocks[i];
    blocks[i] = {b.mi, b.mo, linear->groups, b.woff, linear->w_numel};
  }
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_muon_orthogonalize(tpconv_muon muon, const float* u, float* out, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (!muon || !u || !out) return TPCONV_ERROR_INVALID_VALUE;
  const size_t need = muon_workspace(muon->plan);
  if (bad_workspace(workspace, workspace_bytes, need)) return TPCONV_ERROR_WORKSPACE;
  MuonUpdate a{};
  a.u = u;
  a.out = out;
  return dev(launch_muon(muon->plan, a, workspace, static_cast<hipStream_t>(stream)));
}

tpconv_status tpconv_muon_step(tpconv_muon muon, const tpconv_muon_step_args* args, const float* W,
                               const float* grad, const float* momentum, float* W_out, float* momentum_out,
                               void* W_bf16, void* workspace, size_t workspace_bytes, void* stream) {
  if (!muon || !args || !W || !grad || !momentum || !W_out || !momentum_out) return TPCONV_ERROR_INVALID_VALUE;
  if (!std::isfinite(args->lr) || !std::isfinite(args->weight_decay) || !(args->beta >= 0.f) || !(args->beta < 1.f) ||
      (args->nesterov != 0 && args->nesterov != 1))
    return TPCONV_ERROR_INVALID_VALUE;
  const size_t need = muon_workspace(muon->plan);
  if (bad_workspace(workspace, workspace_bytes, need)) return TPCONV_ERROR_WORKSPACE;
  MuonUpdate a{};
  a.W = W;
  a.grad = grad;
  a.mom = momentum;
  a.out = W_out;
  a.mom_out = momentum_out;
  a.w_bf16 = static_cast<uint16_t*>(W_bf16);
  a.lr = args->lr;
  a.beta = args->beta;
  a.decay = args->weight_decay;
  a.nesterov = args->nesterov;
  return dev(launch_muon(muon->plan, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
