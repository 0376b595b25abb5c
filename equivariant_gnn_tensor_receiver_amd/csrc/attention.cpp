// C ABI of the attention block's operators (declared in
// include/tpconv_attention.h): handles, argument checks, workspace sizes, and
// the launches' argument blocks.
#include "attention.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <vector>

#include "kernels.h"

struct tpconv_attention_s {
  tpconv::AttnSide qk, v;
  int32_t heads = 0;
  float scale = 0.f, cap = 0.f;
  int x_dtype = 0, y_dtype = 0;
};

struct tpconv_embed_s {
  int32_t rows = 0, features = 0;
  float scale = 0.f;
  int w_dtype = 0, y_dtype = 0;
};

struct tpconv_dropout_s {
  tpconv::DropArgs args;
};

namespace tpconv {
namespace {

tpconv_status dev(hipError_t e) { return e == hipSuccess ? TPCONV_SUCCESS : TPCONV_ERROR_DEVICE; }
bool bad_dtype(int t) { return t != TPCONV_F32 && t != TPCONV_BF16; }
bool bad_workspace(const void* ws, size_t bytes, size_t need) {
  return need > 0 && (!ws || bytes < need || reinterpret_cast<uintptr_t>(ws) % 16 != 0);
}
bool bad_count(int64_t n) { return n < 0 || n >= INT32_MAX; }

tpconv_status parse(const char* text, std::vector<Irrep>& ir) {
  if (!text) return TPCONV_ERROR_INVALID_VALUE;
  if (!parse_irreps(text, ir)) return TPCONV_ERROR_IRREPS;
  if ((int)ir.size() > kMaxGroups) return TPCONV_ERROR_UNSUPPORTED;
  int64_t F = 0;
  for (const auto& i : ir) {
    if (i.l > kMaxL) return TPCONV_ERROR_UNSUPPORTED;
    F += (int64_t)i.mul * (2 * i.l + 1);
  }
  return F <= INT32_MAX / 2 ? TPCONV_SUCCESS : TPCONV_ERROR_UNSUPPORTED;
}

tpconv_status parse_side(const char* text, int heads, AttnSide& s) {
  std::vector<Irrep> ir;
  const tpconv_status st = parse(text, ir);
  if (st != TPCONV_SUCCESS) return st;
  std::memset(&s, 0, sizeof(s));
  s.nirr = (int32_t)ir.size();
  s.vec = 1;
  int64_t F = 0, D = 0;
  for (int i = 0; i < s.nirr; ++i) {
    if (ir[i].mul % heads != 0) return TPCONV_ERROR_IRREPS;
    const int32_t cph = ir[i].mul / heads;
    s.ir[i] = {(int32_t)F, ir[i].mul, cph, (int32_t)D};
    if (cph % 4 != 0) s.vec = 0;
    F += (int64_t)ir[i].mul * (2 * ir[i].l + 1);
    D += (int64_t)cph * (2 * ir[i].l + 1);
    if (D > kAttnMaxHead) return TPCONV_ERROR_UNSUPPORTED;
  }
  s.F = (int32_t)F;
  s.D = (int32_t)D;
  return TPCONV_SUCCESS;
}

// What a call of these counts needs: shapes of its launches and the workspace's parts (in floats).
struct AttnPlan {
  AttnShape fwd, q, kv;
  size_t part_o, part_ml;                                         // forward
  size_t delta, gq, gk, gv, qpos, kpos, slope;                    // backward
  size_t floats;
};

// Floats behind one another, each part on a 16-byte boundary.
struct Taker {
  size_t at = 0;
  size_t operator()(size_t n) {
    const size_t o = at;
    at += (n + 3) / 4 * 4;
    return o;
  }
};

int64_t keys_of(const tpconv_attention_batch& b) { return b.key_offsets ? b.num_keys : b.num_queries; }

// Blocks of a launch: their threads must stay below 2^32.
bool too_many(const AttnShape& s, int heads) {
  return s.tiles > (int64_t(1) << 40) / (heads * s.nsplit) ||
         (s.tiles * heads * s.nsplit + 8) * 4 * s.cols >= (int64_t(1) << 32);
}

// saves: a forward that leaves fp32 results (or saves them), in which the sums of a graph's runs fit
tpconv_status plan_of(const tpconv_attention_s& h, int op, const tpconv_attention_batch& b, bool saves, AttnPlan& p) {
  std::memset(&p, 0, sizeof(p));
  const int64_t Nq = b.num_queries, Nk = keys_of(b), H = h.heads;
  const int D = std::max(h.qk.D, h.v.D);
  Taker take;
  if (op == TPCONV_OP_FORWARD) {
    p.fwd = attn_shape(D, Nq, Nk, b.num_graphs, h.heads, h.y_dtype == TPCONV_F32);
    if (too_many(p.fwd, h.heads)) return TPCONV_ERROR_UNSUPPORTED;
    if (p.fwd.nsplit > 1) {
      p.part_o = take((size_t)p.fwd.nsplit * Nq * h.v.F);
      p.part_ml = take((size_t)p.fwd.nsplit * H * Nq * 2);
    } else if (Nk > kAttnRun && !saves) {
      p.part_o = take((size_t)Nq * h.v.F);
    }
  } else {
    p.q = attn_shape(D, Nq, Nk, b.num_graphs, h.heads, true);
    p.kv = attn_shape(D, Nk, Nq, b.num_graphs, h.heads, true);
    if (too_many(p.q, h.heads) || too_many(p.kv, h.heads)) return TPCONV_ERROR_UNSUPPORTED;
    p.delta = take((size_t)H * Nq);
    if (p.q.nsplit > 1) p.gq = take((size_t)p.q.nsplit * Nq * h.qk.F);
    if (p.kv.nsplit > 1) {
      p.gk = take((size_t)p.kv.nsplit * Nk * h.qk.F);
      p.gv = take((size_t)p.kv.nsplit * Nk * h.v.F);
    }
    if (b.pos || (b.key_offsets && b.key_pos)) {
      p.qpos = take((size_t)p.q.nsplit * H * Nq * 3);
      p.kpos = take((size_t)p.kv.nsplit * H * Nk * 3);
      p.slope = take((size_t)p.q.nsplit * H * Nq * 3);
    }
  }
  p.floats = take.at;
  return TPCONV_SUCCESS;
}

tpconv_status check_batch(const tpconv_attention_s* h, const tpconv_attention_batch* b) {
  if (!h || !b || bad_count(b->num_queries) || bad_count(b->num_graphs)) return TPCONV_ERROR_INVALID_VALUE;
  if (!b->offsets && b->num_graphs != 1) return TPCONV_ERROR_INVALID_VALUE;
  if (b->key_offsets && (bad_count(b->num_keys) || !b->offsets)) return TPCONV_ERROR_INVALID_VALUE;
  return TPCONV_SUCCESS;
}

bool bad_stride(int64_t ld, int64_t F) { return ld != 0 && (ld < F || ld > (int64_t(1) << 40)); }

// Checks the tensors of a call and fills what its launches share.
tpconv_status common_args(const tpconv_attention_s& h, const tpconv_attention_batch& b,
                          const tpconv_attention_inputs* in, AttnArgs& a) {
  std::memset(&a, 0, sizeof(a));
  if (!in || bad_stride(in->q_stride, h.qk.F) || bad_stride(in->k_stride, h.qk.F) || bad_stride(in->v_stride, h.v.F))
    return TPCONV_ERROR_INVALID_VALUE;
  const int64_t Nk = keys_of(b);
  if ((b.num_queries > 0 && !in->q) || (Nk > 0 && (!in->k || !in->v))) return TPCONV_ERROR_INVALID_VALUE;
  if (in->slope) {
    if ((b.num_queries > 0 && !b.pos) || (b.key_offsets && Nk > 0 && !b.key_pos)) return TPCONV_ERROR_INVALID_VALUE;
    a.slope = in->slope;
    a.qpos = b.pos;
    a.kpos = b.key_offsets ? b.key_pos : b.pos;
  }
  a.H = h.heads;
  a.G = (int32_t)b.num_graphs;
  a.self = !b.key_offsets;
  a.x_bf16 = h.x_dtype == TPCONV_BF16;
  a.y_bf16 = h.y_dtype == TPCONV_BF16;
  a.scale = h.scale;
  a.cap = h.cap;
  a.Nq = b.num_queries;
  a.Nk = Nk;
  a.qo = b.offsets;
  a.ko = b.key_offsets ? b.key_offsets : b.offsets;
  a.q = in->q;
  a.k = in->k;
  a.v = in->v;
  a.ldq = in->q_stride ? in->q_stride : h.qk.F;
  a.ldk = in->k_stride ? in->k_stride : h.qk.F;
  a.ldv = in->v_stride ? in->v_stride : h.v.F;
  a.sqk = h.qk;
  a.sv = h.v;
  return TPCONV_SUCCESS;
}

}  // namespace
}  // namespace tpconv

using namespace tpconv;

extern "C" {

// ---- attention ----------------------------------------------------------------------

tpconv_status tpconv_attention_create(tpconv_attention* out, const tpconv_attention_desc* desc) {
  if (!out || !desc) return TPCONV_ERROR_INVALID_VALUE;
  *out = nullptr;
  const float cap = desc->score_cap, most = 0x1p100f;  // with these, what the kernels make of them is in range
  if (desc->num_heads < 1 || desc->num_heads > 256 || !(std::fabs(desc->scale) <= most) ||
      !(cap == 0.f || (cap >= 1.f / most && cap <= most && std::isfinite(desc->scale / cap))) ||
      bad_dtype(desc->x_dtype) || bad_dtype(desc->y_dtype))
    return TPCONV_ERROR_INVALID_VALUE;
  try {
    auto h = std::make_unique<tpconv_attention_s>();
    tpconv_status st = parse_side(desc->irreps_qk, desc->num_heads, h->qk);
    if (st == TPCONV_SUCCESS) st = parse_side(desc->irreps_v, desc->num_heads, h->v);
    if (st != TPCONV_SUCCESS) return st;
    h->heads = desc->num_heads;
    h->scale = desc->scale;
    h->cap = cap;
    h->x_dtype = desc->x_dtype;
    h->y_dtype = desc->y_dtype;
    *out = h.release();
    return TPCONV_SUCCESS;
  } catch (...) {
    return TPCONV_ERROR_INVALID_VALUE;
  }
}

tpconv_status tpconv_attention_destroy(tpconv_attention attention) {
  delete attention;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_attention_info(tpconv_attention attention, int64_t* feat_qk, int64_t* feat_v, int32_t* head_qk,
                                    int32_t* head_v) {
  if (!attention) return TPCONV_ERROR_INVALID_VALUE;
  if (feat_qk) *feat_qk = attention->qk.F;
  if (feat_v) *feat_v = attention->v.F;
  if (head_qk) *head_qk = attention->qk.D;
  if (head_v) *head_v = attention->v.D;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_attention_saved_size(tpconv_attention attention, int64_t num_queries, int64_t* values) {
  if (!attention || !values || bad_count(num_queries)) return TPCONV_ERROR_INVALID_VALUE;
  *values = 2 * num_queries * attention->heads;
  if (attention->y_dtype == TPCONV_BF16) *values += num_queries * attention->v.F;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_attention_workspace_size(tpconv_attention attention, int32_t op,
                                              const tpconv_attention_batch* batch, size_t* bytes) {
  tpconv_status st = check_batch(attention, batch);
  if (st != TPCONV_SUCCESS) return st;
  if (!bytes || (op != TPCONV_OP_FORWARD && op != TPCONV_OP_BACKWARD)) return TPCONV_ERROR_INVALID_VALUE;
  AttnPlan p;
  st = plan_of(*attention, op, *batch, attention->y_dtype == TPCONV_F32, p);
  if (st == TPCONV_SUCCESS) *bytes = p.floats * sizeof(float);
  return st;
}

tpconv_status tpconv_attention_forward(tpconv_attention attention, const tpconv_attention_batch* batch,
                                       const tpconv_attention_inputs* in, void* out, float* saved, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  tpconv_status st = check_batch(attention, batch);
  if (st != TPCONV_SUCCESS) return st;
  AttnArgs a;
  st = common_args(*attention, *batch, in, a);
  if (st != TPCONV_SUCCESS) return st;
  if (a.Nq == 0 || a.G == 0) return TPCONV_SUCCESS;
  if (!out) return TPCONV_ERROR_INVALID_VALUE;
  AttnPlan p;
  st = plan_of(*attention, TPCONV_OP_FORWARD, *batch, saved || !a.y_bf16, p);
  if (st != TPCONV_SUCCESS) return st;
  if (bad_workspace(workspace, workspace_bytes, p.floats * sizeof(float))) return TPCONV_ERROR_WORKSPACE;
  float* ws = static_cast<float*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.out = out;
  a.stat = saved;
  if (saved && a.y_bf16) a.out32 = saved + 2 * a.Nq * a.H;
  const bool parts = p.fwd.nsplit > 1;
  a.sums = parts || (a.y_bf16 && !saved) ? ws + p.part_o : a.y_bf16 ? a.out32 : static_cast<float*>(out);
  a.put_f32 = parts || !a.y_bf16 || saved;
  a.put_bf16 = !parts && a.y_bf16;
  a.part_ml = ws + p.part_ml;
  st = dev(launch_attn_forward(a, p.fwd, s));
  if (st == TPCONV_SUCCESS && parts) st = dev(launch_attn_combine(a, p.fwd, s));
  return st;
}

tpconv_status tpconv_attention_backward(tpconv_attention attention, const tpconv_attention_batch* batch,
                                        const tpconv_attention_inputs* in, const void* out, const float* saved,
                                        const float* grad_out, const tpconv_attention_grads* grads,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  tpconv_status st = check_batch(attention, batch);
  if (st != TPCONV_SUCCESS) return st;
  const tpconv_attention_s& h = *attention;
  AttnArgs a;
  st = common_args(h, *batch, in, a);
  if (st != TPCONV_SUCCESS) return st;
  if (!grads || bad_stride(grads->q_stride, h.qk.F) || bad_stride(grads->k_stride, h.qk.F) ||
      bad_stride(grads->v_stride, h.v.F))
    return TPCONV_ERROR_INVALID_VALUE;
  const tpconv_attention_grads& g = *grads;
  const bool pos = g.grad_pos || g.grad_key_pos;
  if (!g.grad_q && !g.grad_k && !g.grad_v && !g.grad_slope && !pos) return TPCONV_ERROR_INVALID_VALUE;
  if (((pos || g.grad_slope) && !a.slope) || (g.grad_key_pos && a.self)) return TPCONV_ERROR_INVALID_VALUE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.G == 0 || (a.Nq == 0 && a.Nk == 0)) return g.grad_slope ? dev(launch_fill(g.grad_slope, a.H, 0.f, s)) : TPCONV_SUCCESS;
  if (a.Nq > 0 && (!out || !saved || !grad_out)) return TPCONV_ERROR_INVALID_VALUE;
  AttnPlan p;
  st = plan_of(h, TPCONV_OP_BACKWARD, *batch, true, p);
  if (st != TPCONV_SUCCESS) return st;
  if (bad_workspace(workspace, workspace_bytes, p.floats * sizeof(float))) return TPCONV_ERROR_WORKSPACE;
  float* ws = static_cast<float*>(workspace);
  a.stat = const_cast<float*>(saved);
  a.go = grad_out;
  a.o = a.y_bf16 ? saved + 2 * a.Nq * a.H : static_cast<const float*>(out);
  a.delta = ws + p.delta;

  AttnJoinArgs j;
  std::memset(&j, 0, sizeof(j));
  j.H = a.H;
  j.G = a.G;
  j.nsplit_q = p.q.nsplit;
  j.nsplit_k = p.kv.nsplit;
  j.Nq = a.Nq;
  j.Nk = a.Nk;
  j.qo = a.qo;
  j.ko = a.ko;
  j.gq = g.grad_q;
  j.gk = g.grad_k;
  j.gv = g.grad_v;
  j.ldgq = g.q_stride ? g.q_stride : h.qk.F;
  j.ldgk = g.k_stride ? g.k_stride : h.qk.F;
  j.ldgv = g.v_stride ? g.v_stride : h.v.F;
  j.Fqk = h.qk.F;
  j.Fv = h.v.F;
  j.gpos = g.grad_pos;
  j.gkpos = g.grad_key_pos;
  j.gslope = g.grad_slope;

  // the queries' side: also what the keys' side reads of every query (delta)
  const bool keys = g.grad_k || g.grad_v || (pos && (a.self || g.grad_key_pos));
  if (a.Nq > 0) {
    AttnArgs b = a;
    if (g.grad_q) {
      if (p.q.nsplit > 1) {
        b.gq = ws + p.gq;
        b.ldgq = h.qk.F;
        j.part_gq = b.gq;
      } else {
        b.gq = g.grad_q;
        b.ldgq = j.ldgq;
      }
    }
    if (g.grad_pos) j.part_qpos = b.part_pos = ws + p.qpos;
    if (g.grad_slope) j.part_slope = b.part_slope = ws + p.slope;
    st = dev(launch_attn_grad_q(b, p.q, s));
    if (st != TPCONV_SUCCESS) return st;
  }
  if (keys && a.Nk > 0) {
    AttnArgs b = a;
    const bool parts = p.kv.nsplit > 1;
    if (g.grad_k) {
      b.gk = parts ? ws + p.gk : g.grad_k;
      b.ldgk = parts ? h.qk.F : j.ldgk;
      if (parts) j.part_gk = b.gk;
    }
    if (g.grad_v) {
      b.gv = parts ? ws + p.gv : g.grad_v;
      b.ldgv = parts ? h.v.F : j.ldgv;
      if (parts) j.part_gv = b.gv;
    }
    if (pos && (a.self || g.grad_key_pos)) j.part_kpos = b.part_pos = ws + p.kpos;
    st = dev(launch_attn_grad_kv(b, p.kv, s));
    if (st != TPCONV_SUCCESS) return st;
  }
  if (j.part_gq || j.part_gk || j.part_gv || pos || g.grad_slope) st = dev(launch_attn_join(j, s));
  return st;
}

// ---- embedding ------------------------------------------------------------------------

tpconv_status tpconv_embed_create(tpconv_embed* out, const tpconv_embed_desc* desc) {
  if (!out || !desc) return TPCONV_ERROR_INVALID_VALUE;
  *out = nullptr;
  if (desc->num_rows < 1 || desc->num_rows > (1 << 24) || desc->features < 1 || desc->features > 65536 ||
      !std::isfinite(desc->scale) || bad_dtype(desc->w_dtype) || bad_dtype(desc->y_dtype))
    return TPCONV_ERROR_INVALID_VALUE;
  try {
    auto h = std::make_unique<tpconv_embed_s>();
    h->rows = desc->num_rows;
    h->features = desc->features;
    h->scale = desc->scale;
    h->w_dtype = desc->w_dtype;
    h->y_dtype = desc->y_dtype;
    *out = h.release();
    return TPCONV_SUCCESS;
  } catch (...) {
    return TPCONV_ERROR_INVALID_VALUE;
  }
}

tpconv_status tpconv_embed_destroy(tpconv_embed embed) {
  delete embed;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_embed_workspace_size(tpconv_embed embed, int64_t num_nodes, size_t* bytes) {
  if (!embed || !bytes || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  *bytes = embed_workspace(embed->rows, embed->features, num_nodes);
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_embed_forward(tpconv_embed embed, int64_t num_nodes, const int32_t* index, const void* W, void* y,
                                   void* stream) {
  if (!embed || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  if (num_nodes == 0) return TPCONV_SUCCESS;
  if (!index || !W || !y) return TPCONV_ERROR_INVALID_VALUE;
  EmbedArgs a{};
  a.rows = embed->rows;
  a.features = embed->features;
  a.w_bf16 = embed->w_dtype == TPCONV_BF16;
  a.y_bf16 = embed->y_dtype == TPCONV_BF16;
  a.scale = embed->scale;
  a.N = num_nodes;
  a.index = index;
  a.W = W;
  a.y = y;
  return dev(launch_embed_forward(a, static_cast<hipStream_t>(stream)));
}

tpconv_status tpconv_embed_backward(tpconv_embed embed, int64_t num_nodes, const int32_t* index, const float* grad_y,
                                    float* grad_W, void* workspace, size_t workspace_bytes, void* stream) {
  if (!embed || bad_count(num_nodes) || !grad_W || (num_nodes > 0 && (!index || !grad_y)))
    return TPCONV_ERROR_INVALID_VALUE;
  if (bad_workspace(workspace, workspace_bytes, embed_workspace(embed->rows, embed->features, num_nodes)))
    return TPCONV_ERROR_WORKSPACE;
  EmbedArgs a{};
  a.rows = embed->rows;
  a.features = embed->features;
  a.scale = embed->scale;
  a.N = num_nodes;
  a.index = index;
  a.gy = grad_y;
  a.gW = grad_W;
  return dev(launch_embed_backward(a, workspace, static_cast<hipStream_t>(stream)));
}

// ---- dropout ----------------------------------------------------------------------------

tpconv_status tpconv_dropout_create(tpconv_dropout* out, const tpconv_dropout_desc* desc) {
  if (!out || !desc) return TPCONV_ERROR_INVALID_VALUE;
  *out = nullptr;
  if (!(desc->p >= 0.f) || !(desc->p <= 1.f) || bad_dtype(desc->x_dtype) || bad_dtype(desc->y_dtype))
    return TPCONV_ERROR_INVALID_VALUE;
  try {
    std::vector<Irrep> ir;
    const tpconv_status st = parse(desc->irreps, ir);
    if (st != TPCONV_SUCCESS) return st;
    auto h = std::make_unique<tpconv_dropout_s>();
    DropArgs& a = h->args;
    std::memset(&a, 0, sizeof(a));
    a.nirr = (int32_t)ir.size();
    for (int i = 0; i < a.nirr; ++i) {
      a.ir[i] = {ir[i].mul, 2 * ir[i].l + 1, (int32_t)a.F, a.groups};
      a.F += (int64_t)ir[i].mul * (2 * ir[i].l + 1);
      a.groups += (ir[i].mul + 7) / 8;
    }
    a.x_bf16 = desc->x_dtype == TPCONV_BF16;
    a.y_bf16 = desc->y_dtype == TPCONV_BF16;
    a.limit = (int32_t)std::nearbyint((double)desc->p * 65536.0);
    a.factor = a.limit < 65536 ? (float)(65536.0 / (65536 - a.limit)) : 0.f;
    *out = h.release();
    return TPCONV_SUCCESS;
  } catch (...) {
    return TPCONV_ERROR_INVALID_VALUE;
  }
}

tpconv_status tpconv_dropout_destroy(tpconv_dropout dropout) {
  delete dropout;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_dropout_info(tpconv_dropout dropout, int64_t* features, float* p) {
  if (!dropout) return TPCONV_ERROR_INVALID_VALUE;
  if (features) *features = dropout->args.F;
  if (p) *p = (float)dropout->args.limit / 65536.f;
  return TPCONV_SUCCESS;
}

tpconv_status tpconv_dropout_forward(tpconv_dropout dropout, int64_t num_nodes, const void* x, const int64_t* rng,
                                     const void* residual, void* y, void* stream) {
  if (!dropout || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  if (num_nodes == 0) return TPCONV_SUCCESS;
  if (!x || !rng || !y || (y == x && dropout->args.x_bf16 != dropout->args.y_bf16)) return TPCONV_ERROR_INVALID_VALUE;
  DropArgs a = dropout->args;
  a.N = num_nodes;
  a.x = x;
  a.rng = rng;
  a.res = residual;
  a.has_res = residual != nullptr;
  a.y = y;
  return dev(launch_dropout(a, static_cast<hipStream_t>(stream)));
}

tpconv_status tpconv_dropout_backward(tpconv_dropout dropout, int64_t num_nodes, const float* grad_y,
                                      const int64_t* rng, float* grad_x, void* stream) {
  if (!dropout || bad_count(num_nodes)) return TPCONV_ERROR_INVALID_VALUE;
  if (num_nodes == 0) return TPCONV_SUCCESS;
  if (!grad_y || !rng || !grad_x) return TPCONV_ERROR_INVALID_VALUE;
  DropArgs a = dropout->args;
  a.x_bf16 = a.y_bf16 = 0;
  a.N = num_nodes;
  a.x = grad_y;
  a.rng = rng;
  a.y = grad_x;
  return dev(launch_dropout(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
