// C ABI of the block join and its gradient: argument validation and launches.
#include <cmath>

#include "api_util.hpp"
#include "join.hpp"
#include "mx4.hpp"

using namespace vggt3::api;
namespace join = vggt3::join;
namespace mx4 = vggt3::mx4;

namespace {

bool valid_norm(int32_t k) { return k == VGGT3_NORM_NONE || k == VGGT3_NORM_RMS || k == VGGT3_NORM_LAYER; }

int check_shape(int64_t n, int32_t C, int32_t dtype) {
  if (!valid_dtype(dtype)) return fail(VGGT3_EINVAL, "dtype %d is not VGGT3_BF16 or VGGT3_F32", dtype);
  if (n < 0) return fail(VGGT3_EINVAL, "n_tokens = %lld < 0", (long long)n);
  if (C < 1) return fail(VGGT3_EINVAL, "channels = %d < 1", C);
  if (C > join::kMaxChannels) return fail(VGGT3_EUNSUPPORTED, "channels = %d, at most %d", C, join::kMaxChannels);
  if (n > (int64_t)1 << 31) return fail(VGGT3_EUNSUPPORTED, "n_tokens = %lld, at most 2^31", (long long)n);
  return VGGT3_OK;
}

// What both directions share: the block's output with its gate and norms. (No
// tokens: f may be the NULL of an empty tensor, so has_f says true there.)
int check_join(bool has_f, const void* gate, int64_t gate_tokens, const float* scale, int32_t post, const float* post_w,
               const float* post_b, int32_t pre, const float* pre_w, const float* pre_b, float eps) {
  if (!valid_norm(post) || !valid_norm(pre)) return fail(VGGT3_EINVAL, "norm kind %d / %d", post, pre);
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(VGGT3_EINVAL, "eps = %g", (double)eps);
  if (!has_f && (gate || scale || post != VGGT3_NORM_NONE))
    return fail(VGGT3_EINVAL, "gate, residual scale and the norm after the block go with a block output f");
  if (gate && gate_tokens < 1) return fail(VGGT3_EINVAL, "gate_tokens = %lld < 1", (long long)gate_tokens);
  if (post == VGGT3_NORM_NONE && (post_w || post_b)) return fail(VGGT3_EINVAL, "post_w / post_b without a norm");
  if (pre == VGGT3_NORM_NONE && (pre_w || pre_b)) return fail(VGGT3_EINVAL, "pre_w / pre_b without a norm");
  return VGGT3_OK;
}

// Tokens that share a gate row: at most all of them.
int64_t tokens_per_gate(const void* gate, int64_t gate_tokens, int64_t n) {
  return gate == nullptr ? 1 : gate_tokens < n ? gate_tokens : n > 0 ? n : 1;
}
int64_t gate_rows(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Workspace of the gradient: [per-workgroup sums | shared gate groups' parts].
struct GradWs {
  size_t edge, total;
};
GradWs grad_ws(const join::GradPlan& p, int C) {
  GradWs l;
  l.edge = round256((size_t)p.blocks * join::kVecs * C * sizeof(float));
  l.total = l.edge + round256((size_t)p.units * 2 * C * sizeof(float));
  return l;
}

}  // namespace

extern "C" {

int vggt3_block_join(const void* x, const void* f, const void* gate, int64_t gate_tokens, const float* scale,
                     int32_t post, const float* post_w, const float* post_b, int32_t pre, const float* pre_w,
                     const float* pre_b, float eps, void* r, void* y, void* y_codes, void* y_scales, int64_t n_tokens,
                     int32_t channels, int32_t dtype, void* stream) {
  int rc = check_shape(n_tokens, channels, dtype);
  if (rc) return rc;
  const bool has_f = f != nullptr || n_tokens == 0;
  rc = check_join(has_f, gate, gate_tokens, scale, post, post_w, post_b, pre, pre_w, pre_b, eps);
  if (rc) return rc;
  if (!has_f && pre == VGGT3_NORM_NONE) return fail(VGGT3_EINVAL, "neither a block output nor a norm: nothing to do");
  if ((y_codes == nullptr) != (y_scales == nullptr)) return fail(VGGT3_EINVAL, "y_codes and y_scales go together");
  if (pre == VGGT3_NORM_NONE ? (y || y_codes) : n_tokens > 0 && (y != nullptr) == (y_codes != nullptr))
    return fail(VGGT3_EINVAL, pre == VGGT3_NORM_NONE ? "y without a norm before the next block"
                                                     : "give y or (y_codes, y_scales), one of them");
  if (n_tokens == 0) return ok();
  const int64_t per = tokens_per_gate(gate, gate_tokens, n_tokens);
  if (x == nullptr) return fail(VGGT3_EINVAL, "x is NULL");
  if (f && r == nullptr) return fail(VGGT3_EINVAL, "r is NULL");
  if (!f && r) return fail(VGGT3_EINVAL, "r goes with a block output f");
  const size_t tb = (size_t)n_tokens * channels * elem_size(dtype), vb = (size_t)channels * sizeof(float);
  const Region rs[] = {{"x", x, tb, false},
                       {"f", f, tb, false},
                       {"gate", gate, gate ? (size_t)gate_rows(n_tokens, per) * channels * elem_size(dtype) : 0, false},
                       {"scale", scale, vb, false},
                       {"post_w", post_w, vb, false},
                       {"post_b", post_b, vb, false},
                       {"pre_w", pre_w, vb, false},
                       {"pre_b", pre_b, vb, false},
                       {"r", r, tb, true},
                       {"y", y, tb, true},
                       {"y_codes", y_codes, (size_t)mx4::code_bytes(n_tokens, channels), true},
                       {"y_scales", y_scales, (size_t)mx4::scale_bytes(n_tokens, channels), true}};
  rc = check_regions(rs, 12, {{0, 8}});  // in place: r may be x
  if (rc) return rc;
  join::Args a{};
  a.x = x; a.f = f; a.gate = gate; a.scale = scale;
  a.post_w = post_w; a.post_b = post_b; a.pre_w = pre_w; a.pre_b = pre_b;
  a.r = r; a.y = y;
  a.y_codes = static_cast<uint8_t*>(y_codes); a.y_scales = static_cast<uint8_t*>(y_scales);
  a.n = n_tokens; a.per = per; a.C = channels; a.post = post; a.pre = pre; a.eps = eps;
  rc = check_hip(join::launch_forward(a, dtype == VGGT3_BF16, static_cast<hipStream_t>(stream)), "block join launch");
  return rc ? rc : ok();
}

size_t vggt3_block_join_grad_workspace_bytes(int64_t n_tokens, int32_t channels, int32_t dtype) {
  if (check_shape(n_tokens, channels, dtype) != VGGT3_OK || n_tokens == 0) return 0;
  return grad_ws(join::grad_plan(n_tokens, channels, dtype == VGGT3_BF16), channels).total;
}

int vggt3_block_join_grad(const void* r, const void* f, const void* gate, int64_t gate_tokens, const float* scale,
                          int32_t post, const float* post_w, const float* post_b, int32_t pre, const float* pre_w,
                          float eps, const void* dr, const void* dy, void* dx, void* df, void* dgate, float* dscale,
                          float* dpost_w, float* dpost_b, float* dpre_w, float* dpre_b, int64_t n_tokens,
                          int32_t channels, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(n_tokens, channels, dtype);
  if (rc) return rc;
  const bool has_f = f != nullptr || n_tokens == 0;
  rc = check_join(has_f, gate, gate_tokens, scale, post, post_w, post_b, pre, pre_w, nullptr, eps);
  if (rc) return rc;
  if (!has_f && (df || dgate || dscale || dpost_w || dpost_b))
    return fail(VGGT3_EINVAL, "gradients of the block output, its gate, scale and norm go with f");
  if (!has_f && pre == VGGT3_NORM_NONE) return fail(VGGT3_EINVAL, "neither a block output nor a norm: nothing to do");
  if (dgate && !gate) return fail(VGGT3_EINVAL, "dgate without a gate");
  if (post == VGGT3_NORM_NONE && (dpost_w || dpost_b)) return fail(VGGT3_EINVAL, "dpost_w / dpost_b without a norm");
  if (pre == VGGT3_NORM_NONE && (dpre_w || dpre_b || dy)) return fail(VGGT3_EINVAL, "dy / dpre_w / dpre_b without a norm");
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* outs[join::kOuts];
  outs[join::kDScale] = dscale;
  outs[join::kDPostW] = dpost_w;
  outs[join::kDPostB] = dpost_b;
  outs[join::kDPreW] = dpre_w;
  outs[join::kDPreB] = dpre_b;
  const size_t vb = (size_t)channels * sizeof(float);
  const join::GradPlan p = n_tokens > 0 ? join::grad_plan(n_tokens, channels, dtype == VGGT3_BF16) : join::GradPlan{};
  const GradWs l = n_tokens > 0 ? grad_ws(p, channels) : GradWs{};
  if (n_tokens > 0) {
    if (pre != VGGT3_NORM_NONE && (r == nullptr || dy == nullptr))
      return fail(VGGT3_EINVAL, "%s is NULL", r == nullptr ? "r" : "dy");
    if (pre == VGGT3_NORM_NONE && dr == nullptr) return fail(VGGT3_EINVAL, "dr is NULL");
    if (workspace == nullptr || workspace_bytes < l.total)
      return fail(VGGT3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, l.total);
  }
  const size_t tb = (size_t)n_tokens * channels * elem_size(dtype);
  const int64_t per = tokens_per_gate(gate, gate_tokens, n_tokens);
  const size_t gb = gate ? (size_t)gate_rows(n_tokens, per) * channels * elem_size(dtype) : 0;
  const Region rs[] = {{"r", r, tb, false},           {"f", f, tb, false},
                       {"gate", gate, gb, false},     {"scale", scale, vb, false},
                       {"post_w", post_w, vb, false}, {"post_b", post_b, vb, false},
                       {"pre_w", pre_w, vb, false},   {"dr", dr, tb, false},
                       {"dy", dy, tb, false},         {"dx", dx, tb, true},
                       {"df", df, tb, true},          {"dgate", dgate, gb, true},
                       {"dscale", dscale, vb, true},  {"dpost_w", dpost_w, vb, true},
                       {"dpost_b", dpost_b, vb, true}, {"dpre_w", dpre_w, vb, true},
                       {"dpre_b", dpre_b, vb, true},  {"workspace", n_tokens > 0 ? workspace : nullptr, l.total, true}};
  rc = check_regions(rs, 18, {{7, 9}});  // in place: dx may be dr
  if (rc) return rc;
  join::Args a{};
  a.x = r; a.f = f; a.gate = gate; a.scale = scale;
  a.post_w = post_w; a.post_b = post_b; a.pre_w = pre_w;
  a.dr = dr; a.dy = dy; a.dx = dx; a.df = df; a.dgate = dgate;
  a.part = static_cast<float*>(workspace);
  a.edge = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.edge);
  a.n = n_tokens; a.per = per; a.C = channels; a.post = post; a.pre = pre; a.eps = eps;
  rc = check_hip(join::launch_grad(a, p, outs, dtype == VGGT3_BF16, s), "block join gradient launch");
  return rc ? rc : ok();
}

}  // extern "C"
