// C ABI of the query/key preparation and its gradient: argument validation and
// launches.
#include <cmath>

#include "api_util.hpp"
#include "qk.hpp"

using namespace vggt3::api;
namespace qk = vggt3::qk;

namespace {

struct Call {
  int64_t n;
  int32_t heads[2], d, dtype, norm;
  float eps;
  const int32_t* pos;
  const int32_t* sections;
  int32_t axes;
  double base;
};

int check_call(const Call& c) {
  if (!valid_dtype(c.dtype)) return fail(VGGT3_EINVAL, "dtype %d is not VGGT3_BF16 or VGGT3_F32", c.dtype);
  if (c.n < 0) return fail(VGGT3_EINVAL, "n_tokens = %lld < 0", (long long)c.n);
  if (c.heads[0] < 1 || c.heads[1] < 0) return fail(VGGT3_EINVAL, "n_heads = %d, n_heads_k = %d", c.heads[0], c.heads[1]);
  if (c.d < 1) return fail(VGGT3_EINVAL, "d_head = %d < 1", c.d);
  if (c.d > qk::kMaxHead) return fail(VGGT3_EUNSUPPORTED, "d_head = %d, at most %d", c.d, qk::kMaxHead);
  if (c.n > (int64_t)1 << 31) return fail(VGGT3_EUNSUPPORTED, "n_tokens = %lld, at most 2^31", (long long)c.n);
  if (c.heads[0] > 4096 || c.heads[1] > 4096) return fail(VGGT3_EUNSUPPORTED, "more than 4096 heads");
  if (c.norm < VGGT3_NORM_NONE || c.norm > VGGT3_NORM_L2) return fail(VGGT3_EINVAL, "norm kind %d", c.norm);
  if (!(c.eps >= 0.0f) || !std::isfinite(c.eps)) return fail(VGGT3_EINVAL, "eps = %g", (double)c.eps);
  if (c.axes < 0) return fail(VGGT3_EINVAL, "n_axes = %d < 0", c.axes);
  if (c.axes > qk::kMaxAxes) return fail(VGGT3_EUNSUPPORTED, "n_axes = %d, at most %d", c.axes, qk::kMaxAxes);
  if (c.axes > 0 && c.sections == nullptr) return fail(VGGT3_EINVAL, "sections is NULL");
  int64_t pairs = 0;
  for (int i = 0; i < c.axes; ++i) {
    if (c.sections[i] < 1) return fail(VGGT3_EINVAL, "axis %d rotates %d pairs", i, c.sections[i]);
    pairs += c.sections[i];
  }
  if (2 * pairs > c.d) return fail(VGGT3_EINVAL, "%lld rotated pairs in heads of %d channels", (long long)pairs, c.d);
  if (c.axes > 0 && (!(c.base > 0.0) || !std::isfinite(c.base))) return fail(VGGT3_EINVAL, "base = %g", c.base);
  if (c.axes > 0 && c.n > 0 && c.pos == nullptr) return fail(VGGT3_EINVAL, "pos is NULL");
  if (c.axes == 0 && c.norm == VGGT3_NORM_NONE) return fail(VGGT3_EINVAL, "neither a norm nor a rotation: nothing to do");
  return VGGT3_OK;
}

int check_side(const Call& c, int i, const char* name, const void* x, int64_t stride, const float* w, const float* b) {
  if (c.heads[i] == 0) return x || w || b ? fail(VGGT3_EINVAL, "%s without key heads", name) : VGGT3_OK;
  if (c.n > 0 && x == nullptr) return fail(VGGT3_EINVAL, "%s is NULL", name);
  if (stride < (int64_t)c.heads[i] * c.d || stride > (int64_t)1 << 31)
    return fail(VGGT3_EINVAL, "rows of %s are %lld apart, %lld long", name, (long long)stride, (long long)c.heads[i] * c.d);
  if ((w || b) && c.norm != VGGT3_NORM_RMS && c.norm != VGGT3_NORM_LAYER)
    return fail(VGGT3_EINVAL, "%s_w / %s_b go with an RMS or layer norm", name, name);
  return VGGT3_OK;
}

qk::Args args_of(const Call& c, int32_t per_axis, int32_t interleaved) {
  qk::Args a{};
  a.pos = c.pos;
  a.n = c.n;
  a.d = c.d;
  a.norm = c.norm;
  a.axes = c.axes;
  for (int i = 0; i < c.axes; ++i) {
    a.pairs[i] = c.sections[i];
    a.rotated += c.sections[i];
  }
  a.per_axis = per_axis != 0;
  a.interleaved = interleaved != 0;
  for (int i = 0; i < c.axes; ++i) {
    const int size = a.per_axis ? c.sections[i] : a.rotated;
    if (i > 0 && size == (a.per_axis ? c.sections[i - 1] : a.rotated)) {
      a.step[i][0] = a.step[i - 1][0];
      a.step[i][1] = a.step[i - 1][1];
      continue;
    }
    const long double step = std::pow((long double)c.base, -1.0L / size);  // 64 bits: the two doubles hold them
    a.step[i][0] = (double)step;
    a.step[i][1] = (double)(step - a.step[i][0]);
  }
  a.eps = c.eps;
  return a;
}

size_t span(const Call& c, int i, int64_t stride) {
  return c.n == 0 || c.heads[i] == 0 ? 0 : ((size_t)(c.n - 1) * stride + (size_t)c.heads[i] * c.d) * elem_size(c.dtype);
}

}  // namespace

extern "C" {

int vggt3_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int32_t norm,
                       const float* q_w, const float* q_b, const float* k_w, const float* k_b, float eps,
                       const int32_t* pos, const int32_t* sections, int32_t n_axes, double base, int32_t per_axis,
                       int32_t interleaved, void* q_out, void* k_out, int64_t n_tokens, int32_t n_heads,
                       int32_t n_heads_k, int32_t d_head, int32_t dtype, void* stream) {
  const Call c{n_tokens, {n_heads, n_heads_k}, d_head, dtype, norm, eps, pos, sections, n_axes, base};
  int rc = check_call(c);
  if (!rc) rc = check_side(c, 0, "q", q, q_stride, q_w, q_b);
  if (!rc) rc = check_side(c, 1, "k", k, k_stride, k_w, k_b);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  if (q_out == nullptr || (n_heads_k > 0 && k_out == nullptr)) return fail(VGGT3_EINVAL, "%s is NULL", q_out ? "k_out" : "q_out");
  if (n_heads_k == 0 && k_out) return fail(VGGT3_EINVAL, "k_out without key heads");
  const size_t e = elem_size(dtype), vb = (size_t)d_head * sizeof(float);
  const int64_t rows[2] = {(int64_t)n_heads * d_head, (int64_t)n_heads_k * d_head};
  const Region rs[] = {{"q", q, span(c, 0, q_stride), false, e},
                       {"k", k, span(c, 1, k_stride), false, e},
                       {"q_w", q_w, vb, false, 4},
                       {"q_b", q_b, vb, false, 4},
                       {"k_w", k_w, vb, false, 4},
                       {"k_b", k_b, vb, false, 4},
                       {"pos", n_axes ? pos : nullptr, (size_t)n_tokens * n_axes * 4, false, 4},
                       {"q_out", q_out, span(c, 0, rows[0]), true, e},
                       {"k_out", k_out, span(c, 1, rows[1]), true, e}};
  // in place where rows are not apart
  if ((q_out == q && q_stride != rows[0]) || (k_out && k_out == k && k_stride != rows[1]))
    return fail(VGGT3_EINVAL, "in place takes rows without gaps");
  rc = check_regions(rs, 9, {{0, 7}, {1, 8}});
  if (rc) return rc;
  qk::Args a = args_of(c, per_axis, interleaved);
  a.s[0] = qk::Side{q, nullptr, q_out, q_w, q_b, q_stride, n_heads};
  a.s[1] = qk::Side{k, nullptr, k_out, k_w, k_b, k_stride, n_heads_k};
  rc = check_hip(qk::launch_forward(a, dtype == VGGT3_BF16, static_cast<hipStream_t>(stream)), "query/key launch");
  return rc ? rc : ok();
}

size_t vggt3_qk_norm_rope_grad_workspace_bytes(int64_t n_tokens, int32_t d_head) {
  if (n_tokens < 1 || d_head < 1 || d_head > qk::kMaxHead) return 0;
  return round256((size_t)qk::grad_blocks(n_tokens) * 4 * d_head * sizeof(float));
}

int vggt3_qk_norm_rope_grad(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* dq_out,
                            const void* dk_out, int32_t norm, const float* q_w, const float* k_w, float eps,
                            const int32_t* pos, const int32_t* sections, int32_t n_axes, double base,
                            int32_t per_axis, int32_t interleaved, void* dq, void* dk, float* dq_w, float* dq_b,
                            float* dk_w, float* dk_b, int64_t n_tokens, int32_t n_heads, int32_t n_heads_k,
                            int32_t d_head, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const Call c{n_tokens, {n_heads, n_heads_k}, d_head, dtype, norm, eps, pos, sections, n_axes, base};
  int rc = check_call(c);
  if (!rc) rc = check_side(c, 0, "q", q, q_stride, q_w, nullptr);
  if (!rc) rc = check_side(c, 1, "k", k, k_stride, k_w, nullptr);
  if (rc) return rc;
  const bool vecs = dq_w || dq_b || dk_w || dk_b;
  if (vecs && norm != VGGT3_NORM_RMS && norm != VGGT3_NORM_LAYER)
    return fail(VGGT3_EINVAL, "gradients of weights and biases go with an RMS or layer norm");
  if (n_heads_k == 0 && (dk_out || dk || dk_w || dk_b)) return fail(VGGT3_EINVAL, "gradients of k without key heads");
  if (n_tokens > 0 && (dq_out == nullptr || (n_heads_k > 0 && dk_out == nullptr)))
    return fail(VGGT3_EINVAL, "%s is NULL", dq_out ? "dk_out" : "dq_out");
  const size_t need = vecs ? vggt3_qk_norm_rope_grad_workspace_bytes(n_tokens, d_head) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(VGGT3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, need);
  const size_t e = elem_size(dtype), vb = (size_t)d_head * sizeof(float);
  const int64_t rows[2] = {(int64_t)n_heads * d_head, (int64_t)n_heads_k * d_head};
  const size_t qb = span(c, 0, rows[0]), kb = span(c, 1, rows[1]);
  const Region rs[] = {{"q", q, span(c, 0, q_stride), false, e},
                       {"k", k, span(c, 1, k_stride), false, e},
                       {"dq_out", dq_out, qb, false, e},
                       {"dk_out", dk_out, kb, false, e},
                       {"q_w", q_w, vb, false, 4},
                       {"k_w", k_w, vb, false, 4},
                       {"pos", n_axes ? pos : nullptr, (size_t)n_tokens * n_axes * 4, false, 4},
                       {"dq", dq, qb, true, e},
                       {"dk", dk, kb, true, e},
                       {"dq_w", dq_w, vb, true, 4},
                       {"dq_b", dq_b, vb, true, 4},
                       {"dk_w", dk_w, vb, true, 4},
                       {"dk_b", dk_b, vb, true, 4},
                       {"workspace", need ? workspace : nullptr, need, true}};
  rc = check_regions(rs, 14, {{2, 7}, {3, 8}});  // in place: dq may be dq_out
  if (rc) return rc;
  qk::Args a = args_of(c, per_axis, interleaved);
  a.s[0] = qk::Side{q, dq_out, dq, q_w, nullptr, q_stride, n_heads};
  a.s[1] = qk::Side{k, dk_out, dk, k_w, nullptr, k_stride, n_heads_k};
  a.part = need ? static_cast<float*>(workspace) : nullptr;
  float* out[4] = {dq_w, dq_b, dk_w, dk_b};
  rc = check_hip(qk::launch_grad(a, out, dtype == VGGT3_BF16, static_cast<hipStream_t>(stream)), "query/key gradient launch");
  return rc ? rc : ok();
}

}  // extern "C"
