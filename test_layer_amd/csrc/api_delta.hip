// C ABI of the gated delta rule: argument validation, workspaces and launches.
#include <cmath>

#include "api_util.hpp"
#include "delta.hpp"

using namespace vggt3::api;
namespace delta = vggt3::delta;

namespace {

struct Shape {
  int64_t n;
  int32_t nseq, hk, hv, dk, dv, dtype;
  size_t keys() const { return (size_t)n * hk * dk * elem_size(dtype); }
  size_t values() const { return (size_t)n * hv * dv * elem_size(dtype); }
  size_t scalars() const { return (size_t)n * hv * sizeof(float); }
  size_t state() const { return (size_t)hv * dk * dv * sizeof(float); }
};

int check_shape(const Shape& s) {
  if (!valid_dtype(s.dtype)) return fail(VGGT3_EINVAL, "dtype %d is not VGGT3_BF16 or VGGT3_F32", s.dtype);
  if (s.n < 0) return fail(VGGT3_EINVAL, "n_tokens = %lld < 0", (long long)s.n);
  if (s.nseq < 1) return fail(VGGT3_EINVAL, "n_seqs = %d < 1", s.nseq);
  if (s.hk < 1 || s.hv < 1 || s.hv % s.hk)
    return fail(VGGT3_EINVAL, "n_heads_v = %d is not a multiple of n_heads = %d", s.hv, s.hk);
  if ((s.dk != 64 && s.dk != 128) || (s.dv != 64 && s.dv != 128))
    return fail(VGGT3_EUNSUPPORTED, "heads of %d x %d; 64 or 128 each way", s.dk, s.dv);
  if (s.n > 0x7FFFFFFF) return fail(VGGT3_EUNSUPPORTED, "n_tokens = %lld, at most 2^31 - 1", (long long)s.n);
  if (s.hv > 1024) return fail(VGGT3_EUNSUPPORTED, "n_heads_v = %d, at most 1024", s.hv);
  return VGGT3_OK;
}

// A launch has at most 2^32 threads a side; these grids are pieces * heads of 256.
int check_grid(int64_t groups) {
  if (groups > (int64_t)0x7FFFFF) return fail(VGGT3_EUNSUPPORTED, "%lld sequences or pieces x heads, at most 8388607", (long long)groups);
  return VGGT3_OK;
}

int64_t longest_of(int64_t max_seqlen, int64_t n) { return max_seqlen > 0 && max_seqlen < n ? max_seqlen : n; }

delta::Plan plan_of(const Shape& s, int64_t max_seqlen) {
  return delta::plan(s.n, s.nseq, longest_of(max_seqlen, s.n), s.hv, s.dk, s.dv);
}

// Workspace of the forward: [chunks' matrices | a piece's R | a piece's M | many sequences'
// first pieces and chunks].
struct Ws {
  size_t seg_n, seg_m, cuts, total;
};
Ws forward_ws(const Shape& s, const delta::Plan& p, bool keep) {
  Ws w;
  w.seg_n = round256((size_t)delta::chunk_slots(s.n, s.nseq) * s.hv * delta::matrix_bytes(keep));
  w.seg_m = w.seg_n + (p.split ? round256((size_t)p.pieces * s.state()) : 0);
  w.cuts = w.seg_m + (p.split ? round256((size_t)p.pieces * s.hv * s.dk * s.dk * sizeof(float)) : 0);
  w.total = w.cuts + (delta::needs_cuts(true, s.nseq) ? round256(2 * (size_t)s.nseq * sizeof(uint32_t)) : 0);
  return w;
}

// Workspace of the gradient: [the forward's | states before chunks | gradients after
// chunks | dq and dk by value head, where these share a key head].
struct GradWs {
  Ws f;
  size_t states, dstates, dq, dk, total;
};
GradWs grad_ws(const Shape& s, const delta::Plan& p) {
  const size_t all = round256((size_t)delta::chunk_slots(s.n, s.nseq) * s.state());
  GradWs w;
  w.f = forward_ws(s, p, true);
  w.states = w.f.total;
  w.dstates = w.states + all;
  w.dq = w.dstates + all;
  const size_t part = s.hv == s.hk ? 0 : round256((size_t)s.n * s.hv * s.dk * sizeof(float));
  w.dk = w.dq + part;
  w.total = w.dk + part;
  return w;
}

// The workspace's matrices and pieces, and the cut.
void place(delta::Args& a, char* ws, const Ws& w, const delta::Plan& p, bool keep) {
  a.mats = ws;
  a.keep = keep;
  a.seg_n = reinterpret_cast<float*>(ws + w.seg_n);
  a.seg_m = reinterpret_cast<float*>(ws + w.seg_m);
  a.cuts = delta::needs_cuts(a.cu != nullptr, a.nseq) ? reinterpret_cast<uint32_t*>(ws + w.cuts) : nullptr;
  a.per = p.per;
  a.pieces = p.pieces;
}

int check_scale(float scale) {
  if (!std::isfinite(scale)) return fail(VGGT3_EINVAL, "scale = %g", (double)scale);
  return VGGT3_OK;
}

int check_seqs(const Shape& s, const int32_t* cu, int64_t max_seqlen) {
  if (cu == nullptr && s.nseq != 1) return fail(VGGT3_EINVAL, "n_seqs = %d without cu_seqlens", s.nseq);
  if (max_seqlen < 0) return fail(VGGT3_EINVAL, "max_seqlen = %lld < 0", (long long)max_seqlen);
  return VGGT3_OK;
}

}  // namespace

extern "C" {

size_t vggt3_gated_delta_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int64_t max_seqlen, int32_t n_heads,
                                         int32_t n_heads_v, int32_t d_k, int32_t d_v, int32_t dtype) {
  const Shape s{n_tokens, n_seqs, n_heads, n_heads_v, d_k, d_v, dtype};
  if (check_shape(s) != VGGT3_OK || max_seqlen < 0) return 0;
  return forward_ws(s, plan_of(s, max_seqlen), false).total;
}

int vggt3_gated_delta(const void* q, const void* k, const void* v, const float* g, const float* beta,
                      const int32_t* cu_seqlens, int64_t max_seqlen, const float* state, float scale, void* o,
                      float* state_out, int64_t n_tokens, int32_t n_seqs, int32_t n_heads, int32_t n_heads_v,
                      int32_t d_k, int32_t d_v, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const Shape s{n_tokens, n_seqs, n_heads, n_heads_v, d_k, d_v, dtype};
  int rc = check_shape(s);
  if (!rc) rc = check_seqs(s, cu_seqlens, max_seqlen);
  if (!rc) rc = check_scale(scale);
  if (rc) return rc;
  if (n_tokens > 0) {
    const void* need[] = {q, k, v, beta, o};
    const char* names[] = {"q", "k", "v", "beta", "o"};
    for (int i = 0; i < 5; ++i)
      if (need[i] == nullptr) return fail(VGGT3_EINVAL, "%s is NULL", names[i]);
  }
  const delta::Plan p = plan_of(s, max_seqlen);
  const Ws w = forward_ws(s, p, false);
  rc = check_grid(p.pieces * s.hv);
  if (!rc) rc = check_grid(delta::chunk_slots(n_tokens, n_seqs) * s.hv / 4);
  if (rc) return rc;
  if (workspace == nullptr || workspace_bytes < w.total)
    return fail(VGGT3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, w.total);
  const size_t states = (size_t)n_seqs * s.state();
  const Region rs[] = {{"q", q, s.keys(), false},
                       {"k", k, s.keys(), false},
                       {"v", v, s.values(), false},
                       {"g", g, s.scalars(), false, 4},
                       {"beta", beta, s.scalars(), false, 4},
                       {"cu_seqlens", cu_seqlens, ((size_t)n_seqs + 1) * sizeof(int32_t), false, 4},
                       {"state", state, states, false},
                       {"o", o, s.values(), true},
                       {"state_out", state_out, states, true},
                       {"workspace", workspace, w.total, true}};
  rc = check_regions(rs, 10, {{6, 8}});  // in place: state_out may be state
  if (rc) return rc;
  delta::Args a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu = cu_seqlens; a.state = state;
  a.o = o; a.state_out = state_out;
  a.n = n_tokens; a.nseq = n_seqs; a.hk = n_heads; a.hv = n_heads_v; a.dk = d_k; a.dv = d_v;
  a.scale = scale;
  place(a, static_cast<char*>(workspace), w, p, false);
  rc = check_hip(delta::launch_forward(a, p, dtype == VGGT3_BF16, static_cast<hipStream_t>(stream)),
                 "gated delta rule launch");
  return rc ? rc : ok();
}

size_t vggt3_gated_delta_grad_workspace_bytes(int64_t n_tokens, int32_t n_seqs, int64_t max_seqlen, int32_t n_heads,
                                              int32_t n_heads_v, int32_t d_k, int32_t d_v, int32_t dtype) {
  const Shape s{n_tokens, n_seqs, n_heads, n_heads_v, d_k, d_v, dtype};
  if (check_shape(s) != VGGT3_OK || max_seqlen < 0) return 0;
  return grad_ws(s, plan_of(s, max_seqlen)).total;
}

int vggt3_gated_delta_grad(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           const int32_t* cu_seqlens, int64_t max_seqlen, const float* state, float scale,
                           const void* d_o, const float* dstate_out, void* dq, void* dk, void* dv, float* dg,
                           float* dbeta, float* dstate, int64_t n_tokens, int32_t n_seqs, int32_t n_heads,
                           int32_t n_heads_v, int32_t d_k, int32_t d_v, int32_t dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const Shape s{n_tokens, n_seqs, n_heads, n_heads_v, d_k, d_v, dtype};
  int rc = check_shape(s);
  if (!rc) rc = check_seqs(s, cu_seqlens, max_seqlen);
  if (!rc) rc = check_scale(scale);
  if (rc) return rc;
  if (n_tokens > 0) {
    const void* need[] = {q, k, v, beta, d_o};
    const char* names[] = {"q", "k", "v", "beta", "d_o"};
    for (int i = 0; i < 5; ++i)
      if (need[i] == nullptr) return fail(VGGT3_EINVAL, "%s is NULL", names[i]);
  }
  if (dg && !g) return fail(VGGT3_EINVAL, "dg without g");
  const delta::Plan p = plan_of(s, max_seqlen);
  const GradWs w = grad_ws(s, p);
  rc = check_grid(p.pieces * s.hv);
  if (!rc) rc = check_grid(delta::chunk_slots(n_tokens, n_seqs) * s.hv);
  if (rc) return rc;
  if (workspace == nullptr || workspace_bytes < w.total)
    return fail(VGGT3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, w.total);
  const size_t states = (size_t)n_seqs * s.state();
  const Region rs[] = {{"q", q, s.keys(), false},
                       {"k", k, s.keys(), false},
                       {"v", v, s.values(), false},
                       {"g", g, s.scalars(), false, 4},
                       {"beta", beta, s.scalars(), false, 4},
                       {"cu_seqlens", cu_seqlens, ((size_t)n_seqs + 1) * sizeof(int32_t), false, 4},
                       {"state", state, states, false},
                       {"d_o", d_o, s.values(), false},
                       {"dstate_out", dstate_out, states, false},
                       {"dq", dq, s.keys(), true},
                       {"dk", dk, s.keys(), true},
                       {"dv", dv, s.values(), true},
                       {"dg", dg, s.scalars(), true, 4},
                       {"dbeta", dbeta, s.scalars(), true, 4},
                       {"dstate", dstate, states, true},
                       {"workspace", workspace, w.total, true}};
  rc = check_regions(rs, 16, {{8, 14}});  // in place: dstate may be dstate_out
  if (rc) return rc;
  char* ws = static_cast<char*>(workspace);
  delta::Args a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu = cu_seqlens; a.state = state;
  a.dout = d_o; a.dlast = dstate_out; a.dfirst = dstate;
  a.states = reinterpret_cast<float*>(ws + w.states);
  a.dstates = reinterpret_cast<float*>(ws + w.dstates);
  a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.dg = dg; a.dbeta = dbeta;
  if (s.hv != s.hk) {
    a.dq_part = reinterpret_cast<float*>(ws + w.dq);
    a.dk_part = reinterpret_cast<float*>(ws + w.dk);
  }
  a.n = n_tokens; a.nseq = n_seqs; a.hk = n_heads; a.hv = n_heads_v; a.dk = d_k; a.dv = d_v;
  a.scale = scale;
  place(a, ws, w.f, p, true);
  const bool bf16 = dtype == VGGT3_BF16;
  hipStream_t st = static_cast<hipStream_t>(stream);
  rc = check_hip(delta::launch_states(a, p, bf16, st), "gated delta states launch");
  if (!rc) rc = check_hip(delta::launch_back(a, p, bf16, st), "gated delta reverse launch");
  if (!rc) rc = check_hip(delta::launch_grad(a, bf16, st), "gated delta gradient launch");
  return rc ? rc : ok();
}

int vggt3_gated_delta_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           float* state, int64_t n_slots, const int32_t* slots, float scale, void* o, int64_t n_rows,
                           int32_t n_heads, int32_t n_heads_v, int32_t d_k, int32_t d_v, int32_t dtype, void* stream) {
  const Shape s{n_rows, 1, n_heads, n_heads_v, d_k, d_v, dtype};
  int rc = check_shape(s);
  if (!rc) rc = check_scale(scale);
  if (!rc) rc = check_grid(n_rows * n_heads_v);
  if (rc) return rc;
  if (n_slots < 0) return fail(VGGT3_EINVAL, "n_slots = %lld < 0", (long long)n_slots);
  if (slots == nullptr && n_rows > n_slots)
    return fail(VGGT3_EINVAL, "%lld rows without slots, %lld states", (long long)n_rows, (long long)n_slots);
  if (n_rows == 0) return ok();
  const void* need[] = {q, k, v, beta, o};
  const char* names[] = {"q", "k", "v", "beta", "o"};
  for (int i = 0; i < 5; ++i)
    if (need[i] == nullptr) return fail(VGGT3_EINVAL, "%s is NULL", names[i]);
  if (state == nullptr && n_slots > 0) return fail(VGGT3_EINVAL, "state is NULL");
  const Region rs[] = {{"q", q, s.keys(), false},
                       {"k", k, s.keys(), false},
                       {"v", v, s.values(), false},
                       {"g", g, s.scalars(), false, 4},
                       {"beta", beta, s.scalars(), false, 4},
                       {"slots", slots, (size_t)n_rows * sizeof(int32_t), false, 4},
                       {"state", state, (size_t)n_slots * s.state(), true},
                       {"o", o, s.values(), true}};
  rc = check_regions(rs, 8, {});
  if (rc) return rc;
  delta::StepArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = state; a.slots = slots; a.o = o;
  a.n_slots = n_slots; a.rows = (int)n_rows; a.hk = n_heads; a.hv = n_heads_v; a.dk = d_k; a.dv = d_v;
  a.scale = scale;
  rc = check_hip(delta::launch_step(a, dtype == VGGT3_BF16, static_cast<hipStream_t>(stream)),
                 "gated delta step launch");
  return rc ? rc : ok();
}

}  // extern "C"
