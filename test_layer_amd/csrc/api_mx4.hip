// C ABI of the microscaled 4-bit operators: argument validation and launch
// sequencing. Every check runs on the host before anything is enqueued.
#include <initializer_list>

#include "api_util.hpp"
#include "mx4.hpp"
#include "wide.hpp"

using namespace vggt3::api;
namespace mx4 = vggt3::mx4;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 20;   // columns of a 4-bit matrix
// Scale tiles of a matrix: the quantiser's workgroups of 256 threads, of which a
// launch may have fewer than 2^32 in all.
constexpr int64_t kMaxTiles = (int64_t)1 << 24;
constexpr int64_t kMaxProductTiles = (int64_t)1 << 31;  // 16 x 16, of C

struct Region {
  const char* name;
  const void* p;
  size_t bytes;
  bool written;
};

// Non-null, 16-byte aligned, and no written region overlapping another one.
int check_regions(std::initializer_list<Region> rs) {
  for (const Region& r : rs) {
    if (r.p == nullptr && r.bytes > 0) return fail(VGGT3_EINVAL, "%s is NULL", r.name);
    if (!aligned16(r.p)) return fail(VGGT3_EINVAL, "%s is not 16-byte aligned", r.name);
  }
  for (const Region* a = rs.begin(); a != rs.end(); ++a)
    for (const Region* b = a + 1; b != rs.end(); ++b)
      if ((a->written || b->written) && overlap(a->p, a->bytes, b->p, b->bytes))
        return fail(VGGT3_EINVAL, "%s and %s overlap", a->name, b->name);
  return VGGT3_OK;
}

int check_matrix(const char* what, int64_t rows, int64_t k) {
  if (rows < 0) return fail(VGGT3_EINVAL, "%s has %lld rows", what, (long long)rows);
  if (k < 1) return fail(VGGT3_EINVAL, "%s has %lld columns", what, (long long)k);
  if (k > kMaxCols) return fail(VGGT3_EUNSUPPORTED, "%s has %lld columns, at most %lld", what, (long long)k,
                                (long long)kMaxCols);
  if (rows > (int64_t)1 << 40 || mx4::row_tiles(rows) * (mx4::padded_k(k) / mx4::kPad) >= kMaxTiles)
    return fail(VGGT3_EUNSUPPORTED, "%s is too large (%lld x %lld)", what, (long long)rows, (long long)k);
  return VGGT3_OK;
}

size_t cbytes(int64_t rows, int64_t k) { return (size_t)mx4::code_bytes(rows, k); }
size_t sbytes(int64_t rows, int64_t k) { return (size_t)mx4::scale_bytes(rows, k); }

bool valid_type(int32_t t) { return valid_dtype(t) || t == VGGT3_MX4; }

size_t tokens_bytes(int64_t rows, int64_t k, int32_t type) {
  return type == VGGT3_MX4 ? cbytes(rows, k) : (size_t)rows * k * elem_size(type);
}

// Workspace of a product: [codes | scales] of A, when it comes as more tokens
// than the product quantises itself.
struct MatmulWs {
  size_t scales, total;
};
MatmulWs matmul_ws(int64_t m, int64_t k, int32_t a_type) {
  MatmulWs l{};
  if (a_type != VGGT3_MX4 && !mx4::takes_tokens(m, (int)k)) {
    l.scales = round256(cbytes(m, k));
    l.total = l.scales + round256(sbytes(m, k));
  }
  return l;
}

int check_matmul_shape(int64_t m, int64_t n, int64_t k, int32_t a_type) {
  if (!valid_type(a_type)) return fail(VGGT3_EINVAL, "A type %d is not VGGT3_BF16, VGGT3_F32 or VGGT3_MX4", a_type);
  int rc = check_matrix("A", m, k);
  if (rc) return rc;
  if (n < 1) return fail(VGGT3_EINVAL, "n = %lld < 1", (long long)n);
  if (n > kMaxCols) return fail(VGGT3_EUNSUPPORTED, "n = %lld, at most %lld", (long long)n, (long long)kMaxCols);
  if (((m + 15) / 16) * ((n + 15) / 16) >= kMaxProductTiles) return fail(VGGT3_EUNSUPPORTED, "m x n is too large");
  return VGGT3_OK;
}

// Workspace of the 4-bit read of the full-width MLP, for chunks of at most
// wide::kChunk tokens: H in 4 bits, then Q (when it comes as more tokens than
// the product quantises itself).
struct ReadWs {
  int64_t ct;
  size_t hs, qc, qs, total;
};
ReadWs read_ws(int64_t n, int32_t q_type) {
  namespace w = vggt3::wide;
  ReadWs l{};
  l.ct = n < w::kChunk ? n : w::kChunk;
  l.hs = round256(cbytes(l.ct, w::kM));
  l.qc = l.total = l.hs + round256(sbytes(l.ct, w::kM));
  if (q_type != VGGT3_MX4 && !mx4::takes_tokens(l.ct, w::kD)) {
    l.qs = l.qc + round256(cbytes(l.ct, w::kD));
    l.total = l.qs + round256(sbytes(l.ct, w::kD));
  }
  return l;
}

int check_read_shape(int64_t n, int32_t H, int32_t d, int32_t m, int32_t q_type) {
  namespace w = vggt3::wide;
  if (n < 0) return fail(VGGT3_EINVAL, "n_tokens = %lld < 0", (long long)n);
  if (H < 1 || d < 1 || m < 1)
    return fail(VGGT3_EINVAL, "n_heads/d_head/d_hidden must be >= 1 (got %d/%d/%d)", H, d, m);
  if (H != 1 || d != w::kD || m != w::kM)
    return fail(VGGT3_EUNSUPPORTED, "4-bit fast weights are those of the %d -> %d -> %d MLP (got %d heads of %d, %d)",
                w::kD, w::kM, w::kD, H, d, m);
  if (q_type != VGGT3_BF16 && q_type != VGGT3_MX4)
    return fail(VGGT3_EUNSUPPORTED, "Q type %d is not VGGT3_BF16 or VGGT3_MX4", q_type);
  return check_matrix("Q", n, d);
}

}  // namespace

extern "C" {

size_t vggt3_mx4_codes_bytes(int64_t rows, int32_t k) {
  return check_matrix("matrix", rows, k) == VGGT3_OK ? cbytes(rows, k) : 0;
}

size_t vggt3_mx4_scales_bytes(int64_t rows, int32_t k) {
  return check_matrix("matrix", rows, k) == VGGT3_OK ? sbytes(rows, k) : 0;
}

int vggt3_mx4_quantize(const void* X, int32_t transposed, void* codes, void* scales, int64_t rows, int32_t k,
                       int32_t dtype, void* stream) {
  if (!valid_dtype(dtype)) return fail(VGGT3_EINVAL, "dtype %d is not VGGT3_BF16 or VGGT3_F32", dtype);
  int rc = check_matrix("X", rows, k);
  if (rc) return rc;
  if (rows == 0) return ok();
  rc = check_regions({{"X", X, tokens_bytes(rows, k, dtype), false},
                      {"codes", codes, cbytes(rows, k), true},
                      {"scales", scales, sbytes(rows, k), true}});
  if (rc) return rc;
  rc = check_hip(mx4::launch_quantize(X, transposed != 0, dtype == VGGT3_BF16, static_cast<uint8_t*>(codes),
                                      static_cast<uint8_t*>(scales), rows, k, static_cast<hipStream_t>(stream)),
                 "quantize launch");
  return rc ? rc : ok();
}

int vggt3_mx4_dequantize(const void* codes, const void* scales, void* X, int64_t rows, int32_t k, int32_t dtype,
                         void* stream) {
  if (!valid_dtype(dtype)) return fail(VGGT3_EINVAL, "dtype %d is not VGGT3_BF16 or VGGT3_F32", dtype);
  int rc = check_matrix("X", rows, k);
  if (rc) return rc;
  if (rows == 0) return ok();
  rc = check_regions({{"X", X, tokens_bytes(rows, k, dtype), true},
                      {"codes", codes, cbytes(rows, k), false},
                      {"scales", scales, sbytes(rows, k), false}});
  if (rc) return rc;
  rc = check_hip(mx4::launch_dequantize(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), X,
                                        dtype == VGGT3_BF16, rows, k, static_cast<hipStream_t>(stream)),
                 "dequantize launch");
  return rc ? rc : ok();
}

size_t vggt3_mx4_matmul_workspace_bytes(int64_t m, int32_t n, int32_t k, int32_t a_type) {
  return check_matmul_shape(m, n, k, a_type) == VGGT3_OK && m > 0 ? matmul_ws(m, k, a_type).total : 0;
}

int vggt3_mx4_matmul(const void* A, const void* A_scales, int32_t a_type, const void* W_codes, const void* W_scales,
                     void* C, int64_t m, int32_t n, int32_t k, int32_t dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype)) return fail(VGGT3_EINVAL, "dtype %d is not VGGT3_BF16 or VGGT3_F32", dtype);
  int rc = check_matmul_shape(m, n, k, a_type);
  if (rc) return rc;
  if (m == 0) return ok();
  const MatmulWs l = matmul_ws(m, k, a_type);
  const bool quantized = a_type == VGGT3_MX4;
  if (!quantized && A_scales != nullptr) return fail(VGGT3_EINVAL, "A_scales goes with a VGGT3_MX4 A only");
  if (l.total > 0 && (workspace == nullptr || workspace_bytes < l.total))
    return fail(VGGT3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0,
                l.total);
  rc = check_regions({{"A", A, tokens_bytes(m, k, a_type), false},
                      {"A_scales", A_scales, quantized ? sbytes(m, k) : 0, false},
                      {"W_codes", W_codes, cbytes(n, k), false},
                      {"W_scales", W_scales, sbytes(n, k), false},
                      {"C", C, (size_t)m * n * elem_size(dtype), true},
                      {"workspace", workspace, l.total, true}});
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const mx4::Matrix w{static_cast<const uint8_t*>(W_codes), static_cast<const uint8_t*>(W_scales)};
  const bool bf16 = dtype == VGGT3_BF16;
  if (!quantized && l.total == 0) {
    rc = check_hip(mx4::launch_gemm_tokens(A, a_type == VGGT3_BF16, w, C, bf16, m, n, k, s), "4-bit product launch");
    return rc ? rc : ok();
  }
  mx4::Matrix a{static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(A_scales)};
  if (!quantized) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a = mx4::Matrix{ws, ws + l.scales};
    rc = check_hip(mx4::launch_quantize(A, false, a_type == VGGT3_BF16, ws, ws + l.scales, m, k, s), "quantize launch");
    if (rc) return rc;
  }
  rc = check_hip(mx4::launch_gemm(a, w, C, bf16, m, n, k, s),
                 "4-bit product launch");
  return rc ? rc : ok();
}

int vggt3_ttt_freeze_mx4(const float* theta, void* gate_codes, void* gate_scales, void* up_codes, void* up_scales,
                         void* down_codes, void* down_scales, int32_t n_heads, int32_t d_head, int32_t d_hidden,
                         void* stream) {
  int rc = check_read_shape(0, n_heads, d_head, d_hidden, VGGT3_MX4);
  if (rc) return rc;
  const int64_t d = d_head, m = d_hidden;
  rc = check_regions({{"theta", theta, (size_t)(3 * d * m) * sizeof(float), false},
                      {"gate_codes", gate_codes, cbytes(m, d), true},
                      {"gate_scales", gate_scales, sbytes(m, d), true},
                      {"up_codes", up_codes, cbytes(m, d), true},
                      {"up_scales", up_scales, sbytes(m, d), true},
                      {"down_codes", down_codes, cbytes(d, m), true},
                      {"down_scales", down_scales, sbytes(d, m), true}});
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto u8 = [](void* p) { return static_cast<uint8_t*>(p); };
  // W_g, W_u [d][m] and W_d [m][d] are all stored with the contraction first.
  rc = check_hip(mx4::launch_quantize(theta, true, false, u8(gate_codes), u8(gate_scales), m, d_head, s), "gate");
  if (rc) return rc;
  rc = check_hip(mx4::launch_quantize(theta + d * m, true, false, u8(up_codes), u8(up_scales), m, d_head, s), "up");
  if (rc) return rc;
  rc = check_hip(mx4::launch_quantize(theta + 2 * d * m, true, false, u8(down_codes), u8(down_scales), d, d_hidden, s),
                 "down");
  return rc ? rc : ok();
}

size_t vggt3_ttt_read_mx4_workspace_bytes(int64_t n_tokens, int32_t n_heads, int32_t d_head, int32_t d_hidden,
                                          int32_t q_type) {
  if (check_read_shape(n_tokens, n_heads, d_head, d_hidden, q_type) != VGGT3_OK || n_tokens == 0) return 0;
  return read_ws(n_tokens, q_type).total;
}

int vggt3_ttt_read_mx4(const void* Q, const void* Q_scales, int32_t q_type, const void* gate_codes,
                       const void* gate_scales, const void* up_codes, const void* up_scales, const void* down_codes,
                       const void* down_scales, void* O, int64_t n_tokens, int32_t n_heads, int32_t d_head,
                       int32_t d_hidden, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_read_shape(n_tokens, n_heads, d_head, d_hidden, q_type);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  const int64_t d = d_head, m = d_hidden;
  const ReadWs l = read_ws(n_tokens, q_type);
  const bool quantized = q_type == VGGT3_MX4;
  if (!quantized && Q_scales != nullptr) return fail(VGGT3_EINVAL, "Q_scales goes with a VGGT3_MX4 Q only");
  if (workspace == nullptr || workspace_bytes < l.total)
    return fail(VGGT3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0,
                l.total);
  rc = check_regions({{"Q", Q, tokens_bytes(n_tokens, d, q_type), false},
                      {"Q_scales", Q_scales, quantized ? sbytes(n_tokens, d) : 0, false},
                      {"gate_codes", gate_codes, cbytes(m, d), false},
                      {"gate_scales", gate_scales, sbytes(m, d), false},
                      {"up_codes", up_codes, cbytes(m, d), false},
                      {"up_scales", up_scales, sbytes(m, d), false},
                      {"down_codes", down_codes, cbytes(d, m), false},
                      {"down_scales", down_scales, sbytes(d, m), false},
                      {"O", O, (size_t)n_tokens * d * 2, true},
                      {"workspace", workspace, l.total, true}});
  if (rc) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto mat = [](const void* c, const void* sc) {
    return mx4::Matrix{static_cast<const uint8_t*>(c), static_cast<const uint8_t*>(sc)};
  };
  const mx4::Matrix wg = mat(gate_codes, gate_scales), wu = mat(up_codes, up_scales),
                    wd = mat(down_codes, down_scales);
  const mx4::Matrix h = mat(ws, ws + l.hs);
  for (int64_t t0 = 0; t0 < n_tokens; t0 += l.ct) {
    const int64_t nc = n_tokens - t0 < l.ct ? n_tokens - t0 : l.ct;
    const uint16_t* tokens = static_cast<const uint16_t*>(Q) + t0 * d;
    if (!quantized && mx4::takes_tokens(nc, d_head)) {
      rc = check_hip(mx4::launch_gemm_swiglu_tokens(tokens, wg, wu, ws, ws + l.hs, nc, d_hidden, d_head, s),
                     "4-bit SwiGLU launch");
    } else {
      mx4::Matrix q;
      if (quantized) {
        // chunks are whole scale tiles, so a chunk's tiles follow those before it
        q = mat(static_cast<const uint8_t*>(Q) + cbytes(t0, d), static_cast<const uint8_t*>(Q_scales) + sbytes(t0, d));
      } else {
        rc = check_hip(mx4::launch_quantize(tokens, false, true, ws + l.qc, ws + l.qs, nc, d_head, s),
                       "quantize launch");
        if (rc) return rc;
        q = mat(ws + l.qc, ws + l.qs);
      }
      rc = check_hip(mx4::launch_gemm_swiglu(q, wg, wu, ws, ws + l.hs, nc, d_hidden, d_head, s),
                     "4-bit SwiGLU launch");
    }
    if (rc) return rc;
    rc = check_hip(mx4::launch_gemm(h, wd, static_cast<uint16_t*>(O) + t0 * d, true, nc, d_head, d_hidden, s),
                   "4-bit product launch");
    if (rc) return rc;
  }
  return ok();
}

}  // extern "C"
