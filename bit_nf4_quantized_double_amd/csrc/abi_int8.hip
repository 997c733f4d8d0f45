// extern "C" entry points of the row-wise operators and the int8 product:
// argument checks on the host, workspace layout and the launch sequence on
// the caller's stream.  Declarations and contracts: include/qlora.h.
#include <climits>
#include <cmath>
#include <exception>

#include "../../include/qlora.h"
#include "abi.h"
#include "common.h"
#include "int8_layout.h"

namespace {

using qlora::aligned16;
using qlora::fail;
using qlora::hip_fail;
using qlora::round_up;

static_assert((int)QLORA_BF16 == qlora::kRowBf16 && (int)QLORA_F16 == qlora::kRowF16 &&
                  (int)QLORA_F32 == qlora::kRowF32,
              "element types");

// No exception leaves a C entry point (building a message can run out of memory).
template <typename F>
int guarded(F f) noexcept {
  try {
    return f();
  } catch (const std::exception&) {
    return QLORA_ERR_HIP;
  } catch (...) {
    return QLORA_ERR_HIP;
  }
}

int done(hipError_t e, const char* where) { return e == hipSuccess ? QLORA_OK : hip_fail(e, where); }

int check_dim(int64_t v, const char* name) {
  if (v < 0) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + " is negative");
  if (v > INT_MAX) return fail(QLORA_ERR_SHAPE, std::string(name) + " exceeds INT_MAX");
  return QLORA_OK;
}

int check_reduction(int64_t v, const char* name) {
  if (v > qlora::kInt8MaxK)
    return fail(QLORA_ERR_SHAPE, std::string(name) + " exceeds 132104, where an int32 sum of products could overflow");
  return QLORA_OK;
}

int check_type(int dtype, bool f32) {
  if (dtype == QLORA_BF16 || dtype == QLORA_F16 || (f32 && dtype == QLORA_F32)) return QLORA_OK;
  return fail(QLORA_ERR_INVALID_ARG, "unsupported element type");
}

// A row-major input whose rows may be apart: present, its stride at least a
// row, its elements aligned to their own size.
int check_rows_in(const void* p, int64_t ld, int64_t m, int64_t k, int dtype, const char* name) {
  if (m == 0 || k == 0) return QLORA_OK;
  if (!p) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (ld < k) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + ": row stride below the row length");
  if (ld > ((int64_t)1 << 40)) return fail(QLORA_ERR_SHAPE, std::string(name) + ": row stride exceeds 2^40 elements");
  const uintptr_t es = dtype == QLORA_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(p) % es) return fail(QLORA_ERR_ALIGN, std::string(name) + " is not aligned to its element size");
  return QLORA_OK;
}

int check_buffer(const void* p, bool needed, const char* name) {
  if (!needed) return QLORA_OK;
  if (!p) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!aligned16(p)) return fail(QLORA_ERR_ALIGN, std::string(name) + " must be 16-byte aligned");
  return QLORA_OK;
}

int check_eps(float eps) {
  // below 1e-12 the reciprocal of a zero row's scale would leave fp32
  if (!(eps >= 1e-12f) || !std::isfinite(eps)) return fail(QLORA_ERR_INVALID_ARG, "eps must be finite and at least 1e-12");
  return QLORA_OK;
}

int check_norm_width(int64_t k) {
  if (k > QLORA_MAX_NORM_WIDTH) return fail(QLORA_ERR_SHAPE, "a normalised row exceeds QLORA_MAX_NORM_WIDTH (32768)");
  return QLORA_OK;
}

// gamma: the row's own 16-bit type, or fp32
int check_gamma(const void* gamma, int gamma_dtype, int dtype, int64_t k) {
  if (gamma_dtype != dtype && gamma_dtype != QLORA_F32)
    return fail(QLORA_ERR_INVALID_ARG, "gamma must have the rows' element type or fp32");
  return check_rows_in(gamma, k, 1, k, gamma_dtype, "gamma");
}

int check_int8_weight(const qlora_int8_weight* w) {
  if (!w) return fail(QLORA_ERR_INVALID_ARG, "weight descriptor is NULL");
  int st;
  if ((st = check_dim(w->n_out, "n_out")) || (st = check_dim(w->k_in, "k_in")) || (st = check_reduction(w->k_in, "k_in")))
    return st;
  const bool some = w->n_out > 0 && w->k_in > 0;
  if ((st = check_buffer(w->codes, some, "weight codes"))) return st;
  if (w->codes_t && (st = check_buffer(w->codes_t, true, "transposed weight codes"))) return st;
  return check_buffer(w->scale, w->n_out > 0, "weight scale");
}

qlora::Int8GemmArgs product_args(const int8_t* wcodes, const float* wscale, int64_t n, int64_t k, const int8_t* xcodes,
                                 const float* xscale, int64_t m, const uint16_t* bias, uint16_t* out, int dtype) {
  qlora::Int8GemmArgs g{};
  g.w = wcodes; g.x = xcodes; g.sw = wscale; g.sx = xscale; g.bias = bias; g.out = out;
  g.m = m; g.n = n; g.k = k;
  g.f16 = dtype == QLORA_F16;
  return g;
}

// The product of quantized rows with a weight's tiles, `n` outputs from a
// reduction over `k`.
int product(const int8_t* wcodes, const float* wscale, int64_t n, int64_t k, const int8_t* xcodes, const float* xscale,
            int64_t m, const uint16_t* bias, uint16_t* out, int dtype, void* part, size_t part_bytes,
            hipStream_t stream) {
  const int cus = qlora::device_compute_units();
  qlora::Int8GemmArgs g = product_args(wcodes, wscale, n, k, xcodes, xscale, m, bias, out, dtype);
  if (part && part_bytes >= qlora::int8_part_bytes(m, n, k, cus)) g.part = static_cast<int32_t*>(part);
  return done(qlora::launch_int8_gemm(g, cus, stream), "int8 product launch");
}

// The arguments of a product whose rows are quantized already.
int check_rows_product(const qlora_int8_weight* w, const int8_t* codes, const float* scale, int64_t M,
                       const uint16_t* bias, const uint16_t* Y, int dtype, const void* ws) {
  int st;
  if ((st = check_int8_weight(w)) || (st = check_dim(M, "M")) || (st = check_type(dtype, false))) return st;
  if (M == 0 || w->n_out == 0) return QLORA_OK;
  if ((st = check_buffer(codes, w->k_in > 0, "codes")) || (st = check_buffer(scale, true, "scale")) ||
      (st = check_buffer(Y, true, "Y")))
    return st;
  if (bias && (st = check_buffer(bias, true, "bias"))) return st;
  if (ws && !aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
  return QLORA_OK;
}

// Workspace of a product that quantizes its rows: [codes][scales][split sums].
struct Int8Ws {
  size_t codes, scale, part, req, total;
};
Int8Ws int8_ws(int64_t m, int64_t n, int64_t k) {
  Int8Ws L{};
  if (qlora::int8_fuses_rows(m, n, k)) return L;
  L.scale = round_up(qlora::int8_rows_bytes(m, k));
  L.part = L.req = L.scale + round_up((size_t)m * 4u);
  L.total = L.part + round_up(qlora::int8_part_bytes(m, n, k, qlora::device_compute_units()));
  return L;
}

int quantized_product(const int8_t* wcodes, const float* wscale, const float* col_scale, int64_t n, int64_t k,
                      const void* X, int64_t ldx, int64_t m, const uint16_t* bias, uint16_t* out, int dtype, void* ws,
                      size_t ws_bytes, hipStream_t stream) {
  qlora::QuantArgs q{};
  q.x = X; q.type = dtype; q.ldx = ldx; q.m = m; q.k = k; q.col_scale = col_scale;
  if (qlora::int8_fuses_rows(m, n, k)) {
    qlora::Int8GemmArgs g{};
    g.w = wcodes; g.sw = wscale; g.bias = bias; g.out = out;
    g.m = m; g.n = n; g.k = k;
    g.f16 = dtype == QLORA_F16;
    return done(qlora::launch_int8_fused(g, q, stream), "int8 product launch");
  }
  const Int8Ws L = int8_ws(m, n, k);
  if (!ws || ws_bytes < L.req) return fail(QLORA_ERR_WORKSPACE, "int8 product workspace too small");
  if (!aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
  char* base = static_cast<char*>(ws);
  q.codes = reinterpret_cast<int8_t*>(base);
  q.scale = reinterpret_cast<float*>(base + L.scale);
  const hipError_t e = qlora::launch_quant_rows(q, qlora::device_compute_units(), stream);
  if (e != hipSuccess) return hip_fail(e, "row quantizer launch");
  return product(wcodes, wscale, n, k, q.codes, q.scale, m, bias, out, dtype, base + L.part, ws_bytes - L.part, stream);
}

}  // namespace

extern "C" {

size_t qlora_int8_weight_bytes(int64_t n_out, int64_t k_in) {
  if (n_out < 0 || k_in < 0 || n_out > INT_MAX || k_in > INT_MAX) return 0;
  return qlora::int8_weight_bytes(n_out, k_in);
}

size_t qlora_int8_rows_bytes(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || M > INT_MAX || K > INT_MAX) return 0;
  return qlora::int8_rows_bytes(M, K);
}

size_t qlora_int8_workspace_bytes(int op, int64_t M, int64_t n_out, int64_t k_in) {
  if (M <= 0 || n_out < 0 || k_in < 0 || M > INT_MAX || n_out > INT_MAX || k_in > INT_MAX) return 0;
  if (op == QLORA_OP_FWD) return int8_ws(M, n_out, k_in).total;
  if (op == QLORA_OP_BWD) return int8_ws(M, k_in, n_out).total;
  return 0;
}

size_t qlora_int8_rows_workspace_bytes(int64_t M, int64_t n_out, int64_t k_in) {
  if (M <= 0 || n_out < 0 || k_in < 0 || M > INT_MAX || n_out > INT_MAX || k_in > INT_MAX) return 0;
  return qlora::int8_part_bytes(M, n_out, k_in, qlora::device_compute_units());
}

size_t qlora_rms_norm_bwd_workspace_bytes(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0 || M > INT_MAX || K > QLORA_MAX_NORM_WIDTH) return 0;
  // rows of partial sums are padded to 16 values
  return (size_t)qlora::norm_bwd_groups(M, K, qlora::device_compute_units()) * (size_t)((K + 15) / 16 * 16) * 4u;
}

int qlora_int8_quantize_weight(const void* W, int dtype, int64_t ldw, int64_t n_out, int64_t k_in, int8_t* codes,
                               float* scale, hipStream_t stream) {
  return guarded([&] {
    const qlora_int8_weight w{n_out, k_in, codes, nullptr, scale};
    int st;
    if ((st = check_int8_weight(&w)) || (st = check_type(dtype, true)) ||
        (st = check_rows_in(W, ldw, n_out, k_in, dtype, "W")))
      return st;
    if (n_out == 0) return (int)QLORA_OK;
    qlora::QuantArgs q{};
    q.x = W; q.type = dtype; q.ldx = ldw; q.m = n_out; q.k = k_in; q.weight = true; q.codes = codes; q.scale = scale;
    return done(qlora::launch_quant_rows(q, qlora::device_compute_units(), stream), "weight quantizer launch");
  });
}

int qlora_int8_pack_weight(const int8_t* W8, int64_t ldw, int64_t n_out, int64_t k_in, int8_t* codes,
                           hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_dim(n_out, "n_out")) || (st = check_dim(k_in, "k_in")) || (st = check_reduction(k_in, "k_in")))
      return st;
    if (n_out == 0 || k_in == 0) return (int)QLORA_OK;
    if (!W8) return fail(QLORA_ERR_INVALID_ARG, "W8 is NULL");
    if (ldw < k_in) return fail(QLORA_ERR_INVALID_ARG, "W8: row stride below the row length");
    if (ldw > ((int64_t)1 << 40)) return fail(QLORA_ERR_SHAPE, "W8: row stride exceeds 2^40 elements");
    if ((st = check_buffer(codes, true, "weight codes"))) return st;
    return done(qlora::launch_int8_pack(W8, ldw, n_out, k_in, codes, stream), "weight pack launch");
  });
}

int qlora_int8_transpose_weight(const qlora_int8_weight* w, int8_t* codes_t, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_int8_weight(w)) || (st = check_reduction(w->n_out, "n_out"))) return st;
    if (w->n_out == 0 || w->k_in == 0) return (int)QLORA_OK;
    if ((st = check_buffer(codes_t, true, "transposed weight codes"))) return st;
    return done(qlora::launch_int8_transpose(w->codes, w->n_out, w->k_in, codes_t, stream), "weight transpose launch");
  });
}

int qlora_int8_dequant_weight(const qlora_int8_weight* w, uint16_t* W16, int dtype, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_int8_weight(w)) || (st = check_type(dtype, false))) return st;
    if (w->n_out == 0 || w->k_in == 0) return (int)QLORA_OK;
    if ((st = check_buffer(W16, true, "output weight"))) return st;
    return done(qlora::launch_int8_dequant(w->codes, w->scale, w->n_out, w->k_in, true, dtype == QLORA_F16, W16, stream),
                "weight dequant launch");
  });
}

int qlora_int8_quantize_rows(const void* X, int dtype, int64_t ldx, int64_t M, int64_t K, const float* col_scale,
                             int8_t* codes, float* scale, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_reduction(K, "K")) ||
        (st = check_type(dtype, true)) || (st = check_rows_in(X, ldx, M, K, dtype, "X")) ||
        (st = check_buffer(codes, M > 0 && K > 0, "codes")) || (st = check_buffer(scale, M > 0, "scale")))
      return st;
    if (reinterpret_cast<uintptr_t>(col_scale) & 3u) return fail(QLORA_ERR_ALIGN, "col_scale is not aligned to its element size");
    if (M == 0) return (int)QLORA_OK;
    qlora::QuantArgs q{};
    q.x = X; q.type = dtype; q.ldx = ldx; q.m = M; q.k = K; q.col_scale = col_scale; q.codes = codes; q.scale = scale;
    return done(qlora::launch_quant_rows(q, qlora::device_compute_units(), stream), "row quantizer launch");
  });
}

int qlora_int8_dequant_rows(const int8_t* codes, const float* scale, int64_t M, int64_t K, uint16_t* X16, int dtype,
                            hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_reduction(K, "K")) ||
        (st = check_type(dtype, false)))
      return st;
    if (M == 0 || K == 0) return (int)QLORA_OK;
    if ((st = check_buffer(codes, true, "codes")) || (st = check_buffer(scale, true, "scale")) ||
        (st = check_buffer(X16, true, "X16")))
      return st;
    return done(qlora::launch_int8_dequant(codes, scale, M, K, false, dtype == QLORA_F16, X16, stream),
                "row dequant launch");
  });
}

int qlora_int8_linear_fwd(const qlora_int8_weight* w, const void* X, int64_t ldx, int64_t M, const uint16_t* bias,
                          uint16_t* Y, int dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_int8_weight(w)) || (st = check_dim(M, "M")) || (st = check_type(dtype, false)) ||
        (st = check_rows_in(X, ldx, M, w->k_in, dtype, "X")))
      return st;
    if (M == 0 || w->n_out == 0) return (int)QLORA_OK;
    if ((st = check_buffer(Y, true, "Y"))) return st;
    if (bias && (st = check_buffer(bias, true, "bias"))) return st;
    return quantized_product(w->codes, w->scale, nullptr, w->n_out, w->k_in, X, ldx, M, bias, Y, dtype, ws, ws_bytes,
                             stream);
  });
}

int qlora_int8_linear_rows(const qlora_int8_weight* w, const int8_t* codes, const float* scale, int64_t M,
                           const uint16_t* bias, uint16_t* Y, int dtype, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_rows_product(w, codes, scale, M, bias, Y, dtype, ws))) return st;
    if (M == 0 || w->n_out == 0) return (int)QLORA_OK;
    return product(w->codes, w->scale, w->n_out, w->k_in, codes, scale, M, bias, Y, dtype, ws, ws_bytes, stream);
  });
}

int qlora_int8_linear_bwd(const qlora_int8_weight* w, const void* dY, int64_t lddy, int64_t M, uint16_t* dX, int dtype,
                          void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_int8_weight(w)) || (st = check_reduction(w->n_out, "n_out")) || (st = check_dim(M, "M")) ||
        (st = check_type(dtype, false)) || (st = check_rows_in(dY, lddy, M, w->n_out, dtype, "dY")))
      return st;
    if (M == 0 || w->k_in == 0) return (int)QLORA_OK;
    if (w->n_out > 0 && !w->codes_t)
      return fail(QLORA_ERR_INVALID_ARG, "the weight has no transposed codes (qlora_int8_transpose_weight)");
    if ((st = check_buffer(dX, true, "dX"))) return st;
    // the channels' scales belong to the reduction here: they go into dY
    return quantized_product(w->codes_t, nullptr, w->scale, w->k_in, w->n_out, dY, lddy, M, nullptr, dX, dtype, ws,
                             ws_bytes, stream);
  });
}

int qlora_int8_plan(int op, int64_t M, int64_t n_out, int64_t k_in, int compute_units, int64_t out[3]) {
  return guarded([&] {
    if (!out) return fail(QLORA_ERR_INVALID_ARG, "out is NULL");
    if (op != QLORA_OP_FWD && op != QLORA_OP_BWD) return fail(QLORA_ERR_INVALID_ARG, "unknown op");
    int st;
    if ((st = check_dim(M, "M")) || (st = check_dim(n_out, "n_out")) || (st = check_dim(k_in, "k_in"))) return st;
    const int64_t n = op == QLORA_OP_FWD ? n_out : k_in, k = op == QLORA_OP_FWD ? k_in : n_out;
    const qlora::Int8Plan p =
        qlora::int8_plan(M, n, k, compute_units > 0 ? compute_units : qlora::device_compute_units());
    out[0] = qlora::int8_tokens(p.kind);
    out[1] = p.ksplit;
    out[2] = qlora::int8_fuses_rows(M, n, k);
    return (int)QLORA_OK;
  });
}

int qlora_debug_int8_linear_rows(const qlora_int8_weight* w, const int8_t* codes, const float* scale, int64_t M,
                                 const uint16_t* bias, uint16_t* Y, int dtype, int tokens, int splits, void* ws,
                                 size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_rows_product(w, codes, scale, M, bias, Y, dtype, ws))) return st;
    qlora::Int8Plan p{};
    for (const qlora::Int8Kind kind : {qlora::kInt8Few16, qlora::kInt8Few32, qlora::kInt8Few64, qlora::kInt8Tile})
      if (qlora::int8_tokens(kind) == tokens) p = qlora::Int8Plan{kind, splits};
    if (p.ksplit == 0 || splits < 1 || splits > 64)
      return fail(QLORA_ERR_INVALID_ARG, "tokens must be 16, 32, 64 or 256, splits 1 to 64");
    if (M == 0 || w->n_out == 0) return (int)QLORA_OK;
    if (splits > 1 && (!ws || ws_bytes < qlora::int8_plan_bytes(p, M, w->n_out)))
      return fail(QLORA_ERR_WORKSPACE, "int8 product workspace too small");
    qlora::Int8GemmArgs g = product_args(w->codes, w->scale, w->n_out, w->k_in, codes, scale, M, bias, Y, dtype);
    if (splits > 1) g.part = static_cast<int32_t*>(ws);
    return done(qlora::launch_int8_plan(g, p, stream), "int8 product launch");
  });
}

int qlora_rms_norm_fwd(const void* X, int64_t ldx, const void* residual, int64_t ldr, const void* gamma,
                       int gamma_dtype, int64_t M, int64_t K, float eps, uint16_t* H, uint16_t* Y, float* rstd,
                       int dtype, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_norm_width(K)) ||
        (st = check_type(dtype, false)) || (st = check_eps(eps)) || (st = check_rows_in(X, ldx, M, K, dtype, "X")) ||
        (st = check_gamma(gamma, gamma_dtype, dtype, K)))
      return st;
    if (residual && (st = check_rows_in(residual, ldr, M, K, dtype, "residual"))) return st;
    if (M == 0 || (K == 0 && !rstd)) return (int)QLORA_OK;
    if ((st = check_buffer(H, residual && K > 0, "H")) || (st = check_buffer(Y, K > 0, "Y")) ||
        (st = check_buffer(rstd, true, "rstd")))
      return st;
    qlora::NormArgs a{};
    a.x = X; a.residual = residual; a.gamma = gamma; a.type = dtype; a.gamma_type = gamma_dtype;
    a.ldx = ldx; a.ldr = ldr; a.m = M; a.k = K; a.eps = eps;
    a.h = residual ? H : nullptr; a.y = Y; a.rstd = rstd;
    return done(qlora::launch_norm(a, qlora::device_compute_units(), stream), "RMS norm launch");
  });
}

int qlora_rms_norm_int8(const void* X, int64_t ldx, const void* residual, int64_t ldr, const void* gamma,
                        int gamma_dtype, int64_t M, int64_t K, float eps, uint16_t* H, int8_t* codes, float* scale,
                        int dtype, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_norm_width(K)) ||
        (st = check_type(dtype, false)) || (st = check_eps(eps)) || (st = check_rows_in(X, ldx, M, K, dtype, "X")) ||
        (st = check_gamma(gamma, gamma_dtype, dtype, K)))
      return st;
    if (residual && (st = check_rows_in(residual, ldr, M, K, dtype, "residual"))) return st;
    if (M == 0 || (K == 0 && !scale)) return (int)QLORA_OK;
    if ((st = check_buffer(H, residual && K > 0, "H")) || (st = check_buffer(codes, K > 0, "codes")) ||
        (st = check_buffer(scale, true, "scale")))
      return st;
    qlora::NormArgs a{};
    a.x = X; a.residual = residual; a.gamma = gamma; a.type = dtype; a.gamma_type = gamma_dtype;
    a.ldx = ldx; a.ldr = ldr; a.m = M; a.k = K; a.eps = eps;
    a.h = residual ? H : nullptr; a.codes = codes; a.scale = scale;
    return done(qlora::launch_norm(a, qlora::device_compute_units(), stream), "RMS norm launch");
  });
}

int qlora_rms_norm_bwd(const void* dY, int64_t lddy, const void* H, int64_t ldh, const float* rstd, const void* gamma,
                       int gamma_dtype, const void* dH, int64_t lddh, int64_t M, int64_t K, uint16_t* dX,
                       float* dgamma, int dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_norm_width(K)) ||
        (st = check_type(dtype, false)) || (st = check_rows_in(dY, lddy, M, K, dtype, "dY")) ||
        (st = check_rows_in(H, ldh, M, K, dtype, "H")) || (st = check_gamma(gamma, gamma_dtype, dtype, K)))
      return st;
    if (dH && (st = check_rows_in(dH, lddh, M, K, dtype, "dH"))) return st;
    if (K == 0) return (int)QLORA_OK;
    if ((st = check_buffer(dgamma, true, "dgamma"))) return st;
    qlora::NormBwdArgs a{};
    a.type = dtype; a.gamma_type = gamma_dtype; a.m = M; a.k = K; a.dgamma = dgamma;
    if (M > 0) {
      if ((st = check_buffer(rstd, true, "rstd")) || (st = check_buffer(dX, true, "dX"))) return st;
      if (!ws || ws_bytes < qlora_rms_norm_bwd_workspace_bytes(M, K))
        return fail(QLORA_ERR_WORKSPACE, "RMS norm backward workspace too small");
      if (!aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    a.dy = dY; a.h = H; a.gamma = gamma; a.dh = dH; a.rstd = rstd;
    a.lddy = lddy; a.ldh = ldh; a.lddh = lddh; a.dx = dX; a.part = static_cast<float*>(ws);
    return done(qlora::launch_norm_bwd(a, qlora::device_compute_units(), stream), "RMS norm backward launch");
  });
}

static int swiglu_args(const void* G, int64_t ldg, const void* U, int64_t ldu, int64_t M, int64_t K, int dtype,
                       bool elementwise, qlora::SwigluArgs* a) {
  int st;
  if ((st = check_dim(M, "M")) || (st = check_dim(K, "K")) || (st = check_type(dtype, false)) ||
      (st = check_rows_in(G, ldg, M, K, dtype, "gate")) || (st = check_rows_in(U, ldu, M, K, dtype, "up")))
    return st;
  // the elementwise kernels count pieces of 16 values in 32 bits
  if (elementwise && M > 0 && (K + 15) / 16 > ((int64_t)UINT32_MAX - 256) / M)
    return fail(QLORA_ERR_SHAPE, "M * K exceeds 2^36 elements");
  a->g = G; a->u = U; a->type = dtype; a->ldg = ldg; a->ldu = ldu; a->m = M; a->k = K;
  return QLORA_OK;
}

int qlora_swiglu_fwd(const void* G, int64_t ldg, const void* U, int64_t ldu, int64_t M, int64_t K, uint16_t* Y,
                     int dtype, hipStream_t stream) {
  return guarded([&] {
    qlora::SwigluArgs a{};
    int st;
    if ((st = swiglu_args(G, ldg, U, ldu, M, K, dtype, true, &a))) return st;
    if (M == 0 || K == 0) return (int)QLORA_OK;
    if ((st = check_buffer(Y, true, "Y"))) return st;
    a.y = Y;
    return done(qlora::launch_swiglu(a, stream), "SwiGLU launch");
  });
}

int qlora_swiglu_int8(const void* G, int64_t ldg, const void* U, int64_t ldu, int64_t M, int64_t K, int8_t* codes,
                      float* scale, int dtype, hipStream_t stream) {
  return guarded([&] {
    qlora::SwigluArgs a{};
    int st;
    if ((st = swiglu_args(G, ldg, U, ldu, M, K, dtype, false, &a)) || (st = check_reduction(K, "K"))) return st;
    if (M == 0) return (int)QLORA_OK;
    if ((st = check_buffer(codes, K > 0, "codes")) || (st = check_buffer(scale, true, "scale"))) return st;
    a.codes = codes; a.scale = scale;
    return done(qlora::launch_swiglu_rows(a, qlora::device_compute_units(), stream), "SwiGLU launch");
  });
}

int qlora_swiglu_bwd(const void* dY, int64_t lddy, const void* G, int64_t ldg, const void* U, int64_t ldu, int64_t M,
                     int64_t K, uint16_t* dG, uint16_t* dU, int dtype, hipStream_t stream) {
  return guarded([&] {
    qlora::SwigluArgs a{};
    int st;
    if ((st = swiglu_args(G, ldg, U, ldu, M, K, dtype, true, &a)) ||
        (st = check_rows_in(dY, lddy, M, K, dtype, "dY")))
      return st;
    if (M == 0 || K == 0) return (int)QLORA_OK;
    if ((st = check_buffer(dG, true, "dG")) || (st = check_buffer(dU, true, "dU"))) return st;
    a.dy = dY; a.lddy = lddy; a.dg = dG; a.du = dU;
    return done(qlora::launch_swiglu_bwd(a, stream), "SwiGLU backward launch");
  });
}

}  // extern "C"
