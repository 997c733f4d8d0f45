// extern "C" entry points of rotary positions, attention and the head's loss:
// argument checks on the host, workspace layout and the launch sequence on
// the caller's stream.  Declarations and contracts: include/qlora.h.
#include <climits>
#include <cmath>
#include <exception>
#include <initializer_list>

#include "../../include/qlora.h"
#include "abi.h"
#include "common.h"
#include "decoder.h"

namespace {

using qlora::aligned16;
using qlora::fail;
using qlora::hip_fail;
using qlora::round_up;

// No exception leaves a C entry point (building a message can run out of memory).
template <typename F>
int guarded(F f) noexcept {
  try {
    return f();
  } catch (...) {
    return QLORA_ERR_HIP;
  }
}

int done(hipError_t e, const char* where) { return e == hipSuccess ? QLORA_OK : hip_fail(e, where); }

int check_range(int64_t v, int64_t most, const char* name) {
  if (v < 0) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + " is negative");
  if (v > most) return fail(QLORA_ERR_SHAPE, std::string(name) + " exceeds " + std::to_string(most));
  return QLORA_OK;
}

int check_type16(int dtype) {
  if (dtype == QLORA_BF16 || dtype == QLORA_F16) return QLORA_OK;
  return fail(QLORA_ERR_INVALID_ARG, "unsupported element type");
}

constexpr int64_t kMostStride = (int64_t)1 << 40, kMostTokenStride = 1 << 23;

// [tokens, heads, d]: there, aligned to `align` bytes, its strides multiples of
// that, and for an output without two elements in one place.
int check_heads(const qlora_heads* x, int64_t tokens, int64_t heads, int64_t d, int align, bool out, const char* name) {
  if (tokens == 0 || heads == 0 || d == 0) return QLORA_OK;
  if (!x || !x->p) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  const int64_t t = tokens > 1 ? x->token_stride : 0, h = heads > 1 ? x->head_stride : 0;
  if (t < 0 || h < 0) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + ": negative stride");
  if (t > kMostStride || h > kMostStride) return fail(QLORA_ERR_SHAPE, std::string(name) + ": a stride exceeds 2^40 elements");
  if (reinterpret_cast<uintptr_t>(x->p) % align || t * 2 % align || h * 2 % align)
    return fail(QLORA_ERR_ALIGN, std::string(name) + " and its strides must be multiples of " + std::to_string(align) + " bytes");
  if (out) {
    const bool by_token = (heads == 1 || h >= d) && (tokens == 1 || t >= (heads - 1) * h + d);
    const bool by_head = (tokens == 1 || t >= d) && (heads == 1 || h >= (tokens - 1) * t + d);
    if (!by_token && !by_head) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + ": an output's elements overlap");
  }
  return QLORA_OK;
}

// the same for attention: 16 bytes at a time, tokens near enough for 32-bit offsets inside a tile
int check_attn_heads(const qlora_heads* x, int64_t tokens, int64_t heads, int64_t d, bool out, const char* name) {
  const int st = check_heads(x, tokens, heads, d, 16, out, name);
  if (st == QLORA_OK && x && tokens > 1 && heads > 0 && x->token_stride > kMostTokenStride)
    return fail(QLORA_ERR_SHAPE, std::string(name) + ": the token stride exceeds 2^23 elements");
  return st;
}

qlora::Heads heads_arg(const qlora_heads* x, int64_t tokens, int64_t heads, int64_t d) {
  if (tokens == 0 || heads == 0 || d == 0) return qlora::Heads{nullptr, 0, 0, 0};
  return qlora::heads_of(x->p, tokens > 1 ? x->token_stride : 0, heads > 1 ? x->head_stride : 0, tokens, heads, d);
}

int check_attention(const qlora_attention* a, bool backward) {
  if (!a) return fail(QLORA_ERR_INVALID_ARG, "attention descriptor is NULL");
  const int64_t most = INT_MAX - 255;
  int st;
  if ((st = check_range(a->tokens_q, most, "tokens_q")) || (st = check_range(a->tokens_k, (1 << 30) - 1, "tokens_k")) ||
      (st = check_range(a->batch, 1 << 24, "batch")) || (st = check_range(a->heads, 65536, "heads")) ||
      (st = check_range(a->kv_heads, 65536, "kv_heads")) ||
      (st = check_range(a->head_dim, QLORA_MAX_HEAD_DIM, "head_dim")) || (st = check_type16(a->dtype)))
    return st;
  if (a->head_dim % 8 || a->head_dim == 0) return fail(QLORA_ERR_SHAPE, "head_dim must be a positive multiple of 8");
  if (a->kv_heads == 0 ? a->heads != 0 : a->heads % a->kv_heads != 0)
    return fail(QLORA_ERR_SHAPE, "heads must be a multiple of kv_heads");
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return fail(QLORA_ERR_INVALID_ARG, "scale must be positive and finite");
  if (!a->cu_q || !a->cu_k) return fail(QLORA_ERR_INVALID_ARG, "cu_q or cu_k is NULL");
  for (const int32_t* p : {a->cu_q, a->cu_k, a->len_q, a->len_k})
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(QLORA_ERR_ALIGN, "cu_q, cu_k, len_q and len_k must be 4-byte aligned");
  if (a->heads) {
    const int64_t group = a->heads / a->kv_heads;
    if (a->tokens_q > most / group) return fail(QLORA_ERR_SHAPE, "tokens_q * heads / kv_heads exceeds 2^31 - 256");
    // workgroups of a launch: fewer than 2^24 (the forward's are of rows of queries only;
    // the backward's of dK and dV and of their join; delta's, at most batch heads / 4 +
    // 2^20, are then fewer too)
    if (((a->tokens_q * group + 31) / 32 + a->batch + 2) * a->kv_heads >= (1 << 24))
      return fail(QLORA_ERR_SHAPE, "too many rows for one launch");
    if (backward && (((a->tokens_k + 127) / 128 + a->batch + 2) * a->heads >= (1 << 24) ||
                     a->tokens_k / 4 + a->batch >= (1 << 24) - 2))
      return fail(QLORA_ERR_SHAPE, "too many keys or sequences for one launch of the backward");
  }
  return QLORA_OK;
}

// Kernels read inputs after they have written outputs of other rows.
int check_apart(std::initializer_list<const qlora_heads*> out, std::initializer_list<const qlora_heads*> in) {
  for (auto o = out.begin(); o != out.end(); ++o) {
    if (!*o || !(*o)->p) continue;
    for (auto x = out.begin(); x != o; ++x)
      if (*x && (*x)->p == (*o)->p) return fail(QLORA_ERR_INVALID_ARG, "two outputs are the same tensor");
    for (const qlora_heads* x : in)
      if (x && x->p == (*o)->p) return fail(QLORA_ERR_INVALID_ARG, "an output is an input");
  }
  return QLORA_OK;
}

qlora::AttnArgs attention_args(const qlora_attention* a) {
  qlora::AttnArgs g{};
  g.cu_q = a->cu_q; g.cu_k = a->cu_k; g.len_q = a->len_q; g.len_k = a->len_k;
  g.tq = a->tokens_q; g.tk = a->tokens_k; g.batch = (int32_t)a->batch;
  g.heads = (int32_t)a->heads; g.kv_heads = (int32_t)a->kv_heads; g.group = (int32_t)(a->heads / a->kv_heads);
  g.d = (int32_t)a->head_dim; g.splits = 1;
  g.scale = a->scale; g.causal = a->causal != 0; g.zero_rest = a->zero_rest != 0; g.f16 = a->dtype == QLORA_F16;
  return g;
}

bool nothing(const qlora_attention* a) { return a->heads == 0 || a->tokens_q + a->tokens_k == 0; }

qlora::AttnPlan plan_of(const qlora_attention* a, int cus) {
  return qlora::attn_plan(a->tokens_q, a->tokens_k, a->batch, a->heads, a->kv_heads, cus);
}

// Workspace of a backward: [delta][lse in base 2][maxima][split sums].
struct BwdWs {
  size_t lse2, top, part, total;
  int splits;
};
BwdWs bwd_ws(const qlora_attention* a) {
  BwdWs L{};
  L.splits = qlora::attn_bwd_splits(a->tokens_k, a->batch, a->heads, a->kv_heads, qlora::device_compute_units());
  L.lse2 = round_up((size_t)a->tokens_q * (size_t)a->heads * 4u);
  L.top = 2 * L.lse2;
  L.part = L.top + 2 * qlora::kAttnTops * 4u;
  L.total = L.part + qlora::attn_bwd_part_bytes(L.splits, a->tokens_k, a->kv_heads, a->head_dim);
  return L;
}

int check_ce_sizes(int64_t M, int64_t K, int64_t V) {
  int st;
  if ((st = check_range(M, INT_MAX, "M")) || (st = check_range(K, 1 << 20, "K")) || (st = check_range(V, 1 << 24, "V")))
    return st;
  if (K < 8 || K % 8) return fail(QLORA_ERR_SHAPE, "K must be a positive multiple of 8");
  if (V < 1) return fail(QLORA_ERR_SHAPE, "V must be at least 1");
  return QLORA_OK;
}

int check_aligned(const void* p, int align, const char* name) {
  if (!p) return fail(QLORA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail(QLORA_ERR_ALIGN, std::string(name) + " must be " + std::to_string(align) + "-byte aligned");
  return QLORA_OK;
}

int run_cross_entropy(const void* X, int64_t ldx, const void* W, int64_t ldw, const int64_t* targets, int64_t M, int64_t K,
                      int64_t V, int64_t ignore_index, const float* dloss, float* loss, float* lse, uint16_t* dX, float* unit,
                      bool units, int dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  int st;
  if ((st = check_ce_sizes(M, K, V)) || (st = check_type16(dtype))) return st;
  if (M == 0) return (int)QLORA_OK;
  if ((st = check_aligned(X, 2, "X")) || (st = check_aligned(W, 16, "W")) || (st = check_aligned(targets, 8, "targets")) ||
      (st = check_aligned(loss, 4, "loss")) || (st = check_aligned(lse, 4, "lse")))
    return st;
  if (dloss && (st = check_aligned(dloss, 4, "dloss"))) return st;
  if (units && (st = check_aligned(unit, 4, "unit"))) return st;
  if ((dX || units) && (st = check_aligned(dX, 16, "dX"))) return st;
  if (M == 1) ldx = K;
  if (V == 1) ldw = K;
  if (ldx < K || ldw < K) return fail(QLORA_ERR_INVALID_ARG, "a row stride is below the row length");
  if (ldx > kMostStride || ldw > (1 << 22)) return fail(QLORA_ERR_SHAPE, "a row stride is too large");
  if (ldw % 8) return fail(QLORA_ERR_ALIGN, "ldw must be a multiple of 8");
  if ((const void*)dX == X && ldx != K) return fail(QLORA_ERR_INVALID_ARG, "dX may be X only where its rows are contiguous");
  const int cus = qlora::device_compute_units();
  if (!ws || ws_bytes < qlora::ce_workspace_bytes(M, K, V, dX != nullptr, cus))
    return fail(QLORA_ERR_WORKSPACE, "cross entropy workspace too small");
  if (!aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
  qlora::CeArgs a{};
  a.x = static_cast<const uint16_t*>(X); a.w = static_cast<const uint16_t*>(W);
  a.ldx = ldx; a.ldw = ldw; a.m = M; a.k = K; a.v = V;
  a.targets = targets; a.ignore = ignore_index; a.dloss = dloss;
  a.loss = loss; a.lse = lse; a.dx = dX; a.unit = unit; a.f16 = dtype == QLORA_F16;
  return done(qlora::launch_ce(a, ws, cus, stream), "cross entropy launch");
}

}  // namespace

extern "C" {

int qlora_rope(const qlora_heads* Q, int64_t heads, const qlora_heads* K, int64_t kv_heads, int64_t tokens,
               int64_t head_dim, int64_t rot, int interleaved, const void* positions, int positions64,
               const uint64_t* turns, float factor, int inverse, const qlora_heads* Qo, const qlora_heads* Ko, int dtype,
               hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_range(heads, 65536, "heads")) || (st = check_range(kv_heads, 65536, "kv_heads")) ||
        (st = check_range(tokens, INT_MAX, "tokens")) || (st = check_range(head_dim, 65536, "head_dim")) ||
        (st = check_type16(dtype)))
      return st;
    if (rot < 0 || rot % 2 || rot > head_dim) return fail(QLORA_ERR_SHAPE, "rot must be even and at most head_dim");
    if (!std::isfinite(factor)) return fail(QLORA_ERR_INVALID_ARG, "factor must be finite");
    if ((st = check_heads(Q, tokens, heads, head_dim, 2, false, "Q")) ||
        (st = check_heads(K, tokens, kv_heads, head_dim, 2, false, "K")) ||
        (st = check_heads(Qo, tokens, heads, head_dim, 2, true, "Qo")) ||
        (st = check_heads(Ko, tokens, kv_heads, head_dim, 2, true, "Ko")))
      return st;
    if (tokens == 0 || heads + kv_heads == 0 || head_dim == 0) return (int)QLORA_OK;
    const auto in_place = [&](const qlora_heads* x, const qlora_heads* y, int64_t h) {
      return h == 0 || x->p != y->p || ((tokens == 1 || x->token_stride == y->token_stride) && (h == 1 || x->head_stride == y->head_stride));
    };
    if (!in_place(Q, Qo, heads) || !in_place(K, Ko, kv_heads))
      return fail(QLORA_ERR_INVALID_ARG, "in place, strides must be the same");
    // heads of one are written while the other's are read
    if (heads > 0 && kv_heads > 0 && (Qo->p == Ko->p || Qo->p == K->p || Ko->p == Q->p))
      return fail(QLORA_ERR_INVALID_ARG, "Qo and Ko must be apart from each other and from the other's input");
    if (rot > 0) {
      if (!positions || !turns) return fail(QLORA_ERR_INVALID_ARG, "positions or turns is NULL");
      if (reinterpret_cast<uintptr_t>(positions) % (positions64 ? 8 : 4) || reinterpret_cast<uintptr_t>(turns) % 8)
        return fail(QLORA_ERR_ALIGN, "positions and turns must be aligned to their element size");
    }
    qlora::RopeArgs a{};
    a.q = heads_arg(Q, tokens, heads, head_dim); a.qo = heads_arg(Qo, tokens, heads, head_dim);
    a.k = heads_arg(K, tokens, kv_heads, head_dim); a.ko = heads_arg(Ko, tokens, kv_heads, head_dim);
    a.t = tokens; a.heads = (int32_t)heads; a.kv_heads = (int32_t)kv_heads; a.d = (int32_t)head_dim; a.rot = (int32_t)rot;
    a.positions = positions; a.turns = turns; a.factor = factor;
    a.pos64 = positions64 != 0; a.interleaved = interleaved != 0; a.inverse = inverse != 0; a.f16 = dtype == QLORA_F16;
    return done(qlora::launch_rope(a, stream), "rotary positions launch");
  });
}

size_t qlora_attention_workspace_bytes(int op, const qlora_attention* a) {
  size_t n = 0;
  guarded([&] {
    if (check_attention(a, op == QLORA_OP_BWD) != QLORA_OK || nothing(a)) return (int)QLORA_OK;
    if (op == QLORA_OP_FWD)
      n = qlora::attn_part_bytes(plan_of(a, qlora::device_compute_units()), a->tokens_q, a->heads, a->head_dim);
    else if (op == QLORA_OP_BWD)
      n = bwd_ws(a).total;
    return (int)QLORA_OK;
  });
  return n;
}

int qlora_attention_plan(const qlora_attention* a, int compute_units, int64_t out[2]) {
  return guarded([&] {
    if (!out) return fail(QLORA_ERR_INVALID_ARG, "out is NULL");
    int st;
    if ((st = check_attention(a, false))) return st;
    const qlora::AttnPlan p = plan_of(a, compute_units > 0 ? compute_units : qlora::device_compute_units());
    out[0] = p.rows;
    out[1] = p.splits;
    return (int)QLORA_OK;
  });
}

int qlora_attention_fwd(const qlora_attention* a, const qlora_heads* Q, const qlora_heads* K, const qlora_heads* V,
                        const qlora_heads* O, float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_attention(a, false))) return st;
    const int64_t d = a->head_dim;
    if ((st = check_attn_heads(Q, a->tokens_q, a->heads, d, false, "Q")) ||
        (st = check_attn_heads(K, a->tokens_k, a->kv_heads, d, false, "K")) ||
        (st = check_attn_heads(V, a->tokens_k, a->kv_heads, d, false, "V")) ||
        (st = check_attn_heads(O, a->tokens_q, a->heads, d, true, "O")))
      return st;
    if (nothing(a) || a->tokens_q == 0) return (int)QLORA_OK;
    if (!lse) return fail(QLORA_ERR_INVALID_ARG, "lse is NULL");
    if (!aligned16(lse)) return fail(QLORA_ERR_ALIGN, "lse must be 16-byte aligned");
    if (ws && !aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
    if ((st = check_apart({O}, {Q, K, V}))) return st;
    qlora::AttnArgs g = attention_args(a);
    g.q = heads_arg(Q, a->tokens_q, a->heads, d); g.k = heads_arg(K, a->tokens_k, a->kv_heads, d);
    g.v = heads_arg(V, a->tokens_k, a->kv_heads, d); g.o = heads_arg(O, a->tokens_q, a->heads, d);
    g.lse = lse;
    qlora::AttnPlan p = plan_of(a, qlora::device_compute_units());
    if (!ws || ws_bytes < qlora::attn_part_bytes(p, a->tokens_q, a->heads, d)) p.splits = 1;
    g.part = static_cast<float*>(ws);
    return done(qlora::launch_attn_fwd(g, p, stream), "attention launch");
  });
}

int qlora_attention_bwd(const qlora_attention* a, const qlora_heads* dO, const qlora_heads* Q, const qlora_heads* K,
                        const qlora_heads* V, const qlora_heads* O, const float* lse, const qlora_heads* dQ,
                        const qlora_heads* dK, const qlora_heads* dV, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_attention(a, true))) return st;
    const int64_t d = a->head_dim, tq = a->tokens_q, tk = a->tokens_k, h = a->heads, hk = a->kv_heads;
    if ((st = check_attn_heads(dO, tq, h, d, false, "dO")) || (st = check_attn_heads(Q, tq, h, d, false, "Q")) ||
        (st = check_attn_heads(K, tk, hk, d, false, "K")) || (st = check_attn_heads(V, tk, hk, d, false, "V")) ||
        (st = check_attn_heads(O, tq, h, d, false, "O")) || (st = check_attn_heads(dQ, tq, h, d, true, "dQ")) ||
        (st = check_attn_heads(dK, tk, hk, d, true, "dK")) || (st = check_attn_heads(dV, tk, hk, d, true, "dV")))
      return st;
    if (nothing(a)) return (int)QLORA_OK;
    if (tq > 0 && !lse) return fail(QLORA_ERR_INVALID_ARG, "lse is NULL");
    if (!aligned16(lse)) return fail(QLORA_ERR_ALIGN, "lse must be 16-byte aligned");
    if (!ws || ws_bytes < qlora_attention_workspace_bytes(QLORA_OP_BWD, a))
      return fail(QLORA_ERR_WORKSPACE, "attention backward workspace too small");
    if (!aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
    if ((st = check_apart({dQ, dK, dV}, {dO, Q, K, V, O}))) return st;
    qlora::AttnArgs g = attention_args(a);
    g.dout = heads_arg(dO, tq, h, d); g.q = heads_arg(Q, tq, h, d); g.k = heads_arg(K, tk, hk, d);
    g.v = heads_arg(V, tk, hk, d); g.o = heads_arg(O, tq, h, d); g.lse = const_cast<float*>(lse);
    g.dq = heads_arg(dQ, tq, h, d); g.dk = heads_arg(dK, tk, hk, d); g.dv = heads_arg(dV, tk, hk, d);
    const BwdWs L = bwd_ws(a);
    char* base = static_cast<char*>(ws);
    return done(qlora::launch_attn_bwd(g, reinterpret_cast<float*>(base), reinterpret_cast<float*>(base + L.lse2),
                                       reinterpret_cast<float*>(base + L.top), reinterpret_cast<float*>(base + L.part), L.splits,
                                       stream),
                "attention backward launch");
  });
}

size_t qlora_cross_entropy_workspace_bytes(int64_t M, int64_t K, int64_t V, int with_gradient) {
  size_t n = 0;
  guarded([&] {
    if (check_ce_sizes(M, K, V) == QLORA_OK && M > 0)
      n = qlora::ce_workspace_bytes(M, K, V, with_gradient != 0, qlora::device_compute_units());
    return (int)QLORA_OK;
  });
  return n;
}

int qlora_cross_entropy(const void* X, int64_t ldx, const void* W, int64_t ldw, const int64_t* targets, int64_t M,
                        int64_t K, int64_t V, int64_t ignore_index, const float* dloss, float* loss, float* lse,
                        uint16_t* dX, int dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    return run_cross_entropy(X, ldx, W, ldw, targets, M, K, V, ignore_index, dloss, loss, lse, dX, nullptr, false, dtype, ws,
                             ws_bytes, stream);
  });
}

int qlora_cross_entropy_units(const void* X, int64_t ldx, const void* W, int64_t ldw, const int64_t* targets, int64_t M,
                              int64_t K, int64_t V, int64_t ignore_index, float* loss, float* lse, uint16_t* dX, float* unit,
                              int dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  return guarded([&] {
    return run_cross_entropy(X, ldx, W, ldw, targets, M, K, V, ignore_index, nullptr, loss, lse, dX, unit, true, dtype, ws,
                             ws_bytes, stream);
  });
}

int qlora_scale_rows(const uint16_t* X, const float* g, int64_t M, int64_t K, uint16_t* Y, int dtype, hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_range(M, INT_MAX, "M")) || (st = check_range(K, 1 << 20, "K")) || (st = check_type16(dtype))) return st;
    if (K % 8) return fail(QLORA_ERR_SHAPE, "K must be a multiple of 8");
    if (M == 0 || K == 0) return (int)QLORA_OK;
    if ((st = check_aligned(X, 16, "X")) || (st = check_aligned(g, 4, "g")) || (st = check_aligned(Y, 16, "Y"))) return st;
    return done(qlora::launch_scale_rows(X, g, M, K, Y, dtype == QLORA_F16, stream), "row scale launch");
  });
}

int qlora_loss_sum(const float* loss, const int64_t* targets, int64_t M, int64_t ignore_index, int mean, float* out,
                   hipStream_t stream) {
  return guarded([&] {
    int st;
    if ((st = check_range(M, INT_MAX, "M"))) return st;
    if (M > 0 && ((st = check_aligned(loss, 4, "loss")) || (st = check_aligned(targets, 8, "targets")))) return st;
    if ((st = check_aligned(out, 4, "out"))) return st;
    return done(qlora::launch_loss_sum(loss, targets, M, ignore_index, mean != 0, out, stream), "loss sum launch");
  });
}

}  // extern "C"
