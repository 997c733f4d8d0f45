// Host-side argument blocks and launchers of what stands between a decoder's
// linears and at its end: rotary positions, attention, the head's loss.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

// A 16-bit tensor [tokens, heads, d], values of a head contiguous.
struct Heads {
  const uint16_t* p;
  int64_t token, head;  // strides in elements
  int64_t n;            // elements from p to the end of the last head
};

inline Heads heads_of(const void* p, int64_t token, int64_t head, int64_t t, int64_t h, int64_t d) {
  return Heads{static_cast<const uint16_t*>(p), token, head, t > 0 && h > 0 ? (t - 1) * token + (h - 1) * head + d : 0};
}

// ---- rotary positions (rope.hip) ----
struct RopeArgs {
  Heads q, k, qo, ko;  // outputs are written
  int64_t t;
  int32_t heads, kv_heads, d, rot;
  const void* positions;  // int32 or int64 [t]
  const uint64_t* turns;  // [rot / 2], 2^-64 of a turn for each position
  float factor;
  bool pos64, interleaved, inverse, f16;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// ---- attention (attention.hip, attention_bwd.hip) ----
struct AttnArgs {
  Heads q, k, v, o, dout, dq, dk, dv;
  float* lse;              // [tq, heads]
  const float *delta, *lse2;  // backward: [tq, heads]
  const float* top;        // fp16 backward: [2 kAttnTops] partial maxima of |dO|, then of |V|
  const int32_t *cu_q, *cu_k, *len_q, *len_k;
  float* part;             // forward, split keys: [splits][tq][heads][d] and then [splits][tq][heads] log-sums;
                           // backward, split query heads: [splits][tk][kv_heads][dK, dV][d]
  int64_t tq, tk;
  int32_t batch, heads, kv_heads, group, d;
  int32_t splits;
  float scale;
  bool causal, zero_rest, f16;
};

constexpr int kAttnTops = 1024;  // partial maxima of the fp16 backward, for each of dO and V

// How a forward runs: rows of a workgroup (128, or 32 whose four waves share
// out the keys) and over how many workgroups a row's keys are split.
struct AttnPlan {
  int rows, splits;
};
AttnPlan attn_plan(int64_t tq, int64_t tk, int64_t batch, int64_t heads, int64_t kv_heads, int compute_units);
size_t attn_part_bytes(const AttnPlan& p, int64_t tq, int64_t heads, int64_t d);

hipError_t launch_attn_fwd(const AttnArgs& a, const AttnPlan& p, hipStream_t stream);
int attn_bwd_splits(int64_t tk, int64_t batch, int64_t heads, int64_t kv_heads, int compute_units);
size_t attn_bwd_part_bytes(int splits, int64_t tk, int64_t kv_heads, int64_t d);
hipError_t launch_attn_bwd(const AttnArgs& a, float* delta, float* lse2, float* top, float* part, int splits,
                           hipStream_t stream);

// ---- the head's cross entropy (cross_entropy.hip) ----
struct CeArgs {
  const uint16_t *x, *w;  // [m, k] (ldx), [v, k] (ldw)
  int64_t ldx, ldw, m, k, v;
  const int64_t* targets;  // [m]
  int64_t ignore;
  const float* dloss;      // [m] or NULL (ones)
  float *loss, *lse;       // [m]
  uint16_t* dx;            // [m, k] contiguous, or NULL: no gradient
  float* unit;             // [m] or NULL: dx times a power of two for each row, written here
  bool f16;
};
size_t ce_workspace_bytes(int64_t m, int64_t k, int64_t v, bool grad, int compute_units);
hipError_t launch_ce(const CeArgs& a, void* ws, int compute_units, hipStream_t stream);
hipError_t launch_scale_rows(const uint16_t* x, const float* g, int64_t m, int64_t k, uint16_t* out, bool f16,
                             hipStream_t stream);
hipError_t launch_loss_sum(const float* loss, const int64_t* targets, int64_t m, int64_t ignore, bool mean, float* out,
                           hipStream_t stream);

}  // namespace qlora
