// Attention of packed sequences, backward.  With P = exp(scale Q K^T - lse) at
// the keys a row sees (0 elsewhere) and delta = sum_d dO O:
//
//   dV = P^T dO,  dS = P (dO V^T - delta),  dQ = scale dS K,  dK = scale dS^T Q,
//
// dK and dV summed over the query heads of a key head.  P is made again from
// the log-sums.  Two kernels: one goes over the queries for a tile of keys (dK,
// dV), one over the keys for a tile of queries (dQ).  That computes the scores
// and dO V^T twice (7 products instead of 5), but every sum has one owner: no
// atomics, the same bits every time.
//
// P and dS are matrix operands in 16 bits.  In fp16 their small values would
// fall below its range, so P is kept times 2^12, and dS times a power of two
// from a bound on it: |dS| <= 2 d max|dO| max|V|, taken to 2^14 at most.  The
// maxima are of the finite values (over the row for dQ, over all for dK).
//
// Masked places: P and dS are set to zero there, whatever the values are, and
// infinities and NaNs of the second products' other operand are kept out of tiles
// that are seen only in part.  dO's are added to dV at the end where they are
// seen; Q's show in dK (and dV) through their rows' lse, which is a NaN; a K that
// is not finite makes the dQ of the rows that see it NaN (and its own dK and dV,
// through rows past the last, also where all scores are -inf).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "attention_common.h"

namespace qlora {
namespace {

constexpr int kDeltaTokens = 4;  // tokens of a delta tile
constexpr int kFewKeys = 32;      // rows that see no more get delta from P and dO V
constexpr float kPShift = 12.f;   // fp16: P times 2^12

template <typename E>
struct IsF16 { static constexpr bool value = false; };
template <>
struct IsF16<F16> { static constexpr bool value = true; };

template <typename E>
__device__ __forceinline__ float finite_max(const uint4& u) {
  const uint4 f = finite_part<E>(u);
  const uint32_t d[4] = {f.x, f.y, f.z, f.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(E::widen((uint16_t)d[i])), fabsf(E::widen((uint16_t)(d[i] >> 16)))));
  return m;
}

__device__ __forceinline__ int tops_of(int64_t tokens, int64_t batch) {
  const int64_t n = attn_tiles(tokens, 1, batch, kDeltaTokens);
  return (int)(n < kAttnTops ? n : kAttnTops);
}

// sum of 8 products
template <typename E>
__device__ __forceinline__ float dot8(const uint4& u, const uint4& v) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s += E::widen((uint16_t)p[i]) * E::widen((uint16_t)q[i]);
    s += E::widen((uint16_t)(p[i] >> 16)) * E::widen((uint16_t)(q[i] >> 16));
  }
  return s;
}

template <typename E>
constexpr float kShift = IsF16<E>::value ? kPShift : 0.f;

// delta of the rows that see few keys, as sum P (dO V) by the matrix cores: O is
// rounded, by up to half a step of itself, and a row's dS is as far off as its
// delta.  (Where a row spreads over many keys, O is small beside the V that it is
// made of.)  Wave w: sequence w / heads, head w % heads.
template <typename E, int DB>
__device__ __forceinline__ void delta_few(const AttnArgs& a, int64_t w, float* delta) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  if (w >= (int64_t)a.batch * a.heads) return;
  const int32_t seq = (int32_t)(w / a.heads), head = (int32_t)(w % a.heads);
  const int64_t start = region_start(a.cu_q, a.batch, a.tq, seq + 1);
  const int64_t size = clampl(region_start(a.cu_q, a.batch, a.tq, seq + 2), start, a.tq) - start;
  const int32_t n = seq_length(a.len_q, seq, a.batch, size);
  const Keys ks = keys_of(a, seq);
  // the rows that see 1 .. kFewKeys keys
  const int32_t shift = ks.n - n;
  const int32_t from = a.causal ? max(0, -shift) : 0;
  const int32_t to = a.causal ? min(n, kFewKeys - shift) : ks.n <= kFewKeys ? n : 0;
  if (ks.n == 0) return;
  const int32_t key = lane & 31, kv_head = head / a.group;
  const bool live = key < ks.n;
  for (int32_t t0 = from; t0 < to; t0 += 32) {
    const int32_t t = t0 + (lane & 31);
    const bool row = t < to;
    const int64_t tok = start + t;
    f32x16 s = (f32x16)(0.f), dp = (f32x16)(0.f);
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) {
      const int c = 16 * i + 8 * half;
      const bool in = c < a.d;
      const uint4 k = load16(a.k, (ks.start + key) * a.k.token + kv_head * a.k.head + c, live && in);
      const uint4 v = load16(a.v, (ks.start + key) * a.v.token + kv_head * a.v.head + c, live && in);
      const uint4 q = load16(a.q, tok * a.q.token + head * a.q.head + c, row && in);
      const uint4 d = load16(a.dout, tok * a.dout.token + head * a.dout.head + c, row && in);
      s = E::mfma32(E::vec(k), E::vec(q), s);
      dp = E::mfma32(E::vec(v), E::vec(d), dp);
    }
    const int64_t at = tok * a.heads + head;
    const bool ok = row && in_bounds(at, 1, a.tq * a.heads);
    const float l = ok ? a.lse[at] * kLog2e : 0.f;
    const int32_t sees = a.causal ? min(ks.n, t + shift + 1) : ks.n;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (8 * (r / 4) + 4 * half + r % 4 < sees)
        sum += __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.scale * kLog2e, -l)) * dp[r];
    sum = half_sum(sum);
    if (ok && half == 0) delta[at] = sum;
  }
}

// delta = sum_d dO O, 16 lanes a row, and lse in base 2, less P's power of two; in
// fp16 (blockIdx.y: dO, V) also the largest finite magnitude of each workgroup's
// rows.  The first `few` workgroups (of blockIdx.y 0) see to the rows with few keys.
// Bound by memory where there are many tokens (8192, 32 heads of 128: 30 to 34 us,
// 4.0 to 4.5 TB/s; tiles of 4 tokens, since tiles of 32 left compute units idle at 2048).
template <typename E, int DB>
__global__ __launch_bounds__(256) void k_attn_delta(AttnArgs a, uint32_t few, float* delta, float* lse2, float* top) {
  const bool isv = blockIdx.y == 1;
  if (blockIdx.x < few) {
    if (!isv) delta_few<E, DB>(a, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), delta);
    return;
  }
  const Heads& x = isv ? a.v : a.dout;
  const int32_t heads = isv ? a.kv_heads : a.heads;
  const int64_t tokens = isv ? a.tk : a.tq, tiles = attn_tiles(tokens, 1, a.batch, kDeltaTokens);
  const int sub = threadIdx.x >> 4, l16 = threadIdx.x & 15;
  float most = 0.f;
  for (int64_t t = blockIdx.x - few; t < tiles; t += gridDim.x - few) {
    const Region rg = find_region(isv ? a.cu_k : a.cu_q, a.batch, tokens, 1, kDeltaTokens, t);
    if (rg.tile < 0) continue;
    const int32_t n = seq_length(isv ? a.len_k : a.len_q, rg.seq, a.batch, rg.size), first = rg.tile * kDeltaTokens;
    const int32_t rows = max(0, min(n - first, kDeltaTokens)) * heads;
    const Keys ks = keys_of(a, rg.seq);
    for (int32_t r = sub; r < rows; r += 16) {
      const int64_t tok = rg.start + first + r / heads, head = r % heads;
      float sum = 0.f;
      for (int c = 8 * l16; c < a.d; c += 128) {
        const uint4 u = load16(x, tok * x.token + head * x.head + c, true);
        if (IsF16<E>::value) most = fmaxf(most, finite_max<E>(u));
        if (!isv) {
          sum += dot8<E>(u, load16(a.o, tok * a.o.token + head * a.o.head + c, true));
        }
      }
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) sum += __shfl_xor(sum, s, 16);
      const int32_t sees = a.causal ? min(ks.n, first + r / heads + ks.n - n + 1) : ks.n;
      if (!isv && l16 == 0 && in_bounds(tok * heads + head, 1, a.tq * heads)) {
        const float l = a.lse[tok * heads + head] * kLog2e;
        if (sees <= 0 || sees > kFewKeys) delta[tok * heads + head] = sum;  // the others: delta_few
        lse2[tok * heads + head] = l == -INFINITY ? INFINITY : l - kShift<E>;  // a row that sees nothing: P = 0
      }
    }
  }
  if constexpr (IsF16<E>::value) {
    __shared__ float s_top[4];
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor(most, s));
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = most;
    __syncthreads();
    const int at = (isv ? kAttnTops : 0) + blockIdx.x - few;
    if (threadIdx.x == 0 && in_bounds(at, 1, 2 * kAttnTops))
      top[at] = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  }
}

// The largest of the partial maxima, in every thread.  All threads take part.
__device__ __forceinline__ float all_tops(const float* top, int n, float* s_top) {
  float m = 0.f;
  for (int i = threadIdx.x; i < n; i += 256) m = fmaxf(m, in_bounds(i, 1, kAttnTops) ? top[i] : 0.f);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
}

// A power of two that takes values up to `bound` to 2^14 at most.
__device__ __forceinline__ float to_range(float bound) {
  const int e = (int)(__builtin_bit_cast(uint32_t, bound) >> 23) - 126;  // bound < 2^e
  return __builtin_bit_cast(float, (uint32_t)(max(-100, min(100, 14 - e)) + 127) << 23);
}

// dQ: 128 rows a workgroup, 32 a wave, tiles of 64 keys.  Q, dO and dQ stay in
// registers.  Bound by the matrix cores, 67 % busy near 1.8 GHz (8192 causal tokens, 32
// heads of 128 on 8: 690 to 770 us, 1.07 to 1.19 PFLOP/s); they wait for operands from
// LDS, one read a product, and share the issue with vector instructions (50 % of the
// cycles).
template <typename E, int DB>
__global__ __launch_bounds__(256, 2) void k_attn_bwd_q(AttnArgs a) {
  constexpr int BN = 64, BM = 128;
  constexpr int CH = Tile<DB>::kChunks, PER = BN * CH / 256, BYTES = BN * Tile<DB>::kPitch;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * BYTES];
  __shared__ int s_bad;  // the first key that is not finite
  __shared__ float s_top[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
  const int32_t kv_head = blockIdx.x % a.kv_heads;
  const int64_t t = attn_tiles(a.tq, a.group, a.batch, BM) - 1 - blockIdx.x / a.kv_heads;
  const Region rg = find_region(a.cu_q, a.batch, a.tq, a.group, BM, t);
  if (rg.tile < 0 || (int64_t)rg.tile * BM >= rg.size * a.group) return;
  const int32_t nq = seq_length(a.len_q, rg.seq, a.batch, rg.size);
  const Keys ks = keys_of(a, rg.seq);
  const int32_t rows = nq * a.group, first = rg.tile * BM, wfirst = first + wave * 32, row = wfirst + (lane & 31);
  const bool live = row < rows;
  const int32_t tok = row / a.group, head = kv_head * a.group + row % a.group;
  const int64_t o_at = (rg.start + tok) * a.dq.token + head * a.dq.head;
  if (a.zero_rest && !live && row < rg.size * a.group)
    for (int c = 8 * half; c < a.d; c += 16)
      if (in_bounds(o_at + c, 8, a.dq.n))
        *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.dq.p) + o_at + c) = make_uint4(0, 0, 0, 0);
  if (first >= rows) return;

  const int32_t shift = ks.n - nq;
  const int32_t last = !live ? -1 : a.causal ? min(ks.n - 1, tok + shift) : ks.n - 1;
  const int32_t end = a.causal ? max(0, min(ks.n, (min(first + BM, rows) - 1) / a.group + shift + 1)) : ks.n;
  const int32_t whole = a.causal ? min(ks.n, first / a.group + shift + 1) : ks.n;
  const int32_t wend = a.causal ? min(ks.n, (min(wfirst + 32, rows) - 1) / a.group + shift + 1) : ks.n;
  const int32_t k1 = (end + BN - 1) / BN;

  uint4 qf[2 * DB], df[2 * DB];
  float most = 0.f;
#pragma unroll
  for (int s = 0; s < 2 * DB; ++s) {
    const int c = 16 * s + 8 * half;
    qf[s] = load16(a.q, (rg.start + tok) * a.q.token + head * a.q.head + c, live && c < a.d);
    df[s] = load16(a.dout, (rg.start + tok) * a.dout.token + head * a.dout.head + c, live && c < a.d);
    if (IsF16<E>::value) most = fmaxf(most, finite_max<E>(df[s]));
  }
  const int64_t r_at = (rg.start + tok) * a.heads + head;
  float lse = INFINITY, delta = 0.f;  // a row that sees nothing: P = 0
  if (live && in_bounds(r_at, 1, a.tq * a.heads)) {
    lse = a.lse2[r_at] + kShift<E>;
    delta = a.delta[r_at];
  }
  float up = 1.f;
  if constexpr (IsF16<E>::value) {
    const float vtop = all_tops(a.top + kAttnTops, tops_of(a.tk, a.batch), s_top);
    up = to_range(2.f * a.d * half_max(most) * vtop);
  }
  const float c2 = a.scale * kLog2e;

  // a thread's pieces of a tile (columns past d: none)
  Tile<DB> at(lane);
  uint4 st[2][PER];
  const auto off = [&](const Heads& x, int u) {
    const uint32_t c = Fill<DB>::column(tid, 256, u);
    return c < (uint32_t)a.d ? ((Fill<DB>::row(tid) + u * (256 / CH)) * (uint32_t)x.token + c) * 2 : kOOB;
  };
  const auto first_key = [&](const Heads& x, int32_t kt) { return (ks.start + (int64_t)kt * BN) * x.token + kv_head * x.head; };
  auto load = [&](int32_t kt) {
    const int64_t left = kt < k1 ? ks.n - (int64_t)kt * BN : 0;
    const __amdgpu_buffer_rsrc_t rk = rows_rsrc(a.k, first_key(a.k, kt), left, a.d), rv = rows_rsrc(a.v, first_key(a.v, kt), left, a.d);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      st[0][u] = buf_load16(rk, off(a.k, u));
      st[1][u] = buf_load16(rv, off(a.v, u));
    }
  };
  auto store = [&](int32_t kt, int buf) {
    uint8_t* const to = lds + buf * 2 * BYTES;
    const bool part = (kt + 1) * BN > whole;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int c = u * 256 + tid;
      if (part && not_finite<E>(st[0][u])) {
        atomicMin(&s_bad, kt * BN + c / CH);
        st[0][u] = finite_part<E>(st[0][u]);
      }
      *reinterpret_cast<uint4*>(to + c * 16) = st[0][u];
      *reinterpret_cast<uint4*>(to + BYTES + c * 16) = st[1][u];
    }
  };

  f32x16 dq[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) dq[b] = (f32x16)(0.f);
  // The scores of a tile's second half are computed beside dS of the first, dQ of
  // the first beside dS of the second; operands come from LDS through a ring of
  // registers, RING products ahead.  MASKED: some of the rows do not see it in full
  auto tile = [&](int32_t kt, const uint8_t* kb, auto MASKED) {
    at.renew();
    const uint8_t* vb = kb + BYTES;
    constexpr int N = 2 * DB, RING = 4, EP = 8 / DB;  // products of each kind, dS beside each of them
    uint4 ring[RING];
    auto fetch = [&](int f) {
      if (f < 4 * N) ring[f % RING] = at.rows(f / N % 2 ? vb : kb, 32 * (f / (2 * N)), f % N);
      else if (f < 6 * N) ring[f % RING] = at.cols(kb, 16 * ((f - 4 * N) / N * 2 + f % 2), f % N / 2);
    };
    f32x16 s[2], dp[2];
    typename E::v8 ds[2][2];
    auto make_ds = [&](int u, int e) {
      s[u][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e], c2, -lse)) * ((dp[u][e] - delta) * up);
      if constexpr (decltype(MASKED)::value)
        if (kt * BN + 32 * u + 8 * (e / 4) + 4 * half + e % 4 > last) s[u][e] = 0.f;
      if (e % 8 == 7) ds[u][e / 8] = pack8<E>(s[u], e / 8 * 8);
    };
#pragma unroll
    for (int f = 0; f < RING; ++f) fetch(f);
#pragma unroll
    for (int u = 0; u < 2; ++u) s[u] = dp[u] = (f32x16)(0.f);
#pragma unroll
    for (int f = 0; f < 4 * N; ++f) {
      const int u = f / (2 * N);
      if (f / N % 2 == 0) s[u] = E::mfma32(E::vec(ring[f % RING]), E::vec(qf[f % N]), s[u]);
      else dp[u] = E::mfma32(E::vec(ring[f % RING]), E::vec(df[f % N]), dp[u]);
      fetch(f + RING);
      if (u == 1) {
#pragma unroll
        for (int e = EP / 2 * (f - 2 * N); e < EP / 2 * (f - 2 * N + 1); ++e) make_ds(0, e);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int f = 4 * N; f < 6 * N; ++f) {
      const int u = (f - 4 * N) / N, b = f % N / 2;
      dq[b] = E::mfma32(E::vec(ring[f % RING]), ds[u][f % 2], dq[b]);
      fetch(f + RING);
      if (u == 0) {
#pragma unroll
        for (int e = EP * (f - 4 * N); e < EP * (f - 4 * N + 1); ++e) make_ds(1, e);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (tid == 0) s_bad = INT_MAX;
  __syncthreads();  // here: where no row sees a key there is no other before s_bad is read
  const int32_t kf = max(0, min(k1, whole / BN));  // the first tile that not all rows see in full
  if (kf > 0) {
    const uint32_t lds0 = lds_offset(lds) + wave * 1024;
    auto direct = [&](int32_t kt, uint32_t to) {
      const LdsSource rk = rows_source(a.k, first_key(a.k, kt), kt < kf ? BN : 0, a.d);
      const LdsSource rv = rows_source(a.v, first_key(a.v, kt), kt < kf ? BN : 0, a.d);
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        load_to_lds16(rk, off(a.k, u), to + u * 4096);
        load_to_lds16(rv, off(a.v, u), to + BYTES + u * 4096);
      }
    };
    direct(0, lds0);
    tile_barrier();
    for (int32_t kt = 0; kt < kf; ++kt) {
      const int buf = kt & 1;
      direct(kt + 1, lds0 + (buf ^ 1) * 2 * BYTES);
      tile(kt, lds + buf * 2 * BYTES, std::false_type{});
      tile_barrier();
    }
  }
  if (kf < k1) {
    __syncthreads();
    load(kf);
    store(kf, 0);
    load(kf + 1);
    __syncthreads();
    for (int32_t kt = kf; kt < k1; ++kt) {
      const int buf = (kt - kf) & 1;
      if (kt + 1 < k1) {
        store(kt + 1, buf ^ 1);
        load(kt + 2);
      }
      if (kt * BN < wend) tile(kt, lds + buf * 2 * BYTES, std::true_type{});
      __syncthreads();
    }
  }
  const float f = s_bad <= last ? NAN : a.scale / up;
#pragma unroll
  for (int b = 0; b < DB; ++b) store_block<E>(a.dq, o_at, live, b, a.d, dq[b], f, lane);
}

// dK and dV: 128 keys a workgroup, 32 a wave, tiles of 32 rows of queries.
// Workgroups of split z take every query head z of a key head's sets of
// group / splits heads; with more than one split their sums go to `part`.
//
// dK and dV take 128 registers, K's operands 32; V's are read from LDS each time
// (in registers they would leave none for operands on their way: slower, as were 64
// keys a wave with 512 registers a lane).  Operands come from LDS through a ring of
// four, ahead of their products (six and eight were slower); exponentials are made
// beside dO V^T and dS beside dV.  Bound by waits for operands, one or two of which
// each product reads from LDS (36 to 40 % busy): matrix cores 48 to 52 % busy (8192 causal tokens,
// 32 heads of 128 on 8: 1.1 to 1.3 ms, 0.85 to 1.0 PFLOP/s), and 14 % of the time the last
// workgroups leave places empty.  Waves that skip row tiles none of whose rows see
// their keys: no faster.
template <typename E, int DB>
__global__ __launch_bounds__(256, 2) void k_attn_bwd_kv(AttnArgs a) {
  constexpr int BQ = 32, BK = 128;
  constexpr int CH = Tile<DB>::kChunks, PER = BQ * CH / 256, BYTES = BQ * Tile<DB>::kPitch;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * BYTES], s_v[BK * Tile<DB>::kPitch];
  __shared__ __attribute__((aligned(16))) float s_lse[2][64], s_delta[2][64];
  __shared__ __attribute__((aligned(16))) int s_last[2][BQ];
  __shared__ NonFinite<32 * DB> s_bad;
  __shared__ float s_top[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
  const int32_t kv_head = blockIdx.x % a.kv_heads, z = blockIdx.x / a.kv_heads % a.splits;
  const Region rg = find_region(a.cu_k, a.batch, a.tk, 1, BK, blockIdx.x / a.kv_heads / a.splits);
  if (rg.tile < 0 || (int64_t)rg.tile * BK >= rg.size) return;
  const int32_t nk = seq_length(a.len_k, rg.seq, a.batch, rg.size);
  const int32_t key0 = rg.tile * BK, key = key0 + wave * 32 + (lane & 31);
  const bool live = key < nk;
  const int64_t tok = rg.start + key;
  const int64_t k_at = tok * a.dk.token + kv_head * a.dk.head, v_at = tok * a.dv.token + kv_head * a.dv.head;
  if (a.zero_rest && z == 0 && !live && key < rg.size)
    for (int c = 8 * half; c < a.d; c += 16) {
      if (in_bounds(k_at + c, 8, a.dk.n))
        *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.dk.p) + k_at + c) = make_uint4(0, 0, 0, 0);
      if (in_bounds(v_at + c, 8, a.dv.n))
        *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.dv.p) + v_at + c) = make_uint4(0, 0, 0, 0);
    }
  if (key0 >= nk) return;

  // the sequence's queries
  const int64_t q0 = region_start(a.cu_q, a.batch, a.tq, rg.seq + 1);
  const int64_t qsize = clampl(region_start(a.cu_q, a.batch, a.tq, rg.seq + 2), q0, a.tq) - q0;
  const int32_t nq = seq_length(a.len_q, rg.seq, a.batch, qsize), off = nk - nq;
  const int32_t group = a.group / a.splits, rows = nq * group, head0 = kv_head * a.group + z * group;
  const int32_t t0 = a.causal ? max(0, key0 - off) : 0;  // the first query that sees the first key
  // tiles of rows: from r0 on; from rf on every row sees all keys here.  (Rows past
  // the last have P = 0, keys past the last are not stored: neither needs a mask.)
  const int64_t tf = a.causal ? max(0, min(key0 + BK, nk) - 1 - off) : 0;
  const int32_t r0 = (int32_t)min((int64_t)t0 * group, (int64_t)rows) / BQ, r1 = (rows + BQ - 1) / BQ;
  const int32_t rf = max(r0, (int32_t)min((tf * group + BQ - 1) / BQ, (int64_t)r1));

  uint4 kf[2 * DB];
#pragma unroll
  for (int s = 0; s < 2 * DB; ++s) {
    const int c = 16 * s + 8 * half;
    kf[s] = load16(a.k, tok * a.k.token + kv_head * a.k.head + c, live && c < a.d);
  }
#pragma unroll
  for (int u = 0; u < BK * CH / 256; ++u) {
    const int c = u * 256 + tid, col = Fill<DB>::column(tid, 256, u);
    const int32_t k = key0 + c / CH;
    *reinterpret_cast<uint4*>(s_v + c * 16) =
        load16(a.v, (rg.start + k) * a.v.token + kv_head * a.v.head + col, k < nk && col < a.d);
  }
  float up = 1.f;
  if constexpr (IsF16<E>::value) {
    const float dtop = all_tops(a.top, tops_of(a.tq, a.batch), s_top);
    up = to_range(2.f * a.d * dtop * all_tops(a.top + kAttnTops, tops_of(a.tk, a.batch), s_top));
  }
  const float ups = up * __builtin_amdgcn_exp2f(-kShift<E>);
  const float c2 = a.scale * kLog2e;

  // a thread's pieces of a tile, of Q and dO: rows tid / CH + u 256 / CH, the same
  // columns ch8 .. + 7 (256 / CH is a multiple of 16: so is the permutation)
  Tile<DB> at(lane);
  const uint32_t ch8 = Fill<DB>::column(tid, 256, 0);
  const int64_t q_at = q0 * a.q.token + head0 * a.q.head, d_at = q0 * a.dout.token + head0 * a.dout.head;
  uint4 st[2][PER];
  float st_lse = 0.f, st_delta = 0.f;
  int st_last = 0;
  // through registers; nothing past the last row
  auto load = [&](int32_t rt) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int32_t r = rt * BQ + (u * 256 + tid) / CH, tok = r / group, head = r % group;
      const bool ok = tok < nq && ch8 < (uint32_t)a.d;
      st[0][u] = load16(a.q, q_at + tok * a.q.token + head * a.q.head + ch8, ok);
      st[1][u] = load16(a.dout, d_at + tok * a.dout.token + head * a.dout.head + ch8, ok);
    }
    if (tid < BQ) {
      const int32_t r = rt * BQ + tid, tok = r / group;
      const int64_t i = (q0 + tok) * a.heads + head0 + r % group;
      st_lse = INFINITY;
      st_delta = 0.f;
      st_last = -1;
      if (tok < nq && in_bounds(i, 1, a.tq * a.heads)) {
        st_lse = a.lse2[i];
        st_delta = a.delta[i];
        st_last = a.causal ? min(nk - 1, tok + off) : nk - 1;
      }
    }
  };
  auto store = [&](int32_t rt, int buf) {
    uint8_t* const to = lds + buf * 2 * BYTES;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int c = u * 256 + tid;
      if (rt < rf) {
        if (not_finite<E>(st[1][u])) {
          const int32_t t = (rt * BQ + c / CH) / group;
          s_bad.template take<E, false>(st[1][u], ch8, a.causal ? min(nk - 1, t + off) : nk - 1);
        }
        if (not_finite<E>(st[0][u])) st[0][u] = finite_part<E>(st[0][u]);
      }
      *reinterpret_cast<uint4*>(to + c * 16) = st[0][u];
      *reinterpret_cast<uint4*>(to + BYTES + c * 16) = st[1][u];
    }
    if (tid < BQ) {
      s_lse[buf][tid] = st_lse;
      s_delta[buf][tid] = st_delta;
      s_last[buf][tid] = st_last;
    }
  };

  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) dk[b] = dv[b] = (f32x16)(0.f);
  auto tile = [&](int32_t rt, int buf, auto MASKED) {
    at.renew();
    constexpr bool kMasked = decltype(MASKED)::value;
    const uint8_t *qb = lds + buf * 2 * BYTES, *db = qb + BYTES, *vb = s_v + 32 * wave * Tile<DB>::kPitch;
    // Operands in the order of their use, each read from LDS into a ring of
    // registers while the products before it run.
    constexpr int N = 2 * DB, RING = 4, EP = 16 / N;
    uint4 ring[RING];
    auto fetch = [&](int f) {
      if (f < N) ring[f % RING] = at.rows(qb, 0, f);
      else if (f < 3 * N) ring[f % RING] = at.rows((f - N) % 2 ? vb : db, 0, (f - N) / 2);
      else if (f < 5 * N) ring[f % RING] = at.cols(f < 4 * N ? db : qb, 16 * (f % 2), f % N / 2);
    };
    // row values (lse, delta) of accumulators EP i .. EP i + EP - 1
    float aux[2][EP];
    auto fetch_rows = [&](const float* v, int i) {
#pragma unroll
      for (int j = 0; j < EP; ++j) {
        const int r = EP * i + j;
        aux[i % 2][j] = v[8 * (r / 4) + 4 * half + r % 4];
      }
    };
    f32x16 s = (f32x16)(0.f), dp = (f32x16)(0.f);
#pragma unroll
    for (int f = 0; f < RING; ++f) fetch(f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s = E::mfma32(E::vec(ring[i % RING]), E::vec(kf[i]), s);
      fetch(i + RING);
      if (i == N - 1) fetch_rows(s_lse[buf], 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    // dO V^T, and P beside it
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = N + 2 * i;
      dp = E::mfma32(E::vec(ring[f % RING]), E::vec(ring[(f + 1) % RING]), dp);
      fetch(f + RING);
      fetch(f + 1 + RING);
      fetch_rows(i + 1 < N ? s_lse[buf] : s_delta[buf], (i + 1) % N);
#pragma unroll
      for (int j = 0; j < EP; ++j) s[EP * i + j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[EP * i + j], c2, -aux[i % 2][j]));
      __builtin_amdgcn_sched_barrier(0);
    }
    bool seen[16];
    if constexpr (kMasked) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        seen[r] = key <= s_last[buf][8 * (r / 4) + 4 * half + r % 4];
        s[r] = seen[r] ? s[r] : 0.f;
      }
    }
    typename E::v8 p[2], ds[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) p[i] = pack8<E>(s, 8 * i);
    // dV, and dS beside it
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dv[i / 2] = E::mfma32(E::vec(ring[(3 * N + i) % RING]), p[i % 2], dv[i / 2]);
      fetch(3 * N + i + RING);
      if (i + 1 < N) fetch_rows(s_delta[buf], i + 1);
#pragma unroll
      for (int j = 0; j < EP; ++j) {
        const int r = EP * i + j;
        dp[r] = s[r] * ((dp[r] - aux[i % 2][j]) * ups);
        if constexpr (kMasked) dp[r] = seen[r] ? dp[r] : 0.f;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) ds[i] = pack8<E>(dp, 8 * i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dk[i / 2] = E::mfma32(E::vec(ring[(4 * N + i) % RING]), ds[i % 2], dk[i / 2]);
      fetch(4 * N + i + RING);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  s_bad.clear(-1);
  __syncthreads();
  // Rows that do not see all keys go through registers, the others straight into
  // LDS, where a workgroup's rows are at the same places in every tile (that is,
  // where the group divides the rows of a piece).
  const bool quick = 256 / CH % group == 0 && (group - 1) * max(a.q.head, a.dout.head) < (1 << 28);
  const int32_t rd = quick ? rf : r1;
  if (r0 < rd) {
    load(r0);
    store(r0, 0);
    load(r0 + 1);
    __syncthreads();
    for (int32_t rt = r0; rt < rd; ++rt) {
      const int buf = (rt - r0) & 1;
      if (rt + 1 < rd) {
        store(rt + 1, buf ^ 1);
        load(rt + 2);
      }
      tile(rt, buf, std::true_type{});
      __syncthreads();
    }
  }
  if (rd < r1) {
    const int32_t mytok = tid / CH / group, myhead = tid / CH % group, ltok = (lane & 31) / group, lhead = (lane & 31) % group;
    const uint32_t q_off = (uint32_t)(mytok * a.q.token + myhead * a.q.head + ch8) * 2;
    const uint32_t d_off = (uint32_t)(mytok * a.dout.token + myhead * a.dout.head + ch8) * 2;
    const uint32_t l_off = (uint32_t)(ltok * a.heads + lhead) * 4;
    const uint32_t lds0 = lds_offset(lds) + wave * 1024, rows0 = lds_offset(wave == 0 ? &s_lse[0][0] : &s_delta[0][0]);
    auto direct = [&](int32_t rt, int buf) {
      const int32_t tok0 = rt * BQ / group, left = rt < r1 ? nq - tok0 : 0;  // whole tokens: group divides BQ
      // (descriptors of the tile's size would check every offset, but cost fp16, whose
      // registers are all taken, 4 %: the bounds-checked build does)
      const int64_t q_tile = left > 0 ? q_at + tok0 * a.q.token : 0, d_tile = left > 0 ? d_at + tok0 * a.dout.token : 0;
      const LdsSource rq = lds_source(a.q.p + q_tile, 0x7fffffff), ro = lds_source(a.dout.p + d_tile, 0x7fffffff);
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int32_t on = u * (256 / CH) / group;
        const bool ok = mytok + on < left && ch8 < (uint32_t)a.d;
        const uint32_t qo = q_off + on * 2 * (uint32_t)a.q.token, go = d_off + on * 2 * (uint32_t)a.dout.token;
        load_to_lds16(rq, ok && in_bounds(q_tile + qo / 2, 8, a.q.n) ? qo : kOOB, lds0 + buf * 2 * BYTES + u * 4096);
        load_to_lds16(ro, ok && in_bounds(d_tile + go / 2, 8, a.dout.n) ? go : kOOB, lds0 + buf * 2 * BYTES + BYTES + u * 4096);
      }
      // rows past the last: zeros, and so P dO and dS Q are zero whatever P is (of a finite K)
      if (wave < 2) {
        const int64_t l_tile = left > 0 ? (q0 + tok0) * a.heads + head0 : 0;
        const LdsSource rl = lds_source((wave == 0 ? a.lse2 : a.delta) + l_tile, 0x7fffffff);
        const bool ok = lane < BQ && ltok < left && in_bounds(l_tile + l_off / 4, 1, a.tq * a.heads);
        load_to_lds4(rl, ok ? l_off : kOOB, rows0 + buf * 256);
      }
    };
    direct(rd, 0);
    tile_barrier();
    for (int32_t rt = rd; rt < r1; ++rt) {
      const int buf = (rt - rd) & 1;
      direct(rt + 1, buf ^ 1);
      tile(rt, buf, std::false_type{});
      tile_barrier();
    }
  }
  if (s_bad.any) {
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) dv[b][r] += s_bad.template seen<false>(32 * b + 8 * (r / 4) + 4 * half + r % 4, key);
  }
  const float fk = a.scale / up, fv = __builtin_amdgcn_exp2f(-kShift<E>);
  if (a.splits == 1) {
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      store_block<E>(a.dk, k_at, live, b, a.d, dk[b], fk, lane);
      store_block<E>(a.dv, v_at, live, b, a.d, dv[b], fv, lane);
    }
    return;
  }
  const int64_t pat = ((z * a.tk + tok) * a.kv_heads + kv_head) * 2 * a.d, n = a.splits * a.tk * a.kv_heads * 2 * a.d;
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 32 * b + 8 * i + 4 * half;
      if (!live || c >= a.d || !in_bounds(pat + c, 4, n) || !in_bounds(pat + a.d + c, 4, n)) continue;
      *reinterpret_cast<float4*>(a.part + pat + c) =
          make_float4(dk[b][4 * i] * fk, dk[b][4 * i + 1] * fk, dk[b][4 * i + 2] * fk, dk[b][4 * i + 3] * fk);
      *reinterpret_cast<float4*>(a.part + pat + a.d + c) =
          make_float4(dv[b][4 * i] * fv, dv[b][4 * i + 1] * fv, dv[b][4 * i + 2] * fv, dv[b][4 * i + 3] * fv);
    }
}

// The splits' sums together: a few keys' values of all key heads a workgroup.
// Bound by memory (8192 keys, 8 heads of 128, two splits: 28 us, 6 TB/s).
template <typename E>
__global__ __launch_bounds__(256) void k_attn_bwd_join(AttnArgs a) {
  const Region rg = find_region(a.cu_k, a.batch, a.tk, 1, kDeltaTokens, blockIdx.x);
  if (rg.tile < 0) return;
  const int32_t n = seq_length(a.len_k, rg.seq, a.batch, rg.size), first = rg.tile * kDeltaTokens;
  const int32_t keys = max(0, min(n - first, kDeltaTokens)), pieces = a.d / 8, width = a.kv_heads * 2 * pieces;
  const int64_t size = a.tk * a.kv_heads * 2 * a.d;
  for (int32_t i = threadIdx.x; i < keys * width; i += 256) {
    const int32_t c = i % pieces * 8, rest = i / pieces, which = rest & 1, head = rest / 2 % a.kv_heads;
    const int64_t tok = rg.start + first + rest / 2 / a.kv_heads;
    const int64_t at = ((tok * a.kv_heads + head) * 2 + which) * a.d + c;
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int z = 0; z < a.splits; ++z) {
      if (!in_bounds(z * size + at, 8, a.splits * size)) continue;
      const float4 x = *reinterpret_cast<const float4*>(a.part + z * size + at);
      const float4 y = *reinterpret_cast<const float4*>(a.part + z * size + at + 4);
      s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
      s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
    }
    const Heads& o = which ? a.dv : a.dk;
    const int64_t to = tok * o.token + head * o.head + c;
    if (in_bounds(to, 8, o.n))
      *reinterpret_cast<uint4*>(const_cast<uint16_t*>(o.p) + to) =
          make_uint4(E::pack2(s[0], s[1]), E::pack2(s[2], s[3]), E::pack2(s[4], s[5]), E::pack2(s[6], s[7]));
  }
}

}  // namespace

// Over how many workgroups the query heads of a key head are split: as few as
// make eight workgroups a compute unit, two of which it runs at a time (under a
// causal mask they differ in length, and the last ones leave units idle).  Forward
// and backward of 8192 tokens, 32 heads on 8: 2.52 ms with two, 2.36 with four, 2.32
// with eight, which takes 268 MB of workspace.
int attn_bwd_splits(int64_t tk, int64_t batch, int64_t heads, int64_t kv_heads, int compute_units) {
  if (heads <= 0 || kv_heads <= 0) return 1;
  const int64_t group = heads / kv_heads, units = kv_heads * std::max<int64_t>((tk + 127) / 128, batch);
  int64_t s = 1;
  while (s < group && (group % s != 0 || units * s < 8 * compute_units)) ++s;
  return (int)s;
}

size_t attn_bwd_part_bytes(int splits, int64_t tk, int64_t kv_heads, int64_t d) {
  return splits > 1 ? (size_t)splits * tk * kv_heads * 2 * d * 4 : 0;
}

hipError_t launch_attn_bwd(const AttnArgs& args, float* delta, float* lse2, float* top, float* part, int splits,
                           hipStream_t stream) {
  AttnArgs a = args;
  a.delta = delta;
  a.lse2 = lse2;
  a.top = top;
  a.part = part;
  a.splits = splits;
  const auto run = [&](auto e, auto db) {
    using E = decltype(e);
    constexpr int DB = decltype(db)::value;
    const int64_t dt = attn_tiles(a.tq, 1, a.batch, kDeltaTokens), vt = attn_tiles(a.tk, 1, a.batch, kDeltaTokens);
    const uint32_t few = a.tq > 0 && a.tk > 0 ? (uint32_t)(((int64_t)a.batch * a.heads + 3) / 4) : 0;
    // fp16: as many workgroups as partial maxima, the same for dO and V
    const int64_t n = a.f16 ? std::min<int64_t>(std::max(dt, vt), kAttnTops) : std::min<int64_t>(dt, 1 << 20);
    k_attn_delta<E, DB><<<dim3(few + (uint32_t)n, a.f16 ? 2 : 1), 256, 0, stream>>>(a, few, delta, lse2, top);
    if (a.tk > 0) {
      k_attn_bwd_kv<E, DB><<<(uint32_t)(attn_tiles(a.tk, 1, a.batch, 128) * a.kv_heads * a.splits), 256, 0, stream>>>(a);
      if (a.splits > 1)
        k_attn_bwd_join<E><<<(uint32_t)attn_tiles(a.tk, 1, a.batch, kDeltaTokens), 256, 0, stream>>>(a);
    }
    if (a.tq > 0)
      k_attn_bwd_q<E, DB><<<(uint32_t)(attn_tiles(a.tq, a.group, a.batch, 128) * a.kv_heads), 256, 0, stream>>>(a);
  };
  const auto typed = [&](auto e) {
    if (a.d <= 64) run(e, std::integral_constant<int, 2>{});
    else run(e, std::integral_constant<int, 4>{});
  };
  if (a.f16) typed(F16{});
  else typed(Bf16{});
  return hipGetLastError();
}

QLORA_OOB_READER(oob_count_attention_bwd)

}  // namespace qlora
