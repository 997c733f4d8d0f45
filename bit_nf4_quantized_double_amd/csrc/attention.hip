// Attention of packed sequences, forward: O = softmax(scale Q K^T) V over the
// keys that a row sees, and the log-sums lse = log sum exp(scale q k).
//
// One pass over the keys with a running reference m and sum l in base 2:
//   p = 2^(c s - m),  c = scale log2 e,  l = sum p,  O = (sum p V) / l.
// bf16: m starts at a row's maximum and moves (and O, l are rescaled) only once the
// maximum is more than 2^8 above: most tiles need no rescaling.  l is summed in fp32
// from the unrounded p; p is rounded to 16 bits because it is a matrix operand (a
// relative 2^-9 or 2^-12 of each term, independent of one another).
// fp16: small p would fall below the type's range and be missing from O but not
// from l.  m is set 2^12 below the maximum, where p is 2^12, and moves once that is
// 2^3 more: p stays at most 2^15, is a normal number from 2^-26 of the row's largest on,
// and nothing above 2^-37 of it is lost.
//
// Scores are computed transposed (keys x queries): a lane then holds scores of
// one query only, so maxima and sums need a single exchange between the
// wave's halves, and the accumulators' order is the operand order of the second
// product (O transposed = V^T P^T) with V read through the transposing LDS load.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "attention_common.h"

namespace qlora {
namespace {

template <typename E>
struct Reference {
  static constexpr float below = 0.f, room = 8.f;  // of the maximum; how far that may rise
};
template <>
struct Reference<F16> {
  static constexpr float below = 12.f, room = 3.f;
};

// One online-softmax step's state of a lane: reference, and the sum over the
// keys of its half of the wave.
struct Running {
  float m, l;
};

// Keys of a split at least: a workgroup with fewer spends its time on finding its
// rows and keys (16 sequences of 1 to 16384 keys, 64 heads on 8: 90 us with 16
// splits whatever the length, 82 with these; 77 since).
constexpr int kLeastKeys = 512;

// KW = 1: 128 rows a workgroup, 32 a wave; tiles of 64 keys, double buffered,
// shared by the waves.  Bound by the matrix cores, 57 % busy near 1.8 GHz, and the
// vector instructions between their products, issued in 60 % of the cycles, the
// products' own issue among them (8192 causal tokens, 32 heads of 128 on 8: 515 to 580
// us, 0.95 to 1.07 PFLOP/s).  Each operand read from LDS serves one product; 64 rows a
// wave would halve the reads (28 % of the cycles), but with 512 registers a lane the half
// that only the matrix instructions can use costs 5 moves a product (440 -> 585 us for
// four turns of a prompt, 64 heads on 8).
// KW = 4 (few rows, many keys): 32 rows a workgroup, whose waves take tiles of 32
// keys in turn, each through its own LDS.  Bound by reading the keys (16 sequences
// of 1 to 16384 keys, 64 heads on 8, 310 MB: 67 to 76 us, 4.1 to 4.6 TB/s; 6 us in
// k_attn_join) and by the longest sequence's workgroups.
template <typename E, int DB, int KW>
__global__ __launch_bounds__(256, 2) void k_attn_fwd(AttnArgs a) {
  constexpr int NU = KW == 1 ? 2 : 1, BN = 32 * NU, BM = KW == 1 ? 128 : 32;
  constexpr int TH = 256 / KW;                       // threads that share a tile
  constexpr int CH = Tile<DB>::kChunks, PER = BN * CH / TH, BYTES = BN * Tile<DB>::kPitch;
  constexpr int NBUF = KW == 1 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * BYTES * NBUF * KW];
  __shared__ NonFinite<32 * DB> s_bad;
  __shared__ float s_m[4][32], s_l[4][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, part_tid = KW == 1 ? tid : lane;
  uint8_t* const mine = lds + (KW == 1 ? 0 : wave * 2 * BYTES);

  // Heads first: workgroups go to the 8 XCDs in turn, so with 8 key heads (or a
  // multiple) an XCD keeps its heads' keys in its cache.  Late tiles first:
  // under a causal mask they are the long ones.
  uint32_t lin = blockIdx.x;
  const int32_t kv_head = lin % a.kv_heads;
  lin /= a.kv_heads;
  const int32_t z = lin % a.splits;
  const int64_t tiles = attn_tiles(a.tq, a.group, a.batch, BM), t = tiles - 1 - lin / a.splits;
  const Region rg = find_region(a.cu_q, a.batch, a.tq, a.group, BM, t);
  if (rg.tile < 0 || (int64_t)rg.tile * BM >= rg.size * a.group) return;
  const int32_t nq = seq_length(a.len_q, rg.seq, a.batch, rg.size);
  const Keys ks = keys_of(a, rg.seq);
  const int32_t rows = nq * a.group, first = rg.tile * BM;

  // this lane's row
  const int32_t row = first + (KW == 1 ? wave * 32 : 0) + (lane & 31);
  const bool live = row < rows, idle = !live && row < rg.size * a.group;
  const int32_t tok = row / a.group, head = kv_head * a.group + row % a.group;
  const int64_t o_at = (rg.start + tok) * a.o.token + head * a.o.head;
  const int64_t r_at = (rg.start + tok) * a.heads + head, r_n = a.tq * a.heads;
  if (a.zero_rest && idle && z == 0 && (KW == 1 || wave == 0)) {
    for (int c = 8 * half; c < a.d; c += 16)
      if (in_bounds(o_at + c, 8, a.o.n))
        *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.o.p) + o_at + c) = make_uint4(0, 0, 0, 0);
    if (half == 0 && in_bounds(r_at, 1, r_n)) a.lse[r_at] = -INFINITY;
  }
  if (first >= rows) return;

  // keys: row sees 0 .. last; the tile up to `end`, all its rows up to `whole`
  const int32_t shift = ks.n - nq;
  const int32_t last = !live ? -1 : a.causal ? min(ks.n - 1, tok + shift) : ks.n - 1;
  const int32_t wfirst = first + (KW == 1 ? wave * 32 : 0);
  const int32_t end = a.causal ? max(0, min(ks.n, (min(first + BM, rows) - 1) / a.group + shift + 1)) : ks.n;
  const int32_t whole = a.causal ? min(ks.n, first / a.group + shift + 1) : ks.n;
  const int32_t wend = a.causal ? min(ks.n, (min(wfirst + 32, rows) - 1) / a.group + shift + 1) : ks.n;
  const int32_t ntiles = (end + BN - 1) / BN, per = max((ntiles + a.splits - 1) / a.splits, kLeastKeys / BN);
  const int32_t k0 = z * per + (KW == 1 ? 0 : wave), k1 = min(ntiles, (z + 1) * per);

  typename E::v8 qf[2 * DB];
#pragma unroll
  for (int s = 0; s < 2 * DB; ++s) {
    const int c = 16 * s + 8 * half;
    qf[s] = E::vec(load16(a.q, (rg.start + tok) * a.q.token + head * a.q.head + c, live && c < a.d));
  }

  // a thread's pieces of a tile, through registers (columns past d: none)
  Tile<DB> at(lane);
  uint4 st[2][PER];
  const auto off = [&](const Heads& x, int u) {
    const uint32_t c = Fill<DB>::column(part_tid, TH, u);
    return c < (uint32_t)a.d ? ((Fill<DB>::row(part_tid) + u * (TH / CH)) * (uint32_t)x.token + c) * 2 : kOOB;
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
    uint8_t* const to = mine + buf * 2 * BYTES;
    const bool part = (kt + 1) * BN > whole;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int c = u * TH + part_tid;
      if (part && not_finite<E>(st[1][u]))
        s_bad.template take<E, true>(st[1][u], Fill<DB>::column(part_tid, TH, u), kt * BN + c / CH);
      *reinterpret_cast<uint4*>(to + c * 16) = st[0][u];
      *reinterpret_cast<uint4*>(to + BYTES + c * 16) = st[1][u];
    }
  };

  Running run{-INFINITY, 0.f};
  f32x16 o[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) o[b] = (f32x16)(0.f);
  const float c2 = a.scale * kLog2e;

  // the largest score of a lane's row so far in a tile -> the reference, and what
  // there is of the sums moved to it
  auto refer = [&](float top) {
    top = half_max(top) * c2 - Reference<E>::below;
    if (__ballot(top > run.m + Reference<E>::room)) {
      const float m = fmaxf(run.m, top);
      const float f = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(run.m - m);
      run.m = m;
      run.l *= f;
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] *= f;
    }
    return run.m == -INFINITY ? 0.f : run.m;
  };

  // a tile by itself.  MASKED: some of the rows do not see it in full
  auto tile = [&](int32_t kt, const uint8_t* kb, auto MASKED) {
    at.renew();
    const uint8_t* vb = kb + BYTES;
    f32x16 s[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      s[u] = (f32x16)(0.f);
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) s[u] = E::mfma32(E::vec(at.rows(kb, 32 * u, i)), qf[i], s[u]);
    }
    if (KW > 1) __builtin_amdgcn_sched_barrier(0);  // fewer operands on their way: nothing spills
    if constexpr (decltype(MASKED)::value) {
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (kt * BN + 32 * u + 8 * (r / 4) + 4 * half + r % 4 > last) s[u][r] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
    const float ref = refer(top);
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[u][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][r], c2, -ref));
        sum += s[u][r];
      }
    run.l += sum;
#pragma unroll
    for (int i = 0; i < 2 * NU; ++i) {
      const typename E::v8 p = pack8<E>(s[i / 2], 8 * (i % 2));
#pragma unroll
      for (int b = 0; b < DB; ++b) o[b] = E::mfma32(E::vec(at.cols(vb, 16 * i, b)), p, o[b]);
      if (KW > 1) __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Whole tiles, one in advance: the scores of the next tile are computed between
  // the exponentials of this one, and their maximum between the products with V.
  // Operands are read from LDS into a ring of registers, RING products ahead.
  // K's next tile is there in full when this one's turn comes, V's own.
  auto scores = [&](const uint8_t* kb, f32x16 (&s)[2]) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      s[u] = (f32x16)(0.f);
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) s[u] = E::mfma32(E::vec(at.rows(kb, 32 * u, i)), qf[i], s[u]);
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
    return top;
  };
  auto step = [&](const uint8_t* kb, const uint8_t* vb, f32x16 (&s)[2], f32x16 (&next)[2], float& top) {
    at.renew();
    constexpr int N = 4 * DB, RING = 4, EP = 32 / N;  // products of each kind, elements beside each
    uint4 ring[RING];
    auto fetch = [&](int f) {
      if (f < N) ring[f % RING] = at.rows(kb, 32 * (f / (2 * DB)), f % (2 * DB));
      else if (f < 2 * N) ring[f % RING] = at.cols(vb, 16 * (f % 4), (f - N) / 4);
    };
#pragma unroll
    for (int f = 0; f < RING; ++f) fetch(f);
    const float ref = refer(top);
    float sum = 0.f;
    typename E::v8 p[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) next[u] = (f32x16)(0.f);
#pragma unroll
    for (int f = 0; f < N; ++f) {
      next[f / (2 * DB)] = E::mfma32(E::vec(ring[f % RING]), qf[f % (2 * DB)], next[f / (2 * DB)]);
      fetch(f + RING);
#pragma unroll
      for (int e = EP * f; e < EP * f + EP; ++e) {
        s[e / 16][e % 16] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 16][e % 16], c2, -ref));
        sum += s[e / 16][e % 16];
      }
      if (EP * (f + 1) % 8 == 0) p[(EP * (f + 1) - 1) / 8] = pack8<E>(s[(EP * f) / 16], (EP * f) / 8 % 2 * 8);
      __builtin_amdgcn_sched_barrier(0);
    }
    run.l += sum;
    top = next[0][0];
#pragma unroll
    for (int f = 0; f < N; ++f) {
      o[f / 4] = E::mfma32(E::vec(ring[(N + f) % RING]), p[f % 4], o[f / 4]);
      fetch(N + f + RING);
#pragma unroll
      for (int e = EP * f; e < EP * f + EP; ++e) top = fmaxf(top, next[e / 16][e % 16]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  s_bad.clear(INT_MAX);
  __syncthreads();
  if constexpr (KW == 1) {
    const int32_t kf = max(k0, min(k1, whole / BN));  // the first tile that not all rows see in full
    if (k0 < kf) {
      // whole tiles: K's buffers first, then V's
      const uint32_t lds0 = lds_offset(lds) + wave * 1024;
      auto direct = [&](const Heads& x, int32_t kt, uint32_t to) {
        const LdsSource src = rows_source(x, first_key(x, kt), kt < kf ? BN : 0, a.d);
#pragma unroll
        for (int u = 0; u < PER; ++u) load_to_lds16(src, off(x, u), to + u * 4096);
      };
      direct(a.k, k0, lds0);
      direct(a.v, k0, lds0 + 2 * BYTES);
      direct(a.k, k0 + 1, lds0 + BYTES);
      tile_barrier();
      f32x16 s[2], next[2];
      float top = scores(lds, s);
      tile_barrier();
      for (int32_t kt = k0; kt < kf; kt += 2) {
        direct(a.k, kt + 2, lds0);
        direct(a.v, kt + 1, lds0 + 3 * BYTES);
        step(lds + BYTES, lds + 2 * BYTES, s, next, top);
        tile_barrier();
        if (kt + 1 >= kf) break;
        direct(a.k, kt + 3, lds0 + BYTES);
        direct(a.v, kt + 2, lds0 + 2 * BYTES);
        step(lds, lds + 3 * BYTES, next, s, top);
        tile_barrier();
      }
    }
    if (kf < k1) {
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
        if (kt * BN < wend) tile(kt, mine + buf * 2 * BYTES, std::true_type{});
        __syncthreads();
      }
    }
  } else {
    load(k0);
    for (int32_t kt = k0; kt < k1; kt += KW) {
      store(kt, 0);
      load(kt + KW);
      own_lds_order();
      if ((kt + 1) * BN <= whole) tile(kt, mine, std::false_type{});
      else tile(kt, mine, std::true_type{});
      own_lds_order();
    }
  }

  run.l = half_sum(run.l);
  float* part = a.part;
  auto finish = [&](int b, f32x16& acc, float m, float l) {
    const float f = l == 0.f ? 0.f : 1.f / l;
    if (s_bad.any) {
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] += s_bad.template seen<true>(32 * b + 8 * (r / 4) + 4 * half + r % 4, last);
    }
    if (a.splits == 1) {
      store_block<E>(a.o, o_at, live, b, a.d, acc, f, lane);
    } else if (l != 0.f) {
      const int64_t at = (z * r_n + r_at) * a.d, n = a.splits * r_n * a.d;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 32 * b + 8 * i + 4 * half;
        if (live && c < a.d && in_bounds(at + c, 4, n))
          *reinterpret_cast<float4*>(part + at + c) =
              make_float4(acc[4 * i] * f, acc[4 * i + 1] * f, acc[4 * i + 2] * f, acc[4 * i + 3] * f);
      }
    }
    if (b == 0 && half == 0 && live) {
      constexpr float below = Reference<E>::below, f = 1.f / (1 << (int)below);
      const float lse = l == 0.f ? -INFINITY : ((m + below) + __log2f(l * f)) * kLn2;
      if (a.splits == 1) {
        if (in_bounds(r_at, 1, r_n)) a.lse[r_at] = lse;
      } else {
        const int64_t at = a.splits * r_n * a.d + z * r_n + r_at;
        if (in_bounds(at, 1, a.splits * r_n * (a.d + 1))) part[at] = lse;
      }
    }
  };
  if constexpr (KW == 1) {
#pragma unroll
    for (int b = 0; b < DB; ++b) finish(b, o[b], run.m, run.l);
  } else {
    // the waves' keys together: block b of the rows' values by wave b
    float* so = reinterpret_cast<float*>(lds);
    static_assert(sizeof(lds) >= (size_t)KW * DB * 16 * 64 * 4 || KW == 1, "sums of all waves");
    if (half == 0) {
      s_m[wave][lane] = run.m;
      s_l[wave][lane] = run.l;
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) so[((wave * DB + b) * 16 + r) * 64 + lane] = o[b][r];
    __syncthreads();
    if (wave >= DB) return;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) m = fmaxf(m, s_m[w][lane & 31]);
    f32x16 acc = (f32x16)(0.f);
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][lane & 31] - (m == -INFINITY ? 0.f : m));
      l += f * s_l[w][lane & 31];
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] += f * so[((w * DB + wave) * 16 + r) * 64 + lane];
    }
    finish(wave, acc, m, l);
  }
}

// The splits of a row together: weights exp(lse_z - lse).  8 values a thread.
template <typename E>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  const int64_t token = blockIdx.x;
  const int lane = threadIdx.x & 63;
  int32_t n = 0;  // sequences that start at the token or before
  for (int32_t i0 = 0; i0 < a.batch + 1; i0 += 64)
    n += __popcll(__ballot(i0 + lane < a.batch + 1 && region_start(a.cu_q, a.batch, a.tq, i0 + lane + 1) <= token));
  n = __builtin_amdgcn_readfirstlane(n);
  if (n < 1 || n > a.batch) return;
  const int64_t start = region_start(a.cu_q, a.batch, a.tq, n);
  const int64_t size = clampl(region_start(a.cu_q, a.batch, a.tq, n + 1), start, a.tq) - start;
  if (token - start >= seq_length(a.len_q, n - 1, a.batch, size)) return;
  const int64_t r_n = a.tq * a.heads;
  const float* sums = a.part + a.splits * r_n * a.d;
  const int pieces = a.d / 8, i = blockIdx.y * 256 + threadIdx.x;
  if (i >= a.heads * pieces) return;
  const int head = i / pieces, c = i % pieces * 8;
  const int64_t r = token * a.heads + head;
  float top = -INFINITY;
#pragma unroll 8
  for (int z = 0; z < a.splits; ++z)
    if (in_bounds(z * r_n + r, 1, a.splits * r_n)) top = fmaxf(top, sums[z * r_n + r]);
  const float ref = top == -INFINITY ? 0.f : top;
  float l = 0.f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int z = 0; z < a.splits; ++z) {
    const float s = in_bounds(z * r_n + r, 1, a.splits * r_n) ? sums[z * r_n + r] : -INFINITY;
    const int64_t at = (z * r_n + r) * a.d + c;
    // a split that sees no key has not written its part
    if (s == -INFINITY || !in_bounds(at, 8, a.splits * r_n * a.d)) continue;
    const float w = __builtin_amdgcn_exp2f((s - ref) * kLog2e);
    l += w;
    const float4 x = *reinterpret_cast<const float4*>(a.part + at), y = *reinterpret_cast<const float4*>(a.part + at + 4);
    acc[0] += w * x.x; acc[1] += w * x.y; acc[2] += w * x.z; acc[3] += w * x.w;
    acc[4] += w * y.x; acc[5] += w * y.y; acc[6] += w * y.z; acc[7] += w * y.w;
  }
  const float f = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = token * a.o.token + head * a.o.head + c;
  if (in_bounds(at, 8, a.o.n))
    *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.o.p) + at) =
        make_uint4(E::pack2(acc[0] * f, acc[1] * f), E::pack2(acc[2] * f, acc[3] * f), E::pack2(acc[4] * f, acc[5] * f),
                   E::pack2(acc[6] * f, acc[7] * f));
  if (c == 0 && in_bounds(r, 1, r_n)) a.lse[r] = l == 0.f ? -INFINITY : ref + __log2f(l) * kLn2;
}

}  // namespace

AttnPlan attn_plan(int64_t tq, int64_t tk, int64_t batch, int64_t heads, int64_t kv_heads, int compute_units) {
  AttnPlan p{128, 1};
  if (tq <= 0 || batch <= 0 || kv_heads <= 0) return p;
  const int64_t rows = tq * (heads / kv_heads);
  if (rows <= 64 * batch) p.rows = 32;
  const int64_t work = kv_heads * std::max<int64_t>((rows + p.rows - 1) / p.rows, batch);
  // Two workgroups a compute unit at a time, two turns of them for the short ones
  // (two and eight turns: 82 and 90 us for 82 in the case above, 114 and 135 for 118
  // with four sequences of 8000 keys, 32 heads).
  const int64_t want = (p.rows == 32 ? 4 : 2) * (int64_t)compute_units;
  const int64_t most = (tk / batch + kLeastKeys - 1) / kLeastKeys;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({want / work, most, 64}));
  return p;
}

size_t attn_part_bytes(const AttnPlan& p, int64_t tq, int64_t heads, int64_t d) {
  return p.splits > 1 ? (size_t)p.splits * tq * heads * (d + 1) * 4 : 0;
}

hipError_t launch_attn_fwd(const AttnArgs& args, const AttnPlan& p, hipStream_t stream) {
  AttnArgs a = args;
  a.splits = p.splits;
  const int64_t blocks = attn_tiles(a.tq, a.group, a.batch, p.rows) * a.kv_heads * a.splits;
  const auto run = [&](auto e, auto db) {
    using E = decltype(e);
    constexpr int DB = decltype(db)::value;
    if (p.rows == 32) k_attn_fwd<E, DB, 4><<<(uint32_t)blocks, 256, 0, stream>>>(a);
    else k_attn_fwd<E, DB, 1><<<(uint32_t)blocks, 256, 0, stream>>>(a);
    if (a.splits > 1) k_attn_join<E><<<dim3((uint32_t)a.tq, (uint32_t)((a.heads * a.d / 8 + 255) / 256)), 256, 0, stream>>>(a);
  };
  const auto typed = [&](auto e) {
    if (a.d <= 64) run(e, std::integral_constant<int, 2>{});
    else run(e, std::integral_constant<int, 4>{});
  };
  if (a.f16) typed(F16{});
  else typed(Bf16{});
  return hipGetLastError();
}

QLORA_OOB_READER(oob_count_attention)

}  // namespace qlora
