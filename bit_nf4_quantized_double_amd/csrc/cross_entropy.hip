// Softmax cross entropy under a frozen output head W [v, k]:
//
//   z = x W^T (fp32, never stored),  lse = log sum_v exp z_v,  loss = lse - z_t,
//   dx = g (softmax(z) - 1_t) W.
//
// One pass over W in pieces of the vocabulary, 4 m k v operations with the
// gradient: softmax(z) W is an average of W's rows, and an average can be
// summed online.  For a piece:
//   k_ce_logits  z by matrix cores; each tile of 128 entries keeps, for each
//                token, a whole number m >= max z log2 e and l = sum 2^(z log2 e - m)
//                and writes p = 2^(z log2 e - m) in 16 bits, in operand order
//   k_ce_stats   the running m of each token, by how much each tile's m is below
//                it (whole numbers), the running l
//   k_ce_grad    acc = acc 2^(old m - new m) + p W, where a tile's distance to
//                the running m is a subtraction from p's exponents: exact
// and at the end dx = g (acc / total - (rest / total) w_t).  The target's own term
// is left out of l and p and added in fp32: 1 - p_t of a token that is known well
// would otherwise lose its digits, and with it the loss and the gradient.
//
// p is rounded to 16 bits because it is a matrix operand (a relative 2^-9 or
// 2^-12 of each term, independent); in fp16 it is kept times 2^15, and what is
// 2^-29 below a token's largest becomes zero.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "decoder.h"
#include "rows_common.h"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kTileM = 256, kTileN = 128;   // of both products: tokens, outputs
constexpr int64_t kChunkM = 8192;           // tokens of one round of launches
constexpr int64_t kPieceBytes = (int64_t)512 << 20;
constexpr float kMost = 1e9f;               // bound of a tile's m: infinities stay outside

// What the kernels of one round of tokens share; all in the workspace.
struct CeRound {
  int64_t m, mp;       // tokens, rounded up to 64
  int64_t kp;          // k rounded up to 64
  int64_t piece;       // vocabulary of a piece, a multiple of 128
  int64_t v0, vn;      // this piece's first entry and how many
  int32_t splits;      // of a piece's entries in k_ce_grad
  uint16_t* xt;        // [mp / 16][kp / 32] tiles of 16 x 32 in operand order
  uint16_t* p;         // [mp / 16][piece / 32] tiles
  float *tile_m, *tile_l;  // [vtiles][mp]
  uint16_t* below;     // [vtiles][mp / 64][16][4]
  float *run_m, *run_l, *shift, *target, *c1, *c2;  // [mp]
  float* acc;          // [splits][token blocks][column blocks] tiles of 256 x 128
  int64_t n_xt, n_p, n_stat, n_below, n_acc;        // elements
};

template <typename E>
struct Half {
  static constexpr bool f16 = false;  // true: p is kept times 2^15
  static constexpr int mant = 7;
};
template <>
struct Half<F16> {
  static constexpr bool f16 = true;
  static constexpr int mant = 10;
};

// x in operand order, padded with zeros: 16 bytes a thread.
template <typename E>
__device__ __forceinline__ void pack(const CeArgs& a, const CeRound& r, int64_t i) {
  const int64_t chunks = r.kp / 32, tile = i >> 6;
  if (tile >= r.mp / 16 * chunks) return;
  const int lane = (int)(i & 63);
  const int64_t row = tile / chunks * 16 + (lane & 15), col = tile % chunks * 32 + 8 * (lane >> 4);
  const int64_t at = row * a.ldx + col, n = a.m > 0 ? (a.m - 1) * a.ldx + a.k : 0;
  Bytes16 u = {0, 0, 0, 0};
  if (row < r.m && col < a.k && in_bounds(at, 8, n)) __builtin_memcpy(&u, a.x + at, 16);
  if (in_bounds(i * 8, 8, r.n_xt)) *reinterpret_cast<uint4*>(r.xt + i * 8) = make_uint4(u.x, u.y, u.z, u.w);
}

// The target's logit of each token, a wave each: sums of k / 64 terms a lane.
// (Where a token is known well its loss is as far off, relative to itself, as
// this logit, and the matrix cores add up k / 32 times in a row.)
template <typename E>
__device__ __forceinline__ void target_logit(const CeArgs& a, const CeRound& r, int64_t m) {
  const int lane = threadIdx.x & 63;
  if (m >= r.m || !in_bounds(m, 1, r.m)) return;
  const int64_t y = a.targets[m];
  if (y == a.ignore || y < 0 || y >= a.v) return;
  float s[2] = {0.f, 0.f};
  for (int64_t c = 8 * lane; c < a.k; c += 512) {
    Bytes16 u = {0, 0, 0, 0};
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in_bounds(m * a.ldx + c, 8, (a.m - 1) * a.ldx + a.k)) __builtin_memcpy(&u, a.x + m * a.ldx + c, 16);
    if (in_bounds(y * a.ldw + c, 8, (a.v - 1) * a.ldw + a.k)) w = *reinterpret_cast<const uint4*>(a.w + y * a.ldw + c);
    const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[0] += E::widen((uint16_t)p[i]) * E::widen((uint16_t)q[i]);
      s[1] += E::widen((uint16_t)(p[i] >> 16)) * E::widen((uint16_t)(q[i] >> 16));
    }
  }
  float sum = s[0] + s[1];
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) sum += __shfl_xor(sum, i);
  if (lane == 0) r.target[m] = sum;
}

// All but the 24 latest of the wave's vector memory loads are there.
__device__ __forceinline__ void wait_loads_but_24() {
  __builtin_amdgcn_s_waitcnt(0x4f78);
  asm volatile("" ::: "memory");
}

// Both in one launch, the targets' workgroups first.
template <typename E>
__global__ __launch_bounds__(256) void k_ce_prepare(CeArgs a, CeRound r, int64_t targets) {
  const int64_t b = block_of(blockIdx.x, blockIdx.y);
  if (b < targets) target_logit<E>(a, r, b * 4 + (threadIdx.x >> 6));
  else pack<E>(a, r, (b - targets) * 256 + threadIdx.x);
}

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Workgroups are dealt round-robin to the 8 XCDs: each gets a contiguous run of
// an order that goes column by column inside bands of 4 token blocks, so that
// the tiles an XCD works on share token and output blocks in its L2.
__device__ __forceinline__ void tile_of(uint32_t lin, uint32_t mt, uint32_t nt, uint32_t& tm, uint32_t& tn) {
  constexpr uint32_t RB = 4;
  const uint32_t total = mt * nt, whole = total & ~7u;
  const uint32_t t = lin < whole ? (lin & 7u) * (whole >> 3) + (lin >> 3) : lin;
  const uint32_t band = t / (RB * nt), rows = min(RB, mt - band * RB), within = t - band * RB * nt;
  tn = within / rows;
  tm = band * RB + within % rows;
}

// p with its exponents lowered by b (halves of d; a value that falls out of
// range becomes zero).
template <typename E>
__device__ __forceinline__ uint32_t lower(uint32_t d, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
  const u16x2 x = __builtin_bit_cast(u16x2, d), y = __builtin_bit_cast(u16x2, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(x, y));
}

// Both products, bound by the matrix cores (8192 tokens, width 4096, 128256 entries:
// four pieces of 1.51 ms for the logits, 1.43 PFLOP/s with the cores 78 % busy, and of
// 1.73 ms for the gradient, 1.25 PFLOP/s, 63 % busy; a plain library product of such a
// piece runs at 1.40 to 1.52).  256 tokens x 128 outputs a workgroup, 4 waves of 64 tokens, in
// 16 x 16 x 32 MFMAs (A: outputs, B: tokens).  The tokens' operand is in tiles of
// 1 KB in lane order and goes straight into registers, three chunks of 32 ahead;
// W's goes straight into LDS, four buffers, three steps of 64 ahead, one barrier a step.
//   TRANS = false: outputs are rows of W, the reduction its columns
//   TRANS = true:  outputs are columns of W, the reduction its rows, read from
//                  LDS through the transposing load; a lane's 8 rows are 4 g .. + 3
//                  and 16 + 4 g .. + 3 of 32, the order in which k_ce_logits holds p
template <typename E, bool TRANS>
struct CeProduct {
  static constexpr int kTile = 128 * 64 * 2;  // bytes of a step's W tile
  static constexpr int kBuffers = 4;
  static constexpr int NS = 8, KC = 2;
  static constexpr int RING = 3;               // chunks of 32 of the tokens' operand
  static constexpr int kRow = TRANS ? 16 : 8;  // 16-byte chunks of a tile's row

  f32x4 acc[NS][4];

  // A tile's chunks are in LDS in the order of rows, permuted inside a row by
  // chunk ^ spread(row): the rows that a read touches at a time (16 of one column;
  // for a transposing one 4 of 32 bytes) fall into different banks.
  static __device__ __forceinline__ uint32_t spread(uint32_t r) {
    return TRANS ? (r & 3) << 2 | (r >> 2 & 1) << 1 : r >> 1 & 7;
  }

  // w: W's tile origin; wrows, wcols: what there is of it from there on.
  // x: the wave's first tile of tokens, whose rows of tiles are `xpitch` bytes
  // apart, xbytes long.  steps: [s0, s1).  below: TRANS, [vtile][16][4] of this wave's tokens,
  // `bpitch` elements apart (n_below 0: a wave without tokens).
  __device__ __forceinline__ void run(uint8_t* lds, const uint16_t* w, int64_t ldw, int64_t wrows, int64_t wcols,
                                      const uint16_t* x, uint32_t xpitch, int64_t xbytes, uint32_t s0, uint32_t s1,
                                      const uint16_t* below, uint32_t bpitch, int64_t n_below) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint4 xf[RING][4], wf[2][4];
    uint2 low[RING];
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds)) + wave * 1024;
    // this thread's chunks of a tile: tid + 256 u, rows 256 / kRow apart
    const uint32_t row0 = tid / kRow, col0 = (tid % kRow ^ spread(row0)) * 8;  // (rows 16 or 32 apart have the same spread)
    const uint32_t woff = (row0 * (uint32_t)ldw + col0) * 2;
    const uint32_t most = (uint32_t)min(wrows, (int64_t)128);
    // (from step s1 on nothing: a buffer without bytes)
    auto load_w = [&](uint32_t s, int buffer) {
      // the buffer moves with the step, so that offsets stay in 32 bits
      const int64_t left = TRANS ? wrows - (int64_t)s * 64 : most;
      const uint32_t rows = s < s1 ? (uint32_t)max(min(left, (int64_t)(TRANS ? 64 : 128)), (int64_t)0) : 0u;
      const LdsSource src = lds_source(TRANS ? w + (int64_t)s * 64 * ldw : w,
                                       (rows * (uint32_t)ldw - ((uint32_t)ldw - (uint32_t)wcols)) * (rows > 0 ? 2u : 0u));
      const uint32_t col = TRANS ? col0 : s * 64 + col0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t off = woff + u * (256 / kRow) * 2 * (uint32_t)ldw + (TRANS ? 0u : s * 128);
        load_to_lds16(src, col < wcols ? off : kOOB, lds0 + buffer * kTile + u * 4096);
      }
    };
    // chunk c (of 32, from this part's first on), into the ring's place j.  (Chunks
    // past the part's last are another's or zeros, and not used.)  Here, too, the
    // buffer moves, and a lane's offsets stay.
    const int32_t xb = (int32_t)min(xbytes, (int64_t)0x7fffffff), lb = (int32_t)max(n_below, (int64_t)0) * 2;
    auto load_x = [&](uint32_t c, int j) {
      c += s0 * KC;
      const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (int64_t)c * 512, (uint32_t)max(xb - (int32_t)(c * 1024), 0));
#pragma unroll
      for (int t = 0; t < 4; ++t) xf[j][t] = buf_load16(rx, t * xpitch + lane * 16u);
      if constexpr (TRANS) {
        const int32_t past = (int32_t)(c / 4 * bpitch);
        low[j] = buf_load8(make_rsrc(below + past, (uint32_t)max(lb - past * 2, 0)), (lane & 15) * 8);
      }
    };
    constexpr int P = NS / 4, Q = KC * P;  // sub-steps of a chunk of 32, and of a step
    // a lane's places in a tile: of its row's chunk (TRANS: of strip k)
    const int g = lane >> 4;
    uint32_t at[TRANS ? 8 : 2];
    if constexpr (TRANS) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t row = 4 * g + (lane >> 2 & 3);
        at[k] = row * 256 + ((2 * k + (lane >> 1 & 1)) ^ spread(row)) * 16 + 8 * (lane & 1);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) at[k] = (lane & 15) * 128 + ((4 * k + g) ^ spread(lane & 15)) * 16;
    }
    auto read_w = [&](const uint8_t* tile, int q, uint4 (&f)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int strip = 4 * (q % P) + i, chunk = q / P;
        if constexpr (!TRANS) {
          f[i] = *reinterpret_cast<const uint4*>(tile + strip * 2048 + at[chunk]);
        } else {
          uint2 h[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            typedef __attribute__((ext_vector_type(4))) short s16x4;
            const uint8_t* p = tile + at[strip] + (32 * chunk + 16 * e) * 256;
            h[e] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
          }
          f[i] = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[i][t] = (f32x4)(0.f);
#pragma unroll
    for (int j = 0; j < 3; ++j) load_w(s0 + j, j);
#pragma unroll
    for (int j = 0; j < RING; ++j) load_x(j, j);
    wait_loads();
    lds_barrier();
    read_w(lds, 0, wf[0]);
    // step s = s0 + 12 n + I: W tile s is in buffer I % 4.  The barrier in its last
    // sub-step ends the reads of that buffer and begins those of the next one.
    auto step = [&](uint32_t s, auto which) {
      constexpr int I = decltype(which)::value, B = I % kBuffers;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = (I * KC + q / P) % RING;
        if (q == Q - 1) {
          // W tile s + 1 is there: since then at least 4 chunks and 2 tiles were loaded, 4 loads each
          wait_loads_but_24();
          lds_barrier();
        }
        if (q < Q - 1) read_w(lds + B * kTile, q + 1, wf[(q + 1) & 1]);
        else read_w(lds + (B + 1) % kBuffers * kTile, 0, wf[0]);
        if constexpr (TRANS) {
          if (q % P == 0) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t l = t < 2 ? low[j].x : low[j].y, b = (t & 1 ? l >> 16 : l & 0xffffu) * 0x10001u;
              uint4& f = xf[j][t];
              f = make_uint4(lower<E>(f.x, b), lower<E>(f.y, b), lower<E>(f.z, b), lower<E>(f.w, b));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[4 * (q % P) + i][t] = E::mfma16(E::vec(wf[q & 1][i]), E::vec(xf[j][t]), acc[4 * (q % P) + i][t]);
        if (q % P == P - 1) load_x((s - s0) * KC + q / P + RING, j);
        if (q == P - 1) load_w(s + 3, (B + 3) % kBuffers);
        // each sub-step's loads stay ahead of its MFMAs
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // (Each step follows one other only, or the compiler has to take the loads that
    // are out for those of any order, and waits for all of them.)
    uint32_t s = s0;
    const auto steps = [&](auto... i) { return (... && (step(s, i), ++s < s1)); };
    if (s < s1)
      while (steps(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{},
                   std::integral_constant<int, 3>{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 5>{},
                   std::integral_constant<int, 6>{}, std::integral_constant<int, 7>{}, std::integral_constant<int, 8>{},
                   std::integral_constant<int, 9>{}, std::integral_constant<int, 10>{}, std::integral_constant<int, 11>{})) {
      }
    wait_loads();
  }
};

// The largest (sum) of the four lanes that share a token.
__device__ __forceinline__ float token_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float token_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

template <typename E, bool GRAD>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_ce_logits(CeArgs a, CeRound r) {
  typedef CeProduct<E, false> G;
  __shared__ __attribute__((aligned(16))) uint8_t lds[G::kBuffers * G::kTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c = lane & 15;
  uint32_t tm, tn;
  tile_of(blockIdx.x, (uint32_t)((r.m + kTileM - 1) / kTileM), (uint32_t)((r.vn + kTileN - 1) / kTileN), tm, tn);
  const int64_t m0 = (int64_t)tm * kTileM + 64 * wave, n0 = (int64_t)tn * kTileN;  // n0: in the piece
  const int64_t left = r.mp - m0;                                                  // tokens from here on, padded
  G p;
  const uint32_t pitch = (uint32_t)(r.kp / 32 * 1024);
  p.run(lds, a.w + (r.v0 + n0) * a.ldw, a.ldw, min(r.vn - n0, (int64_t)kTileN), a.k, r.xt + (left > 0 ? m0 * r.kp : 0), pitch,
        left > 0 ? left / 16 * pitch : 0, 0, (uint32_t)(r.kp / 64), nullptr, 0, 0);
  if (left <= 0) return;

  // lane 16 g + c: token 16 t + c, entries 16 i + 4 g + e
  const int have = (int)min(r.vn - n0, (int64_t)kTileN) - 4 * g;
  if (have < kTileN) {
#pragma unroll
    for (int i = 0; i < G::NS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (16 * i + e >= have)
#pragma unroll
          for (int t = 0; t < 4; ++t) p.acc[i][t][e] = -INFINITY;
  }
  // the target's own entry apart (k_ce_prepare has it)
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t m = m0 + 16 * t + c;
    const int64_t y = m < r.m && in_bounds(m, 1, r.m) ? a.targets[m] : -1;
    const int64_t rel = y == a.ignore ? -1 : y - r.v0 - n0 - 4 * g;
    const int at = rel >= 0 && rel < kTileN && rel < have ? (int)rel : -1;
    if (__ballot(at >= 0)) {
#pragma unroll
      for (int i = 0; i < G::NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at == 16 * i + e) p.acc[i][t][e] = -INFINITY;
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < G::NS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, p.acc[i][t][e]);
    top = fminf(fmaxf(ceilf(token_max(top) * kLog2e), -kMost), kMost);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < G::NS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(p.acc[i][t][e], kLog2e, -top));
        sum += x;
        p.acc[i][t][e] = x;
      }
    sum = token_sum(sum);
    const int64_t m = m0 + 16 * t + c, at = (n0 / kTileN) * r.mp + m;
    if (g == 0 && m < r.mp && in_bounds(at, 1, r.n_stat)) {
      r.tile_m[at] = top;
      r.tile_l[at] = sum;
    }
    if constexpr (GRAD) {
      constexpr float f = Half<E>::f16 ? 32768.f : 1.f;
      const int64_t chunks = r.piece / 32;
#pragma unroll
      for (int q = 0; q < G::NS / 2; ++q) {
        const f32x4 x = p.acc[2 * q][t] * f, y = p.acc[2 * q + 1][t] * f;
        const int64_t to = (((m0 / 16 + t) * chunks + n0 / 32 + q) * 64 + lane) * 8;
        if (m0 + 16 * t < r.mp && in_bounds(to, 8, r.n_p))
          *reinterpret_cast<uint4*>(r.p + to) =
              make_uint4(E::pack2(x[0], x[1]), E::pack2(x[2], x[3]), E::pack2(y[0], y[1]), E::pack2(y[2], y[3]));
      }
    }
  }
}

// 16 tokens a workgroup, 64 threads each: a piece's tiles into the running m and
// l; after the last piece the loss, the log-sum and the gradient's factors.  Bound by
// the latency of its loads, so that many are out at a time (16 tokens, 1002 tiles: 12 us
// for 49 with 16 threads a token; 8192 tokens, 251 tiles: 17 for 21).
constexpr int kStatParts = 64;
template <typename E, bool GRAD>
__global__ __launch_bounds__(16 * kStatParts) void k_ce_stats(CeArgs a, CeRound r, bool first, bool final) {
  const int part = threadIdx.x >> 4, lane16 = threadIdx.x & 15;
  const int64_t m = (int64_t)blockIdx.x * 16 + lane16;
  const int64_t tiles = (r.vn + kTileN - 1) / kTileN;
  __shared__ float s[kStatParts][17];
  const float old_m = first ? -kMost : r.run_m[m], old_l = first ? 0.f : r.run_l[m];
  float top = -kMost;
#pragma unroll 4
  for (int64_t t = part; t < tiles; t += kStatParts)
    if (in_bounds(t * r.mp + m, 1, r.n_stat)) top = fmaxf(top, r.tile_m[t * r.mp + m]);
  s[part][lane16] = top;
  __syncthreads();
  top = old_m;
#pragma unroll 16
  for (int i = 0; i < kStatParts; ++i) top = fmaxf(top, s[i][lane16]);
  __syncthreads();
  float l = 0.f;
#pragma unroll 4
  for (int64_t t = part; t < tiles; t += kStatParts) {
    if (!in_bounds(t * r.mp + m, 1, r.n_stat)) continue;
    const float d = top - r.tile_m[t * r.mp + m];  // a whole number
    l += r.tile_l[t * r.mp + m] * __builtin_amdgcn_exp2f(-d);
    if constexpr (GRAD) {
      constexpr int mant = Half<E>::mant, most = 0xffff >> mant;
      const int64_t at = (t * (r.mp / 64) + m / 64) * 64 + lane16 * 4 + (m / 16 & 3);
      if (in_bounds(at, 1, r.n_below)) r.below[at] = (uint16_t)((int)fminf(d, (float)most) << mant);
    }
  }
  s[part][lane16] = l;
  __syncthreads();
  if (part != 0) return;
  const float shift = __builtin_amdgcn_exp2f(old_m - top);
  l = old_l * shift;
#pragma unroll 16
  for (int i = 0; i < kStatParts; ++i) l += s[i][lane16];
  r.run_m[m] = top;
  r.run_l[m] = l;
  if constexpr (GRAD) r.shift[m] = shift;
  if (!final || m >= r.m) return;
  const int64_t y = in_bounds(m, 1, r.m) ? a.targets[m] : 0;
  const bool ignored = y == a.ignore, bad = !ignored && (y < 0 || y >= a.v);
  // the rest's l is relative to 2^top, the target's term to the larger of both
  const float z = ignored || bad ? -INFINITY : r.target[m];
  const float z2 = z * kLog2e;
  const float ref = fmaxf(l == 0.f ? -kMost : top, ceilf(fminf(fmaxf(z2, -kMost), kMost)));
  const float scale = __builtin_amdgcn_exp2f(top - ref);
  const float rest = l == 0.f ? 0.f : l * scale, mine = __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -ref));
  const float total = rest + mine;
  // ln 2 in two parts: ref is a whole number
  const float lse = __builtin_fmaf(ref, 0.693359375f, __builtin_fmaf(ref, -2.12194440e-4f, logf(total)));
  if (in_bounds(m, 1, r.m)) {
    a.lse[m] = lse;
    a.loss[m] = ignored ? 0.f : bad ? NAN : rest < mine && z < INFINITY ? log1pf(rest / mine) : lse - z;
  }
  if constexpr (GRAD) {
    r.c1[m] = scale / total * (Half<E>::f16 ? 1.f / 32768.f : 1.f);
    r.c2[m] = z == INFINITY ? NAN : rest / total;  // (an infinity less an infinity, as in the loss)
  }
}

template <typename E>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_ce_grad(CeArgs a, CeRound r, bool first) {
  typedef CeProduct<E, true> G;
  __shared__ __attribute__((aligned(16))) uint8_t lds[G::kBuffers * G::kTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t mt = (uint32_t)((r.m + kTileM - 1) / kTileM), nt = (uint32_t)((a.k + kTileN - 1) / kTileN), tiles = mt * nt;
  const uint32_t z = blockIdx.x / tiles;
  uint32_t tm, tn;
  tile_of(blockIdx.x % tiles, mt, nt, tm, tn);
  const int64_t m0 = (int64_t)tm * kTileM + 64 * wave, n0 = (int64_t)tn * kTileN, left = r.mp - m0;
  // this split's entries, in whole tiles of 128 (two steps)
  const uint32_t vt = (uint32_t)((r.vn + kTileN - 1) / kTileN), per = (vt + r.splits - 1) / r.splits;
  const uint32_t s0 = min(z * per, vt) * 2, s1 = min((z + 1) * per, vt) * 2;
  const uint32_t pitch = (uint32_t)(r.piece / 32 * 1024);
  G p;
  p.run(lds, a.w + r.v0 * a.ldw + n0, a.ldw, r.vn, min(a.k - n0, (int64_t)kTileN), r.p + (left > 0 ? m0 * r.piece : 0), pitch,
        left > 0 ? left / 16 * pitch : 0, s0, s1, r.below + (left > 0 ? m0 : 0), r.mp, left > 0 ? r.n_below - m0 : 0);
  if (left <= 0) return;
  float f[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t m = m0 + 16 * t + (lane & 15);
    f[t] = m < r.mp && in_bounds(m, 1, r.mp) ? r.shift[m] : 0.f;
  }
  const int64_t base = (((int64_t)z * tiles + (int64_t)tm * nt + tn) * 4 + wave) * 64 * 128;
#pragma unroll
  for (int i = 0; i < G::NS; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t at = base + ((i * 4 + t) * 64 + lane) * 4;
      if (!in_bounds(at, 4, r.n_acc)) continue;
      f32x4* to = reinterpret_cast<f32x4*>(r.acc + at);
      *to = first ? p.acc[i][t] : *to * f[t] + p.acc[i][t];
    }
}

// What a row of dx with dloss 1 is multiplied by to be stored, where it is only
// multiplied again later: a power of two that takes 1 - p of the target, in [2^-e, 2^-e+1),
// to [1/8, 1/4).  dx is 1 - p times the difference of an average of W's rows and one
// of them, so that it then has the size of W's entries: as far in range as they are.
// At most 2^64 (a row below 2^-67 is as good as zero).
__device__ __forceinline__ float unit_of(float rest) {
  const int e = 127 - (int)(__builtin_bit_cast(uint32_t, rest) >> 23);
  return rest >= 0x1p-67f && rest <= 1.f ? __builtin_bit_cast(float, (uint32_t)(127 - 3 + e) << 23) : rest < 0x1p-67f ? 0x1p64f : 1.f;
}

// dx from the sums: 16 tokens x 16 pieces of 8 columns a workgroup.
template <typename E>
__global__ __launch_bounds__(256) void k_ce_finish(CeArgs a, CeRound r) {
  const int c = threadIdx.x & 15;
  const uint32_t nt = (uint32_t)((a.k + kTileN - 1) / kTileN), mt = (uint32_t)((r.m + kTileM - 1) / kTileM);
  const uint32_t tn = blockIdx.x % nt;
  const int64_t strip = blockIdx.x / nt, m = strip * 16 + c, col = (int64_t)tn * kTileN + 8 * (threadIdx.x >> 4);
  if (m >= r.m || col >= a.k) return;
  const int64_t tile = strip / 16 * nt + tn;
  const int wave = strip / 4 & 3, t = strip & 3, i = threadIdx.x >> 5, g = (threadIdx.x >> 4 & 1) * 2;
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int z = 0; z < r.splits; ++z) {
    const int64_t at = ((((int64_t)z * mt * nt + tile) * 4 + wave) * 32 + i * 4 + t) * 256 + (g * 16 + c) * 4;
    if (!in_bounds(at, 68, r.n_acc)) continue;
    const f32x4 x = *reinterpret_cast<const f32x4*>(r.acc + at), y = *reinterpret_cast<const f32x4*>(r.acc + at + 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] += x[e];
      s[4 + e] += y[e];
    }
  }
  const int64_t y = in_bounds(m, 1, r.m) ? a.targets[m] : a.ignore;
  uint4 out = make_uint4(0, 0, 0, 0);
  float unit = 1.f;
  if (y != a.ignore) {
    const bool bad = y < 0 || y >= a.v;
    const float c1 = r.c1[m], c2 = r.c2[m];
    if (a.unit && !bad) unit = unit_of(c2);
    const float g1 = bad ? NAN : a.dloss ? a.dloss[m] : unit;
    const int64_t at = (bad ? 0 : y) * a.ldw + col;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in_bounds(at, 8, (a.v - 1) * a.ldw + a.k)) w = *reinterpret_cast<const uint4*>(a.w + at);
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = E::pack2(g1 * (s[2 * e] * c1 - c2 * E::widen((uint16_t)d[e])),
                      g1 * (s[2 * e + 1] * c1 - c2 * E::widen((uint16_t)(d[e] >> 16))));
    out = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (in_bounds(m * a.k + col, 8, a.m * a.k)) *reinterpret_cast<uint4*>(a.dx + m * a.k + col) = out;
  if (a.unit && col == 0 && in_bounds(m, 1, a.m)) a.unit[m] = unit;
}

// out = g x, row by row, 8 values a thread.
template <typename E>
__global__ __launch_bounds__(256) void k_scale_rows(const uint16_t* x, const float* g, int64_t m, int64_t k, uint16_t* out) {
  const int64_t i = block_of(blockIdx.x, blockIdx.y) * 256 + threadIdx.x, at = i * 8;
  if (at >= m * k || !in_bounds(at, 8, m * k)) return;
  const uint4 u = *reinterpret_cast<const uint4*>(x + at);
  const float f = g[at / k];
  const uint32_t d[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = E::pack2(f * E::widen((uint16_t)d[e]), f * E::widen((uint16_t)(d[e] >> 16)));
  *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
}

// The losses' sum or mean over the tokens that count, in 64 bits and a fixed
// order: one workgroup (8192 tokens: 4.5 us, most of it the launch).  out[0] the result,
// out[1] what each loss counts in it.
__global__ __launch_bounds__(1024) void k_loss_sum(const float* loss, const int64_t* targets, int64_t m, int64_t ignore, bool mean,
                                                   float* out) {
  __shared__ double s_sum[16];
  __shared__ int64_t s_n[16];
  double sum = 0.0;
  int64_t n = 0;
  for (int64_t i = threadIdx.x; i < m; i += 1024)
    if (targets[i] != ignore) {
      sum += (double)loss[i];
      ++n;
    }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    sum += __shfl_xor(sum, s);
    n += __shfl_xor(n, s);
  }
  if ((threadIdx.x & 63) == 0) {
    s_sum[threadIdx.x >> 6] = sum;
    s_n[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) {
    sum += s_sum[w];
    n += s_n[w];
  }
  out[0] = (float)(mean ? sum / (double)n : sum);
  out[1] = (float)(mean ? 1.0 / (double)n : 1.0);
}

struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) & ~(size_t)255;
    return at;
  }
};

// A round of m tokens: sizes, and pointers into ws.
CeRound ce_round(int64_t m, int64_t k, int64_t v, bool grad, int cus, char* ws, size_t* bytes) {
  CeRound r{};
  r.m = m;
  r.mp = (m + 63) / 64 * 64;
  r.kp = (k + 63) / 64 * 64;
  const int64_t vp = (v + kTileN - 1) / kTileN * kTileN;
  r.piece = grad ? std::min(vp, std::max<int64_t>(kPieceBytes / (2 * r.mp) / kTileN * kTileN, kTileN)) : vp;
  const int64_t pieces = (vp + r.piece - 1) / r.piece;
  r.piece = (vp / kTileN + pieces - 1) / pieces * kTileN;  // of even size
  const int64_t vtiles = r.piece / kTileN;
  const int64_t tiles = ((m + kTileM - 1) / kTileM) * ((k + kTileN - 1) / kTileN);
  // few tiles: the entries of a piece split, to about two workgroups a compute unit
  r.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(2 * cus / std::max<int64_t>(tiles, 1), std::min<int64_t>(vtiles / 4, 64)));
  r.n_xt = r.mp * r.kp;
  r.n_stat = vtiles * r.mp;
  if (grad) {
    r.n_p = r.mp * r.piece;
    r.n_below = vtiles * r.mp;
    r.n_acc = r.splits * tiles * kTileM * kTileN;
  }
  Layout l;
  const size_t xt = l.take(r.n_xt * 2), p = l.take(r.n_p * 2), tm = l.take(r.n_stat * 4), tl = l.take(r.n_stat * 4),
               be = l.take(r.n_below * 2), run = l.take(6 * r.mp * 4), acc = l.take(r.n_acc * 4);
  *bytes = l.bytes;
  r.xt = reinterpret_cast<uint16_t*>(ws + xt);
  r.p = reinterpret_cast<uint16_t*>(ws + p);
  r.tile_m = reinterpret_cast<float*>(ws + tm);
  r.tile_l = reinterpret_cast<float*>(ws + tl);
  r.below = reinterpret_cast<uint16_t*>(ws + be);
  r.run_m = reinterpret_cast<float*>(ws + run);
  r.run_l = r.run_m + r.mp;
  r.shift = r.run_l + r.mp;
  r.target = r.shift + r.mp;
  r.c1 = r.target + r.mp;
  r.c2 = r.c1 + r.mp;
  r.acc = reinterpret_cast<float*>(ws + acc);
  return r;
}

template <typename E, bool GRAD>
void run_round(const CeArgs& a, CeRound r, hipStream_t stream) {
  const int64_t targets = (r.m + 3) / 4;
  k_ce_prepare<E><<<grid_of(targets + (r.n_xt / 8 + 255) / 256), 256, 0, stream>>>(a, r, targets);
  for (int64_t v0 = 0; v0 < a.v; v0 += r.piece) {
    r.v0 = v0;
    r.vn = std::min(r.piece, a.v - v0);
    const int64_t mt = (r.m + kTileM - 1) / kTileM, vt = (r.vn + kTileN - 1) / kTileN;
    k_ce_logits<E, GRAD><<<(uint32_t)(mt * vt), 256, 0, stream>>>(a, r);
    k_ce_stats<E, GRAD><<<(uint32_t)(r.mp / 16), 16 * kStatParts, 0, stream>>>(a, r, v0 == 0, v0 + r.piece >= a.v);
    if constexpr (GRAD)
      k_ce_grad<E><<<(uint32_t)(mt * ((a.k + kTileN - 1) / kTileN) * r.splits), 256, 0, stream>>>(a, r, v0 == 0);
  }
  if constexpr (GRAD)
    k_ce_finish<E><<<(uint32_t)((r.m + 15) / 16 * ((a.k + kTileN - 1) / kTileN)), 256, 0, stream>>>(a, r);
}

}  // namespace

size_t ce_workspace_bytes(int64_t m, int64_t k, int64_t v, bool grad, int compute_units) {
  size_t most = 0;
  // a last, smaller round may split a piece further
  for (const int64_t n : {std::min(m, kChunkM), m % kChunkM}) {
    size_t b = 0;
    if (n > 0) ce_round(n, k, v, grad, compute_units, nullptr, &b);
    most = std::max(most, b);
  }
  return most;
}

hipError_t launch_ce(const CeArgs& args, void* ws, int compute_units, hipStream_t stream) {
  for (int64_t m0 = 0; m0 < args.m; m0 += kChunkM) {
    CeArgs a = args;
    a.m = std::min(kChunkM, args.m - m0);
    a.x += m0 * a.ldx;
    a.targets += m0;
    a.loss += m0;
    a.lse += m0;
    if (a.dloss) a.dloss += m0;
    if (a.dx) a.dx += m0 * a.k;
    if (a.unit) a.unit += m0;
    size_t bytes;
    const CeRound r = ce_round(a.m, a.k, a.v, a.dx != nullptr, compute_units, static_cast<char*>(ws), &bytes);
    if (a.dx) a.f16 ? run_round<F16, true>(a, r, stream) : run_round<Bf16, true>(a, r, stream);
    else a.f16 ? run_round<F16, false>(a, r, stream) : run_round<Bf16, false>(a, r, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_scale_rows(const uint16_t* x, const float* g, int64_t m, int64_t k, uint16_t* out, bool f16,
                             hipStream_t stream) {
  const dim3 grid = grid_of((m * k / 8 + 255) / 256);
  if (f16) k_scale_rows<F16><<<grid, 256, 0, stream>>>(x, g, m, k, out);
  else k_scale_rows<Bf16><<<grid, 256, 0, stream>>>(x, g, m, k, out);
  return hipGetLastError();
}

hipError_t launch_loss_sum(const float* loss, const int64_t* targets, int64_t m, int64_t ignore, bool mean, float* out,
                           hipStream_t stream) {
  k_loss_sum<<<1, 1024, 0, stream>>>(loss, targets, m, ignore, mean, out);
  return hipGetLastError();
}

QLORA_OOB_READER(oob_count_cross_entropy)

}  // namespace qlora
