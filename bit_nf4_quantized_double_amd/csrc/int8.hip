// Matrix product in 8-bit integers:
//
//   out[m][n] = E(sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n])
//
// x and w are int8 codes in operand tiles (int8_layout.h); the sum is exact
// in int32 on the matrix cores, the scales are applied in fp32, token first,
// and the result is rounded once to the 16-bit output type.  w is the A
// operand, x the B operand: a lane then holds consecutive outputs of a token.
#include <algorithm>
#include <type_traits>
#include <climits>

#include "common.h"
#include "int8_layout.h"
#include "rows_common.h"

namespace qlora {
namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

// 16 bytes at any element's address (the hardware takes any; rows of an odd
// number of elements start anywhere).
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4u;
typedef __attribute__((ext_vector_type(4), aligned(1))) uint32_t u32x4b;

__device__ __forceinline__ i32x4 as_i32x4(uint4 u) { return __builtin_bit_cast(i32x4, u); }

// Strips [first, total) of a tiled matrix as a buffer: what lies past its end
// (at most 2^31 bytes on) reads zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t strips_rsrc(const int8_t* p, int64_t first, int64_t total,
                                                              int64_t kp) {
  const int64_t bytes = max((int64_t)0, total - first) * 16 * kp;
  return make_rsrc(p + (first < total ? first : 0) * 16 * kp, (uint32_t)min(bytes, (int64_t)0x7fffffff));
}

// The scales and biases of W consecutive outputs n .. n + W - 1 (n a multiple
// of W; past a.n: zeros).
template <typename E, int W>
struct Outs {
  float s[W], b[W];
  __device__ __forceinline__ void load(const Int8GemmArgs& a, int64_t n) {
    if (n + W <= a.n && in_bounds(n, W, a.n)) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const float4 f = a.sw ? *reinterpret_cast<const float4*>(a.sw + n + i) : make_float4(1.f, 1.f, 1.f, 1.f);
        s[i] = f.x; s[i + 1] = f.y; s[i + 2] = f.z; s[i + 3] = f.w;
        const uint2 u = a.bias ? *reinterpret_cast<const uint2*>(a.bias + n + i) : make_uint2(0, 0);
        b[i] = E::widen((uint16_t)u.x);
        b[i + 1] = E::widen((uint16_t)(u.x >> 16));
        b[i + 2] = E::widen((uint16_t)u.y);
        b[i + 3] = E::widen((uint16_t)(u.y >> 16));
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const bool ok = n + i < a.n && in_bounds(n + i, 1, a.n);
        s[i] = ok ? (a.sw ? a.sw[n + i] : 1.f) : 0.f;
        b[i] = ok && a.bias ? E::widen(a.bias[n + i]) : 0.f;
      }
    }
  }
  // E(sum sx s + b), token scale first
  __device__ __forceinline__ uint32_t pair(int i, int lo, int hi, float sx) const {
    return E::pack2(__builtin_fmaf((float)lo * sx, s[i], b[i]), __builtin_fmaf((float)hi * sx, s[i + 1], b[i + 1]));
  }
  __device__ __forceinline__ uint4 eight(i32x4 lo, i32x4 hi, float sx) const {
    return make_uint4(pair(0, lo[0], lo[1], sx), pair(2, lo[2], lo[3], sx), pair(4, hi[0], hi[1], sx),
                      pair(6, hi[2], hi[3], sx));
  }
};

__device__ __forceinline__ float token_scale(const Int8GemmArgs& a, int64_t m) {
  return m < a.m && in_bounds(m, 1, a.m) ? a.sx[m] : 0.f;
}

// 8 consecutive outputs n .. n + 7 of token m, as far as they exist, packed.
// `stream`: not kept in the second-level cache.
__device__ __forceinline__ void store8(const Int8GemmArgs& a, int64_t m, int64_t n, uint4 u, bool stream = false) {
  if (m >= a.m || n >= a.n) return;
  const int64_t e = m * a.n + n, size = a.m * a.n;
  if (n + 8 <= a.n) {
    const u32x4u v = {u.x, u.y, u.z, u.w};
    if (in_bounds(e, 8, size)) {
      if (stream) __builtin_nontemporal_store(v, reinterpret_cast<u32x4u*>(a.out + e));
      else *reinterpret_cast<u32x4u*>(a.out + e) = v;
    }
  } else {
    const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < a.n && in_bounds(e + i, 1, size)) a.out[e + i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
  }
}

// The split sums of 8 consecutive outputs of token m (rows of `part` are
// padded to 8 outputs).
__device__ __forceinline__ int64_t part_at(const Int8GemmArgs& a, int64_t z, int64_t m, int64_t n) {
  return (z * a.m + m) * ((a.n + 7) & ~(int64_t)7) + n;
}
__device__ __forceinline__ void store_part8(const Int8GemmArgs& a, int64_t z, int64_t m, int64_t n, i32x4 lo, i32x4 hi) {
  const int64_t e = part_at(a, z, m, n);
  if (m < a.m && n < a.n && in_bounds(e, 8, part_at(a, a.ksplit, 0, 0))) {
    *reinterpret_cast<i32x4*>(a.part + e) = lo;
    *reinterpret_cast<i32x4*>(a.part + e + 4) = hi;
  }
}

// Hand-off of LDS between waves: this wave's own LDS operations are done,
// then the barrier.  Global loads stay in flight (a __syncthreads would wait
// for them).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// XCD-aware tile order: workgroups are dealt round-robin to the 8 XCDs, so
// each XCD gets a contiguous run of an order that goes column-major inside
// bands of 4 token blocks: the 64 tiles an XCD works on at a time share 4
// token blocks and 16 output blocks in its L2.  (Few tokens' kernel at 6240 x
// 295 x 7723: 37 us, 44 us in bands of 16, 70 us dealt out token block by token
// block.)
__device__ __forceinline__ void tile_of(uint32_t lin, uint32_t mt, uint32_t nt, uint32_t& tm, uint32_t& tn) {
  constexpr uint32_t RB = 4;
  const uint32_t total = mt * nt, whole = total & ~7u;
  const uint32_t t = lin < whole ? (lin & 7u) * (whole >> 3) + (lin >> 3) : lin;
  const uint32_t band = t / (RB * nt), rows = min(RB, mt - band * RB), within = t - band * RB * nt;
  tn = within / rows;
  tm = band * RB + within % rows;
}

// Many tokens.  Workgroup tile: 256 tokens x 128 outputs, 4 waves of 64 x 128
// (32 accumulators of 16 x 16, 128 registers), two workgroups a compute unit.
// A 128-deep step is 4 sub-steps of 16 MFMAs (16 x 16 x 64): 64 of its columns
// by 64 outputs.
//
// The step's W tile goes through LDS (global -> registers two steps ahead ->
// LDS, double buffered), where the four waves read it; each wave loads its own
// token rows, which no other wave needs, straight into registers, one step
// ahead.  The two workgroups of a compute unit move 96 KB a step through the
// cache and 160 KB through LDS (32 in, 128 out) in 2048 matrix-core cycles:
// neither is the bound by its rate.
//
// 8192 x 14336 x 4096 takes 384 us (2.5 PFLOP/s): 734 thousand cycles at 1.91
// GHz, the matrix cores busy 62 % of them.  The loop without any loads takes 237
// us at 2.18 GHz, so two things cost: waves that wait for an operand or for
// their turn to issue (about 100 us; half of all wave cycles), and the clock,
// which the power limit lowers under this load (about 45 us).  With 32 x 32 x 32
// MFMAs, whose accumulators move twice the registers for the same products, the
// loop without loads takes 307 us.  Tiles of 256 x 256 (8 waves, one
// workgroup a compute unit) take 402 us where these take 392: less traffic, but
// nothing runs beside their epilogue.  128 x 128: 448 us.  8 waves of 64 x 64
// where a tile has its compute unit to itself: 4 % less or more, by the shape.
//
// The barrier of a step stands before its last sub-step: by then the next W
// tile is written and every wave has this one's last operands in registers,
// so the MFMAs of the last sub-step run while the next step's operands come.
//
// ksplit > 1: workgroup z of a tile sums its own range of steps and stores
// the int32 sums to part[z]; k_int8_reduce adds them and finishes.
template <typename E>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_int8_gemm(Int8GemmArgs a) {
  constexpr int kThreads = 256, BM = 256, BN = 128;
  constexpr int KC = 2;                               // chunks of 64 columns in a step
  constexpr int NS = BN / 16;                         // weight strips
  constexpr int kTile = BN * 64 * KC;                 // bytes of a W tile
  constexpr int kStage = kTile / (16 * kThreads);     // 16-byte pieces of it per thread
  constexpr int kPitch = BN + 8;                      // output staging: 16-bit elements per token
  constexpr int kOut = 4 * 64 * kPitch * 2;           // bytes: 64 tokens x 128 outputs per wave
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kTile > kOut ? 2 * kTile : kOut];
  // uniform across the wave: buffer resources made from it stay scalar
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t mt = (uint32_t)((a.m + BM - 1) / BM), nt = (uint32_t)((a.n + BN - 1) / BN);
  const uint32_t tiles = mt * nt;
  const int z = blockIdx.x / tiles;
  uint32_t tm, tn;
  tile_of(blockIdx.x % tiles, mt, nt, tm, tn);
  const int64_t m0 = (int64_t)tm * BM + 64 * wave, n0 = (int64_t)tn * BN;
  const int64_t kp = int8_kp(a.k);
  const uint32_t strip = 16u * (uint32_t)kp;
  // this split's columns, in chunks of 64: [c0, c1)
  const uint32_t chunks = (uint32_t)(kp >> 6), per = (chunks + a.ksplit - 1) / a.ksplit;
  const uint32_t c0 = min(z * per, chunks), c1 = min(c0 + per, chunks), steps = (c1 - c0 + KC - 1) / KC;

  const __amdgpu_buffer_rsrc_t rw = strips_rsrc(a.w, n0 >> 4, int8_weight_strips(a.n), kp);
  const __amdgpu_buffer_rsrc_t rx = strips_rsrc(a.x, m0 >> 4, int8_row_strips(a.m), kp);
  const uint32_t at = (uint32_t)lane * 16u;

  uint4 st[2][kStage], xf[KC][4], wf[2][4];
  auto load_stage = [&](uint32_t s, int d) {
#pragma unroll
    for (int u = 0; u < kStage; ++u) {
      const uint32_t i = u * kThreads + tid, c = c0 + s * KC + i % (64 * KC) / 64;
      st[d][u] = buf_load16(rw, c < c1 ? i / (64 * KC) * strip + c * 1024u + i % 64 * 16u : kOOB);
    }
  };
  auto write_stage = [&](int buf, int d) {
#pragma unroll
    for (int u = 0; u < kStage; ++u)
      *reinterpret_cast<uint4*>(lds + buf * kTile + (u * kThreads + tid) * 16) = st[d][u];
  };
  auto load_x = [&](uint32_t s, int j) {
    const uint32_t c = c0 + s * KC + j;
#pragma unroll
    for (int t = 0; t < 4; ++t) xf[j][t] = buf_load16(rx, c < c1 ? at + t * strip + c * 1024u : kOOB);
  };
  // sub-step q: columns 64 (q / P) .., strips 4 (q % P) .. of the wave's
  constexpr int P = NS / 4, Q = KC * P;  // sub-steps for 64 columns, and in a step
  auto read_w = [&](int buf, int q, uint4 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = *reinterpret_cast<const uint4*>(lds + buf * kTile + at + ((4 * (q % P) + i) * KC + q / P) * 1024);
  };

  i32x4 acc[NS][4];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][t][v] = 0;

  load_stage(0, 0);
#pragma unroll
  for (int j = 0; j < KC; ++j) load_x(0, j);
  write_stage(0, 0);
  load_stage(1, 1);
  load_stage(2, 0);
  lds_barrier();
  read_w(0, 0, wf[0]);
  // step s, B = s % 2: W tile s is in LDS buffer B, s + 1 in st[B ^ 1], s + 2 on its way to st[B]
  auto step = [&](uint32_t s, auto parity) {
    constexpr int B = decltype(parity)::value;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (q == 0) {
        write_stage(B ^ 1, B ^ 1);
        load_stage(s + 3, B ^ 1);
      }
      if (q == Q - 1) lds_barrier();
      if (q < Q - 1) read_w(B, q + 1, wf[(q + 1) & 1]);
      else read_w(B ^ 1, 0, wf[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          acc[4 * (q % P) + i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(as_i32x4(wf[q & 1][i]), as_i32x4(xf[q / P][t]),
                                                                          acc[4 * (q % P) + i][t], 0, 0, 0);
      if (q % P == P - 1) load_x(s + 1, q / P);
      // the scheduler keeps each sub-step's loads ahead of its MFMAs only if
      // it cannot move them across (408 us for the 8192 x 14336 x 4096
      // product without this, 390 with it)
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (uint32_t s = 0; s < steps; s += 2) {
    step(s, std::integral_constant<int, 0>{});
    if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>{});
  }

  // lane 16 g + c: token 16 t + c, outputs 32 p + 8 g .. + 7 in strips 2 p and 2 p + 1
  const int g = lane >> 4, c = lane & 15;
  if (a.ksplit > 1) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int p = 0; p < NS / 2; ++p)
        store_part8(a, z, m0 + 16 * t + c, n0 + 32 * p + 8 * g, acc[2 * p][t], acc[2 * p + 1][t]);
    return;
  }
  // Through LDS, so that a token's outputs leave as whole lines: each wave in
  // its own region (no other wave touches it).
  lds_barrier();  // every wave has read its last operands
  uint16_t* so = reinterpret_cast<uint16_t*>(lds) + wave * 64 * kPitch;
  float sx[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) sx[t] = token_scale(a, m0 + 16 * t + c);
#pragma unroll
  for (int p = 0; p < NS / 2; ++p) {
    Outs<E, 8> os;
    os.load(a, n0 + 32 * p + 8 * g);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      *reinterpret_cast<uint4*>(so + (16 * t + c) * kPitch + 32 * p + 8 * g) = os.eight(acc[2 * p][t], acc[2 * p + 1][t], sx[t]);
  }
  constexpr int kAcross = 2 * NS;  // 16-byte pieces of a token's outputs
  // Whole lines are not kept in the second-level cache, which the operands need
  // (8192 x 14336 x 4096: 3 % less time); where rows start inside a line,
  // that cache has to put the parts together (3549 x 26474 x 224: 59 us, 94
  // without it).
  const bool stream = a.n % 64 == 0;
#pragma unroll
  for (int r = 0; r < kAcross; ++r) {
    const int row = (64 / kAcross) * r + lane / kAcross, col = lane % kAcross * 8;
    store8(a, m0 + row, n0 + col, *reinterpret_cast<const uint4*>(so + row * kPitch + col), stream);
  }
}

// Few tokens, or little of everything: 16 TT tokens against 32 outputs (a
// strip pair) a workgroup, whose 8 waves share out the reduction, 64 columns
// in turn.  A wave reads weight tiles and token tiles straight into the
// MFMA's registers, whole kilobytes at a time, four of its turns in flight, and
// the waves' sums meet in LDS.  Up to 64 tokens the weight is read once, and
// reading it is the bound: 28672 x 8192 for one token 40 us (5.9 TB/s, a copy's
// rate is 5.1), 8192 x 28672 for sixteen 42 us.  More tokens come in
// blocks of 64, up to 940 TOP/s from the cache: 150 x 1000 x 2500 takes 6.1 us,
// and 13 us as tiles with a split reduction.
//
// NP > 0 (TT = 1): x is not quantized yet, and is at most 8192 NP values.
// Every workgroup quantizes all of it into LDS, after its first weight tiles
// are on their way: the rows are a few kilobytes in the second-level cache, and
// a launch of its own for them costs more than the repetition (a call of 1 x
// 28672 x 8192: 41.6 us for 47.9, of 16 x 4096 x 2048: 8.3 for 12.5).
constexpr int kFusedValues = 32768;
constexpr int kFewWaves = 8;
constexpr int kFewAhead = 4;  // turns in flight
__host__ __device__ constexpr int64_t fused_pitch(int64_t k) { return int8_kp(k) + 16; }  // of a token's codes in LDS

template <int TT, int NP, typename E>
__global__ __launch_bounds__(64 * kFewWaves) void k_int8_few(Int8GemmArgs a, QuantSrc<E> src) {
  constexpr bool FUSED = NP > 0;
  constexpr int NW = kFewWaves, U = kFewAhead;
  __shared__ i32x4 s_sum[NW][2 * TT][64];
  __shared__ float s_scale[16];
  __shared__ uint32_t s_top[16];
  extern __shared__ __attribute__((aligned(16))) uint8_t s_codes[];  // FUSED: [m][fused_pitch]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t kp = int8_kp(a.k);
  const uint32_t groups = (uint32_t)((a.n + 31) / 32), blocks = (uint32_t)((a.m + 16 * TT - 1) / (16 * TT));
  const uint32_t lin = (uint32_t)block_of(blockIdx.x, blockIdx.y), z = lin / (blocks * groups);
  if (z >= (uint32_t)a.ksplit) return;
  uint32_t tb, group;
  tile_of(lin % (blocks * groups), blocks, groups, tb, group);
  const uint32_t strip = 16u * (uint32_t)kp;
  const uint32_t chunks = (uint32_t)(kp >> 6), per = (chunks + a.ksplit - 1) / a.ksplit;
  const uint32_t c0 = min(z * per, chunks), c1 = min(c0 + per, chunks);
  const __amdgpu_buffer_rsrc_t rw = strips_rsrc(a.w, 2 * (int64_t)group, int8_weight_strips(a.n), kp);
  const uint32_t at = lane * 16u;
  uint4 w[U][2];
  auto load_w = [&](uint32_t c) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) w[u][i] = buf_load16(rw, c + u * NW < c1 ? i * strip + (c + u * NW) * 1024u + at : kOOB);
  };
  if constexpr (FUSED) {
    load_w(c0 + wave);
    // the tokens' pieces of 16 columns, one after another: a thread has NP of
    // them, and 8 neighbouring threads' are always of one token
    const uint32_t across = (uint32_t)(kp >> 4);
    typename QuantSrc<E>::Raw raw[NP];
    auto value = [&](int i, float (&v)[16]) {
      const uint32_t id = i * 64 * NW + threadIdx.x, m = id / across;
      const int64_t c = (int64_t)(id % across) * 16;
      float none = 0.f;
      if (m < a.m && c < a.k) {
        src.value(raw[i], m, c, a.k, v, none);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
      }
    };
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t id = i * 64 * NW + threadIdx.x;
      // past the end of a row or of the tokens: its (their) last values, dropped below
      src.template load<true>(min((int64_t)(id / across), a.m - 1), min((int64_t)(id % across) * 16, a.k - 16), a.k, raw[i]);
    }
    if (threadIdx.x < 16) s_top[threadIdx.x] = 0;
    lds_barrier();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t id = i * 64 * NW + threadIdx.x, m = id / across;
      const int64_t c = (int64_t)(id % across) * 16;
      if (c < a.k && c + 16 > a.k) raw[i].shift((int)(c + 16 - a.k));
      float v[16];
      value(i, v);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) top = max(top, abs_bits(v[j]));
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
      // a maximum of whole numbers: the order does not matter
      if (lane % 8 == 0 && m < a.m) atomicMax(&s_top[m], top);
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t id = i * 64 * NW + threadIdx.x, m = id / across, p = id % across;
      // unpacked again: kept across the barrier the values would cost half the
      // workgroups that fit a compute unit
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(raw[i].x.d[j]));
      value(i, v);
      if (m < a.m) {
        const uint32_t top = s_top[m];
        const float amax = fmaxf(__builtin_bit_cast(float, top), kAmaxFloor);
        const bool finite = top < 0x7f800000u;
        const RowQuant q = row_quant(finite ? amax : 1.f);
        *reinterpret_cast<uint4*>(s_codes + m * fused_pitch(a.k) + p * 16) = finite ? codes16(q, v) : make_uint4(0, 0, 0, 0);
        if (p == 0) s_scale[m] = finite ? amax / 127.f : __builtin_nanf("");
      }
    }
    lds_barrier();
  }
  const __amdgpu_buffer_rsrc_t rx = strips_rsrc(FUSED ? a.w : a.x, (int64_t)tb * TT, FUSED ? 0 : int8_row_strips(a.m), kp);
  i32x4 acc[2][TT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][t][v] = 0;
  // token rows past m are not read
  uint32_t xat[TT];
  const int64_t m0 = (int64_t)tb * (16 * TT);
#pragma unroll
  for (int t = 0; t < TT; ++t) xat[t] = m0 + 16 * t + (lane & 15) < a.m ? t * strip + at : kOOB;
  for (uint32_t c = c0 + wave; c < c1; c += U * NW) {
    uint4 x[U][TT];
    if (!FUSED || c != c0 + wave) load_w(c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t cc = c + u * NW;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if constexpr (FUSED) {
          x[u][t] = make_uint4(0, 0, 0, 0);
          if ((lane & 15) < a.m && cc < c1)
            x[u][t] = *reinterpret_cast<const uint4*>(s_codes + (lane & 15) * fused_pitch(a.k) + cc * 64 + (lane >> 4) * 16);
        } else {
          x[u][t] = buf_load16(rx, cc < c1 && xat[t] != kOOB ? xat[t] + cc * 1024u : kOOB);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(as_i32x4(w[u][i]), as_i32x4(x[u][t]), acc[i][t], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) s_sum[wave][i * TT + t][lane] = acc[i][t];
  __syncthreads();
  for (int t = wave; t < TT; t += NW) {
    i32x4 lo = s_sum[0][t][lane], hi = s_sum[0][TT + t][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) {
      lo += s_sum[v][t][lane];
      hi += s_sum[v][TT + t][lane];
    }
    const int64_t m = m0 + 16 * t + (lane & 15), n = 32 * (int64_t)group + 8 * (lane >> 4);
    if (a.ksplit > 1) {
      store_part8(a, z, m, n, lo, hi);
    } else {
      Outs<E, 8> os;
      os.load(a, n);
      const float sx = !FUSED ? token_scale(a, m) : m < a.m ? s_scale[m & 15] : 0.f;
      store8(a, m, n, os.eight(lo, hi, sx));
    }
  }
}

// Adds the splits' int32 sums and finishes: 8 outputs a thread.
template <typename E>
__global__ __launch_bounds__(256) void k_int8_reduce(Int8GemmArgs a) {
  const int64_t per = (a.n + 7) / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= per * a.m) return;
  const int64_t m = id / per, n = id % per * 8;
  i32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
  for (int z = 0; z < a.ksplit; ++z) {
    const int64_t e = part_at(a, z, m, n);
    if (in_bounds(e, 8, part_at(a, a.ksplit, 0, 0))) {
      lo += *reinterpret_cast<const i32x4*>(a.part + e);
      hi += *reinterpret_cast<const i32x4*>(a.part + e + 4);
    }
  }
  Outs<E, 8> o;
  o.load(a, n);
  store8(a, m, n, o.eight(lo, hi, token_scale(a, m)));
}

// ---- layouts ----------------------------------------------------------------
// Row-major codes into weight tiles: one 16-byte piece a thread, rows past n
// and columns past k zero.
__global__ __launch_bounds__(256) void k_int8_pack(const int8_t* src, int64_t ld, int64_t n, int64_t k, int8_t* dst,
                                                   int64_t rows) {
  const int64_t kp = int8_kp(k);
  const int64_t row = block_of(blockIdx.x, blockIdx.z) * 16 + (threadIdx.x & 15),
                piece = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 4);
  if (row >= rows || piece * 16 >= kp) return;
  const int64_t c = piece * 16, e = row * ld + c, size = (n - 1) * ld + k;
  uint4 u = make_uint4(0, 0, 0, 0);
  if (row < n) {
    if (c + 16 <= k) {
      if (in_bounds(e, 16, size)) {
        const u32x4b b = *reinterpret_cast<const u32x4b*>(src + e);
        u = make_uint4(b.x, b.y, b.z, b.w);
      }
    } else {
      uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < k && in_bounds(e + i, 1, size)) d[i >> 2] |= (uint32_t)(uint8_t)src[e + i] << (8 * (i & 3));
      u = make_uint4(d[0], d[1], d[2], d[3]);
    }
  }
  const int64_t at = int8_piece(int8_weight_row(row), piece, kp);
  if (in_bounds(at, 16, rows * kp)) *reinterpret_cast<uint4*>(dst + at) = u;
}

// Tiles of w [n x k] into tiles of its transpose [k x n]: 64 x 64 codes a
// workgroup, turned in LDS.
__global__ __launch_bounds__(256) void k_int8_transpose(const int8_t* src, int64_t n, int64_t k, int8_t* dst) {
  __shared__ uint8_t s[64][68];
  const int64_t kp = int8_kp(k), np = int8_kp(n), rows = int8_weight_strips(n) * 16, trows = int8_weight_strips(k) * 16;
  const int64_t n0 = (int64_t)blockIdx.y * 64, k0 = (int64_t)blockIdx.x * 64;
  const int r = threadIdx.x & 63, g = threadIdx.x >> 6;
  uint4 u = make_uint4(0, 0, 0, 0);
  if (n0 + r < n && k0 + 16 * g < kp) {  // rows past n are padding: zero columns of the transpose
    const int64_t at = int8_piece(int8_weight_row(n0 + r), (k0 >> 4) + g, kp);
    if (in_bounds(at, 16, rows * kp)) u = *reinterpret_cast<const uint4*>(src + at);
  }
  uint32_t* o = reinterpret_cast<uint32_t*>(&s[r][16 * g]);
  o[0] = u.x;
  o[1] = u.y;
  o[2] = u.z;
  o[3] = u.w;
  __syncthreads();
  // row r of the transpose (column k0 + r of w), its columns n0 + 16 g ..
  if (k0 + r < trows && n0 + 16 * g < np) {
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i >> 2] |= (uint32_t)s[16 * g + i][r] << (8 * (i & 3));
    const int64_t at = int8_piece(int8_weight_row(k0 + r), (n0 >> 4) + g, np);
    if (in_bounds(at, 16, trows * np)) *reinterpret_cast<uint4*>(dst + at) = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// Tiles back to a row-major 16-bit matrix of the values they stand for; bound by
// memory (8192 x 4096: 20 to 22 us, 4.7 to 5.0 TB/s; 18 us on codes that were just
// written).
template <typename E>
__global__ __launch_bounds__(256) void k_int8_dequant(const int8_t* codes, const float* scale, int64_t m, int64_t k,
                                                      bool weight, uint16_t* out) {
  const int64_t kp = int8_kp(k), rows = (weight ? int8_weight_strips(m) : int8_row_strips(m)) * 16;
  // a strip's columns first: its 16 rows fill up together
  const uint32_t across = (uint32_t)((k + 255) / 256);
  const uint32_t lin = (uint32_t)block_of(blockIdx.x, blockIdx.y);
  const int64_t row = (int64_t)(lin / across) * 16 + (threadIdx.x & 15),
                piece = (int64_t)(lin % across) * 16 + (threadIdx.x >> 4);
  const int64_t c = piece * 16;
  if (row >= m || c >= k) return;
  const int64_t at = int8_piece(weight ? int8_weight_row(row) : row, piece, kp);
  if (!in_bounds(at, 16, rows * kp) || !in_bounds(row, 1, m)) return;
  const uint4 u = *reinterpret_cast<const uint4*>(codes + at);
  const float s = scale[row];
  const uint32_t d[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = d[i >> 1] >> (16 * (i & 1));
    o[i] = E::pack2((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s);
  }
  const int64_t e = row * k + c;
  if (c + 16 <= k) {
    if (in_bounds(e, 16, m * k)) {
      u32x4u* q = reinterpret_cast<u32x4u*>(out + e);
      q[0] = u32x4u{o[0], o[1], o[2], o[3]};
      q[1] = u32x4u{o[4], o[5], o[6], o[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < k && in_bounds(e + i, 1, m * k)) out[e + i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
}

}  // namespace

// Which kernel, and how many splits: the least by a model of their times, in
// microseconds on 256 compute units, fitted to sweeps over 40 to 8192 tokens,
// 64 to 28672 outputs and reductions of 224 to 28672 (it is within 20 % of
// nearly all and picks the fastest or one within 10 % of it).
//   few     a workgroup makes one turn of its loads for each 2048 columns, at
//           1.0, 1.2 or 2.0 us a turn for 16, 32 or 64 tokens; all of them
//           together run at no more than 1000 TOP/s (operands from the cache),
//           with 2.3 us for each further round of workgroups, and read the
//           weight at no more than 5.5 TB/s.
//           72 x 4096 x 4096: 8 us, as tiles 28 us (15 us with 4 splits).
//   tiles   256 x 128, two workgroups a compute unit: 1.72 us a step of 128
//           columns with two, 0.82 us with one.  8192 x 14336 x 4096: 384 us;
//           1024 x 11008 x 4096: 50 us, few tokens' kernel 90 us.
//   either  writes its output at no more than 3.5 TB/s.
//   split   a launch more (3 us), and the int32 sums written and read at
//           5 TB/s.  512 x 4096 x 11008 as tiles: 67, 45, 37 us in 1, 2, 4.
Int8Plan int8_plan(int64_t m, int64_t n, int64_t k, int cus) {
  Int8Plan best{};
  double least = 0;
  const double scale = 256.0 / cus, ops = 2e-6 * (double)n * (double)int8_kp(k), out = 2e-6 * (double)m * (double)n / 3.5;
  const int64_t steps = int8_kp(k) / 128;
  auto consider = [&](Int8Kind kind, int split, double us) {
    us = std::max(us, out);
    if (split > 1) us += 3.0 + 8e-6 * split * (double)m * (double)n / 5.0;
    if (best.ksplit == 0 || us < least) {
      best = Int8Plan{kind, split};
      least = us;
    }
  };
  const Int8Kind few = m <= 16 ? kInt8Few16 : m <= 32 ? kInt8Few32 : kInt8Few64;
  const int64_t rows = m <= 16 ? 16 : m <= 32 ? 32 : 64, blocks = (m + rows - 1) / rows;
  const double turn = m <= 16 ? 1.0 : m <= 32 ? 1.2 : 2.0;
  const int64_t groups = blocks * ((n + 31) / 32), tiles = (m + 255) / 256 * ((n + 127) / 128);
  const int64_t rounds = (groups + 2 * cus - 1) / (2 * cus);
  for (int split = 1; split <= 8; split *= 2) {
    if (split == 1 || groups * split <= cus) {
      const double turns = (double)((steps + 16 * split - 1) / (16 * split));
      const double bulk = scale * std::max(ops * (double)(blocks * rows) / 1000.0, (double)n * (double)k / 5.5e6) +
                          2.3 * (double)(rounds - 1);
      consider(few, split, 2.7 + std::max(turns * turn, bulk));
    }
    if (m > 64 && (split == 1 || tiles * split <= 2 * cus)) {
      const int64_t wgs = tiles * split, full = wgs / (2 * cus), rest = wgs % (2 * cus);
      const double step = 1.72 * (double)full + (rest > cus ? 1.6 : rest > 0 ? 0.82 : 0.0);
      consider(kInt8Tile, split, 5.0 + step * (double)((steps + split - 1) / split));
    }
  }
  return best;
}

size_t int8_plan_bytes(const Int8Plan& p, int64_t m, int64_t n) {
  return p.ksplit > 1 ? (size_t)p.ksplit * (size_t)m * (size_t)((n + 7) & ~(int64_t)7) * 4u : 0;
}

size_t int8_part_bytes(int64_t m, int64_t n, int64_t k, int cus) { return int8_plan_bytes(int8_plan(m, n, k, cus), m, n); }

// The quantizer inside the product costs each workgroup 2.9 us for 32768 values,
// and a launch of its own about as much: worth it while the workgroups, one for
// each 32 outputs, are few or the values are.  This form has no split, and needs
// none: one token, 1024 outputs and a reduction of 28672 take 12.9 us on the GPU,
// quantizer, product split 4 ways and their sum 13.3 (4.1 + 6.5 + 2.7), and a
// call 12.6 us for 19.9.
bool int8_fuses_rows(int64_t m, int64_t n, int64_t k) {
  return m <= 16 && k >= 16 && m * int8_kp(k) <= kFusedValues && (n + 31) / 32 * m * int8_kp(k) <= 256 * kFusedValues;
}

template <typename E>
static hipError_t run_plan(Int8GemmArgs a, const Int8Plan& p, const QuantArgs* rows, hipStream_t st) {
  a.ksplit = a.part ? p.ksplit : 1;
  const bool tile = p.kind == kInt8Tile;
  const int64_t bm = int8_tokens(p.kind), bn = tile ? 128 : 32;
  const int64_t tiles = (a.m + bm - 1) / bm * ((a.n + bn - 1) / bn);
  // tiles count in one dimension, of 2^32 threads: past that lie outputs of 0.5 TB
  if (tiles * a.ksplit > (tile ? (int64_t)INT_MAX / 128 : INT_MAX)) return hipErrorInvalidValue;
  const dim3 gr = tile ? dim3((uint32_t)(tiles * a.ksplit)) : grid_of(tiles * a.ksplit);
  QuantSrc<E> src{};
  if (rows) {
    src = QuantSrc<E>{mat<E>(rows->x, rows->ldx, rows->m, rows->k), rows->col_scale};
    const size_t lds = (size_t)(a.m * fused_pitch(a.k));
    static_assert(kFusedValues == 4 * 16 * 64 * kFewWaves, "values a workgroup quantizes");
    if (a.m * int8_kp(a.k) <= kFusedValues / 4) k_int8_few<1, 1, E><<<gr, 64 * kFewWaves, lds, st>>>(a, src);
    else k_int8_few<1, 4, E><<<gr, 64 * kFewWaves, lds, st>>>(a, src);
  } else {
    switch (p.kind) {
      case kInt8Few16: k_int8_few<1, 0, E><<<gr, 64 * kFewWaves, 0, st>>>(a, src); break;
      case kInt8Few32: k_int8_few<2, 0, E><<<gr, 64 * kFewWaves, 0, st>>>(a, src); break;
      case kInt8Few64: k_int8_few<4, 0, E><<<gr, 64 * kFewWaves, 0, st>>>(a, src); break;
      case kInt8Tile: k_int8_gemm<E><<<gr, 256, 0, st>>>(a); break;
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.ksplit == 1) return e;
  const int64_t blocks = ((a.n + 7) / 8 * a.m + 255) / 256;
  if (blocks >= (int64_t)1 << 24) return hipErrorInvalidValue;  // of 256 threads; plans split only small outputs
  k_int8_reduce<E><<<dim3((uint32_t)blocks), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_int8_plan(const Int8GemmArgs& a, const Int8Plan& p, hipStream_t st) {
  return a.f16 ? run_plan<F16>(a, p, nullptr, st) : run_plan<Bf16>(a, p, nullptr, st);
}

hipError_t launch_int8_gemm(const Int8GemmArgs& a, int cus, hipStream_t st) {
  return launch_int8_plan(a, int8_plan(a.m, a.n, a.k, cus), st);
}

hipError_t launch_int8_fused(const Int8GemmArgs& a, const QuantArgs& rows, hipStream_t st) {
  Int8Plan p{};
  p.kind = kInt8Few16;
  p.ksplit = 1;
  return a.f16 ? run_plan<F16>(a, p, &rows, st) : run_plan<Bf16>(a, p, &rows, st);
}

hipError_t launch_int8_pack(const int8_t* src, int64_t ld, int64_t n, int64_t k, int8_t* dst, hipStream_t st) {
  const int64_t rows = int8_weight_strips(n) * 16;
  const dim3 strips = grid_of(rows / 16), grid(strips.x, (uint32_t)((int8_kp(k) / 16 + 15) / 16), strips.y);
  k_int8_pack<<<grid, 256, 0, st>>>(src, ld, n, k, dst, rows);
  return hipGetLastError();
}

hipError_t launch_int8_transpose(const int8_t* src, int64_t n, int64_t k, int8_t* dst, hipStream_t st) {
  const dim3 grid((uint32_t)((int8_weight_strips(k) * 16 + 63) / 64), (uint32_t)((int8_kp(n) + 63) / 64));
  k_int8_transpose<<<grid, 256, 0, st>>>(src, n, k, dst);
  return hipGetLastError();
}

hipError_t launch_int8_dequant(const int8_t* codes, const float* scale, int64_t m, int64_t k, bool weight, bool f16,
                               uint16_t* out, hipStream_t st) {
  const int64_t blocks = (m + 15) / 16 * ((k + 255) / 256);
  if (blocks > INT_MAX) return hipErrorInvalidValue;
  const dim3 grid = grid_of(blocks);
  if (f16) k_int8_dequant<F16><<<grid, 256, 0, st>>>(codes, scale, m, k, weight, out);
  else k_int8_dequant<Bf16><<<grid, 256, 0, st>>>(codes, scale, m, k, weight, out);
  return hipGetLastError();
}

QLORA_OOB_READER(oob_count_int8)

}  // namespace qlora
