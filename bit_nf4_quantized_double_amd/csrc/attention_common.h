// Shared by the attention kernels: which sequence a workgroup's rows belong
// to, operand tiles in LDS, and matrix-core fragments of them.
//
// Rows.  The queries of a key head's `group` heads are packed: row r of a
// sequence is token r / group, head r % group of the group.  They share their
// keys, so a tile of rows needs one pass over the keys whatever the group is.
//
// Tiles.  Lengths are on the device only, so the host cannot list the tiles.
// Sequences s_0 <= s_1 <= ... take tile numbers from floor(s_i group / rows) + i
// on: no two overlap, since ceil(n / b) <= floor((s + n) / b) - floor(s / b) + 1,
// and about one number a sequence has nothing to do.  The tokens before the
// first sequence and behind the last count as a sequence each (0 and batch + 1),
// whose rows are zeroed or left alone.
#pragma once

#include "common.h"
#include "decoder.h"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

__device__ __forceinline__ int64_t clampl(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// Numbers of tiles of `rows` rows that the launch needs.
__host__ __device__ inline int64_t attn_tiles(int64_t tokens, int64_t group, int64_t batch, int64_t rows) {
  return tokens * group / rows + batch + 2;
}

// Start of region i (0: before the first sequence, batch + 1: behind the last).
__device__ __forceinline__ int64_t region_start(const int32_t* cu, int32_t batch, int64_t tokens, int32_t i) {
  if (i <= 0 || !in_bounds(i - 1, 1, batch + 1)) return 0;
  return clampl(cu[i - 1], 0, tokens);
}

struct Region {
  int64_t start, size;  // tokens
  int32_t tile;         // of the region; < 0: none
  int32_t seq;          // -1: no sequence's
};

// The region of tile number t.  All lanes of the wave take part and get the same.
__device__ __forceinline__ Region find_region(const int32_t* cu, int32_t batch, int64_t tokens, int32_t group, int32_t rows,
                                              int64_t t) {
  const int lane = threadIdx.x & 63;
  int32_t n = 0;  // regions that start at tile t or before
  for (int32_t i0 = 0; i0 < batch + 2; i0 += 64) {
    const int32_t i = i0 + lane;
    const bool yes = i < batch + 2 && region_start(cu, batch, tokens, i) * group / rows + i <= t;
    n += __popcll(__ballot(yes));
  }
  const int32_t i = __builtin_amdgcn_readfirstlane(n - 1);
  Region r;
  r.start = region_start(cu, batch, tokens, i);
  r.size = (i > batch ? tokens : clampl(region_start(cu, batch, tokens, i + 1), r.start, tokens)) - r.start;
  r.tile = (int32_t)(t - (r.start * group / rows + i));
  r.seq = i >= 1 && i <= batch ? i - 1 : -1;
  return r;
}

// Tokens of a sequence: its region, or fewer where lengths are given.
__device__ __forceinline__ int32_t seq_length(const int32_t* len, int32_t seq, int32_t batch, int64_t size) {
  if (seq < 0) return 0;
  if (!len) return (int32_t)size;
  return in_bounds(seq, 1, batch) ? (int32_t)clampl(len[seq], 0, size) : 0;
}

// Keys of a sequence: [start, start + n).
struct Keys {
  int64_t start;
  int32_t n;
};
__device__ __forceinline__ Keys keys_of(const AttnArgs& a, int32_t seq) {
  if (seq < 0) return Keys{0, 0};
  const int64_t s = region_start(a.cu_k, a.batch, a.tk, seq + 1);
  const int64_t e = clampl(region_start(a.cu_k, a.batch, a.tk, seq + 2), s, a.tk);
  return Keys{s, seq_length(a.len_k, seq, a.batch, e - s)};
}

// A tile in LDS: rows of DB * 32 16-bit values (chunks of 16 bytes past d are
// zeros) one after another, as loads straight into LDS leave them; the chunks of a
// row are permuted by chunk ^ spread(row), so that the 16 rows that a wave's b128
// reads of one column touch at a time, and the 4 rows by 64 bytes of its
// transposing reads, fall into different banks (64 of 4 bytes).
template <int DB>
struct Tile {
  static constexpr int kPitch = DB * 64;  // bytes of a row
  static constexpr int kChunks = DB * 4;  // 16-byte chunks of a row
  static __device__ __forceinline__ uint32_t spread(uint32_t r) {
    return (DB == 4 ? (r & 3) << 2 : (r >> 1 & 1) << 2) | (r >> 2 & 3);
  }

  // A lane's places in a tile.  The permutation is an exclusive or, and so is the
  // way from a column to the next: an address is (place ^ constant) + base, one
  // instruction.
  uint32_t row, col;
  __device__ __forceinline__ explicit Tile(int lane) {
    const uint32_t r = lane & 31, t = 4 * (lane >> 5) + ((lane & 15) >> 2);
    row = r * kPitch + ((lane >> 5) ^ spread(r)) * 16;
    col = t * kPitch + ((2 * (lane >> 4 & 1) + ((lane & 3) >> 1)) ^ spread(t)) * 16 + 8 * (lane & 1);
  }
  // To the compiler these change here: it would make all addresses ahead of a
  // loop and keep them in registers that there are not.
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(row), "+v"(col)); }

  // MFMA operand (32 x 16): row r0 + lane % 32, columns 16 step + 8 (lane / 32) .. + 7.  r0 a multiple of 32.
  __device__ __forceinline__ uint4 rows(const uint8_t* tile, int r0, int step) const {
    return *reinterpret_cast<const uint4*>(tile + (row ^ (uint32_t)step << 5) + r0 * kPitch);
  }
  // The transposed operand (32 x 16): column 32 block + lane % 32 of rows r0 ..
  // r0 + 15, in the order in which the accumulators of a 32 x 32 product hold
  // their rows: element e of lane half h is row r0 + 8 (e / 4) + 4 h + e % 4.
  // (ds_read_b64_tr_b16: 16 lanes give the addresses of 4 rows of 16 values, 4 a
  // lane, and each gets one column of them.)  r0 a multiple of 16.
  __device__ __forceinline__ uint4 cols(const uint8_t* tile, int r0, int block) const {
    typedef __attribute__((ext_vector_type(4))) short s16x4;
    uint2 u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      u[i] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(tile + (col ^ (uint32_t)(block << 6 | i << 5)) + (r0 + 8 * i) * kPitch)));
    return make_uint4(u[0].x, u[0].y, u[1].x, u[1].y);
  }
};

// How `threads` threads fill a tile: piece u of thread t is the 16 bytes t + u
// threads of it, of row t / chunks + u step, whose source is this column.
template <int DB>
struct Fill {
  static __device__ __forceinline__ uint32_t row(uint32_t t) { return t / Tile<DB>::kChunks; }
  static __device__ __forceinline__ uint32_t column(uint32_t t, uint32_t threads, uint32_t u) {
    return (t % Tile<DB>::kChunks ^ Tile<DB>::spread(row(t) + u * (threads / Tile<DB>::kChunks))) * 8;
  }
};

// Halves of d that are infinite or NaN: their top bits.
template <typename E>
__device__ __forceinline__ uint32_t not_finite(uint32_t d);
template <>
__device__ __forceinline__ uint32_t not_finite<Bf16>(uint32_t d) {
  return ~((~d & 0x7f807f80u) + 0x7fff7fffu) & 0x80008000u;
}
template <>
__device__ __forceinline__ uint32_t not_finite<F16>(uint32_t d) {
  return ~((~d & 0x7c007c00u) + 0x7fff7fffu) & 0x80008000u;
}
template <typename E>
__device__ __forceinline__ uint32_t not_finite(const uint4& u) {
  return not_finite<E>(u.x) | not_finite<E>(u.y) | not_finite<E>(u.z) | not_finite<E>(u.w);
}
// d with such halves zeroed
template <typename E>
__device__ __forceinline__ uint32_t finite_part(uint32_t d) {
  return d & ~((not_finite<E>(d) >> 15) * 0xffffu);
}
template <typename E>
__device__ __forceinline__ uint4 finite_part(const uint4& u) {
  return make_uint4(finite_part<E>(u.x), finite_part<E>(u.y), finite_part<E>(u.z), finite_part<E>(u.w));
}
// Infinities and NaNs in masked places.  A masked weight is zero, but zero times
// one of them is a NaN, so where rows see only a part of a tile its values that
// are not finite are kept out of LDS (zeros instead) and remembered by column:
// which key is the first (the last query's reach is the furthest) with a +inf, a
// -inf or a NaN.  Since masks are monotone, that is all it takes to add them, at
// the end, to the sums that see them (weights are positive: infinities keep their
// sign).
template <int COLS>
struct NonFinite {
  int at[3][COLS];
  int any;
  // all threads; a barrier has to follow
  __device__ __forceinline__ void clear(int none) {
    for (int i = threadIdx.x; i < 3 * COLS; i += 256) at[i / COLS][i % COLS] = none;
    if (threadIdx.x == 0) any = 0;
  }
  // takes them out of columns c .. c + 7 in u, of the key (or with the reach) `value`
  template <typename E, bool MIN>
  __device__ __forceinline__ void take(uint4& u, int c, int value) {
    const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = i < 2 ? d[0] : i < 4 ? d[1] : i < 6 ? d[2] : d[3];
      const float x = E::widen((uint16_t)(w >> (16 * (i & 1))));
      if (fabsf(x) < INFINITY) continue;
      int* const to = &at[x != x ? 2 : x > 0.f ? 0 : 1][c + i];
      if (MIN) atomicMin(to, value);
      else atomicMax(to, value);
    }
    any = 1;
    u = finite_part<E>(u);
  }
  // what column c's make of a sum: those with a key up to (a reach from) `value` on are seen
  template <bool MIN>
  __device__ __forceinline__ float seen(int c, int value) const {
    bool y[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) y[i] = MIN ? at[i][c] <= value : at[i][c] >= value;
    return y[2] || (y[0] && y[1]) ? NAN : y[0] ? INFINITY : y[1] ? -INFINITY : 0.f;
  }
};

// Between a wave's own writes to LDS and other lanes' reads of them, or the
// reverse: the hardware keeps a wave's LDS operations in order, the compiler has to.
__device__ __forceinline__ void own_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The largest of both halves of the wave, lane by lane % 32; and the sum.
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// A 32 x 32 accumulator block, whose columns (lane % 32) are rows of the
// tensor: values 32 block + 0 .. 31 of the lane's row at element `at`, as far
// as they are below d, times f, rounded.  The halves of the wave trade parts so
// that each lane stores 16 bytes twice.
template <typename E>
__device__ __forceinline__ void store_block(const Heads& o, int64_t at, bool ok, int block, int d, const f32x16& acc, float f,
                                            int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = E::pack2(acc[8 * i + 2 * j] * f, acc[8 * i + 2 * j + 1] * f);
      const uint32_t hi = E::pack2(acc[8 * i + 4 + 2 * j] * f, acc[8 * i + 5 + 2 * j] * f);
      const auto r = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
      w[j] = r[0];
      w[2 + j] = r[1];
    }
    const int c = 32 * block + 16 * i + 8 * (lane >> 5);
    if (ok && c < d && in_bounds(at + c, 8, o.n))
      *reinterpret_cast<uint4*>(const_cast<uint16_t*>(o.p) + at + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// `rows` tokens of one head from element `at` on as a buffer: past its end
// (token strides are at most 2^23 elements, tiles at most 128 tokens) reads zeros.
__device__ __forceinline__ uint32_t rows_bytes(const Heads& x, int64_t rows, int32_t d) {
  const int64_t n = min(rows, (int64_t)128);
  return n > 0 ? (uint32_t)(((n - 1) * x.token + d) * 2) : 0u;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const Heads& x, int64_t at, int64_t rows, int32_t d) {
  return make_rsrc(x.p + (rows > 0 ? at : 0), rows_bytes(x, rows, d));
}
__device__ __forceinline__ LdsSource rows_source(const Heads& x, int64_t at, int64_t rows, int32_t d) {
  return lds_source(x.p + (rows > 0 ? at : 0), rows_bytes(x, rows, d));
}

// Hand-off of LDS between waves: all of this wave's loads and LDS operations are
// done, then the barrier.
__device__ __forceinline__ void tile_barrier() {
  wait_loads();
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint4 load16(const Heads& x, int64_t at, bool ok) {
  return ok && in_bounds(at, 8, x.n) ? *reinterpret_cast<const uint4*>(x.p + at) : make_uint4(0, 0, 0, 0);
}

template <typename E, typename A>
__device__ __forceinline__ typename E::v8 pack8(const A& p, int i) {
  return E::vec(make_uint4(E::pack2(p[i], p[i + 1]), E::pack2(p[i + 2], p[i + 3]), E::pack2(p[i + 4], p[i + 5]),
                           E::pack2(p[i + 6], p[i + 7])));
}

}  // namespace
}  // namespace qlora
