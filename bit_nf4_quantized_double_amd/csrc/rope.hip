// Rotary positions:
//
//   (x_a, x_b) -> factor (x_a cos - x_b sin, x_b cos + x_a sin),  angle = p f
//
// for the pairs (i, i + r/2) or (2i, 2i + 1) of the first r values of a head;
// the others pass through.  The backward is the same with -angle.
//
// The angle.  f comes as a whole number F of 2^-64 turns, so p F modulo 2^64
// is the angle's place in the turn, exact but for F's own rounding: p 2^-65
// turns, 1e-13 of one at a million.  (p f in fp32 is off by 0.06 radians there.)
// Its top bits give the eighth of a turn and a remainder of at most an eighth,
// where sine and cosine are their power series.
//
// Bound by memory: each value is read and written once (8192 tokens, 32 query and
// 8 key heads of 128: 33 to 35 us, 4.9 to 5.1 TB/s, a copy's rate).  A thread
// keeps the sines of its 8 pairs for all the heads it turns, 8 of them; few tokens
// are bound by the launch (16 tokens: 4.5 us), and spread over more threads.
#include <algorithm>

#include "common.h"
#include "decoder.h"
#include "rows_common.h"

namespace qlora {
namespace {

// sine and cosine of a turn's fraction u / 2^32
__device__ __forceinline__ void sincos_turn(uint32_t u, float& s, float& c) {
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(u - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32; |x| <= pi / 4
  const float y = x * x;
  // power series; the terms left out are below x^11 / 11! = 2e-9 and x^12 / 12! = 1e-10
  const float sn = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
  const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 - y * (1.f / 3628800)))));
  const float a = quarter & 1 ? cs : sn, b = quarter & 1 ? sn : cs;
  s = quarter & 2 ? -a : a;
  c = (quarter + 1) & 2 ? -b : b;
}

template <typename E>
__device__ __forceinline__ float half_of(const uint4& u, int i) {
  const uint32_t d = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
  return E::widen((uint16_t)(d >> (16 * (i & 1))));
}

// A thread turns pieces of 8 pairs (16 bytes twice; or, where sizes, strides or
// pointers leave no such pieces, single pairs) of every nth head of a token, and
// copies the same piece of what is not turned.
template <typename E, bool VEC>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a, int32_t pieces, int32_t turned, int32_t lines) {
  constexpr int P = VEC ? 8 : 1;
  const int64_t i = block_of(blockIdx.x, blockIdx.y) * 256 + threadIdx.x;
  const int64_t token = i / (pieces * lines);
  if (token >= a.t) return;
  const int32_t rest = (int32_t)(i - token * (pieces * lines)), piece = rest % pieces, line = rest / pieces;
  const int32_t half = a.rot >> 1;
  const bool turn = piece < turned;
  float sn[P], cs[P];
  if (turn) {
    const int64_t p = !in_bounds(token, 1, a.t) ? 0
                      : a.pos64                 ? static_cast<const int64_t*>(a.positions)[token]
                                                : static_cast<const int32_t*>(a.positions)[token];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int32_t at = piece * P + j;
      const uint64_t f = in_bounds(at, 1, half) ? a.turns[at] : 0;
      sincos_turn((uint32_t)((uint64_t)p * f >> 32), sn[j], cs[j]);
      sn[j] *= a.inverse ? -a.factor : a.factor;
      cs[j] *= a.factor;
    }
  }
  for (int32_t h = line; h < a.heads + a.kv_heads; h += lines) {
    const bool isk = h >= a.heads;
    const Heads &x = isk ? a.k : a.q, &y = isk ? a.ko : a.qo;
    const int32_t head = isk ? h - a.heads : h;
    const int64_t in = token * x.token + head * x.head, out = token * y.token + head * y.head;
    uint16_t* o = const_cast<uint16_t*>(y.p);
    if constexpr (VEC) {
      if (!turn) {
        const int32_t c = a.rot + (piece - turned) * 8;
        if (in_bounds(in + c, 8, x.n) && in_bounds(out + c, 8, y.n))
          *reinterpret_cast<uint4*>(o + out + c) = *reinterpret_cast<const uint4*>(x.p + in + c);
        continue;
      }
      const int32_t c0 = a.interleaved ? piece * 16 : piece * 8, c1 = a.interleaved ? c0 + 8 : half + c0;
      uint4 u = make_uint4(0, 0, 0, 0), v = u;
      if (in_bounds(in + c0, 8, x.n)) u = *reinterpret_cast<const uint4*>(x.p + in + c0);
      if (in_bounds(in + c1, 8, x.n)) v = *reinterpret_cast<const uint4*>(x.p + in + c1);
      float r[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = a.interleaved ? half_of<E>(j < 4 ? u : v, 2 * j & 7) : half_of<E>(u, j);
        const float g = a.interleaved ? half_of<E>(j < 4 ? u : v, (2 * j & 7) + 1) : half_of<E>(v, j);
        const float lo = f * cs[j] - g * sn[j], hi = g * cs[j] + f * sn[j];
        // (constant indexes on both sides: the array stays in registers)
        if (a.interleaved) { r[2 * j] = lo; r[2 * j + 1] = hi; }
        else { r[j] = lo; r[8 + j] = hi; }
      }
      u = make_uint4(E::pack2(r[0], r[1]), E::pack2(r[2], r[3]), E::pack2(r[4], r[5]), E::pack2(r[6], r[7]));
      v = make_uint4(E::pack2(r[8], r[9]), E::pack2(r[10], r[11]), E::pack2(r[12], r[13]), E::pack2(r[14], r[15]));
      if (in_bounds(out + c0, 8, y.n)) *reinterpret_cast<uint4*>(o + out + c0) = u;
      if (in_bounds(out + c1, 8, y.n)) *reinterpret_cast<uint4*>(o + out + c1) = v;
    } else {
      if (!turn) {
        const int32_t c = a.rot + piece - turned;
        if (in_bounds(in + c, 1, x.n) && in_bounds(out + c, 1, y.n)) o[out + c] = x.p[in + c];
        continue;
      }
      const int32_t c0 = a.interleaved ? 2 * piece : piece, c1 = a.interleaved ? c0 + 1 : half + c0;
      const float f = in_bounds(in + c0, 1, x.n) ? E::widen(x.p[in + c0]) : 0.f;
      const float g = in_bounds(in + c1, 1, x.n) ? E::widen(x.p[in + c1]) : 0.f;
      const uint32_t w = E::pack2(f * cs[0] - g * sn[0], g * cs[0] + f * sn[0]);
      if (in_bounds(out + c0, 1, y.n)) o[out + c0] = (uint16_t)w;
      if (in_bounds(out + c1, 1, y.n)) o[out + c1] = (uint16_t)(w >> 16);
    }
  }
}

bool in_pieces(const Heads& x, int64_t h) {
  return h == 0 || (((uintptr_t)x.p & 15) == 0 && x.token % 8 == 0 && x.head % 8 == 0);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  const bool vec = a.rot % 16 == 0 && a.d % 8 == 0 && in_pieces(a.q, a.heads) && in_pieces(a.qo, a.heads) &&
                   in_pieces(a.k, a.kv_heads) && in_pieces(a.ko, a.kv_heads);
  // what is not turned is copied, unless it is there already
  const bool copy = a.q.p != a.qo.p || a.k.p != a.ko.p;
  const int32_t turned = vec ? a.rot / 16 : a.rot / 2;
  const int32_t pieces = turned + (copy ? (vec ? (a.d - a.rot) / 8 : a.d - a.rot) : 0);
  const int64_t all = a.heads + a.kv_heads;
  if (pieces == 0) return hipSuccess;
  // Heads of a thread: 8, whose sines it makes once, but fewer where that
  // would leave compute units idle (a token's heads spread over more threads).
  int64_t lines = std::max<int64_t>((all + 7) / 8, 1);
  while (lines < all && a.t * pieces * lines < 256 * 512) lines = std::min(all, 2 * lines);
  const dim3 grid = grid_of((a.t * pieces * lines + 255) / 256);
  const auto run = [&](auto e) {
    using E = decltype(e);
    if (vec) k_rope<E, true><<<grid, 256, 0, stream>>>(a, pieces, turned, (int32_t)lines);
    else k_rope<E, false><<<grid, 256, 0, stream>>>(a, pieces, turned, (int32_t)lines);
  };
  if (a.f16) run(F16{});
  else run(Bf16{});
  return hipGetLastError();
}

QLORA_OOB_READER(oob_count_rope)

}  // namespace qlora
