// Matrix product in 8-bit integers:
//
//   out[m][n] = E(sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n])
//
// x and w are int8 codes in operand tiles (int8_layout.h); the sum is exact
// in int32 on the matrix cores (v_mfma_i32_32x32x32_i8), the scales are
// applied in fp32, token first, and the result is rounded once to the 16-bit
// output type.  w is the A operand, x the B operand: a lane then holds 16
// consecutive outputs of one token.
#include <algorithm>
#include <climits>

#include "common.h"
#include "int8_layout.h"

namespace qlora {
namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

__device__ __forceinline__ i32x4 as_i32x4(uint4 u) { return __builtin_bit_cast(i32x4, u); }

// Strips [first, total) of a tiled matrix as a buffer: what lies past its end
// (at most 2^31 bytes on) reads zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t strips_rsrc(const int8_t* p, int64_t first, int64_t total,
                                                              int64_t kp) {
  const int64_t bytes = max((int64_t)0, total - first) * 16 * kp;
  return make_rsrc(p + (first < total ? first : 0) * 16 * kp, (uint32_t)min(bytes, (int64_t)0x7fffffff));
}

// Up to 4 consecutive outputs n0 .. n0 + 3 of token m.
template <typename E>
__device__ __forceinline__ void store4(const Int8GemmArgs& a, int64_t m, int64_t n0, const int* acc, float sx,
                                       bool vec) {
  if (m >= a.m || n0 >= a.n) return;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool ok = n0 + i < a.n;
    y[i] = (float)acc[i] * sx;
    if (a.sw) y[i] *= ok && in_bounds(n0 + i, 1, a.n) ? a.sw[n0 + i] : 0.f;
    if (a.bias) y[i] += ok && in_bounds(n0 + i, 1, a.n) ? E::widen(a.bias[n0 + i]) : 0.f;
  }
  const int64_t e = m * a.n + n0;
  const uint32_t lo = E::pack2(y[0], y[1]), hi = E::pack2(y[2], y[3]);
  if (vec && n0 + 4 <= a.n) {
    if (in_bounds(e, 4, a.m * a.n)) *reinterpret_cast<uint2*>(a.out + e) = make_uint2(lo, hi);
  } else {
    const uint32_t d[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.n && in_bounds(e + i, 1, a.m * a.n)) a.out[e + i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
  }
}

// Tile of 128 outputs x 128 tokens, 4 waves of 64 x 64, operands straight
// from memory into registers.
template <typename E>
__global__ __launch_bounds__(256) void k_int8_gemm(Int8GemmArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t kp = int8_kp(a.k);
  const int64_t tn = (a.n + 127) / 128;
  const int64_t n0 = blockIdx.x % tn * 128 + 64 * (wave & 1), m0 = blockIdx.x / tn * 128 + 64 * (wave >> 1);
  const __amdgpu_buffer_rsrc_t rw = strips_rsrc(a.w, n0 >> 4, int8_weight_strips(a.n), kp);
  const __amdgpu_buffer_rsrc_t rx = strips_rsrc(a.x, m0 >> 4, int8_row_strips(a.m), kp);
  // lane l of a 32-row operand: row l & 31, half l >> 5 of 32 columns
  const uint32_t strip = 16u * (uint32_t)kp;
  const uint32_t at = (uint32_t)((lane >> 4) & 1) * strip + (uint32_t)(lane >> 5) * 256u + (uint32_t)(lane & 15) * 16u;
  i32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  for (uint32_t k = 0; k < (uint32_t)kp; k += 32) {
    uint4 w[2], x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = buf_load16(rw, at + 2u * i * strip + (k >> 6) * 1024u + ((k >> 5) & 1u) * 512u);
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = buf_load16(rx, at + 2u * i * strip + (k >> 6) * 1024u + ((k >> 5) & 1u) * 512u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(as_i32x4(w[i]), as_i32x4(x[j]), acc[i][j], 0, 0, 0);
  }
  const bool vec = a.n % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7u) == 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t m = m0 + 32 * j + (lane & 31);
    const float sx = m < a.m && in_bounds(m, 1, a.m) ? a.sx[m] : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        store4<E>(a, m, n0 + 32 * i + 16 * (lane >> 5) + 4 * q, v, sx, vec);
      }
  }
}

// ---- layouts ----------------------------------------------------------------
// Row-major codes into weight tiles: one 16-byte piece a thread, rows past n
// and columns past k zero.
__global__ __launch_bounds__(256) void k_int8_pack(const int8_t* src, int64_t ld, int64_t n, int64_t k, int8_t* dst,
                                                   int64_t rows, bool vec) {
  const int64_t kp = int8_kp(k);
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15), piece = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 4);
  if (row >= rows || piece * 16 >= kp) return;
  const int64_t c = piece * 16, e = row * ld + c, size = (n - 1) * ld + k;
  uint4 u = make_uint4(0, 0, 0, 0);
  if (row < n) {
    if (vec && c + 16 <= k) {
      if (in_bounds(e, 16, size)) u = *reinterpret_cast<const uint4*>(src + e);
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

// Tiles back to a row-major 16-bit matrix of the values they stand for.
template <typename E>
__global__ __launch_bounds__(256) void k_int8_dequant(const int8_t* codes, const float* scale, int64_t m, int64_t k,
                                                      bool weight, uint16_t* out, bool vec) {
  const int64_t kp = int8_kp(k), rows = (weight ? int8_weight_strips(m) : int8_row_strips(m)) * 16;
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15), piece = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 4);
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
  if (vec && c + 16 <= k) {
    if (in_bounds(e, 16, m * k)) {
      uint4* q = reinterpret_cast<uint4*>(out + e);
      q[0] = make_uint4(o[0], o[1], o[2], o[3]);
      q[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < k && in_bounds(e + i, 1, m * k)) out[e + i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace

size_t int8_part_bytes(int64_t, int64_t, int64_t, int) { return 0; }

hipError_t launch_int8_gemm(Int8GemmArgs a, int, hipStream_t st) {
  const int64_t grid = (a.n + 127) / 128 * ((a.m + 127) / 128);
  if (grid > INT_MAX) return hipErrorInvalidValue;
  if (a.f16) k_int8_gemm<F16><<<dim3((uint32_t)grid), 256, 0, st>>>(a);
  else k_int8_gemm<Bf16><<<dim3((uint32_t)grid), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_int8_pack(const int8_t* src, int64_t ld, int64_t n, int64_t k, int8_t* dst, hipStream_t st) {
  const int64_t rows = int8_weight_strips(n) * 16;
  const dim3 grid((uint32_t)(rows / 16), (uint32_t)((int8_kp(k) / 16 + 15) / 16));
  k_int8_pack<<<grid, 256, 0, st>>>(src, ld, n, k, dst, rows, aligned(src, 16) && (n <= 1 || ld % 16 == 0));
  return hipGetLastError();
}

hipError_t launch_int8_transpose(const int8_t* src, int64_t n, int64_t k, int8_t* dst, hipStream_t st) {
  const dim3 grid((uint32_t)((int8_weight_strips(k) * 16 + 63) / 64), (uint32_t)((int8_kp(n) + 63) / 64));
  k_int8_transpose<<<grid, 256, 0, st>>>(src, n, k, dst);
  return hipGetLastError();
}

hipError_t launch_int8_dequant(const int8_t* codes, const float* scale, int64_t m, int64_t k, bool weight, bool f16,
                               uint16_t* out, hipStream_t st) {
  const dim3 grid((uint32_t)((m + 15) / 16), (uint32_t)((k + 255) / 256));
  const bool vec = aligned(out, 16) && (m <= 1 || k % 8 == 0);
  if (f16) k_int8_dequant<F16><<<grid, 256, 0, st>>>(codes, scale, m, k, weight, out, vec);
  else k_int8_dequant<Bf16><<<grid, 256, 0, st>>>(codes, scale, m, k, weight, out, vec);
  return hipGetLastError();
}

QLORA_OOB_READER(oob_count_int8)

}  // namespace qlora
