// Storage of 8-bit matrices: MFMA-operand tiles.
//
// A matrix of R rows by K columns is cut into strips of 16 rows and chunks of
// 64 columns; a (strip, chunk) tile is 1024 bytes, 16 bytes (columns 16 g ..
// 16 g + 15 of row r) at byte 256 g + 16 r.  Lane 16 g + r of a wave that
// loads a tile with one 16-byte load per lane holds what one operand of
// v_mfma_i32_16x16x64_i8 wants: row r, a quarter g of the 64 reduction
// columns.  (Which columns of the tile the instruction pairs up does not
// matter: both operands are stored alike, and a sum has no order.)  The tiles
// of a strip follow each other along K, which is padded to a multiple of 128
// with zero codes; a strip is contiguous, so both products read memory in
// runs of whole kilobytes and LDS without bank conflicts.
//
// A weight is the A operand, so its rows are the rows of D, of which lane
// 16 g + c holds rows 4 g + i (i = 0 .. 3) of column c.  Weight rows are stored
// so that row 4 g + i of strip s of a pair is output 8 g + 4 s + i of the
// pair's 32: a lane then holds 8 consecutive outputs of one token.  The last
// pair is padded.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace qlora {

// The largest reduction whose int32 sum cannot overflow: quantized rows hold
// codes of -127 .. 127, a weight's codes from elsewhere -128 too.
constexpr int64_t kInt8MaxK = 132104;

__host__ __device__ constexpr int64_t int8_kp(int64_t k) { return (k + 127) / 128 * 128; }
__host__ __device__ constexpr int64_t int8_row_strips(int64_t m) { return (m + 15) / 16; }
__host__ __device__ constexpr int64_t int8_weight_strips(int64_t n) { return (n + 31) / 32 * 2; }
constexpr size_t int8_rows_bytes(int64_t m, int64_t k) { return (size_t)int8_row_strips(m) * 16u * (size_t)int8_kp(k); }
constexpr size_t int8_weight_bytes(int64_t n, int64_t k) {
  return (size_t)int8_weight_strips(n) * 16u * (size_t)int8_kp(k);
}

// Stored row of weight row n (see above); activation rows keep their order.
__host__ __device__ constexpr int64_t int8_weight_row(int64_t n) {
  return (n & ~(int64_t)31) | (((n >> 2) & 1) << 4) | (((n >> 3) & 3) << 2) | (n & 3);
}

// Byte offset of 16-column piece `piece` (columns 16 piece ..) of stored row `row`.
__host__ __device__ constexpr int64_t int8_piece(int64_t row, int64_t piece, int64_t kp) {
  return (row >> 4) * (16 * kp) + (piece >> 2) * 1024 + (piece & 3) * 256 + (row & 15) * 16;
}

// Element types of the row operators' inputs, as in include/qlora.h.
enum RowType { kRowBf16 = 0, kRowF16 = 1, kRowF32 = 2 };

struct QuantArgs {  // a matrix to quantize, row by row
  const void* x;
  int type;
  int64_t ldx, m, k;
  const float* col_scale;  // NULL or [k]: multiplies the columns first
  bool weight;             // weight row order and padding
  int8_t* codes;
  float* scale;
};
struct NormArgs {
  const void *x, *residual, *gamma;
  int type, gamma_type;
  int64_t ldx, ldr, m, k;
  float eps;
  uint16_t* h;     // NULL without a residual
  uint16_t* y;     // 16-bit output,
  float* rstd;     // with y; NULL for
  int8_t* codes;   // 8-bit output
  float* scale;
};
struct NormBwdArgs {
  const void *dy, *h, *gamma, *dh;
  const float* rstd;
  int type, gamma_type;
  int64_t lddy, ldh, lddh, m, k;
  uint16_t* dx;
  float *dgamma, *part;
};
struct SwigluArgs {
  const void *g, *u, *dy;
  int type;
  int64_t ldg, ldu, lddy, m, k;
  uint16_t *y, *dg, *du;
  int8_t* codes;
  float* scale;
};

int norm_bwd_groups(int64_t m, int64_t k, int cus);  // partial rows of dgamma
hipError_t launch_quant_rows(const QuantArgs& a, int cus, hipStream_t st);
hipError_t launch_norm(const NormArgs& a, int cus, hipStream_t st);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int cus, hipStream_t st);
hipError_t launch_swiglu_rows(const SwigluArgs& a, int cus, hipStream_t st);  // 8-bit output
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t st);
hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t st);

struct Int8GemmArgs {  // out[m][n] = E(sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n])
  const int8_t *w, *x;
  const float *sw, *sx;  // sw may be NULL (all ones)
  const uint16_t* bias;
  uint16_t* out;
  int64_t m, n, k;
  bool f16;
  int32_t* part;  // room for split sums, or NULL
  int ksplit;
};
// Which kernel a product takes, and over how many workgroups a tile's
// reduction is split (needs `part`; without it one).
enum Int8Kind { kInt8Few16, kInt8Few32, kInt8Few64, kInt8Tile };
constexpr int int8_tokens(Int8Kind kind) {  // of a workgroup
  return kind == kInt8Few16 ? 16 : kind == kInt8Few32 ? 32 : kind == kInt8Few64 ? 64 : 256;
}
struct Int8Plan {
  Int8Kind kind;
  int ksplit;
};
Int8Plan int8_plan(int64_t m, int64_t n, int64_t k, int cus);
size_t int8_plan_bytes(const Int8Plan& p, int64_t m, int64_t n);
size_t int8_part_bytes(int64_t m, int64_t n, int64_t k, int cus);
hipError_t launch_int8_plan(const Int8GemmArgs& a, const Int8Plan& p, hipStream_t st);
hipError_t launch_int8_gemm(const Int8GemmArgs& a, int cus, hipStream_t st);
// Whether a product quantizes its 16-bit rows itself, in one launch (a.x, a.sx
// and a.part are then not used).
bool int8_fuses_rows(int64_t m, int64_t n, int64_t k);
hipError_t launch_int8_fused(const Int8GemmArgs& a, const QuantArgs& rows, hipStream_t st);
hipError_t launch_int8_pack(const int8_t* src, int64_t ld, int64_t n, int64_t k, int8_t* dst, hipStream_t st);
hipError_t launch_int8_transpose(const int8_t* src, int64_t n, int64_t k, int8_t* dst, hipStream_t st);
hipError_t launch_int8_dequant(const int8_t* codes, const float* scale, int64_t m, int64_t k, bool weight, bool f16,
                               uint16_t* out, hipStream_t st);

}  // namespace qlora
