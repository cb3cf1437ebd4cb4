// What the gradients' two ways to dx share (usw_grad.hip, usw_grad_few.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "usw.h"
#include "usw_device.h"
#include "usw_internal.h"

namespace usw {

// Gradients of few rows: dx [N][K] straight from the encoded weights, up to two
// of one shape, whose rows follow each other in D's columns, and the values' of
// fp16 weights straight from D and X.
struct FewCall {
  const usw_fmt* f[2];   // the weight of each block of dx's reduction
  int weights, blocks;   // blocks > weights: the weight once more, for D's remainders
  int64_t ldD, lo;       // row length of D; lo > 0: the column where the remainders of its rounding start
  bool frag;             // dx reads F, the fragments of D's columns (below), else D's rows
  const uint16_t *D, *F, *X;
  void *dX, *dV[2];
  bool want_x, want_v;
  int32_t N, out_type;
};

struct FewPlan {
  int splits;    // workgroups per strip of 64 columns
  bool lean;     // five value chunks to a slot
  size_t cb, need;
};

// Most rows of dx, as the kernels' accumulators allow; the expanded product /
// this, with the values' gradient of the fp16 weights: pairs of 11008x4096 N = 128
// 188 / 116 us, INT4 113 / 53.5; 4096x4096 N = 128 51.0 / 45.5; 2048x2048 pairs N =
// 100 44.5 / 37.2; 640x512 N = 100 23.5 / 21.
constexpr int kFewGradRows = 128;
// Most rows of the values', whose d stays in registers; wide / this: pairs of
// 11008x4096 N = 64 101 / 99, 4096x4096 N = 64 41.7 / 25.5, 640x512 N = 33 21.0 / 14.8.
constexpr int kFewValueRows = 64;
constexpr int kLoRows = 32;   // most rows with remainders

// 16-token blocks of a call.  D as fragments: of 32 columns (the reduction) by 16
// tokens, a column's blocks behind each other; lane l of one holds token l % 16,
// columns 8 (l / 16) on.
int few_row_blocks(int N);
FewPlan few_plan(const Geometry& g, const FewCall& c);
usw_status few_launch(const Geometry& g, const FewCall& c, const FewPlan& p, void* ws, void* stream);

}  // namespace usw

namespace usw_dev {

// A row's INT4 scale as 2^e times f with f in [0.5, 1) (e at most 12, so that
// codes times 2^e are fp16 numbers).  A scale that is zero, infinite or NaN is
// all in f.
__device__ __forceinline__ float scale_power(float s) {
  const uint32_t b = __float_as_uint(s) & 0x7FFFFFFFu;
  if (b == 0 || b >= 0x7F800000u) return 1.0f;
  const int e = min(static_cast<int>(b >> 23) - 126, 12);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ float scale_rest(float s) {
  return s * __uint_as_float((254u << 23) - __float_as_uint(scale_power(s)));   // by 2^-e, exact
}

// v with the largest numbers for infinities and NaN: what remainders of d are
// multiplied with.  An infinity is in the product with d itself, where a
// remainder of zero, or of the other sign, would make a NaN of it.  As whole
// numbers +inf and its NaN are the largest signed ones, -inf and its the largest
// unsigned ones.  For the values it costs half a percent (pairs of 11008x4096 N = 8
// 68.3 / 68.9 us).
__device__ __forceinline__ half8_t finite(half8_t v) {
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  typedef unsigned short u16x8_t __attribute__((ext_vector_type(8)));
  const s16x8_t up = __builtin_elementwise_min(__builtin_bit_cast(s16x8_t, v), s16x8_t{} + static_cast<short>(0x7BFF));
  return __builtin_bit_cast(half8_t, __builtin_elementwise_min(__builtin_bit_cast(u16x8_t, up),
                                                               u16x8_t{} + static_cast<unsigned short>(0xFBFF)));
}

typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kTrLd = 72;                     // halves of a row of a tile of 64 columns in LDS: rows 144 bytes apart

// Eight rows 8 (lane / 16) on of column `col` + lane % 16 of the tile.
__device__ __forceinline__ half8_t read_column(const uint8_t* tile, int lane, int col) {
  const uint8_t* p = tile + 2 * ((8 * (lane >> 4) + ((lane >> 2) & 3)) * kTrLd + col + 4 * (lane & 3));
  typedef __attribute__((address_space(3))) s16x4_t* At;
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(p + 2 * 4 * kTrLd));
  return __builtin_bit_cast(half8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

}  // namespace usw_dev
