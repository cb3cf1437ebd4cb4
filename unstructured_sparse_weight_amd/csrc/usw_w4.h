// The dense 4-bit weight's layout and rounding, shared by its host and device
// encoders and its product (the format is described in usw.h).
#pragma once

#include <cstdint>

#include "usw.h"
#include "usw_quant.h"

namespace usw {

constexpr int kW4Rows = 16, kW4Cols = 128;   // a tile

inline int w4_tiles(int64_t K) { return static_cast<int>((K + kW4Cols - 1) / kW4Cols); }   // of a row block

// M at most 2^20 keeps a tile's rows of outputs within 32-bit addresses, M K
// at most 2^34 the encoder's and the expansion's launches below HIP's 2^32 threads.
inline usw_status check_w4_shape(int64_t M, int64_t K, int32_t group) {
  if (M <= 0 || K <= 0 || M % kW4Rows || K % 64) return USW_ERR_BAD_SHAPE;
  if (group != 32 && group != 64 && group != 128) return USW_ERR_BAD_SHAPE;
  if (M > (int64_t(1) << 20) || K > (int64_t(1) << 20) || M * K > (int64_t(1) << 34)) return USW_ERR_UNSUPPORTED;
  return USW_OK;
}

// Bit position in its dword of column i (0..7): nibbles t and t + 4 hold
// columns 2 t and 2 t + 1.
__host__ __device__ inline int w4_shift(int i) { return 4 * ((i >> 1) + 4 * (i & 1)); }

// fp16 bits of a non-negative scale rounded to 8 significant bits, half to
// even, so that its product with a code (at most 3 significant bits, or 8) is
// an fp16 number.  Carries move into the exponent as they should; infinities
// and the quiet NaN have no bits to drop.
__host__ __device__ inline uint16_t w4_round_scale(uint16_t bits) {
  uint32_t m = (bits & 0x3FFu) | (bits >= 0x400u ? 0x400u : 0u);
  int drop = 0;
  while (m >> (8 + drop)) ++drop;
  if (drop == 0) return bits;
  const uint32_t half = (1u << drop) >> 1, odd = (bits >> drop) & 1u;
  return static_cast<uint16_t>((bits + half - 1u + odd) >> drop << drop);
}

// Scale of a group from its largest magnitude's bits.
__host__ __device__ inline uint16_t w4_scale_bits(uint16_t amax_bits) { return w4_round_scale(i4_scale_bits(amax_bits)); }

}  // namespace usw
