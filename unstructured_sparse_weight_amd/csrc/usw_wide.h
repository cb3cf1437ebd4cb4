// Many rows per weight: the weight is expanded once to dense fp16 fragments
// in the workspace and multiplied on the matrix cores (usw_wide.hip).
#pragma once

#include <cstddef>
#include <cstdint>

#include "usw.h"
#include "usw_epilogue.h"
#include "usw_internal.h"

namespace usw {

// Leading workspace bytes that hold `bytes` of counters.  At least 64 KiB, which
// no call uses for anything else, so that calls of different sizes can share a
// workspace whose counters stay zero.
inline size_t counter_zone(size_t bytes) {
  constexpr size_t kLeast = size_t(64) << 10;
  return bytes <= kLeast ? kLeast : (bytes + 255) & ~size_t(255);
}

// One call: a single weight (slots null, one run of S rows) or E weights on
// the runs slots[E+1].  The encodings are as in usw_expert_fmt.
struct WideCall {
  const uint64_t* bitmaps;
  const uint32_t* offsets;
  const uint8_t* values;
  const int64_t* starts;      // null: one weight
  const uint16_t* scales;     // INT4 only
  int64_t values_total;       // bytes of values
  int32_t val_type, E;
  const uint16_t* X;
  const int32_t* slots;
  const int32_t* rows;
  int32_t S, T;
  void* Y;
  usw_dev::Epilogue e;
};

struct WidePlan {
  int group;        // weights expanded and multiplied at a time
  int tiling;       // 0, 1, 2: large, medium, small tiles
  int splits;       // workgroups that share a tile's columns
  int64_t tiles;    // most output tiles of one group
  size_t cb, slots_at, dense_at, need;   // workspace: counters (0: none), partial sums, dense fragments
};

// lone: large tiles also where there is no whole round of them and the estimate has
// them ahead (all their columns are shared then).  Calls with / without, us: gated
// 5120x5120 N = 1500 182 / 200, 2048x8192 N = 2000 144 / 155; gradients of pairs of
// 11008x4096 N = 1024 483 / 561, 8192x2048 N = 2000 323 / 363, INT4 20480x5120 N = 400
// 422 / 617; 4-bit 4096x11008 N = 2047 190 / 210, 5120x20480 N = 512 211 / 283; where
// the estimate has medium tiles ahead both are one, 4-bit 4096x4096 N = 2048 77.6 /
// 76.7.  None was slower by more than 1%; the fused and expert products go without, because sums of
// shared columns are added in another order and their results are kept bit for bit.
WidePlan wide_plan(const Geometry& g, int32_t E, int32_t S, bool lone = false);

// Whether the plan's product is a launch: less than HIP's 2^32 threads, 256 of
// them to each workgroup of the small and medium tiles, whose number is rounded up
// to a multiple of 8; the large tiles' launch is of fixed size, their numbers 32-bit.
inline bool wide_launchable(const WidePlan& p) {
  return p.tiling == 0 ? p.tiles < (int64_t(1) << 31) : p.tiles * p.splits <= (int64_t(1) << 24) - 8;
}
usw_status wide_launch(const WideCall& c, const Geometry& g, const WidePlan& p, void* ws, void* stream);

// The product alone, Y [rows][g.M] from X [rows][g.K] and dense fragments that
// the caller wrote ([64-row strip][64 columns][half][4 fragments][64 lanes], the
// last strip whole), with wide_plan(g, 1, rows).  Of the workspace it uses what
// comes before p.dense_at.
usw_status wide_multiply(const Geometry& g, const WidePlan& p, int32_t rows, const uint16_t* X, void* Y,
                         const usw_dev::Epilogue& e, const void* dense, void* ws, void* stream);

}  // namespace usw
