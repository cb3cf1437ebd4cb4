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

WidePlan wide_plan(const Geometry& g, int32_t E, int32_t S);
usw_status wide_launch(const WideCall& c, const Geometry& g, const WidePlan& p, void* ws, void* stream);

}  // namespace usw
