// The product with an epilogue for many rows per weight, in two steps:
//
//  1. expand_kernel rebuilds the weight's GroupTiles into dense fp16 matrix-
//     core fragments in the workspace, once per call (INT4: the codes; the row
//     scales go into the epilogue).  A wave takes a GroupTile, as in decode;
//     it is bound by the bytes it writes, 2 per element.
//  2. wide_kernel multiplies them, fp32 accumulators in registers, both
//     operands through LDS by LDS-DMA several half columns (32 k) ahead, the
//     fragments of the next half column read between the MFMAs of this one.
//
// Rebuilding inside the product instead would cost LDS time on every column
// for every tile of rows, and LDS is what the product is next bound by: per
// column a wave of the large tiling reads 24 KB of fragments for 64 MFMAs of
// 16 cycles, 0.75 of the matrix time at 128 B a cycle, before any rebuild.
// The large tiling reaches 1180 TFLOP/s on 4096^3 (116 us; the library's dense
// product 1350 on 8192^3), where the clock falls under load.
//
// Fragments in the workspace are in the order a wave reads them (1 KB each),
// so their copies to LDS and the reads from it are contiguous.  Rows of x are
// copied as they lie, gathered rows alike.
//
// Work split, large tiles: they are dealt to one workgroup per compute unit,
// whole rounds of tiles; the GroupTile columns of the tiles left over are
// split evenly (a tile may then be shared by workgroups, which leave fp32
// partial sums; the last to finish adds them in column order, so results do
// not depend on timing).  Smaller tiles are a workgroup each, or a few that
// split the columns.  Consecutive tiles are up to eight tiles of rows by the
// weight's strips, so the workgroups of an XCD share both operands in its L2.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "usw.h"
#include "usw_decode_kernels.h"
#include "usw_internal.h"
#include "usw_wide.h"
#include "usw_wide_kernels.h"

namespace {

constexpr int kBM[3] = {Large::BM, Medium::BM, Small::BM};
constexpr int kBN[3] = {Large::BN, Medium::BN, Small::BN};
constexpr int64_t kComputeUnits = 256;

// Dense fragments held at a time: weights beyond this are expanded and
// multiplied in groups, each with its own pair of launches.
constexpr int64_t kDenseBytes = int64_t(1) << 30;

}  // namespace

namespace usw {

WidePlan wide_plan(const Geometry& g, int32_t E, int32_t S, bool lone) {
  WidePlan p{};
  const int64_t one = g.M * g.K * 2;
  p.group = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(E, kDenseBytes / one)));
  // Expected tiles of a tiling: runs end inside a tile, half a tile each.
  const int64_t runs = std::min<int64_t>(p.group, S);
  auto expected = [&](int t) {
    const int64_t n = p.group == 1 ? (S + kBN[t] - 1) / kBN[t] : std::max<int64_t>(runs, S / kBN[t] + runs / 2);
    return n * ((g.M + kBM[t] - 1) / kBM[t]);
  };
  // Large tiles are the fastest on the matrix cores, but need a whole round
  // of them, and each stands alone on its compute unit: nothing hides its
  // fill and epilogue, nor the sums of the columns shared after the last
  // whole round.  In microseconds of MI355X, fitted to the times below: 1.82 a
  // column and 6 a tile, 35 where tiles are left over, against 0.64 a column
  // of a medium tile.  Expansion included, large / medium: 4096^3 131 / 174,
  // 8192x4096 N = 2048 126 / 147, 20480x2560 N = 2000 224 / 257, 11904x1152
  // N = 2000 108 / 72, 8 experts of 4096x2048 with 500 rows each 155 / 120.
  // Small tiles up to 4e9 multiply-adds, where the grid is short of workgroups,
  // small / medium: 1152x1152 N = 300 13.2 / 17.1, 4096x4096 N = 100 26.2 /
  // 30.4; 5120x5120 N = 200 40.5 / 40.9, N = 300 50.1 / 44.3.
  const int64_t large = expected(0), rounds = large / kComputeUnits;
  const double large_us = 1.82 * large * g.Gc / kComputeUnits + 6.0 * rounds + (large % kComputeUnits ? 35.0 : 0.0);
  const double medium_us = 0.64 * expected(1) * g.Gc / kComputeUnits;
  p.tiling = (rounds > 0 || lone) && large_us < medium_us ? 0 : g.M * g.K * S <= 4000000000ll ? 2 : 1;
  // Splits of the columns, at least eight each, while they fill the chip: up
  // to 256 medium workgroups (4096x11008 N = 512: 2 splits 81.4 us, 1 113.7, 4
  // 87.7) or 704 small ones (2560x2560 N = 160: 4 splits 21.3, 1 27.3;
  // 2048x2048 N = 70: 4 splits 15.8, 1 19.9; 128x16064 N = 669: 16 splits 25.4,
  // 8 26.0, 32 33.1).
  p.splits = 1;
  const int64_t most = p.tiling == 0 ? 0 : p.tiling == 1 ? 256 : 704;
  while (p.splits < 16 && expected(p.tiling) * p.splits * 2 <= most && g.Gc >= 16 * p.splits) p.splits *= 2;
  const int64_t mt = (g.M + kBM[p.tiling] - 1) / kBM[p.tiling];
  p.tiles = (runs + (S - runs) / kBN[p.tiling]) * mt;
  const size_t slot = static_cast<size_t>(4) * kBM[p.tiling] * kBN[p.tiling];
  const size_t slots = p.tiling == 0 ? 2 * kComputeUnits : p.splits > 1 ? p.tiles * p.splits : 0;
  p.slots_at = counter_zone(slots > 0 ? static_cast<size_t>(4) * p.tiles : 0);
  p.cb = slots > 0 ? p.slots_at : 0;
  p.dense_at = p.slots_at + slots * slot;
  p.need = p.dense_at + static_cast<size_t>(p.group) * one;
  return p;
}

usw_status wide_launch(const WideCall& c, const Geometry& g, const WidePlan& p, void* ws, void* stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  ExpandArgs x{};
  x.bitmaps = c.bitmaps;
  x.offsets = c.offsets;
  x.values = c.values;
  x.starts = c.starts;
  x.slots = c.slots;
  x.dense = reinterpret_cast<u32x4_t*>(w + p.dense_at);
  x.values_total = c.values_total;
  x.ngt = g.ngt;
  x.S = c.S;
  WideArgs a{};
  fill_wide(a, p, g, c.S, x.dense, ws);
  a.X = c.X;
  a.Y = c.Y;
  a.scales = c.scales;
  a.slots = c.slots;
  a.rows = c.rows;
  a.e = c.e;
  a.T = c.T;
  a.i4 = c.val_type == USW_VAL_I4;
  if (!wide_launchable(p) || g.ngt / kExpandWaves >= (int64_t(1) << 31) - 1) return USW_ERR_UNSUPPORTED;
  const unsigned gx = static_cast<unsigned>((g.ngt + kExpandWaves - 1) / kExpandWaves);
  for (int e0 = 0; e0 < c.E; e0 += p.group) {
    const int e1 = std::min(c.E, e0 + p.group);
    x.e0 = a.e0 = e0;
    a.e1 = e1;
    const dim3 grid(gx, static_cast<unsigned>(e1 - e0));
    if (a.i4) expand_kernel<true><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    else expand_kernel<false><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    launch_wide<EpilogueFinish>(p, a, s);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

usw_status wide_multiply(const Geometry& g, const WidePlan& p, int32_t rows, const uint16_t* X, void* Y,
                         const usw_dev::Epilogue& e, const void* dense, void* ws, void* stream) {
  if (!wide_launchable(p)) return USW_ERR_UNSUPPORTED;
  WideArgs a{};
  fill_wide(a, p, g, rows, dense, ws);
  a.X = X;
  a.Y = Y;
  a.e = e;
  launch_wide<EpilogueFinish>(p, a, static_cast<hipStream_t>(stream));
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

}  // namespace usw
