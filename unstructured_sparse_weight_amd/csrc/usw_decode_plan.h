// Host side of the decode kernels (usw_decode_kernels.h): launch shapes,
// split factors, workspace sizes and launches, shared by the plain product
// and the products with an epilogue.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "usw.h"
#include "usw_decode_kernels.h"
#include "usw_internal.h"

namespace {

// Decode launch configurations (waves per workgroup, pipeline depth,
// minimum waves per SIMD), each the measured best on MI355X for its case.
using DefaultCfg = Cfg<4, 1, 4>;
// fp16 with five-chunk value slots: 96 VGPRs, so a fifth wave per SIMD fits
// (measured 2% faster than four on the 20480x5120 layer at N = 16).
using DefaultCfgLean = Cfg<4, 1, 5>;
// 17..32 columns of N: twice the accumulators and X fragments, which do not
// fit 128 registers; three waves per SIMD leave room for them.
using DefaultCfg2 = Cfg<4, 1, 3>;
// 33..64 columns of N in one pass (four token blocks): two waves per SIMD.
using DefaultCfg4 = Cfg<4, 1, 2>;
// 65..128 columns in one pass (five, six or eight token blocks; only the fused
// product: by expert there are tiles enough to fill the chip, and two smaller
// ones beat one of 128 rows, 8 experts of 4096x4096 with 100 rows each 91.6
// against 112.5 us): one wave per SIMD, whose 512 registers hold up to 128
// accumulators and two GroupTiles' X fragments.  Two passes rebuild the
// weight twice (MI355X, two passes / one: 4096x11008 N = 77 41.4 / 27.6 us,
// 8192x8192 N = 128 60.8 / 46.4).  Not faster at N = 77: three slots 2.6% behind,
// eight waves of half the columns equal there, spilling above 80 columns.
using DefaultCfg8 = Cfg<4, 1, 1>;
// INT4 values, up to 16 columns of N: a third of the fp16 slot registers
// (85 VGPRs), so a fifth wave per SIMD fits and hides more of the rebuild
// latency (measured 6% faster on the 20480x5120 layer at N = 2).
using DefaultCfgI4 = Cfg<4, 1, 5>;

struct CfgInfo {
  int waves;   // waves per workgroup
  int occ;     // waves per SIMD the configuration allows
};

CfgInfo cfg_info(int nchunk, bool i4, bool lean) {
  if (nchunk > 64) return CfgInfo{DefaultCfg8::kWavesPerGroup, DefaultCfg8::kOcc};
  if (nchunk > 32) return CfgInfo{DefaultCfg4::kWavesPerGroup, DefaultCfg4::kOcc};
  if (nchunk > 16) return CfgInfo{DefaultCfg2::kWavesPerGroup, DefaultCfg2::kOcc};
  if (i4) return CfgInfo{DefaultCfgI4::kWavesPerGroup, DefaultCfgI4::kOcc};
  return lean ? CfgInfo{DefaultCfgLean::kWavesPerGroup, DefaultCfgLean::kOcc}
              : CfgInfo{DefaultCfg::kWavesPerGroup, DefaultCfg::kOcc};
}

// Compute units of MI355X; the automatic split aims at one full round of
// resident workgroups on all of them.
constexpr int64_t kComputeUnits = 256;

struct Plan {
  int splits;     // workgroups per 64-row strip, passes of nchunk tokens
  int nchunk;     // columns of N per kernel pass (pass_chunk)
  int rsplits;    // the same for the last pass when it is shorter (N mod
  int rchunk;     // nchunk tokens in a pass of rchunk), else splits, 0
  int waves;      // waves per workgroup
  bool ring;      // the workgroup-cooperative kernel
};

// LDS slots of the workgroup-cooperative decode: two GroupTiles load while
// one is computed (measured on MI355X: 2 slots 2% slower, 4 slots, which
// leave room for four workgroups per compute unit instead of five, 24%
// slower).
constexpr int kRingDepth = 3;
// Fewest GroupTile columns the automatic split gives a ring workgroup.
constexpr int64_t kRingMinCols = 10;

// The argument structs with an epilogue carry Y's type themselves; it is a
// template argument where the kernel's sums go by it.
template <class A>
void ring_launch(const A& a, bool f16out, dim3 grid, hipStream_t s) {
  if constexpr (!ArgTraits<A>::kEpilogue) {
    if (!f16out) {
      decode_ring_kernel<kRingDepth, false, A><<<grid, kRingThreads, 0, s>>>(a);
      return;
    }
  }
  decode_ring_kernel<kRingDepth, true, A><<<grid, kRingThreads, 0, s>>>(a);
}

// Workgroups of the ring kernel resident per compute unit (registers, LDS).
template <class A>
int ring_resident() {
  int n = 0;
  const hipError_t e =
      hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_ring_kernel<kRingDepth, true, A>, kRingThreads, 0);
  return (e == hipSuccess && n > 0) ? n : 4;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Five 1 KB value chunks per slot when an fp16 matrix is at most 55% dense on
// average (a GroupTile then needs more than five only far in the tail; such
// a wave takes the two-half path), six otherwise.
bool lean_values(const usw_fmt* f, const usw::Geometry& g) {
  return f->val_type == USW_VAL_F16 &&
         static_cast<double>(f->nnz) <= 0.55 * static_cast<double>(g.M) * static_cast<double>(g.K);
}

// Pass size that n tokens take: 16, 32 or 64 tokens or, where passes may be
// as long, 80, 96 or 128.
int pass_chunk(int n, int longest) {
  const int c = n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : n <= 80 ? 80 : n <= 96 ? 96 : 128;
  return std::min(c, longest);
}

// Longest pass: a pass's rows of partial sums are addressed in 32 bits.
template <class A>
constexpr bool kTallPasses = ArgTraits<A>::kEpilogue && !ArgTraits<A>::kExperts;
template <class A>
int longest_pass(const usw::Geometry& g) {
  return kTallPasses<A> && g.M <= (int64_t(1) << 21) ? 128 : 64;
}

// Split factor of the per-wave decode kernel for passes of `chunk` tokens.
int wave_splits(const usw::Geometry& g, int chunk, int splits_req, bool i4, bool lean) {
  const CfgInfo ci = cfg_info(chunk, i4, lean);
  int64_t s = splits_req;
  if (s <= 0) {
    // About one round of resident workgroups (occ waves per SIMD, 4 SIMDs
    // per compute unit), each wave keeping at least 3 GroupTiles to stream.
    // Passes of 64 tokens and more on a matrix with at most one strip per compute
    // unit take as many workgroups as there are compute units, no more: the
    // split partial sums (64 x M fp32 per split, written and read back) then
    // cost more than the second workgroup per compute unit gains (measured
    // on MI355X at N = 64: 11008x4096 31.0 us with 1 split against 37.3 with
    // 3; 4096x11008 27.3 with 4 against 31.0 with 8; 15360x5120 38.1 with 1
    // against 44.5 with 2).
    const int64_t target = kComputeUnits * 4 * ci.occ / ci.waves;
    if (chunk >= 64 && g.Gr <= kComputeUnits)
      s = kComputeUnits / g.Gr;
    else
      s = std::max<int64_t>(1, (target + g.Gr / 2) / g.Gr);
    s = std::min<int64_t>(s, std::max<int64_t>(1, g.Gc / (ci.waves * 3)));
  }
  const int64_t smax = std::max<int64_t>(1, g.Gc / ci.waves);
  // Each wave caches its GroupTile offsets in one register: at most 63
  // GroupTiles per wave.
  const int64_t smin = (g.Gc + 63 * ci.waves - 1) / (63 * ci.waves);
  return static_cast<int>(std::max(smin, std::max<int64_t>(1, std::min(s, smax))));
}

template <class A = Args>
Plan make_plan(const usw::Geometry& g, int N, int splits_req, bool i4, bool lean) {
  Plan p;
  // More tokens than the longest pass: equal passes.
  const int longest = longest_pass<A>(g), passes = static_cast<int>((static_cast<int64_t>(N) + longest - 1) / longest);
  p.nchunk = pass_chunk(longest > 64 ? (N - 1) / passes + 1 : N, longest);
  p.rchunk = 0;
  p.ring = !i4 && lean && N <= 16;
  if (p.ring) {
    // One round of resident workgroups, each keeping at most 63 GroupTiles
    // and, when the matrix has few strips, at least kRingMinCols: a
    // workgroup fills and drains its ring over the first and last steps, so
    // shorter runs lose more to that than a full round gains (measured on
    // MI355X: 5120x5120 at N = 16 13.5 us with 8 splits against 15.5 us with
    // the 16 of a full round).  The factor is clamped to K/256 like the
    // other decode kernel's.
    p.waves = 5;
    static const int resident = ring_resident<A>();
    int64_t s = splits_req > 0 ? splits_req
                               : std::min<int64_t>((kComputeUnits * resident) / g.Gr,
                                                   std::max<int64_t>(1, g.Gc / kRingMinCols));
    const int64_t smax = std::max<int64_t>(1, g.Gc / 4);
    const int64_t smin = (g.Gc + 62) / 63;
    p.splits = static_cast<int>(std::max(smin, std::max<int64_t>(1, std::min(s, smax))));
    p.rsplits = p.splits;
    return p;
  }
  p.waves = cfg_info(p.nchunk, i4, lean).waves;
  p.splits = wave_splits(g, p.nchunk, splits_req, i4, lean);
  // A shorter last pass gets the split factor of its own size.
  const int rem = N > p.nchunk ? N % p.nchunk : 0;
  p.rchunk = rem > 0 ? pass_chunk(rem, longest) : 0;
  p.rsplits = rem > 0 ? wave_splits(g, p.rchunk, splits_req, i4, lean) : p.splits;
  return p;
}

usw_status check_common(const usw_fmt* f, int32_t y_type, int32_t N, usw::Geometry* g) {
  if (!f) return USW_ERR_NULL_ARG;
  usw_status st = usw::make_geometry(f->M, f->K, f->gt_m, f->gt_k, g);
  if (st) return st;
  if (f->val_type != USW_VAL_F16 && f->val_type != USW_VAL_I4) return USW_ERR_BAD_DTYPE;
  if (y_type != USW_OUT_F16 && y_type != USW_OUT_F32) return USW_ERR_BAD_DTYPE;
  if (N < 1) return USW_ERR_BAD_N;
  if (f->reserved != 0) return USW_ERR_BAD_SHAPE;
  if (f->gt_m != kGT || f->gt_k != kGT) return USW_ERR_UNSUPPORTED;
  if (f->nnz < 0 || f->nnz >= (int64_t(1) << 32)) return USW_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(N) * g->M > (int64_t(1) << 40)) return USW_ERR_BAD_SHAPE;
  return USW_OK;
}

// Workspace: per-strip counters (4 B each, padded to 256 B) then the fp32
// partial sums of every split.
size_t counters_bytes(const usw::Geometry& g) { return (static_cast<size_t>(4 * g.Gr) + 255) & ~size_t(255); }

// Partial sums of the largest pass: splits x tokens of the pass x M fp32.
size_t workspace_bytes(const usw::Geometry& g, const Plan& p) {
  const size_t full = p.splits > 1 ? static_cast<size_t>(p.splits) * p.nchunk : 0;
  const size_t last = p.rchunk > 0 && p.rsplits > 1 ? static_cast<size_t>(p.rsplits) * p.rchunk : 0;
  const size_t cols = std::max(full, last);
  if (cols == 0) return 0;
  return counters_bytes(g) + cols * g.M * sizeof(float);
}

template <int NB, bool I4, int CH, class C, class A>
void launch_cfg(const A& a, bool f16out, dim3 grid, hipStream_t s) {
  if constexpr (!ArgTraits<A>::kEpilogue || (I4 && NB == 1)) {
    if (!f16out) {
      decode_kernel<NB, I4, CH, false, C, A><<<grid, C::kThreadsPerGroup, 0, s>>>(a);
      return;
    }
  }
  decode_kernel<NB, I4, CH, true, C, A><<<grid, C::kThreadsPerGroup, 0, s>>>(a);
}

template <int NB, bool I4, int CH, class A>
void launch_decode(const A& a, bool f16out, dim3 grid, hipStream_t s) {
  if constexpr (NB > 4)
    launch_cfg<NB, I4, CH, DefaultCfg8>(a, f16out, grid, s);
  else if constexpr (NB == 4)
    launch_cfg<NB, I4, CH, DefaultCfg4>(a, f16out, grid, s);
  else if constexpr (NB == 2)
    launch_cfg<NB, I4, CH, DefaultCfg2>(a, f16out, grid, s);
  else if constexpr (I4)
    launch_cfg<NB, I4, CH, DefaultCfgI4>(a, f16out, grid, s);
  else if constexpr (CH == 5)
    launch_cfg<NB, I4, CH, DefaultCfgLean>(a, f16out, grid, s);
  else
    launch_cfg<NB, I4, CH, DefaultCfg>(a, f16out, grid, s);
}

// One pass of nb 16-token blocks (1, 2 or 4; the fused product 5, 6 or 8 too).
template <class A>
void launch_pass(const A& a, bool ring, bool i4, bool lean, int nb, bool f16out, dim3 grid, hipStream_t s) {
  if constexpr (kTallPasses<A>) {
    auto tall = [&](auto blocks) {
      constexpr int NB = decltype(blocks)::value;
      if (i4) launch_decode<NB, true, 3>(a, f16out, grid, s);
      else if (lean) launch_decode<NB, false, 5>(a, f16out, grid, s);
      else launch_decode<NB, false, 6>(a, f16out, grid, s);
    };
    if (nb == 5) return tall(std::integral_constant<int, 5>{});
    if (nb == 6) return tall(std::integral_constant<int, 6>{});
    if (nb == 8) return tall(std::integral_constant<int, 8>{});
  }
  if (ring) {
    ring_launch(a, f16out, grid, s);
  } else if (i4) {
    if (nb == 4) launch_decode<4, true, 3>(a, f16out, grid, s);
    else if (nb == 2) launch_decode<2, true, 3>(a, f16out, grid, s);
    else launch_decode<1, true, 3>(a, f16out, grid, s);
  } else if (lean) {
    if (nb == 4) launch_decode<4, false, 5>(a, f16out, grid, s);
    else if (nb == 2) launch_decode<2, false, 5>(a, f16out, grid, s);
    else launch_decode<1, false, 5>(a, f16out, grid, s);
  } else {
    if (nb == 4) launch_decode<4, false, 6>(a, f16out, grid, s);
    else if (nb == 2) launch_decode<2, false, 6>(a, f16out, grid, s);
    else launch_decode<1, false, 6>(a, f16out, grid, s);
  }
}

}  // namespace
