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

namespace {

using namespace usw_dev;

// ---------------------------------------------------------------------------
// Expansion
// ---------------------------------------------------------------------------

struct ExpandArgs {
  const uint64_t* __restrict__ bitmaps;
  const uint32_t* __restrict__ offsets;
  const uint8_t* __restrict__ values;
  const int64_t* __restrict__ starts;
  const int32_t* __restrict__ slots;
  u32x4_t* __restrict__ dense;   // [weight of the group][GroupTile][k half][4 fragments][64 lanes]
  int64_t values_total, ngt;
  int e0, S;
};

// Waits until at most N of this wave's loads are in flight, then the barrier.
template <int N>
__device__ __forceinline__ void ring_barrier() {
  static_assert(N == 2 || N == 4 || N == 8, "one case for each tiling");
  if constexpr (N == 2) USW_PRODUCER_BARRIER(2);
  else if constexpr (N == 4) USW_PRODUCER_BARRIER(4);
  else USW_PRODUCER_BARRIER(8);
}

constexpr int kExpandWaves = 4;

// Value bytes [v0, v0 + *alloc) of weight e, clamped to the buffer.
__device__ __forceinline__ int64_t value_range(const int64_t* starts, int64_t total, int e, uint64_t* alloc) {
  if (!starts) {
    *alloc = static_cast<uint64_t>(total);
    return 0;
  }
  const int64_t v0 = min(max(starts[e], int64_t(0)), total - 16) & ~int64_t(15);
  const int64_t v1 = min(max(starts[e + 1], v0 + 16), total);
  *alloc = static_cast<uint64_t>(v1 - v0) & ~uint64_t(15);
  return v0;
}

template <bool I4>
__global__ __launch_bounds__(64 * kExpandWaves) void expand_kernel(ExpandArgs a) {
  // A GroupTile's values span at most 8 KB (INT4 2 KB) and a partial first
  // piece of 16 bytes; they arrive in 1 KB loads.
  constexpr int kLoads = I4 ? 3 : 9;
  __shared__ __attribute__((aligned(16))) uint32_t lut[I4 ? 512 : 32];
  __shared__ __attribute__((aligned(16))) uint8_t vals[kExpandWaves][kLoads * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t tabs[kExpandWaves][kTabBytes];
  USW_LDS_POISON(vals);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = a.e0 + static_cast<int>(blockIdx.y);
  if (a.slots && min(a.slots[e + 1], a.S) <= max(a.slots[e], 0)) return;   // no rows read this weight (scan_runs)
  if constexpr (I4) {
    for (int i = tid; i < 256; i += 64 * kExpandWaves) reinterpret_cast<u32x2_t*>(lut)[i] = row_byte_selectors(i);
  } else if (tid < 16) {
    u32x2_t s;
    s.x = nibble_selector(tid, 0);
    s.y = nibble_selector(tid, 1);
    reinterpret_cast<u32x2_t*>(lut)[tid] = s;
  }
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kExpandWaves + w;
  uint64_t alloc;
  const uint8_t* values = a.values + value_range(a.starts, a.values_total, e, &alloc);
  const uint64_t top = alloc - 16;
  uint8_t* vb = vals[w];
  const LaneMap lm = lane_map(lane);
  if (g < a.ngt) {
    const uint32_t* off = a.offsets + (a.ngt + 1) * e + g;
    const uint32_t o0 = off[0], o1 = off[1];
    const u32x2_t bm = reinterpret_cast<const u32x2_t*>(a.bitmaps + (a.ngt * e + g) * kBtPerGt)[lane];
    const uint64_t a0 = min(chunk_start<I4>(o0), top);
    const uint32_t pieces = min(chunk_count<I4>(o1, a0), static_cast<uint32_t>(64 * kLoads));
    const uint32_t last = min(pieces > 0 ? pieces - 1 : 0u, static_cast<uint32_t>((top - a0) >> 4));
    const u32x4_t* src = reinterpret_cast<const u32x4_t*>(values + a0);
    for (uint32_t i = 0; 64 * i < pieces; ++i) lds_dma16(src + min(64 * i + lane, last), lds_addr(vb) + 1024 * i);
    tab_write(tabs[w], bm, bitmap_prefix_reg(bm) + chunk_delta<I4>(o0, a0), lane);
  }
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();
  if (g >= a.ngt) return;
  u32x4_t* out = a.dense + (static_cast<int64_t>(blockIdx.y) * a.ngt + g) * 512 + lane;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const u32x2_t t = *reinterpret_cast<const u32x2_t*>(tabs[w] + lm.tab + 256 * f + 128 * ks);
      const uint32_t rb = t.y + __builtin_popcount(t.x & lm.pmask);
      half8_t v = rebuild_row<I4>(vb, lut, rb, __builtin_amdgcn_ubfe(t.x, lm.sh, 8));
      if constexpr (I4) v -= static_cast<_Float16>(kCodeOffset);   // exact: codes and 72 + code are whole
      out[64 * (4 * ks + f)] = __builtin_bit_cast(u32x4_t, v);
    }
}

// ---------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------

// Fewest columns of a streaming workgroup's share: shorter ones cost more in
// partial sums than they save.
constexpr int kStreamMinCols = 16;

// A tile is BM outputs by BN rows: WM x WN waves of 16 MF outputs by 16 NF
// rows, and an LDS ring of RING half columns (32 k).  STREAM: the tiles are
// dealt to one workgroup per compute unit and the rest's columns shared;
// otherwise every tile, or equal share of its columns, is a workgroup.
template <int MF_, int NF_, int WM_, int WN_, int RING_, bool STREAM_>
struct Tiling {
  static constexpr int MF = MF_, NF = NF_, WM = WM_, WN = WN_;
  static constexpr bool kStream = STREAM_;
  static constexpr int W = WM * WN, kThreads = 64 * W;
  static constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
  static constexpr int kA = BM / 16, kB = BN / 16;      // 1 KB loads of a half column
  static constexpr int kLoads = (kA + kB) / W;           // of them a wave issues
  static constexpr int kPlace = 1024 * (kA + kB);        // a ring place
  static constexpr int kRing = RING_;
  static constexpr int kSlot = 4 * BM * BN;              // bytes of a tile's partial sums
  static_assert(kA % W == 0 && kB % W == 0, "every wave issues the same loads");
  static_assert(BM % 64 == 0 && 64 * BN * 4 <= kRing * kPlace, "the epilogue's stage fits the ring");
};

struct WideArgs {
  const u32x4_t* __restrict__ dense;
  const uint16_t* __restrict__ X;
  void* Y;
  const uint16_t* __restrict__ scales;
  const int32_t* __restrict__ slots;
  const int32_t* __restrict__ rows;
  float* __restrict__ part;
  uint32_t* __restrict__ counters;
  Epilogue e;
  int M, K, Gr, Gc, mt;   // mt: tiles of outputs
  int e0, e1, S, T, i4;
  int splits;
};

// The rows of an output tile: expert, its first slot and how many, and the
// tile's first strip.
struct WideTile {
  int e, strip0, row0, n;
};

// Inclusive maximum over the lanes up to this one (wave_inclusive_scan's steps).
__device__ __forceinline__ int wave_inclusive_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));   // row_shr:1, 2, 4, 8
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));   // row_bcast:15, 31
  return max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
}

// Scans the runs of the group's experts, 64 at a time: found(first expert,
// tiles before, this lane's tiles of rows, inclusive tiles up to this lane, its
// run) until it returns true.  Returns the tiles seen.
//
// An offset below one before it counts as that one, so whatever the array
// holds the runs are disjoint parts of [0, S) and make no more tiles than the
// host planned counters and partial sums for.
template <int BN, class Fn>
__device__ __forceinline__ int scan_runs(const WideArgs& a, int lane, Fn found) {
  int before = 0, top = 0;
  for (int b = a.e0; b < a.e1; b += 64) {
    const int e = min(b + lane, a.e1 - 1);
    int lo = 0, hi = a.S;
    if (a.slots) {
      lo = max(top, wave_inclusive_max(min(max(a.slots[e], 0), a.S)));
      hi = max(lo, min(a.slots[e + 1], a.S));
      top = __builtin_amdgcn_readlane(hi, 63);
    }
    if (b + lane >= a.e1) hi = lo;
    const uint32_t nt = static_cast<uint32_t>(hi - lo + BN - 1) / BN;
    const uint32_t incl = wave_inclusive_scan(nt * a.mt);
    if (found(b, before, nt, incl, lo, hi)) break;
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return before;
}

template <class C>
__device__ __forceinline__ WideTile wide_tile(const WideArgs& a, int t, int lane) {
  WideTile r{};
  scan_runs<C::BN>(a, lane, [&](int b, int before, uint32_t nt, uint32_t incl, int lo, int hi) {
    const uint64_t past = __ballot(before + static_cast<int>(incl) > t);
    if (!past) return false;
    const int l = __builtin_ctzll(past);
    const int ntl = __builtin_amdgcn_readlane(nt, l);
    int i = t - (before + static_cast<int>(__builtin_amdgcn_readlane(incl, l)) - ntl * a.mt);
    // Blocks of up to eight tiles of rows by all tiles of outputs, rows first.
    const int blk = i / (8 * a.mt);
    i -= blk * 8 * a.mt;
    const int wide = min(8, ntl - 8 * blk);
    const int m = i / wide, n = 8 * blk + (i - m * wide);
    r.e = b + l;
    r.strip0 = m * (C::BM / kGT);
    r.row0 = __builtin_amdgcn_readlane(lo, l) + n * C::BN;
    r.n = min(C::BN, __builtin_amdgcn_readlane(hi, l) - r.row0);
    return true;
  });
  return r;
}

// The kernel's arguments, read again from where the launch put them: what the
// epilogue needs is then loaded there and holds no register over the product.
typedef const __attribute__((address_space(4))) WideArgs* ArgsAgain;
__device__ __forceinline__ ArgsAgain args_again() {
  ArgsAgain p = (ArgsAgain)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// The epilogue of a tile.  The sums pass through LDS, 64 outputs by BN rows
// at a time, so that a row's 64 outputs are stored together; the 16-byte unit
// u of row n lies at u ^ (n % 16), which keeps writes and reads off each
// other's banks.  A thread stores the same four outputs of several rows, whose
// operands it loads while the sums arrive.  Rows and outputs past the tile's
// are cut by the bounds of the buffer accesses.
template <class C>
__device__ __forceinline__ void wide_finish(uint8_t* smem, const f32x4_t (&acc)[C::MF][C::NF], const WideTile& t,
                                            int wm, int wn, int me) {
  constexpr int MF = C::MF, NF = C::NF;
  constexpr int kStep = C::kThreads / 16, kRows = C::BN / kStep, kBatch = kRows < 8 ? kRows : 8;
  const ArgsAgain z = args_again();
  f32x4_t* stage = reinterpret_cast<f32x4_t*>(smem);
  auto unit = [](int n, int u) { return 16 * n + (u ^ (n & 15)); };
  const int m0 = t.strip0 * kGT, m_end = min(C::BM, z->M - m0);
  // A [rows][ld] operand of the tile from its first element on.
  auto tile_rsrc = [&](const void* p, int64_t ld, int size) {
    const uint8_t* at = static_cast<const uint8_t*>(p) + (t.row0 * ld + m0) * size;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(at), 0,
                                             static_cast<int>(((t.n - 1) * ld + m_end) * size), kBufferRsrcWord3);
  };
  const bool f16out = z->e.f16out, has_mul = z->e.mul != nullptr, has_res = z->e.res != nullptr;
  const int size = f16out ? 2 : 4, ld_mul = static_cast<int>(z->e.ld_mul), ld_res = static_cast<int>(z->e.ld_res);
  const auto ry = tile_rsrc(z->Y, z->M, size);
  const auto rmul = tile_rsrc(z->e.mul, ld_mul, 2), rres = tile_rsrc(z->e.res, ld_res, 2);
  const int act = z->e.act;
#pragma unroll 1
  for (int p = 0; p < C::BM / 64; ++p) {
    asm volatile("" : "+v"(me));
    const int u = me & 15, n0 = me >> 4;
    const int m = 64 * p + 4 * u;
    const bool mine = m < m_end;
    f32x4_t bias = {0.f, 0.f, 0.f, 0.f}, scale = {1.f, 1.f, 1.f, 1.f};
    const int64_t em = static_cast<int64_t>(z->M) * t.e + m0 + m;
    if (mine && z->e.bias) bias = load_half4(z->e.bias + em);
    if (mine && z->i4) scale = load_half4(z->scales + em);
    // Byte offset of row n0 + kStep j, past every bound for outputs that are not ours.
    auto at = [&](int j, int ld, int bytes) { return mine ? ((n0 + kStep * j) * ld + m) * bytes : 0x7FFFFFF0; };
    half4_t mul[kBatch], res[kBatch];
    auto operands = [&](int j0) {
      if (has_mul) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          mul[j] = __builtin_bit_cast(half4_t, __builtin_amdgcn_raw_buffer_load_b64(rmul, at(j0 + j, ld_mul, 2), 0, 0));
      }
      if (has_res) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          res[j] = __builtin_bit_cast(half4_t, __builtin_amdgcn_raw_buffer_load_b64(rres, at(j0 + j, ld_res, 2), 0, 0));
      }
    };
    operands(0);
    const int row = me & 15, kb = (me >> 4) & 3;
#pragma unroll
    for (int f = 0; f < MF; ++f)
      if ((MF * wm + f) / 4 == p) {
#pragma unroll
        for (int nb = 0; nb < NF; ++nb)
          stage[unit(16 * (NF * wn + nb) + row, (4 * (MF * wm + f) + kb) & 15)] = acc[f][nb];
      }
    __syncthreads();
    auto emit = [&](auto kind) {
#pragma unroll 1
      for (int j0 = 0; j0 < kRows; j0 += kBatch) {
        asm volatile("" : "+v"(me));
        if (j0 > 0) operands(j0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          f32x4_t v = stage[unit((me >> 4) + kStep * (j0 + j), me & 15)] * scale + bias;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = activation<decltype(kind)::value>(v[i]);
          if (has_mul) v *= to_float4(mul[j]);
          if (has_res) v += to_float4(res[j]);
          if (f16out)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_half4(v)), ry,
                                                  at(j0 + j, z->M, 2), 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), ry, at(j0 + j, z->M, 4), 0, 0);
        }
      }
    };
    switch (act) {
      case USW_ACT_RELU: emit(std::integral_constant<int, USW_ACT_RELU>{}); break;
      case USW_ACT_GELU: emit(std::integral_constant<int, USW_ACT_GELU>{}); break;
      case USW_ACT_GELU_TANH: emit(std::integral_constant<int, USW_ACT_GELU_TANH>{}); break;
      case USW_ACT_SILU: emit(std::integral_constant<int, USW_ACT_SILU>{}); break;
      default: emit(std::integral_constant<int, USW_ACT_NONE>{});
    }
    __syncthreads();
  }
}

template <class C>
__global__ __launch_bounds__(C::kThreads, 2) void wide_kernel(WideArgs a) {
  constexpr int MF = C::MF, NF = C::NF, W = C::W;
  // The ring: places of a half column (32 k) of both operands, kA KB of
  // weight fragments, then kB blocks of 16 rows of x, 64 bytes a row.
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::kRing * C::kPlace];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w % C::WM, wn = w / C::WM;
  const int row = lane & 15, kb = lane >> 4;

  // Workgroups are dealt to the 8 XCDs in turn; XCD i takes the i-th eighth
  // of the pieces or, streaming, is workgroups i P / 8 on, so that neighbours
  // share their operands in its L2.
  const int tiles = a.slots
                        ? scan_runs<C::BN>(a, lane, [](int, int, uint32_t, uint32_t, int, int) { return false; })
                        : static_cast<int>((static_cast<uint32_t>(a.S) + C::BN - 1) / C::BN) * a.mt;
  const int b = static_cast<int>(blockIdx.x);
  int L;
  // Streaming: R rounds of whole tiles; the U units (tile, column) from B on,
  // of the tiles left over, are shared evenly by Pr workgroups, this one's
  // being [r0, u1).
  int P = 0, R = 0, Pr = 0;
  int64_t B = 0, U = 0, r0 = 0, u1 = 0;
  const int64_t Gc = a.Gc;
  if constexpr (C::kStream) {
    P = static_cast<int>(gridDim.x);
    L = (b & 7) * (P >> 3) + (b >> 3);   // P is a multiple of 8
    R = tiles / P;
    B = static_cast<int64_t>(R) * P * Gc;
    U = static_cast<int64_t>(tiles - R * P) * Gc;
    Pr = min(P, max(tiles - R * P, static_cast<int>(U / kStreamMinCols)));
    if (L < Pr) {
      r0 = B + U * L / Pr;
      u1 = B + U * (L + 1) / Pr;
    }
  } else {
    const int pieces = tiles * a.splits;
    const int per = (pieces + 7) / 8;
    L = (b & 7) * per + (b >> 3);
    if ((b >> 3) >= per || L >= pieces) return;
  }
  // The shared pieces from the last to the first, so that the workgroups of a
  // tile start at both its ends and its sums are added while whole tiles still
  // run; then the whole tiles.
  for (int round = 0; !C::kStream || u1 > r0 || round < R;) {
  int tile, c_begin = 0, c_end = a.Gc, slot = L;
  bool shared;
  if constexpr (C::kStream) {
    if (u1 > r0) {
      tile = static_cast<int>((u1 - 1) / Gc);
      c_end = static_cast<int>(u1 - tile * Gc);
      c_begin = static_cast<int>(max(r0, tile * Gc) - tile * Gc);
      u1 = tile * Gc + c_begin;
      slot = 2 * L + (u1 == r0 ? 0 : 1);
    } else {
      tile = L + round * P;
      ++round;
    }
    shared = c_begin > 0 || c_end < a.Gc;
  } else {
    tile = L / a.splits;
    const int sidx = L - tile * a.splits;
    c_begin = static_cast<int>(Gc * sidx / a.splits);
    c_end = static_cast<int>(Gc * (sidx + 1) / a.splits);
    shared = a.splits > 1;
  }
  const WideTile t = wide_tile<C>(a, tile, lane);

  // This wave's loads of a half column: fragments w, w + W, ... of the weight
  // and blocks w, w + W, ... of x.  Lane 4 j + i of a block's load brings
  // piece (i - j / 4) mod 4 of row j, so piece q of row r lies at
  // (q + r / 4) mod 4 and the 16 rows of a fragment spread over all banks.
  const u32x4_t* wsrc[C::kA / W];
#pragma unroll
  for (int j = 0; j < C::kA / W; ++j) {
    const int i = w + W * j;
    const int strip = min(t.strip0 + (i >> 2), a.Gr - 1);
    wsrc[j] = a.dense + ((static_cast<int64_t>(t.e - a.e0) * a.Gr + strip) * a.Gc + c_begin) * 512 + 64 * (i & 3) + lane;
  }
  const uint16_t* xsrc[C::kB / W];
#pragma unroll
  for (int j = 0; j < C::kB / W; ++j) {
    const int s = t.row0 + min(16 * (w + W * j) + (lane >> 2), t.n - 1);
    const uint32_t xr = min(static_cast<uint32_t>(a.rows ? a.rows[s] : s), static_cast<uint32_t>(a.T - 1));
    xsrc[j] = a.X + static_cast<int64_t>(xr) * a.K + c_begin * kGT + 8 * ((lane - (lane >> 4)) & 3);
  }
  const uint32_t ldst = lds_addr(smem) + 1024 * w;
  const int H = 2 * (c_end - c_begin);   // half columns of the piece
  auto load = [&](int h, uint32_t place) {
#pragma unroll
    for (int j = 0; j < C::kA / W; ++j) lds_dma16(wsrc[j] + static_cast<int64_t>(h) * 256, ldst + place + 1024 * W * j);
#pragma unroll
    for (int j = 0; j < C::kB / W; ++j) lds_dma16(xsrc[j] + 32 * h, ldst + place + 1024 * (C::kA + W * j));
  };

  struct Frags {
    half8_t a[MF], b[NF];
  };
  const uint8_t* abase = smem + 1024 * MF * wm + 16 * lane;
  const uint8_t* bbase = smem + 1024 * (C::kA + NF * wn) + 64 * row + 16 * ((kb + (row >> 2)) & 3);
  auto read = [&](Frags& f, uint32_t place) {
#pragma unroll
    for (int nb = 0; nb < NF; ++nb) f.b[nb] = *reinterpret_cast<const half8_t*>(bbase + place + 1024 * nb);
#pragma unroll
    for (int i = 0; i < MF; ++i) f.a[i] = *reinterpret_cast<const half8_t*>(abase + place + 1024 * i);
  };
  f32x4_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // Half column h: its fragments are in registers; those of h + 1 are read
  // between its MFMAs, and the loads of h + kRing go into its own ring place,
  // whose reads ended before the last barrier.  At the barrier half h + 2 has
  // landed, with the loads of the kRing - 2 after it still in flight.
  uint32_t place = 0;   // of half column h
  auto half_column = [&](int h, const Frags& cur, Frags& nxt) {
    const bool more = h + C::kRing < H;
    if (more) load(h + C::kRing, place);
    place = place == (C::kRing - 1) * C::kPlace ? 0u : place + C::kPlace;
    read(nxt, place);
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int nb = 0; nb < NF; ++nb)
        acc[i][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(cur.a[i], cur.b[nb], acc[i][nb], 0, 0, 0);
    constexpr int kEach = MF * NF / (MF + NF);
#pragma unroll
    for (int i = 0; i < MF + NF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);       // one LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);   // MFMAs
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MF * NF - kEach * (MF + NF), 0);
    if (more) ring_barrier<(C::kRing - 2) * C::kLoads>();
    else USW_PRODUCER_BARRIER(0);
  };
#pragma unroll
  for (int h = 0; h < C::kRing; ++h)
    if (h < H) load(h, h * C::kPlace);
  if (H >= C::kRing) ring_barrier<(C::kRing - 2) * C::kLoads>();
  else USW_PRODUCER_BARRIER(0);
  Frags f0, f1;
  read(f0, 0);
  lds_barrier();   // every wave has read place 0, which half column 0 loads into
  for (int h = 0; h < H; h += 2) {
    half_column(h, f0, f1);
    half_column(h + 1, f1, f0);
  }

  // Lane l of block (f, nb): outputs 16 f + 4 (l / 16) + i, row 16 nb + l % 16
  // of the wave's tile.  The thread's number goes through an empty asm, here
  // and below: what is derived from it is computed where it is used and holds
  // no register over the product.
  int me = tid;
  asm volatile("" : "+v"(me));
  bool finish = true;
  if (shared) {
    // The pieces of a tile leave their accumulators in slots, in register
    // order, with stores that reach the level all XCDs share; the last to
    // finish adds them, every lane its own, in column order.  Streaming, the
    // owners of a tile are the workgroups p with B + U p / Pr <= t0 + Gc - 1
    // and B + U (p + 1) / Pr > t0, t0 its first unit, and a workgroup has a
    // slot for the piece that opens its range and one for that which closes it.
    const int64_t t0 = tile * Gc;
    int q0 = tile * a.splits, np = a.splits;
    if constexpr (C::kStream) {
      q0 = static_cast<int>(((t0 - B + 1) * Pr + U - 1) / U) - 1;
      np = static_cast<int>(((t0 - B + Gc) * Pr + U - 1) / U) - q0;
    }
    auto slot_rsrc = [&](int64_t i) {
      return __builtin_amdgcn_make_buffer_rsrc(a.part + i * (C::kSlot / 4), 0, C::kSlot, kBufferRsrcWord3);
    };
    auto slot_of = [&](int k) -> int64_t {
      const int64_t q = q0 + k;
      if constexpr (C::kStream) return 2 * q + (B + U * q / Pr >= t0 ? 0 : 1);
      else return q;
    };
    const int at = (w * MF * NF * 64 + (me & 63)) * 16;
    const auto own = slot_rsrc(slot);
#pragma unroll
    for (int i = 0; i < MF * NF; ++i)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[i / NF][i % NF]), own, at + 1024 * i, 0,
                                             kCacheSc1);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __syncthreads();
    if (tid == 0)
      last_flag = __hip_atomic_fetch_add(&a.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                  static_cast<uint32_t>(np - 1);
    __syncthreads();
    finish = last_flag != 0;
    __syncthreads();   // last_flag is read; the next piece may write it
    if (finish) {
      if (tid == 0) __hip_atomic_store(&a.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const auto first = slot_rsrc(slot_of(0));
#pragma unroll
      for (int i = 0; i < MF * NF; ++i)
        acc[i / NF][i % NF] =
            __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(first, at + 1024 * i, 0, kCacheSc1));
      constexpr int kBatch = MF * NF < 16 ? MF * NF : 16;
      for (int k = 1; k < np; ++k) {
        const auto r = slot_rsrc(slot_of(k));
#pragma unroll
        for (int i0 = 0; i0 < MF * NF; i0 += kBatch) {
          f32x4_t v[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            v[i] = __builtin_bit_cast(f32x4_t,
                                      __builtin_amdgcn_raw_buffer_load_b128(r, at + 1024 * (i0 + i), 0, kCacheSc1));
#pragma unroll
          for (int i = 0; i < kBatch; ++i) acc[(i0 + i) / NF][(i0 + i) % NF] += v[i];
        }
      }
    }
  }
  if (finish) wide_finish<C>(smem, acc, t, wm, wn, me);
  if constexpr (!C::kStream) return;
  }
}

using Large = Tiling<8, 4, 2, 4, 4, true>;     // 256 x 256, eight waves, one workgroup per compute unit
using Medium = Tiling<4, 4, 2, 2, 3, false>;   // 128 x 128
using Small = Tiling<2, 2, 2, 2, 3, false>;    // 64 x 64

constexpr int kBM[3] = {Large::BM, Medium::BM, Small::BM};
constexpr int kBN[3] = {Large::BN, Medium::BN, Small::BN};
constexpr int64_t kComputeUnits = 256;

// Dense fragments held at a time: weights beyond this are expanded and
// multiplied in groups, each with its own pair of launches.
constexpr int64_t kDenseBytes = int64_t(1) << 30;

}  // namespace

namespace usw {

WidePlan wide_plan(const Geometry& g, int32_t E, int32_t S) {
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
  p.tiling = rounds > 0 && large_us < medium_us ? 0 : g.M * g.K * S <= 4000000000ll ? 2 : 1;
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
  a.dense = x.dense;
  a.X = c.X;
  a.Y = c.Y;
  a.scales = c.scales;
  a.slots = c.slots;
  a.rows = c.rows;
  a.part = reinterpret_cast<float*>(w + p.slots_at);
  a.counters = reinterpret_cast<uint32_t*>(w);
  a.e = c.e;
  a.M = static_cast<int>(g.M);
  a.K = static_cast<int>(g.K);
  a.Gr = static_cast<int>(g.Gr);
  a.Gc = static_cast<int>(g.Gc);
  a.mt = static_cast<int>((g.M + kBM[p.tiling] - 1) / kBM[p.tiling]);
  a.S = c.S;
  a.T = c.T;
  a.i4 = c.val_type == USW_VAL_I4;
  a.splits = p.splits;
  if (p.tiles * p.splits >= (int64_t(1) << 31) || g.ngt / kExpandWaves >= (int64_t(1) << 31) - 1) return USW_ERR_UNSUPPORTED;
  const unsigned gx = static_cast<unsigned>((g.ngt + kExpandWaves - 1) / kExpandWaves);
  const int64_t blocks = p.tiling == 0 ? kComputeUnits : (p.tiles * p.splits + 7) / 8 * 8;
  const dim3 wgrid(static_cast<unsigned>(blocks));
  for (int e0 = 0; e0 < c.E; e0 += p.group) {
    const int e1 = std::min(c.E, e0 + p.group);
    x.e0 = a.e0 = e0;
    a.e1 = e1;
    const dim3 grid(gx, static_cast<unsigned>(e1 - e0));
    if (a.i4) expand_kernel<true><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    else expand_kernel<false><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    if (p.tiling == 0) wide_kernel<Large><<<wgrid, Large::kThreads, 0, s>>>(a);
    else if (p.tiling == 1) wide_kernel<Medium><<<wgrid, Medium::kThreads, 0, s>>>(a);
    else wide_kernel<Small><<<wgrid, Small::kThreads, 0, s>>>(a);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

}  // namespace usw
