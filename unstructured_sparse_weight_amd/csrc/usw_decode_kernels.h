// The bitmap SpMM decode kernels for gfx950, shared by the plain product
// (usw_spmm.hip) and the products with an epilogue, of one weight or grouped by
// expert (usw_fused.hip).
//
// What is computed: Y[n][m] = sum_k W_sp[m][k] X[n][k], W_sp held in the
// TCA-BME bitmap format (blog "SpInfer: How bitmaps make sparse LLMs actually
// fast", section "How TCA-BME addresses the indexing overhead").  Values are
// located by masked popcount (same blog, "Shared Memory Bitmap Decoding").
//
// Two kernels: decode_ring_kernel (fp16 values, N <= 16, matrices at most
// 55% dense), in which a workgroup's waves share each GroupTile through an
// LDS ring filled by a loader wave (described where it is defined), and
// decode_kernel (everything else in decode), described here.  They share
// the rebuild and the split-K epilogue.
//
// Design of decode_kernel (gfx950, wave64):
//   * One workgroup owns one 64-row strip of GroupTiles (64x64) and a range
//     of GroupTile columns; each of its waves streams its own contiguous run
//     of GroupTiles (bitmaps and values of consecutive GroupTiles of a strip
//     are contiguous in memory), so the main loop has no workgroup barrier.
//   * Loads run one GroupTile ahead of the compute: the 16-byte global loads
//     of GroupTile c+1 (bitmaps, the value range [offsets[g], offsets[g+1])
//     from a 16-byte aligned start, and the X^T fragments) sit in registers
//     while GroupTile c, already copied into the wave's private LDS buffer,
//     is rebuilt and multiplied.  Every load is issued unconditionally
//     (clamped indices), so the compiler waits for exactly the slot in use.
//   * Rebuild: v_mfma_f32_16x16x32_f16 gives lane l 8 consecutive columns
//     8*(l/16)..+7 of one row of a 16x32 block, which is exactly one row of
//     one BitmapTile; its kept values are contiguous in the stream.  A
//     fragment is one TCTile row (16 strip rows) by four BitmapTile columns,
//     so the 32 lanes the LDS serves together read rows of a single TCTile,
//     whose values are contiguous (few bank conflicts).  Where each
//     BitmapTile's values start (GroupTile offset + a DPP wave prefix scan of
//     the BitmapTile popcounts) goes with its bitmap words into a small LDS
//     table one GroupTile ahead; a lane reads its row's word and base, adds
//     the popcount of the earlier rows, and expands the row into 8 slots with
//     two aligned LDS windows and v_perm_b32 byte selectors looked up by the
//     row's 4-bit halves (zero for clear bits).
//   * The rebuilt fragment meets the X^T fragment (X is [N][K], so each
//     lane's 8 k values are one 16-byte load) on the matrix cores with fp32
//     accumulation, which leaves the vector ALUs to the rebuild.
//   * Partial sums of the waves of a workgroup are added in LDS in a fixed
//     order.  Split K (several workgroups per strip): each writes its sums to
//     an fp32 workspace with device-coherent stores and the last workgroup of
//     the strip, found with a per-strip counter, adds them in split order, so
//     results do not depend on scheduling.

#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "usw_device.h"
#include "usw_decode_common.h"
#include "usw_epilogue.h"

namespace {

using namespace usw_dev;

// ---------------------------------------------------------------------------
// Arguments of the products with an epilogue, of one weight or by expert
// ---------------------------------------------------------------------------
//
// The kernels below are templates over their argument struct: Args is the
// plain product, FusedArgs adds an epilogue, ExpertArgs runs E weights of one
// shape, each on its own run of rows (slots), with the same epilogue.

template <class A>
struct ArgTraits {
  static constexpr bool kEpilogue = false, kExperts = false;
};

struct FusedArgs : Args {
  Epilogue e;
};
template <>
struct ArgTraits<FusedArgs> {
  static constexpr bool kEpilogue = true, kExperts = false;
};

// A tile is up to 1 << lg_chunk consecutive slots of one expert.  The grid
// has room for the most tiles that S slots over E experts can make; which
// expert and slots tile t is, every workgroup finds from slots[E+1], so the
// runs never have to reach the host.  Workgroups past the last tile leave at
// once.
struct ExpertArgs : FusedArgs {
  const int32_t* __restrict__ slots;    // [E+1] first slot of each expert
  const int32_t* __restrict__ rows;     // [S] row of X of each slot, or null: slot s reads row s
  const int64_t* __restrict__ starts;   // [E+1] byte offset of each expert's values
  int64_t values_total;                 // bytes of all experts' values
  int64_t nbt, noff;                    // bitmap words and offsets of one expert
  int E, S, T, lg_chunk, Gr;
};
template <>
struct ArgTraits<ExpertArgs> {
  static constexpr bool kEpilogue = true, kExperts = true;
};

// Moves a's pointers to tile t: its expert's weight, bias and scales, its
// slots' rows of Y and of the epilogue's operands, its counters and partial
// sums.  Returns the tile's first slot, or -1 past the last tile.  Runs are
// clamped to [0, S) and values to the buffer, whatever the arrays hold.
__device__ __forceinline__ int expert_tile(ExpertArgs& a, int t, int lane) {
  int e = -1, row0 = 0, n = 0;
  for (int e0 = 0, before = 0; e0 < a.E; e0 += 64) {
    const int i = min(e0 + lane, a.E - 1);
    const int lo = min(max(a.slots[i], 0), a.S);
    const int hi = e0 + lane < a.E ? min(max(a.slots[i + 1], lo), a.S) : lo;
    const uint32_t mine = (static_cast<uint32_t>(hi - lo) + (1u << a.lg_chunk) - 1u) >> a.lg_chunk;
    const uint32_t incl = wave_inclusive_scan(mine);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (t < before + total) {
      const uint64_t past = __ballot(before + static_cast<int>(incl) > t);
      const int l = __builtin_ctzll(past);
      const int first = before + __builtin_amdgcn_readlane(incl - mine, l);
      e = e0 + l;
      row0 = __builtin_amdgcn_readlane(lo, l) + ((t - first) << a.lg_chunk);
      n = min(1 << a.lg_chunk, __builtin_amdgcn_readlane(hi, l) - row0);
      break;
    }
    before += total;
  }
  if (e < 0) return -1;
  a.bitmaps += a.nbt * e;
  a.offsets += a.noff * e;
  const int64_t v0 = min(max(a.starts[e], int64_t(0)), a.values_total - 16) & ~int64_t(15);
  const int64_t v1 = min(max(a.starts[e + 1], v0 + 16), a.values_total);
  a.values += v0;
  a.values_alloc = static_cast<uint64_t>(v1 - v0) & ~uint64_t(15);
  if (a.scales) a.scales += static_cast<int64_t>(a.M) * e;
  if (a.e.bias) a.e.bias += static_cast<int64_t>(a.M) * e;
  if (a.e.mul) a.e.mul += a.e.ld_mul * row0;
  if (a.e.res) a.e.res += a.e.ld_res * row0;
  a.Y = static_cast<uint8_t*>(a.Y) + static_cast<int64_t>(row0) * a.M * (a.e.f16out ? 2 : 4);
  if (a.splits > 1) {
    a.part += static_cast<int64_t>(row0) * a.M;
    a.counters += static_cast<int64_t>(t) * a.Gr;
  }
  a.N = n;
  return row0;
}

// The row of X that token n of the pass (n clamped to the pass) reads.
template <class A>
__device__ __forceinline__ int x_row(const A& a, int n, int row0) {
  n = min(n, a.N - 1);
  if constexpr (ArgTraits<A>::kExperts) {
    const int s = row0 + n;
    return min(static_cast<uint32_t>(a.rows ? a.rows[s] : s), static_cast<uint32_t>(a.T - 1));
  } else {
    return n;
  }
}

// finish_strip with an epilogue: writes a strip's finished sums through the
// epilogue to Y or, with split K, to split sidx's partial sums, which the
// strip's last workgroup adds in split order and finishes, AHEAD splits' loads
// in flight.
template <int NB, bool I4, int AHEAD, class A, class SumFn>
__device__ __forceinline__ void finish_strip_fused(const A& a, int gi, int sidx, int nthreads, uint32_t& last_flag,
                                                   SumFn sum_of) {
  const int tid = threadIdx.x;
  const int m0 = gi * kGT;
  auto store_y4 = [&](int n, int ml, f32x4_t v) {
    if constexpr (I4) v *= load_half4(a.scales + m0 + ml);
    epilogue_store4(a.e, a.Y, a.M, n, m0 + ml, v);
  };
  // Partial sums of split s: [rows][M] fp32, a row for every token of the
  // call (by expert: every slot), of which this pass owns a.N.
  auto part_rsrc = [&](int s) {
    int64_t rows = a.N;
    if constexpr (ArgTraits<A>::kExperts) rows = a.S;
    return __builtin_amdgcn_make_buffer_rsrc(a.part + s * rows * a.M, 0, a.N * a.M * 4, kBufferRsrcWord3);
  };
  for (int e = tid; e < 16 * 16 * NB; e += nthreads) {
    const int n = e >> 4;
    const int ml = 4 * (e & 15);
    if (n >= a.N) continue;
    const f32x4_t sum = sum_of(n, ml);
    if (a.splits > 1)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, sum), part_rsrc(sidx),
                                             (n * a.M + m0 + ml) * 4, 0, kCacheSc1);
    else
      store_y4(n, ml, sum);
  }
  if (a.splits <= 1) return;

  // As in finish_strip: partial stores complete before the count, and the
  // last workgroup reads them past its own caches.
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (tid == 0)
    last_flag = __hip_atomic_fetch_add(&a.counters[gi], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                static_cast<uint32_t>(a.splits - 1);
  __syncthreads();
  if (!last_flag) return;
  // Every output of a thread at once (of eight token blocks, half), so that
  // one round trip brings AHEAD splits of all of them (MI355X, 4096x11008 N =
  // 77: the last workgroup takes 3.7 us one output after another, 1.9 together).
  constexpr int kEach = NB == 8 ? 4 : NB;
  for (int e0 = tid; e0 < 16 * a.N; e0 += kEach * nthreads) {
    f32x4_t sum[kEach];
    int off[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = e0 + i * nthreads;
      sum[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      off[i] = e < 16 * a.N ? ((e >> 4) * a.M + m0 + 4 * (e & 15)) * 4 : 0x7FFFFFF0;   // past the bound: zeros
    }
    for (int p0 = 0; p0 < a.splits; p0 += AHEAD) {
      f32x4_t v[AHEAD][kEach];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (p0 + j < a.splits) {
          const auto r = part_rsrc(p0 + j);
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            v[j][i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off[i], 0, kCacheSc1));
        }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (p0 + j < a.splits) {
#pragma unroll
          for (int i = 0; i < kEach; ++i) sum[i] += v[j][i];
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = e0 + i * nthreads;
      if (e < 16 * a.N) store_y4(e >> 4, 4 * (e & 15), sum[i]);
    }
  }
  if (tid == 0) __hip_atomic_store(&a.counters[gi], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Which strip and split a workgroup takes.  Workgroups are dealt to the 8
// XCDs round robin; with remap the splits of one strip land on the same XCD
// (one L2 for their partial sums).  By expert the workgroups of a tile are
// spread over all XCDs, so that the empty tiles at the grid's end idle none.
// Returns false for a workgroup with no tile; row0 is its tile's first slot.
template <class A>
__device__ __forceinline__ bool locate(A& a, int lane, int* gi, int* sidx, int* row0) {
  int nblk = static_cast<int>(gridDim.x);
  int b = static_cast<int>(blockIdx.x);
  *row0 = 0;
  if constexpr (ArgTraits<A>::kExperts) {
    nblk = a.Gr * a.splits;
    const int t = b / nblk;
    b -= t * nblk;
    *row0 = expert_tile(a, t, lane);
    if (*row0 < 0) return false;
  }
  const int L = a.remap ? (b & 7) * (nblk >> 3) + (b >> 3) : b;
  *gi = L / a.splits;
  *sidx = L - *gi * a.splits;
  return true;
}

// Value slot constants: CH 1 KB chunks per GroupTile, i.e. 64 lanes x 16 B
// per chunk.  fp16 takes 5 chunks (GroupTiles up to ~62% dense) when the
// matrix is at most 55% dense on average, else 6 (~74%); INT4 takes 3, which
// every GroupTile fits (<= 2 KB + head).  Denser GroupTiles are staged in two
// halves of two TCTile rows each (<= 4 KB + head).  Every chunk load is
// issued unconditionally, so the loads carry no branches and the compiler
// waits for exactly the slot being consumed.
template <bool I4, int CH>
struct ValTraits {
  static constexpr int kChunks = CH;
  // LDS value buffer per wave: one slot plus the <16 B a window reads past
  // the last value.
  static constexpr int kVbuf = CH * 1024 + 64;
  static constexpr uint32_t kFastLimit = I4 ? 4096u : (16u * 64u * CH - 32u) / 2u;   // values per GroupTile
  static_assert(I4 || kVbuf >= 16 * 257 + 16, "a half GroupTile fits");
  static_assert(!I4 || kFastLimit / 2 + 16 <= 1024 * CH, "every INT4 GroupTile fits");
};

// Registers holding one GroupTile's loads until they are copied into LDS.
template <int NB, bool I4, int CH>
struct Slot {
  u32x4_t v[CH];
  u32x2_t bm;       // lane t: bitmap word t of the GroupTile
  u32x4_t x[2][NB];
  uint32_t nch;     // 16-byte pieces of values spanned (wave-uniform)
  uint32_t delta;   // value elements before the GroupTile's first one in its first piece
  uint64_t a0;      // byte offset of the first piece
};


// Issue the loads of GroupTile c of strip gi, whose values occupy elements
// [o0, o1) of the stream.
template <int NB, bool I4, int CH, class A>
__device__ __forceinline__ void slot_load(Slot<NB, I4, CH>& s, const A& a, int gi, int c, int lane, uint32_t o0,
                                          uint32_t o1, const int (&xrow)[NB]) {
  using VT = ValTraits<I4, CH>;
  const int64_t g = static_cast<int64_t>(gi) * a.Gc + c;
  // Bitmaps first: the bitmap table of a slot is written while its values
  // and X^T fragments may still be in flight.
  s.bm = reinterpret_cast<const u32x2_t*>(a.bitmaps + g * kBtPerGt)[lane];
  // The clamps keep every load inside the padded allocation and every store
  // inside the LDS buffer even for offsets that disagree with the bitmaps.
  const uint64_t top = a.values_alloc - 16;
  s.a0 = min(chunk_start<I4>(o0), top);
  s.delta = chunk_delta<I4>(o0, s.a0);
  s.nch = min(chunk_count<I4>(o1, s.a0), static_cast<uint32_t>((VT::kVbuf - 16) / 16));
  // The values go through buffer resources, one per chunk, that end after
  // the GroupTile's last piece (piece 0 of an empty GroupTile lies inside the
  // padded allocation): pieces past it read as zero, with no clamp per piece
  // and one vector offset (the lane's) for all chunks.
  const uint32_t last = min(s.nch > 0 ? s.nch - 1 : 0u, static_cast<uint32_t>((top - s.a0) >> 4));
  const int span = static_cast<int>(16 * (last + 1));
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.values + s.a0 + 1024 * i), 0,
                                                        max(span - 1024 * i, 0), kBufferRsrcWord3);
    s.v[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc, 16 * lane, 0, 0));
  }
  // X^T fragments.  Columns n >= N of B only feed columns n >= N of the
  // product, which are never stored, so those lanes just repeat row N-1.
  const int row = lane & 15, kb = lane >> 4;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      int n = min(nb * 16 + row, a.N - 1);
      if constexpr (ArgTraits<A>::kExperts) n = xrow[nb];
      s.x[ks][nb] = *reinterpret_cast<const u32x4_t*>(a.X + static_cast<size_t>(n) * a.K + c * kGT + ks * 32 + kb * 8);
    }
}

template <int NB, bool I4, int CH>
__device__ __forceinline__ void slot_commit(const Slot<NB, I4, CH>& s, uint8_t* vb, int lane) {
#pragma unroll
  for (int i = 0; i < CH; ++i) reinterpret_cast<u32x4_t*>(vb)[lane + 64 * i] = s.v[i];
}

// Which rows a lane rebuilds.  Fragment (f, ks) of a GroupTile (f = 0..3,
// ks = 0, 1) is the 16 x 32 block of strip rows 16f .. 16f+15 and GroupTile
// columns 32ks .. 32ks+31.  Lane l with i = l % 16 and g = l / 16 holds row i,
// columns 8g .. 8g+7 of the block, which is row r = i % 8 of the BitmapTile
// in BitmapTile row R = 2f + i / 8 and BitmapTile column C = 4ks + g.  The
// 32 lanes that the LDS serves together (g = 0, 1 or g = 2, 3) thus read the
// rows of one TCTile, whose values are contiguous, so their windows spread
// over few bytes and few bank conflicts; and D row i of fragment f is strip
// row 16f + i.
struct LaneMap {
  uint32_t tab;     // byte offset of the lane's entry for f = ks = 0 in the bitmap table
  uint32_t sh;      // 8 (r % 4): bit offset of row r in its bitmap word
  uint32_t pmask;   // bits of the rows before r in that word
};

__device__ __forceinline__ LaneMap lane_map(int lane) {
  const int i = lane & 15, g = lane >> 4, r = i & 7;
  // BitmapTile (R, C) is number 16 (R / 2) + 4 (C / 2) + 2 (R % 2) + C % 2 in
  // storage order (TCTiles row-major, BitmapTiles row-major inside them);
  // fragment (f, ks) adds 16 f + 8 ks to the BitmapTile number below.
  const int bt = 4 * (g >> 1) + 2 * (i >> 3) + (g & 1);
  LaneMap m;
  m.tab = 16u * static_cast<uint32_t>(bt) + 8u * static_cast<uint32_t>(r >> 2);
  m.sh = 8u * static_cast<uint32_t>(r & 3);
  m.pmask = (1u << m.sh) - 1u;
  return m;
}

constexpr int kTabBytes = 16 * kBtPerGt;

// Bitmap table of a GroupTile in LDS, 16 bytes per BitmapTile, written by
// lane t for BitmapTile t: bitmap rows 0-3, where row 0's values start,
// bitmap rows 4-7, where row 4's values start (value positions counted in
// elements from the start of the staging area).  base is where the
// BitmapTile's values start.
__device__ __forceinline__ void tab_write(uint8_t* tab, u32x2_t bm, uint32_t base, int lane) {
  u32x4_t e;
  e.x = bm.x;
  e.y = base;
  e.z = bm.y;
  e.w = base + __builtin_popcount(bm.x);
  reinterpret_cast<u32x4_t*>(tab)[lane] = e;
}

// Exclusive prefix of the BitmapTile popcounts of a GroupTile from the
// slot's registers (lane t holds bitmap word t).
__device__ __forceinline__ uint32_t bitmap_prefix_reg(u32x2_t bm) {
  const uint32_t pc = __builtin_popcount(bm.x) + __builtin_popcount(bm.y);
  return wave_inclusive_scan(pc) - pc;
}

// How a product of INT4 codes loses the offset that its expanded rows carry
// (code_offset_collect).  The plain product collects the offset's share of the
// sums and takes it out at the end: its sums then round at the scale of
// 72 sum|x| over all of a wave's columns, which grows with them where x is all
// positive, as a ReLU leaves it (512x20480 in one split, 100 rows: 4.6e-4 of
// the output off, an fp16 output's own rounding 2.1e-4; fp32 outputs 4e-6 with
// x of both signs).  The products with an epilogue keep the sums at the scale
// of the codes:
//   kEach: four packed subtractions take it out of every slot, exactly (INT4
//     5120x20480 N = 64: 44.9 us collected, 39.8 so; N = 128: 71.4 / 68.1;
//     N = 24: 30.8 / 30.4; the subtractions serve all token blocks).
//   kStep: one token block with fp16 output, where the subtractions would cost
//     2 to 6% and the matrix cores idle: a product with the offset's negative
//     goes into the same accumulator before each step's own, so no more than
//     72 sum|x| of one step of 32 columns is ever in it: an x leaves at most
//     72 2^-24 |x| = 4e-6 |x| for each rounding of its step, in units where its
//     codes are whole numbers (20480x5120 N = 8: 19.3 us collected, 19.8 so,
//     20.4 by subtractions; 11008x4096 N = 16: 15.7 / 15.9 / 16.4).
enum class CodeOffset { kCollect, kEach, kStep };

// Rebuild and multiply fragments f = F0 .. F1-1 (both ks) of a GroupTile
// whose bitmap table is at tab and whose values are in the LDS staging area
// starting at vals.  INT4 rows carry the expansion's offset: corr collects
// its correction (code_offset_collect, all four fragments of a GroupTile at
// once) unless OFFSET takes it out here.
template <int NB, bool I4, int F0 = 0, int F1 = 4, CodeOffset OFFSET = CodeOffset::kCollect>
__device__ __forceinline__ void tile_mma(const u32x4_t (&x)[2][NB], const uint8_t* vals, const uint8_t* tab,
                                         const uint32_t* lut, f32x4_t (&acc)[4][NB], f32x4_t (&corr)[NB],
                                         const LaneMap& lm) {
  static_assert(!I4 || (F0 == 0 && F1 == 4), "the INT4 correction covers whole GroupTiles");
  if constexpr (I4 && OFFSET == CodeOffset::kCollect) code_offset_collect<NB>(corr, x);
  u32x2_t e[F1 - F0][2];
#pragma unroll
  for (int f = F0; f < F1; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      e[f - F0][ks] = *reinterpret_cast<const u32x2_t*>(tab + lm.tab + 256 * f + 128 * ks);
#pragma unroll
  for (int f = F0; f < F1; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint32_t word = e[f - F0][ks].x;
      const uint32_t rb = e[f - F0][ks].y + __builtin_popcount(word & lm.pmask);
      half8_t a = rebuild_row<I4>(vals, lut, rb, __builtin_amdgcn_ubfe(word, lm.sh, 8));
      if constexpr (I4 && OFFSET == CodeOffset::kEach) a -= static_cast<_Float16>(kCodeOffset);
      if constexpr (I4 && OFFSET == CodeOffset::kStep) {
        const _Float16 m = static_cast<_Float16>(-kCodeOffset);
        const half8_t neg = {m, m, m, m, m, m, m, m};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          acc[f][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(neg, __builtin_bit_cast(half8_t, x[ks][nb]), acc[f][nb],
                                                              0, 0, 0);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        acc[f][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(half8_t, x[ks][nb]), acc[f][nb], 0,
                                                            0, 0);
    }
}

// Launch shape of the decode kernel: waves per workgroup, GroupTiles loaded
// ahead of the one being computed (1 or 2), and the minimum waves per SIMD
// the register allocation must allow.
template <int WAVES_, int DEPTH_, int OCC_>
struct Cfg {
  static constexpr int kWavesPerGroup = WAVES_;
  static constexpr int kDepth = DEPTH_;
  static constexpr int kOcc = OCC_;
  static constexpr int kThreadsPerGroup = 64 * WAVES_;
};

template <int NB, bool I4, int CH, bool OUT_F16, class C, class A = Args>
__global__ __launch_bounds__(C::kThreadsPerGroup, C::kOcc) void decode_kernel(A a) {
  using VT = ValTraits<I4, CH>;
  constexpr int kW = C::kWavesPerGroup;
  constexpr int kThreads = C::kThreadsPerGroup;
  constexpr int kD = C::kDepth;
  constexpr CodeOffset kOffset = !ArgTraits<A>::kEpilogue ? CodeOffset::kCollect
                                 : OUT_F16 && NB == 1     ? CodeOffset::kStep
                                                          : CodeOffset::kEach;
  constexpr bool kCollected = I4 && kOffset == CodeOffset::kCollect;
  // Row selectors: fp16 16 nibble entries of two dwords, INT4 256 byte
  // entries of two dwords.
  __shared__ __attribute__((aligned(16))) uint32_t lut[I4 ? 512 : 32];
  // Staging (per wave: values, then the bitmap table); reused for the final
  // reduction.
  constexpr int kStage = kW * (VT::kVbuf + kTabBytes);
  constexpr int kRed = kW * 4 * NB * 64 * 4 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kStage > kRed ? kStage : kRed];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  // The wave index is uniform across the wave; saying so keeps the wave's
  // GroupTile range, its offsets and the loop control scalar.
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int gi, sidx, row0;
  if (!locate(a, lane, &gi, &sidx, &row0)) return;
  int xrow[NB] = {};
  if constexpr (ArgTraits<A>::kExperts) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) xrow[nb] = x_row(a, nb * 16 + (lane & 15), row0);
  }

  if (tid < 16) {
    if constexpr (!I4) {
      u32x2_t e;
      e.x = nibble_selector(tid, 0);
      e.y = nibble_selector(tid, 1);
      reinterpret_cast<u32x2_t*>(lut)[tid] = e;
    }
  }
  if constexpr (I4) {
    for (int i = tid; i < 256; i += kThreads) reinterpret_cast<u32x2_t*>(lut)[i] = row_byte_selectors(i);
  }
  __syncthreads();

  // Columns of GroupTiles this wave streams.
  const int parts = a.splits * kW;
  const int q = sidx * kW + w;
  const int c_begin = static_cast<int>(static_cast<int64_t>(a.Gc) * q / parts);
  const int c_end = static_cast<int>(static_cast<int64_t>(a.Gc) * (q + 1) / parts);

  const LaneMap lm = lane_map(lane);

  f32x4_t acc[4][NB];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  f32x4_t corr[NB];   // INT4: the expansion offset's correction, same for every row
#pragma unroll
  for (int j = 0; j < NB; ++j) corr[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  uint8_t* vb = smem + w * VT::kVbuf;
  uint8_t* tab = smem + kW * VT::kVbuf + w * kTabBytes;
  // The rebuild addresses the wave's value buffer from smem: its offset, in
  // value elements, is folded into the BitmapTile bases.
  const uint32_t vb_elems = I4 ? static_cast<uint32_t>(w * VT::kVbuf * 2) : static_cast<uint32_t>(w * VT::kVbuf / 2);

  // The wave's GroupTile offsets, one per lane: lane i holds
  // offsets[g_begin + i] for i <= count (the host keeps count <= 63), so a
  // slot's value range comes from two v_readlane.
  const int cnt = c_end - c_begin;
  const int64_t g_begin = static_cast<int64_t>(gi) * a.Gc + c_begin;
  const uint32_t ov = a.offsets[g_begin + min(lane, max(cnt, 0))];
  auto off_at = [&](int c) -> uint32_t { return __builtin_amdgcn_readlane(ov, min(c - c_begin, 63)); };

  // A wave may own no GroupTile column (K < 64 * waves): it only joins the
  // reduction.  A GroupTile whose values span more chunks than a slot holds
  // (fp16 density above ~74%) sends the whole wave down the unpipelined path.
  const uint32_t ov_next = __shfl_down(ov, 1);
  const uint32_t widest = wave_max(lane < cnt ? ov_next - ov : 0u);

  // The bitmap table of the GroupTile in slot s.
  auto write_tab = [&](const Slot<NB, I4, CH>& s) {
    tab_write(tab, s.bm, bitmap_prefix_reg(s.bm) + s.delta + vb_elems, lane);
  };

  if (cnt <= 0) {
    // nothing to stream
  } else if (widest > VT::kFastLimit) {
    if constexpr (!I4) {
      // Unpipelined: per GroupTile, the values of TCTile rows 0-1 (fragments
      // f = 0, 1), then those of TCTile rows 2-3 (f = 2, 3), each staged in
      // the wave's buffer with its own bitmap table bases.
      const uint64_t top = a.values_alloc - 16;
      for (int c = c_begin; c < c_end; ++c) {
        const uint32_t o0 = off_at(c), o1 = off_at(c + 1);
        Slot<NB, I4, CH> s0;
        slot_load(s0, a, gi, c, lane, o0, o1, xrow);
        const uint32_t excl = bitmap_prefix_reg(s0.bm);
        const uint32_t mid = __builtin_amdgcn_readlane(excl, 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hs = o0 + (h ? mid : 0u);
          const uint32_t he = h ? o1 : o0 + mid;
          const uint64_t a0 = min(chunk_start<I4>(hs), top);
          const uint32_t delta = chunk_delta<I4>(hs, a0);
          const uint32_t nch = min(chunk_count<I4>(he, a0), static_cast<uint32_t>((VT::kVbuf - 16) / 16));
          const uint32_t last = static_cast<uint32_t>((top - a0) >> 4);
          const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.values + a0);
          for (uint32_t ch = lane; ch < nch; ch += 64) reinterpret_cast<u32x4_t*>(vb)[ch] = src[min(ch, last)];
          // Entries of the other half get bases that are never read.
          tab_write(tab, s0.bm, excl - (h ? mid : 0u) + delta + vb_elems, lane);
          wave_sync();
          if (h == 0)
            tile_mma<NB, I4, 0, 2>(s0.x, smem, tab, lut, acc, corr, lm);
          else
            tile_mma<NB, I4, 2, 4>(s0.x, smem, tab, lut, acc, corr, lm);
          wave_sync();
        }
      }
    }
  } else if constexpr (kD == 0) {
    // One register slot: GroupTile c is copied into LDS, then the loads of
    // c+1 are issued into the same registers while c is rebuilt and
    // multiplied.  Fewer registers, more waves per SIMD.
    const int c_last = c_end - 1;
    Slot<NB, I4, CH> s0;
    slot_load(s0, a, gi, c_begin, lane, off_at(c_begin), off_at(c_begin + 1), xrow);
    write_tab(s0);
    for (int c = c_begin; c < c_end; ++c) {
      slot_commit(s0, vb, lane);
      u32x4_t xc[2][NB];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) xc[ks][nb] = s0.x[ks][nb];
      const int cn = min(c + 1, c_last);
      slot_load(s0, a, gi, cn, lane, off_at(cn), off_at(cn + 1), xrow);
      wave_sync();
      tile_mma<NB, I4, 0, 4, kOffset>(xc, smem, tab, lut, acc, corr, lm);
      wave_sync();
      write_tab(s0);
    }
  } else {
    // kD + 1 register slots: GroupTile c is in LDS while c+1 .. c+kD load.
    // Loads past the wave's last GroupTile repeat it (every wave here owns at
    // least one), so each step issues the same loads and waits for exactly
    // one slot.  A step issues the loads of c+kD before it waits for c, and
    // ends by writing the bitmap table of c+1 (the bitmaps are the first
    // load of a slot, long arrived by then).
    constexpr int kS = kD + 1;
    const int c_last = c_end - 1;
    auto load = [&](Slot<NB, I4, CH>& sl, int c) {
      const int cc = min(c, c_last);
      slot_load(sl, a, gi, cc, lane, off_at(cc), off_at(cc + 1), xrow);
    };
    Slot<NB, I4, CH> s[kS];
#pragma unroll
    for (int j = 0; j < kD; ++j) load(s[j], c_begin + j);
    write_tab(s[0]);
    // The loads go out at a raised wave priority, so a wave that reaches
    // them is not held behind the other waves' rebuild work (measured on
    // MI355X: INT4 20480x5120 N = 2 19.5 -> 19.0 us, N = 32 41.4 -> 40.1,
    // 11008x4096 N = 64 30.7 -> 28.3).
    auto step = [&](Slot<NB, I4, CH>& cur, int c, Slot<NB, I4, CH>& nxt, const Slot<NB, I4, CH>& after) {
      __builtin_amdgcn_s_setprio(2);
      load(nxt, c + kD);
      __builtin_amdgcn_s_setprio(0);
      slot_commit(cur, vb, lane);
      wave_sync();
      tile_mma<NB, I4, 0, 4, kOffset>(cur.x, smem, tab, lut, acc, corr, lm);
      wave_sync();
      write_tab(after);
    };
    int c = c_begin;
    for (; c + kS <= c_end; c += kS) {
#pragma unroll
      for (int j = 0; j < kS; ++j) step(s[j], c + j, s[(j + kD) % kS], s[(j + 1) % kS]);
    }
#pragma unroll
    for (int j = 0; j < kD; ++j)
      if (c + j < c_end) step(s[j], c + j, s[(j + kD) % kS], s[(j + 1) % kS]);
  }

  // Workgroup reduction over waves (fixed order).
  if constexpr (kCollected) code_offset_finish<NB>(corr);
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);   // [waves][4][NB][64 lanes][4]
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      *reinterpret_cast<f32x4_t*>(red + (((w * 4 + f) * NB + nb) * 64 + lane) * 4) =
          kCollected ? acc[f][nb] + corr[nb] : acc[f][nb];
  __syncthreads();

  auto sum_of = [&](int n, int ml) {
    // Strip rows ml .. ml+3 are D rows 4g .. 4g+3 (g = (ml / 4) % 4) of
    // fragment ml / 16: registers 0-3 of lane 16 g + n % 16.
    const int f = ml >> 4;
    const int ln = 16 * ((ml >> 2) & 3) + (n & 15);
    const int nb = n >> 4;
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ww = 0; ww < kW; ++ww)
      sum += *reinterpret_cast<const f32x4_t*>(red + (((ww * 4 + f) * NB + nb) * 64 + ln) * 4);
    return sum;
  };
  if constexpr (ArgTraits<A>::kEpilogue)
    finish_strip_fused<NB, I4, NB == 1 ? 8 : 4>(a, gi, sidx, kThreads, last_flag, sum_of);
  else
    finish_strip<NB, I4, OUT_F16>(a, gi, sidx, kThreads, last_flag, sum_of);
}

// ---------------------------------------------------------------------------
// Workgroup-cooperative decode: fp16 values, N <= 16, matrices at most 55%
// dense on average
// ---------------------------------------------------------------------------
//
// One workgroup is four compute waves and two loader waves over one strip's
// range of GroupTile columns; all six pass one barrier per GroupTile.
//  * Wave 4 moves each GroupTile's values and X^T column, and the bitmap
//    words of the GroupTile after, straight into a ring of R LDS slots with
//    global_load_lds_dwordx4, R - 1 GroupTiles ahead, so no register holds
//    them in flight.  It waits for its own loads with explicit vmcnt counts
//    before each barrier.
//  * Wave 5 writes the bitmap table of the next GroupTile into its slot.
//  * Compute wave q (0-3) rebuilds fragments f = 2 (q / 2) and 2 (q / 2) + 1
//    for ks = q % 2: two rows per lane per GroupTile, and multiplies them
//    with its X^T fragment, which wave 4 also stages in the slot.  The MFMA B
//    layout puts a different token in each of four consecutive lanes, so as
//    a global load every compute wave's fragment would cost four times the
//    address-unit cycles of a contiguous one; the compute waves issue no
//    global loads at all.
// A workgroup whose range holds a GroupTile too wide for a slot runs the
// range unpipelined, half a GroupTile (two TCTile rows) at a time in slot 0.

constexpr int kRingVals = 5 * 1024 + 64;                 // value bytes per slot
constexpr int kRingX = 2048;                             // X^T of one GroupTile column, 16 tokens
constexpr int kRingSlot = kRingVals + 512 + kTabBytes + kRingX;   // + bitmap words, table, X^T
constexpr uint32_t kRingPieces = 5 * 64;                 // 16-byte value pieces a slot takes
constexpr uint32_t kRingFast = (16u * kRingPieces - 32u) / 2u;   // values per GroupTile that fit a slot
constexpr int kRingThreads = 384;
static_assert(kRingSlot % 16 == 0, "slots keep 16-byte alignment");
static_assert(16 * kRingPieces + 16 <= kRingVals, "windows past the last piece stay in the slot");

template <int R, bool OUT_F16, class A = Args>
__global__ __launch_bounds__(kRingThreads, 5) void decode_ring_kernel(A a) {
  constexpr int NB = 1;
  constexpr int kRed = 2 * 4 * 64 * 16;          // [ks][f][64 lanes][4] fp32
  constexpr int kRing = R * kRingSlot;
  __shared__ __attribute__((aligned(16))) uint32_t lut[32];
  __shared__ __attribute__((aligned(16))) uint8_t smem[kRing > kRed ? kRing : kRed];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int gi, sidx, row0;
  if (!locate(a, lane, &gi, &sidx, &row0)) return;
  // By expert: the row of X that the loader's lane brings in for token lane / 4.
  int xrow = 0;
  if constexpr (ArgTraits<A>::kExperts) xrow = x_row(a, lane >> 2, row0);

  if (tid < 16) {
    u32x2_t e;
    e.x = nibble_selector(tid, 0);
    e.y = nibble_selector(tid, 1);
    reinterpret_cast<u32x2_t*>(lut)[tid] = e;
  }
  __syncthreads();

  // The workgroup's GroupTile columns (the host keeps 1 <= count <= 63) and
  // their offsets, lane i holding offsets[g_begin + i].
  const int c_begin = static_cast<int>(static_cast<int64_t>(a.Gc) * sidx / a.splits);
  const int c_end = static_cast<int>(static_cast<int64_t>(a.Gc) * (sidx + 1) / a.splits);
  const int cnt = c_end - c_begin;
  const int64_t g_begin = static_cast<int64_t>(gi) * a.Gc + c_begin;
  const uint32_t ov = a.offsets[g_begin + min(lane, cnt)];
  auto off_at = [&](int c) -> uint32_t { return __builtin_amdgcn_readlane(ov, min(c - c_begin, 63)); };
  // The shuffle runs in all lanes (a lane reading an inactive one gets 0).
  const uint32_t ov_next = __shfl_down(ov, 1);
  const uint32_t widest = wave_max(lane < cnt ? ov_next - ov : 0u);

  const int role = w < 4 ? 0 : w - 3;   // 0 compute, 1 loads, 2 bitmap tables
  const uint64_t top = a.values_alloc - 16;
  auto slot_vals = [&](int s) { return smem + s * kRingSlot; };
  auto slot_bm = [&](int s) { return smem + s * kRingSlot + kRingVals; };
  auto slot_tab = [&](int s) { return smem + s * kRingSlot + kRingVals + 512; };
  auto slot_x = [&](int s) { return smem + s * kRingSlot + kRingVals + 512 + kTabBytes; };

  // Loader: the bitmap words of GroupTile c (lanes 0-31, 16 bytes each) into
  // slot s; one load.
  auto issue_bm = [&](int c, int s) {
    const int64_t g = static_cast<int64_t>(gi) * a.Gc + c;
    if (lane < 32) lds_dma16_tracked(a.bitmaps + g * kBtPerGt + 2 * lane, slot_bm(s));
  };
  // Loader: value elements [e0, e1) into slot s, from the 16-byte piece
  // holding e0 on; returns the number of loads (1 KB each).  Pieces past the
  // range repeat its last one, and the range is cut to what a slot takes.
  auto issue_vals = [&](uint32_t e0, uint32_t e1, int s) -> int {
    const uint64_t a0 = min(chunk_start<false>(e0), top);
    const uint32_t pieces = min(chunk_count<false>(e1, a0), kRingPieces);
    const uint32_t last = min(pieces > 0 ? pieces - 1 : 0u, static_cast<uint32_t>((top - a0) >> 4));
    const int nl = static_cast<int>((pieces + 63) / 64);
    const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.values + a0);
    for (int i = 0; i < nl; ++i) lds_dma16_tracked(src + min(64u * i + lane, last), slot_vals(s) + 1024 * i);
    return nl;
  };
  // Loader: X^T of GroupTile column c (16 tokens x 64 k) into slot s, two
  // loads of 1 KB, one per k half.  Four consecutive lanes read one token's
  // 64 contiguous bytes of the half (one address-unit cycle, where the MFMA
  // B layout would take four); their pieces are rotated by token / 4 so that
  // the compute waves' 16-lane reads of B fragments fall in 16 different
  // bank groups.  Lane 4j + t holds piece (t - j/4) mod 4 of token j.
  auto issue_x = [&](int c, int s) {
    const int j = lane >> 2, t = lane & 3;
    const int piece = (t - (j >> 2)) & 3;
    int n = min(j, a.N - 1);
    if constexpr (ArgTraits<A>::kExperts) n = xrow;
    const uint16_t* src = a.X + static_cast<size_t>(n) * a.K + c * kGT + piece * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) lds_dma16_tracked(src + 32 * i, slot_x(s) + 1024 * i);
  };
  // The bitmap table of the value range starting at element e0 whose bitmaps
  // are in slot s; `skip` values of the GroupTile precede the range.  Its LDS
  // accesses are asm, so that in the wave that issues the LDS-DMA loads they
  // do not wait for those in flight.
  auto build_tab = [&](uint32_t e0, uint32_t skip, int s) {
    const u32x2_t bm = lds_load_b64(lds_addr(slot_bm(s)) + 8 * lane);
    const uint64_t a0 = min(chunk_start<false>(e0), top);
    const uint32_t base = bitmap_prefix_reg(bm) - skip + chunk_delta<false>(e0, a0) + (s * kRingSlot) / 2;
    u32x4_t e;
    e.x = bm.x;
    e.y = base;
    e.z = bm.y;
    e.w = base + __builtin_popcount(bm.x);
    lds_store_b128(lds_addr(slot_tab(s)) + 16 * lane, e);
  };

  // Compute waves.
  const int ks = w & 1;
  const int f0 = 2 * (w >> 1);
  const LaneMap lm = lane_map(lane);
  const uint32_t toff = lm.tab + 256u * f0 + 128u * ks;
  f32x4_t acc[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
  // The lane's B fragment (token n = lane % 16, k group g = lane / 16 of half
  // ks) in a slot's X^T area: position 4n + (g + n/4) mod 4 of the half.
  const uint32_t xoff = 1024u * ks + 16u * (4 * (lane & 15) + (((lane >> 4) + ((lane & 15) >> 2)) & 3));
  auto compute = [&](int s) {
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(slot_x(s) + xoff);
    const uint8_t* tab = slot_tab(s);
    u32x2_t e[2];
    e[0] = *reinterpret_cast<const u32x2_t*>(tab + toff);
    e[1] = *reinterpret_cast<const u32x2_t*>(tab + toff + 256);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t rb = e[j].y + __builtin_popcount(e[j].x & lm.pmask);
      const half8_t av = rebuild_row<false>(smem, lut, rb, __builtin_amdgcn_ubfe(e[j].x, lm.sh, 8));
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, __builtin_bit_cast(half8_t, x), acc[j], 0, 0, 0);
    }
  };

  // The offsets load completes here, before the loader's first LDS-DMA: the
  // compiler does not count those, so a later wait for it would wait for
  // them too.
  asm volatile("" : : "v"(ov));
  if constexpr (ArgTraits<A>::kExperts) asm volatile("" : : "v"(xrow));
  // The roles are separate uniform paths (a branch taken by the whole wave).
  // Lowered as a divergent branch, one role's code would follow another's,
  // and the compute waves' LDS reads would wait for the loader's LDS-DMA
  // loads.  All pass the same number of barriers: two before the first
  // GroupTile, then one per GroupTile (four per GroupTile unpipelined).
  const bool fast = widest <= kRingFast;
  const int rl = __builtin_amdgcn_readfirstlane(role);
  if (rl == 1) {
    // The two loader waves run at a higher wave priority than the compute
    // waves: a step ends only when their loads are issued and their tables
    // written, so their instructions go first when several waves of a SIMD
    // are ready (measured on MI355X: 27.8 against 28.9 us on 20480x5120,
    // N = 16).
    __builtin_amdgcn_s_setprio(3);
    if (fast) {
      // Step c issues the values and X^T of c+R-1 and the bitmaps of c+R,
      // then waits until those issued R-2 steps before (values and X^T of
      // c+1, bitmaps of c+2) have landed.  pend[j]: loads issued by step
      // c-R+2+j.
      auto step_loads = [&](int c) -> int {
        const int sv = (c + R - 1 - c_begin) % R;
        int n = 0;
#ifdef USW_DEBUG
        // The areas this step loads into hold NaNs until the loads land:
        // slot sv's values and X^T, the next slot's bitmap words.
        auto poison = [&](uint8_t* p, int bytes) {
          const u32x4_t v = {kLdsPoison, kLdsPoison, kLdsPoison, kLdsPoison};
          for (int off = 16 * lane; off < bytes; off += 1024) lds_store_b128(lds_addr(p) + off, v);
        };
        if (c + R - 1 < c_end) {
          poison(slot_vals(sv), kRingVals);
          poison(slot_x(sv), kRingX);
        }
        if (c + R < c_end) poison(slot_bm(sv == R - 1 ? 0 : sv + 1), 512);
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
#endif
        if (c + R - 1 < c_end) {
          issue_x(c + R - 1, sv);
          n += 2 + issue_vals(off_at(c + R - 1), off_at(c + R), sv);
        }
        if (c + R < c_end) {
          issue_bm(c + R, sv == R - 1 ? 0 : sv + 1);
          ++n;
        }
        return n;
      };
      // Before the first GroupTile: the bitmaps of c_begin, then steps
      // c_begin-R+1 .. c_begin-1.
      issue_bm(c_begin, 0);
      int pend[R - 1];
#pragma unroll
      for (int j = 0; j < R - 1; ++j) pend[j] = step_loads(c_begin - R + 1 + j);
      int later = 0;
#pragma unroll
      for (int j = 0; j < R - 1; ++j) later += pend[j];
      wait_vm(later);                              // bitmaps of c_begin
      lds_barrier();
      later -= pend[0];
      wait_vm(later);                              // values and X^T of c_begin, bitmaps of c_begin+1
      lds_barrier();
      for (int c = c_begin; c < c_end; ++c) {
#pragma unroll
        for (int j = 0; j < R - 2; ++j) pend[j] = pend[j + 1];
        pend[R - 2] = step_loads(c);
        later = 0;
#pragma unroll
        for (int j = 1; j < R - 1; ++j) later += pend[j];
        wait_vm(later);                            // values and X^T of c+1, bitmaps of c+2
        lds_barrier();
      }
    } else {
      // Unpipelined: per GroupTile, its bitmaps, then the values of TCTile
      // rows 0-1 and of rows 2-3 in turn (each at most 4 KB + head), all in
      // slot 0; two barriers per half.
      lds_barrier();
      lds_barrier();
      for (int c = c_begin; c < c_end; ++c) {
        const uint32_t o0 = off_at(c), o1 = off_at(c + 1);
        issue_bm(c, 0);
        wait_vm(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x2_t bm = lds_load_b64(lds_addr(slot_bm(0)) + 8 * lane);
          const uint32_t mid = __builtin_amdgcn_readlane(bitmap_prefix_reg(bm), 32);
          const uint32_t hs = o0 + (h ? mid : 0u);
          if (h == 0) issue_x(c, 0);
          issue_vals(hs, h ? o1 : o0 + mid, 0);
          wait_vm(0);
          build_tab(hs, h ? mid : 0u, 0);
          lds_barrier();
          lds_barrier();
        }
      }
    }
  } else if (rl == 2) {
    __builtin_amdgcn_s_setprio(3);
    // The bitmap table of c+1 (its bitmaps landed before the barrier that
    // opened step c) goes into its slot during step c.
    lds_barrier();
    if (fast) build_tab(off_at(c_begin), 0, 0);
    lds_barrier();
    if (fast) {
      for (int c = c_begin; c < c_end; ++c) {
        if (c + 1 < c_end) build_tab(off_at(c + 1), 0, (c + 1 - c_begin) % R);
        lds_barrier();
      }
    } else {
      for (int c = c_begin; c < c_end; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lds_barrier();
          lds_barrier();
        }
    }
  } else {
    lds_barrier();
    lds_barrier();
    if (fast) {
      int s = 0;
      for (int c = c_begin; c < c_end; ++c) {
        compute(s);
        s = s + 1 == R ? 0 : s + 1;
        lds_barrier();
      }
    } else {
      for (int c = c_begin; c < c_end; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lds_barrier();
          if (f0 == 2 * h) compute(0);
          lds_barrier();
        }
      }
    }
  }

  // Sum the two k halves of every fragment (fixed order) and finish.
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  if (role == 0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<f32x4_t*>(red + ((ks * 4 + f0 + j) * 64 + lane) * 4) = acc[j];
  }
  __syncthreads();
  auto sum_of = [&](int n, int ml) {
    const int f = ml >> 4;
    const int ln = 16 * ((ml >> 2) & 3) + (n & 15);
    return *reinterpret_cast<const f32x4_t*>(red + (f * 64 + ln) * 4) +
           *reinterpret_cast<const f32x4_t*>(red + ((4 + f) * 64 + ln) * 4);
  };
  if constexpr (ArgTraits<A>::kEpilogue)
    finish_strip_fused<NB, false, 4>(a, gi, sidx, kRingThreads, last_flag, sum_of);
  else
    finish_strip<NB, false, OUT_F16>(a, gi, sidx, kRingThreads, last_flag, sum_of);
}

}  // namespace
