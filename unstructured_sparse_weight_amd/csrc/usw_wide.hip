// The product with an epilogue for many rows per weight, in two steps:
//
//  1. expand_kernel rebuilds the weight's GroupTiles into dense fp16 matrix-
//     core fragments in the workspace, once per call (INT4: the codes; the row
//     scales go into the epilogue).  A wave takes a GroupTile, as in decode;
//     it is bound by the bytes it writes, 2 per element.
//  2. wide_kernel multiplies them: tiles of 256 outputs by 256 rows, eight
//     waves of 128 x 64 each, fp32 accumulators in registers, both operands
//     through LDS by LDS-DMA a GroupTile column ahead.
//
// Rebuilding inside the product instead costs LDS time on every column for
// every tile of rows, and LDS is what bounds the product: per column a wave
// reads 16 KB of weight and 8 KB of x fragments for 64 MFMAs of 16 cycles,
// 0.75 of the matrix time at 128 B a cycle, before any rebuild.
//
// Fragments in the workspace are in the order a wave reads them (1 KB each),
// so their copies to LDS and the reads from it are contiguous.  Rows of x are
// copied as they lie (eight lanes per 128-byte piece of a row, gathered rows
// alike), the 16-byte pieces of row r rotated by xor with (r / 2) % 8, which
// spreads a fragment's 16 rows over all banks.
//
// Work split: the tiles are dealt to one workgroup per compute unit, whole
// rounds of tiles first; the GroupTile columns of the tiles left over are
// split evenly (a tile may then be shared by workgroups, which leave fp32
// partial sums; the last to finish adds them in column order, so results do
// not depend on timing).  Consecutive tiles are up to eight tiles of rows by
// the weight's strips, so the 32 workgroups of an XCD share both operands in
// its L2.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

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
  if (a.slots && min(a.slots[e + 1], a.S) <= max(a.slots[e], 0)) return;   // no rows read this weight
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

constexpr int kWideM = 256, kWideN = 256;
constexpr int kWideThreads = 512;
constexpr int kWideSlot = kWideM * kWideN;   // fp32 partial sums of a tile
constexpr int64_t kComputeUnits = 256;
// Fewest GroupTile columns of a split tile's piece: shorter ones cost more in
// partial sums than the workgroup's share of the columns.
constexpr int kWideMinCols = 16;

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
  int remap;
};

// The rows of an output tile: expert, its first slot and how many, and the
// tile's first strip.
struct WideTile {
  int e, strip0, row0, n;
};

__device__ __forceinline__ void run_of(const WideArgs& a, int e, int* lo, int* hi) {
  if (!a.slots) {
    *lo = 0;
    *hi = a.S;
    return;
  }
  *lo = min(max(a.slots[e], 0), a.S);
  *hi = min(max(a.slots[e + 1], *lo), a.S);
}

// Tiles of the group's experts before expert lane e, and their number: every
// wave scans the runs, 64 experts at a time.
template <class Fn>
__device__ __forceinline__ int scan_runs(const WideArgs& a, int lane, Fn found) {
  int before = 0;
  for (int b = a.e0; b < a.e1; b += 64) {
    const int e = min(b + lane, a.e1 - 1);
    int lo, hi;
    run_of(a, e, &lo, &hi);
    if (b + lane >= a.e1) hi = lo;
    const uint32_t nt = static_cast<uint32_t>(hi - lo + kWideN - 1) / kWideN;
    const uint32_t incl = wave_inclusive_scan(nt * a.mt);
    if (found(b, before, nt, incl, lo, hi)) return before;
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return before;
}

__device__ __forceinline__ WideTile wide_tile(const WideArgs& a, int t, int lane) {
  WideTile r{};
  scan_runs(a, lane, [&](int b, int before, uint32_t nt, uint32_t incl, int lo, int hi) {
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
    r.strip0 = m * (kWideM / kGT);
    const int row0 = __builtin_amdgcn_readlane(lo, l) + n * kWideN;
    r.row0 = row0;
    r.n = min(kWideN, __builtin_amdgcn_readlane(hi, l) - row0);
    return true;
  });
  return r;
}

__global__ __launch_bounds__(kWideThreads, 2) void wide_kernel(WideArgs a) {
  // A ring of four half columns (32 k) of both operands, each 16 KB of A
  // (4 strips x 4 fragments x 1 KB) and 16 KB of B (256 rows x 64 B).
  __shared__ __attribute__((aligned(16))) uint8_t smem[4][32768];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w & 1, wn = w >> 1;
  const int row = lane & 15, kb = lane >> 4;
  const int P = static_cast<int>(gridDim.x);
  const int b = static_cast<int>(blockIdx.x);
  const int L = a.remap ? (b & 7) * (P >> 3) + (b >> 3) : b;
  const int64_t Gc = a.Gc;

  const int tiles = a.slots ? scan_runs(a, lane, [](int, int, uint32_t, uint32_t, int, int) { return false; })
                            : (a.S + kWideN - 1) / kWideN * a.mt;
  const int R = tiles / P;
  const int64_t B = static_cast<int64_t>(R) * P * Gc;          // units (tile, column) of the whole rounds
  const int64_t U = static_cast<int64_t>(tiles - R * P) * Gc;  // units of the tiles left over
  const int64_t Pr = min(static_cast<int64_t>(P), max(int64_t(1), U / kWideMinCols));   // workgroups that share them
  int64_t r0 = 0, r1 = 0;
  if (L < Pr) {
    r0 = B + U * L / Pr;
    r1 = B + U * (L + 1) / Pr;
  }

  // Stores four sums: row n of the tile, outputs m .. m+3.
  auto store4 = [&](const WideTile& t, int n, int m, f32x4_t v) {
    if (n >= t.n || m >= a.M) return;
    if (a.i4) v *= load_half4(a.scales + static_cast<int64_t>(a.M) * t.e + m);
    Epilogue e = a.e;
    if (e.bias) e.bias += static_cast<int64_t>(a.M) * t.e;
    epilogue_store4(e, a.Y, a.M, static_cast<int64_t>(t.row0) + n, m, v);
  };

  // The pieces of the shared range from the last to the first, so that the
  // workgroups of a tile start at both its ends and its sums are added while
  // whole tiles still run; then the whole tiles.
  int64_t u1 = r1;
  for (int r = 0; u1 > r0 || r < R;) {
    int tile, c_begin = 0, c_end = a.Gc;
    if (u1 > r0) {
      tile = static_cast<int>((u1 - 1) / Gc);
      c_end = static_cast<int>(u1 - tile * Gc);
      c_begin = static_cast<int>(max(r0, tile * Gc) - tile * Gc);
      u1 = tile * Gc + c_begin;
    } else {
      tile = L + r * P;
      ++r;
    }
    const WideTile t = wide_tile(a, tile, lane);
    const int64_t t0 = tile * Gc;
    const bool full = c_begin == 0 && c_end == a.Gc;

    // This wave's share of a half column: two fragments and two blocks of 16
    // rows of x, 1 KB a load.  Lane 4 j + i of a block's load brings piece
    // (i - j / 4) mod 4 of row j, so piece q of row r lies at (q + r / 4) mod 4
    // and the 16 rows of a fragment spread over all banks.
    const int strip = min(t.strip0 + (w >> 1), a.Gr - 1);
    const u32x4_t* wsrc = a.dense + ((static_cast<int64_t>(t.e - a.e0) * a.Gr + strip) * Gc + c_begin) * 512 + 128 * (w & 1) + lane;
    const uint16_t* xsrc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = t.row0 + min(16 * (2 * w + j) + (lane >> 2), t.n - 1);
      const uint32_t xr = min(static_cast<uint32_t>(a.rows ? a.rows[s] : s), static_cast<uint32_t>(a.T - 1));
      xsrc[j] = a.X + static_cast<int64_t>(xr) * a.K + c_begin * kGT + 8 * ((lane - (lane >> 4)) & 3);
    }
    const uint32_t ldst = lds_addr(smem[0]) + 2048 * w;
    const int H = 2 * (c_end - c_begin);   // half columns of the piece
    auto load = [&](int h) {
      const uint32_t dst = ldst + 32768 * (h & 3);
      const u32x4_t* ws = wsrc + static_cast<int64_t>(h) * 256;
      lds_dma16(ws, dst);
      lds_dma16(ws + 64, dst + 1024);
      lds_dma16(xsrc[0] + 32 * h, dst + 16384);
      lds_dma16(xsrc[1] + 32 * h, dst + 16384 + 1024);
    };

    struct Frags {
      half8_t a[8], b[4];
    };
    const uint8_t* abase = smem[0] + 8192 * wm + 16 * lane;
    const uint8_t* bbase = smem[0] + 16384 + 64 * (64 * wn + row) + 16 * ((kb + (row >> 2)) & 3);
    auto read = [&](Frags& f, int h) {
      const int at = 32768 * (h & 3);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) f.b[nb] = *reinterpret_cast<const half8_t*>(bbase + at + 1024 * nb);
#pragma unroll
      for (int i = 0; i < 8; ++i) f.a[i] = *reinterpret_cast<const half8_t*>(abase + at + 1024 * i);
    };
    f32x4_t acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Half column h: its fragments are in registers; those of h + 1 are read
    // between its MFMAs, and the loads of h + 4 go into the ring place that
    // the reads of h left before the last barrier.  At the barrier half
    // h + 2 has landed, with the loads of h + 3 and h + 4 still in flight.
    auto half_column = [&](int h, const Frags& cur, Frags& nxt) {
      const bool more = h + 4 < H;
      if (more) load(h + 4);
      read(nxt, h + 1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          acc[i][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(cur.a[i], cur.b[nb], acc[i][nb], 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 12; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);   // two MFMAs
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
      if (more) USW_PRODUCER_BARRIER(8);
      else USW_PRODUCER_BARRIER(0);
    };
    for (int h = 0; h < min(4, H); ++h) load(h);
    if (H >= 4) USW_PRODUCER_BARRIER(8);
    else USW_PRODUCER_BARRIER(0);
    Frags f0, f1;
    read(f0, 0);
    for (int h = 0; h < H; h += 2) {
      half_column(h, f0, f1);
      half_column(h + 1, f1, f0);
    }

    // Lane l of block (f, nb): outputs 16 f + 4 (l / 16) + i, row 16 nb + l % 16 of the wave's 128 x 64.
    // The thread's number goes through an empty asm: the addresses derived
    // from it are computed here, not kept in registers over the product.
    int me = tid;
    asm volatile("" : "+v"(me));
    const int64_t x0 = t0 - B;
    int q0 = 0, np = 0;
    if (!full) {
      // A shared tile: the accumulators go to a slot in register order with
      // stores that reach the level all XCDs share; the piece that completes
      // the tile's count adds the slots in column order.  Owners of the tile:
      // workgroups p with B + U p / Pr <= t0 + Gc - 1 and B + U (p + 1) / Pr > t0.
      const int slot = 2 * L + (t0 + c_begin == r0 ? 0 : 1);
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(a.part + static_cast<int64_t>(slot) * kWideSlot, 0,
                                                          kWideSlot * 4, kBufferRsrcWord3);
#pragma unroll
      for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[f][nb]), rsrc,
                                                 (((w * 8 + f) * 4 + nb) * 64 + (me & 63)) * 16, 0, kCacheSc1);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_waitcnt(0);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __syncthreads();
      q0 = static_cast<int>(((x0 + 1) * Pr + U - 1) / U) - 1;
      np = static_cast<int>(((x0 + Gc) * Pr + U - 1) / U) - q0;
      if (tid == 0)
        last_flag = __hip_atomic_fetch_add(&a.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                    static_cast<uint32_t>(np - 1);
      __syncthreads();
      const bool last = last_flag != 0;
      __syncthreads();   // last_flag is read; the next piece may write it
      if (!last) continue;
      if (tid == 0) __hip_atomic_store(&a.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    // Through LDS, 128 outputs by 256 rows at a time, so that a row's 128
    // outputs are stored together; the 16-byte unit u of row n lies at
    // u ^ (n % 32), which keeps writes and reads off each other's banks.
    f32x4_t* tile4 = reinterpret_cast<f32x4_t*>(smem);
    auto unit = [](int n, int u) { return 32 * n + (u ^ (n & 31)); };
    for (int h = 0; h < 2; ++h) {
      if (full) {
        if (wm == h) {
#pragma unroll
          for (int f = 0; f < 8; ++f)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb)
              tile4[unit(64 * wn + 16 * nb + (me & 15), 4 * f + ((me >> 4) & 3))] = acc[f][nb];
        }
      } else {
        // Eight elements per thread and round; element el is lane el % 64 of
        // block (f, nb) of wave wv, el = ((wv * 8 + f) * 4 + nb) * 64 + lane;
        // the half's waves are wv = h, h + 2, ...
        for (int v0 = 0; v0 < 4; v0 += 2) {
          f32x4_t sum[8], u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          for (int k = 0; k < np; ++k) {
            const int64_t q = q0 + k;
            const int64_t s = 2 * q + (B + U * q / Pr >= t0 ? 0 : 1);
            const auto r = __builtin_amdgcn_make_buffer_rsrc(a.part + s * kWideSlot, 0, kWideSlot * 4, kBufferRsrcWord3);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int el = (2 * (v0 + (j >> 2)) + h) * 2048 + 512 * (j & 3) + me;
              u[j] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, el * 16, 0, kCacheSc1));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += u[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int in = 512 * (j & 3) + me;   // element of wave 2 (v0 + j / 4) + h
            const int ln = in & 63, nb = (in >> 6) & 3, f = in >> 8;
            tile4[unit(64 * (v0 + (j >> 2)) + 16 * nb + (ln & 15), 4 * f + (ln >> 4))] = sum[j];
          }
        }
      }
      __syncthreads();
      for (int i = me; i < 32 * kWideN; i += kWideThreads) {
        const int n = i >> 5, u = i & 31;
        store4(t, n, t.strip0 * kGT + 128 * h + 4 * u, tile4[unit(n, u)]);
      }
      __syncthreads();
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Dense fragments held at a time: weights beyond this are expanded and
// multiplied in groups, each with its own pair of launches.
constexpr int64_t kDenseBytes = int64_t(1) << 30;

}  // namespace

namespace usw {

WidePlan wide_plan(const Geometry& g, int32_t E, int32_t S) {
  WidePlan p{};
  const int64_t one = g.M * g.K * 2;
  p.group = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(E, kDenseBytes / one)));
  const int64_t mt = (g.M + kWideM - 1) / kWideM;
  const int64_t active = std::min<int64_t>(p.group, S);
  p.tiles = (active + (S - active) / kWideN) * mt;
  p.wgs = static_cast<int>(kComputeUnits);
  p.cb = align256(static_cast<size_t>(4) * p.tiles);
  p.slots_at = p.cb;
  p.dense_at = p.slots_at + static_cast<size_t>(2) * p.wgs * kWideSlot * sizeof(float);
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
  a.mt = static_cast<int>((g.M + kWideM - 1) / kWideM);
  a.S = c.S;
  a.T = c.T;
  a.i4 = c.val_type == USW_VAL_I4;
  a.remap = p.wgs % 8 == 0;
  const unsigned gx = static_cast<unsigned>((g.ngt + kExpandWaves - 1) / kExpandWaves);
  for (int e0 = 0; e0 < c.E; e0 += p.group) {
    const int e1 = std::min(c.E, e0 + p.group);
    x.e0 = a.e0 = e0;
    a.e1 = e1;
    const dim3 grid(gx, static_cast<unsigned>(e1 - e0));
    if (a.i4) expand_kernel<true><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    else expand_kernel<false><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    wide_kernel<<<p.wgs, kWideThreads, 0, s>>>(a);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

}  // namespace usw
