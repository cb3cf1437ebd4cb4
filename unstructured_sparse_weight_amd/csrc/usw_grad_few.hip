// Gradients of few rows.
//
//   dx[n][k] = sum_m W_sp[m][k] d[n][m]
//
// straight from the encoding, as the decode kernel (usw_decode_kernels.h) down
// the columns of GroupTiles instead of along the rows: a workgroup owns a strip
// of 64 columns of W, each of its waves streams a run of the strip's GroupTiles,
// one ahead in registers, and the workgroups of a strip join their fp32 sums in
// split order.  What differs is the matrix operand: the reduction runs over W's
// rows, and a lane needs eight rows of one column where a rebuilt BitmapTile row
// is eight columns of one row.  So 32 rebuilt rows at a time pass through a tile
// in LDS, written as they are rebuilt and read by ds_read_b64_tr_b16, which hands
// each of 16 lanes one column of four rows.  The tile's rows are 144 bytes apart,
// so neither access has bank conflicts.
//
//   dV[i] = sum_n d[n][m_i] x[n][k_i]
//
// is bound by its own bytes and by the latency of each GroupTile.  A workgroup
// keeps four strips' d in registers, one to a wave, and goes along the columns,
// the next 64 columns of x on their way.  d and x are read as they lie and
// transposed on the way from LDS.
//
// Where both are wanted they are one launch, the workgroups of dx first: the one
// waits on memory where the other compacts.  MI355X, both, as two launches / one:
// 5120x5120 N = 20, dx and dV in fp32, 37.2 / 28.5 us; pairs of 4096x4096 N = 10
// 39.6 / 31.0, of 11008x4096 N = 8 72.9 / 65 (3.1 TB/s of the 203 MB it reads
// and writes), of 2048x2048 N = 60 29.7 / 23.5.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "usw.h"
#include "usw_decode_plan.h"
#include "usw_grad.h"
#include "usw_grad_values.h"
#include "usw_internal.h"
#include "usw_wide.h"

namespace {

using namespace usw_dev;

// M: columns of W (the outputs), K: row length of d, Gc: GroupTile rows of all
// blocks (the reduction).
struct ColumnArgs : FusedArgs {
  const uint64_t* wbitmaps[2];
  const uint32_t* woffsets[2];
  const uint8_t* wvalues[2];
  const uint16_t* wscales[2];
  uint64_t walloc[2];
  int rows;   // GroupTile rows of a block
  int lo;     // LO: column of d's remainders
  bool frag;
};
template <>
struct ArgTraits<ColumnArgs> : ArgTraits<FusedArgs> {};

constexpr int kTrBytes = 32 * kTrLd * 2;

// Rebuilds rows 32 H .. 32 H + 31 of a GroupTile into the wave's tile.  scale:
// INT4, that of the lane's row of each fragment, whose power of two it takes.
template <bool I4, int H>
__device__ __forceinline__ void column_rows(const uint8_t* vals, const uint8_t* tab, const uint32_t* lut, uint8_t* tile,
                                            const uint32_t (&scale)[4], const LaneMap& lm, int lane) {
#pragma unroll
  for (int f = 2 * H; f < 2 * H + 2; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const u32x2_t e = *reinterpret_cast<const u32x2_t*>(tab + lm.tab + 256 * f + 128 * ks);
      const uint32_t rb = e.y + __builtin_popcount(e.x & lm.pmask);
      half8_t v = rebuild_row<I4>(vals, lut, rb, __builtin_amdgcn_ubfe(e.x, lm.sh, 8));
      if constexpr (I4) {
        v -= static_cast<_Float16>(kCodeOffset);   // exact, and so is the power of two
        v *= static_cast<_Float16>(scale_power(static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(scale[f])))));
      }
      *reinterpret_cast<half8_t*>(tile + 2 * ((16 * (f - 2 * H) + (lane & 15)) * kTrLd + 32 * ks + 8 * (lane >> 4))) = v;
    }
  wave_sync();
}

// Multiplies the tile's columns with those rows of d.
template <int NB>
__device__ __forceinline__ void column_mma(const u32x4_t (&x)[NB], const uint8_t* tile, f32x4_t (&acc)[4][NB], int lane) {
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const half8_t w = read_column(tile, lane, 16 * f);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      acc[f][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, __builtin_bit_cast(half8_t, x[nb]), acc[f][nb], 0, 0, 0);
  }
  wave_sync();
}
// And with its remainders.  GUARD: infinite weights are left to d itself.
template <int NB, bool GUARD>
__device__ __forceinline__ void column_mma(const u32x4_t (&x)[NB], const u32x4_t (&lo)[NB], const uint8_t* tile,
                                           f32x4_t (&acc)[4][NB], int lane) {
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const half8_t w = read_column(tile, lane, 16 * f);
    const half8_t wf = GUARD ? finite(w) : w;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      acc[f][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, __builtin_bit_cast(half8_t, x[nb]), acc[f][nb], 0, 0, 0);
      acc[f][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf, __builtin_bit_cast(half8_t, lo[nb]), acc[f][nb], 0, 0, 0);
    }
  }
  wave_sync();
}

// Waves per SIMD as registers allow.
template <int NB, int CH, bool LO>
using ColumnCfg = Cfg<4, 1, NB <= 4 && !(NB == 2 && CH == 6 && LO) ? 3 : 2>;

template <int NB, bool I4, int CH>
struct ColumnLds {
  static constexpr int kLut = I4 ? 2048 : 128;
  static constexpr int kStage = 4 * (ValTraits<I4, CH>::kVbuf + kTabBytes + kTrBytes), kRed = 2 * 4 * NB * 1024;
  static constexpr int kBytes = kLut + (kStage > kRed ? kStage : kRed);
};

// Workgroup b of blocks.  FRAG: d lies in the order of its matrix fragments.
template <int NB, bool I4, int CH, bool LO, bool FRAG>
__device__ __forceinline__ void column_body(const ColumnArgs& a, uint8_t* lds, uint32_t& last_flag, int b, int blocks) {
  using VT = ValTraits<I4, CH>;
  constexpr int kW = 4, kThreads = 64 * kW;
  uint32_t* lut = reinterpret_cast<uint32_t*>(lds);
  uint8_t* smem = lds + ColumnLds<NB, I4, CH>::kLut;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // As the decode kernel's: the splits of a strip on one XCD.
  const int L = a.remap ? (b & 7) * (blocks >> 3) + (b >> 3) : b;
  const int gi = L / a.splits, sidx = L - gi * a.splits;
  if constexpr (I4) {
    for (int i = tid; i < 256; i += kThreads) reinterpret_cast<u32x2_t*>(lut)[i] = row_byte_selectors(i);
  } else if (tid < 16) {
    u32x2_t e;
    e.x = nibble_selector(tid, 0);
    e.y = nibble_selector(tid, 1);
    reinterpret_cast<u32x2_t*>(lut)[tid] = e;
  }
  __syncthreads();

  // The wave's GroupTiles c of the strip: block c / rows, GroupTile row
  // c % rows, their first and last values one to a lane (the host keeps the
  // count at 63 or fewer).
  const int parts = a.splits * kW, q = sidx * kW + w;
  const int c_begin = static_cast<int>(static_cast<int64_t>(a.Gc) * q / parts);
  const int c_end = static_cast<int>(static_cast<int64_t>(a.Gc) * (q + 1) / parts);
  const int cnt = c_end - c_begin, cols = a.M / kGT;
  const LaneMap lm = lane_map(lane);
  f32x4_t acc[4][NB];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  uint8_t* vb = smem + w * VT::kVbuf;
  uint8_t* tab = smem + kW * VT::kVbuf + w * kTabBytes;
  uint8_t* tile = smem + kW * (VT::kVbuf + kTabBytes) + w * kTrBytes;
  const uint32_t vb_elems = I4 ? static_cast<uint32_t>(w * VT::kVbuf * 2) : static_cast<uint32_t>(w * VT::kVbuf / 2);
  uint32_t first = 0, past = 0;
  if (cnt > 0) {
    const int c = c_begin + min(lane, cnt - 1), e = c >= a.rows ? 1 : 0;
    const uint32_t* off = (e ? a.woffsets[1] : a.woffsets[0]) + static_cast<int64_t>(c - e * a.rows) * cols + gi;
    first = off[0];
    past = off[1];
  }
  const uint32_t widest = wave_max(past - first);
  // Loads of GroupTile c: weight, d of its rows 32 h on, d's remainders.
  auto load_w = [&](Slot<NB, I4, CH>& s, uint32_t (&scale)[4], int c) {
    c = min(c, c_end - 1);
    const uint32_t o0 = __builtin_amdgcn_readlane(first, c - c_begin), o1 = __builtin_amdgcn_readlane(past, c - c_begin);
    const int e = c >= a.rows ? 1 : 0, i = c - e * a.rows;
    slot_load_weight(s, (e ? a.wbitmaps[1] : a.wbitmaps[0]) + (static_cast<int64_t>(i) * cols + gi) * kBtPerGt,
                     e ? a.wvalues[1] : a.wvalues[0], e ? a.walloc[1] : a.walloc[0], lane, o0, o1);
    if constexpr (I4) {
      const uint16_t* sc = (e ? a.wscales[1] : a.wscales[0]) + i * kGT + (lane & 15);
#pragma unroll
      for (int f = 0; f < 4; ++f) scale[f] = sc[16 * f];
    }
  };
  // Tokens past the last repeat it (FRAG: are zeros): their products are not
  // stored.
  auto load_d = [&](u32x4_t (&d)[NB], int c, int h, int at) {
    c = min(c, c_end - 1);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (FRAG)
        d[nb] = reinterpret_cast<const u32x4_t*>(a.X)[((static_cast<size_t>(at) / kGT + c) * 2 + h) * (64 * NB) + 64 * nb + lane];
      else
        d[nb] = *reinterpret_cast<const u32x4_t*>(a.X + static_cast<size_t>(min(nb * 16 + (lane & 15), a.N - 1)) * a.K + at +
                                                  c * kGT + h * 32 + (lane >> 4) * 8);
    }
  };
  auto write_tab = [&](const Slot<NB, I4, CH>& s) {
    tab_write(tab, s.bm, bitmap_prefix_reg(s.bm) + s.delta + vb_elems, lane);
  };
  // As in the decode kernel: the values of half a GroupTile at a time.
  auto by_halves = [&](auto guard) {
    constexpr bool GUARD = decltype(guard)::value;
    for (int c = c_begin; c < c_end; ++c) {
      Slot<NB, I4, CH> s0;
      uint32_t none[4];
      load_w(s0, none, c);
      const int e = c >= a.rows ? 1 : 0;
      const uint8_t* values = e ? a.wvalues[1] : a.wvalues[0];
      const uint64_t top = (e ? a.walloc[1] : a.walloc[0]) - 16;
      const uint32_t o0 = __builtin_amdgcn_readlane(first, c - c_begin), o1 = __builtin_amdgcn_readlane(past, c - c_begin);
      const uint32_t excl = bitmap_prefix_reg(s0.bm);
      const uint32_t mid = __builtin_amdgcn_readlane(excl, 32);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t d[NB];
        load_d(d, c, h, 0);
        const uint32_t hs = o0 + (h ? mid : 0u), he = h ? o1 : o0 + mid;
        const uint64_t a0 = min(chunk_start<I4>(hs), top);
        const uint32_t delta = chunk_delta<I4>(hs, a0);
        const uint32_t nch = min(chunk_count<I4>(he, a0), static_cast<uint32_t>((VT::kVbuf - 16) / 16));
        const uint32_t last = static_cast<uint32_t>((top - a0) >> 4);
        const u32x4_t* src = reinterpret_cast<const u32x4_t*>(values + a0);
        for (uint32_t ch = lane; ch < nch; ch += 64) reinterpret_cast<u32x4_t*>(vb)[ch] = src[min(ch, last)];
        // Entries of the other half get bases that are never read.
        tab_write(tab, s0.bm, excl - (h ? mid : 0u) + delta + vb_elems, lane);
        wave_sync();
        if (h == 0) column_rows<I4, 0>(smem, tab, lut, tile, none, lm, lane);
        else column_rows<I4, 1>(smem, tab, lut, tile, none, lm, lane);
        if constexpr (LO) {
          u32x4_t dlo[NB];
          load_d(dlo, c, h, a.lo);
          column_mma<NB, GUARD>(d, dlo, tile, acc, lane);
        } else {
          column_mma<NB>(d, tile, acc, lane);
        }
      }
    }
  };
  if (cnt <= 0) {
    // nothing to stream
  } else if (widest > VT::kFastLimit) {
    if constexpr (!I4) by_halves(std::false_type{});
  } else if constexpr (NB > 2) {
    // Registers for three waves per SIMD (more than 64 tokens two): half a
    // GroupTile's d at a time, and the next weight in one slot, asked for where
    // this one's second half starts.  Loads are in the order in which they are
    // waited for.  Against two slots as below, a wave less: dx and dV of 4096x4096
    // N = 64 25.0 -> 19.8 us, INT4 dx of 5120x20480 N = 60 53.1 -> 42.6.
    Slot<NB, I4, CH> s;
    uint32_t scale[4], next[4];
    u32x4_t d[NB];
    load_w(s, next, c_begin);
    load_d(d, c_begin, 0, 0);
    for (int c = c_begin; c < c_end; ++c) {
      slot_commit(s, vb, lane);
      write_tab(s);
      if constexpr (I4) {
#pragma unroll
        for (int f = 0; f < 4; ++f) scale[f] = next[f];
      }
      wave_sync();
      column_rows<I4, 0>(smem, tab, lut, tile, scale, lm, lane);
      column_mma<NB>(d, tile, acc, lane);
      load_d(d, c, 1, 0);
      load_w(s, next, c + 1);
      column_rows<I4, 1>(smem, tab, lut, tile, scale, lm, lane);
      column_mma<NB>(d, tile, acc, lane);
      load_d(d, c + 1, 0, 0);
    }
  } else {
    // As the decode kernel with two register slots.
    struct Ahead {
      Slot<NB, I4, CH> s;
      u32x4_t d[2][NB], lo[2][NB];
      uint32_t scale[4];
    };
    Ahead s[2];
    auto load = [&](Ahead& t, int c) {
      load_w(t.s, t.scale, c);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load_d(t.d[h], c, h, 0);
        if constexpr (LO) load_d(t.lo[h], c, h, a.lo);
      }
    };
    load(s[0], c_begin);
    write_tab(s[0].s);
    auto step = [&](int c, int cur) {
      __builtin_amdgcn_s_setprio(2);
      load(s[cur ^ 1], c + 1);
      __builtin_amdgcn_s_setprio(0);
      slot_commit(s[cur].s, vb, lane);
      wave_sync();
      column_rows<I4, 0>(smem, tab, lut, tile, s[cur].scale, lm, lane);
      if constexpr (LO) column_mma<NB, false>(s[cur].d[0], s[cur].lo[0], tile, acc, lane);
      else column_mma<NB>(s[cur].d[0], tile, acc, lane);
      column_rows<I4, 1>(smem, tab, lut, tile, s[cur].scale, lm, lane);
      if constexpr (LO) column_mma<NB, false>(s[cur].d[1], s[cur].lo[1], tile, acc, lane);
      else column_mma<NB>(s[cur].d[1], tile, acc, lane);
      write_tab(s[cur ^ 1].s);
    };
    int c = c_begin;
    for (; c + 2 <= c_end; c += 2) {
      step(c, 0);
      step(c + 1, 1);
    }
    if (c < c_end) step(c, 0);
  }
  if constexpr (LO && !I4) {
    // An infinite weight times a remainder of zero, or of the other sign than d's,
    // has left a NaN: the wave's GroupTiles once more, guarded.  Guarding each
    // weight from the start costs 2 to 4% (pairs of 11008x4096 N = 8 68.3 / 69.7
    // us, of 20480x5120 N = 20 150 / 156).
    bool nan = false;
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= acc[f][nb][i] != acc[f][nb][i];
    if (__ballot(nan)) {
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[f][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      by_halves(std::true_type{});
    }
  }

  // Workgroup reduction over waves (fixed order), the last two into the first.
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);   // [2 waves][4][NB][64 lanes][4]
  auto place = [&](int f, int nb) {
    return reinterpret_cast<f32x4_t*>(red + ((((w & 1) * 4 + f) * NB + nb) * 64 + lane) * 4);
  };
  if (w >= 2) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) *place(f, nb) = acc[f][nb];
  }
  __syncthreads();
  if (w < 2) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) *place(f, nb) += acc[f][nb];
  }
  __syncthreads();
  auto sum_of = [&](int n, int ml) {
    const int f = ml >> 4, ln = 16 * ((ml >> 2) & 3) + (n & 15), nb = n >> 4;
    const f32x4_t* at = reinterpret_cast<const f32x4_t*>(red + ((f * NB + nb) * 64 + ln) * 4);
    return at[0] + at[4 * NB * 64];
  };
  finish_strip_fused<NB, false, NB == 1 ? 8 : 4>(a, gi, sidx, kThreads, last_flag, sum_of);
}

struct FewValuesArgs {
  ValueWeights v;
  const uint16_t* d;   // [N][ldd], the second weight's M columns behind the first's
  const uint16_t* X;   // [N][K]
  int64_t ldd, lo;     // lo > 0: d's remainders lie this many columns on
  int M, K, N, splits;
  bool two;
};

// H: 32-row halves of d and x.
template <int H, typename T, bool LO>
constexpr int kFewResident = H == 1 ? (LO ? 4 : 5) : sizeof(T) == 2 ? 3 : 2;   // workgroups per compute unit

// Two tiles of x and the waves' runs; before them, a tile of d for each wave.
template <int H, typename T>
struct ValuesLds {
  static constexpr int kTile = 32 * H * kTrLd * 2, kWave = kKeptBytes<T, 4>, kUsed = 2 * kTile + 4 * kWave;
  static constexpr int kBytes = kUsed > 4 * kTile ? kUsed : 4 * kTile;
};

// Workgroup b: four strips, a part of the columns.
template <int H, typename T, bool LO>
__device__ __forceinline__ void values_body(const FewValuesArgs& a, uint8_t* smem, int b) {
  static_assert(!LO || 32 * H <= usw::kLoRows, "rows with remainders");
  constexpr int P = LO ? 2 : 1;   // parts of d
  constexpr int kTile = ValuesLds<H, T>::kTile, kWave = ValuesLds<H, T>::kWave;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int quad = b / a.splits, part = b - quad * a.splits;
  const int c0 = static_cast<int>(static_cast<int64_t>(a.v.cols) * part / a.splits);
  const int c1 = static_cast<int>(static_cast<int64_t>(a.v.cols) * (part + 1) / a.splits);
  const int all = a.two ? 2 * a.v.strips : a.v.strips;

  const int vs = min(4 * quad + w, all - 1);
  const int second = vs >= a.v.strips ? 1 : 0, r = vs - second * a.v.strips;
  T* dv = static_cast<T*>(second ? a.v.dv[1] : a.v.dv[0]);
  const uint64_t* bitmaps = (second ? a.v.bitmaps[1] : a.v.bitmaps[0]) + static_cast<int64_t>(r) * a.v.cols * kBtPerGt;
  const uint32_t* offsets = (second ? a.v.offsets[1] : a.v.offsets[0]) + static_cast<int64_t>(r) * a.v.cols;
  const int64_t nnz = 4 * quad + w < all && dv ? (second ? a.v.nnz[1] : a.v.nnz[0]) : 0;
  uint8_t* lds = smem + 2 * kTile + w * kWave;

  // Rows past the last are loaded from it and become zeros, as d's there are (an
  // infinity times one would be a NaN); columns past the last repeat it.  Strips
  // past the last run along with the last one's bitmaps and store nothing.
  u32x4_t xr[H];
  u32x2_t bm;
  uint32_t first;
  auto load = [&](int c) {
    c = min(c, c1 - 1);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int p = tid + 256 * i;
      xr[i] = *reinterpret_cast<const u32x4_t*>(a.X + static_cast<int64_t>(min(p >> 3, a.N - 1)) * a.K + kGT * c + 8 * (p & 7));
    }
    bm = reinterpret_cast<const u32x2_t*>(bitmaps + static_cast<int64_t>(c) * kBtPerGt)[lane];
    first = offsets[c];
  };
  // 16-byte piece p of 64 columns: row p / 8, columns 8 (p % 8) on.
  auto put = [&](uint8_t* tile, int p, u32x4_t v) {
    *reinterpret_cast<u32x4_t*>(tile + 2 * ((p >> 3) * kTrLd + 8 * (p & 7))) = v;
  };
  auto commit = [&](uint8_t* tile) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int p = tid + 256 * i;
      put(tile, p, (p >> 3) < a.N ? xr[i] : u32x4_t{0u, 0u, 0u, 0u});
    }
  };
  load(c0);
  // The wave's d, 8 rows to a load, through its tile.
  half8_t d[P][4][H];
  u32x4_t dr[P][4 * H];
  const uint16_t* dsrc = a.d + (second ? a.M + r * kGT : r * kGT) + 8 * (lane & 7);
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int i = 0; i < 4 * H; ++i) {
      const int n = (lane >> 3) + 8 * i;
      dr[q][i] = u32x4_t{0u, 0u, 0u, 0u};
      if (n < a.N) dr[q][i] = *reinterpret_cast<const u32x4_t*>(dsrc + n * a.ldd + q * a.lo);
    }
#pragma unroll
  for (int q = 0; q < P; ++q) {
    uint8_t* tile = smem + w * kTile;
#pragma unroll
    for (int i = 0; i < 4 * H; ++i) put(tile, lane + 64 * i, dr[q][i]);
    wave_sync();
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int h = 0; h < H; ++h) d[q][f][h] = read_column(tile + 2 * 32 * h * kTrLd, lane, 16 * f);
    wave_sync();
  }
  __syncthreads();
  kept_selectors(lds, lane);
  commit(smem);
  lds_barrier();
  // Only LDS is shared: the barrier leaves stores in flight.
  for (int c = c0; c < c1; ++c) {
    const uint8_t* tile = smem + kTile * ((c - c0) & 1);
    const u32x2_t bits = bm;
    const uint32_t at = first;
    load(c + 1);
    f32x4_t acc[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const half8_t x = read_column(tile + 2 * 32 * h * kTrLd, lane, 16 * n);
        const half8_t xf = LO ? finite(x) : x;
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int q = 0; q < P; ++q)
            acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q ? xf : x, d[q][f][h], h + q ? acc[f][n] : f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      }
    const Kept<T> k = kept_of<T>(bits, at, nnz, dv, lds, lane);
#pragma unroll
    for (int f = 0; f < 4; ++f) store_kept<T, 4>(k, acc[f], f, 0, lds, lane);
    commit(smem + kTile * ((c + 1 - c0) & 1));
    lds_barrier();
  }
}

// ---------------------------------------------------------------------------
// Kernels: dx alone, dV alone, both
// ---------------------------------------------------------------------------

template <int NB, bool I4, int CH, bool LO, bool FRAG>
__global__ __launch_bounds__(256, (ColumnCfg<NB, CH, LO>::kOcc)) void column_kernel(ColumnArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[ColumnLds<NB, I4, CH>::kBytes];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);
  column_body<NB, I4, CH, LO, FRAG>(a, smem, last_flag, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
}

template <int H, typename T, bool LO>
__global__ __launch_bounds__(256, (kFewResident<H, T, LO>)) void few_values_kernel(FewValuesArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[ValuesLds<H, T>::kBytes];
  USW_LDS_POISON(smem);
  values_body<H, T, LO>(a, smem, static_cast<int>(blockIdx.x));
}

struct BothArgs {
  ColumnArgs x;
  FewValuesArgs v;
  int first;   // workgroups of dx
};

template <int NB, int CH, typename T, bool LO, bool FRAG>
__global__ __launch_bounds__(256, (ColumnCfg<NB, CH, LO>::kOcc)) void both_kernel(BothArgs a) {
  constexpr int H = (NB + 1) / 2;
  constexpr int kX = ColumnLds<NB, false, CH>::kBytes, kV = ValuesLds<H, T>::kBytes;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kX > kV ? kX : kV];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);
  const int b = static_cast<int>(blockIdx.x);
  if (b < a.first) column_body<NB, false, CH, LO, FRAG>(a.x, smem, last_flag, b, a.first);
  else values_body<H, T, LO>(a.v, smem, b - a.first);
}

// As many columns to a workgroup as one round of resident workgroups leaves
// it; one less where they are few and the round a tenth over.  dx and dV, splits of
// dV's columns: 5120x5120 N = 20 in fp32 5 65.5 us, 10 45.9, 20 38.4, 40 35.8;
// 4096x11008 N = 1 16 53.8, 32 43.0, 80 39.0; 11008x4096 N = 8 29 43.5, 32 40.9.
int value_splits(int64_t quads, int64_t cols, int64_t resident) {
  int64_t each = (cols * quads + resident - 1) / resident;
  const auto splits = [&](int64_t n) { return (cols + n - 1) / n; };
  if ((each == 2 || each == 3) && splits(each - 1) * quads * 10 <= resident * 11) --each;
  return static_cast<int>(splits(each));
}

// Launches with the types that the call's rows and outputs ask for.  x, v: null
// where not wanted.
template <int NB>
void launch_few(const ColumnArgs* x, FewValuesArgs* v, bool i4, bool lean, bool f16, hipStream_t s) {
  constexpr bool kLo = 16 * NB <= usw::kLoRows;   // d of as many rows has remainders where it is made, of INT4 weights always
  const dim3 gx(x ? static_cast<unsigned>(x->M / kGT * x->splits) : 0);
  if constexpr (16 * NB <= usw::kFewValueRows) {
    constexpr int H = (NB + 1) / 2;
    if (v) {
      auto go = [&](auto zero, auto remainders, auto fragments) {
        constexpr bool LO = decltype(remainders)::value, F = decltype(fragments)::value;
        using T = decltype(zero);
        const int64_t quads = ((v->two ? 2 : 1) * v->v.strips + 3) / 4;
        v->splits = value_splits(quads, v->v.cols, kComputeUnits * kFewResident<H, T, LO>);
        const unsigned blocks = static_cast<unsigned>(quads * v->splits);
        if (!x) {
          few_values_kernel<H, T, LO><<<blocks, 256, 0, s>>>(*v);
          return;
        }
        const BothArgs b{*x, *v, static_cast<int>(gx.x)};
        if (lean) both_kernel<NB, 5, T, LO, F><<<gx.x + blocks, 256, 0, s>>>(b);
        else both_kernel<NB, 6, T, LO, F><<<gx.x + blocks, 256, 0, s>>>(b);
      };
      // A gated block's gradients are fp16, and its d has remainders or is both in
      // rows and as fragments.
      if (v->two) go(_Float16(0), std::integral_constant<bool, kLo>{}, std::integral_constant<bool, !kLo>{});
      else if (f16) go(_Float16(0), std::false_type{}, std::false_type{});
      else go(0.0f, std::false_type{}, std::false_type{});
      return;
    }
  }
  // dx alone.  INT4's d is always made, with remainders up to kLoRows rows.
  if (i4) {
    column_kernel<NB, true, 3, kLo, true><<<gx, 256, 0, s>>>(*x);
    return;
  }
  auto go = [&](auto remainders, auto fragments) {
    constexpr bool LO = decltype(remainders)::value, F = decltype(fragments)::value;
    if (lean) column_kernel<NB, false, 5, LO, F><<<gx, 256, 0, s>>>(*x);
    else column_kernel<NB, false, 6, LO, F><<<gx, 256, 0, s>>>(*x);
  };
  // And a gated block's.
  if (x->frag) go(std::integral_constant<bool, kLo>{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
}

}  // namespace

namespace usw {

int few_row_blocks(int N) {
  const int nb = (N + 15) / 16;
  return nb <= 4 ? nb : nb <= 6 ? 6 : 8;
}

FewPlan few_plan(const Geometry& g, const FewCall& c) {
  FewPlan p{};
  const int nb = few_row_blocks(c.N);
  p.lean = true;
  for (int h = 0; h < c.blocks; ++h) p.lean = p.lean && lean_values(c.f[h], g);
  // One round of resident workgroups, each wave keeping at least 3 GroupTiles,
  // at most 63: INT4 pairs of 11008x4096 N = 77 4 splits 56 us, 8 46, 12 60;
  // 11008x4096 INT4 N = 8 8 splits 22.0, 12 20.9, 24 24.8.  d in rows of more than 64
  // tokens, which come from the L2 in half lines: one to a compute unit, 4096x4096 N
  // = 128 4 splits 43, 8 48.  Where dV's workgroups
  // fill the rest of the chip, one to a compute unit: dx and dV of 4096x4096
  // pairs N = 10 2 splits 39.5, 4 31.0, 12 36.8; 5120x5120 N = 20 1 43.5, 3 28.5, 10
  // 32.8; 4096x11008 N = 16 1 32.9, 4 36.8; 8192x1024 N = 20 4 22.2, 12 16.5.
  const int64_t rows = c.blocks * g.Gr, strips = g.Gc;
  const int64_t resident = kComputeUnits * (c.want_v || (nb > 4 && !c.frag) ? 1 : nb <= 4 ? 3 : 2);
  int64_t s = std::max<int64_t>(1, (resident + strips / 2) / strips);
  s = std::min(s, std::max<int64_t>(1, rows / 12));
  p.splits = static_cast<int>(std::max((rows + 63 * 4 - 1) / (63 * 4), std::min(s, std::max<int64_t>(1, rows / 4))));
  if (p.splits > 1) {
    p.cb = counter_zone(4 * strips);
    p.need = p.cb + static_cast<size_t>(p.splits) * c.N * g.K * sizeof(float);
  }
  return p;
}

usw_status few_launch(const Geometry& g, const FewCall& c, const FewPlan& p, void* ws, void* stream) {
  const bool i4 = c.f[0]->val_type == USW_VAL_I4, f16 = c.out_type == USW_OUT_F16;
  ColumnArgs a{};
  if (c.want_x) {
    for (int h = 0; h < c.blocks; ++h) {
      const usw_fmt* f = c.f[h];
      a.wbitmaps[h] = f->bitmaps;
      a.woffsets[h] = f->offsets;
      a.wvalues[h] = static_cast<const uint8_t*>(f->values);
      a.wscales[h] = f->scales;
      a.walloc[h] = values_alloc_bytes(f->val_type, f->nnz);
    }
    a.rows = static_cast<int>(g.Gr);
    a.X = c.frag ? c.F : c.D;
    a.Y = c.dX;
    a.e = Epilogue{nullptr, nullptr, nullptr, g.K, g.K, USW_ACT_NONE, f16 ? 1 : 0};
    a.counters = static_cast<uint32_t*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.cb);
    a.M = static_cast<int>(g.K);
    a.K = static_cast<int>(c.ldD);
    a.lo = static_cast<int>(c.lo);
    a.frag = c.frag;
    a.N = c.N;
    a.Gc = static_cast<int>(c.blocks * g.Gr);
    a.splits = p.splits;
    a.remap = g.Gc * p.splits % 8 == 0 ? 1 : 0;
  }
  FewValuesArgs v{};
  if (c.want_v) {
    v.v = value_weights(c.f, c.dV, c.weights, g);
    v.d = c.D;
    v.X = c.X;
    v.ldd = c.ldD;
    v.lo = c.lo;
    v.M = static_cast<int>(g.M);
    v.K = static_cast<int>(g.K);
    v.N = c.N;
    v.two = c.weights == 2;
  }
  const ColumnArgs* x = c.want_x ? &a : nullptr;
  FewValuesArgs* vp = c.want_v ? &v : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (few_row_blocks(c.N)) {
    case 1: launch_few<1>(x, vp, i4, p.lean, f16, s); break;
    case 2: launch_few<2>(x, vp, i4, p.lean, f16, s); break;
    case 3: launch_few<3>(x, vp, i4, p.lean, f16, s); break;
    case 4: launch_few<4>(x, vp, i4, p.lean, f16, s); break;
    case 6: launch_few<6>(x, vp, i4, p.lean, f16, s); break;
    default: launch_few<8>(x, vp, i4, p.lean, f16, s);
  }
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

}  // namespace usw
