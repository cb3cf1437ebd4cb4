// The gated feed-forward block's first half in one product (usw_spmm_gated):
//
//   g = Wg x + bg,  u = Wu x + bu,  h = act(g) * u,
//
// both weights sparse, of one shape.  g and u stay in fp32 until h is rounded;
// a training step has them written in fp16 too, for the backward pass
// (usw_grad.hip).
//
// Few rows run on the decode kernels (usw_decode_kernels.h) over a grid of
// both weights' strips, interleaved, so one launch streams both at the full
// chip and x is read while it is in the caches.  The last workgroup of a pair
// of strips joins their sums; neither projection reaches memory as an output
// (11008x4096 N = 1: 102 MB in 25.4 us, 4.0 TB/s).
//
// More rows, up to 128, run on a kernel of the same kind (tall_kernel) that takes
// half a GroupTile's columns at a time, so that two or three waves of a SIMD have
// registers for a pass of 48 to 128 rows.
//
// Many rows run on the expanded product (usw_wide_kernels.h).  The expansion
// interleaves the two weights by fragments of 16 outputs, gate then up, so a
// lane of the product holds both sums of an output in neighbouring
// accumulators and multiplies them in registers (11008x4096 N = 2048, g and u kept:
// 350 us, 1.06 PFLOP/s, after 47 of expansion).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "usw.h"
#include "usw_decode_plan.h"
#include "usw_internal.h"
#include "usw_wide.h"
#include "usw_wide_kernels.h"

namespace {

using namespace usw_dev;

constexpr int64_t kMaxElements = int64_t(1) << 34;   // of a weight: launches stay below HIP's 2^32 threads

// ---------------------------------------------------------------------------
// 33 to 128 rows
// ---------------------------------------------------------------------------

template <int NB>
constexpr int kTallResident = NB <= 4 ? 3 : 2;   // workgroups per compute unit

// As decode_kernel (usw_decode_kernels.h), its waves' steps half a GroupTile wide:
// 32 columns of x, 64 bytes of a token, pass through a tile in LDS, which four
// lanes to a token fill (as the matrix operand lies, each would be of another
// token and cost the address unit four times as much) while the half before is
// multiplied; the four fragments of the half's weights are rebuilt into
// registers and each of x's read once for them.  The next weight is asked for a
// GroupTile ahead, in one slot.  Bound by latency and the rebuild's instructions;
// decode_kernel with one or two waves per SIMD / this, 11008x4096, us: N = 64 53 / 45.5,
// INT4 46 / 33.7, N = 77 66 / 59, N = 128 98 / 78, INT4 91 / 58.5.
template <int NB, bool I4, int CH>
__global__ __launch_bounds__(256, kTallResident<NB>) void tall_kernel(GatedArgs a) {
  using VT = ValTraits<I4, CH>;
  constexpr int kW = 4, kThreads = 64 * kW, kX = 1024 * NB;
  constexpr int kStage = kW * (VT::kVbuf + kTabBytes + kX), kRed = 2 * 4 * NB * 1024;
  __shared__ __attribute__((aligned(16))) uint32_t lut[I4 ? 512 : 32];
  __shared__ __attribute__((aligned(16))) uint8_t smem[kStage > kRed ? kStage : kRed];
  __shared__ uint32_t last_flag;
  USW_LDS_POISON(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int gi, sidx, row0;
  if (!locate(a, lane, &gi, &sidx, &row0)) return;
  if constexpr (I4) {
    for (int i = tid; i < 256; i += kThreads) reinterpret_cast<u32x2_t*>(lut)[i] = row_byte_selectors(i);
  } else if (tid < 16) {
    u32x2_t e;
    e.x = nibble_selector(tid, 0);
    e.y = nibble_selector(tid, 1);
    reinterpret_cast<u32x2_t*>(lut)[tid] = e;
  }
  __syncthreads();

  // The wave's GroupTile columns; offsets one to a lane (the host keeps the count
  // at 63 or fewer).
  const int parts = a.splits * kW, q = sidx * kW + w;
  const int c_begin = static_cast<int>(static_cast<int64_t>(a.Gc) * q / parts);
  const int c_end = static_cast<int>(static_cast<int64_t>(a.Gc) * (q + 1) / parts);
  const int cnt = c_end - c_begin;
  const LaneMap lm = lane_map(lane);
  f32x4_t acc[4][NB];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[f][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint8_t* vb = smem + w * VT::kVbuf;
  uint8_t* tab = smem + kW * VT::kVbuf + w * kTabBytes;
  uint8_t* xt = smem + kW * (VT::kVbuf + kTabBytes) + w * kX;
  const uint32_t vb_elems = I4 ? static_cast<uint32_t>(w * VT::kVbuf * 2) : static_cast<uint32_t>(w * VT::kVbuf / 2);
  const int64_t g_begin = static_cast<int64_t>(gi) * a.Gc + c_begin;
  const uint32_t ov = a.offsets[g_begin + min(lane, max(cnt, 0))];
  const uint32_t ov_next = __shfl_down(ov, 1);
  const uint32_t widest = wave_max(lane < cnt ? ov_next - ov : 0u);

  auto load_w = [&](Slot<NB, I4, CH>& s, int c) {
    c = min(c, c_end - 1);
    slot_load_weight(s, a.bitmaps + (static_cast<int64_t>(gi) * a.Gc + c) * kBtPerGt, a.values, a.values_alloc, lane,
                     __builtin_amdgcn_readlane(ov, c - c_begin), __builtin_amdgcn_readlane(ov, c + 1 - c_begin));
  };
  // Tokens past the last repeat it: their products are not stored.
  auto load_x = [&](u32x4_t (&x)[NB], int c, int ks) {
    c = min(c, c_end - 1);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      x[nb] = *reinterpret_cast<const u32x4_t*>(a.X + static_cast<size_t>(min(16 * nb + (lane >> 2), a.N - 1)) * a.K +
                                                c * kGT + 32 * ks + 8 * (lane & 3));
  };
  // Piece p of token t lies at p ^ (t / 2 % 4) of its four, which keeps the
  // writes and the reads off each other's banks.
  uint8_t* xput = xt + 64 * (lane >> 2) + 16 * ((lane & 3) ^ ((lane >> 3) & 3));
  const uint8_t* xget = xt + 64 * (lane & 15) + 16 * ((lane >> 4) ^ ((lane >> 1) & 3));
  auto put_x = [&](const u32x4_t (&x)[NB]) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) *reinterpret_cast<u32x4_t*>(xput + 1024 * nb) = x[nb];
  };
  auto rebuilt = [&](int f, int ks) {
    const u32x2_t e = *reinterpret_cast<const u32x2_t*>(tab + lm.tab + 256 * f + 128 * ks);
    const uint32_t rb = e.y + __builtin_popcount(e.x & lm.pmask);
    half8_t v = rebuild_row<I4>(smem, lut, rb, __builtin_amdgcn_ubfe(e.x, lm.sh, 8));
    if constexpr (I4) v -= static_cast<_Float16>(kCodeOffset);   // exact
    return v;
  };
  // Fragments F0 on of the columns 32 ks on, by all tokens.
  auto multiply = [&](auto first, auto count, int ks) {
    constexpr int F0 = decltype(first)::value, F = decltype(count)::value;
    half8_t v[F];
#pragma unroll
    for (int f = 0; f < F; ++f) v[f] = rebuilt(F0 + f, ks);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const half8_t x = *reinterpret_cast<const half8_t*>(xget + 1024 * nb);
#pragma unroll
      for (int f = 0; f < F; ++f)
        acc[F0 + f][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[f], x, acc[F0 + f][nb], 0, 0, 0);
    }
    wave_sync();
  };
  using std::integral_constant;
  u32x4_t x[NB];
  if (cnt <= 0) {
    // nothing to stream
  } else if (widest > VT::kFastLimit) {
    if constexpr (!I4) {
      // As in decode_kernel: the values of half a GroupTile's rows at a time.
      const uint64_t top = a.values_alloc - 16;
      for (int c = c_begin; c < c_end; ++c) {
        Slot<NB, I4, CH> s;
        load_w(s, c);
        const uint32_t o0 = __builtin_amdgcn_readlane(ov, c - c_begin), o1 = __builtin_amdgcn_readlane(ov, c + 1 - c_begin);
        const uint32_t excl = bitmap_prefix_reg(s.bm);
        const uint32_t mid = __builtin_amdgcn_readlane(excl, 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hs = o0 + (h ? mid : 0u), he = h ? o1 : o0 + mid;
          const uint64_t a0 = min(chunk_start<I4>(hs), top);
          const uint32_t delta = chunk_delta<I4>(hs, a0);
          const uint32_t nch = min(chunk_count<I4>(he, a0), static_cast<uint32_t>((VT::kVbuf - 16) / 16));
          const uint32_t last = static_cast<uint32_t>((top - a0) >> 4);
          const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.values + a0);
          for (uint32_t ch = lane; ch < nch; ch += 64) reinterpret_cast<u32x4_t*>(vb)[ch] = src[min(ch, last)];
          // Entries of the other half get bases that are never read.
          tab_write(tab, s.bm, excl - (h ? mid : 0u) + delta + vb_elems, lane);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            load_x(x, c, ks);
            put_x(x);
            wave_sync();
            if (h == 0) multiply(integral_constant<int, 0>{}, integral_constant<int, 2>{}, ks);
            else multiply(integral_constant<int, 2>{}, integral_constant<int, 2>{}, ks);
          }
        }
      }
    }
  } else {
    // Loads are in the order in which they are waited for.
    Slot<NB, I4, CH> s;
    load_w(s, c_begin);
    load_x(x, c_begin, 0);
    for (int c = c_begin; c < c_end; ++c) {
      slot_commit(s, vb, lane);
      tab_write(tab, s.bm, bitmap_prefix_reg(s.bm) + s.delta + vb_elems, lane);
      put_x(x);
      wave_sync();
      load_x(x, c, 1);
      load_w(s, c + 1);
      multiply(integral_constant<int, 0>{}, integral_constant<int, 4>{}, 0);
      put_x(x);
      wave_sync();
      load_x(x, c + 1, 0);
      multiply(integral_constant<int, 0>{}, integral_constant<int, 4>{}, 1);
    }
  }

  // Workgroup reduction over waves (fixed order), the last two into the first.
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem) + (w & 1) * (4 * NB * 64) + lane;   // [2 waves][4][NB][64 lanes]
  if (w >= 2) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) red[(f * NB + nb) * 64] = acc[f][nb];
  }
  __syncthreads();
  if (w < 2) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) red[(f * NB + nb) * 64] += acc[f][nb];
  }
  __syncthreads();
  auto sum_of = [&](int n, int ml) {
    const f32x4_t* at = reinterpret_cast<const f32x4_t*>(smem) + ((ml >> 4) * NB + (n >> 4)) * 64 + 16 * ((ml >> 2) & 3) + (n & 15);
    return at[0] + at[4 * NB * 64];
  };
  finish_strip_gated<NB, I4>(a, gi, sidx, kThreads, last_flag, sum_of);
}

// 16-token blocks of a pass.
int tall_blocks(int N) {
  const int nb = (N + 15) / 16;
  return nb == 7 ? 8 : nb;
}

// Workgroups per strip, each wave of them with at least two GroupTiles: the least
// work to a compute unit, as many workgroups as its fullest has, each of 1 / s of a
// strip, where one alone hides less of its latency and each split's sums cost
// (pairs, us: 11008x4096 N = 64 1 / 2 / 3 / 4 splits 52 / 45 / 52 / 51, N = 77 58 / 62 /
// 65 / 63; 4096x4096 N = 48 2 / 3 / 4 / 5 / 6 22.7 / 22.1 / 19.9 / 22.2 / 21.5;
// 5120x2560 N = 44 2 / 3 / 4 20.0 / 18.6 / 19.9; 2048x2048 N = 40 2 / 4 / 8 15.4 /
// 14.2 / 16.6).
int tall_splits(const usw::Geometry& pair, int N) {
  const int resident = tall_blocks(N) <= 4 ? 3 : 2;
  int64_t best = 1;
  double least = 0;
  for (int64_t s = 1; s == 1 || (s <= pair.Gc / 8 && pair.Gr * s <= resident * kComputeUnits); ++s) {
    const int64_t fullest = (pair.Gr * s + kComputeUnits - 1) / kComputeUnits;
    const double cost = static_cast<double>(fullest) / s * (fullest == 1 ? 1.15 : 1.0) + 0.01 * s;
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return static_cast<int>(std::max((pair.Gc + 63 * 4 - 1) / (63 * 4), best));
}

void launch_tall(const GatedArgs& a, bool i4, bool lean, dim3 grid, hipStream_t s) {
  auto go = [&](auto blocks) {
    constexpr int NB = decltype(blocks)::value;
    if (i4) tall_kernel<NB, true, 3><<<grid, 256, 0, s>>>(a);
    else if (lean) tall_kernel<NB, false, 5><<<grid, 256, 0, s>>>(a);
    else tall_kernel<NB, false, 6><<<grid, 256, 0, s>>>(a);
  };
  switch (tall_blocks(a.N)) {
    case 3: go(std::integral_constant<int, 3>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 5: go(std::integral_constant<int, 5>{}); break;
    case 6: go(std::integral_constant<int, 6>{}); break;
    default: go(std::integral_constant<int, 8>{});
  }
}

// ---------------------------------------------------------------------------
// Many rows: both weights expanded, interleaved
// ---------------------------------------------------------------------------

struct PairExpandArgs {
  const uint64_t* bitmaps[2];
  const uint32_t* offsets[2];
  const uint8_t* values[2];
  uint64_t alloc[2];
  u32x4_t* __restrict__ dense;
  int64_t ngt;
  int Gc;
};

// GroupTile (i, c) of weight e = blockIdx.y: fragment f goes to strip
// 2 i + f / 2 of the interleaved weight, as its fragment 2 (f % 2) + e.
template <bool I4>
__global__ __launch_bounds__(64 * kExpandWaves) void expand_pair_kernel(PairExpandArgs a) {
  __shared__ __attribute__((aligned(16))) ExpandLds<I4> s;
  USW_LDS_POISON(s.vals);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = static_cast<int>(blockIdx.y);
  expand_selectors<I4>(s.lut, tid);
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kExpandWaves + w;
  if (g < a.ngt)
    expand_load<I4>(s, (e ? a.bitmaps[1] : a.bitmaps[0]) + g * kBtPerGt, (e ? a.offsets[1] : a.offsets[0]) + g,
                    e ? a.values[1] : a.values[0], e ? a.alloc[1] : a.alloc[0], w, lane);
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();
  if (g >= a.ngt) return;
  const LaneMap lm = lane_map(lane);
  const int64_t i = g / a.Gc, c = g - i * a.Gc;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    u32x4_t* out = a.dense + ((2 * i + (f >> 1)) * a.Gc + c) * 512 + 64 * (2 * (f & 1) + e) + lane;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) out[256 * ks] = __builtin_bit_cast(u32x4_t, expand_row<I4>(s, lm, w, f, ks));
  }
}

struct GatedWideArgs : WideArgs {
  GatedOperands g;
};

// Accumulators 2 q and 2 q + 1 of a wave are the two sums of the same outputs.
// What is stored (h, and g and u where they are kept) passes through LDS as in
// wide_finish, so that a row's outputs are stored together.
struct GatedFinish {
  using Args = GatedWideArgs;
  template <class C>
  __device__ static __forceinline__ void finish(uint8_t* smem, f32x4_t (&acc)[C::MF][C::NF], const WideTile& t, int wm,
                                                int wn, int me) {
    constexpr int MP = C::MF / 2, NF = C::NF;
    constexpr int kGroups = C::BM < 128 ? 1 : C::BM / 128;   // of 64 outputs
    constexpr int kStep = C::kThreads / 16, kRows = C::BN / kStep;
    const auto z = args_again<GatedWideArgs>();
    f32x4_t* stage = reinterpret_cast<f32x4_t*>(smem);
    auto unit = [](int n, int u) { return 16 * n + (u ^ (n & 15)); };
    const int M = z->M / 2, m0 = t.strip0 * (kGT / 2), m_end = min(C::BM / 2, M - m0);
    const int row = me & 15, kb = (me >> 4) & 3;
    const bool i4 = z->i4;
#pragma unroll
    for (int q = 0; q < MP; ++q) {
      const int m = 16 * (MP * wm + q) + 4 * kb;
      if (m < m_end) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i4) {
            const f32x4_t s = load_half4(z->g.scales[h] + m0 + m);
#pragma unroll
            for (int nb = 0; nb < NF; ++nb) acc[2 * q + h][nb] *= s;
          }
          if (z->g.bias[h]) {
            const f32x4_t b = load_half4(z->g.bias[h] + m0 + m);
#pragma unroll
            for (int nb = 0; nb < NF; ++nb) acc[2 * q + h][nb] += b;
          }
        }
      }
    }
    // Stores one fp32 value of each output, value(q, nb) from the accumulators.
    auto emit = [&](void* to, bool f16, auto value) {
      const int size = f16 ? 2 : 4;
      uint8_t* at0 = static_cast<uint8_t*>(to) + (static_cast<int64_t>(t.row0) * M + m0) * size;
      const auto r = __builtin_amdgcn_make_buffer_rsrc(at0, 0, ((t.n - 1) * M + m_end) * size, kBufferRsrcWord3);
#pragma unroll 1
      for (int p = 0; p < kGroups; ++p) {
        asm volatile("" : "+v"(me));
#pragma unroll
        for (int q = 0; q < MP; ++q)
          if ((MP * wm + q) / 4 == p) {
#pragma unroll
            for (int nb = 0; nb < NF; ++nb)
              stage[unit(16 * (NF * wn + nb) + row, (4 * (MP * wm + q) + kb) & 15)] = value(q, nb);
          }
        __syncthreads();
        const int u = me & 15, n0 = me >> 4, m = 64 * p + 4 * u;
#pragma unroll 4
        for (int j = 0; j < kRows; ++j) {
          const int n = n0 + kStep * j;
          const f32x4_t v = stage[unit(n, u)];
          const int off = m < m_end ? (n * M + m) * size : 0x7FFFFFF0;   // past every bound
          if (f16)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_half4(v)), r, off, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, off, 0, 0);
        }
        __syncthreads();
      }
    };
    if (z->g.pre[0]) emit(z->g.pre[0], true, [&](int q, int nb) { return acc[2 * q][nb]; });
    if (z->g.pre[1]) emit(z->g.pre[1], true, [&](int q, int nb) { return acc[2 * q + 1][nb]; });
    auto multiply = [&](auto kind) {
#pragma unroll
      for (int q = 0; q < MP; ++q)
#pragma unroll
        for (int nb = 0; nb < NF; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[2 * q][nb][i] = activation<decltype(kind)::value>(acc[2 * q][nb][i]) * acc[2 * q + 1][nb][i];
    };
    switch (z->e.act) {
      case USW_ACT_RELU: multiply(std::integral_constant<int, USW_ACT_RELU>{}); break;
      case USW_ACT_GELU: multiply(std::integral_constant<int, USW_ACT_GELU>{}); break;
      case USW_ACT_GELU_TANH: multiply(std::integral_constant<int, USW_ACT_GELU_TANH>{}); break;
      case USW_ACT_SILU: multiply(std::integral_constant<int, USW_ACT_SILU>{}); break;
      default: multiply(std::integral_constant<int, USW_ACT_NONE>{});
    }
    emit(z->Y, z->e.f16out, [&](int q, int nb) { return acc[2 * q][nb]; });
  }
};

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

struct GatedPlan {
  bool wide, tall, lean;   // many rows; 33 and more; five value chunks to a slot
  Plan p;
  usw::Geometry pair;   // both weights as one, of 2 M outputs
  usw::WidePlan w;
  size_t need, cb;
};

// Rows up to which the weights are read as they are.  tall_kernel / expanded, us:
// 11008x4096 N = 128 78 / 115, INT4 58 / 101; 4096x4096 N = 128 31.5 / 40; 2048x2048
// N = 64 15.4 / 22.4, N = 128 21.0 / 21.6; 640x512 N = 128 16.2 / 16.7.  Few strips of
// many columns leave compute units idle unless their sums are joined from many
// splits: 512x2048 N = 60 14.0 / 17.1, INT4 N = 128 21.3 / 17.9; 256x4096 N = 128 23.4 /
// 17.5.
int few_rows(const usw::Geometry& g) { return g.M < 1024 && g.K >= 2048 ? 64 : 128; }

GatedPlan plan_gated(const usw_fmt* gate, const usw_fmt* up, const usw::Geometry& g, int32_t N) {
  GatedPlan c{};
  c.pair = g;
  c.pair.M *= 2;
  c.pair.Gr *= 2;
  c.pair.ngt *= 2;
  c.wide = N > few_rows(g);
  if (c.wide) {
    c.w = usw::wide_plan(c.pair, 1, N, true);
    c.need = c.w.need;
    c.cb = c.w.cb;
    return c;
  }
  c.lean = lean_values(gate, g) && lean_values(up, g);
  c.tall = N > 32;
  if (c.tall) {
    c.p.splits = tall_splits(c.pair, N);
  } else {
    c.p = make_plan<GatedArgs>(c.pair, N, 0, gate->val_type == USW_VAL_I4, c.lean);
  }
  c.cb = usw::counter_zone(counters_bytes(g));
  c.need = c.cb + 2 * static_cast<size_t>(c.p.splits) * N * g.M * sizeof(float);
  return c;
}

// Checks the pair without its pointers.
usw_status check_pair(const usw_fmt* gate, const usw_fmt* up, int32_t y_type, int32_t N, usw::Geometry* g) {
  usw_status st = check_common(gate, y_type, N, g);
  if (st) return st;
  usw::Geometry gu;
  st = check_common(up, y_type, N, &gu);
  if (st) return st;
  if (up->M != gate->M || up->K != gate->K) return USW_ERR_BAD_SHAPE;
  if (up->val_type != gate->val_type) return USW_ERR_BAD_DTYPE;
  return g->M > kMaxLd || g->M * g->K > kMaxElements ? USW_ERR_UNSUPPORTED : USW_OK;
}

usw_status gated_impl(const usw_fmt* gate, const usw_fmt* up, const uint16_t* X, void* Y, int32_t y_type, int32_t N,
                      const usw_gated* ep, void* ws, size_t ws_bytes, void* stream) {
  usw::Geometry g;
  usw_status st = check_pair(gate, up, y_type, N, &g);
  if (st) return st;
  const bool i4 = gate->val_type == USW_VAL_I4;
  const usw_fmt* both[2] = {gate, up};
  if (!X || !Y) return USW_ERR_NULL_ARG;
  for (const usw_fmt* f : both)
    if (!f->bitmaps || !f->offsets || !f->values || (i4 && !f->scales)) return USW_ERR_NULL_ARG;
  GatedOperands o{};
  int act = USW_ACT_SILU;
  if (ep) {
    if (ep->act < USW_ACT_NONE || ep->act > USW_ACT_SILU) return USW_ERR_BAD_DTYPE;
    if (ep->reserved != 0) return USW_ERR_BAD_SHAPE;
    act = ep->act;
    o.bias[0] = ep->gate_bias;
    o.bias[1] = ep->up_bias;
    o.pre[0] = ep->pre_gate;
    o.pre[1] = ep->pre_up;
  }
  if (!aligned16(X) || !aligned16(Y)) return USW_ERR_MISALIGNED;
  for (int h = 0; h < 2; ++h) {
    const usw_fmt* f = both[h];
    if (!aligned16(f->bitmaps) || !aligned16(f->values) || (reinterpret_cast<uintptr_t>(f->offsets) & 3u) ||
        (i4 && !aligned16(f->scales)) || !aligned16(o.bias[h]) || !aligned16(o.pre[h]))
      return USW_ERR_MISALIGNED;
    o.scales[h] = i4 ? f->scales : nullptr;
  }
  const GatedPlan c = plan_gated(gate, up, g, N);
  if (c.wide && !usw::wide_launchable(c.w)) return USW_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < c.need) return USW_ERR_WORKSPACE;
  if (!aligned16(ws)) return USW_ERR_MISALIGNED;
  const Epilogue e{nullptr, nullptr, nullptr, g.M, g.M, act, y_type == USW_OUT_F16 ? 1 : 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint64_t alloc[2];
  for (int h = 0; h < 2; ++h) alloc[h] = usw::values_alloc_bytes(both[h]->val_type, both[h]->nnz);
  if (c.wide) {
    PairExpandArgs x{};
    for (int h = 0; h < 2; ++h) {
      x.bitmaps[h] = both[h]->bitmaps;
      x.offsets[h] = both[h]->offsets;
      x.values[h] = static_cast<const uint8_t*>(both[h]->values);
      x.alloc[h] = alloc[h];
    }
    x.dense = reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(ws) + c.w.dense_at);
    x.ngt = g.ngt;
    x.Gc = static_cast<int>(g.Gc);
    const dim3 grid(static_cast<unsigned>((g.ngt + kExpandWaves - 1) / kExpandWaves), 2);
    if (i4) expand_pair_kernel<true><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    else expand_pair_kernel<false><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    GatedWideArgs a{};
    fill_wide(a, c.w, c.pair, N, x.dense, ws);
    a.X = X;
    a.Y = Y;
    a.e = e;
    a.i4 = i4;
    a.g = o;
    launch_wide<GatedFinish>(c.w, a, s);
    return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
  }
  const int64_t nblk = c.pair.Gr * c.p.splits;
  GatedArgs a{};
  a.bitmaps = gate->bitmaps;
  a.offsets = gate->offsets;
  a.values = static_cast<const uint8_t*>(gate->values);
  a.values_alloc = alloc[0];
  a.up_bitmaps = up->bitmaps;
  a.up_offsets = up->offsets;
  a.up_values = static_cast<const uint8_t*>(up->values);
  a.up_alloc = alloc[1];
  a.X = X;
  a.Y = Y;
  a.counters = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + c.cb);
  a.M = static_cast<int>(g.M);
  a.K = static_cast<int>(g.K);
  a.N = N;
  a.Gc = static_cast<int>(g.Gc);
  a.splits = c.p.splits;
  a.remap = nblk % 8 == 0 ? 1 : 0;
  a.e = e;
  a.g = o;
  const dim3 grid(static_cast<unsigned>(nblk));
  if (c.tall) launch_tall(a, i4, c.lean, grid, s);
  else launch_pass(a, c.p.ring, i4, c.lean, c.p.nchunk / 16, e.f16out, grid, s);
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

}  // namespace

extern "C" {

usw_status usw_spmm_gated_workspace(const usw_fmt* gate, const usw_fmt* up, int32_t N, size_t* bytes,
                                    size_t* counter_bytes) {
  if (!bytes || !counter_bytes) return USW_ERR_NULL_ARG;
  usw::Geometry g;
  usw_status st = check_pair(gate, up, USW_OUT_F16, N, &g);
  if (st) return st;
  const GatedPlan c = plan_gated(gate, up, g, N);
  if (c.wide && !usw::wide_launchable(c.w)) return USW_ERR_UNSUPPORTED;
  *bytes = c.need;
  *counter_bytes = c.cb;
  return USW_OK;
}

usw_status usw_spmm_gated(const usw_fmt* gate, const usw_fmt* up, const uint16_t* X, void* Y, int32_t y_type, int32_t N,
                          const usw_gated* ep, void* ws, size_t ws_bytes, void* stream) {
  return gated_impl(gate, up, X, Y, y_type, N, ep, ws, ws_bytes, stream);
}

}  // extern "C"
