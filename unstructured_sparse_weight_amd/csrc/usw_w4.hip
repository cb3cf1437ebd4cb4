// The dense 4-bit weight with a scale for each group of a row's columns
// (usw_w4_*): encoder, and the product with an epilogue
//
//   y[n][m] = res[n][m] + mul[n][m] * act(sum_k w[m][k] x[n][k] + bias[m]),
//   w[m][k] = fp16(code[m][k] * scale[m][k / group]),
//
// for the layers that pruning leaves dense.  The scales that the encoder makes
// have 8 significant bits and codes at most 4, so w is the product itself and
// nothing is rounded before the fp32 sums.
//
// Few rows (w4_kernel): bound by the codes' bytes.  A tile of the format, 16
// rows by 128 columns, is the 1 KB that one load of a wave brings, and lane
// 16 g + r holds the 32 codes of row r, columns 32 g on: eight columns are one
// dword and one lane's share of a v_mfma_f32_16x16x32_f16 operand, whose
// reduction index is any order of columns that x's fragment has too.  So codes
// go from memory to the matrix cores through registers alone.
//   * Unpacking: nibbles t and t + 4 of a dword are columns 2 t and 2 t + 1;
//     masked into the mantissas of 1024 or 64 they are fp16 numbers, and one
//     packed subtraction and one packed multiplication by the scale, both
//     exact, make two weights.
//   * x goes through LDS, so that four lanes read 64 bytes of a token.
//   * The waves of a workgroup share a strip of 16 R rows and split its
//     columns; their sums meet in LDS in a fixed order, so no such call needs a
//     workspace and results do not depend on timing.
// 20480x5120 N = 16: 57 MB in 15.2 us, 3.7 TB/s; 11008x4096 N = 1 8.2.
// Many rows: the weight is expanded to dense fp16 fragments and multiplied as
// the sparse weights are (usw_wide.hip).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "usw.h"
#include "usw_checks.h"
#include "usw_device.h"
#include "usw_epilogue.h"
#include "usw_internal.h"
#include "usw_quant.h"
#include "usw_w4.h"
#include "usw_wide.h"

namespace {

using namespace usw_dev;

constexpr int kTileRows = usw::kW4Rows, kTileCols = usw::kW4Cols;

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

// The eight weights of a dword of codes (stored plus 8) under scale s.
__device__ __forceinline__ half8_t unpack8(uint32_t c, half2_t s) {
  const half2_t k1032 = {static_cast<_Float16>(1032.0f), static_cast<_Float16>(1032.0f)};
  const half2_t k72 = {static_cast<_Float16>(72.0f), static_cast<_Float16>(72.0f)};
  u32x4_t w;
#pragma unroll
  for (int t = 0; t < 4; t += 2) {
    const uint32_t v = c >> (4 * t);
    // 0x6400 | u is 1024 + u, 0x5400 | u << 4 is 64 + u.
    const half2_t a = __builtin_bit_cast(half2_t, (v & 0x000F000Fu) | 0x64006400u) - k1032;
    const half2_t b = __builtin_bit_cast(half2_t, (v & 0x00F000F0u) | 0x54005400u) - k72;
    w[t] = __builtin_bit_cast(uint32_t, a * s);
    w[t + 1] = __builtin_bit_cast(uint32_t, b * s);
  }
  return __builtin_bit_cast(half8_t, w);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------

struct W4Args {
  const u32x4_t* __restrict__ codes;
  const uint16_t* __restrict__ scales;
  const uint16_t* __restrict__ X;
  void* Y;
  Epilogue e;
  int M, K, N, tiles;    // tiles: of a row block
  int lg_groups;         // log2 of the groups of a tile
};

// What a wave loads for one tile column: codes and scales of R row blocks, and
// x, piece 4 i + l % 4 of token 16 nb + l / 4 in lane l.
template <int R, int NB>
struct W4Slot {
  u32x4_t c[R];
  uint32_t s[R];
  u32x4_t x[NB][4];
};

constexpr uint32_t kBehind = 0x7FFFFE00u;   // past every buffer here

// D: tile columns loaded ahead.
template <int R, int NB, int W, int D>
__global__ __launch_bounds__(64 * W) void w4_kernel(W4Args a) {
  constexpr int kX = 4096 * NB;
  constexpr int kRed = W * R * NB * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t smem[W * kX > kRed ? W * kX : kRed];
  USW_LDS_POISON(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int b0 = static_cast<int>(blockIdx.x) * R, blocks = a.M / kTileRows;
  const int t0 = static_cast<int>(static_cast<int64_t>(a.tiles) * w / W);
  const int t1 = static_cast<int>(static_cast<int64_t>(a.tiles) * (w + 1) / W);

  // Row blocks past the last repeat it; nothing of theirs is stored.
  const u32x4_t* csrc[R];
  const uint16_t* ssrc[R];
  const int group = (g << a.lg_groups) >> 2;   // the lane's group of a tile
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t b = static_cast<int64_t>(min(b0 + i, blocks - 1)) * a.tiles;
    csrc[i] = a.codes + b * 64 + lane;
    ssrc[i] = a.scales + ((b << a.lg_groups) + group) * kTileRows + r;
  }
  // x through a buffer: tokens past the last and columns past the row read as
  // zeros, whatever lies behind them.  Four lanes read 64 bytes of a token; as
  // the matrix operand lies, each would be of another token and cost the
  // address unit four times as much.
  const auto xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.X), 0, a.N * a.K * 2, kBufferRsrcWord3);
  const int xn = lane >> 2, xp = lane & 3;
  uint32_t xoff[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int n = 16 * nb + xn;
    xoff[nb] = n < a.N ? static_cast<uint32_t>(n * a.K + 8 * xp) * 2u : kBehind;
  }
  auto load = [&](W4Slot<R, NB>& s, int t) {
    t = min(t, t1 - 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s.c[i] = __builtin_nontemporal_load(csrc[i] + static_cast<int64_t>(t) * 64);
      s.s[i] = ssrc[i][static_cast<int64_t>(t) * (kTileRows << a.lg_groups)];
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // K is a multiple of 64: a tile's half is in the row or is not.  The
        // scalar offset is the tile's start, inside x: the bound is taken less it.
        const uint32_t at = (i < 2 || kTileCols * t + 64 < a.K ? xoff[nb] : kBehind) + 64u * i;
        s.x[nb][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xr, static_cast<int>(at), 256 * t, 0));
      }
  };
  // The wave's x tile in LDS: token n's piece p at p ^ (4 (n % 4) + n / 4 % 4) of
  // its 16, which keeps both the writes and the reads below off each other's
  // banks.
  uint8_t* xt = smem + w * kX;
  uint8_t* xput = xt + 256 * xn;
  const int xflip = 4 * (xn & 3) + (xn >> 2), rflip = 4 * (r & 3) + (r >> 2);
  const uint8_t* xget = xt + 256 * r;

  f32x4_t acc[R][NB];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[i][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const W4Slot<R, NB>& s) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x4_t*>(xput + 4096 * nb + 16 * ((4 * i + xp) ^ xflip)) = s.x[nb][i];
    wave_sync();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      half8_t x[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        x[nb] = *reinterpret_cast<const half8_t*>(xget + 4096 * nb + 16 * ((4 * g + j) ^ rflip));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const _Float16 h = __builtin_bit_cast(_Float16, static_cast<uint16_t>(s.s[i]));
        const half8_t v = unpack8(s.c[i][j], half2_t{h, h});
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          acc[i][nb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, x[nb], acc[i][nb], 0, 0, 0);
      }
    }
    wave_sync();
  };
  if (t0 < t1) {
    W4Slot<R, NB> s[D + 1];
#pragma unroll
    for (int i = 0; i < D; ++i) load(s[i], t0 + i);
    int t = t0;
    for (; t + D < t1; t += D + 1) {
#pragma unroll
      for (int i = 0; i <= D; ++i) {
        load(s[(i + D) % (D + 1)], t + i + D);
        multiply(s[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (t + i < t1) multiply(s[i]);
  }
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem);   // [W][R][NB][64 lanes]
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) red[((w * R + i) * NB + nb) * 64 + lane] = acc[i][nb];
  __syncthreads();
  // Thread e takes outputs 16 (b0 + i) + 4 q on of token n: lane 16 q + n % 16
  // of block (i, n / 16).
  for (int e = tid; e < R * NB * 64; e += 64 * W) {
    const int n = e / (4 * R), mq = e - n * (4 * R), i = mq >> 2;
    if (n >= a.N || b0 + i >= blocks) continue;
    const int at = (i * NB + (n >> 4)) * 64 + 16 * (mq & 3) + (n & 15);
    f32x4_t sum = red[at];
#pragma unroll
    for (int ww = 1; ww < W; ++ww) sum += red[ww * R * NB * 64 + at];
    epilogue_store4(a.e, a.Y, a.M, n, b0 * kTileRows + 4 * mq, sum);
  }
}

// ---------------------------------------------------------------------------
// Many rows: the weight expanded
// ---------------------------------------------------------------------------

constexpr int kExpandW4Waves = 4;

// A wave takes one tile: quarter g of lane 16 g + r is half column g % 2 of
// GroupTile column 2 t + g / 2, dword j the lane 16 j + r of its fragment.
// Row blocks past the last, up to the end of its strip, are zeros.
__global__ __launch_bounds__(64 * kExpandW4Waves) void expand_w4_kernel(const u32x4_t* __restrict__ codes,
                                                                        const uint16_t* __restrict__ scales,
                                                                        u32x4_t* __restrict__ dense, int blocks,
                                                                        int tiles, int Gc, int lg_groups) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kExpandW4Waves + (threadIdx.x >> 6);
  const int b = static_cast<int>(id / tiles), t = static_cast<int>(id - static_cast<int64_t>(b) * tiles);
  if (b >= (blocks + 3) / 4 * 4) return;
  const int c = 2 * t + (g >> 1);
  if (c >= Gc) return;
  u32x4_t v = {0u, 0u, 0u, 0u};
  half2_t scale = {};
  if (b < blocks) {
    v = codes[id * 64 + lane];
    const _Float16 h = __builtin_bit_cast(_Float16, scales[((id << lg_groups) + ((g << lg_groups) >> 2)) * kTileRows + r]);
    scale = half2_t{h, h};
  }
  u32x4_t* out = dense + (static_cast<int64_t>(b >> 2) * Gc + c) * 512 + 64 * (4 * (g & 1) + (b & 3)) + r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const half8_t w = b < blocks ? unpack8(v[j], scale) : half8_t{};
    out[16 * j] = __builtin_bit_cast(u32x4_t, w);
  }
}

// ---------------------------------------------------------------------------
// Encoder
// ---------------------------------------------------------------------------

// A wave takes one tile, lane 16 g + r the 32 columns from 32 g on of row r: the
// group's largest magnitude comes from the lanes 16 or 32 apart.  Columns past
// the row count as zeros.
__global__ __launch_bounds__(256) void w4_encode_kernel(const uint16_t* __restrict__ W, u32x4_t* __restrict__ codes,
                                                        uint16_t* __restrict__ scales, int64_t all, int tiles, int K,
                                                        int lg_groups) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (id >= all) return;
  const int64_t b = id / tiles;
  const int t = static_cast<int>(id - b * tiles);
  const int k0 = kTileCols * t + 32 * g;
  u32x4_t v[4];
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = u32x4_t{0u, 0u, 0u, 0u};
    if (k0 < K) v[j] = *reinterpret_cast<const u32x4_t*>(W + (b * kTileRows + r) * K + k0 + 8 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) most = max(most, max(v[j][i] & 0x7FFFu, (v[j][i] >> 16) & 0x7FFFu));
  }
  if (lg_groups < 2) most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 16)));
  if (lg_groups < 1) most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 32)));
  const uint16_t bits = usw::w4_scale_bits(static_cast<uint16_t>(most));
  const double s = usw::f16_to_f64(bits);
  u32x4_t q;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t x = static_cast<uint16_t>(v[j][i >> 1] >> (16 * (i & 1)));
      d |= static_cast<uint32_t>(usw::i4_code(x, s) + 8) << usw::w4_shift(i);
    }
    q[j] = d;
  }
  codes[id * 64 + lane] = q;
  const int per = 4 >> lg_groups;   // lanes of a row's group
  if ((g & (per - 1)) == 0) scales[((id << lg_groups) + ((g << lg_groups) >> 2)) * kTileRows + r] = bits;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

struct W4Plan {
  bool wide;
  usw::Geometry g;
  usw::WidePlan w;
  size_t need, cb;
};

// Rows of a pass over the codes, and up to which such passes are taken (MI355X,
// passes / expanded, us: 8192x8192 N = 192 65 / 74, 193 84 / 74; 11008x4096 N = 192
// 46 / 58, 193 60 / 58; 16384x4096 N = 192 57 / 69, 193 74 / 69; fewer outputs leave
// compute units without a row block: 4096x11008 N = 128 52 / 51, 160 75 / 57;
// 4096x4096 N = 128 25.0 / 26.8, 160 35 / 31; 2048x1024 N = 128 14.7 / 16.1, 160
// 17.7 / 15.8).  A dense weight of more than 192 MiB, with the codes, does not stay in
// the 256 MB cache between its expansion and its product: 20480x5120 N = 256 100 /
// 139, 320 125 / 143, 16384x8192 N = 320 154 / 228, 28672x8192 N = 320 285 / 350,
// 28672x4096 N = 256 136 / 156, 320 170 / 168; just below, 24576x4096 N = 193 112 /
// 100, 12288x8192 N = 256 106 / 115.  With few columns a pass is mostly its start:
// 65536x2048 N = 193 175 / 137, 40960x2560 N = 320 152 / 142.
constexpr int kPassRows = 64;
int few_rows(int64_t outputs, int64_t columns) {
  if (outputs < 8192) return 128;
  return columns >= 4096 && outputs * columns * 2 > int64_t(192) << 20 ? 320 : 192;
}

W4Plan plan_w4(const usw_w4_fmt* f, int32_t N) {
  W4Plan p{};
  p.wide = N > few_rows(f->M, f->K);
  if (!p.wide) return p;
  p.g.M = f->M;
  p.g.K = f->K;
  p.g.Gr = (f->M + kGT - 1) / kGT;
  p.g.Gc = f->K / kGT;
  p.w = usw::wide_plan(p.g, 1, N, true);
  p.cb = p.w.cb;
  p.need = p.w.dense_at + static_cast<size_t>(p.g.Gr) * kGT * f->K * 2;
  return p;
}

usw_status check_w4(const usw_w4_fmt* f, int32_t y_type, int32_t N) {
  if (!f) return USW_ERR_NULL_ARG;
  usw_status st = usw::check_w4_shape(f->M, f->K, f->group);
  if (st) return st;
  if (f->reserved != 0) return USW_ERR_BAD_SHAPE;
  if (y_type != USW_OUT_F16 && y_type != USW_OUT_F32) return USW_ERR_BAD_DTYPE;
  if (N < 1) return USW_ERR_BAD_N;
  if (static_cast<int64_t>(N) * f->M > (int64_t(1) << 40)) return USW_ERR_BAD_SHAPE;
  return USW_OK;
}

// Row blocks of a workgroup: more of them share x's way through LDS, fewer spread
// the codes over the compute units.  A workgroup's time is about R + share, and
// each round of one to a compute unit adds that (MI355X, R = 1 / 2 / 3 / 4 / 5, us;
// N = 16: 20480x5120 21.8 / 18.0 / 16.0 / 20.2 / 15.1, 16384x4096 14.9 / 10.8 / 12.7
// / 10.7 / 13.5, 8192x8192 16.0 / 11.1 / 12.7 / 15.1 / 17.9; N = 32: 20480x5120 33.2 /
// 28.3 / 24.2 / 26.3 / 21.5, 11008x4096 19.0 / 15.5 / 12.9 / 13.1 / 16.7; N = 64:
// 20480x5120 62.8 / 42.5 / 36.7 / 41.4 / 29.1, 11008x4096 33.0 / 23.7 / 17.6 / 19.9 /
// 22.0).  More than five are behind two rounds of fewer: 28672x4096 N = 4 18.1 with
// three, 18.5 with seven.  Of up to 16 rows, more than one round is of workgroups of
// three or four (128256x4096 N = 1 48.8 / 50.2, with five 53.6, N = 16 60.2 / 57.3 and
// 59.3).
constexpr int kComputeUnits = 256;
int row_blocks(int64_t blocks, int NB) {
  const double share = NB == 1 ? 1.5 : NB == 2 ? 2.5 : 4.0;
  const int most = NB == 1 && blocks > 5 * kComputeUnits ? 4 : 5;
  int best = 1;
  double least = 0;
  for (int r = 1; r <= most; ++r) {
    const double rounds = static_cast<double>((blocks + kComputeUnits * r - 1) / (kComputeUnits * r));
    const double cost = rounds * (r + share);
    if (r == 1 || cost < least) {
      best = r;
      least = cost;
    }
  }
  return best;
}

template <int R, int NB, int W, int D>
void launch_w4_as(const W4Args& a, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(a.M / kTileRows);
  w4_kernel<R, NB, W, D><<<(blocks + R - 1) / R, 64 * W, 0, s>>>(a);
}

// Waves: eight, or four where two workgroups or more come to a compute unit, or
// the rows' accumulators leave no registers for eight (us, four / eight waves: N = 1,
// R = 4: 28672x4096 15.0 / 19.0, 28672x8192 28.5 / 31.6, 65536x4096 27.3 / 37.1;
// one workgroup to a compute unit 20480x5120, R = 5, 15.3 / 12.7; N = 32, R = 2:
// 11008x4096 14.2 / 17.4).  Sixteen are behind eight (N = 1: 2048x1024 3.3 / 2.7,
// 1024x28672 15.4 / 15.4, N = 32: 1024x4096 8.3 / 7.1).
// One tile ahead.  Two where a workgroup has one row block of up to 16 rows, and
// a wave two tiles or more (one / two ahead, N = 1: 4096x11008 9.8 / 8.6,
// 1024x28672 18.6 / 15.4, 4096x2048 3.9 / 3.6, of one tile each 4096x1024 3.1 / 3.3;
// of more row blocks 28672x4096, R = 2, 18.6 / 18.1, 11008x4096 9.9 / 10.5; N = 32:
// 4096x11008 15.5 / 16.6).
template <int NB>
void launch_w4(const W4Args& a, hipStream_t s) {
  const int64_t blocks = a.M / kTileRows;
  const int r = row_blocks(blocks, NB);
  if constexpr (NB == 1) {
    // Two or five row blocks are one round here, three and four also more.
    const bool one = blocks <= kComputeUnits * r;
    switch (r) {
      case 1: return a.tiles >= 16 ? launch_w4_as<1, NB, 8, 2>(a, s) : launch_w4_as<1, NB, 8, 1>(a, s);
      case 2: return launch_w4_as<2, NB, 8, 1>(a, s);
      case 3: return one ? launch_w4_as<3, NB, 8, 1>(a, s) : launch_w4_as<3, NB, 4, 1>(a, s);
      case 4: return one ? launch_w4_as<4, NB, 8, 1>(a, s) : launch_w4_as<4, NB, 4, 1>(a, s);
      default: return launch_w4_as<5, NB, 8, 1>(a, s);
    }
  } else {
    switch (r) {
      case 1: return launch_w4_as<1, NB, 8, 1>(a, s);
      case 2: return launch_w4_as<2, NB, 4, 1>(a, s);
      case 3: return launch_w4_as<3, NB, 4, 1>(a, s);
      case 4: return launch_w4_as<4, NB, 4, 1>(a, s);
      default: return launch_w4_as<5, NB, 4, 1>(a, s);
    }
  }
}

usw_status w4_impl(const usw_w4_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N, const usw_epilogue* ep,
                   void* ws, size_t ws_bytes, void* stream) {
  usw_status st = check_w4(f, y_type, N);
  if (st) return st;
  if (!X || !Y || !f->codes || !f->scales) return USW_ERR_NULL_ARG;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(f->codes) || !aligned16(f->scales)) return USW_ERR_MISALIGNED;
  Epilogue e;
  st = make_epilogue(ep, f->M, y_type, &e);
  if (st) return st;
  const W4Plan p = plan_w4(f, N);
  if (p.wide && !usw::wide_launchable(p.w)) return USW_ERR_UNSUPPORTED;
  if (p.need > 0) {
    if (!ws || ws_bytes < p.need) return USW_ERR_WORKSPACE;
    if (!aligned16(ws)) return USW_ERR_MISALIGNED;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tiles = usw::w4_tiles(f->K), lg = f->group == 32 ? 2 : f->group == 64 ? 1 : 0;
  if (p.wide) {
    void* dense = static_cast<uint8_t*>(ws) + p.w.dense_at;
    const int64_t all = p.g.Gr * 4 * tiles;
    expand_w4_kernel<<<static_cast<unsigned>((all + kExpandW4Waves - 1) / kExpandW4Waves), 64 * kExpandW4Waves, 0, s>>>(
        static_cast<const u32x4_t*>(f->codes), f->scales, static_cast<u32x4_t*>(dense), f->M / kTileRows, tiles,
        static_cast<int>(p.g.Gc), lg);
    return usw::wide_multiply(p.g, p.w, N, X, Y, e, dense, ws, stream);
  }
  // Passes of equal length, up to 64 rows.
  const int passes = (N + kPassRows - 1) / kPassRows;
  for (int i = 0; i < passes; ++i) {
    const int n0 = static_cast<int>(static_cast<int64_t>(N) * i / passes), n1 = static_cast<int>(static_cast<int64_t>(N) * (i + 1) / passes);
    W4Args a{};
    a.codes = static_cast<const u32x4_t*>(f->codes);
    a.scales = f->scales;
    a.X = X + static_cast<int64_t>(n0) * f->K;
    a.Y = static_cast<uint8_t*>(Y) + static_cast<int64_t>(n0) * f->M * (e.f16out ? 2 : 4);
    a.e = e;
    if (e.mul) a.e.mul += e.ld_mul * n0;
    if (e.res) a.e.res += e.ld_res * n0;
    a.M = f->M;
    a.K = f->K;
    a.N = n1 - n0;
    a.tiles = tiles;
    a.lg_groups = lg;
    if (a.N <= 16) launch_w4<1>(a, s);
    else if (a.N <= 32) launch_w4<2>(a, s);
    else launch_w4<4>(a, s);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

}  // namespace

extern "C" {

usw_status usw_w4_encode_device(const uint16_t* W, int32_t M, int32_t K, int32_t group, void* codes, uint16_t* scales,
                                void* stream) {
  usw_status st = usw::check_w4_shape(M, K, group);
  if (st) return st;
  if (!W || !codes || !scales) return USW_ERR_NULL_ARG;
  if (!aligned16(W) || !aligned16(codes) || !aligned16(scales)) return USW_ERR_MISALIGNED;
  const int tiles = usw::w4_tiles(K);
  const int64_t all = static_cast<int64_t>(M / kTileRows) * tiles;
  w4_encode_kernel<<<static_cast<unsigned>((all + 3) / 4), 256, 0, static_cast<hipStream_t>(stream)>>>(
      W, static_cast<u32x4_t*>(codes), scales, all, tiles, K, group == 32 ? 2 : group == 64 ? 1 : 0);
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

usw_status usw_w4_matmul_workspace(const usw_w4_fmt* f, int32_t N, size_t* bytes, size_t* counter_bytes) {
  if (!bytes || !counter_bytes) return USW_ERR_NULL_ARG;
  usw_status st = check_w4(f, USW_OUT_F16, N);
  if (st) return st;
  const W4Plan p = plan_w4(f, N);
  if (p.wide && !usw::wide_launchable(p.w)) return USW_ERR_UNSUPPORTED;
  *bytes = p.need;
  *counter_bytes = p.cb;
  return USW_OK;
}

usw_status usw_w4_matmul(const usw_w4_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N,
                         const usw_epilogue* ep, void* ws, size_t ws_bytes, void* stream) {
  return w4_impl(f, X, Y, y_type, N, ep, ws, ws_bytes, stream);
}

}  // extern "C"
