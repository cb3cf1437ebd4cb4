// Gradients of the sparse products, of one weight (usw_spmm_backward) and of
// the gated block (usw_spmm_gated_backward).  With d the gradient of the
// sums y = W_sp x + b (one row per token),
//
//   dx[n][k] = sum_m W_sp[m][k] d[n][m],
//   dV[i]    = sum_n d[n][m_i] x[n][k_i]   for the kept value i at (m_i, k_i),
//   db[m]    = sum_n d[n][m],
//
// and for h = act(g) * u:  dg = dh u act'(g),  du = dh act(g), whose dx add up.
//
// Few rows have kernels of their own (usw_grad_few.hip).  Of many, both large sums
// are the expanded product (usw_wide_kernels.h) on other operands, so they run at
// its rate (pairs of 11008x4096 N = 2048: dx 340 us, 1.09 PFLOP/s, dV 357):
//   * dx takes the weight's GroupTiles expanded in transposed order.  The two
//     weights of a gated block lie behind each other along the reduction, as
//     dg and du do, and one product adds them.
//   * dV takes x transposed as the "weight" and d transposed as the rows; its
//     tiles cover the whole matrix, and the epilogue keeps the values whose
//     bitmap bits are set (sampling inside the product would leave most of a
//     matrix instruction idle at the densities of this format).
// One pass over dh, g and u makes d in the orders that are asked for, x's
// transpose and the biases' sums.
//
// Precision: sums, activations and their slopes are fp32.  The matrix cores
// take fp16: dg and du are rounded once (d of a single product is an input,
// exact).  INT4 rows keep their code's power of two in the weight and the rest
// of their scale, in [0.5, 1), in d, which is rounded once then.  A rounding of d
// is as large as that of the result, and independent: sqrt(2) of its error alone.
// Up to 32 rows the remainders go along as more columns of d, which costs a
// second matrix operation on each rebuilt weight (pairs of 4096x4096 N = 10 5%);
// where INT4's dx is fp32 and the rows are more, as a second block with the weight
// once more.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "usw.h"
#include "usw_checks.h"
#include "usw_grad.h"
#include "usw_grad_values.h"
#include "usw_internal.h"
#include "usw_wide.h"
#include "usw_wide_kernels.h"

namespace {

using namespace usw_dev;

constexpr int64_t kMaxElements = int64_t(1) << 34;   // of a weight, and tokens by outputs or columns: launches
constexpr int64_t kMaxD = int64_t(1) << 35;          // stay below HIP's 2^32 threads (check_back has d's pass)

// ---------------------------------------------------------------------------
// d in the orders of the two products
// ---------------------------------------------------------------------------

// The activation and its slope.  p is the logistic function of v (SiLU) or of
// 2 z (GELU's tanh form), or the normal distribution's (GELU).  A g beyond fp16 is
// kept as an infinity, where p is 0 or 1 and its product with v, or 1 - p's, would be
// a NaN: there the limits are taken, by v's nearest finite fp16 numbers.  A NaN is
// in p.
template <int ACT>
__device__ __forceinline__ void act_and_slope(float v, float* a, float* s) {
  const float left = fmaxf(v, -65504.0f), near = fminf(left, 65504.0f);
  if constexpr (ACT == USW_ACT_RELU) {
    *a = v < 0.0f ? 0.0f : v;
    *s = v > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == USW_ACT_GELU) {
    const float p = 0.5f * erfcf(v * -0.70710678118654752f);
    *a = left * p;
    *s = p + near * (0.39894228040143268f * __expf(-0.5f * v * v));
  } else if constexpr (ACT == USW_ACT_GELU_TANH) {
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    *a = left * p;
    *s = p + near * (1.5957691216057308f * (1.0f + 0.134145f * near * near)) * (p * (1.0f - p));
  } else if constexpr (ACT == USW_ACT_SILU) {
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
    *a = left * p;
    *s = p + near * (p * (1.0f - p));
  } else {
    *a = v;
    *s = 1.0f;
  }
}

struct PrepArgs {
  const uint16_t* __restrict__ dY;      // [N][M]
  const uint16_t* __restrict__ g;       // gated: [N][M] pre-activations
  const uint16_t* __restrict__ u;
  const uint16_t* __restrict__ scales[2];   // INT4
  uint16_t* __restrict__ D;             // [N][ldD] rows for dx or few rows' dV, or null
  uint16_t* __restrict__ F;             // fragments of frag blocks of 16 tokens for few rows' dx, or null
  int frag;
  uint16_t* __restrict__ T;             // d transposed for dV, [weights * M][64 chunks], or null
  float* __restrict__ sums;             // [64-token chunk][weights * M] for db
  float* db[2];                         // or null; with one chunk its sums are final
  const uint16_t* __restrict__ X;       // [N][K] and
  u32x4_t* __restrict__ xt;             // its transpose's fragments, for dV
  int64_t N, ldD;
  int M, K, Gr, chunks;
  int lo;                               // > 0: the remainders of D's rounding go this many columns on
};

constexpr int kPrepLd = 72;   // halves of an LDS row: 64 and a pad that keeps 16-byte pieces aligned

// 64 tokens by 64 columns of x to its transpose, zeros behind token N: fragment
// (f, ks) of strip `block`, 64-token column `chunk`, whose lane l holds column
// 16 f + l % 16, tokens 32 ks + 8 (l / 16) on.
__device__ __forceinline__ void transpose_x(const PrepArgs& a, uint16_t* tile, int block, int chunk, int tid) {
  const int col = 8 * (tid & 7), k0 = block * kGT, lane = tid & 63, w = tid >> 6;
  const int64_t n0 = static_cast<int64_t>(chunk) * kGT;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (tid >> 3) + 32 * i;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (n0 + r < a.N) v = *reinterpret_cast<const u32x4_t*>(a.X + (n0 + r) * a.K + k0 + col);
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[(col + j) * kPrepLd + r] = static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1)));
  }
  __syncthreads();
  u32x4_t* out = a.xt + (static_cast<int64_t>(block) * a.chunks + chunk) * 512 + lane;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = w + 4 * i, f = p & 3, ks = p >> 2;
    out[64 * p] = *reinterpret_cast<const u32x4_t*>(&tile[(16 * f + (lane & 15)) * kPrepLd + 32 * ks + 8 * (lane >> 4)]);
  }
}

// A workgroup takes 64 tokens by 64 outputs; a thread two pieces of 8 outputs,
// 32 tokens apart.  Bound by memory: reads 2 (gated 6) bytes for each element
// and writes 2 for each order and weight (11008 outputs, 2048 tokens, with x's
// transpose of 4096 columns: 349 MB in 60 us, 5.8 TB/s).  Workgroups behind the
// outputs' transpose x.
template <bool GATED, int ACT>
__global__ __launch_bounds__(256) void prep_kernel(PrepArgs a) {
  constexpr int NW = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) _Float16 tile[NW][kGT * kPrepLd];
  __shared__ float red[NW][4][kGT];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int m0 = static_cast<int>(blockIdx.x) * kGT, col = 8 * (tid & 7);
  const int chunk = static_cast<int>(blockIdx.y);
  if (static_cast<int>(blockIdx.x) >= a.Gr) {
    transpose_x(a, reinterpret_cast<uint16_t*>(tile[0]), static_cast<int>(blockIdx.x) - a.Gr, chunk, tid);
    return;
  }
  float sum[NW][8], scale[NW][8];
#pragma unroll
  for (int h = 0; h < NW; ++h) {
    half8_t s;
    if (a.scales[h]) s = *reinterpret_cast<const half8_t*>(a.scales[h] + m0 + col);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum[h][j] = 0.0f;
      if (a.scales[h]) scale[h][j] = scale_rest(static_cast<float>(s[j]));
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (tid >> 3) + 32 * i;
    const int64_t n = static_cast<int64_t>(chunk) * kGT + r;
    float d[NW][8];
    if (n < a.N) {
      const int64_t at = n * a.M + m0 + col;
      const half8_t dy = *reinterpret_cast<const half8_t*>(a.dY + at);
      if constexpr (GATED) {
        const half8_t g = *reinterpret_cast<const half8_t*>(a.g + at), u = *reinterpret_cast<const half8_t*>(a.u + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float act, slope;
          act_and_slope<ACT>(static_cast<float>(g[j]), &act, &slope);
          const float dh = static_cast<float>(dy[j]);
          d[0][j] = dh * static_cast<float>(u[j]) * slope;
          d[1][j] = dh * act;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[0][j] = static_cast<float>(dy[j]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < NW; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[h][j] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < NW; ++h) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[h][j] += d[h][j];
      if ((a.D && n < a.N) || (a.F && n < 16 * a.frag)) {   // fragments: zeros behind the last token
        half8_t v, rest;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = a.scales[h] ? d[h][j] * scale[h][j] : d[h][j];
          v[j] = static_cast<_Float16>(x);
          const float seen = static_cast<float>(v[j]);
          rest[j] = static_cast<_Float16>(__builtin_isinf(seen) ? 0.0f : x - seen);   // not inf - inf
        }
        const int64_t at = static_cast<int64_t>(h) * a.M + m0 + col;
        if (a.D && n < a.N) {
          uint16_t* out = a.D + n * a.ldD + at;
          *reinterpret_cast<half8_t*>(out) = v;
          if (a.lo) *reinterpret_cast<half8_t*>(out + a.lo) = rest;
        }
        if (a.F) {
          uint16_t* out = a.F + ((at >> 5) * a.frag + (n >> 4)) * 512 + 128 * ((at >> 3) & 3) + 8 * (n & 15);
          *reinterpret_cast<half8_t*>(out) = v;
          if (a.lo) *reinterpret_cast<half8_t*>(out + static_cast<int64_t>(16) * a.frag * a.lo) = rest;
        }
      }
      if (a.T) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[h][(col + j) * kPrepLd + r] = static_cast<_Float16>(d[h][j]);
      }
    }
  }
  const bool bias = a.db[0] || a.db[1];
  if (bias) {
    // Over the 8 lanes of a wave with the same columns, then over the waves.
#pragma unroll
    for (int h = 0; h < NW; ++h)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = sum[h][j];
        v += __shfl_xor(v, 8);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (lane < 8) red[h][w][col + j] = v;
      }
  }
  __syncthreads();
  if (bias && tid < kGT * NW) {
    const int h = tid >> 6, m = tid & 63;
    float* to = h ? a.db[1] : a.db[0];
    if (a.chunks > 1) to = a.sums + (static_cast<int64_t>(chunk) * NW + h) * a.M;
    if (to) to[m0 + m] = (red[h][0][m] + red[h][1][m]) + (red[h][2][m] + red[h][3][m]);
  }
  if (a.T) {
#pragma unroll
    for (int h = 0; h < NW; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = (tid >> 3) + 32 * i;
        *reinterpret_cast<u32x4_t*>(a.T + (static_cast<int64_t>(h) * a.M + m0 + m) * a.chunks * kGT + chunk * kGT + col) =
            *reinterpret_cast<const u32x4_t*>(&tile[h][m * kPrepLd + col]);
      }
  }
}

// db[m] = the chunks' sums in order.
__global__ __launch_bounds__(256) void bias_kernel(const float* __restrict__ sums, float* db0, float* db1, int M, int nw,
                                                   int chunks) {
  const int i = static_cast<int>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= nw * M) return;
  float v = 0.0f;
  for (int c = 0; c < chunks; ++c) v += sums[static_cast<int64_t>(c) * nw * M + i];
  float* db = i < M ? db0 : db1;
  if (db) db[i < M ? i : i - M] = v;
}

// ---------------------------------------------------------------------------
// The weight's transpose
// ---------------------------------------------------------------------------

struct ExpandTArgs {
  const uint64_t* bitmaps[2];
  const uint32_t* offsets[2];
  const uint8_t* values[2];
  const uint16_t* scales[2];
  uint64_t alloc[2];
  u32x4_t* __restrict__ dense;
  int64_t ngt;
  int Gr, Gc, blocks;   // blocks: of Gr columns each of the transposed weights
};

// GroupTile (i, c) of block e = blockIdx.y is strip c, column e Gr + i of the
// transposed weights.  The wave's rows pass through LDS: written as they are
// rebuilt (8 columns of an output), read 8 outputs of a column.  Bound by memory:
// two weights of 11008x4096 283 MB in 50 us, 5.7 TB/s.
template <bool I4>
__global__ __launch_bounds__(64 * kExpandWaves) void expand_t_kernel(ExpandTArgs a) {
  constexpr int kTile = 2 * kGT * kPrepLd;   // 9 KB
  __shared__ __attribute__((aligned(16))) ExpandLds<I4> s;
  __shared__ __attribute__((aligned(16))) uint8_t extra[I4 ? kExpandWaves * kTile : 16];
  static_assert(I4 || sizeof(s.vals[0]) >= kTile, "the rows overwrite the values, read by then");
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
  const int r16 = lane & 15, q = lane >> 4;
  half8_t rows[4][2];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) rows[f][ks] = expand_row<I4>(s, lm, w, f, ks);
  if constexpr (I4) {
    const uint16_t* scales = (e ? a.scales[1] : a.scales[0]) + i * kGT + r16;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const float p = scale_power(static_cast<float>(__builtin_bit_cast(_Float16, scales[16 * f])));
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) rows[f][ks] *= static_cast<_Float16>(p);   // exact
    }
  }
  wave_sync();
  uint8_t* tile = I4 ? extra + w * kTile : s.vals[w];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      *reinterpret_cast<half8_t*>(tile + 2 * ((16 * f + r16) * kPrepLd + 32 * ks + 8 * q)) = rows[f][ks];
  wave_sync();
  u32x4_t* out = a.dense + ((c * a.blocks + e) * a.Gr + i) * 512 + lane;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      half8_t v;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = *reinterpret_cast<const _Float16*>(tile + 2 * ((32 * ks + 8 * q + j) * kPrepLd + 16 * f + r16));
      out[64 * (4 * ks + f)] = __builtin_bit_cast(u32x4_t, v);
    }
}

// ---------------------------------------------------------------------------
// The values' gradient
// ---------------------------------------------------------------------------

struct SampleArgs : WideArgs {
  ValueWeights v;
};

// A tile covers whole GroupTiles, outputs the weights' columns, rows their rows,
// and a wave's fragments whole runs, so the waves finish independently.
struct SampleFinish {
  using Args = SampleArgs;

  template <class C, typename T>
  __device__ static __forceinline__ void emit(uint8_t* smem, f32x4_t (&acc)[C::MF][C::NF], const WideTile& t, int wm,
                                              int wn, int me) {
    constexpr int MF = C::MF, NF = C::NF, kCols = MF < 4 ? MF : 4, kBytes = kKeptBytes<T, kCols>;
    static_assert(C::W * kBytes <= C::kRing * C::kPlace, "the waves' buffers fit the ring");
    const auto z = args_again<SampleArgs>();
    const int lane = me & 63, w = __builtin_amdgcn_readfirstlane(me >> 6);
    const int strips = z->v.strips, cols = z->v.cols;
    uint8_t* lds = smem + w * kBytes;
    kept_selectors(lds, lane);
    // The wave's GroupTile row; second: of the second weight.
    const int vs = t.row0 / kGT + NF * wn / 4;
    const int second = vs >= strips ? 1 : 0, r = vs - second * strips;
    T* dv = static_cast<T*>(second ? z->v.dv[1] : z->v.dv[0]);
    const bool mine = vs * kGT < z->S && dv != nullptr;
#pragma unroll
    for (int f0 = 0; f0 < MF; f0 += kCols) {
      const int c = t.strip0 + (MF * wm + f0) / 4;
      if (!mine || c >= cols) continue;
      const int64_t gt = static_cast<int64_t>(r) * cols + c;
      const u32x2_t bm = reinterpret_cast<const u32x2_t*>((second ? z->v.bitmaps[1] : z->v.bitmaps[0]) + gt * kBtPerGt)[lane];
      const Kept<T> k = kept_of<T>(bm, (second ? z->v.offsets[1] : z->v.offsets[0])[gt],
                                   second ? z->v.nnz[1] : z->v.nnz[0], dv, lds, lane);
#pragma unroll
      for (int nb = 0; nb < NF; ++nb) {
        f32x4_t sums[kCols];
#pragma unroll
        for (int n = 0; n < kCols; ++n) sums[n] = acc[f0 + n][nb];
        store_kept<T, kCols>(k, sums, (NF * wn + nb) & 3, (MF * wm) & 3, lds, lane);
      }
    }
    __syncthreads();
  }

  template <class C>
  __device__ static __forceinline__ void finish(uint8_t* smem, f32x4_t (&acc)[C::MF][C::NF], const WideTile& t, int wm,
                                                int wn, int me) {
    if (args_again<SampleArgs>()->e.f16out) emit<C, _Float16>(smem, acc, t, wm, wn, me);
    else emit<C, float>(smem, acc, t, wm, wn, me);
  }
};

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

struct Back {
  int nw;                  // weights: 1, or 2 of a gated block
  const usw_fmt* f[2];
  const uint16_t *X, *dY, *g, *u;
  void* dX;
  void* dV[2];
  float* db[2];
  int32_t N, act, out_type;
  bool i4, want_x, want_v, want_b;
};

struct BackPlan {
  int blocks;              // blocks of M columns of the reduction, each with its weight
  int64_t ldD;             // row length of D
  bool lo;                 // D's remainders follow its blocks
  int chunks;              // 64-token chunks
  bool prep;
  bool few, few_v;         // few rows: dx straight from the encodings, dV straight from d and x
  bool own_d;              // d is made, in rows, else dY is d
  int frag;                // > 0: it is made for few rows' dx, as fragments of as many 16-token blocks
  usw::FewPlan fx;
  usw::Geometry gx, gv;
  usw::WidePlan px, pv;
  size_t cb, D, F, dense, T, xt, sums, need;   // offsets in the workspace
};

usw::Geometry product(int64_t M, int64_t K) {
  usw::Geometry g{};
  g.M = M;
  g.K = K;
  g.Gr = M / kGT;
  g.Gc = K / kGT;
  g.ngt = g.Gr * g.Gc;
  return g;
}

usw::FewCall few_call(const Back& b, const BackPlan& p, const usw::Geometry& g) {
  usw::FewCall c{};
  c.f[0] = b.f[0];
  c.f[1] = b.f[b.nw - 1];
  c.weights = b.nw;
  c.blocks = p.blocks;
  c.ldD = p.own_d || p.frag ? p.ldD : g.M;
  c.lo = p.lo ? b.nw * g.M : 0;
  c.frag = p.frag > 0;
  c.X = b.X;
  c.dX = p.few ? b.dX : nullptr;
  for (int h = 0; h < b.nw; ++h) c.dV[h] = p.few_v ? b.dV[h] : nullptr;
  c.want_x = p.few;
  c.want_v = p.few_v;
  c.N = b.N;
  c.out_type = b.out_type;
  return c;
}

BackPlan plan_back(const Back& b, const usw::Geometry& g) {
  BackPlan p{};
  const bool own_x = b.want_x && (b.nw == 2 || b.i4);
  p.lo = (own_x || (b.nw == 2 && b.want_v)) && b.N <= usw::kLoRows;
  p.blocks = b.nw == 1 && b.i4 && b.out_type == USW_OUT_F32 && !p.lo ? 2 : b.nw;
  p.ldD = (p.lo ? 2 : 1) * p.blocks * g.M;
  p.chunks = (b.N + kGT - 1) / kGT;
  p.gx = product(g.K, p.blocks * g.M);
  p.gv = product(g.K, static_cast<int64_t>(p.chunks) * kGT);
  size_t base = 0;
  p.few = b.want_x && b.N <= usw::kFewGradRows;
  p.few_v = b.want_v && b.N <= usw::kFewValueRows;
  // Few rows' dx reads a d that is made as fragments, dV in rows.  Both are worth
  // their writes from 33 rows: pairs of 11008x4096 N = 60 84.5 us from rows, 79.6
  // from both; N = 8 64.2 and 65.2, of 20480x5120 N = 20 151 and 153.
  p.frag = own_x && p.few && !(p.few_v && b.N <= usw::kLoRows) ? usw::few_row_blocks(b.N) : 0;
  p.own_d = (own_x && !p.frag) || (b.nw == 2 && p.few_v);
  if (p.few) {
    p.fx = usw::few_plan(g, few_call(b, p, g));
    p.cb = p.fx.cb;
    p.px.slots_at = p.fx.cb;
    p.px.dense_at = std::max(p.fx.cb, p.fx.need);
  } else if (b.want_x) {
    p.px = usw::wide_plan(p.gx, 1, b.N, true);
    p.cb = p.px.cb;
  }
  if (b.want_v && !p.few_v) {
    p.pv = usw::wide_plan(p.gv, 1, static_cast<int32_t>(b.nw * g.M), true);
    p.cb = std::max(p.cb, p.pv.cb);
  }
  // One zone of counters and one of partial sums for both products.
  const size_t slots_at = std::max({p.px.slots_at, p.pv.slots_at, usw::counter_zone(0)});
  base = slots_at + std::max(p.px.dense_at - p.px.slots_at, p.pv.dense_at - p.pv.slots_at);
  p.px.slots_at = p.pv.slots_at = p.fx.cb = slots_at;
  auto take = [&](bool wanted, size_t bytes) {
    const size_t at = base = (base + 255) & ~size_t(255);
    if (wanted) base += bytes;
    return at;
  };
  const bool tall_v = b.want_v && !p.few_v;
  p.prep = p.own_d || p.frag || tall_v || b.want_b;
  p.D = take(p.own_d, static_cast<size_t>(b.N) * p.ldD * 2);
  p.F = take(p.frag > 0, static_cast<size_t>(16) * p.frag * p.ldD * 2);
  p.dense = take(b.want_x && !p.few, static_cast<size_t>(g.K) * p.blocks * g.M * 2);
  p.T = take(tall_v, static_cast<size_t>(b.nw) * g.M * p.chunks * kGT * 2);
  p.xt = take(tall_v, static_cast<size_t>(g.K) * p.chunks * kGT * 2);
  p.sums = take(b.want_b && p.chunks > 1, static_cast<size_t>(p.chunks) * b.nw * g.M * 4);
  p.need = base;
  return p;
}

template <bool GATED>
void launch_prep(const PrepArgs& a, int act, dim3 grid, hipStream_t s) {
  if constexpr (!GATED) {
    prep_kernel<false, USW_ACT_NONE><<<grid, 256, 0, s>>>(a);
  } else {
    switch (act) {
      case USW_ACT_RELU: prep_kernel<true, USW_ACT_RELU><<<grid, 256, 0, s>>>(a); break;
      case USW_ACT_GELU: prep_kernel<true, USW_ACT_GELU><<<grid, 256, 0, s>>>(a); break;
      case USW_ACT_GELU_TANH: prep_kernel<true, USW_ACT_GELU_TANH><<<grid, 256, 0, s>>>(a); break;
      case USW_ACT_SILU: prep_kernel<true, USW_ACT_SILU><<<grid, 256, 0, s>>>(a); break;
      default: prep_kernel<true, USW_ACT_NONE><<<grid, 256, 0, s>>>(a);
    }
  }
}

usw_status check_back(const Back& b, usw::Geometry* g) {
  for (int h = 0; h < b.nw; ++h) {
    usw_status st = check_common(b.f[h], b.out_type, b.N, g);
    if (st) return st;
  }
  if (b.nw == 2 && (b.f[1]->M != b.f[0]->M || b.f[1]->K != b.f[0]->K)) return USW_ERR_BAD_SHAPE;
  if (b.nw == 2 && b.f[1]->val_type != b.f[0]->val_type) return USW_ERR_BAD_DTYPE;
  if (g->M > kMaxLd || g->K > kMaxLd || g->M * g->K > kMaxElements) return USW_ERR_UNSUPPORTED;
  // The codes of INT4 values have no gradient.
  if (b.i4 && b.want_v) return USW_ERR_UNSUPPORTED;
  // dg and du are rounded to fp16 for the products, so their fp32 results would not be.
  if (b.nw == 2 && b.out_type != USW_OUT_F16) return USW_ERR_UNSUPPORTED;
  // 64-token chunks are the second dimension of d's pass, which takes 256 threads
  // to one by 64 outputs and, where x's transpose is asked for, by 64 columns.
  const int64_t chunks = (static_cast<int64_t>(b.N) + kGT - 1) / kGT;
  if (chunks > 65535 || static_cast<int64_t>(b.N) * std::max(g->M, g->K) > kMaxD ||
      chunks * (g->Gr + (b.want_v ? g->Gc : 0)) >= int64_t(1) << 24)
    return USW_ERR_UNSUPPORTED;
  return USW_OK;
}

bool products_launchable(const Back& b, const BackPlan& p) {
  return (!b.want_x || p.few || usw::wide_launchable(p.px)) && (!b.want_v || p.few_v || usw::wide_launchable(p.pv));
}

// Whether an output lies on another one or on something that the call reads.
bool outputs_overlap(const Back& b, const usw::Geometry& g, const void* ws, size_t ws_bytes) {
  struct Span {
    uintptr_t at;
    size_t bytes;
  };
  Span out[5], in[13];
  int no = 0, ni = 0;
  const auto span = [](const void* p, size_t bytes) { return Span{reinterpret_cast<uintptr_t>(p), p ? bytes : 0}; };
  const size_t size = b.out_type == USW_OUT_F16 ? 2 : 4, rows = static_cast<size_t>(b.N);
  out[no++] = span(b.dX, rows * g.K * size);
  in[ni++] = span(b.want_v ? b.X : nullptr, rows * g.K * 2);
  in[ni++] = span(b.dY, rows * g.M * 2);
  in[ni++] = span(b.g, rows * g.M * 2);
  in[ni++] = span(b.u, rows * g.M * 2);
  in[ni++] = span(ws, ws_bytes);
  for (int h = 0; h < b.nw; ++h) {
    const usw_fmt* f = b.f[h];
    out[no++] = span(b.dV[h], static_cast<size_t>(f->nnz) * size);
    out[no++] = span(b.db[h], static_cast<size_t>(g.M) * 4);
    in[ni++] = span(f->bitmaps, static_cast<size_t>(g.M) * g.K / 8);
    in[ni++] = span(f->offsets, static_cast<size_t>(g.ngt + 1) * 4);
    in[ni++] = span(f->values, usw::values_alloc_bytes(f->val_type, f->nnz));
    in[ni++] = span(b.i4 ? f->scales : nullptr, static_cast<size_t>(g.M) * 2);
  }
  const auto meet = [](const Span& a, const Span& c) {
    return a.bytes > 0 && c.bytes > 0 && a.at < c.at + c.bytes && c.at < a.at + a.bytes;
  };
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (meet(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
  }
  return false;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

usw_status back_impl(const Back& b, void* ws, size_t ws_bytes, void* stream) {
  usw::Geometry g;
  usw_status st = check_back(b, &g);
  if (st) return st;
  if (!b.dY || (b.want_v && !b.X) || (b.nw == 2 && (!b.g || !b.u))) return USW_ERR_NULL_ARG;
  if (!aligned16(b.X) || !aligned16(b.dY) || !aligned16(b.g) || !aligned16(b.u) || !aligned16(b.dX))
    return USW_ERR_MISALIGNED;
  for (int h = 0; h < b.nw; ++h) {
    const usw_fmt* f = b.f[h];
    if (!f->bitmaps || !f->offsets || !f->values || (b.i4 && !f->scales)) return USW_ERR_NULL_ARG;
    if (!aligned16(f->bitmaps) || !aligned16(f->values) || !aligned4(f->offsets) || (b.i4 && !aligned16(f->scales)) ||
        !aligned4(b.dV[h]) || !aligned4(b.db[h]))
      return USW_ERR_MISALIGNED;
  }
  const BackPlan p = plan_back(b, g);
  if (!products_launchable(b, p)) return USW_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < p.need) return USW_ERR_WORKSPACE;
  if (!aligned16(ws)) return USW_ERR_MISALIGNED;
  if (outputs_overlap(b, g, ws, p.need)) return USW_ERR_UNSUPPORTED;
  uint8_t* at = static_cast<uint8_t*>(ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool tall_v = b.want_v && !p.few_v;
  const uint16_t* d = p.own_d ? reinterpret_cast<const uint16_t*>(at + p.D) : b.dY;
  if (p.prep) {
    PrepArgs a{};
    a.dY = b.dY;
    a.g = b.g;
    a.u = b.u;
    for (int h = 0; h < b.nw; ++h) a.scales[h] = b.i4 ? b.f[h]->scales : nullptr;
    if (p.own_d) a.D = reinterpret_cast<uint16_t*>(at + p.D);
    if (tall_v) a.T = reinterpret_cast<uint16_t*>(at + p.T);
    a.sums = reinterpret_cast<float*>(at + p.sums);
    for (int h = 0; h < b.nw; ++h) a.db[h] = b.db[h];
    a.X = b.X;
    a.xt = reinterpret_cast<u32x4_t*>(at + p.xt);
    a.N = b.N;
    if (p.frag) a.F = reinterpret_cast<uint16_t*>(at + p.F);
    a.ldD = p.ldD;
    a.frag = p.frag;
    a.M = static_cast<int>(g.M);
    a.K = static_cast<int>(g.K);
    a.Gr = static_cast<int>(g.Gr);
    a.chunks = p.chunks;
    a.lo = p.ldD > b.nw * g.M ? static_cast<int>(b.nw * g.M) : 0;
    const dim3 grid(static_cast<unsigned>(g.Gr + (tall_v ? g.Gc : 0)), static_cast<unsigned>(p.chunks));
    if (b.nw == 2) launch_prep<true>(a, b.act, grid, s);
    else launch_prep<false>(a, b.act, grid, s);
    if (b.want_b && p.chunks > 1)
      bias_kernel<<<static_cast<unsigned>((b.nw * g.M + 255) / 256), 256, 0, s>>>(a.sums, b.db[0], b.db[1], a.M, b.nw,
                                                                                  p.chunks);
  }
  if (p.few || p.few_v) {
    usw::FewCall c = few_call(b, p, g);
    c.D = d;
    c.F = p.frag ? reinterpret_cast<const uint16_t*>(at + p.F) : nullptr;
    st = usw::few_launch(g, c, p.fx, ws, stream);
    if (st) return st;
  }
  if (b.want_x && !p.few) {
    ExpandTArgs x{};
    for (int h = 0; h < p.blocks; ++h) {
      const usw_fmt* f = b.f[h < b.nw ? h : 0];
      x.bitmaps[h] = f->bitmaps;
      x.offsets[h] = f->offsets;
      x.values[h] = static_cast<const uint8_t*>(f->values);
      x.scales[h] = f->scales;
      x.alloc[h] = usw::values_alloc_bytes(f->val_type, f->nnz);
    }
    x.dense = reinterpret_cast<u32x4_t*>(at + p.dense);
    x.ngt = g.ngt;
    x.Gr = static_cast<int>(g.Gr);
    x.Gc = static_cast<int>(g.Gc);
    x.blocks = p.blocks;
    const dim3 grid(static_cast<unsigned>((g.ngt + kExpandWaves - 1) / kExpandWaves), static_cast<unsigned>(p.blocks));
    if (b.i4) expand_t_kernel<true><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    else expand_t_kernel<false><<<grid, 64 * kExpandWaves, 0, s>>>(x);
    const Epilogue e{nullptr, nullptr, nullptr, g.K, g.K, USW_ACT_NONE, b.out_type == USW_OUT_F16 ? 1 : 0};
    st = usw::wide_multiply(p.gx, p.px, b.N, d, b.dX, e, x.dense, ws, stream);
    if (st) return st;
  }
  if (tall_v) {
    SampleArgs a{};
    fill_wide(a, p.pv, p.gv, static_cast<int>(b.nw * g.M), at + p.xt, ws);
    a.X = reinterpret_cast<const uint16_t*>(at + p.T);
    a.e.f16out = b.out_type == USW_OUT_F16 ? 1 : 0;
    a.v = value_weights(b.f, b.dV, b.nw, g);
    launch_wide<SampleFinish>(p.pv, a, s);
  }
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

Back single(const usw_fmt* f, int32_t N, int32_t out_type) {
  Back b{};
  b.nw = 1;
  b.f[0] = f;
  b.N = N;
  b.act = USW_ACT_NONE;
  b.out_type = out_type;
  b.i4 = f->val_type == USW_VAL_I4;
  return b;
}

Back pair(const usw_fmt* gate, const usw_fmt* up, int32_t N) {
  Back b{};
  b.nw = 2;
  b.f[0] = gate;
  b.f[1] = up;
  b.N = N;
  b.out_type = USW_OUT_F16;
  b.i4 = gate->val_type == USW_VAL_I4;
  return b;
}

usw_status workspace_of(Back b, int32_t grads, size_t* bytes, size_t* counter_bytes) {
  if (!bytes || !counter_bytes) return USW_ERR_NULL_ARG;
  if (grads & ~(USW_GRAD_X | USW_GRAD_VALUES | USW_GRAD_BIAS)) return USW_ERR_BAD_DTYPE;
  b.want_x = grads & USW_GRAD_X;
  b.want_v = grads & USW_GRAD_VALUES;
  b.want_b = grads & USW_GRAD_BIAS;
  usw::Geometry g;
  usw_status st = check_back(b, &g);
  if (st) return st;
  const BackPlan p = plan_back(b, g);
  if (!products_launchable(b, p)) return USW_ERR_UNSUPPORTED;
  *bytes = p.need;
  *counter_bytes = p.cb;
  return USW_OK;
}

}  // namespace

extern "C" {

usw_status usw_spmm_backward_workspace(const usw_fmt* f, int32_t N, int32_t out_type, int32_t grads, size_t* bytes,
                                       size_t* counter_bytes) {
  if (!f) return USW_ERR_NULL_ARG;
  return workspace_of(single(f, N, out_type), grads, bytes, counter_bytes);
}

usw_status usw_spmm_backward(const usw_fmt* f, const uint16_t* X, const uint16_t* dY, int32_t N, void* dX, void* dvalues,
                             float* dbias, int32_t out_type, void* ws, size_t ws_bytes, void* stream) {
  if (!f) return USW_ERR_NULL_ARG;
  Back b = single(f, N, out_type);
  b.X = X;
  b.dY = dY;
  b.dX = dX;
  b.dV[0] = dvalues;
  b.db[0] = dbias;
  b.want_x = dX != nullptr;
  b.want_v = dvalues != nullptr;
  b.want_b = dbias != nullptr;
  return back_impl(b, ws, ws_bytes, stream);
}

usw_status usw_spmm_gated_backward_workspace(const usw_fmt* gate, const usw_fmt* up, int32_t N, int32_t grads,
                                             size_t* bytes, size_t* counter_bytes) {
  if (!gate || !up) return USW_ERR_NULL_ARG;
  return workspace_of(pair(gate, up, N), grads, bytes, counter_bytes);
}

usw_status usw_spmm_gated_backward(const usw_fmt* gate, const usw_fmt* up, const uint16_t* X, int32_t N,
                                   const usw_gated_grad* d, void* ws, size_t ws_bytes, void* stream) {
  if (!gate || !up || !d) return USW_ERR_NULL_ARG;
  if (d->act < USW_ACT_NONE || d->act > USW_ACT_SILU) return USW_ERR_BAD_DTYPE;
  if (d->reserved != 0) return USW_ERR_BAD_SHAPE;
  Back b = pair(gate, up, N);
  b.X = X;
  b.dY = d->dY;
  b.g = d->pre_gate;
  b.u = d->pre_up;
  b.act = d->act;
  b.dX = d->dX;
  b.dV[0] = d->dgate_values;
  b.dV[1] = d->dup_values;
  b.db[0] = d->dgate_bias;
  b.db[1] = d->dup_bias;
  b.want_x = b.dX != nullptr;
  b.want_v = b.dV[0] || b.dV[1];
  b.want_b = b.db[0] || b.db[1];
  return back_impl(b, ws, ws_bytes, stream);
}

}  // extern "C"
