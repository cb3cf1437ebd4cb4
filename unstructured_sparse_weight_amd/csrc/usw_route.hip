// The router of the expert products (usw_expert_route) and the sum that joins
// their rows again (usw_expert_combine).
//
// Routing.  Of token t's E logits the k largest are chosen (equal logits: the
// lower expert first; -inf and NaN are never chosen), and their weights are
// exp(l - l_max) over the sum of the same over the chosen, or over all,
// experts.  The chosen (token, expert) pairs, the slots, are then sorted by
// (expert, token): a token chooses an expert at most once, so a slot's place
// is the first slot of its expert plus the number of earlier tokens that
// chose it.  A block of tokens keeps one bit per token for each expert, so
// that number is a masked popcount inside the block plus the counts of the
// blocks before; no atomics decide an order, and equal inputs give equal
// plans.
//
// Up to 256 tokens one workgroup does all of it in one launch, since there
// the launches are the time.  Above, blocks of 64 tokens (one bitmap word
// per expert) choose and count, a scan adds the counts down the blocks, and
// the blocks place their slots.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "usw.h"
#include "usw_device.h"
#include "usw_internal.h"

namespace {

using namespace usw_dev;

constexpr int kMaxRouteExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kOneTokens = 256;    // tokens the one-workgroup kernel takes
constexpr int kBlockTokens = 64;   // tokens per workgroup above that

struct RouteArgs {
  const void* __restrict__ logits;
  int64_t ld;
  int32_t* __restrict__ ids;       // [T][k]
  float* __restrict__ weights;     // [T][k]
  int32_t* __restrict__ slots;     // [E+1]
  int32_t* __restrict__ rows;      // [T k]
  int32_t* __restrict__ pos;       // [T][k]
  int32_t* __restrict__ counts;    // [blocks][E], then [E] totals
  int T, E, k, blocks, f16, renormalize;
};

// A float as an unsigned integer in the same order; NaN and -inf become 0,
// which is below every value that can be chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);   // -0 becomes +0
  const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return v > -__builtin_inff() ? key : 0u;
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __builtin_bit_cast(float, (key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// exp(v - top) for a top that is the maximum: equal infinities count 1.
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.0f : expf(v - top); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The choice of one token by one wave; PER = experts per lane.  Lane j < k
// ends with the j-th chosen expert in *id (-1: none left) and its weight.
template <int PER>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int lane, int* id, float* weight) {
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    key[i] = 0;
    if (e < a.E) {
      const int64_t at = t * a.ld + e;
      key[i] = order_key(a.f16 ? static_cast<float>(static_cast<const _Float16*>(a.logits)[at])
                               : static_cast<const float*>(a.logits)[at]);
    }
  }
  float top = 0.0f, total = 0.0f, mine = 0.0f;
  int chosen = -1;
  for (int j = 0; j < a.k; ++j) {
    // The largest key, the lowest expert among equals: the maximum of
    // (key, ~expert) over the lanes.
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t c = (static_cast<uint64_t>(key[i]) << 32) | ~static_cast<uint32_t>(lane + 64 * i);
      best = c > best ? c : best;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const uint64_t o = __shfl_xor(best, d);
      best = o > best ? o : best;
    }
    const uint32_t bkey = static_cast<uint32_t>(best >> 32);
    if (bkey == 0) break;
    const int e = static_cast<int>(~static_cast<uint32_t>(best));
    const float v = key_value(bkey);
    if (j == 0) {
      top = v;
      if (!a.renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (key[i]) total += exp_below(key_value(key[i]), top);
        total = wave_sum(total);
      }
    }
    const float p = exp_below(v, top);
    if (a.renormalize) total += p;
    if (lane == j) {
      chosen = e;
      mine = p;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i == e) key[i] = 0;
  }
  *id = chosen;
  *weight = chosen >= 0 ? mine / total : 0.0f;
}

__device__ __forceinline__ void choose_any(const RouteArgs& a, int t, int lane, int* id, float* weight) {
  if (a.E <= 64) choose<1>(a, t, lane, id, weight);
  else if (a.E <= 128) choose<2>(a, t, lane, id, weight);
  else if (a.E <= 256) choose<4>(a, t, lane, id, weight);
  else choose<16>(a, t, lane, id, weight);
}

// Chooses for the block's tokens [t0, t0 + n), n <= 64 WORDS, and leaves each
// expert's bitmap of the tokens that chose it in bits[WORDS][E].
template <int WAVES, int WORDS>
__device__ __forceinline__ void choose_block(const RouteArgs& a, int t0, int n, uint32_t* bits) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int i = tid; i < 2 * WORDS * a.E; i += 64 * WAVES) bits[i] = 0u;
  __syncthreads();
  for (int i = w; i < n; i += WAVES) {
    int id;
    float weight;
    choose_any(a, t0 + i, lane, &id, &weight);
    if (lane < a.k) {
      const int64_t at = static_cast<int64_t>(t0 + i) * a.k + lane;
      a.ids[at] = id;
      a.weights[at] = weight;
      if (id >= 0) atomicOr(&bits[(i >> 5) * a.E + id], 1u << (i & 31));
    }
  }
  __syncthreads();
}

// Tokens of the block before token i that chose expert e.
__device__ __forceinline__ int rank_in(const uint32_t* bits, int E, int e, int i) {
  int r = __builtin_popcount(bits[(i >> 5) * E + e] & ((1u << (i & 31)) - 1u));
  for (int q = 0; q < (i >> 5); ++q) r += __builtin_popcount(bits[q * E + e]);
  return r;
}

// Exclusive prefix of v[0 .. E) in place by the first wave, v[E] = the total.
__device__ __forceinline__ void scan_experts(int32_t* v, int E) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    uint32_t before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const uint32_t c = e0 + lane < E ? static_cast<uint32_t>(v[e0 + lane]) : 0u;
      const uint32_t incl = wave_inclusive_scan(c);
      if (e0 + lane < E) v[e0 + lane] = static_cast<int32_t>(before + incl - c);
      before += __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) v[E] = static_cast<int32_t>(before);
  }
  __syncthreads();
}

__global__ __launch_bounds__(1024) void route_one_kernel(RouteArgs a) {
  extern __shared__ uint32_t lds[];   // bits [8][E], first slots [E + 1]
  uint32_t* bits = lds;
  int32_t* first = reinterpret_cast<int32_t*>(lds + 8 * a.E);
  const int tid = threadIdx.x;
  choose_block<16, 4>(a, 0, a.T, bits);
  for (int e = tid; e < a.E; e += 1024) {
    int c = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) c += __builtin_popcount(bits[q * a.E + e]);
    first[e] = c;
  }
  __syncthreads();
  scan_experts(first, a.E);
  for (int e = tid; e <= a.E; e += 1024) a.slots[e] = first[e];
  const int n = a.T * a.k, live = first[a.E];
  for (int i = tid; i < n; i += 1024) {
    // The ids this workgroup stored: written before the barrier, read back
    // from the same compute unit.
    const int id = a.ids[i], t = i / a.k;
    int p = -1;
    if (id >= 0) {
      p = first[id] + rank_in(bits, a.E, id, t);
      a.rows[p] = t;
    }
    a.pos[i] = p;
    if (i >= live) a.rows[i] = -1;
  }
}

// Blocks of 64 tokens: choose, count, and leave each slot's rank inside the
// block in pos.
__global__ __launch_bounds__(1024) void route_choose_kernel(RouteArgs a) {
  extern __shared__ uint32_t lds[];   // bits [2][E]
  const int t0 = static_cast<int>(blockIdx.x) * kBlockTokens;
  const int n = min(kBlockTokens, a.T - t0);
  choose_block<16, 1>(a, t0, n, lds);
  const int tid = threadIdx.x;
  for (int e = tid; e < a.E; e += 1024)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = __builtin_popcount(lds[e]) + __builtin_popcount(lds[a.E + e]);
  for (int i = tid; i < n * a.k; i += 1024) {
    const int64_t at = static_cast<int64_t>(t0) * a.k + i;
    const int id = a.ids[at];
    a.pos[at] = id >= 0 ? rank_in(lds, a.E, id, i / a.k) : -1;
  }
}

// One wave per expert: its counts down the blocks become exclusive prefixes,
// and its total goes behind them.
__global__ __launch_bounds__(64) void route_scan_kernel(RouteArgs a) {
  const int e = static_cast<int>(blockIdx.x), lane = threadIdx.x;
  uint32_t before = 0;
  for (int b0 = 0; b0 < a.blocks; b0 += 64) {
    const int b = b0 + lane;
    int32_t* at = a.counts + static_cast<int64_t>(b) * a.E + e;
    const uint32_t c = b < a.blocks ? static_cast<uint32_t>(*at) : 0u;
    const uint32_t incl = wave_inclusive_scan(c);
    if (b < a.blocks) *at = static_cast<int32_t>(before + incl - c);
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  if (lane == 0) a.counts[static_cast<int64_t>(a.blocks) * a.E + e] = static_cast<int32_t>(before);
}

__global__ __launch_bounds__(256) void route_place_kernel(RouteArgs a) {
  extern __shared__ uint32_t lds[];   // first slots [E + 1]
  int32_t* first = reinterpret_cast<int32_t*>(lds);
  const int tid = threadIdx.x;
  for (int e = tid; e < a.E; e += 256) first[e] = a.counts[static_cast<int64_t>(a.blocks) * a.E + e];
  __syncthreads();
  scan_experts(first, a.E);
  if (blockIdx.x == 0)
    for (int e = tid; e <= a.E; e += 256) a.slots[e] = first[e];
  const int t0 = static_cast<int>(blockIdx.x) * kBlockTokens;
  const int n = min(kBlockTokens, a.T - t0) * a.k, live = first[a.E];
  const int32_t* before = a.counts + static_cast<int64_t>(blockIdx.x) * a.E;
  for (int i = tid; i < n; i += 256) {
    const int64_t at = static_cast<int64_t>(t0) * a.k + i;
    const int id = a.ids[at];
    if (id >= 0) {
      const int p = first[id] + before[id] + a.pos[at];
      a.rows[p] = t0 + i / a.k;
      a.pos[at] = p;
    }
    if (at >= live) a.rows[at] = -1;
  }
}

// ---------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------
//
// out[t] = res[t] + sum over j = 0 .. k-1, in that order, of
// weights[t][j] * y[pos[t][j]].  Bound by the bytes of y: a thread owns eight
// columns of one token and has the loads of up to eight slots in flight.

struct CombineArgs {
  const void* __restrict__ y;
  const int32_t* __restrict__ pos;
  const float* __restrict__ weights;
  const uint16_t* res;
  void* out;
  int64_t ld_res;
  int64_t total;   // T * M / 8
  int S, M8, k;
};

struct Eight {
  f32x4_t lo, hi;
};

template <bool F16>
__device__ __forceinline__ Eight load8(const void* p, int64_t at) {
  Eight r;
  if constexpr (F16) {
    const half8_t h = *reinterpret_cast<const half8_t*>(static_cast<const _Float16*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.lo[i] = static_cast<float>(h[i]);
      r.hi[i] = static_cast<float>(h[4 + i]);
    }
  } else {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at);
    r.lo = q[0];
    r.hi = q[1];
  }
  return r;
}

template <bool Y16, bool OUT16>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.total) return;
  const int64_t t = a.total <= 0xFFFFFFFFll ? static_cast<uint32_t>(i) / static_cast<uint32_t>(a.M8) : i / a.M8;
  const int col = 8 * static_cast<int>(i - t * a.M8);
  const int64_t M = 8ll * a.M8;
  Eight sum = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    Eight v[8];
    float w[8];
    bool has[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = t * a.k + min(j0 + j, a.k - 1);
      const int p = a.pos[at];
      has[j] = j0 + j < a.k && static_cast<uint32_t>(p) < static_cast<uint32_t>(a.S);
      w[j] = a.weights[at];
      if (has[j]) v[j] = load8<Y16>(a.y, p * M + col);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (has[j]) {
        sum.lo += w[j] * v[j].lo;
        sum.hi += w[j] * v[j].hi;
      }
  }
  if (a.res) {
    const Eight r = load8<true>(a.res, t * a.ld_res + col);
    sum.lo += r.lo;
    sum.hi += r.hi;
  }
  const int64_t o = t * M + col;
  if constexpr (OUT16) {
    half8_t h;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      h[q] = static_cast<_Float16>(sum.lo[q]);
      h[4 + q] = static_cast<_Float16>(sum.hi[q]);
    }
    *reinterpret_cast<half8_t*>(static_cast<_Float16*>(a.out) + o) = h;
  } else {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + o);
    q[0] = sum.lo;
    q[1] = sum.hi;
  }
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

usw_status check_route(int32_t T, int32_t E, int32_t k) {
  if (T < 0) return USW_ERR_BAD_N;
  if (E < 1 || k < 1 || k > E) return USW_ERR_BAD_SHAPE;
  if (E > kMaxRouteExperts || k > kMaxTopK) return USW_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(T) * k >= (int64_t(1) << 31)) return USW_ERR_UNSUPPORTED;
  return USW_OK;
}

size_t route_bytes(int32_t T, int32_t E) {
  if (T <= kOneTokens) return 0;
  const int64_t blocks = (static_cast<int64_t>(T) + kBlockTokens - 1) / kBlockTokens;
  return static_cast<size_t>(4) * (blocks + 1) * E;
}

}  // namespace

extern "C" {

usw_status usw_expert_route_workspace(int32_t T, int32_t E, int32_t k, size_t* bytes) {
  if (!bytes) return USW_ERR_NULL_ARG;
  const usw_status st = check_route(T, E, k);
  if (st) return st;
  *bytes = route_bytes(T, E);
  return USW_OK;
}

usw_status usw_expert_route(const void* logits, int32_t l_type, int64_t ld, int32_t T, int32_t E, int32_t k,
                            int32_t renormalize, int32_t* ids, float* weights, int32_t* slots, int32_t* rows,
                            int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
  const usw_status st = check_route(T, E, k);
  if (st) return st;
  if (l_type != USW_OUT_F16 && l_type != USW_OUT_F32) return USW_ERR_BAD_DTYPE;
  if (ld == 0) ld = E;
  if (ld < E || ld > (int64_t(1) << 31)) return USW_ERR_BAD_SHAPE;
  if (!slots || (T > 0 && (!logits || !ids || !weights || !rows || !pos))) return USW_ERR_NULL_ARG;
  if (!aligned(logits, l_type == USW_OUT_F16 ? 2 : 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(slots, 4) || !aligned(rows, 4) || !aligned(pos, 4))
    return USW_ERR_MISALIGNED;
  const size_t need = route_bytes(T, E);
  if (need > 0) {
    if (!ws || ws_bytes < need) return USW_ERR_WORKSPACE;
    if (!aligned(ws, 4)) return USW_ERR_MISALIGNED;
  }
  RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.weights = weights;
  a.slots = slots;
  a.rows = rows;
  a.pos = pos;
  a.counts = static_cast<int32_t*>(ws);
  a.T = T;
  a.E = E;
  a.k = k;
  a.f16 = l_type == USW_OUT_F16;
  a.renormalize = renormalize != 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T <= kOneTokens) {
    route_one_kernel<<<1, 1024, (9 * E + 1) * sizeof(uint32_t), s>>>(a);
  } else {
    a.blocks = (T + kBlockTokens - 1) / kBlockTokens;
    route_choose_kernel<<<a.blocks, 1024, 2 * E * sizeof(uint32_t), s>>>(a);
    route_scan_kernel<<<E, 64, 0, s>>>(a);
    route_place_kernel<<<a.blocks, 256, (E + 1) * sizeof(uint32_t), s>>>(a);
  }
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

usw_status usw_expert_combine(const void* Y, int32_t y_type, int32_t S, int32_t M, const int32_t* pos,
                              const float* weights, int32_t T, int32_t k, const uint16_t* res, int64_t ld_res,
                              void* out, int32_t out_type, void* stream) {
  if (T < 0 || S < 0) return USW_ERR_BAD_N;
  if (M < 1 || M % 8 || k < 1) return USW_ERR_BAD_SHAPE;
  if ((y_type != USW_OUT_F16 && y_type != USW_OUT_F32) || (out_type != USW_OUT_F16 && out_type != USW_OUT_F32))
    return USW_ERR_BAD_DTYPE;
  if (ld_res == 0) ld_res = M;
  if (ld_res < M || ld_res > (int64_t(1) << 31)) return USW_ERR_BAD_SHAPE;
  if (T > 0 && (!pos || !weights || !out || (S > 0 && !Y))) return USW_ERR_NULL_ARG;
  if (!aligned(Y, 16) || !aligned(out, 16) || !aligned(res, 16) || (res && ld_res % 8) || !aligned(pos, 4) ||
      !aligned(weights, 4))
    return USW_ERR_MISALIGNED;
  if (T == 0) return USW_OK;
  CombineArgs a{};
  a.y = Y;
  a.pos = pos;
  a.weights = weights;
  a.res = res;
  a.out = out;
  a.ld_res = ld_res;
  a.S = S;
  a.M8 = M / 8;
  a.k = k;
  a.total = static_cast<int64_t>(T) * a.M8;
  const int64_t blocks = (a.total + 255) / 256;
  if (blocks >= (int64_t(1) << 31)) return USW_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool y16 = y_type == USW_OUT_F16, o16 = out_type == USW_OUT_F16;
  if (y16 && o16) combine_kernel<true, true><<<grid, 256, 0, s>>>(a);
  else if (y16) combine_kernel<true, false><<<grid, 256, 0, s>>>(a);
  else if (o16) combine_kernel<false, true><<<grid, 256, 0, s>>>(a);
  else combine_kernel<false, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

}  // extern "C"
