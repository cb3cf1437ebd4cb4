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
// Choosing is bound by the instructions it issues: k rounds of a maximum over
// the experts, the lowest expert that has it (fp16 logits: part of the
// maximum), and its removal.  Four tokens share a wave, 16 lanes (a DPP row)
// to a token, so that the moves across lanes serve four tokens each.
//
// Up to 64 tokens one workgroup does all of it in one launch, since there
// the launches are the time (64 experts, k 8, 64 tokens: 5.0 us, a second
// launch adds 2).  Above, blocks of tokens choose and count, and in a second
// launch each block adds the counts of the blocks before it and places its
// slots.  From 256 blocks on, where every block would read a long table, a
// launch between them turns the counts into prefixes.
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
constexpr int kOneTokens = 64;     // tokens the one-workgroup kernel takes
constexpr int kFineTokens = 4096;  // above that, blocks of 32 tokens up to here, then of 64
constexpr int kMaxRouteTokens = (1 << 28) - 64;   // their blocks of 64 make less than HIP's 2^32 threads
constexpr int kAddBlocks = 256;    // most blocks whose counts every block adds itself

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
  int per;                         // tokens to a block
  int lg_e;                        // log2 of E rounded up to a power of two
};

// Blocks of 32 tokens choose sooner (256 experts, k 8, 256 tokens: 9.5 us
// against 11.8), but leave twice the counts to add (512 experts, k 2, 4000
// tokens: 15.1 us against 14.6, and the table grows with the square of T).
constexpr int block_tokens(int32_t T) { return T <= kFineTokens ? 32 : 64; }

// A float as an unsigned integer in the same order; NaN and -inf become 0,
// which is below every value that can be chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);   // -0 becomes +0
  const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return v > -__builtin_inff() ? key : 0u;
}

// An fp16 logit's key ends in bits that are all alike, so its last ten hold
// the expert instead, the lower expert above: such keys are all different, and
// a maximum is the choice itself (64 tokens of 256 experts, k 8: 9.3 us, fp32
// logits 11.1).
constexpr uint32_t kExpertBits = 0x3FFu;
static_assert(kMaxRouteExperts <= kExpertBits + 1);

template <bool UNIQUE>
__device__ __forceinline__ float key_value(uint32_t key) {
  if constexpr (UNIQUE) key = (key & 0x80000000u) ? key & ~kExpertBits : key | kExpertBits;
  return __builtin_bit_cast(float, (key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// exp(v - top) for a top that is the maximum: equal infinities count 1.
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.0f : expf(v - top); }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}

__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t as_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

// Maximum and sum over the L lanes of a token, in each of them.  Over 16 lanes
// by rotations of a DPP row: every lane adds the same pairs, so all have the
// same sum.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 64) {
    return wave_max(v);
  } else {
    v = max(v, dpp<0x128, 0xf>(v));   // row_ror:8, 4, 2, 1
    v = max(v, dpp<0x124, 0xf>(v));
    v = max(v, dpp<0x122, 0xf>(v));
    return max(v, dpp<0x121, 0xf>(v));
  }
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L == 64) {
    v += as_float(dpp<0x111, 0xf>(as_bits(v)));   // row_shr:1, 2, 4, 8
    v += as_float(dpp<0x112, 0xf>(as_bits(v)));
    v += as_float(dpp<0x114, 0xf>(as_bits(v)));
    v += as_float(dpp<0x118, 0xf>(as_bits(v)));
    v += as_float(dpp<0x142, 0xa>(as_bits(v)));   // row_bcast:15, 31
    v += as_float(dpp<0x143, 0xc>(as_bits(v)));
    return as_float(__builtin_amdgcn_readlane(as_bits(v), 63));
  } else {
    v += as_float(dpp<0x128, 0xf>(as_bits(v)));
    v += as_float(dpp<0x124, 0xf>(as_bits(v)));
    v += as_float(dpp<0x122, 0xf>(as_bits(v)));
    return v + as_float(dpp<0x121, 0xf>(as_bits(v)));
  }
}

// Chooses for the block's tokens [t0, t0 + n), L lanes to a token and PER
// logits to a lane (expert c + L i), and sets their bits in bits.
template <bool F16, int WAVES, int L, int PER>
__device__ __forceinline__ void choose_tokens(const RouteArgs& a, int t0, int n, uint32_t* bits) {
  constexpr bool kUnique = F16 && PER < 32;   // keys that hold the expert (with 32 a register would spill)
  const int c = threadIdx.x & (L - 1);
  for (int i = threadIdx.x / L; i - static_cast<int>(threadIdx.x & 63) / L < n; i += 64 * WAVES / L) {
    const int64_t row = (t0 + min(i, n - 1)) * a.ld;
    uint32_t key[PER], top = 0, mine = 0;
    float all = 0.0f;
    int id = -1;
    float v[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int64_t at = row + min(c + L * q, a.E - 1);
      if constexpr (F16) v[q] = static_cast<float>(static_cast<const _Float16*>(a.logits)[at]);
      else v[q] = static_cast<const float*>(a.logits)[at];
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      key[q] = c + L * q < a.E ? order_key(v[q]) : 0u;
      if (kUnique && key[q]) key[q] = (key[q] | kExpertBits) - static_cast<uint32_t>(c + L * q);
    }
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int q = 1; q < PER; ++q) best = max(best, key[q]);
      best = lanes_max<L>(best);
      if (j == 0) {
        top = best;
        if (!a.renormalize) {
#pragma unroll
          for (int q = 0; q < PER; ++q)
            if (key[q]) all += exp_below(key_value<kUnique>(key[q]), key_value<kUnique>(top));
        }
      }
      if constexpr (kUnique) {
        mine = c == j ? best : mine;
#pragma unroll
        for (int q = 0; q < PER; ++q) key[q] = key[q] == best ? 0u : key[q];
      } else {
        // The lowest expert that has it, as the largest complement.
        uint32_t at = 0;
#pragma unroll
        for (int q = PER - 1; q >= 0; --q) at = key[q] == best ? ~static_cast<uint32_t>(L * q) - c : at;
        const int e = static_cast<int>(~lanes_max<L>(at));
        if (c == j && best != 0) {
          id = e;
          mine = best;
        }
#pragma unroll
        for (int q = 0; q < PER; ++q) key[q] = e - c == L * q ? 0u : key[q];
      }
    }
    if (kUnique && mine) id = static_cast<int>(kExpertBits - (mine & kExpertBits));
    const float p = mine ? exp_below(key_value<kUnique>(mine), key_value<kUnique>(top)) : 0.0f;
    const float total = lanes_sum<L>(a.renormalize ? p : all);
    if (i < n && c < a.k) {
      const int64_t at = static_cast<int64_t>(t0 + i) * a.k + c;
      a.ids[at] = id;
      a.weights[at] = mine ? p / total : 0.0f;
      if (id >= 0) atomicOr(&bits[(i >> 5) * a.E + id], 1u << (i & 31));
    }
  }
}

template <bool F16, int WAVES>
__device__ __forceinline__ void choose_in(const RouteArgs& a, int t0, int n, uint32_t* bits) {
  // 16 lanes to a token issue the fewest instructions (64 tokens, 256 experts,
  // k 8: 9.3 us against 13.4 with 64 lanes), 64 lanes have the shorter chain
  // where one token is all a wave has (1 token: 4.3 us against 5.9).  Above 512
  // experts the two are equal at 64 tokens, and 64 lanes keep fewer registers.
  if (a.E > 512) choose_tokens<F16, WAVES, 64, 16>(a, t0, n, bits);
  else if (n <= WAVES && a.E > 256) choose_tokens<F16, WAVES, 64, 8>(a, t0, n, bits);
  else if (n <= WAVES && a.E > 128) choose_tokens<F16, WAVES, 64, 4>(a, t0, n, bits);
  else if (n <= WAVES && a.E > 64) choose_tokens<F16, WAVES, 64, 2>(a, t0, n, bits);
  else if (a.E <= 16) choose_tokens<F16, WAVES, 16, 1>(a, t0, n, bits);
  else if (a.E <= 32) choose_tokens<F16, WAVES, 16, 2>(a, t0, n, bits);
  else if (a.E <= 64) choose_tokens<F16, WAVES, 16, 4>(a, t0, n, bits);
  else if (a.E <= 128) choose_tokens<F16, WAVES, 16, 8>(a, t0, n, bits);
  else if (a.E <= 256) choose_tokens<F16, WAVES, 16, 16>(a, t0, n, bits);
  else choose_tokens<F16, WAVES, 16, 32>(a, t0, n, bits);
}

// Chooses for the block's tokens [t0, t0 + n), n <= 4 WAVES, and leaves each
// expert's bitmap of the tokens that chose it in bits[WAVES / 8][E].
template <int WAVES>
__device__ __forceinline__ void choose_block(const RouteArgs& a, int t0, int n, uint32_t* bits) {
  for (int i = threadIdx.x; i < WAVES / 8 * a.E; i += 64 * WAVES) bits[i] = 0u;
  __syncthreads();
  if (a.f16) choose_in<true, WAVES>(a, t0, n, bits);
  else choose_in<false, WAVES>(a, t0, n, bits);
  __syncthreads();
}

// Tokens of the block before token i that chose expert e.
__device__ __forceinline__ int rank_in(const uint32_t* bits, int E, int e, int i) {
  const int r = __builtin_popcount(bits[(i >> 5) * E + e] & ((1u << (i & 31)) - 1u));
  return i >> 5 ? r + __builtin_popcount(bits[e]) : r;
}

// Tokens of the block that chose expert e.
template <int WORDS>
__device__ __forceinline__ int chose(const uint32_t* bits, int E, int e) {
  int c = __builtin_popcount(bits[e]);
  if constexpr (WORDS == 2) c += __builtin_popcount(bits[E + e]);
  return c;
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
  extern __shared__ uint32_t lds[];   // bits [2][E], first slots [E + 1]
  uint32_t* bits = lds;
  int32_t* first = reinterpret_cast<int32_t*>(lds + 2 * a.E);
  const int tid = threadIdx.x;
  choose_block<16>(a, 0, a.T, bits);
  for (int e = tid; e < a.E; e += 1024) {
    first[e] = chose<2>(bits, a.E, e);
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

// Blocks of 4 WAVES tokens: choose, count, and leave each slot's rank inside
// the block in pos.
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void route_choose_kernel(RouteArgs a) {
  extern __shared__ uint32_t lds[];   // bits [WAVES / 8][E]
  const int t0 = static_cast<int>(blockIdx.x) * 4 * WAVES;
  const int n = min(4 * WAVES, a.T - t0);
  choose_block<WAVES>(a, t0, n, lds);
  const int tid = threadIdx.x;
  for (int e = tid; e < a.E; e += 64 * WAVES)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = chose<WAVES / 8>(lds, a.E, e);
  for (int i = tid; i < n * a.k; i += 64 * WAVES) {
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

// PREFIXED: the scan has run.  Otherwise the block adds the counts of all
// blocks, and of those before it, itself: its threads in groups of E rounded
// up to a power of two, each group every n-th block.
template <bool PREFIXED>
__global__ __launch_bounds__(1024) void route_place_kernel(RouteArgs a) {
  extern __shared__ uint32_t lds[];   // first slots [E + 1], then [E] slots before this block
  int32_t* first = reinterpret_cast<int32_t*>(lds);
  int32_t* before = first + a.E + 1;
  const int tid = threadIdx.x, blk = static_cast<int>(blockIdx.x);
  if constexpr (PREFIXED) {
    for (int e = tid; e < a.E; e += 1024) {
      first[e] = a.counts[static_cast<int64_t>(a.blocks) * a.E + e];
      before[e] = a.counts[static_cast<int64_t>(blk) * a.E + e];
    }
  } else {
    for (int e = tid; e < a.E; e += 1024) first[e] = before[e] = 0;
    __syncthreads();
    const int groups = 1024 >> a.lg_e, e = tid & ((1 << a.lg_e) - 1);
    if (e < a.E) {
      int all = 0, mine = 0;
#pragma unroll 8
      for (int b = tid >> a.lg_e; b < a.blocks; b += groups) {
        const int c = a.counts[static_cast<int64_t>(b) * a.E + e];
        all += c;
        mine += b < blk ? c : 0;
      }
      if (all) atomicAdd(&first[e], all);       // integer sums: their order does not matter
      if (mine) atomicAdd(&before[e], mine);
    }
  }
  __syncthreads();
  scan_experts(first, a.E);
  if (blk == 0)
    for (int e = tid; e <= a.E; e += 1024) a.slots[e] = first[e];
  const int t0 = blk * a.per;
  const int n = min(a.per, a.T - t0) * a.k, live = first[a.E];
  for (int i = tid; i < n; i += 1024) {
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
// weights[t][j] * y[pos[t][j]].  Bound by the bytes of y: a wave owns 512
// columns of one token, so slots and weights are scalar loads and the rows'
// loads, up to eight in flight, go without a mask.
struct CombineArgs {
  const void* __restrict__ y;
  const int32_t* __restrict__ pos;
  const float* __restrict__ weights;
  const uint16_t* res;
  void* out;
  int64_t ld_res;
  uint32_t waves;        // tokens of the launch * parts
  int S, M8, k, parts;   // parts: waves per token
};

constexpr int64_t kCombineWaves = int64_t(1) << 25;   // most waves of a launch

struct Eight {
  f32x4_t lo, hi;
};

template <bool F16>
struct Raw8;   // eight columns as they lie in memory
template <>
struct Raw8<true> {
  half8_t h;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    h = *reinterpret_cast<const half8_t*>(static_cast<const _Float16*>(p) + at);
  }
  __device__ __forceinline__ Eight value() const {
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.lo[i] = static_cast<float>(h[i]);
      r.hi[i] = static_cast<float>(h[4 + i]);
    }
    return r;
  }
};
template <>
struct Raw8<false> {
  Eight v;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at);
    v.lo = q[0];
    v.hi = q[1];
  }
  __device__ __forceinline__ Eight value() const { return v; }
};

template <bool Y16, bool OUT16>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const uint32_t i = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (i >= a.waves) return;
  const int64_t t = i / static_cast<uint32_t>(a.parts);
  const int unit = 64 * static_cast<int>(i - t * a.parts) + (threadIdx.x & 63);
  if (unit >= a.M8) return;
  const int col = 8 * unit;
  const int64_t M = 8ll * a.M8;
  Raw8<true> r;
  if (a.res) r.load(a.res, t * a.ld_res + col);
  Eight sum = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    Raw8<Y16> v[8];
    bool has[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = a.pos[t * a.k + min(j0 + j, a.k - 1)];
      has[j] = j0 + j < a.k && static_cast<uint32_t>(p) < static_cast<uint32_t>(a.S);
      if (has[j]) v[j].load(a.y, p * M + col);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (has[j]) {
        const float w = a.weights[t * a.k + j0 + j];
        const Eight e = v[j].value();
        sum.lo += w * e.lo;
        sum.hi += w * e.hi;
      }
  }
  if (a.res) {
    const Eight e = r.value();
    sum.lo += e.lo;
    sum.hi += e.hi;
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
  if (E > kMaxRouteExperts || k > kMaxTopK || T > kMaxRouteTokens) return USW_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(T) * k >= (int64_t(1) << 31)) return USW_ERR_UNSUPPORTED;
  return USW_OK;
}

size_t route_bytes(int32_t T, int32_t E) {
  if (T <= kOneTokens) return 0;
  const int64_t blocks = (static_cast<int64_t>(T) + block_tokens(T) - 1) / block_tokens(T);
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
    route_one_kernel<<<1, 1024, (3 * E + 1) * sizeof(uint32_t), s>>>(a);
  } else {
    a.per = block_tokens(T);
    a.blocks = static_cast<int>((static_cast<int64_t>(T) + a.per - 1) / a.per);
    if (a.per == 32) route_choose_kernel<8><<<a.blocks, 512, E * sizeof(uint32_t), s>>>(a);
    else route_choose_kernel<16><<<a.blocks, 1024, 2 * E * sizeof(uint32_t), s>>>(a);
    const size_t lds = (2 * E + 1) * sizeof(uint32_t);
    while ((1 << a.lg_e) < E) ++a.lg_e;
    if (a.blocks > kAddBlocks) {
      route_scan_kernel<<<E, 64, 0, s>>>(a);
      route_place_kernel<true><<<a.blocks, 1024, lds, s>>>(a);
    } else {
      route_place_kernel<false><<<a.blocks, 1024, lds, s>>>(a);
    }
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
  a.ld_res = ld_res;
  a.S = S;
  a.M8 = M / 8;
  a.k = k;
  a.parts = (a.M8 + 63) / 64;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool y16 = y_type == USW_OUT_F16, o16 = out_type == USW_OUT_F16;
  // As many tokens a launch as stay under its 2^32 threads.
  const int64_t most = std::max<int64_t>(1, kCombineWaves / a.parts);
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    const int64_t n = std::min(most, T - t0);
    a.pos = pos + t0 * k;
    a.weights = weights + t0 * k;
    a.res = res ? res + t0 * ld_res : nullptr;
    a.out = static_cast<uint8_t*>(out) + t0 * M * (o16 ? 2 : 4);
    a.waves = static_cast<uint32_t>(n * a.parts);
    const dim3 grid((a.waves + 3) / 4);
    if (y16 && o16) combine_kernel<true, true><<<grid, 256, 0, s>>>(a);
    else if (y16) combine_kernel<true, false><<<grid, 256, 0, s>>>(a);
    else if (o16) combine_kernel<false, true><<<grid, 256, 0, s>>>(a);
    else combine_kernel<false, false><<<grid, 256, 0, s>>>(a);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

}  // extern "C"
