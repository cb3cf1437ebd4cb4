// The sparse product with an epilogue, of one weight (usw_spmm_fused) and of
// E expert weights over ragged runs of rows (usw_expert_spmm):
//
//   y[n][m] = res[n][m] + mul[n][m] * act(sum_k W_sp[m][k] x[n][k] + bias[m]).
//
// Few rows run on the decode kernels (usw_decode_kernels.h), instantiated
// with arguments that carry the epilogue: it costs no launch and no pass over
// memory, since it works on the fp32 sums a strip's last workgroup holds.
// Many rows run on the expanded weight (usw_wide.hip).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "usw.h"
#include "usw_decode_plan.h"
#include "usw_internal.h"
#include "usw_wide.h"

namespace {

using namespace usw_dev;

constexpr int kMaxExperts = 1024;
// Most outputs of an expanded weight, and longest stride of such a weight's
// epilogue operands: the expanded product addresses a tile's rows with 32 bits.
constexpr int64_t kMaxLd = int64_t(1) << 20;
// Most outputs of a weight: a pass addresses its partial sums with 32 bits.
// Also the longest stride where a weight has too many outputs to be expanded;
// the passes address the operands with 64 bits.
constexpr int64_t kMaxM = int64_t(1) << 22;

// HIP's limit on a launch is 2^32 threads.
bool launchable(int64_t workgroups, bool ring) {
  return workgroups < (int64_t(1) << 32) / (ring ? kRingThreads : DefaultCfg::kThreadsPerGroup);
}
static_assert(DefaultCfg::kThreadsPerGroup == 256 && DefaultCfg8::kThreadsPerGroup == 256, "every per-wave configuration alike");

// Checks an epilogue for rows of M outputs and fills the kernels' copy.
usw_status make_epilogue(const usw_epilogue* ep, int64_t M, int32_t y_type, Epilogue* e) {
  *e = Epilogue{nullptr, nullptr, nullptr, M, M, USW_ACT_NONE, y_type == USW_OUT_F16 ? 1 : 0};
  if (!ep) return USW_OK;
  if (ep->act < USW_ACT_NONE || ep->act > USW_ACT_SILU) return USW_ERR_BAD_DTYPE;
  if (ep->reserved != 0) return USW_ERR_BAD_SHAPE;
  e->act = ep->act;
  e->bias = ep->bias;
  e->mul = ep->mul;
  e->res = ep->res;
  if (ep->mul && ep->ld_mul != 0) e->ld_mul = ep->ld_mul;
  if (ep->res && ep->ld_res != 0) e->ld_res = ep->ld_res;
  const int64_t longest = M <= kMaxLd ? kMaxLd : kMaxM;
  if (e->ld_mul < M || e->ld_res < M || (ep->mul && e->ld_mul > longest) || (ep->res && e->ld_res > longest))
    return USW_ERR_BAD_SHAPE;
  if (!aligned16(ep->bias) || !aligned16(ep->mul) || !aligned16(ep->res) || e->ld_mul % 8 || e->ld_res % 8)
    return USW_ERR_MISALIGNED;
  return USW_OK;
}

// ---------------------------------------------------------------------------
// One weight
// ---------------------------------------------------------------------------

struct FusedPlan {
  bool wide;
  Plan p;               // decode passes
  usw::WidePlan w;
  size_t need, cb;
};

bool fits_wide(const usw::Geometry& g) { return g.M <= kMaxLd; }

// Rows from which the weight is expanded; fewer take passes of up to 128 rows
// that rebuild it each time (MI355X, passes / expanded).  Weights of up to
// 2^22 elements, whose expansion is short: 640x640 N = 96 11.8 / 9.9 us,
// 2048x2048 N = 72 17.9 / 17.0, N = 128 24.0 / 17.4.  Above, one pass is ahead:
// 4096x4096 N = 128 26.3 / 27.0, 11008x4096 N = 96 32.7 / 50.8, N = 128 41.4 /
// 51.2; two are not, 4096x4096 N = 160 36.5 / 31.8, 11008x4096 N = 192 64.1 /
// 59.8, except on the largest fp16 weights: 20480x5120 N = 160 130 / 149, N =
// 192 149 / 170, N = 256 194 / 189; INT4, whose expansion reads less, N = 160
// 136 / 132.  A caller's split factor asks for the passes.
bool use_wide(const usw_fmt* f, const usw::Geometry& g, int32_t N, int splits_req) {
  const int64_t elements = g.M * g.K;
  const bool largest = elements > (int64_t(1) << 26) && f->val_type == USW_VAL_F16;
  const int from = elements <= (int64_t(1) << 22) ? 64 : largest ? 192 : 128;
  return N > from && splits_req <= 0 && fits_wide(g);
}

FusedPlan plan_fused(const usw_fmt* f, const usw::Geometry& g, int32_t N, int splits_req) {
  FusedPlan c{};
  c.wide = use_wide(f, g, N, splits_req);
  if (c.wide) {
    c.w = usw::wide_plan(g, 1, N);
    c.need = c.w.need;
    c.cb = c.w.cb;
    return c;
  }
  c.p = make_plan<FusedArgs>(g, N, splits_req, f->val_type == USW_VAL_I4, lean_values(f, g));
  c.need = workspace_bytes(g, c.p);
  if (c.need > 0) {
    c.cb = usw::counter_zone(counters_bytes(g));
    c.need += c.cb - counters_bytes(g);
  }
  return c;
}

usw_status fused_impl(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N, const usw_epilogue* ep,
                      int splits_req, void* ws, size_t ws_bytes, void* stream) {
  usw::Geometry g;
  usw_status st = check_common(f, y_type, N, &g);
  if (st) return st;
  if (!X || !Y || !f->bitmaps || !f->offsets || !f->values) return USW_ERR_NULL_ARG;
  const bool i4 = f->val_type == USW_VAL_I4;
  if (i4 && !f->scales) return USW_ERR_NULL_ARG;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(f->bitmaps) || !aligned16(f->values) ||
      (reinterpret_cast<uintptr_t>(f->offsets) & 3u) || (i4 && !aligned16(f->scales)))
    return USW_ERR_MISALIGNED;
  if (g.M > kMaxM) return USW_ERR_UNSUPPORTED;
  Epilogue e;
  st = make_epilogue(ep, g.M, y_type, &e);
  if (st) return st;
  const FusedPlan c = plan_fused(f, g, N, splits_req);
  if (!c.wide && !launchable(g.Gr * std::max(c.p.splits, c.p.rsplits), c.p.ring)) return USW_ERR_UNSUPPORTED;
  if (c.need > 0) {
    if (!ws || ws_bytes < c.need) return USW_ERR_WORKSPACE;
    if (!aligned16(ws)) return USW_ERR_MISALIGNED;
  }
  if (c.wide) {
    usw::WideCall w{};
    w.bitmaps = f->bitmaps;
    w.offsets = f->offsets;
    w.values = static_cast<const uint8_t*>(f->values);
    w.scales = f->scales;
    w.values_total = static_cast<int64_t>(usw::values_alloc_bytes(f->val_type, f->nnz));
    w.val_type = f->val_type;
    w.E = 1;
    w.X = X;
    w.S = w.T = N;
    w.Y = Y;
    w.e = e;
    return usw::wide_launch(w, g, c.w, ws, stream);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Plan& p = c.p;
  const bool lean = lean_values(f, g);
  for (int n0 = 0; n0 < N; n0 += p.nchunk) {
    const int nc = std::min(p.nchunk, N - n0);
    const int splits = (p.rchunk > 0 && n0 + p.nchunk > N) ? p.rsplits : p.splits;
    const int64_t nblk = g.Gr * splits;
    FusedArgs a{};
    a.bitmaps = f->bitmaps;
    a.offsets = f->offsets;
    a.values = static_cast<const uint8_t*>(f->values);
    a.scales = i4 ? f->scales : nullptr;
    a.X = X + static_cast<size_t>(n0) * g.K;
    a.Y = static_cast<uint8_t*>(Y) + static_cast<size_t>(n0) * g.M * (e.f16out ? 2 : 4);
    if (c.need) {
      a.counters = static_cast<uint32_t*>(ws);
      a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + c.cb);
    }
    a.values_alloc = usw::values_alloc_bytes(f->val_type, f->nnz);
    a.M = static_cast<int>(g.M);
    a.K = static_cast<int>(g.K);
    a.N = nc;
    a.Gc = static_cast<int>(g.Gc);
    a.splits = splits;
    a.remap = (splits > 1 && nblk % 8 == 0) ? 1 : 0;
    a.e = e;
    if (e.mul) a.e.mul += e.ld_mul * n0;
    if (e.res) a.e.res += e.ld_res * n0;
    const int nb = pass_chunk(nc, p.nchunk) / 16;
    launch_pass(a, p.ring, i4, lean, nb, e.f16out, dim3(static_cast<unsigned>(nblk)), s);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

// ---------------------------------------------------------------------------
// By expert
// ---------------------------------------------------------------------------

struct ExpertPlan {
  bool wide;
  usw::WidePlan w;
  int lg_chunk;      // slots per tile: 16, 32 or 64
  int64_t tiles;     // most tiles the slots can make
  int splits;        // workgroups per tile and 64-row strip
  bool ring, lean;
  size_t need, cb;
};

usw_status check_expert(const usw_expert_fmt* f, int32_t y_type, int32_t S, usw::Geometry* g) {
  if (!f) return USW_ERR_NULL_ARG;
  usw_status st = usw::make_geometry(f->M, f->K, kGT, kGT, g);
  if (st) return st;
  if (f->E < 1 || f->reserved != 0) return USW_ERR_BAD_SHAPE;
  if (f->E > kMaxExperts || g->M > kMaxM) return USW_ERR_UNSUPPORTED;
  if (f->val_type != USW_VAL_F16 && f->val_type != USW_VAL_I4) return USW_ERR_BAD_DTYPE;
  if (y_type != USW_OUT_F16 && y_type != USW_OUT_F32) return USW_ERR_BAD_DTYPE;
  if (S < 0) return USW_ERR_BAD_N;
  if (f->nnz < 0 || f->nnz > f->E * g->M * g->K || f->values_bytes < 16 * int64_t(f->E) || f->values_bytes % 16)
    return USW_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(S) * g->M > (int64_t(1) << 40)) return USW_ERR_BAD_SHAPE;
  return USW_OK;
}

ExpertPlan plan_expert(const usw_expert_fmt* f, const usw::Geometry& g, int32_t S) {
  ExpertPlan p{};
  const bool i4 = f->val_type == USW_VAL_I4;
  // By the bank's mean density, the one that the host has.  An expert above
  // 62% in a bank below 55% takes the unpipelined path (8 of 11008x4096 with 8
  // rows each, seven 50% and one 70% dense: 149 us; the six-chunk kernels 94,
  // and all at 54% 100).
  p.lean = !i4 && static_cast<double>(f->nnz) <= 0.55 * static_cast<double>(f->E) * g.M * g.K;
  const int64_t active = std::min<int64_t>(f->E, S);
  const int64_t mean = S / std::max<int64_t>(1, active);
  // Rows per expert from which expanding pays (MI355X, fp16): with weights of
  // up to 2^26 elements in all, where the passes leave compute units idle,
  // 128 (8 experts of 2048x2048: 43.9 us in passes, 42.9 expanded; 16 of
  // 2048x1024, 250 rows each: 69.8 / 50.9); above, 224 (8 of 11008x4096, 200
  // rows each: 428 / 481; 8 of 4096x11008, 500 rows each: 800 / 684).  With up
  // to 4 GroupTile columns, less than one for each wave of a split, 80 (26 of
  // 8192x256, 88 rows each: 82.2 / 65.5; 8 of 8192x256, 64 rows: 25.4 / 27.8),
  // with one column 32 (8 of 4096x64, 32 rows each: 10.2 / 10.4; 26 of
  // 12672x64, 88 rows: 107 / 48.3).
  const int from = g.Gc == 1 ? 32 : g.Gc <= 4 ? 80 : f->E * g.M * g.K <= (int64_t(1) << 26) ? 128 : 224;
  p.wide = mean >= from && fits_wide(g);
  if (p.wide) {
    p.w = usw::wide_plan(g, f->E, S);
    p.need = p.w.need;
    p.cb = p.w.cb;
    return p;
  }
  p.lg_chunk = mean <= 8 ? 4 : mean <= 24 ? 5 : 6;
  const int chunk = 1 << p.lg_chunk;
  p.tiles = active + (S - active) / chunk;
  p.ring = p.lean && chunk == 16;
  // One round of resident workgroups over the tiles, as the plain product
  // splits a matrix with that many strips.  Where it takes a workgroup per
  // compute unit, half as many more: runs fill about two thirds of the tiles
  // that p.tiles bounds (26 experts of 256x12288 with 38 rows each 66.7 us
  // with 256 workgroups, 44.0 with 384; 8 of 1024x8192 with 38 rows 47.9 /
  // 39.3; 512 or more no better there, 4 of 512x16384 with 50 rows 33.0 / 27.4
  // / 32.2 with 512).
  usw::Geometry gt = g;
  gt.Gr = g.Gr * p.tiles;
  int64_t want = 0;
  if (chunk == 64 && gt.Gr <= kComputeUnits)
    want = std::min<int64_t>(kComputeUnits * 3 / 2 / gt.Gr, std::max<int64_t>(1, g.Gc / 12));
  const Plan one = make_plan<ExpertArgs>(gt, chunk, static_cast<int>(want), i4, p.lean);
  p.splits = one.splits;
  if (p.splits > 1) {
    p.cb = usw::counter_zone(static_cast<size_t>(4) * p.tiles * g.Gr);
    p.need = p.cb + static_cast<size_t>(p.splits) * S * g.M * sizeof(float);
  }
  return p;
}

usw_status expert_impl(const usw_expert_fmt* f, const uint16_t* X, int32_t T, const int32_t* slots,
                       const int32_t* rows, int32_t S, void* Y, int32_t y_type, const usw_epilogue* ep, void* ws,
                       size_t ws_bytes, void* stream) {
  usw::Geometry g;
  usw_status st = check_expert(f, y_type, S, &g);
  if (st) return st;
  const bool i4 = f->val_type == USW_VAL_I4;
  if (T < 0 || (!rows && T < S) || (S > 0 && T == 0)) return USW_ERR_BAD_N;
  if (!f->bitmaps || !f->offsets || !f->values || !f->starts || (i4 && !f->scales) || !slots) return USW_ERR_NULL_ARG;
  if (S > 0 && (!X || !Y)) return USW_ERR_NULL_ARG;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(f->bitmaps) || !aligned16(f->values) ||
      ((reinterpret_cast<uintptr_t>(f->offsets) | reinterpret_cast<uintptr_t>(slots) |
        reinterpret_cast<uintptr_t>(rows)) & 3u) ||
      (reinterpret_cast<uintptr_t>(f->starts) & 7u) || (i4 && !aligned16(f->scales)))
    return USW_ERR_MISALIGNED;
  Epilogue e;
  st = make_epilogue(ep, g.M, y_type, &e);
  if (st) return st;
  if (S == 0) return USW_OK;
  const ExpertPlan p = plan_expert(f, g, S);
  const int64_t per = g.Gr * p.splits;   // workgroups of a tile
  if (!p.wide && !launchable(p.tiles * per, p.ring)) return USW_ERR_UNSUPPORTED;
  if (p.need > 0) {
    if (!ws || ws_bytes < p.need) return USW_ERR_WORKSPACE;
    if (!aligned16(ws)) return USW_ERR_MISALIGNED;
  }
  if (p.wide) {
    usw::WideCall w{};
    w.bitmaps = f->bitmaps;
    w.offsets = f->offsets;
    w.values = static_cast<const uint8_t*>(f->values);
    w.starts = f->starts;
    w.scales = f->scales;
    w.values_total = f->values_bytes;
    w.val_type = f->val_type;
    w.E = f->E;
    w.X = X;
    w.slots = slots;
    w.rows = rows;
    w.S = S;
    w.T = T;
    w.Y = Y;
    w.e = e;
    return usw::wide_launch(w, g, p.w, ws, stream);
  }
  ExpertArgs a{};
  a.bitmaps = f->bitmaps;
  a.offsets = f->offsets;
  a.values = static_cast<const uint8_t*>(f->values);
  a.scales = i4 ? f->scales : nullptr;
  a.X = X;
  a.Y = Y;
  if (p.need) {
    a.counters = static_cast<uint32_t*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.cb);
  }
  a.M = static_cast<int>(g.M);
  a.K = static_cast<int>(g.K);
  a.Gc = static_cast<int>(g.Gc);
  a.splits = p.splits;
  a.remap = per % 8 == 0 ? 1 : 0;
  a.e = e;
  a.slots = slots;
  a.rows = rows;
  a.starts = f->starts;
  a.values_total = f->values_bytes;
  a.nbt = g.nbt;
  a.noff = g.ngt + 1;
  a.E = f->E;
  a.S = S;
  a.T = T;
  a.lg_chunk = p.lg_chunk;
  a.Gr = static_cast<int>(g.Gr);
  launch_pass(a, p.ring, i4, p.lean, 1 << (p.lg_chunk - 4), e.f16out, dim3(static_cast<unsigned>(p.tiles * per)),
              static_cast<hipStream_t>(stream));
  return hipGetLastError() == hipSuccess ? USW_OK : USW_ERR_HIP;
}

}  // namespace

extern "C" {

usw_status usw_spmm_fused_workspace(const usw_fmt* f, int32_t N, int32_t splits, size_t* bytes, size_t* counter_bytes) {
  if (!bytes || !counter_bytes) return USW_ERR_NULL_ARG;
  usw::Geometry g;
  usw_status st = check_common(f, USW_OUT_F16, N, &g);
  if (st) return st;
  const FusedPlan c = plan_fused(f, g, N, splits < 0 ? 0 : splits);
  *bytes = c.need;
  *counter_bytes = c.cb;
  return USW_OK;
}

usw_status usw_spmm_fused(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N,
                          const usw_epilogue* ep, int32_t splits, void* ws, size_t ws_bytes, void* stream) {
  return fused_impl(f, X, Y, y_type, N, ep, splits < 0 ? 0 : splits, ws, ws_bytes, stream);
}

usw_status usw_expert_spmm_workspace(const usw_expert_fmt* f, int32_t S, size_t* bytes, size_t* counter_bytes) {
  if (!bytes || !counter_bytes) return USW_ERR_NULL_ARG;
  usw::Geometry g;
  usw_status st = check_expert(f, USW_OUT_F16, S, &g);
  if (st) return st;
  *bytes = *counter_bytes = 0;
  if (S == 0) return USW_OK;
  const ExpertPlan p = plan_expert(f, g, S);
  *bytes = p.need;
  *counter_bytes = p.cb;
  return USW_OK;
}

usw_status usw_expert_spmm(const usw_expert_fmt* f, const uint16_t* X, int32_t T, const int32_t* slots,
                           const int32_t* rows, int32_t S, void* Y, int32_t y_type, const usw_epilogue* ep, void* ws,
                           size_t ws_bytes, void* stream) {
  return expert_impl(f, X, T, slots, rows, S, Y, y_type, ep, ws, ws_bytes, stream);
}

}  // extern "C"
