// Device half of libusw: the usw_spmm dispatcher of the bitmap SpMM decode kernels
// (usw_decode_kernels.h) and of the prefill kernels (usw_prefill.hip).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "usw.h"
#include "usw_internal.h"
#include "usw_decode_plan.h"

// Scratch of usw_spmm_noalloc (see scratch_address below): split-K counters
// and partial sums, one copy per GPU, kept until the process ends.
static __device__ __align__(256) uint8_t scratch[size_t(16) << 20];

namespace {

using namespace usw_dev;

// ---------------------------------------------------------------------------
// Host dispatch
// ---------------------------------------------------------------------------

// fp16 values with more than this many tokens take the prefill kernels;
// fewer take the decode kernels in passes of up to 64 tokens, which re-read
// the weight per pass but beat the 256-token prefill tiles up to 128 tokens
// on MI355X (at 128: 59.5 against 84.5 us on 11008x4096, 53.0 against 77.8
// on 4096x11008, 115.8 against 154.6 on 20480x5120; at 192 the prefill
// kernel is as fast or faster).
constexpr int kDecodeMaxN = 128;

bool use_prefill(const usw_fmt* f, int32_t N) { return f->val_type == USW_VAL_F16 && N > kDecodeMaxN; }

// Argument checks of a product call (nothing is written or launched).
usw_status check_call(const usw_fmt* f, const uint16_t* X, const void* Y, int32_t y_type, int32_t N,
                      usw::Geometry* g) {
  usw_status st = check_common(f, y_type, N, g);
  if (st) return st;
  if (!X || !Y || !f->bitmaps || !f->offsets || !f->values) return USW_ERR_NULL_ARG;
  if (f->val_type == USW_VAL_I4 && !f->scales) return USW_ERR_NULL_ARG;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(f->bitmaps) || !aligned16(f->values) ||
      (reinterpret_cast<uintptr_t>(f->offsets) & 3u))
    return USW_ERR_MISALIGNED;
  return USW_OK;
}

// Kernel choice, split factor and workspace of one call.
struct CallPlan {
  bool prefill;
  usw::PrefillPlan pp;   // prefill
  Plan p;                // decode
  size_t need;           // workspace bytes (0: none)
  size_t cb;             // leading counter bytes of the workspace
};

CallPlan make_call_plan(const usw_fmt* f, const usw::Geometry& g, int32_t N, int splits_req, bool tiles512 = true) {
  CallPlan c{};
  c.prefill = use_prefill(f, N);
  if (c.prefill) {
    c.pp = usw::prefill_plan(g, N, splits_req, tiles512);
    c.need = usw::prefill_workspace_bytes(g, N, c.pp);
    c.cb = usw::prefill_counter_bytes(g, c.pp);
  } else {
    c.p = make_plan(g, N, splits_req, f->val_type == USW_VAL_I4, lean_values(f, g));
    c.need = workspace_bytes(g, c.p);
    c.cb = c.need > 0 ? counters_bytes(g) : 0;
  }
  return c;
}

// Enqueue a planned call.  counters (c.cb bytes, zero at the start) and part
// (c.need - c.cb bytes) are used only when c.need > 0.
usw_status launch_call(const usw_fmt* f, const usw::Geometry& g, const CallPlan& c, const uint16_t* X, void* Y,
                       int32_t y_type, int32_t N, uint32_t* counters, float* part, void* stream) {
  if (c.prefill) return usw::prefill_launch(f, g, X, Y, y_type == USW_OUT_F16, N, counters, part, c.pp, stream);
  const Plan& p = c.p;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int M = static_cast<int>(g.M), K = static_cast<int>(g.K), Gc = static_cast<int>(g.Gc);
  const size_t ybytes = y_type == USW_OUT_F16 ? 2 : 4;
  const bool f16out = y_type == USW_OUT_F16;
  const bool i4 = f->val_type == USW_VAL_I4;
  const bool lean = lean_values(f, g);

  for (int n0 = 0; n0 < N; n0 += p.nchunk) {
    const int nc = std::min(p.nchunk, N - n0);
    // The shorter last pass of a multi-pass call has its own split factor.
    const int splits = (p.rchunk > 0 && n0 + p.nchunk > N) ? p.rsplits : p.splits;
    const int64_t nblk = g.Gr * splits;
    const dim3 grid(static_cast<unsigned>(nblk));
    Args a{};
    a.bitmaps = f->bitmaps;
    a.offsets = f->offsets;
    a.values = static_cast<const uint8_t*>(f->values);
    a.scales = i4 ? f->scales : nullptr;
    a.X = X + static_cast<size_t>(n0) * K;
    a.Y = static_cast<uint8_t*>(Y) + static_cast<size_t>(n0) * M * ybytes;
    a.counters = c.need ? counters : nullptr;
    a.part = c.need ? part : nullptr;
    a.values_alloc = usw::values_alloc_bytes(f->val_type, f->nnz);
    a.M = M;
    a.K = K;
    a.N = nc;
    a.Gc = Gc;
    a.splits = splits;
    a.remap = (splits > 1 && nblk % 8 == 0) ? 1 : 0;
    const int nb = nc > 32 ? 4 : nc > 16 ? 2 : 1;   // 16-token blocks of this pass
    launch_pass(a, p.ring, i4, lean, nb, f16out, grid, s);
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return USW_OK;
}

usw_status spmm_impl(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N, void* ws,
                     size_t ws_bytes, void* stream, int splits_req) {
  usw::Geometry g;
  usw_status st = check_call(f, X, Y, y_type, N, &g);
  if (st) return st;
  const CallPlan c = make_call_plan(f, g, N, splits_req);
  if (c.need > 0) {
    if (!ws || ws_bytes < c.need) return USW_ERR_WORKSPACE;
    if (!aligned16(ws)) return USW_ERR_MISALIGNED;
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  return launch_call(f, g, c, X, Y, y_type, N, reinterpret_cast<uint32_t*>(w),
                     c.need ? reinterpret_cast<float*>(w + c.cb) : nullptr, stream);
}

// ---------------------------------------------------------------------------
// Scratch-backed calls (usw_spmm_noalloc)
// ---------------------------------------------------------------------------
//
// The split-K counters and partial sums of usw_spmm_noalloc live in one
// statically allocated device array per GPU instead of a caller workspace:
// counters in its first kScratchCounterBytes, partial sums after them.  In
// host code the array's name is only a stand-in; its device address on the
// current GPU comes from hipGetSymbolAddress, taken once per device and kept.

constexpr size_t kScratchBytes = size_t(16) << 20;          // the whole array: 16 MiB
constexpr size_t kScratchCounterBytes = size_t(16) << 10;   // counters: up to 4096 tiles
constexpr int kMaxDevices = 64;
static_assert(sizeof(scratch) == kScratchBytes, "the scratch array has the stated size");

// Clears n 32-bit words (the counters a call needs at zero) with ordinary
// vector stores; a kernel, so that the call can be captured in a HIP graph.
__global__ __launch_bounds__(256) void scratch_clear_kernel(uint32_t* __restrict__ p, uint32_t n) {
  for (uint32_t i = threadIdx.x + blockIdx.x * 256u; i < n; i += 256u * gridDim.x) p[i] = 0u;
}

std::mutex g_scratch_mu;
uint8_t* g_scratch_ptr[kMaxDevices] = {};

// Device address of the scratch array on the current device.
usw_status scratch_address(uint8_t** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return USW_ERR_HIP;
  if (dev >= kMaxDevices) return USW_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return USW_ERR_HIP;
    g_scratch_ptr[dev] = static_cast<uint8_t*>(p);
  }
  *out = g_scratch_ptr[dev];
  return USW_OK;
}

usw_status spmm_noalloc_impl(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N,
                             int32_t splits, void* stream) {
  usw::Geometry g;
  usw_status st = check_call(f, X, Y, y_type, N, &g);
  if (st) return st;
  auto fits = [](const CallPlan& c) {
    return c.cb <= kScratchCounterBytes && c.need - c.cb <= kScratchBytes - kScratchCounterBytes;
  };
  CallPlan c = make_call_plan(f, g, N, splits < 0 ? 0 : splits);
  // The automatic factor falls back to 1 when its partial sums do not fit,
  // and N > 256 to the 256-token prefill kernel when the 512-token kernel's
  // copy of X does not.
  if (splits <= 0 && !fits(c)) c = make_call_plan(f, g, N, 1);
  if (splits <= 1 && c.prefill && !fits(c)) c = make_call_plan(f, g, N, 1, false);
  if (!fits(c)) return USW_ERR_WORKSPACE;
  uint8_t* base = nullptr;
  if (c.need > 0) {
    st = scratch_address(&base);
    if (st) return st;
    // The counters must be zero when the kernels start.  Every call leaves
    // them zero, but a call that overlapped another on this GPU may not.
    hipStream_t s = static_cast<hipStream_t>(stream);
    scratch_clear_kernel<<<1, 256, 0, s>>>(reinterpret_cast<uint32_t*>(base), static_cast<uint32_t>(c.cb / 4));
    if (hipGetLastError() != hipSuccess) return USW_ERR_HIP;
  }
  return launch_call(f, g, c, X, Y, y_type, N, reinterpret_cast<uint32_t*>(base),
                     c.need ? reinterpret_cast<float*>(base + kScratchCounterBytes) : nullptr, stream);
}

}  // namespace

extern "C" {

usw_status usw_spmm_workspace(const usw_fmt* f, int32_t N, size_t* bytes) {
  return usw_spmm_workspace_ex(f, N, 0, bytes);
}

usw_status usw_spmm(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N, void* ws,
                    size_t ws_bytes, void* stream) {
  return spmm_impl(f, X, Y, y_type, N, ws, ws_bytes, stream, 0);
}

usw_status usw_spmm_workspace_ex(const usw_fmt* f, int32_t N, int32_t splits, size_t* bytes) {
  if (!bytes) return USW_ERR_NULL_ARG;
  usw::Geometry g;
  usw_status st = check_common(f, USW_OUT_F16, N, &g);
  if (st) return st;
  const int sr = splits < 0 ? 0 : splits;
  if (use_prefill(f, N))
    *bytes = usw::prefill_workspace_bytes(g, N, usw::prefill_plan(g, N, sr));
  else
    *bytes = workspace_bytes(g, make_plan(g, N, sr, f->val_type == USW_VAL_I4, lean_values(f, g)));
  return USW_OK;
}

usw_status usw_spmm_counter_bytes(const usw_fmt* f, int32_t N, int32_t splits, size_t* bytes) {
  if (!bytes) return USW_ERR_NULL_ARG;
  usw::Geometry g;
  usw_status st = check_common(f, USW_OUT_F16, N, &g);
  if (st) return st;
  const int sr = splits < 0 ? 0 : splits;
  if (use_prefill(f, N)) {
    *bytes = usw::prefill_counter_bytes(g, usw::prefill_plan(g, N, sr));
  } else {
    const Plan p = make_plan(g, N, sr, f->val_type == USW_VAL_I4, lean_values(f, g));
    *bytes = workspace_bytes(g, p) > 0 ? counters_bytes(g) : 0;
  }
  return USW_OK;
}

usw_status usw_spmm_ex(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N, int32_t splits,
                       void* ws, size_t ws_bytes, void* stream) {
  return spmm_impl(f, X, Y, y_type, N, ws, ws_bytes, stream, splits < 0 ? 0 : splits);
}

usw_status usw_spmm_noalloc(const usw_fmt* f, const uint16_t* X, void* Y, int32_t y_type, int32_t N, int32_t splits,
                            void* stream) {
  return spmm_noalloc_impl(f, X, Y, y_type, N, splits, stream);
}

}  // extern "C"
