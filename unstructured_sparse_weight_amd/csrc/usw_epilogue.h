// The epilogue of the fused products: what happens to the fp32 sums of an
// output tile before they are rounded and stored,
//
//   y[n][m] = res[n][m] + mul[n][m] * act(scale[m] * sum + bias[m]),
//
// each operand optional.  Everything is computed in fp32 on the sums where
// the kernel already holds them, so the output is rounded once and neither
// the pre-activation nor any intermediate reaches memory.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "usw.h"
#include "usw_device.h"

namespace usw_dev {

struct Epilogue {
  const uint16_t* __restrict__ bias;   // fp16 [M] or null
  const uint16_t* __restrict__ mul;    // fp16 [rows][ld_mul] or null
  const uint16_t* __restrict__ res;    // fp16 [rows][ld_res] or null
  int64_t ld_mul, ld_res;
  int act;                             // usw_act
  int f16out;                          // y is fp16, else fp32
};

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

// GELU by erfc, which keeps its relative accuracy where v is negative; 1 + erf
// would cancel there (v = -5: 4% off).  It is the dearer of the two
// (11008x4096 N = 2048 242 us against 232, few rows equal).
//
// GELU's tanh form is v times the logistic function of 2z, z = sqrt(2/pi)
// (v + 0.044715 v^3), because (1 + tanh z) / 2 = 1 / (1 + exp(-2z)).  For
// very negative v the exponential overflows to infinity and the product is
// the limit, -0.  ReLU keeps NaN.  __expf is off by its argument's rounding,
// z 2^-24 relative, which only shows where the output is a small e^z.  The
// hardware's reciprocal is within one unit in the last place, where an IEEE
// quotient would take ten instructions more for each output (11008x4096
// N = 2048, SiLU and mul: 220.6 us, with the quotient 226.8).
template <int ACT>
__device__ __forceinline__ float activation(float v) {
  if constexpr (ACT == USW_ACT_RELU) return v < 0.0f ? 0.0f : v;
  else if constexpr (ACT == USW_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  else if constexpr (ACT == USW_ACT_GELU_TANH)
    return v * __builtin_amdgcn_rcpf(1.0f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
  else if constexpr (ACT == USW_ACT_SILU) return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
  else return v;
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case USW_ACT_RELU: return activation<USW_ACT_RELU>(v);
    case USW_ACT_GELU: return activation<USW_ACT_GELU>(v);
    case USW_ACT_GELU_TANH: return activation<USW_ACT_GELU_TANH>(v);
    case USW_ACT_SILU: return activation<USW_ACT_SILU>(v);
    default: return v;
  }
}

__device__ __forceinline__ f32x4_t to_float4(half4_t h) {
  return f32x4_t{static_cast<float>(h.x), static_cast<float>(h.y), static_cast<float>(h.z), static_cast<float>(h.w)};
}
__device__ __forceinline__ f32x4_t load_half4(const uint16_t* p) { return to_float4(*reinterpret_cast<const half4_t*>(p)); }

__device__ __forceinline__ half4_t to_half4(f32x4_t v) {
  half4_t h;
  h.x = static_cast<_Float16>(v.x);
  h.y = static_cast<_Float16>(v.y);
  h.z = static_cast<_Float16>(v.z);
  h.w = static_cast<_Float16>(v.w);
  return h;
}

// Stores four outputs, rounded to y's type, at y + at.
__device__ __forceinline__ void store_out4(void* y, int64_t at, int f16out, f32x4_t v) {
  if (f16out) {
    *reinterpret_cast<half4_t*>(static_cast<_Float16*>(y) + at) = to_half4(v);
  } else {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(y) + at) = v;
  }
}

// Applies the epilogue to the sums of row n, outputs m .. m+3 (m a multiple
// of 4), and stores them at y + n M + m.
__device__ __forceinline__ void epilogue_store4(const Epilogue& e, void* y, int M, int64_t n, int m, f32x4_t v) {
  if (e.bias) v += load_half4(e.bias + m);
  if (e.act != USW_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = activate(v[j], e.act);
  }
  if (e.mul) v *= load_half4(e.mul + n * e.ld_mul + m);
  if (e.res) v += load_half4(e.res + n * e.ld_res + m);
  store_out4(y, n * M + m, e.f16out, v);
}

}  // namespace usw_dev
