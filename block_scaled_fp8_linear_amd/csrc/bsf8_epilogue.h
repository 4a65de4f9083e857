// Device code that the products with an epilogue and by expert share: the
// epilogue, y = act(v + bias) + residual_scale * residual in F32, and the exact
// decoding of codes.  Not part of the ABI.
#pragma once

#include "bsf8_internal.h"

namespace bsf8 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// eight E4M3 codes as BF16 (exact: three of eight significand bits are used)
__device__ __forceinline__ v8bf decode8(uint32_t lo, uint32_t hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The activations keep their relative accuracy where the result is small (no
// 1 + tanh or 1 + erf near -1): gelu through erfc, the two others through 1 /
// (1 + exp).
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case BSF8_ACT_RELU: return fmaxf(v, 0.f);
    case BSF8_ACT_SILU: return v / (1.f + expf(-v));
    case BSF8_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case BSF8_ACT_GELU_TANH: {
      const float u = 1.5957691216057308f * (v + 0.044715f * v * v * v);   // 2 sqrt(2 / pi) (...)
      return v / (1.f + expf(-u));
    }
    default: return v;
  }
}

__device__ __forceinline__ float load_real(const void* p, int bf16, int64_t i) {
  if (bf16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
  return static_cast<const float*>(p)[i];
}

// one output: row r, column n of y
__device__ __forceinline__ float epilogue(const EpilogueDev& e, float v, int64_t r, int64_t n) {
  if (e.bias) v += load_real(e.bias, e.bias_bf16, n);
  v = activate(v, e.act);
  if (e.res) v = fmaf(e.alpha, load_real(e.res, e.res_bf16, r * e.ldr + n), v);
  return v;
}

}  // namespace bsf8
