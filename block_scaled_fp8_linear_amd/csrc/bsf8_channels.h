// Device code that the operators on rows of channels share: eight consecutive channels
// per lane, loaded and stored 16 bytes at a time where addresses allow it, and the E4M3
// quantization of a 128-channel group.  Not part of the ABI.
#pragma once

#include "bsf8_internal.h"

namespace bsf8 {

constexpr int EPL = 8;                   // channels per lane and vector
constexpr int LPG = kBlock / EPL;        // lanes per 128-channel scale group
constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 1e-10f;

// EPL raw values: 16 bytes of BF16 or 32 of F32
template <bool BF16>
struct Raw {
  uint32_t w[BF16 ? EPL / 2 : EPL];
};

// EPL values from element off; zeros from element `valid` on
template <bool BF16>
__device__ __forceinline__ void load_raw(const void* p, int64_t off, int valid, bool vec, Raw<BF16>& r) {
  constexpr int W = BF16 ? EPL / 2 : EPL;
#pragma unroll
  for (int i = 0; i < W; ++i) r.w[i] = 0;
  if (valid <= 0) return;
  if (valid == EPL && vec) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + off * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 u = q[i];
      r.w[4 * i] = u.x;
      r.w[4 * i + 1] = u.y;
      r.w[4 * i + 2] = u.z;
      r.w[4 * i + 3] = u.w;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < EPL; ++e) {
    if (e >= valid) continue;
    if (BF16)
      r.w[e >> 1] |= uint32_t(static_cast<const uint16_t*>(p)[off + e]) << (16 * (e & 1));
    else
      r.w[e] = static_cast<const uint32_t*>(p)[off + e];
  }
}

template <bool BF16>
__device__ __forceinline__ float value(const Raw<BF16>& r, int e) {
  if (BF16) return __uint_as_float((e & 1) ? r.w[e >> 1] & 0xFFFF0000u : r.w[e >> 1] << 16);
  return __uint_as_float(r.w[e]);
}

// a per-channel vector (norm weight, bias, gate) of either type
__device__ __forceinline__ void load_vec(const void* p, int bf16, int64_t off, int valid, bool vec, float (&v)[EPL]) {
  if (bf16) {
    Raw<true> r;
    load_raw<true>(p, off, valid, vec, r);
#pragma unroll
    for (int e = 0; e < EPL; ++e) v[e] = value<true>(r, e);
  } else {
    Raw<false> r;
    load_raw<false>(p, off, valid, vec, r);
#pragma unroll
    for (int e = 0; e < EPL; ++e) v[e] = value<false>(r, e);
  }
}

typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const v2bf16 r = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ void store_row(void* p, bool bf16, int64_t off, int valid, bool vec, const float (&v)[EPL]) {
  if (valid <= 0) return;
  if (bf16) {
    uint16_t* q = static_cast<uint16_t*>(p) + off;
    const uint32_t w[4] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    if (valid == EPL && vec) {
      *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        if (e < valid) q[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* q = static_cast<float*>(p) + off;
    if (valid == EPL && vec) {
      reinterpret_cast<float4*>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        if (e < valid) q[e] = v[e];
    }
  }
}

// The rounding to F32.  The compiler must not see past it: it would merge it
// with a rounding to BF16 that follows into one from F64, which lands on the
// other side where the F32 value is a BF16 midpoint, so the stored BF16 would
// not be the rounding of the F32 value that the codes are made of (and the
// merged form takes nine instructions more).
__device__ __forceinline__ float to_f32(double v) {
  float f = static_cast<float>(v);
  asm("" : "+v"(f));
  return f;
}

// The scale of a group, max(amax, 1e-10) / 448, and EPL codes, bit for bit what
// the IEEE divisions of the activation quantizer give, without dividing.  With r
// = RN(1 / b), q0 = a * r and the exact remainder e = a - q0 * b (one FMA), RN(q0
// + e * r) is the correctly rounded quotient a / b (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990).  For
// the scale r is a constant.  For the codes r comes from the hardware's F64
// reciprocal and two Newton steps (relative error below 2^-52; 1 / s is at least
// 2^-49 from a midpoint of two F32 values), rounded to F32.  The remainder is
// exact for |n| >= 2^-100; below, n / s < 2^-57 and its code is zero whatever
// its last bit.  A negative zero passes the remainder as +0, so the sign of n
// is put back.  No clamp: |n| <= amax makes the quotient at most 448 (1 +
// 2^-23), which rounds to the code of 448.
__device__ __forceinline__ void encode(const float (&n)[EPL], float amax, float& s, uint32_t (&packed)[EPL / 4]) {
  const float a = fmaxf(amax, kAmaxFloor);
  constexpr float kInv = 1.0f / kE4M3Max;
  const float s0 = a * kInv;
  s = fmaf(fmaf(-s0, kE4M3Max, a), kInv, s0);
  const double sd = double(s);
  double rd = __builtin_amdgcn_rcp(sd);
  rd = fma(fma(-sd, rd, 1.0), rd, rd);
  rd = fma(fma(-sd, rd, 1.0), rd, rd);
  const float r = static_cast<float>(rd);
#pragma unroll
  for (int q = 0; q < EPL / 4; ++q) {
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = n[4 * q + e];
      const float f0 = v * r;
      f[e] = copysignf(fmaf(fmaf(-f0, s, v), r, f0), v);
    }
    int pk = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    pk = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], pk, true);
    packed[q] = uint32_t(pk);
  }
}

// 1 / sqrt(x) to within an F64 rounding or two: the hardware's estimate and two Newton steps
__device__ __forceinline__ double rsqrt64(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(0.5 * y, fma(-x * y, y, 1.0), y);
  return y;
}

}  // namespace bsf8
