// Device code that the products with an epilogue and by expert share: the
// epilogue, y = act(v + bias) + residual_scale * residual in F32, the exact
// decoding of codes, and the experts' row runs.  Not part of the ABI.
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

// The activations from the hardware's exp2 and reciprocal (each within a unit or
// two in the last place), in F32, without a division: with the library's expf and
// the IEEE division a 256 x 256 tile's activations took 8 us, a tenth of it.  The
// error is below 4 * 2^-24 |v|: the exponent's rounding, |u| 2^-24 relative, meets
// sigma(u) <= 1 / (1 + |u|) where u is negative and 1 - sigma where it is positive.
// Relative to the result it is below (6 + 1.5 |u|) 2^-24, and u's own error for a u
// that is computed, down to 2^-118 (exp2 and the reciprocal know no denormals).
__device__ __forceinline__ float times_sigmoid(float v, float u) {   // v / (1 + exp(-u))
  return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u * -1.4426950408889634f));
}
__device__ __forceinline__ float relu(float v) { return v < 0.f ? 0.f : v; }   // (NaN stays NaN)
__device__ __forceinline__ float silu(float v) { return times_sigmoid(v, v); }
__device__ __forceinline__ float gelu_tanh(float v) {   // u = 2 sqrt(2 / pi) (v + 0.044715 v^3)
  return times_sigmoid(v, v * fmaf(v * v, 0.071354816272600248f, 1.5957691216057308f));
}
// v Phi(v) with the tail |v| Phi(-|v|) = |v| / 2 * erfc(|v| / sqrt(2)), and
// erfc(|v| / sqrt(2)) = exp(-v^2 / 2) t P(t - 1/2), t = 1 / (1 + 0.35 |v|).  P is a
// polynomial of degree eight, fitted to the least relative error over 0 <= |v| <= 14
// (2^-24.9; the result is below 2^-126 beyond).  The error is relative to the tail, so
// it shrinks with the result where v is negative: below (19 + 1.25 v^2) 2^-24 of it,
// v^2 from the roundings of the exponent, 9 from those of t (the tail's slope in t is
// 2.3 at 0), the rest from the polynomial and the products.  (A form with an absolute
// bound on erfc was wrong by 1e-2 of the result at -7, three bits of a BF16 output.)
__device__ __forceinline__ float gelu(float v) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(v), 0.35f, 1.f));
  const float s = t - 0.5f;
  float p = fmaf(s, -0.0582918764f, 0.0547759776f);
  p = fmaf(s, p, 0.0883303399f);
  p = fmaf(s, p, -0.112277419f);
  p = fmaf(s, p, -0.163480295f);
  p = fmaf(s, p, 0.16374165f);
  p = fmaf(s, p, 0.568791597f);
  p = fmaf(s, p, 0.685983216f);
  p = fmaf(s, p, 0.506488546f);
  const float tail = 0.5f * v * t * p * __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);
  // (at +inf the tail is inf * 0: the smaller of v - NaN and v is v)
  return v >= 0.f ? fminf(v - tail, v) : tail;
}
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case BSF8_ACT_RELU: return relu(v);
    case BSF8_ACT_SILU: return silu(v);
    case BSF8_ACT_GELU: return gelu(v);
    case BSF8_ACT_GELU_TANH: return gelu_tanh(v);
    default: return v;
  }
}
// The same over an array: one branch for all of it, four values at a time (as
// many as keep the latencies covered; the scheduler would interleave all of them,
// and their intermediates would crowd out the tile).
template <int N, typename F>
__device__ __forceinline__ void by_fours(float (&v)[N], F f) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i + e] = f(v[i + e]);
    __builtin_amdgcn_sched_barrier(0);
  }
}
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  if (act == BSF8_ACT_RELU) by_fours(v, relu);
  else if (act == BSF8_ACT_SILU) by_fours(v, silu);
  else if (act == BSF8_ACT_GELU) by_fours(v, gelu);
  else if (act == BSF8_ACT_GELU_TANH) by_fours(v, gelu_tanh);
}

// element i of a BF16 or F32 array as raw bits, and their value
__device__ __forceinline__ uint32_t load_bits(const void* p, int bf16, int64_t i) {
  if (bf16) return static_cast<const uint16_t*>(p)[i];
  return static_cast<const uint32_t*>(p)[i];
}
__device__ __forceinline__ float widen(uint32_t bits, int bf16) { return __uint_as_float(bf16 ? bits << 16 : bits); }

__device__ __forceinline__ float load_real(const void* p, int bf16, int64_t i) {
  if (bf16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
  return static_cast<const float*>(p)[i];
}

// four outputs of one row, columns that follow each other (nvalid of them
// exist): bias values b, the residual from element `at` on
typedef float bsf8_f4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bsf8_f4 finish4(const EpilogueDev& e, bsf8_f4 v, const float (&b)[4], int64_t at, int nvalid) {
  float r[4] = {0.f, 0.f, 0.f, 0.f};
  if (e.res) {
    if (e.res_bf16) {
      const uint16_t* p = static_cast<const uint16_t*>(e.res) + at;
      if (nvalid == 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        r[0] = __uint_as_float(u.x << 16);
        r[1] = __uint_as_float(u.x & 0xFFFF0000u);
        r[2] = __uint_as_float(u.y << 16);
        r[3] = __uint_as_float(u.y & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < nvalid) r[i] = __uint_as_float(uint32_t(p[i]) << 16);
      }
    } else {
      const float* p = static_cast<const float*>(e.res) + at;
      if (nvalid == 4 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        r[0] = u.x;
        r[1] = u.y;
        r[2] = u.z;
        r[3] = u.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < nvalid) r[i] = p[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = activate(v[i] + b[i], e.act);
  if (e.res) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(e.alpha, r[i], v[i]);
  }
  return v;
}

// Experts' row runs as the kernels take them.  Each expert's rows are cut into
// tiles of T; all tiles of all experts, times the weight's row tiles, are the
// blocks that have work.  The runs lie in device memory, so each wave counts the
// tiles of 64 experts at a time and sums across its lanes.  Offsets are clamped
// to [0, R], so nothing in device memory can lead an access out of bounds.
__device__ __forceinline__ int run_tiles(const int32_t* offsets, int E, int R, int T, int e, int& lo, int& hi) {
  const int i = min(e, E - 1);
  lo = min(max(offsets[i], 0), R);
  hi = min(max(offsets[i + 1], lo), R);
  return e < E ? (hi - lo + T - 1) / T : 0;
}
// 64 experts' tiles, one expert per lane: rows, tiles, and the tiles up to and with it.
struct Runs {
  int lo, hi, n, sum;
};
__device__ __forceinline__ Runs runs_of(const int32_t* offsets, int E, int R, int T, int base) {
  const int lane = threadIdx.x & 63;
  Runs r;
  r.n = run_tiles(offsets, E, R, T, base + lane, r.lo, r.hi);
  r.sum = r.n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(r.sum, d, 64);
    if (lane >= d) r.sum += up;
  }
  return r;
}
// Tiles of all experts; `first` keeps those of the first 64 experts.  Ascending
// offsets make at most min(E, R) + R / T of them, and the count ends there, so
// that overlapping runs (descending offsets) cannot pass 32 bits.
__device__ __forceinline__ int all_run_tiles(const int32_t* offsets, int E, int R, int T, Runs& first) {
  first = runs_of(offsets, E, R, T, 0);
  int sum = __builtin_amdgcn_readlane(first.sum, 63);
  const int most = min(E, R) + R / T;
  for (int base = 64; base < E && sum < most; base += 64) {
    const Runs r = runs_of(offsets, E, R, T, base);
    sum += __builtin_amdgcn_readlane(r.sum, 63);
  }
  return min(sum, most);
}
// The expert that holds tile `tile`, -1 past the last: its rows [lo, hi), its
// tiles, and the tiles of the experts before it.
__device__ __forceinline__ int find_run(const int32_t* offsets, int E, int R, int T, Runs r, int tile, int& lo, int& hi,
                                        int& tiles, int& before) {
  before = 0;
  for (int base = 0; base < E; base += 64) {
    if (base) r = runs_of(offsets, E, R, T, base);
    const uint64_t past = __ballot(before + r.sum > tile);
    if (past) {
      const int at = __builtin_ctzll(past);
      lo = __builtin_amdgcn_readlane(r.lo, at);
      hi = __builtin_amdgcn_readlane(r.hi, at);
      tiles = __builtin_amdgcn_readlane(r.n, at);
      before += __builtin_amdgcn_readlane(r.sum, at) - tiles;
      return base + at;
    }
    before += __builtin_amdgcn_readlane(r.sum, 63);
  }
  return -1;
}

}  // namespace bsf8
