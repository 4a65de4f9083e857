// The step between two blocks of a residual stream (gfx950): the block's output
// (or the router-weighted sum of its experts' rows), an optional norm of it,
// a gate, the scaled residual add, the norm before the next block, and the
// E4M3 quantization that the next W8A8 product reads, in one pass.
//
//   o  = x[m]                          or  sum_j p[m, j] * x[slot[m, j]]
//   o' = o                             or  norm(o) * wp + bp
//   h  = a * res[m] + g * o'           rounded to F32 and then to h's type
//   n  = norm(h) * w + b               rounded to F32; codes and scales from it
//
// norm is the RMS norm v / sqrt(mean(v^2) + eps) or the layer norm
// (v - mean) / sqrt(var + eps), the variance taken about the mean in a second
// sweep of the registers.  Everything between the inputs and the two stated
// roundings is F64, in the registers of the block that owns the row.  A code
// lies next to a border: with F32 statistics (relative error some 2^-23) about
// one value in a million changes its code with the order of a sum, by a whole
// E4M3 step; with F64 the chance is 2^-29 of that, so codes are reproducible
// from the formula, as the quantizer's are.  gfx950 runs F64 FMAs at the rate
// of F32 ones.  The next norm reads h as it is stored, so the fused call gives
// what its parts in separate calls give.
//
// One block (or one wave, for short rows) per row; a row stays in registers
// from its only read to its last write: 8 consecutive channels per lane and
// vector, so a 128-channel scale group is 16 lanes, and every access is 16
// bytes wide where addresses allow it.  Sums go through a wave butterfly and
// one LDS exchange per statistic, in a fixed order.
#include <hip/hip_runtime.h>

#include "bsf8_internal.h"

namespace bsf8 {
namespace {

constexpr int EPL = 8;                   // channels per lane and vector
constexpr int LPG = kBlock / EPL;        // lanes per 128-channel scale group
constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 1e-10f;
constexpr int kSmallBlock = 256;         // threads per block where a row takes one wave

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

// Sum over the threads of a row, the same value in each: a butterfly within the
// wave, then the waves' sums in wave order.
template <int T>
__device__ __forceinline__ double row_sum(double s, double* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
  if (T == 64) return s;
  __syncthreads();   // the exchange before this one has been read
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) t += lds[w];
  return t;
}

// mean (0 for the RMS norm) and 1 / sqrt(mean square about it + eps) of a row
template <int T, int V>
__device__ __forceinline__ void row_stats(const double (&v)[V][EPL], const int (&valid)[V], bool layer, int K,
                                          double eps, double* lds, double& mean, double& rstd) {
  mean = 0.0;
  if (layer) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) s += v[i][e];   // zeros past K
    mean = row_sum<T>(s, lds) / double(K);
  }
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const double d = e < valid[i] ? v[i][e] - mean : 0.0;
      q = fma(d, d, q);
    }
  rstd = 1.0 / sqrt(row_sum<T>(q, lds) / double(K) + eps);
}

// T threads per row (64: four rows per block), V vectors of EPL channels each.
template <int T, int V, bool XBF16, bool HBF16>
__global__ __launch_bounds__(T == 64 ? kSmallBlock : T) void quant_norm_kernel(NormDev a) {
  __shared__ double lds[T / 64];
  const int t = threadIdx.x & (T - 1);
  const int64_t m = T == 64 ? int64_t(blockIdx.x) * (kSmallBlock / 64) + (threadIdx.x >> 6) : int64_t(blockIdx.x);
  if (T == 64 && m >= a.M) return;   // whole waves; a wave-wide row meets no barrier
  const int K = a.K;
  int k[V], valid[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    k[i] = (t + T * i) * EPL;
    valid[i] = max(0, min(EPL, K - k[i]));
  }

  // ---- the residual's loads go out first; they are used last
  Raw<HBF16> res[V];
  if (a.res != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) load_raw<HBF16>(a.res, m * a.ldr + k[i], valid[i], a.res_vec, res[i]);
  }

  // ---- the block's output
  double v[V][EPL];
  if (a.slots == nullptr) {
    Raw<XBF16> x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) load_raw<XBF16>(a.x, m * a.ldx + k[i], valid[i], a.x_vec, x[i]);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = double(value<XBF16>(x[i], e));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = 0.0;
    for (int j = 0; j < a.top; ++j) {
      const int slot = a.slots[m * a.top + j];
      if (slot < 0 || slot >= a.R) continue;   // the same for the whole row
      const double p = double(a.probs[m * a.top + j]);
      Raw<XBF16> x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) load_raw<XBF16>(a.x, int64_t(slot) * a.ldx + k[i], valid[i], a.x_vec, x[i]);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < EPL; ++e) v[i][e] = fma(p, double(value<XBF16>(x[i], e)), v[i][e]);
    }
  }

  // ---- its norm
  if (a.post_w != nullptr) {
    double mean, rstd;
    row_stats<T, V>(v, valid, a.layer, K, a.eps, lds, mean, rstd);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float w[EPL], b[EPL] = {};
      load_vec(a.post_w, a.post_bf16, k[i], valid[i], a.post_vec, w);
      if (a.post_b != nullptr) load_vec(a.post_b, a.post_bf16, k[i], valid[i], a.post_vec, b);
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = fma((v[i][e] - mean) * rstd, double(w[e]), double(b[e]));
    }
  }

  // ---- gate, residual, the stored stream
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.gate != nullptr) {
      float g[EPL];
      load_vec(a.gate, a.gate_bf16, m * a.ldg + k[i], valid[i], a.gate_vec, g);
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] *= double(g[e]);
    }
    if (a.res != nullptr) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = fma(a.alpha, double(value<HBF16>(res[i], e)), v[i][e]);
    }
    float h[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      h[e] = to_f32(v[i][e]);
      if (HBF16) h[e] = float(static_cast<__bf16>(h[e]));
      v[i][e] = e < valid[i] ? double(h[e]) : 0.0;
    }
    if (a.h != nullptr) store_row(a.h, HBF16, m * a.ldh + k[i], valid[i], a.h_vec, h);
  }

  // ---- the next block's norm, and its codes
  double mean, rstd;
  row_stats<T, V>(v, valid, a.layer, K, a.eps, lds, mean, rstd);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float w[EPL], b[EPL] = {}, n[EPL];
    load_vec(a.w, a.w_bf16, k[i], valid[i], a.w_vec, w);
    if (a.b != nullptr) load_vec(a.b, a.w_bf16, k[i], valid[i], a.w_vec, b);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      n[e] = to_f32(fma((v[i][e] - mean) * rstd, double(w[e]), double(b[e])));
      if (e < valid[i]) amax = fmaxf(amax, fabsf(n[e]));
    }
    if (a.n != nullptr) store_row(a.n, a.n_bf16, m * a.ldn + k[i], valid[i], a.n_vec, n);
    if (a.xq == nullptr) continue;
#pragma unroll
    for (int d = LPG / 2; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d, LPG));
    // as the activation quantizer: the F64 product with fl64(1 / s) rounds to
    // the IEEE F32 quotient n / s
    const float s = fmaxf(amax, kAmaxFloor) / kE4M3Max;
    const double rs = 1.0 / static_cast<double>(s);
    uint32_t packed[EPL / 4];
#pragma unroll
    for (int q = 0; q < EPL / 4; ++q) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f[e] = fminf(fmaxf(static_cast<float>(static_cast<double>(n[4 * q + e]) * rs), -kE4M3Max), kE4M3Max);
      int pk = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
      pk = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], pk, true);
      packed[q] = uint32_t(pk);
    }
    if (valid[i] > 0) {
      uint8_t* q = a.xq + m * a.ldq + k[i];
      if (valid[i] == EPL && a.q_vec) {
        *reinterpret_cast<uint2*>(q) = make_uint2(packed[0], packed[1]);
      } else {
#pragma unroll
        for (int e = 0; e < EPL; ++e)
          if (e < valid[i]) q[e] = uint8_t(packed[e >> 2] >> (8 * (e & 3)));
      }
      if ((t & (LPG - 1)) == 0) a.xs[m * a.xs_sm + int64_t(k[i] / kBlock) * a.xs_sk] = s;
    }
  }
}

using Kern = void (*)(NormDev);

template <int T, int V>
Kern pick(bool x_bf16, bool h_bf16) {
  return x_bf16 ? (h_bf16 ? quant_norm_kernel<T, V, true, true> : quant_norm_kernel<T, V, true, false>)
                : (h_bf16 ? quant_norm_kernel<T, V, false, true> : quant_norm_kernel<T, V, false, false>);
}

}  // namespace

bsf8_status launch_quant_norm(const NormDev& a, bool x_bf16, bool h_bf16, hipStream_t stream) {
  const int vecs = (a.K + EPL - 1) / EPL;
  Kern kern;
  int T;
  if (vecs <= 64) {
    T = 64;
    kern = pick<64, 1>(x_bf16, h_bf16);
  } else if (vecs <= 1024) {
    T = 256;
    kern = vecs <= 256 ? pick<256, 1>(x_bf16, h_bf16)
           : vecs <= 512 ? pick<256, 2>(x_bf16, h_bf16)
           : vecs <= 768 ? pick<256, 3>(x_bf16, h_bf16)
                         : pick<256, 4>(x_bf16, h_bf16);
  } else {
    T = 1024;
    kern = vecs <= 2048 ? pick<1024, 2>(x_bf16, h_bf16) : pick<1024, 4>(x_bf16, h_bf16);
  }
  const int rows = T == 64 ? kSmallBlock / 64 : 1;
  hipLaunchKernelGGL(kern, dim3(unsigned((a.M + rows - 1) / rows)), dim3(T == 64 ? kSmallBlock : T), 0, stream, a);
  return device_status(hipGetLastError(), "quant_norm launch");
}

}  // namespace bsf8
