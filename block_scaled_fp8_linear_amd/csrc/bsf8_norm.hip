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

// T threads per row (64: four rows per block), V vectors of EPL channels each.
template <int T, int V, bool XBF16, bool HBF16>
__global__ __launch_bounds__(T == 64 ? kSmallBlock : T) void quant_norm_kernel(NormDev a) {
  __shared__ double lds[T / 64];
  const int t = threadIdx.x & (T - 1);
  const int64_t m = T == 64 ? a.m0 + int64_t(blockIdx.x) * (kSmallBlock / 64) + (threadIdx.x >> 6) : a.m0 + int64_t(blockIdx.x);
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
    float s;
    uint32_t packed[EPL / 4];
    encode(n, amax, s, packed);
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

// ---------------------------------------------------------------------------
// Rows whose length is a multiple of EPL, up to 16384, and whose addresses all
// allow 16-byte accesses: no tests inside a vector.  One row per block of
// blockDim.x threads with V vectors each; only the last vector can lie past K,
// and it then reads the row's first vector and is zeroed.
//
// What bounds it: some 20 to 45 instructions per channel at about 5 cycles per
// wave and instruction (F64 FMAs and the conversions run at the F32 rate) lie
// close to the time of the memory traffic, so the two must overlap, and waves
// in flight are what overlaps them: the test-free form at 128 registers (four
// waves per SIMD) takes [8192, 7168] BF16 with residual, post norm and gate in
// 111 us and with the residual alone in 82-85 us (410 MB; a copy of as much takes
// 84 us), [8192, 5120] in 76 and 60 us.  Tried and slower: the general kernel
// above for these rows (205 us; two waves per SIMD and a branch around every
// load), blocks that stay and prefetch their next row (175 us; the registers of
// the second row halve the waves), two rows per block sharing the weights'
// conversions (155 us), one vector per thread (132 us; more waves wait at each
// barrier), IEEE divisions in place of encode() and 1 / sqrt() in place of
// rsqrt64().  One row takes 3.5 us.
// ---------------------------------------------------------------------------

// NT: non-temporal, for rows that are read once and then dead (the block's output and the old stream): they leave the
// caches to what the next call reads (rows from memory, [1024, 5120] 16.2 -> 14.2 us, [8192, 7168] 113 -> 111 us).  The
// new stream is stored as usual: the next step reads it.  Experts' rows are loaded as usual too: behind the product that
// wrote them both forms take 18.4 us (1024 tokens, 8 rows of 4096 each), from the cache 17.8 against 19.0 us.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void load_wide(const void* p, int64_t off, Raw<BF16>& r) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const u4* q = reinterpret_cast<const u4*>(static_cast<const uint8_t*>(p) + off * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    const u4 u = NT ? __builtin_nontemporal_load(q + i) : q[i];
    r.w[4 * i] = u[0];
    r.w[4 * i + 1] = u[1];
    r.w[4 * i + 2] = u[2];
    r.w[4 * i + 3] = u[3];
  }
}

template <bool BF16>
__device__ __forceinline__ void clear(Raw<BF16>& r) {
#pragma unroll
  for (int i = 0; i < (BF16 ? EPL / 2 : EPL); ++i) r.w[i] = 0;
}

// s moved by a DPP control word, 0.0 where no lane is the source
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double s) {
  const int2 v = __builtin_bit_cast(int2, s);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, v.x, CTRL, ROWS, 0xf, false),
                                              __builtin_amdgcn_update_dpp(0, v.y, CTRL, ROWS, 0xf, false)));
}

__device__ __forceinline__ double lane_value(double s, int lane) {
  const int2 v = __builtin_bit_cast(int2, s);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(v.x, lane), __builtin_amdgcn_readlane(v.y, lane)));
}

// Sum over the block, in every thread: lanes through DPP (rows of 16, then the
// rows' last lanes onwards; lane 63 ends with the wave's sum), waves through
// LDS in wave order.  Two exchange rows taken in turn: a row is written again
// only after the barrier of the sum between, which every thread reaches after
// it has read the row.
__device__ __forceinline__ double block_sum(double s, double (*lds)[16], int& turn) {
  s += dpp<0x111, 0xf>(s);   // row_shr:1
  s += dpp<0x112, 0xf>(s);   // row_shr:2
  s += dpp<0x114, 0xf>(s);   // row_shr:4
  s += dpp<0x118, 0xf>(s);   // row_shr:8
  s += dpp<0x142, 0xa>(s);   // row_bcast:15 into rows 1 and 3
  s += dpp<0x143, 0xc>(s);   // row_bcast:31 into rows 2 and 3
  s = lane_value(s, 63);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return s;
  turn ^= 1;
  const int lane = threadIdx.x & 63;
  if (lane == 0) lds[turn][threadIdx.x >> 6] = s;
  __syncthreads();
  s = (lane & 15) < waves ? lds[turn][lane & 15] : 0.0;
  s += dpp<0x111, 0xf>(s);
  s += dpp<0x112, 0xf>(s);
  s += dpp<0x114, 0xf>(s);
  s += dpp<0x118, 0xf>(s);
  return lane_value(s, 15);
}

// 1 / sqrt(x) to within an F64 rounding or two: the hardware's estimate and two Newton steps
__device__ __forceinline__ double rsqrt64(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(0.5 * y, fma(-x * y, y, 1.0), y);
  return y;
}

// norm(v) as (v - mean) * rstd, or v * rstd in the RMS norm; `on`: the last
// vector lies in the row.  The difference is taken before the scaling: in v *
// rstd - mean * rstd the rounding of mean * rstd is left where v is near the
// mean, and a row of one value would not be zero.  The mean is the quotient sum /
// K with its remainder put back, so that K equal values have exactly that value
// as their mean.
template <bool LAYER>
__device__ __forceinline__ double centred(double v, double mean) {
  return LAYER ? v - mean : v;
}
template <bool LAYER, int V>
__device__ __forceinline__ void wide_stats(const double (&v)[V][EPL], bool on, const NormDev& a, double inv_k,
                                           double (*lds)[16], int& turn, double& rstd, double& mean) {
  double q = 0.0;
  mean = 0.0;
  if constexpr (LAYER) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) s += v[i][e];
    s = block_sum(s, lds, turn);
    mean = s * inv_k;
    mean = fma(fma(-mean, double(a.K), s), inv_k, mean);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i == V - 1 && !on) continue;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const double d = v[i][e] - mean;
        q = fma(d, d, q);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) q = fma(v[i][e], v[i][e], q);
  }
  rstd = rsqrt64(fma(block_sum(q, lds, turn), inv_k, a.eps));
}

// COMBINE: x holds the experts' rows.  LAYER: the layer norm; a kernel that tests
// for it held 96 to 107 registers, four or five waves per SIMD, where one for the
// RMS norm holds 78 and six waves ([8192, 7168] with post norm and gate 127 us at
// 107 registers against 111).
template <int V, bool COMBINE, bool XBF16, bool HBF16, bool WBF16, bool LAYER>
__global__ __launch_bounds__(V == 1 ? 128 : 1024) void quant_norm_wide_kernel(NormDev a) {
  __shared__ double lds[2][16];
  int turn = 0;
  const int t = threadIdx.x;
  const int K = a.K;
  int k[V];
#pragma unroll
  for (int i = 0; i < V; ++i) k[i] = (t + int(blockDim.x) * i) * EPL;
  const bool on = k[V - 1] < K;
  if (!on) k[V - 1] = 0;
  const double inv_k = 1.0 / double(K);
  const int64_t m = a.m0 + int64_t(blockIdx.x);

  // ---- the block's output; the residual's loads go out with it
  Raw<HBF16> res[V];
  double v[V][EPL];
  if constexpr (!COMBINE) {
    Raw<XBF16> x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) load_wide<XBF16, true>(a.x, m * a.ldx + k[i], x[i]);
    if (a.res != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) load_wide<HBF16, true>(a.res, m * a.ldr + k[i], res[i]);
    }
    if (!on) clear(x[V - 1]);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = double(value<XBF16>(x[i], e));
  } else {
    if (a.res != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) load_wide<HBF16, true>(a.res, m * a.ldr + k[i], res[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = 0.0;
    // four choices at a time: their rows' loads are in flight together
    constexpr int J = 4;
    for (int j0 = 0; j0 < a.top; j0 += J) {
      Raw<XBF16> xj[J][V];
      double p[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int64_t at = m * a.top + min(j0 + j, a.top - 1);
        const int slot = a.slots[at];
        const bool ok = j0 + j < a.top && slot >= 0 && slot < a.R;
        p[j] = ok ? double(a.probs[at]) : 0.0;
        if (ok) {
#pragma unroll
          for (int i = 0; i < V; ++i) load_wide<XBF16>(a.x, int64_t(slot) * a.ldx + k[i], xj[j][i]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) clear(xj[j][i]);
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (i == V - 1 && !on) clear(xj[j][i]);
#pragma unroll
          for (int e = 0; e < EPL; ++e) v[i][e] = fma(p[j], double(value<XBF16>(xj[j][i], e)), v[i][e]);
        }
    }
  }
  Raw<WBF16> w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) load_wide<WBF16>(a.w, k[i], w[i]);
  // lanes past the row: weight zero, so that n is 0 and leaves the group's amax to the others
  if (!on) clear(w[V - 1]);

  // ---- norm of the block's output
  if (a.post_w != nullptr) {
    Raw<WBF16> wp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) load_wide<WBF16>(a.post_w, k[i], wp[i]);
    double rstd, mean;
    wide_stats<LAYER, V>(v, on, a, inv_k, lds, turn, rstd, mean);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = centred<LAYER>(v[i][e], mean) * rstd * double(value<WBF16>(wp[i], e));
    if (a.post_b != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        load_wide<WBF16>(a.post_b, k[i], wp[i]);
#pragma unroll
        for (int e = 0; e < EPL; ++e) v[i][e] += double(value<WBF16>(wp[i], e));
      }
    }
  }
  // ---- gate
  if (a.gate != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Raw<WBF16> g;
      load_wide<WBF16>(a.gate, m * a.ldg + k[i], g);
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] *= double(value<WBF16>(g, e));
    }
  }
  // ---- residual, the stored stream
  if (a.res != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = fma(a.alpha, double(value<HBF16>(res[i], e)), v[i][e]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool past = i == V - 1 && !on;
    float h[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      h[e] = to_f32(v[i][e]);
      if (past) h[e] = 0.f;
    }
    if (HBF16) {
      const uint32_t p[4] = {bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3]), bf16_pair(h[4], h[5]), bf16_pair(h[6], h[7])};
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        v[i][e] = double(__uint_as_float((e & 1) ? p[e >> 1] & 0xFFFF0000u : p[e >> 1] << 16));
      if (a.h != nullptr && !past)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + m * a.ldh + k[i]) = make_uint4(p[0], p[1], p[2], p[3]);
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[i][e] = double(h[e]);
      if (a.h != nullptr && !past) store_row(a.h, false, m * a.ldh + k[i], EPL, true, h);
    }
  }

  // ---- the next block's norm, and its codes
  double rstd, mean;
  wide_stats<LAYER, V>(v, on, a, inv_k, lds, turn, rstd, mean);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool past = i == V - 1 && !on;
    float n[EPL];
    if (a.b != nullptr) {
      Raw<WBF16> b;
      load_wide<WBF16>(a.b, k[i], b);
      if (past) clear(b);
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        n[e] = to_f32(fma(centred<LAYER>(v[i][e], mean) * rstd, double(value<WBF16>(w[i], e)), double(value<WBF16>(b, e))));
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e) n[e] = to_f32(centred<LAYER>(v[i][e], mean) * rstd * double(value<WBF16>(w[i], e)));
    }
    if (a.n != nullptr && !past) store_row(a.n, a.n_bf16, m * a.ldn + k[i], EPL, true, n);
    if (a.xq == nullptr) continue;
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) amax = fmaxf(amax, fabsf(n[e]));
#pragma unroll
    for (int d = LPG / 2; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d, LPG));
    float s;
    uint32_t q[EPL / 4];
    encode(n, amax, s, q);
    if (!past) {
      *reinterpret_cast<uint2*>(a.xq + m * a.ldq + k[i]) = make_uint2(q[0], q[1]);
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

template <int V, bool COMBINE, bool LAYER>
Kern pick_wide(bool x_bf16, bool h_bf16, bool w_bf16) {
#define BSF8_WIDE(X, H) \
  (w_bf16 ? quant_norm_wide_kernel<V, COMBINE, X, H, true, LAYER> : quant_norm_wide_kernel<V, COMBINE, X, H, false, LAYER>)
  return x_bf16 ? (h_bf16 ? BSF8_WIDE(true, true) : BSF8_WIDE(true, false))
                : (h_bf16 ? BSF8_WIDE(false, true) : BSF8_WIDE(false, false));
#undef BSF8_WIDE
}
template <int V>
Kern pick_wide(const NormDev& a, bool x_bf16, bool h_bf16) {
  if (a.slots) return a.layer ? pick_wide<V, true, true>(x_bf16, h_bf16, a.w_bf16) : pick_wide<V, true, false>(x_bf16, h_bf16, a.w_bf16);
  return a.layer ? pick_wide<V, false, true>(x_bf16, h_bf16, a.w_bf16) : pick_wide<V, false, false>(x_bf16, h_bf16, a.w_bf16);
}

}  // namespace

bsf8_status launch_quant_norm(const NormDev& args, bool x_bf16, bool h_bf16, hipStream_t stream) {
  NormDev a = args;
  const int vecs = (a.K + EPL - 1) / EPL;
  Kern kern;
  int threads, rows;
  if (a.wide && vecs <= 2048) {
    // a block's first vector must lie in the row, so fewer than 128 vectors take one each
    rows = 1;
    threads = vecs < 128 ? (vecs + 63) / 64 * 64 : ((vecs + 1) / 2 + 63) / 64 * 64;
    kern = vecs < 128 ? pick_wide<1>(a, x_bf16, h_bf16) : pick_wide<2>(a, x_bf16, h_bf16);
  } else if (vecs <= 64) {
    threads = kSmallBlock;
    rows = kSmallBlock / 64;
    kern = pick<64, 1>(x_bf16, h_bf16);
  } else {
    threads = vecs <= 1024 ? 256 : 1024;
    rows = 1;
    kern = vecs <= 1024 ? pick<256, 4>(x_bf16, h_bf16) : pick<1024, 4>(x_bf16, h_bf16);
  }
  // a launch holds fewer than 2^32 threads, so rows go out by 2^22 blocks (four rows each in the short rows' kernel)
  bsf8_status st = BSF8_OK;
  for (int64_t step = (int64_t(1) << 22) * rows - rows; a.m0 < a.M && st == BSF8_OK; a.m0 += step) {
    const int64_t here = a.M - a.m0 < step ? a.M - a.m0 : step;
    hipLaunchKernelGGL(kern, dim3(unsigned((here + rows - 1) / rows)), dim3(threads), 0, stream, a);
    st = device_status(hipGetLastError(), "quant_norm launch");
  }
  return st;
}

}  // namespace bsf8
