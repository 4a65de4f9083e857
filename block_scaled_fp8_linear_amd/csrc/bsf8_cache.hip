// Rotary positions, and a paged cache of keys and values written and read back (gfx950).
//
// heads_kernel: rows of head_dim channels (queries, keys, values of a token's heads) with
// the head norm, the rotation and, for the cache, the E4M3 quantization.
//   x' = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// Everything is F64 up to one rounding to F32, as in the norm step: a code next to a border
// changes by a whole step with the last bit of an F32 sum, and F64 FMAs run at the F32 rate
// here.  Memory bounds rows that only turn (4096 tokens of 48 heads of 128 F32 channels to BF16,
// 151 MB: 30.5 us, 4.9 TB/s; 8192 of BF16, 201 MB: 41); where codes are made the vector
// instructions take about as long as the bytes (8192 tokens' keys, turned, and values, 8 heads of
// 128 each, 51 MB: 17.5 us, into BF16 rows, 67 MB, 14.6).  So a pass over values alone skips the
// arithmetic, a lane past its row is left out only where it would count, and the largest of a
// group is found by lane exchanges in the adder's path, not by LDS (20.5 -> 17.5 us together).
// The head norm is bound by vector instructions and by its registers, 138 to 146 of a lane where the turn
// alone takes 73 to 84 (three waves per SIMD for five or six): weights become F64 and multiply both channels
// of a pair row by row, and the squares' sum is a chain of F64 exchanges through LDS.  1024 tokens of 48 heads
// of 128 BF16 channels 15.3 us with it, 11.7 without, 4.8 in a copy; 4096 39 and 22 of 19; 2048 tokens of
// 24 + 4 + 4 heads of 256 into codes 27 and 18 of 12.
//
// A row is LPR = 8, 16 or 32 lanes of 8 channels (head_dim up to 64, 128, 256), so that a
// 128-channel scale group is 16 lanes, and a wave holds 64 / LPR rows, all of one token:
// a lane has the same channels in every row it takes, so its angles' sines and cosines are
// there once for all the heads of the wave.  The pair's other channel is loaded a second time
// rather than exchanged between lanes: it is in the cache line that the row's own lanes ask
// for.  An output may be its input: a row's stores need values of all the loads of its wave.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "bsf8_channels.h"
#include "bsf8_fused.h"

namespace bsf8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

enum Pairs { kNone, kHalf, kHalfOdd, kAdjacent };   // kHalfOdd: R / 2 is no multiple of a lane's channels

// sine and cosine of an angle below 2^31: r = t - n pi / 2 by two FMAs with pi / 2 in two
// parts (W. J. Cody and W. Waite, "Software Manual for the Elementary Functions", 1980),
// |r| <= pi / 4, and the Taylor sums of both up to a remainder below 2^-57.
__device__ __forceinline__ void sine_cosine(double t, double& s, double& c) {
  const double n = rint(t * 0.63661977236758138);
  double r = fma(-n, 1.5707963267948966, t);
  r = fma(-n, 6.123233995736766e-17, r);
  const double z = r * r;
  double p = 1.0 / 355687428096000.0;
  p = fma(p, z, -1.0 / 1307674368000.0);
  p = fma(p, z, 1.0 / 6227020800.0);
  p = fma(p, z, -1.0 / 39916800.0);
  p = fma(p, z, 1.0 / 362880.0);
  p = fma(p, z, -1.0 / 5040.0);
  p = fma(p, z, 1.0 / 120.0);
  p = fma(p, z, -1.0 / 6.0);
  const double sr = fma(r * z, p, r);
  double q = 1.0 / 20922789888000.0;
  q = fma(q, z, -1.0 / 87178291200.0);
  q = fma(q, z, 1.0 / 479001600.0);
  q = fma(q, z, -1.0 / 3628800.0);
  q = fma(q, z, 1.0 / 40320.0);
  q = fma(q, z, -1.0 / 720.0);
  q = fma(q, z, 1.0 / 24.0);
  const double cr = fma(z * z, q, fma(z, -0.5, 1.0));
  const int k = static_cast<int>(n);
  s = (k & 1) ? cr : sr;
  c = (k & 1) ? sr : cr;
  if (k & 2) s = -s;
  if ((k + 1) & 2) c = -c;
}

__device__ __forceinline__ double position(const HeadsJob& a, int axis, int64_t m) {
  const int64_t at = axis * a.ld_axis + m;
  return a.pos64 ? double(static_cast<const int64_t*>(a.pos)[at]) : double(static_cast<const int32_t*>(a.pos)[at]);
}

// the angle of pair i of token m; p0: the token's position on axis 0
__device__ __forceinline__ double angle(const HeadsJob& a, int i, int64_t m, double p0) {
  double p = p0;
  if (a.n_axes > 1) p = position(a, (a.axis[i >> 3] >> (4 * (i & 7))) & 15, m);
  return p * double(a.inv_freq[i]);
}

// The turn of a lane's channels c0 .. c0 + 7 for token m: y[e] = cs[e] x[e] + sn[e] partner[e];
// the sign of the sine is the channel's.  A wave's lanes make the token's R / 2 cosines and
// sines between them, one or two each, and take theirs from `lds` (the wave's own), where each
// lane made its own eight before: 8 times the work for 128 channels, a third of the time of
// 8192 tokens' keys into the cache.
struct Turn {
  double c, s;
};
constexpr int kMostPairs = BSF8_CACHE_MAX_HEAD_DIM / 2;
template <int PAIRS>
__device__ __forceinline__ void turn_factors(const HeadsJob& a, int c0, int64_t m, Turn* lds, double (&cs)[EPL], double (&sn)[EPL]) {
  const int R = a.R, half = R >> 1;
  if (PAIRS != kHalf) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      cs[e] = 1.0;
      sn[e] = 0.0;
    }
  }
  if (PAIRS == kNone) return;
  const double p0 = a.n_axes == 1 ? position(a, 0, m) : 0.0;
  for (int i = threadIdx.x & 63; i < half; i += 64) {
    Turn t;
    sine_cosine(angle(a, i, m, p0), t.s, t.c);
    t.s *= a.scale;
    t.c *= a.scale;
    lds[i] = t;
  }
  // the wave's stores are before its loads: LDS takes a wave's instructions in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  if (PAIRS == kHalf) {
    // a lane's channels are all of one half; those that do not turn take the first ones and leave them unused
    const uint64_t sign = c0 >= half ? 0 : uint64_t(1) << 63;
    const int i0 = c0 >= R ? 0 : c0 >= half ? c0 - half : c0;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const Turn t = lds[i0 + e];
      cs[e] = t.c;
      sn[e] = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, t.s) ^ sign);
    }
    return;
  }
  if (c0 >= R) return;
  if (PAIRS == kAdjacent) {
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
      if (c0 + e >= R) continue;
      const Turn t = lds[(c0 + e) >> 1];
      cs[e] = cs[e + 1] = t.c;
      sn[e + 1] = t.s;
      sn[e] = -t.s;
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const int ch = c0 + e;
      if (ch >= R) continue;
      const bool second = ch >= half;
      const Turn t = lds[second ? ch - half : ch];
      cs[e] = t.c;
      sn[e] = second ? t.s : -t.s;
    }
  }
}

// Eight channels at an address that a lane has picked among several: named as global memory,
// since the compiler takes a pointer that it cannot trace for one that may be LDS (flat accesses
// took 1.7 times as long).
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) u4v* GlobalVec;
template <bool BF16>
__device__ __forceinline__ void load_global(uint64_t at, Raw<BF16>& r) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    const u4v u = reinterpret_cast<GlobalVec>(at)[i];
#pragma unroll
    for (int y = 0; y < 4; ++y) r.w[4 * i + y] = u[y];
  }
}
__device__ __forceinline__ void store_global(uint64_t row, bool bf16, int c0, const float (&f)[EPL]) {
  GlobalVec p = reinterpret_cast<GlobalVec>(row + uint64_t(c0 * (bf16 ? 2 : 4)));
  if (bf16) {
    p[0] = u4v{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
  } else {
    p[0] = u4v{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    p[1] = u4v{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
  }
}

// A row of keys or values into the cache; the lanes of a row call it together.
struct CacheRow {   // of a token: addresses of its keys, values and their scales
  uint64_t k, v, ks, vs;
};
__device__ __forceinline__ CacheRow cache_row(const CacheDev& c, int64_t slot) {
  if (slot < 0) return CacheRow{0, 0, 0, 0};
  const uint32_t page = c.page_of(uint32_t(slot)), row = uint32_t(slot) - page * uint32_t(c.page_size);
  const uint64_t at = uint64_t(int64_t(page) * c.page + int64_t(row) * c.row), s = uint64_t(int64_t(page) * c.s_page + int64_t(row) * c.s_row) * 4;
  return CacheRow{uint64_t(c.k) + at, uint64_t(c.v) + at, uint64_t(c.k_scale) + s, uint64_t(c.v_scale) + s};
}
// the largest of 8 or 16 neighbouring lanes: exchanged in pairs, in fours, and mirrored in eights and sixteens
template <int LANES>
__device__ __forceinline__ float max_of_group(float x) {
  const auto with = [](float v, auto control) {
    return fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), decltype(control)::value, 0xF, 0xF, true)));
  };
  x = with(x, std::integral_constant<int, 0xB1>{});
  x = with(x, std::integral_constant<int, 0x4E>{});
  x = with(x, std::integral_constant<int, 0x141>{});
  if (LANES == 16) x = with(x, std::integral_constant<int, 0x140>{});
  return x;
}
template <int LPR>
__device__ __forceinline__ void store_cached(const CacheDev& c, const CacheRow& to, bool is_v, int h, int c0, bool on,
                                             const float (&f)[EPL]) {
  uint64_t out = to.k, scale = to.ks;
  if (is_v) out = to.v, scale = to.vs;
  out += uint64_t(int64_t(h) * c.head);
  if (!c.e4m3) {
    if (on) store_global(out, true, c0, f);
    return;
  }
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < EPL; ++e) amax = fmaxf(amax, fabsf(f[e]));
  amax = max_of_group<LPR < LPG ? LPR : LPG>(on ? amax : 0.f);
  float s;
  uint32_t packed[EPL / 4];
  encode(f, amax, s, packed);
  if (!on) return;
  typedef uint32_t u2v __attribute__((ext_vector_type(2)));
  *reinterpret_cast<__attribute__((address_space(1))) u2v*>(out + uint64_t(c0)) = u2v{packed[0], packed[1]};
  if (c0 % kBlock == 0)
    reinterpret_cast<__attribute__((address_space(1))) float*>(scale)[int64_t(h) * c.s_head + int64_t(c0 / kBlock) * c.s_group] = s;
}

// the slot of token m, -1 where it has none
__device__ __forceinline__ int64_t slot_of(const HeadsJob& a, int64_t m) {
  if (!a.to_cache) return -1;
  const int64_t s = a.slot64 ? static_cast<const int64_t*>(a.slots)[m] : int64_t(static_cast<const int32_t*>(a.slots)[m]);
  return s < a.cache.rows ? max(s, int64_t(-1)) : -1;
}

template <int LPR, int PAIRS>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsJob a) {
  __shared__ Turn turn[kWaves][PAIRS == kNone ? 1 : kMostPairs];
  constexpr int RPP = 64 / LPR;                     // rows of a wave
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * kWaves + uint32_t(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const uint32_t tok = wave / uint32_t(a.parts), part = wave - tok * uint32_t(a.parts);
  if (tok >= uint32_t(a.M)) return;                 // whole waves; nothing here waits for another
  const int64_t m = a.m0 + tok;
  const int D = a.D, R = a.R, half = R >> 1;
  const int c0 = (lane & (LPR - 1)) * EPL;
  const int on = c0 < D ? EPL : 0;                  // D is a multiple of a lane's channels
  const bool turns = PAIRS != kNone && c0 < R;

  double cs[EPL], sn[EPL];
  turn_factors<PAIRS>(a, c0, m, turn[threadIdx.x >> 6], cs, sn);

  const int64_t slot = slot_of(a, m);
  const CacheRow to = cache_row(a.cache, slot);

  const int heads = a.q.heads + a.k.heads + a.v.heads;
  const int first = int(part) * a.per_part, last = min(heads, first + a.per_part);
  for (int at = first + lane / LPR; at < last; at += RPP) {
    const bool is_q = at < a.q.heads, is_v = at >= a.q.heads + a.k.heads;
    const HeadsDev& src = is_q ? a.q : is_v ? a.v : a.k;
    const int h = at - (is_q ? 0 : is_v ? a.q.heads + a.k.heads : a.q.heads);
    const bool skip = a.to_cache && !is_q && slot < 0;
    const int64_t base = m * src.token + int64_t(h) * src.head;
    float x[EPL];
    load_vec(src.p, src.bf16, base + c0, skip ? 0 : on, src.vec, x);
    float f[EPL];
    if (is_v) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) f[e] = x[e];
    } else {
      const void* w = is_q ? a.qw : a.kw;
      float xp[EPL] = {}, wp[EPL] = {};
      int pc = 0;
      if (PAIRS == kHalf) {
        pc = c0 < half ? c0 + half : c0 - half;
        load_vec(src.p, src.bf16, base + pc, turns && !skip ? EPL : 0, src.vec, xp);
      } else if (PAIRS == kHalfOdd) {
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
          const int ch = c0 + e;
          if (ch < R && !skip) xp[e] = load_real(src.p, src.bf16, base + (ch < half ? ch + half : ch - half));
        }
      } else if (PAIRS == kAdjacent) {
#pragma unroll
        for (int e = 0; e < EPL; ++e) xp[e] = x[e ^ 1];
      }
      double v[EPL], vp[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        v[e] = double(x[e]);
        vp[e] = double(xp[e]);
      }
      if (w != nullptr) {
        float wv[EPL];
        load_vec(w, a.w_bf16, c0, on, a.w_vec, wv);
        if (PAIRS == kHalf) {
          load_vec(w, a.w_bf16, pc, turns ? EPL : 0, a.w_vec, wp);
        } else if (PAIRS == kHalfOdd) {
#pragma unroll
          for (int e = 0; e < EPL; ++e) {
            const int ch = c0 + e;
            if (ch < R) wp[e] = load_real(w, a.w_bf16, ch < half ? ch + half : ch - half);
          }
        } else if (PAIRS == kAdjacent) {
#pragma unroll
          for (int e = 0; e < EPL; ++e) wp[e] = wv[e ^ 1];
        }
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < EPL; ++e) sum = fma(v[e], v[e], sum);   // zeros past D
#pragma unroll
        for (int d = LPR / 2; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
        const double rstd = 1.0 / sqrt(sum / double(D) + a.eps);
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
          v[e] = v[e] * rstd * double(wv[e]);
          vp[e] = vp[e] * rstd * double(wp[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        double y = v[e];
        // (beside the sum: a channel that does not turn keeps its zero's sign)
        if (PAIRS != kNone && (PAIRS == kHalf ? turns : c0 + e < R)) y = fma(cs[e], v[e], sn[e] * vp[e]);
        f[e] = to_f32(y);
      }
    }
    if (is_q || !a.to_cache) {
      const HeadsDev& dst = is_q ? a.q_out : a.k_out;
      store_row(const_cast<void*>(dst.p), dst.bf16, m * dst.token + int64_t(h) * dst.head + c0, on, dst.vec, f);
      continue;
    }
    if (!skip) store_cached<LPR>(a.cache, to, is_v, h, c0, on != 0, f);
  }
}

// The rows of a token in one numbering: queries, keys, values.
struct Kinds {
  int keys, values;   // the first key's and the first value's number
  __device__ __forceinline__ bool is_q(int at) const { return at < keys; }
  __device__ __forceinline__ bool is_v(int at) const { return at >= values; }
  __device__ __forceinline__ int head(int at) const { return at - (at < keys ? 0 : at < values ? keys : values); }
};
// The one of three values that a row's kind asks for.  By value, and not as a choice between
// variables: of those the compiler makes a choice between their addresses, and puts them in memory.
__device__ __forceinline__ uint64_t pick(Kinds kinds, int at, uint64_t q, uint64_t k, uint64_t v) {
  return at < kinds.keys ? q : at < kinds.values ? k : v;
}

// The same for inputs of one type whose rows, and the outputs', allow 16-byte accesses, and
// pairs whose halves begin at a lane's first channel: the next rows are asked for before the
// ones at hand are turned, and nothing branches around a load.
template <int LPR, int PAIRS, bool XBF16, bool NORM>
__global__ __launch_bounds__(kThreads) void heads_wide_kernel(HeadsJob a) {
  __shared__ Turn turn[kWaves][PAIRS == kNone ? 1 : kMostPairs];
  constexpr int RPP = 64 / LPR;
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * kWaves + uint32_t(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const uint32_t tok = wave / uint32_t(a.parts), part = wave - tok * uint32_t(a.parts);
  if (tok >= uint32_t(a.M)) return;
  const int64_t m = a.m0 + tok;
  const int D = a.D, R = a.R, half = R >> 1;
  const int c0 = (lane & (LPR - 1)) * EPL, at0 = c0 < D ? c0 : 0;   // (lanes past the row read its first channels)
  const bool on = c0 < D, turns = PAIRS != kNone && c0 < R;
  const int pc = PAIRS == kHalf && turns ? (c0 < half ? c0 + half : c0 - half) : at0;

  const int q_heads = a.q.heads, k_heads = a.k.heads, heads = q_heads + k_heads + a.v.heads;
  const int first = int(part) * a.per_part, last = min(heads, first + a.per_part);
  // a lane's rows are of three kinds: it picks the token's address and the heads' distance
  constexpr int XB = XBF16 ? 2 : 4;
  const auto token_of = [&](const HeadsDev& h, int64_t bytes) { return uint64_t(h.p) + uint64_t(m * h.token * bytes); };
  const uint64_t q_at = token_of(a.q, XB), k_at = token_of(a.k, XB), v_at = token_of(a.v, XB);
  const int64_t q_step = a.q.head * XB, k_step = a.k.head * XB, v_step = a.v.head * XB;
  const Kinds kinds{q_heads, q_heads + k_heads};
  Raw<XBF16> next_x, next_p;
  const auto fetch = [=](int at, Raw<XBF16>& x, Raw<XBF16>& p) __attribute__((always_inline)) {
    at = min(at, last - 1);
    const uint64_t row = pick(kinds, at, q_at, k_at, v_at) + uint64_t(int64_t(kinds.head(at)) * int64_t(pick(kinds, at, uint64_t(q_step), uint64_t(k_step), uint64_t(v_step))));
    load_global(row + uint64_t(at0 * XB), x);
    if (PAIRS == kHalf) load_global(row + uint64_t(pc * XB), p);
  };
  fetch(first + lane / LPR, next_x, next_p);
  float wq[EPL], wk[EPL], wqp[EPL], wkp[EPL];
  if (NORM) {
    const void* any = a.qw ? a.qw : a.kw;
    load_vec(a.qw ? a.qw : any, a.w_bf16, at0, EPL, a.w_vec, wq);
    load_vec(a.kw ? a.kw : any, a.w_bf16, at0, EPL, a.w_vec, wk);
    if (PAIRS == kHalf) {
      load_vec(a.qw ? a.qw : any, a.w_bf16, pc, EPL, a.w_vec, wqp);
      load_vec(a.kw ? a.kw : any, a.w_bf16, pc, EPL, a.w_vec, wkp);
    }
  }
  const int64_t slot = slot_of(a, m);
  const CacheRow to = cache_row(a.cache, slot);
  const uint64_t qo_at = token_of(a.q_out, a.q_out.bf16 ? 2 : 4), ko_at = token_of(a.k_out, a.k_out.bf16 ? 2 : 4);
  const int64_t qo_step = a.q_out.head * (a.q_out.bf16 ? 2 : 4), ko_step = a.k_out.head * (a.k_out.bf16 ? 2 : 4);
  const uint64_t qo_bf16 = a.q_out.bf16, ko_bf16 = a.k_out.bf16;
  double cs[EPL], sn[EPL];
  turn_factors<PAIRS>(a, c0, m, turn[threadIdx.x >> 6], cs, sn);

  for (int pass = first; pass < last; pass += RPP) {
    const int at = pass + lane / LPR;
    if (at >= last) break;
    const Raw<XBF16> x = next_x, p = next_p;
    fetch(at + RPP, next_x, next_p);
    const bool is_q = kinds.is_q(at), is_v = kinds.is_v(at);
    const int h = kinds.head(at);
    float f[EPL];   // (of lanes past the row: its first channels, left unused)
#pragma unroll
    for (int e = 0; e < EPL; ++e) f[e] = value<XBF16>(x, e);
    if ((PAIRS != kNone || NORM) && pass < kinds.values) {   // not values alone: one choice for the wave
      double v[EPL], vp[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        v[e] = double(f[e]);
        vp[e] = PAIRS == kHalf ? double(value<XBF16>(p, e)) : 0.0;
      }
      if (NORM && (is_q ? a.qw : a.kw) != nullptr) {
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < EPL; ++e) sum = fma(v[e], v[e], sum);
        sum = on ? sum : 0.0;
#pragma unroll
        for (int d = LPR / 2; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
        const double rstd = rsqrt64(fma(sum, 1.0 / double(D), a.eps));
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
          v[e] = v[e] * rstd * double(is_q ? wq[e] : wk[e]);
          if (PAIRS == kHalf) vp[e] = vp[e] * rstd * double(is_q ? wqp[e] : wkp[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        // (chosen beside the sum: a channel that does not turn keeps its zero's sign)
        const bool turned = PAIRS == kHalf ? turns : PAIRS == kAdjacent && c0 + e < R;
        const double y = fma(cs[e], v[e], sn[e] * (PAIRS == kHalf ? vp[e] : v[e ^ 1]));
        if (NORM) f[e] = is_v ? f[e] : to_f32(turned ? y : v[e]);
        else f[e] = is_v || !turned ? f[e] : to_f32(y);
      }
    }
    if (is_q || !a.to_cache) {
      const uint64_t to_row = pick(kinds, at, qo_at, ko_at, ko_at) +
                              uint64_t(int64_t(h) * int64_t(pick(kinds, at, uint64_t(qo_step), uint64_t(ko_step), uint64_t(ko_step))));
      if (on) store_global(to_row, pick(kinds, at, qo_bf16, ko_bf16, ko_bf16) != 0, c0, f);
    } else if (slot >= 0) {
      store_cached<LPR>(a.cache, to, is_v, h, c0, on, f);
    }
  }
}

// Rows of the cache back: a wave takes per_wave rows that follow each other, 64 / LPR heads
// at a time, keys and values together.
// Bound by memory: 13000 rows of 8 heads of 128 E4M3 channels as BF16, 81 MB, 18 us, 4.4 TB/s;
// 9000 of 5 heads of 96 BF16 channels as F32, 52 MB, 14 us, 3.6 TB/s.
struct ReadJob {
  CacheDev cache;
  HeadsDev k, v;              // outputs
  const int32_t* table;
  const int32_t* starts;
  const int32_t* offsets;
  int64_t ld_table, r0;
  int32_t B, pages, R, per_wave;
};

__device__ __forceinline__ void read_codes(const CacheDev& c, const uint8_t* p, float scale, bool there, float (&f)[EPL]) {
#pragma unroll
  for (int e = 0; e < EPL; ++e) f[e] = 0.f;
  if (!there) return;
  if (!c.e4m3) {
    Raw<true> r;
    load_raw<true>(p, 0, EPL, true, r);
#pragma unroll
    for (int e = 0; e < EPL; ++e) f[e] = value<true>(r, e);
    return;
  }
  typedef float f2 __attribute__((ext_vector_type(2)));
  const uint2 u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int w = int(q ? u.y : u.x);
    const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[4 * q] = lo[0] * scale;
    f[4 * q + 1] = lo[1] * scale;
    f[4 * q + 2] = hi[0] * scale;
    f[4 * q + 3] = hi[1] * scale;
  }
}

template <int LPR>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(ReadJob a) {
  constexpr int RPP = 64 / LPR;
  const int lane = threadIdx.x & 63;
  const int64_t r_begin = a.r0 + (int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * a.per_wave;
  if (r_begin >= a.R) return;
  const int r_end = int(min(int64_t(a.R), r_begin + a.per_wave));
  const CacheDev& c = a.cache;
  const int c0 = (lane & (LPR - 1)) * EPL;
  const bool on = c0 < c.head_dim;
  // the last sequence whose range begins at or before the first row
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= int(r_begin)) lo = mid;
    else hi = mid;
  }
  int b = lo;
  for (int r = int(r_begin); r < r_end; ++r) {
    while (b + 1 < a.B && a.offsets[b + 1] <= r) ++b;
    const int begin = max(a.offsets[b], 0);
    if (r < begin || r >= min(a.offsets[b + 1], a.R)) continue;   // no sequence's row
    const int64_t pos = int64_t(a.starts ? a.starts[b] : 0) + (r - begin);
    bool there = pos >= 0 && pos < int64_t(a.pages) * c.page_size;
    const uint32_t col = there ? c.page_of(uint32_t(pos)) : 0;
    const int32_t page = there ? a.table[int64_t(b) * a.ld_table + col] : -1;
    there = page >= 0 && page < c.n_pages;
    const int64_t row = there ? pos - int64_t(col) * c.page_size : 0;
    const int64_t at = there ? int64_t(page) * c.page + row * c.row : 0;
    const int64_t s_at = there && c.e4m3 ? int64_t(page) * c.s_page + row * c.s_row : 0;
    for (int h = lane / LPR; h < c.heads; h += RPP) {
      const int64_t off = at + int64_t(h) * c.head + int64_t(c0) * (c.e4m3 ? 1 : 2);
      float ks = 1.f, vs = 1.f;
      if (there && on && c.e4m3) {
        const int64_t so = s_at + int64_t(h) * c.s_head + int64_t(c0 / kBlock) * c.s_group;
        if (a.k.p) ks = c.k_scale[so];
        if (a.v.p) vs = c.v_scale[so];
      }
      float kf[EPL], vf[EPL];
      read_codes(c, c.k + off, ks, there && on && a.k.p, kf);
      read_codes(c, c.v + off, vs, there && on && a.v.p, vf);
      if (a.k.p) store_row(const_cast<void*>(a.k.p), a.k.bf16, int64_t(r) * a.k.token + int64_t(h) * a.k.head + c0, on ? EPL : 0, a.k.vec, kf);
      if (a.v.p) store_row(const_cast<void*>(a.v.p), a.v.bf16, int64_t(r) * a.v.token + int64_t(h) * a.v.head + c0, on ? EPL : 0, a.v.vec, vf);
    }
  }
}

// Waves that fill the device: a token is split over more of them only up to here, since each makes
// the token's sines and cosines again (1024 tokens of 48 heads of 128 BF16 channels with norms, 25 MB, 4.8
// us in a copy: 4096 waves 15 us, 8192 19.4; 4096 tokens with their cache rows 25, 25 and, at 16384, 29).
// Rows read back share nothing.
constexpr int64_t kEnoughWaves = 4096, kReadWaves = 8192;
constexpr int64_t kMostWaves = int64_t(1) << 25;    // of one launch (2^31 threads)

template <int LPR>
void launch_heads_pairs(const HeadsJob& a, int pairs, unsigned blocks, hipStream_t stream) {
  switch (pairs) {
    case kNone: hipLaunchKernelGGL((heads_kernel<LPR, kNone>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
    case kHalf: hipLaunchKernelGGL((heads_kernel<LPR, kHalf>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
    case kHalfOdd: hipLaunchKernelGGL((heads_kernel<LPR, kHalfOdd>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
    default: hipLaunchKernelGGL((heads_kernel<LPR, kAdjacent>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
  }
}

template <int LPR, int PAIRS>
void launch_heads_wide(const HeadsJob& a, bool x_bf16, unsigned blocks, hipStream_t stream) {
  const bool norm = a.qw || a.kw;
  const dim3 grid(blocks), block(kThreads);
  if (x_bf16 && norm) hipLaunchKernelGGL((heads_wide_kernel<LPR, PAIRS, true, true>), grid, block, 0, stream, a);
  else if (x_bf16) hipLaunchKernelGGL((heads_wide_kernel<LPR, PAIRS, true, false>), grid, block, 0, stream, a);
  else if (norm) hipLaunchKernelGGL((heads_wide_kernel<LPR, PAIRS, false, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((heads_wide_kernel<LPR, PAIRS, false, false>), grid, block, 0, stream, a);
}
template <int LPR>
void launch_heads_any(const HeadsJob& a, int pairs, bool wide, unsigned blocks, hipStream_t stream) {
  const bool x_bf16 = (a.q.heads ? a.q : a.k).bf16 != 0;
  if (!wide) launch_heads_pairs<LPR>(a, pairs, blocks, stream);
  else if (pairs == kNone) launch_heads_wide<LPR, kNone>(a, x_bf16, blocks, stream);
  else if (pairs == kHalf) launch_heads_wide<LPR, kHalf>(a, x_bf16, blocks, stream);
  else launch_heads_wide<LPR, kAdjacent>(a, x_bf16, blocks, stream);
}

}  // namespace

bsf8_status launch_heads(HeadsJob a, int64_t M, hipStream_t stream) {
  const int heads = a.q.heads + a.k.heads + a.v.heads;
  if (heads == 0) return BSF8_OK;
  const int lpr = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32, rows = 64 / lpr;
  const int pairs = a.R == 0 ? kNone : !a.half ? kAdjacent : (a.R / 2) % EPL == 0 ? kHalf : kHalfOdd;
  bool wide = pairs != kHalfOdd;
  for (const HeadsDev* h : {&a.q, &a.q_out, &a.k, &a.k_out, &a.v})
    if (h->heads) wide = wide && h->vec && (h == &a.q_out || h == &a.k_out || h->bf16 == (a.q.heads ? a.q : a.k).bf16);
  const int64_t passes = (heads + rows - 1) / rows;
  int64_t per = M * passes / kEnoughWaves;
  per = per < 1 ? 1 : per > passes ? passes : per;
  a.per_part = int(per) * rows;
  a.parts = int((passes + per - 1) / per);
  const int64_t tokens = kMostWaves / a.parts > 0 ? kMostWaves / a.parts : 1;
  for (int64_t m0 = 0; m0 < M; m0 += tokens) {
    a.m0 = m0;
    a.M = int32_t(M - m0 < tokens ? M - m0 : tokens);
    const unsigned blocks = unsigned((int64_t(a.M) * a.parts + kWaves - 1) / kWaves);
    if (lpr == 8) launch_heads_any<8>(a, pairs, wide, blocks, stream);
    else if (lpr == 16) launch_heads_any<16>(a, pairs, wide, blocks, stream);
    else launch_heads_any<32>(a, pairs, wide, blocks, stream);
    const bsf8_status st = device_status(hipGetLastError(), "rope / cache_write launch");
    if (st != BSF8_OK) return st;
  }
  return BSF8_OK;
}

bsf8_status launch_cache_read(const CacheDev& cache, int64_t B, const int32_t* table, int64_t ld_table, int64_t pages,
                              const int32_t* starts, const int32_t* offsets, int64_t R, const HeadsDev& k,
                              const HeadsDev& v, hipStream_t stream) {
  ReadJob a{};
  a.cache = cache;
  a.k = k;
  a.v = v;
  a.table = table;
  a.starts = starts;
  a.offsets = offsets;
  a.ld_table = ld_table;
  a.B = int32_t(B);
  a.pages = int32_t(pages);
  a.R = int32_t(R);
  const int64_t per = R / kReadWaves;
  a.per_wave = int32_t(per < 1 ? 1 : per > 16 ? 16 : per);
  for (int64_t r0 = 0; r0 < R; r0 += kMostWaves * a.per_wave) {
    a.r0 = r0;
    const int64_t n = R - r0 < kMostWaves * a.per_wave ? R - r0 : kMostWaves * a.per_wave;
    const unsigned blocks = unsigned((n + int64_t(kWaves) * a.per_wave - 1) / (int64_t(kWaves) * a.per_wave));
    if (cache.head_dim <= 64) hipLaunchKernelGGL(cache_read_kernel<8>, dim3(blocks), dim3(kThreads), 0, stream, a);
    else if (cache.head_dim <= 128) hipLaunchKernelGGL(cache_read_kernel<16>, dim3(blocks), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(cache_read_kernel<32>, dim3(blocks), dim3(kThreads), 0, stream, a);
    const bsf8_status st = device_status(hipGetLastError(), "cache_read launch");
    if (st != BSF8_OK) return st;
  }
  return BSF8_OK;
}

}  // namespace bsf8
