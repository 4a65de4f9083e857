// Attention of one new token per sequence over a paged cache (gfx950).
//
//   s_t = scale q.k_t,  o = sum_t 2^(c s_t - m) v_t / sum_t 2^(c s_t - m),  c = log2(e)
// with a running maximum m, in one pass over the sequence's keys and values.  The cache's
// bytes bound it: with G query heads per key head there are 4 G operations per element read,
// and up to 16 query heads share one read of the keys and values.
//
// A wave takes 32 tokens at a time, for 16 query heads, and keeps everything in registers:
//  * logits, transposed: S^T[token, head] = K[token, ch] Q^T[ch, head] by
//    v_mfma_f32_16x16x32_bf16, keys as they lie in memory as the A operand (a lane holds 8
//    channels of one token), queries as B.  A lane then holds one head's logits of 8 tokens:
//    4 g .. 4 g + 3 and 16 + 4 g .. of the tile, g its lane group.
//  * which is a B operand of the second product, O^T[ch, head] = V^T[ch, token] P^T[token, head],
//    if its k index (8 g + e) means those tokens: the sum over tokens has no order of its own.
//    The head stays the lane, so maximum, sum and rescaling are per lane.
//  * values: a lane loads 8 channels of each of its 8 tokens (a load instruction covers four
//    whole rows of 128 channels) and transposes the 8 x 8 block with v_perm_b32 in its own
//    registers; channel 8 i + j of the head is row i of the j-th product.
// No LDS and no barrier until a segment ends.
//
// Split over the length: a batch's (sequence, head) items are cut into tiles of 128 tokens
// (32 per wave), numbered through, and every block of a fixed grid takes an equal range of
// tiles, whatever the lengths are: long sequences spread over many blocks, short ones share
// one.  A block that holds an item whole stores its result; parts go to the workspace (at most
// two per block: its first and its last item) and the second kernel adds them, in an order that
// the lengths alone decide.
// The blocks find their ranges by a sum over the lengths, so nothing is read on the host.
#include <hip/hip_runtime.h>

#include <climits>

#include "bsf8_channels.h"
#include "bsf8_fused.h"

namespace bsf8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kWaveTokens = 32;
constexpr int kTile = kWaves * kWaveTokens;   // tokens
constexpr int kRows = 16;                     // query heads of an item

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) int32_t* ConstInts;   // read by the scalar unit

struct AttentionDev {
  CacheDev c;
  HeadsDev q, out;
  const int32_t* table;
  const int32_t* lens;
  float* lse;
  float* part;          // partial results: slots of kRows x chunks x 128 floats, then kRows maxima and kRows sums
  int64_t ld_table;
  int32_t B, pages;
  int32_t G;            // query heads per key head
  int32_t row_tiles;    // ceil(G / 16)
  int32_t items;        // of a sequence: key heads x row tiles
  int32_t window;       // 0: none
  int32_t bound;        // pages * page_size
  int32_t uniform;      // 16 tokens that start at a multiple of 16 are on one page
  int32_t scale_vec;    // four of a page's scales that follow each other are one aligned load
  int32_t blocks;       // grid of the first kernel
  float scale;          // log2(e) included
};

__device__ __forceinline__ int first_token(const AttentionDev& a, int n) { return a.window ? max(0, n - a.window) : 0; }
__device__ __forceinline__ int length(const AttentionDev& a, int b) {
  return min(max(((ConstInts)(a.lens))[b], 0), a.bound);
}
// tiles of a sequence of n tokens (one, all of it masked, where there is none), and the first one's number
__device__ __forceinline__ int tiles_of(const AttentionDev& a, int n, int& first) {
  first = first_token(a, n) / kTile;
  return n > 0 ? (n - 1) / kTile - first + 1 : 1;
}

// sums of a lane's value over the lanes up to it
__device__ __forceinline__ int running_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(v, d, 64);
    if (lane >= d) v += up;
  }
  return v;
}
__device__ __forceinline__ int lane_tiles(const AttentionDev& a, int b) {
  int first;
  const int n = b < a.B ? min(max(a.lens[b], 0), a.bound) : 0;
  return b < a.B ? tiles_of(a, n, first) : 0;
}
// tiles of the whole batch for one item per sequence
__device__ __forceinline__ int all_tiles(const AttentionDev& a) {
  int sum = 0;
  for (int base = 0; base < a.B; base += 64)
    sum += __builtin_amdgcn_readlane(running_sum(lane_tiles(a, base + int(threadIdx.x & 63))), 63);
  return sum;
}
// the sequence that holds tile `u` of that numbering, and the tiles before it
__device__ __forceinline__ int find_sequence(const AttentionDev& a, int u, int& before) {
  before = 0;
  for (int base = 0; base < a.B; base += 64) {
    const int n = lane_tiles(a, base + int(threadIdx.x & 63)), sum = running_sum(n);
    const uint64_t past = __ballot(before + sum > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      before += __builtin_amdgcn_readlane(sum - n, at);
      return base + at;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return a.B - 1;
}
// the tiles before sequence b
__device__ __forceinline__ int tiles_before(const AttentionDev& a, int b) {
  int sum = 0;
  for (int base = 0; base < b; base += 64) {
    const int i = base + int(threadIdx.x & 63);
    sum += __builtin_amdgcn_readlane(running_sum(i < b ? lane_tiles(a, i) : 0), 63);
  }
  return sum;
}

// the largest of the four lanes that hold a head (lanes 16 and 32 apart)
__device__ __forceinline__ float max_of_groups(float x) {
  u2 r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_of_groups(float x) {
  u2 r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Four channels of a head's result: o / l, and with channel 0 the log of the sum (natural, from
// base 2); zeros and -inf where there was no token.
__device__ __forceinline__ void store_result(const AttentionDev& a, int b, int head, int ch, f4 o, float m, float l) {
  const bool none = m == -INFINITY;
  float v[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] = none ? 0.f : o[x] / l;
  const int64_t at = int64_t(b) * a.out.token + int64_t(head) * a.out.head + ch;
  void* p = const_cast<void*>(a.out.p);
  if (a.out.bf16) {
    uint16_t* q = static_cast<uint16_t*>(p) + at;
    const uint32_t lo = bf16_pair(v[0], v[1]), hi = bf16_pair(v[2], v[3]);
    if (a.out.vec) {
      *reinterpret_cast<u2*>(q) = u2{lo, hi};
    } else {
      q[0] = uint16_t(lo);
      q[1] = uint16_t(lo >> 16);
      q[2] = uint16_t(hi);
      q[3] = uint16_t(hi >> 16);
    }
  } else {
    float* q = static_cast<float*>(p) + at;
    if (a.out.vec) {
      *reinterpret_cast<f4*>(q) = f4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) q[x] = v[x];
    }
  }
  if (a.lse && ch == 0)
    a.lse[int64_t(b) * a.q.heads + head] = none ? -INFINITY : 0.69314718055994531f * m + logf(l);
}

__device__ __forceinline__ v8bf as_bf16(u4 v) { return __builtin_bit_cast(v8bf, v); }

// eight F32 values as N BF16 terms whose sum they are (to 8 N bits)
template <int N>
__device__ __forceinline__ void split(const float (&x)[8], v8bf (&t)[N]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float rest = x[e];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const __bf16 b = static_cast<__bf16>(rest);
      t[i][e] = b;
      rest -= static_cast<float>(b);
    }
  }
}

// Blocks per compute unit (waves per SIMD) that the registers allow.
template <bool E4M3, int NG>
struct Shape {
  static constexpr int kBlocksPerCu = NG == 2 ? 1 : 2;
  static constexpr int kChannels = NG * 128;
  static constexpr int kSlot = kRows * kChannels + 2 * kRows;   // floats of a partial result
};

// NG: 128-channel groups of a head.  QT: BF16 terms of a query (1: BF16 queries, 3: F32);
// PT: of a softmax weight.  A weight in one term would be off by 2^-9 of itself, as much as
// the rounding of a BF16 output; two leave 2^-17, three 2^-25.
template <bool E4M3, int NG, int QT, int PT>
__global__ __launch_bounds__(kThreads, QT > 1 ? 1 : (Shape<E4M3, NG>::kBlocksPerCu)) void attention_kernel(AttentionDev a) {
  using S = Shape<E4M3, NG>;
  constexpr int KV = E4M3 ? 2 * NG : 4 * NG;   // 16-byte key loads per token and lane
  constexpr int PITCH = S::kChannels + 4;
  __shared__ float lds_o[kWaves][kRows][PITCH];
  __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int D = a.c.head_dim;

  const int total = all_tiles(a) * a.items;
  const int per = (total + a.blocks - 1) / a.blocks;
  const int t_begin = int(blockIdx.x) * per, t_end = min(total, t_begin + per);
  if (t_begin >= t_end) return;
  int before;
  int b = find_sequence(a, t_begin / a.items, before);
  int n = length(a, b), first;
  int n_tiles = tiles_of(a, n, first);
  int item = (t_begin - before * a.items) / n_tiles, j = (t_begin - before * a.items) - item * n_tiles;

  // byte offsets of a lane's pieces within a row; channels past head_dim are read as others
  // that exist (queries are zero there, and outputs are not stored)
  uint32_t k_off[KV], v_off[NG];
#pragma unroll
  for (int s = 0; s < KV; ++s) {
    const int ch = E4M3 ? min(s * 64 + g * 16, D - 16) : min(s * 32 + g * 8, D - 8);
    k_off[s] = uint32_t(i16) * uint32_t(a.c.row) + uint32_t(ch) * (E4M3 ? 1 : 2);
  }
#pragma unroll
  for (int c = 0; c < NG; ++c)
    v_off[c] = uint32_t(4 * g) * uint32_t(a.c.row) + uint32_t(min(c * 128 + i16 * 8, D - 8)) * (E4M3 ? 1 : 2);

  for (int t = t_begin; t < t_end;) {
    const int j_end = min(n_tiles, j + (t_end - t));
    const int h = item / a.row_tiles, row0 = (item - h * a.row_tiles) * kRows;
    const int rows = min(kRows, a.G - row0), head0 = h * a.G + row0;
    const int start = first_token(a, n), stop = min(n, (first + j_end) * kTile);

    // queries: the B operand, in the channel order of the keys' pieces
    v8bf qf[E4M3 ? 2 * KV : KV][QT];
#pragma unroll
    for (int s = 0; s < (E4M3 ? 2 * KV : KV); ++s) {
      const int ch = E4M3 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
      float x[8];
      load_vec(a.q.p, a.q.bf16, int64_t(b) * a.q.token + int64_t(head0 + i16) * a.q.head + ch, i16 < rows && ch < D ? 8 : 0,
               a.q.vec, x);
      split<QT>(x, qf[s]);
    }

    const uint8_t* k_base = a.c.k + int64_t(h) * a.c.head;
    const uint8_t* v_base = a.c.v + int64_t(h) * a.c.head;
    const float* ks_base = E4M3 ? a.c.k_scale + int64_t(h) * a.c.s_head : nullptr;
    const float* vs_base = E4M3 ? a.c.v_scale + int64_t(h) * a.c.s_head : nullptr;
    ConstInts table = (ConstInts)(a.table + int64_t(b) * a.ld_table);

    f4 o[NG][8];
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
      for (int x = 0; x < 8; ++x) o[c][x] = f4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    // ---- the pages of a wave's 32 tokens: two halves on a page each, or a token per lane
    struct Where {
      uint32_t mask;        // bit x: token x of the 32 exists
      int fast;             // both halves' pages are named by e0 / e1, r0 / r1 (page and row of their first token)
      int e0, e1, r0, r1;
      int le, lr;           // page and row of token lane & 31
    };
    const auto locate = [&](int pos, Where& w) {
      // (columns past the table's end are not read: tokens there do not exist)
      if (a.uniform) {
        const uint32_t p0 = a.c.page_of(uint32_t(pos)), p1 = a.c.page_of(uint32_t(pos + 16));
        w.r0 = pos - int(p0) * a.c.page_size;
        w.r1 = pos + 16 - int(p1) * a.c.page_size;
        w.e0 = table[min(int(p0), a.pages - 1)];
        w.e1 = table[min(int(p1), a.pages - 1)];
        w.fast = pos >= start && pos + kWaveTokens <= stop && uint32_t(w.e0) < uint32_t(a.c.n_pages) &&
                 uint32_t(w.e1) < uint32_t(a.c.n_pages);
        w.le = (lane & 16) ? w.e1 : w.e0;
        w.lr = ((lane & 16) ? w.r1 : w.r0) + i16;
      } else {
        const uint32_t p = a.c.page_of(uint32_t(pos + (lane & 31)));
        w.fast = 0;
        w.e0 = w.e1 = w.r0 = w.r1 = 0;
        w.le = a.table[int64_t(b) * a.ld_table + min(int(p), a.pages - 1)];
        w.lr = pos + (lane & 31) - int(p) * a.c.page_size;
      }
      w.mask = ~0u;
      if (!w.fast) {
        const int tok = pos + (lane & 31);
        const bool there = tok >= start && tok < stop && uint32_t(w.le) < uint32_t(a.c.n_pages);
        w.mask = uint32_t(__ballot(there));
        if (!there) w.le = w.lr = 0;   // row 0 of page 0 is read in its place and left out
      }
    };

    u4 kr[2][KV];
    float ksc[NG][2][4], vsc[NG][2][4];
    const auto load_keys = [&](const Where& w) {
      if (w.fast) {
        const uint8_t* p0 = k_base + int64_t(w.e0) * a.c.page + int64_t(w.r0) * a.c.row;
        const uint8_t* p1 = k_base + int64_t(w.e1) * a.c.page + int64_t(w.r1) * a.c.row;
#pragma unroll
        for (int s = 0; s < KV; ++s) {
          if (s * (E4M3 ? 64 : 32) >= D) continue;
          kr[0][s] = *reinterpret_cast<const u4*>(p0 + k_off[s]);
          kr[1][s] = *reinterpret_cast<const u4*>(p1 + k_off[s]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int e = __shfl(w.le, 16 * x + i16, 64), r = __shfl(w.lr, 16 * x + i16, 64);
          const uint8_t* p = k_base + int64_t(e) * a.c.page + int64_t(r - i16) * a.c.row;
#pragma unroll
          for (int s = 0; s < KV; ++s) {
            if (s * (E4M3 ? 64 : 32) >= D) continue;
            kr[x][s] = *reinterpret_cast<const u4*>(p + int64_t(k_off[s]));
          }
        }
      }
    };
    // scales of a lane's eight tokens
    const auto load_scales = [&](const Where& w, const float* base, float (&sc)[NG][2][4]) {
#pragma unroll
      for (int c = 0; c < NG; ++c) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float* p = base + int64_t(c) * a.c.s_group;
          if (w.fast) {
            p += int64_t(x ? w.e1 : w.e0) * a.c.s_page + int64_t(x ? w.r1 : w.r0) * a.c.s_row;
            if (a.scale_vec) {
              const f4 v = *reinterpret_cast<const f4*>(p + 4 * g);
#pragma unroll
              for (int r = 0; r < 4; ++r) sc[c][x][r] = v[r];
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r) sc[c][x][r] = p[int64_t(4 * g + r) * a.c.s_row];
            }
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int tok = 16 * x + 4 * g + r;
              sc[c][x][r] = p[int64_t(__shfl(w.le, tok, 64)) * a.c.s_page + int64_t(__shfl(w.lr, tok, 64)) * a.c.s_row];
            }
          }
        }
      }
    };
    u4 vr[NG][8];   // (E4M3: the first two words)
    const auto load_values = [&](const Where& w) {
      const auto piece = [&](const uint8_t* p, u4& v) {
        if (E4M3) {
          const u2 x = *reinterpret_cast<const u2*>(p);
          v[0] = x[0];
          v[1] = x[1];
        } else {
          v = *reinterpret_cast<const u4*>(p);
        }
      };
      if (w.fast) {
        const uint8_t* p0 = v_base + int64_t(w.e0) * a.c.page + int64_t(w.r0) * a.c.row;
        const uint8_t* p1 = v_base + int64_t(w.e1) * a.c.page + int64_t(w.r1) * a.c.row;
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int c = 0; c < NG; ++c)
            piece((e < 4 ? p0 : p1) + int64_t(e & 3) * a.c.row + v_off[c], vr[c][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int tok = (e >> 2) * 16 + 4 * g + (e & 3);
          const int pe = __shfl(w.le, tok, 64), r = __shfl(w.lr, tok, 64);
          const uint8_t* p = v_base + int64_t(pe) * a.c.page + int64_t(r - 4 * g) * a.c.row;
#pragma unroll
          for (int c = 0; c < NG; ++c)
            piece(p + int64_t(v_off[c]), vr[c][e]);
        }
      }
    };

    int pos = (first + j) * kTile + wave * kWaveTokens;
    Where w, next;
    if (pos < stop) {
      locate(pos, w);
      load_keys(w);
      if (E4M3) load_scales(w, ks_base, ksc);
      load_values(w);
      if (E4M3) load_scales(w, vs_base, vsc);
    }
    for (; pos < stop; pos += kTile) {
      const bool more = pos + kTile < stop;
      if (more) locate(pos + kTile, next);

      // ---- logits of 8 tokens and one head per lane
      float s[8];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        f4 acc[NG];
#pragma unroll
        for (int c = 0; c < NG; ++c) acc[c] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < KV; ++p) {
          if (p * (E4M3 ? 64 : 32) >= D) continue;
          constexpr int PARTS = E4M3 ? 2 : 1;
#pragma unroll
          for (int y = 0; y < PARTS; ++y) {
            const v8bf kf = E4M3 ? decode8(kr[x][p][2 * y], kr[x][p][2 * y + 1]) : as_bf16(kr[x][p]);
            f4& to = acc[E4M3 ? p / 2 : 0];
#pragma unroll
            for (int q = 0; q < QT; ++q) to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[p * PARTS + y][q], to, 0, 0, 0);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v = acc[0][r];
          if (E4M3) {
            v *= ksc[0][x][r];
            if (NG == 2) v = fmaf(acc[NG - 1][r], ksc[NG - 1][x][r], v);
          }
          s[4 * x + r] = v * a.scale;
        }
      }
      if (more) {
        load_keys(next);
        if (E4M3) load_scales(next, ks_base, ksc);
      }
      if (w.mask != ~0u) {
        const uint32_t mine = w.mask >> (4 * g);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((mine >> ((e >> 2) * 16 + (e & 3))) & 1)) s[e] = -INFINITY;
      }

      // ---- running maximum and sum
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
      top = fmaxf(m, max_of_groups(top));
      if (__ballot(top > m)) {
        const float f = top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - top);
        l *= f;
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
          for (int x = 0; x < 8; ++x) o[c][x] *= f;
        m = top;
      }
      const float ref = m == -INFINITY ? 0.f : m;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(s[e] - ref);
        l += p[e];
      }

      // ---- values: rows of tokens that do not exist may hold anything
      if (w.mask != ~0u) {
        const uint32_t mine = w.mask >> (4 * g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool there = (mine >> ((e >> 2) * 16 + (e & 3))) & 1;
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            if (E4M3 && !there) vsc[c][e >> 2][e & 3] = 0.f;
#pragma unroll
            for (int x = 0; x < (E4M3 ? 2 : 4); ++x) vr[c][e][x] = there ? vr[c][e][x] : 0u;
          }
        }
      }
      v8bf pt[E4M3 ? NG : 1][PT];
      if (E4M3) {
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            float ps[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) ps[e] = p[e] * vsc[c][e >> 2][e & 3];
          split<PT>(ps, pt[c]);
        }
      } else {
        split<PT>(p, pt[0]);
      }
#pragma unroll
      for (int c = 0; c < NG; ++c) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {   // channels 2 x and 2 x + 1 of each lane's eight
          uint32_t pair[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            pair[e] = E4M3 ? __builtin_bit_cast(uint32_t, (x & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vr[c][e][x >> 1], 1.0f, true)
                                                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vr[c][e][x >> 1], 1.0f, false))
                           : vr[c][e][x];
          u4 lo, hi;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            lo[e] = __builtin_amdgcn_perm(pair[2 * e + 1], pair[2 * e], 0x05040100u);
            hi[e] = __builtin_amdgcn_perm(pair[2 * e + 1], pair[2 * e], 0x07060302u);
          }
#pragma unroll
          for (int q = 0; q < PT; ++q) {
            o[c][2 * x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(lo), pt[E4M3 ? c : 0][q], o[c][2 * x], 0, 0, 0);
            o[c][2 * x + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(hi), pt[E4M3 ? c : 0][q], o[c][2 * x + 1], 0, 0, 0);
          }
        }
      }
      if (more) {
        load_values(next);
        if (E4M3) load_scales(next, vs_base, vsc);
        w = next;
      }
    }

    // ---- the waves' parts of the segment
    l = sum_of_groups(l);
    if (g == 0) {
      lds_m[wave][i16] = m;
      lds_l[wave][i16] = l;
    }
    __syncthreads();
    float top = lds_m[0][i16];
#pragma unroll
    for (int x = 1; x < kWaves; ++x) top = fmaxf(top, lds_m[x][i16]);
    const float mine = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          f4 v;
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = o[c][4 * y + x][r] * mine;
          *reinterpret_cast<f4*>(&lds_o[wave][i16][c * 128 + (4 * g + r) * 8 + 4 * y]) = v;
        }
    __syncthreads();
    const bool whole = j == 0 && j_end == n_tiles;
    float* part = a.part + (int64_t(blockIdx.x) * 2 + (t == t_begin ? 0 : 1)) * S::kSlot;
    for (int x = threadIdx.x; x < kRows * (S::kChannels / 4); x += kThreads) {
      const int row = x / (S::kChannels / 4), ch = 4 * (x % (S::kChannels / 4));
      if (row >= rows || ch >= D) continue;
      f4 v = *reinterpret_cast<const f4*>(&lds_o[0][row][ch]);
#pragma unroll
      for (int y = 1; y < kWaves; ++y) v += *reinterpret_cast<const f4*>(&lds_o[y][row][ch]);
      float all_m = lds_m[0][row], all_l = 0.f;
#pragma unroll
      for (int y = 1; y < kWaves; ++y) all_m = fmaxf(all_m, lds_m[y][row]);
#pragma unroll
      for (int y = 0; y < kWaves; ++y)
        all_l += all_m == -INFINITY ? 0.f : lds_l[y][row] * __builtin_amdgcn_exp2f(lds_m[y][row] - all_m);
      if (whole) {
        store_result(a, b, head0 + row, ch, v, all_m, all_l);
      } else {
        *reinterpret_cast<f4*>(part + row * S::kChannels + ch) = v;
        if (ch == 0) {
          part[kRows * S::kChannels + row] = all_m;
          part[kRows * S::kChannels + kRows + row] = all_l;
        }
      }
    }
    __syncthreads();

    t += j_end - j;
    j = 0;
    if (++item == a.items && t < t_end) {
      item = 0;
      n = length(a, ++b);
      n_tiles = tiles_of(a, n, first);
    }
  }
}

// Adds the parts of the items that lie in more than one block, a query head per block of this
// grid: groups of lanes take every so many parts, with a maximum of their own.
template <int NG>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttentionDev a) {
  using S = Shape<false, NG>;   // (a slot has one size for both types of cache)
  constexpr int LANES = S::kChannels / 4, GROUPS = kThreads / LANES, FLIGHT = 4;
  __shared__ float lds_o[GROUPS][S::kChannels], lds_m[GROUPS], lds_l[GROUPS];
  const int heads = a.G * a.c.heads;
  const int b = int(blockIdx.x / unsigned(heads)), head = int(blockIdx.x) - b * heads;
  const int h = head / a.G, in_group = head - h * a.G, item = h * a.row_tiles + in_group / kRows, row = in_group % kRows;
  int first;
  const int n_tiles = tiles_of(a, length(a, b), first);
  const int total = all_tiles(a) * a.items, per = (total + a.blocks - 1) / a.blocks;
  const int begin = tiles_before(a, b) * a.items + item * n_tiles;
  const int from = begin / per, to = (begin + n_tiles - 1) / per;
  if (from == to) return;   // one block had all of it
  const int group = threadIdx.x / LANES, ch = 4 * (threadIdx.x % LANES);
  const bool on = ch < a.c.head_dim;
  float m = -INFINITY, l = 0.f;
  f4 o = f4{0.f, 0.f, 0.f, 0.f};
  for (int x = from + group; x <= to; x += GROUPS * FLIGHT) {
    f4 v[FLIGHT];
    float pm[FLIGHT], pl[FLIGHT];
#pragma unroll
    for (int y = 0; y < FLIGHT; ++y) {
      const int blk = min(x + y * GROUPS, to);
      // its block's first item, unless the block begins before it
      const float* p = a.part + (int64_t(blk) * 2 + (blk == from && begin > from * per ? 1 : 0)) * S::kSlot;
      v[y] = on ? *reinterpret_cast<const f4*>(p + row * S::kChannels + ch) : f4{0.f, 0.f, 0.f, 0.f};
      pm[y] = x + y * GROUPS <= to ? p[kRows * S::kChannels + row] : -INFINITY;
      pl[y] = p[kRows * S::kChannels + kRows + row];
    }
    float top = m;
#pragma unroll
    for (int y = 0; y < FLIGHT; ++y) top = fmaxf(top, pm[y]);
    if (top == -INFINITY) continue;
    float f = __builtin_amdgcn_exp2f(m - top);
    l *= f;
    o *= f;
#pragma unroll
    for (int y = 0; y < FLIGHT; ++y) {
      f = __builtin_amdgcn_exp2f(pm[y] - top);
      if (f == 0.f) continue;   // (a part without a token)
      l = fmaf(pl[y], f, l);
      o += v[y] * f;
    }
    m = top;
  }
  *reinterpret_cast<f4*>(&lds_o[group][ch]) = o;
  if (ch == 0) {
    lds_m[group] = m;
    lds_l[group] = l;
  }
  __syncthreads();
  if (group != 0 || !on) return;
  float top = lds_m[0], sum = 0.f;
#pragma unroll
  for (int y = 1; y < GROUPS; ++y) top = fmaxf(top, lds_m[y]);
  f4 v = f4{0.f, 0.f, 0.f, 0.f};
  if (top != -INFINITY) {
#pragma unroll
    for (int y = 0; y < GROUPS; ++y) {
      const float f = __builtin_amdgcn_exp2f(lds_m[y] - top);
      sum = fmaf(lds_l[y], f, sum);
      v += *reinterpret_cast<const f4*>(&lds_o[y][ch]) * f;
    }
  }
  store_result(a, b, head, ch, v, top, sum);
}

int compute_units() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  static thread_local int known_dev = -1, known = 0;
  if (dev != known_dev) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    known = cus;
    known_dev = dev;
  }
  return known;
}

// Blocks of the first kernel: as many as the device holds at once, or a block per tile.
int64_t grid_blocks(const CacheDev& c, int64_t B, int32_t q_heads, int64_t bound) {
  const int64_t row_tiles = (q_heads / c.heads + kRows - 1) / kRows;
  const int64_t most = B * c.heads * row_tiles * (bound / kTile + 2);
  const int64_t held = int64_t(compute_units()) * (c.head_dim > 128 ? Shape<false, 2>::kBlocksPerCu
                                                   : c.e4m3         ? Shape<true, 1>::kBlocksPerCu
                                                                    : Shape<false, 1>::kBlocksPerCu);
  return most < held ? most : held;
}

template <bool E4M3, int NG>
void launch_attention_kernel(const AttentionDev& a, bool f32, hipStream_t stream) {
  if (f32)
    hipLaunchKernelGGL((attention_kernel<E4M3, NG, 3, 3>), dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((attention_kernel<E4M3, NG, 1, 2>), dim3(unsigned(a.blocks)), dim3(kThreads), 0, stream, a);
}

}  // namespace

int64_t attention_tiles(const CacheDev& c, int64_t B, int32_t q_heads, int64_t bound) {
  return B * c.heads * ((q_heads / c.heads + kRows - 1) / kRows) * (bound / kTile + 2);
}

size_t attention_workspace_bytes(const CacheDev& c, int64_t B, int32_t q_heads, int64_t bound) {
  if (bound <= kTile || B == 0) return 0;   // no item is ever split
  const size_t slot = c.head_dim > 128 ? Shape<false, 2>::kSlot : Shape<false, 1>::kSlot;
  return size_t(grid_blocks(c, B, q_heads, bound)) * 2 * slot * sizeof(float);
}

bsf8_status launch_attention(const CacheDev& c, const HeadsDev& q, const HeadsDev& out, int64_t B, const int32_t* table,
                             int64_t ld_table, int64_t pages, const int32_t* lens, int64_t window, double scale, float* lse,
                             void* ws, hipStream_t stream) {
  AttentionDev a{};
  a.c = c;
  a.q = q;
  a.out = out;
  a.table = table;
  a.lens = lens;
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.ld_table = ld_table;
  a.B = int32_t(B);
  a.pages = int32_t(pages);
  a.G = q.heads / c.heads;
  a.row_tiles = (a.G + kRows - 1) / kRows;
  a.items = c.heads * a.row_tiles;
  a.bound = int32_t(pages * c.page_size);
  a.window = window >= a.bound ? 0 : int32_t(window);
  a.uniform = c.page_size % 16 == 0 ? 1 : 0;
  a.scale_vec = c.e4m3 && c.s_row == 1 && ((c.s_page | c.s_head | c.s_group) & 3) == 0 &&
                        ((reinterpret_cast<uintptr_t>(c.k_scale) | reinterpret_cast<uintptr_t>(c.v_scale)) & 15) == 0
                    ? 1 : 0;
  a.blocks = int32_t(grid_blocks(c, B, q.heads, a.bound));
  a.scale = float(scale * 1.4426950408889634);
  const bool f32 = !q.bf16 || !out.bf16, wide = c.head_dim > 128;
  if (c.e4m3 && wide) launch_attention_kernel<true, 2>(a, f32, stream);
  else if (c.e4m3) launch_attention_kernel<true, 1>(a, f32, stream);
  else if (wide) launch_attention_kernel<false, 2>(a, f32, stream);
  else launch_attention_kernel<false, 1>(a, f32, stream);
  bsf8_status st = device_status(hipGetLastError(), "paged_attention launch");
  if (st != BSF8_OK || a.bound <= kTile) return st;
  const unsigned rows = unsigned(B * q.heads);
  if (wide) hipLaunchKernelGGL(attention_join_kernel<2>, dim3(rows), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(attention_join_kernel<1>, dim3(rows), dim3(kThreads), 0, stream, a);
  return device_status(hipGetLastError(), "paged_attention join launch");
}

}  // namespace bsf8
