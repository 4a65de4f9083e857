// Attention of one new token per sequence over a paged cache (gfx950).
//
//   s_t = scale q.k_t,  o = sum_t 2^(c s_t - m) v_t / sum_t 2^(c s_t - m),  c = log2(e)
// with a running maximum m, in one pass over the sequence's keys and values.  The cache's
// bytes bound it: with G query heads per key head there are 4 G operations per element read,
// and up to 16 query heads share one read of the keys and values.
//
// A wave takes 32 tokens at a time, for 16 query heads, and keeps them in registers (what does not
// fit goes to scratch: with BF16 queries 37 registers of the instances of 256 BF16 channels and, where
// pages are no multiple of 16 rows, 71 to 82, 25 to 27 of those of 128 BF16 channels and 10 to 23 of
// 256 codes; 3 to 9 in heads of 129 to 255 codes; one with F32 queries of 256 codes; no others):
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
// two per block: its first and its last item) and a second kernel adds them, in an order that
// the lengths alone decide.  The blocks find their ranges by a sum over the lengths, so nothing
// is read on the host; the block that holds an item's beginning leaves a note of where its
// parts are, so that the second kernel need not find them again.
//
// Measured (kernels alone, joining apart): 64 sequences to 8192, 8 key heads of 128 E4M3 channels,
// 379 MB: 82 + 6 us, 4.6 TB/s; 256 to 1000, 24 heads of 80 BF16 channels, 661 MB: 125 us, 5.3 TB/s,
// what a copy reaches; one of 131072, 4 key heads of E4M3, 138 MB: 28 + 5; F32 queries of 7 to 5000
// (window 2048, 256 BF16 channels, 38 MB): 21.5 + 4, a tile or two for each compute unit, so that
// the time is that of a wave's chain from lengths over table and rows to the products.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "bsf8_channels.h"
#include "bsf8_fused.h"

namespace bsf8 {
namespace {

constexpr int kMostWaves = 8;                 // of a block; four or eight
constexpr int kWaveTokens = 32;
constexpr int kRows = 16;                     // query heads of an item
constexpr int kWholeTokens = 512;             // up to here an item is a block's
constexpr float kDown = 0x1p-64f;             // of queries, where the scale is very small

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) int32_t* ConstInts;   // read by the scalar unit

struct Task;

struct AttentionDev {
  CacheDev c;
  HeadsDev q, out;
  const int32_t* table;
  const int32_t* lens;
  float* lse;
  float* part;          // partial results: slots of kRows x chunks x 128 floats, then kRows maxima and kRows sums
  Task* tasks;   // what is to be joined: by item if there are no more items than blocks, else by block
  int32_t by_item;
  int64_t ld_table;
  int32_t B, pages;
  int32_t G;            // query heads per key head
  int32_t row_tiles;    // ceil(G / 16)
  int32_t items;        // of a sequence: key heads x row tiles
  int32_t window;       // 0: none
  int32_t bound;        // pages * page_size
  int32_t blocks;       // grid of the first kernel
  int32_t whole;        // a block per item, nothing to join
  int32_t tile_shift;   // a tile is 1 << tile_shift tokens: 32 for each wave of a block
  int32_t negative;     // the scale is: queries change their sign, and `scale` is its size
  int32_t small;        // and very small: queries are taken down by 2^64, and `scale` is up by it
  float scale;          // log2(e) included; not zero
  double natural;       // the size of the scale, for such queries
};

// An item whose parts lie in blocks `slot / 2` .. `to`: the first in `slot`, the others in the
// first slot of their blocks.
struct Task {
  int32_t b, head0, rows, slot, to;   // rows 0: nothing to join
  int32_t unused[3];
};

__device__ __forceinline__ int first_token(const AttentionDev& a, int n) { return a.window ? max(0, n - a.window) : 0; }
// tiles of a sequence of n tokens (one, all of it masked, where there is none), and the first one's number
__device__ __forceinline__ int tiles_of(const AttentionDev& a, int n, int& first) {
  first = first_token(a, n) >> a.tile_shift;
  return n > 0 ? ((n - 1) >> a.tile_shift) - first + 1 : 1;
}

// 64 sequences, one per lane: their lengths, tiles, and the tiles up to and with them.
struct Lengths {
  int n, tiles, sum;
};
__device__ __forceinline__ Lengths lengths_of(const AttentionDev& a, int base) {
  const int lane = threadIdx.x & 63, b = base + lane;
  Lengths x;
  x.n = min(max(a.lens[min(b, a.B - 1)], 0), a.bound);
  int first;
  x.tiles = b < a.B ? tiles_of(a, x.n, first) : 0;
  x.sum = x.tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(x.sum, d, 64);
    if (lane >= d) x.sum += up;
  }
  return x;
}
// the sequence that holds tile `u` (of one item per sequence), and the tiles before it; x: those of the first 64 at first
__device__ __forceinline__ int find_sequence(const AttentionDev& a, Lengths& x, int& base, int u, int& before) {
  before = 0;
  for (base = 0;; base += 64) {
    if (base) x = lengths_of(a, base);
    const uint64_t past = __ballot(before + x.sum > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      before += __builtin_amdgcn_readlane(x.sum - x.tiles, at);
      return base + at;
    }
    if (base + 64 >= a.B) return a.B - 1;   // (u is a tile of the batch: not reached)
    before += __builtin_amdgcn_readlane(x.sum, 63);
  }
}

// Block w's tiles begin at begin_of(w): `few` or, the first `more` blocks, few + 1 tiles each.
// (Ranges of one size would leave blocks without work: 4096 tiles over 768 blocks in sixes.)
struct Ranges {
  int few, more;
  __device__ __forceinline__ Ranges(int total, int blocks) : few(total / blocks), more(total - few * blocks) {}
  __device__ __forceinline__ int begin_of(int w) const { return w * few + min(w, more); }
  __device__ __forceinline__ int block_of(int t) const {
    const int big = more * (few + 1);
    return t < big ? t / (few + 1) : more + (t - big) / few;
  }
};

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

// Four channels of a head's result: o / l, and with channel 0 the log of the sum, the maximum's
// part of it in F64 (it can be large); zeros and -inf where there was no token, which is where the
// sum is zero (logits of nothing but NaN leave the maximum at -inf and the sum NaN).
__device__ __forceinline__ void store_result(const AttentionDev& a, int b, int head, int ch, f4 o, float m, float l) {
  const bool none = l == 0.f;
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
    a.lse[int64_t(b) * a.q.heads + head] = none ? -INFINITY : static_cast<float>(a.natural * double(m) + double(logf(l)));
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

// What an instance is made for.
// DIM: channels that its pieces cover (64, 128, 256).  FULL: a head has exactly DIM of them, so
// that offsets are constants and rows are whole cache lines, which are read non-temporally: each
// once (64 sequences to 8192 of 128 BF16 channels 147 -> 134 us, of E4M3 91 -> 84; rows that
// share lines lose by it, 80 channels 185 -> 218.  Keys left to the cache, the values alone
// non-temporal, both sides three times in turn, each within 1 %: one sequence of 131072 33.0 -> 31.4
// us, of 32768 34.2 -> 30.0, but the batch 85.3 -> 88.3, of BF16 132.6 -> 136.1, 32 of 256 BF16 channels
// 90.5 -> 99.3).
// QT: BF16 terms of a query (1: BF16 queries, 3: F32).  PT: of a softmax weight.  A weight in one
// term would be off by up to 2^-8 of itself, as much as the rounding of a BF16 output; two leave 2^-17,
// three nothing of its 24 bits.
// PAGES: kAny, each lane looks up a token's page; kHalves, pages are a multiple of 16 rows, so
// that each half of a wave's 32 tokens is on one page, whose rows all exist: addresses are
// scalar, and rows past the length are read and left out; kHalvesWide, also four scales are
// one load.  (A choice inside the kernel would be a branch around loads, and where its sides
// meet the compiler waits for all of them.)
enum Pages { kAny, kHalves, kHalvesWide };
template <bool E4M3_, int DIM_, bool FULL_, int QT_, int PT_, int PAGES_>
struct Config {
  static constexpr bool E4M3 = E4M3_, FULL = FULL_, PAGES16 = PAGES_ != kAny;
  static constexpr int DIM = DIM_, QT = QT_, PT = PT_, PAGES = PAGES_;
  static constexpr int NG = DIM > 128 ? 2 : 1;         // 128-channel groups
  // HP 2: a row of the keys' operand is half a line of a token, 64 bytes, so that one load of the
  // wave covers eight tokens' whole lines where it would touch half of sixteen and every line be
  // asked for twice; the matrix instructions double.  (Both sides three times in turn, each within 1 %:
  // 256 sequences to 1000 of 80 BF16 channels 148 -> 124 us, 64 to 8192 of 128 E4M3 ones 86.7 -> 85.3,
  // 32 of 256 BF16 ones, which spill, 93.9 -> 90.5, one of 32768 36.6 -> 34.2.  Not where rows are
  // 64 bytes, nor where the instructions tell: 256 E4M3 channels 53 -> 57, F32 queries 62 -> 65.)
  static constexpr int HP = QT > 1 || (E4M3 && DIM != 128) ? 1 : 2;
  static constexpr int LN = DIM * (E4M3 ? 1 : 2) / (64 * HP);   // 16-byte loads per lane and row of the operand
  static constexpr int X = 2 * HP;                     // operands of 32 tokens
  static constexpr int PER = 4 / HP;                   // tokens of a lane's logits in one of them
  static constexpr int QS = DIM / 32;                  // query pieces: 32 channels each
  static constexpr int CHANNELS = NG * 128;
  static constexpr int PITCH = CHANNELS + 4;           // floats of a row in LDS
  static constexpr int SLOT = kRows * CHANNELS + 2 * kRows;   // floats of a partial result
};
// Waves per SIMD that the registers allow.
constexpr int waves_per_simd(int dim, bool f32) { return dim > 128 ? (f32 ? 1 : 2) : f32 ? 2 : 3; }
// Waves of a block: wide heads with F32 queries take half of a SIMD's registers and more.
constexpr int most_waves(int dim, bool f32) { return dim > 128 && f32 ? 4 : kMostWaves; }
constexpr int slot_floats(int dim) { return Config<false, 128, false, 1, 2, kAny>::SLOT + (dim > 128 ? kRows * 128 : 0); }

template <bool NT, typename T>
__device__ __forceinline__ T fetch(const uint8_t* p) {
  if (NT) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  return *reinterpret_cast<const T*>(p);
}

// Queries of 16 heads: the B operand, in the channel order of the keys' pieces; zeros for heads
// past `rows` and channels past head_dim.  begin() asks for them, end() makes the operand.
template <class C>
struct Queries {
  static constexpr int W = C::QT == 1 ? 1 : 2;
  u4 raw[C::QS][W];       // BF16 values, or F32 ones
  __device__ __forceinline__ static int channel(int s) {
    const int g = (threadIdx.x & 63) >> 4;
    return C::E4M3 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
  }
  __device__ __forceinline__ void begin(const AttentionDev& a, int b, int head0, int rows) {
    const int D = C::FULL ? C::DIM : a.c.head_dim;
    const int64_t base = int64_t(b) * a.q.token + int64_t(head0 + min(int(threadIdx.x & 15), rows - 1)) * a.q.head;
    if (a.q.vec && (C::QT == 1 || !a.q.bf16)) {
#pragma unroll
      for (int s = 0; s < C::QS; ++s)
#pragma unroll
        for (int y = 0; y < W; ++y)
          raw[s][y] = reinterpret_cast<const u4*>(static_cast<const uint8_t*>(a.q.p) +
                                                  (base + min(channel(s), D - 8)) * (C::QT == 1 ? 2 : 4))[y];
      return;
    }
#pragma unroll
    for (int s = 0; s < C::QS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = load_real(a.q.p, a.q.bf16, base + min(channel(s), D - 8) + e);
        if (C::QT == 1) raw[s][0][e >> 1] = (e & 1) ? raw[s][0][e >> 1] | __float_as_uint(x) : __float_as_uint(x) >> 16;
        else raw[s][e >> 2][e & 3] = __float_as_uint(x);
      }
  }
  __device__ __forceinline__ void end(const AttentionDev& a, int rows, v8bf (&qf)[C::QS][C::QT]) const {
    const int D = C::FULL ? C::DIM : a.c.head_dim;
#pragma unroll
    for (int s = 0; s < C::QS; ++s) {
      const bool there = int(threadIdx.x & 15) < rows && channel(s) < D;
      const uint32_t sign = a.negative ? (C::QT == 1 ? 0x80008000u : 0x80000000u) : 0u;
      if (C::QT == 1) {
        u4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = there ? raw[s][0][x] ^ sign : 0u;
        if (a.small) {
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = bf16_pair(__uint_as_float(v[x] << 16) * kDown, __uint_as_float(v[x] & 0xFFFF0000u) * kDown);
        }
        qf[s][0] = as_bf16(v);
      } else {
        float x[8];
        const float by = a.small ? kDown : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = there ? __uint_as_float(raw[s][(e >> 2) % W][e & 3] ^ sign) * by : 0.f;
        split<C::QT>(x, qf[s]);
      }
    }
  }
};

template <class C>
__global__ __launch_bounds__(64 * most_waves(C::DIM, C::QT > 1), waves_per_simd(C::DIM, C::QT > 1)) void attention_kernel(AttentionDev a) {
  constexpr bool E4M3 = C::E4M3, PAGES16 = C::PAGES16;
  constexpr int NG = C::NG, QT = C::QT, PT = C::PT, QS = C::QS, HP = C::HP, LN = C::LN, X = C::X, PER = C::PER;
  constexpr int PITCH = C::PITCH;
  // a wave's part of a result: its sums (kRows x PITCH), and for all waves maxima and sums of weights
  extern __shared__ __attribute__((aligned(16))) float lds_o[];
  __shared__ float lds_m[kMostWaves][kRows], lds_l[kMostWaves][kRows];
  const int waves = int(blockDim.x >> 6), tile_tokens = 1 << a.tile_shift;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int D = C::FULL ? C::DIM : a.c.head_dim;

  // the block's tiles, and the item of the first: sequence, key head, first query head of the key head's, tile
  int t_begin, t_end, b, n, first, n_tiles, item, j, base = 0;
  Lengths seq;
  Ranges ranges(0, 1);
  if (a.whole) {
    b = int(blockIdx.x / unsigned(a.items));
    item = int(blockIdx.x) - b * a.items;
    n = min(max(((ConstInts)a.lens)[b], 0), a.bound);
    n_tiles = tiles_of(a, n, first);
    t_begin = j = 0;
    t_end = n_tiles;
  } else {
    seq = lengths_of(a, 0);
    int total = __builtin_amdgcn_readlane(seq.sum, 63);
    for (int at = 64; at < a.B; at += 64) total += __builtin_amdgcn_readlane(lengths_of(a, at).sum, 63);
    total *= a.items;
    ranges = Ranges(total, a.blocks);
    t_begin = ranges.begin_of(int(blockIdx.x));
    t_end = ranges.begin_of(int(blockIdx.x) + 1);
    if (t_begin >= t_end) {
      if (!a.by_item && threadIdx.x == 0) a.tasks[blockIdx.x].rows = 0;
      return;
    }
    int before;
    b = find_sequence(a, seq, base, t_begin / a.items, before);
    n = __builtin_amdgcn_readlane(seq.n, b - base);
    n_tiles = tiles_of(a, n, first);
    item = (t_begin - before * a.items) / n_tiles;
    j = (t_begin - before * a.items) - item * n_tiles;
  }
  int h = item / a.row_tiles, row0 = (item - h * a.row_tiles) * kRows;

  // byte offsets of a lane's pieces within a row, with its token's among the operand's; channels
  // past head_dim are read as others that exist (queries are zero there, and outputs are not stored)
  const uint32_t k_row = PAGES16 ? uint32_t(i16 / HP) * uint32_t(a.c.row) : 0, v_row = PAGES16 ? uint32_t(PER * g) * uint32_t(a.c.row) : 0;
  const auto key_offset = [&](int ln) {
    const int at = ln * 64 * HP + (i16 % HP) * 64 + g * 16;
    return k_row + uint32_t(C::FULL ? at : min(at, (D - (E4M3 ? 16 : 8)) * (E4M3 ? 1 : 2)));
  };
  const auto value_offset = [&](int c) { return v_row + uint32_t(min(c * 128 + i16 * 8, D - 8)) * (E4M3 ? 1 : 2); };
  // the lane's eight tokens of the 32: PER of each operand; the rest of their numbers is PER * g
  const auto token = [](int e) constexpr { return e / PER * (16 / HP) + e % PER; };

  for (int t = t_begin; t < t_end;) {
    // the item's tiles j .. j_end - 1 are this block's
    const int j_end = min(n_tiles, j + (t_end - t));
    const int rows = min(kRows, a.G - row0), head0 = h * a.G + row0;
    const int start = first_token(a, n), stop = min(n, (first + j_end) << a.tile_shift);

    // ---- where a wave's 32 tokens lie.  Entries of the table are asked for a tile before they are needed
    struct Entries {
      int e0, e1;           // pages of the halves; or e0: page of token lane & 31
      int r0, r1;           // their rows
    };
    const auto entries = [&](int pos) {
      // (columns past the table's end are not read: tokens there do not exist)
      Entries e;
      if (PAGES16) {
        const int p0 = int(__umulhi(uint32_t(pos), a.c.magic) >> (a.c.shift - 32));   // (shift is 35 or more)
        e.r0 = pos - p0 * a.c.page_size;
        const bool same = e.r0 + 16 < a.c.page_size;
        e.r1 = same ? e.r0 + 16 : 0;
        ConstInts table = (ConstInts)(a.table + int64_t(b) * a.ld_table);
        e.e0 = table[min(p0, a.pages - 1)];
        e.e1 = table[min(same ? p0 : p0 + 1, a.pages - 1)];
      } else {
        const int tok = pos + (lane & 31), p = int(a.c.page_of(uint32_t(tok)));
        e.r0 = tok - p * a.c.page_size;
        e.e0 = a.table[int64_t(b) * a.ld_table + min(p, a.pages - 1)];
        e.e1 = e.r1 = 0;
      }
      return e;
    };
    struct Where {
      uint32_t mask;              // bit x: token x of the 32 exists
      int64_t at[2], s_at[2];     // of the halves: bytes, elements of scales; at[0] and s_at[0] of the head alone where
      int le, lr;                 // each lane has a page and row of token lane & 31
    };
    const auto locate = [&](int pos, Entries e, Where& w) {
      w.at[0] = int64_t(h) * a.c.head;
      if (E4M3) w.s_at[0] = int64_t(h) * a.c.s_head;
      if (PAGES16) {
        const auto below = [](int x) { return x >= 32 ? ~0u : x <= 0 ? 0u : (1u << x) - 1u; };
        w.mask = below(stop - pos) & ~below(start - pos);
        // a page outside the cache: page 0 is read in its place and left out
        if (uint32_t(e.e0) >= uint32_t(a.c.n_pages)) {
          e.e0 = 0;
          w.mask &= 0xFFFF0000u;
        }
        if (uint32_t(e.e1) >= uint32_t(a.c.n_pages)) {
          e.e1 = 0;
          w.mask &= 0xFFFFu;
        }
        w.at[1] = w.at[0] + uint64_t(uint32_t(e.e1)) * uint32_t(a.c.page) + uint64_t(uint32_t(e.r1)) * uint32_t(a.c.row);
        w.at[0] += uint64_t(uint32_t(e.e0)) * uint32_t(a.c.page) + uint64_t(uint32_t(e.r0)) * uint32_t(a.c.row);
        if (E4M3) {
          w.s_at[1] = w.s_at[0] + uint64_t(uint32_t(e.e1)) * uint32_t(a.c.s_page) + uint64_t(uint32_t(e.r1)) * uint32_t(a.c.s_row);
          w.s_at[0] += uint64_t(uint32_t(e.e0)) * uint32_t(a.c.s_page) + uint64_t(uint32_t(e.r0)) * uint32_t(a.c.s_row);
        }
      } else {
        const int tok = pos + (lane & 31);
        w.le = e.e0;
        w.lr = e.r0;
        const bool there = tok >= start && tok < stop && uint32_t(w.le) < uint32_t(a.c.n_pages);
        w.mask = uint32_t(__ballot(there));
        if (!there) w.le = w.lr = 0;
      }
    };
    // the place of token `tok` where each lane looks up one
    const auto lane_at = [&](const Where& w, int tok) {
      return w.at[0] + int64_t(__shfl(w.le, tok, 64)) * a.c.page + int64_t(__shfl(w.lr, tok, 64)) * a.c.row;
    };

    u4 kr[X][LN];
    float ksc[NG][8], vsc[NG][8];
    const auto load_keys = [&](const Where& w) {
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const uint8_t* p = a.c.k + (PAGES16 ? w.at[x / HP] + uint64_t(uint32_t(x % HP * 8)) * uint32_t(a.c.row)
                                            : lane_at(w, x * (16 / HP) + i16 / HP));
#pragma unroll
        for (int ln = 0; ln < LN; ++ln) kr[x][ln] = fetch<C::FULL, u4>(p + key_offset(ln));
      }
    };
    // scales of a lane's eight tokens
    const auto load_scales = [&](const Where& w, const float* of, float (&sc)[NG][8]) {
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const float* p = of + int64_t(c) * a.c.s_group;
          if (C::PAGES == kHalvesWide) {
            typedef float fper __attribute__((ext_vector_type(PER)));
            const fper v = *reinterpret_cast<const fper*>(p + w.s_at[x / HP] + x % HP * 8 + PER * g);
#pragma unroll
            for (int r = 0; r < PER; ++r) sc[c][x * PER + r] = v[r];
          } else if (PAGES16) {
#pragma unroll
            for (int r = 0; r < PER; ++r)
              sc[c][x * PER + r] = (p + w.s_at[x / HP])[uint32_t(x % HP * 8 + PER * g + r) * uint32_t(a.c.s_row)];
          } else {
#pragma unroll
            for (int r = 0; r < PER; ++r) {
              const int tok = token(x * PER + r) + PER * g;
              sc[c][x * PER + r] = p[w.s_at[0] + int64_t(__shfl(w.le, tok, 64)) * a.c.s_page + int64_t(__shfl(w.lr, tok, 64)) * a.c.s_row];
            }
          }
        }
    };
    constexpr int VW = E4M3 ? 2 : 4;
    typedef uint32_t vw __attribute__((ext_vector_type(VW)));
    vw vr[NG][8];
    const auto load_values = [&](const Where& w) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint8_t* p = a.c.v + (PAGES16 ? w.at[token(e) / 16] + uint64_t(uint32_t(token(e) % 16)) * uint32_t(a.c.row)
                                            : lane_at(w, token(e) + PER * g));
#pragma unroll
        for (int c = 0; c < NG; ++c) vr[c][e] = fetch<C::FULL, vw>(p + value_offset(c));
      }
    };


    int pos = ((first + j) << a.tile_shift) + wave * kWaveTokens;
    Where w;
    Entries ahead;
    Queries<C> queries;
    if (pos < stop) ahead = entries(pos);
    queries.begin(a, b, head0, rows);
    if (pos < stop) {
      locate(pos, ahead, w);
      if (E4M3) load_scales(w, a.c.k_scale, ksc);
      load_keys(w);
      if (E4M3) load_scales(w, a.c.v_scale, vsc);
      load_values(w);
      ahead = entries(pos + tile_tokens);
    }
    v8bf qf[QS][QT];
    queries.end(a, rows, qf);
    f4 o[NG][8];
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
      for (int x = 0; x < 8; ++x) o[c][x] = f4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    // one tile's products and, behind the registers' last use, the next one's loads
    const auto tile = [&](auto loads) {
      constexpr bool LOADS = decltype(loads)::value;
      const uint32_t mask = w.mask;
      if (LOADS) {
        locate(pos + tile_tokens, ahead, w);
        ahead = entries(pos + 2 * tile_tokens);
      }

      // ---- logits of 8 tokens and one head per lane.  Each operand meets the queries of either half;
      // of the rows that are tokens' first halves the one sum counts, of the second ones the other
      float s[8];
#pragma unroll
      for (int x = 0; x < X; ++x) {
        f4 acc[HP][NG], small[HP][NG];   // (an F32 query's lower terms by themselves: a third of the roundings of the sum)
#pragma unroll
        for (int hh = 0; hh < HP; ++hh)
#pragma unroll
          for (int c = 0; c < NG; ++c) acc[hh][c] = small[hh][c] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ln = 0; ln < LN; ++ln) {
          constexpr int PARTS = E4M3 ? 2 : 1;
          const int c = E4M3 ? ln * 64 * HP / 128 : 0;
#pragma unroll
          for (int y = 0; y < PARTS; ++y) {
            const v8bf kf = E4M3 ? decode8(kr[x][ln][2 * y], kr[x][ln][2 * y + 1]) : as_bf16(kr[x][ln]);
#pragma unroll
            for (int hh = 0; hh < HP; ++hh) {
              const int piece = (ln * HP + hh) * PARTS + y;
              acc[hh][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[piece][0], acc[hh][c], 0, 0, 0);
#pragma unroll
              for (int q = 1; q < QT; ++q)
                small[hh][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[piece][q], small[hh][c], 0, 0, 0);
            }
          }
        }
        if (QT > 1) {
#pragma unroll
          for (int hh = 0; hh < HP; ++hh)
#pragma unroll
            for (int c = 0; c < NG; ++c) acc[hh][c] += small[hh][c];
        }
#pragma unroll
        for (int r = 0; r < PER; ++r) {
          const auto sum = [&](int c) { return HP == 1 ? acc[0][c][r] : acc[0][c][(2 * r) & 3] + acc[HP - 1][c][(2 * r + 1) & 3]; };
          float v = sum(0);
          if (E4M3) {
            v *= ksc[0][x * PER + r];
            if (NG == 2) v = fmaf(sum(NG - 1), ksc[NG - 1][x * PER + r], v);
          }
          s[x * PER + r] = v;
        }
      }
      if (LOADS) {
        if (E4M3) load_scales(w, a.c.k_scale, ksc);
        load_keys(w);
      }
      if (mask != ~0u) {
        const uint32_t mine = mask >> (PER * g);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((mine >> token(e)) & 1)) s[e] = -INFINITY;
      }

      // ---- running maximum and sum, of logits that are not scaled yet: a difference of two
      // that matter is exact, and its scaling rounds it relative to the difference
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
      top = fmaxf(m, max_of_groups(top));
      if (__ballot(top > m)) {
        const float f = top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - top) * a.scale);
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
        p[e] = __builtin_amdgcn_exp2f((s[e] - ref) * a.scale);
        l += p[e];
      }

      // ---- values: rows of tokens that do not exist may hold anything
      if (mask != ~0u) {
        const uint32_t mine = mask >> (PER * g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool there = (mine >> token(e)) & 1;
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            if (E4M3 && !there) vsc[c][e] = 0.f;
#pragma unroll
            for (int x = 0; x < VW; ++x) vr[c][e][x] = there ? vr[c][e][x] : 0u;
          }
        }
      }
      v8bf pt[E4M3 ? NG : 1][PT];
      if (E4M3) {
#pragma unroll
        for (int c = 0; c < NG; ++c) {
          float ps[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) ps[e] = p[e] * vsc[c][e];
          split<PT>(ps, pt[c]);
        }
      } else {
        split<PT>(p, pt[0]);
      }
#pragma unroll
      for (int c = 0; c < NG; ++c) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {   // channels 2 x and 2 x + 1 of each lane's eight
          u4 lo, hi;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (E4M3) {
              // both tokens' bytes of the two channels side by side, then two conversions
              const uint32_t both = __builtin_amdgcn_perm(vr[c][2 * e + 1][x >> 1], vr[c][2 * e][x >> 1],
                                                          (x & 1) ? 0x07030602u : 0x05010400u);
              lo[e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(both, 1.0f, false));
              hi[e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(both, 1.0f, true));
            } else {
              lo[e] = __builtin_amdgcn_perm(vr[c][2 * e + 1][x % VW], vr[c][2 * e][x % VW], 0x05040100u);
              hi[e] = __builtin_amdgcn_perm(vr[c][2 * e + 1][x % VW], vr[c][2 * e][x % VW], 0x07060302u);
            }
          }
#pragma unroll
          for (int q = 0; q < PT; ++q) {
            o[c][2 * x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(lo), pt[E4M3 ? c : 0][q], o[c][2 * x], 0, 0, 0);
            o[c][2 * x + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(hi), pt[E4M3 ? c : 0][q], o[c][2 * x + 1], 0, 0, 0);
          }
        }
      }
      if (LOADS) {
        if (E4M3) load_scales(w, a.c.v_scale, vsc);
        load_values(w);
      }
    };
    for (; pos + tile_tokens < stop; pos += tile_tokens) tile(std::true_type{});
    if (pos < stop) tile(std::false_type{});

    // ---- the waves' parts of the segment: maxima, then sums brought to the common one
    l = sum_of_groups(l);
    if (g == 0) lds_m[wave][i16] = m;
    __syncthreads();
    float top = lds_m[0][i16];
    for (int y = 0; y < waves; y += 4)
#pragma unroll
      for (int x = 0; x < 4; ++x) top = fmaxf(top, lds_m[y + x][i16]);
    const float mine = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - top) * a.scale);
    if (g == 0) lds_l[wave][i16] = l * mine;
    if (i16 < rows) {
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            f4 v;
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = o[c][4 * y + x][r] * mine;
            *reinterpret_cast<f4*>(&lds_o[(wave * kRows + i16) * PITCH + c * 128 + (4 * g + r) * 8 + 4 * y]) = v;
          }
    }
    __syncthreads();
    const bool whole = j == 0 && j_end == n_tiles;
    const int slot = int(blockIdx.x) * 2 + (t == t_begin ? 0 : 1);
    if (a.tasks && threadIdx.x == 0 && (a.by_item ? j == 0 : t + j_end - j == t_end)) {
      Task* task = a.tasks + (a.by_item ? b * a.items + h * a.row_tiles + row0 / kRows : int(blockIdx.x));
      const bool begins = j == 0 && !whole;
      task->b = b;
      task->head0 = head0;
      task->rows = begins ? rows : 0;
      task->slot = slot;
      task->to = begins ? ranges.block_of(t + n_tiles - 1) : 0;
    }
    float* part = a.part + int64_t(slot) * C::SLOT;
    for (int x = threadIdx.x; x < kRows * (C::CHANNELS / 4); x += int(blockDim.x)) {
      const int row = x / (C::CHANNELS / 4), ch = 4 * (x % (C::CHANNELS / 4));
      if (row >= rows || ch >= D) continue;
      f4 v = f4{0.f, 0.f, 0.f, 0.f};
      float all_m = -INFINITY, all_l = 0.f;
      for (int y = 0; y < waves; y += 4)
#pragma unroll
        for (int z = y; z < y + 4; ++z) {
          v += *reinterpret_cast<const f4*>(&lds_o[(z * kRows + row) * PITCH + ch]);
          all_m = fmaxf(all_m, lds_m[z][row]);
          all_l += lds_l[z][row];
        }
      if (whole) {
        store_result(a, b, head0 + row, ch, v, all_m, all_l);
      } else {
        *reinterpret_cast<f4*>(part + row * C::CHANNELS + ch) = v;
        if (ch == 0) {
          part[kRows * C::CHANNELS + row] = all_m;
          part[kRows * C::CHANNELS + kRows + row] = all_l;
        }
      }
    }
    __syncthreads();

    t += j_end - j;
    j = 0;
    if ((row0 += kRows) >= a.G) {
      row0 = 0;
      ++h;
    }
    if (h == a.c.heads && t < t_end) {
      h = 0;
      if (++b == base + 64) {
        base = b;
        seq = lengths_of(a, base);
      }
      n = __builtin_amdgcn_readlane(seq.n, b - base);
      n_tiles = tiles_of(a, n, first);
    }
  }
}

// Adds the parts of the items that lie in more than one block, a query head per block of this
// kernel: groups of lanes take every so many parts, with a maximum of their own.
// Bound by latency: the note, then the parts, then the groups' sums.  64 sequences of 40 heads
// take 6 us, 32 heads of hundreds of parts each 5 with 1024 threads.
template <int DIM, int THREADS>
__global__ __launch_bounds__(THREADS) void attention_join_kernel(AttentionDev a) {
  using C = Config<false, DIM, false, 1, 2, kAny>;   // (a slot has one size for both types of cache)
  constexpr int LANES = C::CHANNELS / 4, GROUPS = THREADS / LANES, FLIGHT = 8;
  __shared__ float lds_o[GROUPS][C::CHANNELS], lds_m[GROUPS], lds_l[GROUPS];
  const Task task = a.tasks[blockIdx.x];
  const int row = int(blockIdx.y);
  if (row >= task.rows) return;
  const int from = task.slot >> 1, to = task.to;
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
      const float* p = a.part + int64_t(blk == from ? task.slot : 2 * blk) * C::SLOT;
      v[y] = on ? *reinterpret_cast<const f4*>(p + row * C::CHANNELS + ch) : f4{0.f, 0.f, 0.f, 0.f};
      pm[y] = p[kRows * C::CHANNELS + row];
      pl[y] = p[kRows * C::CHANNELS + kRows + row];
    }
#pragma unroll
    for (int y = 1; y < FLIGHT; ++y)
      if (x + y * GROUPS > to) {   // (read again, not counted again)
        pm[y] = -INFINITY;
        pl[y] = 0.f;
        v[y] = f4{0.f, 0.f, 0.f, 0.f};
      }
    float top = m;
#pragma unroll
    for (int y = 0; y < FLIGHT; ++y) top = fmaxf(top, pm[y]);
    const float ref = top == -INFINITY ? 0.f : top;   // (parts without a token count nothing, and those of NaN NaN)
    float f = __builtin_amdgcn_exp2f((m - ref) * a.scale);
    l *= f;
    o *= f;
#pragma unroll
    for (int y = 0; y < FLIGHT; ++y) {
      f = __builtin_amdgcn_exp2f((pm[y] - ref) * a.scale);
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
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int y = 0; y < GROUPS; ++y) {
    const float f = __builtin_amdgcn_exp2f((lds_m[y] - ref) * a.scale);
    sum = fmaf(lds_l[y], f, sum);
    v += *reinterpret_cast<const f4*>(&lds_o[y][ch]) * f;
  }
  store_result(a, task.b, task.head0 + row, ch, v, top, sum);
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

// How a call is cut up, from what the host knows.
struct Plan {
  int64_t items;     // of the batch
  int64_t blocks;
  int32_t whole, waves;
};
Plan plan_of(const CacheDev& c, int64_t B, int32_t q_heads, int64_t bound, bool f32) {
  Plan p{};
  p.items = B * c.heads * ((q_heads / c.heads + kRows - 1) / kRows);
  const int64_t held = compute_units() * waves_per_simd(c.head_dim, f32);   // blocks of four waves that run at once
  p.waves = 4;
  const int64_t tiles = bound / (p.waves * kWaveTokens) + 1;
  // A block per item where the longest is short (one sequence of 200 tokens 13.4 -> 10.0 us, with
  // eight waves) or where so many items follow each other on a compute unit that they even out (8
  // key heads: 256 sequences to 1000 88 -> 77 us, to 2000 149 -> 146, but to 4000 260 -> 282; 64 to
  // 1000 29.0 -> 29.7, to 2000 44 -> 54; 24 key heads of 80, 256 to 1000 165 -> 124).  These lengths grow
  // as a square; the host knows the table's width alone, so other batches pay for it where one block's item
  // is far longer than the rest: 256 sequences of 24 key heads under a table of 8000, one of them of 7999 and the
  // others of 200, 103.5 -> 110, eight of 7999 187 -> 209, all of 700 244 -> 233.
  p.whole = bound <= kWholeTokens || tiles * held <= 8 * p.items ? 1 : 0;
  if (p.whole) {
    p.blocks = p.items;
    if (2 * p.items < held && tiles > 1) p.waves = most_waves(c.head_dim, f32);
    return p;
  }
  const int64_t most = p.items * (tiles + 1);
  p.blocks = most < held ? most : held;
  return p;
}

template <bool E4M3, int DIM, bool FULL, int QT, int PT>
void launch_pages(const AttentionDev& a, bool scale_vec, hipStream_t stream) {
  using Any = Config<E4M3, DIM, FULL, QT, PT, kAny>;
  const int waves = 1 << (a.tile_shift - 5);
  const dim3 grid{unsigned(a.blocks)}, block{unsigned(64 * waves)};
  const unsigned lds = unsigned(waves * kRows * Any::PITCH * sizeof(float));
  if (a.c.page_size % 16)
    hipLaunchKernelGGL((attention_kernel<Any>), grid, block, lds, stream, a);
  else if (!E4M3 || scale_vec)   // (BF16: no scales)
    hipLaunchKernelGGL((attention_kernel<Config<E4M3, DIM, FULL, QT, PT, kHalvesWide>>), grid, block, lds, stream, a);
  else if constexpr (E4M3)
    hipLaunchKernelGGL((attention_kernel<Config<E4M3, DIM, FULL, QT, PT, kHalves>>), grid, block, lds, stream, a);
}
template <bool E4M3>
void launch_dims(const AttentionDev& a, bool f32, bool scale_vec, hipStream_t stream) {
  const int D = a.c.head_dim;
  if (f32 && D > 128) launch_pages<E4M3, 256, false, 3, 3>(a, scale_vec, stream);
  else if (f32) launch_pages<E4M3, 128, false, 3, 3>(a, scale_vec, stream);
  else if (D == 64) launch_pages<E4M3, 64, true, 1, 2>(a, scale_vec, stream);
  else if (D == 128) launch_pages<E4M3, 128, true, 1, 2>(a, scale_vec, stream);
  else if (D == 256) launch_pages<E4M3, 256, true, 1, 2>(a, scale_vec, stream);
  else if (D > 128) launch_pages<E4M3, 256, false, 1, 2>(a, scale_vec, stream);
  else launch_pages<E4M3, 128, false, 1, 2>(a, scale_vec, stream);
}

}  // namespace

int64_t attention_tiles(const CacheDev& c, int64_t B, int32_t q_heads, int64_t bound) {
  return B * c.heads * ((q_heads / c.heads + kRows - 1) / kRows) * (bound / (4 * kWaveTokens) + 2);
}

size_t attention_workspace_bytes(const CacheDev& c, int64_t B, int32_t q_heads, int64_t bound) {
  const Plan p = plan_of(c, B, q_heads, bound, false);   // (F32 calls have fewer blocks, or none to join, not more)
  return p.whole ? 0 : size_t(p.blocks) * (2 * slot_floats(c.head_dim) * sizeof(float) + sizeof(Task));
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
  const bool scale_vec = c.s_row == 1 && ((c.s_page | c.s_head | c.s_group) & 3) == 0 &&
                         ((reinterpret_cast<uintptr_t>(c.k_scale) | reinterpret_cast<uintptr_t>(c.v_scale)) & 15) == 0;
  const bool f32 = !q.bf16 || !out.bf16;
  const Plan plan = plan_of(c, B, q.heads, a.bound, f32);
  a.blocks = int32_t(plan.blocks);
  a.whole = plan.whole;
  a.tile_shift = plan.waves == 8 ? 8 : 7;
  if (!plan.whole) {
    a.tasks = reinterpret_cast<Task*>(a.part + size_t(a.blocks) * 2 * slot_floats(c.head_dim));
    a.by_item = plan.items <= a.blocks ? 1 : 0;
  }
  a.negative = scale < 0.0 ? 1 : 0;
  a.natural = scale < 0.0 ? -scale : scale;
  constexpr double kLog2e = 1.4426950408889634;
  // A scale below 2^-100 makes logits of products so large that their differences leave F32: queries
  // 2^64 times smaller under a scale as much larger are the same logits.  (A query's bits below 2^-126
  // of F32 go, 2^8 channels times 2^-126 times keys up to 2^128 times the scale's 2^-36: 2^-26 of a
  // logit at most.)  Below 2^-126 then, zero among them, differences of up to 2^65 leave all weights 1.
  a.small = a.natural * kLog2e < 0x1p-100 ? 1 : 0;
  if (a.small) a.natural *= 0x1p64;
  a.scale = float(a.natural * kLog2e);
  if (!(a.scale > FLT_MIN)) a.scale = FLT_MIN;   // (-inf times it stays -inf)
  if (a.scale > FLT_MAX) a.scale = FLT_MAX;      // (the largest logit's weight is 1 there, and 0 times it stays 0)
  if (c.e4m3) launch_dims<true>(a, f32, scale_vec, stream);
  else launch_dims<false>(a, f32, scale_vec, stream);
  bsf8_status st = device_status(hipGetLastError(), "paged_attention launch");
  if (st != BSF8_OK || plan.whole) return st;
  const unsigned rows = unsigned(a.G < kRows ? a.G : kRows);
  const dim3 grid(unsigned(a.by_item ? plan.items : plan.blocks), rows);
  // hundreds of parts to an item: all of them in flight at once
  const bool many = plan.blocks > 32 * plan.items;
  if (c.head_dim > 128) {
    if (many) hipLaunchKernelGGL((attention_join_kernel<256, 1024>), grid, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((attention_join_kernel<256, 256>), grid, dim3(256), 0, stream, a);
  } else {
    if (many) hipLaunchKernelGGL((attention_join_kernel<128, 1024>), grid, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((attention_join_kernel<128, 256>), grid, dim3(256), 0, stream, a);
  }
  return device_status(hipGetLastError(), "paged_attention join launch");
}

}  // namespace bsf8
