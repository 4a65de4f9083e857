// W8A8 products of few rows: the projection with an epilogue at few tokens, and
// the experts' products, whose rows come in ragged runs.
//
// As in the tile GEMM, 16 weight rows are an MFMA's A operand and 16 rows of
// codes its B operand, and the sum over one 128-wide scale block is scaled by
// (activation scale x weight scale) in F32.  The sum is four
// v_mfma_f32_16x16x32_bf16 on codes decoded to BF16, which is exact: the FP8
// instruction adds its products in fewer bits than F32 holds (measured on random
// codes: 5.1e-5 of the result's norm, up to 2^-12 of the sum of magnitudes,
// against 7.7e-8 and 2^-22), and here, where the weight's bytes set the time,
// twice the matrix instructions cost nothing.
//
// A block takes 16 RT weight rows and up to 16 TJ rows of codes; its waves take K
// blocks wave, wave + WAVES, ..., each on its own, and their partial tiles are
// added through LDS in wave order, so results do not depend on timing.  Eight
// lanes load one row's 128 bytes of a K block: what bounds the kernel is the
// weight's bytes, and the memory system streams whole 128-byte lines of few rows
// faster than the fragments' own layout (16 bytes of each of 16 rows, four lanes
// to 64 bytes).  The rows pass through the wave's own part of LDS into the
// fragments' layout, without a barrier; the next K block's loads go out as soon
// as the registers of this one are in LDS, before its arithmetic.  Sixteen waves
// of a compute unit then have 96 KiB in flight (up to 16 rows of codes; 114 registers).
//
// W [5120, 5120] with bias and residual takes 7.8 / 9.7 / 16.3 / 17.6 us at 1 / 16 / 48
// / 64 tokens (26 MB: 3.4 TB/s at one token, launch and ramp included; fragments
// loaded straight into registers took 11.4 us); 8 of 64 experts [1536, 2048] at one
// token 9.3 us.  Four waves where K has at most 16 blocks, eight beyond: 4 tokens
// of 8 of 64 experts at K = 2048 12.4 against 17.2 us, [5120, 17408] at one token 28.7
// against 18.7 us.
//
// Experts: the row runs lie in device memory, so every wave finds the (expert,
// run of 16 TJ rows) of its block itself: 64 experts' runs are counted at a time
// and summed across the lanes.  The grid covers the most runs that R rows of E
// experts can make, min(E, R) + R / (16 TJ); blocks past the last run leave at
// once.  Offsets are clamped to [0, R] and a gather row outside the tokens reads
// as zeros, so nothing in device memory can lead an access out of bounds.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <string>

#include "bsf8_fused.h"

namespace bsf8 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef u4v __attribute__((aligned(1))) u4v_any;   // (the hardware loads 16 bytes from any address)

constexpr int KB = 128;

struct RowsArgs {
  WeightDev w;                      // expert 0's members
  EpilogueDev ep;
  int32_t rt0[kMaxMembers + 1];     // first row tile (16 RT rows) of each member
  const int32_t* offsets;           // experts: their row runs; null: one weight, all rows
  const int32_t* rows;              // gather: the token of each row, or null
  const uint8_t* xq;
  const float* xs;
  void* y;
  int64_t ldq, xs_sm, xs_sk, ldy;
  int32_t M;                        // tokens (rows of xq)
  int32_t R;                        // rows of y
  int32_t E;
  int32_t y_bf16;
};

__device__ __forceinline__ void blank(uint4& v, bool all) {
  v.x = all ? 0u : v.x;
  v.y = all ? 0u : v.y;
  v.z = all ? 0u : v.z;
  v.w = all ? 0u : v.w;
}

// How a row's 16-byte pieces are read.
enum Access {
  kAligned,     // K and every row a multiple of 16
  kUnaligned,   // K >= 16: loads at any byte address, the last piece ending at K
  kBytes        // K < 16
};

// 16 bytes at p + k of a row of K bytes; a piece that does not lie in the row is
// read as the row's last 16 bytes and put right by clip().
template <Access ACCESS, bool NT>
__device__ __forceinline__ uint4 load_piece(const uint8_t* p, int k, int K) {
  if constexpr (ACCESS == kAligned) {
    const u4v* q = reinterpret_cast<const u4v*>(p + min(k, K - 16));
    const u4v v = NT ? __builtin_nontemporal_load(q) : *q;
    return make_uint4(v.x, v.y, v.z, v.w);
  } else if constexpr (ACCESS == kUnaligned) {
    const u4v v = *reinterpret_cast<const u4v_any*>(p + min(k, K - 16));
    return make_uint4(v.x, v.y, v.z, v.w);
  } else {
    uint32_t b[4] = {0, 0, 0, 0};
    for (int i = 0; i < K; ++i)
      if (k == 0) b[i >> 2] |= uint32_t(p[i]) << (8 * (i & 3));
    return make_uint4(b[0], b[1], b[2], b[3]);
  }
}
// The piece at k of what load_piece read: bytes past K become zeros.
template <Access ACCESS>
__device__ __forceinline__ void clip(uint4& v, int k, int K) {
  if constexpr (ACCESS == kAligned) {
    blank(v, k >= K);
  } else if constexpr (ACCESS == kUnaligned) {
    const int d = k - min(k, K - 16);   // the piece starts d bytes into what was read
    const int s = 8 * (d & 7);
    uint64_t lo = uint64_t(v.x) | uint64_t(v.y) << 32, hi = uint64_t(v.z) | uint64_t(v.w) << 32;
    if (d & 8) {
      lo = hi;
      hi = 0;
    }
    if (s) {
      lo = lo >> s | hi << (64 - s);
      hi >>= s;
    }
    v = make_uint4(uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32));
    blank(v, d >= 16);
  }
}

// a lane's 32 codes of a K block as the four steps' operands
struct Operand {
  v8bf s[4];
};
__device__ __forceinline__ Operand operand(const uint4 (&p)[2]) {
  return Operand{{decode8(p[0].x, p[0].y), decode8(p[0].z, p[0].w), decode8(p[1].x, p[1].y), decode8(p[1].z, p[1].w)}};
}

// A wave's LDS: its 16 RT weight rows and 16 TJ rows of codes of one K block.
template <int RT, int TJ>
constexpr int wave_lds() { return (RT + TJ) * 16 * KB; }

// 16-byte piece p of row r sits at piece p ^ s(r), s a permutation of r & 7 that
// sends even rows to {0, 1, 4, 5} and odd rows to {2, 3, 6, 7}: a fragment read's
// 16 rows over two lane groups then hit all 64 banks once.
__device__ __forceinline__ int at_piece(int row, int p) {
  return row * KB + ((p ^ (((row & 1) << 1) | ((row >> 1) & 1) | (row & 4))) << 4);
}

// One block's tile: 16 RT weight rows from n0 of member `mem`, rows [first, end)
// of codes, which fill TJ column tiles.  No branch around a load: the compiler
// would wait for all of them there.  The loads issued in the last round repeat
// the last K block and are not used.
template <int WAVES, int RT, int TJ, Access ACCESS, bool KFULL, bool SBF16>
__device__ __forceinline__ void tile(const RowsArgs& a, const MemberDev& mem, int expert, int n0, int first, int end,
                                     uint8_t* lds) {
  constexpr int THREADS = WAVES * 64;
  const int K = a.w.K, Kb = a.w.Kb;
  const int nb = (mem.rows + 127) >> 7;
  const uint8_t* wbase = mem.w + int64_t(expert) * mem.rows * K;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int lr = lane >> 3, lp = lane & 7;   // row and piece of a load: 8 lanes read one row's 128 bytes
  uint8_t* const wl = lds + wave * wave_lds<RT, TJ>();
  uint8_t* const xl = wl + RT * 16 * KB;

  // rows past the member's end repeat its last one and are not stored; rows past
  // the run repeat its first, and rows without a token read token 0
  const uint8_t* wrow[2 * RT];
#pragma unroll
  for (int q = 0; q < 2 * RT; ++q) wrow[q] = wbase + int64_t(min(n0 + 8 * q + lr, mem.rows - 1)) * K;
  auto token = [&](int i) {
    const int r = first + i < end ? first + i : first;
    const int tok = a.rows ? a.rows[r] : r;
    return tok < 0 || tok >= a.M ? 0 : tok;
  };
  const uint8_t* xrow[2 * TJ];
#pragma unroll
  for (int q = 0; q < 2 * TJ; ++q) xrow[q] = a.xq + int64_t(token(8 * q + lr)) * a.ldq;
  const float* srow[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) srow[j] = a.xs + int64_t(token(16 * j + l16)) * a.xs_sm;
  // the scale row of the row tiles (16 RT divides 128, so they lie in one)
  const int64_t s_off = (a.w.s_rs ? int64_t(expert) * nb * Kb : 0) + int64_t(n0 >> 7) * a.w.s_rs;

  v4f acc[RT][TJ];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // What the store needs besides the sums is loaded before everything else, so
  // that no memory latency follows the last sum: thread tid finishes outputs o =
  // tid + THREADS u, row o % (16 RT) of the weight tile, row o / (16 RT) of codes.
  constexpr int OUT = (RT * TJ * 256 + THREADS - 1) / THREADS;
  // (Raw bits, widened at their use: a conversion here would wait for the load.)
  uint32_t bias[OUT], res[OUT];
  int out_tok[OUT];
#pragma unroll
  for (int u = 0; u < OUT; ++u) {
    const int o = tid + THREADS * u;
    const int n = min(n0 + o % (16 * RT), mem.rows - 1), r = min(first + o / (16 * RT), end - 1);
    bias[u] = a.ep.bias ? load_bits(a.ep.bias, a.ep.bias_bf16, mem.col0 + n) : 0;
    res[u] = a.ep.res ? load_bits(a.ep.res, a.ep.res_bf16, int64_t(r) * a.ep.ldr + mem.col0 + n) : 0;
    out_tok[u] = a.rows ? a.rows[r] : 0;
  }
  __builtin_amdgcn_sched_barrier(0);

  uint4 wr[2 * RT], xr[2 * TJ];
  float sa[TJ];
  // The weight scales of the wave's K blocks, one per lane: block wave + WAVES
  // (64 h + lane) for h-th 64 rounds.
  uint32_t swr = 0;
  auto load_scales = [&](int h) {
    const int c = min(wave + WAVES * (64 * h + lane), Kb - 1);
    swr = load_bits(mem.s, SBF16, s_off + int64_t(c) * a.w.s_cs);
  };
  load_scales(0);
  __builtin_amdgcn_sched_barrier(0);
  auto issue = [&](int c) __attribute__((always_inline)) {
    const int cc = min(c, Kb - 1);
    const int k = cc * KB + 16 * lp;
#pragma unroll
    for (int j = 0; j < TJ; ++j) sa[j] = srow[j][int64_t(cc) * a.xs_sk];
#pragma unroll
    for (int q = 0; q < 2 * TJ; ++q) xr[q] = load_piece<ACCESS, false>(xrow[q], k, K);
#pragma unroll
    for (int q = 0; q < 2 * RT; ++q) wr[q] = load_piece<ACCESS, true>(wrow[q], k, K);
  };
  issue(wave);
  __builtin_amdgcn_sched_barrier(0);
  int round = 0;
  for (int c = wave; c < Kb; c += WAVES, ++round) {
    if (round == 64) {   // (K beyond 65536)
      load_scales(c / (WAVES * 64));
      round = 0;
    }
    const float sw = widen(__builtin_amdgcn_readlane(swr, round), SBF16);
    // bytes past K: zeros on both sides (a NaN code times zero is NaN)
    if (!KFULL && ACCESS != kBytes && c == Kb - 1) {
      const int k = c * KB + 16 * lp;
#pragma unroll
      for (int q = 0; q < 2 * RT; ++q) clip<ACCESS>(wr[q], k, K);
#pragma unroll
      for (int q = 0; q < 2 * TJ; ++q) clip<ACCESS>(xr[q], k, K);
    }
#pragma unroll
    for (int q = 0; q < 2 * RT; ++q) *reinterpret_cast<uint4*>(wl + at_piece(8 * q + lr, lp)) = wr[q];
#pragma unroll
    for (int q = 0; q < 2 * TJ; ++q) *reinterpret_cast<uint4*>(xl + at_piece(8 * q + lr, lp)) = xr[q];
    float s[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) s[j] = sa[j] * sw;
    // the registers are free: the next loads go out before this block's arithmetic
    __builtin_amdgcn_sched_barrier(0);
    issue(c + WAVES);
    __builtin_amdgcn_sched_barrier(0);
    auto fragment = [&](const uint8_t* base, int row) {
      const uint4 p[2] = {*reinterpret_cast<const uint4*>(base + at_piece(row, 2 * g)),
                          *reinterpret_cast<const uint4*>(base + at_piece(row, 2 * g + 1))};
      return operand(p);
    };
    Operand w[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) w[i] = fragment(wl, 16 * i + l16);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const Operand x = fragment(xl, 16 * j + l16);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        v4f p = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i].s[q], x.s[q], p, 0, 0, 0);
        acc[i][j] += p * s[j];
      }
    }
  }

  // ---- the waves' partial tiles in wave order, the epilogue, the store
  float(*red)[RT * TJ][64][4] = reinterpret_cast<float(*)[RT * TJ][64][4]>(lds);
  static_assert(RT * TJ * 1024 <= wave_lds<RT, TJ>(), "partial tiles fit the waves' LDS");
  __syncthreads();   // every wave is done with its rows
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) *reinterpret_cast<v4f*>(&red[wave][i * TJ + j][lane][0]) = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < OUT; ++u) {
    const int o = tid + THREADS * u;
    const int row = o % (16 * RT), col = o / (16 * RT);
    const int n = n0 + row, r = first + col;
    if (o >= RT * TJ * 256 || n >= mem.rows || r >= end) continue;
    const int t = (row >> 4) * TJ + (col >> 4), ln = 16 * ((row & 15) >> 2) + (col & 15);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) v += red[q][t][ln][row & 3];
    if (out_tok[u] < 0 || out_tok[u] >= a.M) v = 0.f;
    v = activate(v + widen(bias[u], a.ep.bias_bf16), a.ep.act);
    if (a.ep.res) v = fmaf(a.ep.alpha, widen(res[u], a.ep.res_bf16), v);
    const int64_t at = int64_t(r) * a.ldy + mem.col0 + n;
    if (a.y_bf16)
      static_cast<__bf16*>(a.y)[at] = static_cast<__bf16>(v);
    else
      static_cast<float*>(a.y)[at] = v;
  }
}

// Up to TJ column tiles; a block runs the code of as many as its rows fill.
template <int WAVES, int RT, int TJ, Access ACCESS, bool KFULL, bool SBF16>
__global__ __launch_bounds__(WAVES * 64) void w8a8_rows_kernel(RowsArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * wave_lds<RT, TJ>()];
  const int rt_total = a.rt0[a.w.n_members];
  const int item = blockIdx.x / rt_total;
  int R_tile = blockIdx.x - item * rt_total, expert = 0, first = item * 16 * TJ, end = a.R;
  if (a.offsets != nullptr) {
    // an expert's runs of one weight tile follow each other
    int lo, tiles, before;
    expert = find_run(a.offsets, a.E, a.R, 16 * TJ, runs_of(a.offsets, a.E, a.R, 16 * TJ, 0), item, lo, end, tiles, before);
    if (expert < 0) return;
    const int u = blockIdx.x - before * rt_total;
    R_tile = u / tiles;
    first = lo + (u - R_tile * tiles) * 16 * TJ;
  }
  end = min(end, first + 16 * TJ);
  int mi = 0;
  while (mi + 1 < a.w.n_members && R_tile >= a.rt0[mi + 1]) ++mi;
  const MemberDev mem = a.w.m[mi];
  const int n0 = (R_tile - a.rt0[mi]) * 16 * RT;
  const int tiles = (end - first + 15) / 16;
  if (TJ == 1 || tiles == 1)
    tile<WAVES, RT, 1, ACCESS, KFULL, SBF16>(a, mem, expert, n0, first, end, lds);
  else if (TJ == 2 || tiles == 2)
    tile<WAVES, RT, TJ < 2 ? TJ : 2, ACCESS, KFULL, SBF16>(a, mem, expert, n0, first, end, lds);
  else
    tile<WAVES, RT, TJ, ACCESS, KFULL, SBF16>(a, mem, expert, n0, first, end, lds);
}

template <int WAVES, int RT, int TJ, bool SBF16>
auto pick(bool aligned, int K) -> void (*)(RowsArgs) {
  const bool kfull = K % KB == 0;
  if (aligned)
    return kfull ? w8a8_rows_kernel<WAVES, RT, TJ, kAligned, true, SBF16> : w8a8_rows_kernel<WAVES, RT, TJ, kAligned, false, SBF16>;
  if constexpr (WAVES == 4)
    if (K < 16) return w8a8_rows_kernel<WAVES, RT, TJ, kBytes, false, SBF16>;
  // (any K: unaligned rows with K a multiple of 128 take it too)
  return w8a8_rows_kernel<WAVES, RT, TJ, kUnaligned, false, SBF16>;
}

template <int WAVES, int RT, int TJ>
bsf8_status launch(const RowsArgs& base, bool aligned, int64_t items, hipStream_t stream) {
  RowsArgs a = base;
  int r = 0;
  for (int i = 0; i < kMaxMembers; ++i) {
    a.rt0[i] = r;
    if (i < a.w.n_members) r += (a.w.m[i].rows + 16 * RT - 1) / (16 * RT);
  }
  a.rt0[kMaxMembers] = r;
  const int64_t grid = items * r;
  if (grid * WAVES * 64 > UINT32_MAX) {
    set_error("UNSUPPORTED: %lld blocks", (long long)grid);
    return BSF8_E_UNSUPPORTED;
  }
  void (*kern)(RowsArgs) = a.w.scale_bf16 ? pick<WAVES, RT, TJ, true>(aligned, a.w.K) : pick<WAVES, RT, TJ, false>(aligned, a.w.K);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(WAVES * 64), 0, stream, a);
  return device_status(hipGetLastError(), "w8a8_rows launch");
}

// The kernel that takes R rows of E weights (E = 1: one weight).
bsf8_status launch_rows(const RowsArgs& a, bool aligned, hipStream_t stream) {
  const int64_t R = a.R, E = a.offsets ? a.E : 1;
  const auto items = [&](int64_t T) { return a.offsets ? std::min(E, R) + R / T : (R + T - 1) / T; };
  const bool few = R <= 16 * E, w4 = a.w.Kb <= 16;
  if (few) return w4 ? launch<4, 2, 1>(a, aligned, items(16), stream) : launch<8, 2, 1>(a, aligned, items(16), stream);
  return w4 ? launch<4, 2, 4>(a, aligned, items(64), stream) : launch<8, 2, 4>(a, aligned, items(64), stream);
}

}  // namespace

bsf8_status launch_w8a8_rows(const WeightDev& w, bool aligned, const uint8_t* xq, int64_t ldq, const float* xs,
                             int64_t xs_sm, int64_t xs_sk, int64_t M, const EpilogueDev& ep, void* y, bool y_bf16,
                             int64_t ldy, hipStream_t stream) {
  RowsArgs a{};
  a.w = w;
  a.ep = ep;
  a.xq = xq;
  a.xs = xs;
  a.y = y;
  a.ldq = ldq;
  a.xs_sm = xs_sm;
  a.xs_sk = xs_sk;
  a.ldy = ldy;
  a.M = int32_t(M);
  a.R = int32_t(M);
  a.y_bf16 = y_bf16;
  return launch_rows(a, aligned, stream);
}

bsf8_status launch_w8a8_expert_rows(const WeightDev& w, int64_t E, bool aligned, const uint8_t* xq, int64_t ldq,
                                const float* xs, int64_t xs_sm, int64_t xs_sk, int64_t M, const int32_t* offsets,
                                const int32_t* rows, int64_t R, void* y, bool y_bf16, int64_t ldy, hipStream_t stream) {
  RowsArgs a{};
  a.w = w;
  a.offsets = offsets;
  a.rows = rows;
  a.xq = xq;
  a.xs = xs;
  a.y = y;
  a.ldq = ldq;
  a.xs_sm = xs_sm;
  a.xs_sk = xs_sk;
  a.ldy = ldy;
  a.M = int32_t(M);
  a.R = int32_t(R);
  a.E = int32_t(E);
  a.y_bf16 = y_bf16;
  return launch_rows(a, aligned, stream);
}

std::string describe_w8a8_rows(bool few, bool aligned) {
  char buf[256];
  snprintf(buf, sizeof(buf), "arithmetic=e4m3 codes decoded exactly to bf16, mfma_f32_16x16x32_bf16, f32 per-128-K epilogue | "
           "kernel=w8a8_rows rows<=%d path=%s", few ? 16 : 64, aligned ? "aligned16" : "unaligned");
  return buf;
}

}  // namespace bsf8
