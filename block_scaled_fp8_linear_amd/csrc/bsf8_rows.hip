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
// Nothing goes through LDS on the way in: a lane's 32 bytes of a K block are two
// 16-byte loads straight into the registers that are decoded.  The sum over K
// does not care which K a register holds so long as both operands agree, so lane
// group g takes bytes [16 g, 16 g + 16) of each half of the block instead of [32
// g, 32 g + 32): four lanes then read 64 contiguous bytes per instruction.  The
// weight is what there is to read, and every byte of it is read once per 16 TJ
// rows of codes.
//
// A block takes 16 RT weight rows and up to 16 TJ rows of codes; its eight waves
// take K blocks wave, wave + 8, ... (neighbouring waves read neighbouring 128
// bytes of a row) with D blocks in flight each, and their partial tiles are
// added through LDS in wave order, so results do not depend on timing.
//
// Experts: the row runs lie in device memory, so every wave finds the (expert,
// run of 16 TJ rows) of its block itself: 64 experts' runs are counted at a time
// and summed across the lanes.  The grid covers the most runs that R rows of E
// experts can make, min(E, R) + R / (16 TJ); blocks past the last run leave at
// once.  Offsets are clamped to [0, R] and a gather row outside the tokens reads
// as zeros, so nothing in device memory can lead an access out of bounds.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <string>

#include "bsf8_epilogue.h"

namespace bsf8 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

constexpr int WAVES = 8;
constexpr int THREADS = WAVES * 64;
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

// Run number `item` of the experts' runs of T rows: the expert and its rows
// [first, end); false past the last run.  All lanes of a wave agree.
__device__ __forceinline__ bool find_run(const int32_t* offsets, int E, int R, int T, int item, int& expert, int& first,
                                         int& end) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < E; base += 64) {
    const int e = min(base + lane, E - 1);
    const int lo = min(max(offsets[e], 0), R), hi = min(max(offsets[e + 1], lo), R);
    const int runs = base + lane < E ? (hi - lo + T - 1) / T : 0;
    int sum = runs;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d, 64);
      if (lane >= d) sum += up;
    }
    const uint64_t past = __ballot(sum > item);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int run = item - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(runs, l));
      expert = base + l;
      end = __builtin_amdgcn_readlane(hi, l);
      first = __builtin_amdgcn_readlane(lo, l) + run * T;
      end = min(end, first + T);
      return true;
    }
    item -= __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// 16 bytes at p + k of a row of K bytes.  ALIGNED: K and p are multiples of 16;
// past the row's end the last 16 bytes (zeroed by the caller).  Else byte by
// byte, zeros past the end.
template <bool ALIGNED, bool NT>
__device__ __forceinline__ uint4 load_piece(const uint8_t* p, int k, int K) {
  if constexpr (ALIGNED) {
    const u4v* q = reinterpret_cast<const u4v*>(p + min(k, K - 16));
    const u4v v = NT ? __builtin_nontemporal_load(q) : *q;
    return make_uint4(v.x, v.y, v.z, v.w);
  } else {
    uint32_t b[4] = {0, 0, 0, 0};
    const int n = min(16, K - k);
    for (int i = 0; i < n; ++i) b[i >> 2] |= uint32_t(p[k + i]) << (8 * (i & 3));
    return make_uint4(b[0], b[1], b[2], b[3]);
  }
}

// a lane's 32 codes of a K block as the four steps' operands
struct Operand {
  v8bf s[4];
};
__device__ __forceinline__ Operand operand(const uint4 (&p)[2]) {
  return Operand{{decode8(p[0].x, p[0].y), decode8(p[0].z, p[0].w), decode8(p[1].x, p[1].y), decode8(p[1].z, p[1].w)}};
}

template <int RT, int TJ, int D, bool ALIGNED>
__global__ __launch_bounds__(THREADS) void w8a8_rows_kernel(RowsArgs a) {
  __shared__ float red[WAVES][RT * TJ][64][4];
  const int rt_total = a.rt0[a.w.n_members];
  const int item = blockIdx.x / rt_total, R_tile = blockIdx.x - item * rt_total;
  int expert = 0, first, end;
  if (a.offsets != nullptr) {
    if (!find_run(a.offsets, a.E, a.R, 16 * TJ, item, expert, first, end)) return;
  } else {
    first = item * 16 * TJ;
    end = min(a.R, first + 16 * TJ);
  }
  int mi = 0;
  while (mi + 1 < a.w.n_members && R_tile >= a.rt0[mi + 1]) ++mi;
  const MemberDev mem = a.w.m[mi];
  const int K = a.w.K, Kb = a.w.Kb;
  const int n0 = (R_tile - a.rt0[mi]) * 16 * RT;
  const int nb = (mem.rows + 127) >> 7;
  const uint8_t* wbase = mem.w + int64_t(expert) * mem.rows * K;
  const int64_t s_expert = int64_t(expert) * nb * a.w.Kb;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;

  // rows past the member's end repeat its last one and are not stored
  const uint8_t* wrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) wrow[i] = wbase + int64_t(min(n0 + 16 * i + l16, mem.rows - 1)) * K;
  // the column's row of codes; rows past the run and rows without a token read
  // token 0 and are not stored, or stored as zeros
  const uint8_t* xrow[TJ];
  const float* srow[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int r = first + 16 * j + l16;
    int tok = r < end ? (a.rows ? a.rows[r] : r) : 0;
    if (tok < 0 || tok >= a.M) tok = 0;
    xrow[j] = a.xq + int64_t(tok) * a.ldq;
    srow[j] = a.xs + int64_t(tok) * a.xs_sm;
  }
  const int tiles = (end - first + 15) / 16;      // column tiles that hold rows
  // the scale row of each row tile (a tile lies in one: 16 RT divides 128)
  const int64_t s_off = s_expert * (a.w.s_rs ? 1 : 0) + int64_t(n0 >> 7) * a.w.s_rs;

  v4f acc[RT][TJ];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  uint4 wr[D][RT][2], xr[D][TJ][2];
  float sa[D][TJ], sw[D];
  auto issue = [&](int c, int d) __attribute__((always_inline)) {
    const int cc = min(c, Kb - 1);
    const int k = cc * KB + 16 * g;
    sw[d] = load_real(mem.s, a.w.scale_bf16, s_off + int64_t(cc) * a.w.s_cs);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (j >= tiles) continue;
      sa[d][j] = srow[j][int64_t(cc) * a.xs_sk];
      xr[d][j][0] = load_piece<ALIGNED, false>(xrow[j], k, K);
      xr[d][j][1] = load_piece<ALIGNED, false>(xrow[j], k + 64, K);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      wr[d][i][0] = load_piece<ALIGNED, TJ == 1>(wrow[i], k, K);
      wr[d][i][1] = load_piece<ALIGNED, TJ == 1>(wrow[i], k + 64, K);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    issue(wave + WAVES * d, d);
    __builtin_amdgcn_sched_barrier(0);
  }
  const bool ragged = ALIGNED && K % KB != 0;
  for (int c0 = wave; c0 < Kb; c0 += WAVES * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int c = c0 + WAVES * d;
      if (c >= Kb) break;
      if (ragged && c == Kb - 1) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c * KB + 64 * h + 16 * g >= K) {
#pragma unroll
            for (int i = 0; i < RT; ++i) wr[d][i][h] = zero;
#pragma unroll
            for (int j = 0; j < TJ; ++j) xr[d][j][h] = zero;
          }
      }
      Operand w[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) w[i] = operand(wr[d][i]);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if (j >= tiles) continue;
        const Operand x = operand(xr[d][j]);
        const float s = sa[d][j] * sw[d];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          v4f p = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i].s[q], x.s[q], p, 0, 0, 0);
          acc[i][j] += p * s;
        }
      }
      issue(c + WAVES * D, d);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // ---- the waves' partial tiles in wave order, the epilogue, the store
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) *reinterpret_cast<v4f*>(&red[wave][i * TJ + j][lane][0]) = acc[i][j];
  __syncthreads();
  for (int o = tid; o < RT * TJ * 256; o += THREADS) {
    const int row = o % (16 * RT), col = o / (16 * RT);   // weight row and row of codes of the block
    const int n = n0 + row, r = first + col;
    if (n >= mem.rows || r >= end) continue;
    const int t = (row >> 4) * TJ + (col >> 4), ln = 16 * ((row & 15) >> 2) + (col & 15);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) v += red[q][t][ln][row & 3];
    if (a.rows) {
      const int tok = a.rows[r];
      if (tok < 0 || tok >= a.M) v = 0.f;
    }
    const int64_t at = int64_t(r) * a.ldy + mem.col0 + n;
    v = epilogue(a.ep, v, r, mem.col0 + n);
    if (a.y_bf16)
      static_cast<__bf16*>(a.y)[at] = static_cast<__bf16>(v);
    else
      static_cast<float*>(a.y)[at] = v;
  }
}

template <int RT, int TJ, int D>
bsf8_status launch(const RowsArgs& base, bool aligned, int64_t items, hipStream_t stream) {
  RowsArgs a = base;
  int r = 0;
  for (int i = 0; i < kMaxMembers; ++i) {
    a.rt0[i] = r;
    if (i < a.w.n_members) r += (a.w.m[i].rows + 16 * RT - 1) / (16 * RT);
  }
  a.rt0[kMaxMembers] = r;
  const int64_t grid = items * r;
  if (grid > INT32_MAX) {
    set_error("UNSUPPORTED: %lld blocks", (long long)grid);
    return BSF8_E_UNSUPPORTED;
  }
  if (aligned)
    hipLaunchKernelGGL((w8a8_rows_kernel<RT, TJ, D, true>), dim3(unsigned(grid)), dim3(THREADS), 0, stream, a);
  else
    hipLaunchKernelGGL((w8a8_rows_kernel<RT, TJ, 1, false>), dim3(unsigned(grid)), dim3(THREADS), 0, stream, a);
  return device_status(hipGetLastError(), "w8a8_rows launch");
}

bsf8_status launch_rows(RowsArgs& a, bool aligned, int64_t items1, int64_t items4, bool few, hipStream_t stream) {
  return few ? launch<1, 1, 4>(a, aligned, items1, stream) : launch<1, 4, 2>(a, aligned, items4, stream);
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
  return launch_rows(a, aligned, (M + 15) / 16, (M + 63) / 64, M <= 16, stream);
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
  const int64_t used = E < R ? E : R;
  return launch_rows(a, aligned, used + R / 16, used + R / 64, R <= 16 * E, stream);
}

std::string describe_w8a8_rows(bool few, bool aligned) {
  char buf[256];
  snprintf(buf, sizeof(buf), "arithmetic=e4m3 codes decoded exactly to bf16, mfma_f32_16x16x32_bf16, f32 per-128-K epilogue | "
           "kernel=w8a8_rows rows<=%d path=%s", few ? 16 : 64, aligned ? "aligned16" : "bytewise");
  return buf;
}

}  // namespace bsf8
