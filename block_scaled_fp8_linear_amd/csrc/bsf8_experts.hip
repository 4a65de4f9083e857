// The experts' products (gfx950): which kernel takes a call, and the tile GEMM's
// instances for ragged row runs.
#include <cmath>
#include <cstdio>
#include <string>

#include "bsf8_tile.h"

namespace bsf8 {
namespace {

// Which kernel: 0 the few-row kernel, else the tile size.  The host knows the
// rows R and the experts E, not the runs, and takes about R / T + E / 2 tiles of
// T rows, at least one for each expert that can have rows.  Times in
// microseconds, fitted to calls timed on all kernels (2 to 128 experts, 8 to 16384
// rows, N 300 to 5120, K 512 to 7168):
//  * few rows: a block of 32 weight rows and 16 or 64 rows of codes takes 0.6 +
//    0.67 or 15.6 + 1.15 ns of the device per K block (0.67 ns for 4 KiB of weight
//    is 6 TB/s), at least its waves' own chain of K blocks;
//  * 128 x 128 tiles: 3.4 ns per block and K block, 0.85 us while few blocks run;
//    F32 outputs (one block per compute unit) 1.1 us per round of blocks;
//  * 256 x 256 tiles: 1.6 us per round of blocks and K block.
// 64 experts [1536, 2048] and 8 / 256 / 512 / 1024 / 8192 rows take 9 / 26 / 38 / 54 /
// 187 us few-row, 18 / 30 / 44 / 45 / 79 us in 128 x 128 and 21 / 30 / 53 / 53 / 62 us in
// 256 x 256 tiles.
int choose(const WeightDev& w, int64_t E, bool aligned, int64_t R, int64_t M, int64_t ldq, int64_t xs_extent, bool y_bf16) {
  // the tile kernel's 32-bit offsets: one expert's member, the tokens' codes and scales
  bool fits = M * ldq < (int64_t(1) << 31) && xs_extent * 4 < (int64_t(1) << 31) && w.Kb <= F_MAX_KB;
  for (int i = 0; i < w.n_members; ++i) fits = fits && int64_t(w.m[i].rows) * w.K < (int64_t(1) << 31);
  if (!aligned || !fits) return 0;
  const double used = double(E < R ? E : R);
  const auto blocks = [&](int rows, int T) {
    double rt = 0;
    for (int i = 0; i < w.n_members; ++i) rt += (w.m[i].rows + rows - 1) / rows;
    return rt * std::max(used, double(R) / T + 0.5 * used);
  };
  const double cus = device_cus(), kb = w.Kb;
  const bool few = R <= 16 * E;
  const double by_rows = 3.0 + std::max(blocks(32, few ? 16 : 64) * (few ? 0.6e-3 + 0.67e-3 * kb : 15.6e-3 + 1.15e-3 * kb),
                                        0.9 * kb / (kb <= 16 ? 4 : 8));
  const double b128 = blocks(128, 128);
  const double t128 = 4.5 + kb * (y_bf16 ? std::max(0.85, 3.4e-3 * b128) : 1.1 * std::ceil(b128 / cus));
  const double t256 = y_bf16 ? 5.0 + kb * 1.6 * std::ceil(blocks(256, 256) / cus) : 1e30;
  return by_rows <= std::min(t128, t256) ? 0 : t128 <= t256 ? 128 : 256;
}

}  // namespace

bsf8_status launch_w8a8_experts(const WeightDev& w, int64_t E, bool aligned, const uint8_t* xq, int64_t ldq,
                                const float* xs, int64_t xs_sm, int64_t xs_sk, int64_t M, const int32_t* offsets,
                                const int32_t* rows, int64_t R, void* y, bool y_bf16, int64_t ldy, hipStream_t stream) {
  const int T = choose(w, E, aligned, R, M, ldq, (M - 1) * xs_sm + (w.Kb - 1) * xs_sk + 1, y_bf16);
  if (T == 0)
    return launch_w8a8_expert_rows(w, E, aligned, xq, ldq, xs, xs_sm, xs_sk, M, offsets, rows, R, y, y_bf16, ldy, stream);
  FusedArgs a{};
  a.w = w;
  int r = 0;
  for (int i = 0; i <= kMaxMembers; ++i) {
    a.rt0[i] = r;
    if (i < w.n_members) r += (w.m[i].rows + T - 1) / T;
  }
  a.rt_total = r;
  a.xq = xq;
  a.xs = xs;
  a.y = y;
  a.ldq = ldq;
  a.xs_sm = xs_sm;
  a.xs_sk = xs_sk;
  a.ldy = ldy;
  a.M = int32_t(M);
  a.y_bf16 = y_bf16 ? 1 : 0;
  const int64_t esz = y_bf16 ? 2 : 4;
  bool vec = (reinterpret_cast<uintptr_t>(y) & 15) == 0 && (ldy * esz) % 16 == 0;
  for (int i = 0; i < w.n_members; ++i) vec = vec && (w.m[i].col0 * esz) % 16 == 0;
  a.y_vec = vec ? 1 : 0;
  a.y_nt = R * int64_t(w.m[w.n_members - 1].col0 + w.m[w.n_members - 1].rows) * esz > (int64_t(128) << 20) ? 1 : 0;
  a.offsets = offsets;
  a.rows = rows;
  a.E = int32_t(E);
  a.R = int32_t(R);
  // the most tiles that R rows of E experts can make; blocks past the last one leave
  const int64_t grid = ((E < R ? E : R) + R / T) * r;
  if (grid * FTHREADS > UINT32_MAX) {
    set_error("UNSUPPORTED: %lld blocks", (long long)grid);
    return BSF8_E_UNSUPPORTED;
  }
  const bool kfull = w.K % KBYTES == 0;
  const auto kern = y_bf16 ? tile_kernel<kExperts, false>(T, w.scale_bf16 != 0, kfull)
                           : tile_kernel<kExperts, true>(T, w.scale_bf16 != 0, kfull);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(FTHREADS), 0, stream, a);
  return device_status(hipGetLastError(), "w8a8_experts launch");
}

// (For packed tokens whose codes and scales stay below 2 GiB: farther ones take the few-row kernel.)
std::string describe_w8a8_experts(const WeightDev& w, int64_t E, bool aligned, int64_t R) {
  char n[64];
  snprintf(n, sizeof(n), " | R=%lld", (long long)R);
  std::string out = "arm=w8a8-experts";
  for (const bool bf16 : {true, false}) {
    const int T = choose(w, E, aligned, R, 1, w.K, w.Kb, bf16);
    char buf[256];
    snprintf(buf, sizeof(buf), "arithmetic=%s, f32 per-128-K epilogue | kernel=w8a8_gemm_fast<experts> tile=%dx%d",
             bf16 ? "e4m3xe4m3 mfma_f32_16x16x128_f8f6f4" : "e4m3 codes decoded exactly to bf16, mfma_f32_16x16x32_bf16", T, T);
    out += std::string(bf16 ? " | bf16 outputs: " : " | f32 outputs: ") +
           (T == 0 ? describe_w8a8_rows(R <= 16 * E, aligned) : std::string(buf));
  }
  return out + n;
}

}  // namespace bsf8
