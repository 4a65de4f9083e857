// The experts' products (gfx950): which kernel takes a call, and the tile GEMM's
// instances for ragged row runs.
#include <cstdio>
#include <cstdlib>
#include <string>

#include "bsf8_tile.h"

namespace bsf8 {
namespace {

// The host knows the rows R and the experts E, not the runs: the choice goes by
// the mean run R / E.
bool by_rows(const WeightDev& w, int64_t E, bool aligned, int64_t R, int64_t M, int64_t ldq, int64_t xs_extent) {
  // the tile kernel's 32-bit offsets: one expert's member, the tokens' codes and scales
  bool fits = M * ldq < (int64_t(1) << 31) && xs_extent * 4 < (int64_t(1) << 31) && w.Kb <= F_MAX_KB;
  for (int i = 0; i < w.n_members; ++i) fits = fits && int64_t(w.m[i].rows) * w.K < (int64_t(1) << 31);
  return !aligned || !fits || R <= (getenv("XR") ? atoi(getenv("XR")) : 16) * E;
}

int tile_of(int64_t E, int64_t R, bool y_bf16) { if (getenv("XT")) return y_bf16 ? atoi(getenv("XT")) : 128; return y_bf16 && R >= 256 * E ? 256 : 128; }

}  // namespace

bsf8_status launch_w8a8_experts(const WeightDev& w, int64_t E, bool aligned, const uint8_t* xq, int64_t ldq,
                                const float* xs, int64_t xs_sm, int64_t xs_sk, int64_t M, const int32_t* offsets,
                                const int32_t* rows, int64_t R, void* y, bool y_bf16, int64_t ldy, hipStream_t stream) {
  if (by_rows(w, E, aligned, R, M, ldq, (M - 1) * xs_sm + (w.Kb - 1) * xs_sk + 1))
    return launch_w8a8_expert_rows(w, E, aligned, xq, ldq, xs, xs_sm, xs_sk, M, offsets, rows, R, y, y_bf16, ldy, stream);
  const int T = tile_of(E, R, y_bf16);
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
  if (grid > INT32_MAX) {
    set_error("UNSUPPORTED: %lld blocks", (long long)grid);
    return BSF8_E_UNSUPPORTED;
  }
  const bool kfull = w.K % KBYTES == 0;
  const auto kern = y_bf16 ? tile_kernel<kExperts, false>(T, w.scale_bf16 != 0, kfull)
                           : tile_kernel<kExperts, true>(T, w.scale_bf16 != 0, kfull);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(FTHREADS), 0, stream, a);
  return device_status(hipGetLastError(), "w8a8_experts launch");
}

std::string describe_w8a8_experts(const WeightDev& w, int64_t E, bool aligned, int64_t R) {
  char n[64];
  snprintf(n, sizeof(n), " | R=%lld", (long long)R);
  if (by_rows(w, E, aligned, R, 1, w.K, w.Kb)) return "arm=w8a8-experts " + describe_w8a8_rows(R <= 16 * E, aligned) + n;
  char buf[320];
  snprintf(buf, sizeof(buf),
           "arm=w8a8-experts arithmetic=bf16 outputs e4m3xe4m3 mfma_f32_16x16x128_f8f6f4, f32 outputs codes decoded "
           "exactly to bf16, f32 per-128-K epilogue | kernel=w8a8_gemm_fast<experts> tile=%dx%d (f32 outputs 128x128)",
           tile_of(E, R, true), tile_of(E, R, true));
  return std::string(buf) + n;
}

}  // namespace bsf8
