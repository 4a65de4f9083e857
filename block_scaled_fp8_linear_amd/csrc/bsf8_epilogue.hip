// The W8A8 product with bias, activation and residual (gfx950): which kernel
// takes a call, and the tile GEMM's instances with an epilogue.
#include <cstdio>
#include <string>

#include "bsf8_tile.h"

namespace bsf8 {
namespace {

// Up to this many tokens the few-row kernel, which has four 16-token tiles.  At 64
// tokens with a residual it takes 17.6 us against the tile GEMM's 19.3 on [5120,
// 5120], 17.7 against 19.0 on [5000, 4000], 11.8 / 11.9 on [1000, 2000]; the tile GEMM is
// ahead on wide and on long weights, 47.5 against 48.3 on [17408, 5120] and 35.7 against
// 39.7 on [5120, 17408], which this rule does not see.  At 100 tokens, where the few-row
// kernel reads the weight twice, it takes 26.9 against 20.6 on [5120, 5120].
constexpr int64_t kRowsMaxM = 64;

bool by_rows(const Plan& p, int64_t M) { return !p.fast || M <= kRowsMaxM; }

// F32 outputs sum the codes exactly (128 x 128 tiles); BF16 outputs take the FP8 MFMA.
Plan plan_of(const WeightDev& w, bool aligned, int64_t M, int64_t ldq, int64_t xs_extent, bool y_bf16) {
  return make_plan(w, aligned, M, ldq, xs_extent, !y_bf16);
}

}  // namespace

// (the larger of the two output types' plans)
size_t w8a8_epilogue_workspace_bytes(const WeightDev& w, int64_t M) {
  if (M <= kRowsMaxM) return 0;
  return std::max(plan_of(w, true, M, w.K, -1, true).ws_bytes, plan_of(w, true, M, w.K, -1, false).ws_bytes);
}

bsf8_status launch_w8a8_epilogue(const WeightDev& w, bool aligned, const uint8_t* xq, int64_t ldq, const float* xs,
                                 int64_t xs_sm, int64_t xs_sk, int64_t M, const EpilogueDev& ep, void* y, bool y_bf16,
                                 int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  const Plan p = plan_of(w, aligned, M, ldq, (M - 1) * xs_sm + (w.Kb - 1) * xs_sk + 1, y_bf16);
  if (by_rows(p, M))
    return launch_w8a8_rows(w, aligned, xq, ldq, xs, xs_sm, xs_sk, M, ep, y, y_bf16, ldy, stream);
  return y_bf16 ? launch_fast<kEpilogue>(p, w, xq, ldq, xs, xs_sm, xs_sk, M, y, y_bf16, ldy, ws, ws_bytes, stream, &ep)
                : launch_fast<kEpilogue, true>(p, w, xq, ldq, xs, xs_sm, xs_sk, M, y, y_bf16, ldy, ws, ws_bytes, stream, &ep);
}

// (Both output types' plans, for tokens packed at a pitch of K.)
std::string describe_w8a8_epilogue(const WeightDev& w, bool aligned, int64_t M) {
  char m[64];
  snprintf(m, sizeof(m), " | M=%lld", (long long)M);
  if (by_rows(plan_of(w, aligned, M, w.K, -1, true), M)) return "arm=w8a8-epilogue " + describe_w8a8_rows(M <= 16, aligned) + m;
  std::string out = "arm=w8a8-epilogue";
  for (const bool bf16 : {true, false}) {
    const Plan p = plan_of(w, aligned, M, w.K, -1, bf16);
    char buf[320];
    snprintf(buf, sizeof(buf),
             "arithmetic=%s, f32 per-128-K epilogue | kernel=w8a8_gemm_fast tile=%dx%d split_k=%d split_row_tiles=%d",
             bf16 ? "e4m3xe4m3 mfma_f32_16x16x128_f8f6f4" : "e4m3 codes decoded exactly to bf16, mfma_f32_16x16x32_bf16",
             p.tile, p.tile, p.splits, p.rt_total - p.rt_split0);
    out += std::string(bf16 ? " | bf16 outputs: " : " | f32 outputs: ") + buf;
  }
  return out + m;
}

}  // namespace bsf8
