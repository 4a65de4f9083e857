// Host side of libbsf8: status names, the header-only validator, weight handles,
// argument checks and dispatch to the kernel launchers.  No device memory is
// touched here except through the launchers.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <new>
#include <string>

#include "bsf8_internal.h"

namespace bsf8 {

// fixed buffers: reporting a failure allocates nothing, so it cannot throw
static thread_local char g_last_error[560];
static thread_local char g_describe[1536];

void set_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
}

bsf8_status device_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return BSF8_OK;
  set_error("%s: %s", what, hipGetErrorString(e));
  return BSF8_E_DEVICE;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

static bsf8_status fail(bsf8_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  snprintf(g_last_error, sizeof(g_last_error), "%s: %s", bsf8_status_name(s), buf);
  return s;
}

// The member's scale leaf: the block grid, or the per-tensor weight_scale.
static const bsf8_tensor_desc* scale_leaf(const bsf8_member_desc& m) { return m.scale_inv ? m.scale_inv : m.scale; }

static bool shape_is(const bsf8_tensor_desc* t, int64_t a, int64_t b) {
  return t->rank == 2 && t->shape[0] == a && t->shape[1] == b;
}

// Header-only validation.  The order of the checks is the precedence the ABI
// documents, so every bad input has exactly one status.
static bsf8_status validate_impl(const bsf8_decl* decl, const bsf8_member_desc* members, int32_t n) {
  if (decl == nullptr || (members == nullptr && n > 0)) return fail(BSF8_E_INVALID_ARG, "null descriptor");
  if (n < 1 || n > kMaxMembers) return fail(BSF8_E_GROUP, "%d members (1..%d allowed)", n, kMaxMembers);
  const bool per_tensor = decl->quant_method_fp8 && decl->block_n == 0 && decl->block_k == 0;
  if (!decl->quant_method_fp8 || (!per_tensor && (decl->block_n != kBlock || decl->block_k != kBlock)))
    return fail(BSF8_E_DECL,
                "declaration is not quant_method fp8 with weight_block_size [128,128] or per-tensor (got fp8=%d, [%d,%d])",
                decl->quant_method_fp8, decl->block_n, decl->block_k);
  for (int i = 0; i < n; ++i) {
    const bsf8_member_desc& m = members[i];
    const bsf8_tensor_desc& w = m.weight;
    if (w.rank < 0 || w.rank > 4) return fail(BSF8_E_INVALID_ARG, "member %d: weight rank %d", i, w.rank);
    if (w.dtype == BSF8_DT_F8_E5M2) return fail(BSF8_E_WEIGHT_E5M2, "member %d: E5M2 weight", i);
    if (w.dtype != BSF8_DT_F8_E4M3) return fail(BSF8_E_WEIGHT_DTYPE, "member %d: weight dtype %d is not F8_E4M3", i, w.dtype);
    if (w.rank != 2) return fail(BSF8_E_WEIGHT_RANK, "member %d: weight rank %d", i, w.rank);
    if (w.shape[0] <= 0 || w.shape[1] <= 0)
      return fail(BSF8_E_WEIGHT_EMPTY, "member %d: weight shape [%lld,%lld]", i, (long long)w.shape[0], (long long)w.shape[1]);
    if (m.scale_inv == nullptr && m.scale == nullptr) return fail(BSF8_E_SCALE_MISSING, "member %d: FP8 weight without a scale", i);
    if (m.scale_inv != nullptr && m.scale != nullptr)
      return fail(BSF8_E_SCALE_AMBIGUOUS, "member %d: both a block grid and a row/tensor scale", i);
    const bsf8_tensor_desc* leaf = m.scale_inv ? m.scale_inv : m.scale;
    if (leaf->rank < 0 || leaf->rank > 4) return fail(BSF8_E_INVALID_ARG, "member %d: scale rank %d", i, leaf->rank);
    if (per_tensor) {
      // one weight_scale value for the whole tensor (rank 0, or rank 1 of one element)
      if (m.scale_inv != nullptr)
        return fail(BSF8_E_DECL, "member %d: a weight_scale_inv grid under a per-tensor declaration", i);
      if (leaf->rank == 1 && leaf->shape[0] != 1) return fail(BSF8_E_SCALE_ROWWISE, "member %d: rank-1 (row-wise) scale", i);
      if (leaf->rank > 1) return fail(BSF8_E_SCALE_RANK, "member %d: per-tensor scale of rank %d", i, leaf->rank);
      if (leaf->dtype != BSF8_DT_BF16 && leaf->dtype != BSF8_DT_F32)
        return fail(BSF8_E_SCALE_DTYPE, "member %d: scale dtype %d is not BF16/F32", i, leaf->dtype);
      continue;
    }
    if (leaf->rank == 1) return fail(BSF8_E_SCALE_ROWWISE, "member %d: rank-1 (row-wise) scale", i);
    if (leaf->rank == 0 && m.scale != nullptr) return fail(BSF8_E_SCALE_PER_TENSOR, "member %d: per-tensor scale", i);
    if (leaf->rank != 2) return fail(BSF8_E_SCALE_RANK, "member %d: scale rank %d", i, leaf->rank);
    if (leaf->dtype != BSF8_DT_BF16 && leaf->dtype != BSF8_DT_F32)
      return fail(BSF8_E_SCALE_DTYPE, "member %d: scale dtype %d is not BF16/F32", i, leaf->dtype);
    const int64_t nb = ceil_div(w.shape[0], kBlock), kb = ceil_div(w.shape[1], kBlock);
    if (!shape_is(leaf, nb, kb) && shape_is(leaf, kb, nb))
      return fail(BSF8_E_SCALE_TRANSPOSED, "member %d: grid [%lld,%lld] is the transpose of [%lld,%lld]", i,
                  (long long)leaf->shape[0], (long long)leaf->shape[1], (long long)nb, (long long)kb);
    if (!shape_is(leaf, nb, kb))
      return fail(BSF8_E_SCALE_GRID, "member %d: grid [%lld,%lld] != [%lld,%lld]", i, (long long)leaf->shape[0],
                  (long long)leaf->shape[1], (long long)nb, (long long)kb);
    if (m.scale != nullptr)
      return fail(BSF8_E_SCALE_GRID, "member %d: a block-shaped weight_scale leaf is not a weight_scale_inv grid", i);
  }
  const int64_t k0 = members[0].weight.shape[1];
  const int32_t dt0 = scale_leaf(members[0])->dtype;
  for (int i = 1; i < n; ++i) {
    if (members[i].weight.shape[1] != k0) return fail(BSF8_E_GROUP, "member %d: K differs from member 0", i);
    if (scale_leaf(members[i])->dtype != dt0) return fail(BSF8_E_GROUP, "member %d: scale dtype differs from member 0", i);
  }
  for (int i = 0; i < n; ++i) {
    const uintptr_t wa = reinterpret_cast<uintptr_t>(members[i].weight.data);
    if (wa % 16 != 0) return fail(BSF8_E_ALIGNMENT, "member %d: weight address not 16-byte aligned", i);
    const uintptr_t sa = reinterpret_cast<uintptr_t>(scale_leaf(members[i])->data);
    const uintptr_t esz = scale_leaf(members[i])->dtype == BSF8_DT_BF16 ? 2 : 4;
    if (sa % esz != 0) return fail(BSF8_E_ALIGNMENT, "member %d: scale address not element aligned", i);
  }
  return BSF8_OK;
}

// A describe line, `text()` followed by the handle's geometry, in the thread's
// buffer; the geometry alone where the host's memory ends.
template <typename F>
static const char* described(const char* geo, const F& text) {
  try {
    const std::string s = text();
    snprintf(g_describe, sizeof(g_describe), "%s%s", s.c_str(), geo);
  } catch (const std::exception&) {
    snprintf(g_describe, sizeof(g_describe), "out of host memory%s", geo);
  }
  return g_describe;
}

static bool dtype_ok(int32_t dt, bool f32, bool bf16) {
  return (f32 && dt == BSF8_DT_F32) || (bf16 && dt == BSF8_DT_BF16);
}

}  // namespace bsf8

using namespace bsf8;

extern "C" {

int32_t bsf8_abi_version(void) { return BSF8_ABI_VERSION; }

const char* bsf8_status_name(bsf8_status s) {
  switch (s) {
    case BSF8_OK: return "OK";
    case BSF8_E_INVALID_ARG: return "INVALID_ARG";
    case BSF8_E_GROUP: return "GROUP";
    case BSF8_E_DECL: return "DECL";
    case BSF8_E_WEIGHT_E5M2: return "WEIGHT_E5M2";
    case BSF8_E_WEIGHT_DTYPE: return "WEIGHT_DTYPE";
    case BSF8_E_WEIGHT_RANK: return "WEIGHT_RANK";
    case BSF8_E_WEIGHT_EMPTY: return "WEIGHT_EMPTY";
    case BSF8_E_SCALE_MISSING: return "SCALE_MISSING";
    case BSF8_E_SCALE_AMBIGUOUS: return "SCALE_AMBIGUOUS";
    case BSF8_E_SCALE_ROWWISE: return "SCALE_ROWWISE";
    case BSF8_E_SCALE_PER_TENSOR: return "SCALE_PER_TENSOR";
    case BSF8_E_SCALE_RANK: return "SCALE_RANK";
    case BSF8_E_SCALE_DTYPE: return "SCALE_DTYPE";
    case BSF8_E_SCALE_TRANSPOSED: return "SCALE_TRANSPOSED";
    case BSF8_E_SCALE_GRID: return "SCALE_GRID";
    case BSF8_E_ALIGNMENT: return "ALIGNMENT";
    case BSF8_E_UNSUPPORTED: return "UNSUPPORTED";
    case BSF8_E_WORKSPACE: return "WORKSPACE";
    case BSF8_E_DEVICE: return "DEVICE";
  }
  return "UNKNOWN";
}

const char* bsf8_last_error(void) { return g_last_error; }

bsf8_status bsf8_validate(const bsf8_decl* decl, const bsf8_member_desc* members, int32_t n_members) {
  return validate_impl(decl, members, n_members);
}

bsf8_status bsf8_weight_create(const bsf8_decl* decl, const bsf8_member_desc* members, int32_t n_members,
                               bsf8_weight** out) {
  if (out == nullptr) return fail(BSF8_E_INVALID_ARG, "out is NULL");
  *out = nullptr;
  bsf8_status st = validate_impl(decl, members, n_members);
  if (st != BSF8_OK) return st;
  const int64_t K = members[0].weight.shape[1];
  int64_t total = 0;
  for (int i = 0; i < n_members; ++i) {
    if (members[i].weight.data == nullptr || scale_leaf(members[i])->data == nullptr)
      return fail(BSF8_E_INVALID_ARG, "member %d: a handle needs device addresses", i);
    total += members[i].weight.shape[0];
  }
  if (K > INT32_MAX / 2 || total > INT32_MAX / 2)
    return fail(BSF8_E_UNSUPPORTED, "N or K beyond 2^30");
  bsf8_weight* h = new (std::nothrow) bsf8_weight();
  if (h == nullptr) return fail(BSF8_E_UNSUPPORTED, "out of host memory");
  std::memset(&h->dev, 0, sizeof(h->dev));
  h->dev.n_members = n_members;
  h->dev.K = static_cast<int32_t>(K);
  h->dev.Kb = static_cast<int32_t>(ceil_div(K, kBlock));
  h->dev.scale_bf16 = scale_leaf(members[0])->dtype == BSF8_DT_BF16 ? 1 : 0;
  h->per_tensor = members[0].scale_inv == nullptr;
  h->dev.s_rs = h->per_tensor ? 0 : h->dev.Kb;
  h->dev.s_cs = h->per_tensor ? 0 : 1;
  h->aligned16 = (K % 16) == 0;
  int64_t col = 0, srow = 0;
  for (int i = 0; i < n_members; ++i) {
    const int64_t rows = members[i].weight.shape[0];
    h->dev.m[i].w = static_cast<const uint8_t*>(members[i].weight.data);
    h->dev.m[i].s = scale_leaf(members[i])->data;
    h->dev.m[i].rows = static_cast<int32_t>(rows);
    h->dev.m[i].col0 = static_cast<int32_t>(col);
    h->rows[i] = rows;
    h->col0[i] = col;
    h->srow0[i] = srow;
    col += rows;
    srow += h->per_tensor ? 1 : ceil_div(rows, kBlock);
  }
  h->n_total = total;
  *out = h;
  return BSF8_OK;
}

void bsf8_weight_destroy(bsf8_weight* w) { delete w; }

bsf8_status bsf8_weight_geometry(const bsf8_weight* w, int64_t* n_total, int64_t* k, int32_t* n_members) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (n_total) *n_total = w->n_total;
  if (k) *k = w->dev.K;
  if (n_members) *n_members = w->dev.n_members;
  return BSF8_OK;
}

bsf8_status bsf8_weight_scale_row(const bsf8_weight* w, int64_t n, int32_t* member, int64_t* local_row,
                                  int64_t* stacked_row) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (n < 0 || n >= w->n_total) return fail(BSF8_E_INVALID_ARG, "row %lld outside [0,%lld)", (long long)n, (long long)w->n_total);
  for (int i = w->dev.n_members - 1; i >= 0; --i) {
    if (n >= w->col0[i]) {
      const int64_t r = w->per_tensor ? 0 : (n - w->col0[i]) / kBlock;
      if (member) *member = i;
      if (local_row) *local_row = r;
      if (stacked_row) *stacked_row = w->srow0[i] + r;
      return BSF8_OK;
    }
  }
  return fail(BSF8_E_INVALID_ARG, "row not found");
}

// The two accepted activation scale layouts: token-major (xs_sk == 1, rows of
// at least Kb) and K-major (xs_sm == 1, rows of at least M).
static bool scale_layout_ok(int64_t M, int64_t Kb, int64_t xs_sm, int64_t xs_sk) {
  return (xs_sk == 1 && xs_sm >= Kb) || (xs_sm == 1 && xs_sk >= M);
}

bsf8_status bsf8_quant_act(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, uint8_t* xq,
                           int64_t ldq, float* xs, int64_t xs_sm, int64_t xs_sk, void* stream) {
  if (M < 0 || K < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (!dtype_ok(x_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "x dtype %d (F32 or BF16)", x_dtype);
  if (M == 0 || K == 0) return BSF8_OK;
  if (x == nullptr || xq == nullptr || xs == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldx < K || ldq < K) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (!scale_layout_ok(M, ceil_div(K, kBlock), xs_sm, xs_sk))
    return fail(BSF8_E_INVALID_ARG, "xs strides (%lld, %lld): neither token-major nor K-major", (long long)xs_sm,
                (long long)xs_sk);
  if (M > INT32_MAX || K > INT32_MAX / 2) return fail(BSF8_E_UNSUPPORTED, "M or K too large");
  const size_t esz = x_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % esz || reinterpret_cast<uintptr_t>(xs) % 4)
    return fail(BSF8_E_ALIGNMENT, "x or xs not element aligned");
  return launch_quant_act(x, x_dtype == BSF8_DT_BF16, M, K, ldx, xq, ldq, xs, xs_sm, xs_sk,
                          static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_quant_glu(const void* y, int32_t y_dtype, int64_t M, int64_t F, int64_t ldy, uint8_t* xq,
                           int64_t ldq, float* xs, int64_t xs_sm, int64_t xs_sk, void* stream) {
  if (M < 0 || F < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0 || F == 0) return BSF8_OK;
  if (y == nullptr || xq == nullptr || xs == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldy < 2 * F || ldq < F) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (!scale_layout_ok(M, ceil_div(F, kBlock), xs_sm, xs_sk))
    return fail(BSF8_E_INVALID_ARG, "xs strides (%lld, %lld): neither token-major nor K-major", (long long)xs_sm,
                (long long)xs_sk);
  if (M > INT32_MAX || F > INT32_MAX / 4) return fail(BSF8_E_UNSUPPORTED, "M or F too large");
  const size_t esz = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(y) % esz || reinterpret_cast<uintptr_t>(xs) % 4)
    return fail(BSF8_E_ALIGNMENT, "y or xs not element aligned");
  return launch_quant_glu(y, y_dtype == BSF8_DT_BF16, M, F, ldy, xq, ldq, xs, xs_sm, xs_sk,
                          static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_glu_act(const void* y, int32_t y_dtype, int64_t M, int64_t F, int64_t ldy, float* h, int64_t ldh,
                         void* stream) {
  if (M < 0 || F < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0 || F == 0) return BSF8_OK;
  if (y == nullptr || h == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldy < 2 * F || ldh < F) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (M > INT32_MAX || F > INT32_MAX / 4) return fail(BSF8_E_UNSUPPORTED, "M or F too large");
  const size_t esz = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(y) % esz || reinterpret_cast<uintptr_t>(h) % 4)
    return fail(BSF8_E_ALIGNMENT, "y or h not element aligned");
  return launch_glu_act(y, y_dtype == BSF8_DT_BF16, M, F, ldy, h, ldh, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_quant_norm(const bsf8_norm_args* p, void* stream) {
  if (p == nullptr) return fail(BSF8_E_INVALID_ARG, "null arguments");
  const bsf8_norm_args& q = *p;
  if (q.M < 0 || q.K < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (q.kind != BSF8_NORM_RMS && q.kind != BSF8_NORM_LAYER) return fail(BSF8_E_INVALID_ARG, "norm kind %d", q.kind);
  if (!(q.eps > 0.0) || !std::isfinite(q.eps) || !std::isfinite(q.residual_scale))
    return fail(BSF8_E_INVALID_ARG, "eps %g (positive) or residual_scale %g", q.eps, q.residual_scale);
  if (!dtype_ok(q.x_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "x dtype %d (F32 or BF16)", q.x_dtype);
  if (!dtype_ok(q.h_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "h dtype %d (F32 or BF16)", q.h_dtype);
  if (!dtype_ok(q.weight_dtype, true, true) || (q.post_weight && !dtype_ok(q.post_dtype, true, true)) ||
      (q.gate && !dtype_ok(q.gate_dtype, true, true)) || (q.n && !dtype_ok(q.n_dtype, true, true)))
    return fail(BSF8_E_INVALID_ARG, "weight, post, gate or n dtype (F32 or BF16)");
  if ((q.slots == nullptr) != (q.probs == nullptr)) return fail(BSF8_E_INVALID_ARG, "slots and probs: both or neither");
  if (q.slots && (q.top < 1 || q.x_rows < 0)) return fail(BSF8_E_INVALID_ARG, "top %d or x_rows %lld", q.top, (long long)q.x_rows);
  if ((q.xq == nullptr) != (q.xs == nullptr)) return fail(BSF8_E_INVALID_ARG, "xq and xs: both or neither");
  if (q.M == 0 || q.K == 0) return BSF8_OK;
  // an experts' output without a row may have no address
  if ((q.x == nullptr && !(q.slots && q.x_rows == 0)) || q.weight == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (q.n == nullptr && q.xq == nullptr) return fail(BSF8_E_INVALID_ARG, "neither n nor xq is given");
  if (q.residual && !q.h) return fail(BSF8_E_INVALID_ARG, "a residual without h");
  if (q.post_bias && !q.post_weight) return fail(BSF8_E_INVALID_ARG, "post_bias without post_weight");
  if (q.ldx < q.K || (q.residual && q.ldr < q.K) || (q.h && q.ldh < q.K) || (q.n && q.ldn < q.K) ||
      (q.xq && q.ldq < q.K) || (q.gate && q.ldg != 0 && q.ldg < q.K))
    return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (q.xq && !scale_layout_ok(q.M, ceil_div(q.K, kBlock), q.xs_sm, q.xs_sk))
    return fail(BSF8_E_INVALID_ARG, "xs strides (%lld, %lld): neither token-major nor K-major", (long long)q.xs_sm,
                (long long)q.xs_sk);
  if (q.K > BSF8_NORM_MAX_K || q.M > INT32_MAX || (q.slots && q.x_rows > INT32_MAX))
    return fail(BSF8_E_UNSUPPORTED, "K beyond %d, or M or x_rows too large", BSF8_NORM_MAX_K);
  NormDev a{};
  bool misaligned = false;
  // element alignment is required; 16-byte rows are taken where they are there
  const auto vec = [&](const void* ptr, bool bf16, int64_t ld) -> int32_t {
    const uintptr_t at = reinterpret_cast<uintptr_t>(ptr);
    const int64_t esz = bf16 ? 2 : 4;
    misaligned = misaligned || at % uintptr_t(esz) != 0;
    return at % 16 == 0 && (ld * esz) % 16 == 0 ? 1 : 0;
  };
  const bool x_bf16 = q.x_dtype == BSF8_DT_BF16, h_bf16 = q.h_dtype == BSF8_DT_BF16;
  a.M = int32_t(q.M);
  a.K = int32_t(q.K);
  a.layer = q.kind == BSF8_NORM_LAYER ? 1 : 0;
  a.top = q.top;
  a.R = q.slots ? int32_t(q.x_rows) : 0;
  a.post_bf16 = q.post_dtype == BSF8_DT_BF16;
  a.gate_bf16 = q.gate_dtype == BSF8_DT_BF16;
  a.w_bf16 = q.weight_dtype == BSF8_DT_BF16;
  a.n_bf16 = q.n_dtype == BSF8_DT_BF16;
  a.x_vec = vec(q.x, x_bf16, q.ldx);
  a.res_vec = vec(q.residual, h_bf16, q.ldr);
  a.h_vec = vec(q.h, h_bf16, q.ldh);
  a.n_vec = vec(q.n, a.n_bf16 != 0, q.ldn);
  a.post_vec = vec(q.post_weight, a.post_bf16 != 0, 0) & vec(q.post_bias, a.post_bf16 != 0, 0);
  a.gate_vec = vec(q.gate, a.gate_bf16 != 0, q.ldg);
  a.w_vec = vec(q.weight, a.w_bf16 != 0, 0) & vec(q.bias, a.w_bf16 != 0, 0);
  a.q_vec = reinterpret_cast<uintptr_t>(q.xq) % 8 == 0 && q.ldq % 8 == 0 ? 1 : 0;
  a.wide = q.K % 8 == 0 && a.x_vec && a.res_vec && a.h_vec && a.n_vec && a.q_vec && a.post_vec && a.gate_vec && a.w_vec &&
                   (!q.post_weight || a.post_bf16 == a.w_bf16) && (!q.gate || a.gate_bf16 == a.w_bf16)
               ? 1 : 0;
  misaligned = misaligned || reinterpret_cast<uintptr_t>(q.xs) % 4 || reinterpret_cast<uintptr_t>(q.slots) % 4 ||
               reinterpret_cast<uintptr_t>(q.probs) % 4;
  if (misaligned) return fail(BSF8_E_ALIGNMENT, "an address is not element aligned");
  a.eps = q.eps;
  a.alpha = q.residual_scale;
  a.x = q.x;
  a.slots = q.slots;
  a.probs = q.probs;
  a.post_w = q.post_weight;
  a.post_b = q.post_bias;
  a.gate = q.gate;
  a.res = q.residual;
  a.w = q.weight;
  a.b = q.bias;
  a.h = q.h;
  a.n = q.n;
  a.xq = q.xq;
  a.xs = q.xs;
  a.ldx = q.ldx;
  a.ldg = q.ldg;
  a.ldr = q.ldr;
  a.ldh = q.ldh;
  a.ldn = q.ldn;
  a.ldq = q.ldq;
  a.xs_sm = q.xs_sm;
  a.xs_sk = q.xs_sk;
  return launch_quant_norm(a, x_bf16, h_bf16, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_expert_plan(const void* ids, int32_t ids_bytes, int64_t M, int64_t top, int64_t n_experts,
                             int32_t* offsets, int32_t* rows, int32_t* slots, void* stream) {
  if (M < 0 || top < 1 || n_experts < 1) return fail(BSF8_E_INVALID_ARG, "M %lld, top %lld or n_experts %lld",
                                                     (long long)M, (long long)top, (long long)n_experts);
  if (ids_bytes != 4 && ids_bytes != 8) return fail(BSF8_E_INVALID_ARG, "ids of %d bytes (4 or 8)", ids_bytes);
  if (offsets == nullptr || (M > 0 && (ids == nullptr || rows == nullptr || slots == nullptr)))
    return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (top > INT32_MAX || M > INT32_MAX / top || n_experts > 65535)
    return fail(BSF8_E_UNSUPPORTED, "M * top beyond 2^31 - 1, or n_experts beyond 65535");
  if (reinterpret_cast<uintptr_t>(ids) % uintptr_t(ids_bytes) || reinterpret_cast<uintptr_t>(offsets) % 4 ||
      reinterpret_cast<uintptr_t>(rows) % 4 || reinterpret_cast<uintptr_t>(slots) % 4)
    return fail(BSF8_E_ALIGNMENT, "ids or an output not element aligned");
  return launch_expert_plan(ids, ids_bytes == 8, M, top, n_experts, offsets, rows, slots,
                            static_cast<hipStream_t>(stream));
}

// ---- heads of tokens and the paged cache

// Whether `n` dimensions of `size` elements at `stride` above `width` adjacent elements keep all elements apart:
// ordered by stride, each steps over what lies within it.
static bool strides_apart(int64_t width, const int64_t* size, const int64_t* stride, int n) {
  bool used[4] = {};
  int64_t within = width;   // elements from the first to the last address of what is inside, counted with it
  for (int k = 0; k < n; ++k) {
    int at = -1;
    for (int i = 0; i < n; ++i)
      if (!used[i] && (at < 0 || stride[i] < stride[at] || (stride[i] == stride[at] && size[i] < size[at]))) at = i;
    used[at] = true;
    if (size[at] <= 1) continue;
    if (stride[at] < within) return false;
    if (stride[at] > (INT64_MAX / 8 - within) / (size[at] - 1)) return false;   // (no memory has as many bytes)
    within += stride[at] * (size[at] - 1);
  }
  return true;
}

static bsf8_status cache_checks(const bsf8_cache* p, CacheDev* out) {
  if (p == nullptr) return fail(BSF8_E_INVALID_ARG, "null cache");
  const bsf8_cache& c = *p;
  const bool e4m3 = c.dtype == BSF8_DT_F8_E4M3;
  if (!e4m3 && c.dtype != BSF8_DT_BF16) return fail(BSF8_E_INVALID_ARG, "cache dtype %d (F8_E4M3 or BF16)", c.dtype);
  if (c.heads < 1 || c.head_dim < 1 || c.page_size < 1 || c.n_pages < 1)
    return fail(BSF8_E_INVALID_ARG, "cache of %d heads of %d, %lld pages of %d rows", c.heads, c.head_dim,
                (long long)c.n_pages, c.page_size);
  if (c.k == nullptr || c.v == nullptr) return fail(BSF8_E_INVALID_ARG, "null cache pointer");
  if (e4m3 != (c.k_scale != nullptr) || e4m3 != (c.v_scale != nullptr))
    return fail(BSF8_E_INVALID_ARG, "an E4M3 cache has k_scale and v_scale, a BF16 cache neither");
  if (c.head_dim % 16 || c.head_dim > BSF8_CACHE_MAX_HEAD_DIM)
    return fail(BSF8_E_UNSUPPORTED, "head_dim %d (a multiple of 16 up to %d)", c.head_dim, BSF8_CACHE_MAX_HEAD_DIM);
  if (c.n_pages > INT32_MAX / c.page_size) return fail(BSF8_E_UNSUPPORTED, "n_pages * page_size beyond 2^31 - 1");
  const int64_t size[4] = {c.n_pages, c.page_size, c.heads, ceil_div(c.head_dim, kBlock)};
  const int64_t at[3] = {c.page, c.row, c.head}, s_at[4] = {c.s_page, c.s_row, c.s_head, c.s_group};
  for (int i = 0; i < 3; ++i)
    if (at[i] < 0 || at[i] > INT64_MAX / 16) return fail(BSF8_E_INVALID_ARG, "cache stride %lld", (long long)at[i]);
  if (!strides_apart(c.head_dim, size, at, 3)) return fail(BSF8_E_INVALID_ARG, "cache strides let elements share an address");
  const int64_t esz = e4m3 ? 1 : 2;
  if (reinterpret_cast<uintptr_t>(c.k) % 16 || reinterpret_cast<uintptr_t>(c.v) % 16 || c.page * esz % 16 ||
      c.row * esz % 16 || c.head * esz % 16)
    return fail(BSF8_E_ALIGNMENT, "cache addresses and strides are multiples of 16 bytes");
  if (c.row > (int64_t(1) << 27) / esz || c.page > UINT32_MAX / esz)
    return fail(BSF8_E_UNSUPPORTED, "cache rows further apart than 2^27 bytes, or pages than 2^32 - 1");
  CacheDev d{};
  if (e4m3) {
    for (int i = 0; i < 4; ++i)
      if (s_at[i] < 0) return fail(BSF8_E_INVALID_ARG, "negative scale stride");
    if (!strides_apart(1, size, s_at, 4)) return fail(BSF8_E_INVALID_ARG, "scale strides let elements share an address");
    if (reinterpret_cast<uintptr_t>(c.k_scale) % 4 || reinterpret_cast<uintptr_t>(c.v_scale) % 4)
      return fail(BSF8_E_ALIGNMENT, "a scale address is not element aligned");
    if (c.s_row > (int64_t(1) << 25) || c.s_page > UINT32_MAX)
      return fail(BSF8_E_UNSUPPORTED, "scale rows further apart than 2^25 elements, or pages than 2^32 - 1");
    d.k_scale = c.k_scale;
    d.v_scale = c.v_scale;
    d.s_page = c.s_page;
    d.s_row = c.s_row;
    d.s_head = c.s_head;
    d.s_group = c.s_group;
  }
  if (out == nullptr) return BSF8_OK;
  d.k = static_cast<uint8_t*>(c.k);
  d.v = static_cast<uint8_t*>(c.v);
  d.page = c.page * esz;
  d.row = c.row * esz;
  d.head = c.head * esz;
  d.heads = c.heads;
  d.head_dim = c.head_dim;
  d.page_size = c.page_size;
  d.n_pages = int32_t(c.n_pages);
  d.rows = int32_t(c.n_pages * c.page_size);
  d.e4m3 = e4m3 ? 1 : 0;
  // T. Granlund and P. Montgomery, "Division by invariant integers using multiplication", 1994
  int l = 0;
  while ((int64_t(1) << l) < c.page_size) ++l;
  d.magic = uint32_t((uint64_t(1) << (31 + l)) / uint64_t(c.page_size) + 1);
  d.shift = uint32_t(31 + l);
  *out = d;
  return BSF8_OK;
}

bsf8_status bsf8_cache_validate(const bsf8_cache* cache) { return cache_checks(cache, nullptr); }

// Heads of M tokens: M > 0.  heads < 0: any number; out: no two elements at one address.
static bsf8_status heads_checks(const char* name, const bsf8_heads& h, int64_t M, int32_t D, int32_t heads, bool out,
                                HeadsDev* dev) {
  if (!dtype_ok(h.dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "%s dtype %d (F32 or BF16)", name, h.dtype);
  if (h.heads < 1 || (heads >= 0 && h.heads != heads)) return fail(BSF8_E_INVALID_ARG, "%s has %d heads", name, h.heads);
  if (h.data == nullptr) return fail(BSF8_E_INVALID_ARG, "%s is null", name);
  if (h.token < 0 || h.head < 0) return fail(BSF8_E_INVALID_ARG, "%s has a negative stride", name);
  if (M > INT32_MAX / h.heads) return fail(BSF8_E_UNSUPPORTED, "%s: M * heads beyond 2^31 - 1", name);
  const int64_t size[2] = {M, h.heads}, stride[2] = {h.token, h.head};
  if (out && !strides_apart(D, size, stride, 2)) return fail(BSF8_E_INVALID_ARG, "%s: elements share an address", name);
  if (h.token > INT64_MAX / 8 / M || h.head > INT64_MAX / 8 / h.heads)
    return fail(BSF8_E_INVALID_ARG, "%s: strides beyond any memory", name);
  const int64_t esz = h.dtype == BSF8_DT_BF16 ? 2 : 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(h.data);
  if (at % uintptr_t(esz)) return fail(BSF8_E_ALIGNMENT, "%s is not element aligned", name);
  dev->p = h.data;
  dev->token = h.token;
  dev->head = h.head;
  dev->heads = h.heads;
  dev->bf16 = esz == 2 ? 1 : 0;
  dev->vec = at % 16 == 0 && (M == 1 || h.token * esz % 16 == 0) && (h.heads == 1 || h.head * esz % 16 == 0) ? 1 : 0;
  return BSF8_OK;
}

// What bsf8_rope and bsf8_cache_write have in common: the rotation and the queries.  keys: the rope has keys of its own.
static bsf8_status rope_checks(const bsf8_rope_args& r, bool keys, HeadsJob* a) {
  if (r.M < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (r.head_dim < 1 || r.rotary_dim < 0 || r.rotary_dim > r.head_dim || r.rotary_dim % 2)
    return fail(BSF8_E_INVALID_ARG, "rotary_dim %d of head_dim %d (even, up to head_dim)", r.rotary_dim, r.head_dim);
  if (r.head_dim % 16 || r.head_dim > BSF8_CACHE_MAX_HEAD_DIM)
    return fail(BSF8_E_UNSUPPORTED, "head_dim %d (a multiple of 16 up to %d)", r.head_dim, BSF8_CACHE_MAX_HEAD_DIM);
  if (r.pairing != BSF8_PAIR_HALF && r.pairing != BSF8_PAIR_ADJACENT) return fail(BSF8_E_INVALID_ARG, "pairing %d", r.pairing);
  if (!keys && (r.k.data || r.k_out.data)) return fail(BSF8_E_INVALID_ARG, "the keys of a cache write are its own");
  if (r.q_weight || r.k_weight) {
    if (!dtype_ok(r.weight_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "weight dtype %d (F32 or BF16)", r.weight_dtype);
    if (!(r.eps > 0.0) || !std::isfinite(r.eps)) return fail(BSF8_E_INVALID_ARG, "eps %g (positive)", r.eps);
  }
  if (r.rotary_dim) {
    if (r.n_axes < 1 || r.n_axes > BSF8_ROPE_MAX_AXES) return fail(BSF8_E_INVALID_ARG, "%d axes (1 to %d)", r.n_axes, BSF8_ROPE_MAX_AXES);
    if (r.position_bytes != 4 && r.position_bytes != 8) return fail(BSF8_E_INVALID_ARG, "positions of %d bytes (4 or 8)", r.position_bytes);
    if (!std::isfinite(r.scale)) return fail(BSF8_E_INVALID_ARG, "scale %g", r.scale);
    if (r.axis)
      for (int i = 0; i < r.rotary_dim / 2; ++i)
        if (r.axis[i] >= r.n_axes) return fail(BSF8_E_INVALID_ARG, "pair %d is on axis %d of %d", i, r.axis[i], r.n_axes);
  }
  a->D = r.head_dim;
  a->R = r.rotary_dim;
  a->half = r.pairing == BSF8_PAIR_HALF ? 1 : 0;
  if (r.M == 0) return BSF8_OK;
  // (heads of no tokens may have no address: only from here on is NULL what is absent)
  if (r.q.data == nullptr && r.q_out.data != nullptr) return fail(BSF8_E_INVALID_ARG, "q_out without q");
  if (r.q.data == nullptr && r.q_weight) return fail(BSF8_E_INVALID_ARG, "q_weight without q");
  if (keys && r.k.data == nullptr && (r.k_out.data || r.k_weight)) return fail(BSF8_E_INVALID_ARG, "k_out or k_weight without k");
  if (r.M > INT32_MAX) return fail(BSF8_E_UNSUPPORTED, "M too large");
  if (r.rotary_dim) {
    if (r.positions == nullptr || r.inv_freq == nullptr) return fail(BSF8_E_INVALID_ARG, "null positions or inv_freq");
    if (r.ld_axis < 0 || (r.n_axes > 1 && r.ld_axis > INT64_MAX / 32)) return fail(BSF8_E_INVALID_ARG, "ld_axis %lld", (long long)r.ld_axis);
    if (reinterpret_cast<uintptr_t>(r.positions) % uintptr_t(r.position_bytes) || reinterpret_cast<uintptr_t>(r.inv_freq) % 4)
      return fail(BSF8_E_ALIGNMENT, "positions or inv_freq not element aligned");
    a->n_axes = r.axis ? r.n_axes : 1;
    a->pos64 = r.position_bytes == 8 ? 1 : 0;
    a->ld_axis = r.ld_axis;
    a->pos = r.positions;
    a->inv_freq = r.inv_freq;
    a->scale = r.scale;
    if (r.axis)
      for (int i = 0; i < r.rotary_dim / 2; ++i) a->axis[i / 8] |= uint32_t(r.axis[i]) << (4 * (i % 8));
  }
  if (r.q_weight || r.k_weight) {
    a->w_bf16 = r.weight_dtype == BSF8_DT_BF16 ? 1 : 0;
    const uintptr_t both = reinterpret_cast<uintptr_t>(r.q_weight) | reinterpret_cast<uintptr_t>(r.k_weight);
    if (both % (a->w_bf16 ? 2 : 4)) return fail(BSF8_E_ALIGNMENT, "a weight is not element aligned");
    a->w_vec = both % 16 == 0 ? 1 : 0;
    a->qw = r.q_weight;
    a->kw = r.k_weight;
    a->eps = r.eps;
  }
  if (r.q.data) {
    bsf8_status st = heads_checks("q", r.q, r.M, r.head_dim, -1, false, &a->q);
    if (st == BSF8_OK) st = heads_checks("q_out", r.q_out, r.M, r.head_dim, r.q.heads, true, &a->q_out);
    if (st != BSF8_OK) return st;
  }
  if (r.k.data) {
    bsf8_status st = heads_checks("k", r.k, r.M, r.head_dim, -1, false, &a->k);
    if (st == BSF8_OK) st = heads_checks("k_out", r.k_out, r.M, r.head_dim, r.k.heads, true, &a->k_out);
    if (st != BSF8_OK) return st;
  }
  if (int64_t(a->q.heads) + a->k.heads > INT32_MAX / 4 || r.M > INT32_MAX / (int64_t(a->q.heads) + a->k.heads + 1))
    return fail(BSF8_E_UNSUPPORTED, "M * heads beyond 2^31 - 1");
  return BSF8_OK;
}

bsf8_status bsf8_rope(const bsf8_rope_args* args, void* stream) {
  if (args == nullptr) return fail(BSF8_E_INVALID_ARG, "null arguments");
  HeadsJob a{};
  const bsf8_status st = rope_checks(*args, true, &a);
  if (st != BSF8_OK || args->M == 0) return st;
  if (a.q.heads == 0 && a.k.heads == 0) return fail(BSF8_E_INVALID_ARG, "neither q nor k is given");
  return launch_heads(a, args->M, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_cache_write(const bsf8_cache* cache, int64_t M, const bsf8_heads* k, const bsf8_heads* v, const void* slots,
                             int32_t slot_bytes, const bsf8_rope_args* rope, void* stream) {
  HeadsJob a{};
  bsf8_status st = cache_checks(cache, &a.cache);
  if (st != BSF8_OK) return st;
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (slot_bytes != 4 && slot_bytes != 8) return fail(BSF8_E_INVALID_ARG, "slots of %d bytes (4 or 8)", slot_bytes);
  if (rope) {
    if (rope->M != M || rope->head_dim != cache->head_dim)
      return fail(BSF8_E_INVALID_ARG, "rope of M %lld, head_dim %d", (long long)rope->M, rope->head_dim);
    st = rope_checks(*rope, false, &a);
    if (st != BSF8_OK) return st;
  }
  if (M == 0) return BSF8_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (M > INT32_MAX / (2 * int64_t(cache->heads) + a.q.heads + 1)) return fail(BSF8_E_UNSUPPORTED, "M * heads beyond 2^31 - 1");
  st = heads_checks("k", *k, M, cache->head_dim, cache->heads, false, &a.k);
  if (st == BSF8_OK) st = heads_checks("v", *v, M, cache->head_dim, cache->heads, false, &a.v);
  if (st != BSF8_OK) return st;
  if (reinterpret_cast<uintptr_t>(slots) % uintptr_t(slot_bytes)) return fail(BSF8_E_ALIGNMENT, "slots not element aligned");
  a.D = cache->head_dim;
  a.to_cache = 1;
  a.slots = slots;
  a.slot64 = slot_bytes == 8 ? 1 : 0;
  return launch_heads(a, M, static_cast<hipStream_t>(stream));
}

static bsf8_status table_checks(const bsf8_cache& c, int64_t B, const int32_t* table, int64_t ld_table, int64_t pages) {
  if (table == nullptr) return fail(BSF8_E_INVALID_ARG, "null table");
  if (pages < 1 || (B > 1 && ld_table < pages)) return fail(BSF8_E_INVALID_ARG, "table of %lld pages, pitch %lld", (long long)pages, (long long)ld_table);
  if (reinterpret_cast<uintptr_t>(table) % 4) return fail(BSF8_E_ALIGNMENT, "table not element aligned");
  if (B > INT32_MAX || pages > INT32_MAX / c.page_size) return fail(BSF8_E_UNSUPPORTED, "B, or pages * page_size, beyond 2^31 - 1");
  if (B > 1 && ld_table > INT64_MAX / 8 / B) return fail(BSF8_E_INVALID_ARG, "table pitch beyond any memory");
  return BSF8_OK;
}

bsf8_status bsf8_cache_read(const bsf8_cache* cache, int64_t B, const int32_t* table, int64_t ld_table, int64_t pages,
                            const int32_t* starts, const int32_t* offsets, int64_t R, const bsf8_heads* k_out,
                            const bsf8_heads* v_out, void* stream) {
  CacheDev c{};
  bsf8_status st = cache_checks(cache, &c);
  if (st != BSF8_OK) return st;
  if (B < 0 || R < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (B == 0 || R == 0) return BSF8_OK;
  HeadsDev k{}, v{};
  if ((k_out == nullptr || k_out->data == nullptr) && (v_out == nullptr || v_out->data == nullptr))
    return fail(BSF8_E_INVALID_ARG, "neither k_out nor v_out is given");
  if (offsets == nullptr) return fail(BSF8_E_INVALID_ARG, "null offsets");
  st = table_checks(*cache, B, table, ld_table, pages);
  if (st == BSF8_OK && k_out && k_out->data) st = heads_checks("k_out", *k_out, R, cache->head_dim, cache->heads, true, &k);
  if (st == BSF8_OK && v_out && v_out->data) st = heads_checks("v_out", *v_out, R, cache->head_dim, cache->heads, true, &v);
  if (st != BSF8_OK) return st;
  if (k.p && v.p && k.bf16 != v.bf16) return fail(BSF8_E_INVALID_ARG, "k_out and v_out of different types");
  if (reinterpret_cast<uintptr_t>(offsets) % 4 || reinterpret_cast<uintptr_t>(starts) % 4)
    return fail(BSF8_E_ALIGNMENT, "offsets or starts not element aligned");
  return launch_cache_read(c, B, table, ld_table, pages, starts, offsets, R, k, v, static_cast<hipStream_t>(stream));
}

// Shape checks that the attention and its workspace share; q_heads per key head whole.
static bsf8_status attention_shape(const bsf8_cache& cache, const CacheDev& c, int64_t B, int32_t q_heads, int64_t pages) {
  if (B < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (q_heads < 1 || q_heads % cache.heads) return fail(BSF8_E_INVALID_ARG, "%d query heads over %d", q_heads, cache.heads);
  if (pages < 1) return fail(BSF8_E_INVALID_ARG, "table of %lld pages", (long long)pages);
  if (B > INT32_MAX / q_heads || B * q_heads > (int64_t(1) << 24) - 1 || pages > (INT32_MAX - 4096) / cache.page_size ||
      attention_tiles(c, B, q_heads, pages * cache.page_size) > INT32_MAX / 2)
    return fail(BSF8_E_UNSUPPORTED, "B * heads, pages * page_size, or their product, too large");
  return BSF8_OK;
}

bsf8_status bsf8_attention_workspace_size(const bsf8_cache* cache, int64_t B, int32_t q_heads, int64_t pages, size_t* bytes) {
  if (bytes == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  *bytes = 0;
  CacheDev c{};
  bsf8_status st = cache_checks(cache, &c);
  if (st == BSF8_OK) st = attention_shape(*cache, c, B, q_heads, pages);
  if (st == BSF8_OK) *bytes = attention_workspace_bytes(c, B, q_heads, pages * cache->page_size);
  return st;
}

bsf8_status bsf8_paged_attention(const bsf8_cache* cache, const bsf8_attention_args* args, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  CacheDev c{};
  bsf8_status st = cache_checks(cache, &c);
  if (st != BSF8_OK) return st;
  if (args == nullptr) return fail(BSF8_E_INVALID_ARG, "null arguments");
  const bsf8_attention_args& a = *args;
  if (a.B < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (a.window < 0) return fail(BSF8_E_INVALID_ARG, "window %lld (0 or more)", (long long)a.window);
  if (!std::isfinite(a.scale)) return fail(BSF8_E_INVALID_ARG, "scale %g", a.scale);
  if (a.B == 0) return BSF8_OK;
  st = attention_shape(*cache, c, a.B, a.q.heads, a.pages);
  if (st != BSF8_OK) return st;
  HeadsDev q{}, out{};
  st = heads_checks("q", a.q, a.B, cache->head_dim, -1, false, &q);
  if (st == BSF8_OK) st = heads_checks("out", a.out, a.B, cache->head_dim, a.q.heads, true, &out);
  if (st == BSF8_OK) st = table_checks(*cache, a.B, a.table, a.ld_table, a.pages);
  if (st != BSF8_OK) return st;
  if (a.lens == nullptr) return fail(BSF8_E_INVALID_ARG, "null lens");
  if (reinterpret_cast<uintptr_t>(a.lens) % 4 || reinterpret_cast<uintptr_t>(a.lse) % 4)
    return fail(BSF8_E_ALIGNMENT, "lens or lse not element aligned");
  const size_t need = attention_workspace_bytes(c, a.B, a.q.heads, a.pages * cache->page_size);
  if (need) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(BSF8_E_WORKSPACE, "%zu bytes of workspace needed, %zu given", need, workspace ? workspace_bytes : size_t(0));
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(BSF8_E_ALIGNMENT, "workspace not 256-byte aligned");
  }
  return launch_attention(c, q, out, a.B, a.table, a.ld_table, a.pages, a.lens, a.window, a.scale, a.lse, workspace,
                          static_cast<hipStream_t>(stream));
}

// Workspace of the two-step form of bsf8_linear_w8a8_dynamic: the codes (row
// pitch K rounded up to 16 bytes), the K-major scales, then the W8A8 call's own
// workspace, each from a 256-byte boundary.
struct DynLayout {
  int64_t ldq;
  size_t xs_off, gemm_off, gemm_bytes, total;
};
static size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
static DynLayout dyn_layout(const WeightDev& d, int64_t M) {
  DynLayout L{};
  L.ldq = (int64_t(d.K) + 15) & ~int64_t(15);
  L.xs_off = round256(size_t(M) * size_t(L.ldq));
  L.gemm_off = L.xs_off + round256(size_t(M) * size_t(d.Kb) * sizeof(float));
  L.gemm_bytes = w8a8_workspace_bytes(d, M);
  L.total = L.gemm_off + L.gemm_bytes;
  return L;
}

bsf8_status bsf8_workspace_size(const bsf8_weight* w, int32_t arm, int64_t M, size_t* bytes) {
  if (w == nullptr || bytes == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative M");
  if (arm == BSF8_ARM_W8A16) *bytes = M ? w8a16_workspace_bytes(w->dev, M) : 0;
  else if (arm == BSF8_ARM_W8A8) *bytes = M ? w8a8_workspace_bytes(w->dev, M) : 0;
  else if (arm == BSF8_ARM_DENSE) *bytes = M ? dense_workspace_bytes(w->n_total, w->dev.K, M) : 0;
  else if (arm == BSF8_ARM_W8A8_DYNAMIC) *bytes = M ? dyn_layout(w->dev, M).total : 0;
  else if (arm == BSF8_ARM_W8A8_EPILOGUE) *bytes = M ? w8a8_epilogue_workspace_bytes(w->dev, M) : 0;
  else return fail(BSF8_E_INVALID_ARG, "arm %d", arm);
  return BSF8_OK;
}

bsf8_status bsf8_upcast(const bsf8_weight* w, void* out, int32_t out_dtype, int64_t ldo, void* stream) {
  if (w == nullptr || out == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (!dtype_ok(out_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "out dtype %d (F32 or BF16)", out_dtype);
  if (ldo < w->dev.K) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  const size_t esz = out_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(out) % esz) return fail(BSF8_E_ALIGNMENT, "out not element aligned");
  const bool vec = w->aligned16 && reinterpret_cast<uintptr_t>(out) % 16 == 0 && (ldo * int64_t(esz)) % 16 == 0;
  return launch_upcast(w->dev, w->n_total, vec, out, out_dtype == BSF8_DT_BF16, ldo, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_dense_workspace_size(int64_t N, int64_t K, int64_t M, size_t* bytes) {
  if (bytes == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (N <= 0 || K <= 0 || M < 0) return fail(BSF8_E_INVALID_ARG, "sizes N=%lld K=%lld M=%lld", (long long)N,
                                             (long long)K, (long long)M);
  *bytes = dense_workspace_bytes(N, K, M);
  return BSF8_OK;
}

bsf8_status bsf8_linear_dense(const uint16_t* wd, int64_t N, int64_t K, const uint16_t* x, int64_t M, int64_t ldx,
                              void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (N <= 0 || K <= 0 || M < 0) return fail(BSF8_E_INVALID_ARG, "sizes N=%lld K=%lld M=%lld", (long long)N,
                                             (long long)K, (long long)M);
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0) return BSF8_OK;
  if (wd == nullptr || x == nullptr || y == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldx < K || ldy < N) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  const size_t ye = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (K % 8 || ldx % 8 || reinterpret_cast<uintptr_t>(wd) % 16 || reinterpret_cast<uintptr_t>(x) % 16)
    return fail(BSF8_E_ALIGNMENT, "dense GEMM needs K and ldx multiples of 8 and 16-byte aligned wd and x");
  if (reinterpret_cast<uintptr_t>(y) % ye) return fail(BSF8_E_ALIGNMENT, "y not element aligned");
  if (M == 1) ldx = K;   // one row has no pitch
  if (!dense_supported(N, K, M, ldx))
    return fail(BSF8_E_UNSUPPORTED, "dense GEMM shape N=%lld K=%lld M=%lld ldx=%lld (K <= 65536 and operands "
                "below 2 GiB)", (long long)N, (long long)K, (long long)M, (long long)ldx);
  const size_t need = dense_workspace_bytes(N, K, M);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(BSF8_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
  if (workspace != nullptr && reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(BSF8_E_ALIGNMENT, "workspace not 256-byte aligned");
  return launch_dense(wd, N, K, x, M, ldx, y, y_dtype == BSF8_DT_BF16, ldy, workspace, workspace_bytes,
                      static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_linear_w8a16(const bsf8_weight* w, const void* x, int32_t x_dtype, int64_t M, int64_t ldx,
                              void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative M");
  if (!dtype_ok(x_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "x dtype %d (F32 or BF16)", x_dtype);
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0) return BSF8_OK;
  if (x == nullptr || y == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldx < w->dev.K || ldy < w->n_total) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (M > INT32_MAX / 2) return fail(BSF8_E_UNSUPPORTED, "M too large");
  const size_t xe = x_dtype == BSF8_DT_F32 ? 4 : 2, ye = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % xe || reinterpret_cast<uintptr_t>(y) % ye)
    return fail(BSF8_E_ALIGNMENT, "x or y not element aligned");
  const size_t need = w8a16_workspace_bytes(w->dev, M);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(BSF8_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
  if (workspace != nullptr && reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(BSF8_E_ALIGNMENT, "workspace not 256-byte aligned");
  const bool aligned = w->aligned16 && (reinterpret_cast<uintptr_t>(x) % 16 == 0) && ((ldx * xe) % 16 == 0);
  return launch_w8a16(w->dev, aligned, x, x_dtype == BSF8_DT_BF16, M, ldx, y, y_dtype == BSF8_DT_BF16, ldy,
                      workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_linear_w8a8(const bsf8_weight* w, const uint8_t* xq, int64_t ldq, const float* xs, int64_t xs_sm,
                             int64_t xs_sk,
                             int64_t M, void* y, int32_t y_dtype, int64_t ldy, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative M");
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0) return BSF8_OK;
  if (xq == nullptr || xs == nullptr || y == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldq < w->dev.K || ldy < w->n_total) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (!scale_layout_ok(M, w->dev.Kb, xs_sm, xs_sk))
    return fail(BSF8_E_INVALID_ARG, "xs strides (%lld, %lld): neither token-major nor K-major", (long long)xs_sm,
                (long long)xs_sk);
  if (M > INT32_MAX / 2) return fail(BSF8_E_UNSUPPORTED, "M too large");
  const size_t ye = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(xs) % 4 || reinterpret_cast<uintptr_t>(y) % ye)
    return fail(BSF8_E_ALIGNMENT, "xs or y not element aligned");
  const size_t need = w8a8_workspace_bytes(w->dev, M);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(BSF8_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
  if (workspace != nullptr && reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(BSF8_E_ALIGNMENT, "workspace not 256-byte aligned");
  const bool aligned = w->aligned16 && (reinterpret_cast<uintptr_t>(xq) % 16 == 0) && (ldq % 16 == 0);
  return launch_w8a8(w->dev, aligned, xq, ldq, xs, xs_sm, xs_sk, M, y, y_dtype == BSF8_DT_BF16, ldy, workspace,
                     workspace_bytes, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_linear_w8a8_dynamic(const bsf8_weight* w, const void* x, int32_t x_dtype, int64_t M, int64_t ldx,
                                     void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative M");
  if (!dtype_ok(x_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "x dtype %d (F32 or BF16)", x_dtype);
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0) return BSF8_OK;
  if (x == nullptr || y == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldx < w->dev.K || ldy < w->n_total) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (M > INT32_MAX / 2) return fail(BSF8_E_UNSUPPORTED, "M too large");
  const size_t xe = x_dtype == BSF8_DT_F32 ? 4 : 2, ye = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % xe || reinterpret_cast<uintptr_t>(y) % ye)
    return fail(BSF8_E_ALIGNMENT, "x or y not element aligned");
  const bool x_bf16 = x_dtype == BSF8_DT_BF16, y_bf16 = y_dtype == BSF8_DT_BF16;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool aligned = w->aligned16 && (reinterpret_cast<uintptr_t>(x) % 16 == 0) && ((ldx * int64_t(xe)) % 16 == 0);
  if (w8a8_dyn_stream_applies(w->dev, aligned, M, ldx * int64_t(xe)))
    return launch_w8a8_dyn_stream(w->dev, x, x_bf16, M, ldx, y, y_bf16, ldy, st);
  // two steps: the quantizer into the workspace, then the W8A8 kernels
  const DynLayout L = dyn_layout(w->dev, M);
  if (workspace == nullptr || workspace_bytes < L.total)
    return fail(BSF8_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", L.total, workspace ? workspace_bytes : 0);
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(BSF8_E_ALIGNMENT, "workspace not 256-byte aligned");
  uint8_t* base = static_cast<uint8_t*>(workspace);
  uint8_t* xq = base;
  float* xs = reinterpret_cast<float*>(base + L.xs_off);
  const bsf8_status s1 = launch_quant_act(x, x_bf16, M, w->dev.K, ldx, xq, L.ldq, xs, 1, M, st);
  if (s1 != BSF8_OK) return s1;
  return launch_w8a8(w->dev, w->aligned16, xq, L.ldq, xs, 1, M, M, y, y_bf16, ldy,
                     L.gemm_bytes ? base + L.gemm_off : nullptr, L.gemm_bytes, st);
}

bsf8_status bsf8_linear_w8a8_epilogue(const bsf8_weight* w, const uint8_t* xq, int64_t ldq, const float* xs,
                                      int64_t xs_sm, int64_t xs_sk, int64_t M, const bsf8_epilogue* e, void* y,
                                      int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (e == nullptr) return fail(BSF8_E_INVALID_ARG, "null epilogue");
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative M");
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (e->activation < BSF8_ACT_NONE || e->activation > BSF8_ACT_GELU_TANH)
    return fail(BSF8_E_INVALID_ARG, "activation %d", e->activation);
  if ((e->bias && !dtype_ok(e->bias_dtype, true, true)) || (e->residual && !dtype_ok(e->residual_dtype, true, true)))
    return fail(BSF8_E_INVALID_ARG, "bias or residual dtype (F32 or BF16)");
  if (M == 0) return BSF8_OK;
  if (xq == nullptr || xs == nullptr || y == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (ldq < w->dev.K || ldy < w->n_total || (e->residual && e->ldr < w->n_total))
    return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (!scale_layout_ok(M, w->dev.Kb, xs_sm, xs_sk))
    return fail(BSF8_E_INVALID_ARG, "xs strides (%lld, %lld): neither token-major nor K-major", (long long)xs_sm,
                (long long)xs_sk);
  if (M > INT32_MAX / 2) return fail(BSF8_E_UNSUPPORTED, "M too large");
  const size_t ye = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(xs) % 4 || reinterpret_cast<uintptr_t>(y) % ye ||
      reinterpret_cast<uintptr_t>(e->bias) % (e->bias_dtype == BSF8_DT_BF16 ? 2 : 4) ||
      reinterpret_cast<uintptr_t>(e->residual) % (e->residual_dtype == BSF8_DT_BF16 ? 2 : 4))
    return fail(BSF8_E_ALIGNMENT, "xs, y, bias or residual not element aligned");
  EpilogueDev ep{};
  ep.bias = e->bias;
  ep.res = e->residual;
  ep.ldr = e->ldr;
  ep.alpha = e->residual_scale;
  ep.bias_bf16 = e->bias_dtype == BSF8_DT_BF16;
  ep.res_bf16 = e->residual_dtype == BSF8_DT_BF16;
  ep.act = e->activation;
  const size_t need = w8a8_epilogue_workspace_bytes(w->dev, M);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(BSF8_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
  if (workspace != nullptr && reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(BSF8_E_ALIGNMENT, "workspace not 256-byte aligned");
  const bool aligned = w->aligned16 && (reinterpret_cast<uintptr_t>(xq) % 16 == 0) && (ldq % 16 == 0);
  return launch_w8a8_epilogue(w->dev, aligned, xq, ldq, xs, xs_sm, xs_sk, M, ep, y, y_dtype == BSF8_DT_BF16, ldy,
                              workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

bsf8_status bsf8_experts_create(const bsf8_decl* decl, const bsf8_member_desc* members, int32_t n_members,
                                bsf8_experts** out) {
  if (out == nullptr) return fail(BSF8_E_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (decl == nullptr || (members == nullptr && n_members > 0)) return fail(BSF8_E_INVALID_ARG, "null descriptor");
  if (n_members < 1 || n_members > kMaxMembers)
    return fail(BSF8_E_GROUP, "%d members (1..%d allowed)", n_members, kMaxMembers);
  if (decl->block_n == 0 && decl->block_k == 0) return fail(BSF8_E_DECL, "experts need weight_block_size [128,128]");
  // one expert's slice of every member; a descriptor of another rank becomes
  // one that the slice's checks refuse by rank
  bsf8_member_desc slice[kMaxMembers];
  bsf8_tensor_desc grid[kMaxMembers][2];
  const auto cut = [](const bsf8_tensor_desc& t) {
    bsf8_tensor_desc s = t;
    s.rank = t.rank == 3 ? 2 : (t.rank < 0 || t.rank > 4 ? t.rank : 3);
    for (int d = 0; d + 1 < 4; ++d) s.shape[d] = t.shape[d + 1];
    return s;
  };
  for (int i = 0; i < n_members; ++i) {
    slice[i].weight = cut(members[i].weight);
    slice[i].scale_inv = slice[i].scale = nullptr;
    if (members[i].scale_inv) {
      grid[i][0] = cut(*members[i].scale_inv);
      slice[i].scale_inv = &grid[i][0];
    }
    if (members[i].scale) {
      grid[i][1] = cut(*members[i].scale);
      slice[i].scale = &grid[i][1];
    }
  }
  const bsf8_status st = validate_impl(decl, slice, n_members);
  if (st != BSF8_OK) return st;
  const int64_t E = members[0].weight.shape[0], K = slice[0].weight.shape[1];
  int64_t total = 0;
  for (int i = 0; i < n_members; ++i) {
    const bsf8_member_desc& m = members[i];
    if (m.weight.shape[0] <= 0) return fail(BSF8_E_WEIGHT_EMPTY, "member %d: %lld experts", i, (long long)m.weight.shape[0]);
    if (m.weight.shape[0] != E) return fail(BSF8_E_GROUP, "member %d: another number of experts than member 0", i);
    if (scale_leaf(m)->shape[0] != E) return fail(BSF8_E_SCALE_GRID, "member %d: grids of %lld experts, weights of %lld", i,
                                                  (long long)scale_leaf(m)->shape[0], (long long)E);
    if (m.weight.data == nullptr || scale_leaf(m)->data == nullptr)
      return fail(BSF8_E_INVALID_ARG, "member %d: a handle needs device addresses", i);
    total += m.weight.shape[1];
  }
  if (K > INT32_MAX / 2 || total > INT32_MAX / 2 || E > 65535)
    return fail(BSF8_E_UNSUPPORTED, "N or K beyond 2^30, or more than 65535 experts");
  bsf8_experts* h = new (std::nothrow) bsf8_experts();
  if (h == nullptr) return fail(BSF8_E_UNSUPPORTED, "out of host memory");
  std::memset(&h->dev, 0, sizeof(h->dev));
  h->dev.n_members = n_members;
  h->dev.K = int32_t(K);
  h->dev.Kb = int32_t(ceil_div(K, kBlock));
  h->dev.scale_bf16 = scale_leaf(members[0])->dtype == BSF8_DT_BF16 ? 1 : 0;
  h->dev.s_rs = h->dev.Kb;
  h->dev.s_cs = 1;
  h->n_experts = E;
  h->n_total = total;
  h->aligned16 = K % 16 == 0;
  int64_t col = 0;
  for (int i = 0; i < n_members; ++i) {
    h->dev.m[i].w = static_cast<const uint8_t*>(members[i].weight.data);
    h->dev.m[i].s = scale_leaf(members[i])->data;
    h->dev.m[i].rows = int32_t(members[i].weight.shape[1]);
    h->dev.m[i].col0 = int32_t(col);
    col += members[i].weight.shape[1];
  }
  *out = h;
  return BSF8_OK;
}

void bsf8_experts_destroy(bsf8_experts* w) { delete w; }

bsf8_status bsf8_experts_geometry(const bsf8_experts* w, int64_t* n_experts, int64_t* n_total, int64_t* k) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (n_experts) *n_experts = w->n_experts;
  if (n_total) *n_total = w->n_total;
  if (k) *k = w->dev.K;
  return BSF8_OK;
}

bsf8_status bsf8_linear_w8a8_experts(const bsf8_experts* w, const uint8_t* xq, int64_t ldq, const float* xs,
                                     int64_t xs_sm, int64_t xs_sk, int64_t M, const int32_t* offsets,
                                     const int32_t* rows, int64_t R, void* y, int32_t y_dtype, int64_t ldy,
                                     void* stream) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (M < 0 || R < 0) return fail(BSF8_E_INVALID_ARG, "negative M or R");
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (R == 0) return BSF8_OK;
  // (M == 0 with rows: every row is one without a token, and there is nothing to point at)
  if (M == 0) return fail(BSF8_E_INVALID_ARG, "%lld rows of no tokens", (long long)R);
  if (xq == nullptr || xs == nullptr || offsets == nullptr || y == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (rows == nullptr && M < R) return fail(BSF8_E_INVALID_ARG, "%lld tokens for %lld rows without gather rows", (long long)M, (long long)R);
  if (ldq < w->dev.K || ldy < w->n_total) return fail(BSF8_E_INVALID_ARG, "leading dimension too small");
  if (!scale_layout_ok(M, w->dev.Kb, xs_sm, xs_sk))
    return fail(BSF8_E_INVALID_ARG, "xs strides (%lld, %lld): neither token-major nor K-major", (long long)xs_sm,
                (long long)xs_sk);
  if (M > INT32_MAX / 2 || R > INT32_MAX / 2) return fail(BSF8_E_UNSUPPORTED, "M or R too large");
  const size_t ye = y_dtype == BSF8_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(xs) % 4 || reinterpret_cast<uintptr_t>(y) % ye ||
      reinterpret_cast<uintptr_t>(offsets) % 4 || reinterpret_cast<uintptr_t>(rows) % 4)
    return fail(BSF8_E_ALIGNMENT, "xs, offsets, rows or y not element aligned");
  const bool aligned = w->aligned16 && (reinterpret_cast<uintptr_t>(xq) % 16 == 0) && (ldq % 16 == 0);
  return launch_w8a8_experts(w->dev, w->n_experts, aligned, xq, ldq, xs, xs_sm, xs_sk, M, offsets, rows, R, y,
                             y_dtype == BSF8_DT_BF16, ldy, static_cast<hipStream_t>(stream));
}

const char* bsf8_experts_describe(const bsf8_experts* w, int64_t R) {
  if (w == nullptr) return nullptr;
  char geo[256];
  snprintf(geo, sizeof(geo), " | experts E=%lld N=%lld K=%d members=%d scales=%s", (long long)w->n_experts,
           (long long)w->n_total, w->dev.K, w->dev.n_members, w->dev.scale_bf16 ? "bf16" : "f32");
  return described(geo, [&] { return describe_w8a8_experts(w->dev, w->n_experts, w->aligned16, R > 0 ? R : 1); });
}

bsf8_status bsf8_linear_w8a8_noalloc(const bsf8_weight* w, const uint8_t* xq, int64_t ldq, const float* xs,
                                     int64_t xs_sm, int64_t xs_sk, int64_t M, void* y, int32_t y_dtype, int64_t ldy,
                                     void* stream) {
  if (w == nullptr) return fail(BSF8_E_INVALID_ARG, "null handle");
  if (M < 0) return fail(BSF8_E_INVALID_ARG, "negative M");
  if (!dtype_ok(y_dtype, true, true)) return fail(BSF8_E_INVALID_ARG, "y dtype %d (F32 or BF16)", y_dtype);
  if (M == 0) return BSF8_OK;
  const size_t need = w8a8_workspace_bytes(w->dev, M);
  if (need > size_t(BSF8_NOALLOC_SCRATCH_BYTES))
    return fail(BSF8_E_WORKSPACE,
                "this call needs %zu bytes of split-K partials; the no-allocation entry point holds %zu "
                "(BSF8_NOALLOC_SCRATCH_BYTES): call bsf8_linear_w8a8 with a workspace instead",
                need, size_t(BSF8_NOALLOC_SCRATCH_BYTES));
  void* scratch = nullptr;
  const bsf8_status st = w8a8_noalloc_scratch(&scratch);
  if (st != BSF8_OK) return st;
  return bsf8_linear_w8a8(w, xq, ldq, xs, xs_sm, xs_sk, M, y, y_dtype, ldy, scratch,
                          size_t(BSF8_NOALLOC_SCRATCH_BYTES), stream);
}

bsf8_status bsf8_read_stream(const void* p, int64_t bytes, uint32_t* sink, void* stream) {
  if (p == nullptr || sink == nullptr) return fail(BSF8_E_INVALID_ARG, "null pointer");
  if (bytes < 0) return fail(BSF8_E_INVALID_ARG, "negative size");
  if (reinterpret_cast<uintptr_t>(p) % 16 || bytes % 16 || reinterpret_cast<uintptr_t>(sink) % 4)
    return fail(BSF8_E_ALIGNMENT, "read_stream needs a 16-byte aligned pointer and size");
  if (bytes == 0) return BSF8_OK;
  return launch_read_stream(p, bytes, sink, static_cast<hipStream_t>(stream));
}

const char* bsf8_describe(const bsf8_weight* w, int32_t arm, int64_t M) {
  if (w == nullptr) return nullptr;
  char geo[256];
  snprintf(geo, sizeof(geo), " | weight N=%lld K=%d members=%d scales=%s%s", (long long)w->n_total, w->dev.K,
           w->dev.n_members, w->dev.scale_bf16 ? "bf16" : "f32", w->per_tensor ? " per-tensor" : "");
  return described(geo, [&]() -> std::string {
    switch (arm) {
      case BSF8_ARM_W8A16: return describe_w8a16(w->dev, w->aligned16, M);
      case BSF8_ARM_W8A8: return describe_w8a8(w->dev, w->aligned16, M);
      case BSF8_ARM_DENSE: return describe_dense(w->n_total, w->dev.K, M);
      case BSF8_ARM_W8A8_DYNAMIC:
        return w8a8_dyn_stream_applies(w->dev, w->aligned16, M > 0 ? M : 1, int64_t(w->dev.K) * 4)
                   ? describe_w8a8_dyn_stream(w->dev, M > 0 ? M : 1)
                   : "quant_act into the workspace (K-major scales), then " + describe_w8a8(w->dev, w->aligned16, M);
      case BSF8_ARM_W8A8_EPILOGUE: return describe_w8a8_epilogue(w->dev, w->aligned16, M > 0 ? M : 1);
      default: geo[0] = 0; return "unknown arm";
    }
  });
}

}  // extern "C"
