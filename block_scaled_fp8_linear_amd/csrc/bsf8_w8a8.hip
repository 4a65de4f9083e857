// W8A8 block-scaled GEMM on the gfx950 FP8 matrix cores.
//
// ("Module w8a8_prefill", section "WHY (#917 / #928)": FP8 x FP8 products
//  accumulated in F32, each 128-wide K slice rescaled by the token's group scale
//  times the weight block scale in an F32 epilogue; "FP8 Native Serving",
//  section "Native FP8 vs dequant-to-BF16": FP8 operands go straight into the
//  matrix unit and results become BF16 only when written back.)
//
// Design for CDNA4:
//  * Y^T tile = W tile . Xq^T: the weight rows are the MFMA A operand (16 rows
//    of N) and the quantized tokens the B operand (16 columns of M).  Both are
//    K-contiguous in HBM, exactly what v_mfma_f32_16x16x128_f8f6f4 reads per
//    lane (32 consecutive K bytes of one row), so neither operand is repacked.
//  * One 16x16x128 MFMA covers exactly one 128-wide scale block, so its result
//    is the block partial P of the method; the epilogue is one FMA per output
//    per K block: acc += P * (sa[m,kb] * sw[row block,kb]).
//  * Block tile 256 (N) x 128 (M), four waves of 128 x 64.  Tiles are laid out
//    member by member from each member's own row 0, so a wave's 128 rows are
//    exactly one row of that member's scale grid: sw is one scalar per wave and
//    K block (member-local origins come for free).
//  * Operands are staged through LDS, double-buffered, 128 bytes per row per K
//    block with the 16-byte chunks XOR-swizzled by (row & 7), which makes both
//    the staging writes and the MFMA fragment reads bank-conflict free.
//  * Tails: rows past a member's end, tokens past M and K bytes past K are
//    loaded as zeros (so a NaN code beyond K can never reach a product) and
//    never stored.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdio>
#include <mutex>
#include <string>

#include "bsf8_tile.h"

namespace bsf8 {
namespace {

constexpr int THREADS = 256;
constexpr int WN = 128;        // rows per wave
constexpr int WM = 64;         // tokens per wave
constexpr int TI = WN / 16;    // 8 MFMA row tiles per wave
constexpr int TJ = WM / 16;    // 4 MFMA column tiles per wave
constexpr int A_CHUNKS = BN * KBYTES / 16 / THREADS;  // 8 16-byte chunks per thread
constexpr int B_CHUNKS = BM * KBYTES / 16 / THREADS;  // 4
constexpr int STAGE_BYTES = (BN + BM) * KBYTES;        // 48 KiB

struct GemmArgs {
  WeightDev w;
  TileMap tm;
  const uint8_t* xq;
  const float* xs;
  void* y;
  int64_t ldq;
  int64_t xs_sm;   // activation scale (m, kb) at xs[m * xs_sm + kb * xs_sk]
  int64_t xs_sk;
  int64_t ldy;
  int32_t M;
  int32_t m_tiles;
  int32_t y_bf16;
};
template <bool ALIGNED>
__global__ __launch_bounds__(THREADS) void w8a8_gemm_kernel(GemmArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE_BYTES];

  // ---- tile of this block: member, row tile, token tile
  const int t = blockIdx.x;
  int mi = 0;
  while (mi + 1 < a.w.n_members && t >= a.tm.tile0[mi + 1]) ++mi;
  const int local = t - a.tm.tile0[mi];
  const int nt = local % a.tm.n_tiles[mi];
  const int mt = local / a.tm.n_tiles[mi];
  const MemberDev mem = a.w.m[mi];
  const int n0 = nt * BN;
  const int m0 = mt * BM;
  const int K = a.w.K, Kb = a.w.Kb, M = a.M;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wn = wave & 1, wm = wave >> 1;
  const int l16 = lane & 15, g = lane >> 4;

  // ---- staging geometry: each thread owns fixed (row, chunk) slots
  // Thread tid always stages chunk (tid & 7) of rows (tid >> 3) + 32 i.
  const int ch16 = (tid & 7) * 16;
  const uint8_t* a_row[A_CHUNKS];
  bool a_ok[A_CHUNKS];
  int a_dst[A_CHUNKS];
#pragma unroll
  for (int i = 0; i < A_CHUNKS; ++i) {
    const int c = tid + THREADS * i, row = c >> 3, ch = c & 7;
    a_ok[i] = (n0 + row) < mem.rows;
    a_row[i] = mem.w + int64_t(a_ok[i] ? n0 + row : 0) * K;
    a_dst[i] = swz(row, ch);
  }
  const uint8_t* b_row[B_CHUNKS];
  bool b_ok[B_CHUNKS];
  int b_dst[B_CHUNKS];
#pragma unroll
  for (int i = 0; i < B_CHUNKS; ++i) {
    const int c = tid + THREADS * i, row = c >> 3, ch = c & 7;
    b_ok[i] = (m0 + row) < M;
    b_row[i] = a.xq + int64_t(b_ok[i] ? m0 + row : 0) * a.ldq;
    b_dst[i] = BN * KBYTES + swz(row, ch);
  }

  // ---- scales: one weight scale per wave and K block, one token scale per column tile
  const int srow = (n0 + wn * WN) >> 7;
  const int nb = (mem.rows + 127) >> 7;
  const bool srow_ok = srow < nb;
  const int64_t s_base = int64_t(srow_ok ? srow : 0) * a.w.s_rs;
  const float* xs_row[TJ];
  bool m_ok[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int m = m0 + wm * WM + 16 * j + l16;
    m_ok[j] = m < M;
    xs_row[j] = a.xs + int64_t(m_ok[j] ? m : 0) * a.xs_sm;
  }

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  uint4 ra[A_CHUNKS], rb[B_CHUNKS];
  auto gload = [&](int kb) {
    const int k = kb * KBYTES + ch16;
#pragma unroll
    for (int i = 0; i < A_CHUNKS; ++i) ra[i] = load_chunk<ALIGNED>(a_row[i], k, K, a_ok[i]);
#pragma unroll
    for (int i = 0; i < B_CHUNKS; ++i) rb[i] = load_chunk<ALIGNED>(b_row[i], k, K, b_ok[i]);
  };
  auto lstore = [&](int stage) {
    uint8_t* base = smem + stage * STAGE_BYTES;
#pragma unroll
    for (int i = 0; i < A_CHUNKS; ++i) *reinterpret_cast<uint4*>(base + a_dst[i]) = ra[i];
#pragma unroll
    for (int i = 0; i < B_CHUNKS; ++i) *reinterpret_cast<uint4*>(base + b_dst[i]) = rb[i];
  };

  gload(0);
  lstore(0);
  __syncthreads();

  float sw_next = srow_ok ? load_scale(mem.s, s_base, a.w.scale_bf16) : 0.f;
  float sa_next[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) sa_next[j] = m_ok[j] ? xs_row[j][0] : 0.f;

  for (int kb = 0; kb < Kb; ++kb) {
    const int stage = kb & 1;
    const bool more = kb + 1 < Kb;
    if (more) gload(kb + 1);
    float s[TJ];
    const float sw = sw_next;
#pragma unroll
    for (int j = 0; j < TJ; ++j) s[j] = sa_next[j] * sw;
    if (more) {
      sw_next = srow_ok ? load_scale(mem.s, s_base + int64_t(kb + 1) * a.w.s_cs, a.w.scale_bf16) : 0.f;
#pragma unroll
      for (int j = 0; j < TJ; ++j) sa_next[j] = m_ok[j] ? xs_row[j][int64_t(kb + 1) * a.xs_sk] : 0.f;
    }

    const uint8_t* As = smem + stage * STAGE_BYTES;
    const uint8_t* Bs = As + BN * KBYTES;
    v8i bf[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int r = wm * WM + 16 * j + l16;
      const uint4 lo = *reinterpret_cast<const uint4*>(Bs + swz(r, 2 * g));
      const uint4 hi = *reinterpret_cast<const uint4*>(Bs + swz(r, 2 * g + 1));
      bf[j] = v8i{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int r = wn * WN + 16 * i + l16;
      const uint4 lo = *reinterpret_cast<const uint4*>(As + swz(r, 2 * g));
      const uint4 hi = *reinterpret_cast<const uint4*>(As + swz(r, 2 * g + 1));
      const v8i af = v8i{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af, bf[j], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                                       0, 0, 0);
        acc[i][j] += p * s[j];
      }
    }
    if (more) lstore(stage ^ 1);
    __syncthreads();
  }

  // ---- store: lane holds rows 4*(lane/16)+r of each 16x16 tile, column lane%16
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int m = m0 + wm * WM + 16 * j + l16;
    if (m >= M) continue;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int n = n0 + wn * WN + 16 * i + 4 * g;
      const int nvalid = mem.rows - n;
      if (nvalid <= 0) continue;
      store4(a.y, a.y_bf16, int64_t(m) * a.ldy + mem.col0 + n, nvalid, acc[i][j]);
    }
  }
}

}  // namespace

// An upper bound over the paths a call may take: the split plan of the fast
// kernel for packed activations (the register-staged kernel needs none).
size_t w8a8_workspace_bytes(const WeightDev& w, int64_t M) {
  if (M <= 0) return 0;
  return make_plan(w, true, M, w.K).ws_bytes;
}

std::string describe_w8a8(const WeightDev& w, bool aligned, int64_t M) {
  if (w8a8_stream_applies(w, aligned, M > 0 ? M : 1, w.K)) return describe_w8a8_stream(w, M > 0 ? M : 1);
  const Plan p = make_plan(w, aligned, M > 0 ? M : 1, w.K);
  char buf[320];
  if (p.fast)
    snprintf(buf, sizeof(buf),
             "arm=w8a8 arithmetic=e4m3xe4m3 mfma_f32_16x16x128_f8f6f4, f32 per-128-K epilogue | "
             "kernel=w8a8_gemm_fast tile=%dx%d waves=8 lds=2x%dKiB (two stage arrays) buffer_load_lds "
             "xcd_groups=%d split_k=%d split_row_tiles=%d | M=%lld blocks=%d",
             p.tile, p.tile, (p.tile == 256 ? FTile<256>::STAGE : FTile<128>::STAGE) / 1024,
             group_rows_for(p.m_tiles, p.rt_total * p.m_tiles, device_cus()), p.splits,
             p.rt_total - p.rt_split0, (long long)M, p.blocks);
  else
    snprintf(buf, sizeof(buf),
             "arm=w8a8 arithmetic=e4m3xe4m3 mfma_f32_16x16x128_f8f6f4, f32 per-128-K epilogue | "
             "kernel=w8a8_gemm tile=%dx%d waves=4 lds=2x%dKiB path=%s | M=%lld blocks=%d",
             BN, BM, STAGE_BYTES / 1024, aligned ? "aligned16" : "bytewise", (long long)M, p.blocks);
  return buf;
}

namespace {

// The dense BF16 weight [N, K] as the fast kernel's single member: rows of
// 2K bytes, no scales.
WeightDev dense_weight(const uint16_t* wd, int64_t N, int64_t K) {
  WeightDev w{};
  w.m[0].w = reinterpret_cast<const uint8_t*>(wd);
  w.m[0].s = nullptr;
  w.m[0].rows = int32_t(N);
  w.m[0].col0 = 0;
  w.n_members = 1;
  w.K = int32_t(2 * K);
  w.Kb = int32_t((2 * K + KBYTES - 1) / KBYTES);
  return w;
}

}  // namespace

bool dense_supported(int64_t N, int64_t K, int64_t M, int64_t ldx) {
  if (N <= 0 || K <= 0 || N > INT32_MAX || 2 * K > int64_t(F_MAX_KB) * KBYTES) return false;
  return make_plan(dense_weight(nullptr, N, K), true, M > 0 ? M : 1, 2 * ldx).fast;
}

size_t dense_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  if (M <= 0 || !dense_supported(N, K, M, K)) return 0;
  return make_plan(dense_weight(nullptr, N, K), true, M, 2 * K).ws_bytes;
}

std::string describe_dense(int64_t N, int64_t K, int64_t M) {
  const int64_t m = M > 0 ? M : 1;
  if (!dense_supported(N, K, m, K)) return "arm=dense unsupported shape";
  const Plan p = make_plan(dense_weight(nullptr, N, K), true, m, 2 * K);
  char buf[320];
  snprintf(buf, sizeof(buf),
           "arm=dense arithmetic=bf16xbf16 mfma_f32_16x16x32_bf16 (two per 128-byte K block), f32 accumulate | "
           "kernel=w8a8_gemm_fast<dense> tile=%dx%d waves=8 buffer_load_lds xcd_groups=%d split_k=%d "
           "split_row_tiles=%d | M=%lld blocks=%d | dense weight N=%lld K=%lld bf16",
           p.tile, p.tile, group_rows_for(p.m_tiles, p.rt_total * p.m_tiles, device_cus()), p.splits,
           p.rt_total - p.rt_split0, (long long)m, p.blocks, (long long)N,
           (long long)K);
  return buf;
}

bsf8_status launch_dense(const uint16_t* wd, int64_t N, int64_t K, const uint16_t* x, int64_t M, int64_t ldx,
                         void* y, bool y_bf16, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  const WeightDev w = dense_weight(wd, N, K);
  const Plan p = make_plan(w, true, M, 2 * ldx);
  if (!p.fast) {
    set_error("UNSUPPORTED: dense GEMM shape N=%lld K=%lld M=%lld", (long long)N, (long long)K, (long long)M);
    return BSF8_E_UNSUPPORTED;
  }
  if (p.blocks == 0) return BSF8_OK;
  return launch_fast<kDense>(p, w, reinterpret_cast<const uint8_t*>(x), 2 * ldx, nullptr, 0, 0, M, y, y_bf16, ldy,
                     ws, ws_bytes, stream);
}

// ---------------------------------------------------------------------------
// Scratch of the no-allocation entry point (bsf8_linear_w8a8_noalloc): the
// split-K partial tiles go here instead of a caller workspace.  Each device
// holds its own copy of this array from the library's load until the process
// ends.  Its name is only a host-side stand-in: kernels are given the device
// address hipGetSymbolAddress returns for the current device, looked up once
// per device and kept.  Nothing in it needs to start at zero (every split
// writes the whole partial tile it later reads), and calls that overlap in
// time on one device share it, so they race.
// ---------------------------------------------------------------------------
static __device__ __align__(256) uint8_t scratch[BSF8_NOALLOC_SCRATCH_BYTES];

namespace {
constexpr int kScratchDevices = 64;
std::atomic<void*> g_scratch[kScratchDevices];
std::mutex g_scratch_mu;
}  // namespace

bsf8_status w8a8_noalloc_scratch(void** ptr) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return device_status(e, "hipGetDevice");
  if (dev < 0 || dev >= kScratchDevices) {
    set_error("DEVICE: device index %d beyond the %d the no-allocation scratch table covers", dev, kScratchDevices);
    return BSF8_E_DEVICE;
  }
  void* p = g_scratch[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
      e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
      if (e != hipSuccess) return device_status(e, "hipGetSymbolAddress(scratch)");
      if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 255) != 0) {
        set_error("DEVICE: the no-allocation scratch has no 256-byte aligned device address");
        return BSF8_E_DEVICE;
      }
      g_scratch[dev].store(p, std::memory_order_release);
    }
  }
  *ptr = p;
  return BSF8_OK;
}

bsf8_status launch_w8a8(const WeightDev& w, bool aligned, const uint8_t* xq, int64_t ldq, const float* xs,
                        int64_t xs_sm, int64_t xs_sk, int64_t M, void* y, bool y_bf16, int64_t ldy, void* ws,
                        size_t ws_bytes, hipStream_t stream) {
  if (w8a8_stream_applies(w, aligned, M, ldq))
    return launch_w8a8_stream(w, xq, ldq, xs, xs_sm, xs_sk, M, y, y_bf16, ldy, stream);
  const Plan p = make_plan(w, aligned, M, ldq, (M - 1) * xs_sm + (w.Kb - 1) * xs_sk + 1);
  if (p.blocks == 0) return BSF8_OK;
  if (p.fast) return launch_fast<kPlain>(p, w, xq, ldq, xs, xs_sm, xs_sk, M, y, y_bf16, ldy, ws, ws_bytes, stream);
  GemmArgs a{};
  a.w = w;
  a.tm = p.tm;
  a.xq = xq;
  a.xs = xs;
  a.y = y;
  a.ldq = ldq;
  a.xs_sm = xs_sm;
  a.xs_sk = xs_sk;
  a.ldy = ldy;
  a.M = int32_t(M);
  a.m_tiles = p.m_tiles;
  a.y_bf16 = y_bf16 ? 1 : 0;
  if (aligned)
    hipLaunchKernelGGL(w8a8_gemm_kernel<true>, dim3(p.blocks), dim3(THREADS), 0, stream, a);
  else
    hipLaunchKernelGGL(w8a8_gemm_kernel<false>, dim3(p.blocks), dim3(THREADS), 0, stream, a);
  return device_status(hipGetLastError(), "w8a8_gemm launch");
}

}  // namespace bsf8
