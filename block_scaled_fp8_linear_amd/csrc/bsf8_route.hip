// Router choices -> the expert product's row order (gfx950): a stable counting
// sort of M * top expert numbers, in one launch without atomics.
//
// One block per expert e.  Its waves each take a contiguous part of the
// choices; a first sweep counts, per wave, the choices below e and those equal
// to e; the sum of the former is offsets[e], and offsets[e] plus the counts of
// the waves before gives each wave's first place.  A second sweep places the
// wave's choices in order, by ballots.  Blocks share nothing, so the result
// does not depend on timing, and every block reads all the choices twice (from
// the cache: 256 KiB for 65536 of them), which is cheaper than a second launch
// or a chain of blocks waiting for each other's counts.
// The operator moves 12 bytes per choice; what bounds it is the launch (2.5 us up
// to some thousand choices) and then the two sweeps' instructions, two comparisons
// per choice and block with the counts on the scalar unit, and the places: 65536
// choices of 128 experts 11.5-13.6 us (24 us with a test around every load, 17.5 us with
// the counts on the vector unit, 13.8 us with a division by top).  Groups of 8 or
// 16 steps' loads in place of 4 take as long or longer.
#include <hip/hip_runtime.h>

#include "bsf8_internal.h"

namespace bsf8 {
namespace {

constexpr int THREADS = 1024;
constexpr int WAVES = THREADS / 64;
constexpr int PER_LANE = 4;                    // consecutive choices per lane and step
constexpr int STEP = 64 * PER_LANE;

constexpr int GROUP = 4;                       // steps whose loads go out together

struct PlanArgs {
  const void* ids;
  int32_t* offsets;
  int32_t* rows;
  int32_t* slots;
  int32_t n;         // M * top
  int32_t E;
  uint32_t magic;    // i / top = i * magic >> shift
  int32_t shift;
};

// A lane's choices of one step.  16 bytes at a time from any address: the choices
// need only be element aligned.
template <typename T>
struct Ids {
  static constexpr int W = int(sizeof(T) * PER_LANE / 16);
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  typedef u4 __attribute__((aligned(4))) u4_any;
  u4 w[W];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const u4_any*>(p)[i];
  }
  // choice j as an unsigned number; 2^32 - 1 for one outside 32 bits (no expert: experts are below 65535)
  __device__ __forceinline__ uint32_t number(int j) const {
    if (sizeof(T) == 4) return w[0][j];
    return w[(j >> 1) % W][2 * (j & 1) + 1] ? ~0u : w[(j >> 1) % W][2 * (j & 1)];
  }
};

template <typename T>
__global__ __launch_bounds__(THREADS) void expert_plan_kernel(PlanArgs a) {
  __shared__ int32_t less[WAVES], equal[WAVES];
  const uint32_t e = blockIdx.x, E = uint32_t(a.E);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const T* ids = static_cast<const T*>(a.ids);
  // a wave's part: whole steps; only the choices' last step can be short
  const int steps_all = a.n / STEP + (a.n % STEP != 0), part = (steps_all + WAVES - 1) / WAVES;
  const int s_begin = min(steps_all, wave * part), s_end = min(steps_all, s_begin + part);
  const int s_full = min(s_end, a.n / STEP);
  const bool has_short = s_begin <= a.n / STEP && a.n / STEP < s_end;
  const auto at_lane = [&](int s) { return int64_t(s) * STEP + lane * PER_LANE; };
  // the short step's choices of this lane; `live`: choice j exists
  const auto live = [&](int j) { return at_lane(a.n / STEP) + j < a.n; };
  uint32_t tail_id[PER_LANE];
  if (has_short)
    for (int j = 0; j < PER_LANE; ++j) {
      tail_id[j] = ~0u;
      if (live(j)) {
        const T v = ids[at_lane(a.n / STEP) + j];
        tail_id[j] = v >= 0 && v < T(E) ? uint32_t(v) : ~0u;
      }
    }

  // counts by ballots: two comparisons per choice, the rest on the scalar unit
  int n_less = 0, n_equal = 0;
  const auto count = [&](uint32_t id) {
    n_less += __popcll(__ballot(id < e));
    n_equal += __popcll(__ballot(id == e));
  };
  int s = s_begin;
  for (; s + GROUP <= s_full; s += GROUP) {
    Ids<T> g[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) g[i].load(ids + at_lane(s + i));
#pragma unroll
    for (int i = 0; i < GROUP; ++i)
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j) count(g[i].number(j));
  }
  for (; s < s_full; ++s) {
    Ids<T> g;
    g.load(ids + at_lane(s));
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) count(g.number(j));
  }
  if (has_short)
    for (int j = 0; j < PER_LANE; ++j) count(tail_id[j]);
  if (lane == 0) {
    less[wave] = n_less;
    equal[wave] = n_equal;
  }
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    at += less[w] + (w < wave ? equal[w] : 0);
    all += less[w] + equal[w];
  }
  if (threadIdx.x == 0) {
    a.offsets[e] = at;                              // wave 0: the choices below e
    if (e == E - 1) a.offsets[a.E] = all;
  }
  if (n_equal == 0 && e != 0) return;               // nothing of this wave's part to place

  const auto place = [&](const uint32_t (&id)[PER_LANE], int64_t i0) {
    uint64_t hit[PER_LANE];
    int before = 0, total = 0;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      hit[j] = __ballot(id[j] == e);
      before = int(__builtin_amdgcn_mbcnt_hi(uint32_t(hit[j] >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(hit[j]), uint32_t(before))));
      total += __popcll(hit[j]);
    }
    if (total) {
      int p = at + before;
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j)
        if (id[j] == e) {
          a.rows[p] = int32_t(uint64_t(uint32_t(i0 + j)) * a.magic >> a.shift);
          a.slots[i0 + j] = p++;
        }
      at += total;
    }
    if (e == 0) {                                   // choices without an expert have no slot
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j)
        if (id[j] >= E && i0 + j < a.n) a.slots[i0 + j] = -1;
    }
  };
  s = s_begin;
  for (; s + GROUP <= s_full; s += GROUP) {
    Ids<T> g[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) g[i].load(ids + at_lane(s + i));
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      uint32_t id[PER_LANE];
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j) id[j] = g[i].number(j);
      place(id, at_lane(s + i));
    }
  }
  for (; s < s_full; ++s) {
    Ids<T> g;
    g.load(ids + at_lane(s));
    uint32_t id[PER_LANE];
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) id[j] = g.number(j);
    place(id, at_lane(s));
  }
  if (has_short) place(tail_id, at_lane(a.n / STEP));
}

}  // namespace

bsf8_status launch_expert_plan(const void* ids, bool ids64, int64_t M, int64_t top, int64_t E, int32_t* offsets,
                               int32_t* rows, int32_t* slots, hipStream_t stream) {
  PlanArgs a{};
  a.ids = ids;
  a.offsets = offsets;
  a.rows = rows;
  a.slots = slots;
  a.n = int32_t(M * top);
  a.E = int32_t(E);
  // The quotient of i < 2^31 by top without a division (T. Granlund and P. Montgomery, "Division by
  // invariant integers using multiplication", 1994): 2^l >= top, magic = floor(2^(31 + l) / top) + 1.
  int l = 0;
  while ((int64_t(1) << l) < top) ++l;
  a.magic = uint32_t((uint64_t(1) << (31 + l)) / uint64_t(top) + 1);
  a.shift = 31 + l;
  if (ids64)
    hipLaunchKernelGGL(expert_plan_kernel<int64_t>, dim3(unsigned(E)), dim3(THREADS), 0, stream, a);
  else
    hipLaunchKernelGGL(expert_plan_kernel<int32_t>, dim3(unsigned(E)), dim3(THREADS), 0, stream, a);
  return device_status(hipGetLastError(), "expert_plan launch");
}

}  // namespace bsf8
