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
// or a chain of blocks waiting for each other's counts.  The operator moves 12
// bytes per choice and is bound by latency at every size a router meets.
#include <hip/hip_runtime.h>

#include "bsf8_internal.h"

namespace bsf8 {
namespace {

constexpr int THREADS = 1024;
constexpr int WAVES = THREADS / 64;
constexpr int PER_LANE = 4;                    // consecutive choices per lane and step
constexpr int STEP = 64 * PER_LANE;

struct PlanArgs {
  const void* ids;
  int32_t* offsets;
  int32_t* rows;
  int32_t* slots;
  int32_t n;         // M * top
  int32_t top;
  int32_t E;
  int32_t vec;       // 16-byte loads of the choices
};

// PER_LANE choices from i0 on; -2 past the end (no expert, and no slot to write)
template <typename T>
__device__ __forceinline__ void load_ids(const PlanArgs& a, int64_t i0, int64_t end, int (&id)[PER_LANE]) {
  const T* p = static_cast<const T*>(a.ids);
  if (a.vec && i0 + PER_LANE <= end) {
    T v[PER_LANE];
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * PER_LANE / 16); ++i)
      reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(p + i0)[i];
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) id[j] = v[j] >= 0 && v[j] < a.E ? int(v[j]) : -1;
  } else {
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      id[j] = -2;
      if (i0 + j < end) {
        const T v = p[i0 + j];
        id[j] = v >= 0 && v < a.E ? int(v) : -1;
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(THREADS) void expert_plan_kernel(PlanArgs a) {
  __shared__ int32_t less[WAVES], equal[WAVES];
  const int e = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // a wave's part: whole steps, so that its loads stay aligned
  const int64_t part = (int64_t(a.n) + int64_t(WAVES) * STEP - 1) / (int64_t(WAVES) * STEP) * STEP;
  const int64_t begin = min(int64_t(a.n), wave * part), end = min(int64_t(a.n), begin + part);

  int n_less = 0, n_equal = 0;
#pragma unroll 4
  for (int64_t i = begin; i < end; i += STEP) {
    int id[PER_LANE];
    load_ids<T>(a, i + lane * PER_LANE, end, id);
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      n_less += id[j] >= 0 && id[j] < e ? 1 : 0;
      n_equal += id[j] == e ? 1 : 0;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    n_less += __shfl_xor(n_less, d, 64);
    n_equal += __shfl_xor(n_equal, d, 64);
  }
  if (lane == 0) {
    less[wave] = n_less;
    equal[wave] = n_equal;
  }
  __syncthreads();
  int at = 0, all = 0;
  for (int w = 0; w < WAVES; ++w) {
    at += less[w] + (w < wave ? equal[w] : 0);
    all += less[w] + equal[w];
  }
  if (threadIdx.x == 0) {
    a.offsets[e] = at;                              // wave 0: the choices below e
    if (e == a.E - 1) a.offsets[a.E] = all;
  }

  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (int64_t i = begin; i < end; i += STEP) {
    int id[PER_LANE];
    const int64_t i0 = i + lane * PER_LANE;
    load_ids<T>(a, i0, end, id);
    int before = 0, total = 0;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const uint64_t hit = __ballot(id[j] == e);
      before += __popcll(hit & below);
      total += __popcll(hit);
    }
    int place = at + before;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      if (id[j] == e) {
        a.rows[place] = int32_t((i0 + j) / a.top);
        a.slots[i0 + j] = place++;
      } else if (e == 0 && id[j] == -1) {
        a.slots[i0 + j] = -1;                       // no expert: no slot
      }
    }
    at += total;
  }
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
  a.top = int32_t(top);
  a.E = int32_t(E);
  a.vec = reinterpret_cast<uintptr_t>(ids) % 16 == 0 ? 1 : 0;
  if (ids64)
    hipLaunchKernelGGL(expert_plan_kernel<int64_t>, dim3(unsigned(E)), dim3(THREADS), 0, stream, a);
  else
    hipLaunchKernelGGL(expert_plan_kernel<int32_t>, dim3(unsigned(E)), dim3(THREADS), 0, stream, a);
  return device_status(hipGetLastError(), "expert_plan launch");
}

}  // namespace bsf8
