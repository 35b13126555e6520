// Device helpers shared by the selective scan's kernels.
#pragma once

#include "layer_util.cuh"
#include "kernels.h"
#include "state_space.h"

namespace wkv7 {

// log(1 + exp(v)) without overflow or cancellation, and its derivative's companion sigmoid.
__device__ __forceinline__ float softplus_of(float v) { return log1pf(expf(-fabsf(v))) + fmaxf(v, 0.f); }

// The step d_t of token row `bt` (= b T + t) for head h, and (optionally) its argument.
template <typename T>
__device__ __forceinline__ float step_of(const SsmArgs& p, int64_t bt, int64_t h, float* raw = nullptr) {
  float v = rows_ok(bt * p.dt_ld + h, 1, p.B * p.T, p.dt_ld, p.H, p.status) ? Elt<T>::to_f32(static_cast<const T*>(p.dt)[bt * p.dt_ld + h]) : 0.f;
  if (p.dt_bias) v += __ldg(p.dt_bias + h);
  if (raw) *raw = v;
  return p.softplus ? softplus_of(v) : v;
}

// A decay exp(d A) that is zero in fp32 (below 2^-150) cuts like a reset: nothing of what is before the token is left.
__device__ __forceinline__ bool cuts(float d, float A) { return d * A < -103.97208f; }

__host__ __device__ __forceinline__ int64_t chunks_of(int64_t T) { return (T + kSsmChunk - 1) / kSsmChunk; }

// Reverse sums inside segments over the 128 tokens of a chunk held by one warp, 4 consecutive tokens per lane:
// out[i] = sum of v from the token to the last token of its segment.  `cut` bit i: a new segment starts right after
// token i of this lane.
__device__ __forceinline__ void segmented_suffix(const double (&v)[4], unsigned cut, double (&out)[4]) {
  const unsigned lane = threadIdx.x & 31;
  double sum = 0.0;   // from this lane's first token to the first cut after it
  int open = 1;       // no cut met yet
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (open) sum += v[i];
    if (cut >> i & 1u) open = 0;
  }
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const double s2 = __shfl_down_sync(0xffffffffu, sum, o);
    const int o2 = __shfl_down_sync(0xffffffffu, open, o);
    if (lane + o < 32 && open) {
      sum += s2;
      open = o2;
    }
  }
  double run = __shfl_down_sync(0xffffffffu, sum, 1);
  if (lane == 31) run = 0.0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    run = (cut >> i & 1u) ? v[i] : run + v[i];
    out[i] = run;
  }
}

}  // namespace wkv7
