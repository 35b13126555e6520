// Device helpers shared by the state-space layer's streaming kernels.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace wkv7 {

// Debug build: elements [off, off + n) inside `rows` rows of `width` elements whose starts are `ld` apart.
__device__ __forceinline__ bool rows_ok(int64_t off, int64_t n, int64_t rows, int64_t ld, int64_t width, int* status) {
  return range_ok(off, n, (rows - 1) * ld + width, status);
}

// sigmoid(v), from which silu(v) = v sigmoid(v).  The 16-bit types use the hardware's exponential and reciprocal, five
// instructions instead of a dozen; fp32 uses the accurate ones.  Relative error: 2^-21 of the two, and for negative v up to
// |v| 2^-23 of rounding the exponent (2^-19 at -12, 2^-16.7 at -80): far below the half step of a 16-bit output.  The fp32
// gradients of the filter and the norm's weight that belong to 16-bit inputs have it in each of their terms.
// exp(-v) = inf for very negative v gives 0.
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
template <typename T>
__device__ __forceinline__ float sigmoid_of(float v) {
  if (sizeof(T) == 4) return 1.f / (1.f + expf(-v));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  return rcp_fast(1.f + e);
}

// N consecutive elements of T at p (N * sizeof(T) = 8 or 16 bytes, so aligned) as fp32, and back.
template <typename T, int N>
__device__ __forceinline__ void unpack(const T* e, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = Elt<T>::to_f32(e[i]);
}
template <int BYTES> struct Raw;
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };
template <typename T, int N>
struct VecOf {
  using R = typename Raw<N * int(sizeof(T))>::type;
  static __device__ __forceinline__ R load(const T* p) { return __ldg(reinterpret_cast<const R*>(p)); }
  static __device__ __forceinline__ void get(const R& raw, float (&v)[N]) { unpack<T, N>(reinterpret_cast<const T*>(&raw), v); }
  static __device__ __forceinline__ R pack(const float (&v)[N]) {
    R raw;
    T* q = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < N; i += 2) store2(q + i, make_float2(v[i], v[i + 1]));
    return raw;
  }
  static __device__ __forceinline__ void put(T* p, const R& raw) { *reinterpret_cast<R*>(p) = raw; }
  static __device__ __forceinline__ void store(T* p, const float (&v)[N]) { put(p, pack(v)); }
};

// Column sums of partial results: out(c) = sum over r < rows of in[r * ld + c], c < cols, in a fixed order (32
// threads share a column, each adding every 32nd row; then a tree), so that repeated calls give the same bits.
// `put(c, sum)` stores.
template <typename F>
__device__ __forceinline__ void column_sums(const float* in, int64_t rows, int64_t ld, int64_t cols, F put) {
  __shared__ float part[32][33];
  const int tc = threadIdx.x & 31, tr = threadIdx.x >> 5;   // 1024 threads
  const int64_t c = int64_t(blockIdx.x) * 32 + tc;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  if (c < cols) {
    int64_t r = tr;
    for (; r + 96 < rows; r += 128) {
      s0 += in[r * ld + c];
      s1 += in[(r + 32) * ld + c];
      s2 += in[(r + 64) * ld + c];
      s3 += in[(r + 96) * ld + c];
    }
    for (; r < rows; r += 32) s0 += in[r * ld + c];
  }
  part[tr][tc] = (s0 + s1) + (s2 + s3);
  __syncthreads();
  float v = part[tc][tr];   // warp tr now holds column tr, lane = row slice
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t co = int64_t(blockIdx.x) * 32 + tr;
  if (tc == 0 && co < cols) put(co, v);
}

}  // namespace wkv7
