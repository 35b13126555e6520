// RMS norm over equal slices of each row, with the residual's addition or a SiLU gate before it and an optional
// e4m3 output (wkv7_rms_forward / wkv7_rms_backward):
//   h = x | round(x + other) | x silu(other),   out = h rstd weight,   rstd = 1 / sqrt(mean(h^2) + eps)
// and, with g = dout weight and m = mean(g h rstd) over the slice,
//   dh = rstd (g - h rstd m) [+ the gradient reaching h directly],   dweight = sum over rows of dout h rstd,
//   gate: dx = dh silu(z), dz = dh x silu'(z).
//
// HBM-bound: every input is read once and every output written once.  A slice is held in the registers of TPS
// threads (1, 2 or 4 16-byte vectors each), so both reductions and the outputs come from one
// read.  Up to 32 threads reduce by shuffles alone; wider slices add one pass through shared memory.  Short
// slices share a CTA of 128 threads; CTAs are that small so that several independent ones per SM cover each other's
// reductions.  Measured for bf16, 67 M elements, slices of 2048: forward with residual 86 us (6.2 TB/s), plain 55 us (4.9),
// backward 85 us (4.7); slices of 64 48 us; the same bytes in fp32: 83, 47, 77 and 46 us.  Wide slices are slower: of 8192 plain,
// with residual and backward 3.9, 5.7 and 4.4 TB/s (fp32 5.6, 6.1, 3.2), of 16384 3.3, 5.2 and 3.6 (fp32 4.3, 5.2, 2.9).  One of
// 16384 bf16 takes 512 threads with four vectors each and 92 (backward 126) registers: an SM holds one such CTA, which loads,
// reduces and stores with nothing else under way (a quarter of the warps, issue slots 32 and 50 % busy); of 8192 it holds two.
#include <cuda_fp8.h>

#include "kernels.h"
#include "layer_util.cuh"
#include "state_space.h"

namespace wkv7 {
namespace {

enum Mode { kPlain = 0, kResidual = 1, kGate = 2 };
constexpr int kCta = 128;
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 7.888609052210118e-31f;   // 2^-100: its reciprocal and the scaled values stay finite

// Maximum that keeps a NaN, so that a block that holds one gets a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float scale_of(float top) { return top == 0.f ? 1.f : max_nan(top * (1.f / kE4m3Max), kMinScale); }

// Sums (or, of the first, the maximum) over the TPS threads of a slice of COUNT = 1 or 2 values at once.  All threads
// of the CTA call it together.
struct Pair { float a, b; };
template <bool MAXA, int COUNT>
__device__ __forceinline__ Pair slice_reduce(Pair v, int tps, float (*sm)[2]) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (o >= tps) continue;
    const float a = __shfl_xor_sync(0xffffffffu, v.a, o);
    v.a = MAXA ? max_nan(v.a, a) : v.a + a;
    if (COUNT == 2) v.b += __shfl_xor_sync(0xffffffffu, v.b, o);
  }
  if (tps <= 32) return v;
  const int warp = threadIdx.x >> 5, nw = tps >> 5, first = blockDim.x == tps ? 0 : warp & ~(nw - 1);
  __syncthreads();   // the last use of `sm` is over
  if ((threadIdx.x & 31) == 0) *reinterpret_cast<float2*>(sm[warp]) = make_float2(v.a, v.b);
  __syncthreads();
  float2 r = *reinterpret_cast<const float2*>(sm[first]);
  for (int i = 1; i < nw; ++i) {
    const float2 q = *reinterpret_cast<const float2*>(sm[first + i]);
    r.x = MAXA ? max_nan(r.x, q.x) : r.x + q.x;
    if (COUNT == 2) r.y += q.y;
  }
  return Pair{r.x, r.y};
}

// Threads of a CTA at most: slices have up to 64, 1024 and (L <= 16384) 16384 / V vectors with 1, 2 and 4 per thread.
template <typename T, int VPT>
constexpr int kMaxThreads = VPT == 1 ? kCta : VPT == 2 ? 512 : 16384 / Vec16<T>::n / 4;

// Two neighbouring values of an array, for the packed fp32 instructions: the kernels are close to bound by their issue.
template <int V>
__device__ __forceinline__ float2& two(float (&a)[V], int e) { return *reinterpret_cast<float2*>(&a[e]); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

struct Shape {
  int64_t L, slices;   // channels of a slice; rows * groups
  int tps, spc;        // threads per slice, slices per CTA: with several, a slice has a power of two
  int log_tps;
  float inv_l;         // 1 / L
};

template <typename T, int V>
__device__ __forceinline__ void store_e4m3(uint8_t* o, const float (&q)[V]) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if (V == 8) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[V / 4 - 1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
}

template <typename T, int VPT, int MODE, int QUANT>   // QUANT: 0 none, 1 per 128 channels, 2 per slice
__global__ void __launch_bounds__(kMaxThreads<T, VPT>) rms_fwd_kernel(const RmsArgs p, const Shape s) {
  constexpr int V = Vec16<T>::n;
  using VT = VecOf<T, V>;
  __shared__ __align__(8) float sm[32][2];
  const int sub = s.spc == 1 ? 0 : threadIdx.x >> s.log_tps, lane = threadIdx.x - sub * s.tps;
  const int64_t nv = s.L / V, total = p.rows * p.D;
  for (int64_t s0 = int64_t(blockIdx.x) * s.spc; s0 < s.slices; s0 += int64_t(gridDim.x) * s.spc) {
    const int64_t slice = s0 + sub;
    const int64_t row = p.groups == 1 ? slice : slice / p.groups, g = p.groups == 1 ? 0 : slice - row * p.groups;
    const int64_t base = row * p.D + g * s.L;
    typename VT::R rx[VPT], rz[VPT];
    bool act[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = i * s.tps + lane;
      act[i] = slice < s.slices && v < nv && range_ok(base + v * V, V, total, p.status);
      if (act[i]) {
        rx[i] = VT::load(static_cast<const T*>(p.x) + base + v * V);
        if (MODE != kPlain) rz[i] = VT::load(static_cast<const T*>(p.other) + base + v * V);
      }
    }
    float h[VPT][V];
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (act[i]) {
        VT::get(rx[i], h[i]);
        if (MODE != kPlain) {
          float z[V];
          VT::get(rz[i], z);
#pragma unroll
          for (int e = 0; e < V; e += 2)
            two(h[i], e) = MODE == kResidual ? add2(two(h[i], e), two(z, e))
                                             : mul2(two(h[i], e), mul2(two(z, e), make_float2(sigmoid_of<T>(z[e]), sigmoid_of<T>(z[e + 1]))));
          if (MODE == kResidual) {   // the stored sum is normalised, so that the backward, which reads it, sees the same h
            rx[i] = VT::pack(h[i]);
            VT::get(rx[i], h[i]);
            VT::put(static_cast<T*>(p.h_out) + base + (i * s.tps + lane) * V, rx[i]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) h[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; e += 2) s2 = fma2(two(h[i], e), two(h[i], e), s2);
    }
    const float rstd = rsqrtf(fmaf(slice_reduce<false, 1>(Pair{s2.x + s2.y, 0.f}, s.tps, sm).a, s.inv_l, p.eps));
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = i * s.tps + lane;
      if (act[i]) {
        const float4* w = reinterpret_cast<const float4*>(p.weight + g * s.L + v * V);
#pragma unroll
        for (int u = 0; u < V / 4; ++u) {
          const float4 w4 = __ldg(w + u);
          two(h[i], 4 * u) = mul2(two(h[i], 4 * u), mul2(both(rstd), make_float2(w4.x, w4.y)));
          two(h[i], 4 * u + 2) = mul2(two(h[i], 4 * u + 2), mul2(both(rstd), make_float2(w4.z, w4.w)));
        }
        if (QUANT == 0) VT::store(static_cast<T*>(p.out) + base + v * V, h[i]);
      }
      if (QUANT) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) m = max_nan(m, fabsf(h[i][e]));
        if (QUANT == 1) {   // 128 channels are 128 / V neighbouring threads (tps >= that many)
#pragma unroll
          for (int o = 64 / V; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float sc = scale_of(m);
          const float inv = rcp_fast(sc);   // sc >= 2^-100, or NaN
          if (act[i]) {
            float q[V];
#pragma unroll
            for (int e = 0; e < V; e += 2) two(q, e) = mul2(two(h[i], e), both(inv));
            store_e4m3<T, V>(static_cast<uint8_t*>(p.out) + base + v * V, q);
            if ((lane & (128 / V - 1)) == 0 && range_ok((base + v * V) >> 7, 1, total >> 7, p.status)) p.scale[(base + v * V) >> 7] = sc;
          }
        }
        top = max_nan(top, m);
      }
    }
    if (QUANT == 2) {
      top = slice_reduce<true, 1>(Pair{top, 0.f}, s.tps, sm).a;
      const float sc = scale_of(top);
      const float inv = rcp_fast(sc);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (act[i]) {
          float q[V];
#pragma unroll
          for (int e = 0; e < V; e += 2) two(q, e) = mul2(two(h[i], e), both(inv));
          store_e4m3<T, V>(static_cast<uint8_t*>(p.out) + base + (i * s.tps + lane) * V, q);
        }
      if (lane == 0 && slice < s.slices && range_ok(slice, 1, p.rows * p.groups, p.status)) p.scale[slice] = sc;
    }
  }
}

// Backward.  A CTA stays on one group of channels (blockIdx.x % groups), so a thread keeps its channels' dweight
// in registers over all its rows; the CTA's sum goes to its row of scratch, and column_sums adds those rows.
template <typename T, int VPT, bool GATE>
__global__ void __launch_bounds__(kMaxThreads<T, VPT>, kMaxThreads<T, VPT> < 512 ? 512 / kMaxThreads<T, VPT> : 1)
rms_bwd_kernel(const RmsArgs p, const Shape s, int64_t nb) {
  constexpr int V = Vec16<T>::n;
  using VT = VecOf<T, V>;
  __shared__ __align__(8) float sm[32][2];
  extern __shared__ float acc[];   // [spc][L] when a CTA holds several slices
  const int sub = s.spc == 1 ? 0 : threadIdx.x >> s.log_tps, lane = threadIdx.x - sub * s.tps;
  const int64_t nv = s.L / V, total = p.rows * p.D;
  const int64_t g = blockIdx.x % p.groups, blk = blockIdx.x / p.groups;
  float dw[VPT][V] = {};
  // The weight stays in registers too, except with four vectors: it is read again, from the L1, for each row.
  constexpr bool HOLD = VPT < 4;
  float held[HOLD ? VPT : 1][V];
  auto weight_of = [&](int i, float (&w)[V]) {
    const int64_t v = i * s.tps + lane;
#pragma unroll
    for (int u = 0; u < V / 4; ++u) {
      const float4 w4 = v < nv ? __ldg(reinterpret_cast<const float4*>(p.weight + g * s.L + v * V) + u) : make_float4(0, 0, 0, 0);
      w[4 * u] = w4.x; w[4 * u + 1] = w4.y; w[4 * u + 2] = w4.z; w[4 * u + 3] = w4.w;
    }
  };
  if (HOLD)
#pragma unroll
    for (int i = 0; i < VPT; ++i) weight_of(i, held[HOLD ? i : 0]);
  // The next row's loads are under way while this one is reduced (bf16, 67 M elements, slices of 2048: 85 us, 118 without),
  // except with four vectors, which take too many registers.
  constexpr bool AHEAD = VPT < 4;
  typename VT::R nx[VPT], nz[VPT], ng[VPT];
  auto fetch = [&](int64_t row) {
    const int64_t base = row * p.D + g * s.L;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = i * s.tps + lane, o = base + v * V;
      if (row < p.rows && v < nv && range_ok(o, V, total, p.status)) {
        nx[i] = VT::load(static_cast<const T*>(p.x) + o);
        ng[i] = VT::load(static_cast<const T*>(p.dout) + o);
        if (GATE) nz[i] = VT::load(static_cast<const T*>(p.other) + o);
        else if (p.dh) nz[i] = VT::load(static_cast<const T*>(p.dh) + o);
      }
    }
  };
  if (AHEAD) fetch(blk * s.spc + sub);
  for (int64_t r0 = blk * s.spc; r0 < p.rows; r0 += nb * s.spc) {
    const int64_t row = r0 + sub;
    const int64_t base = row * p.D + g * s.L;
    typename VT::R rx[VPT], rz[VPT], rg[VPT];
    bool act[VPT];
    if (!AHEAD) fetch(row);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = i * s.tps + lane;
      act[i] = row < p.rows && v < nv && range_ok(base + v * V, V, total, p.status);
      rx[i] = nx[i];
      rg[i] = ng[i];
      rz[i] = nz[i];
    }
    if (AHEAD) fetch(row + nb * s.spc);
    float2 ss = make_float2(0.f, 0.f), gh = ss;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (act[i]) {
        float x[V], z[V], d[V], wt[V];
        VT::get(rx[i], x);
        VT::get(rg[i], d);
        if (!HOLD) weight_of(i, wt);
        if (GATE) VT::get(rz[i], z);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          float2 h = two(x, e);
          if (GATE) h = mul2(h, mul2(two(z, e), make_float2(sigmoid_of<T>(z[e]), sigmoid_of<T>(z[e + 1]))));
          ss = fma2(h, h, ss);
          gh = fma2(mul2(two(d, e), HOLD ? two(held[HOLD ? i : 0], e) : two(wt, e)), h, gh);
        }
      }
    const Pair r = slice_reduce<false, 2>(Pair{ss.x + ss.y, gh.x + gh.y}, s.tps, sm);
    const float rstd = rsqrtf(fmaf(r.a, s.inv_l, p.eps));
    const float m = r.b * rstd * rstd * s.inv_l;   // mean(g xhat) rstd: dh = rstd (g - h m)
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (act[i]) {
        const int64_t o = base + (i * s.tps + lane) * V;
        float x[V], z[V], d[V], dx[V], dz[V], wt[V];
        VT::get(rx[i], x);
        if (!HOLD) weight_of(i, wt);
        VT::get(rg[i], d);
        if (GATE || p.dh) VT::get(rz[i], z);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 x2 = two(x, e), d2 = two(d, e);
          float2 h = x2, sg = make_float2(0.f, 0.f), sz = sg;
          if (GATE) {
            sg = make_float2(sigmoid_of<T>(z[e]), sigmoid_of<T>(z[e + 1]));
            sz = mul2(two(z, e), sg);
            h = mul2(x2, sz);
          }
          two(dw[i], e) = fma2(d2, mul2(h, both(rstd)), two(dw[i], e));
          const float2 gw = mul2(d2, HOLD ? two(held[HOLD ? i : 0], e) : two(wt, e));
          const float2 dh = mul2(both(rstd), fma2(h, both(-m), gw));
          if (GATE) {
            two(dx, e) = mul2(dh, sz);
            two(dz, e) = mul2(mul2(dh, x2), mul2(sg, fma2(two(z, e), sub2(both(1.f), sg), both(1.f))));
          } else {
            two(dx, e) = p.dh ? add2(dh, two(z, e)) : dh;
          }
        }
        VT::store(static_cast<T*>(p.dx) + o, dx);
        if (GATE) VT::store(static_cast<T*>(p.dother) + o, dz);
      }
  }
  if (!p.scratch || !range_ok(blk * p.D + g * s.L, s.L, nb * p.D, p.status)) return;
  float* out = p.scratch + blk * p.D + g * s.L;
  if (s.spc == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = i * s.tps + lane;
      if (v < nv)
#pragma unroll
        for (int u = 0; u < V / 4; ++u)
          *reinterpret_cast<float4*>(out + v * V + 4 * u) =
              make_float4(dw[i][4 * u], dw[i][4 * u + 1], dw[i][4 * u + 2], dw[i][4 * u + 3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int64_t v = i * s.tps + lane;
    if (v < nv)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[sub * s.L + v * V + e] = dw[i][e];
  }
  __syncthreads();
  for (int64_t c = threadIdx.x; c < s.L; c += blockDim.x) {
    float t = 0.f;
    for (int i = 0; i < s.spc; ++i) t += acc[i * s.L + c];
    out[c] = t;
  }
}

__global__ void __launch_bounds__(1024) rms_dw_kernel(const float* scratch, int64_t rows, int64_t D, float* dweight) {
  column_sums(scratch, rows, D, D, [&](int64_t c, float v) { dweight[c] = v; });
}

// Threads of a slice of nv vectors: one vector each up to 64 vectors, two up to 1024, four above.
int vectors_per_thread(int64_t nv) { return nv <= 64 ? 1 : nv <= 1024 ? 2 : 4; }
Shape shape_of(const RmsArgs& p, int64_t nv, int vpt) {
  Shape s;
  s.L = p.D / p.groups;
  s.slices = p.rows * p.groups;
  s.tps = 1;
  s.log_tps = 0;
  while (int64_t(s.tps) * vpt < nv) {
    s.tps *= 2;
    ++s.log_tps;
  }
  s.inv_l = 1.f / float(s.L);
  s.spc = s.tps < kCta ? kCta / s.tps : 1;
  if (s.spc == 1) s.tps = int((nv + vpt * 32 - 1) / (vpt * 32)) * 32;   // whole warps (2560 channels of bf16: 4.3 TB/s, a power of two 3.4)
  return s;
}
constexpr int64_t kFwdCtas = 148 * 16;   // grid-stride over the rest

// CTAs per group of the backward, its scratch rows: one wave.  An SM holds 512 threads of the backward's 128 registers, or,
// of the 32-bit kernel with four vectors, the 1024 of its 64.
int64_t bwd_blocks(int64_t rows, int64_t groups, const Shape& s, bool wide) {
  const int64_t per_sm = (wide ? 1024 : 512) / (int64_t(s.tps) * s.spc);
  const int64_t cap = 148 * per_sm / groups, need = (rows + s.spc - 1) / s.spc;
  const int64_t nb = need < cap ? need : cap;
  return nb < 1 ? 1 : nb;
}

template <typename T, int VPT, int MODE, int QUANT>
cudaError_t fwd(const RmsArgs& p, const Shape& s, cudaStream_t st) {
  const int64_t need = (s.slices + s.spc - 1) / s.spc;
  rms_fwd_kernel<T, VPT, MODE, QUANT><<<unsigned(need < kFwdCtas ? need : kFwdCtas), s.tps * s.spc, 0, st>>>(p, s);
  return cudaGetLastError();
}
template <typename T, int VPT, int MODE>
cudaError_t fwd_q(const RmsArgs& p, const Shape& s, cudaStream_t st) {
  return p.quant_block == 0 ? fwd<T, VPT, MODE, 0>(p, s, st)
         : p.quant_block > 0 ? fwd<T, VPT, MODE, 1>(p, s, st)
                             : fwd<T, VPT, MODE, 2>(p, s, st);
}
template <typename T, int VPT>
cudaError_t fwd_mode(const RmsArgs& p, const Shape& s, cudaStream_t st) {
  return !p.other ? fwd_q<T, VPT, kPlain>(p, s, st) : p.gate ? fwd_q<T, VPT, kGate>(p, s, st) : fwd_q<T, VPT, kResidual>(p, s, st);
}
template <typename T, int VPT>
cudaError_t bwd(const RmsArgs& p, const Shape& s, cudaStream_t st) {
  const int64_t nb = bwd_blocks(p.rows, p.groups, s, kMaxThreads<T, VPT> > 512);
  if (nb * p.groups > 2147483647) return cudaErrorInvalidValue;
  const size_t smem = s.spc > 1 ? size_t(s.spc) * s.L * 4 : 0;   // at most 128 threads * 16 floats = 8 KiB
  const dim3 grid(unsigned(nb * p.groups)), block(unsigned(s.tps * s.spc));
  if (p.other) rms_bwd_kernel<T, VPT, true><<<grid, block, smem, st>>>(p, s, nb);
  else rms_bwd_kernel<T, VPT, false><<<grid, block, smem, st>>>(p, s, nb);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dweight) return e;
  rms_dw_kernel<<<unsigned((p.D + 31) / 32), 1024, 0, st>>>(p.scratch, nb, p.D, p.dweight);
  return cudaGetLastError();
}
template <typename T>
cudaError_t run(const RmsArgs& p, bool backward, cudaStream_t st) {
  const int64_t nv = p.D / p.groups / Vec16<T>::n;
  const int vpt = vectors_per_thread(nv);
  const Shape s = shape_of(p, nv, vpt);
  if (s.tps > 1024) return cudaErrorInvalidValue;
  if (backward) return vpt == 1 ? bwd<T, 1>(p, s, st) : vpt == 2 ? bwd<T, 2>(p, s, st) : bwd<T, 4>(p, s, st);
  return vpt == 1 ? fwd_mode<T, 1>(p, s, st) : vpt == 2 ? fwd_mode<T, 2>(p, s, st) : fwd_mode<T, 4>(p, s, st);
}
cudaError_t run_dtype(const RmsArgs& p, int dtype, bool backward, cudaStream_t st) {
  switch (dtype) {
    case 0: return run<float>(p, backward, st);
    case 1: return run<__nv_bfloat16>(p, backward, st);
    case 2: return run<__half>(p, backward, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Enough for every dtype: the fewest threads per slice give the most rows of scratch.
int64_t rms_scratch_floats(int64_t rows, int64_t D, int64_t groups) {
  if (rows == 0 || D == 0) return 0;
  int64_t most = 0;
  for (int n : {4, 8}) {
    const int64_t nv = D / groups / n;
    RmsArgs p{};
    p.rows = rows; p.D = D; p.groups = groups;
    const int vpt = vectors_per_thread(nv);
    const int64_t nb = bwd_blocks(rows, groups, shape_of(p, nv, vpt), vpt == 4 && n == 4);
    most = nb > most ? nb : most;
  }
  return most * D;
}

cudaError_t launch_rms_fwd(const RmsArgs& p, int dtype, cudaStream_t s) { return run_dtype(p, dtype, false, s); }
cudaError_t launch_rms_bwd(const RmsArgs& p, int dtype, cudaStream_t s) { return run_dtype(p, dtype, true, s); }

}  // namespace wkv7
