// Short causal convolution per channel, with optional SiLU (wkv7_conv_forward / _backward / _step).
//   u_t = bias + sum_{j<W} w[W-1-j] x_{t-j},   y_t = silu(u_t) or u_t
// A reset at t cuts the taps before t: zeroing the window of earlier inputs there is the same thing, and the
// window after the last token is the state that a decode step continues from.
//
// HBM-bound: x is read and y written once (2 D elements per token).  One thread owns four
// channels and a run of tokens, so the window stays in registers and every input element is loaded once per run
// plus W - 1 tokens of run-in (in L2: the neighbouring run has just read them).  The run length is chosen so
// that the grid still fills the machine: long runs save run-in, short ones keep small calls parallel.
#include <type_traits>

#include "kernels.h"
#include "layer_util.cuh"
#include "state_space.h"

namespace wkv7 {
namespace {

constexpr int kThreads = 256, kRunThreads = 128;   // decode step; forward and backward
constexpr int kV = 4;            // channels of a thread: 8 per thread (16-byte loads of bf16) took 108 registers and 0.142 ms
                                 // for B=8 T=4096 D=2304
constexpr int kBatch = 4;        // tokens whose loads are issued together
static_assert(kBatch == 4, "the tokens of a batch are picked by hand where one is a reset");
constexpr int kNoReset = 1 << 20;

template <int W, int V>
__device__ __forceinline__ void load_filter(const ConvArgs& p, int64_t d0, float (&w)[W][V], float (&bias)[V]) {
  float flat[W * V];   // [V][W] in memory; V W floats are a multiple of 16 bytes
#pragma unroll
  for (int i = 0; i < W * V / 4; ++i) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p.weight + d0 * W) + i);
    flat[4 * i] = f.x; flat[4 * i + 1] = f.y; flat[4 * i + 2] = f.z; flat[4 * i + 3] = f.w;
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) w[j][e] = flat[e * W + (W - 1 - j)];   // w[j] multiplies x_{t-j}
#pragma unroll
  for (int e = 0; e < V; ++e) bias[e] = p.bias ? __ldg(p.bias + d0 + e) : 0.f;
}

// Inputs before token t0 that its taps may see (win[j] = x_{t0-1-j}, zero where a reset cuts them off) and the
// number of tokens since the last reset before t0.
template <typename T, int W, int V>
__device__ __forceinline__ int load_window(const ConvArgs& p, int64_t b, int64_t t0, int64_t d0, float (&win)[W - 1][V]) {
  int age = kNoReset;
#pragma unroll
  for (int j = W - 2; j >= 0; --j) {
    const int64_t t = t0 - 1 - j;
    float v[V] = {};
    if (t >= 0) {
      const int64_t off = (b * p.T + t) * p.x_ld + d0;
      if (range_ok(off, V, (p.B * p.T - 1) * p.x_ld + p.D, p.status))
        VecOf<T, V>::get(VecOf<T, V>::load(static_cast<const T*>(p.x) + off), v);
      if (p.reset && p.reset[b * p.T + t]) {
        age = 0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
          if (i > j)
#pragma unroll
            for (int e = 0; e < V; ++e) win[i][e] = 0.f;
      } else if (age < kNoReset) {
        ++age;
      }
    } else if (p.s0) {
      const int64_t off = (b * (W - 1) + (W - 1 + t)) * p.D + d0;
      if (range_ok(off, V, p.B * (W - 1) * p.D, p.status))
        VecOf<T, V>::get(VecOf<T, V>::load(static_cast<const T*>(p.s0) + off), v);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) win[j][e] = v[e];
  }
  return age;
}

// CTAs per SM of the forward that the registers are held to: seven (72 registers) for the 16-bit types, whose loads are
// half as long (B=8 T=4096 D=2304: bf16 72 us, 81 unbound; fp32 167 us, 137 unbound).
template <typename T>
constexpr int kFwdMinCtas = sizeof(T) == 2 ? 7 : 1;

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kRunThreads, kFwdMinCtas<T>) conv_fwd_kernel(const ConvArgs p, int64_t run, int64_t runs) {
  constexpr int V = kV;
  using VT = VecOf<T, V>;
  const int64_t nv = p.D / V;
  const int64_t id = int64_t(blockIdx.x) * kRunThreads + threadIdx.x;
  const int64_t br = id / nv, d0 = (id - br * nv) * V, b = br / runs;
  if (b >= p.B) return;
  const int64_t t0 = (br - b * runs) * run, t1 = min64(t0 + run, p.T);
  float w[W][V], bias[V], win[W - 1][V];
  load_filter<W, V>(p, d0, w, bias);
  load_window<T, W, V>(p, b, t0, d0, win);
  const T* x = static_cast<const T*>(p.x) + b * p.T * p.x_ld + d0;
  T* y = static_cast<T*>(p.y) + b * p.T * p.D + d0;
  const uint8_t* reset = p.reset ? p.reset + b * p.T : nullptr;
  auto load = [&](int64_t t) {
    return rows_ok((b * p.T + t) * p.x_ld + d0, V, p.B * p.T, p.x_ld, p.D, p.status) ? VT::load(x + t * p.x_ld) : typename VT::R{};
  };
  auto token = [&](const typename VT::R& raw, int64_t t) {   // u_t from its input and the window, which moves on
    float v[V], u[V];
    VT::get(raw, v);
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      float2 a = fma2(make_float2(w[0][e], w[0][e + 1]), make_float2(v[e], v[e + 1]), make_float2(bias[e], bias[e + 1]));
#pragma unroll
      for (int j = 1; j < W; ++j)
        a = fma2(make_float2(w[j][e], w[j][e + 1]), make_float2(win[j - 1][e], win[j - 1][e + 1]), a);
      u[e] = SILU ? a.x * sigmoid_of<T>(a.x) : a.x;
      u[e + 1] = SILU ? a.y * sigmoid_of<T>(a.y) : a.y;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = W - 2; j > 0; --j) win[j][e] = win[j - 1][e];
      win[0][e] = v[e];
    }
    if (range_ok((b * p.T + t) * p.D + d0, V, p.B * p.T * p.D, p.status)) VT::store(y + t * p.D, u);
  };
  int64_t t = t0;
  typename VT::R next[kBatch];   // loads run one batch ahead
  if (t + kBatch <= t1)
#pragma unroll
    for (int i = 0; i < kBatch; ++i) next[i] = load(t + i);
  for (; t + kBatch <= t1; t += kBatch) {
    typename VT::R raw[kBatch];
    unsigned cut = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) raw[i] = next[i];
    if (t + 2 * kBatch <= t1)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) next[i] = load(t + kBatch + i);
    if (reset)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) cut |= reset[t + i] ? 1u << i : 0u;
    if (cut == 0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) token(raw[i], t + i);
    } else {
#pragma unroll 1
      for (int i = 0; i < kBatch; ++i) {
        if (cut >> i & 1u)
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) win[j][e] = 0.f;
        token(i == 0 ? raw[0] : i == 1 ? raw[1] : i == 2 ? raw[2] : raw[3], t + i);
      }
    }
  }
  for (; t < t1; ++t) {
    if (reset && reset[t])
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) win[j][e] = 0.f;
    token(load(t), t);
  }
  if (p.s_out && t1 == p.T)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {   // slot W-2-j holds x_{T-1-j}
      const int64_t off = (b * (W - 1) + (W - 2 - j)) * p.D + d0;
      if (range_ok(off, V, p.B * (W - 1) * p.D, p.status)) VT::store(static_cast<T*>(p.s_out) + off, win[j]);
    }
}

// Backward: with du_t = dy_t silu'(u_t) (u recomputed), dx_t = sum_j w[j] du_{t+j} over the taps that no reset
// cuts, dw[j] = sum_t du_t x_{t-j}, dbias = sum_t du_t.  A thread owns 4 channels (the filter's gradient stays in
// registers beside the windows) and a run of tokens; it walks W - 1 tokens past its run for the gradients that
// reach back into it.  The filter's partial sums per run go to scratch and are added by column_sums.  As
// in the forward, batches of tokens whose taps all count take a path without tests, and their loads run one batch ahead:
// B=8 T=4096 D=2304 with the filter's gradient: bf16 157 us (2.9 TB/s), 321 us with every token on the general path; fp32
// 286 us (3.2 TB/s).  Without the filter's gradient 140 and 270.

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kRunThreads) conv_bwd_kernel(const ConvArgs p, int64_t run, int64_t runs) {
  constexpr int V = kV;
  using VT = VecOf<T, V>;
  const int64_t nv = p.D / V;
  const int64_t id = int64_t(blockIdx.x) * kRunThreads + threadIdx.x;
  const int64_t br = id / nv, d0 = (id - br * nv) * V, b = br / runs;
  if (b >= p.B) return;
  const int64_t t0 = (br - b * runs) * run, t1 = min64(t0 + run, p.T);
  float w[W][V], bias[V], win[W - 1][V];
  load_filter<W, V>(p, d0, w, bias);
  int age = load_window<T, W, V>(p, b, t0, d0, win);
  float dxp[W][V] = {};        // partial dx of tokens t, t-1, .., t-W+1
  float dw[W][V] = {}, dbias[V] = {};
  const T* x = static_cast<const T*>(p.x) + b * p.T * p.x_ld + d0;
  const T* dy = static_cast<const T*>(p.dy) + b * p.T * p.D + d0;
  const uint8_t* reset = p.reset ? p.reset + b * p.T : nullptr;
  T* dx = static_cast<T*>(p.dx) + b * p.T * p.D + d0;
  auto load = [&](int64_t t, typename VT::R& rx, typename VT::R& rg) {
    if (rows_ok((b * p.T + t) * p.x_ld + d0, V, p.B * p.T, p.x_ld, p.D, p.status)) rx = VT::load(x + t * p.x_ld);
    if (range_ok((b * p.T + t) * p.D + d0, V, p.B * p.T * p.D, p.status)) rg = VT::load(dy + t * p.D);
  };
  // One token: the gradient of u_t, which goes to the filter and to the inputs behind its taps; then the input that is
  // W - 1 tokens back is complete.  PLAIN: a token of this run, all of whose taps count, and that input is of this run too.
  auto token = [&](const typename VT::R& rx, const typename VT::R& rg, int64_t t, auto plain) {
    constexpr bool PLAIN = decltype(plain)::value;
    float v[V], g[V];
#pragma unroll
    for (int j = W - 1; j > 0; --j)
#pragma unroll
      for (int e = 0; e < V; ++e) dxp[j][e] = dxp[j - 1][e];
#pragma unroll
    for (int e = 0; e < V; ++e) dxp[0][e] = 0.f;
    if (PLAIN || t < p.T) {
      VT::get(rx, v);
      VT::get(rg, g);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 v2 = make_float2(v[e], v[e + 1]);
        float2 g2 = make_float2(g[e], g[e + 1]);
        auto at = [&](float (&a)[V]) -> float2& { return *reinterpret_cast<float2*>(&a[e]); };
        if (SILU) {
          float2 u = fma2(at(w[0]), v2, at(bias));
#pragma unroll
          for (int j = 1; j < W; ++j) u = fma2(at(w[j]), at(win[j - 1]), u);
          const float sx = sigmoid_of<T>(u.x), sy = sigmoid_of<T>(u.y);
          g2.x *= sx * fmaf(u.x, 1.f - sx, 1.f);
          g2.y *= sy * fmaf(u.y, 1.f - sy, 1.f);
        }
        if (PLAIN || t < t1) {
          at(dbias) = add2(at(dbias), g2);
          at(dw[0]) = fma2(g2, v2, at(dw[0]));
#pragma unroll
          for (int j = 1; j < W; ++j) at(dw[j]) = fma2(g2, at(win[j - 1]), at(dw[j]));
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (PLAIN || j <= age) at(dxp[j]) = fma2(at(w[j]), g2, at(dxp[j]));
#pragma unroll
        for (int j = W - 2; j > 0; --j) at(win[j]) = at(win[j - 1]);
        at(win[0]) = v2;
      }
    }
    const int64_t td = t - (W - 1);
    if (PLAIN) {
      if (range_ok((b * p.T + td) * p.D + d0, V, p.B * p.T * p.D, p.status)) VT::store(dx + td * p.D, dxp[W - 1]);
      return;
    }
    if (td < t0 && !(t0 == 0 && td < 0)) return;
    if (p.dsT && td >= p.T - (W - 1) && p.T - 1 - td <= age) {   // it is in s_out, not cut off
      float s[V] = {};
      const int64_t off = (b * (W - 1) + td - (p.T - (W - 1))) * p.D + d0;
      if (range_ok(off, V, p.B * (W - 1) * p.D, p.status)) VT::get(VT::load(static_cast<const T*>(p.dsT) + off), s);
#pragma unroll
      for (int e = 0; e < V; ++e) dxp[W - 1][e] += s[e];
    }
    if (td >= 0) {
      if (range_ok((b * p.T + td) * p.D + d0, V, p.B * p.T * p.D, p.status)) VT::store(dx + td * p.D, dxp[W - 1]);
    } else if (p.ds0) {
      const int64_t off = (b * (W - 1) + W - 1 + td) * p.D + d0;
      if (range_ok(off, V, p.B * (W - 1) * p.D, p.status)) VT::store(static_cast<T*>(p.ds0) + off, dxp[W - 1]);
    }
  };
  auto slow = [&](int64_t t) {   // any token, also behind the run or the row
    typename VT::R rx{}, rg{};
    if (t < p.T) {
      load(t, rx, rg);
      if (reset && reset[t]) {
        age = 0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) win[j][e] = 0.f;
      } else if (age < kNoReset) {
        ++age;
      }
    }
    token(rx, rg, t, std::false_type{});
  };
  const int64_t tend = t1 + W - 1;
  const int64_t plain_end = p.dsT ? min64(t1, p.T - (W - 1)) : t1;   // behind it an input may be part of s_out
  int64_t t = t0;
#pragma unroll 1
  for (; t < min64(t0 + W - 1, tend); ++t) slow(t);
  typename VT::R nx[kBatch], ng[kBatch];   // loads run one batch ahead
  auto ahead = [&](int64_t t) {
    if (t + kBatch <= plain_end)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) load(t + i, nx[i], ng[i]);
  };
  ahead(t);
#pragma unroll 1
  for (; t + kBatch <= plain_end; t += kBatch) {
    typename VT::R rx[kBatch], rg[kBatch];
    bool cut = false;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      rx[i] = nx[i];
      rg[i] = ng[i];
      cut |= reset && reset[t + i];
    }
    ahead(t + kBatch);
    if (!cut && age >= W - 2) {   // (age counts the tokens since the last reset; the batch's first one adds one more)
      age = min(age + kBatch, kNoReset);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) token(rx[i], rg[i], t + i, std::true_type{});
    } else {
#pragma unroll 1
      for (int i = 0; i < kBatch; ++i) slow(t + i);
    }
  }
#pragma unroll 1
  for (; t < tend; ++t) slow(t);
  if (p.scratch && range_ok(br * (W + 1) * p.D + d0, W * p.D + V, p.B * runs * (W + 1) * p.D, p.status)) {   // [run][W + 1][D]: dw of weight[.][0..W-1], then dbias
    float* o = p.scratch + br * (W + 1) * p.D + d0;
#pragma unroll
    for (int j = 0; j < W; ++j)
      *reinterpret_cast<float4*>(o + (W - 1 - j) * p.D) = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    *reinterpret_cast<float4*>(o + W * p.D) = make_float4(dbias[0], dbias[1], dbias[2], dbias[3]);
  }
}

__global__ void __launch_bounds__(1024) conv_dw_kernel(const ConvArgs p, int64_t rows) {
  const int W = p.W;
  column_sums(p.scratch, rows, (W + 1) * p.D, (W + 1) * p.D, [&](int64_t c, float v) {
    const int64_t k = c / p.D, d = c - k * p.D;
    if (k < W) {
      if (p.dweight) p.dweight[d * W + k] = v;
    } else if (p.dbias) {
      p.dbias[d] = v;
    }
  });
}

// Decode: one thread per (row, 16-byte vector of channels); the window is the state.
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvArgs p) {
  constexpr int V = Vec16<T>::n;
  using VT = VecOf<T, V>;
  const int64_t nv = p.D / V;
  const int64_t id = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t b = id / nv, d0 = (id - b * nv) * V;
  if (b >= p.B) return;
  if (!range_ok(b * p.D + d0, V, p.B * p.D, p.status) || !rows_ok(b * p.x_ld + d0, V, p.B, p.x_ld, p.D, p.status) ||
      !range_ok((b * (W - 1) + W - 2) * p.D + d0, V, p.B * (W - 1) * p.D, p.status))
    return;
  T* y = static_cast<T*>(p.y) + b * p.D + d0;
  if (p.active && !p.active[b]) {
    const float zero[V] = {};
    VT::store(y, zero);
    return;
  }
  T* st = static_cast<T*>(p.state) + b * (W - 1) * p.D + d0;
  typename VT::R raw[W - 1];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) raw[i] = *reinterpret_cast<const typename VT::R*>(st + i * p.D);
  const typename VT::R rx = VT::load(static_cast<const T*>(p.x) + b * p.x_ld + d0);
  float w[W][V], bias[V], v[V], u[V];
  load_filter<W, V>(p, d0, w, bias);
  VT::get(rx, v);
#pragma unroll
  for (int e = 0; e < V; ++e) u[e] = fmaf(w[0][e], v[e], bias[e]);
#pragma unroll
  for (int j = 1; j < W; ++j) {
    VT::get(raw[W - 1 - j], v);
#pragma unroll
    for (int e = 0; e < V; ++e) u[e] = fmaf(w[j][e], v[e], u[e]);
  }
  if (SILU)
#pragma unroll
    for (int e = 0; e < V; ++e) u[e] *= sigmoid_of<T>(u[e]);
  VT::store(y, u);
#pragma unroll
  for (int i = 0; i < W - 2; ++i) *reinterpret_cast<typename VT::R*>(st + i * p.D) = raw[i + 1];
  *reinterpret_cast<typename VT::R*>(st + (W - 2) * p.D) = rx;
}

// Tokens of a run: the longest of 64, 32, 16, 8 (backward) or 32, 16, 8, 4 that leaves `want` threads.
int64_t run_length(int64_t B, int64_t T, int64_t vecs, int64_t longest, int64_t want) {
  int64_t run = longest;
  for (int i = 0; i < 3 && B * ((T + run - 1) / run) * vecs < want; ++i) run /= 2;
  return run;
}
constexpr int64_t kFwdWant = 148 * 1024, kBwdWant = 148 * 512;

template <typename T, int W, bool SILU>
cudaError_t fwd(const ConvArgs& p, cudaStream_t s) {
  const int64_t nv = p.D / kV, run = run_length(p.B, p.T, nv, 32, kFwdWant), runs = (p.T + run - 1) / run;
  const int64_t blocks = (p.B * runs * nv + kRunThreads - 1) / kRunThreads;
  if (blocks > 2147483647) return cudaErrorInvalidValue;
  conv_fwd_kernel<T, W, SILU><<<unsigned(blocks), kRunThreads, 0, s>>>(p, run, runs);
  return cudaGetLastError();
}
template <typename T, int W, bool SILU>
cudaError_t bwd(const ConvArgs& p, cudaStream_t s) {
  const int64_t nv = p.D / kV, run = run_length(p.B, p.T, nv, 64, kBwdWant), runs = (p.T + run - 1) / run;
  const int64_t blocks = (p.B * runs * nv + kRunThreads - 1) / kRunThreads;
  if (blocks > 2147483647) return cudaErrorInvalidValue;
  conv_bwd_kernel<T, W, SILU><<<unsigned(blocks), kRunThreads, 0, s>>>(p, run, runs);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.scratch) return e;
  conv_dw_kernel<<<unsigned(((W + 1) * p.D + 31) / 32), 1024, 0, s>>>(p, p.B * runs);
  return cudaGetLastError();
}
template <typename T, int W, bool SILU>
cudaError_t step(const ConvArgs& p, cudaStream_t s) {
  const int64_t blocks = (p.B * (p.D / Vec16<T>::n) + kThreads - 1) / kThreads;
  if (blocks > 2147483647) return cudaErrorInvalidValue;
  conv_step_kernel<T, W, SILU><<<unsigned(blocks), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

enum Kind { kFwd, kBwd, kStep };
template <typename T, int W, bool SILU>
cudaError_t run_kind(Kind k, const ConvArgs& p, cudaStream_t s) {
  return k == kFwd ? fwd<T, W, SILU>(p, s) : k == kBwd ? bwd<T, W, SILU>(p, s) : step<T, W, SILU>(p, s);
}
template <typename T, int W>
cudaError_t run_silu(Kind k, const ConvArgs& p, cudaStream_t s) {
  return p.silu ? run_kind<T, W, true>(k, p, s) : run_kind<T, W, false>(k, p, s);
}
template <typename T>
cudaError_t run_w(Kind k, const ConvArgs& p, cudaStream_t s) {
  return p.W == 2 ? run_silu<T, 2>(k, p, s) : p.W == 3 ? run_silu<T, 3>(k, p, s) : run_silu<T, 4>(k, p, s);
}
cudaError_t run(Kind k, const ConvArgs& p, int dtype, cudaStream_t s) {
  if (p.W < 2 || p.W > 4) return cudaErrorInvalidValue;
  switch (dtype) {
    case 0: return run_w<float>(k, p, s);
    case 1: return run_w<__nv_bfloat16>(k, p, s);
    case 2: return run_w<__half>(k, p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int64_t conv_scratch_floats(int64_t B, int64_t T, int64_t D, int W) {
  if (B == 0 || T == 0 || D == 0) return 0;
  const int64_t run = run_length(B, T, D / kV, 64, kBwdWant);
  return B * ((T + run - 1) / run) * (W + 1) * D;
}

cudaError_t launch_conv_fwd(const ConvArgs& p, int dtype, cudaStream_t s) { return run(kFwd, p, dtype, s); }
cudaError_t launch_conv_bwd(const ConvArgs& p, int dtype, cudaStream_t s) { return run(kBwd, p, dtype, s); }
cudaError_t launch_conv_step(const ConvArgs& p, int dtype, cudaStream_t s) { return run(kStep, p, dtype, s); }

}  // namespace wkv7
