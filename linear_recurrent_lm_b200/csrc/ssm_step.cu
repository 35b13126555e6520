// Decode step of the selective scan on B*H resident fp32 states [64][N], in place: a pure stream over the state
// (32 KiB read and written per head at N = 128), HBM-bound.  Like the WKV-7 step: a persistent grid of CTAs of 512
// threads walks the heads; 8 threads per row, each with every eighth float4 of it, so a warp's access is whole
// 128-byte lines; the output needs three shuffles; inactive rows touch nothing but y = 0; consecutive steps overlap
// launch and tail by programmatic dependent launch.
#include <atomic>

#include "ssm.cuh"

namespace wkv7 {
namespace {

constexpr int kThreads = 8 * kHeadP;
constexpr int kMaxDevices = 64;

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 3) ssm_step_kernel(const SsmArgs p) {
  constexpr int NI = N / 32;
  // everything this grid reads or writes may belong to the grid launched before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = threadIdx.x >> 3, q = threadIdx.x & 7;
  const int64_t units = p.B * p.H, hg = p.H / p.G;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t b = unit / p.H, h = unit - b * p.H, g = h / hg;
    if (!range_ok((unit * kHeadP + i) * N, N, units * kHeadP * N, p.status) ||
        !rows_ok(b * p.x_ld + h * kHeadP + i, 1, p.B, p.x_ld, p.H * kHeadP, p.status) ||
        !rows_ok(b * p.b_ld + g * N, N, p.B, p.b_ld, p.G * N, p.status) || !rows_ok(b * p.c_ld + g * N, N, p.B, p.c_ld, p.G * N, p.status))
      continue;
    T* y = static_cast<T*>(p.y) + unit * kHeadP;
    if (p.active && !p.active[b]) {
      if (q == 0) y[i] = Elt<T>::from_f32(0.f);
      continue;
    }
    float4* row = reinterpret_cast<float4*>(p.state + (unit * kHeadP + i) * N) + q;
    float4 S[NI];
#pragma unroll
    for (int u = 0; u < NI; ++u) S[u] = row[8 * u];
    const T* bp = static_cast<const T*>(p.b) + b * p.b_ld + g * N + 4 * q;
    const T* cp = static_cast<const T*>(p.c) + b * p.c_ld + g * N + 4 * q;
    const float x = Elt<T>::to_f32(static_cast<const T*>(p.x)[b * p.x_ld + h * kHeadP + i]);
    const float d = step_of<T>(p, b, h);
    const float f = expf(d * __ldg(p.A + h)), u0 = d * x;
    float a = 0.f;
#pragma unroll
    for (int u = 0; u < NI; ++u) {
      const float2 b0 = load2(bp + 32 * u), b1 = load2(bp + 32 * u + 2);
      const float2 c0 = load2(cp + 32 * u), c1 = load2(cp + 32 * u + 2);
      S[u].x = fmaf(S[u].x, f, u0 * b0.x);
      S[u].y = fmaf(S[u].y, f, u0 * b0.y);
      S[u].z = fmaf(S[u].z, f, u0 * b1.x);
      S[u].w = fmaf(S[u].w, f, u0 * b1.y);
      row[8 * u] = S[u];
      a = fmaf(S[u].x, c0.x, a);
      a = fmaf(S[u].y, c0.y, a);
      a = fmaf(S[u].z, c1.x, a);
      a = fmaf(S[u].w, c1.y, a);
    }
    a += __shfl_xor_sync(0xffffffffu, a, 1);
    a += __shfl_xor_sync(0xffffffffu, a, 2);
    a += __shfl_xor_sync(0xffffffffu, a, 4);
    if (q == 0) y[i] = Elt<T>::from_f32(p.Dw ? fmaf(__ldg(p.Dw + h), x, a) : a);
  }
}

template <typename T, int N>
cudaError_t launch(const SsmArgs& p, cudaStream_t stream) {
  static std::atomic<int> cached[kMaxDevices];   // SMs x resident CTAs per SM; 0 = not looked up yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int slots = (dev >= 0 && dev < kMaxDevices) ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (slots == 0) {
    int sms = 0, per_sm = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, ssm_step_kernel<T, N>, kThreads, 0)) != cudaSuccess) return e;
    slots = sms * (per_sm > 0 ? per_sm : 1);
    if (dev >= 0 && dev < kMaxDevices) cached[dev].store(slots, std::memory_order_relaxed);
  }
  const int64_t units = p.B * p.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units < slots ? units : slots));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, ssm_step_kernel<T, N>, p)) != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs& p, int dtype, cudaStream_t s) {
  const bool n128 = p.N == 128;
  switch (dtype) {
    case 0: return n128 ? launch<float, 128>(p, s) : launch<float, 64>(p, s);
    case 1: return n128 ? launch<__nv_bfloat16, 128>(p, s) : launch<__nv_bfloat16, 64>(p, s);
    case 2: return n128 ? launch<__half, 128>(p, s) : launch<__half, 64>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace wkv7
