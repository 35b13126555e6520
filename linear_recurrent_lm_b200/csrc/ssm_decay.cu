// Last step of the selective scan's backward: from per-token scalars to the gradients of dt, A, D and dt_bias.
//
// The log decay a_t = d_t A of token t multiplies every path from a token (or state) before t to one at or after t.
// With W_ts the weight of the path from s to t (its contribution to the loss, s < t),
//   dL/da_t = sum over paths crossing into t = E + sum_{s >= t in the chunk} (row_s - d_s col_s)
// where row_s sums the paths that end at s (from other tokens or the state), d_s col_s those that start at s, and
// E = <state after the chunk, gradient of it> the paths that leave the chunk.  A reset ends every path, so the sum runs
// to the end of t's segment, E belongs to the last segment only, and the reset token's own decay has no gradient.  The
// paths that neither start nor end at t cancel in the difference, so it is summed in fp64; the path from a token to
// itself is in neither sum (it would cancel too, at a far larger size where little is remembered).  What leaves the chunk
// is in E and in col: the chunked backward hands that part of col over on its own (`far`) and E without it, so that the
// same numbers are added here and cancel exactly.
//   dL/dd_t = A dL/da_t + col_t + own_t,   own_t = (x . dy)(b . c);   ddt = dL/dd sigmoid(dt + bias)
//
// One warp per (b, h, chunk), 4 tokens per lane.  Per token and head it reads the sums (8 + 8 + 4 + 4 bytes, 4 more where
// `far` is apart) and dt, and writes ddt: 34 bytes in all for bf16 CHUNKED, 36 MB and 24 us for B=8 T=4096 H=32, as the tokens of
// dt and ddt are H elements apart; the sums per head after it, one warp each, 8 us.
#include "ssm.cuh"

namespace wkv7 {
namespace {

template <typename T, bool CHUNKED>
__global__ void __launch_bounds__(256) decay_kernel(const SsmArgs p, const SsmScratch sc, float* part) {
  const int lane = threadIdx.x & 31;
  const int64_t nc = chunks_of(p.T), tp = nc * kSsmChunk;
  const int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= p.B * p.H * nc) return;
  const int64_t unit = w / nc, c = w - unit * nc, b = unit / p.H, h = unit - b * p.H;
  const float A = __ldg(p.A + h);
  const int64_t t0 = c * kSsmChunk + 4 * lane, o = unit * tp + t0;
  const bool in = range_ok(o, 4, p.B * p.H * tp, p.status) && (t0 >= p.T || range_ok((b * p.T + t0) * p.H + h, 1, p.B * p.T * p.H, p.status));
  if (kDebugChecks && !__all_sync(0xffffffffu, in)) return;
  const double *rows = reinterpret_cast<const double*>(p.scratch + sc.row) + o, *cols = reinterpret_cast<const double*>(p.scratch + sc.col) + o;
  const float4 own = *reinterpret_cast<const float4*>(p.scratch + sc.own + o);
  const float4 xd = *reinterpret_cast<const float4*>(p.scratch + sc.xdy + o);
  const float owns[4] = {own.x, own.y, own.z, own.w}, xds[4] = {xd.x, xd.y, xd.z, xd.w};
  float d[4] = {}, sg[4] = {};
  double v[4], suf[4], cs[4] = {}, leave = 0.0;
  float fr[4] = {};
  if (CHUNKED) {
    const float4 f4 = *reinterpret_cast<const float4*>(p.scratch + sc.far + o);
    fr[0] = f4.x; fr[1] = f4.y; fr[2] = f4.z; fr[3] = f4.w;
  }
  unsigned rst = 0, cut = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = 0.0;
    if (t0 + i < p.T) {
      float raw;
      d[i] = step_of<T>(p, b * p.T + t0 + i, h, &raw);
      sg[i] = p.softplus ? 1.f / (1.f + expf(-raw)) : 1.f;
      cs[i] = CHUNKED ? cols[i] + double(fr[i]) : cols[i];
      v[i] = rows[i] - double(d[i]) * cs[i];
      if (CHUNKED) leave += double(d[i]) * double(fr[i]);
      // a decay that is zero cuts like a reset: what is left of its sums is rounding, which a large A would blow up
      if ((p.reset && p.reset[b * p.T + t0 + i]) || cuts(d[i], A)) rst |= 1u << i;
    }
  }
  cut = rst >> 1;   // token i ends its segment where token i + 1 is a reset
  const unsigned next = __shfl_down_sync(0xffffffffu, rst, 1);
  if (lane < 31 && (next & 1u)) cut |= 8u;
  if (CHUNKED)
#pragma unroll
    for (int s = 16; s; s >>= 1) leave += __shfl_xor_sync(0xffffffffu, leave, s);
  if (lane == 31) v[3] += leave + reinterpret_cast<const double*>(p.scratch + sc.anchor)[w];   // the chunk's last token carries E
  segmented_suffix(v, cut, suf);
  double dA = 0.0, dB = 0.0, dD = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + i < p.T) {
      const double da = (rst >> i & 1u) ? 0.0 : suf[i];
      const double g = (double(A) * da + cs[i] + double(owns[i])) * double(sg[i]);
      static_cast<T*>(p.ddt)[(b * p.T + t0 + i) * p.H + h] = Elt<T>::from_f32(float(g));
      dA += double(d[i]) * da;
      dB += g;
      dD += double(xds[i]);
    }
#pragma unroll
  for (int s = 16; s; s >>= 1) {
    dA += __shfl_xor_sync(0xffffffffu, dA, s);
    dB += __shfl_xor_sync(0xffffffffu, dB, s);
    dD += __shfl_xor_sync(0xffffffffu, dD, s);
  }
  if (lane == 0) {
    part[3 * w] = float(dA);
    part[3 * w + 1] = float(dD);
    part[3 * w + 2] = float(dB);
  }
}

// Sums of the (b, chunk) partials per head, in a fixed order: one warp per head and gradient.
__global__ void __launch_bounds__(96) decay_sum_kernel(const SsmArgs p, const float* part) {
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t h = blockIdx.x, nc = chunks_of(p.T);
  double s = 0.0;
  for (int64_t i = lane; i < p.B * nc; i += 32) {
    const int64_t b = i / nc, c = i - b * nc;
    s += double(part[3 * ((b * p.H + h) * nc + c) + k]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  float* out = k == 0 ? p.dA : k == 1 ? p.dD : p.ddt_bias;
  if (lane == 0 && out) out[h] = float(s);
}

}  // namespace

cudaError_t launch_ssm_decay(const SsmArgs& p, int dtype, bool chunked, cudaStream_t s) {
  const SsmScratch sc = ssm_scratch(p.B, p.T, p.H, p.G, p.N, chunked);
  const int64_t warps = p.B * p.H * chunks_of(p.T);
  const unsigned grid = unsigned((warps + 7) / 8);
  float* part = p.scratch + sc.part;
  switch (dtype) {
    case 0: decay_kernel<float, false><<<grid, 256, 0, s>>>(p, sc, part); break;
    case 1:
      if (chunked) decay_kernel<__nv_bfloat16, true><<<grid, 256, 0, s>>>(p, sc, part);
      else decay_kernel<__nv_bfloat16, false><<<grid, 256, 0, s>>>(p, sc, part);
      break;
    case 2: decay_kernel<__half, false><<<grid, 256, 0, s>>>(p, sc, part); break;
    default: return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(p.dA || p.dD || p.ddt_bias)) return e;
  decay_sum_kernel<<<unsigned(p.H), 96, 0, s>>>(p, part);
  return cudaGetLastError();
}

SsmScratch ssm_scratch(int64_t B, int64_t T, int64_t H, int64_t G, int N, bool chunked) {
  const int64_t nc = chunks_of(T), tok = B * H * nc * kSsmChunk, state = int64_t(kHeadP) * N;
  SsmScratch s{};
  int64_t o = 0;
  auto take = [&](int64_t n) { const int64_t at = o; o += (n + 3) / 4 * 4; return at; };
  s.row = take(2 * tok);
  s.col = take(2 * tok);
  if (chunked) s.far = take(tok);
  s.own = take(tok);
  s.xdy = take(tok);
  s.anchor = take(2 * B * H * nc);
  s.part = take(3 * B * H * nc);
  if (chunked) {
    s.dstate = take(B * H * nc * state);
    s.seg = take(ssm_segment_floats(B, T, H, N));
    // heads of a group per CTA: as few splits as leave every SM its share within a tenth
    const int64_t units = B * nc * G, hg = H / G;
    s.splits = 1;
    double best = 1e300;
    for (int64_t k = 1; k <= hg && k <= 32; k *= 2) {
      const int64_t per = (hg + k - 1) / k, rounds = (units * k + 147) / 148;
      const double cost = double(rounds * per) + 0.05 * double(units * k) / 148.0;   // a part's sums cost about 1/20 head
      if (cost < best * 0.97) {
        best = cost;
        s.splits = k;
      }
    }
    if (s.splits > 1) {
      s.db_part = take(s.splits * B * T * G * N);
      s.dc_part = take(s.splits * B * T * G * N);
    }
  } else {
    s.dstate = take(2 * B * H * nc * state);
    s.seg = take(5 * ssm_run_floats(B, T, H, N));   // of three scans, two of them in fp64
    s.state_t = take(2 * B * H * (nc + 1) * state);
    s.dcp = take(2 * B * T * H * N);
    s.dbp = take(2 * B * T * H * N);
  }
  s.total = o;
  return s;
}

}  // namespace wkv7
