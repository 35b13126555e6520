// Selective state space scan, token by token on FP32 cores (algo SCAN; every dtype, exact fp32 arithmetic).
//
// All four passes of a training step are one recurrence.  With f_t the decay applied before token t,
//   past_t[r] = sum_k f_t Z_{t-1}[r][k] con_t[k],    Z_t = f_t Z_{t-1} + i_t rin_t kin_t^T   (R x K)
// walked forward or in reverse:
//   y:   forward, Z = S      (64 x N):  rin = x, kin = b, con = c, i = d    -> past + (b.c) d x + D x
//   dc:  forward, Z = S^T    (N x 64):  rin = b, kin = x, con = dy, i = d   -> past, per head
//   dx:  reverse, Z = dS     (64 x N):  rin = dy, kin = c, con = b          -> d (past + (b.c) dy) + D dy
//   db:  reverse, Z = dS^T   (N x 64):  rin = c, kin = dy, con = x          -> past, per head
// In reverse f is the decay of the token after (the gradient passes through it on its way back).  The transposed scans
// leave a token's own term out of `past`: the gradient of the decays is made of the paths between different tokens alone, and
// where little is remembered they are far smaller than the own term that would absorb them.
//
// A decay of zero (a reset) drops what it is applied to instead of scaling it, so that nothing of the tokens behind it
// is left, not even a NaN.
//
// Bound by shared memory and shuffles rather than by its 3 R K operations per token and head (decay, output, update).  One
// CTA per (b, h); a thread owns 4 rows and every eighth 16-byte vector of the columns, so a token's K-vectors are read from
// shared memory as whole 128-byte lines, each serves 16 rows of the warp, and the outputs of 4 rows need four shuffles
// (two rows per thread: 61 us instead of 38 for bf16 B=64 T=16 H=32 N=64).  B=8 T=1024 H=32 fp32 forward: N=64 325 us, N=128
// 486 us; backward, three scans, 1.41 ms and 2.76 ms.  Tokens move in tiles: the next tile's loads are
// in flight while this one is computed.
//
// The two scans behind the decay's gradient (dc and db) run in fp64, at half the rate: that gradient is a sum of
// differences between what ends and what starts at a token, in which most paths cancel, and the rounding of a long
// carried fp32 state does not cancel with it (measured: dA off by 5e-6 to 2e-5 of its size in fp32).
#include <type_traits>

#include "ssm.cuh"

namespace wkv7 {
namespace {

struct ScanOp {
  const void *rin, *kin, *con;           // token rows of R, K, K elements
  int64_t rin_ld, kin_ld, con_ld;        // token strides
  bool rin_g, kin_g, con_g;              // the row's vector is the group's (b, c), not the head's
  const float *init;                     // [B,H,64,N] entering state (or gradient), or null
  bool scale_in, scale_out;              // i_t = d_t, o_t = d_t
  const float* skip;                     // [H] or null
  void* out;                             // [B,T,H,R]: T, or double (past alone) for the transposed scans
  void* chunk_state;                     // Z before (forward) or after (reverse) each chunk, as [R][K] of fp32 (transposed
                                         // scans: fp64): [B,H,stride], or null
  int64_t chunk_stride;
  float* last;                           // [B,H,R,K]: Z after the walk (reverse: carried through token 0's decay), or null
  // The walk may be cut into `segments` runs of `per` tokens: a first pass (LOCAL) leaves each run's end state from
  // zero and its total decay, and the second starts every run from what those before it left.
  int64_t segments, per;
  void* seg_state;                       // [B,H,segments] states [R][K], fp32 (transposed scans: fp64)
  double* seg_decay;                     // [B,H,segments] decays: of a run's many tokens they may leave fp32's range where
                                         // what they multiply brings the product back
};

// 16 bytes of staged values.
__device__ __forceinline__ void load_pair(const float* p, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void load_pair(const double* p, double (&v)[2]) {
  const double2 f = *reinterpret_cast<const double2*>(p);
  v[0] = f.x; v[1] = f.y;
}

// One 16-byte vector of columns of one row: decay, update, output; the transposed scans' output is taken before the update.
__device__ __forceinline__ void advance(float* z, const float (&k)[4], const float (&c)[4], float f, float u, float2& a) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    float2& v = *reinterpret_cast<float2*>(z + e);
    v = fma2(make_float2(u, u), make_float2(k[e], k[e + 1]), mul2(v, make_float2(f, f)));
    a = fma2(v, make_float2(c[e], c[e + 1]), a);
  }
}
__device__ __forceinline__ void advance(double* z, const double (&k)[2], const double (&c)[2], double f, double u, double2& a) {
  z[0] *= f; z[1] *= f;
  a.x = fma(z[0], c[0], a.x); a.y = fma(z[1], c[1], a.y);
  z[0] = fma(u, k[0], z[0]); z[1] = fma(u, k[1], z[1]);
}

constexpr int kRows = 4;   // state rows of a thread

// TR: the transposed scans (R = N, K = 64), in double.
template <typename T, int R, int K, bool REV, bool TR, bool LOCAL>
__global__ void __launch_bounds__(8 * R / kRows) scan_kernel(const SsmArgs p, const ScanOp op) {
  using F = typename std::conditional<TR, double, float>::type;
  using F2 = typename std::conditional<TR, double2, float2>::type;
  constexpr int kTile = TR ? 8 : 16, EV = 16 / int(sizeof(F)), NI = K / (8 * EV);
  constexpr int V = Vec16<T>::n, NT = 8 * R / kRows;
  constexpr int VR = R / V, VK = K / V, kVecs = kTile * (VR + 2 * VK), kPer = (kVecs + NT - 1) / NT;
  __shared__ __align__(16) F s_r[2][kTile][R], s_k[2][kTile][K], s_c[2][kTile][K];
  __shared__ __align__(16) F s_fio[2][kTile][4];   // decay, factor of the input, factor of the output
  __shared__ unsigned s_special[2];                // tokens of the tile with a decay of zero or a state to store
  __shared__ __align__(16) F s_out[kTile][R];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // see `launch`
  const int tid = threadIdx.x, lane8 = tid & 7, r0 = (tid >> 3) * kRows;
  const int64_t unit = blockIdx.x / op.segments, seg = blockIdx.x - unit * op.segments;
  const int64_t b = unit / p.H, h = unit - b * p.H, g = h / (p.H / p.G);
  const int64_t T_ = p.T, first = seg * op.per, end = min64(first + op.per, T_);   // positions of the walk
  const float A = __ldg(p.A + h);
  const float skip = op.skip ? __ldg(op.skip + h) : 0.f;

  F Z[kRows][NI * EV];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int u = 0; u < NI; ++u)
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const int row = r0 + i, col = (8 * u + lane8) * EV + e;   // init is [64][N]: transposed where R = N
        const int64_t at = unit * R * K + (TR ? col * R + row : row * K + col);
        Z[i][EV * u + e] = !LOCAL && op.init && range_ok(at, 1, p.B * p.H * R * K, p.status) ? F(__ldg(op.init + at)) : F(0);
      }
  if (!LOCAL)
    for (int64_t j = unit * op.segments; j < unit * op.segments + seg; ++j) {
      const double f = op.seg_decay[j];
      const F* z = static_cast<const F*>(op.seg_state) + j * (R * K);
      auto join = [&](auto g) {   // Z = g Z + z
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int u = 0; u < NI; ++u)
#pragma unroll
            for (int e = 0; e < EV; ++e) {
              F& v = Z[i][EV * u + e];
              v = F(g * v) + z[(r0 + i) * K + (8 * u + lane8) * EV + e];
            }
      };
      if (f == 0.0) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int e = 0; e < NI * EV; ++e) Z[i][e] = F(0);
      }
      if (f < 1e37 && (f > 1e-37 || f == 0.0)) join(F(f));
      else join(f);   // (f16 B=3 T=777 H=6 forward: 36 us, 39 with this throughout)
    }
  double total = 1.0;
  auto put_state = [&](auto* dst, F f) {
    using D = std::remove_pointer_t<decltype(dst)>;
    using D2 = typename std::conditional<sizeof(D) == 8, double2, float2>::type;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int u = 0; u < NI; ++u)
#pragma unroll
        for (int e = 0; e < EV; e += 2)
          *reinterpret_cast<D2*>(dst + (r0 + i) * K + (8 * u + lane8) * EV + e) =
              f == F(0) ? D2{} : D2{D(f * Z[i][EV * u + e]), D(f * Z[i][EV * u + e + 1])};
  };
  auto decay = [&](float d) -> F { return TR ? F(exp(double(d) * double(A))) : F(expf(d * A)); };

  uint4 raw[kPer];
  F tf = 0, ti = 0, to = 0;
  bool special = false;
  auto token = [&](int64_t pos) { return REV ? T_ - 1 - pos : pos; };
  auto stores = [&](int64_t t) { return REV ? t % kSsmChunk == kSsmChunk - 1 || t == T_ - 1 : t % kSsmChunk == 0; };
  auto fetch = [&](int64_t pos0) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int v = tid + q * NT;
      raw[q] = make_uint4(0, 0, 0, 0);
      if (v < kVecs) {
        const int tok = v / (VR + 2 * VK), o = v % (VR + 2 * VK);
        if (pos0 + tok < end) {
          const int64_t bt = b * T_ + token(pos0 + tok);
          const int which = o < VR ? 0 : o < VR + VK ? 1 : 2;
          const int j = o - (which == 0 ? 0 : which == 1 ? VR : VR + VK), width = which == 0 ? R : K;
          const void* base = which == 0 ? op.rin : which == 1 ? op.kin : op.con;
          const int64_t ld = which == 0 ? op.rin_ld : which == 1 ? op.kin_ld : op.con_ld;
          const bool grp = which == 0 ? op.rin_g : which == 1 ? op.kin_g : op.con_g;
          const int64_t off = bt * ld + (grp ? g : h) * width + j * V;
          if (rows_ok(off, V, p.B * T_, ld, (grp ? p.G : p.H) * width, p.status))
            raw[q] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(base) + off));
        }
      }
    }
    special = false;
    if (tid < kTile && pos0 + tid < end) {
      const int64_t t = token(pos0 + tid), bt = b * T_ + t;
      const float d = step_of<T>(p, bt, h);
      const int64_t td = REV ? t + 1 : t;   // the decay between this token and the one walked before it
      if (REV && td == T_) tf = 1;
      else if (p.reset && p.reset[b * T_ + td]) tf = 0;
      else tf = decay(REV ? step_of<T>(p, bt + 1, h) : d);
      ti = op.scale_in ? d : 1.f;
      to = op.scale_out ? d : 1.f;
      special = tf == F(0) || (!LOCAL && op.chunk_state && stores(t));
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int v = tid + q * NT;
      if (v < kVecs) {
        const int tok = v / (VR + 2 * VK), o = v % (VR + 2 * VK);
        float f[V];
        unpack16<T>(raw[q], f);
        F* dst = o < VR ? &s_r[buf][tok][o * V] : o < VR + VK ? &s_k[buf][tok][(o - VR) * V] : &s_c[buf][tok][(o - VR - VK) * V];
#pragma unroll
        for (int e = 0; e < V; e += 2) *reinterpret_cast<F2*>(dst + e) = F2{F(f[e]), F(f[e + 1])};
      }
    }
    if (tid < 32) {
      const unsigned m = __ballot_sync(0xffffffffu, special);
      if (tid == 0) s_special[buf] = m;
    }
    if (tid < kTile) {
      s_fio[buf][tid][0] = tf;
      s_fio[buf][tid][1] = ti;
      s_fio[buf][tid][2] = to;
    }
  };

  fetch(first);
  stage(0);
  __syncthreads();
  int buf = 0;
  for (int64_t pos0 = first; pos0 < end; pos0 += kTile, buf ^= 1) {
    const int n = int(min64(kTile, end - pos0));
    if (pos0 + kTile < end) fetch(pos0 + kTile);
    auto one = [&](int i, unsigned mark) {
      const F f = s_fio[buf][i][0], in = s_fio[buf][i][1];
      if (mark >> i & 1u) {
        const int64_t t = token(pos0 + i);
        if (!LOCAL && op.chunk_state && stores(t) && range_ok(t / kSsmChunk, 1, op.chunk_stride, p.status))
          put_state(static_cast<F*>(op.chunk_state) + (unit * op.chunk_stride + t / kSsmChunk) * (R * K), REV ? f : F(1));
        if (f == F(0))
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < NI * EV; ++e) Z[r][e] = F(0);
      }
      F u[kRows];
#pragma unroll
      for (int r = 0; r < kRows; r += 2) {
        const F2 v = *reinterpret_cast<const F2*>(&s_r[buf][i][r0 + r]);
        u[r] = in * v.x;
        u[r + 1] = in * v.y;
      }
      if (LOCAL) total *= f;
      F2 a[kRows] = {};
#pragma unroll
      for (int q = 0; q < NI; ++q) {
        F k[EV], c[EV];
        load_pair(&s_k[buf][i][(8 * q + lane8) * EV], k);
        load_pair(&s_c[buf][i][(8 * q + lane8) * EV], c);
#pragma unroll
        for (int r = 0; r < kRows; ++r) advance(&Z[r][EV * q], k, c, f, u[r], a[r]);   // (LOCAL: the outputs fall away)
      }
      if (LOCAL) return;
      // sums over the 8 threads of the rows: each exchange halves the rows that a thread holds
      const bool hi4 = lane8 & 4, hi2 = lane8 & 2;
      F o[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) o[r] = a[r].x + a[r].y;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const F give = hi4 ? o[r] : o[r + 2];
        o[r] = (hi4 ? o[r + 2] : o[r]) + __shfl_xor_sync(0xffffffffu, give, 4);
      }
      const F give = hi2 ? o[0] : o[1];
      F sum = (hi2 ? o[1] : o[0]) + __shfl_xor_sync(0xffffffffu, give, 2);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      if (!(lane8 & 1)) {
        const int row = r0 + (lane8 >> 1);   // (bit 2 of the lane chose the pair of rows, bit 1 the row)
        s_out[i][row] = TR ? sum : s_fio[buf][i][2] * sum + F(skip) * s_r[buf][i][row];
      }
    };
    if (n == kTile && s_special[buf] == 0) {   // no branches between the tokens, so that they overlap
#pragma unroll 4
      for (int i = 0; i < kTile; ++i) one(i, 0);
    } else {
#pragma unroll 1
      for (int i = 0; i < n; ++i) one(i, s_special[buf]);
    }
    if (pos0 + kTile < end) stage(buf ^ 1);
    __syncthreads();
    if constexpr (LOCAL) continue;
    if constexpr (TR) {
      for (int v = tid; v < n * (R / 2); v += NT) {
        const int i = v / (R / 2), j = v % (R / 2);
        const int64_t off = ((b * T_ + token(pos0 + i)) * p.H + h) * R + 2 * j;
        if (range_ok(off, 2, p.B * T_ * p.H * R, p.status))
          *reinterpret_cast<double2*>(static_cast<double*>(op.out) + off) = *reinterpret_cast<const double2*>(&s_out[i][2 * j]);
      }
    } else {
      for (int v = tid; v < n * VR; v += NT) {
        const int i = v / VR, j = v % VR;
        const int64_t off = ((b * T_ + token(pos0 + i)) * p.H + h) * R + j * V;
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = s_out[i][j * V + e];
        if (range_ok(off, V, p.B * T_ * p.H * R, p.status)) VecOf<T, V>::store(static_cast<T*>(op.out) + off, f);
      }
    }
    __syncthreads();
  }
  if (LOCAL) {
    put_state(static_cast<F*>(op.seg_state) + blockIdx.x * int64_t(R * K), F(1));
    if (tid == 0) op.seg_decay[blockIdx.x] = total;
  } else if (seg == op.segments - 1) {
    if (op.last) {
      F f = 1;
      if (REV && T_ > 0) f = (p.reset && p.reset[b * T_]) ? F(0) : decay(step_of<T>(p, b * T_, h));
      put_state(op.last + unit * (R * K), f);
    }
    if (!REV && op.chunk_state) put_state(static_cast<F*>(op.chunk_state) + (unit * op.chunk_stride + chunks_of(T_)) * (R * K), F(1));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // see `launch`
}

// Runs of a row's tokens: with fewer rows of heads than two per SM, as many as fill those slots, of at least 32 tokens.  A
// cut row is walked twice, so it takes three runs to gain (forward, N=64: B=2 T=512 H=12 fp32 34 us, 130 whole; B=1 T=96 H=32, three
// runs, 19 us, 28 whole).
int64_t scan_segments(int64_t units, int64_t T) {
  const int64_t fit = units > 0 ? 296 / units : 1, most = T / 32, k = fit < most ? fit : most;
  return k >= 3 ? k : 1;
}

// One pass of a scan.  `beside`: it needs nothing of the launch before it, so it may start once that one's CTAs have all
// started (programmatic dependent launch) and run beside it; it ends after it, so that whatever follows has both.
template <typename T, int R, int K, bool REV, bool TR, bool LOCAL>
cudaError_t launch(const SsmArgs& p, const ScanOp& op, bool beside, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.B * p.H * op.segments));
  cfg.blockDim = dim3(8 * R / kRows);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, scan_kernel<T, R, K, REV, TR, LOCAL>, p, op);
}
// Cuts the walk into runs where `seg`, scratch for their states and decays, is given.
template <int R, int K, bool TR>
void cut(const SsmArgs& p, ScanOp* op, float* seg) {
  using F = typename std::conditional<TR, double, float>::type;
  const int64_t units = p.B * p.H, k = seg ? scan_segments(units, p.T) : 1;
  op->per = (p.T + k - 1) / k;
  op->segments = op->per > 0 ? (p.T + op->per - 1) / op->per : 1;
  op->seg_state = seg;
  op->seg_decay = reinterpret_cast<double*>(reinterpret_cast<F*>(seg) + units * op->segments * R * K);
}

template <typename T, int N>
cudaError_t fwd(const SsmArgs& p, cudaStream_t s) {
  ScanOp op{};
  op.rin = p.x; op.rin_ld = p.x_ld;
  op.kin = p.b; op.kin_ld = p.b_ld; op.kin_g = true;
  op.con = p.c; op.con_ld = p.c_ld; op.con_g = true;
  op.init = p.s0;
  op.scale_in = true;
  op.skip = p.Dw;
  op.out = p.y;
  op.chunk_state = p.ckpt;
  op.chunk_stride = chunks_of(p.T) + 1;
  op.last = p.s_out;
  cut<kHeadP, N, false>(p, &op, p.ckpt ? p.ckpt + p.B * p.H * (chunks_of(p.T) + 1) * kHeadP * N : nullptr);
  if (op.segments > 1) {
    const cudaError_t e = launch<T, kHeadP, N, false, false, true>(p, op, false, s);
    if (e != cudaSuccess) return e;
  }
  return launch<T, kHeadP, N, false, false, false>(p, op, false, s);
}

// Sums over the heads of a group: with the scans' past parts Pc, Pb per head and q = x . dy,
//   dc = sum_h Pc + d q b,   db = sum_h d (Pb + q c),
// and the per-token scalars of the decay's gradient.  One warp per (b, t, group).
template <typename T, int N>
__global__ void __launch_bounds__(256) heads_kernel(const SsmArgs p, const SsmScratch sc) {
  constexpr int E = N / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5), total = p.B * p.T * p.G;
  if (w >= total) return;
  const int64_t bt = w / p.G, g = w - bt * p.G, b = bt / p.T, t = bt - b * p.T, hg = p.H / p.G;
  const int64_t tp = chunks_of(p.T) * kSsmChunk;
  if (!rows_ok(bt * p.b_ld + g * N, N, p.B * p.T, p.b_ld, p.G * N, p.status) ||
      !rows_ok(bt * p.c_ld + g * N, N, p.B * p.T, p.c_ld, p.G * N, p.status) ||
      !rows_ok(bt * p.x_ld + g * hg * kHeadP, hg * kHeadP, p.B * p.T, p.x_ld, p.H * kHeadP, p.status) ||
      !range_ok((bt * p.H + g * hg) * N, hg * N, p.B * p.T * p.H * N, p.status) || !range_ok(w * N, N, total * N, p.status))
    return;
  float bv[E], cv[E], db[E] = {}, dc[E] = {}, bc = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bv[e] = Elt<T>::to_f32(static_cast<const T*>(p.b)[bt * p.b_ld + g * N + 32 * e + lane]);
    cv[e] = Elt<T>::to_f32(static_cast<const T*>(p.c)[bt * p.c_ld + g * N + 32 * e + lane]);
    bc = fmaf(bv[e], cv[e], bc);
  }
  const double *dcp = reinterpret_cast<const double*>(p.scratch + sc.dcp), *dbp = reinterpret_cast<const double*>(p.scratch + sc.dbp);
  auto warp_sum = [](auto v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  bc = warp_sum(bc);
#pragma unroll 4
  for (int64_t h = g * hg; h < (g + 1) * hg; ++h) {
    const float d = step_of<T>(p, bt, h);
    const float2 x2 = load2(static_cast<const T*>(p.x) + bt * p.x_ld + h * kHeadP + 2 * lane);
    const float2 y2 = load2(static_cast<const T*>(p.dy) + (bt * p.H + h) * kHeadP + 2 * lane);
    const float q = warp_sum(fmaf(x2.x, y2.x, x2.y * y2.y));
    double row = 0.0, col = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t o = (bt * p.H + h) * N + 32 * e + lane;
      const double pc = dcp[o], pb = dbp[o];
      dc[e] += fmaf(d * q, bv[e], float(pc));
      db[e] = fmaf(d, fmaf(q, cv[e], float(pb)), db[e]);
      row += double(cv[e]) * pc;
      col += double(bv[e]) * pb;
    }
    row = warp_sum(row);
    col = warp_sum(col);
    if (lane == 0) {
      const int64_t o = (b * p.H + h) * tp + t;
      reinterpret_cast<double*>(p.scratch + sc.row)[o] = row;
      reinterpret_cast<double*>(p.scratch + sc.col)[o] = col;
      p.scratch[sc.own + o] = q * bc;
      p.scratch[sc.xdy + o] = q;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t o = (bt * p.G + g) * N + 32 * e + lane;
    static_cast<T*>(p.db)[o] = Elt<T>::from_f32(db[e]);
    static_cast<T*>(p.dc)[o] = Elt<T>::from_f32(dc[e]);
  }
}

// <state after the chunk, its gradient> per (b, h, chunk), from the fp64 scans' states: one CTA of 256 threads each.
__global__ void __launch_bounds__(256) anchor_kernel(const SsmArgs p, const SsmScratch sc) {
  __shared__ double part[8];
  const int64_t nc = chunks_of(p.T), u = blockIdx.x, unit = u / nc, c = u - unit * nc, n = int64_t(kHeadP) * p.N;
  const double2* S = reinterpret_cast<const double2*>(p.scratch + sc.state_t) + (unit * (nc + 1) + c + 1) * (n / 2);
  const double2* dS = reinterpret_cast<const double2*>(p.scratch + sc.dstate) + u * (n / 2);
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < n / 2; i += 256) {
    const double2 x = __ldg(S + i), y = __ldg(dS + i);
    a += x.x * y.x + x.y * y.y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < 8; ++i) s += part[i];
    reinterpret_cast<double*>(p.scratch + sc.anchor)[u] = s;
  }
}

template <typename T, int N>
cudaError_t bwd(const SsmArgs& p, cudaStream_t s) {
  const SsmScratch sc = ssm_scratch(p.B, p.T, p.H, p.G, N, false);
  const int64_t nc = chunks_of(p.T);
  const int64_t run = ssm_run_floats(p.B, p.T, p.H, N);
  float* seg = p.scratch + sc.seg;   // dx, then dc and db in fp64
  ScanOp dc{};   // forward again, transposed
  dc.rin = p.b; dc.rin_ld = p.b_ld; dc.rin_g = true;
  dc.kin = p.x; dc.kin_ld = p.x_ld;
  dc.con = p.dy; dc.con_ld = p.H * kHeadP;
  dc.init = p.s0;
  dc.scale_in = true;
  dc.out = p.scratch + sc.dcp;
  dc.chunk_state = p.scratch + sc.state_t; dc.chunk_stride = nc + 1;
  ScanOp dx{};
  dx.rin = p.dy; dx.rin_ld = p.H * kHeadP;
  dx.kin = p.c; dx.kin_ld = p.c_ld; dx.kin_g = true;
  dx.con = p.b; dx.con_ld = p.b_ld; dx.con_g = true;
  dx.init = p.dsT;
  dx.scale_out = true;
  dx.skip = p.Dw;
  dx.out = p.dx;
  dx.last = p.ds0;
  ScanOp db{};
  db.rin = p.c; db.rin_ld = p.c_ld; db.rin_g = true;
  db.kin = p.dy; db.kin_ld = p.H * kHeadP;
  db.con = p.x; db.con_ld = p.x_ld;
  db.init = p.dsT;
  db.out = p.scratch + sc.dbp;
  db.chunk_state = p.scratch + sc.dstate; db.chunk_stride = nc;
  cut<kHeadP, N, false>(p, &dx, seg);
  cut<N, kHeadP, true>(p, &dc, seg + run);
  cut<N, kHeadP, true>(p, &db, seg + 3 * run);
  cudaError_t e;
  if (dc.segments > 1) {
    if ((e = launch<T, N, kHeadP, false, true, true>(p, dc, false, s)) != cudaSuccess) return e;
    if ((e = launch<T, kHeadP, N, true, false, true>(p, dx, true, s)) != cudaSuccess) return e;
    if ((e = launch<T, N, kHeadP, true, true, true>(p, db, true, s)) != cudaSuccess) return e;
  }
  if ((e = launch<T, N, kHeadP, false, true, false>(p, dc, false, s)) != cudaSuccess) return e;
  if ((e = launch<T, kHeadP, N, true, false, false>(p, dx, true, s)) != cudaSuccess) return e;
  if ((e = launch<T, N, kHeadP, true, true, false>(p, db, true, s)) != cudaSuccess) return e;
  heads_kernel<T, N><<<unsigned((p.B * p.T * p.G + 7) / 8), 256, 0, s>>>(p, sc);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  anchor_kernel<<<unsigned(p.B * p.H * nc), 256, 0, s>>>(p, sc);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const SsmArgs& p, bool backward, cudaStream_t s) {
  if (p.N == 128) return backward ? bwd<T, 128>(p, s) : fwd<T, 128>(p, s);
  return backward ? bwd<T, 64>(p, s) : fwd<T, 64>(p, s);
}
cudaError_t run_dtype(const SsmArgs& p, int dtype, bool backward, cudaStream_t s) {
  switch (dtype) {
    case 0: return run<float>(p, backward, s);
    case 1: return run<__nv_bfloat16>(p, backward, s);
    case 2: return run<__half>(p, backward, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// fp32 elements of the runs' states and (fp64) decays, enough for twice as much where the states are fp64 too; whole 16
// bytes, as several follow one another.
int64_t ssm_run_floats(int64_t B, int64_t T, int64_t H, int N) {
  const int64_t k = scan_segments(B * H, T);
  return k > 1 ? (B * H * k * (kHeadP * N + 2) + 3) / 4 * 4 : 0;
}

cudaError_t launch_ssm_scan_fwd(const SsmArgs& p, int dtype, cudaStream_t s) { return run_dtype(p, dtype, false, s); }
cudaError_t launch_ssm_scan_bwd(const SsmArgs& p, int dtype, cudaStream_t s) { return run_dtype(p, dtype, true, s); }

}  // namespace wkv7
