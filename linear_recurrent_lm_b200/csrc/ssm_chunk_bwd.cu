// Backward of the chunked selective scan (see ssm_chunk.cu for the forward's formulas and names).  With dS the gradient
// of the state after the chunk (from the reversed state pass), L_ts = e^{Lambda_t - Lambda_s} (s <= t in one segment) and
// K = dY X^T:
//   dX = d [ (L o G)^T dY + diag(out) B dS^T ] + D dY
//   dB = sum over heads of (L o K diag(d))^T C + diag(d out) X dS,   dC = sum of (L o K diag(d)) B + diag(in) dY S
// and, for the gradient of the decays (ssm_decay.cu), with W = L o G o K:
//   row_t = sum_{s<t} d_s W_ts + in_t dy_t . (S c_t),   col_s = sum_{t>s} W_ts,   far_s = out_s x_s . (dS b_s),
//   own_t = G_tt K_tt,   xdy_t = K_tt,   anchor = e^{Lambda_end} <S, dS>.
// Everything is computed transposed (rows s, columns t >= s), so that (L o G)^T and (L o K)^T come out as A operands.
//
// Precision: G and K are products of the bf16 inputs themselves, so W is an fp32 result, and its row and column sums, most
// of which cancel against each other in the decays' gradient, are taken in fp64 (in fp32 dA was off by 4e-6); S and dS enter the
// products behind row and far in three bf16 parts (2^-26) and those behind dB and dC in two (2^-18), as do L o G and L o K off
// the diagonal and the scaled dY and X: with one part each, db and dc were off by as much again as their own rounding.
//
// One CTA per (b, chunk, group, part of the group's heads); b and c tiles stay in shared memory while it walks the heads,
// and dB, dC accumulate in TMEM over them.  Sixteen warps work in the same phase (ssm_chunk.cu says why):
//   A  S into bf16 parts, in_t dy_t          (while G and K are computed)
//   W  G and K from TMEM: L o G back to TMEM, d L o K to shared memory, the sums
//   B  d_s out_s x_s, dS into bf16 parts (once the products with S are done)
//   E  dX; the second parts of d L o K and of d_s out_s x_s, each in the place of the first once that has been read (that of
//      in_t dy_t is in A, in a half of the place of d L o K)
// while further warps issue MMAs (16), load tiles (17), prepare the decays (18) and, from the sums that the working warps
// leave, write the per-token scalars of the head before (19).
// TMEM: [0,128) G, then both parts of L o G, each 16 columns in the place of theirs, then B dS^T (64); [128,256) K, then C S^T
// (64) and (L o G)^T dY (64); dB; dC.
// What bounds it: phase W, by the instructions of one scheduler.  A warp reaches the TMEM lanes of its number modulo four,
// which is its scheduler too, so the first quadrant's four warps share the eight 16-column units of the longest rows (550
// instructions each before the second parts, a third of them fp64): 5000 of about 19000 cycles per chunk and head; the others
// wait for them.
// The MMA work is 7100 cycles at N = 128, at the rates measured for these shapes.  B=8 T=4096 H=32 N=128: 808 us, and with the
// reversed state pass and the sums behind it 960 (830 with one part each: nearly all of the difference is W's instructions, as
// the second products run beside them).
#include "ssm_chunk.h"
#include "ssm_tc.cuh"

namespace wkv7 {
namespace {

using namespace stc;

constexpr int kWorkers = 16, kThreads = 32 * (kWorkers + 4);   // 20 warps of 96 registers; a 21st would leave 80
constexpr uint32_t kTG = 0, kTXi = 0, kTK = 128, kTY2 = 128, kTX1 = 192, kTdB = 256, kTdC = 384;

template <int N>
struct Smem {
  static constexpr int kNB = N / 64, kPart = N * 128;          // bytes of one bf16 part of a state, rows n of 64 p
  static constexpr int kB = 0, kC = kB + kNB * kTileBytes, kX = kC + kNB * kTileBytes, kdY = kX + kTileBytes;
  static constexpr int kM1 = kdY + kTileBytes, kS = kM1 + 2 * kTileBytes, kSc = kS + 3 * kPart, kEnd = kSc + kTileBytes;
  struct Tail {
    Decays dec[3];
    double rowp[4][kQ];            // row sums of W from the rows of each quadrant
    double colp[4][kQ];            // col, dy . (S c) and x . (dS b) from the quadrant's four warps
    float rp[4][kQ], fp[4][kQ];
    float own_g[kQ], own_k[kQ];
    double sds[kWorkers];
    unsigned long long bc_full, xy_full, xy_free, gk_full, s_ready, w_ready, y2_full, m_done, ds_ready, xi_full, xs_done, m2_ready,
        x2_ready, e_full, ab_free, dec_full[3], dec_free[3], sums_free, sc_free, drained;
    uint32_t tmem;
    int dead;
  };
  static constexpr int kBytes = kEnd + int(sizeof(Tail)) + 1024;
};

__device__ __forceinline__ void prefetch_l2(const float* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Sums of 16 values over the 32 lanes: lane l gets that of value l & 15.
__device__ __forceinline__ double lane_sums(double (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 8; h; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const double keep = up ? v[i + h] : v[i], give = up ? v[i] : v[i + h];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) ssm_chunk_bwd_kernel(const SsmArgs p, const SsmScratch sc,
                                                                      const __grid_constant__ TileMaps tm) {
  using SM = Smem<N>;
  constexpr int NB = SM::kNB, PP = 64 * N / (32 * kWorkers);   // state elements of a thread: PP rows of one column
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  auto& tl = *reinterpret_cast<typename SM::Tail*>(sm + SM::kEnd);
  const uint32_t base = smem_addr(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t nc = chunks_of(p.T), hg = p.H / p.G, splits = sc.splits, per = (hg + splits - 1) / splits;
  int64_t id = blockIdx.x;
  const int64_t part = id % splits; id /= splits;
  const int64_t g = id % p.G; id /= p.G;
  const int64_t c = id % nc, b = id / nc;
  const int64_t h0 = g * hg + part * per;
  const int64_t left = hg - part * per;
  const int n = left > 0 ? int(min64(per, left)) : 0;   // heads of this CTA (none: its sums are zero)
  const int t0 = int(c * kQ);

  if (threadIdx.x == 0) {
    tl.dead = 0;
    unsigned long long* one[] = {&tl.bc_full, &tl.xy_full, &tl.gk_full, &tl.y2_full, &tl.m_done, &tl.xi_full, &tl.e_full,
                                 &tl.sums_free, &tl.sc_free, &tl.xs_done, &tl.drained};
    for (auto* bar : one) mbar_init(bar, 1);
    unsigned long long* all[] = {&tl.xy_free, &tl.s_ready, &tl.w_ready, &tl.ds_ready, &tl.m2_ready, &tl.x2_ready, &tl.ab_free};
    for (auto* bar : all) mbar_init(bar, kWorkers);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&tl.dec_full[i], 1);
      mbar_init(&tl.dec_free[i], kWorkers + 1);
    }
  }
  // the half of (L o K)^T behind the diagonal blocks stays zero
  for (int i = threadIdx.x; i < 2 * kTileBytes / 16; i += kThreads) reinterpret_cast<uint4*>(sm + SM::kM1)[i] = make_uint4(0, 0, 0, 0);
  if (warp == 16) {
    tc::alloc(&tl.tmem, 512);
    tc::relinquish();
  }
  tc::fence_smem_to_async();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tl.tmem;
  const Wait wait{&tl.dead, p.status};
  auto ph = [](int i) { return unsigned(i) & 1u; };
  int bc_loads = 0, xy_loads = 0;

  if (warp == 17) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && n > 0 && in_bounds(t0 < p.T && b < p.B && h0 + n <= p.H, p.status)) {
      mbar_arrive_expect_tx(&tl.bc_full, 2 * NB * kTileBytes);
      for (int j = 0; j < NB; ++j) {
        tma_load_4d(sm + SM::kB + j * kTileBytes, &tm.b, 64 * j, int(g), t0, int(b), &tl.bc_full);
        tma_load_4d(sm + SM::kC + j * kTileBytes, &tm.c, 64 * j, int(g), t0, int(b), &tl.bc_full);
      }
      ++bc_loads;
      auto ahead = [&](int i) {   // a head's state and its gradient into the L2
        if (i >= n) return;
        const int64_t unit = b * p.H + h0 + i;
        prefetch_l2(p.ckpt + (unit * (nc + 1) + c) * 64 * N, 64 * N * 4);
        prefetch_l2(p.scratch + sc.dstate + (unit * nc + c) * 64 * N, 64 * N * 4);
      };
      ahead(0);
      for (int i = 0; i < n; ++i) {
        ahead(i + 1);
        if (i >= 1 && !wait(&tl.xy_free, ph(i - 1))) break;
        mbar_arrive_expect_tx(&tl.xy_full, 2 * kTileBytes);
        tma_load_4d(sm + SM::kX, &tm.x, 0, int(h0 + i), t0, int(b), &tl.xy_full);
        tma_load_4d(sm + SM::kdY, &tm.dy, 0, int(h0 + i), t0, int(b), &tl.xy_full);
        ++xy_loads;
      }
    }
  } else if (warp == 19) {
    // ------------------------------------------------------------ the per-token scalars, from the working warps' sums
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int64_t unit = b * p.H + h0 + i;
      if (!(ok = wait.warp(&tl.dec_full[i % 3], unsigned(i / 3) & 1u) && wait.warp(&tl.ab_free, ph(i)))) break;
      const Decays& dec = tl.dec[i % 3];
      double row[4], col[4];   // all of it is read first: the working warps wait for that
      float far[4], own[4], xdy[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = 32 * q + lane;
        double rs = 0.0;
#pragma unroll
        for (int j = 0; j <= q; ++j) rs += tl.rowp[j][t];
        row[q] = rs + double(dec.in[t] * ((tl.rp[0][t] + tl.rp[1][t]) + (tl.rp[2][t] + tl.rp[3][t])));
        col[q] = (tl.colp[0][t] + tl.colp[1][t]) + (tl.colp[2][t] + tl.colp[3][t]);
        far[q] = dec.out[t] * ((tl.fp[0][t] + tl.fp[1][t]) + (tl.fp[2][t] + tl.fp[3][t]));
        xdy[q] = tl.own_k[t];
        own[q] = tl.own_g[t] * xdy[q];
      }
      double s = lane < kWorkers ? tl.sds[lane] : 0.0;
      const float gam = dec.total;
      __syncwarp();
      if (lane == 0) {
        arrive(&tl.dec_free[i % 3]);
        arrive(&tl.sums_free);
      }
      const int64_t o = unit * nc * kQ + t0 + lane;
      if (!range_ok(o - lane, kQ, p.B * p.H * nc * kQ, p.status)) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        reinterpret_cast<double*>(p.scratch + sc.row)[o + 32 * q] = row[q];
        reinterpret_cast<double*>(p.scratch + sc.col)[o + 32 * q] = col[q];
        p.scratch[sc.far + o + 32 * q] = far[q];
        p.scratch[sc.own + o + 32 * q] = own[q];
        p.scratch[sc.xdy + o + 32 * q] = xdy[q];
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      if (lane == 0) reinterpret_cast<double*>(p.scratch + sc.anchor)[unit * nc + c] = double(gam) * s;
    }
  } else if (warp == 18) {
    // ------------------------------------------------------------ decays
    RawSteps raw;
    if (n > 0) raw.load(p, b, h0, c);
    for (int i = 0; i < n; ++i) {
      const float A = __ldg(p.A + h0 + i), bias = p.dt_bias ? __ldg(p.dt_bias + h0 + i) : 0.f;
      if (i >= 3 && !wait.warp(&tl.dec_free[i % 3], unsigned(i / 3 - 1) & 1u)) break;
      const RawSteps now = raw;
      if (i + 1 < n) raw.load(p, b, h0 + i + 1, c);
      chunk_decays<kBackward>(p, A, bias, c, now, tl.dec[i % 3]);
      __syncwarp();
      if (lane == 0) arrive(&tl.dec_full[i % 3]);
    }
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issue: one elected lane of a warp that stays together
    const uint64_t dBk = desc(base + SM::kB, 16), dCk = desc(base + SM::kC, 16), dBm = desc(base + SM::kB, kTileBytes),
                   dCm = desc(base + SM::kC, kTileBytes), dX = desc(base + SM::kX, 16), ddY = desc(base + SM::kdY, 16),
                   dM1k = desc(base + SM::kM1, 16), dM1m = desc(base + SM::kM1, kTileBytes), dS = desc(base + SM::kS, 16),
                   dSc = desc(base + SM::kSc, 16);
    constexpr uint32_t kIdG = tc::idesc_bf16(128, 128, 0, 0), kIdY = tc::idesc_bf16(128, 64, 0, 1), kIdN = tc::idesc_bf16(128, N, 0, 0),
                       kIddB = tc::idesc_bf16(128, N, 0, 1), kIddC = tc::idesc_bf16(128, N, 1, 1);
    // q groups of four K steps: A `ka` bytes apart in the step and `ga` in the group (mod `wrap` groups), B likewise
    auto products = [&](uint32_t d, uint64_t a, uint32_t ka, uint32_t ga, int wrap, uint64_t bd, uint32_t kb, uint32_t gb, int q,
                        uint32_t idesc, bool add) {
#pragma unroll 1
      for (int j = 0; j < q; ++j) {
        const uint64_t aj = a + ((j & (wrap - 1)) * ga >> 4), bj = bd + (j * gb >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::mma_bf16(d, aj + (k * ka >> 4), bj + (k * kb >> 4), idesc, add || j + k > 0);
      }
    };
    bool ok = n == 0 || wait.warp(&tl.bc_full, 0);
    for (int i = 0; ok && i < n; ++i) {
      if (!(ok = wait.warp(&tl.xy_full, ph(i)) && (i == 0 || wait.warp(&tl.ab_free, ph(i - 1))))) break;
      tc::fence_after_sync();
      if (elected()) {   // K^T = X dY^T, G^T = B C^T
        products(tmem + kTK, dX, 32, 0, 1, ddY, 32, 0, 1, kIdG, false);
        products(tmem + kTG, dBk, 32, kTileBytes, NB, dCk, 32, kTileBytes, NB, kIdG, false);
        tc::commit(&tl.gk_full);
      }
      __syncwarp();
      if (!(ok = wait.warp(&tl.s_ready, ph(i)))) break;
      tc::fence_after_sync();
      if (elected()) {   // dC += (in dY) S: the second part with the first of S, the first with two of S
        products(tmem + kTdC, dM1k + (kTileBytes >> 4), 32, 0, 1, dS + (2 * SM::kPart >> 4), 32, 0, 1, kIdN, i > 0);
        products(tmem + kTdC, dSc, 32, 0, 1, dS + (SM::kPart >> 4), 32, SM::kPart, 2, kIdN, true);
        tc::commit(&tl.sc_free);
      }
      __syncwarp();
      if (!(ok = wait.warp(&tl.w_ready, ph(i)))) break;
      tc::fence_after_sync();
      if (elected()) {
        products(tmem + kTY2, dCk, 32, kTileBytes, NB, dS, 2048, 8192, 3 * NB, kIdY, false);   // C S^T, three parts
        tc::commit(&tl.y2_full);
#pragma unroll 1
        for (int k = 0; k < 16; ++k)   // (L o G)^T dY, the second part first
          mma_bf16_ts(tmem + kTX1, tmem + kTG + 16 * (k & 7) + (k < 8 ? 8 : 0), mn_step(ddY, k & 7), kIdY, k > 0);
        products(tmem + kTdB, dM1k, 32, kTileBytes, 2, dCm, 2048, 8192, 2, kIddB, i > 0);      // dB += (L o K d)^T C
        products(tmem + kTdC, dM1m, 2048, 8192, 2, dBm, 2048, 8192, 2, kIddC, true);           // dC += (L o K d) B
        tc::commit(&tl.m_done);
      }
      __syncwarp();
      if (!(ok = wait.warp(&tl.ds_ready, ph(i)) && wait.warp(&tl.m_done, ph(i)))) break;   // (L o G has been read)
      tc::fence_after_sync();
      if (elected()) {
        products(tmem + kTXi, dBk, 32, kTileBytes, NB, dS, 2048, 8192, 3 * NB, kIdY, false);   // B dS^T, three parts
        tc::commit(&tl.xi_full);
        products(tmem + kTdB, dSc, 32, 0, 1, dS + (SM::kPart >> 4), 32, SM::kPart, 2, kIdN, true);   // dB += (d out X) dS, two
        tc::commit(&tl.xs_done);
      }
      __syncwarp();
      if (!(ok = wait.warp(&tl.m2_ready, ph(i)))) break;
      tc::fence_after_sync();
      if (elected()) {   // the second part of L o K d
        products(tmem + kTdB, dM1k, 32, kTileBytes, 2, dCm, 2048, 8192, 2, kIddB, true);
        products(tmem + kTdC, dM1m, 2048, 8192, 2, dBm, 2048, 8192, 2, kIddC, true);
      }
      __syncwarp();
      if (!(ok = wait.warp(&tl.x2_ready, ph(i)))) break;
      tc::fence_after_sync();
      if (elected()) {   // the second part of d out X, with the first of dS
        products(tmem + kTdB, dSc, 32, 0, 1, dS + (2 * SM::kPart >> 4), 32, 0, 1, kIdN, true);
        tc::commit(&tl.e_full);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ the working warps
    const int w = warp & 3, r = warp >> 2, row = 32 * w + lane;
    const uint32_t lanes = tmem + (uint32_t(32 * w) << 16);
    const int sn = threadIdx.x % N, sp = threadIdx.x / N * PP;   // this thread's state column and first state row
    bool ok = true;
    // the state (or its gradient) of this thread into three bf16 parts, the smallest first: the tensor core cuts its sums
    // off below their leading bits, which the large part then meets in its own steps only
    auto fetch = [&](const float* src, float (&v)[PP]) {
#pragma unroll
      for (int q = 0; q < PP; ++q) v[q] = __ldg(src + (sp + q) * N + sn);
    };
    auto parts = [&](float (&v)[PP]) {
#pragma unroll
      for (int q = 0; q < PP; ++q) asm volatile("" : "+f"(v[q]));   // not before the wait in front: the loads run until here
#pragma unroll
      for (int j = 0; j < PP / 8; ++j) {
        uint32_t o[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 f = make_float2(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]);
          o[0][k] = split(f);
          o[1][k] = split(f);
          o[2][k] = pack(f.x, f.y);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<uint4*>(sm + SM::kS + (2 - q) * SM::kPart + swz(sn, sp / 8 + j)) =
              make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
      }
    };
    // this thread's 16 channels of its token row of `tile`, scaled, into the scaled tile (the first part), and the second
    // part into `second`, if there is one
    auto scaled = [&](int tile, float f, int second) {
#pragma unroll 1
      for (int j = 2 * r; j < 2 * r + 2; ++j) {
        const uint32_t o = swz(row, j);
        const uint4 v = *reinterpret_cast<const uint4*>(sm + tile + o);
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
        uint32_t out[4], rest[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 q = mul2(stc::unpack(in[k]), make_float2(f, f));
          out[k] = split(q);
          rest[k] = pack(q.x, q.y);
        }
        *reinterpret_cast<uint4*>(sm + SM::kSc + o) = make_uint4(out[0], out[1], out[2], out[3]);
        if (second >= 0) *reinterpret_cast<uint4*>(sm + second + o) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
      }
    };
    auto hand_over = [&](unsigned long long* bar) {
      tc::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) arrive(bar);
    };
    float S[PP];   // this thread's part of the state, fetched a phase ahead
    if (n > 0) fetch(p.ckpt + ((b * p.H + h0) * (nc + 1) + c) * 64 * N, S);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int64_t unit = b * p.H + h0 + i;
      const Decays& dec = tl.dec[i % 3];
      // ---- A: S, in dY
      if (i > 0 && !(ok = wait.warp(&tl.e_full, ph(i - 1)))) break;   // the last head's products with both buffers are done
      parts(S);
      if (!(ok = wait.warp(&tl.dec_full[i % 3], unsigned(i / 3) & 1u) && wait.warp(&tl.xy_full, ph(i)))) break;
      const float in = dec.in[row], out = dec.out[row], d = dec.d[row];
      scaled(SM::kdY, in, SM::kM1 + kTileBytes);
      hand_over(&tl.s_ready);
      // ---- W: columns t of row s, 16 at a time from the diagonal block on
      if (!(ok = wait.warp(&tl.gk_full, ph(i)) && (i == 0 || wait.warp(&tl.sums_free, ph(i - 1))))) break;
      tc::fence_after_sync();
      double col = 0.0;
      uint32_t ma[8], mb[8];   // the second parts of d L o K
      {
        const float hi = dec.hi[row], lo = dec.lo[row], fs = decay_between(dec.hi[32 * w + 31], dec.lo[32 * w + 31], hi, lo);
        const bool grow = dec.growing != 0, resets = dec.resets != 0;
        const float* far = dec.far + 32 * (w == 0 ? 0 : w == 1 ? 3 : 5) - 32 * (w + 1);   // indexed by t
#pragma unroll 1
        for (int it = 0; it < 2; ++it) {
          const int c0 = 32 * w + 16 * (r + 4 * it);
          if (c0 >= kQ) break;
          float gv[16], kv[16];
          double wv[16];
          ld16(lanes + kTG + c0, gv);
          ld16(lanes + kTK + c0, kv);
          float L[16] = {};
          if (grow) {   // decays above one: the two factors could overflow where their product does not
#pragma unroll 1
            for (int s = 0; s < 16; ++s) {
              const float l = c0 + s >= row ? decay_between(dec.hi[c0 + s], dec.lo[c0 + s], hi, lo) : 0.f;
#pragma unroll
              for (int e = 0; e < 16; ++e) L[e] = e == s ? l : L[e];
            }
          } else if (c0 < 32 * w + 32) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {   // (the exponent is masked, not the result: no branch around the exponential)
              const float x = (dec.hi[c0 + e] - hi) + (dec.lo[c0 + e] - lo);
              L[e] = ex2(c0 + e >= row ? x : -1e30f);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) L[e] = fs * far[c0 + e];
          }
          if (resets)
#pragma unroll
            for (int e = 0; e < 16; ++e) L[e] = row >= dec.start[c0 + e] ? L[e] : 0.f;
          tc::wait_ld();
          if (c0 < 32 * w + 32) {   // the token itself: its part of (L o G) and of W is handled in fp32
            float og = 0.f, ok_ = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const bool me = c0 + e == row;
              og = me ? gv[e] : og;
              ok_ = me ? kv[e] : ok_;
              gv[e] = me ? 0.f : gv[e];
            }
            if (row >> 4 == c0 >> 4) {
              tl.own_g[row] = og;
              tl.own_k[row] = ok_;
            }
          }
          uint32_t m[8], gm[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 l2 = make_float2(L[2 * e], L[2 * e + 1]), k2 = make_float2(kv[2 * e], kv[2 * e + 1]);
            float2 lg = mul2(l2, make_float2(gv[2 * e], gv[2 * e + 1]));
            float2 kd = mul2(mul2(l2, k2), make_float2(d, d));
            const float2 wd = mul2(lg, k2);
            wv[2 * e] = double(wd.x);
            wv[2 * e + 1] = double(wd.y);
            col += wv[2 * e] + wv[2 * e + 1];
            wv[2 * e] *= double(d);
            wv[2 * e + 1] *= double(d);
            gm[e] = split(lg);
            gm[8 + e] = pack(lg.x, lg.y);
            m[e] = split(kd);
            if (it == 0) ma[e] = pack(kd.x, kd.y);
            else mb[e] = pack(kd.x, kd.y);
          }
          if (it == 0 && !(ok = wait.warp(&tl.sc_free, ph(i)))) break;   // the second part of in dY has been read
          st16(lanes + kTG + c0, gm);   // in the place of these columns of G, which no other warp reads
          uint8_t* m1 = sm + SM::kM1 + (c0 >> 6) * kTileBytes;
          *reinterpret_cast<uint4*>(m1 + swz(row, (c0 & 63) >> 3)) = make_uint4(m[0], m[1], m[2], m[3]);
          *reinterpret_cast<uint4*>(m1 + swz(row, ((c0 & 63) >> 3) + 1)) = make_uint4(m[4], m[5], m[6], m[7]);
          const double rs = lane_sums(wv);
          if (lane < 16) tl.rowp[w][c0 + lane] = rs;
        }
      }
      if (!(ok = ok && wait.warp(&tl.sc_free, ph(i)))) break;
      if (w == 3) *reinterpret_cast<uint4*>(sm + SM::kM1 + kTileBytes + swz(row, r)) = make_uint4(0, 0, 0, 0);   // it lay there too
      tl.colp[r][row] = col;
      {
        const uint32_t zero[16] = {};
        for (int z = 16 * r; z < 32 * w; z += 64) st16(lanes + kTG + z, zero);
        tc::wait_st();
      }
      tc::fence_before_sync();
      hand_over(&tl.w_ready);
      // ---- B: d out X (the product with the scaled dY is done), dS (those with S are)
      float S2[PP], dS[PP];   // S again, for <S, dS>: kept since phase A it would be 16 registers through W
      fetch(p.ckpt + (unit * (nc + 1) + c) * 64 * N, S2);
      fetch(p.scratch + sc.dstate + (unit * nc + c) * 64 * N, dS);
      scaled(SM::kX, d * out, -1);
      if (!(ok = wait.warp(&tl.y2_full, ph(i)))) break;
      tc::fence_after_sync();
      float y2[16];
      ld16(lanes + kTY2 + 16 * r, y2);
      double sds;
      {
        parts(dS);
        float a = 0.f;
#pragma unroll
        for (int q = 0; q < PP; ++q) a = fmaf(S2[q], dS[q], a);
        sds = double(a);
      }
      hand_over(&tl.ds_ready);
      // ---- E: this thread's 16 channels of x and dy, then the tiles may be loaded anew
      uint32_t xv[8], yv[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 a = *reinterpret_cast<const uint4*>(sm + SM::kX + swz(row, 2 * r + j));
        const uint4 q = *reinterpret_cast<const uint4*>(sm + SM::kdY + swz(row, 2 * r + j));
        xv[4 * j] = a.x; xv[4 * j + 1] = a.y; xv[4 * j + 2] = a.z; xv[4 * j + 3] = a.w;
        yv[4 * j] = q.x; yv[4 * j + 1] = q.y; yv[4 * j + 2] = q.z; yv[4 * j + 3] = q.w;
      }
      tc::wait_ld();
      {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) a = fma2(stc::unpack(yv[k]), make_float2(y2[2 * k], y2[2 * k + 1]), a);
        tl.rp[r][row] = a.x + a.y;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sds += __shfl_xor_sync(0xffffffffu, sds, o);
      if (lane == 0) tl.sds[warp] = sds;
      if (!(ok = wait.warp(&tl.m_done, ph(i)))) break;
      __syncwarp();
      if (lane == 0) arrive(&tl.xy_free);
#pragma unroll
      for (int it = 0; it < 2; ++it) {   // the second parts of d L o K take the place of the first
        const int c0 = 32 * w + 16 * (r + 4 * it);
        const uint32_t(&m)[8] = it == 0 ? ma : mb;
        if (c0 < kQ) {
          uint8_t* m1 = sm + SM::kM1 + (c0 >> 6) * kTileBytes;
          *reinterpret_cast<uint4*>(m1 + swz(row, (c0 & 63) >> 3)) = make_uint4(m[0], m[1], m[2], m[3]);
          *reinterpret_cast<uint4*>(m1 + swz(row, ((c0 & 63) >> 3) + 1)) = make_uint4(m[4], m[5], m[6], m[7]);
        }
      }
      hand_over(&tl.m2_ready);
      if (!(ok = wait.warp(&tl.xi_full, ph(i)))) break;
      tc::fence_after_sync();
      const int64_t t = t0 + row;
      {
        float x1[16], xi[16];
        ld16(lanes + kTX1 + 16 * r, x1);
        ld16(lanes + kTXi + 16 * r, xi);
        const float skip = (p.Dw ? __ldg(p.Dw + h0 + i) : 0.f) + d * tl.own_g[row], od = d * out;
        tc::wait_ld();
        tc::fence_before_sync();
        float2 a = make_float2(0.f, 0.f);
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = make_float2(xi[2 * k], xi[2 * k + 1]);
          a = fma2(stc::unpack(xv[k]), f, a);
          float2 q = mul2(make_float2(d, d), make_float2(x1[2 * k], x1[2 * k + 1]));
          q = fma2(make_float2(od, od), f, q);
          q = fma2(make_float2(skip, skip), stc::unpack(yv[k]), q);
          o[k] = pack(q.x, q.y);
        }
        tl.fp[r][row] = a.x + a.y;
        // (an arrival waits for the stores before it, so dX is stored behind these)
        __syncwarp();
        if (lane == 0) {
          arrive(&tl.dec_free[i % 3]);
          arrive(&tl.ab_free);
        }
        if (!(ok = wait.warp(&tl.xs_done, ph(i)))) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // the second part of d out X takes the place of the first
          uint32_t q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 f = mul2(stc::unpack(xv[4 * j + k]), make_float2(od, od));
            split(f);
            q[k] = pack(f.x, f.y);
          }
          *reinterpret_cast<uint4*>(sm + SM::kSc + swz(row, 2 * r + j)) = make_uint4(q[0], q[1], q[2], q[3]);
        }
        hand_over(&tl.x2_ready);
        if (t < p.T && range_ok(t, 1, p.T, p.status)) {
          uint4* dx = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dx) + ((b * p.T + t) * p.H + h0 + i) * 64 + 16 * r);
          dx[0] = make_uint4(o[0], o[1], o[2], o[3]);
          dx[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      if (i + 1 < n) fetch(p.ckpt + ((unit + 1) * (nc + 1) + c) * 64 * N, S);   // the next head's state, under way
    }
    // ---- dB and dC
    if (ok && n > 0) ok = wait.warp(&tl.e_full, ph(n - 1));
    if (ok) {
      tc::fence_after_sync();
      const int64_t t = t0 + row, at = ((b * p.T + t) * p.G + g) * N;
      const bool live = t < p.T && range_ok(t, 1, p.T, p.status);
#pragma unroll 1
      for (int q = r; q < 2 * N / 16; q += 4) {
        const bool second = q >= N / 16;
        const int c0 = 16 * (second ? q - N / 16 : q);
        float v[16];
        if (n > 0) {
          ld16(lanes + (second ? kTdC : kTdB) + c0, v);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0.f;
        }
        if (!live) continue;
        if (splits > 1) {
          float4* o = reinterpret_cast<float4*>(p.scratch + (second ? sc.dc_part : sc.db_part) + part * p.B * p.T * p.G * N + at + c0);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
          uint32_t m[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = pack(v[2 * e], v[2 * e + 1]);
          uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(second ? p.dc : p.db) + at + c0);
          o[0] = make_uint4(m[0], m[1], m[2], m[3]);
          o[1] = make_uint4(m[4], m[5], m[6], m[7]);
        }
      }
      tc::fence_before_sync();
    }
  }
  // ------------------------------------------------------------ end: nothing of this CTA may be in flight
  __syncwarp();
  if (lane == 0 && *reinterpret_cast<volatile int*>(&tl.dead)) {   // a wait was given up: loads and MMAs may be under way
    const unsigned long long began = global_ns();
    auto drain = [&](unsigned long long* bar, unsigned parity) {
      while (!mbar_try_wait(bar, parity) && global_ns() - began < kWaitLimitNs) {}
    };
    if (warp == 17) {
      if (bc_loads) drain(&tl.bc_full, 0);
      if (xy_loads) drain(&tl.xy_full, ph(xy_loads - 1));
    } else if (warp == 16) {
      tc::commit(&tl.drained);
      drain(&tl.drained, 0);
    }
  }
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 16) tc::dealloc(tmem, 512);
}

// dB and dC from the sums of the splits: one thread per 4 values.
__global__ void __launch_bounds__(256) split_sums_kernel(const SsmArgs p, const SsmScratch sc) {
  const int64_t n = p.B * p.T * p.G * p.N, i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= 2 * n) return;
  const bool second = i >= n;
  const int64_t at = second ? i - n : i;
  const float* src = p.scratch + (second ? sc.dc_part : sc.db_part) + at;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t k = 0; k < sc.splits; ++k) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(src + k * n));
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(second ? p.dc : p.db) + at) = make_uint2(pack(s.x, s.y), pack(s.z, s.w));
}

template <int N>
cudaError_t run(const SsmArgs& p, const SsmScratch& sc, const TileMaps& tm, cudaStream_t s) {
  static_assert(Smem<N>::kBytes <= 232448, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(ssm_chunk_bwd_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<N>::kBytes);
  if (e != cudaSuccess) return e;
  ssm_chunk_bwd_kernel<N><<<unsigned(p.B * chunks_of(p.T) * p.G * sc.splits), kThreads, Smem<N>::kBytes, s>>>(p, sc, tm);
  if ((e = cudaGetLastError()) != cudaSuccess || sc.splits == 1) return e;
  split_sums_kernel<<<unsigned((p.B * p.T * p.G * N / 2 + 255) / 256), 256, 0, s>>>(p, sc);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_chunk_bwd(const SsmArgs& p, const TileMaps& tm, cudaStream_t s) {
  const SsmScratch sc = ssm_scratch(p.B, p.T, p.H, p.G, p.N, true);
  const cudaError_t e = launch_ssm_chunk_dstate(p, tm, p.scratch + sc.dstate, p.scratch + sc.seg, s);
  if (e != cudaSuccess) return e;
  return p.N == 128 ? run<128>(p, sc, tm, s) : run<64>(p, sc, tm, s);
}

}  // namespace wkv7
