// Selective state space scan in chunks of 128 tokens on the tensor cores (algo CHUNKED, bf16).
//
// In a chunk with entering state S, Lambda_t the log decay from the chunk's start through token t, and d_t the steps:
//   G = C B^T,   M_ts = G_ts e^{Lambda_t - Lambda_s} d_s   (s <= t in the same segment),
//   Y = M X + diag(in_t) C S^T + D X,          in_t = e^{Lambda_t}           (0 behind a reset)
//   S' = e^{Lambda_end} S + X^T diag(d_s out_s) B,  out_s = e^{Lambda_end - Lambda_s}  (0 before a reset)
// The gradient of the state runs the same last line backwards: dS' = e^{Lambda_end} dS + dY^T diag(in_t) C, so one
// kernel serves both (REV), without the outputs (OUT = false).
//
// Precision: x, b, c enter the products as the bf16 they are; accumulators, decays and the carried state are fp32
// (Lambda fp64).  What is rounded: M off its diagonal to two bf16 parts (2^-18; one part alone put 2^-9 of every term into y,
// as much again as its own rounding) and S to two in C S^T (2^-18); the weighted x to three in the state's update (2^-26),
// so that states are fp32 results.
//
// One CTA per (b, h) and segment of its chunks, one CTA per SM (its tiles fill the shared memory).  Sixteen warps work,
// four per quadrant of TMEM lanes, all through the same phases of a chunk:
//   M     thread = token row, 16 columns at a time, dealt to the quadrant's warps up to the diagonal.  G comes from TMEM, M
//         goes back there as the A operand of M X; off the diagonal blocks the decay is a product of a row and a column
//         factor, both relative to the row block's start (so at most one), which leaves 32 exponentials per row, not 128
//   S     thread = state column, 16 fp32 rows of it in registers: add U, and write the bf16 parts for C S^T
//   XS    thread = token row, a quarter of it: the weighted x in three bf16 parts
//   Y     thread = token row, a quarter of it: Y1 + in Y2 + (D + M_tt) x, in the place of x
// while warp 16 issues the MMAs (one phase ahead of what is read), warp 17 loads tiles and stores y (TMA, 128-byte swizzle) and
// warps 18 and 19 prepare the decays (fp64 prefix sums), every other chunk each, up to three ahead.
//
// What bounds it: instruction fetch.  Code beyond the few KB of a scheduler's own cache arrives at 5.5 cycles per
// instruction (measured on straight-line FMAs), once for all warps of the scheduler that run it together.  Roles on
// separate warps (M, state, XS) therefore ran at 7300 to 11600 cycles per chunk; all warps in the same phase, loops rolled,
// share the fetches: about 6500.  MMA work per chunk and head at N = 128, in cycles at the rates measured for these shapes
// (a product of 64 columns with A in shared memory is bound by reading it): G 512, C S^T 784, M X 520, state 1176.
// B=8 T=4096 H=32 N=128: 238 us (219 with M in one part; 256 rows of heads on 148 SMs: 1.73 rounds cost two), the reversed
// state pass 137 us.
#include "ssm_chunk.h"
#include "ssm_tc.cuh"

namespace wkv7 {
namespace {

using namespace stc;

constexpr int kWorkers = 16, kDecayWarps = 2, kThreads = 32 * (kWorkers + 2 + kDecayWarps);

template <int N, bool OUT>
struct Smem {
  static constexpr int kNB = N / 64;             // 64-column tiles of b and c
  static constexpr int kX = 0, kB = kX + 2 * kTileBytes, kC = kB + 2 * kNB * kTileBytes;
  // The parts of the weighted x: twice for the states alone, where those of the next chunk are made while this one's product
  // runs.  With the outputs' work once, behind Y, whose buffer of x is then free sooner (N = 64, B=8 T=4096 H=32, measured with M in
  // one part: 213 us, 261 with two).
  static constexpr int kXSets = OUT ? 1 : 2;
  static constexpr int kXS = kC + (OUT ? kNB * kTileBytes : 0), kSH = kXS + kXSets * 3 * kTileBytes;
  static constexpr int kEnd = kSH + (OUT ? 2 * N * 128 : 0);
  struct Tail {
    Decays dec[3];
    float own[2][kQ];
    unsigned long long x_full[2], x_free[2], b_full[2], u_full[2], c_full, y2_done, g_full, m_ready[2], y_full[2],
        sh_ready[2], xs_ready[2], dec_full[3], dec_free[3];
    unsigned long long drained;
    uint32_t tmem;
    int dead;
  };
  static constexpr int kBytes = kEnd + int(sizeof(Tail)) + 1024;
};
// TMEM columns.  kTY2: two of 64.  kTU: two of 64 for the states alone; with the outputs one, as XS waits for the state
// then, and the second part of M behind it.
constexpr uint32_t kTG = 0, kTM = 128, kTY1 = 192, kTY2 = 256, kTU = 384, kTM2 = 448;

template <int N, bool OUT, bool REV>
__global__ void __launch_bounds__(kThreads, 1) ssm_chunk_kernel(const SsmArgs p, const __grid_constant__ TileMaps tm, const ChunkOp op) {
  using SM = Smem<N, OUT>;
  constexpr int NB = SM::kNB;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  auto& tl = *reinterpret_cast<typename SM::Tail*>(sm + SM::kEnd);
  const uint32_t base = smem_addr(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x / op.segments, seg = blockIdx.x - unit * op.segments;
  const int64_t b = unit / p.H, h = unit - b * p.H, g = h / (p.H / p.G);
  const int64_t nc = chunks_of(p.T);
  const int64_t pos0 = seg * op.per_segment;
  const int n = int(min64(op.per_segment, nc - pos0));   // chunks of this CTA, at least 1
  auto chunk = [&](int i) { return REV ? nc - 1 - (pos0 + i) : pos0 + i; };

  if (threadIdx.x == 0) {
    tl.dead = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tl.x_full[i], 1);
      mbar_init(&tl.x_free[i], kWorkers);
      mbar_init(&tl.b_full[i], 1);
      mbar_init(&tl.u_full[i], 1);
      mbar_init(&tl.m_ready[i], kWorkers);
      mbar_init(&tl.y_full[i], 1);
      mbar_init(&tl.sh_ready[i], kWorkers);
      mbar_init(&tl.xs_ready[i], kWorkers);
    }
    mbar_init(&tl.c_full, 1);
    mbar_init(&tl.g_full, 1);
    mbar_init(&tl.y2_done, 1);
    mbar_init(&tl.drained, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&tl.dec_full[i], 1);
      mbar_init(&tl.dec_free[i], kWorkers);
    }
  }
  if (warp == 16) {
    tc::alloc(&tl.tmem, 512);
    tc::relinquish();
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tl.tmem;
  const Wait wait{&tl.dead, p.status};
  auto ph = [](int i) { return unsigned(i >> 1) & 1u; };      // phase of a [2] barrier's use i
  auto ph3 = [](int i) { return unsigned(i / 3) & 1u; };
  int x_loads = 0, b_loads = 0, c_loads = 0;                  // loader: what has been asked for

  if (warp == 17) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      const CUtensorMap* mx = REV ? &tm.dy : &tm.x;
      const CUtensorMap* mb = REV ? &tm.c : &tm.b;
      // y of a chunk takes the place of its x (each thread that writes 16 channels of a row there has read those of x), and
      // goes out as a tile: as two 16-byte stores per row and thread it took 1800 cycles of the store path per chunk.
      auto store_y = [&](int i) {
        if (!wait(&tl.x_free[i & 1], ph(i))) return false;
        tma_store_4d(&tm.y, sm + SM::kX + (i & 1) * kTileBytes, 0, int(h), int(chunk(i) * kQ), int(b));
        tma_store_read();
        return true;
      };
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        ok = false;
        const int t0 = int(chunk(i) * kQ), s = i & 1;
        if (!in_bounds(t0 >= 0 && t0 < p.T && b < p.B && g < p.G, p.status)) break;
        if (i >= 2 && !wait(&tl.u_full[s], ph(i - 2))) break;
        mbar_arrive_expect_tx(&tl.b_full[s], NB * kTileBytes);
        for (int j = 0; j < NB; ++j)
          tma_load_4d(sm + SM::kB + (s * NB + j) * kTileBytes, mb, 64 * j, int(g), t0, int(b), &tl.b_full[s]);
        ++b_loads;
        if (OUT) {
          if (i >= 1 && !wait(&tl.y2_done, unsigned(i - 1) & 1u)) break;
          mbar_arrive_expect_tx(&tl.c_full, NB * kTileBytes);
          for (int j = 0; j < NB; ++j) tma_load_4d(sm + SM::kC + j * kTileBytes, &tm.c, 64 * j, int(g), t0, int(b), &tl.c_full);
          ++c_loads;
        }
        if (i >= 2 && !(OUT ? store_y(i - 2) : wait(&tl.x_free[s], ph(i - 2)))) break;
        mbar_arrive_expect_tx(&tl.x_full[s], kTileBytes);
        tma_load_4d(sm + SM::kX + s * kTileBytes, mx, 0, int(h), t0, int(b), &tl.x_full[s]);
        ++x_loads;
        ok = true;
      }
      if (OUT) {
        for (int i = n >= 2 ? n - 2 : 0; ok && i < n; ++i) ok = store_y(i);
        tma_store_done();
      }
    }
  } else if (warp >= 18) {
    // ------------------------------------------------------------ decays
    const float A = __ldg(p.A + h), bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
    RawSteps raw;
    const int first = warp - 18;
    if (first < n) raw.load(p, b, h, chunk(first));
    for (int i = first; i < n; i += kDecayWarps) {
      if (i >= 3 && !wait.warp(&tl.dec_free[i % 3], ph3(i - 3))) break;
      const RawSteps now = raw;
      if (i + kDecayWarps < n) raw.load(p, b, h, chunk(i + kDecayWarps));
      chunk_decays<OUT ? kForward : REV ? kReversed : kStates>(p, A, bias, chunk(i), now, tl.dec[i % 3]);
      __syncwarp();
      if (lane == 0) arrive(&tl.dec_full[i % 3]);
    }
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issue
    // The warp stays together and one elected lane issues (49 cycles per 128 x 64 x 16 MMA, 60 from lane 0 alone).
    const uint64_t dC = desc(base + SM::kC, 16), dSH = desc(base + SM::kSH, 16), dXS = desc(base + SM::kXS, 16);
    const uint64_t dBk = desc(base + SM::kB, 16), dBm = desc(base + SM::kB, kTileBytes), dX = desc(base + SM::kX, 16);
    constexpr uint32_t kIdG = tc::idesc_bf16(128, 128, 0, 0), kIdY = tc::idesc_bf16(128, 64, 0, 1), kIdU = tc::idesc_bf16(N, 64, 1, 1);
    // q groups of four K steps: A `ka` bytes apart in the step and `ga` in the group (mod `wrap` groups), B likewise
    auto products = [&](uint32_t d, uint64_t a, uint32_t ka, uint32_t ga, int wrap, uint64_t b, uint32_t kb, uint32_t gb, int q,
                        uint32_t id, unsigned long long* done) {
      tc::fence_after_sync();
      if (elected()) {
#pragma unroll 1
        for (int j = 0; j < q; ++j) {
          const uint64_t aj = a + ((j & (wrap - 1)) * ga >> 4), bj = b + (j * gb >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::mma_bf16(d, aj + (k * ka >> 4), bj + (k * kb >> 4), id, j + k > 0);
        }
        tc::commit(done);
      }
      __syncwarp();
    };
    bool ok = true;
    for (int i = -1; i < n; ++i) {
      if (OUT && i >= 0) {
        if (!(ok = wait.warp(&tl.m_ready[i & 1], ph(i)) && wait.warp(&tl.x_full[i & 1], ph(i)))) break;
        tc::fence_after_sync();
        if (elected()) {   // Y1(i) = M X, the smaller part of M first (all warps have read Y1(i - 1))
          const uint64_t dx = dX + ((i & 1) * kTileBytes >> 4);
#pragma unroll 1
          for (int k = 0; k < 2 * (kQ / 16); ++k)
            mma_bf16_ts(tmem + kTY1, tmem + (k < 8 ? kTM2 : kTM) + 8 * (k & 7), mn_step(dx, k & 7), kIdY, k > 0);
          tc::commit(&tl.y_full[i & 1]);
        }
        __syncwarp();
      }
      const int e = i + 1;
      if (e == n) break;
      if (!(ok = wait.warp(&tl.b_full[e & 1], ph(e)))) break;
      const uint32_t bt = (e & 1) * NB * kTileBytes >> 4;
      if (OUT) {
        if (!(ok = wait.warp(&tl.c_full, unsigned(e) & 1u))) break;   // G(e) = C B^T (all warps have read G(e - 1))
        products(tmem + kTG, dC, 32, kTileBytes, NB, dBk + bt, 32, kTileBytes, NB, kIdG, &tl.g_full);
        if (!(ok = wait.warp(&tl.sh_ready[e & 1], ph(e)))) break;     // Y2(e) = C S^T: both parts of S
        products(tmem + kTY2 + 64 * (e & 1), dC, 32, kTileBytes, NB, dSH, 2048, 8192, 2 * NB, kIdY, &tl.y2_done);
      }
      if (!(ok = wait.warp(&tl.xs_ready[e & 1], ph(e)))) break;       // U(e) = B^T (w X), transposed state [N][64]: three parts
      products(tmem + kTU + (OUT ? 0 : 64 * (e & 1)), dBm + bt, 2048, 8192, 2, dXS + (e % SM::kXSets * 3 * kTileBytes >> 4), 2048, 8192, 6, kIdU,
               &tl.u_full[e & 1]);
    }
  } else {
    // ------------------------------------------------------------ the working warps
    const int w = warp & 3, r = warp >> 2, row = 32 * w + lane;
    const uint32_t lanes = tmem + (uint32_t(32 * w) << 16);
    const float D = p.Dw ? __ldg(p.Dw + h) : 0.f;
    // state column of this thread: all 128 lanes hold one, or (N = 64, M = 64 accumulator) the first 16 of each warp
    const bool mine = N == 128 || lane < 16;
    const int col = N == 128 ? row : 16 * w + (lane & 15);
    const int64_t at = int64_t(16 * r) * N + col;   // state rows 16 r .. of this column
    float S[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) S[q] = mine && !op.local && op.init ? __ldg(op.init + unit * 64 * N + at + q * N) : 0.f;
    if (mine && !op.local)   // what the segments before this one leave
      for (int64_t j = 0; j < seg; ++j) {
        const float f = __ldg(op.seg_decay + unit * op.segments + j);
        const float* u = op.seg_state + (unit * op.segments + j) * 64 * N + at;
#pragma unroll
        for (int q = 0; q < 16; ++q) S[q] = fmaf(f, S[q], __ldg(u + q * N));
      }
    if (OUT && r > w) {   // the blocks of M behind the diagonal stay zero
      const uint32_t zero[8] = {};
#pragma unroll
      for (int k = 0; k < 16; k += 8) {
        st8(lanes + kTM + 16 * r + k, zero);
        st8(lanes + kTM2 + 16 * r + k, zero);
      }
      tc::wait_st();
    }
    auto put = [&](float* dst, int q0 = 0, int q1 = 16) {   // [64][N]
      if (mine && range_ok(at, 15 * N + 1, 64 * N, p.status))
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (q >= q0 && q < q1) dst[at + q * N] = S[q];
    };
    // The state that enters chunk e, four of a thread's sixteen rows at a time: its stores are spread over the phases, as
    // they would fill the store queue at once (256 of 128 bytes per CTA).
    auto put_part = [&](int e, int k) {
      if (op.states && range_ok(chunk(e), 1, op.stride, p.status)) put(op.states + (unit * op.stride + chunk(e)) * 64 * N, 4 * k, 4 * k + 4);
    };
    // The weighted x of chunk e in three bf16 parts (its buffer has been read).  The smallest part first: the tensor core
    // cuts its sums off below their leading bits, which the large part then meets in its own eight steps only.
    auto weigh = [&](int e) {
      if (!wait.warp(&tl.dec_full[e % 3], ph3(e)) || !wait.warp(&tl.x_full[e & 1], ph(e))) return false;
      const Decays& nd = tl.dec[e % 3];
      const float wt = REV ? nd.in[row] : nd.d[row] * nd.out[row];
      uint8_t* xs = sm + SM::kXS + e % SM::kXSets * 3 * kTileBytes;
#pragma unroll 1
      for (int j = 2 * r; j < 2 * r + 2; ++j) {
        const uint32_t o = swz(row, j);
        const uint4 v = *reinterpret_cast<const uint4*>(sm + SM::kX + (e & 1) * kTileBytes + o);
        const uint32_t xi[4] = {v.x, v.y, v.z, v.w};
        uint32_t part[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 f = mul2(stc::unpack(xi[k]), make_float2(wt, wt));
          part[0][k] = split(f);
          part[1][k] = split(f);
          part[2][k] = pack(f.x, f.y);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<uint4*>(xs + (2 - q) * kTileBytes + o) = make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]);
      }
      tc::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) {
        arrive(&tl.xs_ready[e & 1]);
        if (!OUT) arrive(&tl.x_free[e & 1]);
      }
      return true;
    };
    float total = 1.f;
    bool ok = SM::kXSets == 1 || weigh(0);
#pragma unroll 1
    for (int i = -1; ok && i < n; ++i) {
      const Decays& dec = tl.dec[(i + 3) % 3];
      float in = 0.f;
      if (i >= 0) {
        in = dec.in[row];
        if (OUT) {
          // ---- M(i)
          if (!(ok = wait.warp(&tl.g_full, unsigned(i) & 1u))) break;
          tc::fence_after_sync();
          const bool resets = dec.resets != 0;
          const int start = dec.start[row];
          const float hi = dec.hi[row], lo = dec.lo[row];
          const float rt = ex2(dec.rel[row]);
          const float* back = dec.far + 16 * w * (w - 1);
          const bool grow = dec.growing != 0;
#pragma unroll 1
          for (int c = 16 * r; c < 32 * w + 32; c += 64) {
            float v[16];
            ld16(lanes + kTG + c, v);
            tc::wait_ld();
            if (c >= 32 * w) {   // the diagonal block
              float own = 0.f;   // M_tt stays out of the product: the largest term where little is remembered
#pragma unroll
              for (int s = 0; s < 16; s += 4) {
                const float4 h4 = *reinterpret_cast<const float4*>(dec.hi + c + s), l4 = *reinterpret_cast<const float4*>(dec.lo + c + s);
                const float4 d4 = *reinterpret_cast<const float4*>(dec.d + c + s);
                const float hs[4] = {h4.x, h4.y, h4.z, h4.w}, ls[4] = {l4.x, l4.y, l4.z, l4.w}, ds[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float gd = v[s + e] * ds[e];
                  own = c + s + e <= row ? gd : own;   // the last one is M_tt, if it is in these columns
                  const float x = (hi - hs[e]) + (lo - ls[e]);   // (the exponent is masked, not the result: no branch)
                  v[s + e] = gd * ex2(c + s + e < row ? x : -1e30f);
                }
              }
              if ((row & 127) >> 4 == c >> 4) tl.own[i & 1][row] = own;
            } else if (!grow) {
#pragma unroll
              for (int s = 0; s < 16; s += 4) {
                const float4 f4 = *reinterpret_cast<const float4*>(back + c + s);
                v[s] *= f4.x * rt; v[s + 1] *= f4.y * rt; v[s + 2] *= f4.z * rt; v[s + 3] *= f4.w * rt;
              }
            } else {   // decays above one: the two factors could overflow where their product does not
#pragma unroll 1
              for (int s = 0; s < 16; ++s) {
                const float m = dec.d[c + s] * decay_between(hi, lo, dec.hi[c + s], dec.lo[c + s]);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= e == s ? m : 1.f;
              }
            }
            if (resets)
#pragma unroll
              for (int s = 0; s < 16; ++s) v[s] = c + s >= start ? v[s] : 0.f;
            uint32_t m[8], m2[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float2 f = make_float2(v[2 * e], v[2 * e + 1]);
              m[e] = split(f);
              m2[e] = pack(f.x, f.y);
            }
            st8(lanes + kTM + (c >> 1), m);
            st8(lanes + kTM2 + (c >> 1), m2);
          }
          tc::wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) arrive(&tl.m_ready[i & 1]);
          put_part(i, 3);
        }
        if (SM::kXSets == 2 && i + 1 < n && !(ok = weigh(i + 1))) break;   // (U(i - 1) has read that buffer)
        // ---- S(i + 1) = e^{Lambda_end} S(i) + U(i)
        const float gam = dec.total;
        total *= gam;
        __syncwarp();
        if (lane == 0) arrive(&tl.dec_free[i % 3]);
        if (!(ok = wait.warp(&tl.u_full[i & 1], ph(i)))) break;
        tc::fence_after_sync();
        float u[16];
        ld16(lanes + kTU + (OUT ? 0 : 64 * (i & 1)) + 16 * r, u);
        tc::wait_ld();
        tc::fence_before_sync();
#pragma unroll
        for (int q = 0; q < 16; ++q) S[q] = fmaf(gam, S[q], u[q]);
      }
      const int e = i + 1;
      if (e < n) {
        if (OUT) {   // the bf16 parts of the state that enters chunk e
          if (i >= 0 && !(ok = wait.warp(&tl.y2_done, unsigned(i) & 1u))) break;
          if (mine)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float2 v = make_float2(S[8 * j + 2 * k], S[8 * j + 2 * k + 1]);
                hi[k] = split(v);
                lo[k] = pack(v.x, v.y);
              }
              uint8_t* sh = sm + SM::kSH + swz(col, 2 * r + j);
              *reinterpret_cast<uint4*>(sh + N * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(sh) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          tc::fence_smem_to_async();
          __syncwarp();
          if (lane == 0) arrive(&tl.sh_ready[e & 1]);
          put_part(e, 0);
        } else if (op.states && range_ok(chunk(e), 1, op.stride, p.status)) {
          put(op.states + (unit * op.stride + chunk(e)) * 64 * N);
        }
      }
      if (OUT && i >= 0) {
        // ---- Y(i) = Y1 + in Y2 + (D + M_tt) x
        if (!(ok = wait.warp(&tl.y_full[i & 1], ph(i)))) break;
        tc::fence_after_sync();
        const float dx = D + tl.own[i & 1][row];
        float y1[16], y2[16];
        ld16(lanes + kTY1 + 16 * r, y1);
        ld16(lanes + kTY2 + 64 * (i & 1) + 16 * r, y2);
        tc::wait_ld();
        tc::fence_before_sync();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint4* tile = reinterpret_cast<uint4*>(sm + SM::kX + (i & 1) * kTileBytes + swz(row, 2 * r + j));
          const uint4 xv = *tile;
          const uint32_t xi[4] = {xv.x, xv.y, xv.z, xv.w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int q = 8 * j + 2 * k;
            const float2 f = fma2(make_float2(in, in), make_float2(y2[q], y2[q + 1]), make_float2(y1[q], y1[q + 1]));
            const float2 y = fma2(make_float2(dx, dx), stc::unpack(xi[k]), f);
            o[k] = pack(y.x, y.y);
          }
          *tile = make_uint4(o[0], o[1], o[2], o[3]);
        }
        tc::fence_smem_to_async();
        __syncwarp();
        if (lane == 0) arrive(&tl.x_free[i & 1]);   // (to the loader: y is there)
      }
      // (U(i) has read its parts.  Behind Y(i), which frees a buffer of x for the loader two chunks ahead.)
      if (OUT && e < n) put_part(e, 1);
      if (SM::kXSets == 1 && e < n && !(ok = weigh(e))) break;
      if (OUT && e < n) put_part(e, 2);
    }
    if (ok) {
      if (op.local) {
        put(op.seg_state + (unit * op.segments + seg) * 64 * N);
        if (threadIdx.x == 0) op.seg_decay[unit * op.segments + seg] = total;
      } else if (seg == op.segments - 1) {
        if (op.last) put(op.last + unit * 64 * N);
        if (!REV && op.states) put(op.states + (unit * op.stride + nc) * 64 * N);
      }
    }
  }
  // ------------------------------------------------------------ end: nothing of this CTA may be in flight
  __syncwarp();
  if (lane == 0 && *reinterpret_cast<volatile int*>(&tl.dead)) {   // a wait was given up: loads and MMAs may be under way
    const unsigned long long t0 = global_ns();
    auto drain = [&](unsigned long long* bar, unsigned parity) {
      while (!mbar_try_wait(bar, parity) && global_ns() - t0 < kWaitLimitNs) {}
    };
    if (warp == 17) {
      for (int i = x_loads > 2 ? x_loads - 2 : 0; i < x_loads; ++i) drain(&tl.x_full[i & 1], ph(i));
      for (int i = b_loads > 2 ? b_loads - 2 : 0; i < b_loads; ++i) drain(&tl.b_full[i & 1], ph(i));
      if (c_loads) drain(&tl.c_full, unsigned(c_loads - 1) & 1u);
    } else if (warp == 16) {
      tc::commit(&tl.drained);
      drain(&tl.drained, 0);
    }
  }
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 16) tc::dealloc(tmem, 512);
}

template <int N, bool OUT, bool REV>
cudaError_t run(const SsmArgs& p, const TileMaps& tm, const ChunkOp& op, cudaStream_t s) {
  static_assert(Smem<N, OUT>::kBytes <= 232448, "shared memory of a CTA");
  auto* k = ssm_chunk_kernel<N, OUT, REV>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<N, OUT>::kBytes);
  if (e != cudaSuccess) return e;
  k<<<unsigned(p.B * p.H * op.segments), kThreads, Smem<N, OUT>::kBytes, s>>>(p, tm, op);
  return cudaGetLastError();
}
template <bool OUT, bool REV>
cudaError_t run_n(const SsmArgs& p, const TileMaps& tm, const ChunkOp& op, cudaStream_t s) {
  return p.N == 128 ? run<128, OUT, REV>(p, tm, op, s) : run<64, OUT, REV>(p, tm, op, s);
}

}  // namespace

// Runs that a row's chunks are cut into: with fewer rows of heads than SMs, as many as fill them, of at least 2 chunks.  A
// cut row is walked twice, first for the state that each run leaves (without the outputs' work), then from it on, so it
// takes three runs to gain.  B=1 H=32 N=128: T=1024 28 us against 34 whole, T=2048 38 against 58, T=4096 57 against 106.
int64_t ssm_segments(int64_t units, int64_t nc) {
  const int64_t fit = units > 0 ? 148 / units : 1, most = nc / 2, k = fit < most ? fit : most;
  return k >= 3 ? k : 1;
}
int64_t ssm_segment_floats(int64_t B, int64_t T, int64_t H, int N) {
  const int64_t k = ssm_segments(B * H, chunks_of(T));
  return k > 1 ? B * H * k * (64 * N + 1) : 0;
}

namespace {
template <bool OUT, bool REV>
cudaError_t walk(const SsmArgs& p, const TileMaps& tm, ChunkOp op, float* seg, cudaStream_t s) {
  const int64_t nc = chunks_of(p.T), k = seg ? ssm_segments(p.B * p.H, nc) : 1;
  op.per_segment = (nc + k - 1) / k;
  op.segments = (nc + op.per_segment - 1) / op.per_segment;
  if (op.segments > 1) {
    op.seg_state = seg;
    op.seg_decay = seg + p.B * p.H * op.segments * 64 * p.N;
    ChunkOp first = op;
    first.local = true;
    first.states = nullptr;
    first.last = nullptr;
    const cudaError_t e = run_n<false, REV>(p, tm, first, s);
    if (e != cudaSuccess) return e;
  }
  return run_n<OUT, REV>(p, tm, op, s);
}
}  // namespace

cudaError_t launch_ssm_chunk_fwd(const SsmArgs& p, const TileMaps& tm, cudaStream_t s) {
  const int64_t nc = chunks_of(p.T);
  ChunkOp op{};
  op.init = p.s0;
  op.states = p.ckpt;
  op.stride = nc + 1;
  op.last = p.s_out;
  return walk<true, false>(p, tm, op, p.ckpt ? p.ckpt + p.B * p.H * (nc + 1) * 64 * p.N : nullptr, s);
}

// The gradient of the state after each chunk into the backward's scratch, and of the initial state.
cudaError_t launch_ssm_chunk_dstate(const SsmArgs& p, const TileMaps& tm, float* dstate, float* seg, cudaStream_t s) {
  ChunkOp op{};
  op.init = p.dsT;
  op.states = dstate;
  op.stride = chunks_of(p.T);
  op.last = p.ds0;
  return walk<false, true>(p, tm, op, seg, s);
}

}  // namespace wkv7
