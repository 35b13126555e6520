// Tensor-core side of the chunked selective scan: swizzled tiles, their matrix descriptors, tensor maps, bounded
// waits, and the per-token decay factors of a chunk.  Beside tc05.cuh (allocation, fences, MMA issue).
//
// Tiles hold rows of 64 bf16 (128 bytes) in the 128-byte swizzle that TMA writes: 16-byte piece j of row r sits at
// r * 128 + ((j ^ (r & 7)) << 4), 8 rows make one 1024-byte atom.  A tile serves both ways round:
//   * rows = M or N, columns = K ("K-major"): 8-row groups 1024 bytes apart, one MMA's K = 16 is 32 bytes along the row;
//   * rows = K, columns = M or N ("MN-major"): one MMA's K = 16 is two 8-row groups, 2048 bytes along; columns beyond 64
//     are in the next tile.
#pragma once

#include "ssm.cuh"
#include "tc05.cuh"

namespace wkv7 {
namespace stc {

constexpr int kQ = kSsmChunk;                  // tokens of a chunk = rows of a token tile
constexpr int kTileBytes = kQ * 128;           // [128][64] bf16

__device__ __forceinline__ int swz(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t mn_block_bytes) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t((mn_block_bytes >> 4) & 0x3FFFu) << 16)   // start; distance of 64-column blocks
         | (uint64_t(1024 >> 4) << 32)                                                           // distance of 8-row groups
         | (uint64_t(1) << 46) | (uint64_t(2) << 61);                                            // version, 128-byte swizzle
}
// Operand `step` (K = 16 each) of an MN-major operand (K along the rows), from the descriptor of its start: the address sits
// in the low bits, in units of 16 bytes.
__device__ __forceinline__ uint64_t mn_step(uint64_t d, int step) { return d + ((step * 2048) >> 4); }

// D[tmem] (+)= A[tmem, bf16 pairs] * B[smem desc], kind::f16
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(0u)
      : "memory");
}

// 16 columns of 32 lanes: thread l of warp w reaches lane 32 (w % 4) + l.  While MMAs run, one such move holds up its
// quadrant for about 80 cycles whether it moves 8 columns or 32 (measured), so narrower ones cost the same.
__device__ __forceinline__ void ld16(uint32_t taddr, float (&v)[16]) { tc::ld_32x32b_x16(taddr, v); }
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
      "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// 2^x, 2^-22 relative; results below the normal range are zero
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^(hi + lo): the integer part goes into the exponent, so that only a fraction is rounded
__device__ __forceinline__ float ex2_pair(float hi, float lo) {
  const float n = fmaxf(rintf(hi), -200.f);
  return ex2((hi - n) + lo) * ex2(n);   // the second is exact (0 below 2^-126, inf above 2^127)
}

// ---- pairs of bf16 in a register
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
// v = hi + mid (+ lo): bf16 parts, 8 significant bits each.
__device__ __forceinline__ uint32_t split(float2& v) {
  const uint32_t h = pack(v.x, v.y);
  v = sub2(v, unpack(h));
  return h;
}

// ---- waits: bounded, and given up by everyone once one has run out.  A poll may suspend the thread for a millisecond
// (spinning warps take issue slots and instruction fetches from the working ones).
__device__ __forceinline__ bool try_wait_ms(unsigned long long* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
static __device__ __noinline__ bool wait_slow(unsigned long long* bar, unsigned parity, int* dead, int* status) {
  const unsigned long long t0 = global_ns();
  while (!try_wait_ms(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(dead)) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile int*>(dead) = 1;
      atomicOr(status, kStatusWaitTimeout);
      return false;
    }
  }
  return true;
}
struct Wait {
  int* dead;          // shared: set once a wait has run out
  int* status;        // the device status word
  __device__ __forceinline__ bool operator()(unsigned long long* bar, unsigned parity) const {   // one thread
    return try_wait_ms(bar, parity) || wait_slow(bar, parity, dead, status);
  }
  __device__ __forceinline__ bool warp(unsigned long long* bar, unsigned parity) const {         // all lanes, one answer
    return __all_sync(0xffffffffu, (*this)(bar, parity));
  }
};
__device__ __forceinline__ void arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ---- token tiles by TMA: {64, heads or groups, T, B}, box {64, 1, 128, 1}; tokens past T read as zeros
struct TileMaps {
  CUtensorMap x, b, c, dy, y;   // dy: backward; y, written: forward
};
// A tile back to global memory (rows past T are left out), and the wait until it has been read, or written.
__device__ __forceinline__ void tma_store_4d(const void* map, const void* src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(
                   reinterpret_cast<unsigned long long>(map)),
               "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---- decays of one chunk.  Lambda_t: sum of log2 decays from the chunk's start up to and with token t, summed in fp64
// and kept as a pair of floats; r_t: a reset (or a decay of zero) at or before t in the chunk.  Everything is zero behind the row's end.
struct alignas(16) Decays {   // (its rows are read four floats at a time, in arrays of these)
  float hi[kQ], lo[kQ];   // Lambda_t
  float d[kQ];            // step
  float in[kQ];           // 2^Lambda_t, 0 where r_t: what is left at t of the state that enters the chunk
  float out[kQ];          // 2^(Lambda_end - Lambda_t), 0 if a reset follows: what is left of token t at the chunk's end
  float rel[kQ];          // Lambda_t - Lambda at the start of t's block of 32
  int start[kQ];          // first token of t's segment in the chunk
  // Off the diagonal 32 x 32 blocks the decay is a product of two factors, both relative to the row block w:
  float far[192];         // forward: d_s 2^(Lambda before block w - Lambda_s) for the tokens s before block w = 1, 2, 3;
                          // backward: 2^(Lambda_t - Lambda at the end of block w) for the tokens t after block w = 0, 1, 2
  float total;            // 2^Lambda_end, 0 with a reset
  int resets;             // any reset in the chunk
  int growing;            // any decay above one
};

// 2^(Lambda_a - Lambda_b) of two tokens (or of the chunk's start: zero).
__device__ __forceinline__ float decay_between(float ahi, float alo, float bhi, float blo) {
  return ex2_pair(ahi - bhi, alo - blo);
}

// The raw steps and resets of tokens 4 lane + k of chunk c (loads only, so that they can be under way early).
struct RawSteps {
  unsigned short v[4];   // bf16 as loaded: a conversion here would wait for the load
  uint8_t rst[4];
  __device__ __forceinline__ void load(const SsmArgs& p, int64_t b, int64_t h, int64_t c) {
    const int64_t t0 = c * kQ + 4 * (threadIdx.x & 31), bt = b * p.T + t0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool ok = t0 + k < p.T && rows_ok((bt + k) * p.dt_ld + h, 1, p.B * p.T, p.dt_ld, p.H, p.status);
      v[k] = ok ? static_cast<const unsigned short*>(p.dt)[(bt + k) * p.dt_ld + h] : 0;
      rst[k] = ok && p.reset ? p.reset[bt + k] : 0;
    }
  }
};

// Who reads the decays: the forward, the backward, or a pass over the states alone (forward or reversed).
enum Reader { kForward, kBackward, kStates, kReversed };

// One warp fills `o` for chunk c, four tokens per lane: their chains overlap, and one scan over the lanes serves all 128
// tokens (32 tokens at a time took 7000 cycles, which bounded the reversed state pass: 194 us for B=8 T=4096 H=32 N=128,
// now 140).
template <int READER>
__device__ __forceinline__ void chunk_decays(const SsmArgs& p, float A, float bias, int64_t c, const RawSteps& raw, Decays& o) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = c * kQ + 4 * lane;
  const double A2 = double(A) * 1.4426950408889634074;
  float d[4];
  double l[4], sum = 0.0;
  int st[4], last = -1;
  bool grow = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float v = __uint_as_float(unsigned(raw.v[k]) << 16) + bias;
    d[k] = t0 + k < p.T ? (p.softplus ? softplus_of(v) : v) : 0.f;
    // A step that leaves nothing is a reset and not a term of the sum, which would lose the decays behind it.
    const bool cut = cuts(d[k], A);
    const double x = cut ? 0.0 : double(d[k]) * A2;
    grow |= x > 0.0;
    sum += x;
    l[k] = sum;
    if (raw.rst[k] || cut) last = 4 * lane + k;
    st[k] = last;
  }
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const double u = __shfl_up_sync(0xffffffffu, sum, s);
    const int m = __shfl_up_sync(0xffffffffu, last, s);
    if (lane >= s) {
      sum += u;
      last = m > last ? m : last;
    }
  }
  double ex = __shfl_up_sync(0xffffffffu, sum, 1);   // Lambda and the last reset before this lane's tokens
  int before = __shfl_up_sync(0xffffffffu, last, 1);
  if (lane == 0) {
    ex = 0.0;
    before = -1;
  }
  const double block = __shfl_sync(0xffffffffu, ex, lane & 24), end = __shfl_sync(0xffffffffu, sum, 31);
  last = __shfl_sync(0xffffffffu, last, 31);
  const float ehi = float(end), elo = float(end - double(ehi));
  float hi[4], lo[4], rel[4], in[4], out[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    l[k] += ex;
    hi[k] = float(l[k]);
    lo[k] = float(l[k] - double(hi[k]));
    rel[k] = float(l[k] - block);
    st[k] = st[k] < 0 ? before : st[k];
    in[k] = st[k] < 0 ? ex2_pair(hi[k], lo[k]) : 0.f;
    if (READER != kReversed) out[k] = 4 * lane + k >= last ? decay_between(ehi, elo, hi[k], lo[k]) : 0.f;
    st[k] = st[k] < 0 ? 0 : st[k];
  }
  auto put = [&](float* dst, const float (&v)[4]) { *reinterpret_cast<float4*>(dst + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]); };
  if (READER != kReversed) {
    put(o.d, d);
    put(o.out, out);
  }
  if (READER != kStates) put(o.in, in);
  if (READER == kForward || READER == kBackward) {
    put(o.hi, hi);
    put(o.lo, lo);
    put(o.rel, rel);
    *reinterpret_cast<int4*>(o.start + 4 * lane) = make_int4(st[0], st[1], st[2], st[3]);
#pragma unroll
    for (int j = 1; j < 4; ++j) {   // relative to token 32 j - 1: the start of row block j, the end of row block j - 1
      const float mh = __shfl_sync(0xffffffffu, hi[3], 8 * j - 1), ml = __shfl_sync(0xffffffffu, lo[3], 8 * j - 1);
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = READER == kForward ? d[k] * decay_between(mh, ml, hi[k], lo[k]) : decay_between(hi[k], lo[k], mh, ml);
      if (READER == kForward) {
        if (lane < 8 * j) put(o.far + 16 * j * (j - 1), v);
      } else if (lane >= 8 * j) {
        put(o.far + (j == 1 ? 0 : j == 2 ? 96 : 160) - 32 * j, v);
      }
    }
  }
  const unsigned any_grow = __ballot_sync(0xffffffffu, grow);
  if (lane == 0) {
    o.total = last < 0 ? ex2_pair(ehi, elo) : 0.f;
    o.resets = last >= 0;
    o.growing = any_grow != 0;
  }
}

}  // namespace stc
}  // namespace wkv7
