// C ABI of the state-space layer (include/wkv7.h, "state-space layer"): argument checks and dispatch for the short
// convolution, the selective scan and the RMS norm.  Nothing here allocates memory or keeps state between calls.
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "ssm_chunk.h"
#include "ssm_tc.cuh"
#include "state_space.h"
#include "wkv7.h"

namespace {

constexpr int64_t kMaxGrid = 2147483647;

bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0 || (a != 0 && b > INT64_MAX / a)) return false;
  *out = a * b;
  return true;
}
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int64_t elt(const wkv7_desc_t* d) { return d->dtype == WKV7_F32 ? 4 : 2; }

// Flags, dtype, sizes; `rows` = B * T.
wkv7_status_t check_common(const wkv7_desc_t* d, int64_t* rows) {
  if (!d) return WKV7_ERR_NULL;
  if ((d->flags & ~WKV7_FLAG_CHECK_FINITE) != 0u) return WKV7_ERR_UNSUPPORTED;
  if (d->dtype != WKV7_F32 && d->dtype != WKV7_BF16 && d->dtype != WKV7_F16) return WKV7_ERR_DTYPE;
  if (d->B < 0 || d->T < 0 || d->H < 0 || d->B > kMaxGrid || !mul_ok(d->B, d->T, rows)) return WKV7_ERR_SHAPE;
  return WKV7_OK;
}

// A token stride: 0 means dense; at least the row's size; whole 16-byte units where `vec`.
wkv7_status_t check_ld(int64_t ld, int64_t width, int64_t rows, int64_t es, bool vec, int64_t* out) {
  *out = ld == 0 ? width : ld;
  int64_t n;
  if (*out < width || !mul_ok(rows, *out, &n) || !mul_ok(n, es, &n)) return WKV7_ERR_SHAPE;
  return vec && rows > 1 && (*out * es) % 16 != 0 ? WKV7_ERR_ALIGN : WKV7_OK;
}

wkv7_status_t check_ptrs(bool need, std::initializer_list<const void*> ptrs, uintptr_t align = 16) {
  for (const void* p : ptrs) {
    if (!p) {
      if (need) return WKV7_ERR_NULL;
      continue;
    }
    if (!aligned(p, align)) return WKV7_ERR_ALIGN;
  }
  return WKV7_OK;
}

struct Output {
  const void* ptr;
  int64_t n;
  int dtype;
};
wkv7_status_t finish(const wkv7_desc_t* d, cudaError_t launched, std::initializer_list<Output> outs, int* status, cudaStream_t s) {
  if (launched != cudaSuccess) return WKV7_ERR_CUDA;
  if (!(d->flags & WKV7_FLAG_CHECK_FINITE)) return WKV7_OK;
  for (const Output& o : outs)
    if (wkv7::launch_finite_scan(o.ptr, o.n, o.dtype, status, s) != cudaSuccess) return WKV7_ERR_CUDA;
  return WKV7_OK;
}

// The status word, for the kernels that write it only in the debug build: not looked up where nothing would use it.
bool status_word(const wkv7_desc_t* d, int** out) {
  *out = nullptr;
  return (!wkv7::kDebugChecks && d->flags == 0) || wkv7::device_status_ptr(out) == cudaSuccess;
}

bool zero(void* p, int64_t bytes, cudaStream_t s) {
  return !p || bytes == 0 || cudaMemsetAsync(p, 0, size_t(bytes), s) == cudaSuccess;
}
// dst = src, or zeros where src is NULL.
bool copy(void* dst, const void* src, int64_t bytes, cudaStream_t s) {
  if (!dst || bytes == 0 || dst == src) return true;
  if (!src) return zero(dst, bytes, s);
  return cudaMemcpyAsync(dst, src, size_t(bytes), cudaMemcpyDeviceToDevice, s) == cudaSuccess;
}

#define TRY(expr)                          \
  do {                                     \
    const wkv7_status_t st_ = (expr);      \
    if (st_ != WKV7_OK) return st_;        \
  } while (0)

// ------------------------------------------------------------------ convolution
wkv7_status_t check_conv(const wkv7_desc_t* d, const wkv7_conv_t* cv, wkv7::ConvArgs* a, bool sizes_only = false) {
  int64_t rows, n;
  TRY(check_common(d, &rows));
  if (!cv) return WKV7_ERR_NULL;
  if (cv->W < 2 || cv->W > 4 || cv->D % 8 != 0) return WKV7_ERR_UNSUPPORTED;
  if (cv->D < 0 || !mul_ok(d->B, 3 * 4, &n) || cv->D > (int64_t(1) << 31) || !mul_ok(n, cv->D, &n)) return WKV7_ERR_SHAPE;
  if (!mul_ok(rows, cv->D, &n) || !mul_ok(n, 4 * (cv->W + 1), &n)) return WKV7_ERR_SHAPE;
  *a = wkv7::ConvArgs{};
  TRY(check_ld(cv->x_ld, cv->D, rows, elt(d), true, &a->x_ld));
  a->B = d->B; a->T = d->T; a->D = cv->D; a->W = cv->W;
  a->silu = cv->silu != 0;
  a->weight = cv->weight; a->bias = cv->bias;
  if (sizes_only) return WKV7_OK;
  TRY(check_ptrs(cv->D > 0 && d->B > 0, {cv->weight}));
  return check_ptrs(false, {cv->bias});
}

// ------------------------------------------------------------------ scan
wkv7_status_t check_ssm(const wkv7_desc_t* d, const wkv7_ssm_t* sp, wkv7::SsmArgs* a, bool sizes_only = false) {
  int64_t rows, n;
  TRY(check_common(d, &rows));
  if (!sp) return WKV7_ERR_NULL;
  if (d->N != 64 && d->N != 128) return WKV7_ERR_UNSUPPORTED;
  if (d->algo != WKV7_ALGO_AUTO && d->algo != WKV7_ALGO_SCAN && d->algo != WKV7_ALGO_CHUNKED) return WKV7_ERR_UNSUPPORTED;
  if (d->algo == WKV7_ALGO_CHUNKED && d->dtype != WKV7_BF16) return WKV7_ERR_UNSUPPORTED;
  if (sp->G < 1 || d->H % sp->G != 0) return WKV7_ERR_UNSUPPORTED;
  // every byte count of inputs, states, checkpoints and scratch, and every grid, fits
  const int64_t nc = (d->T + wkv7::kSsmChunk - 1) / wkv7::kSsmChunk;
  if (!mul_ok(d->B, d->H, &n) || n > kMaxGrid || !mul_ok(n, nc + 2, &n) || n > kMaxGrid || !mul_ok(n, 128 * 128 * 32, &n))
    return WKV7_ERR_SHAPE;
  if (!mul_ok(rows, sp->G, &n) || n > kMaxGrid) return WKV7_ERR_SHAPE;
  *a = wkv7::SsmArgs{};
  const int64_t es = elt(d);
  if (!mul_ok(d->H, wkv7::kHeadP, &n)) return WKV7_ERR_SHAPE;
  TRY(check_ld(sp->x_ld, n, rows, es, true, &a->x_ld));
  TRY(check_ld(sp->dt_ld, d->H, rows, es, false, &a->dt_ld));
  if (!mul_ok(sp->G, d->N, &n)) return WKV7_ERR_SHAPE;
  TRY(check_ld(sp->b_ld, n, rows, es, true, &a->b_ld));
  TRY(check_ld(sp->c_ld, n, rows, es, true, &a->c_ld));
  a->B = d->B; a->T = d->T; a->H = d->H; a->G = sp->G; a->N = d->N;
  a->A = sp->A; a->Dw = sp->D; a->dt_bias = sp->dt_bias;
  a->softplus = sp->softplus != 0;
  if (sizes_only) return WKV7_OK;
  if (d->B > 0 && d->H > 0 && !sp->A) return WKV7_ERR_NULL;
  return check_ptrs(false, {sp->A, sp->D, sp->dt_bias}, 4);
}

// AUTO: the tensor cores for bf16, but not in the forward of a few tokens, which would fill a 128-token chunk with zeros.
// Forward, us, token order against chunks, B=8 H=32 N=64: T=8 7.8 / 20, T=16 10 / 20, T=32 16 / 20, T=64 27 / 20; N=128: 11 / 22,
// 15 / 22, 23 / 22, 39 / 22; B=1 N=64: T=16 7.4 / 10.5, T=32 11.3 / 10.4.  Backward, B=8 H=32 N=64: T=1 52 / 46, T=128 249 / 53.
bool chunked(const wkv7_desc_t* d, bool forward) {
  return d->dtype == WKV7_BF16 && d->algo != WKV7_ALGO_SCAN && !(forward && d->algo == WKV7_ALGO_AUTO && d->T <= 16);
}

// ------------------------------------------------------------------ norm
wkv7_status_t check_rms(const wkv7_desc_t* d, const wkv7_rms_t* rn, wkv7::RmsArgs* a, bool sizes_only = false) {
  int64_t rows, n;
  TRY(check_common(d, &rows));
  if (!rn) return WKV7_ERR_NULL;
  if (rn->D < 0) return WKV7_ERR_SHAPE;
  if (rn->groups < 1 || rn->D % rn->groups != 0 || (rn->D / rn->groups) % 8 != 0 || rn->D / rn->groups > 16384) return WKV7_ERR_UNSUPPORTED;
  if (!(rn->eps > 0.f) || !(rn->eps < 1e30f)) return WKV7_ERR_UNSUPPORTED;   // also refuses NaN
  if (rn->quant_block != 0 && rn->quant_block != 128 && rn->quant_block != -1) return WKV7_ERR_UNSUPPORTED;
  if (rn->quant_block == 128 && (rn->D / rn->groups) % 128 != 0) return WKV7_ERR_UNSUPPORTED;
  if (!mul_ok(rows, rn->D, &n) || !mul_ok(n, 4, &n) || rn->groups > (int64_t(1) << 24)) return WKV7_ERR_SHAPE;
  *a = wkv7::RmsArgs{};
  a->rows = rows; a->D = rn->D; a->groups = rn->groups; a->weight = rn->weight; a->eps = rn->eps;
  a->gate = rn->gate != 0;
  a->quant_block = rn->quant_block;
  return sizes_only ? WKV7_OK : check_ptrs(rows > 0 && rn->D > 0, {rn->weight});
}

}  // namespace

extern "C" {

wkv7_status_t wkv7_conv_forward(const wkv7_desc_t* d, const wkv7_conv_t* cv, const void* x, const void* s0,
                                const uint8_t* reset, void* y, void* s_out, void* stream) {
  wkv7::ConvArgs a;
  TRY(check_conv(d, cv, &a));
  const int64_t n = d->B * d->T * cv->D, st = d->B * (cv->W - 1) * cv->D;
  TRY(check_ptrs(n > 0, {x, y}));
  TRY(check_ptrs(false, {s0, s_out}));
  if (s_out && s_out == s0 && st > 0) return WKV7_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (st == 0) return WKV7_OK;
  if (n == 0) return copy(s_out, s0, st * elt(d), s) ? WKV7_OK : WKV7_ERR_CUDA;
  if (!status_word(d, &a.status)) return WKV7_ERR_CUDA;
  a.x = x; a.s0 = s0; a.reset = reset; a.y = y; a.s_out = s_out;
  return finish(d, wkv7::launch_conv_fwd(a, d->dtype, s), {{y, n, d->dtype}, {s_out, st, d->dtype}}, a.status, s);
}

size_t wkv7_conv_scratch_bytes(const wkv7_desc_t* d, const wkv7_conv_t* cv) {
  wkv7::ConvArgs a;
  if (check_conv(d, cv, &a, true) != WKV7_OK) return 0;
  return size_t(wkv7::conv_scratch_floats(d->B, d->T, cv->D, cv->W)) * 4;
}

wkv7_status_t wkv7_conv_backward(const wkv7_desc_t* d, const wkv7_conv_t* cv, const void* x, const void* s0,
                                 const uint8_t* reset, const void* dy, const void* dsT, void* dx, float* dweight,
                                 float* dbias, void* ds0, void* scratch, void* stream) {
  wkv7::ConvArgs a;
  TRY(check_conv(d, cv, &a));
  const int64_t n = d->B * d->T * cv->D, st = d->B * (cv->W - 1) * cv->D;
  TRY(check_ptrs(n > 0, {x, dy, dx}));
  TRY(check_ptrs(false, {s0, dsT, ds0, scratch, dweight, dbias}));
  const bool want = dweight || dbias;
  if (n > 0 && want && !scratch) return WKV7_ERR_WORKSPACE;
  if (n > 0 && ds0 && ds0 == dsT) return WKV7_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    const bool ok = zero(dweight, cv->D * cv->W * 4, s) && zero(dbias, cv->D * 4, s) && copy(ds0, dsT, st * elt(d), s);
    return ok ? WKV7_OK : WKV7_ERR_CUDA;
  }
  if (!status_word(d, &a.status)) return WKV7_ERR_CUDA;
  a.x = x; a.s0 = s0; a.reset = reset; a.dy = dy; a.dsT = dsT; a.dx = dx; a.ds0 = ds0;
  a.dweight = dweight; a.dbias = dbias;
  a.scratch = want ? static_cast<float*>(scratch) : nullptr;
  return finish(d, wkv7::launch_conv_bwd(a, d->dtype, s),
                {{dx, n, d->dtype}, {ds0, st, d->dtype}, {dweight, cv->D * cv->W, WKV7_F32}, {dbias, cv->D, WKV7_F32}}, a.status, s);
}

wkv7_status_t wkv7_conv_step(const wkv7_desc_t* d, const wkv7_conv_t* cv, const void* x, void* state,
                             const uint8_t* active, void* y, void* stream) {
  wkv7::ConvArgs a;
  TRY(check_conv(d, cv, &a));
  if (d->T != 1) return WKV7_ERR_UNSUPPORTED;
  const int64_t n = d->B * cv->D;
  TRY(check_ptrs(n > 0, {x, state, y}));
  if (n == 0) return WKV7_OK;
  if (!status_word(d, &a.status)) return WKV7_ERR_CUDA;
  a.x = x; a.state = state; a.active = active; a.y = y;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(d, wkv7::launch_conv_step(a, d->dtype, s), {{y, n, d->dtype}, {state, n * (cv->W - 1), d->dtype}}, a.status, s);
}

// The workspace: nc + 1 states per (b, h), which are all that the backward reads, then the segments of the forward's form.
size_t wkv7_ssm_workspace_bytes(const wkv7_desc_t* d, const wkv7_ssm_t* sp) {
  wkv7::SsmArgs a;
  if (check_ssm(d, sp, &a, true) != WKV7_OK || d->T == 0) return 0;
  const int64_t nc = (d->T + wkv7::kSsmChunk - 1) / wkv7::kSsmChunk;
  return size_t(d->B * d->H * (nc + 1) * wkv7::kHeadP * d->N +
                (chunked(d, true) ? wkv7::ssm_segment_floats(d->B, d->T, d->H, d->N) : wkv7::ssm_run_floats(d->B, d->T, d->H, d->N))) * 4;
}

wkv7_status_t wkv7_ssm_forward(const wkv7_desc_t* d, const wkv7_ssm_t* sp, const void* x, const void* dt, const void* b,
                               const void* c, const float* s0, const uint8_t* reset, void* y, float* s_out,
                               void* workspace, void* stream) {
  wkv7::SsmArgs a;
  TRY(check_ssm(d, sp, &a));
  const int64_t units = d->B * d->H, n = units * d->T * wkv7::kHeadP, st = units * wkv7::kHeadP * d->N;
  TRY(check_ptrs(n > 0, {x, b, c, y}));
  TRY(check_ptrs(n > 0, {dt}, elt(d)));
  TRY(check_ptrs(false, {s0, s_out, workspace}));
  if (n > 0 && s_out && s_out == s0) return WKV7_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (units == 0) return WKV7_OK;
  if (d->T == 0) return copy(s_out, s0, st * 4, s) ? WKV7_OK : WKV7_ERR_CUDA;
  if (wkv7::device_status_ptr(&a.status) != cudaSuccess) return WKV7_ERR_CUDA;
  a.x = x; a.dt = dt; a.b = b; a.c = c; a.s0 = s0; a.reset = reset; a.y = y; a.s_out = s_out;
  a.ckpt = static_cast<float*>(workspace);
  cudaError_t e;
  if (chunked(d, true)) {
    wkv7::stc::TileMaps tm;
    if (!wkv7::encode_ssm_maps(a, false, &tm)) return WKV7_ERR_CUDA;
    e = wkv7::launch_ssm_chunk_fwd(a, tm, s);
  } else {
    e = wkv7::launch_ssm_scan_fwd(a, d->dtype, s);
  }
  return finish(d, e, {{y, n, d->dtype}, {s_out, st, WKV7_F32}}, a.status, s);
}

size_t wkv7_ssm_scratch_bytes(const wkv7_desc_t* d, const wkv7_ssm_t* sp) {
  wkv7::SsmArgs a;
  if (check_ssm(d, sp, &a, true) != WKV7_OK || d->T == 0) return 0;
  return size_t(wkv7::ssm_scratch(d->B, d->T, d->H, sp->G, d->N, chunked(d, false)).total) * 4;
}

wkv7_status_t wkv7_ssm_backward(const wkv7_desc_t* d, const wkv7_ssm_t* sp, const void* x, const void* dt, const void* b,
                                const void* c, const float* s0, const uint8_t* reset, const void* dy, const float* dsT,
                                const void* workspace, void* dx, void* ddt, void* db, void* dc, float* dA, float* dD,
                                float* ddt_bias, float* ds0, void* scratch, void* stream) {
  wkv7::SsmArgs a;
  TRY(check_ssm(d, sp, &a));
  const int64_t units = d->B * d->H, n = units * d->T * wkv7::kHeadP, st = units * wkv7::kHeadP * d->N;
  const int64_t nb = d->B * d->T * sp->G * d->N;
  TRY(check_ptrs(n > 0, {x, b, c, dy, dx, ddt, db, dc}));
  TRY(check_ptrs(n > 0, {dt}, elt(d)));
  TRY(check_ptrs(false, {s0, dsT, ds0, workspace, scratch, dA, dD, ddt_bias}));
  if (n > 0 && (!scratch || (!workspace && chunked(d, false)))) return WKV7_ERR_WORKSPACE;   // token order walks from s0 again
  if (n > 0 && ds0 && ds0 == dsT) return WKV7_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {   // no tokens: the parameters have no gradient, the state's passes through
    const bool ok = zero(dA, d->H * 4, s) && zero(dD, d->H * 4, s) && zero(ddt_bias, d->H * 4, s) && copy(ds0, dsT, st * 4, s);
    return ok ? WKV7_OK : WKV7_ERR_CUDA;
  }
  if (wkv7::device_status_ptr(&a.status) != cudaSuccess) return WKV7_ERR_CUDA;
  a.x = x; a.dt = dt; a.b = b; a.c = c; a.s0 = s0; a.reset = reset; a.dy = dy; a.dsT = dsT;
  a.ckpt = static_cast<float*>(const_cast<void*>(workspace));
  a.dx = dx; a.ddt = ddt; a.db = db; a.dc = dc; a.dA = dA; a.dD = dD; a.ddt_bias = ddt_bias; a.ds0 = ds0;
  a.scratch = static_cast<float*>(scratch);
  cudaError_t e;
  if (chunked(d, false)) {
    wkv7::stc::TileMaps tm;
    if (!wkv7::encode_ssm_maps(a, true, &tm)) return WKV7_ERR_CUDA;
    e = wkv7::launch_ssm_chunk_bwd(a, tm, s);
  } else {
    e = wkv7::launch_ssm_scan_bwd(a, d->dtype, s);
  }
  if (e == cudaSuccess) e = wkv7::launch_ssm_decay(a, d->dtype, chunked(d, false), s);
  return finish(d, e,
                {{dx, n, d->dtype}, {ddt, units * d->T, d->dtype}, {db, nb, d->dtype}, {dc, nb, d->dtype}, {dA, d->H, WKV7_F32},
                 {dD, d->H, WKV7_F32}, {ddt_bias, d->H, WKV7_F32}, {ds0, st, WKV7_F32}},
                a.status, s);
}

wkv7_status_t wkv7_ssm_step(const wkv7_desc_t* d, const wkv7_ssm_t* sp, const void* x, const void* dt, const void* b,
                            const void* c, float* state, const uint8_t* active, void* y, void* stream) {
  wkv7::SsmArgs a;
  TRY(check_ssm(d, sp, &a));
  if (d->T != 1) return WKV7_ERR_UNSUPPORTED;
  const int64_t units = d->B * d->H, n = units * wkv7::kHeadP;
  TRY(check_ptrs(n > 0, {x, b, c, state, y}));
  TRY(check_ptrs(n > 0, {dt}, elt(d)));
  if (n == 0) return WKV7_OK;
  if (!status_word(d, &a.status)) return WKV7_ERR_CUDA;
  a.x = x; a.dt = dt; a.b = b; a.c = c; a.state = state; a.active = active; a.y = y;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(d, wkv7::launch_ssm_step(a, d->dtype, s), {{y, n, d->dtype}, {state, n * d->N, WKV7_F32}}, a.status, s);
}

wkv7_status_t wkv7_rms_forward(const wkv7_desc_t* d, const wkv7_rms_t* rn, const void* x, const void* other, void* h_out,
                               void* out, float* scale, void* stream) {
  wkv7::RmsArgs a;
  TRY(check_rms(d, rn, &a));
  const int64_t n = a.rows * a.D;
  const bool sum = other && !a.gate;
  TRY(check_ptrs(n > 0, {x, out}));
  TRY(check_ptrs(n > 0 && sum, {h_out}));
  TRY(check_ptrs(n > 0 && a.quant_block != 0, {scale}));
  TRY(check_ptrs(false, {other}));
  if (h_out && !sum) return WKV7_ERR_UNSUPPORTED;
  if (a.gate && !other && n > 0) return WKV7_ERR_NULL;
  if (n == 0) return WKV7_OK;
  if (!status_word(d, &a.status)) return WKV7_ERR_CUDA;
  a.x = x; a.other = other; a.h_out = h_out; a.out = out; a.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = wkv7::launch_rms_fwd(a, d->dtype, s);
  // e4m3 codes have no dtype of the scan: a NaN among them shows in its block's scale
  if (a.quant_block == 0) return finish(d, e, {{out, n, d->dtype}, {h_out, n, d->dtype}}, a.status, s);
  const int64_t ns = a.quant_block > 0 ? n / 128 : a.rows * a.groups;
  return finish(d, e, {{scale, ns, WKV7_F32}, {h_out, n, d->dtype}}, a.status, s);
}

size_t wkv7_rms_scratch_bytes(const wkv7_desc_t* d, const wkv7_rms_t* rn) {
  wkv7::RmsArgs a;
  if (check_rms(d, rn, &a, true) != WKV7_OK) return 0;
  return size_t(wkv7::rms_scratch_floats(d->B * d->T, rn->D, rn->groups)) * 4;
}

wkv7_status_t wkv7_rms_backward(const wkv7_desc_t* d, const wkv7_rms_t* rn, const void* x, const void* other,
                                const void* dout, const void* dh, void* dx, void* dother, float* dweight,
                                void* scratch, void* stream) {
  wkv7::RmsArgs a;
  TRY(check_rms(d, rn, &a));
  const int64_t n = a.rows * a.D;
  if (a.quant_block != 0) return WKV7_ERR_UNSUPPORTED;
  if (!a.gate && (other || dother)) return WKV7_ERR_UNSUPPORTED;
  if (a.gate && dh) return WKV7_ERR_UNSUPPORTED;
  TRY(check_ptrs(n > 0, {x, dout, dx}));
  TRY(check_ptrs(n > 0 && a.gate, {other, dother}));
  TRY(check_ptrs(false, {dh, scratch, dweight}));
  if (n > 0 && dweight && !scratch) return WKV7_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) return zero(dweight, a.D * 4, s) ? WKV7_OK : WKV7_ERR_CUDA;
  if (!status_word(d, &a.status)) return WKV7_ERR_CUDA;
  a.x = x; a.other = a.gate ? other : nullptr; a.dout = dout; a.dh = dh; a.dx = dx; a.dother = dother; a.dweight = dweight;
  a.scratch = dweight ? static_cast<float*>(scratch) : nullptr;
  return finish(d, wkv7::launch_rms_bwd(a, d->dtype, s),
                {{dx, n, d->dtype}, {a.gate ? dother : nullptr, n, d->dtype}, {dweight, a.D, WKV7_F32}}, a.status, s);
}

}  // extern "C"
