// Launch interface of the state-space layer's kernels (short convolution, selective scan, RMS norm)
// behind state_space_api.cu.  dtype codes as in kernels.h: 0 = f32, 1 = bf16, 2 = f16.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "wkv7.h"

namespace wkv7 {

constexpr int kHeadP = 64;       // channels of a head of the selective scan (state rows)
constexpr int kSsmChunk = 128;   // tokens of a chunk: one checkpointed state each

struct ConvArgs {
  int64_t B, T, D, x_ld;
  int W;
  bool silu;
  const float *weight, *bias;
  const void *x, *s0;
  const uint8_t* reset;
  void *y, *s_out;
  // backward
  const void *dy, *dsT;
  void *dx, *ds0;
  float *dweight, *dbias, *scratch;
  // step
  void* state;
  const uint8_t* active;
  int* status;
};
cudaError_t launch_conv_fwd(const ConvArgs& p, int dtype, cudaStream_t s);
cudaError_t launch_conv_bwd(const ConvArgs& p, int dtype, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& p, int dtype, cudaStream_t s);
// fp32 elements of scratch the backward's partial sums need.
int64_t conv_scratch_floats(int64_t B, int64_t T, int64_t D, int W);

struct RmsArgs {
  int64_t rows, D, groups;
  const float* weight;
  float eps;
  bool gate;
  int quant_block;
  const void *x, *other;
  void *h_out, *out;
  float* scale;
  // backward
  const void *dout, *dh;
  void *dx, *dother;
  float *dweight, *scratch;
  int* status;
};
cudaError_t launch_rms_fwd(const RmsArgs& p, int dtype, cudaStream_t s);
cudaError_t launch_rms_bwd(const RmsArgs& p, int dtype, cudaStream_t s);
int64_t rms_scratch_floats(int64_t rows, int64_t D, int64_t groups);

struct SsmArgs {
  int64_t B, T, H, G;
  int N;
  const float *A, *Dw, *dt_bias;
  bool softplus;
  int64_t x_ld, dt_ld, b_ld, c_ld;
  const void *x, *dt, *b, *c;
  const float* s0;
  const uint8_t* reset;
  void* y;
  float* s_out;
  float* ckpt;        // [B,H,nc+1,64,N] state before each chunk, then the last one, or null
  // backward
  const void* dy;
  const float* dsT;
  void *dx, *ddt, *db, *dc;
  float *dA, *dD, *ddt_bias, *ds0;
  float* scratch;
  // step
  float* state;
  const uint8_t* active;
  int* status;
};

// Parts of the backward's scratch, as offsets in fp32 elements (16-byte aligned); `d`: fp64 values.
struct SsmScratch {
  int64_t row, col;        // d [B,H,nc*128] per token: see ssm_decay.cu
  int64_t far;             // [B,H,nc*128] per token: CHUNKED: the part of col that leaves the chunk (not in `col` then)
  int64_t own, xdy;        // [B,H,nc*128] per token: (x . dy)(b . c) and x . dy
  int64_t anchor;          // d [B,H,nc] <state after the chunk, gradient of it> (CHUNKED: without what `far` starts)
  int64_t part;            // [B,H,nc,3] partial dA, dD, ddt_bias
  int64_t dstate;          // [B,H,nc] gradient of the state after each chunk (SCAN: d, transposed)
  int64_t state_t;         // SCAN: d [B,H,nc+1] states before each chunk and the last, transposed as dstate
  int64_t dcp, dbp;        // SCAN: d [B,T,H,N] the past's part of dc and db per head
  int64_t seg;             // end states and decays of the segments of a cut row
  int64_t db_part, dc_part;   // CHUNKED: [splits][B,T,G,N] sums over the heads of a split, where there are several
  int64_t splits;             // CHUNKED: parts that a group's heads are cut into
  int64_t total;
};
SsmScratch ssm_scratch(int64_t B, int64_t T, int64_t H, int64_t G, int N, bool chunked);
// fp32 elements of the part `seg` (the forward's is behind its checkpoints): CHUNKED; SCAN (twice that in the backward).
int64_t ssm_segment_floats(int64_t B, int64_t T, int64_t H, int N);
int64_t ssm_run_floats(int64_t B, int64_t T, int64_t H, int N);

cudaError_t launch_ssm_scan_fwd(const SsmArgs& p, int dtype, cudaStream_t s);
cudaError_t launch_ssm_scan_bwd(const SsmArgs& p, int dtype, cudaStream_t s);
// From the per-token scalars in scratch: ddt, dA, dD, ddt_bias (the last step of every backward).
cudaError_t launch_ssm_decay(const SsmArgs& p, int dtype, bool chunked, cudaStream_t s);
cudaError_t launch_ssm_step(const SsmArgs& p, int dtype, cudaStream_t s);

}  // namespace wkv7
