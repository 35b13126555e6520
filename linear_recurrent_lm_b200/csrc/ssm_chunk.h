// Launch interface of the chunked (tensor-core) selective scan.
#pragma once

#include "state_space.h"

namespace wkv7 {

namespace stc {
struct TileMaps;
}

// One pass over the chunks of every (b, h), each row cut into `segments` runs of `per_segment` chunks.
struct ChunkOp {
  int64_t segments, per_segment;
  bool local;            // segments start from zero and leave their end state and total decay; else they start from
                         // what the segments before them left
  const float* init;     // [B,H,64,N] entering state of the row (gradient: of the last one), or null
  float* states;         // [B,H,stride,64,N]: the state that enters each chunk (and the final one, forward), or null
  int64_t stride;
  float* last;           // [B,H,64,N] state after the walk, or null
  float *seg_state, *seg_decay;   // [B,H,segments,64,N], [B,H,segments]
};

cudaError_t launch_ssm_chunk_fwd(const SsmArgs& p, const stc::TileMaps& tm, cudaStream_t s);
cudaError_t launch_ssm_chunk_dstate(const SsmArgs& p, const stc::TileMaps& tm, float* dstate, float* seg, cudaStream_t s);
// Everything of the backward but the decays' gradients (which follow from the scalars it leaves in scratch).
cudaError_t launch_ssm_chunk_bwd(const SsmArgs& p, const stc::TileMaps& tm, cudaStream_t s);
// Tensor maps of the bf16 token tensors (see ssm_tc.cuh); false if the driver refuses one.
bool encode_ssm_maps(const SsmArgs& p, bool backward, stc::TileMaps* tm);

}  // namespace wkv7
