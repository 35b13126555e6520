// Tensor maps of the chunked selective scan's token tensors.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "ssm_chunk.h"
#include "ssm_tc.cuh"

namespace wkv7 {
namespace {

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime (no link to libcuda).
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Rows of `heads` x `width` bf16, `ld` elements apart, as {width, heads, T, B} with a {64, 1, 128, 1} box.
bool encode(PFN_cuTensorMapEncodeTiled_v12000 enc, const SsmArgs& p, const void* ptr, int64_t width, int64_t heads, int64_t ld,
            CUtensorMap* m) {
  if (!ptr) return true;
  if (p.B * p.T == 1) ld = width * heads;   // one row: its distance to the next is not looked at, but must be encodable
  const cuuint64_t dims[4] = {cuuint64_t(width), cuuint64_t(heads), cuuint64_t(p.T), cuuint64_t(p.B)};
  const cuuint64_t strides[3] = {cuuint64_t(width) * 2, cuuint64_t(ld) * 2, cuuint64_t(p.T) * cuuint64_t(ld) * 2};
  const cuuint32_t box[4] = {64, 1, cuuint32_t(kSsmChunk), 1}, one[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_ssm_maps(const SsmArgs& p, bool backward, stc::TileMaps* tm) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_tiled();
  if (!enc) return false;
  const bool ok = encode(enc, p, p.x, kHeadP, p.H, p.x_ld, &tm->x) && encode(enc, p, p.b, p.N, p.G, p.b_ld, &tm->b) &&
            encode(enc, p, p.c, p.N, p.G, p.c_ld, &tm->c);
  return ok && encode(enc, p, backward ? p.dy : p.y, kHeadP, p.H, p.H * kHeadP, backward ? &tm->dy : &tm->y);
}

}  // namespace wkv7
