// Streaming row kernels for fp32 tensors (norm_stream.cuh).
#include "norm_stream.cuh"

namespace fvx {

fvx_status stream_rows_f32(const char* name, RowOp op, int iters, const StreamArgs& a, int blocks, size_t smem,
                           cudaStream_t s) {
  return stream_rows<float>(name, op, iters, a, blocks, smem, s);
}

}  // namespace fvx
