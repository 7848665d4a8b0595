// Streaming row kernels for bf16 tensors (norm_stream.cuh).
#include "norm_stream.cuh"

namespace fvx {

fvx_status stream_rows_bf16(const char* name, RowOp op, int iters, const StreamArgs& a, int blocks, size_t smem,
                           cudaStream_t s) {
  return stream_rows<__nv_bfloat16>(name, op, iters, a, blocks, smem, s);
}

}  // namespace fvx
