// Heads normed and turned in bf16 (rotary.cuh).
#include "rotary.cuh"

namespace fvx {

fvx_status run_heads_bf16(const char* name, HeadCall& c, HeadOp op, int jobs, const fvx_head_tensor_t* t, HeadDw* dw,
                         cudaStream_t s, Scratch* scr) {
  return run_heads<__nv_bfloat16>(name, c, op, jobs, t, dw, s, scr);
}

}  // namespace fvx
