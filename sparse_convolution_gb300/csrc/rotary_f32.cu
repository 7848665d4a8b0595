// Heads normed and turned in fp32 (rotary.cuh).
#include "rotary.cuh"

namespace fvx {

fvx_status run_heads_f32(const char* name, HeadCall& c, HeadOp op, int jobs, const fvx_head_tensor_t* t, HeadDw* dw,
                        cudaStream_t s, Scratch* scr) {
  return run_heads<float>(name, c, op, jobs, t, dw, s, scr);
}

}  // namespace fvx
