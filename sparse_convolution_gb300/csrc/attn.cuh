// Shared by the cross-attention kernels (attn.cu: fp32 arithmetic on the CUDA
// cores, reductions and the C entry points; attn_tc.cu: bf16 on the tensor
// cores; attn_few.cu: a few rows per key head).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "fvx_internal.cuh"

namespace fvx {

constexpr int kInlineItems = 64;  // batch elements whose offsets travel in the kernel's arguments

// Arrays of items + 1 values that describe a ragged batch to a kernel, held in
// its arguments or (more items) in device memory.  Which arrays follow the
// offsets depends on the kernel.
enum AttnArray {
  kItemQ = 0,      // first query token
  kItemK = 1,      // first key token
  kItemUnit = 2,   // first work unit
  kItemTile = 3,   // backward: first row tile
  kItemRows = 4,   // backward: ranges that the item's row tiles are cut into
  kItemKeys = 5,   // backward: ranges that its key tiles are cut into
  kItemKeyTile = 6,  // backward: first key tile
  kItemRowSlab = 7,  // backward: first slab of dQ's partial sums, one per key range and row tile
  kItemKeySlab = 8,  // backward: first slab of dK's and dV's, one per row range and key tile
  kItemArrays = 9
};
struct AttnItems {
  const int32_t* ptr;
  int32_t items;
  int32_t in[kItemArrays * (kInlineItems + 1)];
#ifdef __CUDACC__
  __device__ __forceinline__ int at(int array, int b) const {
    const int i = array * (items + 1) + b;
    return ptr ? __ldg(ptr + i) : in[i];
  }
  __device__ __forceinline__ int q0(int b) const { return at(kItemQ, b); }
  __device__ __forceinline__ int k0(int b) const { return at(kItemK, b); }
  __device__ __forceinline__ int u0(int b) const { return at(kItemUnit, b); }
  // the item whose range of the (rising) array holds value v
  __device__ __forceinline__ int find(int array, int v) const {
    int lo = 0, hi = items;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at(array, mid) <= v) lo = mid;
      else hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ int item_of(int u) const { return find(kItemUnit, u); }
#endif
};

struct HeadsView {  // [tokens, heads, d] with the last dimension dense; strides in elements
  const void* p;
  int64_t token, head;
};

struct AttnCall {
  fvx_dtype dt;
  HeadsView q, k, v, dout;
  const int64_t* q_offsets;  // host
  const int64_t* kv_offsets;
  int items, heads, kv_heads, shared, d;  // shared: query heads per key head
  int64_t nq, nk;
  const uint8_t* mask;
  float scale;
  void* out;  // [nq, heads, d]; the backward pass reads it
  float* lse; // [nq, heads]
  void *dq, *dk, *dv;
};

// The bf16 tensor-core kernels (attn_tc.cu) take a call when this says so.
bool attn_tc_serves(const AttnCall& c, bool backward);
fvx_status attn_tc_forward(const AttnCall& c, cudaStream_t s, Scratch& scr);
fvx_status attn_tc_backward(const AttnCall& c, cudaStream_t s, Scratch& scr);

// The kernel for a few rows per key head (attn_few.cu).
bool attn_few_serves(const AttnCall& c);
fvx_status attn_few_forward(const AttnCall& c, cudaStream_t s, Scratch& scr);

// attn.cu helpers that the others use
// more: the arrays after the offsets, `arrays - 2` times items + 1 values
fvx_status attn_items(const AttnCall& c, const int32_t* more, int arrays, cudaStream_t s, Scratch& scr,
                      AttnItems* out);
// out = softmax-weighted join of `splits` partial results over ranges of keys
fvx_status attn_join(const AttnCall& c, const float* part, const float* top, const float* total, int splits,
                     cudaStream_t s);

}  // namespace fvx
