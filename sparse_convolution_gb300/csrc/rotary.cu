// Rotary positions of attention heads, and norms of queries and keys per head
// with the rotation in the same pass.
//
// A head of d values has R = 2P rotated ones in P pairs (halves: p and p + P;
// interleaved: 2p and 2p + 1), the rest pass.  Pair p turns by t = pos[axis(p)] f_p:
//   (u, v) -> m (u cos t - v sin t, v cos t + u sin t)
// and its gradient is the transposed matrix, the same with -t.
// With the norm:  y = R(x rstd w),  rstd = 1 / sqrt(sum x^2 / d + eps)
// Backward, g = R' dy:  dx = rstd (g w - x rstd^2 sum(g w x) / d),  dw = sum over tokens and heads of g x rstd
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "rotary.cuh"

namespace fvx {
namespace {

// dw of both tensors from their blocks' parts, in a fixed order: 32 channels per block.
__global__ void __launch_bounds__(1024) k_heads_dw(const __grid_constant__ HeadDw a) {
  __shared__ float sh[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx, which = blockIdx.y;
  float s = 0.0f;
  if (c < a.d && a.dw[which]) {
    constexpr int kAtOnce = 8;
    for (int p = ty; p < a.parts[which]; p += 32 * kAtOnce) {
      float x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = p + 32 * k;
        x[k] = i < a.parts[which] ? __ldg(a.part[which] + (int64_t)i * a.d + c) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) s += x[k];
    }
  }
  sh[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || c >= a.d || !a.dw[which]) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) s += sh[k][tx];
  a.dw[which][c] = s;
}

fvx_status bad(const char* who, const char* what) {
  set_error("%s: %s", who, what);
  return FVX_ERR_INVALID_ARG;
}

fvx_status check_view(const char* who, const char* name, const void* p, int64_t token, int64_t head, int64_t n, int elem) {
  if ((n > 0 && !p) || reinterpret_cast<uintptr_t>(p) % elem) {
    set_error("%s: %s is NULL or not aligned to its elements", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  if (token < 0 || head < 0) {
    set_error("%s: %s has a negative stride", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  return FVX_OK;
}

// Results must not lie over each other.
bool apart(int64_t n, int64_t heads, int64_t d, int64_t token, int64_t head) {
  if (n == 1) return heads <= 1 || head >= d;
  if (heads <= 1) return token >= d;
  return token <= head ? token >= d && head >= (n - 1) * token + d : head >= d && token >= (heads - 1) * head + d;
}

fvx_status prepare(const char* who, fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count,
                   const fvx_rotary_t* r, bool back, HeadCall* c) {
  if (dt != FVX_F32 && dt != FVX_BF16) return bad(who, "dtype must be FVX_F32 or FVX_BF16");
  if (d < 1 || d > kMaxHead) return bad(who, "the head size must be in 1..256");
  if (count < 1 || count > 2 || !t) return bad(who, "one or two tensors are taken");
  const int elem = dt == FVX_F32 ? 4 : 2;
  HeadArgs& a = c->a;
  a.job[0] = a.job[1] = {};
  a.d = d;
  a.inv_d = 1.0f / (float)d;
  a.sign = 1.0f;
  a.magnitude = 1.0f;
  a.pairs = a.axis1 = a.axis2 = 0;
  c->interleaved = false;
  if (r) {
    int64_t pairs = 0;
    for (int i = 0; i < 3; ++i) {
      if (r->pairs[i] < 0) return bad(who, "negative number of rotated pairs");
      pairs += r->pairs[i];
    }
    if (pairs < 1 || 2 * pairs > d) return bad(who, "the rotated pairs must be at least one and fit into the head");
    if (!r->turns) return bad(who, "NULL turns");
    if (!(fabsf(r->magnitude) <= 3.0e38f)) return bad(who, "the rotation's magnitude must be finite");
    a.pairs = (int)pairs;
    a.axis1 = r->pairs[0];
    a.axis2 = r->pairs[0] + r->pairs[1];
    a.magnitude = r->magnitude;
    std::copy(r->turns, r->turns + pairs, a.turns);
    c->interleaved = r->interleaved != 0;
  }
  const int axes = !r ? 0 : r->pairs[2] ? 3 : r->pairs[1] ? 2 : 1;
  // the widest vectors (16 bytes) that the pairs, the values that pass, every base and every stride are multiples of
  int vec = 16 / elem;
  auto fits = [&](int64_t x) {
    while (x % vec) vec >>= 1;
  };
  auto view = [&](const fvx_head_tensor_t& x, const void* p, int64_t token, int64_t head) {
    fits((int64_t)(reinterpret_cast<uintptr_t>(p) / elem));
    if (x.n > 1) fits(token);
    if (x.heads > 1) fits(head);
  };
  fits(a.pairs);
  fits(d - 2 * a.pairs);
  c->head_rows = 0;
  for (int i = 0; i < count; ++i) {
    const fvx_head_tensor_t& x = t[i];
    if (x.n < 0 || x.heads < 1) return bad(who, "tokens must not be negative, heads at least 1");
    if (x.n > ((int64_t)1 << 30) / x.heads) {
      set_error("%s: more than 2^30 rows (tokens * heads)", who);
      return FVX_ERR_RANGE;
    }
    FVX_TRY(check_view(who, back ? "the gradient" : "the tensor", x.in, x.in_token, x.in_head, x.n, elem));
    if (back) FVX_TRY(check_view(who, "x", x.x, x.x_token, x.x_head, x.n, elem));
    FVX_TRY(check_view(who, "out", x.out, x.out_token, x.out_head, x.n, elem));
    if (x.n > 0 && !apart(x.n, x.heads, d, x.out_token, x.out_head)) return bad(who, "the strides of out lay heads over each other");
    if (reinterpret_cast<uintptr_t>(x.weight) % 4 || reinterpret_cast<uintptr_t>(x.dweight) % 4)
      return bad(who, "weight or dweight is not aligned to 4 bytes");
    if (r && ((x.n > 0 && !x.positions) || reinterpret_cast<uintptr_t>(x.positions) % 4))
      return bad(who, "positions is NULL or not aligned to 4 bytes");
    if (r && (x.pos_token < 0 || (axes > 1 && x.pos_axis < 0))) return bad(who, "positions has a negative stride");
    HeadJob& j = a.job[i];
    j = {};
    auto source = [&](const void* p, int64_t token, int64_t head) {
      HeadSource s = {};
      s.p = p;
      s.token = x.n > 1 ? token : 0;
      s.head = x.heads > 1 ? head : 0;
      return s;
    };
    j.in[0] = source(x.in, x.in_token, x.in_head);
    if (back) j.in[1] = source(x.x, x.x_token, x.x_head);
    j.out = x.out;
    j.out_token = x.out_token;
    j.out_head = x.out_head;
    j.w = x.weight;
    j.pos = x.positions;
    j.pos_token = x.pos_token;
    j.pos_axis = x.pos_axis;
    j.heads = (int)x.heads;
    j.n = (int)x.n;
    c->head_rows += x.n * x.heads;
    if (x.n == 0) continue;
    view(x, x.in, x.in_token, x.in_head);
    if (back) view(x, x.x, x.x_token, x.x_head);
    view(x, x.out, x.out_token, x.out_head);
  }
  c->vec = vec;
  a.items_turned = a.pairs / vec;
  a.items = a.items_turned + (d - 2 * a.pairs + 2 * vec - 1) / (2 * vec);
  a.lanes = lanes_of_head(a.items, items_of_lane(dt == FVX_F32, vec));  // 32 at most: 256 values in eights or sixteens
  a.axes = axes;
  a.fours = vec == 8 && !c->interleaved;
  a.pair_lanes = 1;
  while (a.pair_lanes < a.pairs) a.pair_lanes *= 2;
  return FVX_OK;
}

fvx_status run(const char* name, fvx_dtype dt, HeadCall& c, HeadOp op, int jobs, const fvx_head_tensor_t* t, HeadDw* dw,
               fvx_stream stream, Scratch* scr) {
  if (c.head_rows == 0) return FVX_OK;
  return (dt == FVX_F32 ? run_heads_f32 : run_heads_bf16)(name, c, op, jobs, t, dw, (cudaStream_t)stream, scr);
}

}  // namespace
}  // namespace fvx

using namespace fvx;

extern "C" {

fvx_status fvx_rotary_turns(const int32_t pairs[3], double base, fvx_rotary_scaling scaling, double factor, double length,
                            uint64_t* turns, float* magnitude) {
  const char* who = "fvx_rotary_turns";
  EntryScope entry(who);
  if (!pairs || !turns || !magnitude) return bad(who, "NULL argument");
  int64_t all = 0;
  for (int a = 0; a < 3; ++a) {
    if (pairs[a] < 0) return bad(who, "negative number of rotated pairs");
    all += pairs[a];
  }
  if (all < 1 || all > kMaxPairs) return bad(who, "the rotated pairs must be 1..128 in all");
  if (!(base > 1.0 && base <= 1e300)) return bad(who, "base must be above 1 and finite");
  if (scaling < FVX_ROTARY_PLAIN || scaling > FVX_ROTARY_PARTS) return bad(who, "unknown scaling");
  if (scaling != FVX_ROTARY_PLAIN && !(factor >= 1.0 && factor <= 1e9)) return bad(who, "factor must be in 1..1e9");
  if (scaling == FVX_ROTARY_PARTS && !(length >= 1.0 && length <= 1e18)) return bad(who, "length must be in 1..1e18");
  constexpr double kTwoPi = 6.283185307179586476925;
  for (int a = 0; a < 3; ++a)
    for (int i = 0; i < pairs[a]; ++i) {
      double b = base;
      if (scaling == FVX_ROTARY_BASE && pairs[a] > 1) b *= pow(factor, (double)pairs[a] / (pairs[a] - 1));
      double f = pow(b, -(double)i / pairs[a]);
      if (scaling == FVX_ROTARY_LINEAR) f /= factor;
      if (scaling == FVX_ROTARY_PARTS) {
        const double keep = std::min(1.0, std::max(0.0, (length * f / kTwoPi - 1.0) / 31.0));
        f *= keep + (1.0 - keep) / factor;
      }
      *turns++ = (uint64_t)ldexp(f / kTwoPi, 64);  // below 2^64: f <= 1
    }
  *magnitude = scaling == FVX_ROTARY_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return FVX_OK;
}

fvx_status fvx_rotate_heads(fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count, const fvx_rotary_t* rotary,
                            int32_t transposed, fvx_stream stream) {
  const char* who = "fvx_rotate_heads";
  EntryScope entry(who);
  HeadCall c;
  if (!rotary) return bad(who, "NULL rotary");
  FVX_TRY(prepare(who, dt, d, t, count, rotary, false, &c));
  c.a.sign = transposed ? -1.0f : 1.0f;
  return run("rotate_heads", dt, c, kRotate, count, t, nullptr, stream, nullptr);
}

fvx_status fvx_norm_rotate_heads(fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count,
                                 const fvx_rotary_t* rotary, float eps, fvx_stream stream) {
  const char* who = "fvx_norm_rotate_heads";
  EntryScope entry(who);
  HeadCall c;
  if (!(eps >= 0.0f)) return bad(who, "eps must not be negative");
  FVX_TRY(prepare(who, dt, d, t, count, rotary, false, &c));
  c.a.eps = eps;
  return run("norm_rotate_heads", dt, c, kNormRotate, count, t, nullptr, stream, nullptr);
}

fvx_status fvx_norm_rotate_heads_backward(fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count,
                                          const fvx_rotary_t* rotary, float eps, fvx_stream stream) {
  const char* who = "fvx_norm_rotate_heads_backward";
  EntryScope entry(who);
  HeadCall c;
  if (!(eps >= 0.0f)) return bad(who, "eps must not be negative");
  FVX_TRY(prepare(who, dt, d, t, count, rotary, true, &c));
  c.a.eps = eps;
  c.a.sign = -1.0f;
  cudaStream_t s = (cudaStream_t)stream;
  bool sums = false;
  for (int i = 0; i < count; ++i) {
    if (t[i].n == 0 && t[i].dweight) FVX_CUDA(cudaMemsetAsync(t[i].dweight, 0, (size_t)d * 4, s));
    sums |= t[i].n > 0 && t[i].dweight;
  }
  if (c.head_rows == 0) return FVX_OK;
  Scratch scr(s);
  HeadDw w = {};
  w.d = d;
  FVX_TRY(run("norm_rotate_heads_bwd", dt, c, kNormRotateBack, count, t, &w, stream, &scr));
  if (!sums) return FVX_OK;
  LaunchScope ls("norm_rotate_heads_dw", s);
  k_heads_dw<<<dim3((unsigned)((d + 31) / 32), (unsigned)count), 1024, 0, s>>>(w);
  return check_launch("norm_rotate_heads_dw");
}

}  // extern "C"
