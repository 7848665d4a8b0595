// Rotary positions of attention heads, and norms of queries and keys per head
// with the rotation in the same pass.
//
// A head of d values has R = 2P rotated ones in P pairs (halves: p and p + P;
// interleaved: 2p and 2p + 1), the rest pass.  Pair p turns by t = pos[axis(p)] f_p:
//   (u, v) -> m (u cos t - v sin t, v cos t + u sin t)
// and its gradient is the transposed matrix, the same with -t.
// With the norm:  y = R(x rstd w),  rstd = 1 / sqrt(sum x^2 / d + eps)
// Backward, g = R' dy:  dx = rstd (g w - x rstd^2 sum(g w x) / d),  dw = sum over tokens and heads of g x rstd
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "fvx_internal.cuh"
#include "norm.cuh"

namespace fvx {
namespace {

constexpr int kMaxHead = 256;
constexpr int kMaxPairs = kMaxHead / 2;

// One of the call's tensors.
struct HeadJob {
  const void* in;  // forward: x; backward: the gradient of the result
  const void* x;   // norm backward: the forward pass's input
  void* out;
  const float* w;
  const int32_t* pos;
  float* part;  // norm backward: [blocks][d] partial sums of dw
  int64_t in_token, in_head, x_token, x_head, out_token, out_head, pos_token, pos_axis;
  int units, heads, chunks;  // a unit is up to HC heads (chunk, chunk + chunks, ...) of a token
  int block0;                // the job's first block
};
struct HeadArgs {
  HeadJob job[2];
  uint64_t turns[kMaxPairs];  // turns per position step, in 2^-64
  int jobs, d, pairs, axis1, axis2;  // pairs from axis1 (axis2) on belong to the second (third) axis
  int items, items_turned, lanes;    // vectors of pairs, of passing values; lanes that share a head
  float magnitude, sign, eps, inv_d;
};

// A turn's fraction in 2^-32: the product wraps at whole turns by itself, so a
// position of any size loses nothing that its step does not.
__device__ __forceinline__ uint32_t turn_of(uint64_t step, int pos) {
  return (uint32_t)((step * (uint64_t)(int64_t)pos) >> 32);
}
// Sine and cosine of a fraction of a turn: the nearest quarter is taken off
// exactly, and the Taylor series end where they are below 2e-9 on the 1/8 turn left.
__device__ __forceinline__ void sincos_turn(uint32_t t, float& s, float& c) {
  const uint32_t q = (t + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(t - (q << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float a = fmaf(x2, 2.75573192239858907e-6f, -1.98412698412698413e-4f);
  a = fmaf(x2, a, 8.33333333333333333e-3f);
  a = fmaf(x2, a, -1.66666666666666667e-1f);
  a = fmaf(x * x2, a, x);
  float b = fmaf(x2, -2.75573192239858907e-7f, 2.48015873015873016e-5f);
  b = fmaf(x2, b, -1.38888888888888889e-3f);
  b = fmaf(x2, b, 4.16666666666666667e-2f);
  b = fmaf(x2, b, -0.5f);
  b = fmaf(x2, b, 1.0f);
  const bool swap = q & 1u;
  s = swap ? b : a;
  c = swap ? a : b;
  if (q & 2u) s = -s;
  if ((q + 1u) & 2u) c = -c;
}

// What a lane holds of a head: ITEMS items of two vectors of V values each, a
// pair's partners in the same lane.
template <typename T, int V, int ITEMS, bool INTERLEAVED>
struct Place {
  int a[ITEMS], b[ITEMS], p[ITEMS];  // offsets of the two vectors, first pair (or -1: values that pass)
  bool has_a[ITEMS], has_b[ITEMS];
  __device__ __forceinline__ Place(const HeadArgs& args, int lane) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int item = lane + i * args.lanes;
      const bool turned = item < args.items_turned;
      p[i] = turned ? item * V : -1;
      a[i] = turned ? (INTERLEAVED ? 2 : 1) * item * V : 2 * args.pairs + (item - args.items_turned) * 2 * V;
      b[i] = turned && !INTERLEAVED ? a[i] + args.pairs : a[i] + V;
      has_a[i] = item < args.items;
      has_b[i] = has_a[i] && b[i] < args.d;
      if (!has_a[i]) p[i] = -1;
    }
  }
};

template <int V, int ITEMS>
struct Angles {
  float c[ITEMS][V], s[ITEMS][V];
};
template <int V, int ITEMS, typename P>
__device__ __forceinline__ void angles_at(const HeadArgs& a, const HeadJob& j, const P& pl, int64_t token,
                                          const uint64_t (&step)[ITEMS][V], Angles<V, ITEMS>& out) {
  const int32_t* at = j.pos + token * j.pos_token;
  int pos[3];
  pos[0] = __ldg(at);
  pos[1] = a.axis1 < a.pairs ? __ldg(at + j.pos_axis) : 0;
  pos[2] = a.axis2 < a.pairs ? __ldg(at + 2 * j.pos_axis) : 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int p = pl.p[i] + k;
      const int at_axis = p >= a.axis2 ? pos[2] : p >= a.axis1 ? pos[1] : pos[0];
      float s, c;
      sincos_turn(turn_of(step[i][k], at_axis), s, c);
      out.c[i][k] = c * a.magnitude;
      out.s[i][k] = s * a.magnitude * a.sign;
    }
}

// (u, v) of a lane's pairs, as stored in its two vectors, turned.
template <int V, bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&x)[2 * V], const float (&c)[V], const float (&s)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int iu = INTERLEAVED ? 2 * k : k, iv = INTERLEAVED ? 2 * k + 1 : V + k;
    const float u = x[iu], v = x[iv];
    x[iu] = fmaf(u, c[k], -(v * s[k]));
    x[iv] = fmaf(v, c[k], u * s[k]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void join(const Pack<T, V>& a, const Pack<T, V>& b, float (&f)[2 * V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    f[k] = Elem<T>::get(a.v[k]);
    f[V + k] = Elem<T>::get(b.v[k]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void split_store(T* p, int a, int b, bool has_a, bool has_b, const float (&f)[2 * V]) {
  Pack<T, V> u, v;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    u.v[k] = Elem<T>::put(f[k]);
    v.v[k] = Elem<T>::put(f[V + k]);
  }
  if (has_a) *reinterpret_cast<Pack<T, V>*>(p + a) = u;
  if (has_b) *reinterpret_cast<Pack<T, V>*>(p + b) = v;
}

template <typename T, int V, int ITEMS, bool INTERLEAVED, bool NORM, int HC>
__global__ void __launch_bounds__(kThreads) k_heads(const __grid_constant__ HeadArgs args) {
  const HeadJob& j = args.job[args.jobs > 1 && (int)blockIdx.x >= args.job[1].block0];
  const int lane = threadIdx.x & (args.lanes - 1);
  const int unit = (blockIdx.x - j.block0) * (kThreads / args.lanes) + threadIdx.x / args.lanes;
  const bool live = unit < j.units;
  const int token = live ? unit / j.chunks : 0, h0 = unit - token * j.chunks;
  const Place<T, V, ITEMS, INTERLEAVED> pl(args, lane);
  Pack<T, V> xa[HC][ITEMS], xb[HC][ITEMS];
  const T* in = reinterpret_cast<const T*>(j.in) + token * j.in_token;
#pragma unroll
  for (int h = 0; h < HC; ++h) {
    const int head = h0 + h * j.chunks;
    const bool mine = live && head < j.heads;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      xa[h][i] = mine && pl.has_a[i] ? raw_vec<T, V>(in + head * j.in_head + pl.a[i]) : no_vec<T, V>();
      xb[h][i] = mine && pl.has_b[i] ? raw_vec<T, V>(in + head * j.in_head + pl.b[i]) : no_vec<T, V>();
    }
  }
  uint64_t step[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) step[i][k] = pl.p[i] >= 0 ? args.turns[pl.p[i] + k] : 0;
  Angles<V, ITEMS> an;
  if (args.pairs) angles_at<V, ITEMS>(args, j, pl, token, step, an);
  float w[ITEMS][2 * V];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        w[i][k] = j.w && pl.has_a[i] ? __ldg(j.w + pl.a[i] + k) : 1.0f;
        w[i][V + k] = j.w && pl.has_b[i] ? __ldg(j.w + pl.b[i] + k) : 1.0f;
      }
  }
#pragma unroll
  for (int h = 0; h < HC; ++h) {
    const int head = h0 + h * j.chunks;
    const bool mine = live && head < j.heads;
    float x[ITEMS][2 * V], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      join<T, V>(xa[h][i], xb[h][i], x[i]);
      if constexpr (NORM) {
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) sum = fmaf(x[i][k], x[i][k], sum);
      }
    }
    float rstd = 1.0f;
    if constexpr (NORM) rstd = rsqrtf(fmaf(lanes_sum(sum, args.lanes), args.inv_d, args.eps));
    T* out = reinterpret_cast<T*>(j.out) + token * j.out_token + head * j.out_head;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if constexpr (NORM) {
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) x[i][k] *= rstd * w[i][k];
      }
      if (pl.p[i] >= 0) turn<V, INTERLEAVED>(x[i], an.c[i], an.s[i]);
      split_store<T, V>(out, pl.a[i], pl.b[i], mine && pl.has_a[i], mine && pl.has_b[i], x[i]);
    }
  }
}

// The norm's gradients.  Blocks stay and walk their job's units; a lane keeps
// its channels, so its part of dw stays in registers until the end.
template <typename T, int V, int ITEMS, bool INTERLEAVED, int HC>
__global__ void __launch_bounds__(kThreads) k_heads_bwd(const __grid_constant__ HeadArgs args) {
  extern __shared__ float sh[];  // [kThreads / lanes][d]
  const int which = args.jobs > 1 && (int)blockIdx.x >= args.job[1].block0;
  const HeadJob& j = args.job[which];
  const int block = blockIdx.x - j.block0;
  const int blocks = (which + 1 < args.jobs ? args.job[1].block0 : (int)gridDim.x) - j.block0;
  const int lane = threadIdx.x & (args.lanes - 1), group = threadIdx.x / args.lanes, groups = kThreads / args.lanes;
  const Place<T, V, ITEMS, INTERLEAVED> pl(args, lane);
  uint64_t step[ITEMS][V];
  float w[ITEMS][2 * V], dw[ITEMS][2 * V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      step[i][k] = pl.p[i] >= 0 ? args.turns[pl.p[i] + k] : 0;
      w[i][k] = j.w && pl.has_a[i] ? __ldg(j.w + pl.a[i] + k) : 1.0f;
      w[i][V + k] = j.w && pl.has_b[i] ? __ldg(j.w + pl.b[i] + k) : 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) dw[i][k] = 0.0f;
  }
  // every group of a warp takes the same number of turns: they sum together
  for (int64_t first = (int64_t)block * groups; first < j.units; first += (int64_t)blocks * groups) {
    const int64_t unit = first + group;
    const bool live = unit < j.units;
    const int token = live ? (int)unit / j.chunks : 0, h0 = (int)unit - token * j.chunks;
    Pack<T, V> xa[HC][ITEMS], xb[HC][ITEMS], ga[HC][ITEMS], gb[HC][ITEMS];
    const T* in = reinterpret_cast<const T*>(j.in) + token * j.in_token;
    const T* xs = reinterpret_cast<const T*>(j.x) + token * j.x_token;
#pragma unroll
    for (int h = 0; h < HC; ++h) {
      const int head = h0 + h * j.chunks;
      const bool mine = live && head < j.heads;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const bool a = mine && pl.has_a[i], b = mine && pl.has_b[i];
        xa[h][i] = a ? raw_vec<T, V>(xs + head * j.x_head + pl.a[i]) : no_vec<T, V>();
        xb[h][i] = b ? raw_vec<T, V>(xs + head * j.x_head + pl.b[i]) : no_vec<T, V>();
        ga[h][i] = a ? raw_vec<T, V>(in + head * j.in_head + pl.a[i]) : no_vec<T, V>();
        gb[h][i] = b ? raw_vec<T, V>(in + head * j.in_head + pl.b[i]) : no_vec<T, V>();
      }
    }
    Angles<V, ITEMS> an;
    if (args.pairs) angles_at<V, ITEMS>(args, j, pl, token, step, an);
#pragma unroll
    for (int h = 0; h < HC; ++h) {
      const int head = h0 + h * j.chunks;
      const bool mine = live && head < j.heads;
      float x[ITEMS][2 * V], g[ITEMS][2 * V], xx = 0.0f, gx = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        join<T, V>(xa[h][i], xb[h][i], x[i]);
        join<T, V>(ga[h][i], gb[h][i], g[i]);
        if (pl.p[i] >= 0) turn<V, INTERLEAVED>(g[i], an.c[i], an.s[i]);
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) {
          xx = fmaf(x[i][k], x[i][k], xx);
          gx = fmaf(g[i][k] * w[i][k], x[i][k], gx);
        }
      }
      const float rstd = rsqrtf(fmaf(lanes_sum(xx, args.lanes), args.inv_d, args.eps));
      const float back = lanes_sum(gx, args.lanes) * args.inv_d * rstd * rstd;
      T* out = reinterpret_cast<T*>(j.out) + token * j.out_token + head * j.out_head;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) {
          const float xr = x[i][k] * rstd;
          if (mine) dw[i][k] = fmaf(g[i][k], xr, dw[i][k]);
          g[i][k] = rstd * fmaf(-x[i][k], back, g[i][k] * w[i][k]);
        }
        split_store<T, V>(out, pl.a[i], pl.b[i], mine && pl.has_a[i], mine && pl.has_b[i], g[i]);
      }
    }
  }
  if (!j.part) return;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (pl.has_a[i]) sh[group * args.d + pl.a[i] + k] = dw[i][k];
      if (pl.has_b[i]) sh[group * args.d + pl.b[i] + k] = dw[i][V + k];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < args.d; c += kThreads) {
    float s = 0.0f;
    for (int k = 0; k < groups; ++k) s += sh[k * args.d + c];
    j.part[(int64_t)block * args.d + c] = s;
  }
}

// dw of both tensors from their blocks' parts, in a fixed order: 32 channels per block.
struct DwArgs {
  const float* part[2];
  float* dw[2];
  int parts[2];
  int d;
};
__global__ void __launch_bounds__(1024) k_heads_dw(const __grid_constant__ DwArgs a) {
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

// ---------------------------------------------------------------- host
fvx_status bad(const char* who, const char* what) {
  set_error("%s: %s", who, what);
  return FVX_ERR_INVALID_ARG;
}

struct Call {
  HeadArgs a;
  int vec;
  bool interleaved;
  int64_t head_rows;
};

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
  if (n <= 1) return heads <= 1 || head >= d;
  if (heads <= 1) return token >= d;
  return token <= head ? token >= d && head >= (n - 1) * token + d : head >= d && token >= (heads - 1) * head + d;
}

fvx_status prepare(const char* who, fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count,
                   const fvx_rotary_t* r, bool back, Call* c) {
  if (dt != FVX_F32 && dt != FVX_BF16) return bad(who, "dtype must be FVX_F32 or FVX_BF16");
  if (d < 1 || d > kMaxHead) return bad(who, "the head size must be in 1..256");
  if (count < 1 || count > 2 || !t) return bad(who, "one or two tensors are taken");
  const int elem = dt == FVX_F32 ? 4 : 2;
  HeadArgs& a = c->a;
  a.jobs = count;
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
    if (!apart(x.n, x.heads, d, x.out_token, x.out_head)) return bad(who, "the strides of out lay heads over each other");
    if (reinterpret_cast<uintptr_t>(x.weight) % 4 || reinterpret_cast<uintptr_t>(x.dweight) % 4)
      return bad(who, "weight or dweight is not aligned to 4 bytes");
    if (r && ((x.n > 0 && !x.positions) || reinterpret_cast<uintptr_t>(x.positions) % 4))
      return bad(who, "positions is NULL or not aligned to 4 bytes");
    if (r && (x.pos_token < 0 || (axes > 1 && x.pos_axis < 0))) return bad(who, "positions has a negative stride");
    HeadJob& j = a.job[i];
    j = {};
    j.in = x.in;
    j.in_token = x.in_token;
    j.in_head = x.in_head;
    j.x = x.x;
    j.x_token = x.x_token;
    j.x_head = x.x_head;
    j.out = x.out;
    j.out_token = x.out_token;
    j.out_head = x.out_head;
    j.w = x.weight;
    j.pos = x.positions;
    j.pos_token = x.pos_token;
    j.pos_axis = x.pos_axis;
    j.heads = (int)x.heads;
    j.units = (int)x.n;  // times chunks, below
    c->head_rows += x.n * x.heads;
    if (x.n == 0) continue;
    view(x, x.in, x.in_token, x.in_head);
    if (back) view(x, x.x, x.x_token, x.x_head);
    view(x, x.out, x.out_token, x.out_head);
  }
  c->vec = vec;
  a.items_turned = a.pairs / vec;
  a.items = a.items_turned + (d - 2 * a.pairs + 2 * vec - 1) / (2 * vec);
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes < a.items) a.lanes *= 2;
  return FVX_OK;
}

// f<T, V, ITEMS, INTERLEAVED>() for the call's type, vectors and layout
template <typename F>
fvx_status by_shape(fvx_dtype dt, const Call& c, F&& f) {
  auto layout = [&]<typename T, int V, int ITEMS>() -> fvx_status {
    return c.interleaved ? f.template operator()<T, V, ITEMS, true>() : f.template operator()<T, V, ITEMS, false>();
  };
  const bool one = c.a.items <= c.a.lanes;
  if (dt == FVX_F32) {
    if (c.vec == 4) return layout.template operator()<float, 4, 1>();
    if (c.vec == 2) return one ? layout.template operator()<float, 2, 1>() : layout.template operator()<float, 2, 2>();
    return one ? layout.template operator()<float, 1, 1>() : layout.template operator()<float, 1, 4>();
  }
  if (c.vec == 8) return layout.template operator()<__nv_bfloat16, 8, 1>();
  if (c.vec == 4) return layout.template operator()<__nv_bfloat16, 4, 1>();
  if (c.vec == 2) return one ? layout.template operator()<__nv_bfloat16, 2, 1>() : layout.template operator()<__nv_bfloat16, 2, 2>();
  return one ? layout.template operator()<__nv_bfloat16, 1, 1>() : layout.template operator()<__nv_bfloat16, 1, 4>();
}

// Cuts the tensors into units of up to hc heads; blocks for all of them, at most `most` if given.
int cut(HeadArgs& a, int hc, int most) {
  const int per_block = kThreads / a.lanes;
  int64_t all = 0;
  for (int i = 0; i < a.jobs; ++i) {
    HeadJob& j = a.job[i];
    j.chunks = (j.heads + hc - 1) / hc;
    j.units *= j.chunks;
    all += ((int64_t)j.units + per_block - 1) / per_block;
  }
  int at = 0;
  for (int i = 0; i < a.jobs; ++i) {
    HeadJob& j = a.job[i];
    j.block0 = at;
    int64_t b = ((int64_t)j.units + per_block - 1) / per_block;
    if (most && all > most && b > 0) b = std::max<int64_t>(1, b * most / all);
    at += (int)b;
  }
  return at;
}

fvx_status run_heads(const char* name, fvx_dtype dt, Call& c, bool norm, cudaStream_t s) {
  if (c.head_rows == 0) return FVX_OK;
  return by_shape(dt, c, [&]<typename T, int V, int ITEMS, bool IL>() -> fvx_status {
    int sms = 0;
    FVX_TRY(device_sm_count(&sms));
    const bool many = c.head_rows * c.a.lanes >= (int64_t)sms * 2048 * 2;
    constexpr int kMany = ITEMS == 1 ? 2 : 1;
    const int blocks = cut(c.a, many ? kMany : 1, 0);
    LaunchScope ls(name, s);
    if (norm) {
      if (many) k_heads<T, V, ITEMS, IL, true, kMany><<<blocks, kThreads, 0, s>>>(c.a);
      else k_heads<T, V, ITEMS, IL, true, 1><<<blocks, kThreads, 0, s>>>(c.a);
    } else {
      if (many) k_heads<T, V, ITEMS, IL, false, kMany><<<blocks, kThreads, 0, s>>>(c.a);
      else k_heads<T, V, ITEMS, IL, false, 1><<<blocks, kThreads, 0, s>>>(c.a);
    }
    return check_launch(name);
  });
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
  Call c;
  if (!rotary) return bad(who, "NULL rotary");
  FVX_TRY(prepare(who, dt, d, t, count, rotary, false, &c));
  c.a.sign = transposed ? -1.0f : 1.0f;
  return run_heads("rotate_heads", dt, c, false, (cudaStream_t)stream);
}

fvx_status fvx_norm_rotate_heads(fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count,
                                 const fvx_rotary_t* rotary, float eps, fvx_stream stream) {
  const char* who = "fvx_norm_rotate_heads";
  EntryScope entry(who);
  Call c;
  if (!(eps >= 0.0f)) return bad(who, "eps must not be negative");
  FVX_TRY(prepare(who, dt, d, t, count, rotary, false, &c));
  c.a.eps = eps;
  return run_heads("norm_rotate_heads", dt, c, true, (cudaStream_t)stream);
}

fvx_status fvx_norm_rotate_heads_backward(fvx_dtype dt, int32_t d, const fvx_head_tensor_t* t, int32_t count,
                                          const fvx_rotary_t* rotary, float eps, fvx_stream stream) {
  const char* who = "fvx_norm_rotate_heads_backward";
  EntryScope entry(who);
  Call c;
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
  DwArgs w = {};
  w.d = d;
  FVX_TRY(by_shape(dt, c, [&]<typename T, int V, int ITEMS, bool IL>() -> fvx_status {
    int sms = 0;
    FVX_TRY(device_sm_count(&sms));
    const int blocks = cut(c.a, 1, 4 * sms);
    for (int i = 0; i < count; ++i) {
      if (t[i].n == 0 || !t[i].dweight) continue;
      w.parts[i] = (i + 1 < count ? c.a.job[1].block0 : blocks) - c.a.job[i].block0;
      w.dw[i] = t[i].dweight;
      if (!(c.a.job[i].part = scr.get<float>((size_t)w.parts[i] * d))) return FVX_ERR_ALLOC;
      w.part[i] = c.a.job[i].part;
    }
    const size_t smem = (size_t)(kThreads / c.a.lanes) * d * 4;  // a lane holds 16 values at most: 16 KB (passing ones 32)
    LaunchScope ls("norm_rotate_heads_bwd", s);
    k_heads_bwd<T, V, ITEMS, IL, 1><<<blocks, kThreads, smem, s>>>(c.a);
    return check_launch("norm_rotate_heads_bwd");
  }));
  if (!sums) return FVX_OK;
  LaunchScope ls("norm_rotate_heads_dw", s);
  k_heads_dw<<<dim3((unsigned)((d + 31) / 32), (unsigned)count), 1024, 0, s>>>(w);
  return check_launch("norm_rotate_heads_dw");
}

}  // extern "C"
