// Cross attention from the voxels of each batch element to that element's
// encoder states, forward and backward: the C entry points, the fp32 kernels
// on the CUDA cores, and the reductions that the tensor-core kernels
// (attn_tc.cu) share.
//
// For query row i and the kept keys j of its batch element:
//   s_ij = scale q_i . k_j;  lse_i = log sum_j exp s_ij;  p_ij = exp(s_ij - lse_i);  out_i = sum_j p_ij v_j
// and backward, with delta_i = dout_i . out_i:
//   dv_j = sum_i p_ij dout_i;  ds_ij = p_ij (dout_i . v_j - delta_i) scale;
//   dq_i = sum_j ds_ij k_j;    dk_j = sum_i ds_ij q_i
// A row without kept keys has out = 0, lse = -inf and no gradient.  A masked
// key takes part in nothing: whatever its row holds (infinities, NaN) is read
// as zeros, and its gradients are zero.  The maximum and the sum of a row run
// along its keys (Milakov and Gimelshein 2018).
//
// `shared` query heads read one key head.  They are rows of one tile (row =
// token * shared + head within the group), so that keys and values are fetched
// once for all of them and their gradients sum inside the tile's products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "attn.cuh"
#include "tc.cuh"

namespace fvx {
namespace {

constexpr int kMaxD = 128;
constexpr int kFmaThreads = 256;

template <typename T>
__device__ __forceinline__ float as_f32(T v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The fp32 kernels: tiles of 16 I rows by 16 J keys (64 x 64, and 16 or 32 rows
// or 16 keys where a sample has no more) in shared memory, row after row with a
// pitch of 4 more words than a row has, so that the 16 byte reads of
// neighbouring rows lie in different banks.  Thread (ty, tx) of 16 x 16 owns the
// scores of rows ty + 16 i and keys tx + 16 j, and of the results the columns
// 4 tx .. 4 tx + 3 of every 64 in the same rows.  Products run on pairs: over
// even and odd dimensions for the scores, over neighbouring columns for the
// results.  Shared memory's bandwidth and the multiplications bound a long tile
// about equally (8 reads of 16 bytes for 32 paired products of a thread); what
// bounds a small call is the latency of a tile's loads, so inner loops are
// split until there are two blocks per multiprocessor.  Measured: 8000 rows x
// 500 keys and 5000 x 900, 8 heads of 64, forward 525 us, 33 TFLOP/s, backward
// 1682 us, 26; 1208 rows x 6 heads on 219 keys, 3 key heads of 40, 19 and 35 us.
struct FmaArgs {
  AttnItems items;
  HeadsView q, k, v, dout;
  const uint8_t* mask;
  const float* delta;
  const float* lse_in;
  void* out;                  // forward: out (one split); backward: dq (one split)
  void *dk, *dv;              // one split
  float* lse;
  float *part, *top, *total;  // several splits: [split][nq * heads][d], [split][nq * heads]
  float *dk_part, *dv_part;   // several splits: [split][nk * kv_heads][d]
  int64_t nq, nk;
  int heads, kv_heads, shared, d;
  int splits, key_splits;     // ranges that a row tile's keys and a key tile's rows are cut into
  int key_units;              // backward: the first units are key tiles, the others row tiles
  int vec;                    // rows can be read four values at a time
  float scale;
};

constexpr int pitch_of(int columns) { return columns + 4; }

// values [c, c + 4) of a row of d, zeros past the end
template <typename T>
__device__ __forceinline__ float4 load4(const T* row, int c, int d, bool vec) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (vec) {
    if (c < d) {
      if constexpr (sizeof(T) == 4) {
        v = __ldg(reinterpret_cast<const float4*>(row + c));
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + c));
        v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                        __uint_as_float(u.y & 0xffff0000u));
      }
    }
    return v;
  }
  if (c < d) v.x = as_f32<T>(row[c]);
  if (c + 1 < d) v.y = as_f32<T>(row[c + 1]);
  if (c + 2 < d) v.z = as_f32<T>(row[c + 2]);
  if (c + 3 < d) v.w = as_f32<T>(row[c + 3]);
  return v;
}
template <typename T>
__device__ __forceinline__ void store4(void* dst, int64_t row, int c, int d, const float (&v)[4]) {
  T* const p = reinterpret_cast<T*>(dst) + row * d + c;
  if (d % 4 == 0) {
    if (c >= d) return;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < d) p[i] = from_f32<T>(v[i]);
}

// rows [r0, r0 + ROWS) of an item's (token, shared head) rows, zeros past the end;
// copies of fp32 rows are under way until copies_wait
template <typename T, int DP, int ROWS>
__device__ __forceinline__ void load_rows(const FmaArgs& a, float* dst, const HeadsView& t, int token0, int r0,
                                          int rows, int head0) {
  constexpr int kQuads = DP / 4;
  if constexpr (sizeof(T) == 4) {
    if (a.vec) {
#pragma unroll
      for (int e = threadIdx.x; e < ROWS * kQuads; e += kFmaThreads) {
        const int r = e / kQuads, c = (e % kQuads) * 4;
        const bool in = r0 + r < rows && c < a.d;
        const int at = in ? r0 + r : 0, tok = at / a.shared, g = at - tok * a.shared;
        tc::copy16(tc::smem_u32(dst + r * pitch_of(DP) + c),
                   reinterpret_cast<const T*>(t.p) + (int64_t)(token0 + tok) * t.token + (int64_t)(head0 + g) * t.head +
                       (in ? c : 0),
                   in);
      }
      return;
    }
  }
#pragma unroll
  for (int e = threadIdx.x; e < ROWS * kQuads; e += kFmaThreads) {
    const int r = e / kQuads, c = (e % kQuads) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r0 + r < rows) {
      const int tok = (r0 + r) / a.shared, g = (r0 + r) - tok * a.shared;
      v = load4<T>(reinterpret_cast<const T*>(t.p) + (int64_t)(token0 + tok) * t.token + (int64_t)(head0 + g) * t.head,
                   c, a.d, a.vec);
    }
    *reinterpret_cast<float4*>(dst + r * pitch_of(DP) + c) = v;
  }
}
// keys [j0, j0 + KEYS) of head h; a key that is masked or past the end reads as
// zeros (a masked one's row is fetched beside its mask, and not used)
template <typename T, int DP, int KEYS>
__device__ __forceinline__ void load_keys(const FmaArgs& a, float* dst, const HeadsView& t, int key0, int j0, int keys,
                                          int h) {
  constexpr int kQuads = DP / 4;
  if constexpr (sizeof(T) == 4) {
    if (a.vec) {
      constexpr int kTurns = KEYS * kQuads / kFmaThreads;
      static_assert(KEYS * kQuads % kFmaThreads == 0, "every thread copies as much");
      bool in[kTurns];
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int e = threadIdx.x + i * kFmaThreads;
        in[i] = j0 + e / kQuads < keys;
      }
      if (a.mask) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          const int j = (threadIdx.x + i * kFmaThreads) / kQuads;
          in[i] = in[i] && __ldg(a.mask + key0 + min(j0 + j, keys - 1));
        }
      }
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int e = threadIdx.x + i * kFmaThreads, j = e / kQuads, c = (e % kQuads) * 4;
        const bool here = in[i] && c < a.d;
        tc::copy16(tc::smem_u32(dst + j * pitch_of(DP) + c),
                   reinterpret_cast<const T*>(t.p) + (int64_t)(key0 + (here ? j0 + j : 0)) * t.token +
                       (int64_t)h * t.head + (here ? c : 0),
                   here);
      }
      return;
    }
  }
#pragma unroll
  for (int e = threadIdx.x; e < KEYS * kQuads; e += kFmaThreads) {
    const int j = e / kQuads, c = (e % kQuads) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j0 + j < keys) {
      const int64_t key = key0 + j0 + j;
      const bool keep = !a.mask || __ldg(a.mask + key);
      v = load4<T>(reinterpret_cast<const T*>(t.p) + key * t.token + (int64_t)h * t.head, c, a.d, a.vec);
      if (!keep) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    *reinterpret_cast<float4*>(dst + j * pitch_of(DP) + c) = v;
  }
}

// acc[i][j] = sum_d a[ty + 16 i][d] b[tx + 16 j][d]
template <int DP, int I, int J>
__device__ __forceinline__ void tile_dot(const float* a, const float* b, int ty, int tx, int d, float (&acc)[I][J]) {
  uint64_t sum[I][J];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) sum[i][j] = tc::pair(0.0f, 0.0f);
  a += ty * pitch_of(DP);
  b += tx * pitch_of(DP);
#pragma unroll 2
  for (int c = 0; c < d; c += 4) {
    ulonglong2 x[I], y[J];
#pragma unroll
    for (int i = 0; i < I; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(a + 16 * i * pitch_of(DP) + c);
#pragma unroll
    for (int j = 0; j < J; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(b + 16 * j * pitch_of(DP) + c);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) sum[i][j] = tc::fma2(x[i].y, y[j].y, tc::fma2(x[i].x, y[j].x, sum[i][j]));
  }
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float lo, hi;
      tc::unpair(sum[i][j], lo, hi);
      acc[i][j] = lo + hi;
    }
}

// acc[i][2 n], acc[i][2 n + 1]: pairs of the columns 4 tx + 64 n .. of row
// ty + 16 i; adds sum_t p[ty + 16 i][t] x[t][column] over t < count, where p (its
// rows PITCH apart) and x hold zeros up to a multiple of 4
template <int DP, int PITCH, int I>
__device__ __forceinline__ void tile_accumulate(const float* p, const float* x, int ty, int tx, int count,
                                                uint64_t (&acc)[I][DP / 32]) {
  p += ty * PITCH;
  x += 4 * tx;
  for (int t = 0; t < count; t += 4) {
    float4 u[I];
#pragma unroll
    for (int i = 0; i < I; ++i) u[i] = *reinterpret_cast<const float4*>(p + 16 * i * PITCH + t);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int n = 0; n < DP / 64; ++n) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(x + (t + k) * pitch_of(DP) + 64 * n);
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const float f = k == 0 ? u[i].x : k == 1 ? u[i].y : k == 2 ? u[i].z : u[i].w;
          const uint64_t ff = tc::pair(f, f);
          acc[i][2 * n] = tc::fma2(ff, w.x, acc[i][2 * n]);
          acc[i][2 * n + 1] = tc::fma2(ff, w.y, acc[i][2 * n + 1]);
        }
      }
    }
  }
}
template <int DP, int I>
__device__ __forceinline__ void clear(uint64_t (&acc)[I][DP / 32]) {
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int n = 0; n < DP / 32; ++n) acc[i][n] = tc::pair(0.0f, 0.0f);
}
// four columns of a row's results, times f
__device__ __forceinline__ void columns(uint64_t lo, uint64_t hi, float f, float (&v)[4]) {
  tc::unpair(lo, v[0], v[1]);
  tc::unpair(hi, v[2], v[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= f;
}

// true when key j0 + j of the item takes part
__device__ __forceinline__ bool kept(const FmaArgs& a, int key0, int j, int keys) {
  return j < keys && (!a.mask || a.mask[key0 + j]);
}

// reductions over the 16 threads that share a row
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct FmaUnit {
  int b, tile, h, split, q0, rows, key0, keys;
};
// Units of an item: tile fastest (neighbours read the same keys), then key
// head, then split.  `array` holds the items' first units.
template <int I, int J>
__device__ __forceinline__ FmaUnit fma_unit(const FmaArgs& a, int u, int array) {
  FmaUnit w;
  w.b = a.items.find(array, u);
  w.q0 = a.items.q0(w.b);
  w.rows = (a.items.q0(w.b + 1) - w.q0) * a.shared;
  w.key0 = a.items.k0(w.b);
  w.keys = a.items.k0(w.b + 1) - w.key0;
  const int tiles = array == kItemTile ? (w.keys + 16 * J - 1) / (16 * J) : (w.rows + 16 * I - 1) / (16 * I);
  int i = u - a.items.at(array, w.b);
  w.tile = i % tiles;
  i /= tiles;
  w.h = i % a.kv_heads;
  w.split = i / a.kv_heads;
  return w;
}
__device__ __forceinline__ int64_t row_of(const FmaArgs& a, const FmaUnit& w, int r) {
  const int tok = r / a.shared, g = r - tok * a.shared;
  return (int64_t)(w.q0 + tok) * a.heads + w.h * a.shared + g;
}

template <typename T, int DP, int I, int J>
__global__ void __launch_bounds__(kFmaThreads, DP > 64 && I * J > 8 ? 1 : 2) k_attn_fma(const __grid_constant__ FmaArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int kRows = 16 * I * pitch_of(DP), kKeys = 16 * J * pitch_of(DP), kScorePitch = pitch_of(16 * J);
  float *qs = sm, *ks = qs + kRows, *vs = ks + kKeys, *ps = vs + kKeys;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const FmaUnit w = fma_unit<I, J>(a, blockIdx.x, kItemUnit);
  const int r0 = w.tile * 16 * I;
  load_rows<T, DP, 16 * I>(a, qs, a.q, w.q0, r0, w.rows, w.h * a.shared);
  uint64_t acc[I][DP / 32];
  clear<DP>(acc);
  float top[I], total[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    top[i] = -INFINITY;
    total[i] = 0.0f;
  }
  const int kt = (w.keys + 16 * J - 1) / (16 * J);
  const int t0 = (int)((int64_t)kt * w.split / a.splits), t1 = (int)((int64_t)kt * (w.split + 1) / a.splits);
  for (int t = t0; t < t1; ++t) {
    const int j0 = t * 16 * J;
    __syncthreads();
    load_keys<T, DP, 16 * J>(a, ks, a.k, w.key0, j0, w.keys, w.h);
    load_keys<T, DP, 16 * J>(a, vs, a.v, w.key0, j0, w.keys, w.h);
    bool keep[J];
#pragma unroll
    for (int j = 0; j < J; ++j) keep[j] = kept(a, w.key0, j0 + tx + 16 * j, w.keys);
    tc::copies_wait();
    __syncthreads();
    float s[I][J];
    tile_dot<DP, I, J>(qs, ks, ty, tx, a.d, s);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[i][j] = keep[j] ? s[i][j] * a.scale : -INFINITY;
        m = fmaxf(m, s[i][j]);
      }
      m = fmaxf(max16(m), top[i]);
      const float base = m == -INFINITY ? 0.0f : m;  // nothing kept so far: every exp below is 0
      const float fade = expf(top[i] - base);
      float add = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[i][j] = expf(s[i][j] - base);
        add += s[i][j];
        ps[(ty + 16 * i) * kScorePitch + tx + 16 * j] = s[i][j];
      }
      top[i] = m;
      total[i] = total[i] * fade + sum16(add);
#pragma unroll
      for (int n = 0; n < DP / 32; ++n) acc[i][n] = tc::mul2(acc[i][n], tc::pair(fade, fade));
    }
    __syncthreads();
    tile_accumulate<DP, kScorePitch>(ps, vs, ty, tx, min(16 * J, w.keys - j0), acc);
  }
  tc::copies_wait();  // of a range without tiles
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int r = r0 + ty + 16 * i;
    if (r >= w.rows) continue;
    const int64_t row = row_of(a, w, r);
    float v[4];
    if (a.splits == 1) {
      const float inv = total[i] > 0.0f ? 1.0f / total[i] : 0.0f;
      if (tx == 0) a.lse[row] = top[i] + logf(total[i]);
#pragma unroll
      for (int n = 0; n < DP / 64; ++n) {
        columns(acc[i][2 * n], acc[i][2 * n + 1], inv, v);
        store4<T>(a.out, row, 4 * tx + 64 * n, a.d, v);
      }
    } else {
      const int64_t at = (int64_t)w.split * a.nq * a.heads + row;
      if (tx == 0) {
        a.top[at] = top[i];
        a.total[at] = total[i];
      }
#pragma unroll
      for (int n = 0; n < DP / 64; ++n) {
        columns(acc[i][2 * n], acc[i][2 * n + 1], 1.0f, v);
        store4<float>(a.part, at, 4 * tx + 64 * n, a.d, v);
      }
    }
  }
}

// p and ds of one tile: s and dp in, both overwritten
template <int I, int J>
__device__ __forceinline__ void tile_gradient(const FmaArgs& a, float (&s)[I][J], float (&dp)[I][J],
                                              const bool (&keep)[J], const float (&lse)[I], const float (&delta)[I]) {
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float p = keep[j] && lse[i] != -INFINITY ? expf(s[i][j] * a.scale - lse[i]) : 0.0f;
      s[i][j] = p;
      dp[i][j] = p * (dp[i][j] - delta[i]) * a.scale;
    }
}
__device__ __forceinline__ void row_constants(const FmaArgs& a, const FmaUnit& w, int r, float* lse, float* delta) {
  *lse = -INFINITY;
  *delta = 0.0f;
  if (r < w.rows) {
    const int64_t row = row_of(a, w, r);
    *lse = __ldg(a.lse_in + row);
    *delta = __ldg(a.delta + row);
  }
}

// dq of one tile of rows over a range of key tiles
template <typename T, int DP, int I, int J>
__device__ __forceinline__ void fma_dq(const FmaArgs& a, float* sm, int unit) {
  constexpr int kRows = 16 * I * pitch_of(DP), kKeys = 16 * J * pitch_of(DP), kScorePitch = pitch_of(16 * J);
  float *qs = sm, *os = qs + kRows, *ks = os + kRows, *vs = ks + kKeys, *ps = vs + kKeys;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const FmaUnit w = fma_unit<I, J>(a, unit, kItemUnit);
  const int r0 = w.tile * 16 * I;
  load_rows<T, DP, 16 * I>(a, qs, a.q, w.q0, r0, w.rows, w.h * a.shared);
  load_rows<T, DP, 16 * I>(a, os, a.dout, w.q0, r0, w.rows, w.h * a.shared);
  uint64_t acc[I][DP / 32];
  clear<DP>(acc);
  float lse[I], delta[I];
#pragma unroll
  for (int i = 0; i < I; ++i) row_constants(a, w, r0 + ty + 16 * i, &lse[i], &delta[i]);
  const int kt = (w.keys + 16 * J - 1) / (16 * J);
  const int t0 = (int)((int64_t)kt * w.split / a.splits), t1 = (int)((int64_t)kt * (w.split + 1) / a.splits);
  for (int t = t0; t < t1; ++t) {
    const int j0 = t * 16 * J;
    __syncthreads();
    load_keys<T, DP, 16 * J>(a, ks, a.k, w.key0, j0, w.keys, w.h);
    load_keys<T, DP, 16 * J>(a, vs, a.v, w.key0, j0, w.keys, w.h);
    bool keep[J];
#pragma unroll
    for (int j = 0; j < J; ++j) keep[j] = kept(a, w.key0, j0 + tx + 16 * j, w.keys);
    tc::copies_wait();
    __syncthreads();
    float s[I][J], dp[I][J];
    tile_dot<DP, I, J>(qs, ks, ty, tx, a.d, s);
    tile_dot<DP, I, J>(os, vs, ty, tx, a.d, dp);
    tile_gradient(a, s, dp, keep, lse, delta);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) ps[(ty + 16 * i) * kScorePitch + tx + 16 * j] = dp[i][j];
    __syncthreads();
    tile_accumulate<DP, kScorePitch>(ps, ks, ty, tx, min(16 * J, w.keys - j0), acc);
  }
  tc::copies_wait();  // of a range without tiles
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int r = r0 + ty + 16 * i;
    if (r >= w.rows) continue;
    const int64_t row = row_of(a, w, r);
#pragma unroll
    for (int n = 0; n < DP / 64; ++n) {
      float v[4];
      columns(acc[i][2 * n], acc[i][2 * n + 1], 1.0f, v);
      if (a.splits == 1) store4<T>(a.out, row, 4 * tx + 64 * n, a.d, v);
      else store4<float>(a.part, (int64_t)w.split * a.nq * a.heads + row, 4 * tx + 64 * n, a.d, v);
    }
  }
}

// dk and dv of one tile of keys over a range of row tiles; the scores go to
// shared memory with the keys in rows
template <typename T, int DP, int I, int J>
__device__ __forceinline__ void fma_dkv(const FmaArgs& a, float* sm, int unit) {
  constexpr int kRows = 16 * I * pitch_of(DP), kKeys = 16 * J * pitch_of(DP), kScorePitch = pitch_of(16 * I);
  float *qs = sm, *os = qs + kRows, *ks = os + kRows, *vs = ks + kKeys, *ps = vs + kKeys,
        *ds = ps + 16 * J * kScorePitch;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const FmaUnit w = fma_unit<I, J>(a, unit, kItemTile);
  const int j0 = w.tile * 16 * J;
  load_keys<T, DP, 16 * J>(a, ks, a.k, w.key0, j0, w.keys, w.h);
  load_keys<T, DP, 16 * J>(a, vs, a.v, w.key0, j0, w.keys, w.h);
  uint64_t dk[J][DP / 32], dv[J][DP / 32];
  clear<DP>(dk);
  clear<DP>(dv);
  bool keep[J], keep_out[J];  // of the scores' columns, of the rows written
#pragma unroll
  for (int i = 0; i < J; ++i) {
    keep[i] = kept(a, w.key0, j0 + tx + 16 * i, w.keys);
    keep_out[i] = kept(a, w.key0, j0 + ty + 16 * i, w.keys);
  }
  const int rt = (w.rows + 16 * I - 1) / (16 * I);
  const int t0 = (int)((int64_t)rt * w.split / a.key_splits), t1 = (int)((int64_t)rt * (w.split + 1) / a.key_splits);
  for (int t = t0; t < t1; ++t) {
    const int r0 = t * 16 * I;
    __syncthreads();
    load_rows<T, DP, 16 * I>(a, qs, a.q, w.q0, r0, w.rows, w.h * a.shared);
    load_rows<T, DP, 16 * I>(a, os, a.dout, w.q0, r0, w.rows, w.h * a.shared);
    float lse[I], delta[I];
#pragma unroll
    for (int i = 0; i < I; ++i) row_constants(a, w, r0 + ty + 16 * i, &lse[i], &delta[i]);
    tc::copies_wait();
    __syncthreads();
    float s[I][J], dp[I][J];
    tile_dot<DP, I, J>(qs, ks, ty, tx, a.d, s);
    tile_dot<DP, I, J>(os, vs, ty, tx, a.d, dp);
    tile_gradient(a, s, dp, keep, lse, delta);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        ps[(tx + 16 * j) * kScorePitch + ty + 16 * i] = s[i][j];
        ds[(tx + 16 * j) * kScorePitch + ty + 16 * i] = dp[i][j];
      }
    __syncthreads();
    const int count = min(16 * I, w.rows - r0);
    tile_accumulate<DP, kScorePitch>(ps, os, ty, tx, count, dv);
    tile_accumulate<DP, kScorePitch>(ds, qs, ty, tx, count, dk);
  }
  tc::copies_wait();  // of a range without tiles
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int j = j0 + ty + 16 * i;
    if (j >= w.keys) continue;
    const int64_t row = (int64_t)(w.key0 + j) * a.kv_heads + w.h, at = (int64_t)w.split * a.nk * a.kv_heads + row;
#pragma unroll
    for (int n = 0; n < DP / 64; ++n) {
      float v[4], u[4];
      columns(dk[i][2 * n], dk[i][2 * n + 1], 1.0f, v);
      columns(dv[i][2 * n], dv[i][2 * n + 1], 1.0f, u);
      if (!keep_out[i]) v[0] = v[1] = v[2] = v[3] = u[0] = u[1] = u[2] = u[3] = 0.0f;
      if (a.key_splits == 1) {
        store4<T>(a.dk, row, 4 * tx + 64 * n, a.d, v);
        store4<T>(a.dv, row, 4 * tx + 64 * n, a.d, u);
      } else {
        store4<float>(a.dk_part, at, 4 * tx + 64 * n, a.d, v);
        store4<float>(a.dv_part, at, 4 * tx + 64 * n, a.d, u);
      }
    }
  }
}

// The blocks of the key tiles, which take longer, come first.
template <typename T, int DP, int I, int J>
__global__ void __launch_bounds__(kFmaThreads, DP > 64 && I * J > 4 ? 1 : 2) k_attn_fma_bwd(const __grid_constant__ FmaArgs a) {
  extern __shared__ __align__(16) float sm[];
  if ((int)blockIdx.x < a.key_units) fma_dkv<T, DP, I, J>(a, sm, blockIdx.x);
  else fma_dq<T, DP, I, J>(a, sm, blockIdx.x - a.key_units);
}

// ---------------------------------------------------------------- reductions
// One warp per row: the partial results over ranges of keys, each relative to
// its own maximum, brought to the common one and divided by the common sum.
template <typename T>
__global__ void __launch_bounds__(kFmaThreads) k_attn_join(const float* __restrict__ part,
                                                           const float* __restrict__ top,
                                                           const float* __restrict__ total, int splits, int64_t rows,
                                                           int d, T* __restrict__ out, float* __restrict__ lse) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kFmaThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, __ldg(top + s * rows + row));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  float acc[kMaxD / 32] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < splits; ++s) {
    const float f = expf(__ldg(top + s * rows + row) - base), t = __ldg(total + s * rows + row);
    if (t == 0.0f) continue;  // no kept key in this range; a NaN goes on
    l = fmaf(f, t, l);
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i)
      if (lane + 32 * i < d) acc[i] = fmaf(f, __ldg(part + (s * rows + row) * d + lane + 32 * i), acc[i]);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  if (lane == 0) lse[row] = m + logf(l);
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i)
    if (lane + 32 * i < d) out[row * d + lane + 32 * i] = from_f32<T>(acc[i] * inv);
}

// Up to three arrays (blockIdx.y), each the sum of partial results in their order.
struct SumArgs {
  const float* part[3];
  void* dst[3];
  int64_t n[3];
  int splits[3];
};
template <typename T>
__global__ void __launch_bounds__(kFmaThreads) k_attn_sum(const __grid_constant__ SumArgs a) {
  const float* const part = a.part[blockIdx.y];
  const int64_t n = a.n[blockIdx.y];
  T* const dst = reinterpret_cast<T*>(a.dst[blockIdx.y]);
  const int splits = a.splits[blockIdx.y];
  for (int64_t i = (int64_t)blockIdx.x * kFmaThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kFmaThreads) {
    float s = 0.0f;
#pragma unroll 8
    for (int k = 0; k < splits; ++k) s += __ldg(part + k * n + i);
    dst[i] = from_f32<T>(s);
  }
}

// delta of each row: one warp per row, dout and out dense along d
template <typename T>
__global__ void __launch_bounds__(kFmaThreads) k_attn_delta(HeadsView dout, const T* __restrict__ out, int64_t rows,
                                                            int heads, int d, float* __restrict__ delta) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kFmaThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int64_t tok = row / heads;
  const int h = (int)(row - tok * heads);
  const T* p = reinterpret_cast<const T*>(dout.p) + tok * dout.token + h * dout.head;
  float s = 0.0f;
  for (int c = lane; c < d; c += 32) s = fmaf(as_f32<T>(p[c]), as_f32<T>(out[row * d + c]), s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) delta[row] = s;
}

// Offsets of more items than the arguments hold, written a piece at a time.
struct Piece {
  int32_t v[960];
};
__global__ void k_attn_offsets(const __grid_constant__ Piece p, int n, int32_t* dst) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = p.v[i];
}

// ---------------------------------------------------------------- host
fvx_status bad(const char* who, const char* what) {
  set_error("%s: %s", who, what);
  return FVX_ERR_INVALID_ARG;
}

size_t elem_size(fvx_dtype dt) { return dt == FVX_F32 ? 4 : 2; }

fvx_status check_offsets(const char* who, const char* name, const int64_t* o, int32_t B, int64_t* total) {
  if (!o) {
    set_error("%s: NULL %s", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  if (o[0] != 0) {
    set_error("%s: %s must start at 0", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  for (int b = 0; b < B; ++b)
    if (o[b + 1] < o[b]) {
      set_error("%s: %s must be monotone", who, name);
      return FVX_ERR_INVALID_ARG;
    }
  *total = o[B];
  return FVX_OK;
}

fvx_status check_heads(const char* who, const char* name, fvx_dtype dt, const HeadsView& t, int64_t n) {
  if ((n > 0 && !t.p) || reinterpret_cast<uintptr_t>(t.p) % elem_size(dt)) {
    set_error("%s: %s is NULL or not aligned to its elements", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  if (t.token < 0 || t.head < 0) {
    set_error("%s: %s has a negative stride", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  return FVX_OK;
}

fvx_status check_call(const char* who, AttnCall& c, int32_t B, int32_t heads, int32_t kv_heads, int32_t d) {
  if (c.dt != FVX_F32 && c.dt != FVX_BF16) return bad(who, "dtype must be FVX_F32 or FVX_BF16");
  if (B < 1) return bad(who, "B must be at least 1");
  if (heads < 1 || kv_heads < 1 || heads % kv_heads) return bad(who, "heads must be a positive multiple of kv_heads");
  if (d < 1 || d > kMaxD) return bad(who, "the head size must be in 1..128");
  if (!(fabsf(c.scale) <= 3.0e38f)) return bad(who, "scale must be finite");
  FVX_TRY(check_offsets(who, "q_offsets", c.q_offsets, B, &c.nq));
  FVX_TRY(check_offsets(who, "kv_offsets", c.kv_offsets, B, &c.nk));
  c.items = B;
  c.heads = heads;
  c.kv_heads = kv_heads;
  c.shared = heads / kv_heads;
  c.d = d;
  // rows and work units are counted in 32 bits
  if (c.nq > ((int64_t)1 << 30) / heads || c.nk > ((int64_t)1 << 30) / kv_heads) {
    set_error("%s: more than 2^30 rows (tokens times heads)", who);
    return FVX_ERR_RANGE;
  }
  // the stride of a dimension of one element says nothing
  auto dense = [&](HeadsView& t, int64_t tokens, int h) {
    if (h == 1) t.head = d;
    if (tokens <= 1) t.token = (int64_t)h * d;
  };
  dense(c.q, c.nq, heads);
  dense(c.dout, c.nq, heads);
  dense(c.k, c.nk, kv_heads);
  dense(c.v, c.nk, kv_heads);
  FVX_TRY(check_heads(who, "q", c.dt, c.q, c.nq));
  FVX_TRY(check_heads(who, "k", c.dt, c.k, c.nk));
  FVX_TRY(check_heads(who, "v", c.dt, c.v, c.nk));
  if (c.nq > 0 && (!c.out || !c.lse)) return bad(who, "NULL out or lse");
  if (reinterpret_cast<uintptr_t>(c.out) % 16) return bad(who, "out is not aligned to 16 bytes");
  if (reinterpret_cast<uintptr_t>(c.lse) % 4) return bad(who, "lse is not aligned to 4 bytes");
  return FVX_OK;
}

// Rows and keys of a tile.
struct FmaTile {
  int rows, keys;
};
// Prefix of the items' units; `splits` gives each tile that many.
std::vector<int32_t> unit_prefix(const AttnCall& c, FmaTile t, bool by_keys, int splits, int64_t* units) {
  std::vector<int32_t> p((size_t)c.items + 1);
  int64_t n = 0;
  const int tile = by_keys ? t.keys : t.rows;
  for (int b = 0; b < c.items; ++b) {
    p[b] = (int32_t)n;
    const int64_t len = by_keys ? c.kv_offsets[b + 1] - c.kv_offsets[b] : (c.q_offsets[b + 1] - c.q_offsets[b]) * c.shared;
    n += (len + tile - 1) / tile * c.kv_heads * splits;
  }
  p[c.items] = (int32_t)n;
  *units = n;
  return p;
}

// Splits of the inner loops, at most 32, with the least time in tiles: that of
// the longest unit while the units that have work (a sample's loop has no more
// ranges than tiles) fit one wave of two blocks per multiprocessor, past that
// their share and half the longest unit; a unit's start and end and the kernel
// that adds the ranges up (`join`; backward, one for all three gradients) count as
// tiles.  9 samples of 8 to 26 rows on 1400 to
// 2600 keys, 5 key heads of 100: 6 splits, 270 units, 107 us; 7, 315 units, 151.
int pick_splits(const AttnCall& c, FmaTile t, bool by_keys, int sms, double join) {
  constexpr double kEnds = 2.0;
  const int outer = by_keys ? t.keys : t.rows, inner = by_keys ? t.rows : t.keys;
  int splits = 1;
  double best = 1e300;
  for (int s = 1; s <= 32; ++s) {
    int64_t units = 0, longest = 0, tiles = 0;
    for (int b = 0; b < c.items; ++b) {
      const int64_t rows = (c.q_offsets[b + 1] - c.q_offsets[b]) * c.shared, keys = c.kv_offsets[b + 1] - c.kv_offsets[b];
      const int64_t loop = ((by_keys ? rows : keys) + inner - 1) / inner;
      const int64_t n = ((by_keys ? keys : rows) + outer - 1) / outer * c.kv_heads;
      units += n * std::min<int64_t>(s, loop);
      tiles += n * loop;
      if (n > 0) longest = std::max(longest, (loop + s - 1) / s);
    }
    const double unit = (double)longest + kEnds, wave = 2.0 * sms;
    const double time = (units <= wave ? unit : ((double)tiles + kEnds * (double)units) / wave + 0.5 * unit) +
                        (s > 1 ? join : 0.0);
    if (time < best) {
      best = time;
      splits = s;
    }
    if (longest <= 1 || (double)units > 4.0 * wave) break;  // more ranges than that are never the least
  }
  return splits;
}

// four values at a time: 16 bytes of fp32, 8 of bf16
bool loads4(const AttnCall& c, const HeadsView& t) {
  return reinterpret_cast<uintptr_t>(t.p) % (4 * elem_size(c.dt)) == 0 && t.token % 4 == 0 && t.head % 4 == 0;
}

FmaArgs fma_args(const AttnCall& c) {
  FmaArgs a = {};
  a.q = c.q;
  a.k = c.k;
  a.v = c.v;
  a.dout = c.dout;
  a.mask = c.mask;
  a.nq = c.nq;
  a.nk = c.nk;
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.shared = c.shared;
  a.d = c.d;
  a.vec = c.d % 4 == 0 && loads4(c, c.q) && loads4(c, c.k) && loads4(c, c.v) && loads4(c, c.dout);
  a.scale = c.scale;
  return a;
}

template <auto kernel>
fvx_status fma_launch(const char* name, int64_t units, size_t smem, cudaStream_t s, const FmaArgs& a) {
  static std::atomic<uint64_t> allowed{0};
  FVX_TRY(allow_smem((const void*)kernel, (int)smem, allowed));
  LaunchScope ls(name, s);
  kernel<<<(unsigned)units, kFmaThreads, smem, s>>>(a);
  return check_launch(name);
}
// bytes of tiles of rows and of keys and of `scores` tiles of scores
constexpr size_t fma_smem(int dp, FmaTile t, int row_tiles, int key_tiles, int scores) {
  const int score = std::max(t.rows * pitch_of(t.keys), t.keys * pitch_of(t.rows));
  return (size_t)((t.rows * row_tiles + t.keys * key_tiles) * pitch_of(dp) + scores * score) * 4;
}

template <typename T, int DP, int I, int J>
fvx_status fma_forward(const AttnCall& c, cudaStream_t s, Scratch& scr, int sms) {
  constexpr FmaTile tile{16 * I, 16 * J};
  FmaArgs a = fma_args(c);
  a.splits = pick_splits(c, tile, false, sms, 2.0);
  int64_t units = 0;
  const std::vector<int32_t> prefix = unit_prefix(c, tile, false, a.splits, &units);
  FVX_TRY(attn_items(c, prefix.data(), 3, s, scr, &a.items));
  a.out = c.out;
  a.lse = c.lse;
  const int64_t rows = c.nq * c.heads;
  if (a.splits > 1) {
    a.part = scr.get<float>((size_t)a.splits * rows * c.d);
    a.top = scr.get<float>((size_t)a.splits * rows);
    a.total = scr.get<float>((size_t)a.splits * rows);
    if (!a.part || !a.top || !a.total) return FVX_ERR_ALLOC;
  }
  constexpr auto kernel = k_attn_fma<T, DP, I, J>;
  FVX_TRY(fma_launch<kernel>("attn_fma", units, fma_smem(DP, tile, 1, 2, 1), s, a));
  return a.splits > 1 ? attn_join(c, a.part, a.top, a.total, a.splits, s) : FVX_OK;
}

template <typename T, int DP, int I, int J>
fvx_status fma_backward(const AttnCall& c, const float* delta, cudaStream_t s, Scratch& scr, int sms) {
  constexpr FmaTile tile{16 * I, 16 * J};
  FmaArgs a = fma_args(c);
  a.delta = delta;
  a.lse_in = c.lse;
  a.out = c.dq;
  a.dk = c.dk;
  a.dv = c.dv;
  a.splits = pick_splits(c, tile, false, sms, 0.5);
  a.key_splits = pick_splits(c, tile, true, sms, 0.5);
  int64_t row_units = 0, key_units = 0;
  std::vector<int32_t> prefix = unit_prefix(c, tile, false, a.splits, &row_units);
  const std::vector<int32_t> by_keys = unit_prefix(c, tile, true, a.key_splits, &key_units);
  prefix.insert(prefix.end(), by_keys.begin(), by_keys.end());
  FVX_TRY(attn_items(c, prefix.data(), 4, s, scr, &a.items));
  a.key_units = (int)key_units;
  const int64_t q_values = c.nq * c.heads * c.d, k_values = c.nk * c.kv_heads * c.d;
  if (a.splits > 1 && !(a.part = scr.get<float>((size_t)a.splits * q_values))) return FVX_ERR_ALLOC;
  if (a.key_splits > 1 && k_values > 0) {
    a.dk_part = scr.get<float>((size_t)a.key_splits * k_values);
    a.dv_part = scr.get<float>((size_t)a.key_splits * k_values);
    if (!a.dk_part || !a.dv_part) return FVX_ERR_ALLOC;
  }
  constexpr auto kernel = k_attn_fma_bwd<T, DP, I, J>;
  FVX_TRY(fma_launch<kernel>("attn_fma_bwd", key_units + row_units, fma_smem(DP, tile, 2, 2, 2), s, a));
  SumArgs sum = {};
  int arrays = 0;
  auto add = [&](const float* part, void* dst, int64_t n, int splits) {
    if (splits == 1 || n == 0) return;
    sum.part[arrays] = part;
    sum.dst[arrays] = dst;
    sum.n[arrays] = n;
    sum.splits[arrays++] = splits;
  };
  add(a.part, c.dq, q_values, a.splits);
  add(a.dk_part, c.dk, k_values, a.key_splits);
  add(a.dv_part, c.dv, k_values, a.key_splits);
  if (arrays == 0) return FVX_OK;
  const int64_t longest = std::max(sum.n[0], std::max(sum.n[1], sum.n[2]));
  const dim3 grid((unsigned)std::min<int64_t>((longest + kFmaThreads - 1) / kFmaThreads, sms * 16), (unsigned)arrays);
  LaunchScope ls("attn_sum", s);
  k_attn_sum<T><<<grid, kFmaThreads, 0, s>>>(sum);
  return check_launch("attn_sum");
}

// Calls f with the type, the head's size rounded up and the tile: 16 or 32 rows
// or 16 keys where no sample has more of them.  That tile or 64 x 64, forward and
// backward: 9 samples of 4 to 12 rows on 1400 to 2600 keys, 2 heads of 64, 36 or
// 46 us and 60 or 81; 32 rows on 7400 keys, 4 heads of 128, 52 or 60 and 101 or
// 128; 4600 rows on 16 keys, 4 heads of 64, 12 or 14 and 42 or 58 (17 keys, 64 x
// 64: 14 and 58).
//
// bf16 heads that are no multiple of 8 come here as well, since neither TMA nor
// 16-byte loads read their rows: 9014 rows on 500 keys, 8 heads of 100, 829 and
// 2272 us, 17 TFLOP/s (8 heads of 104 on the tensor cores: 33 and 132).  Their
// probabilities stay fp32.
template <typename F>
fvx_status by_shape(const AttnCall& c, F&& f) {
  if (c.dt != FVX_F32)
    return c.d <= 64 ? f.template operator()<__nv_bfloat16, 64, 4, 4>() : f.template operator()<__nv_bfloat16, 128, 4, 4>();
  int64_t rows = 0, keys = 0;
  for (int b = 0; b < c.items; ++b) {
    rows = std::max(rows, (c.q_offsets[b + 1] - c.q_offsets[b]) * c.shared);
    keys = std::max(keys, c.kv_offsets[b + 1] - c.kv_offsets[b]);
  }
  auto with = [&]<int DP>() {
    if (keys <= 16 && rows > 16) return f.template operator()<float, DP, 4, 1>();
    if (rows <= 16) return f.template operator()<float, DP, 1, 4>();
    if (rows <= 32) return f.template operator()<float, DP, 2, 4>();
    return f.template operator()<float, DP, 4, 4>();
  };
  return c.d <= 64 ? with.template operator()<64>() : with.template operator()<128>();
}

}  // namespace

fvx_status attn_items(const AttnCall& c, const int32_t* more, int arrays, cudaStream_t s, Scratch& scr,
                      AttnItems* out) {
  const int n = c.items + 1;
  out->items = c.items;
  out->ptr = nullptr;
  auto value = [&](int i) {
    return i < n ? (int32_t)c.q_offsets[i] : i < 2 * n ? (int32_t)c.kv_offsets[i - n] : more[i - 2 * n];
  };
  if (c.items <= kInlineItems) {
    for (int i = 0; i < arrays * n; ++i) out->in[i] = value(i);
    return FVX_OK;
  }
  int32_t* dev = scr.get<int32_t>((size_t)arrays * n);
  if (!dev) return FVX_ERR_ALLOC;
  constexpr int kPiece = (int)(sizeof(Piece) / 4);
  for (int i = 0; i < arrays * n; i += kPiece) {
    Piece p;
    const int m = std::min(kPiece, arrays * n - i);
    for (int j = 0; j < m; ++j) p.v[j] = value(i + j);
    LaunchScope ls("attn_offsets", s);
    k_attn_offsets<<<1, kFmaThreads, 0, s>>>(p, m, dev + i);
    FVX_TRY(check_launch("attn_offsets"));
  }
  out->ptr = dev;
  return FVX_OK;
}

fvx_status attn_join(const AttnCall& c, const float* part, const float* top, const float* total, int splits,
                     cudaStream_t s) {
  const int64_t rows = c.nq * c.heads;
  const unsigned grid = (unsigned)((rows + kFmaThreads / 32 - 1) / (kFmaThreads / 32));
  LaunchScope ls("attn_join", s);
  if (c.dt == FVX_F32)
    k_attn_join<float><<<grid, kFmaThreads, 0, s>>>(part, top, total, splits, rows, c.d, (float*)c.out, c.lse);
  else
    k_attn_join<__nv_bfloat16>
        <<<grid, kFmaThreads, 0, s>>>(part, top, total, splits, rows, c.d, (__nv_bfloat16*)c.out, c.lse);
  return check_launch("attn_join");
}

}  // namespace fvx

using namespace fvx;

extern "C" {

fvx_status fvx_cross_attention(fvx_dtype dt, const void* q, int64_t q_token, int64_t q_head, const void* k,
                               int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                               const int64_t* q_offsets, const int64_t* kv_offsets, int32_t B, int32_t heads,
                               int32_t kv_heads, int32_t d, const uint8_t* key_mask, float scale, void* out,
                               float* lse, fvx_stream stream) {
  const char* who = "fvx_cross_attention";
  EntryScope entry(who);
  try {
    AttnCall c = {};
    c.dt = dt;
    c.q = HeadsView{q, q_token, q_head};
    c.k = HeadsView{k, k_token, k_head};
    c.v = HeadsView{v, v_token, v_head};
    c.q_offsets = q_offsets;
    c.kv_offsets = kv_offsets;
    c.mask = key_mask;
    c.scale = scale;
    c.out = out;
    c.lse = lse;
    FVX_TRY(check_call(who, c, B, heads, kv_heads, d));
    if (c.nq == 0) return FVX_OK;
    cudaStream_t s = (cudaStream_t)stream;
    int sms = 0;
    FVX_TRY(device_sm_count(&sms));
    Scratch scr(s);
    if (attn_few_serves(c)) return attn_few_forward(c, s, scr);
    if (attn_tc_serves(c, false)) return attn_tc_forward(c, s, scr);
    return by_shape(c, [&]<typename T, int DP, int I, int J>() { return fma_forward<T, DP, I, J>(c, s, scr, sms); });
  } catch (const std::exception& e) {
    set_error("%s: %s", who, e.what());
    return FVX_ERR_ALLOC;
  }
}

fvx_status fvx_cross_attention_backward(fvx_dtype dt, const void* dout, int64_t do_token, int64_t do_head,
                                        const void* q, int64_t q_token, int64_t q_head, const void* k,
                                        int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                                        int64_t v_head, const void* out, const float* lse, const int64_t* q_offsets,
                                        const int64_t* kv_offsets, int32_t B, int32_t heads, int32_t kv_heads,
                                        int32_t d, const uint8_t* key_mask, float scale, void* dq, void* dk, void* dv,
                                        fvx_stream stream) {
  const char* who = "fvx_cross_attention_backward";
  EntryScope entry(who);
  try {
    AttnCall c = {};
    c.dt = dt;
    c.q = HeadsView{q, q_token, q_head};
    c.k = HeadsView{k, k_token, k_head};
    c.v = HeadsView{v, v_token, v_head};
    c.dout = HeadsView{dout, do_token, do_head};
    c.q_offsets = q_offsets;
    c.kv_offsets = kv_offsets;
    c.mask = key_mask;
    c.scale = scale;
    c.out = const_cast<void*>(out);
    c.lse = const_cast<float*>(lse);
    c.dq = dq;
    c.dk = dk;
    c.dv = dv;
    FVX_TRY(check_call(who, c, B, heads, kv_heads, d));
    FVX_TRY(check_heads(who, "dout", dt, c.dout, c.nq));
    if ((c.nq > 0 && !dq) || (c.nk > 0 && (!dk || !dv))) return bad(who, "NULL dq, dk or dv");
    if (reinterpret_cast<uintptr_t>(dq) % 16 || reinterpret_cast<uintptr_t>(dk) % 16 ||
        reinterpret_cast<uintptr_t>(dv) % 16)
      return bad(who, "dq, dk or dv is not aligned to 16 bytes");
    cudaStream_t s = (cudaStream_t)stream;
    const size_t kv_bytes = (size_t)c.nk * kv_heads * d * elem_size(dt);
    if (c.nq == 0) {
      if (c.nk > 0) {
        FVX_CUDA(cudaMemsetAsync(dk, 0, kv_bytes, s));
        FVX_CUDA(cudaMemsetAsync(dv, 0, kv_bytes, s));
      }
      return FVX_OK;
    }
    int sms = 0;
    FVX_TRY(device_sm_count(&sms));
    Scratch scr(s);
    if (attn_tc_serves(c, true)) return attn_tc_backward(c, s, scr);
    const int64_t rows = c.nq * heads;
    float* delta = scr.get<float>((size_t)rows);
    if (!delta) return FVX_ERR_ALLOC;
    {
      const unsigned grid = (unsigned)((rows + kFmaThreads / 32 - 1) / (kFmaThreads / 32));
      LaunchScope ls("attn_delta", s);
      if (dt == FVX_F32)
        k_attn_delta<float><<<grid, kFmaThreads, 0, s>>>(c.dout, (const float*)out, rows, heads, d, delta);
      else
        k_attn_delta<__nv_bfloat16>
            <<<grid, kFmaThreads, 0, s>>>(c.dout, (const __nv_bfloat16*)out, rows, heads, d, delta);
      FVX_TRY(check_launch("attn_delta"));
    }
    return by_shape(c, [&]<typename T, int DP, int I, int J>() {
      return fma_backward<T, DP, I, J>(c, delta, s, scr, sms);
    });
  } catch (const std::exception& e) {
    set_error("%s: %s", who, e.what());
    return FVX_ERR_ALLOC;
  }
}

}  // extern "C"
