// Layer norm over voxel features (forward and backward) and activation
// checkpoints in 8 bits.
//
// Forward, per row x[0..C):   mean = sum x / C;  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//                             y = (x - mean) rstd w + b
// Backward, xh = (x - mean) rstd and g = dy w:
//                             dx = rstd (g - sum(g) / C - xh sum(g xh) / C)
//                             dw = sum over rows of dy xh;  db = sum over rows of dy
// Checkpoint, per group of G channels of a row: top = max |x|, step = top / 127,
// code = round-half-even(x (127 / top)), the value held is code * step.  A group
// with top < 2^-100 holds zeros; a group with an infinity or a NaN holds NaN, so
// that an overflow is still seen by whoever reads the values back.
//
// All of it moves a few bytes per value and computes a few operations on them:
// memory bounds it.  So each row is read once, stays in registers between its
// two reductions, and the checkpoint is written by the pass that reads x.
// Statistics, products and sums are fp32 whatever the storage type.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fvx_internal.cuh"

namespace fvx {
namespace {

constexpr int kThreads = 256;
constexpr int kRegCols = 1024;      // widest row held in a warp's registers
constexpr int64_t kMaxCols = 65536;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  const Pack<T, VEC> u = *reinterpret_cast<const Pack<T, VEC>*>(p);
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = Elem<T>::get(u.v[j]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  Pack<T, VEC> u;
#pragma unroll
  for (int j = 0; j < VEC; ++j) u.v[j] = Elem<T>::put(f[j]);
  *reinterpret_cast<Pack<T, VEC>*>(p) = u;
}

// Sum over the `width` lanes (a power of two) that share a row.
__device__ __forceinline__ float lanes_sum(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Magnitudes are compared as integers: the same order as the floats', with
// infinity above every number and NaN above infinity.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct CodeScale {
  float inv, step;
};
__device__ __forceinline__ CodeScale code_scale(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  CodeScale s;
  if (top_bits >= 0x7f800000u) {
    s.inv = 0.0f;
    s.step = __uint_as_float(0x7fc00000u);
  } else if (top < kTiny) {
    s.inv = 0.0f;
    s.step = 0.0f;
  } else {
    s.inv = __fdiv_rn(127.0f, top);
    s.step = __fdiv_rn(top, 127.0f);
  }
  return s;
}
__device__ __forceinline__ int8_t code_of(float x, float inv) {
  // inv is 0 for a group of zeros or of NaN; x * 0 may be NaN there and converts to 0
  return (int8_t)__float2int_rn(__fmul_rn(x, inv));
}

struct RowArgs {
  const void* x;       // [n, c], row pitch ldx
  const int8_t* codes; // or 8-bit codes [n, c]
  const float* steps;  // [n, groups]
  const void* dy;
  const float* w;  // [c] or null
  const float* b;
  const float* mean_in;
  const float* rstd_in;
  void* y;  // forward output or dx
  int8_t* codes_out;
  float* steps_out;
  float* mean;
  float* rstd;
  float* part;  // backward: [gridDim.x][2][c] partial sums of dw, db (null: not wanted)
  int64_t n, ldx, lddy, ldy;
  int c, groups, group_shift;
  int lanes;  // lanes that share a row (power of two)
  float eps;
};

// Group maxima for the codes.  Lane l of a row holds vectors l, l + 32, ...
// (or one vector when the row has at most 32).  A group is 2^group_shift
// values: a run of lanes of one vector index, or (narrow vectors) all lanes of
// 2 or 4 consecutive indices.
template <int VEC, int ITER>
__device__ __forceinline__ void group_tops(uint32_t (&top)[ITER], int group_shift, int lanes) {
  const int per = (1 << group_shift) / VEC;  // vectors of a group
  const int width = min(per, lanes);
#pragma unroll
  for (int i = 0; i < ITER; ++i)
    for (int o = width >> 1; o > 0; o >>= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
  if constexpr (ITER >= 2) {
    if (per >= 64) {
#pragma unroll
      for (int i = 0; i < ITER; i += 2) top[i] = top[i + 1] = max(top[i], top[i + 1]);
    }
  }
  if constexpr (ITER >= 4) {
    if (per >= 128) {
#pragma unroll
      for (int i = 0; i < ITER; i += 4) top[i] = top[i + 1] = top[i + 2] = top[i + 3] = max(top[i], top[i + 2]);
    }
  }
}

// Rows of up to 1024 values: `lanes` lanes per row, ITER vectors per lane.
// CODES: the checkpoint is written too.
template <typename T, int VEC, int ITER, bool CODES>
__global__ void __launch_bounds__(kThreads) k_norm_rows(const __grid_constant__ RowArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1);
  const int per_block = kThreads / a.lanes;
  const int sub = threadIdx.x / a.lanes;
  const int nv = a.c / VEC;
  const float inv_c = 1.0f / (float)a.c;
  float w[ITER][VEC], b[ITER][VEC];
#pragma unroll
  for (int i = 0; i < ITER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int at = (i * 32 + lane) * VEC + j;
      w[i][j] = a.w && at < a.c ? __ldg(a.w + at) : 1.0f;
      b[i][j] = a.b && at < a.c ? __ldg(a.b + at) : 0.0f;
    }
  // every lane of a warp takes the same number of turns (the shuffles need them all)
  const int64_t turns = (a.n + (int64_t)gridDim.x * per_block - 1) / ((int64_t)gridDim.x * per_block);
  int64_t row = (int64_t)blockIdx.x * per_block + sub;
  for (int64_t t = 0; t < turns; ++t, row += (int64_t)gridDim.x * per_block) {
    const bool live = row < a.n;
    const T* px = reinterpret_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
    float x[ITER][VEC];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = i * 32 + lane;
      if (live && v < nv) {
        load_vec<T, VEC>(px + v * VEC, x[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[i][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += x[i][j];
    }
    const float mean = lanes_sum(s, a.lanes) * inv_c;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      if (i * 32 + lane < nv) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) q += (x[i][j] - mean) * (x[i][j] - mean);
      }
    const float rstd = rsqrtf(lanes_sum(q, a.lanes) * inv_c + a.eps);
    if (live && lane == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    if constexpr (CODES) {
      uint32_t top[ITER];
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        top[i] = 0u;
#pragma unroll
        for (int j = 0; j < VEC; ++j) top[i] = max(top[i], mag_bits(x[i][j]));
      }
      group_tops<VEC, ITER>(top, a.group_shift, a.lanes);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = i * 32 + lane;
        if (!live || v >= nv) continue;
        const CodeScale cs = code_scale(top[i]);
        Pack<int8_t, VEC> u;
#pragma unroll
        for (int j = 0; j < VEC; ++j) u.v[j] = code_of(x[i][j], cs.inv);
        *reinterpret_cast<Pack<int8_t, VEC>*>(a.codes_out + row * a.c + v * VEC) = u;
        if (((v * VEC) & ((1 << a.group_shift) - 1)) == 0)
          a.steps_out[row * a.groups + ((v * VEC) >> a.group_shift)] = cs.step;
      }
    }
    if (live) {
      T* py = reinterpret_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = i * 32 + lane;
        if (v >= nv) continue;
        float y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] = (x[i][j] - mean) * rstd * w[i][j] + b[i][j];
        store_vec<T, VEC>(py + v * VEC, y);
      }
    }
  }
}

// One vector of x, from the tensor or from its checkpoint.
template <typename T, int VEC, bool CODES>
__device__ __forceinline__ void load_x(const RowArgs& a, int64_t row, int v, float (&x)[VEC]) {
  if constexpr (CODES) {
    const Pack<int8_t, VEC> u = *reinterpret_cast<const Pack<int8_t, VEC>*>(a.codes + row * a.c + v * VEC);
    const float step = __ldg(a.steps + row * a.groups + ((v * VEC) >> a.group_shift));
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = (float)u.v[j] * step;
  } else {
    load_vec<T, VEC>(reinterpret_cast<const T*>(a.x) + row * a.ldx + v * VEC, x);
  }
}

// Backward of rows of up to 1024 values.  A lane keeps the same channels for
// all its rows, so its parts of dw and db stay in registers; the block adds
// its lanes' parts in a fixed order and writes them once.
template <typename T, int VEC, int ITER, bool CODES>
__global__ void __launch_bounds__(kThreads) k_norm_rows_bwd(const __grid_constant__ RowArgs a) {
  extern __shared__ float sh[];  // [kThreads / lanes][c]
  const int lane = threadIdx.x & (a.lanes - 1);
  const int per_block = kThreads / a.lanes;
  const int sub = threadIdx.x / a.lanes;
  const int nv = a.c / VEC;
  const float inv_c = 1.0f / (float)a.c;
  float w[ITER][VEC], dw[ITER][VEC], db[ITER][VEC];
#pragma unroll
  for (int i = 0; i < ITER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int at = (i * 32 + lane) * VEC + j;
      w[i][j] = a.w && at < a.c ? __ldg(a.w + at) : 1.0f;
      dw[i][j] = db[i][j] = 0.0f;
    }
  const int64_t turns = (a.n + (int64_t)gridDim.x * per_block - 1) / ((int64_t)gridDim.x * per_block);
  int64_t row = (int64_t)blockIdx.x * per_block + sub;
  for (int64_t t = 0; t < turns; ++t, row += (int64_t)gridDim.x * per_block) {
    const bool live = row < a.n;
    const int64_t r = live ? row : 0;
    const float mean = __ldg(a.mean_in + r), rstd = __ldg(a.rstd_in + r);
    float xh[ITER][VEC], g[ITER][VEC];
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = i * 32 + lane;
      if (live && v < nv) {
        load_x<T, VEC, CODES>(a, r, v, xh[i]);
        load_vec<T, VEC>(reinterpret_cast<const T*>(a.dy) + r * a.lddy + v * VEC, g[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = mean;
          g[i][j] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (live && i * 32 + lane < nv) {
          xh[i][j] = (xh[i][j] - mean) * rstd;
          dw[i][j] += g[i][j] * xh[i][j];
          db[i][j] += g[i][j];
          g[i][j] *= w[i][j];
          sg += g[i][j];
          sgx += g[i][j] * xh[i][j];
        }
      }
    sg = lanes_sum(sg, a.lanes) * inv_c;
    sgx = lanes_sum(sgx, a.lanes) * inv_c;
    if (live) {
      T* py = reinterpret_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = i * 32 + lane;
        if (v >= nv) continue;
        float d[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = rstd * (g[i][j] - sg - xh[i][j] * sgx);
        store_vec<T, VEC>(py + v * VEC, d);
      }
    }
  }
  if (!a.part) return;
  for (int pass = 0; pass < 2; ++pass) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int at = (i * 32 + lane) * VEC + j;
        if (at < a.c) sh[sub * a.c + at] = pass ? db[i][j] : dw[i][j];
      }
    __syncthreads();
    for (int at = threadIdx.x; at < a.c; at += kThreads) {
      float s = 0.0f;
      for (int k = 0; k < per_block; ++k) s += sh[k * a.c + at];
      a.part[((int64_t)blockIdx.x * 2 + pass) * a.c + at] = s;
    }
  }
}

// dw, db = sums of the blocks' parts: 32 channels per block, 8 rows of threads
// over the parts, added in a fixed order.
__global__ void __launch_bounds__(kThreads) k_norm_sum_parts(const float* __restrict__ part, int parts, int c,
                                                             float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sh[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int at = blockIdx.x * 32 + tx;  // over 2c values: dw, then db
  float s = 0.0f;
  if (at < 2 * c)
    for (int p = ty; p < parts; p += 8) s += __ldg(part + (int64_t)p * 2 * c + at);
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && at < 2 * c) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += sh[k][tx];
    float* out = at < c ? dw : db;
    if (out) out[at < c ? at : at - c] = t;
  }
}

// ---------------------------------------------------------------- rows wider than 1024
__device__ __forceinline__ float block_sum(float v, float* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = lanes_sum(v, 32);
  __syncthreads();
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) s += sh[k];
  return s;
}

// One block per row; the row is read again from cache for each of its passes.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_norm_wide(const __grid_constant__ RowArgs a) {
  __shared__ float sh[kThreads / 32];
  const int nv = a.c / VEC;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* px = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    float s = 0.0f;
    for (int v = threadIdx.x; v < nv; v += kThreads) {
      float x[VEC];
      load_vec<T, VEC>(px + v * VEC, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += x[j];
    }
    const float mean = block_sum(s, sh) / (float)a.c;
    float q = 0.0f;
    for (int v = threadIdx.x; v < nv; v += kThreads) {
      float x[VEC];
      load_vec<T, VEC>(px + v * VEC, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) q += (x[j] - mean) * (x[j] - mean);
    }
    const float rstd = rsqrtf(block_sum(q, sh) / (float)a.c + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    T* py = reinterpret_cast<T*>(a.y) + row * a.ldy;
    for (int v = threadIdx.x; v < nv; v += kThreads) {
      float x[VEC];
      load_vec<T, VEC>(px + v * VEC, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int at = v * VEC + j;
        x[j] = (x[j] - mean) * rstd * (a.w ? __ldg(a.w + at) : 1.0f) + (a.b ? __ldg(a.b + at) : 0.0f);
      }
      store_vec<T, VEC>(py + v * VEC, x);
    }
  }
}

template <typename T, int VEC, bool CODES>
__global__ void __launch_bounds__(kThreads) k_norm_wide_dx(const __grid_constant__ RowArgs a) {
  __shared__ float sh[kThreads / 32];
  const int nv = a.c / VEC;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const float mean = __ldg(a.mean_in + row), rstd = __ldg(a.rstd_in + row);
    const T* pd = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
    float sg = 0.0f, sgx = 0.0f;
    for (int v = threadIdx.x; v < nv; v += kThreads) {
      float x[VEC], g[VEC];
      load_x<T, VEC, CODES>(a, row, v, x);
      load_vec<T, VEC>(pd + v * VEC, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        g[j] *= a.w ? __ldg(a.w + v * VEC + j) : 1.0f;
        sg += g[j];
        sgx += g[j] * ((x[j] - mean) * rstd);
      }
    }
    sg = block_sum(sg, sh) / (float)a.c;
    sgx = block_sum(sgx, sh) / (float)a.c;
    T* py = reinterpret_cast<T*>(a.y) + row * a.ldy;
    for (int v = threadIdx.x; v < nv; v += kThreads) {
      float x[VEC], g[VEC];
      load_x<T, VEC, CODES>(a, row, v, x);
      load_vec<T, VEC>(pd + v * VEC, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        g[j] = rstd * (g[j] * (a.w ? __ldg(a.w + v * VEC + j) : 1.0f) - sg - (x[j] - mean) * rstd * sgx);
      store_vec<T, VEC>(py + v * VEC, g);
    }
  }
}

// Parts of dw and db: block (channel slab, row range), one channel vector per thread.
template <typename T, int VEC, bool CODES>
__global__ void __launch_bounds__(kThreads) k_norm_wide_dw(const __grid_constant__ RowArgs a) {
  const int v = blockIdx.x * kThreads + threadIdx.x;
  if (v >= a.c / VEC) return;
  float dw[VEC], db[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) dw[j] = db[j] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    const float mean = __ldg(a.mean_in + row), rstd = __ldg(a.rstd_in + row);
    float x[VEC], g[VEC];
    load_x<T, VEC, CODES>(a, row, v, x);
    load_vec<T, VEC>(reinterpret_cast<const T*>(a.dy) + row * a.lddy + v * VEC, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      dw[j] += g[j] * ((x[j] - mean) * rstd);
      db[j] += g[j];
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    a.part[((int64_t)blockIdx.y * 2) * a.c + v * VEC + j] = dw[j];
    a.part[((int64_t)blockIdx.y * 2 + 1) * a.c + v * VEC + j] = db[j];
  }
}

// ---------------------------------------------------------------- checkpoints
// Pack: `lanes` lanes per group of a row, SPAN vectors per lane.
template <typename T, int VEC, int SPAN>
__global__ void __launch_bounds__(kThreads) k_ck_pack(const __grid_constant__ RowArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1);
  const int per_block = kThreads / a.lanes;
  const int64_t units = a.n * a.groups;
  const int64_t turns = (units + (int64_t)gridDim.x * per_block - 1) / ((int64_t)gridDim.x * per_block);
  int64_t u = (int64_t)blockIdx.x * per_block + threadIdx.x / a.lanes;
  for (int64_t t = 0; t < turns; ++t, u += (int64_t)gridDim.x * per_block) {
    const bool live = u < units;
    const int64_t row = live ? (a.groups == 1 ? u : u / a.groups) : 0;
    const int grp = live ? (int)(u - row * a.groups) : 0;
    const T* px = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    float x[SPAN][VEC];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
      const int at = (grp << a.group_shift) + (i * 32 + lane) * VEC;
      const bool in = live && (i * 32 + lane) * VEC < (1 << a.group_shift) && at < a.c;
      if (in) {
        load_vec<T, VEC>(px + at, x[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[i][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) top = max(top, mag_bits(x[i][j]));
    }
    for (int o = a.lanes >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!live) continue;
    const CodeScale cs = code_scale(top);
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
      const int at = (grp << a.group_shift) + (i * 32 + lane) * VEC;
      if ((i * 32 + lane) * VEC >= (1 << a.group_shift) || at >= a.c) continue;
      Pack<int8_t, VEC> p;
#pragma unroll
      for (int j = 0; j < VEC; ++j) p.v[j] = code_of(x[i][j], cs.inv);
      *reinterpret_cast<Pack<int8_t, VEC>*>(a.codes_out + row * a.c + at) = p;
    }
    if (lane == 0) a.steps_out[u] = cs.step;
  }
}

// Restore, and (NORM) the layer norm of the restored rows with given statistics.
template <typename T, int VEC, bool NORM>
__global__ void __launch_bounds__(kThreads) k_ck_restore(const __grid_constant__ RowArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1);
  const int per_block = kThreads / a.lanes;
  const int nv = a.c / VEC;
  for (int64_t row = (int64_t)blockIdx.x * per_block + threadIdx.x / a.lanes; row < a.n;
       row += (int64_t)gridDim.x * per_block) {
    float mean = 0.0f, rstd = 1.0f;
    if constexpr (NORM) {
      mean = __ldg(a.mean_in + row);
      rstd = __ldg(a.rstd_in + row);
    }
    for (int v = lane; v < nv; v += a.lanes) {
      float x[VEC];
      load_x<T, VEC, true>(a, row, v, x);
      if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int at = v * VEC + j;
          x[j] = (x[j] - mean) * rstd * (a.w ? __ldg(a.w + at) : 1.0f) + (a.b ? __ldg(a.b + at) : 0.0f);
        }
      }
      store_vec<T, VEC>(reinterpret_cast<T*>(a.y) + row * a.ldy + v * VEC, x);
    }
  }
}

// ---------------------------------------------------------------- host
// Widest vector (in elements) that the channel count, the pitches and the
// bases allow: 16 bytes; for bf16 also 4 bytes, so that an even channel count
// still moves 128 bytes per warp and load.
bool aligned(const void* p, int64_t ld, int elem, int vec) {
  return !p || ((reinterpret_cast<uintptr_t>(p) % (size_t)(elem * vec)) == 0 && ld % vec == 0);
}
int pick_vec(fvx_dtype dt, int64_t c, const RowArgs& a) {
  const int elem = dt == FVX_F32 ? 4 : 2;
  for (int vec : {16 / elem, elem == 2 ? 2 : 1, 1}) {
    if (c % vec == 0 && aligned(a.x, a.ldx, elem, vec) && aligned(a.dy, a.lddy, elem, vec) &&
        aligned(a.y, a.ldy, elem, vec) && aligned(a.codes, c, 1, vec) && aligned(a.codes_out, c, 1, vec))
      return vec;
  }
  return 1;
}
int pow2_at_least(int64_t v, int most) {
  int p = 1;
  while (p < v && p < most) p <<= 1;
  return p;
}
int iters_for(int64_t c, int vec) { return (int)((c / vec + 31) / 32); }

// Blocks for `units` units of `per_block`, at most `per_sm` per multiprocessor.
int grid_for(int64_t units, int per_block, int sms, int per_sm) {
  const int64_t need = (units + per_block - 1) / per_block;
  return (int)std::max<int64_t>(1, std::min<int64_t>(need, (int64_t)sms * per_sm));
}

template <typename K>
fvx_status launch(const char* name, K kernel, dim3 grid, size_t smem, cudaStream_t s, const RowArgs& a) {
  LaunchScope ls(name, s);
  kernel<<<grid, kThreads, smem, s>>>(a);
  return check_launch(name);
}

// Calls f.template operator()<T, VEC, ITER>() for the row's vector width.
template <typename F>
fvx_status by_row_shape(fvx_dtype dt, int vec, int iters, F&& f) {
  if (dt == FVX_F32) {
    if (vec == 4) {
      if (iters <= 1) return f.template operator()<float, 4, 1>();
      if (iters <= 2) return f.template operator()<float, 4, 2>();
      return f.template operator()<float, 4, 8>();
    }
    if (iters <= 1) return f.template operator()<float, 1, 1>();
    if (iters <= 4) return f.template operator()<float, 1, 4>();
    return f.template operator()<float, 1, 32>();
  }
  if (vec == 8) {
    if (iters <= 1) return f.template operator()<__nv_bfloat16, 8, 1>();
    if (iters <= 2) return f.template operator()<__nv_bfloat16, 8, 2>();
    return f.template operator()<__nv_bfloat16, 8, 4>();
  }
  if (vec == 2) {
    if (iters <= 1) return f.template operator()<__nv_bfloat16, 2, 1>();
    if (iters <= 4) return f.template operator()<__nv_bfloat16, 2, 4>();
    return f.template operator()<__nv_bfloat16, 2, 16>();
  }
  if (iters <= 1) return f.template operator()<__nv_bfloat16, 1, 1>();
  if (iters <= 4) return f.template operator()<__nv_bfloat16, 1, 4>();
  return f.template operator()<__nv_bfloat16, 1, 32>();
}
template <typename F>
fvx_status by_vec(fvx_dtype dt, int vec, F&& f) {
  if (dt == FVX_F32) return vec == 4 ? f.template operator()<float, 4>() : f.template operator()<float, 1>();
  if (vec == 8) return f.template operator()<__nv_bfloat16, 8>();
  return vec == 2 ? f.template operator()<__nv_bfloat16, 2>() : f.template operator()<__nv_bfloat16, 1>();
}

fvx_status bad(const char* who, const char* what) {
  set_error("%s: %s", who, what);
  return FVX_ERR_INVALID_ARG;
}

fvx_status check_rows(const char* who, fvx_dtype dt, int64_t n, int64_t c) {
  if (dt != FVX_F32 && dt != FVX_BF16) return bad(who, "dtype must be FVX_F32 or FVX_BF16");
  if (n < 0) return bad(who, "negative row count");
  if (c < 1 || c > kMaxCols) return bad(who, "channels must be in 1..65536");
  return FVX_OK;
}
fvx_status check_matrix(const char* who, const char* name, fvx_dtype dt, const void* p, int64_t ld, int64_t n,
                        int64_t c) {
  if (n > 0 && !p) {
    set_error("%s: NULL %s", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  if (ld < c) {
    set_error("%s: the row pitch of %s is below the channel count", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  if (reinterpret_cast<uintptr_t>(p) % (dt == FVX_F32 ? 4 : 2)) {
    set_error("%s: %s is not aligned to its elements", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  return FVX_OK;
}
fvx_status check_f32(const char* who, const char* name, const float* p, bool required) {
  if ((required && !p) || reinterpret_cast<uintptr_t>(p) % 4) {
    set_error("%s: %s is NULL or not aligned to 4 bytes", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  return FVX_OK;
}
// group 0: no checkpoint
fvx_status check_group(const char* who, int32_t group, int64_t n, const void* codes, const float* steps, int* shift) {
  if (group != 32 && group != 64 && group != 128) return bad(who, "the checkpoint's group must be 32, 64 or 128");
  if (n > 0 && !codes) return bad(who, "NULL codes");
  FVX_TRY(check_f32(who, "steps", steps, n > 0));
  *shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  return FVX_OK;
}

fvx_status pack_launch(fvx_dtype dt, RowArgs a, cudaStream_t s, int sms) {
  RowArgs only = a;
  only.y = nullptr;
  only.dy = nullptr;
  const int vec = pick_vec(dt, a.c, only);
  const int64_t in_group = std::min<int64_t>(a.c, 1 << a.group_shift);
  a.lanes = pow2_at_least((in_group + vec - 1) / vec, 32);
  const int span = (int)((in_group + vec * 32 - 1) / (vec * 32));
  const int grid = grid_for(a.n * a.groups, kThreads / a.lanes, sms, 8);
  return by_vec(dt, vec, [&]<typename T, int VEC>() {
    if constexpr (VEC * sizeof(T) == 16) {
      return launch("ck_pack", k_ck_pack<T, VEC, 1>, dim3(grid), 0, s, a);
    } else {
      return span <= 1 ? launch("ck_pack", k_ck_pack<T, VEC, 1>, dim3(grid), 0, s, a)
                       : launch("ck_pack", k_ck_pack<T, VEC, 4>, dim3(grid), 0, s, a);
    }
  });
}

}  // namespace
}  // namespace fvx

using namespace fvx;

extern "C" {

fvx_status fvx_layer_norm(fvx_dtype dt, const void* x, int64_t ldx, int64_t n, int64_t c, const float* w,
                          const float* b, float eps, void* y, int64_t ldy, float* mean, float* rstd, int32_t group,
                          int8_t* codes, float* steps, fvx_stream stream) {
  const char* who = "fvx_layer_norm";
  EntryScope entry(who);
  FVX_TRY(check_rows(who, dt, n, c));
  FVX_TRY(check_matrix(who, "x", dt, x, ldx, n, c));
  FVX_TRY(check_matrix(who, "y", dt, y, ldy, n, c));
  FVX_TRY(check_f32(who, "weight", w, false));
  FVX_TRY(check_f32(who, "bias", b, false));
  FVX_TRY(check_f32(who, "mean", mean, n > 0));
  FVX_TRY(check_f32(who, "rstd", rstd, n > 0));
  if (!(eps >= 0.0f)) return bad(who, "eps must not be negative");
  int shift = 5;
  if (group != 0) FVX_TRY(check_group(who, group, n, codes, steps, &shift));
  if (n == 0) return FVX_OK;
  cudaStream_t s = (cudaStream_t)stream;
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  RowArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.n = n;
  a.c = (int)c;
  a.w = w;
  a.b = b;
  a.eps = eps;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.group_shift = shift;
  a.groups = (int)((c + (1 << shift) - 1) >> shift);
  if (group) {
    a.codes_out = codes;
    a.steps_out = steps;
  }
  const int vec = pick_vec(dt, c, a);
  if (c <= kRegCols) {
    a.lanes = pow2_at_least(c / vec, 32);
    const int grid = grid_for(n, kThreads / a.lanes, sms, 8);
    return by_row_shape(dt, vec, iters_for(c, vec), [&]<typename T, int VEC, int ITER>() {
      return group ? launch("norm_rows", k_norm_rows<T, VEC, ITER, true>, dim3(grid), 0, s, a)
                   : launch("norm_rows", k_norm_rows<T, VEC, ITER, false>, dim3(grid), 0, s, a);
    });
  }
  const int grid = grid_for(n, 1, sms, 8);
  FVX_TRY(by_vec(dt, vec, [&]<typename T, int VEC>() {
    return launch("norm_wide", k_norm_wide<T, VEC>, dim3(grid), 0, s, a);
  }));
  return group ? pack_launch(dt, a, s, sms) : FVX_OK;
}

fvx_status fvx_layer_norm_backward(fvx_dtype dt, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                   int32_t group, const int8_t* codes, const float* steps, int64_t n, int64_t c,
                                   const float* w, const float* mean, const float* rstd, void* dx, int64_t lddx,
                                   float* dw, float* db, fvx_stream stream) {
  const char* who = "fvx_layer_norm_backward";
  EntryScope entry(who);
  FVX_TRY(check_rows(who, dt, n, c));
  FVX_TRY(check_matrix(who, "dy", dt, dy, lddy, n, c));
  FVX_TRY(check_matrix(who, "dx", dt, dx, lddx, n, c));
  int shift = 5;
  if (group != 0) {
    if (x) return bad(who, "x and a checkpoint are both given");
    FVX_TRY(check_group(who, group, n, codes, steps, &shift));
  } else {
    FVX_TRY(check_matrix(who, "x", dt, x, ldx, n, c));
  }
  FVX_TRY(check_f32(who, "weight", w, false));
  FVX_TRY(check_f32(who, "mean", mean, n > 0));
  FVX_TRY(check_f32(who, "rstd", rstd, n > 0));
  FVX_TRY(check_f32(who, "dweight", dw, false));
  FVX_TRY(check_f32(who, "dbias", db, false));
  cudaStream_t s = (cudaStream_t)stream;
  if (n == 0) {
    if (dw) FVX_CUDA(cudaMemsetAsync(dw, 0, (size_t)c * 4, s));
    if (db) FVX_CUDA(cudaMemsetAsync(db, 0, (size_t)c * 4, s));
    return FVX_OK;
  }
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  Scratch scr(s);
  RowArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.codes = group ? codes : nullptr;
  a.steps = steps;
  a.dy = dy;
  a.lddy = lddy;
  a.n = n;
  a.c = (int)c;
  a.w = w;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.y = dx;
  a.ldy = lddx;
  a.group_shift = shift;
  a.groups = (int)((c + (1 << shift) - 1) >> shift);
  const int vec = pick_vec(dt, c, a);
  const bool sums = dw || db;
  int parts = 0;
  if (c <= kRegCols) {
    a.lanes = pow2_at_least(c / vec, 32);
    parts = grid_for(n, kThreads / a.lanes, sms, 4);
    if (sums && !(a.part = scr.get<float>((size_t)parts * 2 * c))) return FVX_ERR_ALLOC;
    const size_t smem = (size_t)(kThreads / a.lanes) * c * 4;  // at most 8 * 1024 or 256 * 8 values
    FVX_TRY(by_row_shape(dt, vec, iters_for(c, vec), [&]<typename T, int VEC, int ITER>() {
      return group ? launch("norm_rows_bwd", k_norm_rows_bwd<T, VEC, ITER, true>, dim3(parts), smem, s, a)
                   : launch("norm_rows_bwd", k_norm_rows_bwd<T, VEC, ITER, false>, dim3(parts), smem, s, a);
    }));
  } else {
    const int grid = grid_for(n, 1, sms, 8);
    const int slabs = (int)((c / vec + kThreads - 1) / kThreads);
    parts = (int)std::min<int64_t>(n, std::max(1, 4 * sms / slabs));
    if (sums && !(a.part = scr.get<float>((size_t)parts * 2 * c))) return FVX_ERR_ALLOC;
    FVX_TRY(by_vec(dt, vec, [&]<typename T, int VEC>() -> fvx_status {
      FVX_TRY(group ? launch("norm_wide_dx", k_norm_wide_dx<T, VEC, true>, dim3(grid), 0, s, a)
                    : launch("norm_wide_dx", k_norm_wide_dx<T, VEC, false>, dim3(grid), 0, s, a));
      if (!sums) return FVX_OK;
      return group ? launch("norm_wide_dw", k_norm_wide_dw<T, VEC, true>, dim3(slabs, parts), 0, s, a)
                   : launch("norm_wide_dw", k_norm_wide_dw<T, VEC, false>, dim3(slabs, parts), 0, s, a);
    }));
  }
  if (!sums) return FVX_OK;
  LaunchScope ls("norm_sum_parts", s);
  k_norm_sum_parts<<<(unsigned)((2 * c + 31) / 32), kThreads, 0, s>>>(a.part, parts, (int)c, dw, db);
  return check_launch("norm_sum_parts");
}

fvx_status fvx_checkpoint_pack(fvx_dtype dt, const void* x, int64_t ldx, int64_t n, int64_t c, int32_t group,
                               int8_t* codes, float* steps, fvx_stream stream) {
  const char* who = "fvx_checkpoint_pack";
  EntryScope entry(who);
  FVX_TRY(check_rows(who, dt, n, c));
  FVX_TRY(check_matrix(who, "x", dt, x, ldx, n, c));
  int shift = 5;
  FVX_TRY(check_group(who, group, n, codes, steps, &shift));
  if (n == 0) return FVX_OK;
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  RowArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.n = n;
  a.c = (int)c;
  a.codes_out = codes;
  a.steps_out = steps;
  a.group_shift = shift;
  a.groups = (int)((c + group - 1) >> shift);
  return pack_launch(dt, a, (cudaStream_t)stream, sms);
}

fvx_status fvx_checkpoint_restore(fvx_dtype dt, int32_t group, const int8_t* codes, const float* steps, int64_t n,
                                  int64_t c, const float* mean, const float* rstd, const float* w, const float* b,
                                  void* out, int64_t ldo, fvx_stream stream) {
  const char* who = "fvx_checkpoint_restore";
  EntryScope entry(who);
  FVX_TRY(check_rows(who, dt, n, c));
  FVX_TRY(check_matrix(who, "out", dt, out, ldo, n, c));
  int shift = 5;
  FVX_TRY(check_group(who, group, n, codes, steps, &shift));
  if ((mean == nullptr) != (rstd == nullptr)) return bad(who, "mean and rstd must both be given or both be NULL");
  if (!mean && (w || b)) return bad(who, "weight and bias need mean and rstd");
  FVX_TRY(check_f32(who, "mean", mean, false));
  FVX_TRY(check_f32(who, "rstd", rstd, false));
  FVX_TRY(check_f32(who, "weight", w, false));
  FVX_TRY(check_f32(who, "bias", b, false));
  if (n == 0) return FVX_OK;
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  cudaStream_t s = (cudaStream_t)stream;
  RowArgs a = {};
  a.codes = codes;
  a.steps = steps;
  a.n = n;
  a.c = (int)c;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.w = w;
  a.b = b;
  a.y = out;
  a.ldy = ldo;
  a.group_shift = shift;
  a.groups = (int)((c + group - 1) >> shift);
  const int vec = pick_vec(dt, c, a);
  a.lanes = pow2_at_least(c / vec, kThreads);
  const int grid = grid_for(n, kThreads / a.lanes, sms, 8);
  return by_vec(dt, vec, [&]<typename T, int VEC>() {
    return mean ? launch("ck_restore", k_ck_restore<T, VEC, true>, dim3(grid), 0, s, a)
                : launch("ck_restore", k_ck_restore<T, VEC, false>, dim3(grid), 0, s, a);
  });
}

}  // extern "C"
