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
// memory bounds it.  So each row of up to 1024 channels is read once, stays in
// registers between its two reductions, and the checkpoint is written by the
// pass that reads x.
// Statistics, products and sums are fp32 whatever the storage type.  Measured
// (bf16, time and bandwidth): 4,000,000 x 64 forward 182 us, 5.6 TB/s, backward
// 266, 5.8; 10,000,000 x 32 packed in 195 us, 4.9 TB/s, restored in 164, 5.9;
// 150,001 x 256 forward with codes 51 us, 3.8 TB/s, backward from codes 57, 3.4
// (both bound by the instructions of the codes), normed again 23, 5.1.
#include "norm.cuh"

namespace fvx {
namespace {

template <typename T, int VEC, int ITER, int OP>
__global__ void __launch_bounds__(kThreads) k_rows(const __grid_constant__ RowArgs a) {
  extern __shared__ float sh[];  // backward: [kThreads / lanes][c]
  Rows<T, VEC, ITER, OP, 0> rows(a);
  const int per_block = kThreads / a.lanes;
  rows.direct((int64_t)blockIdx.x * per_block, (int64_t)gridDim.x * per_block, a.n);
  if constexpr (OpIs<OP>::kBack) rows.write_parts(sh, kThreads);
}

// dw, db = sums of the blocks' parts: 32 channels per block, 32 rows of threads
// over the parts, added in a fixed order.  Latency is all of it: with eight rows
// of threads, four loads of each at once, 608 parts took 10 us.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) k_norm_sum_parts(const float* __restrict__ part, int parts, int c,
                                                                  float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sh[kSumRows][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int at = blockIdx.x * 32 + tx;  // over 2c values: dw, then db
  float s = 0.0f;
  if (at < 2 * c) {
    constexpr int kAtOnce = 10;
    for (int p = ty; p < parts; p += kAtOnce * kSumRows) {
      float x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = p + k * kSumRows;
        x[k] = i < parts ? __ldg(part + (int64_t)i * 2 * c + at) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) s += x[k];
    }
  }
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && at < 2 * c) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kSumRows; ++k) t += sh[k][tx];
    float* out = at < c ? dw : db;
    if (out) out[at < c ? at : at - c] = t;
  }
}

// ---------------------------------------------------------------- rows wider than 1024
// One vector of x, from the tensor or from its checkpoint.
template <typename T, int VEC, bool CODES>
__device__ __forceinline__ void load_x(const RowArgs& a, int64_t row, int v, float (&x)[VEC]) {
  if constexpr (CODES) {
    codes_to_float<VEC>(raw_vec<int8_t, VEC>(a.codes + row * a.c + v * VEC), x);
    const float step = __ldg(a.steps + row * a.groups + ((v * VEC) >> a.group_shift));
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] *= step;
  } else {
    load_vec<T, VEC>(reinterpret_cast<const T*>(a.x) + row * a.ldx + v * VEC, x);
  }
}

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

// One block per row; the row is read again from cache for each of its passes,
// the checkpoint and the parts of dw and db take a kernel of their own each.
// 20,000 x 4096 bf16 (fp32): forward 184 us, 1.8 TB/s (141, 4.6), with codes 258
// (244), backward 265, 1.9 (288, 3.4), packed in 74, 3.3 (107, 3.8), restored in
// 47, 5.2 (76, 5.4); 20,000 x 1026 fp32 53, 115, 114, 64 and 31.  Bound by
// latency: in bf16 k_norm_wide and k_norm_wide_dx (181, 184 us) issue in 34 and
// 39% of the cycles, k_norm_wide_dw (59 us) reads at 71% of the DRAM's rate.
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
// Pack of rows wider than 1024 values: `lanes` lanes per group of a row, SPAN
// vectors per lane.
template <typename T, int VEC, int SPAN>
__global__ void __launch_bounds__(kThreads) k_ck_pack_wide(const __grid_constant__ RowArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1);
  const int per_block = kThreads / a.lanes;
  const int64_t units = a.n * a.groups, step = (int64_t)gridDim.x * per_block;
  const int64_t turns = (units + step - 1) / step;
  int64_t unit = (int64_t)blockIdx.x * per_block + threadIdx.x / a.lanes;
  for (int64_t t = 0; t < turns; ++t, unit += step) {
    const bool live = unit < units;
    const int64_t row = live ? unit / a.groups : 0;
    const int first = live ? (int)(unit - row * a.groups) << a.group_shift : 0;
    const int left = live ? min(a.c - first, 1 << a.group_shift) : 0;
    const T* px = reinterpret_cast<const T*>(a.x) + row * a.ldx + first;
    float x[SPAN][VEC];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
      const int at = (i * 32 + lane) * VEC;
      widen<T, VEC>(at < left ? raw_vec<T, VEC>(px + at) : no_vec<T, VEC>(), x[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) top = max(top, mag_bits(x[i][j]));
    }
    for (int o = a.lanes >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const CodeScale cs = code_scale(top);
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
      const int at = (i * 32 + lane) * VEC;
      if (at >= left) continue;
      float q[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) q[j] = __fadd_rn(__fmul_rn(x[i][j], cs.inv), kMagic);
      store_codes<VEC>(a.codes_out + row * a.c + first + at, q, cs.inv == 0.0f);
    }
    if (lane == 0 && live) a.steps_out[unit] = cs.step;
  }
}

// Restore of rows wider than 1024 values, one block per row.
template <typename T, int VEC, bool NORM>
__global__ void __launch_bounds__(kThreads) k_ck_wide(const __grid_constant__ RowArgs a) {
  const int nv = a.c / VEC;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const float mean = NORM ? __ldg(a.mean_in + row) : 0.0f, rstd = NORM ? __ldg(a.rstd_in + row) : 1.0f;
    for (int v = threadIdx.x; v < nv; v += kThreads) {
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
// bases allow: 16 bytes, or two values, so that an even channel count still moves
// 128 bytes or more per warp and load.
bool aligned(const void* p, int64_t ld, int elem, int vec) {
  return !p || ((reinterpret_cast<uintptr_t>(p) % (size_t)(elem * vec)) == 0 && ld % vec == 0);
}
int pick_vec(fvx_dtype dt, int64_t c, const RowArgs& a) {
  const int elem = dt == FVX_F32 ? 4 : 2;
  for (int vec : {16 / elem, 2, 1}) {
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
// Lanes of a row and vectors per lane: one each of 16 bytes while that fits a
// warp, and four of the narrower ones, since a row's shuffles and bookkeeping
// then cost more instructions than its few values.
int lanes_for(fvx_dtype dt, int64_t c, int vec) {
  const int each = vec * (dt == FVX_F32 ? 4 : 2) == 16 ? 1 : 4;
  return pow2_at_least((c / vec + each - 1) / each, 32);
}
int iters_for(fvx_dtype dt, int64_t c, int vec) {
  const int lanes = lanes_for(dt, c, vec);
  return (int)((c / vec + lanes - 1) / lanes);
}

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

// Calls f.template operator()<T, VEC, ITER>() for the row's vector width, with
// the least power of two of vectors per lane that holds the row (vectors that a
// row does not have cost nearly as much as those it has: 263,657 x 179 bf16 with
// 32 in place of 8 took 641 us forward).
template <typename T, int VEC, int ITER, typename F>
fvx_status by_iters(int iters, F&& f) {
  if constexpr (VEC * 32 * ITER < kRegCols) {
    if (iters > ITER) return by_iters<T, VEC, 2 * ITER>(iters, f);
  }
  return f.template operator()<T, VEC, ITER>();
}
template <typename F>
fvx_status by_row_shape(fvx_dtype dt, int vec, int iters, F&& f) {
  if (dt == FVX_F32) {
    if (vec == 4) return by_iters<float, 4, 1>(iters, f);
    return vec == 2 ? by_iters<float, 2, 1>(iters, f) : by_iters<float, 1, 1>(iters, f);
  }
  if (vec == 8) return by_iters<__nv_bfloat16, 8, 1>(iters, f);
  return vec == 2 ? by_iters<__nv_bfloat16, 2, 1>(iters, f) : by_iters<__nv_bfloat16, 1, 1>(iters, f);
}
// The same for the kernels of wider rows.  What their launches count in vectors
// is counted in f by its VEC, never by the width that was asked for.
template <typename F>
fvx_status by_vec(fvx_dtype dt, int vec, F&& f) {
  if (dt == FVX_F32) {
    if (vec == 4) return f.template operator()<float, 4>();
    return vec == 2 ? f.template operator()<float, 2>() : f.template operator()<float, 1>();
  }
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

fvx_status pack_wide(fvx_dtype dt, RowArgs a, cudaStream_t s, int sms) {
  RowArgs only = a;
  only.y = nullptr;
  only.dy = nullptr;
  const int vec = pick_vec(dt, a.c, only);
  return by_vec(dt, vec, [&]<typename T, int VEC>() {
    const int in_group = 1 << a.group_shift;
    a.lanes = pow2_at_least(in_group / VEC, 32);
    const int grid = grid_for(a.n * a.groups, kThreads / a.lanes, sms, 32);
    if constexpr (VEC * sizeof(T) == 16) {
      return launch("ck_pack", k_ck_pack_wide<T, VEC, 1>, dim3(grid), 0, s, a);
    } else {
      return in_group <= 32 * VEC ? launch("ck_pack", k_ck_pack_wide<T, VEC, 1>, dim3(grid), 0, s, a)
                                  : launch("ck_pack", k_ck_pack_wide<T, VEC, 4>, dim3(grid), 0, s, a);
    }
  });
}

// Blocks of the row kernels; the backward ones write a part of dw and db each.
struct RowGrid {
  int blocks;
  bool stream;
  StreamArgs args;
};
// Rows of 16-byte vectors, dense or nearly so, enough of them for every block to
// take several stages, are streamed through shared memory.
template <int OP>
RowGrid row_grid(fvx_dtype dt, int vec, const RowArgs& a, int sms) {
  using Is = OpIs<OP>;
  const int elem = dt == FVX_F32 ? 4 : 2;
  RowGrid g = {};
  g.blocks = grid_for(a.n, kThreads / a.lanes, sms, Is::kBack ? 4 : 16);
  auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (vec * elem != 16) return g;
  // Rows a little apart are copied with what lies between them.  At a quarter
  // apart the bytes begin to cost what the copies save: 1,500,000 x 64 bf16 with
  // a pitch of 80, streamed or not, forward 86 or 100 us, backward 128 or 190,
  // packed in 68 or 70; 1,250,000 x 64 with 96, 78 or 88, 124 or 169, but 66 or
  // 61; 937,500 x 64 with 128, 70 or 64, 114 or 122, 61 or 45.
  auto close = [&](int64_t ld) { return ld <= a.c + a.c / 4; };
  if (!Is::kFromCodes && !(close(a.ldx) && at16(a.x))) return g;
  if (Is::kFromCodes && !(at16(a.codes) && at16(a.steps))) return g;
  if (Is::kBack && !(close(a.lddy) && at16(a.dy))) return g;
  if (Is::kStats && !(at16(a.mean_in) && at16(a.rstd_in))) return g;
  const int x_row = Is::kFromCodes ? a.c : (int)a.ldx * elem, dy_row = Is::kBack ? (int)a.lddy * elem : 0;
  const int row = x_row + dy_row;
  StreamArgs& s = g.args;
  s.r = a;
  // Two vectors of 16 lanes instead of one of 32 halve the steps of a row's sums
  // (300,000 x 256 bf16: forward 61 to 55 us, backward 88 to 86; x 200: 64 to
  // 56; 150,001 x 256 forward with codes 51 both ways, and the same order of the
  // sums as without codes); from codes the registers of two vectors cost a
  // block per multiprocessor (150,001 x 256 backward 57 to 74 us).
  if ((Is::kNorm || OP == kBackward) && dt == FVX_BF16 && a.lanes == 32 && a.c <= 32 * vec) s.r.lanes = 16;
  const int per_block = kThreads / s.r.lanes;
  // a multiple of the rows of a turn (eight at least: the small arrays' copies
  // are then multiples of 16 bytes), about 10 KB
  s.rows = per_block * std::max(1, 10240 / (per_block * row));
  // the tensor's last row ends with its last channel
  const bool apart = (!Is::kFromCodes && a.ldx > a.c) || (Is::kBack && a.lddy > a.c);
  s.stages = (apart ? std::max<int64_t>(a.n - 1, 0) : a.n) / s.rows;
  auto up = [](int v) { return (v + 15) & ~15; };
  s.off_dy = up(s.rows * x_row);
  s.off_steps = s.off_dy + up(s.rows * dy_row);
  s.off_mean = s.off_steps + (Is::kFromCodes ? up(s.rows * a.groups * 4) : 0);
  s.off_rstd = s.off_mean + (Is::kStats ? up(s.rows * 4) : 0);
  s.stage_bytes = (s.off_rstd + (Is::kStats ? up(s.rows * 4) : 0) + 127) & ~127;
  const int per_sm = std::min(Is::kBack ? 3 : 4, 227 * 1024 / (kStreamStages * s.stage_bytes + 128 + 1024));
  // Four stages for every block.  160,000 x 64 bf16, 4 stages each forward,
  // streamed or not: 14 or 18 us, backward 26 or 34, restored in 10 or 12, packed
  // in 14 both ways; 40,000 x 64, one each: 10 both ways, 20 or 22, 8 and 8.
  if (per_sm < 1 || s.stages < (int64_t)sms * per_sm * 4) return g;
  s.status = device_status_word();
  if (!s.status) return g;
  g.stream = true;
  g.blocks = sms * per_sm;
  return g;
}
template <int OP>
fvx_status rows_launch(const char* name, fvx_dtype dt, int vec, const RowArgs& a, const RowGrid& g, cudaStream_t s) {
  constexpr bool kBack = OpIs<OP>::kBack;
  const size_t parts = kBack ? (size_t)(kThreads / (g.stream ? g.args.r.lanes : a.lanes)) * a.c * 4 : 0;  // at most 8 * 1024 or 256 * 8 values
  if (g.stream) {
    const size_t smem = 128 + std::max((size_t)kStreamStages * g.args.stage_bytes, parts);
    StreamArgs args = g.args;
    const int lanes = args.r.lanes;
    args.r = a;
    args.r.lanes = lanes;
    return (dt == FVX_F32 ? stream_rows_f32 : stream_rows_bf16)(name, (RowOp)OP, (a.c / vec + lanes - 1) / lanes, args, g.blocks,
                                                                smem, s);
  }
  return by_row_shape(dt, vec, iters_for(dt, a.c, vec), [&]<typename T, int VEC, int ITER>() -> fvx_status {
    return launch(name, k_rows<T, VEC, ITER, OP>, dim3(g.blocks), parts, s, a);
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
    a.lanes = lanes_for(dt, c, vec);
    return group ? rows_launch<kForwardCodes>("norm_rows", dt, vec, a, row_grid<kForwardCodes>(dt, vec, a, sms), s)
                 : rows_launch<kForward>("norm_rows", dt, vec, a, row_grid<kForward>(dt, vec, a, sms), s);
  }
  const int grid = grid_for(n, 1, sms, 8);
  FVX_TRY(by_vec(dt, vec, [&]<typename T, int VEC>() {
    return launch("norm_wide", k_norm_wide<T, VEC>, dim3(grid), 0, s, a);
  }));
  return group ? pack_wide(dt, a, s, sms) : FVX_OK;
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
    a.lanes = lanes_for(dt, c, vec);
    const RowGrid g = group ? row_grid<kBackwardCodes>(dt, vec, a, sms) : row_grid<kBackward>(dt, vec, a, sms);
    parts = g.blocks;
    if (sums && !(a.part = scr.get<float>((size_t)parts * 2 * c))) return FVX_ERR_ALLOC;
    FVX_TRY(group ? rows_launch<kBackwardCodes>("norm_rows_bwd", dt, vec, a, g, s)
                  : rows_launch<kBackward>("norm_rows_bwd", dt, vec, a, g, s));
  } else {
    const int grid = grid_for(n, 1, sms, 8);
    FVX_TRY(by_vec(dt, vec, [&]<typename T, int VEC>() -> fvx_status {
      const int slabs = (int)((c / VEC + kThreads - 1) / kThreads);
      parts = (int)std::min<int64_t>(n, std::max(1, 4 * sms / slabs));
      if (sums && !(a.part = scr.get<float>((size_t)parts * 2 * c))) return FVX_ERR_ALLOC;
      // dw before dx, which may lie in dy's memory
      if (sums)
        FVX_TRY(group ? launch("norm_wide_dw", k_norm_wide_dw<T, VEC, true>, dim3(slabs, parts), 0, s, a)
                      : launch("norm_wide_dw", k_norm_wide_dw<T, VEC, false>, dim3(slabs, parts), 0, s, a));
      return group ? launch("norm_wide_dx", k_norm_wide_dx<T, VEC, true>, dim3(grid), 0, s, a)
                   : launch("norm_wide_dx", k_norm_wide_dx<T, VEC, false>, dim3(grid), 0, s, a);
    }));
  }
  if (!sums) return FVX_OK;
  LaunchScope ls("norm_sum_parts", s);
  k_norm_sum_parts<<<(unsigned)((2 * c + 31) / 32), 32 * kSumRows, 0, s>>>(a.part, parts, (int)c, dw, db);
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
  if (c > kRegCols) return pack_wide(dt, a, (cudaStream_t)stream, sms);
  const int vec = pick_vec(dt, c, a);
  a.lanes = lanes_for(dt, c, vec);
  return rows_launch<kPack>("ck_pack", dt, vec, a, row_grid<kPack>(dt, vec, a, sms), (cudaStream_t)stream);
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
  if (c <= kRegCols) {
    a.lanes = lanes_for(dt, c, vec);
    return mean ? rows_launch<kRestoreNorm>("ck_restore", dt, vec, a, row_grid<kRestoreNorm>(dt, vec, a, sms), s)
                : rows_launch<kRestore>("ck_restore", dt, vec, a, row_grid<kRestore>(dt, vec, a, sms), s);
  }
  const int grid = grid_for(n, 1, sms, 8);
  return by_vec(dt, vec, [&]<typename T, int VEC>() {
    return mean ? launch("ck_restore", k_ck_wide<T, VEC, true>, dim3(grid), 0, s, a)
                : launch("ck_restore", k_ck_wide<T, VEC, false>, dim3(grid), 0, s, a);
  });
}

}  // extern "C"
