// Rows of up to 1024 values: what norm.cu (any layout) and norm_stream_*.cu
// (long dense tensors) do with each.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "fvx_internal.cuh"
#include "tc.cuh"

namespace fvx {

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

// What is done with a row.
enum RowOp { kForward, kForwardCodes, kPack, kBackward, kBackwardCodes, kRestore, kRestoreNorm };

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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width) v += __shfl_xor_sync(0xffffffffu, v, o);
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
  // Both quotients rounded once, as division does, at a third of its work: a
  // first quotient by an approximate reciprocal, corrected by its exact
  // remainder (Markstein 1990; by a constant, Brisebarre, Muller and Raina
  // 2004).  They equal the division for every fp32 value from 2^-100 to
  // 2^126 (all compared); beyond, the reciprocal leaves the normal range.
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(top));
  const float p = __fmul_rn(127.0f, y), q = __fmul_rn(top, 1.0f / 127.0f);
  s.inv = __fmaf_rn(__fmaf_rn(-top, p, 127.0f), y, p);
  s.step = __fmaf_rn(__fmaf_rn(-127.0f, q, top), 1.0f / 127.0f, q);
  if (top_bits - __float_as_uint(kTiny) >= 0x7e800000u - __float_as_uint(kTiny)) {  // not in [2^-100, 2^126)
    if (top < kTiny) s.inv = s.step = 0.0f;
    else s.inv = top_bits >= 0x7f800000u ? 0.0f : __fdiv_rn(127.0f, top);
    if (top_bits >= 0x7f800000u) s.step = __uint_as_float(0x7fc00000u);
  }
  return s;
}
// Codes without the conversion instructions, which run at a sixteenth of the
// rate of the arithmetic: a sum with 1.5 * 2^23 rounds to an integer, half to
// even, and holds it in its low bits; a byte b below the bits of 2^23 is the
// float 2^23 + b.
constexpr float kMagic = 12582912.0f;
// q: x * inv + kMagic, rounded after each; none: a group of zeros, or of NaN,
// whose products are no numbers
template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* p, const float (&q)[VEC], bool none) {
  uint32_t bits[VEC];
  const uint32_t keep = none ? 0u : 0xffffffffu;
#pragma unroll
  for (int j = 0; j < VEC; ++j) bits[j] = __float_as_uint(q[j]);
  if constexpr (VEC % 4 == 0) {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j)
      w[j] = __byte_perm(__byte_perm(bits[4 * j], bits[4 * j + 1], 0x0040), __byte_perm(bits[4 * j + 2], bits[4 * j + 3], 0x0040),
                         0x5410) & keep;
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
    Pack<int8_t, VEC> u;
#pragma unroll
    for (int j = 0; j < VEC; ++j) u.v[j] = (int8_t)(bits[j] & keep & 255u);
    *reinterpret_cast<Pack<int8_t, VEC>*>(p) = u;
  }
}
template <int VEC>
__device__ __forceinline__ void codes_to_float(const Pack<int8_t, VEC>& u, float (&f)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      uint32_t w;
      memcpy(&w, &u.v[j], 4);
      w ^= 0x80808080u;  // code + 128
#pragma unroll
      for (int k = 0; k < 4; ++k) f[j + k] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + k)) - 8388736.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = (float)u.v[j];
  }
}


// Group maxima for the codes.  Lane l of a row holds vectors l, l + lanes, ...
// A group is 2^group_shift values: a run of lanes of one vector index, or (few
// lanes or narrow vectors) all lanes of 2, 4 or more consecutive indices.
template <int PER, int ITER>
__device__ __forceinline__ void group_tops_of(uint32_t (&top)[ITER], int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < PER && o < lanes) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    }
#pragma unroll
  for (int d = 1; d < ITER; d <<= 1) {
    if (PER >= 2 * d * lanes) {
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        if ((i & d) == 0) top[i] = top[i ^ d] = max(top[i], top[i ^ d]);
    }
  }
}
template <int VEC, int ITER>
__device__ __forceinline__ void group_tops(uint32_t (&top)[ITER], int group_shift, int lanes) {
  if (group_shift == 5) group_tops_of<32 / VEC, ITER>(top, lanes);
  else if (group_shift == 6) group_tops_of<64 / VEC, ITER>(top, lanes);
  else group_tops_of<128 / VEC, ITER>(top, lanes);
}

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> raw_vec(const T* p) {
  return *reinterpret_cast<const Pack<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> no_vec() {
  Pack<T, VEC> u;
  memset(&u, 0, sizeof(u));
  return u;
}
template <typename T, int VEC>
__device__ __forceinline__ void widen(const Pack<T, VEC>& u, float (&f)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = Elem<T>::get(u.v[j]);
}

template <int OP>
struct OpIs {
  static constexpr bool kNorm = OP == kForward || OP == kForwardCodes;
  static constexpr bool kBack = OP == kBackward || OP == kBackwardCodes;
  static constexpr bool kFromCodes = OP == kBackwardCodes || OP == kRestore || OP == kRestoreNorm;
  static constexpr bool kToCodes = OP == kForwardCodes || OP == kPack;
  static constexpr bool kStats = kBack || OP == kRestoreNorm;  // mean and rstd are read
};

// A lane's part of a row as stored.
template <typename T, int VEC, int ITER, int OP>
struct RowIn {
  using X = std::conditional_t<OpIs<OP>::kFromCodes, int8_t, T>;
  Pack<X, VEC> x[ITER];
  Pack<T, VEC> dy[OpIs<OP>::kBack ? ITER : 1];
  float step[ITER], mean, rstd;
};

// Values in the pairs that the fp32 units take two at a time (VEC 1: one).
template <int VEC>
struct Lane {
  using E = std::conditional_t<VEC == 1, float, uint64_t>;
  static constexpr int N = VEC == 1 ? 1 : VEC / 2;
};
__device__ __forceinline__ float e_add(float a, float b) { return a + b; }
__device__ __forceinline__ float e_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float e_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float e_sum(float a) { return a; }
__device__ __forceinline__ uint64_t e_add(uint64_t a, uint64_t b) { return tc::add2(a, b); }
__device__ __forceinline__ uint64_t e_mul(uint64_t a, uint64_t b) { return tc::mul2(a, b); }
__device__ __forceinline__ uint64_t e_fma(uint64_t a, uint64_t b, uint64_t c) { return tc::fma2(a, b, c); }
__device__ __forceinline__ float e_sum(uint64_t a) {
  float x, y;
  tc::unpair(a, x, y);
  return x + y;
}
template <typename E>
__device__ __forceinline__ E e_all(float v) {
  if constexpr (sizeof(E) == 4) return v;
  else return tc::pair(v, v);
}
template <int VEC>
__device__ __forceinline__ void to_pairs(const float (&f)[VEC], typename Lane<VEC>::E (&e)[Lane<VEC>::N]) {
  if constexpr (VEC == 1) {
    e[0] = f[0];
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) e[j] = tc::pair(f[2 * j], f[2 * j + 1]);
  }
}
template <int VEC>
__device__ __forceinline__ void from_pairs(const typename Lane<VEC>::E (&e)[Lane<VEC>::N], float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = e[0];
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) tc::unpair(e[j], f[2 * j], f[2 * j + 1]);
  }
}

// Rows of up to 1024 values, `lanes` lanes per row, ITER vectors per lane.  A
// lane keeps the same channels for all its rows: its weights and its parts of
// dw and db stay in registers.  What bounds these kernels beside memory is the
// number of instructions per value, hence the arithmetic in pairs.
// LANES: lanes of a row where the kernel knows them, else 0.
template <typename T, int VEC, int ITER, int OP, int LANES>
struct Rows {
  using Is = OpIs<OP>;
  using In = RowIn<T, VEC, ITER, OP>;
  using E = typename Lane<VEC>::E;
  static constexpr int N = Lane<VEC>::N;
  const RowArgs& a;
  const int lanes, lane, nv;
  const float inv_c;  // means are products with it: half an ulp more than a division, off a row's critical path
  E w[ITER][N], b[ITER][N];    // backward: b unused
  E dw[ITER][N], db[ITER][N];  // backward

  __device__ __forceinline__ Rows(const RowArgs& args)
      : a(args),
        lanes(LANES ? LANES : args.lanes),
        lane(threadIdx.x & (lanes - 1)),
        nv(args.c / VEC),
        inv_c(1.0f / (float)args.c) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int at = (i * lanes + lane) * VEC + j;
        f[j] = a.w && at < a.c ? __ldg(a.w + at) : 1.0f;
      }
      to_pairs<VEC>(f, w[i]);
      if constexpr (!Is::kBack) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int at = (i * lanes + lane) * VEC + j;
          f[j] = a.b && at < a.c ? __ldg(a.b + at) : 0.0f;
        }
        to_pairs<VEC>(f, b[i]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = e_all<E>(0.0f);
      }
    }
  }

  // one row per group of lanes; every lane of the warp takes part in the sums.
  // Lanes without a vector hold zeros (backward: dy's zeros keep them out).
  __device__ __forceinline__ void turn(const In& in, int64_t row, bool live) {
    E x[ITER][N];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float f[VEC];
      if constexpr (Is::kFromCodes) codes_to_float<VEC>(in.x[i], f);
      else widen<T, VEC>(in.x[i], f);
      to_pairs<VEC>(f, x[i]);
      if constexpr (Is::kFromCodes) {
        const E step = e_all<E>(in.step[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) x[i][j] = e_mul(x[i][j], step);
      }
    }
    if constexpr (Is::kToCodes) {
      uint32_t top[ITER];
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        top[i] = 0u;
        if constexpr (sizeof(T) == 2 && VEC >= 2) {
          // the magnitudes of two bf16 values are compared as two 16-bit integers
          uint32_t words[VEC / 2];
          memcpy(words, &in.x[i], sizeof(words));
#pragma unroll
          for (int j = 0; j < VEC / 2; ++j) top[i] = __vmaxu2(top[i], words[j] & 0x7fff7fffu);
          top[i] = max(top[i] << 16, top[i] & 0xffff0000u);
        } else {
          float f[VEC];
          from_pairs<VEC>(x[i], f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) top[i] = max(top[i], mag_bits(f[j]));
        }
      }
      group_tops<VEC, ITER>(top, a.group_shift, lanes);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = i * lanes + lane;
        if (!live || v >= nv) continue;
        const CodeScale cs = code_scale(top[i]);
        float f[VEC];
        from_pairs<VEC>(x[i], f);
        // one by one: a product and a sum in pairs may be contracted to one rounding
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = __fadd_rn(__fmul_rn(f[j], cs.inv), kMagic);
        store_codes<VEC>(a.codes_out + row * a.c + v * VEC, f, cs.inv == 0.0f);
        if (((v * VEC) & ((1 << a.group_shift) - 1)) == 0)
          a.steps_out[row * a.groups + ((v * VEC) >> a.group_shift)] = cs.step;
      }
    }
    if constexpr (Is::kNorm) {
      E s = e_all<E>(0.0f), q = e_all<E>(0.0f);
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) s = e_add(s, x[i][j]);
      const float mean = lanes_sum(e_sum(s), lanes) * inv_c;
      const E minus = e_all<E>(-mean);
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        if (i * lanes + lane < nv) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const E d = e_add(x[i][j], minus);
            q = e_fma(d, d, q);
          }
        }
      const float rstd = rsqrtf(lanes_sum(e_sum(q), lanes) * inv_c + a.eps);
      if (live && lane == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
      }
      apply(x, mean, rstd);
    }
    if constexpr (OP == kRestoreNorm) apply(x, in.mean, in.rstd);
    if constexpr (Is::kBack) {
      const E minus = e_all<E>(-in.mean), scale = e_all<E>(in.rstd);
      E g[ITER][N], sum_g = e_all<E>(0.0f), sum_gx = e_all<E>(0.0f);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        float f[VEC];
        widen<T, VEC>(in.dy[i], f);
        to_pairs<VEC>(f, g[i]);
        if (live && i * lanes + lane < nv) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            x[i][j] = e_mul(e_add(x[i][j], minus), scale);
            dw[i][j] = e_fma(g[i][j], x[i][j], dw[i][j]);
            db[i][j] = e_add(g[i][j], db[i][j]);
            g[i][j] = e_mul(g[i][j], w[i][j]);
            sum_g = e_add(g[i][j], sum_g);
            sum_gx = e_fma(g[i][j], x[i][j], sum_gx);
          }
        }
      }
      const E mean_g = e_all<E>(-lanes_sum(e_sum(sum_g), lanes) * inv_c),
              mean_gx = e_all<E>(-lanes_sum(e_sum(sum_gx), lanes) * inv_c);
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) x[i][j] = e_mul(scale, e_fma(x[i][j], mean_gx, e_add(g[i][j], mean_g)));
    }
    if constexpr (OP != kPack) {
      if (!live) return;
      T* py = reinterpret_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = i * lanes + lane;
        float f[VEC];
        from_pairs<VEC>(x[i], f);
        if (v < nv) store_vec<T, VEC>(py + v * VEC, f);
      }
    }
  }
  __device__ __forceinline__ void apply(E (&x)[ITER][N], float mean, float rstd) {
    const E minus = e_all<E>(-mean), scale = e_all<E>(rstd);
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) x[i][j] = e_fma(e_mul(e_add(x[i][j], minus), scale), w[i][j], b[i][j]);
  }

  // the row from global memory; zeros where there is none
  __device__ __forceinline__ void fetch(In& in, int64_t row, bool live) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = i * lanes + lane;
      const bool here = live && v < nv;
      in.step[i] = 0.0f;
      if constexpr (Is::kFromCodes) {
        in.x[i] = here ? raw_vec<int8_t, VEC>(a.codes + row * a.c + v * VEC) : no_vec<int8_t, VEC>();
        if (here) in.step[i] = __ldg(a.steps + row * a.groups + ((v * VEC) >> a.group_shift));
      } else {
        in.x[i] = here ? raw_vec<T, VEC>(reinterpret_cast<const T*>(a.x) + row * a.ldx + v * VEC) : no_vec<T, VEC>();
      }
      if constexpr (Is::kBack)
        in.dy[i] = here ? raw_vec<T, VEC>(reinterpret_cast<const T*>(a.dy) + row * a.lddy + v * VEC) : no_vec<T, VEC>();
    }
    in.mean = in.rstd = 0.0f;
    if constexpr (Is::kStats) {
      if (live) {
        in.mean = __ldg(a.mean_in + row);
        in.rstd = __ldg(a.rstd_in + row);
      }
    }
  }

  // rows first, first + step, ... of [0, n), one per group of lanes and turn
  __device__ __forceinline__ void direct(int64_t first, int64_t step, int64_t n) {
    // every lane of a warp takes the same number of turns (the shuffles need them all)
    const int64_t row0 = first + threadIdx.x / lanes;
    const int64_t turns = first < n ? (n - first + step - 1) / step : 0;
    for (int64_t t = 0; t < turns; ++t) {
      const int64_t row = row0 + t * step;
      In in;
      fetch(in, row, row < n);
      turn(in, row, row < n);
    }
  }

  // dw and db of the block, its groups of lanes added in a fixed order
  __device__ __forceinline__ void write_parts(float* sh, int threads) {
    if (!a.part) return;
    const int groups = threads / lanes, sub = threadIdx.x / lanes;
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
      if ((int)threadIdx.x < threads) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          float f[VEC];
          from_pairs<VEC>(pass ? db[i] : dw[i], f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int at = (i * lanes + lane) * VEC + j;
            if (at < a.c) sh[sub * a.c + at] = f[j];
          }
        }
      }
      __syncthreads();
      for (int at = threadIdx.x; at < a.c; at += blockDim.x) {
        float s = 0.0f;
        for (int k = 0; k < groups; ++k) s += sh[k * a.c + at];
        a.part[((int64_t)blockIdx.x * 2 + pass) * a.c + at] = s;
      }
    }
  }
};

}  // namespace

constexpr int kStreamStages = 6;
struct StreamArgs {
  RowArgs r;
  int64_t stages;  // full stages of the tensor
  int rows;        // of a stage
  int stage_bytes;
  int off_dy, off_steps, off_mean, off_rstd;  // behind x or the codes
  uint32_t* status;
};
// The streaming kernels of one storage type (norm_stream_f32.cu, norm_stream_bf16.cu).
fvx_status stream_rows_f32(const char* name, RowOp op, int iters, const StreamArgs& a, int blocks, size_t smem,
                           cudaStream_t s);
fvx_status stream_rows_bf16(const char* name, RowOp op, int iters, const StreamArgs& a, int blocks, size_t smem,
                            cudaStream_t s);

}  // namespace fvx
