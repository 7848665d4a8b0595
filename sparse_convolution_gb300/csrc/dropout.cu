// Dropout from a counter-based generator: the mask is never stored, the
// backward pass draws it again.
//
//   y = residual + (kept ? x / (1 - drop / 65536) : 0),   kept iff bits(i) >= drop
// in one fused multiply-add, whichever kernel runs.
// bits(i): 16 bits for value i of the row-major tensor, eight values per
// counter of Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw 2011):
// counter words (i / 8, offset), key words seed, value i % 8 the i % 8-th
// sixteen bits, low ones first.  They depend on the place in the tensor alone,
// whatever its type, pitch or alignment.
//
// Memory bounds it, and where little of it moves per value the multiplications
// of the counters (twenty 32 x 32 bit products for eight values).  Sixteen bits
// for a value, not thirty-two, halve those: a probability is met to 2^-17.
// Measured: 10,000,000 x 32 bf16 with a residual 273 us (7.0 TB/s), without 224
// (5.7; the products), 5,000,000 x 32 fp32 272 and 187 (7.1, 6.8); 3,000,000 x 101
// bf16 with a residual out of rows of 134 564 us (3.2), 1,000,000 x 257 out of 265
// 341 (3.0; single loads of two bytes).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "fvx_internal.cuh"
#include "norm.cuh"

namespace fvx {
namespace {

struct DropArgs {
  const void* x;
  const void* residual;  // or null
  void* y;
  int64_t total, ldx, ldr, ldy;
  const uint64_t* state;  // seed and offset on the device, or null
  uint64_t seed, offset;
  uint32_t c, vecs, magic, drop;  // vecs: vectors of 8 per row
  float scale;
};

struct Key {
  uint32_t k0, k1, c2, c3;
  __device__ __forceinline__ Key(const DropArgs& a) {
    uint64_t seed = a.seed, offset = a.offset;
    if (a.state) {
      seed = __ldg(reinterpret_cast<const unsigned long long*>(a.state));
      offset += __ldg(reinterpret_cast<const unsigned long long*>(a.state) + 1);
    }
    k0 = (uint32_t)seed;
    k1 = (uint32_t)(seed >> 32);
    c2 = (uint32_t)offset;
    c3 = (uint32_t)(offset >> 32);
  }
};
__device__ __forceinline__ uint4 philox(const Key& key, uint64_t at) {
  uint32_t c0 = (uint32_t)at, c1 = (uint32_t)(at >> 32), c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}
// Bit k: value k of the counter stays.
__device__ __forceinline__ uint32_t kept_bits(uint4 r, uint32_t drop) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m |= (w[k] & 0xffffu) >= drop ? 1u << (2 * k) : 0u;
    m |= (w[k] >> 16) >= drop ? 2u << (2 * k) : 0u;
  }
  return m;
}

// The value kept or dropped: one rounding, the same in every kernel.
template <bool ADD>
__device__ __forceinline__ float dropped(bool keep, float x, float scale, float add) {
  if constexpr (ADD) return keep ? fmaf(x, scale, add) : add;
  return keep ? x * scale : 0.0f;
}

// Vectors of eight values; LINE: the tensors are dense, so the place of value i is i.
template <typename T, bool LINE, bool ADD>
__global__ void __launch_bounds__(kThreads, 6) k_dropout(const __grid_constant__ DropArgs a) {
  const Key key(a);
  const int64_t whole = a.total >> 3, step = (int64_t)gridDim.x * kThreads;
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* res = reinterpret_cast<const T*>(a.residual);
  T* y = reinterpret_cast<T*>(a.y);
  const uint32_t first_kept = a.drop << 16;  // 65536, all dropped, passes the end
  const bool some = a.drop < 65536u;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < whole; i += step) {
    int64_t ax = i * 8, ar = ax, ay = ax;
    if constexpr (!LINE) {
      const int64_t row = whole >> 32 ? i / a.vecs : (uint32_t)i / a.vecs;  // 32-bit division where it will do
      const int64_t col = (i - row * a.vecs) * 8;
      ax = row * a.ldx + col;
      ar = row * a.ldr + col;
      ay = row * a.ldy + col;
    }
    float f[8], g[8];
    load_vec<T, 8>(x + ax, f);
    if constexpr (ADD) load_vec<T, 8>(res + ar, g);
    const uint4 r = philox(key, (uint64_t)i);
    const uint32_t words[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // either half is compared in the upper one's place
      const bool keep = (k & 1 ? words[k / 2] : words[k / 2] << 16) >= first_kept;
      f[k] = dropped<ADD>(keep && some, f[k], a.scale, ADD ? g[k] : 0.0f);
    }
    store_vec<T, 8>(y + ay, f);
  }
  if (LINE && blockIdx.x == 0 && threadIdx.x < (a.total & 7)) {
    const int64_t at = whole * 8 + threadIdx.x;
    const uint32_t m = kept_bits(philox(key, (uint64_t)whole), a.drop);
    const float add = ADD ? Elem<T>::get(res[at]) : 0.0f;
    y[at] = Elem<T>::put(dropped<ADD>((m >> threadIdx.x) & 1u, Elem<T>::get(x[at]), a.scale, add));
  }
}

// x or residual of any pitch and alignment, rows of at least eight values, into
// a dense y: a thread reads its counter's eight values one by one, from one row
// or the end of one and the start of the next, and writes them at once.  Lanes
// sixteen bytes apart use every byte of the lines that they touch.  (Consecutive
// lanes on consecutive values, whose addresses and bits cost more: 3,000,000 x 101
// bf16 of 134 with a residual 659 us, this way 564; 1,000,000 x 257 of 265 476,
// 341; fp32 of half as many rows 343, 299 and 242, 179.)
template <typename T, bool ADD>
__global__ void __launch_bounds__(kThreads, 5) k_dropout_rows(const __grid_constant__ DropArgs a) {
  const Key key(a);
  const int64_t counters = (a.total + 7) >> 3, step = (int64_t)gridDim.x * kThreads;
  const bool small = a.total >> 32 == 0;  // 32-bit division will do
  const uint32_t first_kept = a.drop << 16;
  const bool some = a.drop < 65536u;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < counters; i += step) {
    const int64_t row = small ? (uint32_t)(i * 8) / a.c : i * 8 / a.c;
    const uint32_t col = (uint32_t)(i * 8 - row * a.c);
    const int left = (int)min((int64_t)8, a.total - i * 8);
    auto read = [&](const void* from, int64_t ld, T (&v)[8]) {
      const T* p = reinterpret_cast<const T*>(from) + row * ld + col;
      const T* q = p + (ld - (int64_t)a.c);  // the next row's values, as far on
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) v[k] = (col + k < a.c ? p : q)[k];
    };
    T x[8], g[8];
    read(a.x, a.ldx, x);
    if constexpr (ADD) read(a.residual, a.ldr, g);
    const uint4 r = philox(key, (uint64_t)i);
    const uint32_t words[4] = {r.x, r.y, r.z, r.w};
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool keep = (k & 1 ? words[k / 2] : words[k / 2] << 16) >= first_kept;
      f[k] = k < left ? Elem<T>::get(x[k]) : 0.0f;
      const float add = ADD && k < left ? Elem<T>::get(g[k]) : 0.0f;
      f[k] = dropped<ADD>(keep && some, f[k], a.scale, add);
    }
    T* y = reinterpret_cast<T*>(a.y) + i * 8;
    if (left == 8) {
      store_vec<T, 8>(y, f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) y[k] = Elem<T>::put(f[k]);
    }
  }
}

// Any pitch and alignment of y too: a warp takes 256 consecutive values, 32 at a time;
// lane l draws their l-th counter and hands out its bits.  NEAR: the rows of 256
// values lie within 2^30 values of their first, and offsets from it take 32 bits.
template <typename T, bool ADD, bool NEAR>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const __grid_constant__ DropArgs a) {
  using Off = std::conditional_t<NEAR, uint32_t, int64_t>;
  const Key key(a);
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), spans = (a.total + 255) >> 8;
  const bool small = a.total >> 32 == 0;  // 32-bit division will do
  for (int64_t span = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); span < spans; span += warps) {
    const int64_t row0 = small ? (uint32_t)(span << 8) / a.c : (span << 8) / a.c;
    const uint32_t col0 = (uint32_t)((span << 8) - row0 * a.c) + lane;
    const int left = (int)min((int64_t)256, a.total - (span << 8)) - lane;
    const T* x = reinterpret_cast<const T*>(a.x) + row0 * a.ldx;
    const T* res = reinterpret_cast<const T*>(a.residual) + (ADD ? row0 * a.ldr : 0);
    T* y = reinterpret_cast<T*>(a.y) + row0 * a.ldy;
    // rows below: fewer than 256 columns past a start below c
    auto down_of = [&](uint32_t at) { return a.c >= 512u ? (at >= a.c ? 1u : 0u) : a.c == 1u ? at : __umulhi(at, a.magic); };
    T f[8], g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t at = col0 + 32 * k, down = down_of(at), col = at - down * a.c;
      if (32 * k < left) {
        f[k] = x[(Off)down * (Off)a.ldx + col];
        if constexpr (ADD) g[k] = res[(Off)down * (Off)a.ldr + col];
      }
    }
    const uint32_t m = kept_bits(philox(key, (uint64_t)span * 32 + lane), a.drop);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t bits = __shfl_sync(0xffffffffu, m, 4 * k + (lane >> 3));
      if (32 * k < left) {
        const uint32_t at = col0 + 32 * k, down = down_of(at);
        const float v = dropped<ADD>((bits >> (lane & 7)) & 1u, Elem<T>::get(f[k]), a.scale, ADD ? Elem<T>::get(g[k]) : 0.0f);
        y[(Off)down * (Off)a.ldy + (at - down * a.c)] = Elem<T>::put(v);
      }
    }
  }
}

fvx_status bad(const char* who, const char* what) {
  set_error("%s: %s", who, what);
  return FVX_ERR_INVALID_ARG;
}
fvx_status check_rows_of(const char* who, const char* name, const void* p, int64_t ld, int64_t n, int64_t c, int elem) {
  if (reinterpret_cast<uintptr_t>(p) % elem) {
    set_error("%s: %s is not aligned to its elements", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  if (n > 1 && ld < c) {
    set_error("%s: the row pitch of %s is below the channel count", who, name);
    return FVX_ERR_INVALID_ARG;
  }
  return FVX_OK;
}

template <typename T>
fvx_status run(const DropArgs& a, bool vectors, bool line, bool to_line, int sms, cudaStream_t s) {
  const int64_t threads = vectors || to_line ? (a.total + 7) >> 3 : ((a.total + 255) >> 8) * 32;
  const int blocks = (int)std::min<int64_t>((threads + kThreads - 1) / kThreads, (int64_t)sms * 64);
  // rows that a span of 256 values reaches below its first
  const int64_t rows = 256 / (int64_t)a.c + 2, most = ((int64_t)1 << 30) / rows;
  const bool near = a.ldx < most && a.ldy < most && (!a.residual || a.ldr < most);
  LaunchScope ls("dropout", s);
  auto go = [&]<bool ADD>() {
    if (!vectors && to_line) k_dropout_rows<T, ADD><<<blocks, kThreads, 0, s>>>(a);
    else if (!vectors && near) k_dropout_any<T, ADD, true><<<blocks, kThreads, 0, s>>>(a);
    else if (!vectors) k_dropout_any<T, ADD, false><<<blocks, kThreads, 0, s>>>(a);
    else if (line) k_dropout<T, true, ADD><<<blocks, kThreads, 0, s>>>(a);
    else k_dropout<T, false, ADD><<<blocks, kThreads, 0, s>>>(a);
  };
  if (a.residual) go.template operator()<true>();
  else go.template operator()<false>();
  return check_launch("dropout");
}

}  // namespace
}  // namespace fvx

using namespace fvx;

extern "C" fvx_status fvx_dropout(fvx_dtype dt, const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t n,
                                  int64_t c, double p, uint64_t seed, uint64_t offset, const uint64_t* state, void* y,
                                  int64_t ldy, fvx_stream stream) {
  const char* who = "fvx_dropout";
  EntryScope entry(who);
  if (dt != FVX_F32 && dt != FVX_BF16) return bad(who, "dtype must be FVX_F32 or FVX_BF16");
  if (n < 0 || c < 1) return bad(who, "rows must not be negative, channels at least 1");
  if (c > (int64_t)1 << 60 || n > ((int64_t)1 << 60) / c) return bad(who, "more than 2^60 values");
  if (!(p >= 0.0 && p <= 1.0)) return bad(who, "p must be in 0..1");
  const int elem = dt == FVX_F32 ? 4 : 2;
  if (n > 0 && (!x || !y)) return bad(who, "NULL x or y");
  FVX_TRY(check_rows_of(who, "x", x, ldx, n, c, elem));
  FVX_TRY(check_rows_of(who, "y", y, ldy, n, c, elem));
  if (residual) FVX_TRY(check_rows_of(who, "residual", residual, ldr, n, c, elem));
  if (reinterpret_cast<uintptr_t>(state) % 8) return bad(who, "state is not aligned to 8 bytes");
  if (n == 0) return FVX_OK;
  const bool line = n <= 1 || (ldx == c && ldy == c && (!residual || ldr == c));
  if (!line && c > 0x7fffffff) return bad(who, "rows with gaps must be shorter than 2^31 values");
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  DropArgs a = {};
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.total = n * c;
  // without gaps any cut into rows is as good
  if (line) c = ldx = ldr = ldy = 1 << 20;
  const bool to_line = ldy == c && c >= 8 && reinterpret_cast<uintptr_t>(y) % (8 * elem) == 0;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.state = state;
  a.seed = seed;
  a.offset = offset;
  a.c = (uint32_t)c;
  a.vecs = (uint32_t)(c / 8);
  a.magic = c > 1 ? (uint32_t)(((uint64_t)1 << 32) / (uint64_t)c + 1) : 0;
  a.drop = (uint32_t)lrint(p * 65536.0);
  a.scale = a.drop < 65536 ? (float)(65536.0 / (65536 - (int)a.drop)) : 0.0f;
  auto wide = [&](const void* q, int64_t ld) {
    return reinterpret_cast<uintptr_t>(q) % (8 * elem) == 0 && ld % 8 == 0;
  };
  const bool vectors = wide(x, ldx) && wide(y, ldy) && (!residual || wide(residual, ldr)) && c % 8 == 0;
  return dt == FVX_F32 ? run<float>(a, vectors, line, to_line, sms, (cudaStream_t)stream)
                       : run<__nv_bfloat16>(a, vectors, line, to_line, sms, (cudaStream_t)stream);
}
