// Cross attention of a few query rows per key head (a query token or a few of
// each sample, times the heads that share a key head): the single-token form.
//
// Each key and value is read once and meets at most eight rows, so memory
// bounds the call, and the tensor cores' tiles of 128 rows would mostly be
// empty.  A work unit is a key head of a sample; its keys are cut into equal
// ranges for the blocks of a cluster (and, for very long samples, for several
// clusters), a block's range is dealt to its warps, and LK lanes hold one key.
// What bounds the kernel then is the number of instructions per key, so the dot
// products of a turn (rows x keys in flight) are summed over the lanes by
// exchanging halves, which leaves each lane one of them, one power to take and
// one sum to keep; the accumulators are brought to a new maximum only when it
// exceeds the old by 2^8.  Groups, warps and the cluster's blocks join their
// results through shuffles, shared and distributed shared memory, in a fixed
// order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "attn.cuh"
#include "tc.cuh"

namespace fvx {
namespace {

namespace cg = cooperative_groups;

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 8;     // most rows of a unit
constexpr int kFewCluster = 8;  // most blocks of a cluster (the portable limit)
constexpr float kLazy = 8.0f;   // growth of the maximum (in powers of 2) that the sums may lag behind
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct FewArgs {
  AttnItems items;
  HeadsView q, k, v;
  const uint8_t* mask;
  void* out;
  float* lse;
  float *part, *top, *total;  // several clusters per unit: [range][nq * heads][d], [range][nq * heads]
  int64_t all_rows;
  int heads, kv_heads, shared, d, ranges, blocks;  // ranges: clusters per unit; blocks of a cluster
  float c;                                         // scale * log2(e)
};

// 16 bytes as pairs of fp32 values
template <typename T>
__device__ __forceinline__ void widen16(uint4 u, uint64_t* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 4) {
    f[0] = tc::pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
    f[1] = tc::pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = tc::pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}

template <typename T, int LK, int R>
__global__ void __launch_bounds__(kFewThreads, R <= 4 ? 2 : 1) k_attn_few(const __grid_constant__ FewArgs a) {
  constexpr int V = 16 / sizeof(T), P = V / 2;  // values and pairs of a lane
  constexpr int kGroups = 32 / LK;              // keys of a warp at once
  constexpr int D = LK * V;                     // the head's size, rounded up
  constexpr int F = R <= 2 ? 8 : 4;             // keys of a lane group in flight
  constexpr int N = R * F;                      // dot products of a turn, number r * F + i
  constexpr int M = N > LK ? N / LK : 1;        // that a lane keeps
  constexpr int kShare = N > LK ? 1 : LK / N;   // lanes that keep the same one
  constexpr int kRowLanes = LK / R;             // lanes that keep a row's
  static_assert(R <= LK, "a lane keeps products of one row");
  __shared__ float s_acc[kFewWarps][R][D], s_top[kFewWarps][R], s_sum[kFewWarps][R];
  __shared__ float b_acc[R][D], b_top[R], b_sum[R];  // the block's result
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane % LK, group = lane / LK;
  const int rank = blockIdx.x % a.blocks;
  int u = blockIdx.x / a.blocks;
  const int range = u % a.ranges;
  u /= a.ranges;
  const int b = a.items.item_of(u);
  const int h = u - a.items.u0(b);
  const int q0 = a.items.q0(b), rows = (a.items.q0(b + 1) - q0) * a.shared;
  const int key0 = a.items.k0(b), keys = a.items.k0(b + 1) - key0;
  const int pieces = a.ranges * a.blocks, piece = range * a.blocks + rank;
  const int from = (int)((int64_t)keys * piece / pieces), to = (int)((int64_t)keys * (piece + 1) / pieces);
  const bool mine = part * V < a.d;

  uint64_t q[R][P], acc2[R][P];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && mine) {
      const int tok = r / a.shared, g = r - tok * a.shared;
      w = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q.p) + (int64_t)(q0 + tok) * a.q.token +
                                          (int64_t)(h * a.shared + g) * a.q.head + part * V);
    }
    widen16<T>(w, q[r]);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      q[r][j] = tc::mul2(q[r][j], tc::pair(a.c, a.c));
      acc2[r][j] = tc::pair(0.0f, 0.0f);
    }
  }
  float my_top = -INFINITY, my_sum = 0.0f;  // of the row whose products this lane keeps
  const T* const pk = reinterpret_cast<const T*>(a.k.p) + (int64_t)h * a.k.head + part * V;
  const T* const pv = reinterpret_cast<const T*>(a.v.p) + (int64_t)h * a.v.head + part * V;
  constexpr int kStep = kFewWarps * kGroups * F;
  for (int j0 = from + warp * kGroups * F + group; j0 - group < to; j0 += kStep) {
    uint4 kw[F], vw[F];
    uint32_t kept = 0;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int j = j0 + i * kGroups;
      kw[i] = vw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (j < to) kept |= 1u << i;
      if (j < to && mine) {
        kw[i] = __ldg(reinterpret_cast<const uint4*>(pk + (int64_t)(key0 + j) * a.k.token));
        vw[i] = __ldg(reinterpret_cast<const uint4*>(pv + (int64_t)(key0 + j) * a.v.token));
      }
    }
    if (a.mask) {
      // the rows of dropped keys are fetched, not waited for, and read as zeros
#pragma unroll
      for (int i = 0; i < F; ++i)
        if (((kept >> i) & 1u) && __ldg(a.mask + key0 + j0 + i * kGroups) == 0) kept &= ~(1u << i);
#pragma unroll
      for (int i = 0; i < F; ++i)
        if (!((kept >> i) & 1u)) kw[i] = vw[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    float s[N];
#pragma unroll
    for (int i = 0; i < F; ++i) {
      uint64_t k[P];
      widen16<T>(kw[i], k);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint64_t x = tc::mul2(q[r][0], k[0]);
#pragma unroll
        for (int j = 1; j < P; ++j) x = tc::fma2(q[r][j], k[j], x);
        float lo, hi;
        tc::unpair(x, lo, hi);
        s[r * F + i] = lo + hi;
      }
    }
    // sums over the LK lanes: each step sends the half that the other lane keeps
#pragma unroll
    for (int o = LK / 2, count = N; o > 0; o >>= 1) {
      if (count > 1) {
        count /= 2;
        const bool upper = (part & o) != 0;
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          if (k >= count) break;
          const float send = upper ? s[k] : s[k + count], keep = upper ? s[k + count] : s[k];
          s[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const int number = N > LK ? part * M + k : part / kShare;
      if (!((kept >> (number % F)) & 1u)) s[k] = -INFINITY;
      m = fmaxf(m, s[k]);
    }
#pragma unroll
    for (int o = kRowLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, m > my_top + kLazy)) {
      const float top = fmaxf(m, my_top), fade = my_top == -INFINITY ? 0.0f : tc::exp2_fast(my_top - top);
      my_top = top;
      my_sum *= fade;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xffffffffu, fade, group * LK + r * kRowLanes);
#pragma unroll
        for (int j = 0; j < P; ++j) acc2[r][j] = tc::mul2(acc2[r][j], tc::pair(f, f));
      }
    }
    const float base = my_top == -INFINITY ? 0.0f : my_top;
#pragma unroll
    for (int k = 0; k < M; ++k) {
      s[k] = tc::exp2_fast(s[k] - base);
      my_sum += s[k];
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
      uint64_t v[P];
      widen16<T>(vw[i], v);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int number = r * F + i;
        const float w = __shfl_sync(0xffffffffu, s[number % M], group * LK + (N > LK ? number / M : number * kShare));
#pragma unroll
        for (int j = 0; j < P; ++j) acc2[r][j] = tc::fma2(v[j], tc::pair(w, w), acc2[r][j]);
      }
    }
  }
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) my_sum += __shfl_xor_sync(0xffffffffu, my_sum, o);
  my_sum *= 1.0f / kShare;
  float top[R], sum[R], acc[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    top[r] = __shfl_sync(0xffffffffu, my_top, group * LK + r * kRowLanes);
    sum[r] = __shfl_sync(0xffffffffu, my_sum, group * LK + r * kRowLanes);
#pragma unroll
    for (int j = 0; j < P; ++j) tc::unpair(acc2[r][j], acc[r][2 * j], acc[r][2 * j + 1]);
  }
  // the warp's lane groups
#pragma unroll
  for (int o = LK; o < 32; o <<= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float other = __shfl_xor_sync(0xffffffffu, top[r], o);
      const float m = fmaxf(top[r], other), base = m == -INFINITY ? 0.0f : m;
      const float f = tc::exp2_fast(top[r] - base), g = tc::exp2_fast(other - base);
      // the same sum in the same order on both sides: low lanes first
      const bool low = (lane & o) == 0;
      const float so = __shfl_xor_sync(0xffffffffu, sum[r], o);
      sum[r] = low ? fmaf(sum[r], f, so * g) : fmaf(so, g, sum[r] * f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = __shfl_xor_sync(0xffffffffu, acc[r][j], o);
        acc[r][j] = low ? fmaf(acc[r][j], f, x * g) : fmaf(x, g, acc[r][j] * f);
      }
      top[r] = m;
    }
  }
  if (group == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int j = 0; j < V; ++j) s_acc[warp][r][part * V + j] = acc[r][j];
      if (part == 0) {
        s_top[warp][r] = top[r];
        s_sum[warp][r] = sum[r];
      }
    }
  }
  __syncthreads();
  // the block's warps
  for (int e = threadIdx.x; e < R * D; e += kFewThreads) {
    const int r = e / D, col = e - r * D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, s_top[w][r]);
    const float base = m == -INFINITY ? 0.0f : m;
    float x = 0.0f, t = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float f = tc::exp2_fast(s_top[w][r] - base);
      x = fmaf(s_acc[w][r][col], f, x);
      t = fmaf(s_sum[w][r], f, t);
    }
    b_acc[r][col] = x;
    if (col == 0) {
      b_top[r] = m;
      b_sum[r] = t;
    }
  }
  // the cluster's blocks: each writes its share of the columns
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int e = rank * kFewThreads + threadIdx.x; e < R * D; e += a.blocks * kFewThreads) {
    const int r = e / D, col = e - r * D;
    if (r >= rows || col >= a.d) continue;
    float tops[kFewCluster], m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewCluster; ++w) {
      tops[w] = w < a.blocks ? *cluster.map_shared_rank(&b_top[r], w) : -INFINITY;
      m = fmaxf(m, tops[w]);
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float x = 0.0f, t = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewCluster; ++w) {
      if (w >= a.blocks) break;
      const float f = tc::exp2_fast(tops[w] - base);
      x = fmaf(*cluster.map_shared_rank(&b_acc[r][col], w), f, x);
      t = fmaf(*cluster.map_shared_rank(&b_sum[r], w), f, t);
    }
    const int tok = r / a.shared, g = r - tok * a.shared;
    const int64_t row = (int64_t)(q0 + tok) * a.heads + h * a.shared + g;
    if (a.ranges == 1) {
      const float y = t > 0.0f ? x / t : x * 0.0f;  // a NaN stays one
      if constexpr (sizeof(T) == 4) reinterpret_cast<float*>(a.out)[row * a.d + col] = y;
      else reinterpret_cast<__nv_bfloat16*>(a.out)[row * a.d + col] = __float2bfloat16_rn(y);
      if (col == 0) a.lse[row] = (m + log2f(t)) * kLn2;
    } else {
      const int64_t at = (int64_t)range * a.all_rows + row;
      a.part[at * a.d + col] = x;
      if (col == 0) {
        a.top[at] = m * kLn2;
        a.total[at] = t;
      }
    }
  }
  cluster.sync();  // nobody leaves while its memory is read
}

template <typename T, int LK, int R>
fvx_status launch_few(const FewArgs& a, int64_t grid, cudaStream_t s) {
  LaunchScope ls("attn_few", s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)a.blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  FVX_CUDA(cudaLaunchKernelEx(&cfg, k_attn_few<T, LK, R>, a));
  return check_launch("attn_few");
}
template <typename T, int LK>
fvx_status few_by_rows(const FewArgs& a, int rows, int64_t grid, cudaStream_t s) {
  if (rows <= 1) return launch_few<T, LK, 1>(a, grid, s);
  if (rows <= 2) return launch_few<T, LK, 2>(a, grid, s);
  if (rows <= 4) return launch_few<T, LK, 4>(a, grid, s);
  return launch_few<T, LK, 8>(a, grid, s);
}

int64_t most_rows(const AttnCall& c) {
  int64_t most = 0;
  for (int b = 0; b < c.items; ++b) most = std::max(most, (c.q_offsets[b + 1] - c.q_offsets[b]) * c.shared);
  return most;
}

bool loads16(const HeadsView& t, int elem) {
  const int per = 16 / elem;
  return reinterpret_cast<uintptr_t>(t.p) % 16 == 0 && t.token % per == 0 && t.head % per == 0;
}

}  // namespace

// At most eight rows per key head of every sample, and rows that 16-byte loads
// can read.
bool attn_few_serves(const AttnCall& c) {
  const int elem = c.dt == FVX_F32 ? 4 : 2;
  if (c.d % (16 / elem) || c.nk == 0 || most_rows(c) > kFewRows) return false;
  return loads16(c.q, elem) && loads16(c.k, elem) && loads16(c.v, elem);
}

fvx_status attn_few_forward(const AttnCall& c, cudaStream_t s, Scratch& scr) {
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  FewArgs a;
  std::vector<int32_t> prefix((size_t)c.items + 1);
  int64_t units = 0, longest = 0;
  for (int b = 0; b < c.items; ++b) {
    prefix[b] = (int32_t)units;
    if (c.q_offsets[b + 1] == c.q_offsets[b]) continue;
    units += c.kv_heads;
    longest = std::max(longest, c.kv_offsets[b + 1] - c.kv_offsets[b]);
  }
  prefix[c.items] = (int32_t)units;
  FVX_TRY(attn_items(c, prefix.data(), 3, s, scr, &a.items));
  // Blocks of at least 128 keys (a turn of all warps), at most two per
  // multiprocessor; several clusters per unit, whose results another kernel
  // joins, only where one each leaves multiprocessors idle.
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(2 * sms / std::max<int64_t>(units, 1), (longest + 127) / 128));
  a.blocks = want >= 8 ? 8 : want >= 4 ? 4 : want >= 2 ? 2 : 1;
  a.ranges = units * kFewCluster < sms ? (int)std::min<int64_t>(64, want / a.blocks) : 1;
  a.q = c.q;
  a.k = c.k;
  a.v = c.v;
  a.mask = c.mask;
  a.out = c.out;
  a.lse = c.lse;
  a.part = a.top = a.total = nullptr;
  a.all_rows = c.nq * c.heads;
  if (a.ranges > 1) {
    a.part = scr.get<float>((size_t)a.ranges * a.all_rows * c.d);
    a.top = scr.get<float>((size_t)a.ranges * a.all_rows);
    a.total = scr.get<float>((size_t)a.ranges * a.all_rows);
    if (!a.part || !a.top || !a.total) return FVX_ERR_ALLOC;
  }
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.shared = c.shared;
  a.d = c.d;
  a.c = c.scale * kLog2e;
  const int64_t grid = units * a.ranges * a.blocks;
  const int rows = (int)most_rows(c);
  fvx_status st;
  if (c.dt == FVX_F32) {
    if (c.d <= 32) st = few_by_rows<float, 8>(a, rows, grid, s);
    else if (c.d <= 64) st = few_by_rows<float, 16>(a, rows, grid, s);
    else st = few_by_rows<float, 32>(a, rows, grid, s);
  } else {
    if (c.d <= 64) st = few_by_rows<__nv_bfloat16, 8>(a, rows, grid, s);
    else st = few_by_rows<__nv_bfloat16, 16>(a, rows, grid, s);
  }
  FVX_TRY(st);
  return a.ranges > 1 ? attn_join(c, a.part, a.top, a.total, a.ranges, s) : FVX_OK;
}

}  // namespace fvx
