// Cross attention of a few query rows per key head (a query token or a few of
// each sample, times the heads that share a key head): the single-token form.
//
// Each key and value is read once and meets at most eight rows, so memory
// bounds the call, and the 128 rows of a tcgen05 product would mostly be empty.
// A work unit is a key head of a sample; its keys are cut into equal ranges for
// the blocks of a cluster (and, for very long samples, for several clusters),
// and a block's range is dealt to its warps.  A warp copies the keys and values
// of its next turns into its own ring in shared memory while it computes, and
// nothing but its own copies makes it wait.  The running maximum of a row is
// raised only when a score exceeds it by 2^8, so the accumulators are rarely
// touched; powers come from the special function unit in fp32 too (relative
// error about 2^-22; the rounding of a score of 10 makes 2^-21); warps and the cluster's blocks join their results through shared and
// distributed shared memory, in a fixed order.
//
// bf16: the products are m16n8k16 with the keys as the 16 and the rows as the
// 8: S' = K Q', then O' = V' P', whose accumulators lie in the same lanes as
// the scores of their rows.  That is a third of the instructions of scalar
// products, which are what bounded the call before.
// fp32: LK lanes hold one key; the dot products of a turn (rows x keys) are
// summed over the lanes by exchanging halves, which leaves each lane one of
// them, one power to take and one sum to keep.
//
// Measured: 8 samples of one token on 777 to 4096 keys, 16 heads on 4 key heads
// of 128, 18 us (2.6 TB/s; a block has eight turns, so the latencies of the
// first loads and of the joins are most of it); 32 samples on 8192 keys, 4 key
// heads of 128, one row each 94 us (5.7 TB/s), eight rows 99; the same in fp32
// with one row 170 us (6.3 TB/s).
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

constexpr int kFewThreads = 128, kFewWarps = kFewThreads / 32;
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

// What a block computes: a range of a key head's keys.
struct FewPiece {
  int rank, range, h, q0, rows, key0, from, to;
};
__device__ __forceinline__ FewPiece few_piece(const FewArgs& a) {
  FewPiece p;
  p.rank = blockIdx.x % a.blocks;
  int u = blockIdx.x / a.blocks;
  p.range = u % a.ranges;
  u /= a.ranges;
  const int b = a.items.item_of(u);
  p.h = u - a.items.u0(b);
  p.q0 = a.items.q0(b);
  p.rows = (a.items.q0(b + 1) - p.q0) * a.shared;
  p.key0 = a.items.k0(b);
  const int keys = a.items.k0(b + 1) - p.key0;
  const int pieces = a.ranges * a.blocks, piece = p.range * a.blocks + p.rank;
  p.from = (int)((int64_t)keys * piece / pieces);
  p.to = (int)((int64_t)keys * (piece + 1) / pieces);
  return p;
}

// The results of the block's warps, each [rows][D] at w * pitch floats, its
// maxima (in powers of 2) and sums, joined, and then those of the cluster's
// blocks, each of which writes its share of the columns.  b_acc: shared memory
// for [kFewRows][D].
template <typename T, int D>
__device__ __forceinline__ void few_join(const FewArgs& a, const FewPiece& p, const float* w_acc, int pitch,
                                         const float (*w_top)[kFewRows], const float (*w_sum)[kFewRows], float* b_acc,
                                         float* b_top, float* b_sum) {
  __syncthreads();
  for (int e = threadIdx.x; e < p.rows * D; e += kFewThreads) {
    const int r = e / D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, w_top[w][r]);
    const float base = m == -INFINITY ? 0.0f : m;
    float x = 0.0f, t = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float f = tc::exp2_fast(w_top[w][r] - base);
      x = fmaf(w_acc[w * pitch + e], f, x);
      t = fmaf(w_sum[w][r], f, t);
    }
    b_acc[e] = x;
    if (e % D == 0) {
      b_top[r] = m;
      b_sum[r] = t;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int e = p.rank * kFewThreads + threadIdx.x; e < p.rows * D; e += a.blocks * kFewThreads) {
    const int r = e / D, col = e - r * D;
    if (col >= a.d) continue;
    float tops[kFewCluster], m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewCluster; ++w) {
      tops[w] = w < a.blocks ? *cluster.map_shared_rank(b_top + r, w) : -INFINITY;
      m = fmaxf(m, tops[w]);
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float x = 0.0f, t = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewCluster; ++w) {
      if (w >= a.blocks) break;
      const float f = tc::exp2_fast(tops[w] - base);
      x = fmaf(*cluster.map_shared_rank(b_acc + e, w), f, x);
      t = fmaf(*cluster.map_shared_rank(b_sum + r, w), f, t);
    }
    const int tok = r / a.shared, g = r - tok * a.shared;
    const int64_t row = (int64_t)(p.q0 + tok) * a.heads + p.h * a.shared + g;
    if (a.ranges == 1) {
      const float y = t > 0.0f ? x / t : x * 0.0f;  // a NaN stays one
      if constexpr (sizeof(T) == 4) reinterpret_cast<float*>(a.out)[row * a.d + col] = y;
      else reinterpret_cast<__nv_bfloat16*>(a.out)[row * a.d + col] = __float2bfloat16_rn(y);
      if (col == 0) a.lse[row] = (m + log2f(t)) * kLn2;
    } else {
      const int64_t at = (int64_t)p.range * a.all_rows + row;
      a.part[at * a.d + col] = x;
      if (col == 0) {
        a.top[at] = m * kLn2;
        a.total[at] = t;
      }
    }
  }
  cluster.sync();  // nobody leaves while its memory is read
}

// ---------------------------------------------------------------- fp32

constexpr int kF32Stages = 3;                        // turns of a warp's ring: one that is read, two under way
constexpr int kFlight = 4;                           // keys of a lane group in a turn
constexpr int kF32Stage = kFlight * 2 * 32 * 16;     // bytes of a turn
constexpr int kF32Ring = kF32Stages * kF32Stage;     // of a warp

__device__ __forceinline__ void widen16(uint4 u, uint64_t* f) {
  f[0] = tc::pair(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = tc::pair(__uint_as_float(u.z), __uint_as_float(u.w));
}

template <int LK, int R>
__global__ void __launch_bounds__(kFewThreads, R <= 4 ? 4 : 2) k_attn_few_f32(const __grid_constant__ FewArgs a) {
  constexpr int V = 4, P = 2;                   // values and pairs of a lane
  constexpr int kGroups = 32 / LK;              // keys of a warp at once
  constexpr int D = LK * V;                     // the head's size, rounded up
  constexpr int F = kFlight;
  constexpr int N = R * F;                      // dot products of a turn, number r * F + i
  constexpr int M = N > LK ? N / LK : 1;        // that a lane keeps
  constexpr int kShare = N > LK ? 1 : LK / N;   // lanes that keep the same one
  constexpr int kRowLanes = LK / R;             // lanes that keep a row's
  constexpr int kStages = kF32Stages, kStageBytes = kF32Stage, kRing = kF32Ring;
  static_assert(R <= LK, "a lane keeps products of one row");
  static_assert(R * D * 4 <= kRing, "a warp's result lies over its own ring");
  extern __shared__ uint4 ring[];
  __shared__ float s_top[kFewWarps][kFewRows], s_sum[kFewWarps][kFewRows];
  __shared__ float b_acc[R * D], b_top[kFewRows], b_sum[kFewRows];  // the block's result
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane % LK, group = lane / LK;
  const FewPiece p = few_piece(a);
  const bool mine = part * V < a.d;

  uint64_t q[R][P], acc2[R][P];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < p.rows && mine) {
      const int tok = r / a.shared, g = r - tok * a.shared;
      w = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(a.q.p) + (int64_t)(p.q0 + tok) * a.q.token +
                                          (int64_t)(p.h * a.shared + g) * a.q.head + part * V);
    }
    widen16(w, q[r]);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      q[r][j] = tc::mul2(q[r][j], tc::pair(a.c, a.c));
      acc2[r][j] = tc::pair(0.0f, 0.0f);
    }
  }
  float my_top = -INFINITY, my_sum = 0.0f;  // of the row whose products this lane keeps
  const float* const pk = reinterpret_cast<const float*>(a.k.p) + (int64_t)p.h * a.k.head + part * V;
  const float* const pv = reinterpret_cast<const float*>(a.v.p) + (int64_t)p.h * a.v.head + part * V;
  constexpr int kStep = kFewWarps * kGroups * F;
  // A lane copies what it will read itself, so a turn waits for the lane's own
  // copies only.
  uint4* const mine_ring = ring + warp * (kRing / 16) + lane;
  const int first = p.from + warp * kGroups * F + group;
  auto fetch = [&](int j0, int stage, uint32_t& kept) {
    uint4* const dst = mine_ring + stage * (kStageBytes / 16);
    kept = 0;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int j = j0 + i * kGroups;
      const bool in = j < p.to;
      const int64_t at = p.key0 + (in ? j : 0);
      if (mine) {
        tc::copy16(tc::smem_u32(dst + i * 32), pk + at * a.k.token, in);
        tc::copy16(tc::smem_u32(dst + (F + i) * 32), pv + at * a.v.token, in);
      }
      if (in) kept |= (a.mask ? (uint32_t)__ldg(a.mask + at) : 1u) << (8 * i);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  static_assert(F <= 4, "a mask's bytes lie in a word");
  if (!mine) {
#pragma unroll
    for (int i = 0; i < kStages * 2 * F; ++i) mine_ring[i * 32] = make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t bytes[kStages - 1];
#pragma unroll
  for (int p = 0; p < kStages - 1; ++p) fetch(first + p * kStep, p, bytes[p]);
  int stage = 0;
  for (int j0 = first; j0 - group < p.to; j0 += kStep) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    const uint32_t now = bytes[0];
#pragma unroll
    for (int p = 0; p + 2 < kStages; ++p) bytes[p] = bytes[p + 1];
    // into the stage that the last turn has read
    fetch(j0 + (kStages - 1) * kStep, stage == 0 ? kStages - 1 : stage - 1, bytes[kStages - 2]);
    uint4* const src = mine_ring + stage * (kStageBytes / 16);
    uint32_t kept = 0;
#pragma unroll
    for (int i = 0; i < F; ++i) kept |= (now >> (8 * i) & 0xffu) ? 1u << i : 0u;
    uint4 kw[F], vw[F];
#pragma unroll
    for (int i = 0; i < F; ++i) {
      kw[i] = src[i * 32];
      vw[i] = src[(F + i) * 32];
      if (!((kept >> i) & 1u)) vw[i] = make_uint4(0u, 0u, 0u, 0u);  // a dropped value may be anything
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float s[N];
#pragma unroll
    for (int i = 0; i < F; ++i) {
      uint64_t k[P];
      widen16(kw[i], k);
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
      widen16(vw[i], v);
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
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  auto s_acc = [&](int w) { return reinterpret_cast<float*>(ring + w * kRing / 16); };  // [R][D]
  if (group == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int j = 0; j < V; ++j) s_acc(warp)[r * D + part * V + j] = acc[r][j];
      if (part == 0) {
        s_top[warp][r] = top[r];
        s_sum[warp][r] = sum[r];
      }
    }
  }
  few_join<float, D>(a, p, reinterpret_cast<const float*>(ring), kRing / 4, s_top, s_sum, b_acc, b_top, b_sum);
}

// ---------------------------------------------------------------- bf16

constexpr int kTurn = 16;  // keys of a warp's turn
template <int DP>
struct FewBf16 {
  static constexpr int kStages = DP > 64 ? 3 : 4;  // turns of a warp's ring: one that is read, the others under way
  static constexpr int kTile = kTurn * DP * 2;     // bytes of a turn's keys, and of its values
  static constexpr int kRing = kStages * 2 * kTile;
};

__device__ __forceinline__ void load4(uint32_t (&f)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void load4_transposed(uint32_t (&f)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void product(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Lane l of a warp holds, of the scores and of the results, the rows
// 2 (l % 4) and 2 (l % 4) + 1; of the scores the keys l / 4 and l / 4 + 8 of a
// turn, of the results the dimensions l / 4 and l / 4 + 8 of every 16.
template <int DP>
__global__ void __launch_bounds__(kFewThreads, DP > 64 ? 2 : 3) k_attn_few_bf16(const __grid_constant__ FewArgs a) {
  using C = FewBf16<DP>;
  constexpr int kStages = C::kStages;
  constexpr int kChunks = DP / 8;             // pieces of 16 bytes of a key
  constexpr int kAtOnce = 32 / kChunks;       // keys that the warp copies at once
  constexpr int kCopies = kTurn / kAtOnce;
  static_assert(kFewRows * DP * 4 <= C::kRing, "a warp's result lies over its own ring");
  extern __shared__ uint4 ring[];
  __shared__ float s_top[kFewWarps][kFewRows], s_sum[kFewWarps][kFewRows];
  __shared__ float b_acc[kFewRows * DP], b_top[kFewRows], b_sum[kFewRows];  // the block's result
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const FewPiece p = few_piece(a);

  // copies: a lane's piece of a key, and the key among those copied at once; a
  // key's pieces are permuted by its number, so that eight keys' pieces of one
  // number lie in different banks
  const int chunk = lane % kChunks, sub = lane / kChunks;
  const bool mine = chunk * 8 < a.d;
  const __nv_bfloat16* pk = reinterpret_cast<const __nv_bfloat16*>(a.k.p) + (int64_t)p.h * a.k.head + chunk * 8;
  const __nv_bfloat16* pv = reinterpret_cast<const __nv_bfloat16*>(a.v.p) + (int64_t)p.h * a.v.head + chunk * 8;
  const uint32_t my_ring = tc::smem_u32(ring) + warp * C::kRing;
  constexpr int kStep = kFewWarps * kTurn;
  const int first = p.from + warp * kTurn;
  const uint8_t* const mask = a.mask ? a.mask + p.key0 : nullptr;
  // bit i: key j0 + i is in range and kept
  auto flag = [&](int j0) -> uint32_t {
    const int j = j0 + lane;
    if (lane >= kTurn || j >= p.to) return 0u;
    return mask ? (uint32_t)__ldg(mask + j) : 1u;
  };
  auto fetch = [&](int j0, int stage, uint32_t kept) {
    const uint32_t dst = my_ring + stage * 2 * C::kTile;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int key = i * kAtOnce + sub;
      const bool in = ((kept >> key) & 1u) && mine;  // zeros for what is dropped, whatever lies there
      const int64_t at = p.key0 + (in ? j0 + key : 0);
      const uint32_t to = dst + key * (DP * 2) + ((chunk ^ (key & 7)) * 16);
      tc::copy16(to, pk + at * a.k.token, in);
      tc::copy16(to + C::kTile, pv + at * a.v.token, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint32_t kept[kStages - 1];
  uint32_t raw[kStages - 1];
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) raw[t] = flag(first + t * kStep);
  uint32_t next = flag(first + (kStages - 1) * kStep);
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) {
    kept[t] = __ballot_sync(0xffffffffu, raw[t] != 0);
    fetch(first + t * kStep, t, kept[t]);
  }

  uint32_t q[DP / 16][2];
  {
    const int r = lane / 4;
    const int tok = r / a.shared, g = r - tok * a.shared;
    const __nv_bfloat16* const pq = reinterpret_cast<const __nv_bfloat16*>(a.q.p) +
                                    (int64_t)(p.q0 + (r < p.rows ? tok : 0)) * a.q.token +
                                    (int64_t)(p.h * a.shared + (r < p.rows ? g : 0)) * a.q.head;
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) {
      const int d0 = i * 8 + (lane % 4) * 2;
      q[i / 2][i % 2] = r < p.rows && d0 < a.d ? *reinterpret_cast<const uint32_t*>(pq + d0) : 0u;
    }
  }
  float acc[DP / 16][4];
#pragma unroll
  for (int i = 0; i < DP / 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
  float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};

  // this lane's row of the 8 x 8 matrices that a load reads: keys in rows for
  // K (two of 8 keys, then the next dimensions), and the same for V'
  const int k_key = lane % 16, k_half = lane / 16;
  const int v_key = lane % 8 + (lane / 16) * 8, v_half = (lane / 8) % 2;
  int stage = 0;
  for (int j0 = first; j0 < p.to; j0 += kStep) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    const uint32_t now = kept[0];
#pragma unroll
    for (int t = 0; t + 2 < kStages; ++t) kept[t] = kept[t + 1];
    kept[kStages - 2] = __ballot_sync(0xffffffffu, next != 0);
    // into the stage that the last turn has read
    fetch(j0 + (kStages - 1) * kStep, stage == 0 ? kStages - 1 : stage - 1, kept[kStages - 2]);
    next = flag(j0 + kStages * kStep);
    const uint32_t at = my_ring + stage * 2 * C::kTile;
    stage = stage + 1 == kStages ? 0 : stage + 1;

    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      uint32_t f[4];
      load4(f, at + k_key * (DP * 2) + (((i * 2 + k_half) ^ (k_key & 7)) * 16));
      product(s, f, q[i][0], q[i][1]);
    }
    const bool low = (now >> (lane / 4)) & 1u, high = (now >> (lane / 4 + 8)) & 1u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[e] = low ? s[e] * a.c : -INFINITY;
      s[2 + e] = high ? s[2 + e] * a.c : -INFINITY;
    }
    float m[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
    if (__any_sync(0xffffffffu, m[0] > top[0] + kLazy || m[1] > top[1] + kLazy)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o));
        m[e] = fmaxf(m[e], top[e]);
        const float fade = top[e] == -INFINITY ? 0.0f : tc::exp2_fast(top[e] - m[e]);
        top[e] = m[e];
        sum[e] *= fade;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          acc[i][e] *= fade;
          acc[i][2 + e] *= fade;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float base = top[e] == -INFINITY ? 0.0f : top[e];
      s[e] = tc::exp2_fast(s[e] - base);
      s[2 + e] = tc::exp2_fast(s[2 + e] - base);
      sum[e] += s[e] + s[2 + e];
    }
    // the probabilities as the product's operand, in bf16 like the values they meet
    const uint32_t p0 = transposed(tc::pack_bf16(s[0], s[1])), p1 = transposed(tc::pack_bf16(s[2], s[3]));
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      uint32_t f[4];
      load4_transposed(f, at + C::kTile + v_key * (DP * 2) + (((i * 2 + v_half) ^ (v_key & 7)) * 16));
      product(acc[i], f, p0, p1);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  float* const w_acc = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
    const int r = (lane % 4) * 2 + e;
    float* const mine_acc = w_acc + warp * (C::kRing / 4) + r * DP + lane / 4;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      mine_acc[i * 16] = acc[i][e];
      mine_acc[i * 16 + 8] = acc[i][2 + e];
    }
    if (lane < 4) {
      s_top[warp][r] = top[e];
      s_sum[warp][r] = sum[e];
    }
  }
  few_join<__nv_bfloat16, DP>(a, p, w_acc, C::kRing / 4, s_top, s_sum, b_acc, b_top, b_sum);
}

template <auto kernel>
fvx_status launch_few(int smem, const FewArgs& a, int64_t grid, cudaStream_t s) {
  LaunchScope ls("attn_few", s);
  static std::atomic<uint64_t> allowed{0};
  FVX_TRY(allow_smem((const void*)kernel, smem, allowed));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)a.blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  FVX_CUDA(cudaLaunchKernelEx(&cfg, kernel, a));
  return check_launch("attn_few");
}
template <int LK>
fvx_status few_f32(const FewArgs& a, int rows, int64_t grid, cudaStream_t s) {
  constexpr int kSmem = kFewWarps * kF32Ring;
  if (rows <= 1) return launch_few<k_attn_few_f32<LK, 1>>(kSmem, a, grid, s);
  if (rows <= 2) return launch_few<k_attn_few_f32<LK, 2>>(kSmem, a, grid, s);
  if (rows <= 4) return launch_few<k_attn_few_f32<LK, 4>>(kSmem, a, grid, s);
  return launch_few<k_attn_few_f32<LK, 8>>(kSmem, a, grid, s);
}
template <int DP>
fvx_status few_bf16(const FewArgs& a, int64_t grid, cudaStream_t s) {
  return launch_few<k_attn_few_bf16<DP>>(kFewWarps * FewBf16<DP>::kRing, a, grid, s);
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
// can read.  Against the tensor cores' tiles of 128 rows (bf16): the 8 samples
// above 18 us and 37 with their join; 4 samples of two rows on 77 to 300 keys 10
// and 18; eight rows on 8192 keys, 32 samples, 100 and 100.
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
  // As many blocks as two per multiprocessor hold, of at least a turn of their
  // warps (64 keys); of long samples up to four times as many, of at least 1024
  // keys, which evens out samples of different lengths.  Several clusters per
  // unit, whose results another kernel joins, only where one each leaves
  // multiprocessors idle.
  const int64_t per = std::max<int64_t>(units, 1);
  const int64_t want = std::max<int64_t>(1, std::max(std::min<int64_t>(2 * sms / per, (longest + 63) / 64),
                                                     std::min<int64_t>(8 * sms / per, longest / 1024)));
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
    if (c.d <= 32) st = few_f32<8>(a, rows, grid, s);
    else if (c.d <= 64) st = few_f32<16>(a, rows, grid, s);
    else st = few_f32<32>(a, rows, grid, s);
  } else {
    st = c.d <= 64 ? few_bf16<64>(a, grid, s) : few_bf16<128>(a, grid, s);
  }
  FVX_TRY(st);
  return a.ranges > 1 ? attn_join(c, a.part, a.top, a.total, a.ranges, s) : FVX_OK;
}

}  // namespace fvx
