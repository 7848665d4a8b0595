// Cross attention in bf16 on the tcgen05 tensor cores (the formulas are in attn.cu).
//
// Forward.  One persistent block per multiprocessor; a work unit is a pair of
// 128-row query tiles of one key head of one batch element, and a range of its
// 128-key tiles.  A query tile's rows are (token, shared head) pairs, so all
// query heads of a key head meet its keys in one product.  Warp roles:
//   warps 0-3, 4-7  softmax of the pair's first / second tile, one row per
//                   thread: scores out of tensor memory, running maximum and
//                   sum in registers, probabilities back to tensor memory as
//                   bf16 (the A operand of the second product), the row's
//                   result at the end
//   warp 8          finds the block's units and publishes them in shared memory;
//                   TMA loads: queries, and a ring of key and value tiles
//   warps 9, 10     issue the products S = Q K^T and O += P V
// While one tile is in its softmax, the other's products run.  For 64-wide
// heads each tile has a warp that issues its products (with one warp for both,
// each waited for the other's softmax: 16,384 rows x 1200 keys x 8 heads took
// 133 us, not 115).  For 128-wide heads, where the products are the longer
// part, one warp issues both tiles' in turn: two warps drew the tiles into
// step, and the tensor cores idled while both were in their softmax (65,536
// rows x 2048 keys x 8 heads: 498 us, not 391).
//
// The accumulated O is relative to the running maximum m_ref of its row.  It
// is brought to a new maximum only when that exceeds m_ref by more than 2^8
// (in the exponent's base 2): until then p <= 2^8, far inside bf16's and
// fp32's range, and the final division by the sum removes the factor exactly.
// (Two tiles in turn and late corrections are steps that published attention
// kernels for this hardware take; the layout, the roles and the code are this
// file's own.)
//
// Roundings below fp32: the probabilities enter the second product as bf16, the
// type of the values they meet, since the product takes no wider one beside
// them; their sum is taken before that rounding.  Against 64 bits `out` is 0.0020
// to 0.0024 off (2-norm), where its own rounding to bf16 makes 0.0017.  Two
// parts per probability would bring that back for half as many products again.
//
// Measured: 65,536 rows x 2048 keys x 8 heads of 128, 395 us, 1390 TFLOP/s (the
// softmax's warps and the products' issue both take most of that time); 17,001
// rows x 1024 keys and 15,800 x 1500, 8 heads of 64, 124 us, 680 TFLOP/s: with
// half the products per score the exponentials are its longest part (72 us at
// the special function units' 4.6e12 a second; the products take 45), and the
// rest are the waits between the two.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "attn.cuh"
#include "tc.cuh"

namespace fvx {
namespace {

using namespace tc;

constexpr int kM = 128;             // rows of a query tile, keys of a key tile
constexpr int kAtom = kM * 128;     // bytes of 128 rows of 64 bf16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;       // growth of the maximum (in powers of 2) that O may lag behind

constexpr int kFwdThreads = 384;  // warp 11 only gives its registers away
constexpr int kFwdLoad = 8, kFwdMma = 9;

template <int DP>
struct Fwd {
  static constexpr int kAtoms = DP / 64;
  static constexpr int kTileBytes = kAtoms * kAtom;
  // 64-wide heads leave tensor memory for probabilities of their own (the next
  // scores are computed while the probabilities are still read) and shared
  // memory for a second set of queries; 128-wide ones put the probabilities
  // over the scores.
  static constexpr bool kOwnP = DP == 64;
  static constexpr int kPerWarp = kOwnP ? 1 : 2;  // tiles whose products one warp issues
  static constexpr int kQBufs = DP == 64 ? 2 : 1;
  static constexpr int kRing = DP == 64 ? 8 : 5;
  static constexpr int kS = 0, kO = 256, kP = kOwnP ? 384 : 0, kPStep = kOwnP ? 64 : 128;
  static constexpr size_t kHead = (size_t)(2 * kQBufs + kRing) * kTileBytes, kSmem = kHead + 512 + 800;
};

struct alignas(128) FwdArgs {
  CUtensorMap tq, tk, tv;
  AttnItems items;
  const uint8_t* mask;
  __nv_bfloat16* out;
  float* lse;
  float *part, *top, *total;
  uint32_t* status;
  int64_t all_rows;  // nq * heads
  int units, splits, heads, kv_heads, shared, d;
  int tile_rows;     // rows of a query tile in use: shared * floor(128 / shared)
  int wide_out;      // rows of out start at multiples of 32 bytes
  float c;           // scale * log2(e)
};

struct FwdUnit {
  int q0, rows, key0, keys, r0, h, split, t0, t1, valid;
};
// items: the offsets and unit prefix in shared memory (or where the items are
// many, in global memory); b: the item of the unit before, units only rise.
__device__ __forceinline__ FwdUnit fwd_unit(const FwdArgs& a, const int32_t* items, int u, int& b) {
  const int n = a.items.items + 1;
  while (items[2 * n + b + 1] <= u) ++b;
  FwdUnit w;
  w.q0 = items[b];
  w.rows = (items[b + 1] - w.q0) * a.shared;
  w.key0 = items[n + b];
  w.keys = items[n + b + 1] - w.key0;
  const int pairs = (w.rows + 2 * a.tile_rows - 1) / (2 * a.tile_rows);
  int i = u - items[2 * n + b];
  w.h = i / pairs;
  w.r0 = (i - w.h * pairs) * 2 * a.tile_rows;
  const int kt = (w.keys + kM - 1) / kM;
  w.split = 0;
  w.t0 = 0;
  w.t1 = kt;
  if (a.splits > 1) {
    w.split = w.h / a.kv_heads;
    w.h -= w.split * a.kv_heads;
    w.t0 = (int)((int64_t)kt * w.split / a.splits);
    w.t1 = (int)((int64_t)kt * (w.split + 1) / a.splits);
  }
  w.valid = 1;
  return w;
}

// Kept keys of tile t of a unit, four words of 32; warp-uniform.
struct Kept {
  uint32_t w[4];
  __device__ __forceinline__ bool all() const { return (w[0] & w[1] & w[2] & w[3]) == 0xffffffffu; }
  // words up to the last that keeps a key, at least one: the rest is not computed
  __device__ __forceinline__ int used() const { return w[3] ? 4 : w[2] ? 3 : w[1] ? 2 : 1; }
};
// Whether tile t may drop keys at all; the common tile takes no mask arithmetic.
__device__ __forceinline__ bool may_drop(const uint8_t* mask, int keys, int t) {
  return mask != nullptr || keys - t * kM < kM;
}
__device__ __forceinline__ void mask_bytes(const uint8_t* mask, int key0, int keys, int t, int lane, uint8_t (&b)[4]) {
  if (!mask) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = t * kM + 32 * i + lane;
    b[i] = j < keys ? __ldg(mask + key0 + j) : 0;
  }
}
__device__ __forceinline__ Kept kept_keys(const uint8_t* mask, int keys, int t, const uint8_t (&b)[4]) {
  Kept k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = keys - t * kM - 32 * i;
    k.w[i] = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
    if (mask) k.w[i] &= __ballot_sync(0xffffffffu, b[i] != 0);
  }
  return k;
}
// Zeros in the rows of a key or value tile that take no part: a probability of
// 0 times an infinity or a NaN would not be 0.  One warp; the products read
// shared memory through the async proxy, hence the fence.
template <int ATOMS>
__device__ __forceinline__ void zero_dropped(unsigned char* tile, const Kept& k, int words, int lane) {
  // Eight lanes write a row, four rows at once.  The loop is unrolled for 64-wide
  // heads only: the warp that issues the wide heads' products does so slower
  // with the long code beside them (65,536 rows x 2048 keys 420 us, not 396).
  auto four_rows = [&](int r) {
    unsigned char* const at = tile + r * 128 + (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < words && !((k.w[i] >> r) & 1u)) {
#pragma unroll
        for (int x = 0; x < ATOMS; ++x) *reinterpret_cast<uint4*>(at + x * kAtom + i * 4096) = make_uint4(0u, 0u, 0u, 0u);
      }
  };
  if constexpr (ATOMS == 1) {
#pragma unroll
    for (int r = 0; r < 32; r += 4) four_rows(r + (lane >> 3));
  } else {
#pragma unroll 1
    for (int r = lane >> 3; r < 32; r += 4) four_rows(r);
  }
  fence_proxy_async();
  __syncwarp();
}

struct FwdHead {
  uint64_t kv_full[8], kv_empty[8], q_full[2][2], q_empty[2][2];
  uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2], o_free[2];
  uint64_t info_full[2], info_free[2];
  uint32_t tmem;
  FwdUnit info[2];
};
constexpr int kFwdItems = 512;  // behind the head: the items' offsets
static_assert(sizeof(FwdHead) <= kFwdItems, "the shared-memory layout holds 512 bytes for it");

// The k-th unit of the block, as the loading warp published it; the whole warp.
__device__ __forceinline__ FwdUnit fwd_take(FwdHead& h, uint32_t k, int lane, uint32_t* status) {
  mbar_wait(smem_u32(&h.info_full[k & 1u]), (k >> 1) & 1u, status);
  FwdUnit w = *const_cast<const FwdUnit*>(&h.info[k & 1u]);
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&h.info_free[k & 1u]));
  return w;
}

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1) k_attn_tc_fwd(const __grid_constant__ FwdArgs a) {
  using C = Fwd<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* const ring = sm + (size_t)2 * C::kQBufs * C::kTileBytes;
  FwdHead& h = *reinterpret_cast<FwdHead*>(sm + C::kHead);
  int32_t* const items = reinterpret_cast<int32_t*>(sm + C::kHead + kFwdItems);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* const status = a.status;
  // The tiles fill shared memory to within a few hundred bytes, so its base
  // must sit on the swizzle's 1024-byte period by itself.
  if (smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) report_device_error(status, DEV_CHECK);
    return;
  }
  if (!a.items.ptr)
    for (int i = threadIdx.x; i < 3 * (a.items.items + 1); i += kFwdThreads) items[i] = a.items.in[i];

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(smem_u32(&h.kv_full[i]), 1);
      mbar_init(smem_u32(&h.kv_empty[i]), 2 / C::kPerWarp);
    }
    for (int s = 0; s < 2; ++s) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&h.q_full[s][b]), 1);
        mbar_init(smem_u32(&h.q_empty[s][b]), 1);
      }
      mbar_init(smem_u32(&h.s_full[s]), 1);
      mbar_init(smem_u32(&h.s_free[s]), 4);
      mbar_init(smem_u32(&h.p_ready[s]), 4);
      mbar_init(smem_u32(&h.pv_done[s]), 1);
      mbar_init(smem_u32(&h.o_free[s]), 4);
      mbar_init(smem_u32(&h.info_full[s]), 1);
      mbar_init(smem_u32(&h.info_free[s]), 8 + 2 / C::kPerWarp);
    }
    mbar_init_fence();
  }
  if (warp == kFwdMma) tmem_alloc(smem_u32(&h.tmem), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = h.tmem;

  // Registers: 384 threads at 168 are launched, 64,512: 256 at 200 and 128 at 104.
  if (warp < 8) {
    setmaxnreg_inc<200>();
    // ---------------------------------------------------------------- softmax
    const int slot = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + C::kS + slot * 128, to = tmem + lanes + C::kO + slot * DP,
                   tp = tmem + lanes + C::kP + slot * C::kPStep;
    const uint32_t s_full = smem_u32(&h.s_full[slot]), s_free = smem_u32(&h.s_free[slot]),
                   p_ready = smem_u32(&h.p_ready[slot]), pv_done = smem_u32(&h.pv_done[slot]),
                   o_free = smem_u32(&h.o_free[slot]);
    const int row = (warp & 3) * 32 + lane;
    // A scale that is not positive: its sign, or zero, goes into the scores, so that c > 0.
    const bool negate = !(a.c > 0.0f);
    const float sign = a.c < 0.0f ? -1.0f : 0.0f, c = a.c > 0.0f ? a.c : a.c < 0.0f ? -a.c : 1.0f;
    uint32_t step = 0;
    for (uint32_t uk = 0;; ++uk) {
      const FwdUnit w = fwd_take(h, uk, lane, status);
      if (!w.valid) break;
      const int r0 = w.r0 + slot * a.tile_rows;
      if (r0 >= w.rows) continue;  // the pair's second tile has no rows
      const int n = w.t1 - w.t0, r = r0 + row;
      const bool live = row < a.tile_rows && r < w.rows;
      float m_ref = -INFINITY, total = 0.0f;
      uint8_t mb[4];
      if (n > 0) mask_bytes(a.mask, w.key0, w.keys, w.t0, lane, mb);
      for (int j = 0; j < n; ++j, ++step) {
        mbar_wait(s_full, step & 1u, status);
        __syncwarp();
        fence_after();
        uint32_t r[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, r + 32 * i);
        tmem_ld_wait(r);
        if constexpr (C::kOwnP) {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
        }
        int used = 4;
        if (negate) {
#pragma unroll
          for (int i = 0; i < 128; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * sign);
        }
        if (may_drop(a.mask, w.keys, w.t0 + j)) {
          const Kept kept = kept_keys(a.mask, w.keys, w.t0 + j, mb);
          if (j + 1 < n) mask_bytes(a.mask, w.key0, w.keys, w.t0 + j + 1, lane, mb);
          used = kept.used();
          if (!kept.all()) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (!((kept.w[i >> 5] >> (i & 31)) & 1u)) r[i] = 0xff800000u;  // -infinity
          }
        }
        // Probabilities relative to `base`: their sum, and as bf16 into tensor
        // memory; m8, if given, collects the scores' maximum in the same pass.
        auto top_of = [&](float* m8) {
          return fmaxf(max3(max3(m8[0], m8[1], m8[2]), m8[3], m8[4]), max3(m8[5], m8[6], m8[7])) * c;
        };
        uint64_t add0, add1;
        auto powers = [&](float base, float* m8) {
          const uint64_t c2 = pair(c, c), b2 = pair(-base, -base);
          add0 = add1 = pair(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= used) break;
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float s0 = __uint_as_float(r[32 * i + 2 * k]), s1 = __uint_as_float(r[32 * i + 2 * k + 1]);
              const float s2 = __uint_as_float(r[32 * i + 2 * k + 2]), s3 = __uint_as_float(r[32 * i + 2 * k + 3]);
              if (m8) {
                m8[k % 8] = max3(m8[k % 8], s0, s1);
                m8[k % 8 + 1] = max3(m8[k % 8 + 1], s2, s3);
              }
              float x, y, z, t;
              unpair(fma2(pair(s0, s1), c2, b2), x, y);
              unpair(fma2(pair(s2, s3), c2, b2), z, t);
              x = exp2_fast(x);
              y = exp2_fast(y);
              z = exp2_fast(z);
              t = exp2_fast(t);
              add0 = add2(add0, pair(x, y));
              add1 = add2(add1, pair(z, t));
              p[k] = pack_bf16(x, y);
              p[k + 1] = pack_bf16(z, t);
            }
            tmem_st16(tp + 16 * i, p);
          }
        };
        bool done = false;
        float mx;
        if (C::kOwnP && j > 0) {
          // the previous product has read the previous probabilities
          mbar_wait(pv_done, (step - 1) & 1u, status);
          __syncwarp();
          fence_after();
          // Most tiles bring no new maximum worth a rescale: the powers are
          // taken relative to the old one while the new one is still being
          // found, and taken again in the few tiles where it matters.
          float m8[8] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
          powers(m_ref == -INFINITY ? 0.0f : m_ref, m8);
          mx = live ? top_of(m8) : -INFINITY;  // a row that is none holds anything
          done = !__any_sync(0xffffffffu, mx > m_ref + kLazy);
        } else {
          float m8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) m8[k] = fmaxf(__uint_as_float(r[k]), __uint_as_float(r[k + 8]));
#pragma unroll
          for (int i = 16; i < 128; i += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = max3(m8[k], __uint_as_float(r[i + k]), __uint_as_float(r[i + k + 8]));
          mx = C::kOwnP && !live ? -INFINITY : top_of(m8);
        }
        if (j == 0) {
          m_ref = mx;
        } else if (!done && __any_sync(0xffffffffu, mx > m_ref + kLazy)) {
          if (!C::kOwnP) {
            mbar_wait(pv_done, (step - 1) & 1u, status);
            __syncwarp();
            fence_after();
          }
          const float m_new = fmaxf(mx, m_ref);
          const float f = m_ref == -INFINITY ? 0.0f : exp2_fast(m_ref - m_new);
          total *= f;
          m_ref = m_new;
#pragma unroll 1
          for (int cc = 0; cc < DP; cc += 16) {
            uint32_t o[16];
            tmem_ld16(to + cc, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(to + cc, o);
          }
        }
        if (!done) powers(m_ref == -INFINITY ? 0.0f : m_ref, nullptr);
        {
          float x, y;
          unpair(add2(add0, add1), x, y);
          total += x + y;
        }
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }
      // ---- the rows' results
      const int tok = a.shared == 1 ? r : r / a.shared, g = r - tok * a.shared;
      const int64_t at = (int64_t)(w.q0 + tok) * a.heads + w.h * a.shared + g;
      const int64_t pat = (int64_t)w.split * a.all_rows + at;
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
      if (live) {
        if (a.splits == 1) {
          a.lse[at] = (m_ref + log2f(total)) * kLn2;
        } else {
          a.top[pat] = m_ref * kLn2;
          a.total[pat] = total;
        }
      }
      if (n == 0) {
        // no keys: zeros (a range without keys joins with total 0, its sums are not read)
        if (live && a.splits == 1)
          for (int cc = 0; cc < a.d; cc += 8) *reinterpret_cast<uint4*>(a.out + at * a.d + cc) = make_uint4(0, 0, 0, 0);
        __syncwarp();
        continue;
      }
      mbar_wait(pv_done, (step - 1) & 1u, status);
      __syncwarp();
      fence_after();
#pragma unroll 1
      for (int cc = 0; cc < DP; cc += 32) {
        uint32_t o[32];
        tmem_ld32(to + cc, o);
        tmem_ld_wait(o);
        if (cc + 32 >= DP) {
          // read: the next unit's product may overwrite it
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        if (live && a.splits == 1) {
          __nv_bfloat16* out = a.out + at * a.d + cc;
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = pack_bf16(__uint_as_float(o[k + 2 * i]) * inv, __uint_as_float(o[k + 2 * i + 1]) * inv);
            if (a.wide_out) {
              if (cc + k < a.d) store32(out + k, v);
            } else {
              if (cc + k < a.d) *reinterpret_cast<uint4*>(out + k) = make_uint4(v[0], v[1], v[2], v[3]);
              if (cc + k + 8 < a.d) *reinterpret_cast<uint4*>(out + k + 8) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        } else if (live) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            if (cc + k >= a.d) break;
            *reinterpret_cast<uint4*>(a.part + pat * a.d + cc + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        __syncwarp();  // the tensor-memory loads need the whole warp
      }
    }
  } else {
    setmaxnreg_dec<104>();
    if (warp == kFwdLoad) {
      // -------------------------------------------------------------- units and loads
      if (lane == 0) {
        tma_prefetch_map(&a.tq);
        tma_prefetch_map(&a.tk);
        tma_prefetch_map(&a.tv);
        uint32_t e = 0, nq[2] = {0, 0}, uk = 0;
        auto publish = [&](const FwdUnit& w) {
          const uint32_t i = uk & 1u;
          if (uk >= 2) mbar_wait(smem_u32(&h.info_free[i]), ((uk >> 1) - 1) & 1u, status);
          h.info[i] = w;
          mbar_arrive(smem_u32(&h.info_full[i]));
          ++uk;
        };
        auto load_kv = [&](const CUtensorMap* map, const FwdUnit& w, int t) {
          const uint32_t i = e % C::kRing, round = e / C::kRing;
          if (round > 0) mbar_wait(smem_u32(&h.kv_empty[i]), (round - 1) & 1u, status);
          const uint32_t bar = smem_u32(&h.kv_full[i]);
          mbar_expect_tx(bar, C::kTileBytes);
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
            tma_tile3d(smem_u32(ring) + i * C::kTileBytes + at * kAtom, map, 64 * at, w.h, w.key0 + t * kM, bar);
          ++e;
        };
        const int32_t* const at_items = a.items.ptr ? a.items.ptr : items;
        int b = 0;
        for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
          const FwdUnit w = fwd_unit(a, at_items, u, b);
          publish(w);
          if (w.t0 == w.t1) continue;
          for (int s = 0; s < 2; ++s) {
            const int r0 = w.r0 + s * a.tile_rows;
            if (r0 >= w.rows) continue;
            const uint32_t i = nq[s] % C::kQBufs, round = nq[s] / C::kQBufs;
            ++nq[s];
            if (round > 0) mbar_wait(smem_u32(&h.q_empty[s][i]), (round - 1) & 1u, status);
            const uint32_t bar = smem_u32(&h.q_full[s][i]);
            mbar_expect_tx(bar, (uint32_t)(C::kAtoms * a.tile_rows * 128));
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              tma_tile3d(smem_u32(sm) + (s * C::kQBufs + i) * C::kTileBytes + at * kAtom, &a.tq, 64 * at,
                         w.h * a.shared, w.q0 + r0 / a.shared, bar);
          }
          // in the order of their use: K0, K1, V0, K2, V1, ..., V(n-1)
          load_kv(&a.tk, w, w.t0);
          for (int t = w.t0; t < w.t1; ++t) {
            if (t + 1 < w.t1) load_kv(&a.tk, w, t + 1);
            load_kv(&a.tv, w, t);
          }
        }
        FwdUnit end = {};
        publish(end);
        // after a give-up, let the copies in flight land before the block exits
        for (uint32_t k = 0; k < C::kRing && k < e; ++k) {
          const uint32_t x = e - 1 - k;
          mbar_drain(smem_u32(&h.kv_full[x % C::kRing]), (x / C::kRing) & 1u);
        }
        for (int s = 0; s < 2; ++s)
          for (uint32_t k = 0; k < C::kQBufs && k < nq[s]; ++k) {
            const uint32_t x = nq[s] - 1 - k;
            mbar_drain(smem_u32(&h.q_full[s][x % C::kQBufs]), (x / C::kQBufs) & 1u);
          }
      }
      __syncwarp();
    } else if (warp >= kFwdMma && warp < kFwdMma + 2 / C::kPerWarp) {
      // -------------------------------------------------------------- products
      constexpr uint32_t kIdO = idesc(kM, DP) | kMnB;
      const uint32_t sq = smem_u32(sm), sr = smem_u32(ring);
      // Everything in this loop is in the way of the tensor cores, so it keeps
      // running indices and phases and touches masks only where keys may drop.
      struct Ring {
        uint32_t i, phase;
        __device__ __forceinline__ void next() {
          if (++i == (uint32_t)C::kRing) {
            i = 0;
            phase ^= 1u;
          }
        }
      } at = {0, 0};
      constexpr int kN = C::kPerWarp;
      const int slot0 = kN == 1 ? warp - kFwdMma : 0;
      uint32_t nq[kN] = {}, qk[kN] = {}, pv[kN] = {}, opened[kN] = {};
      // the step whose second product is still to come
      bool pend = false, first = false, pend_drop = false, pend_mine[kN] = {};
      Kept pend_kept = {};
      auto wait_full = [&](const Ring& x) {
        mbar_wait(smem_u32(&h.kv_full[x.i]), x.phase, status);
        __syncwarp();
      };
      // this warp's products have read a ring position, or never will
      auto release = [&](uint32_t i, bool used) {
        if (elect()) {
          if (used) commit(smem_u32(&h.kv_empty[i]));
          else mbar_arrive(smem_u32(&h.kv_empty[i]));
        }
        __syncwarp();
      };
      auto do_qk = [&](int i, uint32_t qi, uint32_t ki, uint32_t id) {
        const int s = slot0 + i;
        if (C::kOwnP && qk[i] > 0) mbar_wait(smem_u32(&h.s_free[s]), (qk[i] - 1) & 1u, status);
        __syncwarp();
        fence_after();
        if (elect()) {
          const uint64_t qd = desc_k(sq + (s * C::kQBufs + qi) * C::kTileBytes), kd = desc_k(sr + ki * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint32_t off = (uint32_t)((k >> 2) * (kAtom >> 4) + (k & 3) * 2);
            mma_ss(tmem + C::kS + s * 128, qd + off, kd + off, id, k > 0);
          }
          commit(smem_u32(&h.s_full[s]));
        }
        ++qk[i];
      };
      auto do_pv = [&](int i, uint32_t vi) {
        const int s = slot0 + i;
        mbar_wait(smem_u32(&h.p_ready[s]), pv[i] & 1u, status);
        if (first) {
          if (opened[i] > 0) mbar_wait(smem_u32(&h.o_free[s]), (opened[i] - 1) & 1u, status);
          ++opened[i];
        }
        __syncwarp();
        fence_after();
        if (elect()) {
          const uint64_t vd = desc_mn(sr + vi * C::kTileBytes, kAtom);
          const uint32_t to = tmem + C::kO + s * DP, tp = tmem + C::kP + s * C::kPStep;
          mma_ts(to, tp, vd, kIdO, !first);
          if (!pend_drop) {
#pragma unroll
            for (int k = 1; k < kM / 16; ++k) mma_ts(to, tp + 8 * k, vd + (uint32_t)(k * 128), kIdO, 1u);
          } else {
            const int steps = 2 * pend_kept.used();
#pragma unroll 1
            for (int k = 1; k < steps; ++k) mma_ts(to, tp + 8 * k, vd + (uint32_t)(k * 128), kIdO, 1u);
          }
          commit(smem_u32(&h.pv_done[s]));
        }
        ++pv[i];
      };
      // The value tile of the pending products, dropped keys' rows zeroed (by
      // both warps where there are two: they write the same).
      auto take_v = [&](const Ring& x) {
        wait_full(x);
        if (pend_drop && !pend_kept.all() && pend_mine[0])
          zero_dropped<C::kAtoms>(ring + (size_t)x.i * C::kTileBytes, pend_kept, pend_kept.used(), lane);
      };
      auto flush = [&]() {
        if (!pend) return;
        take_v(at);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (pend_mine[i]) do_pv(i, at.i);
        release(at.i, pend_mine[0]);
        at.next();
        pend = false;
      };
      for (uint32_t uk = 0;; ++uk) {
        const FwdUnit w = fwd_take(h, uk, lane, status);
        if (!w.valid) break;
        const int n = w.t1 - w.t0;
        if (n == 0) {
          // The softmax warps of the unit before wait for its last product,
          // and units are published at most two ahead of them.
          flush();
          continue;
        }
        bool mine[kN];
        uint32_t qi[kN], qp[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          mine[i] = w.r0 + (slot0 + i) * a.tile_rows < w.rows;
          qi[i] = nq[i] % C::kQBufs;
          qp[i] = (nq[i] / C::kQBufs) & 1u;
        }
        uint8_t mb[4];
        mask_bytes(a.mask, w.key0, w.keys, w.t0, lane, mb);
        for (int j = 0; j < n; ++j) {
          Kept kept;
          const bool drop = may_drop(a.mask, w.keys, w.t0 + j);
          uint32_t id = idesc(kM, kM);
          if (drop) {
            kept = kept_keys(a.mask, w.keys, w.t0 + j, mb);
            if (j + 1 < n) mask_bytes(a.mask, w.key0, w.keys, w.t0 + j + 1, lane, mb);
            id = idesc(kM, 32 * kept.used());
          }
          if (j == 0) {
            // Ring order: V of the unit before, then this unit's K.  With
            // probabilities of their own the scores can go first, if their
            // operands are there; the unit before waits for its last product.
            Ring kx = at;
            if (pend) kx.next();
            const bool ahead = C::kOwnP && pend &&
                               __all_sync(0xffffffffu, (!mine[0] || mbar_try(smem_u32(&h.q_full[slot0][qi[0]]), qp[0])) &&
                                                           mbar_try(smem_u32(&h.kv_full[kx.i]), kx.phase));
            if (!ahead) {
              flush();
              wait_full(kx);
            }
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (mine[i]) {
                mbar_wait(smem_u32(&h.q_full[slot0 + i][qi[i]]), qp[i], status);
                do_qk(i, qi[i], kx.i, id);
              }
            release(kx.i, mine[0]);
            if (ahead) flush();
            at = kx;
          } else {
            // ring order: K of this step, V of the one before
            const uint32_t ki = at.i;
            wait_full(at);
            at.next();
            if (C::kOwnP) {
              if (mine[0]) do_qk(0, qi[0], ki, id);
              release(ki, mine[0]);
            }
            take_v(at);
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (mine[i]) {
                do_pv(i, at.i);
                if (!C::kOwnP) do_qk(i, qi[i], ki, id);
              }
            release(at.i, mine[0]);
            if (!C::kOwnP) release(ki, true);
          }
          at.next();
          if (j == n - 1) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (mine[i] && elect()) commit(smem_u32(&h.q_empty[slot0 + i][qi[i]]));
            __syncwarp();
          }
          pend = true;
#pragma unroll
          for (int i = 0; i < kN; ++i) pend_mine[i] = mine[i];
          pend_drop = drop;
          if (drop) pend_kept = kept;
          first = j == 0;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) nq[i] += mine[i];
      }
      flush();
      // every product has completed before tensor memory is freed
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (pv[i] > 0) mbar_drain(smem_u32(&h.pv_done[slot0 + i]), (pv[i] - 1) & 1u);
      __syncwarp();
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kFwdMma) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

// ================================================================ backward
// Scores are computed transposed, keys in the lanes and query rows in the
// columns: then P^T and dS^T are A operands straight from tensor memory for
//   dV += P^T dO   and   dK += dS^T Q
// and only dQ = dS K needs dS through shared memory.  A work unit is a range of
// key tiles and a range of row tiles of one key head: for each key tile (K and
// V resident, dK and dV accumulating in tensor memory) it walks its row tiles.
// dQ of a row tile collects over the key tiles in fp32 in a workspace that only
// this unit touches, one thread per value, so the order of every sum is fixed;
// units that share keys (or rows) write partial sums that are added in order.
// Roundings below fp32: P in the product of dV and dS in those of dK and dQ are
// bf16, like the operands they meet; delta is taken from the rounded `out`.  The
// gradients are 0.0024 to 0.0027 off (2-norm), 0.0017 of it their own rounding;
// two parts for each would double three of the five products.
// Warp roles:
//   warps 0-15      P and dS, 32 of the tile's columns each (four warps per
//                   scheduler hide the latencies of a step's phases; with two,
//                   64 columns each, a step took more than twice the
//                   products' time); at the end of a key tile dV and dK out of
//                   tensor memory
//   warps 16-19     dQ out of tensor memory
//   warp 20         TMA loads
//   warp 21         issues the five products
//
// Measured: 17,001 rows x 1024 keys and 15,800 x 1500, 8 heads of 64, 300 us, 702
// TFLOP/s; 2 x 16,384 rows x 2048 keys, 8 heads of 128, 830 us, 830 TFLOP/s.  A
// step takes 3400 cycles of a multiprocessor (64-wide heads), of which the five
// products are 1400: each waits for what the step's phases before it made, with
// some 400 cycles from a product's end to the next one's start.  Without the
// softmax's arithmetic and the writes of dQ (a value is added to for every key
// tile) the first took 266 us where the whole took 321.
constexpr int kBwdThreads = 768;  // warps 22, 23 only give their registers away
constexpr int kBwdLoad = 20, kBwdMma = 21;

template <int DP>
struct Bwd {
  static constexpr int kAtoms = DP / 64;
  static constexpr int kTileBytes = kAtoms * kAtom;
  static constexpr bool kWide = DP == 128;
  static constexpr int kKvBufs = kWide ? 1 : 2;
  static constexpr int kStages = kWide ? 2 : 3;
  // tensor memory: P over the scores.  64-wide heads: dS and dQ in columns of
  // their own; 128-wide: dS over dP, and dQ over both once dK has read dS.
  static constexpr int kS = 0, kDp = 128, kDv = 256, kDk = kWide ? 384 : 320, kDq = kWide ? 128 : 384,
                       kDs = kWide ? 128 : 448, kDsStep = kWide ? 32 : 16;  // per 32 rows
  static constexpr size_t kKv = 0, kQ = (size_t)2 * kKvBufs * kTileBytes,
                          kSmDs = kQ + (size_t)2 * kStages * kTileBytes, kStats = kSmDs + 2 * kAtom,
                          kHead = kStats + (size_t)kStages * 1024, kSmem = kHead + 512;
};

struct alignas(128) BwdArgs {
  CUtensorMap tq, tdo, tk, tv;
  AttnItems items;
  const uint8_t* mask;
  const float* stats;  // [row tile][key head][-lse2 of 128 rows, -delta of 128 rows]
  // An item's partial sums: its slabs from kItemRowSlab (kItemKeySlab) on, range
  // after range.  Only items whose sums need them have any.
  float* dq_sum;             // [key range, row tile][key head][DP / 4][128][4]
  float *dk_part, *dv_part;  // [row range, key tile][key head][DP / 4][128][4]
  __nv_bfloat16 *dq, *dk, *dv;
  uint32_t* status;
  int units, heads, kv_heads, shared, d, tile_rows;
  float c, scale;
};

struct BwdUnit {
  int q0, rows, key0, keys, h, tile0, i0, i1, t0, t1, r_ranges, key_tiles;
  int row_slab, key_slab;  // of the range's row tile 0, of its key tile 0
};
__device__ __forceinline__ BwdUnit bwd_unit(const BwdArgs& a, int u) {
  BwdUnit w;
  const int b = a.items.item_of(u);
  w.q0 = a.items.q0(b);
  w.rows = (a.items.q0(b + 1) - w.q0) * a.shared;
  w.key0 = a.items.k0(b);
  w.keys = a.items.k0(b + 1) - w.key0;
  w.tile0 = a.items.at(kItemTile, b);
  const int tiles = a.items.at(kItemTile, b + 1) - w.tile0;
  w.key_tiles = (w.keys + kM - 1) / kM;
  w.r_ranges = a.items.at(kItemRows, b);
  const int k_ranges = a.items.at(kItemKeys, b);
  int i = u - a.items.u0(b);
  const int r_range = i % w.r_ranges;
  i /= w.r_ranges;
  const int k_range = i % k_ranges;
  w.h = i / k_ranges;
  w.i0 = (int)((int64_t)tiles * r_range / w.r_ranges);
  w.i1 = (int)((int64_t)tiles * (r_range + 1) / w.r_ranges);
  w.t0 = (int)((int64_t)w.key_tiles * k_range / k_ranges);
  w.t1 = (int)((int64_t)w.key_tiles * (k_range + 1) / k_ranges);
  w.row_slab = a.items.at(kItemRowSlab, b) + k_range * tiles;
  w.key_slab = a.items.at(kItemKeySlab, b) + r_range * w.key_tiles;
  return w;
}

struct BwdHead {
  uint64_t kv_full[2], kv_empty[2], q_full[3], q_empty[3];
  uint64_t s_full, dp_full, p_ready, ds_ready, dq_full, dq_free, acc_full, acc_free;
  uint32_t tmem;
};

// The block's steps in order: units, their key tiles, their row tiles.  Every
// unit has at least one of each.
struct BwdCursor {
  BwdUnit w;
  int u, t, i;
  uint32_t step, tile;  // counted over the block's life
  bool valid;
  __device__ __forceinline__ void start(const BwdArgs& a) {
    u = blockIdx.x;
    step = tile = 0;
    valid = u < a.units;
    if (valid) {
      w = bwd_unit(a, u);
      t = w.t0;
      i = w.i0;
    }
  }
  __device__ __forceinline__ void next(const BwdArgs& a) {
    ++step;
    if (++i < w.i1) return;
    i = w.i0;
    ++tile;
    if (++t < w.t1) return;
    u += gridDim.x;
    valid = u < a.units;
    if (valid) {
      w = bwd_unit(a, u);
      t = w.t0;
      i = w.i0;
    }
  }
  __device__ __forceinline__ bool first() const { return i == w.i0; }
  __device__ __forceinline__ bool last() const { return i + 1 == w.i1; }
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1) k_attn_tc_bwd(const __grid_constant__ BwdArgs a) {
  using C = Bwd<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  BwdHead& h = *reinterpret_cast<BwdHead*>(sm + C::kHead);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* const status = a.status;
  const uint32_t sb = smem_u32(sm);
  // The tiles fill shared memory to within a few hundred bytes, so its base
  // must sit on the swizzle's 1024-byte period by itself.
  if (sb & 1023u) {
    if (threadIdx.x == 0) report_device_error(status, DEV_CHECK);
    return;
  }
  // rows that no copy writes (128 is not a multiple of every group of heads) read as zeros
  for (int e = threadIdx.x; e < (int)(2 * C::kStages * C::kTileBytes / 16); e += kBwdThreads)
    reinterpret_cast<uint4*>(sm + C::kQ)[e] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&h.kv_full[i]), 1);
      mbar_init(smem_u32(&h.kv_empty[i]), 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_u32(&h.q_full[i]), 1);
      mbar_init(smem_u32(&h.q_empty[i]), 1);
    }
    mbar_init(smem_u32(&h.s_full), 1);
    mbar_init(smem_u32(&h.dp_full), 1);
    mbar_init(smem_u32(&h.p_ready), 16);
    mbar_init(smem_u32(&h.ds_ready), 16);
    mbar_init(smem_u32(&h.dq_full), 1);
    mbar_init(smem_u32(&h.dq_free), 4);
    mbar_init(smem_u32(&h.acc_full), 1);
    mbar_init(smem_u32(&h.acc_free), 16);
    mbar_init_fence();
  }
  if (warp == kBwdMma) tmem_alloc(smem_u32(&h.tmem), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = h.tmem;
  const uint32_t q_tile = (uint32_t)C::kTileBytes;

  // Registers: 768 threads at 80 are launched, 61,440: 512 at 88 and 256 at 64.
  if (warp < 16) {
    setmaxnreg_inc<88>();
    // ---------------------------------------------------------------- P and dS
    const int quarter = warp >> 2;
    const int key = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + C::kS + quarter * 32, tdp = tmem + lanes + C::kDp + quarter * 32,
                   tds = tmem + lanes + C::kDs + quarter * C::kDsStep;
    unsigned char* const ds_row = sm + C::kSmDs + (quarter >> 1) * kAtom + key * 128;
    const int chunk0 = (quarter & 1) * 4;
    const uint32_t s_full = smem_u32(&h.s_full), dp_full = smem_u32(&h.dp_full), p_ready = smem_u32(&h.p_ready),
                   ds_ready = smem_u32(&h.ds_ready), dq_full = smem_u32(&h.dq_full);
    const uint64_t c2 = pair(a.c, a.c);
    BwdCursor cur;
    cur.start(a);
    bool kept = false, whole = false;
    uint32_t stage = 0, stage_phase = 0;
    while (cur.valid) {
      const BwdUnit& w = cur.w;
      if (cur.first()) {
        const int j = cur.t * kM + key;
        kept = j < w.keys && (!a.mask || __ldg(a.mask + w.key0 + j) != 0);
        whole = __all_sync(0xffffffffu, kept);
      }
      const uint32_t par = cur.step & 1u;
      const float* st = reinterpret_cast<const float*>(sm + C::kStats + stage * 1024) + quarter * 32;
      // the row constants come with the stage's copies
      mbar_wait(smem_u32(&h.q_full[stage]), stage_phase, status);
      if (++stage == (uint32_t)C::kStages) {
        stage = 0;
        stage_phase ^= 1u;
      }
      mbar_wait(s_full, par, status);
      __syncwarp();
      fence_after();
      float p[32];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t r[16], o[8];
        tmem_ld16(ts + 16 * cc, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 nl = *reinterpret_cast<const float4*>(st + 16 * cc + k);
          float x, y, z, t;
          unpair(fma2(pair(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), c2, pair(nl.x, nl.y)), x, y);
          unpair(fma2(pair(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])), c2, pair(nl.z, nl.w)), z, t);
          p[16 * cc + k] = exp2_fast(x);
          p[16 * cc + k + 1] = exp2_fast(y);
          p[16 * cc + k + 2] = exp2_fast(z);
          p[16 * cc + k + 3] = exp2_fast(t);
        }
        if (!whole) {
          // the scores of a dropped key, whose row reads as zeros, are 0, not -infinity
#pragma unroll
          for (int k = 0; k < 16; ++k) p[16 * cc + k] = kept ? p[16 * cc + k] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = pack_bf16(p[16 * cc + 2 * k], p[16 * cc + 2 * k + 1]);
        tmem_st8(ts + 8 * cc, o);
      }
      tmem_st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);

      mbar_wait(dp_full, par, status);
      // dQ of the step before has read dS from shared memory
      if (cur.step > 0) mbar_wait(dq_full, par ^ 1u, status);
      __syncwarp();
      fence_after();
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t r[16], o[8];
        tmem_ld16(tdp + 16 * cc, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 nd = *reinterpret_cast<const float4*>(st + 128 + 16 * cc + k);  // -delta
          float x, y, z, t;
          unpair(mul2(add2(pair(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), pair(nd.x, nd.y)),
                      pair(p[16 * cc + k], p[16 * cc + k + 1])),
                 x, y);
          unpair(mul2(add2(pair(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])), pair(nd.z, nd.w)),
                      pair(p[16 * cc + k + 2], p[16 * cc + k + 3])),
                 z, t);
          o[k / 2] = pack_bf16(x, y);
          o[k / 2 + 1] = pack_bf16(z, t);
        }
        tmem_st8(tds + 8 * cc, o);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(ds_row + (((chunk0 + 2 * cc + k) ^ (key & 7)) << 4)) =
              make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
      tmem_st_wait();
      fence_proxy_async();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);

      if (cur.last()) {
        // dV (quarters 0, 1) and dK (2, 3) of the key tile, half of the columns each
        const bool is_k = quarter >= 2;
        const int col0 = (quarter & 1) * (DP / 2);
        const float f = is_k ? a.scale : 1.0f;
        const int j = cur.t * kM + key;
        const int64_t row = (int64_t)(w.key0 + j) * a.kv_heads + w.h;
        const bool live = j < w.keys, direct = w.r_ranges == 1;
        __nv_bfloat16* const out = (is_k ? a.dk : a.dv) + row * a.d;
        float* const part = (is_k ? a.dk_part : a.dv_part) +
                            ((int64_t)(w.key_slab + cur.t) * a.kv_heads + w.h) * (kM * DP) + key * 4;
        mbar_wait(smem_u32(&h.acc_full), cur.tile & 1u, status);
        __syncwarp();
        fence_after();
#pragma unroll 1
        for (int cc = col0; cc < col0 + DP / 2; cc += 16) {
          uint32_t r[16];
          tmem_ld16(tmem + lanes + (is_k ? C::kDk : C::kDv) + cc, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int k = 0; k < 16; ++k) r[k] = kept ? __float_as_uint(__uint_as_float(r[k]) * f) : 0u;
          if (!direct) {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4*>(part + (cc + k) / 4 * (kM * 4)) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
          } else if (live) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = pack_bf16(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
            if (cc < a.d) *reinterpret_cast<uint4*>(out + cc) = make_uint4(v[0], v[1], v[2], v[3]);
            if (cc + 8 < a.d) *reinterpret_cast<uint4*>(out + cc + 8) = make_uint4(v[4], v[5], v[6], v[7]);
          }
          __syncwarp();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&h.acc_free));
      }
      cur.next(a);
    }
  } else if (warp < 20) {
    setmaxnreg_dec<64>();
    // ---------------------------------------------------------------- dQ
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tdq = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kDq;
    BwdCursor cur;
    cur.start(a);
    while (cur.valid) {
      const BwdUnit& w = cur.w;
      const int r = cur.i * a.tile_rows + row;
      const bool live = row < a.tile_rows && r < w.rows;
      const int tok = live ? r / a.shared : 0, g = r - tok * a.shared;
      const bool only = w.key_tiles == 1;  // nothing to collect
      __nv_bfloat16* out = a.dq + ((int64_t)(w.q0 + tok) * a.heads + w.h * a.shared + g) * a.d;
      float* sum = a.dq_sum + ((int64_t)(w.row_slab + cur.i) * a.kv_heads + w.h) * (kM * DP) + row * 4;
      mbar_wait(smem_u32(&h.dq_full), cur.step & 1u, status);
      __syncwarp();
      fence_after();
#pragma unroll 1
      for (int cc = 0; cc < DP; cc += 32) {
        uint32_t v[32];
        tmem_ld32(tdq + cc, v);
        tmem_ld_wait(v);
        if (cc + 32 >= DP) {
          // read: what is written below keeps nobody waiting
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&h.dq_free));
        }
        float* const at = sum + cc / 4 * (kM * 4);
        if (only) {
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              if (cc + k >= a.d) break;
              uint4 o;
              uint32_t* po = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                po[x] = pack_bf16(__uint_as_float(v[k + 2 * x]) * a.scale, __uint_as_float(v[k + 2 * x + 1]) * a.scale);
              *reinterpret_cast<uint4*>(out + cc + k) = o;
            }
          }
          __syncwarp();
        } else if (cur.t == w.t0) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<uint4*>(at + k / 4 * (kM * 4)) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 32; k += 4) red4(at + k / 4 * (kM * 4), v + k);
        }
      }
      cur.next(a);
    }
  } else {
    setmaxnreg_dec<64>();
    if (warp == kBwdLoad) {
      // -------------------------------------------------------------- loads
      // Lane l issues copy l of a step: Q and dO (an atom each), the row constants.
      if (lane == 0) {
        tma_prefetch_map(&a.tq);
        tma_prefetch_map(&a.tdo);
        tma_prefetch_map(&a.tk);
        tma_prefetch_map(&a.tv);
      }
      BwdCursor cur;
      cur.start(a);
      uint32_t s = 0, s_phase = 1, b = 0, b_phase = 1;  // the first round waits for nobody
      const uint32_t bytes = (uint32_t)(2 * C::kAtoms * a.tile_rows * 128 + 1024);
      const int tile_tokens = a.tile_rows / a.shared;
      const int atom = lane % C::kAtoms, second = lane / C::kAtoms;
      while (cur.valid) {
        if (cur.first()) {
          const uint32_t bar = smem_u32(&h.kv_full[b]);
          if (cur.tile >= (uint32_t)C::kKvBufs) mbar_wait(smem_u32(&h.kv_empty[b]), b_phase, status);
          __syncwarp();
          if (lane == 0) mbar_expect_tx(bar, 2 * q_tile);
          __syncwarp();
          if (lane < 2 * C::kAtoms)
            tma_tile3d(sb + (uint32_t)C::kKv + (2 * b + second) * q_tile + atom * kAtom, second ? &a.tv : &a.tk, 64 * atom,
                       cur.w.h, cur.w.key0 + cur.t * kM, bar);
          if (++b == (uint32_t)C::kKvBufs) {
            b = 0;
            b_phase ^= 1u;
          }
        }
        const uint32_t bar = smem_u32(&h.q_full[s]);
        if (cur.step >= (uint32_t)C::kStages) mbar_wait(smem_u32(&h.q_empty[s]), s_phase, status);
        __syncwarp();
        if (lane == 0) mbar_expect_tx(bar, bytes);
        __syncwarp();
        if (lane < 2 * C::kAtoms)
          tma_tile3d(sb + (uint32_t)C::kQ + (2 * s + second) * q_tile + atom * kAtom, second ? &a.tdo : &a.tq, 64 * atom,
                     cur.w.h * a.shared, cur.w.q0 + cur.i * tile_tokens, bar);
        else if (lane == 2 * C::kAtoms)
          bulk_load(sb + (uint32_t)C::kStats + s * 1024,
                    a.stats + ((int64_t)(cur.w.tile0 + cur.i) * a.kv_heads + cur.w.h) * 256, 1024, bar);
        if (++s == (uint32_t)C::kStages) {
          s = 0;
          s_phase ^= 1u;
        }
        cur.next(a);
      }
      // after a give-up, let the copies in flight land before the block exits
      for (uint32_t k = 0; k < C::kStages && k < cur.step; ++k) {
        const uint32_t x = cur.step - 1 - k;
        mbar_drain(smem_u32(&h.q_full[x % C::kStages]), (x / C::kStages) & 1u);
      }
      for (uint32_t k = 0; k < C::kKvBufs && k < cur.tile; ++k) {
        const uint32_t x = cur.tile - 1 - k;
        mbar_drain(smem_u32(&h.kv_full[x % C::kKvBufs]), (x / C::kKvBufs) & 1u);
      }
      __syncwarp();
    } else if (warp == kBwdMma) {
      // -------------------------------------------------------------- products
      constexpr uint32_t kIdS = idesc(kM, kM), kIdKv = idesc(kM, DP) | kMnB, kIdQ = idesc(kM, DP) | kMnA | kMnB;
      const uint32_t s_full = smem_u32(&h.s_full), dp_full = smem_u32(&h.dp_full);
      // Where a step's operands are: running indices, as every instruction here
      // is in the way of the tensor cores.
      struct Place {
        uint32_t q, q_phase, kv, kv_phase;
      };
      auto after = [](Place x, bool next_tile) {
        if (++x.q == (uint32_t)C::kStages) {
          x.q = 0;
          x.q_phase ^= 1u;
        }
        if (next_tile && ++x.kv == (uint32_t)C::kKvBufs) {
          x.kv = 0;
          x.kv_phase ^= 1u;
        }
        return x;
      };
      auto k_at = [&](const Place& x) { return sb + (uint32_t)C::kKv + 2 * x.kv * q_tile; };
      auto q_at = [&](const Place& x) { return sb + (uint32_t)C::kQ + 2 * x.q * q_tile; };
      // 128 x 128 scores: K-major operands, 16 values of the head per product
      auto scores = [&](uint32_t d, uint32_t ka, uint32_t qa, uint32_t bar) {
        if (elect()) {
          const uint64_t kd = desc_k(ka), qd = desc_k(qa);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint32_t off = (uint32_t)((k >> 2) * (kAtom >> 4) + (k & 3) * 2);
            mma_ss(tmem + d, kd + off, qd + off, kIdS, k > 0);
          }
          commit(bar);
        }
        __syncwarp();
      };
      // waits for a step's operands and zeros what takes no part
      auto ready = [&](const BwdCursor& x, const Place& at) {
        if (x.first()) {
          mbar_wait(smem_u32(&h.kv_full[at.kv]), at.kv_phase, status);
          __syncwarp();
          if (may_drop(a.mask, x.w.keys, x.t)) {
            uint8_t mb[4];
            mask_bytes(a.mask, x.w.key0, x.w.keys, x.t, lane, mb);
            const Kept kept = kept_keys(a.mask, x.w.keys, x.t, mb);
            if (!kept.all()) {
              // keys meet dS in dQ; values meet dO in dP, which P = 0 must not turn into a NaN
              zero_dropped<C::kAtoms>(sm + C::kKv + 2 * at.kv * C::kTileBytes, kept, 4, lane);
              zero_dropped<C::kAtoms>(sm + C::kKv + (2 * at.kv + 1) * C::kTileBytes, kept, 4, lane);
            }
          }
        }
        mbar_wait(smem_u32(&h.q_full[at.q]), at.q_phase, status);
        __syncwarp();
        const int left = x.w.rows - x.i * a.tile_rows;
        if (left < a.tile_rows) {
          // rows of the next sample, or past the end
          Kept live;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            live.w[i] = left >= 32 * (i + 1) ? 0xffffffffu : left <= 32 * i ? 0u : (1u << (left - 32 * i)) - 1u;
          zero_dropped<C::kAtoms>(sm + C::kQ + 2 * at.q * C::kTileBytes, live, 4, lane);
          zero_dropped<C::kAtoms>(sm + C::kQ + (2 * at.q + 1) * C::kTileBytes, live, 4, lane);
        }
      };
      auto issue_s = [&](const Place& at) { scores(C::kS, k_at(at), q_at(at), s_full); };
      auto issue_dp = [&](const Place& at) { scores(C::kDp, k_at(at) + q_tile, q_at(at) + q_tile, dp_full); };

      BwdCursor nx;  // the step after the current one
      nx.start(a);
      bool valid = nx.valid;
      Place here = {0, 0, 0, 0}, there = here;
      if (valid) {
        ready(nx, here);
        fence_after();
        issue_s(here);
        issue_dp(here);
      }
      uint32_t par = 0, tile = 0;
      bool begun = false;
      while (valid) {
        const bool fresh = nx.first(), last = nx.last();
        nx.next(a);
        there = after(here, last);
        const bool more = nx.valid, defer = C::kKvBufs == 1 && last;  // its keys replace this tile's
        // the next step's operands while this one's probabilities are made
        if (more && !defer) ready(nx, there);
        // ---- dV += P^T dO, and the next scores over the probabilities
        mbar_wait(smem_u32(&h.p_ready), par, status);
        if (fresh && tile > 0) mbar_wait(smem_u32(&h.acc_free), (tile - 1) & 1u, status);
        __syncwarp();
        fence_after();
        if (elect()) {
          const uint64_t od = desc_mn(q_at(here) + q_tile, kAtom);
#pragma unroll
          for (int k = 0; k < kM / 16; ++k)
            mma_ts(tmem + C::kDv, tmem + C::kS + (k >> 1) * 32 + (k & 1) * 8, od + (uint32_t)(k * 128), kIdKv,
                   !(fresh && k == 0));
        }
        __syncwarp();
        if (more && !defer) issue_s(there);
        mbar_wait(smem_u32(&h.ds_ready), par, status);
        __syncwarp();
        fence_after();
        if (!C::kWide && more) issue_dp(there);
        // ---- dK += dS^T Q
        if (elect()) {
          const uint64_t qd = desc_mn(q_at(here), kAtom);
#pragma unroll
          for (int k = 0; k < kM / 16; ++k)
            mma_ts(tmem + C::kDk, tmem + C::kDs + (k >> 1) * C::kDsStep + (k & 1) * 8, qd + (uint32_t)(k * 128), kIdKv,
                   !(fresh && k == 0));
          commit(smem_u32(&h.q_empty[here.q]));
          if (last) commit(smem_u32(&h.acc_full));
        }
        __syncwarp();
        // ---- dQ = dS K
        if (!C::kWide && begun) mbar_wait(smem_u32(&h.dq_free), par ^ 1u, status);
        __syncwarp();
        fence_after();
        if (elect()) {
          const uint64_t sd = desc_mn(sb + (uint32_t)C::kSmDs, kAtom), kd = desc_mn(k_at(here), kAtom);
#pragma unroll
          for (int k = 0; k < kM / 16; ++k)
            mma_ss(tmem + C::kDq, sd + (uint32_t)(k * 128), kd + (uint32_t)(k * 128), kIdQ, k > 0);
          commit(smem_u32(&h.dq_full));
          if (last) commit(smem_u32(&h.kv_empty[here.kv]));
        }
        __syncwarp();
        if (more && defer) {
          ready(nx, there);
          fence_after();
          issue_s(there);
        }
        if (C::kWide && more) {
          mbar_wait(smem_u32(&h.dq_free), par, status);
          __syncwarp();
          fence_after();
          issue_dp(there);
        }
        here = there;
        par ^= 1u;
        tile += last;
        begun = true;
        valid = more;
      }
      // every product has completed before tensor memory is freed
      if (begun) mbar_drain(smem_u32(&h.dq_full), par ^ 1u);
      __syncwarp();
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kBwdMma) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

// -lse in powers of 2 and -delta = -(dout . out) of every row tile's rows, 8
// (16 for 128-wide heads) lanes per row; the places of rows that do not exist
// hold -infinity (a probability of 0) and 0.
template <int DP>
__global__ void __launch_bounds__(256) k_attn_stats(const __grid_constant__ AttnItems items, HeadsView dout,
                                                    const __nv_bfloat16* __restrict__ out,
                                                    const float* __restrict__ lse, int heads, int kv_heads, int shared,
                                                    int tile_rows, int d, float* __restrict__ stats) {
  constexpr int kLanes = DP / 8, kRows = 256 / kLanes;  // rows of a block's turn
  const int part = threadIdx.x % kLanes;
  const int tile = blockIdx.x / kv_heads, kh = blockIdx.x - tile * kv_heads;
  const int b = items.find(kItemTile, tile);
  const int q0 = items.q0(b), rows = (items.q0(b + 1) - q0) * shared, tile0 = items.at(kItemTile, b);
  float* st = stats + (int64_t)blockIdx.x * 256;
#pragma unroll
  for (int row = threadIdx.x / kLanes; row < kM; row += kRows) {
    const int r = (tile - tile0) * tile_rows + row;
    const bool live = row < tile_rows && r < rows;
    float s = 0.0f, nl = -INFINITY;
    if (live) {
      const int t = shared == 1 ? r : r / shared;
      const int64_t tok = q0 + t;
      const int hd = kh * shared + r - t * shared;
      if (part * 8 < d) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(dout.p) +
                                                             tok * dout.token + hd * dout.head + part * 8));
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(out + (tok * heads + hd) * d + part * 8));
        const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s = fmaf(__uint_as_float(u[k] << 16), __uint_as_float(v[k] << 16), s);
          s = fmaf(__uint_as_float(u[k] & 0xffff0000u), __uint_as_float(v[k] & 0xffff0000u), s);
        }
      }
      if (part == 0) nl = -__ldg(lse + tok * heads + hd) * kLog2e;
    }
#pragma unroll
    for (int k = kLanes / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (part == 0) {
      st[row] = nl;
      st[kM + row] = -s;
    }
  }
}

// What the main kernel left as partial sums in fp32, added in the order of their
// ranges, scaled and rounded: the first blocks dQ, one per row tile and key
// head (items of one key tile were written by the main kernel, items without
// keys get zeros), the others dK and dV, one per key tile, key head and 8
// columns (items whose rows were not cut were written; items without rows get
// zeros).  A thread has the loads of a whole range under way at once, or (FINE,
// few row tiles: 48 with 28 ranges took 49 us) those of 16 columns of four.
__device__ __forceinline__ void add_parts(float (&s)[8], const float* src) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(src)), y = __ldg(reinterpret_cast<const float4*>(src + kM * 4));
  s[0] += x.x;
  s[1] += x.y;
  s[2] += x.z;
  s[3] += x.w;
  s[4] += y.x;
  s[5] += y.y;
  s[6] += y.z;
  s[7] += y.w;
}
__device__ __forceinline__ void store_rounded(__nv_bfloat16* dst, const float (&s)[8], float scale) {
  uint4 v;
  uint32_t* pv = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int x = 0; x < 4; ++x) pv[x] = pack_bf16(s[2 * x] * scale, s[2 * x + 1] * scale);
  *reinterpret_cast<uint4*>(dst) = v;
}
template <int DP, bool FINE>
__global__ void __launch_bounds__(256) k_attn_sums_out(const __grid_constant__ BwdArgs a, int row_blocks) {
  const int row = threadIdx.x & 127;
  if ((int)blockIdx.x < row_blocks) {
    constexpr int kPieces = FINE ? DP / 16 : 1, kCols = DP / 16 / kPieces;  // pieces of a tile, 16 columns each or all
    const int block = blockIdx.x / kPieces, piece = blockIdx.x - block * kPieces;
    const int tile = block / a.kv_heads, kh = block - tile * a.kv_heads;
    const int b = a.items.find(kItemTile, tile);
    const int q0 = a.items.q0(b), rows = (a.items.q0(b + 1) - q0) * a.shared;
    const int keys = a.items.k0(b + 1) - a.items.k0(b);
    if (keys > 0 && keys <= kM) return;
    const int ranges = keys > 0 ? a.items.at(kItemKeys, b) : 0;
    const int tile0 = a.items.at(kItemTile, b);
    const int64_t range = (int64_t)(a.items.at(kItemTile, b + 1) - tile0) * a.kv_heads * (kM * DP);
    const int r = (tile - tile0) * a.tile_rows + row;
    if (row >= a.tile_rows || r >= rows) return;
    const int tok = r / a.shared, g = r - tok * a.shared, c0 = (threadIdx.x >> 7) * 8 + piece * 16;
    const float* src = a.dq_sum + ((int64_t)(a.items.at(kItemRowSlab, b) + tile - tile0) * a.kv_heads + kh) * (kM * DP) +
                       c0 * kM + row * 4;
    __nv_bfloat16* out = a.dq + ((int64_t)(q0 + tok) * a.heads + kh * a.shared + g) * a.d;
    float s[kCols][8] = {};
#pragma unroll(FINE ? 4 : 1)
    for (int k = 0; k < ranges; ++k)
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (c0 + 16 * i < a.d) add_parts(s[i], src + k * range + i * 16 * kM);
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (c0 + 16 * i < a.d) store_rounded(out + c0 + 16 * i, s[i], a.scale);
    return;
  }
  const int block = blockIdx.x - row_blocks, part = block / (DP / 8), c0 = (block - part * (DP / 8)) * 8;
  const int tile = part / a.kv_heads, kh = part - tile * a.kv_heads;
  const int b = a.items.find(kItemKeyTile, tile);
  const int ranges = a.items.at(kItemRows, b);
  const int key0 = a.items.k0(b), keys = a.items.k0(b + 1) - key0;
  const int tile0 = a.items.at(kItemKeyTile, b), j = (tile - tile0) * kM + row;
  if (ranges == 1 || j >= keys || c0 >= a.d) return;
  const bool second = threadIdx.x >= 128;
  const int64_t range = (int64_t)(a.items.at(kItemKeyTile, b + 1) - tile0) * a.kv_heads * (kM * DP);
  const float* src = (second ? a.dv_part : a.dk_part) +
                     ((int64_t)(a.items.at(kItemKeySlab, b) + tile - tile0) * a.kv_heads + kh) * (kM * DP) + c0 * kM + row * 4;
  float s[8] = {};
#pragma unroll 4
  for (int k = 0; k < ranges; ++k) add_parts(s, src + k * range);
  store_rounded((second ? a.dv : a.dk) + ((int64_t)(key0 + j) * a.kv_heads + kh) * a.d + c0, s, 1.0f);
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled from the driver through the runtime; null when it has none.
EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
    (void)cudaGetLastError();
  });
  return fn;
}

// [tokens][heads][d] read in boxes of 64 values of `box_heads` heads of
// `box_tokens` tokens; columns past d and tokens past the end read as zeros.
fvx_status encode_heads(CUtensorMap* tm, const HeadsView& t, int64_t tokens, int heads, int d, int box_heads,
                        int box_tokens) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) {
    set_error("%s: the driver has no cuTensorMapEncodeTiled", t_entry);
    return FVX_ERR_CUDA;
  }
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)t.head * 2, (cuuint64_t)t.token * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(t.p), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("%s: tensor map encoding failed (driver error %d)", t_entry, (int)r);
    return FVX_ERR_CUDA;
  }
  return FVX_OK;
}

bool tma_ready(const HeadsView& t) {
  return (reinterpret_cast<uintptr_t>(t.p) % 16) == 0 && t.token % 8 == 0 && t.head % 8 == 0 && t.token > 0 &&
         t.head > 0 && t.token < ((int64_t)1 << 38) && t.head < ((int64_t)1 << 38);
}

int tile_rows(const AttnCall& c) { return c.shared * (kM / c.shared); }

// Units of the forward pass: pairs of query tiles per key head and split.
int64_t fwd_units(const AttnCall& c, int splits, std::vector<int32_t>* prefix) {
  int64_t n = 0;
  for (int b = 0; b < c.items; ++b) {
    if (prefix) (*prefix)[b] = (int32_t)n;
    const int64_t rows = (c.q_offsets[b + 1] - c.q_offsets[b]) * c.shared;
    n += (rows + 2 * tile_rows(c) - 1) / (2 * tile_rows(c)) * c.kv_heads * splits;
  }
  if (prefix) (*prefix)[c.items] = (int32_t)n;
  return n;
}

template <int DP>
fvx_status forward(const AttnCall& c, cudaStream_t s, Scratch& scr) {
  using C = Fwd<DP>;
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  FwdArgs a;
  int64_t longest = 1;
  for (int b = 0; b < c.items; ++b)
    longest = std::max(longest, (c.kv_offsets[b + 1] - c.kv_offsets[b] + kM - 1) / kM);
  const int64_t tiles = fwd_units(c, 1, nullptr);
  // Split the keys only where there are fewer units than multiprocessors.
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>({sms / std::max<int64_t>(tiles, 1), longest, 64}));
  std::vector<int32_t> prefix((size_t)c.items + 1);
  a.units = (int)fwd_units(c, a.splits, &prefix);
  FVX_TRY(attn_items(c, prefix.data(), 3, s, scr, &a.items));
  FVX_TRY(encode_heads(&a.tq, c.q, c.nq, c.heads, c.d, c.shared, kM / c.shared));
  // without any key the maps are never read: the queries' stands in
  a.tk = a.tv = a.tq;
  if (c.nk > 0) {
    FVX_TRY(encode_heads(&a.tk, c.k, c.nk, c.kv_heads, c.d, 1, kM));
    FVX_TRY(encode_heads(&a.tv, c.v, c.nk, c.kv_heads, c.d, 1, kM));
  }
  a.mask = c.mask;
  a.out = (__nv_bfloat16*)c.out;
  a.lse = c.lse;
  a.part = a.top = a.total = nullptr;
  a.all_rows = c.nq * c.heads;
  if (a.splits > 1) {
    a.part = scr.get<float>((size_t)a.splits * a.all_rows * c.d);
    a.top = scr.get<float>((size_t)a.splits * a.all_rows);
    a.total = scr.get<float>((size_t)a.splits * a.all_rows);
    if (!a.part || !a.top || !a.total) return FVX_ERR_ALLOC;
  }
  a.status = device_status_word();
  if (!a.status) {
    set_error("%s: could not set up the device status word", t_entry);
    return FVX_ERR_CUDA;
  }
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.shared = c.shared;
  a.d = c.d;
  a.tile_rows = tile_rows(c);
  a.wide_out = c.d % 16 == 0 && reinterpret_cast<uintptr_t>(c.out) % 32 == 0;
  a.c = c.scale * kLog2e;
  static std::atomic<uint64_t> allowed{0};
  FVX_TRY(allow_smem((const void*)k_attn_tc_fwd<DP>, (int)C::kSmem, allowed));
  {
    LaunchScope ls("attn_tc_fwd", s);
    k_attn_tc_fwd<DP><<<std::min(a.units, sms), kFwdThreads, C::kSmem, s>>>(a);
    FVX_TRY(check_launch("attn_tc_fwd"));
  }
  return a.splits > 1 ? attn_join(c, a.part, a.top, a.total, a.splits, s) : FVX_OK;
}

// Cuts the backward pass into units of ranges of row tiles and key tiles of an
// item and key head.  A cut of the rows costs partial sums of dK and dV for
// every key tile, one of the keys a partial sum of dQ for every row tile, and a
// unit pays for each of its key tiles (loads, results), so the cut that gives
// an item its share of units is the one with the least of
//   steps of the longest unit + its key tiles + the partial sums' traffic,
// in cycles: a step's products and softmax about 1500, a key tile 3000 (with
// partial sums 5000), 25 bytes a cycle and multiprocessor for the sums.
struct BwdPlan {
  std::vector<int32_t> more;  // the arrays from kItemUnit on: items + 1 values each
  int units = 0, tiles = 0, key_tiles = 0, row_slabs = 0, key_slabs = 0;
  bool dq_zeros = false, dkv_zeros = false;
};
BwdPlan bwd_plan(const AttnCall& c, int sms) {
  const int n = c.items + 1;
  BwdPlan p;
  p.more.assign((size_t)(kItemArrays - kItemUnit) * n, 0);
  auto array = [&](AttnArray which) { return p.more.data() + (size_t)(which - kItemUnit) * n; };
  int32_t *units = array(kItemUnit), *tiles = array(kItemTile), *rr = array(kItemRows), *kr = array(kItemKeys),
          *key_tiles = array(kItemKeyTile), *row_slabs = array(kItemRowSlab), *key_slabs = array(kItemKeySlab);
  auto row_tiles = [&](int b) {
    return ((c.q_offsets[b + 1] - c.q_offsets[b]) * c.shared + tile_rows(c) - 1) / tile_rows(c);
  };
  auto tiles_of_keys = [&](int b) { return (c.kv_offsets[b + 1] - c.kv_offsets[b] + kM - 1) / kM; };
  int64_t work = 0, key_work = 0, single = 0;
  for (int b = 0; b < c.items; ++b) {
    const int64_t w = row_tiles(b) * tiles_of_keys(b);
    work += w * c.kv_heads;
    key_work += w > 0 ? tiles_of_keys(b) * c.kv_heads : 0;
    single += w > 0 ? c.kv_heads : 0;
  }
  auto ceil_div = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  // Cycles of a tile of 128 rows by 128 keys and of a key tile (its loads and
  // its gradients' way out, in fp32 where row ranges add up), measured on units
  // of 1 to 40 tiles; and of one 128-row slab of partial sums, shared by all.
  const double tile_cost = c.d <= 64 ? 3500.0 : 7000.0, key_cost = c.d <= 64 ? 5000.0 : 9000.0;
  const double sum_cost = 128.0 * 4 * (c.d <= 64 ? 64 : 128) * c.kv_heads / (sms * 25.0);
  const double share = std::max(((double)work * tile_cost + (double)key_work * key_cost) / sms, tile_cost + key_cost);
  // Main kernel and sums, 17,001 rows on 1024 keys and 15,800 on 1500, 8 heads of
  // 64: rows in 8 and 11 ranges, keys whole, 345 us; rows in 8 and 5, the second's
  // keys in 2, 343; rows whole, keys in 8 and 11, 541 (partial sums of dQ past
  // the L2).  9014 rows x 4 on 77 to 1030 keys, 2 key heads: rows in up to 40
  // ranges, keys whole, 109 us; in up to 6, keys in up to 9, 72.
  // The least room above an equal share of the work in which the units fit one
  // wave; every item then takes the fewest units that stay within it, and among
  // those the ranges with the least partial sums.  With more items than
  // multiprocessors, one unit per item and key head.
  for (double room : {1.0, 1.03, 1.06, 1.1, 1.15, 1.2, 1.3, 1.45, 1.7, 2.1, 2.6, 3.3, 4.5, 1e30}) {
    const double most = share * room;
    int64_t u = 0;
    bool fits = true;
    for (int b = 0; b < c.items && fits; ++b) {
      const int64_t T = row_tiles(b), K = tiles_of_keys(b);
      rr[b] = kr[b] = 0;
      if (T == 0 || K == 0) continue;
      if (single >= sms) {
        rr[b] = kr[b] = 1;
        continue;
      }
      double best = 1e300;
      for (int64_t k = 1; k <= std::min<int64_t>(K, sms); ++k) {
        const double ck = (double)ceil_div(K, k);
        const double rows = std::min((double)T, floor((most - ck * key_cost) / (ck * tile_cost)));
        if (rows < 1.0) continue;
        const int64_t r = ceil_div(T, (int64_t)rows);
        if (r * k * c.kv_heads > std::max<int64_t>(sms, c.kv_heads)) continue;
        const double cost = (double)(r * k) * 1e9 + sum_cost * ((r > 1 ? 4.0 * r * K : 0.0) + (double)(k * T));
        if (cost < best) {
          best = cost;
          rr[b] = (int32_t)r;
          kr[b] = (int32_t)k;
        }
      }
      fits = rr[b] > 0;
      u += (int64_t)rr[b] * kr[b] * c.kv_heads;
    }
    if (fits && (u <= sms || single >= sms)) break;
  }
  // Slabs of partial sums: at most one per row tile and key range of the units,
  // of which there are no more than multiprocessors (or one range each).
  int64_t u = 0, t = 0, kt = 0, row_slab = 0, key_slab = 0;
  for (int b = 0; b < c.items; ++b) {
    const int64_t T = row_tiles(b), K = tiles_of_keys(b);
    units[b] = (int32_t)u;
    tiles[b] = (int32_t)t;
    key_tiles[b] = (int32_t)kt;
    row_slabs[b] = (int32_t)row_slab;
    key_slabs[b] = (int32_t)key_slab;
    t += T;
    kt += K;
    if (T == 0 || K == 0) {
      p.dq_zeros |= T > 0;
      p.dkv_zeros |= K > 0;
      continue;
    }
    u += (int64_t)rr[b] * kr[b] * c.kv_heads;
    if (K > 1) row_slab += kr[b] * T;
    if (rr[b] > 1) key_slab += rr[b] * K;
  }
  p.row_slabs = (int)row_slab;
  p.key_slabs = (int)key_slab;
  units[c.items] = p.units = (int)u;
  tiles[c.items] = p.tiles = (int)t;
  key_tiles[c.items] = p.key_tiles = (int)kt;
  return p;
}

template <int DP>
fvx_status backward(const AttnCall& c, cudaStream_t s, Scratch& scr) {
  using C = Bwd<DP>;
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  const BwdPlan p = bwd_plan(c, sms);
  BwdArgs a;
  FVX_TRY(attn_items(c, p.more.data(), kItemArrays, s, scr, &a.items));
  FVX_TRY(encode_heads(&a.tq, c.q, c.nq, c.heads, c.d, c.shared, kM / c.shared));
  FVX_TRY(encode_heads(&a.tdo, c.dout, c.nq, c.heads, c.d, c.shared, kM / c.shared));
  a.tk = a.tv = a.tq;
  if (c.nk > 0) {
    FVX_TRY(encode_heads(&a.tk, c.k, c.nk, c.kv_heads, c.d, 1, kM));
    FVX_TRY(encode_heads(&a.tv, c.v, c.nk, c.kv_heads, c.d, 1, kM));
  }
  a.mask = c.mask;
  a.dq = (__nv_bfloat16*)c.dq;
  a.dk = (__nv_bfloat16*)c.dk;
  a.dv = (__nv_bfloat16*)c.dv;
  a.units = p.units;
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.shared = c.shared;
  a.d = c.d;
  a.tile_rows = tile_rows(c);
  a.c = c.scale * kLog2e;
  a.scale = c.scale;
  a.dq_sum = a.dk_part = a.dv_part = nullptr;
  a.status = device_status_word();
  if (!a.status) {
    set_error("%s: could not set up the device status word", t_entry);
    return FVX_ERR_CUDA;
  }
  const size_t row_blocks = (size_t)p.tiles * c.kv_heads;
  if (p.units > 0) {
    float* stats = scr.get<float>(row_blocks * 256);
    if (!stats) return FVX_ERR_ALLOC;
    a.stats = stats;
    const size_t slab = (size_t)c.kv_heads * kM * DP;
    if (p.row_slabs > 0 && !(a.dq_sum = scr.get<float>(p.row_slabs * slab))) return FVX_ERR_ALLOC;
    if (p.key_slabs > 0) {
      a.dk_part = scr.get<float>(p.key_slabs * slab);
      a.dv_part = scr.get<float>(p.key_slabs * slab);
      if (!a.dk_part || !a.dv_part) return FVX_ERR_ALLOC;
    }
    {
      LaunchScope ls("attn_stats", s);
      k_attn_stats<DP><<<(unsigned)row_blocks, 256, 0, s>>>(a.items, c.dout, (const __nv_bfloat16*)c.out, c.lse, c.heads,
                                                        c.kv_heads, c.shared, a.tile_rows, c.d, stats);
      FVX_TRY(check_launch("attn_stats"));
    }
    static std::atomic<uint64_t> allowed{0};
    FVX_TRY(allow_smem((const void*)k_attn_tc_bwd<DP>, (int)C::kSmem, allowed));
    LaunchScope ls("attn_tc_bwd", s);
    k_attn_tc_bwd<DP><<<std::min(a.units, sms), kBwdThreads, C::kSmem, s>>>(a);
    FVX_TRY(check_launch("attn_tc_bwd"));
  }
  const bool fine = row_blocks < 4 * (size_t)sms;
  const int64_t dq_blocks = p.row_slabs > 0 || p.dq_zeros ? (int64_t)row_blocks * (fine ? DP / 16 : 1) : 0;
  const int64_t dkv_blocks = p.key_slabs > 0 || p.dkv_zeros ? (int64_t)p.key_tiles * c.kv_heads * (DP / 8) : 0;
  if (dq_blocks + dkv_blocks > 0) {
    LaunchScope ls("attn_sums_out", s);
    if (fine) k_attn_sums_out<DP, true><<<(unsigned)(dq_blocks + dkv_blocks), 256, 0, s>>>(a, (int)dq_blocks);
    else k_attn_sums_out<DP, false><<<(unsigned)(dq_blocks + dkv_blocks), 256, 0, s>>>(a, (int)dq_blocks);
    FVX_TRY(check_launch("attn_sums_out"));
  }
  return FVX_OK;
}

}  // namespace

// The tensor cores take bf16 heads of a multiple of 8 values whose rows TMA
// can read (16-byte aligned bases and strides); anything else runs in fp32
// arithmetic on the CUDA cores.
bool attn_tc_serves(const AttnCall& c, bool backward) {
  if (c.dt != FVX_BF16 || c.d % 8 || c.shared > kM) return false;
  return tma_ready(c.q) && (c.nk == 0 || (tma_ready(c.k) && tma_ready(c.v))) && (!backward || tma_ready(c.dout));
}

fvx_status attn_tc_forward(const AttnCall& c, cudaStream_t s, Scratch& scr) {
  return c.d <= 64 ? forward<64>(c, s, scr) : forward<128>(c, s, scr);
}

fvx_status attn_tc_backward(const AttnCall& c, cudaStream_t s, Scratch& scr) {
  return c.d <= 64 ? backward<64>(c, s, scr) : backward<128>(c, s, scr);
}

}  // namespace fvx
