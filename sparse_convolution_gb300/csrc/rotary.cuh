// Heads normed and turned (formulas: rotary.cu): what a call is and the kernels
// that do it, compiled for one storage type per file (rotary_f32.cu,
// rotary_bf16.cu).
//
// A few bytes and a few operations per value: memory bounds it, if the
// instructions allow.  A kernel that computed a token's angles in every group of
// lanes and kept loads in registers spent 20 instructions per value of bf16 where
// the memory's rate leaves 22 (1,000,000 x 8 + 8 x 64 normed and turned in 1113 us,
// backward 1801).  So a persistent block per multiprocessor divides the work:
//   warps 0-15   workers: a head per group of lanes, 16 values of bf16 (8 of
//                fp32) a lane, out of shared memory, two values at a time; the
//                results go straight to global memory
//   warps 16-23  helpers: copy the next stage's tokens to shared memory, by bulk
//                copies where bases and strides are multiples of 16 bytes, by
//                words else, and compute their angles, once per token for all
//                heads of queries and keys
// 13 instructions per value (17 with the norm; counted over all warps, waits
// included), and copies under way whatever the workers do.
//
// Measured (bf16 unless said, of the copy rate of 6.76 TB/s): 1,000,000 x 8 + 8 x 64
// turned by three coordinates in 626 us (97%), normed and turned 615 (99%),
// backward 975 (93%); 300,000 x 4 + 4 x 256 395 (92%), 386 (94%), 669 (82%);
// 500,000 x 8 + 8 x 80 381 (100%), 484 (78%), 757 (75%); 150,001 x 8 + 2 x 128 out of
// rows of 12 heads 131 (87%), 129 (89%), 234 (73%); 300,000 x 16 + 16 x 64 fp32, 32
// turned, 755 (96%), 722 (101%), 1065 (103%).
// What bounds the rest: two heads of 128 per token need an angle for every four
// values (2,400,000 x 2 x 128 normed 635 us, 57%); halves that only narrow accesses
// read (300,000 x 8 + 8 x 100, of two values, normed 493 us, 58%), and rows that
// only single ones do (x 64 out of rows of odd length 495 us, 37%).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "fvx_internal.cuh"
#include "norm.cuh"

namespace fvx {

constexpr int kMaxHead = 256;
constexpr int kMaxPairs = kMaxHead / 2;

// A block's warps: those that work on the heads, and those that fetch the next
// stages' tensors and compute their angles.
constexpr int kWorkers = 16, kHelpers = 8, kHeadThreads = 32 * (kWorkers + kHelpers);
constexpr int kStages = 2;
constexpr int kMostSmem = 227 * 1024;

// A tensor that is read.  Its part of a stage lies in shared memory as in
// global, in pieces: all of it (tokens that follow one another), the heads of a
// token, or one head.
struct HeadSource {
  const void* p;
  int64_t token, head;
  int s_token, s_head;  // strides in shared memory
  int at;               // where the part begins, in bytes
  int bulk_tiles;       // the first tiles go by bulk copies
  bool whole, by_head;  // the part is one piece; a head is
};
// One of the call's tensors, cut into tiles of `tokens` tokens by `head_block` heads.
struct HeadJob {
  HeadSource in[2];  // forward: x; backward: the gradient of the result, and the forward pass's x
  void* out;
  const float* w;
  const int32_t* pos;
  float* part;  // norm backward: [blocks][d] partial sums of dw
  int64_t out_token, out_head, pos_token, pos_axis;
  int out_token32, out_head32;  // the same within a tile
  int n, heads, tokens, head_block, head_blocks, tiles;
  uint32_t block_magic;  // 2^32 / head_block, rounded up
};
struct HeadArgs {
  HeadJob job[2];
  uint64_t turns[kMaxPairs];  // turns per position step, in 2^-64
  uint32_t* status;
  int shared;  // a stage holds the same tokens of both tensors; else tiles of the first, then of the second
  int d, pairs, axes, axis1, axis2;  // pairs from axis1 (axis2) on belong to the second (third) axis
  int items, items_turned, lanes;    // a head's items: of pairs, of values that pass; lanes that share a head (32 / lanes heads at a time)
  int fours;                         // the angles' order: see AngleThread
  int pair_lanes;                    // helper threads of a token's angles: pairs, to the next power of two
  int angles, stage_bytes;           // of a stage: angles, bytes of the tensors
  float magnitude, sign, eps, inv_d;
};

enum HeadOp { kRotate, kNormRotate, kNormRotateBack };

struct HeadCall {
  HeadArgs a;
  int vec;
  bool interleaved;
  int64_t head_rows;
};

struct HeadDw {
  const float* part[2];
  float* dw[2];
  int parts[2];
  int d;
};

// The call's kernel for its storage type; dw: filled for the sums of dw that remain (backward pass).
fvx_status run_heads_f32(const char* name, HeadCall& c, HeadOp op, int jobs, const fvx_head_tensor_t* t, HeadDw* dw,
                         cudaStream_t s, Scratch* scr);
fvx_status run_heads_bf16(const char* name, HeadCall& c, HeadOp op, int jobs, const fvx_head_tensor_t* t, HeadDw* dw,
                          cudaStream_t s, Scratch* scr);

// Items of a lane: 16 values of bf16, 8 of fp32 and of bf16 one at a time
// (300,000 x 8 + 8 x 100, accesses of two values, normed: 16 values 544 us, 8 639;
// x 40, of four, 311 and 382; the backward pass of x 64 out of odd rows, one at a
// time: 16 values, whose registers spill, 1202 us, 8 667).
constexpr int items_of_lane(bool f32, int vec) { return (f32 || vec == 1 ? 4 : 8) / vec; }
// Lanes of a head of `items` items: a power of two, over which sums are quick,
// unless fewer lanes let a warp take more heads at once (500,000 x 8 + 8 x 80 bf16
// in five lanes, not eight: turned 450 to 380 us, normed 673 to 484, backward 1147
// to 760; in seven for x 100, which gain no head, normed 476 to 571).
constexpr int lanes_of_head(int items, int per_lane) {
  const int least = (items + per_lane - 1) / per_lane;
  int two = 1;
  while (two < least) two *= 2;
  return 32 / least > 32 / two ? least : two;
}

namespace {

// Sines and cosines of two angles.  s: a turn's fraction in 2^-32, plus 1/8: its
// top two bits are the quarter, the rest minus 1/8 lies within 1/8 turn of
// zero, where the Taylor series end below 2e-9.
__device__ __forceinline__ void sincos_two(uint32_t s0, uint32_t s1, float m, float ms, float& sin0, float& cos0, float& sin1,
                                           float& cos1) {
  auto both = [](float v) { return tc::pair(v, v); };
  const uint64_t x = tc::mul2(tc::pair((float)(int32_t)((s0 << 2) ^ 0x80000000u), (float)(int32_t)((s1 << 2) ^ 0x80000000u)),
                              both(3.65729519816789921e-10f));  // 2 pi / 2^34
  const uint64_t x2 = tc::mul2(x, x);
  uint64_t a = tc::fma2(x2, both(2.75573192239858907e-6f), both(-1.98412698412698413e-4f));
  a = tc::fma2(x2, a, both(8.33333333333333333e-3f));
  a = tc::fma2(x2, a, both(-1.66666666666666667e-1f));
  a = tc::fma2(tc::mul2(x, x2), a, x);
  uint64_t b = tc::fma2(x2, both(-2.75573192239858907e-7f), both(2.48015873015873016e-5f));
  b = tc::fma2(x2, b, both(-1.38888888888888889e-3f));
  b = tc::fma2(x2, b, both(4.16666666666666667e-2f));
  b = tc::fma2(x2, b, both(-0.5f));
  b = tc::fma2(x2, b, both(1.0f));
  float a0, a1, b0, b1;
  tc::unpair(a, a0, a1);
  tc::unpair(b, b0, b1);
  auto quarter = [&](uint32_t s, float sine, float cosine, float& sn, float& cs) {
    const bool swap = s & 0x40000000u;
    sn = __uint_as_float(__float_as_uint(swap ? cosine : sine) ^ (s & 0x80000000u)) * ms;
    cs = __uint_as_float(__float_as_uint(swap ? sine : cosine) ^ ((s ^ (s << 1)) & 0x80000000u)) * m;
  };
  quarter(s0, a0, b0, sin0, cos0);
  quarter(s1, a1, b1, sin1, cos1);
}

__device__ __forceinline__ float e_sub(float a, float b) { return a - b; }
__device__ __forceinline__ uint64_t e_sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {  // when this thread's copies have landed
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// tc::mbar_wait for the long waits of a kernel that memory bounds: its polls are
// apart, or those of the warps that wait take the issue slots of the warps that
// work (150 of 300 instructions per 512 values).
__device__ __forceinline__ uint32_t stage_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok;
}
template <int NAP>
__device__ __forceinline__ void stage_wait(uint32_t bar, uint32_t parity, uint32_t* status) {
  if (stage_try(bar, parity)) return;
  unsigned long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    __nanosleep(NAP);
    if (stage_try(bar, parity)) return;
    if ((it & 255u) == 0u) {
      if (t0 == 0) t0 = tc::globaltimer();
      if (tc::globaltimer() - t0 > tc::kWaitNs || *(volatile uint32_t*)status != 0u) {
        report_device_error(status, DEV_TIMEOUT);
        return;
      }
    }
  }
}
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWorkers) : "memory"); }

// A tile: its first token and head, and how many of each exist.
struct HeadTile {
  int token, head, tokens, heads;
};
__device__ __forceinline__ HeadTile head_tile(const HeadJob& j, int tile) {
  const int slab = j.head_blocks == 1 ? tile : tile / j.head_blocks;
  HeadTile s;
  s.head = (tile - slab * j.head_blocks) * j.head_block;
  s.token = slab * j.tokens;
  s.tokens = min(j.tokens, j.n - s.token);
  s.heads = min(j.head_block, j.heads - s.head);
  return s;
}

// 0 or 1: whether a piece starts in the second half of a 4-byte word (bf16 alone)
template <typename T>
__device__ __forceinline__ int odd_start(const HeadSource& src, int token, int head) {
  if constexpr (sizeof(T) == 2) {
    if (src.whole) return 0;
    return (int)(((uint32_t)(reinterpret_cast<uintptr_t>(src.p) >> 1) + (uint32_t)token * (uint32_t)src.token +
                  (uint32_t)head * (uint32_t)src.head) & 1u);
  }
  return 0;
}
template <typename T>
__device__ __forceinline__ uint32_t piece_bytes(const HeadSource& src, const HeadJob& j, const HeadTile& s, int d) {
  const int values = src.whole ? j.tokens * src.s_token : src.by_head ? d : (s.heads - 1) * src.s_head + d;
  return ((uint32_t)values * (uint32_t)sizeof(T) + 15u) & ~15u;
}
template <typename T>
__device__ __forceinline__ uint32_t bulk_bytes(const HeadSource& src, const HeadJob& j, int tile, const HeadTile& s, int d) {
  if (tile >= src.bulk_tiles) return 0u;
  return piece_bytes<T>(src, j, s, d) * (src.whole ? 1 : s.tokens * (src.by_head ? s.heads : 1));
}
// Starts the copies of a tile's part of src to the stage at `to`.
template <typename T>
__device__ __forceinline__ void fetch_source(const HeadSource& src, const HeadJob& j, int tile, const HeadTile& s, int d,
                                             uint32_t to, uint32_t bar, int helper) {
  const int lane = threadIdx.x & 31;
  const T* base = reinterpret_cast<const T*>(src.p);
  const int per_token = src.by_head ? s.heads : 1;
  to += src.at;
  if (tile < src.bulk_tiles) {
    const int pieces = src.whole ? 1 : s.tokens * per_token;
    const uint32_t bytes = piece_bytes<T>(src, j, s, d);
    for (int i = helper + kHelpers * lane; i < pieces; i += 32 * kHelpers) {
      const int t = per_token == 1 ? i : i / per_token, h = i - t * per_token;
      tc::bulk_load(to + (t * src.s_token + h * src.s_head) * (int)sizeof(T),
                    base + (s.token + t) * src.token + (s.head + h) * src.head, bytes, bar);
    }
    return;
  }
  const int values = src.by_head ? d : (s.heads - 1) * src.s_head + d;
  // whole words: the halves of a piece's first and last word that are not its own are copied with them
  for (int i = helper; i < s.tokens * per_token; i += kHelpers) {
    const int t = per_token == 1 ? i : i / per_token, h = i - t * per_token;
    const uintptr_t from = reinterpret_cast<uintptr_t>(base + (s.token + t) * src.token + (s.head + h) * src.head);
    const uint32_t dst = to + (t * src.s_token + h * src.s_head + odd_start<T>(src, s.token + t, s.head + h)) * (int)sizeof(T);
    const int words = (int)((from + values * sizeof(T) + 3) / 4 - from / 4);
    for (int k = lane; k < words; k += 32) copy4((dst & ~3u) + 4 * k, reinterpret_cast<const void*>((from & ~(uintptr_t)3) + 4 * k));
  }
}
// Cosines and sines of a tile's tokens, each computed once for all its heads.  A
// helper thread keeps its pair; the positions of its next four tokens are under
// way while it computes, those of a tile's first ones since before its stage
// was free.
struct AngleThread {
  static constexpr int kAtOnce = 4;
  const HeadArgs& a;
  const int p, first, apart, place;
  const bool has;
  uint32_t lo, hi, c;  // the pair's step, and what the position's bias and the 1/8 turn make
  int at[kAtOnce];

  __device__ __forceinline__ AngleThread(const HeadArgs& args, const uint64_t* turns, int thread)
      : a(args),
        p(thread & (args.pair_lanes - 1)),
        first(thread / args.pair_lanes),
        apart(32 * kHelpers / args.pair_lanes),
        // halves in vectors of eight: the first four pairs of every eight, then the others, as the lanes read them
        place(args.fours ? (p >> 2 & 1) * (args.pairs >> 1) + (p >> 3 << 2) + (p & 3) : p),
        has(p < args.pairs) {
    const uint64_t step = has ? turns[p] : 0;
    lo = (uint32_t)step;
    hi = (uint32_t)(step >> 32);
    c = 0x20000000u - (uint32_t)((step << 31) >> 32);
  }
  // The upper half of step * position modulo 2^64, plus 1/8 turn: the product
  // wraps at whole turns by itself, so a position of any size loses nothing that
  // its step does not.
  __device__ __forceinline__ uint32_t turn(int pos) const {
    const uint32_t u = (uint32_t)pos ^ 0x80000000u;  // pos + 2^31
    return __umulhi(lo, u) + hi * u + c;
  }
  __device__ __forceinline__ const int32_t* positions(const HeadJob& j, const HeadTile& s) const {
    return j.pos + ((p >= a.axis1) + (p >= a.axis2)) * j.pos_axis + (int64_t)(s.token + first) * j.pos_token;
  }
  __device__ __forceinline__ void ahead(const HeadJob& j, const int32_t* pos, int left) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) at[k] = has && k * apart < left ? __ldg(pos + (int64_t)(k * apart) * j.pos_token) : 0;
  }
  __device__ __forceinline__ void start(const HeadJob& j, const HeadTile& s) { ahead(j, positions(j, s), s.tokens - first); }
  __device__ __forceinline__ void compute(const HeadJob& j, const HeadTile& s, float* angles) {
    if (!has) return;
    const float ms = a.magnitude * a.sign;
    const int32_t* pos = positions(j, s);
    float* to = angles + first * a.pairs + place;
    for (int left = s.tokens - first; left > 0; left -= kAtOnce * apart) {
      uint32_t turns[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) turns[k] = turn(at[k]);
      pos += (int64_t)(kAtOnce * apart) * j.pos_token;
      ahead(j, pos, left - kAtOnce * apart);
#pragma unroll
      for (int k = 0; k < kAtOnce; k += 2) {
        float s0, c0, s1, c1;
        sincos_two(turns[k], turns[k + 1], a.magnitude, ms, s0, c0, s1, c1);
        if (k * apart < left) {
          to[0] = c0;
          to[a.angles] = s0;
        }
        to += apart * a.pairs;
        if ((k + 1) * apart < left) {
          to[0] = c1;
          to[a.angles] = s1;
        }
        to += apart * a.pairs;
      }
    }
  }
};

// A lane holds ITEMS items of a head, each two vectors of V values in memory, P
// apart: the first and second partners (u and v) of V pairs (halves), or V / 2
// interleaved pairs each; or up to 2V values that pass, split alike.  So a
// group's lanes always read and write side by side.
// Pairs of fp32 values are computed on two at a time.  FULL: every lane has all
// its items, and all turn.
template <typename T, int V, int ITEMS, bool INTERLEAVED, int OP, bool FULL>
struct Heads {
  static constexpr bool kNorm = OP != kRotate, kBack = OP == kNormRotateBack;
  using E = typename Lane<V>::E;
  static constexpr int N = Lane<V>::N;
  const HeadArgs& a;
  const int lane, group, groups;
  int at[ITEMS], second[ITEMS];
  bool has_a[ITEMS], has_b[ITEMS];
  E dw[kBack ? ITEMS : 1][2][N];

  __device__ __forceinline__ explicit Heads(const HeadArgs& args)
      : a(args), lane((threadIdx.x & 31) % args.lanes), group((threadIdx.x & 31) / args.lanes), groups(32 / args.lanes) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int item = lane + i * a.lanes;
      place(a, item, at[i], second[i]);
      has_a[i] = FULL || item < a.items;
      has_b[i] = FULL || (has_a[i] && second[i] < a.d);
      // what a lane does not have it reads elsewhere and clears
      if (!has_a[i]) at[i] = 0;
      if (!has_b[i]) second[i] = at[i];
    }
    clear();
  }
  __device__ __forceinline__ void clear() {
    if constexpr (kBack) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) dw[i][0][k] = dw[i][1][k] = e_all<E>(0.0f);
    }
  }
  // where an item's two vectors start in the head
  static __device__ __forceinline__ void place(const HeadArgs& a, int item, int& first, int& second) {
    const bool turned = item < a.items_turned;
    if (INTERLEAVED && V == 1 && turned) {
      first = 2 * item;
      second = first + 1;
      return;
    }
    first = turned ? item * V : 2 * a.pairs + (item - a.items_turned) * V;
    second = first + (turned ? a.pairs : (a.items - a.items_turned) * V);
  }
  // the channel of value k of an item's side (0: u, 1: v); d or more: none
  static __device__ __forceinline__ int channel(const HeadArgs& a, int item, int side, int k) {
    int first, second;
    place(a, item, first, second);
    if (!INTERLEAVED || V == 1) return (side ? second : first) + k;
    return (k < V / 2 ? first + 2 * k : second + 2 * k - V) + side;
  }
  // Sums over the lanes that share a head.  Where they are no power of two, each
  // lane adds runs of 1, 2, 4, ... lanes from its own on, around the group: one
  // run for each bit of their number.
  __device__ __forceinline__ void head_sums(float& v, float& w) const {
    if ((a.lanes & (a.lanes - 1)) == 0) {
#pragma unroll 1
      for (int o = a.lanes >> 1; o > 0; o >>= 1) {
        v += __shfl_xor_sync(0xffffffffu, v, o);
        if constexpr (kBack) w += __shfl_xor_sync(0xffffffffu, w, o);
      }
      return;
    }
    float all_v = 0.0f, all_w = 0.0f;
    const int first = group * a.lanes;
    auto from = [&](int ahead) {
      const int l = lane + ahead;
      return first + (l >= a.lanes ? l - a.lanes : l);
    };
    int done = 0;
#pragma unroll 1
    for (int run = 1;; run <<= 1) {
      if (a.lanes & run) {
        const int at = from(done);
        all_v += __shfl_sync(0xffffffffu, v, at);
        if constexpr (kBack) all_w += __shfl_sync(0xffffffffu, w, at);
        done += run;
        if (done == a.lanes) break;
      }
      const int at = from(run);
      v += __shfl_sync(0xffffffffu, v, at);
      if constexpr (kBack) w += __shfl_sync(0xffffffffu, w, at);
    }
    v = all_v;
    w = all_w;
  }

  // A group's head within the tile.  Groups without one take the tile's first and store nothing.
  struct Row {
    int token, head;
    bool live;
  };
  struct In {
    Pack<T, V> x[ITEMS], y[ITEMS];
  };
  __device__ __forceinline__ void read(const HeadSource& src, const unsigned char* stage, const HeadTile& s, const Row& r,
                                       In& in) const {
    int off = r.token * src.s_token + r.head * src.s_head;
    if constexpr (V == 1) off += odd_start<T>(src, s.token + r.token, s.head + (src.by_head ? r.head : 0));
    const T* p = reinterpret_cast<const T*>(stage + src.at) + off;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      in.x[i] = raw_vec<T, V>(p + at[i]);
      in.y[i] = raw_vec<T, V>(p + second[i]);
      if (!FULL && !has_a[i]) in.x[i] = no_vec<T, V>();
      if (!FULL && !has_b[i]) in.y[i] = no_vec<T, V>();
    }
  }
  static __device__ __forceinline__ void split(const In& in, E (&e)[ITEMS][2][N]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float f[2 * V], u[V], v[V];
      if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t words[V];  // two values each
        memcpy(words, &in.x[i], 2 * V);
        memcpy(words + V / 2, &in.y[i], 2 * V);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          f[2 * k] = __uint_as_float(words[k] << 16);
          f[2 * k + 1] = __uint_as_float(words[k] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          f[k] = Elem<T>::get(in.x[i].v[k]);
          f[V + k] = Elem<T>::get(in.y[i].v[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        u[k] = INTERLEAVED ? f[2 * k] : f[k];
        v[k] = INTERLEAVED ? f[2 * k + 1] : f[V + k];
      }
      to_pairs<V>(u, e[i][0]);
      to_pairs<V>(v, e[i][1]);
    }
  }
  // Keeps the compiler from holding the widened values instead: they are twice the registers.
  static __device__ __forceinline__ void keep_narrow(In& in) {
    if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        uint32_t words[V];
        memcpy(words, &in.x[i], 2 * V);
        memcpy(words + V / 2, &in.y[i], 2 * V);
#pragma unroll
        for (int k = 0; k < V; ++k) asm volatile("" : "+r"(words[k]));
        memcpy(&in.x[i], words, 2 * V);
        memcpy(&in.y[i], words + V / 2, 2 * V);
      }
    }
  }
  __device__ __forceinline__ void store(const HeadJob& j, T* out, const Row& r, const E (&e)[ITEMS][2][N]) const {
    out += r.token * j.out_token32 + r.head * j.out_head32;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float u[V], v[V];
      from_pairs<V>(e[i][0], u);
      from_pairs<V>(e[i][1], v);
      Pack<T, V> x, y;
      float f[2 * V];
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) f[k] = INTERLEAVED ? (k & 1 ? v[k / 2] : u[k / 2]) : k < V ? u[k % V] : v[k % V];
      if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t words[V];
#pragma unroll
        for (int k = 0; k < V; ++k) words[k] = tc::pack_bf16(f[2 * k], f[2 * k + 1]);
        memcpy(&x, words, 2 * V);
        memcpy(&y, words + V / 2, 2 * V);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x.v[k] = Elem<T>::put(f[k]);
          y.v[k] = Elem<T>::put(f[V + k]);
        }
      }
      if (r.live && has_a[i]) *reinterpret_cast<Pack<T, V>*>(out + at[i]) = x;
      if (r.live && has_b[i]) *reinterpret_cast<Pack<T, V>*>(out + second[i]) = y;
    }
  }
  // V values in shared memory, in pieces of W that are `apart` apart
  template <int W>
  static __device__ __forceinline__ void vector(const float* p, int apart, E (&e)[N]) {
    float f[V];
#pragma unroll
    for (int k = 0; k < V; k += W) {
      const Pack<float, W> x = raw_vec<float, W>(p + k / W * apart);
#pragma unroll
      for (int n = 0; n < W; ++n) f[k + n] = x.v[n];
    }
    to_pairs<V>(f, e);
  }
  static constexpr int kWide = V > 4 ? 4 : V;
  // Weights: a row of a group's lanes for each item, side and four values, 32 lanes apart.
  static constexpr int kLanes = 32, kWeights = kLanes * ITEMS * 2 * V;
  static __device__ __forceinline__ int weight_place(int lane, int i, int side, int k) {
    return (((i * 2 + side) * (V / kWide) + k / kWide) * kLanes + lane) * kWide + k % kWide;
  }
  __device__ __forceinline__ void weights(const float* w, int i, int side, E (&e)[N]) const {
    vector<kWide>(w + weight_place(0, i, side, 0), kLanes * kWide, e);
  }
  __device__ __forceinline__ void rotate_item(const float* angles, int item, E (&e)[2][N]) const {
    constexpr int W = V == 8 || (INTERLEAVED && V > 1) ? V / 2 : V;
    const float* p = angles + item * W;
    E c[N], s[N];
    vector<W>(p, a.pairs / 2, c);
    vector<W>(p + a.angles, a.pairs / 2, s);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const E u = e[0][k], v = e[1][k];
      e[0][k] = e_sub(e_mul(u, c[k]), e_mul(v, s[k]));
      e[1][k] = e_fma(v, c[k], e_mul(u, s[k]));
    }
  }
  __device__ __forceinline__ void rotate(const float* angles, const Row& r, E (&e)[ITEMS][2][N]) const {
    const float* p = angles + r.token * a.pairs;
    if (FULL || a.items_turned == a.items) {  // the same for all lanes; those without an item turn their zeros
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) rotate_item(p, has_a[i] ? lane + i * a.lanes : 0, e[i]);
    } else {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (lane + i * a.lanes < a.items_turned) rotate_item(p, lane + i * a.lanes, e[i]);
    }
  }

  __device__ __forceinline__ void forward(const HeadJob& j, const unsigned char* stage, const float* angles, const float* w,
                                          const HeadTile& s, const Row& r, T* out) const {
    E e[ITEMS][2][N], sum = e_all<E>(0.0f);
    In in;
    read(j.in[0], stage, s, r, in);
    split(in, e);
    if constexpr (kNorm) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) sum = e_fma(e[i][1][k], e[i][1][k], e_fma(e[i][0][k], e[i][0][k], sum));
      float square = e_sum(sum), none = 0.0f;
      head_sums(square, none);
      const E rstd = e_all<E>(rsqrtf(fmaf(square, a.inv_d, a.eps)));
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          E wt[N];
          weights(w, i, side, wt);
#pragma unroll
          for (int k = 0; k < N; ++k) e[i][side][k] = e_mul(e_mul(e[i][side][k], rstd), wt[k]);
        }
    }
    rotate(angles, r, e);
    store(j, out, r, e);
  }
  __device__ __forceinline__ void backward(const HeadJob& j, const unsigned char* stage, const float* angles, const float* w,
                                           const HeadTile& s, const Row& r, T* out) {
    E g[ITEMS][2][N], xx = e_all<E>(0.0f), gx = xx;
    In in, xs;
    read(j.in[0], stage, s, r, in);
    read(j.in[1], stage, s, r, xs);
    split(in, g);
    rotate(angles, r, g);
    {
      E x[ITEMS][2][N];
      split(xs, x);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          E wt[N];
          weights(w, i, side, wt);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            xx = e_fma(x[i][side][k], x[i][side][k], xx);
            gx = e_fma(e_mul(g[i][side][k], wt[k]), x[i][side][k], gx);
          }
        }
    }
    float square = e_sum(xx), product = e_sum(gx);
    head_sums(square, product);
    const float rstd = rsqrtf(fmaf(square, a.inv_d, a.eps));
    // a group without a head adds nothing to dw
    const E rs = e_all<E>(rstd), mine = e_all<E>(r.live ? rstd : 0.0f), back = e_all<E>(-(product * a.inv_d) * rstd * rstd);
    keep_narrow(xs);
    E x[ITEMS][2][N];
    split(xs, x);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        E wt[N];
        weights(w, i, side, wt);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const E gk = g[i][side][k], xk = x[i][side][k];
          if (kBack) dw[i][side][k] = e_fma(gk, e_mul(xk, mine), dw[i][side][k]);
          g[i][side][k] = e_mul(rs, e_fma(xk, back, e_mul(gk, wt[k])));
        }
      }
    store(j, out, r, g);
  }
  // The block's part of dw: groups of a warp by shuffles, then its warps, in a fixed order.
  __device__ __forceinline__ void write_part(float* sh, float* part) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        float f[V], sum[V];
        from_pairs<V>(dw[i][side], f);
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] = f[k];
        if ((a.lanes & (a.lanes - 1)) == 0) {
#pragma unroll 1
          for (int o = a.lanes; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < V; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
        } else {
#pragma unroll 1
          for (int g = 1; g < groups; ++g)
#pragma unroll
            for (int k = 0; k < V; ++k) sum[k] += __shfl_down_sync(0xffffffffu, f[k], g * a.lanes);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = channel(a, lane + i * a.lanes, side, k);
          if (group == 0 && has_a[i] && c < a.d) sh[(threadIdx.x >> 5) * a.d + c] = sum[k];
        }
      }
    workers_sync();
    if (part)
      for (int c = threadIdx.x; c < a.d; c += 32 * kWorkers) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kWorkers; ++k) s += sh[k * a.d + c];
        part[c] = s;
      }
    workers_sync();
    clear();
  }
};

// Shared memory: barriers, steps, both tensors' weights, the workers' parts of
// dw, then the stages' angles and tensors.
struct HeadLayout {
  int turns, w, parts, angles, stages, bytes;
  __host__ __device__ HeadLayout(const HeadArgs& a, int weights, bool back) {
    turns = 64;
    w = turns + ((a.pairs + 1) & ~1) * 8;
    parts = w + 2 * weights * 4;
    angles = parts + (back ? kWorkers * a.d * 4 : 0);
    stages = (angles + kStages * 2 * a.angles * 4 + 127) & ~127;
    bytes = stages + kStages * a.stage_bytes;
  }
};

template <typename T, int V, int ITEMS, bool INTERLEAVED, int OP, bool FULL>
__global__ void __launch_bounds__(kHeadThreads, 1) k_heads(const __grid_constant__ HeadArgs args) {
  using H = Heads<T, V, ITEMS, INTERLEAVED, OP, FULL>;
  extern __shared__ __align__(128) unsigned char sm[];
  constexpr int weights = H::kNorm ? H::kWeights : 0;
  const HeadLayout lay(args, weights, H::kBack);
  uint64_t* const turns = reinterpret_cast<uint64_t*>(sm + lay.turns);
  float* const w = reinterpret_cast<float*>(sm + lay.w);
  float* const angles = reinterpret_cast<float*>(sm + lay.angles);
  unsigned char* const stages = sm + lay.stages;
  const uint32_t full = tc::smem_u32(sm), empty = full + 8 * kStages;
  const int warp = threadIdx.x >> 5;
  const int tiles = args.shared ? args.job[0].tiles : args.job[0].tiles + args.job[1].tiles;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      // the helpers' threads when their copies have landed, their warps when the angles are there, the bytes of the bulk copies
      tc::mbar_init(full + 8 * i, 32 * kHelpers + kHelpers + 1);
      tc::mbar_init(empty + 8 * i, kWorkers);
    }
    tc::mbar_init_fence();
  }
  for (int p = threadIdx.x; p < args.pairs; p += kHeadThreads) turns[p] = args.turns[p];
  if constexpr (H::kNorm)
    for (int n = threadIdx.x; n < 2 * args.lanes * ITEMS * 2 * V; n += kHeadThreads) {
      const int k = n % V, side = n / V & 1, item = (n / (2 * V)) % (args.lanes * ITEMS), seg = n / (2 * V) / (args.lanes * ITEMS);
      const int c = H::channel(args, item, side, k);
      const float* from = seg ? args.job[1].w : args.job[0].w;
      w[seg * weights + H::weight_place(item % args.lanes, item / args.lanes, side, k)] = from && c < args.d ? __ldg(from + c) : 1.0f;
    }
  __syncthreads();
  uint32_t i = 0, phase = 0, taken = 0;
  auto next_stage = [&]() {
    ++taken;
    if (++i == kStages) {
      i = 0;
      phase ^= 1u;
    }
  };
  // Registers: 768 threads at 80 are launched, 61,440: 512 at 88 and 256 at 64 for the backward pass.
  if (warp >= kWorkers) {
    // ---------------------------------------------------------------- helpers
    if constexpr (H::kBack) tc::setmaxnreg_dec<64>();
    const int helper = warp - kWorkers, lane = threadIdx.x & 31;
    auto fetch = [&](const HeadJob& j, int tile, const HeadTile& s, uint32_t to) {
      fetch_source<T>(j.in[0], j, tile, s, args.d, to, full + 8 * i, helper);
      if constexpr (H::kBack) fetch_source<T>(j.in[1], j, tile, s, args.d, to, full + 8 * i, helper);
    };
    auto bytes = [&](const HeadJob& j, int tile, const HeadTile& s) {
      uint32_t b = bulk_bytes<T>(j.in[0], j, tile, s, args.d);
      if constexpr (H::kBack) b += bulk_bytes<T>(j.in[1], j, tile, s, args.d);
      return b;
    };
    AngleThread angle(args, turns, threadIdx.x - 32 * kWorkers);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const uint32_t to = tc::smem_u32(stages) + i * args.stage_bytes;
      float* const mine = angles + i * 2 * args.angles;
      const bool second = !args.shared && tile >= args.job[0].tiles;
      const int t0 = second ? 0 : tile, t1 = args.shared ? tile : tile - args.job[0].tiles;
      HeadTile s0 = {}, s1 = {};
      if (!second) s0 = head_tile(args.job[0], t0);
      if (second || args.shared) s1 = head_tile(args.job[1], t1);
      if (args.pairs) {
        if (second) angle.start(args.job[1], s1);
        else angle.start(args.job[0], s0);
      }
      if (taken >= kStages) stage_wait<300>(empty + 8 * i, phase ^ 1u, args.status);
      __syncwarp();
      // what was written here by other copies and read is behind; bulk copies come next
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (helper == 0) {
        uint32_t b = 0;
        if (!second) b += bytes(args.job[0], t0, s0);
        if (second || args.shared) b += bytes(args.job[1], t1, s1);
        if (lane == 0) tc::mbar_expect_tx(full + 8 * i, b);
        __syncwarp();
      }
      if (!second) fetch(args.job[0], t0, s0, to);
      if (second || args.shared) fetch(args.job[1], t1, s1, to);
      if (args.pairs) {
        if (second) angle.compute(args.job[1], s1, mine);
        else angle.compute(args.job[0], s0, mine);
      }
      copies_arrive(full + 8 * i);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full + 8 * i);
      next_stage();
    }
    // after a give-up, let the copies in flight land before the block exits
    for (uint32_t k = 1; k <= kStages && k <= taken; ++k)
      tc::mbar_drain(full + 8 * ((taken - k) % kStages), ((taken - k) / kStages) & 1u);
    return;
  }
  // ------------------------------------------------------------------ workers
  if constexpr (H::kBack) tc::setmaxnreg_inc<88>();
  H h(args);
  bool first_done = false;
  auto rows = [&](const HeadJob& j, int tile, const float* seg_weights) {
    const float* const weight = seg_weights + h.lane * H::kWide;
    const HeadTile s = head_tile(j, tile);
    const unsigned char* const stage = stages + i * args.stage_bytes;
    const float* const at = angles + i * 2 * args.angles;
    T* const out = reinterpret_cast<T*>(j.out) + s.token * j.out_token + s.head * j.out_head;
    const int count = s.tokens * j.head_block;
    for (int r0 = warp * h.groups; r0 < count; r0 += kWorkers * h.groups) {
      typename H::Row r;
      const int k = r0 + h.group;
      r.token = j.head_block == 1 ? k : (int)__umulhi((uint32_t)k, j.block_magic);
      r.head = k - r.token * j.head_block;
      r.live = r.token < s.tokens && r.head < s.heads && h.group < h.groups;  // lanes left over have none
      if (!r.live) r.token = r.head = 0;
      if constexpr (H::kBack) h.backward(j, stage, at, weight, s, r, out);
      else h.forward(j, stage, at, weight, s, r, out);
    }
  };
  float* const parts = reinterpret_cast<float*>(sm + lay.parts);
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    stage_wait<40>(full + 8 * i, phase, args.status);
    __syncwarp();
    const bool second = !args.shared && tile >= args.job[0].tiles;
    if (!second) rows(args.job[0], tile, w);
    if (second || args.shared) {
      if constexpr (H::kBack) {
        if (!first_done) {
          first_done = true;
          h.write_part(parts, args.job[0].part ? args.job[0].part + (int64_t)blockIdx.x * args.d : nullptr);
        }
      }
      rows(args.job[1], args.shared ? tile : tile - args.job[0].tiles, w + weights);
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(empty + 8 * i);
    next_stage();
  }
  if constexpr (H::kBack) {
    if (!first_done) h.write_part(parts, args.job[0].part ? args.job[0].part + (int64_t)blockIdx.x * args.d : nullptr);
    h.write_part(parts, args.job[1].part ? args.job[1].part + (int64_t)blockIdx.x * args.d : nullptr);
  }
}

// f<V, ITEMS, INTERLEAVED>() for the call's vectors and layout
template <typename T, typename F>
fvx_status by_shape(const HeadCall& c, F&& f) {
  auto layout = [&]<int V>() -> fvx_status {
    constexpr int kItems = items_of_lane(sizeof(T) == 4, V);
    return c.interleaved ? f.template operator()<V, kItems, true>() : f.template operator()<V, kItems, false>();
  };
  if constexpr (sizeof(T) == 2)
    if (c.vec == 8) return layout.template operator()<8>();
  if (c.vec == 4) return layout.template operator()<4>();
  return c.vec == 2 ? layout.template operator()<2>() : layout.template operator()<1>();
}

uint32_t magic_of(int v) { return (uint32_t)((((uint64_t)1 << 32) + v - 1) / v); }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Heads of a token that a quarter of their size at most lies between go in one piece.
bool near(const HeadSource& s, int d) { return s.head <= d + d / 4; }
// Tokens that follow one another likewise: their tiles are one piece.
bool in_line(const HeadSource& s, const HeadJob& j, int d) {
  return near(s, d) && (j.heads > 1 ? s.token == j.heads * s.head : s.token <= d + d / 4) && s.token >= d;
}

// How a tile's part of a tensor is copied and lies in shared memory; its bytes.
int64_t place_source(HeadSource& s, const HeadJob& j, int d, int elem) {
  auto at16 = [&](int64_t values) { return values * elem % 16 == 0; };
  const bool base16 = reinterpret_cast<uintptr_t>(s.p) % 16 == 0;
  const int64_t slabs = ((int64_t)j.n + j.tokens - 1) / j.tokens;
  s.whole = s.by_head = false;
  s.bulk_tiles = 0;
  if (!near(s, d)) {
    s.by_head = true;
    s.s_head = (int)up(d + 1, 16 / elem);
    s.s_token = s.s_head * j.head_block;
    if (base16 && at16(s.token) && at16(s.head) && at16(d)) s.bulk_tiles = j.tiles;
    return (int64_t)j.tokens * s.s_token * elem;
  }
  s.s_head = (int)s.head;
  const int64_t chunk = (j.head_block - 1) * s.head + d;
  if (j.head_blocks == 1 && in_line(s, j, d) && base16 && at16(j.tokens * s.token)) {
    s.whole = true;
    s.s_token = (int)s.token;
    // a piece must not reach past the last head's end
    s.bulk_tiles = (int)(((j.n - 1) * s.token + chunk) / (j.tokens * s.token));
    return (int64_t)j.tokens * s.s_token * elem;
  }
  s.s_token = (int)up(chunk + 1, 16 / elem);
  if (base16 && at16(s.token) && (j.head_blocks == 1 || at16(j.head_block * s.head))) {
    // Pieces end at multiples of 16 bytes: where the last head of a token does
    // not, that is in the gap to the next token, and past the last one's end.
    const int64_t last = ((j.heads - 1) % j.head_block) * s.head + d;
    const bool gaps = s.token >= (j.heads - 1) * s.head + d;
    s.bulk_tiles = (int)((at16(last) ? slabs : gaps ? (j.n - 1) / j.tokens : 0) * j.head_blocks);
  }
  return (int64_t)j.tokens * s.s_token * elem;
}
// Whether offsets of results within a tile fit 32 bits; sets the strides they are computed from.
bool results_near(HeadJob& j) {
  const int64_t token = j.tokens > 1 ? j.out_token : 0, head = j.head_block > 1 ? j.out_head : 0;
  j.out_token32 = (int)token;
  j.out_head32 = (int)head;
  constexpr int64_t kMost = (int64_t)1 << 30;
  return token < kMost && head < kMost && token * j.tokens + head * j.head_block < kMost;
}

// Cuts a tensor into tiles of whole tokens, or (tokens of more than `room` bytes)
// of heads of one token.
void cut(HeadJob& j, int tokens, int heads) {
  j.tokens = tokens;
  j.head_block = heads;
  j.head_blocks = (j.heads + heads - 1) / heads;
  j.tiles = (int)(((int64_t)j.n + tokens - 1) / tokens * j.head_blocks);
  j.block_magic = heads > 1 ? magic_of(heads) : 0;
}

// Tokens of a stage of `count` tensors: up to `most` and no more than give every
// multiprocessor a stage; of the numbers that fill the workers' last turn the one
// that costs least.  A stage costs its workers' turns and about half of one to
// hand over.  Returns the turns per token.
double stage_tokens(const HeadArgs& a, const HeadJob* jobs, int count, int64_t most, int line, int sms, int* tokens) {
  const int turn = kWorkers * (32 / a.lanes);
  int n = 0, heads = 0;
  for (int k = 0; k < count; ++k) {
    n = std::max(n, jobs[k].n);
    heads = std::max(heads, jobs[k].heads);
  }
  most = std::max<int64_t>(1, std::min<int64_t>({most, ((int64_t)n + sms - 1) / sms, 4096}));
  double best = 1e300;
  auto consider = [&](int64_t t) {
    if (t >= line) t -= t % line;
    if (t < 1) return;
    double turns = 0.6;
    for (int k = 0; k < count; ++k) turns += (double)((t * jobs[k].heads + turn - 1) / turn);
    if (turns / t < best * 0.99) {
      best = turns / t;
      *tokens = (int)t;
    }
  };
  consider(most);
  for (int64_t k = most * heads / turn; k >= 1 && 2 * k * turn >= most * heads; --k) consider(k * turn / heads);
  return best;
}

template <typename T, int V, int ITEMS, bool IL, int OP, bool FULL>
fvx_status launch_heads(const char* name, HeadArgs& a, int jobs, const fvx_head_tensor_t* t, HeadDw* dw, cudaStream_t s,
                        Scratch* scr) {
  using H = Heads<T, V, ITEMS, IL, OP, FULL>;
  constexpr int kElem = (int)sizeof(T), kSources = H::kBack ? 2 : 1;
  int sms = 0;
  FVX_TRY(device_sm_count(&sms));
  a.status = device_status_word();
  if (!a.status) {
    set_error("%s: could not set up the device status word", t_entry);
    return FVX_ERR_CUDA;
  }
  constexpr int weights = H::kNorm ? H::kWeights : 0;
  a.angles = a.stage_bytes = 0;
  const HeadLayout fixed(a, weights, H::kBack);
  // Long stages, since a stage costs its hand-over: two of 110 KB for the backward
  // pass, two of 90 KB forward, where reads too far ahead of the writes cost the
  // memory more than the hand-over (1,000,000 x 8 + 8 x 64 bf16 normed in 612 us
  // with two of 90 KB, 642 of 110, 657 with three of 72; backward 1051, 967,
  // 1010; 300,000 x 4 + 4 x 256 normed 379, 379, 481; 300,000 x 16 + 16 x 64 fp32
  // normed 717, 779, 809).
  const int64_t room = (int64_t)(kMostSmem - fixed.bytes - 256) * 2 / (H::kBack ? 4 : 5) - 512;
  // bytes of a token (its heads from global memory, or one by one) and of its angles
  auto token_bytes = [&](const HeadJob& j, int heads) {
    int64_t b = 0;
    for (int k = 0; k < kSources; ++k)
      b += (near(j.in[k], a.d) ? heads * std::max<int64_t>(j.in[k].head, a.d) + (heads == 1 ? a.d / 4 : 0) + 16 / kElem
                               : (int64_t)heads * (a.d + 16 / kElem)) * kElem;
    return b;
  };
  auto line_of = [&](const HeadJob& j) {
    int line = 1;
    for (int k = 0; k < kSources; ++k)
      if (in_line(j.in[k], j, a.d))
        while (line * j.in[k].token * kElem % 16) line *= 2;
    return line;
  };
  // Queries and keys of the same tokens share a stage and its angles (the
  // backward pass keeps one tensor's dw in registers at a time).
  a.shared = OP != kNormRotateBack && jobs == 2 && a.job[0].n == a.job[1].n && a.job[0].pos == a.job[1].pos &&
             a.job[0].pos_token == a.job[1].pos_token && a.job[0].pos_axis == a.job[1].pos_axis && a.job[0].n > 0;
  const int angle_bytes = 8 * a.pairs;
  if (a.shared) {
    const int64_t bytes = token_bytes(a.job[0], a.job[0].heads) + token_bytes(a.job[1], a.job[1].heads) + angle_bytes;
    if (bytes > room) a.shared = 0;
    else {
      int tokens = 1;
      stage_tokens(a, a.job, 2, room / bytes, std::max(line_of(a.job[0]), line_of(a.job[1])), sms, &tokens);
      for (int i = 0; i < 2; ++i) cut(a.job[i], tokens, a.job[i].heads);
      if (!results_near(a.job[0]) || !results_near(a.job[1])) a.shared = 0;
    }
  }
  // Tensors of their own stages: the angles' part of a stage is what the one or
  // the other needs, or between; the cheapest.
  int64_t angle_room = 0;
  if (!a.shared) {
    double best = 1e300;
    auto needs = [&](const HeadJob& j) {
      return std::max<int64_t>(room * angle_bytes / (token_bytes(j, j.heads) + angle_bytes), angle_bytes);
    };
    const int64_t lo = std::min(needs(a.job[0]), needs(a.job[jobs - 1])), hi = std::max(needs(a.job[0]), needs(a.job[jobs - 1]));
    for (int k = 0; k < (lo == hi ? 1 : 4); ++k) {
      const int64_t angles = lo + (hi - lo) * k / 3;
      double turns = 0.0;
      for (int i = 0; i < jobs; ++i) {
        const HeadJob& j = a.job[i];
        int tokens = 1;
        const int64_t fit = (room - angles) / token_bytes(j, j.heads);
        if (j.n > 0 && fit > 0)
          turns += j.n * stage_tokens(a, &j, 1, angle_bytes ? std::min(fit, angles / angle_bytes) : fit, line_of(j), sms, &tokens);
      }
      if (turns < best) {
        best = turns;
        angle_room = angles;
      }
    }
  }
  for (int i = 0; i < jobs && !a.shared; ++i) {
    HeadJob& j = a.job[i];
    if (j.n == 0) continue;
    const int64_t bytes = token_bytes(j, j.heads);
    if (bytes <= room - angle_room) {
      const int64_t most = (room - angle_room) / bytes;
      int tokens = 1;
      stage_tokens(a, &j, 1, angle_bytes ? std::min(most, angle_room / angle_bytes) : most, line_of(j), sms, &tokens);
      cut(j, tokens, j.heads);
    } else {
      const int turn = kWorkers * (32 / a.lanes);
      int64_t heads = (room - angle_room) / token_bytes(j, 1);
      if (heads > turn) heads -= heads % turn;
      cut(j, 1, (int)std::max<int64_t>(1, std::min<int64_t>(heads, j.heads)));
    }
    if (!results_near(j)) {  // tokens or heads 2^30 values apart: a head at a time
      cut(j, 1, 1);
      results_near(j);
    }
  }
  for (int i = 0; i < jobs; ++i) {
    HeadJob& j = a.job[i];
    if (j.n == 0) continue;
    int64_t at = a.shared && i == 1 ? a.stage_bytes : 0;
    for (int k = 0; k < kSources; ++k) {
      j.in[k].at = (int)at;
      at += up(place_source(j.in[k], j, a.d, kElem), 128);
    }
    a.stage_bytes = (int)std::max<int64_t>(a.stage_bytes, at);
    a.angles = std::max(a.angles, (j.tokens * a.pairs + 3) & ~3);
  }
  const HeadLayout lay(a, weights, H::kBack);
  if (lay.bytes > kMostSmem) {
    set_error("%s: a stage needs %d bytes of shared memory", t_entry, lay.bytes);
    return FVX_ERR_INVALID_ARG;
  }
  const int64_t tiles = a.shared ? a.job[0].tiles : (int64_t)a.job[0].tiles + a.job[1].tiles;
  const int blocks = (int)std::min<int64_t>(tiles, sms);
  for (int i = 0; i < jobs && dw; ++i) {
    if (t[i].n == 0 || !t[i].dweight) continue;
    dw->parts[i] = blocks;
    dw->dw[i] = t[i].dweight;
    if (!(a.job[i].part = scr->get<float>((size_t)blocks * a.d))) return FVX_ERR_ALLOC;
    dw->part[i] = a.job[i].part;
  }
  if constexpr (H::kBack) {
    // The warps' shares of registers must not exceed those that the block is
    // launched with, or they wait for the rest: looked up once.
    static std::atomic<int> registers{0};
    if (registers == 0) {
      cudaFuncAttributes f;
      FVX_CUDA(cudaFuncGetAttributes(&f, (const void*)k_heads<T, V, ITEMS, IL, OP, FULL>));
      registers = f.numRegs;
    }
    if (registers * kHeadThreads < 32 * (kWorkers * 88 + kHelpers * 64)) {
      set_error("%s: the kernel was compiled for %d registers", t_entry, registers.load());
      return FVX_ERR_CUDA;
    }
  }
  static std::atomic<uint64_t> allowed{0};
  FVX_TRY(allow_smem((const void*)k_heads<T, V, ITEMS, IL, OP, FULL>, kMostSmem, allowed));
  LaunchScope ls(name, s);
  k_heads<T, V, ITEMS, IL, OP, FULL><<<blocks, kHeadThreads, lay.bytes, s>>>(a);
  return check_launch(name);
}

template <typename T>
fvx_status run_heads(const char* name, HeadCall& c, HeadOp op, int jobs, const fvx_head_tensor_t* t, HeadDw* dw,
                     cudaStream_t s, Scratch* scr) {
  return by_shape<T>(c, [&]<int V, int ITEMS, bool IL>() -> fvx_status {
    auto go = [&]<bool FULL>() -> fvx_status {
      if (op == kRotate) return launch_heads<T, V, ITEMS, IL, kRotate, FULL>(name, c.a, jobs, t, dw, s, scr);
      if (op == kNormRotate) return launch_heads<T, V, ITEMS, IL, kNormRotate, FULL>(name, c.a, jobs, t, dw, s, scr);
      return launch_heads<T, V, ITEMS, IL, kNormRotateBack, FULL>(name, c.a, jobs, t, dw, s, scr);
    };
    // heads of a multiple of 16 (fp32: 8) values that turn as a whole: no lane asks what it has
    if constexpr (V * sizeof(T) == 16)
      if (c.a.d == c.a.lanes * ITEMS * 2 * V && 2 * c.a.pairs == c.a.d) return go.template operator()<true>();
    return go.template operator()<false>();
  });
}

}  // namespace
}  // namespace fvx
