// Streaming row kernels, instantiated for one storage type per file (norm.cuh).
#pragma once
#include "norm.cuh"

namespace fvx {
namespace {

// Many aligned rows, dense or nearly so: a warp copies stages of rows to shared memory ahead
// of the eight that work on them.  Loads into registers keep at most a few
// vectors per thread under way, and the registers they need cost the warps that
// would hide them (4,000,000 x 64 bf16 backward: 297 us with one row in flight
// per lane, not 264, 307 with two, 461 with the next one fetched early); the copies are
// under way whatever the warps do.
// Blocks per multiprocessor: what the registers of a lane's values allow without
// spills (100,000 x 512 bf16, forward with codes: two 67 us, one 95; backward
// from codes: two, which spill, 106, one 80).
constexpr int kStreamThreads = kThreads + 32;
constexpr int kMostSmem = 227 * 1024;
struct StreamHead {
  uint64_t full[kStreamStages], empty[kStreamStages];
};
template <typename T, int VEC, int ITER, int OP, int LANES>
__global__ void __launch_bounds__(kStreamThreads, VEC * ITER > 16 || (VEC * ITER > 8 && OP == kBackwardCodes) ? 1 : VEC * ITER > 8 ? 2 : OpIs<OP>::kBack ? 3 : 4)
    k_rows_stream(const __grid_constant__ StreamArgs s) {
  using Is = OpIs<OP>;
  using X = std::conditional_t<Is::kFromCodes, int8_t, T>;
  extern __shared__ __align__(128) unsigned char sm[];
  StreamHead& h = *reinterpret_cast<StreamHead*>(sm);
  unsigned char* const ring = sm + 128;
  const RowArgs& a = s.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStreamStages; ++i) {
      tc::mbar_init(tc::smem_u32(&h.full[i]), 1);
      tc::mbar_init(tc::smem_u32(&h.empty[i]), kThreads / 32);
    }
    tc::mbar_init_fence();
  }
  __syncthreads();
  const int x_pitch = Is::kFromCodes ? a.c : (int)a.ldx, dy_pitch = (int)a.lddy;
  Rows<T, VEC, ITER, OP, LANES> rows(a);
  if (warp == kThreads / 32) {
    if (lane == 0) {
      uint32_t i = 0, phase = 1;
      int64_t k = 0;
      const uint32_t x_bytes = (uint32_t)(s.rows * x_pitch * sizeof(X)), dy_bytes = (uint32_t)(s.rows * dy_pitch * sizeof(T)),
                     step_bytes = (uint32_t)(s.rows * a.groups * 4), stat_bytes = (uint32_t)(s.rows * 4);
      uint32_t bytes = x_bytes;
      if constexpr (Is::kBack) bytes += dy_bytes;
      if constexpr (Is::kFromCodes) bytes += step_bytes;
      if constexpr (Is::kStats) bytes += 2 * stat_bytes;
      for (int64_t st = blockIdx.x; st < s.stages; st += gridDim.x, ++k) {
        if (k >= kStreamStages) tc::mbar_wait(tc::smem_u32(&h.empty[i]), phase, s.status);
        const uint32_t bar = tc::smem_u32(&h.full[i]), to = tc::smem_u32(ring) + i * (uint32_t)s.stage_bytes;
        const int64_t row = st * s.rows;
        tc::mbar_expect_tx(bar, bytes);
        if constexpr (Is::kFromCodes) {
          tc::bulk_load(to, a.codes + row * a.c, x_bytes, bar);
          tc::bulk_load(to + s.off_steps, a.steps + row * a.groups, step_bytes, bar);
        } else {
          tc::bulk_load(to, reinterpret_cast<const T*>(a.x) + row * x_pitch, x_bytes, bar);
        }
        if constexpr (Is::kBack)
          tc::bulk_load(to + s.off_dy, reinterpret_cast<const T*>(a.dy) + row * dy_pitch, dy_bytes, bar);
        if constexpr (Is::kStats) {
          tc::bulk_load(to + s.off_mean, a.mean_in + row, stat_bytes, bar);
          tc::bulk_load(to + s.off_rstd, a.rstd_in + row, stat_bytes, bar);
        }
        if (++i == kStreamStages) {
          i = 0;
          phase ^= 1u;
        }
      }
      // after a give-up, let the copies in flight land before the block exits
      for (int64_t x = k > kStreamStages ? k - kStreamStages : 0; x < k; ++x)
        tc::mbar_drain(tc::smem_u32(&h.full[x % kStreamStages]), (uint32_t)(x / kStreamStages) & 1u);
    }
    __syncwarp();
  } else {
    const int per_block = kThreads / LANES, sub = threadIdx.x / LANES;
    uint32_t i = 0, phase = 0;
    for (int64_t st = blockIdx.x; st < s.stages; st += gridDim.x) {
      const unsigned char* from = ring + i * (size_t)s.stage_bytes;
      tc::mbar_wait(tc::smem_u32(&h.full[i]), phase, s.status);
      __syncwarp();
      for (int r = sub; r < s.rows; r += per_block) {
        RowIn<T, VEC, ITER, OP> in;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
          const int v = k * rows.lanes + rows.lane;
          const bool here = v < rows.nv;
          in.x[k] = here ? raw_vec<X, VEC>(reinterpret_cast<const X*>(from) + r * x_pitch + v * VEC) : no_vec<X, VEC>();
          in.step[k] = 0.0f;
          if constexpr (Is::kFromCodes) {
            if (here)
              in.step[k] = reinterpret_cast<const float*>(from + s.off_steps)[r * a.groups + ((v * VEC) >> a.group_shift)];
          }
          if constexpr (Is::kBack)
            in.dy[k] = here ? raw_vec<T, VEC>(reinterpret_cast<const T*>(from + s.off_dy) + r * dy_pitch + v * VEC)
                            : no_vec<T, VEC>();
        }
        in.mean = in.rstd = 0.0f;
        if constexpr (Is::kStats) {
          in.mean = reinterpret_cast<const float*>(from + s.off_mean)[r];
          in.rstd = reinterpret_cast<const float*>(from + s.off_rstd)[r];
        }
        rows.turn(in, st * s.rows + r, true);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&h.empty[i]));
      if (++i == kStreamStages) {
        i = 0;
        phase ^= 1u;
      }
    }
    // the rows behind the last full stage
    if (blockIdx.x == (unsigned)(s.stages % gridDim.x)) rows.direct(s.stages * s.rows, per_block, a.n);
  }
  if constexpr (Is::kBack) rows.write_parts(reinterpret_cast<float*>(ring), kThreads);
}

template <typename T, int ITER, int OP, int LANES>
fvx_status launch_stream(const char* name, const StreamArgs& a, int blocks, size_t smem, cudaStream_t s) {
  auto kernel = k_rows_stream<T, 16 / sizeof(T), ITER, OP, LANES>;
  // The limit belongs to the kernel, not to the launch, and stages differ in
  // size: it is set once, to the most that a block may have, so that no thread
  // lowers it between another's check and launch.
  static std::atomic<uint64_t> allowed{0};
  FVX_TRY(allow_smem((const void*)kernel, kMostSmem, allowed));
  LaunchScope ls(name, s);
  kernel<<<blocks, kStreamThreads, smem, s>>>(a);
  return check_launch(name);
}
template <typename T, int OP>
fvx_status by_shape(const char* name, int iters, const StreamArgs& a, int blocks, size_t smem, cudaStream_t s) {
  if (iters > 2) return launch_stream<T, 16 / sizeof(T) == 8 ? 4 : 8, OP, 32>(name, a, blocks, smem, s);
  if constexpr (sizeof(T) == 2 && (OpIs<OP>::kNorm || OP == kBackward))
    if (iters == 2 && a.r.lanes == 16) return launch_stream<T, 2, OP, 16>(name, a, blocks, smem, s);
  if (iters == 2) return launch_stream<T, 2, OP, 32>(name, a, blocks, smem, s);
  switch (a.r.lanes) {
    case 1: return launch_stream<T, 1, OP, 1>(name, a, blocks, smem, s);
    case 2: return launch_stream<T, 1, OP, 2>(name, a, blocks, smem, s);
    case 4: return launch_stream<T, 1, OP, 4>(name, a, blocks, smem, s);
    case 8: return launch_stream<T, 1, OP, 8>(name, a, blocks, smem, s);
    case 16: return launch_stream<T, 1, OP, 16>(name, a, blocks, smem, s);
    default: return launch_stream<T, 1, OP, 32>(name, a, blocks, smem, s);
  }
}
template <typename T>
fvx_status stream_rows(const char* name, RowOp op, int iters, const StreamArgs& a, int blocks, size_t smem,
                       cudaStream_t s) {
  switch (op) {
    case kForward: return by_shape<T, kForward>(name, iters, a, blocks, smem, s);
    case kForwardCodes: return by_shape<T, kForwardCodes>(name, iters, a, blocks, smem, s);
    case kPack: return by_shape<T, kPack>(name, iters, a, blocks, smem, s);
    case kBackward: return by_shape<T, kBackward>(name, iters, a, blocks, smem, s);
    case kBackwardCodes: return by_shape<T, kBackwardCodes>(name, iters, a, blocks, smem, s);
    case kRestore: return by_shape<T, kRestore>(name, iters, a, blocks, smem, s);
    case kRestoreNorm: return by_shape<T, kRestoreNorm>(name, iters, a, blocks, smem, s);
  }
  return FVX_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace fvx
