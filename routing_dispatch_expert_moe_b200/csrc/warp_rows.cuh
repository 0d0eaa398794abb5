// A warp's rows of fp32, brought into shared memory one ahead: two buffers per warp, filled by
// bulk copies of whole rows (a multiple of 16 bytes, 16-byte aligned) that lane 0 issues, so that
// the next row's latency passes under the work on this one and costs no registers.  Every wait is
// bounded (MOE_DEVERR_PIPE_TIMEOUT).
#pragma once

#include "common.cuh"
#include "tc_prims.cuh"

namespace moe {
namespace {

struct WarpRows {
  uint32_t bar, buf;          // this warp's two mbarriers and two buffers (shared addresses)
  uint8_t* mem;               // the buffers again
  uint32_t bytes;             // of a row; also the buffers' pitch

  __device__ __forceinline__ void init(uint64_t* bars, uint8_t* buffers, uint32_t row_bytes, int lane) {
    bar = smem_u32(bars);
    buf = smem_u32(buffers);
    mem = buffers;
    bytes = row_bytes;
    if (lane == 0) {
      mbar_init(bar, 1);
      mbar_init(bar + 8, 1);
      fence_mbar_init();
    }
    __syncwarp();
  }
  // Lane 0: row number i (0, 1, ...) of the warp from src.
  __device__ __forceinline__ void load(unsigned i, const float* src) const {
    const uint32_t b = bar + 8 * (i & 1u), dst = buf + (i & 1u) * bytes;
    mbar_expect_tx(b, bytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(b)
                 : "memory");
  }
  __device__ __forceinline__ float* row(unsigned i) const { return reinterpret_cast<float*>(mem + (i & 1u) * bytes); }
  // The whole warp: false for every lane when the row did not come in time.
  __device__ __forceinline__ bool wait(unsigned i, volatile int* abort_flag, int* err) const {
    const bool got = mbar_wait(bar + 8 * (i & 1u), (i >> 1) & 1u, abort_flag, err);
    return __all_sync(0xffffffffu, got);
  }
  // Lane 0, before leaving early: rows [i, loaded) land first.
  __device__ __forceinline__ void drain(unsigned i, unsigned loaded, int* err) const {
    for (; i < loaded; ++i) mbar_wait_drain(bar + 8 * (i & 1u), (i >> 1) & 1u, err);
  }
};

}  // namespace
}  // namespace moe
