// Shared pieces of the tensor-core windowed-attention kernels (forward and backward).
#pragma once

#include <cuda.h>

#include "chunk.h"
#include "chunk_common.cuh"
#include "sm100.cuh"
#include "window.cuh"

namespace kdn {
namespace window {

using chunk::kWaitCycles;

constexpr int kT = 128;              // queries and keys per tile
constexpr int kPanel = kT * 128;     // bytes of a swizzled panel: 128 rows of 64 bf16
constexpr int kTcThreads = 320;      // two warpgroups of row threads, one load warp, one product warp
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values times f as one 16-byte word of bf16.
__device__ __forceinline__ uint4 pack8_bf16(const float* x, float f) {
  return make_uint4(pack_bf16(x[0] * f, x[1] * f), pack_bf16(x[2] * f, x[3] * f), pack_bf16(x[4] * f, x[5] * f),
                    pack_bf16(x[6] * f, x[7] * f));
}

// A warp's wait: true when every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, sm100::mbar_wait_bounded(bar, parity, kWaitCycles));
}

// Rows ``first`` .. 127 of a tile of NP panels become zero (one warp), visible to the products that follow: what
// memory holds behind a sequence's end must not meet even a zero weight.
template <int NP>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int first, int lane) {
  const int words = (kT - first) * 8;
  for (int e = lane; e < words * NP; e += 32) {
    const int pn = e / words, w = e % words;
    *reinterpret_cast<uint4*>(tile + pn * kPanel + (first + w / 8) * 128 + (w % 8) * 16) = make_uint4(0, 0, 0, 0);
  }
  sm100::fence_async_smem();
  __syncwarp();
}

// One tile of 128 rows (rows t0 .., of array row ``row``) by TMA.
template <int NP>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int t0, int row) {
#pragma unroll
  for (int pn = 0; pn < NP; ++pn) sm100::tma_load_3d(dst + pn * kPanel, tm, bar, 64 * pn, t0, row);
}

// D[tmem] (+)= A B^T over D coordinates: A and B tiles of 128 rows in shared memory, both K-major.
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a, uint32_t b) {
  constexpr uint32_t id = sm100::idesc_bf16(128, kT, false, false);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t off = (ks / 4) * kPanel + (ks % 4) * 32;
    sm100::mma_bf16(d_tmem, sm100::smem_desc(a + off, 16, 1024), sm100::smem_desc(b + off, 16, 1024), id, ks > 0);
  }
}

// D[tmem] (+)= W B: W 128 x 128 bf16 weights in TMEM (pair columns: the first 64 weights at w, the others at w + second),
// B a tile of 128 rows of D in shared memory.
template <int D>
__device__ __forceinline__ void mma_weights(uint32_t d_tmem, uint32_t w, uint32_t second, uint32_t b, bool accumulate) {
  constexpr uint32_t id = sm100::idesc_bf16(128, D, false, true);
#pragma unroll
  for (int ks = 0; ks < kT / 16; ++ks)
    sm100::mma_bf16_ts(d_tmem, w + 8 * (ks & 3) + (ks >= 4 ? second : 0u), sm100::smem_desc(b + ks * 2048, kPanel, 1024), id,
                       accumulate || ks > 0);
}

}  // namespace window
}  // namespace kdn
