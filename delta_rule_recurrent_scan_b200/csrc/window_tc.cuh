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

// Rows max(t0, len) .. t0 + 127 of a [.., L, D] array become zero (bytes per row a multiple of 16), by ``threads`` threads.
__device__ __forceinline__ void zero_tile(void* dst, size_t row0, int row_bytes, int t0, int len, int L, int tid, int threads) {
  const int first = max(t0, len), last = min(t0 + kT, L), words = row_bytes / 16;
  for (int e = tid; e < (last - first) * words; e += threads)
    static_cast<uint4*>(dst)[(row0 + first) * words + e] = make_uint4(0, 0, 0, 0);
}

// Bit e: whether a query ``back`` tokens behind the first of 32 keys sees the e-th of them; ``sinks`` of the keys are sinks.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }  // bits 0 .. n - 1
__device__ __forceinline__ uint32_t seen_bits(int back, int window, int sinks) {
  return below(back + 1) & (~below(back - window + 1) | below(sinks));
}

// Bit e: whether the e-th of 32 queries sees a key that lies ``ahead`` tokens behind the first of them (< 0: before it).
__device__ __forceinline__ uint32_t seeing_bits(int ahead, int window, bool sink) {
  return ~below(ahead) & (sink ? ~0u : below(ahead + window));
}

// One arrival for a warp, after all its lanes' work (32 single arrivals on one word take turns).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(bar);
}

// 32 bytes to global memory: whole sectors where the array is 32-byte aligned (``wide``; the interface asks for 16).
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
  } else {
    static_cast<uint4*>(p)[0] = a, static_cast<uint4*>(p)[1] = b;
  }
}
__device__ __forceinline__ bool is_wide(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// Division by a number known at launch: q = floor(x / d) for x < 2^31 (multiply by ceil(2^(32 + s) / d), s = ceil(log2 d)).
struct Divisor {
  unsigned d, mul, shift;
  __host__ __device__ __forceinline__ unsigned div(unsigned x, unsigned& rest) const {
#ifdef __CUDA_ARCH__
    const unsigned q = (__umulhi(x, mul) + x) >> shift;
#else
    const unsigned q = (static_cast<unsigned>((unsigned long long)x * mul >> 32) + x) >> shift;
#endif
    rest = x - q * d;
    return q;
  }
};
inline Divisor make_divisor(unsigned d) {
  Divisor v{d, 0, 0};
  while ((1ull << v.shift) < d) ++v.shift;
  v.mul = static_cast<unsigned>((((1ull << v.shift) - d) << 32) / d + 1);
  return v;
}

// The r-th of a call's works for this CTA: every other round runs backwards, so that long and short works meet.
__host__ __device__ __forceinline__ unsigned nth_work(unsigned r, unsigned cta, unsigned ctas) {
  return r * ctas + (r & 1 ? ctas - 1 - cta : cta);
}

// What a warp leaves in the rows that it cannot make any more because a wait gave up: NaN.  (Behind a sequence's end: zero,
// where the call asks for it.)  ``bytes`` from ``at`` on, both multiples of 4; NaN in either type is all ones but the sign.
__host__ __device__ __forceinline__ uint32_t nan_word(int dtype) { return dtype == kBF16 ? 0x7fff7fffu : 0x7fffffffu; }
__host__ __device__ __forceinline__ void fill_words(void* p, size_t at, int bytes, uint32_t word) {
  uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<char*>(p) + at);
  for (int e = 0; e < bytes / 4; ++e) to[e] = word;
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

// Descriptors of a tile of 128 rows: as a K-major operand (rows = M or N), and as the MN-major operand of a product over
// its rows.  A byte offset inside the tile is added to the address field (in 16-byte units), which it cannot overflow.
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile) { return sm100::smem_desc(tile, 16, 1024); }
__device__ __forceinline__ uint64_t cols_desc(uint32_t tile) { return sm100::smem_desc(tile, kPanel, 1024); }

// D[tmem] = A B^T over D coordinates: A and B tiles of 128 rows in shared memory (rows_desc).
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint64_t a, uint64_t b) {
  constexpr uint32_t id = sm100::idesc_bf16(128, kT, false, false);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint64_t off = ((ks / 4) * kPanel + (ks % 4) * 32) >> 4;
    sm100::mma_bf16(d_tmem, a + off, b + off, id, ks > 0);
  }
}

// D[tmem] (+)= W B: W 128 x 128 bf16 weights in TMEM (pair columns: the first 64 weights at w, the others at w + second),
// B a tile of 128 rows of D in shared memory (cols_desc).
template <int D>
__device__ __forceinline__ void mma_weights(uint32_t d_tmem, uint32_t w, uint32_t second, uint64_t b, bool accumulate) {
  constexpr uint32_t id = sm100::idesc_bf16(128, D, false, true);
#pragma unroll
  for (int ks = 0; ks < kT / 16; ++ks)
    sm100::mma_bf16_ts(d_tmem, w + 8 * (ks & 3) + (ks >= 4 ? second : 0u), b + (ks * 2048 >> 4), id, accumulate || ks > 0);
}

}  // namespace window
}  // namespace kdn
