// Visibility and tile arithmetic shared by the windowed-attention kernels.
//
// Token t of a sequence of len tokens sees token j when j <= t and (j > t - window or j < n_sink).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace kdn {
namespace window {

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__host__ __device__ __forceinline__ bool visible(int t, int j, int window, int n_sink) {
  return j <= t && (t - j < window || j < n_sink);
}

// Tokens of sequence b: lens[b] held to [0, L], or L.
__device__ __forceinline__ int seq_len(const WindowArgs& p, int b) {
  if (p.lens == nullptr) return p.L;
  return min(max(p.lens[b], 0), p.L);
}

// Key tiles (of T tokens) that the queries t0 .. t1 of a sequence see: the sink tiles [0, sinks) and the window's
// tiles [lo, hi), with sinks <= lo.  walk(i) gives the i-th tile of the two runs joined.
struct KeyTiles {
  int sinks, lo, hi;
  __host__ __device__ __forceinline__ int count() const { return sinks + hi - lo; }
  __host__ __device__ __forceinline__ int walk(int i) const { return i < sinks ? i : lo + (i - sinks); }
};
template <int T>
__host__ __device__ __forceinline__ KeyTiles key_tiles(int t0, int t1, int window, int n_sink) {
  KeyTiles k;
  const int first = t0 - window + 1;
  k.lo = first > 0 ? first / T : 0;
  k.hi = t1 / T + 1;
  const int s = n_sink > 0 ? (n_sink - 1) / T + 1 : 0;
  k.sinks = s < k.lo ? s : k.lo;
  return k;
}

// Query tiles (of T tokens) of a sequence of len tokens that see a key of j0 .. j1: [lo, hi).
template <int T>
__host__ __device__ __forceinline__ void query_tiles(int j0, int j1, int len, int window, int n_sink, int& lo, int& hi) {
  const int last = len - 1;
  int t1 = last;                                                   // a sink: every later token
  if (j0 >= n_sink && window <= last - j1) t1 = j1 + window - 1;   // (no overflow: window is small here)
  lo = j0 / T;
  hi = t1 / T + 1;
}

}  // namespace window
}  // namespace kdn
