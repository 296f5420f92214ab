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

// Whether the backward makes these queries' delta from the weights instead of from o, in a sweep of its own.  dO . o with o
// rounded to bf16 is off by about 2^-9 |dO| |o|, the same for all keys of a row; against P (dP - delta) that is
// 1 / sqrt(n - 1) of what rounding dS costs for n keys of equal weight, so it shows where rows see few keys (the first
// rows of every sequence hold a third of the gradient's energy: 1.5 times the error of the rounded result instead of
// 1.4), and there the walk is short.  Up to 256 keys, in tiles of T; and, whatever o's type, for queries from t0 on among
// which one sees a single key: with its weight taken as 1 its delta is dP to the bit, and the gradient of a softmax over
// one key the zero that it is.
template <int T>
__device__ __forceinline__ bool exact_delta(const WindowArgs& p, const KeyTiles& k, int t0) {
  return (p.out_dtype == kBF16 && (k.hi - k.lo) * T <= 256) || t0 == 0 || (p.window == 1 && p.n_sink == 0);
}
__device__ __forceinline__ bool sees_one_key(const WindowArgs& p, int t) { return t == 0 || (p.window == 1 && p.n_sink == 0); }

// Query tiles (of T tokens) of a sequence of len tokens that see a key of j0 .. j1: [lo, hi).
template <int T>
__host__ __device__ __forceinline__ void query_tiles(int j0, int j1, int len, int window, int n_sink, int& lo, int& hi) {
  const int last = len - 1;
  int t1 = last;                                                   // a sink: every later token
  if (j0 >= n_sink && window <= last - j1) t1 = j1 + window - 1;   // (no overflow: window is small here)
  lo = j0 / T;
  hi = t1 / T + 1;
}

// The keys' pass of the backward.  The key tiles that hold sinks are seen by every later query; where there are one or two
// of them their walk is cut into parts of a regular tile's length, whose fp32 sums go to ``part`` and are added in order
// by a launch of their own.
struct KeyPass {
  int sinks, parts;  // key tiles that are cut, and into how many parts (0, 1: none)
  float* part;
  int tile, head;    // of this CTA (key_tile_of)
};
// Tiles of K keys walk tiles of Q queries.
template <int K, int Q>
inline KeyPass key_pass(int H, int Hkv, int L, int window, int n_sink) {
  const int tiles = (L + K - 1) / K, walk = (L + Q - 1) / Q;
  const int sinks = n_sink <= 0 ? 0 : n_sink < L ? (n_sink - 1) / K + 1 : tiles;
  KeyPass kp{0, 1, nullptr, 0, 0};
  if (sinks == 0 || sinks > 2 || sinks >= tiles) return kp;
  const int regular = (window + K - 2) / Q + 2;    // query tiles that see a tile within the window
  const long long items = (long long)walk * (H / Hkv);
  long long parts = (walk + regular - 1) / regular;
  if (parts > 64) parts = 64;
  if (parts > items / 4) parts = items / 4;        // a part shorter than four tiles is all start-up
  if (parts < 2) return kp;
  kp.sinks = sinks, kp.parts = static_cast<int>(parts);
  return kp;
}
// Key tile and (sequence, k/v head) of CTA x: the cut walks come first (they are the longest), then the other key tiles.
// True for a cut tile, whose part it is then.
__device__ __forceinline__ bool key_tile_of(KeyPass& kp, int heads, int tiles, unsigned x, int& part) {
  const unsigned cut = (unsigned)heads * kp.sinks * kp.parts;
  part = 0;
  if (x < cut) {
    part = x % kp.parts, x /= kp.parts;
    kp.tile = x % kp.sinks, kp.head = x / kp.sinks;
    return true;
  }
  x -= cut;
  const int rest = tiles - kp.sinks;
  kp.tile = kp.sinks + x % rest, kp.head = x / rest;
  return false;
}

}  // namespace window
}  // namespace kdn
