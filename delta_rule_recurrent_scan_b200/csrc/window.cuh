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
__host__ __device__ __forceinline__ int seq_len(const WindowArgs& p, int b) {
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
// rounded to bf16, or made from bf16 weights (``rounded``), is off by about 2^-9 |dO| |o|, the same for all keys of a row;
// against P (dP - delta) that is 1 / sqrt(n - 1) of what rounding dS costs for n keys of equal weight, so it shows where
// rows see few keys (the first rows of every sequence hold a third of the gradient's energy: 1.5 times the error of the
// rounded result instead of 1.4), and there the walk is short.  So: up to 256 keys of the window, in tiles of T, and no more
// than 128 sinks before them (a row behind those sees them all; backward of 2 sequences of 4096, 16 heads on 4, d 128,
// window 64, 2048 sinks: 464 us, 571 with sweeps over all the sinks' tiles).  And, whatever o is, for queries from t0 on
// among which one sees a single key: with its weight taken as 1 its delta is dP to the bit, and the gradient of a softmax
// over one key the zero that it is.
template <int T>
__host__ __device__ __forceinline__ bool exact_delta(const WindowArgs& p, const KeyTiles& k, int t0, bool rounded) {
  const bool few = (k.hi - k.lo) * T <= 256 && (k.sinks == 0 || p.n_sink <= 128);
  return (rounded && few) || t0 == 0 || (p.window == 1 && p.n_sink == 0);
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

// The keys' pass of the backward.  A CTA has a key tile and walks the query tiles that see it; walks that would be far
// longer than the rest, or too few for the SMs, are cut into parts, one CTA each, whose fp32 sums go to ``part`` and are
// added in order by a launch of their own.
//   - Key tiles that hold sinks are seen by every later query: where there are one or two of them they are cut into parts
//     of the other tiles' length.
//   - Where the tiles leave half of the SMs without a CTA every tile is cut, as far as SMs and items go.  Backward in all,
//     whole walks against cut ones: 1 x 8 heads on 2, 2048 tokens, d 128, window 512: 73 -> 45 us; 2 x 8 on 2, 1000 tokens:
//     92 -> 52; 2 x 16 on 2, 1500 tokens, d 64, 64 sinks: 141 -> 85; fp32, 1 x 2 on 1, 2048 tokens, window 128: 216 -> 57.
struct KeyPass {
  int sinks, parts;  // leading key tiles with a cut of their own, and into how many parts (0, 1: none)
  int others;        // parts of every other key tile
  float* part;       // one slot per CTA of a cut tile
  int tile, head;    // of this CTA (key_tile_of)
};
constexpr int kSms = 148;

inline long long key_ctas(const KeyPass& kp, long long heads, int tiles) {
  return heads * ((long long)kp.sinks * kp.parts + (long long)(tiles - kp.sinks) * kp.others);
}
inline int cut_tiles(const KeyPass& kp, int tiles) { return kp.others > 1 ? tiles : kp.sinks; }
inline long long cut_ctas(const KeyPass& kp, long long heads, int tiles) {
  return kp.others > 1 ? key_ctas(kp, heads, tiles) : heads * kp.sinks * kp.parts;
}

// Tiles of K keys walk tiles of Q queries; ``least``: items of a part where every tile is cut.
template <int K, int Q>
inline KeyPass key_pass(int B, int H, int Hkv, int L, int window, int n_sink, int least) {
  const int tiles = (L + K - 1) / K, walk = (L + Q - 1) / Q, G = H / Hkv;
  const int sinks = n_sink <= 0 ? 0 : n_sink < L ? (n_sink - 1) / K + 1 : tiles;
  const int regular = (window + K - 2) / Q + 2;    // query tiles that see a tile within the window
  const long long heads = (long long)B * Hkv, items = (long long)walk * G;
  const bool few_sinks = sinks > 0 && sinks <= 2 && sinks < tiles;
  // parts of a sink tile that make it as long as the other tiles' parts; not shorter than ``shortest``
  auto sink_parts = [&](int others, int shortest) {
    long long parts = ((long long)walk * others + regular - 1) / regular;
    if (parts > 64) parts = 64;
    if (parts > items / shortest) parts = items / shortest;
    return parts < 1 ? 1 : static_cast<int>(parts);
  };
  KeyPass kp{0, 1, 1, nullptr, 0, 0};
  if (few_sinks && sink_parts(1, 4) > 1)           // a part shorter than four tiles is all start-up
    kp.sinks = sinks, kp.parts = sink_parts(1, 4);
  const long long near = (long long)(regular < walk ? regular : walk) * G;
  long long most = heads > 0 && tiles > 0 ? kSms / (heads * tiles) : 0, longest = near > items / kp.parts ? near : items / kp.parts;
  if (sinks == 0) longest = near;
  if (most > near / least) most = near / least;
  for (int others = 2; others <= most; ++others) {  // the cut whose longest part is shortest
    KeyPass all{0, 1, others, nullptr, 0, 0};
    if (few_sinks) {
      const long long room = (kSms / heads - (long long)(tiles - sinks) * others) / sinks;
      const int wanted = sink_parts(others, least), parts = wanted < room ? wanted : static_cast<int>(room);
      if (parts > others) all.sinks = sinks, all.parts = parts;
    }
    const long long sink_part = sinks == 0 ? 0 : items / (all.sinks ? all.parts : others);
    const long long part = near / others > sink_part ? near / others : sink_part;
    if (part < longest) kp = all, longest = part;
  }
  return kp;
}
// Key tile and (sequence, k/v head) of CTA x: the sinks' tiles come first (theirs are the longest walks), then the others.
// Returns into how many parts the tile is cut; the CTA has part ``part``, whose slot in KeyPass::part is x.
__host__ __device__ __forceinline__ int key_tile_of(KeyPass& kp, int heads, int tiles, unsigned x, int& part) {
  const unsigned cut = (unsigned)heads * kp.sinks * kp.parts;
  if (x < cut) {
    part = x % kp.parts, x /= kp.parts;
    kp.tile = x % kp.sinks, kp.head = x / kp.sinks;
    return kp.parts;
  }
  x -= cut;
  part = x % kp.others, x /= kp.others;
  const int rest = tiles - kp.sinks;
  kp.tile = kp.sinks + x % rest, kp.head = x / rest;
  return kp.others;
}
// The parts of a cut tile: how many, and the first one's slot.
__host__ __device__ __forceinline__ int parts_of(const KeyPass& kp, int heads, int tiles, size_t head, int tile, size_t& slot) {
  if (tile < kp.sinks) {
    slot = (head * kp.sinks + tile) * kp.parts;
    return kp.parts;
  }
  slot = (size_t)heads * kp.sinks * kp.parts + (head * (tiles - kp.sinks) + (tile - kp.sinks)) * kp.others;
  return kp.others;
}

}  // namespace window
}  // namespace kdn
