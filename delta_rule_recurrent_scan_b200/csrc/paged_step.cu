// One new token per sequence against its paged key-value cache: o = sum_j softmax_j(scale q . k_j) v_j over the tokens
// j < len that its window (or the first n_sink) leaves visible; the new token itself is the last of them.
//
// A sequence's visible tokens are cut into ``splits`` parts, one CTA each, which keep their own running maximum m, sum
// l = sum exp(s - m) and o = sum exp(s - m) v; with more than one part a second launch joins them in the order of the
// parts: M = max m_i, o = sum exp(m_i - M) o_i / sum exp(m_i - M) l_i.
//
// A table entry that names no page of the pool is not followed: the sequence's l becomes NaN, and with it its o and lse.
#include <climits>
#include <type_traits>

#include "sm100.cuh"
#include "window.cuh"

namespace kdn {

namespace {

using window::KeyTiles;

struct Part {
  int b, kvh, h0, nh, split;  // sequence, k/v head, first query head and how many of them, part
};

// blockIdx.x = ((sequence, k/v head, block of query heads), part), parts fastest.
template <int HB>
__device__ __forceinline__ Part which(const PagedStepArgs& p) {
  const int G = p.H / p.Hkv, hb = (G + HB - 1) / HB;
  unsigned x = blockIdx.x;
  Part w;
  w.split = x % p.splits, x /= p.splits;
  const int c = x % hb;
  x /= hb;
  w.kvh = x % p.Hkv, w.b = x / p.Hkv;
  w.h0 = w.kvh * G + c * HB;
  w.nh = min(HB, G - c * HB);
  return w;
}

__device__ __forceinline__ size_t part_at(const PagedStepArgs& p, int b, int h, int split) {
  return ((size_t)b * p.H + h) * p.splits + split;
}
__device__ __forceinline__ float* part_max(const PagedStepArgs& p, int dv) { return p.part + (size_t)p.n * p.H * p.splits * dv; }
__device__ __forceinline__ float* part_sum(const PagedStepArgs& p, int dv) {
  return part_max(p, dv) + (size_t)p.n * p.H * p.splits;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------------------------------ fp32 CUDA cores
// Every size and type, kHB = 8, 4 or 2 query heads per CTA.  Each of 4 warps walks units of 8 or 16 tokens with its own running maximum,
// sum and o.  A lane holds 4 coordinates: d / 4 lanes read a token's key as one run of 16-byte words, 128 / d tokens at a
// time, straight into registers; the next unit's keys are in flight while this one's values are used.
//   scores:  4 multiply-adds per lane, token and head, then an exchange over the lanes of a token that halves the number
//            of values with every step, so that 8 tokens cost 9 shuffles per head (40 one by one), leaving a lane with one
//            token's scores;
//   weights: the maxima move only when some score has outgrown them by 2^8 (one vote per unit); the 8 heads' weights go
//            through 16 or 32 bytes of the warp's own shared memory per token;
//   values:  o[8][4] += weight x value, the weights as broadcast reads.
// About 110 instructions per token and warp against 1 KB of fp32 keys and values (d = 128).
constexpr int kWarps = 4, kThr = 32 * kWarps;
constexpr float kSlack = 8.f;  // growth of a maximum (base 2) that weights may keep

// Four coordinates of a key or value.
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  float4 x;
  __device__ __forceinline__ void zero() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) { x = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ float4 get() const { return x; }
};
template <>
struct Quad<__nv_bfloat16> {
  uint2 x;
  __device__ __forceinline__ void zero() { x = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
  }
};

// Sums of N values over LANES neighbouring lanes, halving their number with every step while there are several: lane l is
// left with the sum of value ``index``.
template <int N, int LANES>
__device__ __forceinline__ float fold(float (&x)[N], int lane, int& index) {
  index = 0;
  int n = N;
#pragma unroll
  for (int k = LANES / 2; k >= 1; k >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & k) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i >= n) break;
        const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, k);
      }
      index += up ? n : 0;
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], k);
    }
  }
  return x[0];
}

template <int DK, int DV, int kHB, typename T>
__global__ void __launch_bounds__(kThr, 2) paged_step_kernel(PagedStepArgs p) {
  constexpr int kU = (DK > DV ? DK : DV) > 64 ? 8 : 16;       // tokens of a unit
  constexpr int kKL = DK / 4, kVL = DV / 4;                   // lanes of a key, of a value
  constexpr int kKT = 32 / kKL, kVT = 32 / kVL;               // tokens read at a time
  constexpr int kKN = kU / kKT > 0 ? kU / kKT : 1, kVN = kU / kVT > 0 ? kU / kVT : 1;
  static_assert(kKN * kKT >= kU && kVN * kVT >= kU, "a unit is covered");
  __shared__ __align__(16) float p_s[kWarps][kKN * kKT > kVN * kVT ? kKN * kKT : kVN * kVT][kHB];
  __shared__ __align__(16) float o_s[kWarps][kHB][DV];
  __shared__ float l_s[kWarps][kHB], m_s[kWarps][kHB];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Part w = which<kHB>(p);
  if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = p.row ? p.row[w.b] : w.b;
  int n = 0;
  const int* entries = nullptr;
  bool bad = r < 0 || r >= p.rows;
  if (!bad) {
    n = static_cast<int>(min((long long)max(p.lens[r], 0), (long long)p.max_pages * p.page_size));
    entries = p.table + (size_t)r * p.max_pages;
  }
  const int win = p.window > 0 ? p.window : INT_MAX;
  KeyTiles kt{0, 0, 0};
  if (n > 0) kt = window::key_tiles<kU>(n - 1, n - 1, win, p.n_sink);
  const int u0 = (int)((long long)kt.count() * w.split / p.splits) + warp;
  const int u1 = (int)((long long)kt.count() * (w.split + 1) / p.splits);
  const T* kp = static_cast<const T*>(p.k_pages);
  const T* vp = static_cast<const T*>(p.v_pages);
  const int shift = 31 - __clz(p.page_size), mask = p.page_size - 1;

  // a visible token's place in the pages, in tokens; -1: not to be read
  auto place = [&](int j) -> long long {
    if (j >= n || !window::visible(n - 1, j, win, p.n_sink)) return -1;
    const int page = entries[j >> shift];
    if (page < 0 || page >= p.num_pages) {
      bad = true;
      return -1;
    }
    return (((long long)page * p.Hkv + w.kvh) << shift) + (j & mask);
  };
  Quad<T> kq[kKN], vq[kVN];
  // A unit that lies in one page and is seen whole: its page was looked up a step ahead, its addresses differ by constants.
  const bool one_page = p.page_size >= kU;
  auto look = [&](int u) { return u < u1 && one_page ? entries[(kt.walk(u) * kU) >> shift] : 0; };
  auto whole = [&](int j0) { return one_page && j0 + kU <= n && (n - 1 - j0 < win || j0 + kU <= p.n_sink); };
  auto load = [&](auto& buf, const T* pool, int u, int entry, auto dim) {
    constexpr int D = decltype(dim)::value, L = D / 4, TK = 32 / L, N = kU / TK > 0 ? kU / TK : 1;
    const int j0 = u < u1 ? kt.walk(u) * kU : 0, col = 4 * (lane % L);
    if (u < u1 && whole(j0)) {
      const bool there = entry >= 0 && entry < p.num_pages;
      bad |= !there;
      const T* at = pool + ((((size_t)entry * p.Hkv + w.kvh) << shift) + (j0 & mask) + lane / L) * D + col;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (there && i * TK + lane / L < kU) buf[i].load(at + i * TK * D);
        else buf[i].zero();
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = i * TK + lane / L;
      const long long at = u < u1 && t < kU ? place(j0 + t) : -1;
      if (at >= 0) buf[i].load(pool + at * D + col);
      else buf[i].zero();
    }
  };
  auto load_k = [&](int u, int entry) { load(kq, kp, u, entry, std::integral_constant<int, DK>()); };
  auto load_v = [&](int u, int entry) { load(vq, vp, u, entry, std::integral_constant<int, DV>()); };

  int entry = look(u0), next = look(u0 + kWarps);
  load_k(u0, entry);
  float4 q[kHB];
#pragma unroll
  for (int h = 0; h < kHB; ++h) {
    Quad<T> x;
    x.zero();
    if (h < w.nh) x.load(static_cast<const T*>(p.q) + ((size_t)w.b * p.H + w.h0 + h) * DK + 4 * (lane % kKL));
    q[h] = x.get();
  }
  const float c = p.scale * kLog2e;
  float m[kHB], l[kHB];  // base 2; l: this lane's tokens
  float4 acc[kHB];
#pragma unroll
  for (int h = 0; h < kHB; ++h) m[h] = -INFINITY, l[h] = 0.f, acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int u = u0; u < u1; u += kWarps) {
    load_v(u, entry);
    float s[kHB];
    int index = 0;
#pragma unroll
    for (int h = 0; h < kHB; ++h) {
      float x[kKN];
#pragma unroll
      for (int i = 0; i < kKN; ++i) {
        const float4 k = kq[i].get();
        x[i] = fmaf(k.w, q[h].w, fmaf(k.z, q[h].z, fmaf(k.y, q[h].y, k.x * q[h].x)));
      }
      s[h] = fold<kKN, kKL>(x, lane, index) * c;
    }
    load_k(u + kWarps, next);
    entry = next, next = look(u + 2 * kWarps);
    const int t = index * kKT + lane / kKL, j = kt.walk(u) * kU + t;  // this lane's token (shared by lanes of a fold)
    const bool seen = t < kU && j < n && window::visible(n - 1, j, win, p.n_sink);
    bool grown = false;
#pragma unroll
    for (int h = 0; h < kHB; ++h) {
      if (!seen) s[h] = -INFINITY;
      grown |= s[h] > m[h] + kSlack || (m[h] == -INFINITY && s[h] > -INFINITY);
    }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int h = 0; h < kHB; ++h) {
        float top = s[h];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmaxf(top, m[h]);
        const float keep = m[h] == -INFINITY ? 0.f : exp2_fast(m[h] - top);
        l[h] *= keep;
        acc[h].x *= keep, acc[h].y *= keep, acc[h].z *= keep, acc[h].w *= keep;
        m[h] = top;
      }
    }
    // lanes that share a token write it once
    const bool mine = (lane & (kKN >= kKL ? 0 : kKL / kKN - 1)) == 0;
    float e[kHB];
#pragma unroll
    for (int h = 0; h < kHB; ++h) {
      e[h] = seen ? exp2_fast(s[h] - m[h]) : 0.f;
      if (mine) l[h] += e[h];
    }
    __syncwarp();
    if (mine) {
#pragma unroll
      for (int h = 0; h < kHB; h += 2) *reinterpret_cast<float2*>(&p_s[warp][t][h]) = make_float2(e[h], e[h + 1]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kVN; ++i) {
      const int tv = i * kVT + lane / kVL;
      const float4 v = vq[i].get();
      float pw[kHB];
      if constexpr (kHB >= 4) {
#pragma unroll
        for (int h = 0; h < kHB; h += 4) {
          const float4 a = *reinterpret_cast<const float4*>(&p_s[warp][tv][h]);
          pw[h] = a.x, pw[h + 1] = a.y, pw[h + 2] = a.z, pw[h + 3] = a.w;
        }
      } else {
        const float2 a = *reinterpret_cast<const float2*>(&p_s[warp][tv][0]);
        pw[0] = a.x, pw[1] = a.y;
      }
#pragma unroll
      for (int h = 0; h < kHB; ++h) {
        acc[h].x = fmaf(pw[h], v.x, acc[h].x), acc[h].y = fmaf(pw[h], v.y, acc[h].y);
        acc[h].z = fmaf(pw[h], v.z, acc[h].z), acc[h].w = fmaf(pw[h], v.w, acc[h].w);
      }
    }
  }
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int h = 0; h < kHB; ++h) {
    l[h] = warp_sum(l[h]);
    float4 x = acc[h];
#pragma unroll
    for (int o = kVL; o < 32; o <<= 1) {  // the lane groups that read other tokens
      x.x += __shfl_xor_sync(0xffffffffu, x.x, o), x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
      x.z += __shfl_xor_sync(0xffffffffu, x.z, o), x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
    }
    if (lane < kVL) *reinterpret_cast<float4*>(&o_s[warp][h][4 * lane]) = x;
    if (lane == 0) m_s[warp][h] = m[h], l_s[warp][h] = bad ? NAN : l[h];
  }
  __syncthreads();
  for (int e = tid; e < w.nh * DV; e += kThr) {
    const int h = e / DV, col = e % DV;
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) M = fmaxf(M, m_s[i][h]);
    const float base = M == -INFINITY ? 0.f : M;
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float f = exp2_fast(m_s[i][h] - base);
      sum = fmaf(f, l_s[i][h], sum);
      x = fmaf(f, o_s[i][h][col], x);
    }
    const size_t head = (size_t)w.b * p.H + w.h0 + h;
    if (p.splits == 1) {
      store_elem(p.o, head * DV + col, sum == 0.f ? 0.f : x / sum, p.out_dtype);  // nothing visible: zero
      if (col == 0 && p.lse) p.lse[head] = M * kLn2 + logf(sum);
    } else {
      const size_t at = part_at(p, w.b, w.h0 + h, w.split);
      p.part[at * DV + col] = x;
      if (col == 0) part_max(p, DV)[at] = M * kLn2, part_sum(p, DV)[at] = sum;
    }
  }
}

// ------------------------------------------------------------------------------------------ bf16, warp matrix products
// d_k = d_v = 64 or 128.  The step reads every visible key and value once and does two multiply-adds per element and
// query head, so it is bound by memory; products on whole 128-row tensor-core tiles would be nearly all padding (a k/v
// head has 1 to 16 query heads), the warp's m16 n8 k16 product fits: rows = query heads, columns = tokens, then columns
// = d_v.  Each of 4 warps walks units of 16 tokens with a pipeline of its own (cp.async into kStages swizzled stages,
// no CTA barrier) and its own running maximum, sum and o; the warps are joined through shared memory at the end.
//
// The weights enter the second product as bf16 hi + lo (2^-16 of a weight): with up to 8 query heads the 16 rows hold
// every head twice, rows 0-7 taking hi and rows 8-15 lo, so the pair costs nothing; with 9 to 16 heads two products.
constexpr int kMT = 16, kMWarps = 4, kStages = 3, kMHB = 16;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes, or zeros where !there.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int D>
struct StepSmem {
  static constexpr int kTile = kMT * D * 2;            // 16 tokens of k or of v
  static constexpr int kWarp = kStages * 2 * kTile;
  static constexpr int kTotal = kMWarps * kWarp;
  static_assert(kMWarps * kMHB * D * 4 <= kTotal, "the warps' o are joined in the same memory");
};

template <int D, bool TWICE>
__global__ void __launch_bounds__(32 * kMWarps) paged_step_mma_kernel(PagedStepArgs p, int shift) {
  using Sm = StepSmem<D>;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ float m_s[kMWarps][kMHB], l_s[kMWarps][kMHB];
  constexpr int kChunks = D / 8;                       // 16-byte words of a row
  constexpr int kRows = 32 / kChunks;                  // rows a warp copies at once
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const Part w = which<kMHB>(p);
  if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = p.row ? p.row[w.b] : w.b;
  int n = 0;
  const int* entries = nullptr;
  bool bad = r < 0 || r >= p.rows;
  if (!bad) {
    n = static_cast<int>(min((long long)max(p.lens[r], 0), (long long)p.max_pages << shift));
    entries = p.table + (size_t)r * p.max_pages;
  }
  const int win = p.window > 0 ? p.window : INT_MAX;
  KeyTiles kt{0, 0, 0};
  if (n > 0) kt = window::key_tiles<kMT>(n - 1, n - 1, win, p.n_sink);
  const int u0 = (int)((long long)kt.count() * w.split / p.splits) + warp;
  const int u1 = (int)((long long)kt.count() * (w.split + 1) / p.splits);

  // this lane's rows of the units it copies
  const int chunk = lane % kChunks, row0 = lane / kChunks;
  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(sm)) + warp * Sm::kWarp;
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.k_pages);
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.v_pages);
  const int mask = p.page_size - 1;
  const bool one_page = p.page_size >= kMT;            // a unit lies in one page
  // the page of a unit's first token, looked up a step ahead of its copies
  auto look = [&](int u) { return u < u1 && one_page ? entries[(kt.walk(u) * kMT) >> shift] : 0; };
  auto issue = [&](int u, int stage, int entry) {
    if (u < u1) {
      const int j0 = kt.walk(u) * kMT;
      const uint32_t dst = stage0 + stage * 2 * Sm::kTile;
      const bool full = j0 + kMT <= n && (n - 1 - j0 < win || j0 + kMT <= p.n_sink);
      if (full && one_page) {  // one page, every token: the addresses differ by constants
        const bool there = entry >= 0 && entry < p.num_pages;
        bad |= !there;
        const size_t at = there ? ((((size_t)entry * p.Hkv + w.kvh) << shift) + (j0 & mask) + row0) * D + 8 * chunk : 0;
#pragma unroll
        for (int i = 0; i < kMT / kRows; ++i) {
          const int row = row0 + i * kRows;
          const uint32_t to = dst + row * (D * 2) + ((chunk ^ (row & 7)) << 4);
          copy16_or_zero(to, kp + at + i * kRows * D, there);
          copy16_or_zero(to + Sm::kTile, vp + at + i * kRows * D, there);
        }
      } else {
#pragma unroll
      for (int i = 0; i < kMT / kRows; ++i) {
        const int row = row0 + i * kRows, j = j0 + row;
        bool there = full || (j < n && window::visible(n - 1, j, win, p.n_sink));
        const int page = one_page ? entry : (there ? entries[j >> shift] : 0);
        if (there && (page < 0 || page >= p.num_pages)) bad = true, there = false;
        const size_t at = there ? ((((size_t)page * p.Hkv + w.kvh) << shift) + (j & mask)) * D + 8 * chunk : 0;
        const uint32_t to = dst + row * (D * 2) + ((chunk ^ (row & 7)) << 4);
        copy16_or_zero(to, kp + at, there);
        copy16_or_zero(to + Sm::kTile, vp + at, there);
      }
      }
    }
    async_commit();
  };
  int entry = look(u0);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    const int next = look(u0 + (i + 1) * kMWarps);
    issue(u0 + i * kMWarps, i, entry);
    entry = next;
  }

  // q as the first product's A operand
  uint32_t q[D / 16][4];
  {
    const uint32_t* qp = reinterpret_cast<const uint32_t*>(p.q) + ((size_t)w.b * p.H + w.h0) * (D / 2);
    const int ra = g, rb = TWICE ? g : g + 8;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      q[ks][0] = ra < w.nh ? qp[ra * (D / 2) + 8 * ks + t4] : 0u;
      q[ks][1] = rb < w.nh ? qp[rb * (D / 2) + 8 * ks + t4] : 0u;
      q[ks][2] = ra < w.nh ? qp[ra * (D / 2) + 8 * ks + t4 + 4] : 0u;
      q[ks][3] = rb < w.nh ? qp[rb * (D / 2) + 8 * ks + t4 + 4] : 0u;
    }
  }
  const float c2 = p.scale * kLog2e;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g and g + 8 (base 2); l of this lane's tokens
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  int stage = 0;
  for (int u = u0; u < u1; u += kMWarps) {
    async_wait<kStages - 2>();
    __syncwarp();
    {  // the stage read last is free for all lanes: its copies go out first
      const int ahead = u + (kStages - 1) * kMWarps;
      const int next = look(ahead + kMWarps);
      issue(ahead, stage == 0 ? kStages - 1 : stage - 1, entry);
      entry = next;
    }
    const uint32_t k_at = stage0 + stage * 2 * Sm::kTile, v_at = k_at + Sm::kTile;
    float s[2][4] = {}, s2[2][4] = {};  // two chains of products each
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const int row = ((lane >> 4) << 3) + (lane & 7), c = 2 * ks + ((lane >> 3) & 1);
      uint32_t b[4];
      ldsm4(b, k_at + row * (D * 2) + ((c ^ (row & 7)) << 4));
      mma16816(ks & 1 ? s2[0] : s[0], q[ks], b[0], b[1]);
      mma16816(ks & 1 ? s2[1] : s[1], q[ks], b[2], b[3]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] += s2[i][e];
    const int j0 = kt.walk(u) * kMT;
    if (!(j0 + kMT <= n && (n - 1 - j0 < win || j0 + kMT <= p.n_sink))) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + 8 * i + 2 * t4 + (e & 1);
          if (j >= n || !window::visible(n - 1, j, win, p.n_sink)) s[i][e] = -INFINITY;
        }
    }
    float base[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1])) * c2;
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = fmaxf(top, m[i]);
      base[i] = top == -INFINITY ? 0.f : top;
      const float keep = exp2_fast(m[i] - base[i]);
      if (__any_sync(0xffffffffu, top != m[i])) {
        l[i] *= keep;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) o[d][2 * i] *= keep, o[d][2 * i + 1] *= keep;
      }
      m[i] = top;
    }
    uint32_t hi[4], lo[4];  // P as the second product's A operand: (row g, row g + 8) x (tokens 0-7, 8-15)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = exp2_fast(fmaf(s[i][2 * h], c2, -base[h])), b = exp2_fast(fmaf(s[i][2 * h + 1], c2, -base[h]));
        l[h] += a + b;
        sm100::split2_bf16(a, b, hi[2 * i + h], lo[2 * i + h]);
      }
    if constexpr (TWICE) hi[1] = lo[1], hi[3] = lo[3];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const int row = (((lane >> 3) & 1) << 3) + (lane & 7), c = 2 * d + (lane >> 4);
      uint32_t b[4];
      ldsm4_t(b, v_at + row * (D * 2) + ((c ^ (row & 7)) << 4));
      mma16816(o[2 * d], hi, b[0], b[1]);
      mma16816(o[2 * d + 1], hi, b[2], b[3]);
      if constexpr (!TWICE) {
        mma16816(o[2 * d], lo, b[0], b[1]);
        mma16816(o[2 * d + 1], lo, b[2], b[3]);
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  bad = __syncthreads_or(bad);  // every warp has read its last stage
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (t4 == 0) m_s[warp][g + 8 * i] = m[i], l_s[warp][g + 8 * i] = bad ? NAN : l[i];
  }
  float* o_s = reinterpret_cast<float*>(sm);  // [warp][row][D]
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(o_s + ((size_t)warp * kMHB + g + 8 * i) * D + 8 * d + 2 * t4) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
  __syncthreads();
  for (int e = tid; e < w.nh * D; e += 32 * kMWarps) {
    const int h = e / D, col = e % D;
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMWarps; ++i) M = fmaxf(M, m_s[i][h]);
    const float b = M == -INFINITY ? 0.f : M;
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int i = 0; i < kMWarps; ++i) {
      const float f = exp2_fast(m_s[i][h] - b);
      float v = o_s[(i * kMHB + h) * D + col];
      if constexpr (TWICE) v += o_s[(i * kMHB + h + 8) * D + col];
      sum = fmaf(f, l_s[i][h], sum);
      x = fmaf(f, v, x);
    }
    const size_t head = (size_t)w.b * p.H + w.h0 + h;
    if (p.splits == 1) {
      store_elem(p.o, head * D + col, sum == 0.f ? 0.f : x / sum, p.out_dtype);
      if (col == 0 && p.lse) p.lse[head] = M * kLn2 + logf(sum);
    } else {
      const size_t at = part_at(p, w.b, w.h0 + h, w.split);
      p.part[at * D + col] = x;
      if (col == 0) part_max(p, D)[at] = M * kLn2, part_sum(p, D)[at] = sum;
    }
  }
}

// Joins a head's parts: one CTA per head.  The parts' factors exp(m_i - M) are made once, in shared memory; then 256 / (d_v / 4)
// groups of threads add every group-th part, four columns a thread, and the groups are added in order.
constexpr int kJoin = 256, kMaxParts = 1024;
template <int DV>
__global__ void __launch_bounds__(kJoin) paged_join_kernel(PagedStepArgs p) {
  constexpr int kCols = DV / 4, kGroups = kJoin / kCols;
  __shared__ float f_s[kMaxParts], red[8];
  __shared__ __align__(16) float4 o_s[kJoin];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t head = blockIdx.x;
  const float* pm = part_max(p, DV) + head * p.splits;
  const float* pl = part_sum(p, DV) + head * p.splits;
  const float4* po = reinterpret_cast<const float4*>(p.part + head * p.splits * DV);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the parts are still being made
  float M = -INFINITY;
  for (int i = tid; i < p.splits; i += kJoin) M = fmaxf(M, pm[i]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (lane == 0) red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoin / 32; ++i) M = fmaxf(M, red[i]);
  __syncthreads();
  const float base = M == -INFINITY ? 0.f : M;
  float l = 0.f;
  for (int i = tid; i < p.splits; i += kJoin) {
    const float f = expf(pm[i] - base);
    f_s[i] = f;
    l = fmaf(f, pl[i], l);
  }
  l = warp_sum(l);
  if (lane == 0) red[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kJoin / 32; ++i) l += red[i];
  const int col = tid % kCols, group = tid / kCols;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = group; i < p.splits; i += kGroups) {
    const float4 v = po[(size_t)i * kCols + col];
    const float f = f_s[i];
    a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
  }
  o_s[tid] = a;
  __syncthreads();
  if (tid < DV) {
    float x = 0.f;
    for (int g = 0; g < kGroups; ++g) x += reinterpret_cast<const float*>(o_s)[g * DV + tid];
    store_elem(p.o, head * DV + tid, l == 0.f ? 0.f : x / l, p.out_dtype);
    if (tid == 0 && p.lse) p.lse[head] = M + logf(l);
  }
}

// The join's launch overlaps the end of the kernel before it (its wait is at its top).
template <int DV>
cudaError_t join(const PagedStepArgs& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n * p.H), cfg.blockDim = dim3(kJoin), cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<DV>, p);
}

// Query heads per CTA of the fp32 kernel.
int head_block(int G, int in_dtype) { return in_dtype == kBF16 || G > 4 ? 8 : G > 2 ? 4 : 2; }

template <int DK, int DV>
cudaError_t step(const PagedStepArgs& p, cudaStream_t stream) {
  const int G = p.H / p.Hkv, hb = head_block(G, p.in_dtype);
  const unsigned ctas = (unsigned)((long long)p.n * p.Hkv * ((G + hb - 1) / hb) * p.splits);
  if (p.in_dtype == kBF16) paged_step_kernel<DK, DV, 8, __nv_bfloat16><<<ctas, kThr, 0, stream>>>(p);
  else if (hb == 8) paged_step_kernel<DK, DV, 8, float><<<ctas, kThr, 0, stream>>>(p);
  else if (hb == 4) paged_step_kernel<DK, DV, 4, float><<<ctas, kThr, 0, stream>>>(p);
  else paged_step_kernel<DK, DV, 2, float><<<ctas, kThr, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  return join<DV>(p, stream);
}

bool step_mma_supported(int dk, int dv, int in_dtype) { return in_dtype == kBF16 && dk == dv && (dk == 64 || dk == 128); }

template <int D>
cudaError_t step_mma(const PagedStepArgs& p, cudaStream_t stream) {
  const int G = p.H / p.Hkv;
  const long long ctas = (long long)p.n * p.Hkv * ((G + kMHB - 1) / kMHB) * p.splits;
  int shift = 0;
  while ((1 << shift) < p.page_size) ++shift;
  const auto kernel = G <= 8 ? paged_step_mma_kernel<D, true> : paged_step_mma_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, StepSmem<D>::kTotal);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)ctas, 32 * kMWarps, StepSmem<D>::kTotal, stream>>>(p, shift);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  return join<D>(p, stream);
}

template <typename F>
cudaError_t for_dim(int d, F f) {
  switch (d) {
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int paged_step_splits(int dk, int dv, int in_dtype, int n, int H, int Hkv, long long most_tokens) {
  const int G = H / Hkv;
  // Two CTAs fit an SM.  One wave of parts of at least 128 tokens (below that a part is all start-up); for several
  // sequences, whose lengths differ, up to six waves of parts of at least 512 tokens, which even out.  Measured, 16
  // sequences of up to 16000 tokens on 4 heads, fp32: 111 us, one wave 154 us; 32 of up to 2000 on 8 heads, bf16: 40 us
  // with parts of 512 tokens, 50 us with 285; 64 of up to 8192 on 8 heads: 164 us with six waves, 173 us with three (three
  // CTAs per SM instead of two: 169 us against 165).
  const int hb = step_mma_supported(dk, dv, in_dtype) ? kMHB : head_block(G, in_dtype);
  const long long pairs = (long long)n * Hkv * ((G + hb - 1) / hb), slots = 2 * 148;
  const auto least = [](long long a, long long b) { return a < b ? a : b; };
  long long s = least(slots / pairs, most_tokens / 128);
  if (n > 1) {
    const long long waves = least((6 * slots + pairs - 1) / pairs, most_tokens / 512);
    if (waves > s) s = waves;
  }
  if (s > kMaxParts) s = kMaxParts;
  return s < 1 ? 1 : (int)s;
}

size_t paged_step_part_floats(int dv, int n, int H, int splits) {
  return splits > 1 ? (size_t)n * H * splits * (dv + 2) : 0;
}

cudaError_t launch_paged_step(int dk, int dv, const PagedStepArgs& p, cudaStream_t stream) {
  if (step_mma_supported(dk, dv, p.in_dtype)) return dk == 128 ? step_mma<128>(p, stream) : step_mma<64>(p, stream);
  return for_dim(dk, [&](auto k) { return for_dim(dv, [&](auto v) { return step<k(), v()>(p, stream); }); });
}

}  // namespace kdn
