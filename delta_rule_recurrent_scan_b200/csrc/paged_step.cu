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

// ------------------------------------------------------------------------------------------ fp32 CUDA cores
// Every size and type.  128 threads, 8 query heads, tiles of 32 tokens staged as fp32: warp w has the scores of heads
// 2 w and 2 w + 1 for its lane's token; then thread t has column t % d_v of every head's o.
constexpr int kTok = 32, kThr = 128, kHB = 8;

template <int D>
__device__ __forceinline__ bool stage_tokens(float* dst, const void* pool, const PagedStepArgs& p, const int* entries, int kvh,
                                             int j0, int n) {
  constexpr int Q = D / 4;
  bool bad = false;
  for (int e = threadIdx.x; e < kTok * Q; e += kThr) {
    const int r = e / Q, c = 4 * (e % Q), j = j0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < n) {
      const int page = entries[j / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        bad = true;
      } else {
        const size_t at = (((size_t)page * p.Hkv + kvh) * p.page_size + j % p.page_size) * D + c;
        if (p.in_dtype == kBF16) {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(pool) + at);
          x = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                          __uint_as_float(u.y & 0xffff0000u));
        } else {
          x = *reinterpret_cast<const float4*>(static_cast<const float*>(pool) + at);
        }
      }
    }
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = x;
  }
  return bad;
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThr) paged_step_kernel(PagedStepArgs p) {
  __shared__ __align__(16) float k_s[kTok * (DK + 4)], v_s[kTok * (DV + 4)], q_s[kHB * DK], p_s[kTok * kHB];
  __shared__ float keep_s[kHB], l_s[kHB], m_s[kHB];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Part w = which<kHB>(p);
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
  if (n > 0) kt = window::key_tiles<kTok>(n - 1, n - 1, win, p.n_sink);
  const int it0 = (int)((long long)kt.count() * w.split / p.splits), it1 = (int)((long long)kt.count() * (w.split + 1) / p.splits);
  for (int e = tid; e < kHB * DK; e += kThr)
    q_s[e] = e / DK < w.nh ? load_elem(p.q, ((size_t)w.b * p.H + w.h0) * DK + e, p.in_dtype) * p.scale : 0.f;
  constexpr int kGroups = kThr / DV;  // token groups of the second half (d_v < 128)
  const int col = tid % DV, tg = tid / DV;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[kHB] = {};
  for (int it = it0; it < it1; ++it) {
    const int j0 = kt.walk(it) * kTok;
    __syncthreads();
    bad |= stage_tokens<DK>(k_s, p.k_pages, p, entries, w.kvh, j0, n);
    bad |= stage_tokens<DV>(v_s, p.v_pages, p, entries, w.kvh, j0, n);
    __syncthreads();
    float s[2] = {0.f, 0.f};
#pragma unroll 8
    for (int c = 0; c < DK; c += 4) {
      const float4 k = *reinterpret_cast<const float4*>(k_s + lane * (DK + 4) + c);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(q_s + (2 * warp + i) * DK + c);
        s[i] = fmaf(k.w, q.w, fmaf(k.z, q.z, fmaf(k.y, q.y, fmaf(k.x, q.x, s[i]))));
      }
    }
    const int j = j0 + lane;
    const bool vis = j < n && window::visible(n - 1, j, win, p.n_sink);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!vis) s[i] = -INFINITY;
      float top = fmaxf(m[i], s[i]);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = expf(m[i] - base), e = expf(s[i] - base);
      l[i] = l[i] * keep + warp_sum(e);
      m[i] = top;
      p_s[lane * kHB + 2 * warp + i] = e;
      if (lane == 0) keep_s[2 * warp + i] = keep;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHB; ++h) acc[h] *= keep_s[h];
#pragma unroll 8
    for (int t = tg; t < kTok; t += kGroups) {
      const float v = v_s[t * (DV + 4) + col];
      const float4 a = *reinterpret_cast<const float4*>(p_s + t * kHB), b = *reinterpret_cast<const float4*>(p_s + t * kHB + 4);
      acc[0] = fmaf(a.x, v, acc[0]), acc[1] = fmaf(a.y, v, acc[1]), acc[2] = fmaf(a.z, v, acc[2]), acc[3] = fmaf(a.w, v, acc[3]);
      acc[4] = fmaf(b.x, v, acc[4]), acc[5] = fmaf(b.y, v, acc[5]), acc[6] = fmaf(b.z, v, acc[6]), acc[7] = fmaf(b.w, v, acc[7]);
    }
  }
  bad = __syncthreads_or(bad);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < 2; ++i) m_s[2 * warp + i] = m[i], l_s[2 * warp + i] = bad ? NAN : l[i];
  if constexpr (kGroups > 1) {  // the token groups' sums, in their order
    float* red = k_s;
    static_assert(4 * kThr <= kTok * (DK + 4), "room for four heads' sums");
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // four heads at a time
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 4; ++h) red[h * kThr + tid] = acc[4 * half + h];
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float x = 0.f;
        for (int g = 0; g < kGroups; ++g) x += red[h * kThr + g * DV + col];
        acc[4 * half + h] = x;
      }
    }
  }
  __syncthreads();
  if (tg != 0) return;
#pragma unroll
  for (int h = 0; h < kHB; ++h) {
    if (h >= w.nh) break;
    const size_t head = (size_t)w.b * p.H + w.h0 + h;
    if (p.splits == 1) {
      const float x = l_s[h] == 0.f ? 0.f : acc[h] / l_s[h];  // nothing visible: zero
      store_elem(p.o, head * DV + col, x, p.out_dtype);
      if (col == 0 && p.lse) p.lse[head] = m_s[h] + logf(l_s[h]);
    } else {
      const size_t at = part_at(p, w.b, w.h0 + h, w.split);
      p.part[at * DV + col] = acc[h];
      if (col == 0) part_max(p, DV)[at] = m_s[h], part_sum(p, DV)[at] = l_s[h];
    }
  }
}

// Joins a head's parts: one CTA of d_v threads (at least a warp) per head.
template <int DV>
__global__ void __launch_bounds__(DV < 32 ? 32 : DV) paged_join_kernel(PagedStepArgs p) {
  const size_t head = blockIdx.x;
  const float* pm = part_max(p, DV) + head * p.splits;
  const float* pl = part_sum(p, DV) + head * p.splits;
  const float* po = p.part + head * p.splits * DV;
  float M = -INFINITY;
  for (int i = 0; i < p.splits; ++i) M = fmaxf(M, pm[i]);
  const float base = M == -INFINITY ? 0.f : M;
  float l = 0.f, x = 0.f;
  const int col = threadIdx.x;
  for (int i = 0; i < p.splits; ++i) {
    const float f = expf(pm[i] - base);
    l = fmaf(f, pl[i], l);
    if (col < DV) x = fmaf(f, po[(size_t)i * DV + col], x);
  }
  if (col < DV) store_elem(p.o, head * DV + col, l == 0.f ? 0.f : x / l, p.out_dtype);
  if (col == 0 && p.lse) p.lse[head] = M + logf(l);
}

template <int DK, int DV>
cudaError_t step(const PagedStepArgs& p, cudaStream_t stream) {
  const int G = p.H / p.Hkv;
  const long long ctas = (long long)p.n * p.Hkv * ((G + kHB - 1) / kHB) * p.splits;
  paged_step_kernel<DK, DV><<<(unsigned)ctas, kThr, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  paged_join_kernel<DV><<<p.n * p.H, DV < 32 ? 32 : DV, 0, stream>>>(p);
  return cudaGetLastError();
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
  (void)dk, (void)dv, (void)in_dtype;
  const int G = H / Hkv;
  const long long pairs = (long long)n * Hkv * ((G + kHB - 1) / kHB);
  const long long tiles = (most_tokens + kTok - 1) / kTok;
  // enough parts for four CTAs on each of 148 SMs, of at least four tiles each
  long long s = (4 * 148 + pairs - 1) / pairs;
  if (s > tiles / 4) s = tiles / 4;
  return s < 1 ? 1 : (int)s;
}

size_t paged_step_part_floats(int dv, int n, int H, int splits) {
  return splits > 1 ? (size_t)n * H * splits * (dv + 2) : 0;
}

cudaError_t launch_paged_step(int dk, int dv, const PagedStepArgs& p, cudaStream_t stream) {
  return for_dim(dk, [&](auto k) { return for_dim(dv, [&](auto v) { return step<k(), v()>(p, stream); }); });
}

}  // namespace kdn
