// Windowed attention on the fp32 CUDA cores: every supported size and type.
//
//   vis(t) = { j <= t : j > t - window or j < n_sink },  s_tj = scale q_t . k_j,
//   lse_t = log sum_vis exp s_tj,  o_t = sum_vis exp(s_tj - lse_t) v_j.
//
// One CTA of 256 threads per 64 queries of a head walks the 64-token key tiles that any of them sees (the sinks'
// tiles, then the window's), with the running maximum and sum of the softmax in registers.  A thread holds 4 x 4
// scores (queries ty + 16 i, keys tx + 16 j) and the same 4 queries of o.  Rows are padded by 4 floats in shared
// memory, so that the 16-byte reads of 8 consecutive rows fall into 8 different bank groups.  Per 4 coordinates a
// warp spends 64 multiply-adds against 12 shared-memory wavefronts (16 issue cycles of the SM's four schedulers
// against 12): bound by the fp32 pipe.  Rows past the sequence's end are staged as zeros, whatever memory holds.
#include <cmath>
#include <type_traits>

#include "window.cuh"

namespace kdn {

namespace {

using window::KeyTiles;

constexpr int kThreads = 256;
constexpr int kT = 64;       // queries and keys per tile
constexpr int kLP = kT + 4;  // row stride of the score tile

// Rows t0 .. t0 + 63 of a [L, D] array into shared memory as fp32; rows at or past ``len`` become zero.
template <int D>
__device__ __forceinline__ void stage(float* dst, const void* src, size_t row0, int t0, int len, int dtype) {
  constexpr int Q = D / 4;
  for (int e = threadIdx.x; e < kT * Q; e += kThreads) {
    const int r = e / Q, c = 4 * (e % Q);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t0 + r < len) {
      const size_t at = (row0 + t0 + r) * D + c;
      if (dtype == kBF16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(src) + at);
        x = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                        __uint_as_float(u.y & 0xffff0000u));
      } else {
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
      }
    }
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = x;
  }
}

// acc[i][j] += a[ra + 16 i] . b[rb + 16 j] over D coordinates.
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float* a, int ra, const float* b, int rb) {
  constexpr int S = D + 4;
  float2 sum[4][4] = {};  // even and odd coordinates
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ra + 16 * i) * S + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (rb + 16 * j) * S + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sum[i][j] = window::fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w),
                                 window::fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), sum[i][j]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] += sum[i][j].x + sum[i][j].y;
}

// a[n] += w b[n], two at a time.
template <int N>
__device__ __forceinline__ void axpy(float (&a)[N], float w, const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int n = 0; n < N; n += 2) {
      const float2 r = window::fma2(make_float2(w, w), make_float2(b[n], b[n + 1]), make_float2(a[n], a[n + 1]));
      a[n] = r.x, a[n + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) a[n] = fmaf(w, b[n], a[n]);
  }
}

// Column (of D) that value n (of D / 16) of thread column tx stands for: float4 groups where the row is wide enough.
template <int D>
__device__ __forceinline__ int col_of(int tx, int n) {
  return D >= 64 ? 64 * (n / 4) + 4 * tx + n % 4 : tx + 16 * n;
}
// One row's D / 16 values of a thread.
template <int D>
__device__ __forceinline__ void row_vals(float (&x)[D / 16], const float* row, int tx) {
  if constexpr (D >= 64) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      const float4 u = *reinterpret_cast<const float4*>(row + 64 * g + 4 * tx);
      x[4 * g] = u.x, x[4 * g + 1] = u.y, x[4 * g + 2] = u.z, x[4 * g + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int n = 0; n < D / 16; ++n) x[n] = row[tx + 16 * n];
  }
}

// acc[i][n] += sum_j w[(r + 16 i)][j] b[j][col n]: the row-times-tile product (o += P v, dq += dS k).
template <int D>
__device__ __forceinline__ void rows_times_tile(float (&acc)[4][D / 16], const float* w, int r, const float* b, int tx) {
#pragma unroll 2
  for (int j = 0; j < kT; j += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(w + (r + 16 * i) * kLP + j);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x[D / 16];
      row_vals<D>(x, b + (j + u) * (D + 4), tx);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        axpy(acc[i], u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w, x);
      }
    }
  }
}

// acc[i][n] += sum_t w[t][4 ty + i] b[t][col n]: the transposed product (dv += P^T dO, dk += dS^T q).
template <int D>
__device__ __forceinline__ void cols_times_tile(float (&acc)[4][D / 16], const float* w, int ty, const float* b, int tx) {
#pragma unroll 4
  for (int t = 0; t < kT; ++t) {
    const float4 p = *reinterpret_cast<const float4*>(w + t * kLP + 4 * ty);
    float x[D / 16];
    row_vals<D>(x, b + t * (D + 4), tx);
    axpy(acc[0], p.x, x), axpy(acc[1], p.y, x), axpy(acc[2], p.z, x), axpy(acc[3], p.w, x);
  }
}

// Write a thread's values of one row.
template <int D>
__device__ __forceinline__ void put_row(void* dst, size_t row, const float (&x)[D / 16], float f, int tx, int dtype) {
#pragma unroll
  for (int n = 0; n < D / 16; ++n) store_elem(dst, row * D + col_of<D>(tx, n), x[n] * f, dtype);
}

// Rows t .. t0 + 63 (t = the sequence's end, or t0 where the tile lies behind it) of a [L, D] array become zero.
template <int D>
__device__ __forceinline__ void zero_tile(void* dst, size_t row0, int t0, int len, int L, int dtype) {
  const int first = max(t0, len), last = min(t0 + kT, L), words = D * (dtype == kBF16 ? 2 : 4) / 16;
  for (int e = threadIdx.x; e < (last - first) * words; e += kThreads)
    static_cast<uint4*>(dst)[(row0 + first) * words + e] = make_uint4(0, 0, 0, 0);
}

// Which tile, head and sequence this CTA has: tiles run fastest from the last one down (it has the longest walk).
struct Where {
  int tile, h, b;
};
__device__ __forceinline__ Where where(int tiles, int heads) {
  const unsigned x = blockIdx.x;
  Where w;
  w.tile = tiles - 1 - static_cast<int>(x % tiles);
  const unsigned y = x / tiles;
  w.h = static_cast<int>(y % heads), w.b = static_cast<int>(y / heads);
  return w;
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) window_fwd_kernel(WindowArgs p) {
  extern __shared__ __align__(16) float sm[];
  float* q_s = sm;
  float* k_s = q_s + kT * (DK + 4);
  float* v_s = k_s + kT * (DK + 4);
  float* p_s = v_s + kT * (DV + 4);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Where w = where((p.L + kT - 1) / kT, p.H);
  const int len = window::seq_len(p, w.b), t0 = w.tile * kT;
  const size_t qrow = ((size_t)w.b * p.H + w.h) * p.L;
  if (p.zero_rest && t0 + kT > len) {
    zero_tile<DV>(p.o, qrow, t0, len, p.L, p.out_dtype);
    const int t = max(t0, len) + tid;
    if (t < min(t0 + kT, p.L)) p.lse[qrow + t] = 0.f;
  }
  if (t0 >= len) return;
  const size_t krow = ((size_t)w.b * p.Hkv + w.h / (p.H / p.Hkv)) * p.L;
  const KeyTiles kt = window::key_tiles<kT>(t0, min(t0 + kT, len) - 1, p.window, p.n_sink);
  stage<DK>(q_s, p.q, qrow, t0, len, p.in_dtype);
  float m[4], l[4], acc[4][DV / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int n = 0; n < DV / 16; ++n) acc[i][n] = 0.f;
  }
  for (int it = 0; it < kt.count(); ++it) {
    const int j0 = kt.walk(it) * kT;
    __syncthreads();  // the previous tile has been read
    stage<DK>(k_s, p.k, krow, j0, len, p.in_dtype);
    stage<DV>(v_s, p.v, krow, j0, len, p.in_dtype);
    __syncthreads();
    float s[4][4] = {};
    dot_tile<DK>(s, q_s, ty, k_s, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + ty + 16 * i;
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = window::visible(t, j0 + tx + 16 * j, p.window, p.n_sink) ? s[i][j] * p.scale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = top == -INFINITY ? 0.f : top;  // no key of this row so far
      const float keep = expf(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = expf(s[i][j] - base);
        sum += e;
        p_s[(ty + 16 * i) * kLP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * keep + sum;
      m[i] = top;
#pragma unroll
      for (int n = 0; n < DV / 16; ++n) acc[i][n] *= keep;
    }
    __syncwarp();  // a query row's scores are written and read by the same half-warp
    rows_times_tile<DV>(acc, p_s, ty, v_s, tx);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty + 16 * i;
    if (t >= len) continue;
    put_row<DV>(p.o, qrow + t, acc[i], 1.f / l[i], tx, p.out_dtype);
    if (tx == 0) p.lse[qrow + t] = m[i] + logf(l[i]);
  }
}

// delta_t = dO_t . o_t, one warp per token.
__global__ void __launch_bounds__(256) window_delta_kernel(WindowArgs p, int dv) {
  const size_t row = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;  // nothing of this call has raised it yet
  if (row >= (size_t)p.B * p.H * p.L) return;
  const int b = static_cast<int>(row / ((size_t)p.H * p.L)), t = static_cast<int>(row % p.L);
  if (t >= window::seq_len(p, b)) return;
  float x = 0.f;
  for (int c = lane; c < dv; c += 32)
    x = fmaf(load_elem(p.o, row * dv + c, p.out_dtype), load_elem(p.dO, row * dv + c, p.out_dtype), x);
  x = warp_sum(x);
  if (lane == 0) p.delta[row] = x;
}

// P and dS of one 64 x 64 tile: P = exp(scale q.k - lse), dS = P (dO.v - delta), zero where hidden or past the end.
template <int DK, int DV>
__device__ __forceinline__ void grad_scores(const WindowArgs& p, const float* q_s, const float* k_s, const float* do_s,
                                            const float* v_s, const float* lse_s, const float* delta_s, int t0, int j0,
                                            int len, int tx, int ty, float (&P)[4][4], float (&dS)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) P[i][j] = 0.f, dS[i][j] = 0.f;
  dot_tile<DK>(P, q_s, ty, k_s, tx);
  dot_tile<DV>(dS, do_s, ty, v_s, tx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i, t = t0 + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool vis = t < len && window::visible(t, j0 + tx + 16 * j, p.window, p.n_sink);
      P[i][j] = vis ? expf(fmaf(P[i][j], p.scale, -lse_s[r])) : 0.f;
      dS[i][j] = vis ? P[i][j] * (dS[i][j] - delta_s[r]) : 0.f;
    }
  }
}

__device__ __forceinline__ void stage_rows(const WindowArgs& p, float* lse_s, float* delta_s, size_t qrow, int t0, int len) {
  const int r = threadIdx.x;
  if (r < kT) {
    const bool in = t0 + r < len;
    lse_s[r] = in ? p.lse[qrow + t0 + r] : 0.f;
    delta_s[r] = in ? p.delta[qrow + t0 + r] : 0.f;
  }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) window_dq_kernel(WindowArgs p) {
  extern __shared__ __align__(16) float sm[];
  float* q_s = sm;
  float* do_s = q_s + kT * (DK + 4);
  float* k_s = do_s + kT * (DV + 4);
  float* v_s = k_s + kT * (DK + 4);
  float* ds_s = v_s + kT * (DV + 4);
  float* lse_s = ds_s + kT * kLP;
  float* delta_s = lse_s + kT;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Where w = where((p.L + kT - 1) / kT, p.H);
  const int len = window::seq_len(p, w.b), t0 = w.tile * kT;
  const size_t qrow = ((size_t)w.b * p.H + w.h) * p.L;
  if (p.zero_rest && t0 + kT > len) zero_tile<DK>(p.dq, qrow, t0, len, p.L, p.in_dtype);
  if (t0 >= len) return;
  const size_t krow = ((size_t)w.b * p.Hkv + w.h / (p.H / p.Hkv)) * p.L;
  const KeyTiles kt = window::key_tiles<kT>(t0, min(t0 + kT, len) - 1, p.window, p.n_sink);
  stage<DK>(q_s, p.q, qrow, t0, len, p.in_dtype);
  stage<DV>(do_s, p.dO, qrow, t0, len, p.out_dtype);
  stage_rows(p, lse_s, delta_s, qrow, t0, len);
  float acc[4][DK / 16] = {};
  for (int it = 0; it < kt.count(); ++it) {
    const int j0 = kt.walk(it) * kT;
    __syncthreads();
    stage<DK>(k_s, p.k, krow, j0, len, p.in_dtype);
    stage<DV>(v_s, p.v, krow, j0, len, p.in_dtype);
    __syncthreads();
    float P[4][4], dS[4][4];
    grad_scores<DK, DV>(p, q_s, k_s, do_s, v_s, lse_s, delta_s, t0, j0, len, tx, ty, P, dS);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ds_s[(ty + 16 * i) * kLP + tx + 16 * j] = dS[i][j];
    __syncwarp();
    rows_times_tile<DK>(acc, ds_s, ty, k_s, tx);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty + 16 * i;
    if (t < len) put_row<DK>(p.dq, qrow + t, acc[i], p.scale, tx, p.in_dtype);
  }
}

// One CTA per 64 keys of a k/v head: it walks every query tile that sees them, of every head that shares them, in a
// fixed order, so the sums of a gradient are the same on every run.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) window_dkdv_kernel(WindowArgs p) {
  extern __shared__ __align__(16) float sm[];
  float* k_s = sm;
  float* v_s = k_s + kT * (DK + 4);
  float* q_s = v_s + kT * (DV + 4);
  float* do_s = q_s + kT * (DK + 4);
  float* p_s = do_s + kT * (DV + 4);
  float* ds_s = p_s + kT * kLP;
  float* lse_s = ds_s + kT * kLP;
  float* delta_s = lse_s + kT;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  Where w = where((p.L + kT - 1) / kT, p.Hkv);
  w.tile = (p.L + kT - 1) / kT - 1 - w.tile;  // the first tiles (sinks) have the longest walk
  const int len = window::seq_len(p, w.b), j0 = w.tile * kT;
  const int G = p.H / p.Hkv;
  const size_t krow = ((size_t)w.b * p.Hkv + w.h) * p.L;
  if (p.zero_rest && j0 + kT > len) {
    zero_tile<DK>(p.dk, krow, j0, len, p.L, p.in_dtype);
    zero_tile<DV>(p.dv, krow, j0, len, p.L, p.in_dtype);
  }
  if (j0 >= len) return;
  int lo, hi;
  window::query_tiles<kT>(j0, min(j0 + kT, len) - 1, len, p.window, p.n_sink, lo, hi);
  stage<DK>(k_s, p.k, krow, j0, len, p.in_dtype);
  stage<DV>(v_s, p.v, krow, j0, len, p.in_dtype);
  float dk[4][DK / 16] = {}, dv[4][DV / 16] = {};
  for (int g = 0; g < G; ++g) {
    const size_t qrow = ((size_t)w.b * p.H + w.h * G + g) * p.L;
    for (int qt = lo; qt < hi; ++qt) {
      const int t0 = qt * kT;
      __syncthreads();
      stage<DK>(q_s, p.q, qrow, t0, len, p.in_dtype);
      stage<DV>(do_s, p.dO, qrow, t0, len, p.out_dtype);
      stage_rows(p, lse_s, delta_s, qrow, t0, len);
      __syncthreads();
      float P[4][4], dS[4][4];
      grad_scores<DK, DV>(p, q_s, k_s, do_s, v_s, lse_s, delta_s, t0, j0, len, tx, ty, P, dS);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p_s[(ty + 16 * i) * kLP + tx + 16 * j] = P[i][j];
          ds_s[(ty + 16 * i) * kLP + tx + 16 * j] = dS[i][j];
        }
      __syncthreads();
      cols_times_tile<DV>(dv, p_s, ty, do_s, tx);
      cols_times_tile<DK>(dk, ds_s, ty, q_s, tx);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 4 * ty + i;
    if (j >= len) continue;
    put_row<DK>(p.dk, krow + j, dk[i], p.scale, tx, p.in_dtype);
    put_row<DV>(p.dv, krow + j, dv[i], 1.f, tx, p.in_dtype);
  }
}

template <typename K>
cudaError_t run(K kernel, size_t floats, long long ctas, const WindowArgs& p, cudaStream_t stream) {
  const size_t smem = floats * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t forward(const WindowArgs& p, cudaStream_t stream) {
  const long long tiles = (p.L + kT - 1) / kT;
  return run(window_fwd_kernel<DK, DV>, kT * (2 * (DK + 4) + (DV + 4) + kLP), tiles * p.H * p.B, p, stream);
}

template <int DK, int DV>
cudaError_t backward(const WindowArgs& p, cudaStream_t stream) {
  const long long tiles = (p.L + kT - 1) / kT;
  const size_t base = kT * (2 * (DK + 4) + 2 * (DV + 4) + 2);
  const cudaError_t e = run(window_dq_kernel<DK, DV>, base + kT * kLP, tiles * p.H * p.B, p, stream);
  if (e != cudaSuccess) return e;
  return run(window_dkdv_kernel<DK, DV>, base + 2 * kT * kLP, tiles * p.Hkv * p.B, p, stream);
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

cudaError_t launch_window_attn(int dk, int dv, const WindowArgs& p, cudaStream_t stream) {
  if (window_tc_supported(dk, dv, p.in_dtype)) return launch_window_attn_tc(dk, p, stream);
  return for_dim(dk, [&](auto k) { return for_dim(dv, [&](auto v) { return forward<k(), v()>(p, stream); }); });
}

cudaError_t launch_window_attn_backward(int dk, int dv, const WindowArgs& p, cudaStream_t stream) {
  if (window_tc_supported(dk, dv, p.in_dtype)) return launch_window_bwd_tc(dk, p, stream);
  const size_t rows = (size_t)p.B * p.H * p.L;
  window_delta_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p, dv);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return for_dim(dk, [&](auto k) { return for_dim(dv, [&](auto v) { return backward<k(), v()>(p, stream); }); });
}

}  // namespace kdn
