// Windowed attention on the fp32 CUDA cores: every supported size and type.
//
//   vis(t) = { j <= t : j > t - window or j < n_sink },  s_tj = scale q_t . k_j,
//   lse_t = log sum_vis exp s_tj,  o_t = sum_vis exp(s_tj - lse_t) v_j,
//   dv = P^T dO,  dq = scale dS k,  dk = scale dS^T q,  dS = P (dO v^T - delta),  delta_t = dO_t . o_t.
//
// All three kernels are one scheme.  A CTA of 8 warps owns 8 R rows (queries; keys for dk and dv) and walks the 64-row
// tiles of the other side that they meet, staged in shared memory as fp32.  A warp has R rows, the same for all of its
// lanes, and a lane has 2 of the 64 columns:
//   scores:   s[R][2] += row . column; a row's 16 bytes are one broadcast read for the whole warp, the columns' rows are
//             padded by 4 floats so that 8 consecutive lanes fall into 8 different bank groups.  Per 4 coordinates a warp
//             spends 8 R multiply-adds against R + 8 wavefronts;
//   weights:  exp, masks, row maxima and sums within the warp; the R x 64 weights go to a piece of shared memory of the
//             warp's own (no CTA barrier between scores and products);
//   products: acc[R][d / 32] += weight x tile row, again with the weights as broadcast reads.
// R is 8, or 4 where 8 would leave SMs without a CTA.  The next tiles are copied (cp.async) while these are used, where a
// second set of them costs no CTA on the SM.  Measured (fp32, 3 padded sequences of 1531, 8 heads of 64, window 257, 16
// sinks): forward 108 us, backward 359 us; with one set of tiles 117 and 392 us; 4 x 4 values per thread with the rows
// spread over the lanes (four wavefronts a read): 121 and 615 us; R = 16 (one CTA per SM, longer tail): 163 and 404 us;
// three CTAs per SM (spills): 146 and 464 us.  Bound by latency: 8 to 16 warps an SM, the fp32 pipe about 40 % busy.
// tf32 products in three parts were not taken: warp products run at 260 TFLOP/s of tf32, 87 after the split against 74 of
// the fp32 pipe, with an accumulator that truncates.
//
// Rows past the sequence's end are staged as zeros, whatever memory holds.
#include <cmath>
#include <type_traits>

#include "window.cuh"

namespace kdn {

namespace {

using window::KeyPass;
using window::KeyTiles;

constexpr int kThreads = 256, kWarps = 8;
constexpr int kT = 64;       // rows of a walked tile
constexpr int kLP = kT + 4;  // row stride of the weights
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Rows t0 .. t0 + ROWS - 1 of a [L, D] array into shared memory as fp32; rows at or past ``len`` become zero.
template <int D, int ROWS>
__device__ __forceinline__ void stage(float* dst, const void* src, size_t row0, int t0, int len, int dtype) {
  constexpr int Q = D / 4;
#pragma unroll 4
  for (int e = threadIdx.x; e < ROWS * Q; e += kThreads) {
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

// The same, begun: fp32 rows are copied asynchronously (zeros where there is no row), bf16 rows converted at once.  The
// caller commits, waits and synchronises.
template <int D, int ROWS>
__device__ __forceinline__ void begin_stage(float* dst, const void* src, size_t row0, int t0, int len, int dtype) {
  if (dtype == kBF16) {
    stage<D, ROWS>(dst, src, row0, t0, len, dtype);
    return;
  }
  constexpr int Q = D / 4;
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  const float* from = static_cast<const float*>(src) + (row0 + t0) * D;
#pragma unroll 4
  for (int e = threadIdx.x; e < ROWS * Q; e += kThreads) {
    const int r = e / Q, c = 4 * (e % Q);
    const bool there = t0 + r < len;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (r * (D + 4) + c) * 4),
                 "l"(there ? from + (size_t)r * D + c : static_cast<const float*>(src)), "r"(there ? 16 : 0) : "memory");
  }
}

// Shared memory of a CTA beside ``rest`` floats: one set of the two walked tiles, or two, the next tiles being copied while
// these are used.  With R = 4 (few CTAs) always two, else where they cost no CTA on the SM.
template <int DK, int DV>
constexpr int kWalked = kT * (DK + DV + 8);
constexpr int ctas_per_sm(int floats) { return 227 * 1024 / (floats * 4 + 1024) < 2 ? 227 * 1024 / (floats * 4 + 1024) : 2; }
template <int DK, int DV, int R>
constexpr bool two_sets(int rest) {
  return ctas_per_sm(rest + 2 * kWalked<DK, DV>) >= (R == 4 ? 1 : ctas_per_sm(rest + kWalked<DK, DV>));
}
template <int DK, int DV, int R>
constexpr int total(int rest) { return rest + (two_sets<DK, DV, R>(rest) ? 2 : 1) * kWalked<DK, DV>; }
template <int DK, int DV, int R>
constexpr int kFwdRest = kWarps * R * (DK + 4 + kLP);
template <int DK, int DV, int R>
constexpr int kDqRest = kWarps * R * (DK + DV + 8 + kLP);
template <int DK, int DV, int R>
constexpr int kKeysRest = kWarps * R * (DK + DV + 8 + 2 * kLP);

// s[i][c] = rows[i] . tile[lane + 32 c]
template <int D, int R>
__device__ __forceinline__ void scores(float (&s)[R][2], const float* rows, const float* tile, int lane) {
  constexpr int S = D + 4;
  float2 sum[R][2] = {};  // even and odd coordinates
#pragma unroll 2
  for (int c = 0; c < D; c += 4) {
    const float4 y0 = *reinterpret_cast<const float4*>(tile + lane * S + c);
    const float4 y1 = *reinterpret_cast<const float4*>(tile + (lane + 32) * S + c);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(rows + i * S + c);
      const float2 a = make_float2(x.x, x.y), b = make_float2(x.z, x.w);
      sum[i][0] = window::fma2(b, make_float2(y0.z, y0.w), window::fma2(a, make_float2(y0.x, y0.y), sum[i][0]));
      sum[i][1] = window::fma2(b, make_float2(y1.z, y1.w), window::fma2(a, make_float2(y1.x, y1.y), sum[i][1]));
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) s[i][0] = sum[i][0].x + sum[i][0].y, s[i][1] = sum[i][1].x + sum[i][1].y;
}

// Values of a row that a lane holds: d / 32 consecutive ones; with d = 16 one, the half-warps sharing the tile's rows.
template <int D>
constexpr int kVals = D < 32 ? 1 : D / 32;
template <int D>
__device__ __forceinline__ int first_col(int lane) {
  return D < 32 ? lane % D : lane * kVals<D>;
}

// acc[i] += sum_j w[i][j] tile[j]: the products with the weights of this warp.
template <int D, int R>
__device__ __forceinline__ void products(float (&acc)[R][kVals<D>], const float* w, const float* tile, int lane) {
  constexpr int S = D + 4, V = kVals<D>;
  const float* at = tile + first_col<D>(lane);
  const int j0 = D < 32 ? (lane / D) * (kT / 2) : 0, j1 = D < 32 ? j0 + kT / 2 : kT;
#pragma unroll 2
  for (int j = j0; j < j1; j += 4) {
    float x[4][V];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* row = at + (j + u) * S;
      if constexpr (V == 4) {
        const float4 y = *reinterpret_cast<const float4*>(row);
        x[u][0] = y.x, x[u][1] = y.y, x[u][2] = y.z, x[u][3] = y.w;
      } else if constexpr (V == 2) {
        const float2 y = *reinterpret_cast<const float2*>(row);
        x[u][0] = y.x, x[u][1] = y.y;
      } else {
        x[u][0] = *row;
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 p = *reinterpret_cast<const float4*>(w + i * kLP + j);
      const float pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (V == 1) {
          acc[i][0] = fmaf(pw[u], x[u][0], acc[i][0]);
        } else {
#pragma unroll
          for (int n = 0; n < V; n += 2) {
            const float2 r = window::fma2(make_float2(pw[u], pw[u]), make_float2(x[u][n], x[u][n + 1]),
                                          make_float2(acc[i][n], acc[i][n + 1]));
            acc[i][n] = r.x, acc[i][n + 1] = r.y;
          }
        }
      }
    }
  }
}

// Write a lane's values of one row, times f.
template <int D>
__device__ __forceinline__ void put_row(void* dst, size_t row, const float (&x)[kVals<D>], float f, int lane, int dtype) {
  if constexpr (D < 32) {
    const float y = x[0] + __shfl_xor_sync(0xffffffffu, x[0], D);  // the other half-warp's part
    if (lane < D) store_elem(dst, row * D + lane, y * f, dtype);
  } else {
    const size_t at = row * D + first_col<D>(lane);
#pragma unroll
    for (int n = 0; n < kVals<D>; ++n) store_elem(dst, at + n, x[n] * f, dtype);
  }
}

// For R values of every lane: the warp's maximum (KIND 0) or sum (1) of each, in all lanes.
template <int KIND, int R>
__device__ __forceinline__ void reduce_rows(float (&x)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x[i], o);
      x[i] = KIND == 0 ? fmaxf(x[i], y) : x[i] + y;
    }
}

// Rows max(t0, len) .. t0 + ROWS - 1 of a [L, D] array become zero.
template <int D, int ROWS>
__device__ __forceinline__ void zero_tile(void* dst, size_t row0, int t0, int len, int L, int dtype) {
  const int first = max(t0, len), last = min(t0 + ROWS, L), words = D * (dtype == kBF16 ? 2 : 4) / 16;
  for (int e = threadIdx.x; e < (last - first) * words; e += kThreads)
    static_cast<uint4*>(dst)[(row0 + first) * words + e] = make_uint4(0, 0, 0, 0);
}

// Which tile, head and sequence this CTA has: tiles run fastest from the last one down (it has the longest walk).
struct Where {
  int tile, h, b;
};
__device__ __forceinline__ Where where(unsigned x, int tiles, int heads) {
  Where w;
  w.tile = tiles - 1 - static_cast<int>(x % tiles);
  const unsigned y = x / tiles;
  w.h = static_cast<int>(y % heads), w.b = static_cast<int>(y / heads);
  return w;
}

template <int DK, int DV, int R>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(total<DK, DV, R>(kFwdRest<DK, DV, R>)))
    window_fwd_kernel(WindowArgs p) {
  constexpr int kRows = kWarps * R;
  extern __shared__ __align__(16) float sm[];
  constexpr bool kTwo = two_sets<DK, DV, R>(kFwdRest<DK, DV, R>);
  float* q_s = sm;
  float* p_s = q_s + kRows * (DK + 4);
  float* walked = p_s + kRows * kLP;  // k, then v; the second set behind them
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Where w = where(blockIdx.x, (p.L + kRows - 1) / kRows, p.H);
  const int len = window::seq_len(p, w.b), t0 = w.tile * kRows;
  const size_t qrow = ((size_t)w.b * p.H + w.h) * p.L;
  if (p.zero_rest && t0 + kRows > len) {
    zero_tile<DV, kRows>(p.o, qrow, t0, len, p.L, p.out_dtype);
    const int t = max(t0, len) + tid;
    if (t < min(t0 + kRows, p.L)) p.lse[qrow + t] = 0.f;
  }
  if (t0 >= len) return;
  const size_t krow = ((size_t)w.b * p.Hkv + w.h / (p.H / p.Hkv)) * p.L;
  const KeyTiles kt = window::key_tiles<kT>(t0, min(t0 + kRows, len) - 1, p.window, p.n_sink);
  stage<DK, kRows>(q_s, p.q, qrow, t0, len, p.in_dtype);
  const float c = p.scale * kLog2e;
  const int t_w = t0 + warp * R;  // the warp's first query
  float* w_s = p_s + warp * R * kLP;
  float m[R], l[R], acc[R][kVals<DV>] = {};  // m in base 2; l: this lane's part of the sum
#pragma unroll
  for (int i = 0; i < R; ++i) m[i] = -INFINITY, l[i] = 0.f;
  const int n = kt.count();
  auto begin = [&](int it) {
    float* to = walked + (kTwo ? it & 1 : 0) * kWalked<DK, DV>;
    begin_stage<DK, kT>(to, p.k, krow, kt.walk(it) * kT, len, p.in_dtype);
    begin_stage<DV, kT>(to + kT * (DK + 4), p.v, krow, kt.walk(it) * kT, len, p.in_dtype);
    async_commit();
  };
  begin(0);
  for (int it = 0; it < n; ++it) {
    const int j0 = kt.walk(it) * kT;
    const float* k_s = walked + (kTwo ? it & 1 : 0) * kWalked<DK, DV>;
    const float* v_s = k_s + kT * (DK + 4);
    async_wait<0>();
    __syncthreads();  // this tile is here, and the one before it has been read
    if (kTwo && it + 1 < n) begin(it + 1);
    float s[R][2], top[R];
    scores<DK, R>(s, q_s + warp * R * (DK + 4), k_s, lane);
    const bool all = j0 + kT - 1 <= t_w && (t_w + R - 1 - j0 < p.window || j0 + kT <= p.n_sink);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
        s[i][n] = all || window::visible(t_w + i, j0 + lane + 32 * n, p.window, p.n_sink) ? s[i][n] * c : -INFINITY;
      top[i] = fmaxf(s[i][0], s[i][1]);
    }
    reduce_rows<0>(top);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      top[i] = fmaxf(top[i], m[i]);
      const float base = top[i] == -INFINITY ? 0.f : top[i];  // no key of this row so far
      const float keep = exp2f(m[i] - base);
      const float a = exp2f(s[i][0] - base), b = exp2f(s[i][1] - base);
      w_s[i * kLP + lane] = a, w_s[i * kLP + lane + 32] = b;
      l[i] = fmaf(l[i], keep, a + b);
      m[i] = top[i];
#pragma unroll
      for (int n = 0; n < kVals<DV>; ++n) acc[i][n] *= keep;
    }
    __syncwarp();
    products<DV, R>(acc, w_s, v_s, lane);
    if (!kTwo && it + 1 < n) {
      __syncthreads();
      begin(it + 1);
    }
  }
  reduce_rows<1>(l);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = t_w + i;
    if (t >= len) break;
    put_row<DV>(p.o, qrow + t, acc[i], 1.f / l[i], lane, p.out_dtype);
    if (lane == 0) p.lse[qrow + t] = (m[i] + log2f(l[i])) * kLn2;
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

// A first sweep may make delta = sum P dP, also for the keys' pass (window::exact_delta).
template <int DK, int DV, int R>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(total<DK, DV, R>(kDqRest<DK, DV, R>)))
    window_dq_kernel(WindowArgs p) {
  constexpr int kRows = kWarps * R;
  extern __shared__ __align__(16) float sm[];
  constexpr bool kTwo = two_sets<DK, DV, R>(kDqRest<DK, DV, R>);
  float* q_s = sm;
  float* do_s = q_s + kRows * (DK + 4);
  float* ds_s = do_s + kRows * (DV + 4);
  float* walked = ds_s + kRows * kLP;  // k, then v; the second set behind them
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Where w = where(blockIdx.x, (p.L + kRows - 1) / kRows, p.H);
  const int len = window::seq_len(p, w.b), t0 = w.tile * kRows;
  const size_t qrow = ((size_t)w.b * p.H + w.h) * p.L;
  if (p.zero_rest && t0 + kRows > len) zero_tile<DK, kRows>(p.dq, qrow, t0, len, p.L, p.in_dtype);
  if (t0 >= len) return;
  const size_t krow = ((size_t)w.b * p.Hkv + w.h / (p.H / p.Hkv)) * p.L;
  const KeyTiles kt = window::key_tiles<kT>(t0, min(t0 + kRows, len) - 1, p.window, p.n_sink);
  stage<DK, kRows>(q_s, p.q, qrow, t0, len, p.in_dtype);
  stage<DV, kRows>(do_s, p.dO, qrow, t0, len, p.out_dtype);
  const float c = p.scale * kLog2e;
  const int t_w = t0 + warp * R;
  float* w_s = ds_s + warp * R * kLP;
  float lse[R], delta[R], acc[R][kVals<DK>] = {};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool in = t_w + i < len;
    lse[i] = in ? p.lse[qrow + t_w + i] * kLog2e : 0.f;
    delta[i] = in ? p.delta[qrow + t_w + i] : 0.f;
  }
  const int n = kt.count(), before = window::exact_delta<kT>(p, kt, t0, p.out_dtype == kBF16) ? n : 0;
  float sum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) sum[i] = 0.f;
  auto begin = [&](int it) {
    float* to = walked + (kTwo ? it & 1 : 0) * kWalked<DK, DV>;
    const int j0 = kt.walk(it < 0 ? it + n : it) * kT;
    begin_stage<DK, kT>(to, p.k, krow, j0, len, p.in_dtype);
    begin_stage<DV, kT>(to + kT * (DK + 4), p.v, krow, j0, len, p.in_dtype);
    async_commit();
  };
  begin(-before);
  for (int it = -before; it < n; ++it) {
    const int j0 = kt.walk(it < 0 ? it + n : it) * kT;
    const float* k_s = walked + (kTwo ? it & 1 : 0) * kWalked<DK, DV>;
    const float* v_s = k_s + kT * (DK + 4);
    if (it == 0 && before > 0) {
      reduce_rows<1>(sum);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        delta[i] = sum[i];
        if (lane == 0 && t_w + i < len) p.delta[qrow + t_w + i] = sum[i];
      }
    }
    async_wait<0>();
    __syncthreads();  // this tile is here, and the one before it has been read
    if (kTwo && it + 1 < n) begin(it + 1);
    float s[R][2], dp[R][2];
    scores<DK, R>(s, q_s + warp * R * (DK + 4), k_s, lane);
    scores<DV, R>(dp, do_s + warp * R * (DV + 4), v_s, lane);
    const bool all = j0 + kT - 1 <= t_w && (t_w + R - 1 - j0 < p.window || j0 + kT <= p.n_sink);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float P = window::sees_one_key(p, t_w + i) ? 1.f : exp2f(fmaf(s[i][u], c, -lse[i]));
        const bool seen = all || window::visible(t_w + i, j0 + lane + 32 * u, p.window, p.n_sink);
        if (it < 0)
          sum[i] += seen ? P * dp[i][u] : 0.f;
        else
          w_s[i * kLP + lane + 32 * u] = seen ? P * (dp[i][u] - delta[i]) : 0.f;
      }
    if (it >= 0) {
      __syncwarp();
      products<DK, R>(acc, w_s, k_s, lane);
      __syncwarp();
    }
    if (!kTwo && it + 1 < n) {
      __syncthreads();
      begin(it + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (t_w + i >= len) break;
    put_row<DK>(p.dq, qrow + t_w + i, acc[i], p.scale, lane, p.in_dtype);
  }
}

// The keys' pass: every query tile that sees the CTA's keys, of every head that shares them, in a fixed order, so the sums
// of a gradient are the same on every run.  Tiles may be cut (window::key_pass).
template <int DK, int DV, int R>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(total<DK, DV, R>(kKeysRest<DK, DV, R>)))
    window_dkdv_kernel(WindowArgs p, KeyPass kp) {
  constexpr int kRows = kWarps * R;
  extern __shared__ __align__(16) float sm[];
  constexpr bool kTwo = two_sets<DK, DV, R>(kKeysRest<DK, DV, R>);
  float* k_s = sm;
  float* v_s = k_s + kRows * (DK + 4);
  float* p_s = v_s + kRows * (DV + 4);
  float* ds_s = p_s + kRows * kLP;
  float* walked = ds_s + kRows * kLP;  // q, then dO; the second set behind them
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int part;
  const int parts = window::key_tile_of(kp, p.B * p.Hkv, (p.L + kRows - 1) / kRows, blockIdx.x, part);
  const int tile = kp.tile, h = kp.head % p.Hkv, b = kp.head / p.Hkv;
  const int len = window::seq_len(p, b), j0 = tile * kRows;
  const int G = p.H / p.Hkv;
  const size_t krow = (size_t)kp.head * p.L;
  if (p.zero_rest && part == 0 && j0 + kRows > len) {
    zero_tile<DK, kRows>(p.dk, krow, j0, len, p.L, p.in_dtype);
    zero_tile<DV, kRows>(p.dv, krow, j0, len, p.L, p.in_dtype);
  }
  if (j0 >= len) return;
  int lo, hi;
  window::query_tiles<kT>(j0, min(j0 + kRows, len) - 1, len, p.window, p.n_sink, lo, hi);
  const int per = hi - lo, all_items = per * G;  // (head of the group, query tile), query tiles fastest
  const int first = parts > 1 ? (int)((long long)all_items * part / parts) : 0;
  const int last = parts > 1 ? (int)((long long)all_items * (part + 1) / parts) : all_items;
  stage<DK, kRows>(k_s, p.k, krow, j0, len, p.in_dtype);
  stage<DV, kRows>(v_s, p.v, krow, j0, len, p.in_dtype);
  const float c = p.scale * kLog2e;
  const int j_w = j0 + warp * R;  // the warp's first key
  float* pw_s = p_s + warp * R * kLP;
  float* dw_s = ds_s + warp * R * kLP;
  float dk[R][kVals<DK>] = {}, dv[R][kVals<DV>] = {};
  float lse_next[2], delta_next[2];  // of this lane's queries; behind the end every weight is zero
  auto begin = [&](int item) {
    float* to = walked + (kTwo ? item & 1 : 0) * kWalked<DK, DV>;
    const int t0 = (lo + item % per) * kT;
    const size_t qrow = ((size_t)b * p.H + h * G + item / per) * p.L;
    begin_stage<DK, kT>(to, p.q, qrow, t0, len, p.in_dtype);
    begin_stage<DV, kT>(to + kT * (DK + 4), p.dO, qrow, t0, len, p.out_dtype);
    async_commit();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + lane + 32 * u;
      lse_next[u] = t < len ? p.lse[qrow + t] * kLog2e : INFINITY;
      delta_next[u] = t < len ? p.delta[qrow + t] : 0.f;
    }
  };
  if (first < last) begin(first);
  for (int item = first; item < last; ++item) {
    const int t0 = (lo + item % per) * kT;
    const float* q_s = walked + (kTwo ? item & 1 : 0) * kWalked<DK, DV>;
    const float* do_s = q_s + kT * (DK + 4);
    const float lse[2] = {lse_next[0], lse_next[1]}, delta[2] = {delta_next[0], delta_next[1]};
    async_wait<0>();
    __syncthreads();  // these tiles are here, and the ones before them have been read
    if (kTwo && item + 1 < last) begin(item + 1);
    float s[R][2], dp[R][2];
    scores<DK, R>(s, k_s + warp * R * (DK + 4), q_s, lane);
    scores<DV, R>(dp, v_s + warp * R * (DV + 4), do_s, lane);
    const bool all = t0 >= j_w + R - 1 && (t0 + kT - 1 - j_w < p.window || j_w + R <= p.n_sink);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float P = exp2f(fmaf(s[i][n], c, -lse[n]));
        if (!all && !window::visible(t0 + lane + 32 * n, j_w + i, p.window, p.n_sink)) P = 0.f;
        pw_s[i * kLP + lane + 32 * n] = P;
        dw_s[i * kLP + lane + 32 * n] = P == 0.f ? 0.f : P * (dp[i][n] - delta[n]);
      }
    __syncwarp();
    products<DV, R>(dv, pw_s, do_s, lane);
    products<DK, R>(dk, dw_s, q_s, lane);
    __syncwarp();
    if (!kTwo && item + 1 < last) {
      __syncthreads();
      begin(item + 1);
    }
  }
  if (parts > 1) {  // a slot: [dk, then dv] of the CTA's rows, fp32
    float* out = kp.part + (size_t)blockIdx.x * kRows * (DK + DV);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      put_row<DK>(out, warp * R + i, dk[i], p.scale, lane, kF32);
      put_row<DV>(out + kRows * DK, warp * R + i, dv[i], 1.f, lane, kF32);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (j_w + i >= len) break;
    put_row<DK>(p.dk, krow + j_w + i, dk[i], p.scale, lane, p.in_dtype);
    put_row<DV>(p.dv, krow + j_w + i, dv[i], 1.f, lane, p.in_dtype);
  }
}

// The cut tiles' parts, added in their order; one value per thread.
__global__ void __launch_bounds__(256) window_sum_parts_kernel(WindowArgs p, KeyPass kp, int cut, int rows, int dk, int dv) {
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  const int per = rows * (dk + dv);
  const size_t which = e / per;  // (sequence, k/v head, tile)
  if (which >= (size_t)p.B * p.Hkv * cut) return;
  int x = static_cast<int>(e % per);
  const size_t head = which / cut;
  const int tile = static_cast<int>(which % cut);
  size_t slot;
  const int parts = window::parts_of(kp, p.B * p.Hkv, (p.L + rows - 1) / rows, head, tile, slot);
  const float* from = kp.part + slot * per + x;
  const bool keys = x < rows * dk;
  if (!keys) x -= rows * dk;
  const int d = keys ? dk : dv;
  const int j = tile * rows + x / d;
  if (j >= window::seq_len(p, static_cast<int>(head / p.Hkv))) return;
  float a = 0.f;
  for (int i = 0; i < parts; ++i) a += from[(size_t)i * per];
  store_elem(keys ? p.dk : p.dv, (head * p.L + j) * d + x % d, a, p.in_dtype);
}

template <typename K, typename... A>
cudaError_t run(K kernel, size_t floats, long long ctas, cudaStream_t stream, const A&... args) {
  const size_t smem = floats * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)ctas, kThreads, smem, stream>>>(args...);
  return cudaGetLastError();
}

using window::kSms;
long long row_tiles(const WindowArgs& p, int rows, int heads) { return (long long)p.B * heads * ((p.L + rows - 1) / rows); }

template <int DK, int DV, int R>
cudaError_t forward(const WindowArgs& p, cudaStream_t stream) {
  constexpr int kRows = kWarps * R;
  return run(window_fwd_kernel<DK, DV, R>, total<DK, DV, R>(kFwdRest<DK, DV, R>), row_tiles(p, kRows, p.H), stream, p);
}

template <int DK, int DV, int R>
cudaError_t dq_pass(const WindowArgs& p, cudaStream_t stream) {
  constexpr int kRows = kWarps * R;
  return run(window_dq_kernel<DK, DV, R>, total<DK, DV, R>(kDqRest<DK, DV, R>), row_tiles(p, kRows, p.H), stream, p);
}

// Keys per CTA of the keys' pass, in units of the warps: 4 where 8 would leave SMs without a CTA.
int key_rows(int B, int Hkv, int L) { return (long long)B * Hkv * ((L + 8 * kWarps - 1) / (8 * kWarps)) >= kSms ? 8 : 4; }

template <int R>  // keys per warp
KeyPass cut(int B, int H, int Hkv, int L, int window, int n_sink) {
  return window::key_pass<kWarps * R, kT>(B, H, Hkv, L, window, n_sink, 1);
}

template <int DK, int DV, int R>
cudaError_t keys_pass(const WindowArgs& p, cudaStream_t stream) {
  constexpr int kRows = kWarps * R;
  KeyPass kp = cut<R>(p.B, p.H, p.Hkv, p.L, p.window, p.n_sink);
  kp.part = static_cast<float*>(p.scratch) + ((size_t)p.B * p.H * p.L + 63) / 64 * 64;  // behind delta
  const int heads = p.B * p.Hkv, tiles = (p.L + kRows - 1) / kRows, cut_tiles = window::cut_tiles(kp, tiles);
  const cudaError_t e = run(window_dkdv_kernel<DK, DV, R>, total<DK, DV, R>(kKeysRest<DK, DV, R>),
                            window::key_ctas(kp, heads, tiles), stream, p, kp);
  if (e != cudaSuccess || cut_tiles == 0) return e;
  const size_t values = (size_t)heads * cut_tiles * kRows * (DK + DV);
  window_sum_parts_kernel<<<(unsigned)((values + 255) / 256), 256, 0, stream>>>(p, kp, cut_tiles, kRows, DK, DV);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t backward(const WindowArgs& p, cudaStream_t stream) {
  const cudaError_t e = row_tiles(p, 8 * kWarps, p.H) >= kSms ? dq_pass<DK, DV, 8>(p, stream) : dq_pass<DK, DV, 4>(p, stream);
  if (e != cudaSuccess) return e;
  return key_rows(p.B, p.Hkv, p.L) == 8 ? keys_pass<DK, DV, 8>(p, stream) : keys_pass<DK, DV, 4>(p, stream);
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
  return for_dim(dk, [&](auto k) {
    return for_dim(dv, [&](auto v) {
      return row_tiles(p, 8 * kWarps, p.H) >= kSms ? forward<k(), v(), 8>(p, stream) : forward<k(), v(), 4>(p, stream);
    });
  });
}

size_t window_bwd_scratch_bytes(int B, int H, int Hkv, int L, int dk, int dv, int window, int n_sink) {
  const int w = window < L ? window : L, s = n_sink < L ? n_sink : L, rows = key_rows(B, Hkv, L) * kWarps;
  const KeyPass kp = rows == 8 * kWarps ? cut<8>(B, H, Hkv, L, w, s) : cut<4>(B, H, Hkv, L, w, s);
  const size_t slots = (size_t)window::cut_ctas(kp, (long long)B * Hkv, (L + rows - 1) / rows);
  return (((size_t)B * H * L + 63) / 64 * 64 + slots * rows * (dk + dv)) * sizeof(float);
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
