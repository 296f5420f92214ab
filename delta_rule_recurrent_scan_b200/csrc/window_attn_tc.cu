// Windowed attention on the sm_100a tensor cores: bf16 q, k, v with d_k = d_v = 64 or 128.
//
//   S = q k^T (fp32, TMEM),  P = exp2(S scale log2(e) - m),  O += P v (fp32, TMEM),  o = O / sum P,
//
// one pass over the keys with the running maximum m and sum of every query row.  A CTA holds two tiles of 128 queries
// that read the same k/v head (two heads of a group where the group is even, else two neighbouring tiles of a head) and
// walks the 128-token key tiles they see:
//
//   warp 8      TMA: q once, then k and v tiles through two rings of two slots
//   warp 9      one lane issues the products: S_i of the next key tile right after O_i += P_i v of this one, so that the
//               tensor cores work on one query tile while the other's softmax runs
//   warps 0-3   softmax of query tile 0, one thread per row (its TMEM lane); warps 4-7: tile 1
//
// P (bf16, the type of v, which the product of two operands asks for; its rounding is 2^-8 of a weight at most, the
// row's sum takes the unrounded weights) goes back to TMEM over S as the A operand of the second product, so scores
// never leave the SM.  TMEM: S_0, S_1 (128 columns each), O_0, O_1 (d each).  m moves only when the row's maximum has
// grown by more than 2^8 (weights stay below 2^8, far inside fp32 and bf16): O is then multiplied in place.  The commit
// that announces S_i also covers O_i's previous product, so the row may be rescaled without another wait.
//
// v rows behind a sequence's end are set to zero in shared memory (0 times whatever memory holds there would not be 0);
// k rows behind it only reach hidden scores.
#include "window_tc.cuh"

namespace kdn {

namespace {

using namespace window;

constexpr float kSlack = 8.f;        // growth of the maximum (base 2) that weights may keep

template <int D>
struct Smem {
  static constexpr int kTile = (D / 64) * kPanel;
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kTotal = 6 * kTile;
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    window_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, WindowArgs p) {
  using S = Smem<D>;
  constexpr int kNP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_ready[2], p_ready[2], done;
  __shared__ uint32_t tmem_base;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.H / p.Hkv, tiles = (p.L + kT - 1) / kT;
  // (sequence, k/v head, query tiles from the last down, heads of the group)
  const bool heads = (G & 1) == 0;
  const int tp = heads ? tiles : (tiles + 1) / 2, gp = heads ? G / 2 : G;
  unsigned x = blockIdx.x;
  const int g = x % gp;
  x /= gp;
  const int tb = tp - 1 - static_cast<int>(x % tp);
  x /= tp;
  const int kvh = x % p.Hkv, b = x / p.Hkv;
  const int len = window::seq_len(p, b);
  int qt[2], h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) qt[i] = heads ? tb : 2 * tb + i, h[i] = kvh * G + (heads ? 2 * g + i : g);
  if (qt[0] * kT >= len) return;
  const bool two = qt[1] * kT < len;
  const KeyTiles k0 = window::key_tiles<kT>(qt[0] * kT, min(qt[0] * kT + kT, len) - 1, p.window, p.n_sink);
  KeyTiles k1 = k0, ku = k0;
  if (two) {
    k1 = window::key_tiles<kT>(qt[1] * kT, min(qt[1] * kT + kT, len) - 1, p.window, p.n_sink);
    ku.hi = k1.hi;  // tile 1 starts no earlier and ends no earlier than tile 0
  }
  const int n = ku.count();
  const int n_sinks = p.n_sink > 0 ? (p.n_sink - 1) / kT + 1 : 0;
  auto active = [&](int i, int it) {
    const int j = ku.walk(it);
    return i == 0 ? j < k0.hi : two && (j < n_sinks || j >= k1.lo);
  };

  if (tid == 0) {
    sm100::mbar_init(&q_full, 1);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&k_full[i], 1), sm100::mbar_init(&k_empty[i], 1);
      sm100::mbar_init(&v_full[i], 1), sm100::mbar_init(&v_empty[i], 1);
      sm100::mbar_init(&s_ready[i], 1), sm100::mbar_init(&p_ready[i], 128);
    }
    sm100::mbar_init(&done, 1);
    sm100::fence_mbar_init();
  }
  if (warp == 9) {
    sm100::tmem_alloc(&tmem_base, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool fine = true;

  if (warp == 8) {
    // ------------------------------------------------------------------------------------ loads
    if (lane == 0) {
      sm100::prefetch_tmap(&tm_q), sm100::prefetch_tmap(&tm_k), sm100::prefetch_tmap(&tm_v);
      const int row = b * p.Hkv + kvh;
      sm100::mbar_arrive_expect_tx(&q_full, (two ? 2 : 1) * S::kTile);
      for (int i = 0; i < (two ? 2 : 1); ++i)
        load_tile<kNP>(sm + S::kQ + i * S::kTile, &tm_q, &q_full, qt[i] * kT, b * p.H + h[i]);
      int it = 0;
      for (; it < n; ++it) {
        const int slot = it & 1, round = it >> 1, j0 = ku.walk(it) * kT;
        if (round > 0) fine = sm100::mbar_wait_bounded(&k_empty[slot], (round - 1) & 1, kWaitCycles);
        if (!fine) break;
        sm100::mbar_arrive_expect_tx(&k_full[slot], S::kTile);
        load_tile<kNP>(sm + S::kK + slot * S::kTile, &tm_k, &k_full[slot], j0, row);
        if (round > 0) fine = sm100::mbar_wait_bounded(&v_empty[slot], (round - 1) & 1, kWaitCycles);
        if (!fine) break;
        sm100::mbar_arrive_expect_tx(&v_full[slot], S::kTile);
        load_tile<kNP>(sm + S::kV + slot * S::kTile, &tm_v, &v_full[slot], j0, row);
      }
      if (!fine) {  // nothing of this CTA may be in flight when it ends
        sm100::mbar_wait_bounded(&q_full, 0, kWaitCycles);
        for (int back = it > 1 ? it - 1 : 0; back <= it && back < n; ++back) {
          sm100::mbar_wait_bounded(&k_full[back & 1], (back >> 1) & 1, kWaitCycles);
          if (back < it) sm100::mbar_wait_bounded(&v_full[back & 1], (back >> 1) & 1, kWaitCycles);
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------------------------ products
    const uint32_t q_addr = sm100::smem_u32(sm + S::kQ), k_addr = sm100::smem_u32(sm + S::kK), v_addr = sm100::smem_u32(sm + S::kV);
    auto issue_s = [&](int i, int it) {
      if (lane == 0) {
        mma_rows<D>(tmem + 128 * i, q_addr + i * S::kTile, k_addr + (it & 1) * S::kTile);
        sm100::mma_commit(&s_ready[i]);
      }
    };
    uint32_t p_phase[2] = {0, 0};
    bool begun[2] = {false, false};
    fine = warp_wait(&q_full, 0) && warp_wait(&k_full[0], 0);
    if (fine) {
      if (active(0, 0)) issue_s(0, 0);
      if (active(1, 0)) issue_s(1, 0);
      if (lane == 0) sm100::mma_commit(&k_empty[0]);
    }
    for (int it = 0; it < n && fine; ++it) {
      const int slot = it & 1, round = it >> 1, j0 = ku.walk(it) * kT;
      fine = warp_wait(&v_full[slot], round & 1);
      if (it + 1 < n) fine = fine && warp_wait(&k_full[(it + 1) & 1], ((it + 1) >> 1) & 1);
      if (!fine) break;
      if (j0 + kT > len) zero_rows<kNP>(sm + S::kV + slot * S::kTile, len - j0, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (active(i, it)) {
          fine = warp_wait(&p_ready[i], p_phase[i]);
          if (!fine) break;
          p_phase[i] ^= 1;
          sm100::tc_fence_after();
          if (lane == 0) mma_weights<D>(tmem + 256 + D * i, tmem + 128 * i, 32, v_addr + slot * S::kTile, begun[i]);
          begun[i] = true;
        }
        if (it + 1 < n && active(i, it + 1)) issue_s(i, it + 1);
      }
      if (fine && lane == 0) {
        sm100::mma_commit(&v_empty[slot]);
        if (it + 1 < n) sm100::mma_commit(&k_empty[(it + 1) & 1]);
      }
    }
    if (lane == 0) {
      sm100::mma_commit(&done);
      if (!fine) sm100::mbar_wait_bounded(&done, 0, kWaitCycles);
    }
  } else {
    // ------------------------------------------------------------------------------------ softmax
    const int i = warp >> 2, row = tid & 127;
    const int tq = i == 0 ? qt[0] : qt[1], hq = i == 0 ? h[0] : h[1];
    const int t0 = tq * kT, t = t0 + row;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lanes + 128 * i, t_o = tmem + lanes + 256 + D * i;
    const float c = p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    uint32_t phase = 0;
    const bool mine = i == 0 || two;
    const int w_first = t0 + 32 * (warp & 3), w_last = w_first + 31;  // the warp's rows
    for (int it = 0; it < n && mine; ++it) {
      if (!active(i, it)) continue;
      const int j0 = ku.walk(it) * kT;
      fine = warp_wait(&s_ready[i], phase);
      if (!fine) break;
      phase ^= 1;
      sm100::tc_fence_after();
      float s[4][32];
#pragma unroll
      for (int u = 0; u < 4; ++u) sm100::tmem_ld32(t_s + 32 * u, s[u]);
      sm100::tmem_wait_ld();
      // hidden keys: behind the query, or before its window without being a sink
      const bool all = j0 + kT - 1 <= w_first && (w_last - j0 < p.window || j0 + kT <= p.n_sink);
      if (!all) {
        const int hi = t - j0, lo = hi - p.window, sinks = p.n_sink - j0;  // visible: col <= hi, (col > lo or col < sinks)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int col = 32 * u + e;
            if (col > hi || (col <= lo && col >= sinks)) s[u][e] = -INFINITY;
          }
      }
      float top[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        top[u] = s[u][0];
#pragma unroll
        for (int e = 1; e < 32; ++e) top[u] = fmaxf(top[u], s[u][e]);
      }
      const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;  // c > 0
      // the warp rescales together when one of its rows has to
      if (__any_sync(0xffffffffu, now > m + kSlack || (m == -INFINITY && now > -INFINITY))) {
        const float next = fmaxf(m, now);
        const float f = m == -INFINITY ? 0.f : exp2_fast(m - next);
        if (__any_sync(0xffffffffu, l != 0.f)) {  // some row has weights already: O holds the products so far
          float o[32];
#pragma unroll 1
          for (int u = 0; u < D; u += 32) {
            sm100::tmem_ld32(t_o + u, o);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            sm100::tmem_st32(t_o + u, o);
          }
        }
        l *= f;
        m = next;
      }
      const float base = m == -INFINITY ? 0.f : m;  // no visible key so far: every weight is exp2(-inf) = 0
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float a = exp2_fast(fmaf(s[u][e], c, -base)), d = exp2_fast(fmaf(s[u][e + 1], c, -base));
          sum[(e >> 1) & 3] += a + d;
          w[e / 2] = __uint_as_float(pack_bf16(a, d));
        }
        sm100::tmem_st16(t_s + 16 * u, w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      sm100::tmem_wait_st();
      sm100::tc_fence_before();
      sm100::mbar_arrive(&p_ready[i]);
    }
    const size_t at = ((size_t)b * p.H + hq) * p.L + t;
    if (mine && fine) {
      fine = warp_wait(&done, 0);
      sm100::tc_fence_after();
      if (fine) {
        const float inv = 1.f / l;
        if (t < len) p.lse[at] = (m + log2f(l)) * kLn2;
#pragma unroll 1
        for (int u = 0; u < D; u += 32) {
          float o[32];
          sm100::tmem_ld32(t_o + u, o);
          sm100::tmem_wait_ld();
          if (t >= len) {
          } else if (p.out_dtype == kBF16) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at * D + u);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = pack8_bf16(o + 8 * e, inv);
          } else {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * D + u);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
          }
          __syncwarp();
        }
      }
    }
    if (mine && !fine && t < len) p.lse[at] = NAN;
  }
  if (!fine) raise_status(p.status, kStatusTimeout);
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 9) sm100::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t forward(const WindowArgs& p, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  if (!make_bf16_tmap_rows(&tq, p.q, p.B * p.H, p.L, D, kT) || !make_bf16_tmap_rows(&tk, p.k, p.B * p.Hkv, p.L, D, kT) ||
      !make_bf16_tmap_rows(&tv, p.v, p.B * p.Hkv, p.L, D, kT))
    return cudaErrorInvalidValue;
  const int G = p.H / p.Hkv, tiles = (p.L + kT - 1) / kT;
  const long long ctas = (long long)p.B * p.Hkv * (G % 2 == 0 ? (long long)tiles * (G / 2) : (long long)((tiles + 1) / 2) * G);
  const int smem = Smem<D>::kTotal + 1024;
  const cudaError_t e = cudaFuncSetAttribute(window_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  window_fwd_tc_kernel<D><<<(unsigned)ctas, kTcThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

bool window_tc_supported(int dk, int dv, int in_dtype) { return in_dtype == kBF16 && dk == dv && (dk == 64 || dk == 128); }

cudaError_t launch_window_attn_tc(int d, const WindowArgs& p, cudaStream_t stream) {
  return d == 128 ? forward<128>(p, stream) : forward<64>(p, stream);
}

}  // namespace kdn
