// Backward of the windowed attention on the sm_100a tensor cores: bf16, d_k = d_v = 64 or 128.
//
//   P = exp2(S scale log2(e) - lse log2(e)),  dP = dO v^T,  dS = P (dP - delta),  delta = dO . o per query,
//   dv = P^T dO,  dk = scale dS^T q,  dq = scale dS k.
//
// Two passes over the visible tile pairs, each with its accumulators in TMEM for the whole walk: one CTA per 128 keys
// for dk and dv, one per 128 queries for dq.  Computing S and dP twice (7 products per pair instead of 5) leaves every
// sum in one CTA in a fixed order: no atomics, no fp32 dq in memory, gradients equal from run to run.  In both passes
// the weights go from registers to TMEM as the A operand of the next product and never to shared memory:
//
//   keys:    S^T = k q^T and dP^T = v dO^T have the key on the TMEM lane, so P^T and dS^T lie as dv += P^T dO and
//            dk += dS^T q need them.  TMEM: S^T, dP^T (128 columns each), dv, dk (d each); the weights overlay the scores.
//   queries: S and dP have the query on the lane; dq += dS k.  S is free as soon as it is in registers, so the next
//            tile's S and dP (two buffers) run while this tile's dS is made.
//
// P and dS are rounded to bf16 for their product (the other operand's type; 2^-8 of a weight at most), and so is a dO that
// comes as fp32; the sums are fp32.
// A warpgroup takes half of a tile's columns: thread = (lane, half).  One load warp (TMA rings), one warp whose first
// lane issues the products.  Rows behind a sequence's end are zeroed in shared memory.
//
// Key tiles may be cut into parts (window::key_pass); a part's slot: [2 (dv, dk), 128, D].
#include "window_tc.cuh"

namespace kdn {

namespace {

using namespace window;

template <int D>
struct Smem {
  static constexpr int kTile = (D / 64) * kPanel;
  static constexpr int kFixed = 0;                 // the two tiles a CTA keeps
  static constexpr int kLong = 2 * kTile;          // the walked tiles of two products, kSlots of them
  static constexpr int kShort = 5 * kTile;         // the other walked tiles, two of them
  static constexpr int kTotal = 7 * kTile;
};
// A tile that two products use (q in the keys' pass, k in the queries') leaves its slot only with the second, just before
// the tile two steps on is wanted: with two slots every step waited about 1500 cycles for that copy.  A third one: 2
// sequences of 4096, 16 heads on 4, d 128, window 1024, backward 298 -> 271 us; one of 8192 without a window 1146 -> 1004.
constexpr unsigned kSlots = 3;

// ------------------------------------------------------------------------------------------ per-query scalars
// rows[token] = (-lse log2(e), -delta), and dO as bf16 where it came as fp32.  D / 8 lanes per token.
template <int D>
__global__ void __launch_bounds__(256) window_rows_kernel(WindowArgs p, float2* rows, __nv_bfloat16* dO16) {
  constexpr int kLanes = D / 8;
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x, row = e / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (e == 0) *p.status = 0;  // nothing of this call has raised it yet
  bool live = row < (size_t)p.B * p.H * p.L;
  if (live && p.lens != nullptr) {
    const size_t head = row / p.L;
    live = static_cast<int>(row - head * p.L) < window::seq_len(p, static_cast<int>(head / p.H));
  }
  float x = 0.f;
  if (live) {
    float o[8], g[8];
    const size_t at = row * D + 8 * lane;
    if (p.out_dtype == kBF16) {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o) + at);
      const uint4 c = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dO) + at);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(aw[i] << 16), o[2 * i + 1] = __uint_as_float(aw[i] & 0xffff0000u);
        g[2 * i] = __uint_as_float(cw[i] << 16), g[2 * i + 1] = __uint_as_float(cw[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.o) + at + i);
        const float4 c = *reinterpret_cast<const float4*>(static_cast<const float*>(p.dO) + at + i);
        o[i] = a.x, o[i + 1] = a.y, o[i + 2] = a.z, o[i + 3] = a.w;
        g[i] = c.x, g[i + 1] = c.y, g[i + 2] = c.z, g[i + 3] = c.w;
      }
      *reinterpret_cast<uint4*>(dO16 + at) = pack8_bf16(g, 1.f);  // an operand of two bf16 products
      // delta from the same dO as dP: with the unrounded one P (dP - delta) would not add up to zero along a row.  Error of
      // dq against rounding the exact one, windows of 2 to 16 keys: 1.9 to 2.4; this way 1.66 to 1.76 for every window
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = __bfloat162float(__float2bfloat16_rn(g[i]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x = fmaf(o[i], g[i], x);
  }
#pragma unroll
  for (int i = kLanes / 2; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
  if (live && lane == 0) rows[row] = make_float2(-p.lse[row] * kLog2e, -x);
}

// ------------------------------------------------------------------------------------------ dk, dv
// What a thread (half 0: dv, 1: dk; key) leaves where a wait gave up: NaN in its row of the gradient, or in its row of the
// part's slot, which makes the joined row NaN.
template <int D>
__host__ __device__ void mark_key(const WindowArgs& p, const KeyPass& kp, int parts, unsigned slot, int len, int half, int key) {
  const int j = kp.tile * kT + key;
  if (parts > 1) {
    fill_words(kp.part, (((size_t)slot * 2 + half) * kT + key) * D * 4, 4 * D, nan_word(kF32));
  } else if (j < len) {
    fill_words(half == 0 ? p.dv : p.dk, ((size_t)kp.head * p.L + j) * 2 * D, 2 * D, nan_word(kBF16));
  }
}

struct DkdvState {          // behind the tiles in shared memory: with them it fills the 227 KB of a block
  float rows[2][2][kT];     // -lse log2(e), -delta
  uint64_t kv_full, q_full[kSlots], q_empty[kSlots], do_full[2], do_empty[2], rows_full[2], s_ready, p_ready, dp_ready, ds_ready, done;
  uint32_t tmem_base;
};
template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    window_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, WindowArgs p,
                          const float2* rows, KeyPass kp) {
  using S = Smem<D>;
  constexpr int kNP = D / 64;
  extern __shared__ __align__(1024) uint8_t sm[];
  DkdvState& st = *reinterpret_cast<DkdvState*>(sm + S::kTotal);
  auto& rows_s = st.rows;
  uint64_t &kv_full = st.kv_full, &s_ready = st.s_ready, &p_ready = st.p_ready, &dp_ready = st.dp_ready, &ds_ready = st.ds_ready,
           &done = st.done;
  uint64_t *q_full = st.q_full, *q_empty = st.q_empty, *do_full = st.do_full, *do_empty = st.do_empty, *rows_full = st.rows_full;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.H / p.Hkv, tiles = (p.L + kT - 1) / kT, bh = p.B * p.Hkv;
  int part;
  const int parts = window::key_tile_of(kp, bh, tiles, blockIdx.x, part);
  const int tile = kp.tile, kvh = kp.head % p.Hkv, b = kp.head / p.Hkv;
  const int len = window::seq_len(p, b), j0 = tile * kT;
  if (p.zero_rest && part == 0 && j0 + kT > len) {
    const size_t row0 = (size_t)(b * p.Hkv + kvh) * p.L;
    zero_tile(p.dk, row0, 2 * D, j0, len, p.L, tid, kTcThreads);
    zero_tile(p.dv, row0, 2 * D, j0, len, p.L, tid, kTcThreads);
  }
  if (j0 >= len) return;
  if (sm100::smem_u32(sm) & 1023) {  // never seen; the tiles' layout wants it and there is no room to align them here
    raise_status(p.status, kStatusTimeout);
    if (tid < 2 * kT) mark_key<D>(p, kp, parts, blockIdx.x, len, tid / kT, tid % kT);
    return;
  }
  int lo, hi;
  window::query_tiles<kT>(j0, min(j0 + kT, len) - 1, len, p.window, p.n_sink, lo, hi);
  const int per = hi - lo, all = per * G;  // (head of the group, query tile), query tiles fastest
  const int first = parts > 1 ? (int)((long long)all * part / parts) : 0;
  const int n = (parts > 1 ? (int)((long long)all * (part + 1) / parts) : all) - first;

  if (tid == 0) {
    sm100::mbar_init(&kv_full, 1);
    for (int i = 0; i < (int)kSlots; ++i) sm100::mbar_init(&q_full[i], 1), sm100::mbar_init(&q_empty[i], 1);
    for (int i = 0; i < 2; ++i)
      sm100::mbar_init(&do_full[i], 1), sm100::mbar_init(&do_empty[i], 1), sm100::mbar_init(&rows_full[i], 1);
    sm100::mbar_init(&s_ready, 1), sm100::mbar_init(&p_ready, 8);
    sm100::mbar_init(&dp_ready, 1), sm100::mbar_init(&ds_ready, 8);
    sm100::mbar_init(&done, 1);
    sm100::fence_mbar_init();
  }
  if (warp == 9) {
    sm100::tmem_alloc(&st.tmem_base, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = st.tmem_base;
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + D;
  bool fine = true;

  if (warp == 8) {
    // ------------------------------------------------------------------------------------ loads
    if (lane == 0 && n > 0) {
      sm100::prefetch_tmap(&tm_q), sm100::prefetch_tmap(&tm_do);
      sm100::mbar_arrive_expect_tx(&kv_full, 2 * S::kTile);
      load_tile<kNP>(sm + S::kFixed, &tm_k, &kv_full, j0, b * p.Hkv + kvh);
      load_tile<kNP>(sm + S::kFixed + S::kTile, &tm_v, &kv_full, j0, b * p.Hkv + kvh);
    }
    int it = 0;
    bool q_sent = false, do_sent = false;
    for (; it < n; ++it) {
      const int slot = it & 1, round = it >> 1, qslot = it % kSlots, qround = it / kSlots, item = first + it;
      const int row = b * p.H + kvh * G + item / per, t0 = (lo + item % per) * kT;
      q_sent = do_sent = false;
      if (qround > 0) fine = warp_wait(&q_empty[qslot], (qround - 1) & 1);
      if (!fine) break;
      if (lane == 0) {
        sm100::mbar_arrive_expect_tx(&q_full[qslot], S::kTile);
        load_tile<kNP>(sm + S::kLong + qslot * S::kTile, &tm_q, &q_full[qslot], t0, row);
      }
      q_sent = true;
      float2 v[kT / 32];  // the rows' scalars; behind the end -lse = -inf makes every weight zero
#pragma unroll
      for (int u = 0; u < kT / 32; ++u) {
        const int r = lane + 32 * u;
        v[u] = t0 + r < len ? rows[(size_t)row * p.L + t0 + r] : make_float2(-INFINITY, 0.f);
      }
      if (round > 0) fine = warp_wait(&do_empty[slot], (round - 1) & 1);
      if (!fine) break;
      if (lane == 0) {
        sm100::mbar_arrive_expect_tx(&do_full[slot], S::kTile);
        load_tile<kNP>(sm + S::kShort + slot * S::kTile, &tm_do, &do_full[slot], t0, row);
      }
      do_sent = true;
      // dK(it - 2) has ended, and with it every read of that tile's scalars
      if (it > 1) fine = warp_wait(&q_empty[(it - 2) % kSlots], ((it - 2) / kSlots) & 1);
      if (!fine) break;
#pragma unroll
      for (int u = 0; u < kT / 32; ++u) rows_s[slot][0][lane + 32 * u] = v[u].x, rows_s[slot][1][lane + 32 * u] = v[u].y;
      warp_arrive(&rows_full[slot]);
    }
    if (!fine) {  // nothing of this CTA may be in flight when it ends
      sm100::mbar_wait_bounded(&kv_full, 0, kWaitCycles);
      for (int back = it > 2 ? it - 2 : 0; back <= it && back < n; ++back) {
        if (back < it || q_sent) sm100::mbar_wait_bounded(&q_full[back % kSlots], (back / kSlots) & 1, kWaitCycles);
        if (back < it || do_sent) sm100::mbar_wait_bounded(&do_full[back & 1], (back >> 1) & 1, kWaitCycles);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------------------------ products
    const uint32_t k_addr = sm100::smem_u32(sm + S::kFixed), v_addr = k_addr + S::kTile;
    const uint32_t ring_q = sm100::smem_u32(sm + S::kLong), ring_do = sm100::smem_u32(sm + S::kShort);
    auto q_of = [&](int it) { return ring_q + it % kSlots * S::kTile; };
    auto do_of = [&](int it) { return ring_do + (it & 1) * S::kTile; };
    auto end_of = [&](int it) { return len - (lo + (first + it) % per) * kT; };  // rows of this tile inside the sequence
    auto issue_s = [&](int it) {
      if (end_of(it) < kT) zero_rows<kNP>(sm + S::kLong + it % kSlots * S::kTile, end_of(it), lane);
      if (lane == 0) mma_rows<D>(t_s, rows_desc(k_addr), rows_desc(q_of(it))), sm100::mma_commit(&s_ready);
    };
    auto issue_dp = [&](int it) {
      if (end_of(it) < kT) zero_rows<kNP>(sm + S::kShort + (it & 1) * S::kTile, end_of(it), lane);
      if (lane == 0) mma_rows<D>(t_dp, rows_desc(v_addr), rows_desc(do_of(it))), sm100::mma_commit(&dp_ready);
    };
    if (n > 0) {
      fine = warp_wait(&kv_full, 0) && warp_wait(&q_full[0], 0) && warp_wait(&do_full[0], 0);
      if (fine) issue_s(0), issue_dp(0);
    }
    for (int it = 0; it < n && fine; ++it) {
      const int slot = it & 1, next = (it + 1) & 1, next_round = (it + 1) >> 1;
      fine = warp_wait(&p_ready, it & 1);
      if (!fine) break;
      sm100::tc_fence_after();
      if (lane == 0) {
        mma_weights<D>(t_dv, t_s, 64, cols_desc(do_of(it)), it > 0);
        sm100::mma_commit(&do_empty[slot]);
      }
      if (it + 1 < n) {
        fine = warp_wait(&q_full[(it + 1) % kSlots], ((it + 1) / kSlots) & 1);
        if (!fine) break;
        issue_s(it + 1);
      }
      fine = warp_wait(&ds_ready, it & 1);
      if (!fine) break;
      sm100::tc_fence_after();
      if (lane == 0) {
        mma_weights<D>(t_dk, t_dp, 64, cols_desc(q_of(it)), it > 0);
        sm100::mma_commit(&q_empty[it % kSlots]);
      }
      if (it + 1 < n) {
        fine = warp_wait(&do_full[next], next_round & 1);
        if (!fine) break;
        issue_dp(it + 1);
      }
    }
    if (lane == 0) {
      sm100::mma_commit(&done);
      if (!fine) sm100::mbar_wait_bounded(&done, 0, kWaitCycles);
    }
  } else {
    // ------------------------------------------------------------------------------------ weights
    const int half = warp >> 2, key = tid & 127, j = j0 + key;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float2 c2 = make_float2(p.scale * kLog2e, p.scale * kLog2e);
    const int j_first = j0 + 32 * (warp & 3), j_last = j_first + 31;
    const bool sink = j < p.n_sink;
    for (int it = 0; it < n; ++it) {
      const int t0 = (lo + (first + it) % per) * kT + 64 * half;  // this half's first query
      fine = warp_wait(&rows_full[it & 1], (it >> 1) & 1) && warp_wait(&s_ready, it & 1);  // the row scalars and S^T
      if (!fine) break;
      sm100::tc_fence_after();
      float s[2][32];
      sm100::tmem_ld32(t_s + lanes + 64 * half, s[0]);
      sm100::tmem_ld32(t_s + lanes + 64 * half + 32, s[1]);
      sm100::tmem_wait_ld();
      const float4* ls = reinterpret_cast<const float4*>(&rows_s[it & 1][0][64 * half]);  // four queries a word
      const float4* ds = reinterpret_cast<const float4*>(&rows_s[it & 1][1][64 * half]);
      const bool all_seen = t0 >= j_last && (t0 + 63 - j_first < p.window || j_last < p.n_sink);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 r = ls[8 * u + e / 4];
          const float2 x = fma2(make_float2(s[u][e], s[u][e + 1]), c2, make_float2(r.x, r.y));
          const float2 y = fma2(make_float2(s[u][e + 2], s[u][e + 3]), c2, make_float2(r.z, r.w));
          s[u][e] = exp2_fast(x.x), s[u][e + 1] = exp2_fast(x.y), s[u][e + 2] = exp2_fast(y.x), s[u][e + 3] = exp2_fast(y.y);
        }
      if (!all_seen) {  // query t sees key j: t >= j and (t < j + window or a sink)
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // 32 queries: all of them see the warp's keys, or some do
          const int q0 = t0 + 32 * u;
          if (q0 >= j_last && (q0 + 31 - j_first < p.window || j_last < p.n_sink)) continue;
          const uint32_t seen = seeing_bits(j - q0, p.window, sink);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(seen >> e & 1u)) s[u][e] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __uint_as_float(pack_bf16(s[u][2 * e], s[u][2 * e + 1]));
        sm100::tmem_st16(t_s + lanes + 64 * half + 16 * u, w);
      }
      sm100::tmem_wait_st();
      sm100::tc_fence_before();
      warp_arrive(&p_ready);
      fine = warp_wait(&dp_ready, it & 1);
      if (!fine) break;
      sm100::tc_fence_after();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float dp[32], w[16];
        sm100::tmem_ld32(t_dp + lanes + 64 * half + 32 * u, dp);
        sm100::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 r = ds[8 * u + e / 4];
          const float2 x = mul2(make_float2(s[u][e], s[u][e + 1]), add2(make_float2(dp[e], dp[e + 1]), make_float2(r.x, r.y)));
          const float2 y = mul2(make_float2(s[u][e + 2], s[u][e + 3]), add2(make_float2(dp[e + 2], dp[e + 3]), make_float2(r.z, r.w)));
          w[e / 2] = __uint_as_float(pack_bf16(x.x, x.y)), w[e / 2 + 1] = __uint_as_float(pack_bf16(y.x, y.y));
        }
        sm100::tmem_st16(t_dp + lanes + 64 * half + 16 * u, w);
      }
      sm100::tmem_wait_st();
      sm100::tc_fence_before();
      warp_arrive(&ds_ready);
    }
    if (fine) {
      fine = warp_wait(&done, 0);
      sm100::tc_fence_after();
    }
    if (fine) {  // half 0 writes dv, half 1 dk
      const uint32_t t_out = (half == 0 ? t_dv : t_dk) + lanes;
      const float f = half == 0 ? 1.f : p.scale;
      const size_t at = ((size_t)(b * p.Hkv + kvh) * p.L + j) * D;
      float* cut_out = kp.part + ((size_t)blockIdx.x * 2 + half) * kT * D + key * D;
      const bool wide = is_wide(half == 0 ? p.dv : p.dk);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(half == 0 ? p.dv : p.dk) + at;
#pragma unroll 1
      for (int u = 0; u < D; u += 32) {
        float a[32];
        sm100::tmem_ld32(t_out + u, a);
        sm100::tmem_wait_ld();
        if (n == 0) {  // a part without a tile: nothing was added
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = 0.f;
        }
        if (parts > 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(cut_out + u + 4 * e) = make_float4(a[4 * e] * f, a[4 * e + 1] * f, a[4 * e + 2] * f, a[4 * e + 3] * f);
        } else if (j < len) {
#pragma unroll
          for (int e = 0; e < 32; e += 16) store32(out + u + e, pack8_bf16(a + e, f), pack8_bf16(a + e + 8, f), wide);
        }
        __syncwarp();
      }
    }
    if (!fine) mark_key<D>(p, kp, parts, blockIdx.x, len, half, key);
  }
  if (!fine) raise_status(p.status, kStatusTimeout);
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 9) sm100::tmem_dealloc(tmem, 512);
}

// The cut tiles' parts, added in their order; a thread has 8 consecutive values.
template <int D>
__global__ void __launch_bounds__(256) window_join_kernel(WindowArgs p, KeyPass kp, int cut) {
  constexpr int kWords = 2 * kT * D / 8;
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t which = e / kWords;  // (sequence, k/v head, tile)
  if (which >= (size_t)p.B * p.Hkv * cut) return;
  const int w = static_cast<int>(e % kWords), half = w / (kT * D / 8), key = w / (D / 8) % kT, c = w % (D / 8) * 8;
  const int tile = static_cast<int>(which % cut);
  const size_t head = which / cut;
  const int j = tile * kT + key;
  if (j >= window::seq_len(p, static_cast<int>(head / p.Hkv))) return;
  size_t slot;
  const int parts = window::parts_of(kp, p.B * p.Hkv, (p.L + kT - 1) / kT, head, tile, slot);
  const float* from = kp.part + slot * 2 * kT * D + (half * kT + key) * D + c;
  float a[8] = {};
  for (int i = 0; i < parts; ++i) {
    const float4 u = *reinterpret_cast<const float4*>(from + (size_t)i * 2 * kT * D);
    const float4 v = *reinterpret_cast<const float4*>(from + (size_t)i * 2 * kT * D + 4);
    a[0] += u.x, a[1] += u.y, a[2] += u.z, a[3] += u.w, a[4] += v.x, a[5] += v.y, a[6] += v.z, a[7] += v.w;
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(half == 0 ? p.dv : p.dk) + (head * p.L + j) * D + c) = pack8_bf16(a, 1.f);
}

// ------------------------------------------------------------------------------------------ dq
// One CTA per SM takes work after work (a query tile of a head), the longest first.
struct QueryPass {
  unsigned works;
  int tiles;
  Divisor group, kv_heads, batch;
};
inline QueryPass query_pass(int B, int H, int Hkv, int L) {
  const int tiles = (L + kT - 1) / kT;
  return QueryPass{(unsigned)((long long)B * H * tiles), tiles, make_divisor(H / Hkv), make_divisor(Hkv), make_divisor(B)};
}
struct QueryWork {
  int b, kvh, qrow, t0, len, n;  // n = 0: nothing to do
  int before;                    // key tiles of a first sweep: 0 or n
  KeyTiles kt;
};
__host__ __device__ __forceinline__ QueryWork query_work(const WindowArgs& p, const QueryPass& qp, unsigned x) {
  unsigned g, kvh, b;
  x = qp.group.div(x, g);
  x = qp.kv_heads.div(x, kvh);
  x = qp.batch.div(x, b);
  QueryWork w;
  w.b = b, w.kvh = kvh, w.qrow = b * p.H + kvh * qp.group.d + g;
  w.t0 = (qp.tiles - 1 - static_cast<int>(x)) * kT;
  w.len = window::seq_len(p, b);
  w.kt = window::key_tiles<kT>(w.t0, min(w.t0 + kT, w.len) - 1, p.window, p.n_sink);
  w.n = w.t0 < w.len ? w.kt.count() : 0;
  w.before = window::exact_delta<kT>(p, w.kt, w.t0, true) ? w.n : 0;
  return w;
}
// After a wait of a thread (half of the columns, row) gave up in round r: its part of that work's dq and of all later ones'.
template <int D>
__host__ __device__ void mark_queries(const WindowArgs& p, const QueryPass& qp, unsigned r, unsigned cta, unsigned ctas, int half, int row) {
  for (; r * ctas < qp.works; ++r) {
    const unsigned x = nth_work(r, cta, ctas);
    if (x >= qp.works) continue;
    const QueryWork w = query_work(p, qp, x);
    const int t = w.t0 + row;
    if (t >= p.L || (t >= w.len && !p.zero_rest)) continue;
    fill_words(p.dq, ((size_t)w.qrow * p.L + t) * 2 * D + half * D, D, t < w.len ? nan_word(kBF16) : 0u);
  }
}

// A work may take two sweeps over its key tiles, the first for delta_t = sum_j P_tj dP_tj in fp32, which also replaces the
// value from the rounded o for the keys' pass (window::exact_delta).
template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    window_dq_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, WindowArgs p,
                        float2* rows, QueryPass qp) {
  using S = Smem<D>;
  constexpr int kNP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t q_full, q_empty, k_full[kSlots], k_empty[kSlots], v_full[2], v_empty[2], s_ready, s_free, dp_ready[2], ds_ready[2], delta_ready, done, last;
  __shared__ uint32_t tmem_base;
  __shared__ float delta_s[2][kT];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    sm100::mbar_init(&q_full, 1), sm100::mbar_init(&q_empty, 1);
    for (int i = 0; i < (int)kSlots; ++i) sm100::mbar_init(&k_full[i], 1), sm100::mbar_init(&k_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&v_full[i], 1), sm100::mbar_init(&v_empty[i], 1);
      sm100::mbar_init(&dp_ready[i], 1), sm100::mbar_init(&ds_ready[i], 8);
    }
    sm100::mbar_init(&s_ready, 1), sm100::mbar_init(&s_free, 8), sm100::mbar_init(&delta_ready, 8);
    sm100::mbar_init(&done, 1), sm100::mbar_init(&last, 1);
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
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dq = tmem + 384;  // dP: two buffers of 128 columns
  bool fine = true;

  if (warp == 8) {
    // ------------------------------------------------------------------------------------ loads
    if (lane == 0) {
      sm100::prefetch_tmap(&tm_q), sm100::prefetch_tmap(&tm_do), sm100::prefetch_tmap(&tm_k), sm100::prefetch_tmap(&tm_v);
      unsigned nq = 0, nk = 0, nv = 0;  // copies issued so far
      for (unsigned r = 0; r * gridDim.x < qp.works && fine; ++r) {
        const unsigned x = nth_work(r, blockIdx.x, gridDim.x);
        if (x >= qp.works) continue;
        const QueryWork w = query_work(p, qp, x);
        const int row = w.b * p.Hkv + w.kvh;
        const int steps = w.before + w.n;
        for (int it = 0; it < steps; ++it) {
          const unsigned kslot = nk % kSlots, slot = nv & 1;
          const int j0 = w.kt.walk(it < w.n ? it : it - w.n) * kT;
          if (nk >= kSlots) fine = sm100::mbar_wait_bounded(&k_empty[kslot], (nk / kSlots - 1) & 1, kWaitCycles);
          if (!fine) break;
          sm100::mbar_arrive_expect_tx(&k_full[kslot], S::kTile);
          load_tile<kNP>(sm + S::kLong + kslot * S::kTile, &tm_k, &k_full[kslot], j0, row);
          ++nk;
          if (nv > 1) fine = sm100::mbar_wait_bounded(&v_empty[slot], ((nv >> 1) - 1) & 1, kWaitCycles);
          if (!fine) break;
          sm100::mbar_arrive_expect_tx(&v_full[slot], S::kTile);
          load_tile<kNP>(sm + S::kShort + slot * S::kTile, &tm_v, &v_full[slot], j0, row);
          ++nv;
          if (it == 0) {
            if (nq > 0) fine = sm100::mbar_wait_bounded(&q_empty, (nq - 1) & 1, kWaitCycles);
            if (!fine) break;
            sm100::mbar_arrive_expect_tx(&q_full, 2 * S::kTile);
            load_tile<kNP>(sm + S::kFixed, &tm_q, &q_full, w.t0, w.qrow);
            load_tile<kNP>(sm + S::kFixed + S::kTile, &tm_do, &q_full, w.t0, w.qrow);
            ++nq;
          }
        }
      }
      if (!fine) {  // nothing of this CTA may be in flight when it ends
        if (nq > 0) sm100::mbar_wait_bounded(&q_full, (nq - 1) & 1, kWaitCycles);
        for (unsigned c = nk > kSlots ? nk - kSlots : 0; c < nk; ++c) sm100::mbar_wait_bounded(&k_full[c % kSlots], (c / kSlots) & 1, kWaitCycles);
        for (unsigned c = nv > 2 ? nv - 2 : 0; c < nv; ++c) sm100::mbar_wait_bounded(&v_full[c & 1], (c >> 1) & 1, kWaitCycles);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------------------------ products
    const uint32_t ring_k = sm100::smem_u32(sm + S::kLong), ring_v = sm100::smem_u32(sm + S::kShort);
    const uint64_t q_desc = rows_desc(sm100::smem_u32(sm + S::kFixed)), do_desc = rows_desc(sm100::smem_u32(sm + S::kFixed + S::kTile));
    unsigned c = 0, nq = 0;  // key tiles and works begun
    for (unsigned r = 0; r * gridDim.x < qp.works && fine; ++r) {
      const unsigned x = nth_work(r, blockIdx.x, gridDim.x);
      if (x >= qp.works) continue;
      const QueryWork w = query_work(p, qp, x);
      if (w.n == 0) continue;
      const int steps = w.before + w.n;
      // S and dP of the it-th step, the c-th of this CTA: S is free once step c - 1 is in registers.  k and v rows behind
      // the end are zeroed (their weights are zero).
      auto issue = [&](int it) {
        const unsigned kslot = c % kSlots, slot = c & 1;
        fine = warp_wait(&k_full[kslot], (c / kSlots) & 1) && warp_wait(&v_full[slot], (c >> 1) & 1) &&
               (c == 0 || warp_wait(&s_free, (c - 1) & 1));
        if (!fine) return;
        sm100::tc_fence_after();
        const int inside = w.len - w.kt.walk(it < w.n ? it : it - w.n) * kT;
        if (inside < kT) {
          zero_rows<kNP>(sm + S::kLong + kslot * S::kTile, inside, lane);
          zero_rows<kNP>(sm + S::kShort + slot * S::kTile, inside, lane);
        }
        if (lane == 0) {
          mma_rows<D>(t_s, q_desc, rows_desc(ring_k + kslot * S::kTile));
          sm100::mma_commit(&s_ready);
          mma_rows<D>(t_dp + 128 * slot, do_desc, rows_desc(ring_v + slot * S::kTile));
          sm100::mma_commit(&dp_ready[slot]);
          sm100::mma_commit(&v_empty[slot]);
          if (it + 1 == steps) sm100::mma_commit(&q_empty);
        }
        ++c;
      };
      fine = warp_wait(&q_full, nq & 1);
      ++nq;
      if (fine) issue(0);
      for (int it = 0; it < steps && fine; ++it) {
        const unsigned mine = c - 1, kslot = mine % kSlots, slot = mine & 1;  // step ``it``
        if (it + 1 < steps) issue(it + 1);
        if (!fine) break;
        fine = warp_wait(&ds_ready[slot], (mine >> 1) & 1);
        if (!fine) break;
        sm100::tc_fence_after();
        if (lane == 0) {
          const int sweep = it - w.before;  // >= 0: the tile of the sweep that adds up dq
          if (sweep >= 0) mma_weights<D>(t_dq, t_dp + 128 * slot, 64, cols_desc(ring_k + kslot * S::kTile), sweep > 0);
          sm100::mma_commit(&k_empty[kslot]);
          if (it + 1 == steps) sm100::mma_commit(&done);
        }
      }
    }
    if (!fine && lane == 0) {  // the products in flight read shared memory and write TMEM
      sm100::mma_commit(&last);
      sm100::mbar_wait_bounded(&last, 0, kWaitCycles);
    }
  } else {
    // ------------------------------------------------------------------------------------ weights
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float2 c2 = make_float2(p.scale * kLog2e, p.scale * kLog2e);
    const bool wide = is_wide(p.dq);
    unsigned c = 0, works = 0, sweeps = 0;
    unsigned r = 0;
    for (; r * gridDim.x < qp.works; ++r) {
      const unsigned x = nth_work(r, blockIdx.x, gridDim.x);
      if (x >= qp.works) continue;
      const QueryWork w = query_work(p, qp, x);
      if (p.zero_rest && w.t0 + kT > w.len) zero_tile(p.dq, (size_t)w.qrow * p.L, 2 * D, w.t0, w.len, p.L, tid, 256);
      if (w.n == 0) continue;
      const int t = w.t0 + (tid & 127);
      const int w_first = w.t0 + 32 * (warp & 3), w_last = w_first + 31;
      const float2 row = t < w.len ? rows[(size_t)w.qrow * p.L + t] : make_float2(0.f, 0.f);
      const float2 l2 = make_float2(row.x, row.x);
      const bool one = window::sees_one_key(p, t);
      float2 d2 = make_float2(row.y, row.y), sum = make_float2(0.f, 0.f);
      const int steps = w.before + w.n;
      for (int it = 0; it < steps; ++it, ++c) {
        const int j0 = w.kt.walk(it < w.n ? it : it - w.n) * kT + 64 * half;
        fine = warp_wait(&s_ready, c & 1);
        if (!fine) break;
        sm100::tc_fence_after();
        float s[2][32];
        sm100::tmem_ld32(t_s + lanes + 64 * half, s[0]);
        sm100::tmem_ld32(t_s + lanes + 64 * half + 32, s[1]);
        sm100::tmem_wait_ld();
        sm100::tc_fence_before();
        warp_arrive(&s_free);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = fma2(make_float2(s[u][e], s[u][e + 1]), c2, l2);
            s[u][e] = exp2_fast(y.x), s[u][e + 1] = exp2_fast(y.y);
          }
        const bool all_seen = j0 + 63 <= w_first && (w_last - j0 < p.window || j0 + 64 <= p.n_sink);
        if (!all_seen) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // 32 keys: all of the warp's rows see them, or some do
            const int k0 = j0 + 32 * u;
            if (k0 + 31 <= w_first && (w_last - k0 < p.window || k0 + 32 <= p.n_sink)) continue;
            const uint32_t seen = seen_bits(t - k0, p.window, p.n_sink - k0);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              s[u][e] = !(seen >> e & 1u) ? 0.f : one ? 1.f : s[u][e];
          }
        }
        fine = warp_wait(&dp_ready[c & 1], (c >> 1) & 1);
        if (!fine) break;
        sm100::tc_fence_after();
        const uint32_t t_mine = t_dp + 128 * (c & 1) + lanes + 64 * half;
        if (it < w.before) {  // the first sweep
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float dp[32];
            sm100::tmem_ld32(t_mine + 32 * u, dp);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              sum = fma2(make_float2(s[u][e], s[u][e + 1]), make_float2(dp[e], dp[e + 1]), sum);
          }
          sm100::tc_fence_before();
          warp_arrive(&ds_ready[c & 1]);
          if (it + 1 == w.n) {  // the row's other half of the columns is the other warpgroup's
            // Written again in this CTA's next first sweep only, behind a step whose scores wait (s_free) until all eight
            // warps have gone on from here.
            delta_s[half][tid & 127] = sum.x + sum.y;
            warp_arrive(&delta_ready);
            fine = warp_wait(&delta_ready, sweeps & 1);
            if (!fine) break;
            ++sweeps;
            const float delta = delta_s[0][tid & 127] + delta_s[1][tid & 127];
            d2 = make_float2(-delta, -delta);
            if (half == 0 && t < w.len) rows[(size_t)w.qrow * p.L + t].y = -delta;
          }
          continue;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float dp[32], q[16];
          sm100::tmem_ld32(t_mine + 32 * u, dp);
          sm100::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = mul2(make_float2(s[u][e], s[u][e + 1]), add2(make_float2(dp[e], dp[e + 1]), d2));
            q[e / 2] = __uint_as_float(pack_bf16(y.x, y.y));
          }
          sm100::tmem_st16(t_mine + 16 * u, q);
        }
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        warp_arrive(&ds_ready[c & 1]);
      }
      if (fine) {
        fine = warp_wait(&done, works & 1);
        ++works;
        sm100::tc_fence_after();
      }
      if (!fine) break;
      // each half writes half of the columns
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dq) + ((size_t)w.qrow * p.L + t) * D + half * (D / 2);
#pragma unroll 1
      for (int u = 0; u < D / 2; u += 32) {
        float a[32];
        sm100::tmem_ld32(t_dq + lanes + half * (D / 2) + u, a);
        sm100::tmem_wait_ld();
        if (t < w.len) {
#pragma unroll
          for (int e = 0; e < 32; e += 16) store32(out + u + e, pack8_bf16(a + e, p.scale), pack8_bf16(a + e + 8, p.scale), wide);
        }
        __syncwarp();
      }
      sm100::tc_fence_before();  // dq is read: the next work's first product follows this warp's next arrival
    }
    if (!fine) mark_queries<D>(p, qp, r, blockIdx.x, gridDim.x, half, tid & 127);
  }
  if (!fine) raise_status(p.status, kStatusTimeout);
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 9) sm100::tmem_dealloc(tmem, 512);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Query tiles of a part where every key tile is cut: 1 and 2 measure the same, with 4 short sequences lose (1 of 200, 3
// heads on 1, d 128: 47.7 against 38.7 us).
constexpr int kLeast = 2;
struct Layout {
  size_t rows, dO, part, end;  // byte offsets in the scratch
};
KeyPass cut(int B, int H, int Hkv, int L, int window, int n_sink) {
  return window::key_pass<kT, kT>(B, H, Hkv, L, window, n_sink, kLeast);
}
Layout layout(int B, int H, int Hkv, int L, int D, int out_dtype, const KeyPass& kp) {
  Layout l{};
  const size_t tokens = (size_t)B * H * L;
  l.rows = 0, l.dO = round256(tokens * sizeof(float2));
  l.part = l.dO + (out_dtype == kF32 ? round256(tokens * D * 2) : 0);
  l.end = l.part + (size_t)window::cut_ctas(kp, (long long)B * Hkv, (L + kT - 1) / kT) * 2 * kT * D * sizeof(float);
  return l;
}

template <int D>
cudaError_t backward(const WindowArgs& p, cudaStream_t stream) {
  KeyPass kp = cut(p.B, p.H, p.Hkv, p.L, p.window, p.n_sink);
  const Layout l = layout(p.B, p.H, p.Hkv, p.L, D, p.out_dtype, kp);
  char* scratch = static_cast<char*>(p.scratch);
  float2* rows = reinterpret_cast<float2*>(scratch + l.rows);
  __nv_bfloat16* dO16 = reinterpret_cast<__nv_bfloat16*>(scratch + l.dO);
  kp.part = reinterpret_cast<float*>(scratch + l.part);
  CUtensorMap tq, tk, tv, td;
  if (!make_bf16_tmap_rows(&tq, p.q, p.B * p.H, p.L, D, kT) || !make_bf16_tmap_rows(&tk, p.k, p.B * p.Hkv, p.L, D, kT) ||
      !make_bf16_tmap_rows(&tv, p.v, p.B * p.Hkv, p.L, D, kT) ||
      !make_bf16_tmap_rows(&td, p.out_dtype == kBF16 ? p.dO : dO16, p.B * p.H, p.L, D, kT))
    return cudaErrorInvalidValue;
  const size_t tokens = (size_t)p.B * p.H * p.L;
  window_rows_kernel<D><<<(unsigned)((tokens * (D / 8) + 255) / 256), 256, 0, stream>>>(p, rows, dO16);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem = Smem<D>::kTotal + 1024, key_smem = Smem<D>::kTotal + (int)sizeof(DkdvState), tiles = (p.L + kT - 1) / kT, bh = p.B * p.Hkv;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return cudaErrorInvalidDevice;
  e = cudaFuncSetAttribute(window_dkdv_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, key_smem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(window_dq_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long keys = window::key_ctas(kp, bh, tiles);
  const int cut_tiles = window::cut_tiles(kp, tiles);
  const QueryPass qp = query_pass(p.B, p.H, p.Hkv, p.L);
  // the queries' pass first: it may replace the rows' delta
  const unsigned ctas = qp.works < (unsigned)sms ? qp.works : (unsigned)sms;
  window_dq_tc_kernel<D><<<ctas, kTcThreads, smem, stream>>>(tq, tk, tv, td, p, rows, qp);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  window_dkdv_tc_kernel<D><<<(unsigned)keys, kTcThreads, key_smem, stream>>>(tq, tk, tv, td, p, rows, kp);
  e = cudaGetLastError();
  if (e != cudaSuccess || cut_tiles == 0) return e;
  const size_t words = (size_t)bh * cut_tiles * 2 * kT * D / 8;
  window_join_kernel<D><<<(unsigned)((words + 255) / 256), 256, 0, stream>>>(p, kp, cut_tiles);
  return cudaGetLastError();
}

}  // namespace

size_t window_bwd_tc_scratch_bytes(int B, int H, int Hkv, int L, int d, int out_dtype, int window, int n_sink) {
  return layout(B, H, Hkv, L, d, out_dtype, cut(B, H, Hkv, L, window < L ? window : L, n_sink < L ? n_sink : L)).end;
}

cudaError_t launch_window_bwd_tc(int d, const WindowArgs& p, cudaStream_t stream) {
  return d == 128 ? backward<128>(p, stream) : backward<64>(p, stream);
}

}  // namespace kdn
