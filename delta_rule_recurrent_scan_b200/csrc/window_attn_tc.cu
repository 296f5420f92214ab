// Windowed attention on the sm_100a tensor cores: bf16 q, k, v with d_k = d_v = 64 or 128.
//
//   S = q k^T (fp32, TMEM),  P = exp2(S scale log2(e) - m),  O += P v (fp32, TMEM),  o = O / sum P,
//
// one pass over the keys with the running maximum m and sum of every query row.  One CTA per SM takes work after work: two
// tiles of 128 queries that read the same k/v head (two heads of a group where the group is even, else two neighbouring
// tiles of a head), walked over the 128-token key tiles they see:
//
//   warp 8      TMA: q, and k and v tiles through two rings of two slots
//   warp 9      one lane issues the products: S_i of the next key tile right after O_i += P_i v of this one, so that the
//               tensor cores work on one query tile while the other's softmax runs, and S_i of the next work while this
//               one's o is written
//   warps 0-3   softmax of query tile 0, one thread per row (its TMEM lane); warps 4-7: tile 1
//
// P (bf16, the type of v, which the product of two operands asks for; its rounding is 2^-8 of a weight at most, the
// row's sum takes the unrounded weights) goes back to TMEM over S as the A operand of the second product, so scores
// never leave the SM.  TMEM: S_0, S_1 (128 columns each), O_0, O_1 (d each).  m moves only when the row's maximum has
// grown by more than 2^8 (weights stay below 2^8, far inside fp32 and bf16): O is then multiplied in place.  The commit
// that announces S_i also covers O_i's previous product, so the row may be rescaled without another wait.
//
// A tile that a warp's rows do not all see whole is tested 32 columns at a time: only the columns that some of its rows see
// and some do not are compared.  Scaling, subtraction and sums take two values per instruction: with one warp of each
// tile per scheduler the softmax is bound by the latency of its own instructions, not by a pipe.
//
// Measured, 4 sequences of 4096, 16 heads on 4 k/v heads, d = 128, window 1024, 4 sinks: 151 us (800 TFLOP/s of visible
// pairs; the tiles hold 1.25 times as many).  198 us with one CTA per work (start and end not overlapped, works in the
// heads' order), 167 us with scalar instead of paired arithmetic, 158 us with descriptors built per product.  Without a
// window, 16384 tokens: 1216 TFLOP/s.  A tile pair then takes 3750 cycles: products 2780 (q k^T reads two operands from
// shared memory, 128 bytes a cycle, and runs at 0.6 of the rate of the other), the rest waits for a softmax to begin.
// Moving 1/8 or 1/4 of the exponentials to the fp32 pipe (polynomial) made it 1 to 9 % slower; handing P over in halves 5 %;
// 384 threads with registers moved to the softmax warps (setmaxnreg) 25 to 60 %.  Steps of 32 columns for tiles that only
// sinks make visible: no faster with sinks, 6 % slower without (the softmax warps' code got longer).
//
// A wait that gives up ends a role; the softmax warps then leave NaN in every row that they could not make (mark_rest).
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

// One work: two query tiles of a k/v head and the key tiles they see.
struct Work {
  int b, kvh, len, n, qt[2], h[2];
  bool two;
  KeyTiles k0, k1, ku;
  int n_sinks;
  // whether query tile i reads the it-th key tile
  __device__ __forceinline__ bool active(int i, int it) const {
    const int j = ku.walk(it);
    return i == 0 ? j < k0.hi : two && (j < n_sinks || j >= k1.lo);
  }
};

// The works of a call, numbered (query tiles from the last down; sequence; k/v head; heads of the group): the longest first.
struct Schedule {
  unsigned works;
  int tile_groups;   // two tiles, or the same tile of two heads
  bool heads;
  Divisor group, kv_heads, batch;
};

inline Schedule make_schedule(int B, int H, int Hkv, int L) {
  const int G = H / Hkv, tiles = (L + kT - 1) / kT;
  Schedule sch;
  sch.heads = G % 2 == 0;
  sch.tile_groups = sch.heads ? tiles : (tiles + 1) / 2;
  sch.group = make_divisor(sch.heads ? G / 2 : G), sch.kv_heads = make_divisor(Hkv), sch.batch = make_divisor(B);
  sch.works = (unsigned)((long long)B * Hkv * sch.tile_groups * sch.group.d);
  return sch;
}

// n = 0: nothing to do.
__host__ __device__ __forceinline__ Work make_work(const WindowArgs& p, const Schedule& sch, unsigned x) {
  Work w;
  unsigned g, kvh, b;
  x = sch.group.div(x, g);
  x = sch.kv_heads.div(x, kvh);
  const bool heads = sch.heads;
  const int tb = sch.tile_groups - 1 - static_cast<int>(sch.batch.div(x, b));
  w.kvh = kvh, w.b = b;
  const int G = heads ? 2 * sch.group.d : sch.group.d;
  w.len = window::seq_len(p, w.b);
#pragma unroll
  for (int i = 0; i < 2; ++i) w.qt[i] = heads ? tb : 2 * tb + i, w.h[i] = w.kvh * G + (heads ? 2 * g + i : g);
  w.two = w.qt[1] * kT < w.len;
  w.n_sinks = p.n_sink > 0 ? (p.n_sink - 1) / kT + 1 : 0;
  w.k0 = window::key_tiles<kT>(w.qt[0] * kT, min(w.qt[0] * kT + kT, w.len) - 1, p.window, p.n_sink);
  w.k1 = w.ku = w.k0;
  if (w.two) {
    w.k1 = window::key_tiles<kT>(w.qt[1] * kT, min(w.qt[1] * kT + kT, w.len) - 1, p.window, p.n_sink);
    w.ku.hi = w.k1.hi;  // tile 1 starts no earlier and ends no earlier than tile 0
  }
  w.n = w.qt[0] * kT < w.len ? w.ku.count() : 0;
  return w;
}

// After a wait of softmax group i's thread ``row`` gave up in round r: its rows of that work and of all later ones.
template <int D>
__host__ __device__ void mark_rest(const WindowArgs& p, const Schedule& sch, unsigned r, unsigned cta, unsigned ctas, int i, int row) {
  const int width = D * (p.out_dtype == kBF16 ? 2 : 4);
  for (; r * ctas < sch.works; ++r) {
    const unsigned x = nth_work(r, cta, ctas);
    if (x >= sch.works) continue;
    const Work w = make_work(p, sch, x);
    const int t = w.qt[i] * kT + row;
    if (t >= p.L || (t >= w.len && !p.zero_rest)) continue;
    const size_t at = ((size_t)w.b * p.H + w.h[i]) * p.L + t;
    fill_words(p.o, at * width, width, t < w.len ? nan_word(p.out_dtype) : 0u);
    p.lse[at] = t < w.len ? NAN : 0.f;
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    window_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, WindowArgs p, Schedule sch) {
  using S = Smem<D>;
  constexpr int kNP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2], s_ready[2], p_ready[2], done[2], last;
  __shared__ uint32_t tmem_base;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    sm100::mbar_init(&q_full, 1), sm100::mbar_init(&q_empty, 1), sm100::mbar_init(&last, 1);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&k_full[i], 1), sm100::mbar_init(&k_empty[i], 1);
      sm100::mbar_init(&v_full[i], 1), sm100::mbar_init(&v_empty[i], 1);
      sm100::mbar_init(&s_ready[i], 1), sm100::mbar_init(&p_ready[i], 4), sm100::mbar_init(&done[i], 1);
    }
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

  if (warp >= 8) {
    if (warp == 8 && lane == 0) {
      // ---------------------------------------------------------------------------------- loads
      sm100::prefetch_tmap(&tm_q), sm100::prefetch_tmap(&tm_k), sm100::prefetch_tmap(&tm_v);
      unsigned nq = 0, nk = 0, nv = 0;  // copies issued so far
      auto load_k = [&](const Work& w, int it) {
        const unsigned slot = nk & 1;
        if (nk > 1) fine = sm100::mbar_wait_bounded(&k_empty[slot], ((nk >> 1) - 1) & 1, kWaitCycles);
        if (!fine) return;
        sm100::mbar_arrive_expect_tx(&k_full[slot], S::kTile);
        load_tile<kNP>(sm + S::kK + slot * S::kTile, &tm_k, &k_full[slot], w.ku.walk(it) * kT, w.b * p.Hkv + w.kvh);
        ++nk;
      };
      for (unsigned r = 0; r * gridDim.x < sch.works && fine; ++r) {
        const unsigned x = nth_work(r, blockIdx.x, gridDim.x);
        if (x >= sch.works) continue;
        const Work w = make_work(p, sch, x);
        if (w.n == 0) continue;
        load_k(w, 0);
        if (fine && nq > 0) fine = sm100::mbar_wait_bounded(&q_empty, (nq - 1) & 1, kWaitCycles);
        if (!fine) break;
        sm100::mbar_arrive_expect_tx(&q_full, (w.two ? 2 : 1) * S::kTile);
        for (int i = 0; i < (w.two ? 2 : 1); ++i)
          load_tile<kNP>(sm + S::kQ + i * S::kTile, &tm_q, &q_full, w.qt[i] * kT, w.b * p.H + w.h[i]);
        ++nq;
        for (int it = 0; it < w.n; ++it) {
          if (it > 0) load_k(w, it);
          if (!fine) break;
          const unsigned slot = nv & 1;
          if (nv > 1) fine = sm100::mbar_wait_bounded(&v_empty[slot], ((nv >> 1) - 1) & 1, kWaitCycles);
          if (!fine) break;
          sm100::mbar_arrive_expect_tx(&v_full[slot], S::kTile);
          load_tile<kNP>(sm + S::kV + slot * S::kTile, &tm_v, &v_full[slot], w.ku.walk(it) * kT, w.b * p.Hkv + w.kvh);
          ++nv;
        }
      }
      if (!fine) {  // nothing of this CTA may be in flight when it ends
        if (nq > 0) sm100::mbar_wait_bounded(&q_full, (nq - 1) & 1, kWaitCycles);
        for (unsigned c = nk > 2 ? nk - 2 : 0; c < nk; ++c) sm100::mbar_wait_bounded(&k_full[c & 1], (c >> 1) & 1, kWaitCycles);
        for (unsigned c = nv > 2 ? nv - 2 : 0; c < nv; ++c) sm100::mbar_wait_bounded(&v_full[c & 1], (c >> 1) & 1, kWaitCycles);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------------------------------- products
      const uint64_t q0_desc = rows_desc(sm100::smem_u32(sm + S::kQ)), q1_desc = rows_desc(sm100::smem_u32(sm + S::kQ + S::kTile));
      const uint64_t k0_desc = rows_desc(sm100::smem_u32(sm + S::kK)), k1_desc = rows_desc(sm100::smem_u32(sm + S::kK + S::kTile));
      const uint64_t v0_desc = cols_desc(sm100::smem_u32(sm + S::kV)), v1_desc = cols_desc(sm100::smem_u32(sm + S::kV + S::kTile));
      uint32_t p_phase[2] = {0, 0};
      unsigned nq = 0, nk = 0, nv = 0;  // tiles taken so far
      for (unsigned r = 0; r * gridDim.x < sch.works && fine; ++r) {
        const unsigned x = nth_work(r, blockIdx.x, gridDim.x);
        if (x >= sch.works) continue;
        const Work w = make_work(p, sch, x);
        if (w.n == 0) continue;
        auto issue_s = [&](int i, int it) {
          if (lane == 0) {
            mma_rows<D>(tmem + 128 * i, i ? q1_desc : q0_desc, (nk & 1) ? k1_desc : k0_desc);
            sm100::mma_commit(&s_ready[i]);
          }
        };
        bool begun[2] = {false, false};
        fine = warp_wait(&q_full, nq & 1) && warp_wait(&k_full[nk & 1], (nk >> 1) & 1);
        if (!fine) break;
        ++nq;
        if (w.active(0, 0)) issue_s(0, 0);
        if (w.active(1, 0)) issue_s(1, 0);
        if (lane == 0) {
          sm100::mma_commit(&k_empty[nk & 1]);
          if (w.n == 1) sm100::mma_commit(&q_empty);
        }
        ++nk;
        for (int it = 0; it < w.n; ++it) {
          const unsigned slot = nv & 1;
          const bool more = it + 1 < w.n;
          fine = warp_wait(&v_full[slot], (nv >> 1) & 1);
          if (more) fine = fine && warp_wait(&k_full[nk & 1], (nk >> 1) & 1);
          if (!fine) break;
          const int inside = w.len - w.ku.walk(it) * kT;
          if (inside < kT) zero_rows<kNP>(sm + S::kV + slot * S::kTile, inside, lane);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (w.active(i, it)) {
              fine = warp_wait(&p_ready[i], p_phase[i]);
              if (!fine) break;
              p_phase[i] ^= 1;
              sm100::tc_fence_after();
              if (lane == 0) {
                mma_weights<D>(tmem + 256 + D * i, tmem + 128 * i, 32, slot ? v1_desc : v0_desc, begun[i]);
                // the last key tile is tile 1's (or the only tile's) last; tile 0's may come one before
                if (i == 1 ? !more : w.ku.walk(it) == w.k0.hi - 1) sm100::mma_commit(&done[i]);
              }
              begun[i] = true;
            }
            if (more && w.active(i, it + 1)) issue_s(i, it + 1);
          }
          if (!fine) break;
          if (lane == 0) {
            sm100::mma_commit(&v_empty[slot]);
            if (more) sm100::mma_commit(&k_empty[nk & 1]);
            if (it + 2 == w.n) sm100::mma_commit(&q_empty);
          }
          ++nv;
          if (more) ++nk;
        }
      }
      if (!fine && lane == 0) {  // the products in flight read shared memory and write TMEM
        sm100::mma_commit(&last);
        sm100::mbar_wait_bounded(&last, 0, kWaitCycles);
      }
    }
  } else {
    // ------------------------------------------------------------------------------------ softmax
    const int i = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lanes + 128 * i, t_o = tmem + lanes + 256 + D * i;
    const float c = p.scale * kLog2e;
    uint32_t phase = 0, done_phase = 0;
    unsigned r = 0;
    for (; r * gridDim.x < sch.works; ++r) {
      const unsigned x = nth_work(r, blockIdx.x, gridDim.x);
      if (x >= sch.works) continue;
      const Work w = make_work(p, sch, x);
      const int t0 = (i == 0 ? w.qt[0] : w.qt[1]) * kT, t = t0 + row;
      const size_t head = (size_t)w.b * p.H + (i == 0 ? w.h[0] : w.h[1]);
      if (p.zero_rest && t0 + kT > w.len) {
        zero_tile(p.o, head * p.L, D * (p.out_dtype == kBF16 ? 2 : 4), t0, w.len, p.L, row, 128);
        if (t >= w.len && t < p.L) p.lse[head * p.L + t] = 0.f;
      }
      if (w.n == 0 || (i == 1 && !w.two)) continue;
      const int w_first = t0 + 32 * (warp & 3), w_last = w_first + 31;  // the warp's rows
      float m = -INFINITY, l = 0.f;
      for (int it = 0; it < w.n; ++it) {
        if (!w.active(i, it)) continue;
        const int j0 = w.ku.walk(it) * kT;
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
#pragma unroll
          for (int u = 0; u < 4; ++u) {  // 32 columns: seen by every row of the warp, by none, or by some
            const int j = j0 + 32 * u;
            if (j + 31 <= w_first && (w_last - j < p.window || j + 32 <= p.n_sink)) continue;
            const uint32_t seen = seen_bits(t - j, p.window, p.n_sink - j);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen >> e & 1u)) s[u][e] = -INFINITY;
          }
        }
        float top[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          top[u] = s[u][0];
#pragma unroll
          for (int e = 1; e < 31; e += 2) top[u] = fmaxf(fmaxf(top[u], s[u][e]), s[u][e + 1]);
          top[u] = fmaxf(top[u], s[u][31]);
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
        float2 sum[4] = {};
        const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float q[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 x = fma2(make_float2(s[u][e], s[u][e + 1]), c2, b2);
            x.x = exp2_fast(x.x), x.y = exp2_fast(x.y);
            sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], x);
            q[e / 2] = __uint_as_float(pack_bf16(x.x, x.y));
          }
          sm100::tmem_st16(t_s + 16 * u, q);
        }
        const float2 all_sum = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += all_sum.x + all_sum.y;
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        warp_arrive(&p_ready[i]);
      }
      const size_t at = head * p.L + t;
      if (fine) {
        fine = warp_wait(&done[i], done_phase);
        done_phase ^= 1;
        sm100::tc_fence_after();
      }
      if (!fine) break;
      const bool wide = is_wide(p.o);
      const float inv = 1.f / l;
      if (t < w.len) p.lse[at] = (m + log2f(l)) * kLn2;
#pragma unroll 1
      for (int u = 0; u < D; u += 32) {
        float o[32];
        sm100::tmem_ld32(t_o + u, o);
        sm100::tmem_wait_ld();
        if (t >= w.len) {
        } else if (p.out_dtype == kBF16) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + at * D + u;
#pragma unroll
          for (int e = 0; e < 32; e += 16) store32(dst + e, pack8_bf16(o + e, inv), pack8_bf16(o + e + 8, inv), wide);
        } else {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * D + u);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
        }
        __syncwarp();
      }
      sm100::tc_fence_before();  // O is read: the next work's first product follows this warp's next arrival
    }
    if (!fine) mark_rest<D>(p, sch, r, blockIdx.x, gridDim.x, i, row);
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
  const Schedule sch = make_schedule(p.B, p.H, p.Hkv, p.L);
  const int smem = Smem<D>::kTotal + 1024;
  const cudaError_t e = cudaFuncSetAttribute(window_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return cudaErrorInvalidDevice;
  window_fwd_tc_kernel<D><<<(sch.works < (unsigned)sms ? sch.works : (unsigned)sms), kTcThreads, smem, stream>>>(tq, tk, tv, p, sch);
  return cudaGetLastError();
}

}  // namespace

bool window_tc_supported(int dk, int dv, int in_dtype) { return in_dtype == kBF16 && dk == dv && (dk == 64 || dk == 128); }

cudaError_t launch_window_attn_tc(int d, const WindowArgs& p, cudaStream_t stream) {
  return d == 128 ? forward<128>(p, stream) : forward<64>(p, stream);
}

}  // namespace kdn
