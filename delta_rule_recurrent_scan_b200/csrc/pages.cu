// Upkeep of a paged key-value cache: which pages a sequence holds (table, lens, refs), and the pages' movement.
//
// A row r of the table holds ceil(lens[r] / page_size) pages in its leading entries, -1 behind them; refs[p] counts
// the entries that name page p (0 = free).  New pages are always the lowest free ones, handed out in the order of the
// call's list, so the books depend on nothing but the call.  Only whole pages are shared between rows: a fork gives
// its row a page of its own for a part-filled last page, so a row may always write behind its length.
//
// The books are small (4 bytes per page and table entry) and the steps depend on each other (validate, count, find
// free pages, hand out), so one CTA of 1024 threads does each call: the searches stream refs at 16 KB per step.  A
// call that cannot be served as a whole (a row out of range, listed twice, too long, or no page left) changes nothing
// and says so in the status word, which this CTA stores itself: no separate clearing launch.  The host may well enqueue the
// write of the new tokens before it knows, so a refused reservation also marks its rows, and the write passes over them.
//
// The data movers are bandwidth-bound copies of 16-byte words.
#include "common.cuh"
#include "kernels.h"
#include "pages_need.h"

namespace kdn {

namespace {

constexpr int kBook = 1024;               // threads of a book-keeping CTA
constexpr int kMaxRows = 1 << 18;         // one bit per row in shared memory
constexpr int kPer = 4;                   // consecutive refs per thread and step

struct Shared {
  unsigned seen[kMaxRows / 32];
  int warp_sum[33];
  unsigned bad;
  PageSum need;
};

// Exclusive prefix sum of x over the CTA; total gets the sum.
__device__ __forceinline__ int scan_cta(Shared& s, int x, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) s.warp_sum[warp] = y;
  __syncthreads();
  if (warp == 0) {
    const int v = s.warp_sum[lane];
    int w = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += z;
    }
    s.warp_sum[lane] = w - v;
    if (lane == 31) s.warp_sum[32] = w;
  }
  __syncthreads();
  const int before = s.warp_sum[warp] + y - x;
  total = s.warp_sum[32];
  __syncthreads();  // the sums may be written again
  return before;
}

__device__ __forceinline__ void clear_rows(Shared& s, int rows) {
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += kBook) s.seen[i] = 0;
  if (threadIdx.x == 0) s.bad = 0, s.need = 0;
}
__device__ __forceinline__ bool mark(Shared& s, int r) {  // false: it was marked already
  const unsigned bit = 1u << (r & 31);
  return (atomicOr(&s.seen[r >> 5], bit) & bit) == 0;
}
__device__ __forceinline__ bool unmark(Shared& s, int r) {  // whether it was marked
  const unsigned bit = 1u << (r & 31);
  return (atomicAnd(&s.seen[r >> 5], ~bit) & bit) != 0;
}
__device__ __forceinline__ bool marked(const Shared& s, int r) { return (s.seen[r >> 5] >> (r & 31)) & 1u; }

__device__ __forceinline__ int pages_of(const PagesArgs& p, int len) { return kdn::pages_of(len, p.page_size); }

__device__ __forceinline__ bool in_pool(const PagesArgs& p, int page) { return page >= 0 && page < p.num_pages; }
__device__ __forceinline__ bool in_use(const PagesArgs& p, int page) { return in_pool(p, page) && p.refs[page] > 0; }

// The ``want`` lowest free pages into p.scratch, rising; false when there are fewer.
__device__ bool find_free(const PagesArgs& p, Shared& s, int want) {
  int found = 0;
  for (int base = 0; base < p.num_pages && found < want; base += kBook * kPer) {
    const int at = base + kPer * threadIdx.x;
    bool free_[kPer];
    int n = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      free_[u] = at + u < p.num_pages && p.refs[at + u] == 0;
      n += free_[u];
    }
    int total;
    int pos = found + scan_cta(s, n, total);
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (free_[u]) {
        if (pos < want) p.scratch[pos] = at + u;
        ++pos;
      }
    found += total;
  }
  __syncthreads();
  return found >= want;
}

__global__ void __launch_bounds__(kBook, 1) pages_reserve_kernel(PagesArgs p, int n, const int* rows, const int* counts, int count) {
  __shared__ Shared s;
  clear_rows(s, p.rows);
  __syncthreads();
  const long long most = (long long)p.max_pages * p.page_size;
  PageSum need = 0;
  unsigned bad = 0;
  for (int i = threadIdx.x; i < n; i += kBook) {
    const int r = rows[i], c = counts ? counts[i] : count;
    if (r < 0 || r >= p.rows || c < 0) { bad |= kStatusInvalid; continue; }
    const int len = p.lens[r];
    if (len < 0 || len > most || !mark(s, r)) { bad |= kStatusInvalid; continue; }
    if (len + (long long)c > most) { bad |= kStatusCapacity; continue; }
    need += more_pages(len, c, p.page_size);
  }
  if (bad) atomicOr(&s.bad, bad);
  if (need) atomicAdd(&s.need, need);
  __syncthreads();
  if (threadIdx.x == 0 && pool_too_small(s.need, p.num_pages)) atomicOr(&s.bad, kStatusCapacity);
  __syncthreads();
  const int total = static_cast<int>(s.need);  // within num_pages where it is used
  if (s.bad == 0 && total > 0 && !find_free(p, s, total)) {
    if (threadIdx.x == 0) atomicOr(&s.bad, kStatusCapacity);
  }
  __syncthreads();
  if (threadIdx.x == 0) *p.status = s.bad;
  if (s.bad) {  // the write that was to follow would fall on the rows' older tokens
    for (int i = threadIdx.x; i < n; i += kBook)
      if (rows[i] >= 0 && rows[i] < p.rows) p.refused[rows[i]] = 1;
    return;
  }
  int given = 0;
  for (int base = 0; base < n; base += kBook) {
    const int i = base + threadIdx.x;
    int r = 0, len = 0, c = 0, had = 0, more = 0;
    if (i < n) {
      r = rows[i], c = counts ? counts[i] : count, len = p.lens[r];
      had = pages_of(p, len), more = pages_of(p, len + c) - had;
    }
    int sum;
    const int first = given + scan_cta(s, more, sum);
    given += sum;
    for (int k = 0; k < more; ++k) {
      const int page = p.scratch[first + k];
      p.table[(size_t)r * p.max_pages + had + k] = page;
      p.refs[page] = 1;
    }
    if (i < n) p.lens[r] = len + c, p.refused[r] = 0;
  }
}

__global__ void __launch_bounds__(kBook, 1) pages_fork_kernel(PagesArgs p, int n, const int* src, const int* dst, int2* moves) {
  __shared__ Shared s;
  clear_rows(s, p.rows);
  __syncthreads();
  const long long most = (long long)p.max_pages * p.page_size;
  unsigned bad = 0;
  for (int i = threadIdx.x; i < n; i += kBook) {
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= p.rows || b < 0 || b >= p.rows) { bad |= kStatusInvalid; continue; }
    if (p.lens[a] < 0 || p.lens[a] > most || p.lens[b] != 0 || !mark(s, b)) bad |= kStatusInvalid;
  }
  if (bad) atomicOr(&s.bad, bad);
  __syncthreads();
  const bool rows_fine = s.bad == 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  int need = 0;
  if (rows_fine) {
    for (int i = threadIdx.x; i < n; i += kBook) {
      if (marked(s, src[i])) bad |= kStatusInvalid;  // a row that is written by this call
      need += p.lens[src[i]] % p.page_size != 0;
    }
    for (int i = threadIdx.x >> 5; i < n; i += kBook / 32) {  // one warp per row: every entry names a page in use
      const int held = pages_of(p, p.lens[src[i]]);
      for (int e = lane; e < held; e += 32)
        if (!in_use(p, p.table[(size_t)src[i] * p.max_pages + e])) bad |= kStatusInvalid;
    }
    if (bad) atomicOr(&s.bad, bad);
  }
  int total;
  scan_cta(s, need, total);
  if (s.bad == 0 && total > 0 && !find_free(p, s, total)) {
    if (threadIdx.x == 0) atomicOr(&s.bad, kStatusCapacity);
  }
  __syncthreads();
  const unsigned refused = s.bad;
  if (refused) {
    for (int i = threadIdx.x; i < n; i += kBook) moves[i] = make_int2(-1, -1);
    if (threadIdx.x == 0) *p.status = refused;
    return;
  }
  // the part-filled pages, in the order of the list
  int given = 0;
  for (int base = 0; base < n; base += kBook) {
    const int i = base + threadIdx.x;
    int len = 0;
    if (i < n) len = p.lens[src[i]];
    const int part = len % p.page_size != 0;
    int sum;
    const int at = given + scan_cta(s, part, sum);
    given += sum;
    if (i < n) {
      int2 mv = make_int2(-1, -1);
      if (part) {
        const int full = len / p.page_size, old = p.table[(size_t)src[i] * p.max_pages + full], page = p.scratch[at];
        p.table[(size_t)dst[i] * p.max_pages + full] = page;
        p.refs[page] = 1;
        mv = make_int2(old, page);
      }
      moves[i] = mv;
      p.lens[dst[i]] = len, p.refused[dst[i]] = 0;
    }
  }
  // the full pages are shared: one warp per row
  for (int i = threadIdx.x >> 5; i < n; i += kBook / 32) {
    const int full = p.lens[src[i]] / p.page_size;
    for (int e = lane; e < full; e += 32) {
      const int page = p.table[(size_t)src[i] * p.max_pages + e];
      p.table[(size_t)dst[i] * p.max_pages + e] = page;
      atomicAdd(&p.refs[page], 1);
    }
  }
  if (threadIdx.x == 0) *p.status = 0;
}

// Counts down first: when an entry names no page, or a page more often than it was counted, the counts are put back and
// nothing else has changed.  One warp per row; a row listed twice is the warp's that marks (then unmarks) it first.
__global__ void __launch_bounds__(kBook, 1) pages_free_kernel(PagesArgs p, int n, const int* rows) {
  __shared__ Shared s;
  clear_rows(s, p.rows);
  __syncthreads();
  const long long most = (long long)p.max_pages * p.page_size;
  for (int i = threadIdx.x; i < n; i += kBook) {
    const int r = rows[i];
    if (r < 0 || r >= p.rows || p.lens[r] < 0 || p.lens[r] > most) atomicOr(&s.bad, kStatusInvalid);
  }
  __syncthreads();
  const bool rows_fine = s.bad == 0;
  __syncthreads();
  if (rows_fine) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = warp; i < n; i += kBook / 32) {
      const int r = rows[i];
      if (!__shfl_sync(0xffffffffu, lane == 0 && mark(s, r), 0)) continue;
      const int held = pages_of(p, p.lens[r]);
      for (int e = lane; e < held; e += 32) {
        const int page = p.table[(size_t)r * p.max_pages + e];
        if (!in_pool(p, page) || atomicSub(&p.refs[page], 1) <= 0) atomicOr(&s.bad, kStatusInvalid);
      }
    }
    __syncthreads();
    const bool fine = s.bad == 0;
    for (int i = warp; i < n; i += kBook / 32) {
      const int r = rows[i];
      if (!__shfl_sync(0xffffffffu, lane == 0 && unmark(s, r), 0)) continue;
      const int held = pages_of(p, p.lens[r]);
      for (int e = lane; e < held; e += 32) {
        int& entry = p.table[(size_t)r * p.max_pages + e];
        if (fine) entry = -1;
        else if (in_pool(p, entry)) atomicAdd(&p.refs[entry], 1);
      }
      __syncwarp();
      if (fine && lane == 0) p.lens[r] = 0, p.refused[r] = 0;
    }
  }
  if (threadIdx.x == 0) *p.status = s.bad;
}

// The i-th used page behind the first U (U = number of used pages) goes into the i-th free page before it.
// scratch: [0] U, then the holes, the movers (num_pages / 2 each) and where every page at or behind U goes.
__global__ void __launch_bounds__(kBook, 1) pages_compact_kernel(PagesArgs p, int2* moves) {
  __shared__ Shared s;
  const int half = p.num_pages / 2;
  int* holes = p.scratch + 1;
  int* movers = holes + half;
  int* to = movers + half;
  int mine = 0;
  for (int i = threadIdx.x; i < p.num_pages; i += kBook) mine += p.refs[i] != 0;
  int used;
  scan_cta(s, mine, used);
  int nh = 0, nm = 0;
  for (int base = 0; base < p.num_pages; base += kBook * kPer) {
    const int at = base + kPer * threadIdx.x;
    bool hit[kPer];
    int n = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = at + u;
      const bool live = i < p.num_pages && p.refs[i] != 0;
      hit[u] = i < p.num_pages && (i < used ? !live : live);
      n += hit[u] ? (i < used ? 1 : 1 << 16) : 0;  // at most 4096 of each per step: two counts in one word
    }
    int total;
    const int before = scan_cta(s, n, total);
    int ph = nh + (before & 0xffff), pm = nm + (before >> 16);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = at + u;
      if (i >= p.num_pages) continue;
      if (i < used) {
        if (hit[u]) holes[ph++] = i;
      } else {
        to[i] = i;
        if (hit[u]) movers[pm++] = i;
      }
    }
    nh += total & 0xffff, nm += total >> 16;
  }
  __syncthreads();  // nh == nm: as many holes before U as used pages behind it
  for (int i = threadIdx.x; i < half; i += kBook) {
    if (i >= nm) {
      moves[i] = make_int2(-1, -1);
      continue;
    }
    const int a = movers[i], b = holes[i];
    moves[i] = make_int2(a, b);
    to[a] = b;
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  if (threadIdx.x == 0) p.scratch[0] = used, *p.status = 0;
}

__global__ void __launch_bounds__(256) pages_remap_kernel(PagesArgs p) {
  const int used = p.scratch[0];
  const int* to = p.scratch + 1 + 2 * (p.num_pages / 2);
  const size_t n = (size_t)p.rows * p.max_pages;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
    const int e = p.table[i];
    if (e >= used && e < p.num_pages) p.table[i] = to[e];
  }
}

// Page src -> page dst for every pair, keys and values.  A CTA takes pieces of kPiece bytes.
constexpr int kPiece = 256 * 16 * 4;
__global__ void __launch_bounds__(256) pages_copy_kernel(const int2* moves, long long pieces, int per_k, int per_v, int num_pages,
                                                         size_t k_bytes, size_t v_bytes, char* k, char* v) {
  const int per = per_k + per_v;
  for (long long x = blockIdx.x; x < pieces; x += gridDim.x) {
    const int2 mv = moves[x / per];
    if (mv.x < 0 || mv.y < 0 || mv.x >= num_pages || mv.y >= num_pages || mv.x == mv.y) continue;
    int part = static_cast<int>(x % per);
    const bool keys = part < per_k;
    if (!keys) part -= per_k;
    char* pool = keys ? k : v;
    const size_t bytes = keys ? k_bytes : v_bytes, from = (size_t)part * kPiece;
    const uint4* a = reinterpret_cast<const uint4*>(pool + mv.x * bytes + from);
    uint4* b = reinterpret_cast<uint4*>(pool + mv.y * bytes + from);
    const int words = static_cast<int>(min((size_t)kPiece, bytes - from) / 16);
    uint4 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (threadIdx.x + 256 * u < words) r[u] = __ldcs(a + threadIdx.x + 256 * u);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (threadIdx.x + 256 * u < words) __stcs(b + threadIdx.x + 256 * u, r[u]);
  }
}

// The newest tokens of each listed row into its pages: one 16-byte word per thread and step.
__global__ void __launch_bounds__(256) pages_write_kernel(PagesArgs p, PagesWrite w) {
  const int kw = w.k_row / 16, vw = w.v_row / 16;
  const long long per = (long long)w.tokens * (kw + vw);  // words per (listed row, head)
  const long long total = per * w.heads * w.n;
  for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < total; x += (long long)gridDim.x * 256) {
    const long long ih = x / per;
    int c = static_cast<int>(x % per);
    const int i = static_cast<int>(ih / w.heads), h = static_cast<int>(ih % w.heads);
    const bool keys = c < w.tokens * kw;
    if (!keys) c -= w.tokens * kw;
    const int words = keys ? kw : vw, t = c / words, word = c % words;
    const int r = w.rows[i], count = w.counts ? w.counts[i] : w.tokens;
    if (r < 0 || r >= p.rows || t >= count || count > w.tokens || (p.refused && p.refused[r])) continue;
    const int pos = p.lens[r] - count + t;
    if (pos < 0 || pos / p.page_size >= p.max_pages) continue;
    const int page = p.table[(size_t)r * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) continue;
    const uint4* from = reinterpret_cast<const uint4*>(keys ? w.k_new : w.v_new) + ((size_t)ih * w.tokens + t) * words + word;
    uint4* pool = reinterpret_cast<uint4*>(keys ? w.k_pages : w.v_pages);
    pool[(((size_t)page * w.heads + h) * p.page_size + pos % p.page_size) * words + word] = *from;
  }
}

}  // namespace

int pages_max_rows() { return kMaxRows; }
size_t pages_scratch_ints(int num_pages) { return 1 + 2 * (size_t)(num_pages / 2) + num_pages; }

cudaError_t launch_pages_reserve(const PagesArgs& p, int n, const int* rows, const int* counts, int count, cudaStream_t st) {
  pages_reserve_kernel<<<1, kBook, 0, st>>>(p, n, rows, counts, count);
  return cudaGetLastError();
}
cudaError_t launch_pages_fork(const PagesArgs& p, int n, const int* src, const int* dst, int* moves, cudaStream_t st) {
  pages_fork_kernel<<<1, kBook, 0, st>>>(p, n, src, dst, reinterpret_cast<int2*>(moves));
  return cudaGetLastError();
}
cudaError_t launch_pages_free(const PagesArgs& p, int n, const int* rows, cudaStream_t st) {
  pages_free_kernel<<<1, kBook, 0, st>>>(p, n, rows);
  return cudaGetLastError();
}
cudaError_t launch_pages_compact(const PagesArgs& p, int* moves, cudaStream_t st) {
  pages_compact_kernel<<<1, kBook, 0, st>>>(p, reinterpret_cast<int2*>(moves));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t n = (size_t)p.rows * p.max_pages;
  const size_t ctas = (n + 255) / 256;
  pages_remap_kernel<<<(unsigned)(ctas < 1184 ? ctas : 1184), 256, 0, st>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_pages_copy(const int* moves, int n, int num_pages, size_t k_bytes, size_t v_bytes, void* k, void* v,
                              cudaStream_t st) {
  const int per_k = (int)((k_bytes + kPiece - 1) / kPiece), per_v = (int)((v_bytes + kPiece - 1) / kPiece);
  const long long pieces = (long long)n * (per_k + per_v);
  pages_copy_kernel<<<(unsigned)(pieces < 1184 ? pieces : 1184), 256, 0, st>>>(
      reinterpret_cast<const int2*>(moves), pieces, per_k, per_v, num_pages, k_bytes, v_bytes, static_cast<char*>(k),
      static_cast<char*>(v));
  return cudaGetLastError();
}
cudaError_t launch_pages_write(const PagesArgs& p, const PagesWrite& w, cudaStream_t st) {
  const long long total = (long long)w.n * w.heads * w.tokens * (w.k_row / 16 + w.v_row / 16);
  const long long ctas = (total + 255) / 256;
  pages_write_kernel<<<(unsigned)(ctas < 148 * 16 ? ctas : 148 * 16), 256, 0, st>>>(p, w);
  return cudaGetLastError();
}

}  // namespace kdn
