// C-ABI layer of the windowed attention, the paged decode step and the paged cache: argument validation,
// workspace layout, dispatch (the scans' layer is kdn_api.cu, whose helpers it shares).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "../../include/kdn.h"
#include "api_internal.h"
#include "common.cuh"
#include "kernels.h"

using namespace kdn::api;

#define KDN_TRY(expr)            \
  do {                           \
    kdn_status _s = (expr);      \
    if (_s != KDN_OK) return _s; \
  } while (0)

namespace {

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

kdn_status check_heads(int H, int kv_heads) {
  if (kv_heads < 1 || H % kv_heads != 0) return fail(KDN_ERR_INVALID_ARG, "kv_heads must be >= 1 and divide H");
  return KDN_OK;
}

kdn_status check_window(int window, int least, int n_sink, float scale) {
  if (window < least) return fail(KDN_ERR_INVALID_ARG, "window must be >= " + std::to_string(least));
  if (n_sink < 0) return fail(KDN_ERR_INVALID_ARG, "n_sink must be >= 0");
  if (!(scale > 0.f && scale <= 1e30f)) return fail(KDN_ERR_INVALID_ARG, "scale must be positive and at most 1e30");
  return KDN_OK;
}

kdn_status window_checks(const kdn_dims* d, int kv_heads, int window, int n_sink, float scale) {
  KDN_TRY(check_dims(d));
  KDN_TRY(check_heads(d->H, kv_heads));
  KDN_TRY(check_window(window, 1, n_sink, scale));
  if ((long long)d->B * d->H * ((d->L + 63LL) / 64) > INT_MAX || (long long)d->B * d->H * d->L / 8 >= INT_MAX)
    return fail(KDN_ERR_UNSUPPORTED, "B*H*L too large for one launch");
  return KDN_OK;
}

kdn_status check_workspace(const void* ws, size_t bytes, size_t need) {
  KDN_TRY(check_ptr(ws, "workspace", 256, false));
  if (bytes < need)
    return fail(KDN_ERR_INVALID_ARG, "workspace_bytes " + std::to_string(bytes) + " < required " + std::to_string(need));
  return KDN_OK;
}

// The kernels write parts of an output while others still read the inputs: no output may share memory with an input
// or with another output.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};
kdn_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x != 0 && y != 0 && a.bytes != 0 && b.bytes != 0 && (x < y ? y - x < a.bytes : x - y < b.bytes);
  };
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (meet(*a, *b)) return fail(KDN_ERR_INVALID_ARG, std::string(a->name) + " overlaps " + b->name);
    for (const Span& b : ins)
      if (meet(*a, b)) return fail(KDN_ERR_INVALID_ARG, std::string(a->name) + " overlaps " + b.name);
  }
  return KDN_OK;
}

size_t elem_bytes(kdn_dtype t) { return t == KDN_BF16 ? 2 : 4; }
Span ints(const char* name, const void* p, long long n) { return {name, p, n > 0 ? (size_t)n * sizeof(int) : 0}; }
Span table_of(const kdn_pages* p) { return {"table", p->table, (size_t)p->rows * p->max_pages * sizeof(int)}; }
Span lens_of(const kdn_pages* p) { return ints("lens", p->lens, p->rows); }

// ---------------------------------------------------------------------------------------- paged cache
bool pages_sizes_ok(const kdn_pages* p) {
  return p != nullptr && p->num_pages >= 1 && p->rows >= 1 && p->max_pages >= 1 && p->page_size >= 1 &&
         p->page_size <= 1024 && (p->page_size & (p->page_size - 1)) == 0 &&
         (long long)p->max_pages * p->page_size <= (1LL << 30) && p->num_pages <= (1 << 30) &&
         p->rows <= kdn::pages_max_rows();
}

kdn_status check_pages(const kdn_pages* p) {
  if (p == nullptr) return fail(KDN_ERR_INVALID_ARG, "pages is NULL");
  if (p->num_pages < 1 || p->rows < 1 || p->max_pages < 1)
    return fail(KDN_ERR_INVALID_ARG, "num_pages, rows and max_pages must be >= 1");
  if (p->page_size < 1 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)) != 0)
    return fail(KDN_ERR_UNSUPPORTED, "page_size must be a power of two up to 1024");
  if (!pages_sizes_ok(p))
    return fail(KDN_ERR_UNSUPPORTED, "at most 2^30 pages, 2^30 tokens per row and " + std::to_string(kdn::pages_max_rows()) + " rows");
  return KDN_OK;
}

// The books' workspace: the status word, scratch, and a word per row for refused reservations.
size_t refused_at(const kdn_pages* p) { return kStatusBytes + round256(kdn::pages_scratch_ints(p->num_pages) * sizeof(int)); }

kdn::PagesArgs pages_args(const kdn_pages* p, void* ws) {
  kdn::PagesArgs a{p->num_pages, p->page_size, p->rows, p->max_pages, p->table, p->lens, p->refs, nullptr, nullptr, nullptr};
  if (ws != nullptr) {
    a.status = static_cast<unsigned*>(ws);
    a.scratch = reinterpret_cast<int*>(static_cast<char*>(ws) + kStatusBytes);
    a.refused = reinterpret_cast<int*>(static_cast<char*>(ws) + refused_at(p));
  }
  return a;
}

// A book-keeping call's checks; switches to the table's device.  list: the pairs that it writes; ins: the lists it reads.
kdn_status book_checks(const kdn_pages* p, int n, const void* ws, size_t ws_bytes, const Span& list,
                       std::initializer_list<Span> ins, DeviceGuard& guard) {
  KDN_TRY(check_pages(p));
  if (n < 0) return fail(KDN_ERR_INVALID_ARG, "n must be >= 0");
  KDN_TRY(check_apart({table_of(p), lens_of(p), ints("refs", p->refs, p->num_pages), {"workspace", ws, ws_bytes}, list}, ins));
  KDN_TRY(check_ptr(p->table, "table", 4, false));
  KDN_TRY(check_ptr(p->lens, "lens", 4, false));
  KDN_TRY(check_ptr(p->refs, "refs", 4, false));
  KDN_TRY(check_workspace(ws, ws_bytes, kdn_pages_workspace_bytes(p)));
  return use_device_of(p->table, guard);
}

kdn_status clear_status(void* ws, cudaStream_t st) {
  return cuda_status(cudaMemsetAsync(ws, 0, kStatusBytes, st), "clearing the status word");
}

bool pool_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

kdn_status check_pool(int kv_heads, int dk, int dv, kdn_dtype dtype) {
  if (kv_heads < 1) return fail(KDN_ERR_INVALID_ARG, "kv_heads must be >= 1");
  if (!pool_dim(dk) || !pool_dim(dv)) return fail(KDN_ERR_UNSUPPORTED, "dk and dv must be 16, 32, 64 or 128");
  if (dtype != KDN_F32 && dtype != KDN_BF16) return fail(KDN_ERR_INVALID_ARG, "bad dtype");
  return KDN_OK;
}

// workspace: of the books, or NULL to write whatever the last reservations came to.
kdn_status write_pages(const kdn_pages* pages, int n, const int* rows, const int* counts, int tokens, int kv_heads, int dk,
                       int dv, kdn_dtype dtype, const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                       void* workspace, size_t workspace_bytes, void* stream) {
  KDN_TRY(check_pages(pages));
  if (n < 0 || tokens < 0) return fail(KDN_ERR_INVALID_ARG, "n and tokens must be >= 0");
  if (tokens > 1 << 24) return fail(KDN_ERR_UNSUPPORTED, "tokens must be at most 2^24");
  KDN_TRY(check_pool(kv_heads, dk, dv, dtype));
  const int es = (int)elem_bytes(dtype);
  const size_t fresh = (size_t)n * kv_heads * tokens * es, pool = (size_t)pages->num_pages * kv_heads * pages->page_size * es;
  KDN_TRY(check_apart({{"k_pages", k_pages, pool * dk}, {"v_pages", v_pages, pool * dv}},
                      {{"k_new", k_new, fresh * dk}, {"v_new", v_new, fresh * dv}, table_of(pages), lens_of(pages),
                       ints("rows", rows, n), ints("counts", counts, n),
                       {"workspace", workspace, workspace_bytes}}));
  const bool none = n == 0 || tokens == 0;
  KDN_TRY(check_ptr(pages->table, "table", 4, false));
  KDN_TRY(check_ptr(pages->lens, "lens", 4, false));
  KDN_TRY(check_ptr(rows, "rows", 4, none));
  KDN_TRY(check_ptr(counts, "counts", 4, true));
  KDN_TRY(check_ptr(k_new, "k_new", 16, none));
  KDN_TRY(check_ptr(v_new, "v_new", 16, none));
  KDN_TRY(check_ptr(k_pages, "k_pages", 16, false));
  KDN_TRY(check_ptr(v_pages, "v_pages", 16, false));
  if (workspace != nullptr) KDN_TRY(check_workspace(workspace, workspace_bytes, kdn_pages_workspace_bytes(pages)));
  if (none) return ok();
  DeviceGuard guard;
  KDN_TRY(use_device_of(k_pages, guard));
  const kdn::PagesWrite w{n, kv_heads, tokens, dk * es, dv * es, rows, counts, k_new, v_new, k_pages, v_pages};
  return cuda_status(kdn::launch_pages_write(pages_args(pages, workspace), w, (cudaStream_t)stream), "page write launch");
}

}  // namespace

extern "C" {

size_t kdn_window_workspace_bytes(const kdn_dims* dims, int kv_heads, int window, int n_sink, int backward) {
  if (check_dims(dims) != KDN_OK || check_heads(dims->H, kv_heads) != KDN_OK || window < 1 || n_sink < 0) return 0;
  size_t n = kStatusBytes;
  if (!backward || dims->L == 0) return n;
  if (kdn::window_tc_supported(dims->dk, dims->dv, dims->in_dtype))
    n += round256(kdn::window_bwd_tc_scratch_bytes(dims->B, dims->H, kv_heads, dims->L, dims->dk, dims->out_dtype, window, n_sink));
  else
    n += round256(kdn::window_bwd_scratch_bytes(dims->B, dims->H, kv_heads, dims->L, dims->dk, dims->dv, window, n_sink));
  return n;
}

kdn_status kdn_window_attn(const kdn_dims* dims, int kv_heads, const void* q, const void* k, const void* v,
                           const int* lens, int zero_rest, int window, int n_sink, float scale, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  KDN_TRY(window_checks(dims, kv_heads, window, n_sink, scale));
  const bool none = dims->L == 0;
  const size_t in = elem_bytes(dims->in_dtype), rows = (size_t)dims->B * dims->H * dims->L, keys = rows / dims->H * kv_heads;
  const Span q_{"q", q, rows * dims->dk * in}, k_{"k", k, keys * dims->dk * in}, v_{"v", v, keys * dims->dv * in};
  const Span o_{"o", o, rows * dims->dv * elem_bytes(dims->out_dtype)}, lse_{"lse", lse, rows * 4};
  const Span ws_{"workspace", workspace, workspace_bytes};
  KDN_TRY(check_apart({o_, lse_, ws_}, {q_, k_, v_, ints("lens", lens, dims->B)}));
  KDN_TRY(check_ptr(q, "q", 16, none));
  KDN_TRY(check_ptr(k, "k", 16, none));
  KDN_TRY(check_ptr(v, "v", 16, none));
  KDN_TRY(check_ptr(o, "o", 16, none));
  KDN_TRY(check_ptr(lse, "lse", 4, none));
  KDN_TRY(check_ptr(lens, "lens", 4, true));
  if (workspace != nullptr) KDN_TRY(check_workspace(workspace, workspace_bytes, kStatusBytes));
  if (none && workspace == nullptr) return ok();
  DeviceGuard guard;
  KDN_TRY(use_device_of(none ? workspace : o, guard));
  cudaStream_t st = (cudaStream_t)stream;
  if (workspace != nullptr) KDN_TRY(clear_status(workspace, st));
  if (none) return ok();
  kdn::WindowArgs a{};
  a.q = q, a.k = k, a.v = v, a.in_dtype = dims->in_dtype, a.out_dtype = dims->out_dtype, a.lens = lens, a.zero_rest = zero_rest != 0;
  a.B = dims->B, a.H = dims->H, a.Hkv = kv_heads, a.L = dims->L, a.scale = scale;
  a.window = window < dims->L ? window : dims->L, a.n_sink = n_sink < dims->L ? n_sink : dims->L;  // t - j < L
  a.o = o, a.lse = lse, a.status = static_cast<unsigned*>(workspace);
  return cuda_status(kdn::launch_window_attn(dims->dk, dims->dv, a, st), "windowed attention launch");
}

kdn_status kdn_window_attn_backward(const kdn_dims* dims, int kv_heads, const void* q, const void* k, const void* v,
                                    const int* lens, int zero_rest, int window, int n_sink, float scale, const void* o,
                                    const float* lse, const void* dO, void* dq, void* dk, void* dv, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  KDN_TRY(window_checks(dims, kv_heads, window, n_sink, scale));
  const bool none = dims->L == 0;
  const size_t in = elem_bytes(dims->in_dtype), rows = (size_t)dims->B * dims->H * dims->L, keys = rows / dims->H * kv_heads;
  const Span q_{"q", q, rows * dims->dk * in}, k_{"k", k, keys * dims->dk * in}, v_{"v", v, keys * dims->dv * in};
  const Span o_{"o", o, rows * dims->dv * elem_bytes(dims->out_dtype)}, lse_{"lse", lse, rows * 4};
  const Span ws_{"workspace", workspace, workspace_bytes};
  const Span dO_{"dO", dO, o_.bytes}, dq_{"dq", dq, q_.bytes}, dk_{"dk", dk, k_.bytes}, dv_{"dv", dv, v_.bytes};
  KDN_TRY(check_apart({dq_, dk_, dv_, ws_}, {q_, k_, v_, o_, lse_, dO_, ints("lens", lens, dims->B)}));
  KDN_TRY(check_ptr(q, "q", 16, none));
  KDN_TRY(check_ptr(k, "k", 16, none));
  KDN_TRY(check_ptr(v, "v", 16, none));
  KDN_TRY(check_ptr(o, "o", 16, none));
  KDN_TRY(check_ptr(lse, "lse", 4, none));
  KDN_TRY(check_ptr(dO, "dO", 16, none));
  KDN_TRY(check_ptr(dq, "dq", 16, none));
  KDN_TRY(check_ptr(dk, "dk", 16, none));
  KDN_TRY(check_ptr(dv, "dv", 16, none));
  KDN_TRY(check_ptr(lens, "lens", 4, true));
  KDN_TRY(check_workspace(workspace, workspace_bytes, kdn_window_workspace_bytes(dims, kv_heads, window, n_sink, 1)));
  DeviceGuard guard;
  KDN_TRY(use_device_of(workspace, guard));
  cudaStream_t st = (cudaStream_t)stream;
  if (none) return clear_status(workspace, st);
  kdn::WindowArgs a{};
  a.q = q, a.k = k, a.v = v, a.in_dtype = dims->in_dtype, a.out_dtype = dims->out_dtype, a.lens = lens, a.zero_rest = zero_rest != 0;
  a.B = dims->B, a.H = dims->H, a.Hkv = kv_heads, a.L = dims->L, a.scale = scale;
  a.window = window < dims->L ? window : dims->L, a.n_sink = n_sink < dims->L ? n_sink : dims->L;  // t - j < L
  a.o = const_cast<void*>(o), a.lse = const_cast<float*>(lse), a.status = static_cast<unsigned*>(workspace);
  a.dO = dO, a.dq = dq, a.dk = dk, a.dv = dv;
  a.scratch = static_cast<char*>(workspace) + kStatusBytes;
  a.delta = static_cast<float*>(a.scratch);
  return cuda_status(kdn::launch_window_attn_backward(dims->dk, dims->dv, a, st), "windowed attention backward launch");
}

size_t kdn_pages_workspace_bytes(const kdn_pages* pages) {
  if (!pages_sizes_ok(pages)) return 0;
  return refused_at(pages) + round256((size_t)pages->rows * sizeof(int));
}

kdn_status kdn_pages_reserve(const kdn_pages* pages, int n, const int* rows, const int* counts, int count,
                             void* workspace, size_t workspace_bytes, void* stream) {
  DeviceGuard guard;
  if (counts == nullptr && count < 0) return fail(KDN_ERR_INVALID_ARG, "count must be >= 0");
  KDN_TRY(book_checks(pages, n, workspace, workspace_bytes, {"moves", nullptr, 0}, {ints("rows", rows, n), ints("counts", counts, n)}, guard));
  KDN_TRY(check_ptr(rows, "rows", 4, n == 0));
  KDN_TRY(check_ptr(counts, "counts", 4, true));
  return cuda_status(kdn::launch_pages_reserve(pages_args(pages, workspace), n, rows, counts, count, (cudaStream_t)stream),
                     "page reservation launch");
}

kdn_status kdn_pages_fork(const kdn_pages* pages, int n, const int* src_rows, const int* dst_rows, int* moves,
                          void* workspace, size_t workspace_bytes, void* stream) {
  DeviceGuard guard;
  KDN_TRY(book_checks(pages, n, workspace, workspace_bytes, ints("moves", moves, 2LL * n), {ints("src_rows", src_rows, n), ints("dst_rows", dst_rows, n)}, guard));
  KDN_TRY(check_ptr(src_rows, "src_rows", 4, n == 0));
  KDN_TRY(check_ptr(dst_rows, "dst_rows", 4, n == 0));
  KDN_TRY(check_ptr(moves, "moves", 8, n == 0));
  return cuda_status(kdn::launch_pages_fork(pages_args(pages, workspace), n, src_rows, dst_rows, moves, (cudaStream_t)stream),
                     "page fork launch");
}

kdn_status kdn_pages_free(const kdn_pages* pages, int n, const int* rows, void* workspace, size_t workspace_bytes,
                          void* stream) {
  DeviceGuard guard;
  KDN_TRY(book_checks(pages, n, workspace, workspace_bytes, {"moves", nullptr, 0}, {ints("rows", rows, n)}, guard));
  KDN_TRY(check_ptr(rows, "rows", 4, n == 0));
  return cuda_status(kdn::launch_pages_free(pages_args(pages, workspace), n, rows, (cudaStream_t)stream), "page free launch");
}

kdn_status kdn_pages_compact(const kdn_pages* pages, int* moves, void* workspace, size_t workspace_bytes, void* stream) {
  DeviceGuard guard;
  KDN_TRY(book_checks(pages, 0, workspace, workspace_bytes, ints("moves", moves, pages ? pages->num_pages / 2 * 2LL : 0), {}, guard));
  KDN_TRY(check_ptr(moves, "moves", 8, pages->num_pages < 2));
  return cuda_status(kdn::launch_pages_compact(pages_args(pages, workspace), moves, (cudaStream_t)stream),
                     "page compaction launch");
}

kdn_status kdn_pages_copy(int n, const int* moves, int num_pages, int page_size, int kv_heads, int dk, int dv,
                          kdn_dtype dtype, void* k_pages, void* v_pages, void* stream) {
  if (n < 0 || num_pages < 1) return fail(KDN_ERR_INVALID_ARG, "n must be >= 0 and num_pages >= 1");
  if (page_size < 1 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return fail(KDN_ERR_UNSUPPORTED, "page_size must be a power of two up to 1024");
  KDN_TRY(check_pool(kv_heads, dk, dv, dtype));
  if ((long long)kv_heads * page_size * 128 * 4 > (1LL << 40)) return fail(KDN_ERR_UNSUPPORTED, "page too large");
  const size_t head = (size_t)kv_heads * page_size * elem_bytes(dtype);
  KDN_TRY(check_apart({{"k_pages", k_pages, num_pages * head * dk}, {"v_pages", v_pages, num_pages * head * dv}},
                      {ints("moves", moves, 2LL * n)}));
  KDN_TRY(check_ptr(moves, "moves", 8, n == 0));
  KDN_TRY(check_ptr(k_pages, "k_pages", 16, false));
  KDN_TRY(check_ptr(v_pages, "v_pages", 16, false));
  if (n == 0) return ok();
  DeviceGuard guard;
  KDN_TRY(use_device_of(k_pages, guard));
  return cuda_status(kdn::launch_pages_copy(moves, n, num_pages, head * dk, head * dv, k_pages, v_pages, (cudaStream_t)stream),
                     "page copy launch");
}

kdn_status kdn_pages_write(const kdn_pages* pages, int n, const int* rows, const int* counts, int tokens, int kv_heads,
                           int dk, int dv, kdn_dtype dtype, const void* k_new, const void* v_new, void* k_pages,
                           void* v_pages, void* stream) {
  return write_pages(pages, n, rows, counts, tokens, kv_heads, dk, dv, dtype, k_new, v_new, k_pages, v_pages, nullptr, 0, stream);
}

kdn_status kdn_pages_write_reserved(const kdn_pages* pages, int n, const int* rows, const int* counts, int tokens,
                                    int kv_heads, int dk, int dv, kdn_dtype dtype, const void* k_new, const void* v_new,
                                    void* k_pages, void* v_pages, const void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (workspace == nullptr) return fail(KDN_ERR_INVALID_ARG, "workspace is NULL");
  return write_pages(pages, n, rows, counts, tokens, kv_heads, dk, dv, dtype, k_new, v_new, k_pages, v_pages,
                     const_cast<void*>(workspace), workspace_bytes, stream);
}

size_t kdn_paged_step_workspace_bytes(const kdn_pages* pages, int n, int H, int kv_heads, int dk, int dv,
                                      kdn_dtype in_dtype, int window, int n_sink) {
  if (!pages_sizes_ok(pages) || n < 0 || H < 1 || kv_heads < 1 || H % kv_heads != 0 || !pool_dim(dk) || !pool_dim(dv) ||
      window < 0 || n_sink < 0)
    return 0;
  if (n == 0) return kStatusBytes;
  long long most = (long long)pages->max_pages * pages->page_size;
  if (window > 0 && (long long)window + n_sink < most) most = (long long)window + n_sink;
  const int splits = kdn::paged_step_splits(dk, dv, in_dtype, n, H, kv_heads, most);
  return kStatusBytes + round256(kdn::paged_step_part_floats(dv, n, H, splits) * sizeof(float));
}

kdn_status kdn_paged_attn_step(const kdn_pages* pages, int n, const int* rows, int H, int kv_heads, int dk, int dv,
                               kdn_dtype in_dtype, kdn_dtype out_dtype, const void* q, const void* k_pages,
                               const void* v_pages, int window, int n_sink, float scale, void* o, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  KDN_TRY(check_pages(pages));
  if (n < 0 || H < 1) return fail(KDN_ERR_INVALID_ARG, "n must be >= 0 and H >= 1");
  KDN_TRY(check_pool(kv_heads, dk, dv, in_dtype));
  KDN_TRY(check_heads(H, kv_heads));
  if (out_dtype != KDN_F32 && out_dtype != KDN_BF16) return fail(KDN_ERR_INVALID_ARG, "bad out_dtype");
  KDN_TRY(check_window(window, 0, n_sink, scale));
  if ((long long)n * H > (1 << 24)) return fail(KDN_ERR_UNSUPPORTED, "n*H must be at most 2^24");
  if (rows == nullptr && n > pages->rows) return fail(KDN_ERR_INVALID_ARG, "n exceeds the table's rows");
  const size_t heads = (size_t)n * H, pool = (size_t)pages->num_pages * kv_heads * pages->page_size * elem_bytes(in_dtype);
  KDN_TRY(check_apart({{"o", o, heads * dv * elem_bytes(out_dtype)}, {"lse", lse, heads * 4}, {"workspace", workspace, workspace_bytes}},
                      {{"q", q, heads * dk * elem_bytes(in_dtype)}, {"k_pages", k_pages, pool * dk}, {"v_pages", v_pages, pool * dv},
                       table_of(pages), lens_of(pages), ints("rows", rows, n)}));
  KDN_TRY(check_ptr(pages->table, "table", 4, false));
  KDN_TRY(check_ptr(pages->lens, "lens", 4, false));
  KDN_TRY(check_ptr(rows, "rows", 4, true));
  KDN_TRY(check_ptr(q, "q", 16, n == 0));
  KDN_TRY(check_ptr(k_pages, "k_pages", 16, false));
  KDN_TRY(check_ptr(v_pages, "v_pages", 16, false));
  KDN_TRY(check_ptr(o, "o", 16, n == 0));
  KDN_TRY(check_ptr(lse, "lse", 4, true));
  const size_t need = kdn_paged_step_workspace_bytes(pages, n, H, kv_heads, dk, dv, in_dtype, window, n_sink);
  if (workspace != nullptr || need > kStatusBytes) KDN_TRY(check_workspace(workspace, workspace_bytes, need));
  if (n == 0) return ok();
  DeviceGuard guard;
  KDN_TRY(use_device_of(k_pages, guard));
  kdn::PagedStepArgs a{};
  a.q = q, a.k_pages = k_pages, a.v_pages = v_pages, a.in_dtype = in_dtype, a.out_dtype = out_dtype;
  a.n = n, a.H = H, a.Hkv = kv_heads, a.num_pages = pages->num_pages, a.page_size = pages->page_size;
  a.rows = pages->rows, a.max_pages = pages->max_pages, a.table = pages->table, a.lens = pages->lens, a.row = rows;
  a.window = window, a.n_sink = n_sink, a.scale = scale, a.o = o, a.lse = lse;
  long long most = (long long)pages->max_pages * pages->page_size;
  if (window > 0 && (long long)window + n_sink < most) most = (long long)window + n_sink;
  a.splits = kdn::paged_step_splits(dk, dv, in_dtype, n, H, kv_heads, most);
  if (a.splits > 1) a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kStatusBytes);
  return cuda_status(kdn::launch_paged_step(dk, dv, a, (cudaStream_t)stream), "paged decode step launch");
}

}  // extern "C"
