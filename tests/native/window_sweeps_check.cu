// Host-only check of which query tiles of the windowed attention's backward take a first sweep for delta: the kernel's own
// query_work, compiled for the host.  No GPU call is made.  Exit status 0 when every check holds.
#include "window_bwd_tc.cu"

#include <cstdio>

namespace kdn {
bool make_bf16_tmap_rows(CUtensorMap*, const void*, int, int, int, int) { return false; }  // never called here
}

using namespace kdn;

namespace {
int g_failures = 0;
void check(bool ok, const char* what, int a, int b, int c) {
  if (!ok) std::printf("FAILED: %s (window %d, sinks %d, tile %d)\n", what, a, b, c), ++g_failures;
}
}  // namespace

int main() {
  const int windows[] = {1, 2, 12, 64, 128, 129, 200, 1000, 1 << 20}, sinks[] = {0, 1, 4, 100, 128, 129, 300, 2048, 1 << 20};
  for (int window : windows)
    for (int n_sink : sinks)
      for (int type : {kBF16, kF32}) {
        WindowArgs p{};
        p.B = 1, p.H = 1, p.Hkv = 1, p.L = 4096, p.out_dtype = type;
        p.window = window < p.L ? window : p.L, p.n_sink = n_sink < p.L ? n_sink : p.L;
        const QueryPass qp = query_pass(1, 1, 1, p.L);
        for (unsigned x = 0; x < qp.works; ++x) {
          const QueryWork w = query_work(p, qp, x);
          const int tile = w.t0 / kT, t = w.t0 + kT - 1;
          int most = 0;  // keys that the tile's last row sees
          for (int j = 0; j <= t; ++j) most += visible(t, j, p.window, p.n_sink);
          check(w.before == 0 || w.before == w.n, "a first sweep is whole", window, n_sink, tile);
          if (w.t0 == 0) check(w.before == w.n, "the first rows take one", window, n_sink, tile);
          if (w.before && w.t0) check(w.n <= 3 && most <= 256 + 128, "a first sweep is short, and rows see few keys", window, n_sink, tile);
          if (w.t0 && most <= 128) check(w.before == w.n, "rows that see few keys take one", window, n_sink, tile);
        }
      }
  if (g_failures == 0) std::printf("ok\n");
  return g_failures != 0;
}
