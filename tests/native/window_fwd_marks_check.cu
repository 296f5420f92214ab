// Host-only check of what the windowed attention's forward leaves behind a wait that gave up: mark_rest, the kernel's own
// code compiled for the host, on host arrays.  No GPU call is made.  Exit status 0 when every check holds.
#include "window_attn_tc.cu"

#include <cmath>
#include <cstdio>
#include <vector>

namespace kdn {
bool make_bf16_tmap_rows(CUtensorMap*, const void*, int, int, int, int) { return false; }  // never called here
}

using namespace kdn;

namespace {

constexpr int D = 64;
int g_failures = 0;
void check(bool ok, const char* what, int a, int b) {
  if (!ok) std::printf("FAILED: %s (case %d, %d)\n", what, a, b), ++g_failures;
}

struct Rows {
  std::vector<char> of;  // 'n' NaN, '0' zero, '.' as it was, '?' anything else or o and lse apart
};

struct Case {
  int B, H, Hkv, L, window, n_sink;
  std::vector<int> lens;
  bool zero_rest;
  int out_dtype, ctas;
};

struct Run {
  const Case& c;
  Schedule sch;
  WindowArgs p{};
  std::vector<uint32_t> o;
  std::vector<float> lse;
  explicit Run(const Case& c_) : c(c_) {
    const int G = c.H / c.Hkv, tiles = (c.L + kT - 1) / kT;
    sch = make_schedule(c.B, c.H, c.Hkv, c.L);
    check(sch.works == (unsigned)(c.B * c.Hkv * sch.tile_groups) * sch.group.d && G > 0 && tiles > 0, "number of works", 0, 0);
    p.lens = c.lens.data(), p.zero_rest = c.zero_rest, p.B = c.B, p.H = c.H, p.Hkv = c.Hkv, p.L = c.L;
    p.window = c.window, p.n_sink = c.n_sink, p.out_dtype = c.out_dtype;
  }
  Rows mark(unsigned round, unsigned cta) {
    const int words = D * (c.out_dtype == kBF16 ? 2 : 4) / 4;
    const size_t rows = (size_t)c.B * c.H * c.L;
    o.assign(rows * words, 0x40e040e0u), lse.assign(rows, 7.f);
    p.o = o.data(), p.lse = lse.data();
    for (int i = 0; i < 2; ++i)
      for (int row = 0; row < kT; ++row) mark_rest<D>(p, sch, round, cta, c.ctas, i, row);
    Rows r;
    for (size_t e = 0; e < rows; ++e) {
      char kind = std::isnan(lse[e]) ? 'n' : lse[e] == 0.f ? '0' : lse[e] == 7.f ? '.' : '?';
      const uint32_t want = kind == 'n' ? nan_word(c.out_dtype) : kind == '0' ? 0u : 0x40e040e0u;
      for (int w = 0; w < words; ++w)
        if (o[e * words + w] != want) kind = '?';
      r.of.push_back(kind);
    }
    return r;
  }
};

void run(const Case& c, int number) {
  Run run(c);
  const size_t rows = (size_t)c.B * c.H * c.L;
  std::vector<int> times(rows, 0);
  for (int cta = 0; cta < c.ctas; ++cta) {
    const unsigned rounds = (run.sch.works + c.ctas - 1) / c.ctas;
    Rows later = run.mark(rounds, cta);
    for (char k : later.of) check(k == '.', "nothing behind the last round", number, cta);
    for (int r = (int)rounds - 1; r >= 0; --r) {
      Rows now = run.mark(r, cta);
      std::vector<size_t> pairs;  // (head, tile) of what this work adds
      for (size_t e = 0; e < rows; ++e) {
        check(now.of[e] != '?', "whole rows, o and lse alike", number, cta);
        if (later.of[e] != '.') check(now.of[e] == later.of[e], "a later round's rows are marked too", number, cta);
        if (now.of[e] == later.of[e]) continue;
        ++times[e];
        const size_t pair = e / c.L * 1000 + e % c.L / kT;
        if (pairs.empty() || pairs.back() != pair) pairs.push_back(pair);
      }
      check(pairs.size() <= 2, "a round is one work: two tiles at most", number, cta);
      later = now;
    }
    for (size_t e = 0; e < rows; ++e) {  // from the first work on: every row of this CTA, with the value that belongs there
      const int b = e / ((size_t)c.H * c.L), t = e % c.L, n = c.lens[b] < 0 ? 0 : c.lens[b] > c.L ? c.L : c.lens[b];
      if (later.of[e] != '.') check(later.of[e] == (t < n ? 'n' : '0'), "NaN in the sequence, zero behind it", number, t);
    }
  }
  for (size_t e = 0; e < rows; ++e) {
    const int b = e / ((size_t)c.H * c.L), t = e % c.L, n = c.lens[b] < 0 ? 0 : c.lens[b] > c.L ? c.L : c.lens[b];
    check(times[e] == (t < n || c.zero_rest ? 1 : 0), "every row belongs to one round of one CTA", number, t);
  }
}

}  // namespace

int main() {
  const Case cases[] = {
      {1, 1, 1, 1, 1, 0, {1}, false, kBF16, 1},
      {2, 4, 2, 300, 50, 4, {300, 129}, true, kBF16, 3},
      {3, 3, 1, 515, 100, 0, {515, 0, 1}, false, kF32, 4},
      {2, 6, 2, 257, 1000, 200, {9999, -5}, true, kF32, 5},
      {1, 5, 5, 640, 30, 3, {500}, true, kBF16, 7},
  };
  int number = 0;
  for (const Case& c : cases) run(c, number++);
  if (g_failures == 0) std::printf("ok\n");
  return g_failures != 0;
}
