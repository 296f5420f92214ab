// Host-only check of what the windowed attention's backward leaves behind a wait that gave up: mark_queries and mark_key,
// the kernels' own code compiled for the host, on host arrays.  No GPU call is made.  Exit status 0 when every check holds.
#include "window_bwd_tc.cu"

#include <cstdio>
#include <vector>

namespace kdn {
bool make_bf16_tmap_rows(CUtensorMap*, const void*, int, int, int, int) { return false; }  // never called here
}

using namespace kdn;

namespace {

constexpr int D = 64;
constexpr uint32_t kOld = 0x40e040e0u;
int g_failures = 0;
void check(bool ok, const char* what, int a, int b) {
  if (!ok) std::printf("FAILED: %s (case %d, %d)\n", what, a, b), ++g_failures;
}

struct Case {
  int B, H, Hkv, L, window, n_sink;
  std::vector<int> lens;
  bool zero_rest;
  int ctas;
  bool cut;  // some key tile is cut into parts
};
int length(const Case& c, int b) { return c.lens[b] < 0 ? 0 : c.lens[b] > c.L ? c.L : c.lens[b]; }

WindowArgs args(const Case& c) {
  WindowArgs p{};
  p.lens = c.lens.data(), p.zero_rest = c.zero_rest, p.B = c.B, p.H = c.H, p.Hkv = c.Hkv, p.L = c.L;
  p.window = c.window < c.L ? c.window : c.L, p.n_sink = c.n_sink < c.L ? c.n_sink : c.L, p.in_dtype = p.out_dtype = kBF16;
  return p;
}

void queries(const Case& c, int number) {
  WindowArgs p = args(c);
  const QueryPass qp = query_pass(c.B, c.H, c.Hkv, c.L);
  const int half_words = D / 4;  // half of a row of bf16, in words
  const size_t halves = (size_t)c.B * c.H * c.L * 2;
  std::vector<uint32_t> dq;
  p.dq = nullptr;
  std::vector<int> times(halves, 0);
  auto mark = [&](unsigned round, int cta) {
    dq.assign(halves * half_words, kOld);
    p.dq = dq.data();
    for (int half = 0; half < 2; ++half)
      for (int row = 0; row < kT; ++row) mark_queries<D>(p, qp, round, cta, c.ctas, half, row);
    std::vector<char> r;
    for (size_t e = 0; e < halves; ++e) {
      const uint32_t first = dq[e * half_words];
      bool same = first == kOld || first == 0u || first == nan_word(kBF16);
      for (int w = 1; w < half_words; ++w) same = same && dq[e * half_words + w] == first;
      r.push_back(!same ? '?' : first == kOld ? '.' : first == 0u ? '0' : 'n');
    }
    return r;
  };
  for (int cta = 0; cta < c.ctas; ++cta) {
    const unsigned rounds = (qp.works + c.ctas - 1) / c.ctas;
    std::vector<char> later = mark(rounds, cta);
    for (char k : later) check(k == '.', "nothing behind the last round", number, cta);
    for (int r = (int)rounds - 1; r >= 0; --r) {
      std::vector<char> now = mark(r, cta);
      size_t tile = SIZE_MAX;
      for (size_t e = 0; e < halves; ++e) {
        check(now[e] != '?', "whole halves of rows", number, cta);
        if (later[e] != '.') check(now[e] == later[e], "a later round's rows are marked too", number, cta);
        if (now[e] == later[e]) continue;
        ++times[e];
        const size_t row = e / 2, mine = row / c.L * 1000 + row % c.L / kT;
        check(tile == SIZE_MAX || tile == mine, "a round is one query tile", number, cta);
        tile = mine;
        const int b = row / ((size_t)c.H * c.L), t = row % c.L;
        check(now[e] == (t < length(c, b) ? 'n' : '0'), "NaN in the sequence, zero behind it", number, t);
      }
      later = now;
    }
  }
  for (size_t e = 0; e < halves; ++e) {
    const int b = e / 2 / ((size_t)c.H * c.L), t = e / 2 % c.L;
    check(times[e] == (t < length(c, b) || c.zero_rest ? 1 : 0), "every row belongs to one round of one CTA", number, t);
  }
}

void keys(const Case& c, int number) {
  WindowArgs p = args(c);
  KeyPass plan = cut(c.B, c.H, c.Hkv, c.L, p.window, p.n_sink);
  const int bh = c.B * c.Hkv, tiles = (c.L + kT - 1) / kT;
  const long long ctas = key_ctas(plan, bh, tiles), slots = cut_ctas(plan, bh, tiles);
  check(c.cut == (slots > 0), "this case is cut, or not", number, (int)slots);
  const size_t rows = (size_t)bh * c.L, slot_rows = (size_t)slots * 2 * kT;
  const int words = D / 2;
  std::vector<uint32_t> grad[2];
  std::vector<uint32_t> part(slot_rows * D + 1, kOld);
  for (auto& g : grad) g.assign(rows * words, kOld);
  plan.part = reinterpret_cast<float*>(part.data());
  p.dv = grad[0].data(), p.dk = grad[1].data();
  std::vector<int> times(rows, 0);
  for (long long x = 0; x < ctas; ++x) {
    KeyPass kp = plan;
    int at;
    const int parts = key_tile_of(kp, bh, tiles, (unsigned)x, at);
    const int len = length(c, kp.head / c.Hkv);
    if (kp.tile * kT >= len) continue;  // such a CTA has nothing to do
    for (int half = 0; half < 2; ++half)
      for (int key = 0; key < kT; ++key) mark_key<D>(p, kp, parts, (unsigned)x, len, half, key);
    size_t slot = 0;
    if (parts > 1) {
      check(parts_of(kp, bh, tiles, kp.head, kp.tile, slot) == parts, "the join reads as many parts", number, (int)x);
      check(slot + at == (size_t)x && x < slots, "the join reads this part's slot", number, (int)x);
      for (size_t w = (size_t)x * 2 * kT * D; w < (size_t)(x + 1) * 2 * kT * D; ++w)
        if (part[w] != nan_word(kF32)) check(false, "a cut tile's slot is NaN", number, (int)x);
    }
    for (int key = 0; key < kT && kp.tile * kT + key < len; ++key) times[(size_t)kp.head * c.L + kp.tile * kT + key] = parts > 1 ? 2 : 1;
  }
  check(part.back() == kOld, "nothing behind the slots", number, 0);
  for (size_t e = 0; e < rows; ++e) {
    const int t = e % c.L;
    check((times[e] > 0) == (t < length(c, (int)(e / c.L / c.Hkv))), "every key belongs to a CTA", number, t);
    for (auto& g : grad)
      for (int w = 0; w < words; ++w)
        if (g[e * words + w] != (times[e] == 1 ? nan_word(kBF16) : kOld)) check(false, "whole tiles' keys are NaN, nothing else", number, t);
  }
}

}  // namespace

int main() {
  const Case cases[] = {
      {1, 1, 1, 1, 1, 0, {1}, false, 1, false},
      {2, 4, 2, 300, 50, 4, {300, 129}, true, 3, true},
      {3, 3, 1, 515, 100, 0, {515, 0, 1}, false, 4, true},
      {8, 12, 12, 257, 1000, 200, {9999, -5, 1, 128, 129, 200, 257, 0}, true, 50, false},
      {10, 5, 5, 1000, 30, 3, {500, 1000, 1, 0, 7, 999, 128, 256, 257, 640}, true, 7, true},
  };
  int number = 0;
  for (const Case& c : cases) queries(c, number), keys(c, number), ++number;
  if (g_failures == 0) std::printf("ok\n");
  return g_failures != 0;
}
