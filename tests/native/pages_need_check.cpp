// Host-only check of the sums behind a reservation (no GPU, no CUDA headers): needs that pass 31 and 32 bits are still
// larger than any pool.  Exit status 0 when every check holds; the failing check is printed otherwise.
#include <cstdio>
#include <initializer_list>

#include "pages_need.h"

namespace {
int g_failures = 0;
void check(bool ok, const char* what, long long a, long long b) {
  if (!ok) std::printf("FAILED: %s (%lld, %lld)\n", what, a, b), ++g_failures;
}
kdn::PageSum sum(int rows, int len, int count, int page) {
  kdn::PageSum need = 0;
  for (int r = 0; r < rows; ++r) need += kdn::more_pages(len, count, page);
  return need;
}
}  // namespace

int main() {
  static_assert(sizeof(kdn::PageSum) == 8, "64 bits");
  check(kdn::more_pages(0, 0, 16) == 0 && kdn::more_pages(0, 1, 16) == 1 && kdn::more_pages(15, 1, 16) == 0 &&
            kdn::more_pages(16, 1, 16) == 1 && kdn::more_pages(1, 31, 16) == 1 && kdn::more_pages(1, 32, 16) == 2,
        "pages of one row", 0, 0);
  check(kdn::more_pages(0, 1 << 30, 1) == 1ull << 30 && kdn::more_pages((1 << 30) - 1, 1, 1) == 1, "the longest row", 0, 0);
  // 2^31, 2^32, 2^32 + small, 2^48 pages: a sum of 32 bits would be negative, 0 or small
  const struct { int rows, count; } calls[] = {{2, 1 << 30}, {4, 1 << 30}, {4096, 1 << 20}, {4097, 1 << 20}, {1 << 18, 1 << 30}};
  for (auto c : calls) {
    const kdn::PageSum need = sum(c.rows, 0, c.count, 1);
    check(need == (kdn::PageSum)c.rows * (kdn::PageSum)c.count, "the sum is exact", c.rows, c.count);
    for (int pool : {1, 8, 1 << 20, 1 << 30}) check(kdn::pool_too_small(need, pool), "refused", c.rows, pool);
  }
  for (int pool : {1, 8, 1 << 30}) {
    check(!kdn::pool_too_small(0, pool) && !kdn::pool_too_small((kdn::PageSum)pool, pool), "what fits is not refused", pool, 0);
    check(kdn::pool_too_small((kdn::PageSum)pool + 1, pool), "one too many", pool, 0);
  }
  if (g_failures == 0) std::printf("ok\n");
  return g_failures != 0;
}
