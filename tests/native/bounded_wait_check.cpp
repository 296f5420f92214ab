// Host-only check of kdn::wait_bounded against a fake clock and a fake event (no GPU, no CUDA headers).
// Exit status 0 when every check holds; the failing check is printed otherwise.
#include <cstdio>

#include "bounded_wait.h"

namespace {

long long g_clock = 0;
long long g_held_up = 0;     // clocks that pass between a failed try and the next look at the clock, once
long long g_ready_at = -1;   // the event's time; -1: never
int g_tries = 0;
int g_failures = 0;

bool ready() {
  ++g_tries;
  g_clock += 1;
  return g_ready_at >= 0 && g_clock >= g_ready_at;
}
long long now() {
  if (g_tries >= 2) g_clock += g_held_up, g_held_up = 0;
  return g_clock;
}
bool wait(long long ready_at, long long held_up, long long most) {
  g_clock = 0, g_tries = 0, g_ready_at = ready_at, g_held_up = held_up;
  return kdn::wait_bounded(ready, now, most);
}
void check(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAILED: %s\n", what);
    ++g_failures;
  }
}

}  // namespace

int main() {
  check(wait(0, 0, 100) && g_tries == 1, "an event that is there costs one try");
  check(wait(50, 0, 100), "an event within the limit");
  check(!wait(-1, 0, 100) && g_clock <= 110, "an event that never comes ends at the limit");
  check(!wait(10000, 0, 100), "an event long behind the limit");
  check(wait(60, 5000, 100), "held up past the limit, the event there meanwhile");
  check(!wait(-1, 5000, 100), "held up past the limit, no event");
  if (g_failures == 0) std::printf("ok\n");
  return g_failures != 0;
}
