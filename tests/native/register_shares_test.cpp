// Rule of csrc/register_shares.h: which register counts may run a kernel that splits 72 a thread by role.
#include <cstdio>

#include "register_shares.h"

#define CHECK(x)                                          \
  do {                                                    \
    if (!(x)) {                                           \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #x); \
      return 1;                                           \
    }                                                     \
  } while (0)

int main() {
  int calls = 0;
  auto uses = [&](int n) { return [&calls, n] { return ++calls, n; }; };
  for (int n = 65; n <= 72; ++n) CHECK(la::RegisterShares().fit(0, 72, uses(n)));  // all given 72
  for (int n : {1, 32, 56, 57, 63, 64}) CHECK(!la::RegisterShares().fit(0, 72, uses(n)));
  la::RegisterShares r;
  calls = 0;
  CHECK(!r.fit(0, 72, uses(-1)) && calls == 1);  // a failed query refuses this call ...
  CHECK(r.fit(0, 72, uses(70)) && calls == 2);   // ... and not the next one
  CHECK(r.fit(0, 72, uses(10)) && calls == 2);   // known
  CHECK(!r.fit(1, 72, uses(10)) && calls == 3);  // another device has an answer of its own
  CHECK(r.fit(0, 72, uses(10)) && !r.fit(1, 72, uses(72)) && calls == 3);
  std::puts("ok");
  return 0;
}
