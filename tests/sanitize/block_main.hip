// Host driver for the sanitizer build of the lookup in a block map
// (csrc/block.h): maps held in exactly sized buffers, as callers may hand them
// over, and every index that a launch over moe_max_blocks entries looks at.
// Runs without a GPU.  Test infrastructure only.
#include <stdio.h>

#include <vector>

#include "block.h"

static int g_fail = 0;
#define CHECK(cond)                                                      \
  do {                                                                   \
    if (!(cond)) {                                                       \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                          \
    }                                                                    \
  } while (0)

int main() {
  for (int n : {0, 1, 2, 17}) {
    std::vector<int4> map;
    for (int b = 0; b < n; ++b) map.push_back(make_int4(b, 3 * b, 3, 16));
    map.shrink_to_fit();
    const int32_t length = n;
    for (int b = 0; b < 305; ++b) {
      int4 e = make_int4(-1, -1, -1, -1);
      const bool in = moe::map_entry(map.data(), &length, b, e);
      CHECK(in == (b < n));
      CHECK(in ? e.x == b && e.y == 3 * b && e.z == 3 && e.w == 16 : e.x == -1);
    }
  }
  if (!g_fail) printf("block map sanitizer driver ok\n");
  return g_fail != 0;
}
