// Host-only check of where the rows kernel's CTAs keep the records of cut groups
// (compiled by tests/test_cut_records_cpu.py).  Nothing orders one CTA's writes
// before another's within a launch, so every record must be written by one CTA
// alone: the one that clears it when it starts.
#include <cstdio>
#include <set>
#include <vector>

#include "ops.h"

using namespace pkv;

int main() {
  int fails = 0;
  for (int W : {4, 6, 12}) {
    for (int ctas : {2, 3, 7, 152, 456}) {
      std::vector<int> owner(static_cast<size_t>(W) * ctas, -1);   // the CTA that clears the record
      for (int b = 0; b < ctas; ++b)
        for (int w = 0; w < W; ++w) {
          const int i = cut_record(b, W, true, w);
          if (i < 0 || i >= W * ctas || owner[i] != -1) ++fails;
          else owner[i] = b;
        }
      for (bool solo : {false, true}) {
        std::set<int> used;
        for (int b = 0; b < ctas; ++b)
          for (int w = 0; w < (solo ? W : 1); ++w) {   // (a CTA's record is left by its warp 0)
            const int i = cut_record(b, W, solo, w);
            if (i < 0 || i >= W * ctas || owner[i] != b || !used.insert(i).second) ++fails;
          }
      }
    }
  }
  std::printf(fails ? "FAIL %d\n" : "ok\n", fails);
  return fails != 0;
}
