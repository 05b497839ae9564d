// Index arithmetic of the paged cache (csrc/kv_view.h) on ordinary and hostile
// device arrays: every row, page and position it yields stays inside what the
// call was given.  Built for the host under AddressSanitizer and
// UndefinedBehaviorSanitizer.
#include "../../weight_only_mixed_amd/csrc/kv_view.h"

#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

static int failures = 0;
#define CHECK(c)                                             \
  do {                                                       \
    if (!(c)) {                                              \
      if (++failures < 20) printf("line %d: %s\n", __LINE__, #c); \
    }                                                        \
  } while (0)

using namespace slq;

static unsigned long long state = 12345;
static int rnd(int lo, int hi) {
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return lo + (int)((state >> 33) % (unsigned long long)((long long)hi - lo + 1));
}

int main() {
  const int hostile[] = {INT_MIN, -1000, -1, 0, 1, 15, 16, 17, 1000, INT_MAX};
  for (int round = 0; round < 20000; ++round) {
    const int batch = rnd(1, 4), shift = rnd(4, 8), width = rnd(1, 6), rows = rnd(0, 40);
    const int pages = rnd(0, 8);
    std::vector<int> table(batch * width), lens(batch), cu(batch + 1);
    const bool bad = round & 1;
    for (int &t : table) t = bad && rnd(0, 3) == 0 ? hostile[rnd(0, 9)] : rnd(-1, pages);
    int at = 0;
    for (int b = 0; b <= batch; ++b) {
      cu[b] = bad && rnd(0, 4) == 0 ? hostile[rnd(0, 9)] : at;
      at += rnd(0, 12);
    }
    for (int &l : lens) l = bad && rnd(0, 3) == 0 ? hostile[rnd(0, 9)] : rnd(0, width << shift);
    const SeqView s{table.data(), lens.data(), cu.data(), width, batch, width, rows};
    for (int b = 0; b < batch; ++b) {
      const KvSpan sp = kv_span(s, shift, b);
      CHECK(sp.row0 >= 0 && sp.n >= 0 && sp.row0 + sp.n <= rows);
      CHECK(sp.len >= 0 && sp.len <= width << shift);
      // every existing new row lies in exactly one page's part
      std::vector<int> seen(sp.n > 0 ? sp.n : 1, 0);
      const int first = kv_first_page(sp, shift), last = kv_last_page(sp, shift);
      CHECK(first >= 0 && last - first <= sp.n);
      for (int p = first; p <= last; ++p) {
        const int id = kv_page(s, pages, b, p);
        CHECK(id >= -1 && id < pages);
        const KvPart part = kv_part(sp, shift, p);
        CHECK(part.lo >= 0 && part.hi <= 1 << shift && part.lo < part.hi);
        for (int slot = part.lo; slot < part.hi; ++slot) {
          const int row = part.row + slot - part.lo;
          CHECK(row >= sp.row0 && row < sp.row0 + sp.n);
          if (row >= sp.row0 && row < sp.row0 + sp.n) ++seen[row - sp.row0];
          CHECK((long long)sp.pos0 + (row - sp.row0) == ((long long)p << shift) + slot);
        }
      }
      for (int i = 0; i < sp.n; ++i) CHECK(seen[i] == (sp.pos0 + i >= 0 ? 1 : 0));
      // the tokens that query rows see
      for (int i0 = 0; i0 < sp.n; i0 += 3) {
        const int i1 = i0 + 2 < sp.n ? i0 + 2 : sp.n - 1;
        const int windows[] = {0, 1, 5, 100, INT_MAX};
        for (int w : windows) {
          const KvRange r = kv_visible(sp, w, i0, i1);
          CHECK(r.lo >= 0 && r.lo <= r.hi && r.hi <= sp.len);   // empty ranges too
          if (sp.len > 4096) continue;
          for (int i = i0; i <= i1; ++i)
            for (int t = 0; t < sp.len; ++t) {
              const long long pos = (long long)sp.pos0 + i;
              if (t <= pos && (w == 0 || t > pos - w)) CHECK(t >= r.lo && t < r.hi);
            }
        }
      }
    }
    CHECK(kv_page(s, pages, 0, -1) == -1 && kv_page(s, pages, 0, width) == -1);
  }
  printf("%d failing checks\n", failures);
  return failures != 0;
}
