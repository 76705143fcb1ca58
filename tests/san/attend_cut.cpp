// The rule that cuts the attention over a cache, from the library's own header:
// for sizes over the whole range that a call may have, a row's chunks cover its
// length, the grids are within the launch limits and the partial results within
// the workspace.  Built and run by tests/test_cache_workspace_cpu.py.
#include <cstdio>
#include <vector>

#include "bfly_attend_cut.h"

int main() {
  const int64_t top = 1 << 24;
  std::vector<int> lengths;
  for (int b = 0; b <= 30; ++b)
    for (int64_t v : {(int64_t(1) << b) - 1, int64_t(1) << b, (int64_t(1) << b) + 1, int64_t(3) << b >> 1,
                      (int64_t(5) << b >> 2) + 33})
      if (v >= 1 && v <= (1 << 30)) lengths.push_back((int)v);
  const std::vector<int64_t> rows = {1, 2, 3, 7, 16, 33, 64, 100, 255, 256, 257, 512, 1000, 5000, 8191,
                                     70000, (1 << 20) + 1, top - 1};
  const std::vector<int> kvs = {1, 2, 3, 4, 8, 16, 32, 40, 128, 1000, 4096};
  const std::vector<int> shares = {1, 2, 4, 5, 7, 8, 12, 16, 17, 20, 32, 33, 64, 1000, 65535};
  int64_t calls = 0;
  for (int64_t n : rows)
    for (int kv : kvs)
      for (int share : shares) {
        const int64_t heads = (int64_t)kv * share, blocks = bfly::attend_blocks(share);
        if (heads > 65536 || n * heads >= top) continue;
        const int64_t items = n * kv * blocks;
        for (int d : {64, 128, 256})
          for (int most : lengths) {
            const size_t bytes = bfly::attend_workspace_bytes(n, (int)heads, kv, d, most);
            for (int window : {0, 1, 31, 482, 700, 2047, 30000, 1 << 20, 1 << 29, 0x7FFFFFFF}) {
              const int reach = bfly::attend_reach(most, window);
              const bfly::Cut c = bfly::cut_of(n, items, share, d, reach);
              const int64_t all = (int64_t)c.chunk * c.splits;
              const bool packed = c.splits > 1 && n > 1 && n <= 256 && n * c.splits < 65536;
              const bool ok = c.chunk > 0 && c.splits > 0 && all >= reach && all - c.chunk < reach &&
                              reach <= most && (c.splits == 1 || c.chunk % 128 == 0) &&
                              (packed || c.splits < 65536) && items * 512 < (int64_t(1) << 33) &&
                              n * heads * (c.splits > 16 ? 1024 : 256) < (int64_t(1) << 32) &&
                              (c.splits == 1 || (double)n * heads * c.splits * (d + 4) * 4 <= (double)bytes);
              if (!ok) {
                printf("rows %lld heads %lld kv_heads %d head_dim %d max_len %d window %d: chunk %d splits %d\n",
                       (long long)n, (long long)heads, kv, d, most, window, c.chunk, c.splits);
                return 1;
              }
              ++calls;
            }
          }
      }
  printf("all %lld cuts hold\n", (long long)calls);
  return 0;
}
