// Checks the forward schedule of up to 128 tokens, whose one band is cut into
// up to kSingleMaxSplits column ranges of single-CTA tiles: for any number of
// live rows the partials stay inside their slots, the pacing counters that the
// label scan clears inside theirs, and every tile is in exactly one range.
// Prints "OK <cases>" or the first failure.
#include <cstdio>
#include <initializer_list>
#include <vector>

#include "../../chunked_top_kl_b200/csrc/kd_schedule.h"

using namespace kd;

int main() {
  long cases = 0;
  int most_seen = 0;
  for (long N = 1; N <= 128; ++N)
    for (long V : {1L, 255L, 256L, 257L, 4096L, 32001L, 40961L, 128256L, 201088L, 1000001L})
      for (int G : {1, 74, 132, 148, 160, 200}) {
        const int64_t n_tiles = ceil_div64(V, 256), slots = logp_part_slots(N);
        const int g = (int)(n_tiles < G ? n_tiles : G);
        const int64_t counters = wave_slots_bound(logp_units_bound(N), 0);
        for (long rows = 1; rows <= N; ++rows) {
          int64_t most = kSingleMaxSplits;
          if (slots / rows < most) most = slots / rows;
          unsigned long long best = ~0ull;
          for (int s = 1; s <= most && s <= n_tiles; ++s) {
            const unsigned long long key = ((unsigned long long)split_cost(1, n_tiles, g, s) << 32) | (unsigned)s;
            if (key < best) best = key;
          }
          const Raster r = split_raster(1, n_tiles, g, (int)(unsigned)best, 256 * 2880 * 2, 126l << 20);
          if (r.splits > most_seen) most_seen = r.splits;
          if (r.splits < 1 || r.splits > n_tiles || (int64_t)r.splits * rows > slots || r.num_units != r.splits) {
            printf("FAIL %d ranges of %ld rows in %ld slots\n", r.splits, rows, (long)slots);
            return 1;
          }
          if (wave_slots_bound(r.num_units, 0) > counters) {
            printf("FAIL %d units, counters for %ld\n", r.num_units, (long)counters);
            return 1;
          }
          std::vector<int> seen((size_t)n_tiles, 0);
          for (int u = 0; u < r.num_units; ++u) {
            int m, s, n0, n1;
            decode_unit(r, u, m, s, n0, n1);
            if (m != 0 || s < 0 || s >= r.splits || n0 >= n1 || n0 < 0 || n1 > n_tiles) { printf("FAIL unit %d\n", u); return 1; }
            for (int n = n0; n < n1; ++n) seen[(size_t)n]++;
          }
          for (int v : seen)
            if (v != 1) { printf("FAIL a tile is computed %d times\n", v); return 1; }
          ++cases;
        }
      }
  if (most_seen <= kLogpMaxSplits) { printf("FAIL never more than %d ranges\n", most_seen); return 1; }
  printf("OK %ld\n", cases);
  return 0;
}
