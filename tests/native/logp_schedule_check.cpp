// Checks the schedules of the label log-probabilities: for N tokens of which
// any number of rows takes part, the ranges that the label scan picks keep
// the partials inside their slots, the pacing counters inside theirs, and
// every tile in exactly one unit; and that the dH product's cut keeps its
// parts inside their buffer, its ranges non-empty and the pacing counters
// inside theirs, with the scan's search picking the host's plan.  Prints "OK <cases>" or the first failure.
#include <cstdio>
#include <vector>

#include "../../chunked_top_kl_b200/csrc/kd_schedule.h"

using namespace kd;

int main() {
  long cases = 0;
  const long Ns[] = {1, 2, 255, 256, 257, 511, 512, 700, 1000, 3001, 4096, 8192, 32768, 262144};
  const long Vs[] = {1, 255, 256, 257, 4096, 32001, 128256, 201088};
  const int groups[] = {1, 3, 66, 74};
  for (long N : Ns)
    for (long V : Vs)
      for (int G : groups) {
        const int64_t n_tiles = ceil_div64(V, 256), slots = logp_part_slots(N);
        const int64_t most_units = ceil_div64(N, 256) * n_tiles;
        const int g = (int)(most_units < G ? most_units : G);
        const int64_t counters = wave_slots_bound(logp_units_bound(N), 0);
        for (long k = 0; k <= 40; ++k) {
          long rows = k <= 20 ? k * N / 20 : (k - 20) * 13 + 1;
          if (rows < 1 || rows > N) continue;
          int64_t most = kLogpMaxSplits;
          if (slots / rows < most) most = slots / rows;
          if (most < 1) { printf("FAIL no split for %ld of %ld rows\n", rows, N); return 1; }
          const int64_t m_tiles = ceil_div64(rows, 256);
          // the scan's search: smallest cost, then fewest ranges
          unsigned long long best = ~0ull;
          for (int s = 1; s <= most && s <= n_tiles; ++s) {
            const unsigned long long key = ((unsigned long long)split_cost(m_tiles, n_tiles, g, s) << 32) | (unsigned)s;
            if (key < best) best = key;
          }
          const Raster r = split_raster(m_tiles, n_tiles, g, (int)(unsigned)best, 256 * 2880 * 2, 126l << 20);
          const Raster f = forward_raster(m_tiles, n_tiles, g, 256 * 2880 * 2, 126l << 20, (int)most);
          if (r.splits != f.splits || r.group_m != f.group_m || r.num_units != f.num_units) {
            printf("FAIL another schedule than forward_raster's: N %ld rows %ld V %ld\n", N, rows, V);
            return 1;
          }
          if ((int64_t)r.splits * rows > slots || r.splits > n_tiles || r.splits < 1) {
            printf("FAIL %d ranges of %ld rows in %ld slots\n", r.splits, rows, (long)slots);
            return 1;
          }
          if (wave_slots_bound(r.num_units, 0) > counters) {
            printf("FAIL %d units, counters for %ld\n", r.num_units, (long)counters);
            return 1;
          }
          const JointPlan none{};
          for (int u = 0; u < r.num_units; ++u) {
            int expected = 0;
            const int slot = wave_slot(0, u / g, u % g, g, r.num_units, 0, none, &expected);
            if (slot >= wave_slots_bound(r.num_units, 0) || expected < 0 || expected > g) {
              printf("FAIL slot %d of %d units\n", slot, r.num_units);
              return 1;
            }
          }
          if ((int64_t)r.m_tiles * r.n_tiles <= 40000) {
            std::vector<int> seen((size_t)r.m_tiles * r.n_tiles, 0);
            for (int u = 0; u < r.num_units; ++u) {
              int m, s, n0, n1;
              decode_unit(r, u, m, s, n0, n1);
              if (m < 0 || m >= r.m_tiles || s < 0 || s >= r.splits || n0 >= n1) { printf("FAIL unit %d\n", u); return 1; }
              for (int n = n0; n < n1; ++n) seen[(size_t)m * r.n_tiles + n]++;
            }
            for (int v : seen)
              if (v != 1) { printf("FAIL a tile is computed %d times\n", v); return 1; }
          }
          ++cases;
        }
      }
  const long Cs[] = {1, 60, 256, 257, 1000, 4096, 8192, 12000};
  const long ds[] = {8, 256, 264, 1000, 2048, 2880, 8192};
  for (long C : Cs)
    for (long V : Vs)
      for (long d : ds)
        for (int G : groups)
          for (int with_dW = 0; with_dW < 2; ++with_dW)
            for (long k = 1; k <= 12; ++k) {
              const long rows = k <= 10 ? (k * C + 9) / 10 : (k == 11 ? 1 : C / 2 + 1);
              const int64_t bands = ceil_div64(rows, 256), cols = ceil_div64(d, 256), k0 = ceil_div64(V, 64);
              const int64_t U1 = with_dW ? ceil_div64(V, 256) * cols : 0, k1 = with_dW ? ceil_div64(rows, 64) : 0;
              const int64_t room = dh_part_rows(C);
              const DhPlan p = dh_plan(bands, cols, d, k0, U1, k1, G, room);
              unsigned long long best = ~0ull;
              for (int i = 0; i < 2 * kMaxDhSplits; ++i) {
                bool wide;
                int ks;
                dh_candidate(i, wide, ks);
                const int64_t c = dh_cost(bands, cols, d, k0, U1, k1, G, wide, ks, room);
                if (c >= 0) {
                  if (c >= (int64_t(1) << 32)) { printf("FAIL cost %ld\n", (long)c); return 1; }
                  const unsigned long long key = ((unsigned long long)c << 32) | (unsigned)i;
                  if (key < best) best = key;
                }
              }
              const DhPlan q = dh_plan_of((int)(unsigned)best, cols);
              if (p.k_splits != q.k_splits || p.k_cols != q.k_cols || p.wide_cols != q.wide_cols) {
                printf("FAIL the scan's cut differs: C %ld V %ld d %ld rows %ld\n", C, V, d, rows);
                return 1;
              }
              if (p.k_splits < 1 || p.k_splits > k0 || bands * 256 * p.k_splits > room ||
                  p.k_cols != (p.wide_cols ? ceil_div64(cols, 2) : cols) || (p.wide_cols && p.wide_cols != cols)) {
                printf("FAIL cut %d of %ld K blocks, %ld bands in %ld rows\n", p.k_splits, (long)k0, (long)bands, (long)room);
                return 1;
              }
              const int64_t counters = wave_slots_bound(room / 256 * cols, ceil_div64(V, 256) * cols);
              if (wave_slots_bound(bands * p.k_cols * p.k_splits, U1) > counters) { printf("FAIL counters\n"); return 1; }
              int64_t at = 0;                 // the K ranges follow one another, none empty
              for (int part = 0; part < p.k_splits; ++part) {
                const int64_t a = k0 * part / p.k_splits, b = k0 * (part + 1) / p.k_splits;
                if (a != at || b <= a) { printf("FAIL range %d of %d\n", part, p.k_splits); return 1; }
                at = b;
              }
              if (at != k0) { printf("FAIL ranges end at %ld\n", (long)at); return 1; }
              ++cases;
            }
  printf("OK %ld\n", cases);
  return 0;
}
