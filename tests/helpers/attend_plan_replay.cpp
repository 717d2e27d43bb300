// Replays the work line of chunk attention (csrc/attend_plan.h) on the host, as the
// workgroups of k_attend walk over it and k_attend_join joins it.  Reads calls from
// standard input, one per line:
//   grid rows group kv_heads width slots (cached chunk) x slots
// and prints, for each, how many (slot, head, tile, key step) nobody computes, how many
// are computed more than once, and how many groups' joined records lie outside the spans.
#include <stdint.h>
#include <stdio.h>

#include <map>
#include <tuple>
#include <vector>

#define PLAN_FN static inline
#include "attend_plan.h"

using namespace dspark;

int main() {
  int grid, rows, group, heads, slots;
  long long width;
  while (scanf("%d %d %d %d %lld %d", &grid, &rows, &group, &heads, &width, &slots) == 6) {
    std::vector<SlotWork> work(slots);
    std::vector<int64_t> first(slots + 1, 0);
    int row = 0;
    for (int s = 0; s < slots; ++s) {
      int cached, chunk;
      if (scanf("%d %d", &cached, &chunk) != 2) return 1;
      work[s] = plan_slot(row, row + chunk, cached, width, group, rows, heads);
      row += chunk;
      first[s + 1] = first[s] + work[s].units;
    }
    const int64_t total = first[slots], span = plan_span(total, grid);
    const int64_t spans = (total + span - 1) / span;
    long long missing = 0, twice = 0, outside = spans > grid ? spans - grid : 0;
    std::map<std::tuple<int, int, int>, std::vector<int>> done;
    for (int64_t k = 0; k < spans; ++k) {
      const int64_t x1 = (k + 1) * span < total ? (k + 1) * span : total;
      int s = 0;
      for (int64_t x = k * span; x < x1;) {
        while (x >= first[s + 1]) ++s;
        const PlanPlace at = plan_place(work[s], group, rows, x - first[s]);
        if (at.units == 0) {
          x = first[s] + at.next;
          continue;
        }
        const int64_t start = first[s] + at.start;
        const int64_t from = x - start;
        const int64_t to = at.units < from + (x1 - x) ? at.units : from + (x1 - x);
        if (from == 0 && to < at.units && (start + at.units - 1) / span >= spans) ++outside;
        std::vector<int>& n = done[std::make_tuple(s, at.head, at.tile)];
        n.resize(at.units, 0);
        for (int64_t u = from; u < to; ++u) ++n[u];
        x += to - from;
      }
    }
    for (int s = 0; s < slots; ++s)
      for (int h = 0; h < heads; ++h)
        for (int t = 0; t < work[s].tiles; ++t) {
          std::vector<int>& n = done[std::make_tuple(s, h, t)];
          n.resize(tile_units(work[s], group, rows, t), 0);
          for (int c : n) {
            missing += c == 0;
            twice += c > 1;
          }
        }
    printf("%lld %lld %lld\n", missing, twice, outside);
  }
  return 0;
}
