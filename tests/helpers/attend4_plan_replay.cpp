// Replays the work line of 4-bit chunk attention (csrc/attend_plan.h) on the host, as the
// workgroups of k_attend4 walk over it and its join puts it together.  Reads calls from
// standard input, one per line:
//   grid rows group kv_heads width extra slots (cached chunk) x slots
// and prints, for each, how many (slot, head, tile, key step) nobody computes, how many are computed
// more than once, how many records the join reads that nobody writes or are written twice, and
// whether the groups were cut by themselves.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <map>
#include <tuple>
#include <vector>

#define PLAN_FN static inline
#include "attend_plan.h"

using namespace dspark;

int main() {
  int grid, rows, group, heads, extra, slots;
  long long width;
  while (scanf("%d %d %d %d %lld %d %d", &grid, &rows, &group, &heads, &width, &extra, &slots) == 7) {
    std::vector<SlotWork> work(slots);
    int row = 0;
    int64_t groups = 0, steps = 0;
    bool whole = plan_few((int64_t)slots * heads, grid);
    for (int s = 0; s < slots; ++s) {
      int cached, chunk;
      if (scanf("%d %d", &cached, &chunk) != 2) return 1;
      work[s] = plan_slot(row, row + chunk, cached, width, group, rows, heads, extra);
      row += chunk;
      if (work[s].tiles > 0) {
        groups += heads;
        steps += (int64_t)heads * tile_units(work[s], group, rows, 0);
        whole &= work[s].tiles == 1;
      }
    }
    int target = 0, targets[kTargets];
    if (whole && groups) plan_targets(steps, (int)groups, grid, targets);
    for (int k = kTargets - 1; whole && groups && k >= 0; --k) {
      int64_t pieces = 0;
      for (const SlotWork& w : work)
        if (w.tiles) pieces += (int64_t)heads * plan_pieces(tile_units(w, group, rows, 0), targets[k]);
      if (pieces > 768) return 2;  // the kernel's sums take 16 bits
      if (k == kTargets - 1 || pieces <= grid) target = targets[k];
    }
    std::vector<int64_t> first(slots + 1, 0);
    for (int s = 0; s < slots; ++s) {
      const SlotWork& w = work[s];
      first[s + 1] = first[s] + (!target ? w.units : (w.tiles ? (int64_t)heads * plan_pieces(tile_units(w, group, rows, 0), target) : 0));
    }
    const int64_t total = first[slots], span = target ? 1 : plan_span(total, grid);
    const int64_t spans = (total + span - 1) / span;
    long long missing = 0, twice = 0, bad = spans > grid ? spans - grid : 0;
    typedef std::tuple<int, int, int> Key;
    std::map<Key, std::vector<int>> done;
    std::map<int64_t, Key> written;                            // record -> group
    std::map<Key, std::tuple<int64_t, int64_t, int64_t>> cuts;  // group -> span, first record, last span
    auto visit = [&](int64_t k, int s, int head, int tile, int units, int64_t from, int64_t to, int64_t rec, int64_t last) {
      const Key key(s, head, tile);
      std::vector<int>& n = done[key];
      n.resize(units, 0);
      for (int64_t u = from; u < to; ++u) ++n[u];
      if (from == 0 && to == units) return;
      bad += written.count(rec);
      written[rec] = key;
      if (from == 0) cuts[key] = std::make_tuple(k, rec, last);
    };
    for (int64_t k = 0; k < spans; ++k) {
      const int64_t x0 = k * span, x1 = std::min((k + 1) * span, total);
      int s = 0;
      for (int64_t x = x0; x < x1;) {
        while (x >= first[s + 1]) ++s;
        if (target) {
          const int units = tile_units(work[s], group, rows, 0), n = plan_pieces(units, target);
          const int left = (int)(x - first[s]), head = left / n, j = left % n;
          visit(k, s, head, 0, units, piece_start(units, j, n), piece_start(units, j + 1, n), 2 * k, k + n - 1);
          bad += piece_start(units, j + 1, n) <= piece_start(units, j, n);  // an empty piece
          ++x;
          continue;
        }
        const PlanPlace at = plan_place(work[s], group, rows, x - first[s], extra);
        if (at.units == 0) {
          x = first[s] + at.next;
          continue;
        }
        const int64_t start = first[s] + at.start;
        const int64_t from = std::max(x - start, (int64_t)0), to = std::min((int64_t)at.units, x1 - start);
        if (to <= from) break;
        visit(k, s, at.head, at.tile, at.units, from, to, 2 * k + (x != x0), (start + at.units - 1) / span);
        x = start + to;
      }
    }
    // the join: record `first`, then the first records of the spans behind, up to `last`
    size_t read = 0;
    for (auto& c : cuts) {
      const int64_t k = std::get<0>(c.second), last = std::get<2>(c.second);
      for (int64_t p = k; p <= last; ++p, ++read) {
        auto it = written.find(p == k ? std::get<1>(c.second) : 2 * p);
        bad += p >= spans || it == written.end() || it->second != c.first;
      }
    }
    bad += read != written.size();
    for (int s = 0; s < slots; ++s)
      for (int h = 0; h < heads; ++h)
        for (int t = 0; t < work[s].tiles; ++t) {
          std::vector<int>& n = done[Key(s, h, t)];
          n.resize(tile_units(work[s], group, rows, t), 0);
          for (int c : n) {
            missing += c == 0;
            twice += c > 1;
          }
        }
    printf("%lld %lld %lld %d\n", missing, twice, bad, target > 0);
  }
  return 0;
}
