// Replays how k_attend4 cuts a batch of few groups (csrc/attend_plan.h): 256 threads pack their slots' pieces by all targets
// into one number each, sum these up wave by wave, choose a target, and every workgroup looks its piece up in
// the sums.  Reads calls from standard input, one per line:
//   grid rows group kv_heads width slots (cached chunk) x slots
// and prints, for each, the number of pieces, how many workgroups look up a piece that is not the next one of
// the batch in the order slot, head, piece, how many sums differ from plain ones, and how many pieces are left over.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#define PLAN_FN static inline
#include "attend_plan.h"

using namespace dspark;

constexpr int kThreads = 256, kWave = 64;

int main() {
  int grid, rows, group, heads, slots;
  long long width;
  while (scanf("%d %d %d %d %lld %d", &grid, &rows, &group, &heads, &width, &slots) == 6) {
    if (slots > kThreads || !plan_few((int64_t)slots * heads, grid)) return 1;
    std::vector<SlotWork> work(slots);
    int row = 0, groups = 0;
    int64_t steps = 0;
    std::vector<int> mine(kThreads, 0);
    for (int s = 0; s < slots; ++s) {
      int cached, chunk;
      if (scanf("%d %d", &cached, &chunk) != 2) return 1;
      work[s] = plan_slot(row, row + chunk, cached, width, group, rows, heads);
      row += chunk;
      if (work[s].tiles > 1) return 2;
      if (work[s].tiles > 0) {
        mine[s] = tile_units(work[s], group, rows, 0);
        groups += heads;
        steps += (int64_t)heads * mine[s];
      }
    }
    if (groups == 0) return 3;
    int target[kTargets];
    plan_targets(steps, groups, grid, target);
    // as the waves do it: a sum within each, then the waves' totals
    std::vector<int64_t> x(kThreads), sum(kThreads / kWave, 0);
    int64_t plain[kTargets] = {};
    long long wrong_sums = 0;
    for (int t = 0; t < kThreads; ++t) {
      const int64_t own = plan_packed(mine[t], target, heads);
      for (int k = 0; k < kTargets; ++k) plain[k] += (int64_t)heads * plan_pieces(mine[t], target[k]);
      sum[t / kWave] += own;
      x[t] = sum[t / kWave];
    }
    int64_t total = 0;
    for (int w = 0; w < kThreads / kWave; ++w) {
      for (int t = w * kWave; t < (w + 1) * kWave; ++t) x[t] += total;
      total += sum[w];
    }
    for (int k = 0; k < kTargets; ++k) wrong_sums += plan_unpacked(total, k) != plain[k];
    int units;
    const int best = plan_choice(total, grid, target, units);
    wrong_sums += units != target[best];
    for (int k = 0; k < best; ++k) wrong_sums += plain[k] <= grid;
    std::vector<int64_t> before(kThreads + 1, 0);
    for (int t = 0; t < kThreads; ++t) before[t + 1] = plan_unpacked(x[t], best);
    const int pieces = plan_unpacked(total, best);
    long long wrong = 0;
    int at = 0;
    for (int s = 0; s < slots; ++s)
      for (int h = 0; h < heads && mine[s]; ++h) {
        const int n = plan_pieces(mine[s], units);
        int end = 0;
        for (int j = 0; j < n; ++j, ++at) {
          if (at >= pieces) {
            ++wrong;
            continue;
          }
          const int found = plan_run(before.data(), kThreads, at);
          if (found != s) {
            ++wrong;
            continue;
          }
          const PlanPiece p = plan_piece(mine[s], units, at - (int)before[found]);
          wrong += p.head != h || p.j != j || p.n != n || piece_start(mine[s], j, n) != end;
          end = piece_start(mine[s], j + 1, n);
        }
        wrong += end != mine[s];
      }
    printf("%d %lld %lld %d\n", pieces, wrong, wrong_sums, pieces - at);
  }
  return 0;
}
