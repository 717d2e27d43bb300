// attend_plan.h -- the line of work that chunk attention (attend.hip) cuts into spans.
//
// A group is one (slot, kv head, row tile) and has as many units as its rows see key
// steps.  Row tile i of a slot is put together with the slot's i-th last one: what a
// chunk's later tokens see more than its earlier ones evens out, so that every pair
// has `pair_units` units (a bound; a pair may end before it) and a slot's work has a
// closed form.  All units of the batch lie on a line in the order slot, head, pair; a
// workgroup takes a span of it, a group that spans cut is joined afterwards.
//
// Whole-number arithmetic alone, without a compiler's extensions: the tests replay it on
// the host.  The includer defines PLAN_FN, what stands in front of a function.
#pragma once

#include <stdint.h>

namespace dspark {

constexpr int kKeys = 32;  // keys per step of a wave
// Shortest span of a workgroup in steps, and what a pair of row tiles takes on the line at
// least: a group costs several steps' time before its first one (21 slots of one cached
// and up to 7 new tokens: 24 us if a workgroup takes four such groups, 11 us with one each).
constexpr int kMinSpan = 4;

struct SlotWork {
  int o0, chunk;  // first token row and tokens of the chunk
  int len;        // cached tokens before it
  int keys;       // keys that exist: len + chunk, at most the table's width
  int tiles, pairs;
  int pair_units;
  int64_t units;
};

PLAN_FN int plan_min(int a, int b) { return a < b ? a : b; }
PLAN_FN int plan_max(int a, int b) { return a > b ? a : b; }

// Key steps that the rows up to the end of row tile i see.
PLAN_FN int tile_units(const SlotWork& w, int group, int rows, int i) {
  const int last = plan_min((i + 1) * rows, w.chunk * group) - 1;
  return (plan_min(w.len + last / group + 1, w.keys) + kKeys - 1) / kKeys;
}

// A slot's work.  o0, o1: its token rows, 0 <= o0 <= o1; cached: tokens before them;
// width: positions of the table's row; group: query heads per kv head; rows of a tile.
// extra: what a group takes on the line in front of its first step.
PLAN_FN SlotWork plan_slot(int o0, int o1, int cached, int64_t width, int group, int rows,
                           int kv_heads, int extra = 0) {
  SlotWork w;
  w.o0 = o0;
  w.chunk = o1 - o0;
  const int64_t len = plan_max(cached, 0);
  w.len = (int)(len < width ? len : width);
  const int64_t keys = (int64_t)w.len + w.chunk;
  w.keys = (int)(keys < width ? keys : width);
  w.tiles = (w.chunk * group + rows - 1) / rows;
  w.pairs = (w.tiles + 1) >> 1;
  w.pair_units = 0;
  w.units = 0;
  if (w.tiles > 0) {
    const int last = tile_units(w, group, rows, w.tiles - 1);
    if (w.tiles <= 3) {  // the outer pair; of three tiles the middle one is no larger
      w.pair_units = (w.tiles == 1 ? 0 : tile_units(w, group, rows, 0)) + last;
    } else {
      // Tiles i and tiles - 1 - i end at rows (i + 1) rows and (tiles - i) rows at most, so
      // that they see 2 len + floor(((tiles + 1) rows - 2) / group) + 2 keys at most, and
      // twice `keys` at most; rounding each up to steps adds 31 keys.  (The outer pair is no
      // bound: the last tile may be almost empty, and a table shorter than the chunk cuts
      // what the later tiles see.)
      const int64_t both = 2 * (int64_t)w.len + ((int64_t)(w.tiles + 1) * rows - 2) / group + 2;
      const int64_t most = 2 * (int64_t)w.keys;
      w.pair_units = (int)(((both < most ? both : most) + 2 * (kKeys - 1)) / kKeys);
    }
    w.pair_units = plan_max(w.pair_units, kMinSpan) + (w.tiles > 1 ? 2 : 1) * extra;
    w.units = (int64_t)w.pair_units * w.pairs * kv_heads;
  }
  return w;
}

// Where unit `left` of a slot lies.
struct PlanPlace {
  int head, tile;
  int units;     // of the group, 0 behind its pair's end
  int64_t start; // the group's first unit (of its first step, behind `extra`)
  int64_t next;  // the next pair's first unit
};

// narrow: a division in 32 bits where it can be; one in 64 takes a hundred instructions more.  For groups
// of few steps (4 bits); the branch around it makes the longest tiles' loop over whole elements 11 % longer
// (two chunks of 2,048: 505.5 us, 502.5 without).
PLAN_FN PlanPlace plan_place(const SlotWork& w, int group, int rows, int64_t left, int extra = 0,
                             bool narrow = false) {
  PlanPlace g;
  const bool fits = narrow && left <= INT32_MAX;
  const int64_t pair = fits ? (int64_t)((int32_t)left / w.pair_units) : left / w.pair_units;
  const int off = (int)(left - pair * w.pair_units);
  g.head = (int)(pair / w.pairs);
  const int i = (int)(pair - (int64_t)g.head * w.pairs), j = w.tiles - 1 - i;
  const int ui = tile_units(w, group, rows, i);
  g.next = left - off + w.pair_units;
  g.tile = i;
  g.units = ui;
  g.start = left - off + extra;
  if (off >= ui + extra) {
    const int uj = j > i ? tile_units(w, group, rows, j) : 0;
    g.tile = j;
    g.units = off < ui + uj + 2 * extra ? uj : 0;
    g.start = left - off + ui + 2 * extra;
  }
  return g;
}

// Units of a span if `grid` workgroups share `total`.
PLAN_FN int64_t plan_span(int64_t total, int grid) {
  const int64_t span = (total + grid - 1) / grid;
  return span > kMinSpan ? span : kMinSpan;
}

// Where a batch has few groups, of one row tile each, a group is cut by itself, into pieces of about
// `target` units, so that no workgroup pays what a group costs beside its steps twice.  A group of n units
// takes as long as its longest piece, then as long as the join of its pieces: pieces are no shorter than the
// square root of n, the next power of two (a token over 30,000 of 32 heads on 8: 24.7 -> 20.3 us, of 8 heads
// on one: 37 -> 21, 9 tokens over 4,000: 30 -> 20).
// The target is the least of kTargets, from a little above a workgroup's share of an even line on, by which
// the pieces are no more than workgroups; by the last one they always are (a piece that is not full for
// every group).  (By the last alone: 32 slots of 1 to 17 tokens 44.0 us instead of 42.3, a token over
// 130,000 43.5 instead of 40.5.)
// total, groups: of the batch, groups > 0 (2 groups at most grid).
constexpr int kTargets = 4;
// Both sides of the boundary (cut by themselves, on a line with the charge below; 32 query heads on 8 of 128,
// 512 workgroups): 24 slots of 1 to 17 tokens over 2,100 35.5 and 41 us, 32 slots 40 and 45, 40 slots 44.6
// and 46.5, 48 slots 55 and 52; one token over 8,000 of 32 slots 48 and 48, 33 slots 51 and 46, 60 slots 81
// and 72.
PLAN_FN bool plan_few(int64_t groups, int grid) { return 2 * groups <= grid; }
// What a group costs beside its steps, in steps, where spans hold several groups (`extra` above).  256 slots
// of 17 tokens by the charge: 0 321 us, 8 306, 14 299, 20 298, 30 300.  Without and with it, from the
// boundary on: 33 slots of 1 to 17 tokens over 2,100 48 and 43 us, 60 slots 67 and 57; one token over 8,000
// of 33 slots 49 and 46; a token over 30,000 of a single one of 33 or 128 slots 26 and 22; 96 slots of 17
// tokens over 4,096, 24 heads on 8 of 64, 86 and 74; 128 slots of 9 tokens over 2,000, 16 heads on 2 of 256,
// 99.6 and 98.5; 64 slots of 5 tokens over 1,000, fp32, 57 and 55.  Few groups of several row tiles have none:
// two prompts 458 without and 440 with it, 512 tokens over 8,192 118 and 123, two chunks of 200 over 1,000 in
// fp32 52 and 65.
PLAN_FN int plan_charge(int64_t groups, int grid) { return plan_few(groups, grid) ? 0 : 20; }
PLAN_FN int64_t plan_div(int64_t x, int y) {  // x, y >= 0
  return x >> 31 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
PLAN_FN void plan_targets(int64_t total, int groups, int grid, int (&target)[kTargets]) {
  const int64_t even = plan_div(total + grid - 1, grid);
  const int64_t most = plan_div(total + grid - groups - 1, grid - groups);
  const int64_t mean = plan_div(total, groups);
  int64_t least = kMinSpan;
  while (least * least < mean) least *= 2;
  for (int k = 0; k < kTargets; ++k) {
    const int64_t t = even + ((most - even) * (k + 1) >> 2);
    target[k] = (int)(t > least ? t : least);
  }
}
PLAN_FN int plan_pieces(int units, int target) {
  return (int)(((uint32_t)units + (uint32_t)target - 1u) / (uint32_t)target);
}
// Pieces of a slot's groups by each target, in 16 bits each, so that one sum over the slots counts all of
// them: 768 of a batch at most (an even share for each workgroup, and one that is not full for every group).
PLAN_FN int64_t plan_packed(int units, const int (&target)[kTargets], int kv_heads) {
  int64_t x = 0;
  for (int k = 0; k < kTargets; ++k) x |= (int64_t)(plan_pieces(units, target[k]) * kv_heads) << (16 * k);
  return x;
}
PLAN_FN int plan_unpacked(int64_t x, int k) { return (int)(x >> (16 * k) & 0xFFFF); }
// Which target it is, and its units, by the batch's packed sum.
PLAN_FN int plan_choice(int64_t total, int grid, const int (&target)[kTargets], int& units) {
  int best = kTargets - 1;
  units = target[kTargets - 1];
  for (int k = kTargets - 2; k >= 0; --k)
    if (plan_unpacked(total, k) <= grid) {
      best = k;
      units = target[k];
    }
  return best;
}
// The last of `runs` runs of slots that starts at x or before it (before: what lies in front of each run).
PLAN_FN int plan_run(const int64_t* before, int runs, int64_t x) {
  int lo = 0, hi = runs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// Piece `left` of a slot whose groups have n pieces each: the j-th of head's.
struct PlanPiece {
  int head, j, n;
};
PLAN_FN PlanPiece plan_piece(int units, int target, int left) {
  PlanPiece p;
  p.n = plan_pieces(units, target);
  p.head = left / p.n;
  p.j = left - p.head * p.n;
  return p;
}
// First unit of piece j of n.
PLAN_FN int piece_start(int units, int j, int n) { return (int)((int64_t)units * j / n); }

}  // namespace dspark
