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
PLAN_FN SlotWork plan_slot(int o0, int o1, int cached, int64_t width, int group, int rows,
                           int kv_heads) {
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
    w.pair_units = plan_max(w.pair_units, kMinSpan);
    w.units = (int64_t)w.pair_units * w.pairs * kv_heads;
  }
  return w;
}

// Where unit `left` of a slot lies.
struct PlanPlace {
  int head, tile;
  int units;     // of the group, 0 behind its pair's end
  int64_t start; // the group's first unit
  int64_t next;  // the next pair's first unit
};

PLAN_FN PlanPlace plan_place(const SlotWork& w, int group, int rows, int64_t left) {
  PlanPlace g;
  const int64_t pair = left / w.pair_units;
  const int off = (int)(left - pair * w.pair_units);
  g.head = (int)(pair / w.pairs);
  const int i = (int)(pair - (int64_t)g.head * w.pairs), j = w.tiles - 1 - i;
  const int ui = tile_units(w, group, rows, i);
  g.next = left - off + w.pair_units;
  g.tile = i;
  g.units = ui;
  g.start = left - off;
  if (off >= ui) {
    const int uj = j > i ? tile_units(w, group, rows, j) : 0;
    g.tile = j;
    g.units = off < ui + uj ? uj : 0;
    g.start = left - off + ui;
  }
  return g;
}

// Units of a span if `grid` workgroups share `total`.
PLAN_FN int64_t plan_span(int64_t total, int grid) {
  const int64_t span = (total + grid - 1) / grid;
  return span > kMinSpan ? span : kMinSpan;
}

}  // namespace dspark
