// attend_common.h -- what chunk attention over a paged cache shares between the pools' types
// (attend.hip: bf16 and fp32, attend4.hip: 4 bits): the division of the work, the rules of the running
// maximum, and the join of groups that spans cut.
#pragma once

#include "device_common.h"
#include "kernels.h"
#define PLAN_FN __device__ __forceinline__
#include "attend_plan.h"

namespace dspark {

namespace {

constexpr int kPlanThreads = 256;  // the workgroup's first threads work out the plan
constexpr int kPlanWaves = kPlanThreads / 64;
// All loads have arrived.  Placed where a load's result is first used in a loop or
// behind a branch: the compiler would otherwise wait for it inside the loop, and as
// loads return in order, for the newest ones that the loop has just started.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }
constexpr float kRise = 8.f;      // how far scores may pass the running maximum (in log2) ...
constexpr float kRiseSum = 1024.f;  // ... and the sum of a lane's eight weights
constexpr float kNone = -1e30f;  // maximum of a row that has seen no key
// From here on a maximum, a rounded product of score and scale, is off by a whole or more
// (binary logarithm), and an exact product against it could be anything.
constexpr float kFar = 0x1p24f;

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// What differs between the element types.  `Chunk` is a lane's 16 bytes of an operand.
template <typename E>
struct Ops;

template <>
struct Ops<uint16_t> {
  typedef bf16x8 Chunk;
  static constexpr int kE = 8;
  static constexpr int kVChunks = 1;  // V operands per step and 16 dimensions
  // key of row m of 16-key block u of a step: lane group q's accumulators of both
  // blocks are then keys 8q .. 8q + 7, one 16-byte group of V
  static __device__ __forceinline__ int key_of(int u, int m) { return 8 * (m >> 2) + 4 * u + (m & 3); }
  // first key of the group that lane group q loads for V operand u
  static __device__ __forceinline__ int vkey_of(int, int q) { return 8 * q; }
  // position of accumulator j of block u among the step's keys, for lane group q
  static __device__ __forceinline__ int skey_of(int u, int j, int q) { return 8 * q + 4 * u + j; }
  static __device__ __forceinline__ f32x4 score(Chunk k, Chunk q, f32x4 s) { return mma(k, q, s); }
  static __device__ __forceinline__ Chunk zero() {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (__bf16)0.f;
    return c;
  }
  // elements n .. 7 cleared
  static __device__ __forceinline__ Chunk keep(Chunk c, int n) {
    union { Chunk b; uint32_t w[4]; } x;
    x.b = c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t mask = n >= 2 * i + 2 ? 0xFFFFFFFFu : (n == 2 * i + 1 ? 0x0000FFFFu : 0u);
      x.w[i] &= mask;
    }
    return x.b;
  }
};

template <>
struct Ops<float> {
  typedef f32x4 Chunk;
  static constexpr int kE = 4;
  static constexpr int kVChunks = 2;
  static __device__ __forceinline__ int key_of(int u, int m) { return 16 * u + m; }
  static __device__ __forceinline__ int vkey_of(int u, int q) { return 16 * u + 4 * q; }
  static __device__ __forceinline__ int skey_of(int u, int j, int q) { return 16 * u + 4 * q + j; }
  static __device__ __forceinline__ f32x4 score(Chunk k, Chunk q, f32x4 s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s = __builtin_amdgcn_mfma_f32_16x16x4f32(k[j], q[j], s, 0, 0, 0);
    return s;
  }
  static __device__ __forceinline__ Chunk zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
  static __device__ __forceinline__ Chunk keep(Chunk c, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = i < n ? c[i] : 0.f;
    return c;
  }
};

// ---- the batch's work, cut into equal spans (attend_plan.h) --------------------------
// extra: what a group takes on the line in front of its first step.
__device__ __forceinline__ SlotWork slot_work(const AttendArgs& a, int s, int rows, int extra = 0) {
  const int o0 = min(max(a.offsets[s], 0), a.N);
  const int o1 = min(max(a.offsets[s + 1], o0), a.N);
  return plan_slot(o0, o1, a.c.t.lens[s], (int64_t)a.c.max_pages << a.c.page_shift, a.group, rows,
                   a.c.kv_heads, extra);
}

// Units before each plan thread's run of slots (thread t: slots [t per, t per + per)).
struct Plan {
  int64_t before[kPlanThreads + 1];
  int64_t sum[kPlanWaves];
  int64_t span;
  int spans;
  int per;
};

// By all threads of a workgroup, of which there are kPlanThreads at least.
__device__ __forceinline__ void make_plan(const AttendArgs& a, int rows, Plan& plan) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.c.slots + kPlanThreads - 1) / kPlanThreads;
  const int s0 = tid < kPlanThreads ? tid * per : a.c.slots, s1 = min(s0 + per, a.c.slots);
  int64_t x = 0;
  for (int s = s0; s < s1; ++s) x += slot_work(a, s, rows).units;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63 && wave < kPlanWaves) plan.sum[wave] = x;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < wave) x += plan.sum[w];
    total += plan.sum[w];
  }
  if (tid < kPlanThreads) plan.before[tid + 1] = x;
  if (tid == 0) {
    const int64_t span = plan_span(total, a.grid);
    plan.before[0] = 0;
    plan.span = span;
    plan.spans = (int)((total + span - 1) / span);
    plan.per = per;
  }
  __syncthreads();
}

// The group that unit x lies in.
struct Group {
  SlotWork w;
  int slot, head, tile;
  int units;      // of the group
  int64_t start;  // its first unit on the line
  int64_t next;   // units == 0 (x lies behind its pair's end): the next pair's first unit
  int64_t slot_start, slot_end;
};

// `g` may hold the group before it: a slot is looked up when the line leaves it.  work_of(s):
// the slot's work; extra, narrow: as in slot_work and plan_place.
template <typename F>
__device__ __forceinline__ void find_group(const AttendArgs& a, int rows, const Plan& plan,
                                           int64_t x, Group& g, F work_of, int extra = 0,
                                           bool narrow = false) {
  if (x >= g.slot_end) {
    const int lo = plan_run(plan.before, kPlanThreads, x);
    int64_t start = plan.before[lo];
    int s = lo * plan.per;
    const int end = min(s + plan.per, a.c.slots);
    for (;; ++s) {
      g.w = work_of(s);
      if (x < start + g.w.units || s + 1 >= end) break;
      start += g.w.units;
    }
    g.slot = s;
    g.slot_start = start;
    g.slot_end = start + g.w.units;
  }
  const PlanPlace at = plan_place(g.w, a.group, rows, x - g.slot_start, extra, narrow);
  g.head = at.head;
  g.tile = at.tile;
  g.units = at.units;
  g.start = g.slot_start + at.start;
  g.next = g.slot_start + at.next;
}

template <typename E>
__device__ __forceinline__ void store4(E* to, f32x4 v);
template <>
__device__ __forceinline__ void store4<float>(float* to, f32x4 v) {
  *reinterpret_cast<f32x4*>(to) = v;
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t* to, f32x4 v) {
  // rounded to nearest even, once
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  bf16x4 b;
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (__bf16)v[i];
  *reinterpret_cast<bf16x4*>(to) = b;
}

// Rows that a workgroup of k_attend_join takes, four dimensions a thread.
__host__ __device__ constexpr int join_rows(int D) { return kPlanThreads / (D / 4); }

// Joins the groups that spans cut: workgroup (k, b) the b-th join_rows rows of the group
// that starts in span k and goes on behind it.  Its pieces: record `first`, then the first
// records of spans k + 1 to `last`.  The largest maximum first, then the sums: the pieces'
// loads do not wait for each other (5 groups of 38 pieces: 32 us one after the other).
template <typename E>
__global__ __launch_bounds__(kPlanThreads) void k_attend_join(AttendArgs a, int rows_per_tile) {
  const int k = (int)blockIdx.x;
  if (k >= a.cuts[0].first) return;
  const AttendCut cut = a.cuts[1 + k];
  const int D = a.c.head_dim, G = a.group;
  const int per_row = D / 4;
  const int r = join_rows(D) * (int)blockIdx.y + (int)threadIdx.x / per_row;
  const int c = (int)threadIdx.x % per_row;
  if (r >= cut.rows) return;
  const auto record = [&](int p) {
    return (p == k ? (int64_t)cut.first : 2 * (int64_t)p) * rows_per_tile + r;
  };
  float m = kNone;
#pragma unroll 8
  for (int p = k; p <= cut.last; ++p) m = fmaxf(m, a.part_ml[record(p) * 2]);
  float l = 0.f;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = k; p <= cut.last; ++p) {
    const int64_t o = record(p);
    const float f = __builtin_amdgcn_exp2f(a.part_ml[o * 2] - m);
    l += a.part_ml[o * 2 + 1] * f;
    sum += *reinterpret_cast<const f32x4*>(a.part_o + o * D + 4 * c) * f;
  }
  const int row = cut.row0 + r, token = row / G;
  E* to = static_cast<E*>(a.out) +
          ((int64_t)(cut.token0 + token) * a.heads + cut.head * G + (row - token * G)) * D + 4 * c;
  store4<E>(to, sum * (l > 0.f ? 1.f / l : 0.f));
}

}  // namespace

}  // namespace dspark
