// logprobs.hip -- log probabilities of given tokens, with the entropy of their
// distribution and its most likely tokens, over rows of target logits:
//   lse = m + ln sum_v e^(z_v - m),  logprob = z_x - lse,
//   H   = ln sum_v e^(z_v - m) - (sum_v e^(z_v - m) (z_v - m)) / sum_v e^(z_v - m),
//   top n entries in the order (value descending, index ascending).
// One pass over the row keeps the running sums of both exponentials and the candidates
// for the top n: entries above a bar (a lower bound of the n-th best so far) go to a list
// in LDS, which is cut back to n by bisection over the values' bits when it fills.
//
// Many rows are bound by HBM: 4,352 rows of 151,936 bf16 logits with 20 alternatives take
// 263 us, 5.0 TB/s like a large copy.  Few rows are bound by what a split costs before its
// first and behind its last step (245 rows: 47 us, 1.6 TB/s), and a single row by two
// dependent launches (16 us).
#include "device_common.h"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPer = 16;               // entries per thread and step
constexpr int kStep = kThreads * kPer; // entries per workgroup and step
constexpr int kNoIndex = 0x7FFFFFFF;

__device__ __forceinline__ uint64_t ballot(bool b) { return __builtin_amdgcn_ballot_w64(b); }
// Lanes below this one among those of a mask.
__device__ __forceinline__ int rank_in(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// The larger value; NaN if one is (fmaxf would lose it).  Two of them are one instruction.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}

// Order of the alternatives: larger value first, then the lower index.
__device__ __forceinline__ bool ahead(float v1, int i1, float v2, int i2) {
  return v1 > v2 || (v1 == v2 && i1 < i2);
}

// A value's place among binary32 values as an unsigned number (0: below them all).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// The next value that compares as smaller: below +0 lies -0, which does not.
__device__ __forceinline__ float below(float v) {
  const uint32_t o = order_of(v);
  return value_of(o - (o == 0x80000000u ? 2 : 1));
}

struct Candidate {
  float v;
  int i;
};

// A wave's candidates for the n best of its workgroup's entries: an unordered list in
// LDS of the entries that were above the bar when they came.  The bar is a lower bound
// of the workgroup's n-th best entry so far.  Each wave publishes the n'-th best of its
// own list, n' = ceil(n / waves): at least n entries of the workgroup reach the smallest
// of these.  (n below the number of waves: the n-th best of any wave is a bound, the
// largest is taken.)  A published value only rises, so that an old one is a bound too
// and the waves need not wait for each other.  For logits in no particular order step k
// of a row then has n / k entries above the bar: a step mostly costs a compare, or one
// for each of four groups.  Ranks are found by bisecting the bits of a value, a compare
// per 64 entries and bit: no sorting, no exchange between lanes.  Which entries a list
// holds at some time depends on the waves' timing, its n best do not.
constexpr int kCut = 128;              // entries above which a list is cut to its n best
constexpr int kRoom = kCut + 4 * 64;   // one more group's worth

template <int kBits>                   // of a value that can differ: 16 (bf16) or 32
struct WaveTop {
  Candidate* list;
  volatile float* shared;              // the waves' published values
  int n, rank, count, told;            // told: entries when last published
  float bar;                           // entries not above it are no candidates
  float exact;                         // the list's n-th best value at its last cut

  __device__ void start(Candidate* room, volatile float* published, int places) {
    list = room;
    shared = published;
    n = places;
    rank = n >= kWaves ? (n + kWaves - 1) / kWaves : n;
    count = told = 0;
    bar = exact = -INFINITY;
  }

  // The order of the k-th best of the lanes' values (its upper 16 bits), 0 if fewer
  // than k lanes have a finite one.
  __device__ static uint32_t kth_of_lanes(float v, int k) {
    const uint32_t o = v > -INFINITY ? order_of(v) : 0u;
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
      const uint32_t c = t | (1u << b);
      if (__popcll(ballot(o >= c)) >= k) t = c;
    }
    return t > 0x007FFFFFu ? t : 0u;
  }
  // A wave's first bar, from the lanes' largest entries.
  __device__ void first_bar(float mine) {
    const uint32_t t = kth_of_lanes(mine, n);
    if (t) bar = below(value_of(t));
  }

  // The first bar of all waves, from the lanes' largest entries: `rank` lanes of a wave
  // reach what it publishes.  (Each wave's own n-th largest instead lets a quarter of a
  // step's entries through for n = 64, and the cuts take most of the time.)
  __device__ void first_shared(float mine, int wave) {
    const uint32_t t = kth_of_lanes(mine, rank);
    if ((threadIdx.x & 63) == 0) shared[wave] = t ? value_of(t) : -INFINITY;
    __syncthreads();
    step();
    if (bar == -INFINITY) first_bar(mine);
  }

  // A step begins.  Entries that only equal the n-th best of another wave may have a
  // lower index; those that equal the own n-th best come behind n better ones.
  __device__ void step() {
    const float a = shared[0], b = shared[1], c = shared[2], d = shared[3];
    const float all = rank < n || n == kWaves ? fminf(fminf(a, b), fminf(c, d))
                                              : fmaxf(fmaxf(a, b), fmaxf(c, d));
    if (all > -INFINITY) bar = fmaxf(bar, below(all));
    bar = fmaxf(bar, exact);
  }

  // Appends the lanes' entries above the bar.
  __device__ void add(float v, int i) {
    const uint64_t hit = ballot(v > bar);
    if (!hit) return;
    if (v > bar) list[count + rank_in(hit)] = Candidate{v + 0.f, i};  // + 0: the two zeros are equal
    count += __popcll(hit);
  }

  __device__ void publish(int wave) {
    if (count < rank || count == told) return;
    told = count;
    __builtin_amdgcn_wave_barrier();
    uint32_t t;
    if (count <= 64) {
      uint32_t o[1];
      orders(o);
      t = nth(o, rank);
    } else {
      uint32_t o[kRoom / 64];
      orders(o);
      t = nth(o, rank);
    }
    if ((threadIdx.x & 63) == 0) shared[wave] = value_of(t);
  }

  template <int kR>
  __device__ void orders(uint32_t (&o)[kR]) const {
    const int lane = (int)threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int e = lane + 64 * r;
      o[r] = e < count ? order_of(list[e < count ? e : 0].v) : 0u;
    }
  }

  // The order of the k-th best value of a list of at least k.
  template <int kR>
  __device__ static uint32_t nth(const uint32_t (&o)[kR], int k) {
    uint32_t t = 0;
#pragma unroll 4
    for (int b = 31; b >= 32 - kBits; --b) {
      const uint32_t c = t | (1u << b);
      int m = 0;
#pragma unroll
      for (int r = 0; r < kR; ++r) m += __popcll(ballot(o[r] >= c));
      if (m >= k) t = c;
    }
    // the bits that are the same for all: ones in the order of negative values
    if (kBits < 32 && t < 0x80000000u) t |= (uint32_t)((uint64_t(1) << (32 - kBits)) - 1);
    return t;
  }

  // Keeps the n best of the list: all above the n-th best value, and of those equal to
  // it the lowest indices.
  __device__ void cut() {
    if (count <= n) return;
    if (count <= 64) cut_to<1>();
    else cut_to<kRoom / 64>();
  }
  template <int kR>
  __device__ void cut_to() {
    const int lane = (int)threadIdx.x & 63;
    Candidate e[kR];
    uint32_t o[kR];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool there = lane + 64 * r < count;
      e[r] = list[there ? lane + 64 * r : 0];
      o[r] = there ? order_of(e[r].v) : 0u;
    }
    const uint32_t t = nth(o, n);
    int above = 0, equal = 0;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      above += __popcll(ballot(o[r] > t));
      equal += __popcll(ballot(o[r] == t));
    }
    int last = kNoIndex;  // highest index kept among equal values
    if (above + equal > n) {
      const int want = n - above;
      int low = 0;        // largest number with fewer than `want` equal entries below it
#pragma unroll 1
      for (int b = 25; b >= 0; --b) {
        const int c = low | (1 << b);
        int m = 0;
#pragma unroll
        for (int r = 0; r < kR; ++r) m += __popcll(ballot(o[r] == t && e[r].i < c));
        if (m < want) low = c;
      }
      last = low;
    }
    count = 0;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool keep = o[r] > t || (o[r] == t && e[r].i <= last);
      const uint64_t kept = ballot(keep);
      if (keep) list[count + rank_in(kept)] = e[r];
      count += __popcll(kept);
    }
    __builtin_amdgcn_wave_barrier();
    told = 0;
    exact = value_of(t);
    bar = fmaxf(bar, below(exact));  // until the step's end an equal entry may have a lower index
  }

  // From here on entries may come that lie before the list's: one that equals its n-th
  // best is a candidate.
  __device__ void open() {
    if (exact > -INFINITY) bar = below(exact);
  }

  // The n best, best first (places left over: -inf, kNoIndex), to the wave's lanes.
  __device__ Candidate sorted() {
    cut();
    const int lane = (int)threadIdx.x & 63;
    Candidate c = list[lane < count ? lane : 0];
    if (lane >= count) c = Candidate{-INFINITY, kNoIndex};
    int place = 0;
#pragma unroll 8
    for (int q = 0; q < count; ++q) {
      const Candidate o = list[q];
      place += ahead(o.v, o.i, c.v, c.i) ? 1 : 0;
    }
    __builtin_amdgcn_wave_barrier();
    if (lane < count) list[place] = c;
    __builtin_amdgcn_wave_barrier();
    return lane < count ? list[lane] : Candidate{-INFINITY, kNoIndex};
  }
};

// Sums over entries z of one row: m the largest entry (NaN if one is), and with
// y = z L - k, L = log2 e in binary32, k = ceil(m L): s = sum 2^y, t = sum 2^y y, in
// binary64.  m L is exact in binary64 (24 x 24 bits), and so is k, however far from zero m
// lies.  Sums of two sets are brought to one k by a power of two: exact, and no exponential.
struct RowSums {
  float m;
  double k, s, t;

  __device__ void none() {
    m = -INFINITY;
    k = s = t = 0.0;
  }
  // The sums as those of a set with the largest entry mn >= m (or NaN).
  __device__ void to(float mn) {
    const double kn = ceil((double)mn * (double)kLog2e);
    if (m != -INFINITY && kn != k) {
      const double d = kn - k;
      const int e = (int)fmax(-d, -2000.0);
      t = ldexp(t - d * s, e);
      s = ldexp(s, e);
    }
    m = mn;
    k = kn;
  }
  // k - m L, in [0, 1)
  __device__ double above() const { return k - (double)m * (double)kLog2e; }
};
// Up to here binary32 holds k and every y near 0 without loss, and y is one fma of z.
// Beyond, z is taken from m first (exact for entries that matter): from 2^30 on z L - k
// with a rounded k can be anything, and the lowest binary32 value has no binary32 k at all.
constexpr float kNear = 0x1p20f;

// Maximum and sum over a wave by lane shifts within the vector unit; valid in lane 63.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t shifted(uint32_t old, uint32_t x) {
  return __builtin_amdgcn_update_dpp(old, x, kCtrl, kRows, 0xF, false);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ float step_max(float m) {
  return max_or_nan(m, __uint_as_float(shifted<kCtrl, kRows>(__float_as_uint(m), __float_as_uint(m))));
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double step_sum(double s) {
  const uint64_t b = __double_as_longlong(s);
  const uint64_t o = (uint64_t)shifted<kCtrl, kRows>(0u, (uint32_t)(b >> 32)) << 32 |
                     shifted<kCtrl, kRows>(0u, (uint32_t)b);
  return s + __longlong_as_double(o);
}
__device__ __forceinline__ float wave_max(float m) {  // in every lane
  m = step_max<0x111, 0xF>(m);
  m = step_max<0x112, 0xF>(m);
  m = step_max<0x114, 0xF>(m);
  m = step_max<0x118, 0xF>(m);
  m = step_max<0x142, 0xA>(m);
  m = step_max<0x143, 0xC>(m);
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(m), 63));
}
__device__ __forceinline__ double wave_sum(double s) {  // in lane 63
  s = step_sum<0x111, 0xF>(s);
  s = step_sum<0x112, 0xF>(s);
  s = step_sum<0x114, 0xF>(s);
  s = step_sum<0x118, 0xF>(s);
  s = step_sum<0x142, 0xA>(s);
  return step_sum<0x143, 0xC>(s);
}
// The lanes' sums as one; valid in lane 63.
__device__ __forceinline__ void wave_sums(RowSums& b) {
  const float m = wave_max(b.m);
  if (m != -INFINITY) b.to(m);
  b.s = wave_sum(b.s);
  b.t = wave_sum(b.t);
}

template <typename E>
struct Group;  // 16 bytes of a row
template <>
struct Group<uint16_t> {
  static constexpr int size = 8, count = kPer / size, apart = kThreads * size;
  static constexpr uint32_t masked = 0xFF80FF80u;  // two entries of -inf
  static __device__ __forceinline__ void unpack(u32x4 q, float* x) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Group<float> {
  static constexpr int size = 4, count = kPer / size, apart = kThreads * size;
  static constexpr uint32_t masked = 0xFF800000u;
  static __device__ __forceinline__ void unpack(u32x4 q, float* x) {
    x[0] = __uint_as_float(q.x);
    x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z);
    x[3] = __uint_as_float(q.w);
  }
};

// Group g of a thread's entries in a step lies g * apart behind entry u, so that a
// wave's load instruction covers one contiguous kilobyte.  `u` counts entries from the
// 16-byte boundary at or before the row's start (`skew` entries before it): a row may
// start at any element, and whole groups inside it are still aligned.  Entries outside
// the row are masked.
template <typename E>
__device__ __forceinline__ void load_step(const E* row, int u, int skew, int end,
                                          u32x4 (&q)[Group<E>::count]) {
#pragma unroll
  for (int g = 0; g < Group<E>::count; ++g) {
    const int v = u + Group<E>::apart * g - skew;
    if (v >= 0 && v + Group<E>::size <= end) {
      q[g] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + v));
    } else {
      constexpr uint32_t none = Group<E>::masked;
      union {
        u32x4 q;
        E e[Group<E>::size];
      } part = {u32x4{none, none, none, none}};
#pragma unroll
      for (int i = 0; i < Group<E>::size; ++i)
        if (v + i >= 0 && v + i < end) part.e[i] = row[v + i];
      q[g] = part.q;
    }
  }
}

// The row's results, lane by lane: the sums, and the lane's alternative.  With
// d = k - m L the sums are those of e^(z - m) times 2^-d, so that
//   lse = m + ln s + d ln 2,  H = ln s + d ln 2 - (t / s + d) / L;
// only |z - m| times the rounding of L remains.
__device__ __forceinline__ void finish(const LogprobArgs& a, int r, float given, const RowSums& sums,
                                       const Candidate& best) {
  const int lane = (int)threadIdx.x & 63;
  // no finite entry, or one that is +inf or NaN: no distribution
  const bool none = !(fabsf(sums.m) < INFINITY);
  const double d = sums.above();
  const double ln_s = log(sums.s) + d * 0.69314718055994530942;  // lse - m
  if (lane == 0) {
    a.logprob[r] = none ? NAN : (float)(((double)given - (double)sums.m) - ln_s);
    a.entropy[r] = none ? NAN : (float)(ln_s - (sums.t / sums.s + d) / (double)kLog2e);
  }
  if (lane < a.n_top) {
    const bool there = !none && best.i != kNoIndex;
    a.top_ids[(int64_t)r * a.n_top + lane] = there ? best.i : -1;
    a.top_logprobs[(int64_t)r * a.n_top + lane] =
        none ? NAN : (there ? (float)(((double)best.v - (double)sums.m) - ln_s) : -INFINITY);
  }
}

__device__ __forceinline__ void skip(const LogprobArgs& a, int r) {
  const int lane = (int)threadIdx.x & 63;
  if (lane == 0) {
    a.logprob[r] = NAN;
    a.entropy[r] = NAN;
  }
  if (lane < a.n_top) {
    a.top_ids[(int64_t)r * a.n_top + lane] = -1;
    a.top_logprobs[(int64_t)r * a.n_top + lane] = NAN;
  }
}

// The waves' sums (each in its lane 63) and best entries joined; valid in wave 0.
template <int kBits>
__device__ __forceinline__ Candidate join_waves(WaveTop<kBits>& top, bool with_top, RowSums& b,
                                                Candidate* room, RowSums* parts, int* counts) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  if (with_top) top.cut();
  if (lane == 63) {
    parts[wave] = b;
    counts[wave] = with_top ? top.count : 0;
  }
  __syncthreads();
  Candidate best = {-INFINITY, kNoIndex};
  if (wave != 0) return best;
  float m = parts[0].m;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = max_or_nan(m, parts[w].m);
  b.none();
  if (m != -INFINITY) b.to(m);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    RowSums part = parts[w];
    if (part.m == -INFINITY) continue;
    part.to(m);
    b.s += part.s;
    b.t += part.t;
  }
  if (with_top) {
    top.open();
    for (int w = 1; w < kWaves; ++w) {
      const Candidate c = lane < counts[w] ? room[w * kRoom + lane] : Candidate{-INFINITY, kNoIndex};
      top.add(c.v, c.i);
      if (top.count > kCut) top.cut();
    }
    best = top.sorted();
  }
  return best;
}

// ---- rows cut into splits --------------------------------------------------------------
// About 1,536 workgroups (6 per CU, what the registers hold) share the rows that have a
// token to look up, in whole steps.  Which rows these are is known on the device alone (a
// round emits fewer tokens than it has rows): every wave counts them.  245 of 544 rows of
// 151,936 entries, 20 alternatives: 47 us with 5 or 6 splits, 49 us with 8 (2,048
// workgroups), 70 us with whole rows.
constexpr int kTarget = 1536;
constexpr int kMaxSplitRows = 1024;  // two splits each
constexpr int kUnits = kTarget + kMaxSplitRows / 2;

__host__ __device__ __forceinline__ int steps_per_split(int rows, int steps) {
  int ns = (kTarget + rows / 2) / rows;
  ns = ns < 1 ? 1 : (ns > steps ? steps : ns);
  return (steps + ns - 1) / ns;
}

// Rows to look up, 64 to a word; a.N <= kMaxSplitRows.
struct LiveRows {
  uint64_t word[kMaxSplitRows / 64];
  int count;

  __device__ __forceinline__ void find(const LogprobArgs& a) {
    const int lane = (int)threadIdx.x & 63;
    int id[kMaxSplitRows / 64];
#pragma unroll
    for (int c = 0; c < kMaxSplitRows / 64; ++c)
      if (64 * c < a.N) id[c] = a.ids[min(64 * c + lane, a.N - 1)];
    count = 0;
#pragma unroll
    for (int c = 0; c < kMaxSplitRows / 64; ++c) {
      word[c] = 0;
      if (64 * c < a.N) word[c] = ballot(64 * c + lane < a.N && id[c] >= 0 && id[c] < a.V);
      count += __popcll(word[c]);
    }
  }
  // the n-th one, n < count
  __device__ __forceinline__ int row(int n) const {
    const int lane = (int)threadIdx.x & 63;
    int r = -1;
#pragma unroll
    for (int c = 0; c < kMaxSplitRows / 64; ++c) {
      const int here = __popcll(word[c]);
      if (r < 0 && n < here) {
        const bool hit = (word[c] >> lane & 1) && __popcll(word[c] & ((1ull << lane) - 1)) == n;
        r = 64 * c + __ffsll((unsigned long long)ballot(hit)) - 1;
      }
      n -= here;
    }
    return r;
  }
  // how many lie before row r
  __device__ __forceinline__ int before(int r) const {
    int n = 0;
#pragma unroll
    for (int c = 0; c < kMaxSplitRows / 64; ++c) {
      const int k = r - 64 * c;
      if (k > 0) n += __popcll(k >= 64 ? word[c] : word[c] & ((1ull << k) - 1));
    }
    return n;
  }
};

// One workgroup per row, which it finishes, or (a.steps > 0) per split of a row: it
// leaves the split's sums and best entries to k_logprobs_join.  Held to the registers of
// 7 waves per SIMD (fp32: 6): with 6, 4,352 rows of 151,936 bf16 take 269 us, with 7 263 us.
template <typename E, bool kTop>
__global__ __launch_bounds__(kThreads, sizeof(E) == 2 ? 7 : 6) void k_logprobs(LogprobArgs a) {
  __shared__ Candidate room[kTop ? kWaves * kRoom : 1];
  __shared__ float published[kWaves];
  __shared__ RowSums parts[kWaves];
  __shared__ int counts[kWaves];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  int r = (int)blockIdx.x, split = 0, nsplit = 1, chunk = 0x7FFFFFFF, place = 0;
  if (a.steps > 0) {
    LiveRows rows;
    rows.find(a);
    if (rows.count == 0) return;
    const int per = steps_per_split(rows.count, a.steps);
    nsplit = (a.steps + per - 1) / per;
    chunk = per * kStep;
    split = (int)blockIdx.x / rows.count;
    place = (int)blockIdx.x - split * rows.count;
    if (split >= nsplit) return;
    r = rows.row(place);
  }
  const int id = a.ids[r];
  if (id < 0 || id >= a.V) {
    if (wave == 0) skip(a, r);
    return;
  }
  const E* row = static_cast<const E*>(a.logits) + (int64_t)r * a.ld;
  const int skew = (int)(((uintptr_t)row / sizeof(E)) & (Group<E>::size - 1));
  const int u0 = split * chunk;  // a whole number of steps
  const int u1 = min(a.V + skew - u0, chunk) + u0;
  const int ul = Group<E>::size * (int)threadIdx.x;
  const float given = elem_at(row, id);
  u32x4 q[Group<E>::count];
  load_step(row, u0 + ul, skew, u1 - skew, q);
  WaveTop<8 * (int)sizeof(E)> top;
  if (kTop) {
    top.start(room + wave * kRoom, published, a.n_top);
  }
  // Running sums: each exponent is one fma against a reference k that only rises, by
  // an exact power of two (far from zero: a difference and an fma).  y is held above
  // -200, where 2^y is zero in binary32, so that masked entries add 0 and not 0 * inf.
  RowSums b;
  b.none();
  int steps = 0;
  for (int u = u0; u < u1; u += kStep) {
    float x[kPer];
#pragma unroll
    for (int g = 0; g < Group<E>::count; ++g) Group<E>::unpack(q[g], x + g * Group<E>::size);
    // the next step's entries are on their way while this one is worked on
    if (u + kStep < u1) load_step(row, u + kStep + ul, skew, u1 - skew, q);
    if (kTop && u != u0) top.step();
    float m4[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
      m4[g] = max_or_nan(max_or_nan(max_or_nan(x[4 * g], x[4 * g + 1]), x[4 * g + 2]), x[4 * g + 3]);
    const float mt = max_or_nan(max_or_nan(max_or_nan(m4[0], m4[1]), m4[2]), m4[3]);
    if (!(mt <= b.m)) b.to(max_or_nan(mt, b.m));
    if (b.m != -INFINITY) {
      float s4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
      auto add = [&](int j, float y) {
        y = fmaxf(y, -200.f);
        const float e = __builtin_amdgcn_exp2f(y);
        s4[j & 3] += e;
        t4[j & 3] = fmaf(e, y, t4[j & 3]);
      };
      const bool far = fabsf(b.m) > kNear;
      if (!ballot(far)) {
        const float k = (float)b.k;
#pragma unroll
        for (int j = 0; j < kPer; ++j) add(j, fmaf(x[j], kLog2e, -k));
      } else {
        const float c = far ? b.m : 0.f, k = far ? (float)b.above() : (float)b.k;
#pragma unroll
        for (int j = 0; j < kPer; ++j) add(j, fmaf(x[j] - c, kLog2e, -k));
      }
      b.s += (double)((s4[0] + s4[1]) + (s4[2] + s4[3]));
      b.t += (double)((t4[0] + t4[1]) + (t4[2] + t4[3]));
    }
    if (kTop) {
      if (u == u0) top.first_shared(mt, wave);
      if (ballot(mt > top.bar)) {
        if (top.bar == -INFINITY) top.first_bar(mt);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (ballot(m4[g] > top.bar)) {
#pragma unroll
            for (int j = 4 * g; j < 4 * g + 4; ++j)
              top.add(x[j], u + ul + (j / Group<E>::size) * Group<E>::apart + (j % Group<E>::size) - skew);
            if (top.count > kCut) top.cut();
          }
        }
      }
      // after steps 1, 2, 4, 8, ...: between them the bar falls behind by half at most
      ++steps;
      if ((steps & (steps - 1)) == 0) top.publish(wave);
    }
  }
  wave_sums(b);
  const Candidate best = join_waves(top, kTop, b, room, parts, counts);
  if (wave != 0) return;
  if (a.steps == 0) {
    finish(a, r, given, b, best);
    return;
  }
  const int o = place * nsplit + split;
  if (lane == 0) {
    a.part_m[o] = b.m;
    a.part_st[2 * o] = b.s;
    a.part_st[2 * o + 1] = b.t;
  }
  if (kTop && lane < a.n_top) {  // place by place, so that the splits' best come first
    const int p = (place * a.n_top + lane) * nsplit + split;
    a.part_v[p] = best.v;
    a.part_i[p] = best.i;
  }
}

// One workgroup per row: joins the splits' sums and best entries.
template <typename E, bool kTop>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobArgs a) {
  __shared__ Candidate room[kTop ? kWaves * kRoom : 1];
  __shared__ float published[kWaves];
  __shared__ RowSums parts[kWaves];
  __shared__ int counts[kWaves];
  const int r = (int)blockIdx.x;
  const int id = a.ids[r];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  if (id < 0 || id >= a.V) {
    if (wave == 0) skip(a, r);
    return;
  }
  LiveRows rows;
  rows.find(a);
  const int per = steps_per_split(rows.count, a.steps);
  const int nsplit = (a.steps + per - 1) / per;
  const int o = rows.before(r) * nsplit;
  const float given = elem_at(static_cast<const E*>(a.logits) + (int64_t)r * a.ld, id);
  RowSums b;
  b.none();
  for (int j = (int)threadIdx.x; j < nsplit; j += kThreads) {
    RowSums p = {a.part_m[o + j], 0.0, a.part_st[2 * (o + j)], a.part_st[2 * (o + j) + 1]};
    if (p.m == -INFINITY) continue;
    p.k = ceil((double)p.m * (double)kLog2e);
    const float m = max_or_nan(b.m, p.m);
    p.to(m);
    b.to(m);
    b.s += p.s;
    b.t += p.t;
  }
  wave_sums(b);
  WaveTop<8 * (int)sizeof(E)> top;
  if (kTop) {
    // a wave's share of the entries; they come in no order, so that one that equals the
    // n-th best may still have a lower index: the bar is never made exact
    top.start(room + wave * kRoom, published, a.n_top);
    const int total = nsplit * a.n_top;
    const float* pv = a.part_v + o * a.n_top;
    const int* pi = a.part_i + o * a.n_top;
    constexpr int kRounds = 4;  // on their way together
    for (int c = 0; c < total; c += kRounds * kThreads) {
      float x[kRounds];
      int i[kRounds];
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {
        const int e = c + q * kThreads + (int)threadIdx.x;
        x[q] = e < total ? pv[e] : -INFINITY;
        i[q] = e < total ? pi[e] : kNoIndex;
      }
      if (c == 0) top.first_shared(x[0], wave);
#pragma unroll
      for (int q = 0; q < kRounds; ++q) top.add(x[q], i[q]);
      if (top.count > kCut) top.cut();
    }
  }
  const Candidate best = join_waves(top, kTop, b, room, parts, counts);
  if (wave != 0) return;
  finish(a, r, given, b, best);
}

__global__ __launch_bounds__(256) void k_emitted(int R, int gamma, const int32_t* tokens,
                                                 const int32_t* n_accept, const int32_t* out_token,
                                                 int32_t* ids) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x >= (int64_t)R * (gamma + 1)) return;
  const int r = (int)(x / (gamma + 1)), k = (int)(x % (gamma + 1));
  const int n = min(max(n_accept[r], 0), gamma);
  ids[x] = k < n ? tokens[(int64_t)r * gamma + k] : (k == n ? out_token[r] : -1);
}

template <typename E>
hipError_t launch_typed(const LogprobArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.steps > 0 ? logprob_units(a.N, a.steps) : a.N));
  {
    TimingScope t("logprobs", stream);
    if (a.n_top > 0)
      hipLaunchKernelGGL((k_logprobs<E, true>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((k_logprobs<E, false>), grid, dim3(kThreads), 0, stream, a);
  }
  if (a.steps > 0) {
    TimingScope t("logprobs_join", stream);
    if (a.n_top > 0)
      hipLaunchKernelGGL((k_logprobs_join<E, true>), dim3((unsigned)a.N), dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((k_logprobs_join<E, false>), dim3((unsigned)a.N), dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace

// Steps of a row (4,096 entries) if rows are split, 0 if they stay whole: splits are
// worth it where they shorten a row by more than its join costs.  A step takes 1.5 us,
// the join 5 us, and 8 us for enough rows to fill the CUs.  36 rows of 20,480 (5 steps):
// bf16 14.6 us whole and 16.6 split, f32 16.9 and 15.2; 500 rows of 32,768 (8 steps):
// bf16 22 and 30, f32 26 and 34.
int logprob_steps(int N, int V, int skew) {
  const int steps = (V + skew + kStep - 1) / kStep;
  if (N > kMaxSplitRows) return 0;
  return steps - steps_per_split(N, steps) > (N < 256 ? 4 : 8) ? steps : 0;
}

// Workgroups of a split call: as many as steps_per_split gives for any number of rows up to
// N (rows * ns <= kTarget + rows / 2).
int logprob_units(int N, int steps) {
  return (int64_t)N * steps < kUnits ? N * steps : kUnits;
}

hipError_t launch_logprobs(bool bf16, const LogprobArgs& a, hipStream_t stream) {
  return bf16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
}

hipError_t launch_emitted(int R, int gamma, const int32_t* tokens, const int32_t* n_accept,
                          const int32_t* out_token, int32_t* ids, hipStream_t stream) {
  TimingScope t("emitted_tokens", stream);
  const int64_t n = (int64_t)R * (gamma + 1);
  hipLaunchKernelGGL(k_emitted, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, R, gamma,
                     tokens, n_accept, out_token, ids);
  return hipGetLastError();
}

}  // namespace dspark
