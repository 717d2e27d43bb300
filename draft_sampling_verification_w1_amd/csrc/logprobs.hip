// logprobs.hip -- log probabilities of given tokens, with the entropy of their
// distribution and its most likely tokens, over rows of target logits:
//   lse = m + ln sum_v e^(z_v - m),  logprob = z_x - lse,
//   H   = ln sum_v e^(z_v - m) - (sum_v e^(z_v - m) (z_v - m)) / sum_v e^(z_v - m),
//   top n entries in the order (value descending, index ascending).
// One pass over the row keeps the running sums of both exponentials and a
// sorted candidate list, so that the row is read once.
#include "device_common.h"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPer = 16;                       // entries per thread and step
constexpr int kStep = kThreads * kPer;         // entries per workgroup and step
constexpr int kNoIndex = 0x7FFFFFFF;

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

// A wave's candidates for the n best: an unordered list in LDS of entries that were
// above the bar when they came.  The bar is a lower bound of the n-th best entry so
// far; it rises when the list is cut down to its n best.  For logits in no particular
// order a list of kCut takes the entries of some five steps before its first cut and
// few afterwards, so that most steps cost a compare or seventeen.  The n-th best is
// found by bisecting the bits of its value: a compare per 64 entries and bit, no
// sorting and no exchange between lanes.
constexpr int kCut = 128;            // entries above which a list is cut
constexpr int kRoom = kCut + 64;     // one more instruction's worth
struct Candidate {
  float v;
  int i;
};

template <int kBits>                 // of a value that can differ: 16 (bf16) or 32
struct WaveTop {
  Candidate* list;
  int n, count;
  float bar;       // entries not above it are no candidates
  float exact;     // the n-th best value after a cut, -inf before

  __device__ void start(Candidate* room, int places) {
    list = room;
    n = places;
    count = 0;
    bar = exact = -INFINITY;
  }

  __device__ static float below(float v) { return value_of(order_of(v) - 1); }

  // The first bar: the n-th best of the lanes' largest entries is a lower bound.
  // Its value's upper 16 bits are enough.
  __device__ void first_bar(float mine) {
    const uint32_t o = mine > -INFINITY ? order_of(mine) : 0u;
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
      const uint32_t c = t | (1u << b);
      if (__popcll(__ballot(o >= c)) >= n) t = c;
    }
    // fewer than n lanes with a finite entry: no bound
    if (t > 0x007FFFFFu) bar = below(value_of(t));
  }

  // A step begins: its entries come behind all earlier ones in the vocabulary, so that
  // one that only equals the n-th best is no candidate any more.
  __device__ void step() { bar = fmaxf(bar, exact); }

  __device__ void add(float v, int i) {
    const uint64_t hit = __ballot(v > bar);
    if (!hit) return;
    if (v > bar) {
      const int at = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(hit >> 32),
                                                       __builtin_amdgcn_mbcnt_lo((uint32_t)hit, 0u));
      list[at] = Candidate{v + 0.f, i};  // + 0: the two zeros are equal
    }
    count += __popcll(hit);
    if (count > kCut) cut();
  }

  // Keeps the n best of the list: all above the n-th best value, and of those equal to
  // it the lowest indices.
  __device__ void cut() {
    if (count <= n) return;
    constexpr int kR = kRoom / 64;
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
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 32 - kBits; --b) {
      const uint32_t c = t | (1u << b);
      int m = 0;
#pragma unroll
      for (int r = 0; r < kR; ++r) m += __popcll(__ballot(o[r] >= c));
      if (m >= n) t = c;
    }
    if (kBits < 32 && t < 0x80000000u) t |= (1u << (32 - kBits)) - 1u;  // the low bits of negative values
    int above = 0, equal = 0;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      above += __popcll(__ballot(o[r] > t));
      equal += __popcll(__ballot(o[r] == t));
    }
    int last = kNoIndex;  // highest index kept among equal values
    if (above + equal > n) {
      const int want = n - above;
      int low = 0;        // largest number with fewer than `want` equal entries below it
#pragma unroll
      for (int b = 25; b >= 0; --b) {
        const int c = low | (1 << b);
        int m = 0;
#pragma unroll
        for (int r = 0; r < kR; ++r) m += __popcll(__ballot(o[r] == t && e[r].i < c));
        if (m < want) low = c;
      }
      last = low;
    }
    count = 0;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool keep = o[r] > t || (o[r] == t && e[r].i <= last);
      const uint64_t kept = __ballot(keep);
      if (keep)
        list[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(kept >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)kept, 0u))] = e[r];
      count += __popcll(kept);
    }
    __builtin_amdgcn_wave_barrier();
    exact = value_of(t);
    bar = below(exact);  // until the step's end an equal entry may have a lower index
  }
};

// Sums over entries of one row: m the largest entry, s = sum e^(z - m),
// t = sum e^(z - m) (z - m), in binary64.
struct RowSums {
  float m;
  double s, t;
};

// Joins two sets of entries.
__device__ __forceinline__ void join(RowSums& a, const RowSums& b) {
  if (b.m == -INFINITY) return;
  if (a.m == -INFINITY) {
    a = b;
    return;
  }
  const float m = fmaxf(a.m, b.m);
  const double da = (double)a.m - (double)m, db = (double)b.m - (double)m;
  const double ea = exp(da), eb = exp(db);
  a.t = ea * (a.t + da * a.s) + eb * (b.t + db * b.s);
  a.s = ea * a.s + eb * b.s;
  a.m = m;
}

// A thread's sums, brought to the workgroup's largest entry and added up;
// valid in thread 0.  One binary64 exponential per thread.
__device__ __forceinline__ RowSums block_sums(float m, float kf, double s, double t) {
  __shared__ float sm[kWaves];
  __shared__ double ss[kWaves], st[kWaves];
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  float big = m;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) big = fmaxf(big, __shfl_xor(big, off, 64));
  if (lane == 0) sm[wave] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) big = fmaxf(big, sm[w]);
  if (m != -INFINITY) {
    // s, t hold sum 2^y and sum 2^y y with y = z L - kf; shift y by d = kf - big L
    // to exponents of z - big.  L is the same binary32 constant as in the pass,
    // so that only |z - big| times its rounding remains.
    const double d = (double)kf - (double)big * (double)kLog2e;
    const double f = exp2(d);
    t = f * (t + d * s) * (1.0 / (double)kLog2e);
    s = f * s;
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    s += __shfl_xor(s, off, 64);
    t += __shfl_xor(t, off, 64);
  }
  if (lane == 0) {
    ss[wave] = s;
    st[wave] = t;
  }
  __syncthreads();
  RowSums r = {big, 0.0, 0.0};
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      r.s += ss[w];
      r.t += st[w];
    }
  }
  return r;
}

// The n best of the waves' lists, in order: entry e of the 4 n listed ones goes
// to the place given by how many others are ahead of it.
template <int kBits>
__device__ __forceinline__ void block_top(WaveTop<kBits>& top, int n, float* ov, int* oi) {
  __shared__ float lv[kThreads];
  __shared__ int li[kThreads];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  top.cut();
  __builtin_amdgcn_wave_barrier();
  if (lane < n) {
    const Candidate c = top.list[lane];
    lv[wave * n + lane] = lane < top.count ? c.v : -INFINITY;
    li[wave * n + lane] = lane < top.count ? c.i : kNoIndex;
  }
  __syncthreads();
  const int e = (int)threadIdx.x;
  if (e < kWaves * n) {
    const float v = lv[e];
    const int i = li[e];
    int place = 0;
    for (int q = 0; q < kWaves * n; ++q) {
      // empty places are equal: the lower one is ahead
      place += (ahead(lv[q], li[q], v, i) || (lv[q] == v && li[q] == i && q < e)) ? 1 : 0;
    }
    if (place < n) {
      ov[place] = v;
      oi[place] = i;
    }
  }
}

__device__ __forceinline__ float at_or_masked(const uint16_t* row, int v, int end) {
  return v >= 0 && v < end ? bf16_at(row, v) : -INFINITY;
}
__device__ __forceinline__ float at_or_masked(const float* row, int v, int end) {
  return v >= 0 && v < end ? row[v] : -INFINITY;
}

// Group g of a thread's entries in a step: 16 bytes, so that a wave's load
// instruction covers one contiguous kilobyte.  `u` counts entries from the
// 16-byte boundary at or before the row's start (`skew` entries before it): a
// row may start at any element, and whole groups inside it are still aligned.
__device__ __forceinline__ void load_step(const uint16_t* row, int u, int skew, int end, float* out) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int v = u + 2048 * g - skew;
    if (v >= 0 && v + 8 <= end) {
      const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + v));
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[8 * g + 2 * i] = bf16_lo(w[i]);
        out[8 * g + 2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) out[8 * g + i] = at_or_masked(row, v + i, end);
    }
  }
}
__device__ __forceinline__ void load_step(const float* row, int u, int skew, int end, float* out) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int v = u + 1024 * g - skew;
    if (v >= 0 && v + 4 <= end) {
      const f32x4 q = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(row + v));
      out[4 * g] = q.x;
      out[4 * g + 1] = q.y;
      out[4 * g + 2] = q.z;
      out[4 * g + 3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * g + i] = at_or_masked(row, v + i, end);
    }
  }
}
template <typename E>
struct Group;
template <>
struct Group<uint16_t> {
  static constexpr int size = 8, apart = 2048;
};
template <>
struct Group<float> {
  static constexpr int size = 4, apart = 1024;
};

// The row's results from its sums and best entries (one thread per alternative).
template <typename E>
__device__ __forceinline__ void finish(const LogprobArgs& a, int r, int id, const E* row,
                                       const RowSums& sums, const float* tv, const int* ti) {
  const double ln_s = log(sums.s);
  const double lse = (double)sums.m + ln_s;  // NaN for a row without a finite entry
  const bool none = sums.m == -INFINITY;
  if (threadIdx.x == 0) {
    a.logprob[r] = none ? NAN : (float)((double)elem_at(row, id) - lse);
    a.entropy[r] = none ? NAN : (float)(ln_s - sums.t / sums.s);
  }
  for (int j = (int)threadIdx.x; j < a.n_top; j += kThreads) {
    const bool there = ti[j] != kNoIndex;
    a.top_ids[(int64_t)r * a.n_top + j] = there ? ti[j] : -1;
    a.top_logprobs[(int64_t)r * a.n_top + j] =
        none ? NAN : (there ? (float)((double)tv[j] - lse) : -INFINITY);
  }
}

__device__ __forceinline__ void skip(const LogprobArgs& a, int r) {
  if (threadIdx.x == 0) {
    a.logprob[r] = NAN;
    a.entropy[r] = NAN;
  }
  for (int j = (int)threadIdx.x; j < a.n_top; j += kThreads) {
    a.top_ids[(int64_t)r * a.n_top + j] = -1;
    a.top_logprobs[(int64_t)r * a.n_top + j] = NAN;
  }
}

// One workgroup per (row, vocabulary split).  With one split it finishes the
// row; with more it leaves the split's sums and best entries to k_logprobs_join.
template <typename E, bool kTop>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobArgs a) {
  __shared__ RowSums sums;
  __shared__ float tv[64];
  __shared__ int ti[64];
  __shared__ Candidate room[kTop ? kWaves * kRoom : 1];
  const int r = (int)blockIdx.x;
  const int split = (int)blockIdx.y;
  const int id = a.ids[r];
  if (id < 0 || id >= a.V) {
    if (a.nsplit == 1) skip(a, r);
    return;
  }
  const E* row = static_cast<const E*>(a.logits) + (int64_t)r * a.ld;
  const int skew = (int)(((uintptr_t)row / sizeof(E)) & (Group<E>::size - 1));
  const int u0 = split * a.chunk;  // a whole number of steps
  const int u1 = min(a.V + skew, u0 + a.chunk);
  WaveTop<8 * (int)sizeof(E)> top;
  if (kTop) top.start(room + ((int)threadIdx.x >> 6) * kRoom, a.n_top);
  // Running sums s = sum 2^y, t = sum 2^y y with y = z L - K, against an integer
  // reference K >= max z L that only rises: each exponent is one fma and a rise
  // rescales by an exact power of two.  y is held above -200, where 2^y is zero
  // in binary32, so that masked entries add 0 and not 0 * inf.
  float m = -INFINITY, kf = 0.f;
  double s = 0.0, t = 0.0;
  for (int u = u0; u < u1; u += kStep) {
    float x[kPer];
    const int ul = u + Group<E>::size * (int)threadIdx.x;
    load_step(row, ul, skew, u1 - skew, x);
    float mt = x[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) mt = fmaxf(mt, x[j]);
    if (mt > m) {
      const float kn = ceilf(mt * kLog2e);
      if (m != -INFINITY && kn > kf) {
        const double d = (double)kn - (double)kf;
        const int e = (int)fmax(-d, -2000.0);
        t = ldexp(t - d * s, e);
        s = ldexp(s, e);
      }
      if (m == -INFINITY || kn > kf) kf = kn;
      m = mt;
    }
    if (m != -INFINITY) {
      float e[kPer], y[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        y[j] = fmaxf(fmaf(x[j], kLog2e, -kf), -200.f);
        e[j] = __builtin_amdgcn_exp2f(y[j]);
      }
      float s4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        s4[j & 3] += e[j];
        t4[j & 3] = fmaf(e[j], y[j], t4[j & 3]);
      }
      s += (double)((s4[0] + s4[1]) + (s4[2] + s4[3]));
      t += (double)((t4[0] + t4[1]) + (t4[2] + t4[3]));
    }
    if (kTop) {
      top.step();
      if (__ballot(mt > top.bar)) {
        if (top.bar == -INFINITY) top.first_bar(mt);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          top.add(x[j], ul + (j / Group<E>::size) * Group<E>::apart + (j % Group<E>::size) - skew);
      }
    }
  }
  const RowSums b = block_sums(m, kf, s, t);
  if (threadIdx.x == 0) sums = b;
  if (kTop) block_top(top, a.n_top, tv, ti);
  __syncthreads();
  if (a.nsplit == 1) {
    finish(a, r, id, row, sums, tv, ti);
    return;
  }
  const int64_t o = (int64_t)r * a.nsplit + split;
  if (threadIdx.x == 0) {
    a.part_m[o] = sums.m;
    a.part_st[2 * o] = sums.s;
    a.part_st[2 * o + 1] = sums.t;
  }
  if (kTop && (int)threadIdx.x < a.n_top) {
    a.part_v[o * a.n_top + threadIdx.x] = tv[threadIdx.x];
    a.part_i[o * a.n_top + threadIdx.x] = ti[threadIdx.x];
  }
}

// One workgroup per row: joins the splits' sums and best entries.
template <typename E, bool kTop>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobArgs a) {
  __shared__ RowSums part[kWaves];
  __shared__ RowSums sums;
  __shared__ float tv[64];
  __shared__ int ti[64];
  __shared__ Candidate room[kTop ? kWaves * kRoom : 1];
  const int r = (int)blockIdx.x;
  const int id = a.ids[r];
  if (id < 0 || id >= a.V) {
    skip(a, r);
    return;
  }
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int64_t o = (int64_t)r * a.nsplit;
  RowSums b = {-INFINITY, 0.0, 0.0};
  for (int j = (int)threadIdx.x; j < a.nsplit; j += kThreads)
    join(b, RowSums{a.part_m[o + j], a.part_st[2 * (o + j)], a.part_st[2 * (o + j) + 1]});
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    // the pair's lower lane goes first on both sides, so that they agree
    RowSums lo = b, hi;
    hi.m = __shfl_xor(b.m, off, 64);
    hi.s = __shfl_xor(b.s, off, 64);
    hi.t = __shfl_xor(b.t, off, 64);
    if (lane & off) {
      lo = hi;
      hi = b;
    }
    join(lo, hi);
    b = lo;
  }
  if (lane == 0) part[wave] = b;
  if (kTop) {
    // the splits' entries, a wave's share of the splits at a time; an entry that equals
    // the n-th best may still come with a lower index, so that no step is ever begun
    WaveTop<8 * (int)sizeof(E)> top;
    top.start(room + wave * kRoom, a.n_top);
    const int total = a.nsplit * a.n_top;
    const float* pv = a.part_v + o * a.n_top;
    const int* pi = a.part_i + o * a.n_top;
    for (int c = 64 * wave; c < total; c += kThreads) {
      const int e = c + lane;
      const float x = e < total ? pv[e] : -INFINITY;
      top.add(x, e < total ? pi[e] : kNoIndex);
    }
    block_top(top, a.n_top, tv, ti);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) join(b, part[w]);
    sums = b;
  }
  __syncthreads();
  const E* row = static_cast<const E*>(a.logits) + (int64_t)r * a.ld;
  finish(a, r, id, row, sums, tv, ti);
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
  const dim3 grid((unsigned)a.N, (unsigned)a.nsplit);
  {
    TimingScope t("logprobs", stream);
    if (a.n_top > 0)
      hipLaunchKernelGGL((k_logprobs<E, true>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((k_logprobs<E, false>), grid, dim3(kThreads), 0, stream, a);
  }
  if (a.nsplit > 1) {
    TimingScope t("logprobs_join", stream);
    if (a.n_top > 0)
      hipLaunchKernelGGL((k_logprobs_join<E, true>), dim3((unsigned)a.N), dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((k_logprobs_join<E, false>), dim3((unsigned)a.N), dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace

// Vocabulary splits per row: about 2,048 workgroups in all (8 per CU), whole
// steps of 4,096 entries.
int logprob_splits(int N, int V, int* chunk) {
  const int steps = (V + 7 + kStep - 1) / kStep;  // 7: the largest skew
  int ns = 2048 / N;
  ns = ns < 1 ? 1 : (ns > steps ? steps : ns);
  const int per = (steps + ns - 1) / ns;
  *chunk = per * kStep;
  return (steps + per - 1) / per;
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
