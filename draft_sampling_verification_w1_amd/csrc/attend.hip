// attend.hip -- attention of a chunk of new tokens per slot over a paged cache.
//
// Token i of slot s's chunk sees the keys at positions p <= lens[s] + i:
//   o = sum_p softmax_p(scale q . k_p) v_p,
// computed in one pass over the keys with a running maximum m and sum l:
//   p = 2^(c q.k - m), l += p, O += p v; a rise of m by d scales l and O by 2^-d.
//
// Layout.  A page stores K as [kv_head][D / E][token][E] and V as
// [kv_head][token / E][D][E] (E elements = 16 bytes), which are the matrix cores'
// operand orders: the pass computes S^T = K Q^T and O^T = V^T P^T, so that
//   - a wave's load of a K or V operand is 64 lanes x 16 bytes, 256 contiguous bytes
//     per lane group, and needs no transposition, and
//   - S^T's accumulator already is P^T's operand: a lane holds the scores of one
//     query (column l % 16); which keys it holds is settled by the order in which
//     the key rows of K are loaded (key_of), chosen to match V's 16-byte groups.
//
// Tiles.  A row of a tile is one (token, query head of the kv head's group) pair, so
// that the group shares every key it reads.  A workgroup is RW x KW waves: RW row groups
// of 16 NQ rows, KW parts of the key range whose sums are joined through LDS.  Few rows
// (a decoded token, a short chunk) are bound by HBM: one row group, the keys go from
// memory straight to registers, no LDS and no barrier in the loop.  Many rows are bound
// by the matrix products: the row groups share a step's operands through LDS, where they
// lie in operand order (no bank conflicts), loaded one or two steps ahead.
//
// Work.  Slots and lengths are known on the device only.  The key steps of all
// (slot, kv head, row tile) groups lie on one line, which is cut into equal spans, one
// per workgroup, so that any mix of lengths keeps all CUs busy to the end; each
// workgroup works out the line from lens and offsets (one round trip).  Groups that a
// cut goes through are joined by k_attend_join.
//
// Measured (bf16, 32 heads on 8, 128 dimensions), append + attention + join:
//   32 slots, up to 2,100 cached, 1 to 17 new tokens: 66 us, 2.7 TB/s (attention alone
//     43 us, 4.2 TB/s; the rest are the two other launches);
//   256 slots, up to 4,096 cached, 17 new tokens: 609 us, 4.6 TB/s (a large copy: 5.1);
//   2 prompts, 2,048 tokens behind up to 8,192: 500 us, 907 TFLOP/s (a large library
//     matrix product: 1,240).  The matrix units are busy 39% of the time: a step's
//     exponentials and its products do not overlap within a wave, and two waves per SIMD
//     fill half of the gaps.  Tried without gain: values one step late with 4 waves, one
//     wave per SIMD on 64 rows each, 192- and 256-row tiles (561, 577 us for 494),
//     operands two steps ahead, half of the waves half a step behind the others (545).
#include "attend_common.h"

namespace dspark {

namespace {

// Whether a step's operands go through LDS: several row groups share them.
template <typename E, int D, int RW>
__host__ __device__ constexpr bool staged() {
  return sizeof(E) == 2 && RW > 1;
}
template <typename E, int D>
__host__ __device__ constexpr int step_bytes() {
  return kKeys * D * 2 * (int)sizeof(E);
}
// LDS of a workgroup: two steps' operands of every key part, then (at the same
// place) the outputs of all parts but the first.
template <typename E, int D, int NQ, int RW, int KW>
__host__ __device__ constexpr int lds_bytes() {
  const int stages = staged<E, D, RW>() ? 2 * KW * step_bytes<E, D>() : 0;
  const int join = KW > 1 ? (KW - 1) * 16 * NQ * RW * D * 4 : 16;
  return stages > join ? stages : join;
}

// Key steps [first, end) of a group; `rec`: the record that takes the sums of a group
// that is cut, or -1.  D dimensions; RW x KW waves: RW row groups of NQ 16-row blocks each, KW
// parts of the key range.
// kHalf: pages of 16 tokens under bf16, where one operand spans two pages.
template <typename E, int D, int NQ, int RW, int KW, int kAhead, bool kHalf>
__device__ __forceinline__ void attend_steps(const AttendArgs& a, const Group& it, int first,
                                             int end, int64_t rec, float* sh_ml, int* sh_limit,
                                             uint8_t* sh) {
  typedef Ops<E> Op;
  typedef typename Op::Chunk Chunk;
  constexpr int kE = Op::kE;
  constexpr int kSteps = D / (4 * kE);  // K operands per 16 keys
  constexpr int kDT = D / 16;           // 16-dimension blocks of the output
  constexpr int kVC = Op::kVChunks;
  constexpr int kWaveRows = 16 * NQ;
  constexpr int kRows = kWaveRows * RW;
  constexpr int kThreads = 64 * RW * KW;
  constexpr bool kStaged = staged<E, D, RW>();
  constexpr int kLoads = 2 * kSteps + kVC * kDT;  // operands of a step, 1 KB each
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave / RW;                 // the wave's part of the keys
  const int wrow = (wave % RW) * kWaveRows;   // its first row in the tile
  const int n = lane & 15, quad = lane >> 4;
  const int G = a.group, H = a.c.kv_heads;
  const int row0 = it.tile * kRows, rows = it.w.chunk * G;
  const E* q = static_cast<const E*>(a.q);

  // keys any row of the tile sees, and keys all of them see
  const int last_row = min(row0 + kRows, rows) - 1;
  const int seen = min(it.w.len + last_row / G + 1, it.w.keys);
  const int common = min(it.w.len + row0 / G + 1, it.w.keys);
  // the wave's part of the steps
  const int count = end - first;
  const int t0 = first + count * part / KW, t1 = first + count * (part + 1) / KW;

  f32x4 o[NQ][kDT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    m[i] = kNone;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d) o[i][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // Page ids of 64 consecutive table columns, one per lane; a step reads its two
  // halves' ids from them.  Ids outside the pool count as no page.
  const int shift = a.c.page_shift;
  const int32_t* table = a.c.t.table + (int64_t)it.slot * a.c.max_pages;
  int col0 = (t0 * kKeys) >> shift;
  auto columns = [&](int c0) {
    const int c = c0 + lane;
    const int p = c < a.c.max_pages ? table[c] : -1;
    return p >= 0 && p < a.c.pages ? p : -1;
  };
  int ids = columns(col0);
  // keys that each row sees; read from LDS where they matter, to keep them out of the
  // registers of the pass
  for (int r = threadIdx.x; r < kRows; r += kThreads)
    sh_limit[r] = min(it.w.len + min((row0 + r) / G, it.w.chunk) + 1, it.w.keys);
  // queries as operands: lane (n, quad), operand s: dimensions kE (4 s + quad) ..
  Chunk qo[NQ][kSteps];
  auto load_q = [&]() {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int row = row0 + wrow + 16 * i + n;
      const bool live = row < rows;
      const int token = live ? row / G : 0;
      const E* p = q + ((int64_t)(it.w.o0 + token) * a.heads + it.head * G + (live ? row - token * G : 0)) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        qo[i][s] = live ? *reinterpret_cast<const Chunk*>(p + kE * (4 * s + quad)) : Op::zero();
    }
  };
  const int page = 1 << shift;
  const int64_t page_elems = (int64_t)H * page * D;
  const E* Kh = static_cast<const E*>(a.K) + (int64_t)it.head * page * D;
  const E* Vh = static_cast<const E*>(a.V) + (int64_t)it.head * page * D;
  // ids of the pages of keys [32 t, 32 t + 16) and [32 t + 16, 32 t + 32)
  auto pages_of = [&](int t, int& pa, int& pb) {
    const int ca = (t * kKeys) >> shift, cb = (t * kKeys + 16) >> shift;
    if (cb >= col0 + 64) {
      col0 = ca;
      ids = columns(col0);
      wait_loads();
    }
    pa = __builtin_amdgcn_readlane(ids, ca - col0);
    pb = __builtin_amdgcn_readlane(ids, cb - col0);
  };
  // Operand addresses: a wave-uniform base (page, step, layer) and a lane's 32-bit
  // offset that stays the same through the pass.
  const uint32_t k_lane = (uint32_t)(((Op::key_of(0, n) & (page - 1)) + quad * page) * 16);
  const uint32_t v_lane = (uint32_t)(((Op::vkey_of(0, quad) & (page - 1)) / kE * D + n) * 16);
  const int64_t page_size_bytes = page_elems * (int64_t)sizeof(E);
  const char* Kb = reinterpret_cast<const char*>(Kh);
  const char* Vb = reinterpret_cast<const char*>(Vh);
  auto load_k = [&](int t, int pa, int pb, Chunk (&k)[2][kSteps]) {
    const char* ba = Kb + max(pa, 0) * page_size_bytes;
    const char* bb = Kb + max(pb, 0) * page_size_bytes;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // bf16: the 32 keys of a step lie on one page (kHalf: 16 on each of two);
      // f32: block u's 16 keys do
      const int first = sizeof(E) == 2 ? t * kKeys : t * kKeys + 16 * u;
      const int at = kHalf ? 4 * u : (first & (page - 1)) + (sizeof(E) == 2 ? 4 * u : 0);
      const char* base = sizeof(E) == 2 || u == 0 ? ba : bb;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int64_t to = (int64_t)(4 * s * page + at) * 16;
        if constexpr (kHalf) k[u][s] = *reinterpret_cast<const Chunk*>((n < 8 ? ba : bb) + to + k_lane);
        else k[u][s] = *reinterpret_cast<const Chunk*>(base + to + k_lane);
      }
    }
  };
  auto load_v = [&](int t, int pa, int pb, Chunk (&v)[kVC][kDT]) {
    const char* ba = Vb + max(pa, 0) * page_size_bytes;
    const char* bb = Vb + max(pb, 0) * page_size_bytes;
#pragma unroll
    for (int u = 0; u < kVC; ++u) {
      const int first = t * kKeys + 16 * u;
      const int64_t at = kHalf ? 0 : (int64_t)((first & (page - 1)) / kE) * D * 16;
      const char* base = u == 0 ? ba : bb;
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        const int64_t to = at + 16 * 16 * d;
        if constexpr (kHalf) v[u][d] = *reinterpret_cast<const Chunk*>((quad < 2 ? ba : bb) + to + v_lane);
        else v[u][d] = *reinterpret_cast<const Chunk*>(base + to + v_lane);
      }
    }
  };

  f32x4 s[NQ][2];
  Chunk p[NQ][kVC];
  // scores of a 16-key block with every row block
  auto scores = [&](const Chunk (&k)[kSteps], int u, f32x4 (&s)[NQ][2]) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) s[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
#pragma unroll
      for (int i = 0; i < NQ; ++i) s[i][u] = Op::score(k[c], qo[i][c], s[i][u]);
  };
  // keys that some row does not see: behind its position, or on no page
  auto is_partial = [&](int t, int ma, int mb) {
    return (t + 1) * kKeys > common || ma < 0 || mb < 0;
  };
  auto mask = [&](f32x4 (&s)[NQ][2], int t, int ma, int mb) {
    if (is_partial(t, ma, mb)) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int left = sh_limit[wrow + 16 * i + n] - t * kKeys;  // of this step's keys
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = Op::skey_of(u, j, quad);
            const bool there = key < left && (key < 16 ? ma : mb) >= 0;
            s[i][u][j] = there ? s[i][u][j] : -INFINITY;
          }
      }
    }
  };
  // A step's largest scores; true if one lies far above its row's maximum.
  float mx[NQ], sums[NQ];
  auto largest = [&]() {
    bool risen = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      mx[i] = fmaxf(fmaxf(fmaxf(s[i][0][0], s[i][0][1]), fmaxf(s[i][0][2], s[i][0][3])),
                    fmaxf(fmaxf(s[i][1][0], s[i][1][1]), fmaxf(s[i][1][2], s[i][1][3]))) *
              a.scale_log2;
      risen |= mx[i] > m[i] + kRise;
    }
    return __ballot(risen) != 0;
  };
  // The maxima brought up to a step's scores, and the sums so far scaled down.
  bool far = false;  // some row's maximum lies far from zero
  auto follow = [&]() {
    far = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float mn = fmaxf(m[i], mx[i]);
      mn = fmaxf(mn, __shfl_xor(mn, 16, 64));
      mn = fmaxf(mn, __shfl_xor(mn, 32, 64));
      const float f = __builtin_amdgcn_exp2f(m[i] - mn);
      m[i] = mn;
      far |= mn > kNone && fabsf(mn) > kFar;
      l[i] *= f;
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[i][d] *= f;
    }
    far = __ballot(far) != 0;
  };
  // A step's weights p and their sums, against the maxima as they are; true if a sum
  // shows that some score lies far above its row's maximum.
  auto weights_of = [&](auto exponent) {
    bool risen = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(exponent(s[i][j >> 2][j & 3], m[i]));
      sums[i] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      risen |= sums[i] > kRiseSum;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(E) == 2) p[i][0][j] = (__bf16)e[j];
        else p[i][j >> 2][j & 3] = e[j];
      }
    }
    return __ballot(risen) != 0;
  };
  auto weights = [&]() {
    return weights_of([&](float x, float m) { return fmaf(x, a.scale_log2, -m); });
  };
  // The product rounded as the maximum's was, so that the largest weight is 1.
  auto far_weights = [&]() {
    weights_of([&](float x, float m) {
#pragma clang fp contract(off)
      const float y = x * a.scale_log2;
      return y - m;
    });
  };
  // The maxima move at the first step, and when a score is far above all before it;
  // otherwise they stay behind (the sums are far from binary32's end) and a step needs
  // neither a rescaling nor an exchange between lanes.  Large tiles are bound by
  // arithmetic and learn it from the weights' sums, without a maximum over the scores;
  // the others by memory, and go without keeping scores and weights side by side.
  // Maxima far from zero are rare: such a step's weights are computed again (a choice
  // before them costs 5% of a prompt's attention).
  auto step_weights = [&]() {
    if constexpr (KW == 1) {
      if (__builtin_expect(weights() | far, 0)) {
        largest();
        follow();
        if (far) far_weights();
        else weights();
      }
    } else {
      if (largest()) follow();
      weights();
      if (__builtin_expect(far, 0)) far_weights();
    }
  };
  auto add_sums = [&]() {
#pragma unroll
    for (int i = 0; i < NQ; ++i) l[i] += sums[i];
  };
  // rows of the pages behind the last key seen hold anything: 0 * NaN is NaN.  Keys of
  // V operand u that lane group q may use:
  auto usable = [&](int t, int u, int ma, int mb) {
    const int key = Op::vkey_of(u, quad);
    return (key < 16 ? ma : mb) >= 0 ? min(max(seen - (t * kKeys + key), 0), kE) : 0;
  };
  auto add_values = [&](const Chunk (&v)[kVC][kDT], const Chunk (&p)[NQ][kVC]) {
#pragma unroll
    for (int u = 0; u < kVC; ++u)
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int i = 0; i < NQ; ++i) o[i][d] = Op::score(v[u][d], p[i][u], o[i][d]);
  };

  if constexpr (!kStaged) {
    // one row group: the keys go from memory to the operands' registers, the next
    // step's while this one is worked on
    Chunk k[2][kSteps], v[kVC][kDT];
    int pa = -1, pb = -1;
    if (t0 < t1) {
      pages_of(t0, pa, pb);
      load_k(t0, pa, pb, k);
    }
    load_q();
    __syncthreads();  // the limits are there, and the last group's sums are out of LDS
    wait_loads();
    for (int t = t0; t < t1; ++t) {
      load_v(t, pa, pb, v);
      const int ma = pa, mb = pb;
      const bool partial = is_partial(t, ma, mb);
      scores(k[0], 0, s);
      scores(k[1], 1, s);
      if (t + 1 < t1) {
        pages_of(t + 1, pa, pb);
        load_k(t + 1, pa, pb, k);
      }
      mask(s, t, ma, mb);
      step_weights();
      add_sums();
      if (partial) {
#pragma unroll
        for (int u = 0; u < kVC; ++u) {
          const int keep = usable(t, u, ma, mb);
#pragma unroll
          for (int d = 0; d < kDT; ++d) v[u][d] = Op::keep(v[u][d], keep);
        }
      }
      add_values(v, p);
    }
  } else {
    // RW row groups use the same keys: a part's RW waves load 1 / RW of a step's
    // operands each, kAhead steps ahead in registers and one in LDS, from where all
    // of them read it (operand order: no bank conflicts).
    constexpr int kShare = kLoads / RW;
    static_assert(kShare * RW == kLoads && (2 * kSteps) % kShare == 0, "K or V for each wave");
    const int r = wave % RW;
    const bool keys = r * kShare < 2 * kSteps;
    const int l0 = keys ? r * kShare : r * kShare - 2 * kSteps;
    const char* pool = keys ? Kb : Vb;
    const uint32_t at_lane = keys ? k_lane : v_lane;
    Chunk* const tile = reinterpret_cast<Chunk*>(sh) + part * kLoads * 64 + lane;
    Chunk hold[kAhead][kShare];
    auto fetch = [&](Chunk (&h)[kShare], int t, int pa, int pb) {
      const char* ba = pool + max(pa, 0) * page_size_bytes;
      const char* bb = pool + max(pb, 0) * page_size_bytes;
      const char* mine = kHalf && (keys ? n >= 8 : quad >= 2) ? bb : ba;
      const int first = (t * kKeys) & (page - 1);
#pragma unroll
      for (int i = 0; i < kShare; ++i) {
        const int x = l0 + i;
        const int64_t to = keys ? (int64_t)(4 * (x % kSteps) * page + (kHalf ? 0 : first) + 4 * (x / kSteps)) * 16
                                : (int64_t)((kHalf ? 0 : first / kE * D) + 16 * x) * 16;
        h[i] = *reinterpret_cast<const Chunk*>(mine + to + at_lane);
      }
    };
    auto put = [&](Chunk (&h)[kShare], int buf, int t, int pa, int pb) {
      if (!keys && is_partial(t, pa, pb)) {
        const int keep = usable(t, 0, pa, pb);
#pragma unroll
        for (int i = 0; i < kShare; ++i) h[i] = Op::keep(h[i], keep);
      }
#pragma unroll
      for (int i = 0; i < kShare; ++i) tile[(buf * KW * kLoads + r * kShare + i) * 64] = h[i];
    };
    int ca = -1, cb = -1;          // pages of the step in LDS
    int ha[kAhead], hb[kAhead];    // and of the steps in registers
    if (t0 < t1) {
      pages_of(t0, ca, cb);
      fetch(hold[0], t0, ca, cb);
    }
    load_q();
    __syncthreads();  // the limits are there, and the last group's sums are out of LDS
    wait_loads();
    if (t0 < t1) put(hold[0], 0, t0, ca, cb);
#pragma unroll
    for (int i = 1; i <= kAhead; ++i) {
      ha[i % kAhead] = hb[i % kAhead] = -1;
      if (t0 + i < t1) {
        pages_of(t0 + i, ha[i % kAhead], hb[i % kAhead]);
        fetch(hold[i % kAhead], t0 + i, ha[i % kAhead], hb[i % kAhead]);
      }
    }
    __syncthreads();
    const int stages = (count + KW - 1) / KW;  // of the longest part
    auto values = [&](int buf, const Chunk (&w)[NQ][kVC]) {
      const Chunk* from = tile + buf * KW * kLoads * 64;
      Chunk v[kVC][kDT];
#pragma unroll
      for (int d = 0; d < kDT; ++d) v[0][d] = from[(2 * kSteps + d) * 64];
      add_values(v, w);
    };
    int buf = 0;
    for (int st0 = 0; st0 < stages; st0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int st = st0 + j, t = t0 + st;
        if (st < stages) {
          Chunk(&h)[kShare] = hold[(j + 1) % kAhead];
          int& na = ha[(j + 1) % kAhead];
          int& nb = hb[(j + 1) % kAhead];
          const int xa = na, xb = nb;
          const int next = buf ^ 1;
          if (t + 1 < t1) put(h, next, t + 1, xa, xb);
          if (t + 1 + kAhead < t1) {
            pages_of(t + 1 + kAhead, na, nb);
            fetch(h, t + 1 + kAhead, na, nb);
          }
          if (t < t1) {
            const Chunk* from = tile + buf * KW * kLoads * 64;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              Chunk k[kSteps];
#pragma unroll
              for (int c = 0; c < kSteps; ++c) k[c] = from[(u * kSteps + c) * 64];
              scores(k, u, s);
            }
            mask(s, t, ca, cb);
            step_weights();
            add_sums();
            __builtin_amdgcn_sched_barrier(0);  // V's registers are the scores'
            values(buf, p);
          }
          ca = xa, cb = xb;
          buf = next;
          __syncthreads();
        }
      }
    }
  }

  // ---- the sums of the key parts joined: the other parts leave theirs in LDS in the
  // registers' order, the first part's waves add them and write the rows ----
  f32x4* const sh_o = reinterpret_cast<f32x4*>(sh);
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    l[i] += __shfl_xor(l[i], 16, 64);
    l[i] += __shfl_xor(l[i], 32, 64);
  }
  if constexpr (KW > 1) {
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (quad == 0) {
          sh_ml[(part * kRows + wrow + 16 * i + n) * 2] = m[i];
          sh_ml[(part * kRows + wrow + 16 * i + n) * 2 + 1] = l[i];
        }
#pragma unroll
        for (int d = 0; d < kDT; ++d)
          sh_o[(((wave - RW) * NQ + i) * kDT + d) * 64 + lane] = o[i][d];
      }
    }
    __syncthreads();
    if (part > 0) return;
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    float f[KW], mn = m[i];
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      f[w] = sh_ml[(w * kRows + wrow + 16 * i + n) * 2];
      mn = fmaxf(mn, f[w]);
    }
    f[0] = __builtin_amdgcn_exp2f(m[i] - mn);
    float ls = l[i] * f[0];
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      f[w] = __builtin_amdgcn_exp2f(f[w] - mn);
      ls += sh_ml[(w * kRows + wrow + 16 * i + n) * 2 + 1] * f[w];
    }
    const int r = wrow + 16 * i + n, row = row0 + r;
    if (row >= rows) continue;
    const int token = row / G;
    E* to = static_cast<E*>(a.out) +
            ((int64_t)(it.w.o0 + token) * a.heads + it.head * G + (row - token * G)) * D + 4 * quad;
    float* part_to = a.part_o + (rec * kRows + r) * D + 4 * quad;
    const float norm = ls > 0.f ? 1.f / ls : 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      f32x4 sum = o[i][d] * f[0];
#pragma unroll
      for (int w = 1; w < KW; ++w)
        sum += sh_o[(((w - 1) * RW + wave) * NQ * kDT + i * kDT + d) * 64 + lane] * f[w];
      if (rec < 0) store4<E>(to + 16 * d, sum * norm);
      else *reinterpret_cast<f32x4*>(part_to + 16 * d) = sum;
    }
    if (rec >= 0 && quad == 0) {
      a.part_ml[(rec * kRows + r) * 2] = mn;
      a.part_ml[(rec * kRows + r) * 2 + 1] = ls;
    }
  }
}

// Waves per SIMD that the registers of NQ row blocks of D dimensions leave room for.
template <typename E, int D, int NQ, int RW, int KW>
struct Shape {
  static constexpr int waves = (sizeof(E) == 2 && D <= 128) || RW * KW == 8 ? 2 : 1;
};

template <typename E, int D, int NQ, int RW, int KW, int kAhead, bool kHalf>
__global__ __launch_bounds__(64 * RW * KW, (Shape<E, D, NQ, RW, KW>::waves)) void k_attend(AttendArgs a) {
  constexpr int kRows = 16 * NQ * RW;
  __shared__ Plan plan;
  __shared__ float sh_ml[KW * kRows * 2];
  __shared__ int sh_limit[kRows];
  __shared__ __align__(16) uint8_t sh[lds_bytes<E, D, NQ, RW, KW>()];
  make_plan(a, kRows, plan);
  const int64_t total = plan.before[kPlanThreads];
  // Workgroup ids go to the 8 XCDs in turn; each XCD takes a contiguous run of
  // spans, so that row tiles that read the same keys share its L2.
  if (blockIdx.x == 0 && threadIdx.x == 0) a.cuts[0].first = plan.spans;
  const int per_xcd = (plan.spans + 7) >> 3;
  const int idx = (int)(blockIdx.x >> 3), span = (int)(blockIdx.x & 7) * per_xcd + idx;
  if (idx >= per_xcd || span >= plan.spans) return;
  const int64_t x0 = span * plan.span, x1 = min(x0 + plan.span, total);
  Group g;
  g.slot_end = 0;
  AttendCut cut = {};
  for (int64_t x = x0; x < x1;) {
    find_group(a, kRows, plan, x, g, [&](int s) { return slot_work(a, s, kRows); });
    if (g.units == 0) {
      x = g.next;
      continue;
    }
    const int first = (int)(x - g.start);
    const int end = (int)min((int64_t)g.units, first + (x1 - x));
    // a cut group's record: a span has two at most, of its first and of its last group
    const int64_t rec = first == 0 && end == g.units ? -1 : 2 * (int64_t)span + (x != x0);
    if (first == 0 && end < g.units) {  // it goes on in the next span
      cut.row0 = g.tile * kRows;
      cut.rows = min(kRows, g.w.chunk * a.group - cut.row0);
      cut.token0 = g.w.o0;
      cut.head = g.head;
      cut.first = (int)rec;
      cut.last = (int)((g.start + g.units - 1) / plan.span);
    }
    attend_steps<E, D, NQ, RW, KW, kAhead, kHalf>(a, g, first, end, rec, sh_ml, sh_limit, sh);
    x += end - first;
  }
  if (threadIdx.x == 0) a.cuts[1 + span] = cut;
}

template <typename E, int D, int NQ, int RW, int KW, int kAhead>
void start(const AttendArgs& a, hipStream_t stream) {
  const int grid = a.grid;
  if (sizeof(E) == 2 && a.c.page_shift == 4)
    hipLaunchKernelGGL((k_attend<E, D, NQ, RW, KW, kAhead, sizeof(E) == 2>), dim3(grid), dim3(64 * RW * KW), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((k_attend<E, D, NQ, RW, KW, kAhead, false>), dim3(grid), dim3(64 * RW * KW), 0, stream, a);
}

// Tiles in use: rows (16 NQ RW), NQ, RW, KW, steps held in registers.
#define ATTEND_TILES(X) \
  X(16, 1, 1, 4, 1) X(32, 2, 1, 4, 1) X(64, 2, 2, 2, 1) X(96, 3, 2, 2, 1) X(128, 2, 4, 2, 2) \
  X(192, 3, 4, 2, 1) X(256, 2, 8, 1, 2) X(384, 3, 8, 1, 1)
#define ATTEND_TILES_256(X) X(16, 1, 1, 4, 1) X(32, 1, 2, 2, 2) X(64, 1, 4, 2, 1) X(128, 1, 8, 1, 1)
#define ATTEND_TILES_F32(X) X(16, 1, 1, 4, 1) X(32, 1, 2, 2, 1)

template <typename E, int D>
bool start_rows(int rows, const AttendArgs& a, hipStream_t stream) {
#define ATTEND_CASE(ROWS, NQ, RW, KW, AHEAD) \
  case ROWS: start<E, D, NQ, RW, KW, AHEAD>(a, stream); return true;
  if constexpr (sizeof(E) == 4) {
    switch (rows) { ATTEND_TILES_F32(ATTEND_CASE) }
  } else if constexpr (D == 256) {
    switch (rows) { ATTEND_TILES_256(ATTEND_CASE) }
  } else {
    switch (rows) { ATTEND_TILES(ATTEND_CASE) }
  }
#undef ATTEND_CASE
  return false;
}

}  // namespace

// The largest tile: what the registers hold (the output's accumulators take
// D / 4 registers per 16 rows of a wave, the queries' operands half of that).
int attend_max_rows(bool bf16, int head_dim) { return !bf16 ? 32 : (head_dim == 256 ? 128 : 384); }

// Rows (token, head) of a tile: as many as the longest chunk needs, spread evenly
// over its tiles.
int attend_rows(bool bf16, int head_dim, int group, int max_chunk) {
  const int most = attend_max_rows(bf16, head_dim);
  const int64_t rows = (int64_t)max_chunk * group;
  const int64_t tiles = (rows + most - 1) / most;
  const int need = (int)((rows + tiles - 1) / tiles);
#define ATTEND_SIZE(ROWS, NQ, RW, KW, AHEAD) \
  if (ROWS >= need) return ROWS;
  if (!bf16) {
    ATTEND_TILES_F32(ATTEND_SIZE)
  } else if (head_dim == 256) {
    ATTEND_TILES_256(ATTEND_SIZE)
  } else {
    ATTEND_TILES(ATTEND_SIZE)
  }
#undef ATTEND_SIZE
  return most;
}

// Workgroups, and spans at most: what is resident at once.  Two waves per SIMD (four
// waves of up to 256 registers from each of two workgroups, or one of eight waves),
// one where a wave needs more registers.
int attend_grid(bool bf16, int head_dim, int rows) {
  return bf16 && head_dim <= 128 && rows <= 96 ? 512 : 256;
}

hipError_t launch_attend(bool bf16, int rows, const AttendArgs& a, hipStream_t stream) {
  {
    TimingScope t("attend", stream);
    const int D = a.c.head_dim;
    const bool started =
        bf16 ? (D == 64 ? start_rows<uint16_t, 64>(rows, a, stream)
                        : (D == 128 ? start_rows<uint16_t, 128>(rows, a, stream)
                                    : start_rows<uint16_t, 256>(rows, a, stream)))
             : (D == 64 ? start_rows<float, 64>(rows, a, stream)
                        : (D == 128 ? start_rows<float, 128>(rows, a, stream)
                                    : start_rows<float, 256>(rows, a, stream)));
    if (!started) return hipErrorInvalidValue;
  }
  {
    TimingScope t("attend_join", stream);
    const int per = join_rows(a.c.head_dim);
    const dim3 join((unsigned)a.grid, (unsigned)((rows + per - 1) / per));
    if (bf16)
      hipLaunchKernelGGL(k_attend_join<uint16_t>, join, dim3(kPlanThreads), 0, stream, a, rows);
    else
      hipLaunchKernelGGL(k_attend_join<float>, join, dim3(kPlanThreads), 0, stream, a, rows);
  }
  return hipGetLastError();
}

}  // namespace dspark
