// attend4.hip -- attention of a chunk of new tokens per slot over a paged cache in 4 bits.
//
// The mathematics, the tiles' rows, the division of the work over spans and the join of cut
// groups are those of attend.hip (attend_common.h); the pages' layout is that of
// cache_store.hip.  What differs is how the operands come about:
//   K: a lane's share of a key is D / 4 neighbouring elements, D / 8 bytes in memory; the queries are
//     loaded in the same order, so that the product over the dimensions needs no exchange.
//   V: a lane's 16 bytes are 8 keys x 4 elements.  A conversion takes two neighbouring
//     elements of one key with that key's scale to two bf16 (exact: two significant bits);
//     a byte permutation pairs the keys up as the matrix operand wants them.
// Every wave loads and converts its own operands: no LDS and no barrier in the loop.
#include "attend_common.h"

namespace dspark {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

template <int kSel>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t w, float s) {
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, kSel);
  return __builtin_bit_cast(uint32_t, b);
}
template <int kSel>
__device__ __forceinline__ f32x2 pair_f32(uint32_t w, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, kSel);
}

// A lane's codes of one step as they lie in memory.
template <int D>
struct RawK {  // one 16-key block: D / 4 elements of a key
  uint32_t w[D / 32];
  uint32_t scale[D == 256 ? 2 : 1];
};
template <int D>
struct RawV {  // bf16: 8 keys, f32: 2 x 4 keys, of D / 16 elements
  uint32_t w[D / 64][4];
  uint32_t scale[2];
};

// Key steps [first, end) of a group; `rec`: the record that takes the sums of a group
// that is cut, or -1.  RW x KW waves: RW row groups of NQ 16-row blocks each, KW parts of the
// key range.  kHalf: pages of 16 tokens, two of which a step spans.
template <typename E, int D, int NQ, int RW, int KW, bool kHalf>
__device__ __forceinline__ void attend4_steps(const AttendArgs& a, const Group& it, int first,
                                              int end, int64_t rec, float* sh_ml, int* sh_limit,
                                              f32x4* sh_o) {
  typedef Ops<E> Op;
  typedef typename Op::Chunk Chunk;
  constexpr bool kF32 = sizeof(E) == 4;
  constexpr int kE = Op::kE;
  constexpr int kSteps = D / (4 * kE);  // K operands per 16 keys
  constexpr int kDT = D / 16;           // elements of a lane's dimensions: output operands
  constexpr int kVC = Op::kVChunks;
  constexpr int kWaveRows = 16 * NQ;
  constexpr int kRows = kWaveRows * RW;
  constexpr int kThreads = 64 * RW * KW;
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
  // without key parts nothing else ends a group for all waves, and one may still read its limits
  if constexpr (KW == 1) __syncthreads();
  for (int r = threadIdx.x; r < kRows; r += kThreads)
    sh_limit[r] = min(it.w.len + min((row0 + r) / G, it.w.chunk) + 1, it.w.keys);
  const int page = 1 << shift;
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
  const int64_t page_bytes = a.c.page_bytes;
  const int code_head = it.head * page * (D / 2);
  const int scale_head = H * page * (D / 2) + it.head * page * (D / 32);
  const uint8_t* Kb = static_cast<const uint8_t*>(a.K);
  const uint8_t* Vb = static_cast<const uint8_t*>(a.V);
  // the page that holds a step's key, and the key's place in it
  auto page_of = [&](int key, int pa, int pb) { return (int64_t)max(key < 16 ? pa : pb, 0) * page_bytes; };
  auto load_k = [&](int t, int pa, int pb, RawK<D> (&k)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = Op::key_of(u, n), row = (t * kKeys + key) & (page - 1);
      const uint8_t* blob = Kb + page_of(key, pa, pb);
      const uint8_t* codes = blob + code_head;
      const uint8_t* scales = blob + scale_head;
      if constexpr (D == 64) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(codes + ((quad >> 1) * page + row) * 16 + (quad & 1) * 8);
        k[u].w[0] = w.x;
        k[u].w[1] = w.y;
        k[u].scale[0] = scales[(quad >> 1) * page + row];
      } else {
#pragma unroll
        for (int b = 0; b < D / 128; ++b) {
          const int block = quad * (D / 128) + b;
          const u32x4 w = *reinterpret_cast<const u32x4*>(codes + (block * page + row) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) k[u].w[4 * b + i] = w[i];
          k[u].scale[b] = scales[block * page + row];
        }
      }
    }
  };
  auto load_v = [&](int t, int pa, int pb, RawV<D>& v) {
    const int block = n * D / 512;
    if constexpr (!kF32) {
      const int key = 8 * quad, row = (t * kKeys + key) & (page - 1);
      const uint8_t* blob = Vb + page_of(key, pa, pb);
      const uint8_t* codes = blob + code_head + (row >> 3) * (D / 64 * 256) + n * 16;
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(codes + g * 256);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[g][i] = w[i];
      }
      const u32x2 s = *reinterpret_cast<const u32x2*>(blob + scale_head + block * page + row);
      v.scale[0] = s.x;
      v.scale[1] = s.y;
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = 16 * u + 4 * quad, row = (t * kKeys + key) & (page - 1);
        const uint8_t* blob = Vb + page_of(key, pa, pb);
        const uint8_t* codes = blob + code_head + (row >> 3) * (D / 64 * 256) + n * 16 + (row & 4);
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v.w[g][2 * h + u] = *reinterpret_cast<const uint32_t*>(codes + g * 256 + h * 8);
        v.scale[u] = *reinterpret_cast<const uint32_t*>(blob + scale_head + block * page + row);
      }
    }
  };
  // what a page holds behind the last token seen, or where there is no page, counts as zeros
  auto clear_v = [&](int t, int pa, int pb, RawV<D>& v) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = kF32 ? 16 * u + 4 * quad : 8 * quad + 4 * u;
      const int keep = (key < 16 ? pa : pb) >= 0 ? min(max(seen - (t * kKeys + key), 0), 4) : 0;
      const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        v.w[g][u] &= mask;
        v.w[g][2 + u] &= mask;
      }
      v.scale[u] = (v.scale[u] & mask) | (0x7F7F7F7Fu & ~mask);
    }
  };
  // operands of a 16-key block: lane (n, quad), operand s: elements quad D / 4 + kE s ..
  auto k_operands = [&](const RawK<D>& r, Chunk (&k)[kSteps]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if constexpr (!kF32) {
        const float f = scale_of(r.scale[D == 256 ? s / 4 : 0]);
        const u32x4 w = {pair_bf16<0>(r.w[s], f), pair_bf16<1>(r.w[s], f), pair_bf16<2>(r.w[s], f), pair_bf16<3>(r.w[s], f)};
        k[s] = __builtin_bit_cast(bf16x8, w);
      } else {
        const float f = scale_of(r.scale[D == 256 ? s / 8 : 0]);
        const uint32_t w = r.w[s / 2];
        const f32x2 x = s & 1 ? pair_f32<2>(w, f) : pair_f32<0>(w, f);
        const f32x2 y = s & 1 ? pair_f32<3>(w, f) : pair_f32<1>(w, f);
        k[s] = f32x4{x[0], x[1], y[0], y[1]};
      }
    }
  };
  // operand d: element n D / 16 + d of the lane's keys
  auto v_operands = [&](const RawV<D>& r, Chunk (&v)[kVC][kDT]) {
    float s[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) s[t] = scale_of(r.scale[t >> 2] >> (8 * (t & 3)) & 255u);
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = r.w[g][2 * h], y = r.w[g][2 * h + 1];
        const int d = 4 * g + 2 * h;
        if constexpr (!kF32) {
          const uint32_t p[8] = {pair_bf16<0>(x, s[0]), pair_bf16<1>(x, s[1]), pair_bf16<2>(x, s[2]), pair_bf16<3>(x, s[3]),
                                 pair_bf16<0>(y, s[4]), pair_bf16<1>(y, s[5]), pair_bf16<2>(y, s[6]), pair_bf16<3>(y, s[7])};
          u32x4 lo, hi;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
            hi[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
          }
          v[0][d] = __builtin_bit_cast(bf16x8, lo);
          v[0][d + 1] = __builtin_bit_cast(bf16x8, hi);
        } else {
          const f32x2 p[8] = {pair_f32<0>(x, s[0]), pair_f32<1>(x, s[1]), pair_f32<2>(x, s[2]), pair_f32<3>(x, s[3]),
                              pair_f32<0>(y, s[4]), pair_f32<1>(y, s[5]), pair_f32<2>(y, s[6]), pair_f32<3>(y, s[7])};
#pragma unroll
          for (int u = 0; u < kVC; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              v[u][d + e] = __builtin_bit_cast(Chunk, f32x4{p[4 * u][e], p[4 * u + 1][e], p[4 * u + 2][e], p[4 * u + 3][e]});
        }
      }
  };

  RawK<D> k[2];
  RawV<D> v;
  int pa = -1, pb = -1;
  if (t0 < t1) {
    pages_of(t0, pa, pb);
    load_k(t0, pa, pb, k);
    load_v(t0, pa, pb, v);
  }
  // queries as operands
  Chunk qo[NQ][kSteps];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int row = row0 + wrow + 16 * i + n;
    const bool live = row < rows;
    const int token = live ? row / G : 0;
    const E* p = q + ((int64_t)(it.w.o0 + token) * a.heads + it.head * G + (live ? row - token * G : 0)) * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      qo[i][s] = live ? *reinterpret_cast<const Chunk*>(p + quad * (D / 4) + kE * s) : Op::zero();
  }
  __syncthreads();  // the limits are there, and the last group's sums are out of LDS
  wait_loads();
  for (int t = t0; t < t1; ++t) {
    const int ma = pa, mb = pb;
    const bool partial = (t + 1) * kKeys > common || ma < 0 || mb < 0;
    f32x4 s[NQ][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Chunk ko[kSteps];
      k_operands(k[u], ko);
#pragma unroll
      for (int i = 0; i < NQ; ++i) s[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int i = 0; i < NQ; ++i) s[i][u] = Op::score(ko[c], qo[i][c], s[i][u]);
    }
    RawV<D> w = v;
    if (t + 1 < t1) {
      pages_of(t + 1, pa, pb);
      load_k(t + 1, pa, pb, k);
      load_v(t + 1, pa, pb, v);
    }
    if (partial) {
      clear_v(t, ma, mb, w);
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
    // The maxima move at the first step, and when a score is far above all before it;
    // otherwise they stay behind, and a step needs no rescaling.
    float mx[NQ];
    bool risen = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      mx[i] = fmaxf(fmaxf(fmaxf(s[i][0][0], s[i][0][1]), fmaxf(s[i][0][2], s[i][0][3])),
                    fmaxf(fmaxf(s[i][1][0], s[i][1][1]), fmaxf(s[i][1][2], s[i][1][3]))) * a.scale_log2;
      risen |= mx[i] > m[i] + kRise;
    }
    if (__ballot(risen) != 0) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        float mn = fmaxf(m[i], mx[i]);
        mn = fmaxf(mn, __shfl_xor(mn, 16, 64));
        mn = fmaxf(mn, __shfl_xor(mn, 32, 64));
        const float f = __builtin_amdgcn_exp2f(m[i] - mn);
        m[i] = mn;
        l[i] *= f;
#pragma unroll
        for (int d = 0; d < kDT; ++d) o[i][d] *= f;
      }
    }
    Chunk p[NQ][kVC];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      // Far from zero the maximum is a product rounded by a whole or more: the weights
      // then come from the product rounded as it was, so that the largest is 1.
      const bool far = m[i] > kNone && fabsf(m[i]) > kFar;
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = s[i][j >> 2][j & 3];
        float y;
        {
#pragma clang fp contract(off)
          y = x * a.scale_log2;
          y = y - m[i];
        }
        e[j] = __builtin_amdgcn_exp2f(far ? y : fmaf(x, a.scale_log2, -m[i]));
      }
      l[i] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (!kF32) p[i][0][j] = (__bf16)e[j];
        else p[i][j >> 2][j & 3] = e[j];
      }
    }
    Chunk vo[kVC][kDT];
    v_operands(w, vo);
#pragma unroll
    for (int u = 0; u < kVC; ++u)
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int i = 0; i < NQ; ++i) o[i][d] = Op::score(vo[u][d], p[i][u], o[i][d]);
  }

  // ---- the sums of the key parts joined: the other parts leave theirs in LDS in the
  // registers' order, the first part's waves add them and write the rows ----
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
        for (int d = 0; d < kDT; ++d) sh_o[(((wave - RW) * NQ + i) * kDT + d) * 64 + lane] = o[i][d];
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
    // output operand d, register j: element (4 quad + j) D / 16 + d
    E* to = static_cast<E*>(a.out) +
            ((int64_t)(it.w.o0 + token) * a.heads + it.head * G + (row - token * G)) * D + quad * (D / 4);
    float* part_to = a.part_o + (rec * kRows + r) * D + quad * (D / 4);
    const float norm = rec < 0 ? (ls > 0.f ? 1.f / ls : 0.f) : 1.f;
    f32x4 sum[kDT];
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      sum[d] = o[i][d] * f[0];
#pragma unroll
      for (int w = 1; w < KW; ++w)
        sum[d] += sh_o[(((w - 1) * RW + wave) * NQ * kDT + i * kDT + d) * 64 + lane] * f[w];
      sum[d] *= norm;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int d = 0; d < kDT; d += 4) {
        const f32x4 x = {sum[d][j], sum[d + 1][j], sum[d + 2][j], sum[d + 3][j]};
        if (rec < 0) store4<E>(to + j * kDT + d, x);
        else *reinterpret_cast<f32x4*>(part_to + j * kDT + d) = x;
      }
    if (rec >= 0 && quad == 0) {
      a.part_ml[(rec * kRows + r) * 2] = mn;
      a.part_ml[(rec * kRows + r) * 2 + 1] = ls;
    }
  }
}

template <typename E, int D, int NQ, int RW, int KW>
struct Shape4 {
  static constexpr int waves = (sizeof(E) == 2 && D <= 128) || RW * KW == 8 ? 2 : 1;
};

template <typename E, int D, int NQ, int RW, int KW, bool kHalf>
__global__ __launch_bounds__(64 * RW * KW, (Shape4<E, D, NQ, RW, KW>::waves)) void k_attend4(AttendArgs a) {
  constexpr int kRows = 16 * NQ * RW;
  __shared__ Plan plan;
  __shared__ float sh_ml[KW * kRows * 2];
  __shared__ int sh_limit[kRows];
  __shared__ f32x4 sh_o[KW > 1 ? (KW - 1) * kRows * D / 4 : 1];
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
    find_group(a, kRows, plan, x, g);
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
    attend4_steps<E, D, NQ, RW, KW, kHalf>(a, g, first, end, rec, sh_ml, sh_limit, sh_o);
    x += end - first;
  }
  if (threadIdx.x == 0) a.cuts[1 + span] = cut;
}

template <typename E, int D, int NQ, int RW, int KW>
void start4(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid(a.grid), block(64 * RW * KW);
  if (a.c.page_shift == 4) hipLaunchKernelGGL((k_attend4<E, D, NQ, RW, KW, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_attend4<E, D, NQ, RW, KW, false>), grid, block, 0, stream, a);
}

// Tiles in use: rows (16 NQ RW), NQ, RW, KW.
#define ATTEND4_TILES(X) X(16, 1, 1, 4) X(32, 2, 1, 4) X(64, 2, 2, 2) X(96, 3, 2, 2) X(128, 2, 4, 2) \
  X(192, 3, 4, 2) X(256, 2, 8, 1) X(384, 3, 8, 1)
#define ATTEND4_TILES_256(X) X(16, 1, 1, 4) X(32, 1, 2, 2) X(64, 1, 4, 2) X(128, 1, 8, 1)
#define ATTEND4_TILES_F32(X) X(16, 1, 1, 4) X(32, 1, 2, 2)

template <typename E, int D>
bool start4_rows(int rows, const AttendArgs& a, hipStream_t stream) {
#define ATTEND4_CASE(ROWS, NQ, RW, KW) \
  case ROWS: start4<E, D, NQ, RW, KW>(a, stream); return true;
  if constexpr (sizeof(E) == 4) {
    switch (rows) { ATTEND4_TILES_F32(ATTEND4_CASE) }
  } else if constexpr (D == 256) {
    switch (rows) { ATTEND4_TILES_256(ATTEND4_CASE) }
  } else {
    switch (rows) { ATTEND4_TILES(ATTEND4_CASE) }
  }
#undef ATTEND4_CASE
  return false;
}

}  // namespace

int attend4_max_rows(bool bf16, int head_dim) { return !bf16 ? 32 : (head_dim == 256 ? 128 : 384); }

// Rows (token, head) of a tile: as many as the longest chunk needs, spread evenly
// over its tiles.
int attend4_rows(bool bf16, int head_dim, int group, int max_chunk) {
  const int most = attend4_max_rows(bf16, head_dim);
  const int64_t rows = (int64_t)max_chunk * group;
  const int64_t tiles = (rows + most - 1) / most;
  const int need = (int)((rows + tiles - 1) / tiles);
#define ATTEND4_SIZE(ROWS, NQ, RW, KW) \
  if (ROWS >= need) return ROWS;
  if (!bf16) {
    ATTEND4_TILES_F32(ATTEND4_SIZE)
  } else if (head_dim == 256) {
    ATTEND4_TILES_256(ATTEND4_SIZE)
  } else {
    ATTEND4_TILES(ATTEND4_SIZE)
  }
#undef ATTEND4_SIZE
  return most;
}

// Workgroups, and spans at most: what is resident at once.
int attend4_grid(bool bf16, int head_dim, int rows) {
  return bf16 && head_dim <= 128 && rows <= 96 ? 512 : 256;
}

hipError_t launch_attend4(bool bf16, int rows, const AttendArgs& a, hipStream_t stream) {
  {
    TimingScope t("attend4", stream);
    const int D = a.c.head_dim;
    const bool started =
        bf16 ? (D == 64 ? start4_rows<uint16_t, 64>(rows, a, stream)
                        : (D == 128 ? start4_rows<uint16_t, 128>(rows, a, stream)
                                    : start4_rows<uint16_t, 256>(rows, a, stream)))
             : (D == 64 ? start4_rows<float, 64>(rows, a, stream)
                        : (D == 128 ? start4_rows<float, 128>(rows, a, stream)
                                    : start4_rows<float, 256>(rows, a, stream)));
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
