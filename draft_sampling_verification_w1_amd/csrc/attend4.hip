// attend4.hip -- attention of a chunk of new tokens per slot over a paged cache in 4 bits.
//
// The mathematics, the tiles' rows, the division of the work over spans and the join of cut
// groups are those of attend.hip (attend_common.h); the pages' layout is that of
// cache_store.hip.  What differs is how the operands come about:
//   K, bf16 queries: the codes and scales go into the scaled matrix product as they lie in memory,
//     16 bytes (a block of 32 elements) per lane; the queries are two 8-bit operands (Queries).
//     Where these are too coarse for a row and the keys of a step, both are bf16 operands.
//   K, f32 queries: a lane's D / 4 neighbouring elements of a key, converted to binary32.
//   V: a lane's 16 bytes are 8 keys x 4 elements.  A conversion takes two neighbouring
//     elements of one key with that key's scale to two bf16 (exact: two significant bits);
//     a byte permutation pairs the keys up as the matrix operand wants them.
// Every wave loads and converts its own codes, straight from the pages; the queries lie in LDS as
// operands; the loop over the keys has no barrier.
//
// What bounds it.  A step of 32 keys by 48 rows of 128 dimensions is 12 scaled products of 32 cycles
// (queries in two parts) and 24 of 16, beside 64 conversions and permutations, 24 exponentials and as many
// roundings at 4 to 9 cycles each: both units take about as long, and one wave hardly runs them side by
// side.  Two waves per SIMD do, where one is kept at the matrix products (matrix_first).  256 slots
// of 17 tokens: the matrix units are busy 38 % of the time, the vector units 59 %.
//
// Measured (32 heads on 8, 128 dimensions, bf16), with the join:
//   1 token over 30,000: 20 us (attention 15, join 5), 1.6 TB/s: what a launch, the plan, the page
//     ids and the queries take before the first step (whole elements: 48 us);
//   32 slots, up to 2,100 cached, 1 to 17 new tokens: 41 us, 1.2 TB/s (61);
//   256 slots, up to 4,096 cached, 17 new tokens: 295 us, 2.7 TB/s, 620 TFLOP/s (572);
//   256 slots, up to 4,096 cached, 1 new token: 142 us, 5.0 TB/s;
//   2 prompts, 2,048 tokens behind up to 8,192: 457 us, 990 TFLOP/s (494).
// Tried without gain: one wave per SIMD on 80 rows (492 us for the 324 of then), values converted one step
// late, two waves to a workgroup (343), the next group's pages and queries loaded before a group's join
// (355), values converted once into LDS for 8 waves (461 for 460), tiles of 192, 96 and 256 rows for prompts
// (469, 462, 474).
#include <type_traits>

#include "attend_common.h"

namespace dspark {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int kSel>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t w, float s) {
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, kSel);
  return __builtin_bit_cast(uint32_t, b);
}
template <int kSel>
__device__ __forceinline__ f32x2 pair_f32(uint32_t w, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, kSel);
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A lane's codes of one step as they lie in memory.
template <int D>
struct RawK {  // one 16-key block: blocks of 32 elements of a key (f32: D / 4 elements)
  uint32_t w[D == 256 ? 8 : 4];
  uint32_t scale[D == 256 ? 2 : 1];  // of the key and its neighbours in an aligned four
};
template <int D>
struct RawV {  // bf16: 8 keys, f32: 2 x 4 keys, of D / 16 elements
  uint32_t w[D / 64][4];
  uint32_t scale[2];
};

// A lane's share of a row of queries as matrix operands, left in LDS in 16-byte pieces 64 lanes apart: all key
// parts use them, and a wave has its registers for codes on their way and for the sums.
template <typename E, int D>
struct Queries;

// f32: piece s: elements quad D / 4 + 4 s ..
template <int D>
struct Queries<float, D> {
  static constexpr int kPieces = D / 16;
  u32x4 raw[kPieces];
  __device__ __forceinline__ void load(const float* p, bool live, int quad) {
#pragma unroll
    for (int s = 0; s < kPieces; ++s)
      raw[s] = live ? *reinterpret_cast<const u32x4*>(p + quad * (D / 4) + 4 * s) : u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void put(int, float, u32x4* to, uint32_t*) const {
#pragma unroll
    for (int s = 0; s < kPieces; ++s) to[64 * s] = raw[s];
  }
};

// bf16: the keys' codes are operands as they are, beside two 8-bit numbers per query element whose
// sum it is: hi, its E4M3 rounding (4 significant bits) relative to a power of two that takes the
// row's largest element to [128, 256), and lo, what is left, 16 times finer.  bf16 has 8
// significant bits: the sum is exact for elements above 2^-13 of the row's largest, and off by at most
// 2^-21 of that below.  The product with 4-bit codes and their scales is exact, sums are binary32.
// What the sums are off by, added up over a row (rest), moves its score with a key by no more
// than scale rest max|k|.  16 rows have a limit, the largest scale byte of a key up to which that is below
// kSplit for all of them; steps with larger ones are multiplied in bf16 (exact_scores).
//   operand of 128 dimensions: lane group quad holds elements 16 quad .. + 15 and 64 + 16 quad .. + 15
//   D = 64: hi and lo are the two halves of one operand, the keys' blocks are loaded twice.
// Operand c: pieces 2 c and 2 c + 1; c even hi, odd lo (D = 64: piece 0 hi, 1 lo).  The scale bytes of hi
// and lo are bytes 0 and 1 of a word (D = 64: byte 0 that of the lane group's half), byte 3 is the 16
// rows' limit.
template <int D>
constexpr int kQueryOps = D / 64;
// How far (binary logarithm) the two parts may move a score: 0.034 % of a weight, a twelfth of what its
// rounding to bf16 may take.  Rows whose elements lie within 2^13 of the largest have no limit; of normal
// variates of 128 dimensions one row in 30 has, for keys in the thousands.  Where every step is multiplied
// in bf16, 256 slots of 17 tokens take 687 us instead of 295, a token over 30,000 24 instead of 20.5.
constexpr float kSplit = 0x1p-11f;

template <int D>
struct Queries<uint16_t, D> {
  static constexpr int kPieces = 2 * kQueryOps<D>;
  u32x4 raw[D / 64][2];
  __device__ __forceinline__ void load(const uint16_t* p, bool live, int quad) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        raw[g][h] =
            live ? *reinterpret_cast<const u32x4*>(p + 64 * g + 16 * quad + 8 * h) : u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void put(int quad, float scale_log2, u32x4* to, uint32_t* scale) const {
    // the largest magnitude and the smallest but 0, less a bit
    typedef uint16_t Two __attribute__((ext_vector_type(2)));
    Two large = {0, 0}, small = {0xFFFF, 0xFFFF};
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Two m = __builtin_bit_cast(Two, raw[g][h][i] & 0x7FFF7FFFu);
          large = __builtin_elementwise_max(large, m);
          small = __builtin_elementwise_min(small, m - Two{1, 1});
        }
    uint32_t top = max((uint32_t)large.x, (uint32_t)large.y);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const uint32_t byte = max((int)(top >> 7) - 7, 5);
    const float f = __uint_as_float((254u - byte) << 23);
    float rest = 0.f;  // in units of lo
    const auto split = [&](auto with_rest) {
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        u32x4 his, los;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w0 = raw[g][h][2 * i], w1 = raw[g][h][2 * i + 1];
            const float a = bf16_lo(w0) * f, b = bf16_hi(w0) * f, c = bf16_lo(w1) * f, d = bf16_hi(w1) * f;
            int hi = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, hi, true);
            const float x[4] = {(a - __builtin_amdgcn_cvt_f32_fp8(hi, 0)) * 16.f,
                                (b - __builtin_amdgcn_cvt_f32_fp8(hi, 1)) * 16.f,
                                (c - __builtin_amdgcn_cvt_f32_fp8(hi, 2)) * 16.f,
                                (d - __builtin_amdgcn_cvt_f32_fp8(hi, 3)) * 16.f};
            int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
            if constexpr (decltype(with_rest)::value)
              rest += fabsf(x[0] - __builtin_amdgcn_cvt_f32_fp8(lo, 0)) +
                      fabsf(x[1] - __builtin_amdgcn_cvt_f32_fp8(lo, 1)) +
                      (fabsf(x[2] - __builtin_amdgcn_cvt_f32_fp8(lo, 2)) +
                       fabsf(x[3] - __builtin_amdgcn_cvt_f32_fp8(lo, 3)));
            his[2 * h + i] = (uint32_t)hi;
            los[2 * h + i] = (uint32_t)lo;
          }
        to[64 * (D == 64 ? 0 : g / 2 * 4 + g % 2)] = his;
        to[64 * (D == 64 ? 1 : g / 2 * 4 + 2 + g % 2)] = los;
      }
    };
    int limit = 255;
    // one of the lane's elements is below 2^-6 in units of hi, or no normal number
    if (__ballot(min((uint32_t)small.x, (uint32_t)small.y) + 1u < max((int)byte - 6, 1) << 7)) {
      split(std::true_type());
      rest += __shfl_xor(rest, 16, 64);
      rest += __shfl_xor(rest, 32, 64);
      // 2^(byte - 127) rest / 16 scale_log2 6 2^(limit - 127) <= kSplit, by the exponent of what stands
      // beside the powers of two
      const float x = rest * (scale_log2 * (6.f / kSplit));
      if (x > 0.f) limit = min(max(384 - (int)byte - (int)(__float_as_uint(x) >> 23), 0), 255);
      limit = 255 - (int)max_lanes16((uint32_t)(255 - limit));
    } else {
      split(std::false_type());
    }
    *scale = (D == 64 ? (quad < 2 ? byte : byte - 4) : byte | (byte - 4) << 8) | (uint32_t)limit << 24;
  }
};

// LDS of a workgroup: the queries, then (at the same place) the outputs of all key parts but the first.
template <typename E, int D, int NQ, int RW, int KW>
__host__ __device__ constexpr int lds_pieces() {
  const int queries = NQ * RW * Queries<E, D>::kPieces * 64;
  const int join = (KW - 1) * 16 * NQ * RW * D / 4;
  return queries > join ? queries : join;
}

// Key steps [first, end) of a group; `rec`: the record that takes the sums of a group
// that is cut, or -1.  RW x KW waves: RW row groups of NQ 16-row blocks each, KW parts of the
// key range.  kHalf: pages of 16 tokens, two of which a step spans.
template <typename E, int D, int NQ, int RW, int KW, bool kHalf>
__device__ __forceinline__ void attend4_steps(const AttendArgs& a, const Group& it, int first,
                                              int end, int64_t rec, float* sh_ml, int* sh_limit,
                                              uint32_t* sh_scale, u32x4* sh) {
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
  // Two waves share a SIMD, of one workgroup or of two (ids 256 apart).  Matrix instructions go first, and of
  // two waves at the same place always the same one, so that the waves do not stay side by side in
  // the phases that need the same unit (two prompts: 468 us without, 449 with).
  const int odd = RW * KW == 8 ? wave >> 2 : (int)(blockIdx.x >> 8 & 1);
  auto matrix_first = [&]() {
    if (odd) __builtin_amdgcn_s_setprio(3);
    else __builtin_amdgcn_s_setprio(2);
  };
  auto matrix_done = [&]() {
    if (odd) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
  };
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
  int col0 = ((t0 * kKeys) >> shift) & ~1;
  auto columns = [&](int c0) {
    const int c = c0 + lane;
    const int p = c < a.c.max_pages ? table[c] : -1;
    return p >= 0 && p < a.c.pages ? p : -1;
  };
  int ids = columns(col0), ids_next = columns(col0 + 64);
  // queries as operands, each row block by one key part; on their way beside the page ids
  typedef Queries<E, D> Query;
  constexpr int kMine = (NQ + KW - 1) / KW;
  u32x4* const mine = sh + (wave % RW) * NQ * Query::kPieces * 64 + lane;
  Query rows_of[kMine];
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    const int i = x * KW + part, row = row0 + wrow + 16 * i + n;
    const bool live = i < NQ && row < rows;
    const int token = live ? row / G : 0;
    const int64_t at = (int64_t)(it.w.o0 + token) * a.heads + it.head * G + (live ? row - token * G : 0);
    rows_of[x].load(q + at * D, live, quad);
  }
  __syncthreads();  // the last group's limits, queries and sums are out of LDS
  for (int r = threadIdx.x; r < kRows; r += kThreads)
    sh_limit[r] = min(it.w.len + min((row0 + r) / G, it.w.chunk) + 1, it.w.keys);
  const int page = 1 << shift;
  auto pages_of = [&](int t, int& pa, int& pb) {
    const int ca = (t * kKeys) >> shift, cb = (t * kKeys + 16) >> shift;
    if (ca >= col0 + 64) {  // a step's two columns lie in one window: both are even, or the same
      col0 += 64;
      ids = ids_next;
      ids_next = columns(col0 + 64);
    }
    pa = __builtin_amdgcn_readlane(ids, ca - col0);
    pb = __builtin_amdgcn_readlane(ids, cb - col0);
  };
  // Operand addresses: a wave-uniform base (page, step within the page) and a lane's 32-bit
  // offset that stays the same through the pass.  Pages of 16: the lane's page, no step within.
  const int64_t page_bytes = a.c.page_bytes;
  const uint8_t* Kb = static_cast<const uint8_t*>(a.K) + it.head * page * (D / 2);
  const uint8_t* Vb = static_cast<const uint8_t*>(a.V) + it.head * page * (D / 2);
  // from a page's codes of this head to its scales
  const uint32_t to_scales =
      (uint32_t)(H * page * (D / 2) - it.head * page * (D / 2) + it.head * page * (D / 32));
  const int k_key = Op::key_of(0, n) & (page - 1);
  // the first block, others 4 on (f32: 1 on)
  const int k_block = kF32 ? quad * D / 128 : (D == 64 ? quad & 1 : quad);
  const uint32_t k_lane = (uint32_t)((k_block * page + k_key) * 16 + (kF32 && D == 64 ? (quad & 1) * 8 : 0));
  const uint32_t ks_lane = to_scales + (uint32_t)(k_block * page + (k_key & (kF32 ? ~3 : ~7)));
  const int v_key = (kF32 ? 4 * quad : 8 * quad) & (page - 1);
  const uint32_t v_lane = (uint32_t)((v_key >> 3) * (D / 64 * 256) + n * 16 + (v_key & 4));
  const uint32_t vs_lane = to_scales + (uint32_t)((n * D / 512) * page + v_key);
  // the page of a lane's keys; f32 has 16 keys of a step on each of two pages for all lanes
  auto page_at = [&](const uint8_t* pool, int pa, int pb, bool second) {
    if constexpr (kHalf) return pool + (int64_t)max(second ? pb : pa, 0) * page_bytes;
    else return pool + (int64_t)max(pa, 0) * page_bytes;
  };
  auto load_k = [&](int t, int pa, int pb, RawK<D> (&k)[2]) {
    const int at = kHalf ? 0 : (t * kKeys) & (page - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* base = page_at(Kb, pa, pb, kF32 ? u == 1 : n >= 8);
      const int row = at + (kF32 ? (kHalf ? 0 : 16 * u) : 4 * u);
      if constexpr (kF32 && D == 64) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(base + row * 16 + k_lane);
        k[u].w[0] = w.x;
        k[u].w[1] = w.y;
        k[u].scale[0] = *reinterpret_cast<const uint32_t*>(base + row + ks_lane);
      } else {
#pragma unroll
        for (int b = 0; b < (D + 127) / 128; ++b) {
          const int block = kF32 ? b : 4 * b;
          const u32x4 w = *reinterpret_cast<const u32x4*>(base + (row + block * page) * 16 + k_lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) k[u].w[4 * b + i] = w[i];
          if constexpr (kF32) {
            k[u].scale[b] = *reinterpret_cast<const uint32_t*>(base + row + block * page + ks_lane);
          } else if (u == 0) {  // the lane's two keys are 4 apart, in the same 8
            const u32x2 x = *reinterpret_cast<const u32x2*>(base + row + block * page + ks_lane);
            k[0].scale[b] = x.x;
            k[1].scale[b] = x.y;
          }
        }
      }
    }
  };
  auto load_v = [&](int t, int pa, int pb, RawV<D>& v) {
    const int at = kHalf ? 0 : (t * kKeys) & (page - 1);
    if constexpr (!kF32) {
      const uint8_t* base = page_at(Vb, pa, pb, quad >= 2);
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(base + (at >> 3) * (D / 64 * 256) + g * 256 + v_lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[g][i] = w[i];
      }
      const u32x2 s = *reinterpret_cast<const u32x2*>(base + at + vs_lane);
      v.scale[0] = s.x;
      v.scale[1] = s.y;
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* base = page_at(Vb, pa, pb, u == 1);
        const int row = at + (kHalf ? 0 : 16 * u);
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v.w[g][2 * h + u] = *reinterpret_cast<const uint32_t*>(
                base + (row >> 3) * (D / 64 * 256) + g * 256 + h * 8 + v_lane);
        v.scale[u] = *reinterpret_cast<const uint32_t*>(base + row + vs_lane);
      }
    }
  };
  // What a page holds behind the last token seen, or where there is no page, counts as zeros.  Blocks without
  // a value (scale byte 255) do too, so that the weight 0 of a row that doesn't see the token meets no NaN;
  // true if there are any: bit 8 r + 7 of none[u] is set if one of key r's is.
  auto clear_v = [&](int t, int pa, int pb, RawV<D>& v, uint32_t (&none)[2]) {
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
      none[u] = v.scale[u] & ((v.scale[u] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    }
    if (__ballot((none[0] | none[1]) != 0u) == 0) return false;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t mask = ~((none[u] >> 7) * 255u);
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        v.w[g][u] &= mask;
        v.w[g][2 + u] &= mask;
      }
      v.scale[u] = (v.scale[u] & mask) | (0x7F7F7F7Fu & ~mask);
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) none[u] |= (uint32_t)__shfl_xor((int)none[u], off, 64);
    }
    return true;
  };
  // f32: operands of a 16-key block: lane (n, quad), operand s: elements quad D / 4 + 4 s ..
  auto k_operands = [&](const auto& r, auto (&k)[kSteps]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const float f = scale_of(r.scale[D == 256 ? s / 8 : 0] >> (8 * (n & 3)) & 255u);
      const uint32_t w = r.w[s / 2];
      const f32x2 x = s & 1 ? pair_f32<2>(w, f) : pair_f32<0>(w, f);
      const f32x2 y = s & 1 ? pair_f32<3>(w, f) : pair_f32<1>(w, f);
      k[s] = f32x4{x[0], x[1], y[0], y[1]};
    }
  };
  // operands d and d + 1 (d = 4 g + 2 h): elements n D / 16 + d, .. + 1 of the lane's keys
  auto v_operands = [&](const RawV<D>& r, const float (&s)[8], int g, int h, Chunk (&lo)[kVC],
                        Chunk (&hi)[kVC]) {
    const uint32_t x = r.w[g][2 * h], y = r.w[g][2 * h + 1];
    if constexpr (!kF32) {
      const uint32_t p[8] = {pair_bf16<0>(x, s[0]), pair_bf16<1>(x, s[1]), pair_bf16<2>(x, s[2]),
                             pair_bf16<3>(x, s[3]), pair_bf16<0>(y, s[4]), pair_bf16<1>(y, s[5]),
                             pair_bf16<2>(y, s[6]), pair_bf16<3>(y, s[7])};
      u32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
        b[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
      }
      lo[0] = __builtin_bit_cast(Chunk, a);
      hi[0] = __builtin_bit_cast(Chunk, b);
    } else {
      const f32x2 p[8] = {pair_f32<0>(x, s[0]), pair_f32<1>(x, s[1]), pair_f32<2>(x, s[2]),
                          pair_f32<3>(x, s[3]), pair_f32<0>(y, s[4]), pair_f32<1>(y, s[5]),
                          pair_f32<2>(y, s[6]), pair_f32<3>(y, s[7])};
#pragma unroll
      for (int u = 0; u < kVC; ++u) {
        const f32x2* const z = p + 4 * u;
        lo[u] = __builtin_bit_cast(Chunk, f32x4{z[0][0], z[1][0], z[2][0], z[3][0]});
        hi[u] = __builtin_bit_cast(Chunk, f32x4{z[0][1], z[1][1], z[2][1], z[3][1]});
      }
    }
  };

  // The next step's codes are on their way from where this step's are used last (two steps ahead takes
  // registers and gains nothing: 3 % behind for 48 and 96 rows).  They are started without a condition (behind
  // the end the last step's again), so that the number on their way is known where one is waited for.
  RawK<D> k[2];
  RawV<D> v;
  int pa, pb;
  if (t0 < t1) {
    pages_of(t0, pa, pb);
    load_k(t0, pa, pb, k);
    load_v(t0, pa, pb, v);
  }
#pragma unroll
  for (int x = 0; x < kMine; ++x)
    if (x * KW + part < NQ)
      rows_of[x].put(quad, a.scale_log2, mine + (x * KW + part) * Query::kPieces * 64,
                     &sh_scale[((wave % RW) * NQ + x * KW + part) * 64 + lane]);
  __syncthreads();
  uint32_t q_scale[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) q_scale[i] = kF32 ? 0u : sh_scale[((wave % RW) * NQ + i) * 64 + lane];
  int limit = 255;  // of the wave's rows
#pragma unroll
  for (int i = 0; i < NQ; ++i)
    if constexpr (!kF32) limit = min(limit, __builtin_amdgcn_readfirstlane((int)(q_scale[i] >> 24)));
  wait_loads();
  f32x4 s[NQ][2];
  Chunk p[NQ][kVC];
  float sums[NQ];
  bool far = false;  // some row's maximum lies far from zero
  // A step's weights p and their sums against the maxima as they are; true if a sum shows
  // that some score lies far above its row's maximum.
  auto weights_of = [&](auto exponent) {
    bool risen = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float e[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) e[r] = __builtin_amdgcn_exp2f(exponent(s[i][r >> 2][r & 3], m[i]));
      sums[i] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      risen |= sums[i] > kRiseSum;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if constexpr (!kF32) p[i][0][r] = (__bf16)e[r];
        else p[i][r >> 2][r & 3] = e[r];
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
  // Accumulators stay where the matrix instructions have them outside the rare rescaling: the
  // compiler would otherwise copy them to the other register file before every step's branch.
  auto settle = [&]() {
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        if constexpr (NQ > 3) asm volatile("" : "+a"(o[i][d]));
        else asm volatile("" : "+v"(o[i][d]));
      }
  };
  // The maxima brought up to a step's scores, and the sums so far scaled down.
  auto follow = [&]() {
    far = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const float mx = fmaxf(fmaxf(fmaxf(s[i][0][0], s[i][0][1]), fmaxf(s[i][0][2], s[i][0][3])),
                             fmaxf(fmaxf(s[i][1][0], s[i][1][1]), fmaxf(s[i][1][2], s[i][1][3]))) *
                       a.scale_log2;
      float mn = fmaxf(m[i], mx);
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
  // bf16: a step's scores from bf16 operands: the keys' codes converted, the queries as they are in memory.
  // An operand takes 8 elements of a lane's block.
  auto exact_scores = [&]() {
    constexpr int kOps = D == 64 ? 2 : D / 32;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int row = row0 + wrow + 16 * i + n, token = row < rows ? row / G : 0;
      const int h = it.head * G + (row < rows ? row - token * G : 0);
      const E* from = q + ((int64_t)(it.w.o0 + token) * a.heads + h) * D;
#pragma unroll
      for (int u = 0; u < 2; ++u) s[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kOps; ++c) {
        const int b = c / 4;
        const u32x4 x = *reinterpret_cast<const u32x4*>(
            from + (D == 64 ? 32 * (quad & 1) + 16 * (quad >> 1) + 8 * c : 128 * b + 32 * quad + 8 * (c & 3)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t byte = k[u].scale[b] >> (8 * (n & 3)) & 255u;
          const float f = byte == 255u ? NAN : scale_of(byte);
          const uint32_t w = D == 64 ? (quad < 2 ? k[u].w[c & 1] : k[u].w[2 + (c & 1)]) : k[u].w[c];
          const u32x4 y = {pair_bf16<0>(w, f), pair_bf16<1>(w, f), pair_bf16<2>(w, f), pair_bf16<3>(w, f)};
          if constexpr (!kF32)
            s[i][u] = Op::score(__builtin_bit_cast(Chunk, y), __builtin_bit_cast(Chunk, x), s[i][u]);
        }
      }
    }
  };
  for (int t = t0; t < t1; ++t) {
    const int ahead = min(t + 1, t1 - 1);
    const int ma = pa, mb = pb;
    const bool partial = (t + 1) * kKeys > common || ma < 0 || mb < 0;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    matrix_first();
    if constexpr (kF32) {
      Chunk ko[2][kSteps];
      k_operands(k[0], ko[0]);
      k_operands(k[1], ko[1]);
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          const Chunk x = __builtin_bit_cast(Chunk, mine[(i * Query::kPieces + c) * 64]);
#pragma unroll
          for (int u = 0; u < 2; ++u) s[i][u] = Op::score(ko[u][c], x, s[i][u]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int c = 0; c < kQueryOps<D>; ++c) {
          const int b = D == 256 ? c / 2 : 0;
          const u32x4 x = mine[(i * Query::kPieces + 2 * c) * 64];
          const u32x4 y = mine[(i * Query::kPieces + 2 * c + 1) * 64];
          const i32x8 qo = {(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                            (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t* w = k[u].w + 4 * b;
            const i32x8 ko = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
            const int ks = (int)(k[u].scale[b] >> (8 * (n & 3)));  // its low byte counts
            const int qs = (int)q_scale[i];
            if (D != 64 && (c & 1))
              s[i][u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ko, qo, s[i][u], 4, 0, 0, ks, 1, qs);
            else
              s[i][u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ko, qo, s[i][u], 4, 0, 0, ks, 0, qs);
          }
        }
    }
    matrix_done();
    if constexpr (!kF32) {
      if (limit < 255) {
        uint32_t top[2] = {0u, 0u};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int b = 0; b < (D + 127) / 128; ++b) top[u] = max(top[u], k[u].scale[b] >> (8 * (n & 3)) & 255u);
        if (__builtin_expect(__ballot((int)max(top[0], top[1]) > limit) != 0, 0)) {
          // what no token was written to has no say
          bool large = false;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = Op::key_of(u, n);
            large |= (int)top[u] > limit && key < seen - t * kKeys && (key < 16 ? ma : mb) >= 0;
          }
          if (__ballot(large) != 0) exact_scores();
        }
      }
    }
    pages_of(ahead, pa, pb);
    load_k(ahead, pa, pb, k);
    if (__builtin_expect(partial, 0)) {
      asm volatile("");  // a branch, not selections in every step
      uint32_t none[2];
      if (clear_v(t, ma, mb, v, none)) {
        // rows that see the token are NaN by its score
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              s[i][u][r] = none[u] >> (8 * r + 7) & 1u ? NAN : s[i][u][r];
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        // of this step's keys
        const int left = sh_limit[wrow + 16 * i + n] - t * kKeys;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = Op::skey_of(u, r, quad);
            const bool there = key < left && (key < 16 ? ma : mb) >= 0;
            s[i][u][r] = there ? s[i][u][r] : -INFINITY;
          }
      }
    }
    // The maxima move at the first step, and when a lane's weights show that a score is far
    // above all before it; otherwise they stay behind (the sums are far from binary32's end), and
    // a step needs neither a maximum over its scores nor a rescaling.
    if (__builtin_expect(weights() | far, 0)) {
      settle();
      follow();
      settle();
      if (far) far_weights();
      else weights();
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) l[i] += sums[i];
    matrix_first();
    float vs[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) vs[r] = scale_of(v.scale[r >> 2] >> (8 * (r & 3)) & 255u);
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Chunk lo[kVC], hi[kVC];
        v_operands(v, vs, g, h, lo, hi);
#pragma unroll
        for (int u = 0; u < kVC; ++u)
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            o[i][4 * g + 2 * h] = Op::score(lo[u], p[i][u], o[i][4 * g + 2 * h]);
            o[i][4 * g + 2 * h + 1] = Op::score(hi[u], p[i][u], o[i][4 * g + 2 * h + 1]);
          }
      }
    matrix_done();
    load_v(ahead, pa, pb, v);
  }

  // ---- the sums of the key parts joined: the other parts leave theirs in LDS in the
  // registers' order, the first part's waves add them and write the rows ----
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    l[i] += __shfl_xor(l[i], 16, 64);
    l[i] += __shfl_xor(l[i], 32, 64);
  }
  // Row block i belongs to part i % KW, which adds what the others have of it.
  f32x4* const sh_o = reinterpret_cast<f32x4*>(sh);
  // place of part w's piece of block i, left out where it is the owner's own
  auto piece = [&](int w, int i, int d) {
    const int rank = w < i % KW ? w : w - 1;
    return ((((wave % RW) * NQ + i) * (KW - 1) + rank) * kDT + d) * 64 + lane;
  };
  if constexpr (KW > 1) {
    __syncthreads();  // all parts are done with the queries
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if (quad == 0) {
        sh_ml[(part * kRows + wrow + 16 * i + n) * 2] = m[i];
        sh_ml[(part * kRows + wrow + 16 * i + n) * 2 + 1] = l[i];
      }
      if (i % KW == part) continue;
#pragma unroll
      for (int d = 0; d < kDT; ++d) sh_o[piece(part, i, d)] = o[i][d];
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    if (i % KW != part) continue;
    float f[KW], mn = m[i];
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      f[w] = KW > 1 ? sh_ml[(w * kRows + wrow + 16 * i + n) * 2] : m[i];
      mn = fmaxf(mn, f[w]);
    }
    float ls = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      f[w] = __builtin_amdgcn_exp2f(f[w] - mn);
      ls += (KW > 1 ? sh_ml[(w * kRows + wrow + 16 * i + n) * 2 + 1] : l[i]) * f[w];
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
      sum[d] = o[i][d] * f[i % KW];
#pragma unroll
      for (int w = 0; w < KW; ++w)
        if (w != i % KW) sum[d] += sh_o[piece(w, i, d)] * f[w];
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
  static constexpr int waves = NQ > 3 ? 1 : ((sizeof(E) == 2 && D <= 128) || RW * KW == 8 ? 2 : 1);
};

// The line of work (attend_common.h), or, where it has few groups, their pieces one after the other
// (attend_plan.h, plan_target): before[] and spans then count pieces.
struct Plan4 : Plan {
  int target;  // units of a piece, 0: the line is cut into spans
  int64_t totals[kPlanWaves][2];
  int near[kPlanThreads][3];  // a slot's token rows and length, if there are no more slots
};

__device__ __forceinline__ int charge_of(const AttendArgs& a) {
  return plan_charge((int64_t)a.c.slots * a.c.kv_heads, a.grid);
}

__device__ __forceinline__ SlotWork near_work(const AttendArgs& a, const Plan4& plan, int s, int rows) {
  const auto uniform = [&](int i) { return __builtin_amdgcn_readfirstlane(plan.near[s][i]); };
  return plan_slot(uniform(0), uniform(1), uniform(2), (int64_t)a.c.max_pages << a.c.page_shift, a.group,
                   rows, a.c.kv_heads, charge_of(a));
}

template <int kThreads>
__device__ __forceinline__ void make_plan4(const AttendArgs& a, int rows, Plan4& plan) {
  static_assert(kThreads >= kPlanThreads, "a thread for each run of slots");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.c.slots + kPlanThreads - 1) / kPlanThreads;
  const int s0 = tid < kPlanThreads ? tid * per : a.c.slots, s1 = min(s0 + per, a.c.slots);
  const bool few = plan_few((int64_t)a.c.slots * a.c.kv_heads, a.grid);  // as far as slots tell
  int64_t x = 0, groups = 0, steps = 0;
  int long_chunk = 0, mine = 0;
  for (int s = s0; s < s1; ++s) {
    const SlotWork w = slot_work(a, s, rows, charge_of(a));
    x += w.units;
    if (per == 1) {
      plan.near[s][0] = w.o0;
      plan.near[s][1] = w.o0 + w.chunk;
      plan.near[s][2] = a.c.t.lens[s];
    }
    if (few && w.tiles > 0) {
      mine = tile_units(w, a.group, rows, 0);
      steps += (int64_t)mine * a.c.kv_heads;
      groups += a.c.kv_heads;
      long_chunk |= w.tiles > 1;
    }
  }
  if (tid == 0) {
    plan.before[0] = 0;
    plan.per = per;
    plan.target = 0;
  }
  int target[kTargets];
  bool whole = false;
  if (few) {  // (then there are no more slots than threads)
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      steps += __shfl_xor(steps, off, 64);
      groups += __shfl_xor(groups, off, 64);
    }
    if (lane == 0 && wave < kPlanWaves) {
      plan.totals[wave][0] = steps;
      plan.totals[wave][1] = groups;
    }
    whole = !__syncthreads_or(long_chunk);
    steps = groups = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      steps += plan.totals[w][0];
      groups += plan.totals[w][1];
    }
    whole = whole && groups > 0;
    if (whole) {
      plan_targets(steps, (int)groups, a.grid, target);
      x = plan_packed(mine, target, a.c.kv_heads);
    }
  }
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
  if (whole) {
    int units;
    const int best = plan_choice(total, a.grid, target, units);
    x = plan_unpacked(x, best);
    total = plan_unpacked(total, best);
    if (tid == 0) plan.target = units;
  }
  if (tid < kPlanThreads) plan.before[tid + 1] = x;
  if (tid == 0) {
    const int64_t span = plan.target ? 1 : plan_span(total, a.grid);
    plan.span = span;
    plan.spans = (int)((total + span - 1) / span);
  }
  __syncthreads();
}

// The group of piece x of the batch: its slot is the run of slots that x lies in.  j, n: which piece of how
// many.
__device__ __forceinline__ void find_piece(const AttendArgs& a, int rows, const Plan4& plan, int x,
                                           Group& g, int& j, int& n) {
  const int s = plan_run(plan.before, kPlanThreads, x);
  g.w = near_work(a, plan, s, rows);
  g.slot = s;
  g.tile = 0;
  g.units = tile_units(g.w, a.group, rows, 0);
  const PlanPiece p = plan_piece(g.units, plan.target, x - (int)plan.before[s]);
  g.head = p.head;
  j = p.j;
  n = p.n;
}

template <typename E, int D, int NQ, int RW, int KW, bool kHalf>
__global__ __launch_bounds__(64 * RW * KW, (Shape4<E, D, NQ, RW, KW>::waves)) void k_attend4(AttendArgs a) {
  constexpr int kRows = 16 * NQ * RW;
  __shared__ Plan4 plan;
  __shared__ float sh_ml[KW * kRows * 2];
  __shared__ int sh_limit[kRows];
  __shared__ uint32_t sh_scale[NQ * RW * 64];
  __shared__ u32x4 sh[lds_pieces<E, D, NQ, RW, KW>()];
  make_plan4<64 * RW * KW>(a, kRows, plan);
  const int64_t total = plan.before[kPlanThreads];
  // Workgroup ids go to the 8 XCDs in turn; each XCD takes a contiguous run of
  // spans, so that row tiles that read the same keys share its L2.
  if (blockIdx.x == 0 && threadIdx.x == 0) a.cuts[0].first = plan.spans;
  const int per_xcd = (plan.spans + 7) >> 3;
  const int idx = (int)(blockIdx.x >> 3), span = (int)(blockIdx.x & 7) * per_xcd + idx;
  if (idx >= per_xcd || span >= plan.spans) return;
  const bool pieces = plan.target > 0;
  const int64_t x0 = span * plan.span, x1 = min(x0 + plan.span, total);
  Group g;
  g.slot_end = 0;
  AttendCut cut = {};
  for (int64_t x = x0; x < x1;) {
    int first, end;
    int64_t rec;  // a cut group's record: a span has two at most, of its first and of its last group
    bool goes_on;
    int last;
    if (pieces) {
      int j, n;
      find_piece(a, kRows, plan, span, g, j, n);
      first = piece_start(g.units, j, n);
      end = piece_start(g.units, j + 1, n);
      rec = n == 1 ? -1 : 2 * (int64_t)span;
      goes_on = j == 0 && n > 1;
      last = span + n - 1;
      x = x1;
    } else {
      const auto work_of = [&](int s) {
        return plan.per == 1 ? near_work(a, plan, s, kRows) : slot_work(a, s, kRows, charge_of(a));
      };
      find_group(a, kRows, plan, x, g, work_of, charge_of(a), true);
      if (g.units == 0) {
        x = g.next;
        continue;
      }
      // a span may start, or end, in front of the group's first step
      first = (int)max(x - g.start, (int64_t)0);
      end = (int)min((int64_t)g.units, x1 - g.start);
      if (end <= first) break;
      rec = first == 0 && end == g.units ? -1 : 2 * (int64_t)span + (x != x0);
      goes_on = first == 0 && end < g.units;
      last = goes_on ? (int)((g.start + g.units - 1) / plan.span) : 0;
      x = g.start + end;
    }
    if (goes_on) {
      cut.row0 = g.tile * kRows;
      cut.rows = min(kRows, g.w.chunk * a.group - cut.row0);
      cut.token0 = g.w.o0;
      cut.head = g.head;
      cut.first = (int)rec;
      cut.last = last;
    }
    attend4_steps<E, D, NQ, RW, KW, kHalf>(a, g, first, end, rec, sh_ml, sh_limit, sh_scale, sh);
  }
  if (threadIdx.x == 0) a.cuts[1 + span] = cut;
}

// The join of cut groups (k_attend_join) for tiles of 16 rows, whose groups are few and may go through
// hundreds of spans: a workgroup takes all rows of a group, 1024 / (8 D / 4) of them at once, and its pieces by
// eights, so that their loads do not follow each other (8 groups of 64 pieces: 15 us by
// k_attend_join, 5 so).
template <typename E, int D>
__global__ __launch_bounds__(1024) void k_attend4_join(AttendArgs a, int rows_per_tile) {
  constexpr int kCols = D / 4, kLanes = 8, kAtOnce = 1024 / (kCols * kLanes);
  __shared__ float sh_m[kAtOnce][kLanes], sh_l[kAtOnce][kLanes];
  __shared__ f32x4 sh_o[kLanes][kAtOnce][kCols];
  const int k = (int)blockIdx.x;
  if (k >= a.cuts[0].first) return;
  const AttendCut cut = a.cuts[1 + k];
  if (cut.rows == 0) return;
  const int c = (int)threadIdx.x % kCols, at = (int)threadIdx.x / kCols % kAtOnce;
  const int j = (int)threadIdx.x / (kCols * kAtOnce);
  for (int r0 = 0; r0 < cut.rows; r0 += kAtOnce) {
    const int r = r0 + at;
    const bool live = r < cut.rows;
    const auto record = [&](int p) {
      return (p == k ? (int64_t)cut.first : 2 * (int64_t)p) * rows_per_tile + r;
    };
    float m = kNone;
    if (live) {
#pragma unroll 8
      for (int p = k + j; p <= cut.last; p += kLanes) m = fmaxf(m, a.part_ml[record(p) * 2]);
    }
    __syncthreads();  // the last rows are out of LDS
    if (c == 0) sh_m[at][j] = m;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kLanes; ++x) m = fmaxf(m, sh_m[at][x]);
    float l = 0.f;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (live) {
#pragma unroll 8
      for (int p = k + j; p <= cut.last; p += kLanes) {
        const int64_t o = record(p);
        const float f = __builtin_amdgcn_exp2f(a.part_ml[o * 2] - m);
        l += a.part_ml[o * 2 + 1] * f;
        sum += *reinterpret_cast<const f32x4*>(a.part_o + o * D + 4 * c) * f;
      }
    }
    if (c == 0) sh_l[at][j] = l;
    sh_o[j][at][c] = sum;
    __syncthreads();
    if (j > 0 || !live) continue;
    l = 0.f;
    sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < kLanes; ++x) {
      l += sh_l[at][x];
      sum += sh_o[x][at][c];
    }
    const int G = a.group, token = (cut.row0 + r) / G;
    E* to = static_cast<E*>(a.out) +
            ((int64_t)(cut.token0 + token) * a.heads + cut.head * G + (cut.row0 + r - token * G)) * D + 4 * c;
    store4<E>(to, sum * (l > 0.f ? 1.f / l : 0.f));
  }
}

template <typename E>
void start4_join(int rows, const AttendArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.grid), block(1024);
  switch (a.c.head_dim) {
    case 64: hipLaunchKernelGGL((k_attend4_join<E, 64>), grid, block, 0, stream, a, rows); break;
    case 128: hipLaunchKernelGGL((k_attend4_join<E, 128>), grid, block, 0, stream, a, rows); break;
    default: hipLaunchKernelGGL((k_attend4_join<E, 256>), grid, block, 0, stream, a, rows); break;
  }
}

template <typename E, int D, int NQ, int RW, int KW>
void start4(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid(a.grid), block(64 * RW * KW);
  if (a.c.page_shift == 4) hipLaunchKernelGGL((k_attend4<E, D, NQ, RW, KW, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_attend4<E, D, NQ, RW, KW, false>), grid, block, 0, stream, a);
}

// Tiles in use: rows (16 NQ RW), NQ, RW, KW.
#define ATTEND4_TILES(X) X(16, 1, 1, 4) X(32, 2, 1, 4) X(48, 3, 1, 4) X(64, 2, 2, 2) X(96, 3, 2, 2) \
  X(128, 2, 4, 2) X(192, 3, 4, 2) X(256, 2, 8, 1) X(384, 3, 8, 1)
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

// Workgroups, and spans at most: what is resident at once, two waves per SIMD.  Tiles of 16 rows could have
// four, but their groups are then cut into more pieces (256 slots, one token: 1024 workgroups 170
// us, 512 140, 256 184).
int attend4_grid(int head_dim, int rows) {
  return head_dim <= 128 && rows <= 96 ? 512 : 256;
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
    if (rows == 16 && bf16)
      start4_join<uint16_t>(rows, a, stream);
    else if (rows == 16)
      start4_join<float>(rows, a, stream);
    else if (bf16)
      hipLaunchKernelGGL(k_attend_join<uint16_t>, join, dim3(kPlanThreads), 0, stream, a, rows);
    else
      hipLaunchKernelGGL(k_attend_join<float>, join, dim3(kPlanThreads), 0, stream, a, rows);
  }
  return hipGetLastError();
}

}  // namespace dspark
