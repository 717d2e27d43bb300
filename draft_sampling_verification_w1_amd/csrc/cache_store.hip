// cache_store.hip -- a chunk's keys and values into the pages with the position rotation
// and the conversion to 4 bits on the way, and tokens out of the pages again.
//
// Rotation.  A token at position p turns the pair (a, b) of its key (and of its queries) by
// the angle p f_j, f_j in radians per position:
//   a' = a c - b s,  b' = b c + a s,   c = cos(p f_j), s = sin(p f_j).
// The angle is a binary64 product (p f_j loses everything in binary32 from some 10^5
// positions on); it is reduced by the nearest multiple of pi / 2 (two parts of pi / 2, one
// fma each, exact to 2^-53 or so) and the sine and cosine are their Taylor series on
// [-pi/4, pi/4] (to r^15 and r^16: off by less than 2^-52), rounded to binary32 once.  A workgroup works
// them out for its 8 tokens and all heads use them from LDS: there is no table that ends at some
// longest position and none to read.  The pair's products and sums are rounded one by one
// in binary32 (no fma), so that the 4-bit codes follow from the plain definition bit for bit (but for a
// sine or cosine within 2^-52 of the middle between two binary32 numbers, one in some 10^8).
//
// 4 bits.  32 elements of a token share a power of two 2^e, an element is one of +-{0, 0.5, 1,
// 1.5, 2, 3, 4, 6} 2^e (E2M1 with E8M0 scales, the types of gfx950's conversions and matrix
// instructions).  e is the smallest with max |x| <= 7 * 2^e: what saturates at 6 is then off by
// at most 1, as what is rounded between 4 and 6 is.  The maximum is taken over the bits of
// |x|, whose order as whole numbers puts infinities and NaN above all numbers.
//
// Layout of a 4-bit page (one layer's K or V): the codes of all heads, then their scales.
//   K codes [head][D / 32][token][16 bytes]: a lane's 16 bytes are 32 elements of one key;
//   V codes [head][token / 8][D / 64][16][2][8 tokens]: a byte holds two neighbouring elements of one
//     token, its neighbours the same elements of the other seven; a lane's 16 bytes are 8
//     keys x 4 elements, from where the conversion builds the matrix operand of 8 keys;
//   scales [head][D / 32][token], so that 8 keys' scales are one 8-byte load.
//
// Work.  A workgroup of 8 waves takes an aligned group of 8 positions of a slot (what V stores
// side by side); blockIdx.y shares its heads out where there are few groups.  Each wave works out the angles
// of one token, then the waves take one head of V, K or the queries at a time (two of 64
// dimensions).  V: a lane holds two neighbouring elements of all 8 tokens, which is a
// transposition in registers, and a group that is not full is stored in as few pieces as its
// places make.  K and queries: a lane holds two 8-element pieces of one token that rotate with each
// other, the same ones for all heads, so that its angles stay in registers (read from LDS for each head, their
// bank conflicts took longer than the memory: 35 us against 26 for the chunk below); the next
// head's pieces are on their way while one is turned.
//
// Bound by memory.  Alone on the card: 256 chunks of 17 tokens, 32 heads on 8 of 128 dimensions in bf16,
// 107 MB: 23 us, 4.6 TB/s, on the same inputs again; 28 us where three calls' inputs take turns, 33 where
// six do, of which no cache holds any.  Two chunks of 2048 tokens into 4 bits 17 us, where 88 MB move; the same from
// binary32 42 us (171 MB).
// Small calls are latency: 7 us from one launch to the next, as a launch of two dependent loads takes.
#include "device_common.h"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kGroup = 8;  // positions of a group

__device__ __forceinline__ bool page_ok(const CacheArgs& a, int p) { return p >= 0 && p < a.pages; }

// A group of positions of a slot that some of the call's token rows have.
struct Place {
  int row;       // first token row of the group, -1: there is none
  int n;         // its rows
  int e0;        // place of the first among the group's 8 positions
  int page;      // page id, -1: none
  int at;        // the group's first position in the page
  int64_t pos;   // position of the first row
};

// The workgroup's group (blockIdx.x).  Slot s's groups are numbered from
// offsets[s] / 8 + 3 s on, which leaves room for a group that is cut at either end.  Each thread
// looks at its slots' offsets and start position at once, so that finding the group is one round
// trip, its page another.
template <int kThreads>
__device__ __forceinline__ Place find_place(const CacheArgs& c, int N, const int32_t* offsets,
                                            const int32_t* starts) {
  __shared__ int found[6];
  const int w = blockIdx.x;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < c.slots; s += kThreads) {
    const int o0 = min(max(offsets[s], 0), N), o1 = min(max(offsets[s + 1], o0), N);
    const int start = starts[s], held = c.t.held[s];
    const int first = o0 / kGroup + 3 * s;
    if (o0 < o1 && first <= w && w < o1 / kGroup + 3 * (s + 1)) {
      found[0] = s;
      found[1] = o0;
      found[2] = o1;
      found[3] = w - first;
      found[4] = start;
      found[5] = held;
    }
  }
  __syncthreads();
  Place g = {-1, 0, 0, -1, 0, 0};
  const int s = found[0], o0 = found[1], o1 = found[2], start = found[4];
  if (s < 0) return g;
  const int64_t base = max(start, 0);
  const int64_t first = (base / kGroup + found[3]) * kGroup;  // of the group
  g.e0 = first < base ? (int)(base - first) : 0;
  g.pos = first + g.e0;
  const int64_t row = o0 + (g.pos - base);
  if (row >= o1) return g;
  g.row = (int)row;
  g.n = (int)min((int64_t)(kGroup - g.e0), o1 - row);
  const int64_t j = g.pos >> c.page_shift;
  if (start >= 0 && j < min(found[5], c.max_pages)) {
    const int p = c.t.table[(int64_t)s * c.max_pages + j];
    if (page_ok(c, p)) g.page = p;
  }
  g.at = (int)(first & ((1 << c.page_shift) - 1));
  return g;
}

// 8 elements as they lie in memory, and in binary32.
template <typename E>
struct Eight {
  u32x4 w[sizeof(E) / 2];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(E) / 2; ++h) w[h] = reinterpret_cast<const u32x4*>(p)[h];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2) {
        x[2 * i] = bf16_lo(w[0][i]);
        x[2 * i + 1] = bf16_hi(w[0][i]);
      } else {
        x[i] = __uint_as_float(w[0][i]);
        x[4 + i] = __uint_as_float(w[1][i]);
      }
    }
  }
};
// 8 elements rounded to nearest even.  kPast: past the caches, for rows that are written whole by 16-byte
// stores (queries of 256 chunks of 17 tokens, 35 MB: 33 us against 36; the attention behind reads them as
// fast).  Binary32 takes two stores that the caches put together.
template <bool kPast = false>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  bf16x8 b;
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (__bf16)x[i];
  if constexpr (kPast) __builtin_nontemporal_store(b, reinterpret_cast<bf16x8*>(p));
  else *reinterpret_cast<bf16x8*>(p) = b;
}
template <bool kPast = false>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    reinterpret_cast<f32x4*>(p)[h] = f32x4{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
}

// sin and cos of a binary64 angle (below 2^40 in magnitude), rounded to binary32.
__device__ __forceinline__ float2 cos_sin(double angle) {
  // the nearest whole number, left in the low bits of the sum
  const double sum = fma(angle, 0.63661977236758134, 6755399441055744.0);  // + 1.5 2^52
  const double k = sum - 6755399441055744.0;
  double r = fma(-k, 1.5707963267948966, angle);
  r = fma(-k, 6.123233995736766e-17, r);
  const double z = r * r;
  double s = -7.6471637318198164e-13;  // -1 / 15!
  s = fma(s, z, 1.6059043836821613e-10);
  s = fma(s, z, -2.5052108385441720e-08);
  s = fma(s, z, 2.7557319223985893e-06);
  s = fma(s, z, -1.9841269841269841e-04);
  s = fma(s, z, 8.3333333333333332e-03);
  s = fma(s, z, -1.6666666666666666e-01);
  s = fma(s, z * r, r);
  double c = 4.7794773323873853e-14;  // 1 / 16!
  c = fma(c, z, -1.1470745597729725e-11);
  c = fma(c, z, 2.0876756987868100e-09);
  c = fma(c, z, -2.7557319223985888e-07);
  c = fma(c, z, 2.4801587301587302e-05);
  c = fma(c, z, -1.3888888888888889e-03);
  c = fma(c, z, 4.1666666666666664e-02);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const int q = (int)(__double_as_longlong(sum) & 3);
  const float fs = (float)s, fc = (float)c;
  const float a = (q & 1) ? fs : fc, b = (q & 1) ? fc : fs;
  return make_float2((q == 1 || q == 2) ? -a : a, (q & 2) ? -b : b);
}

// (a, b) turned; every operation rounded.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
#pragma clang fp contract(off)
  const float x = a * cs.x - b * cs.y;
  const float y = b * cs.x + a * cs.y;
  a = x;
  b = y;
}

// The scale byte of a block whose largest |x| has these bits: e + 127 within [7, 252], or
// 255 (every value is NaN) if one is infinite or NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int e = (int)(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x600000u);
  return top >= 0x7F800000u ? 255u : (uint32_t)min(max(e, 7), 252);
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int kSel>
__device__ __forceinline__ uint32_t code2(uint32_t old, float lo, float hi, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, lo, hi, scale, kSel);
}
__device__ __forceinline__ uint32_t code8(const float (&x)[8], float scale) {
  uint32_t w = code2<0>(0u, x[0], x[1], scale);
  w = code2<1>(w, x[2], x[3], scale);
  w = code2<2>(w, x[4], x[5], scale);
  return code2<3>(w, x[6], x[7], scale);
}

// Two neighbouring elements in binary32.
__device__ __forceinline__ float2 load2(const uint16_t* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// Byte of token 0 of the group's 8 in V's codes: elements 2 i and 2 i + 1.
template <int D>
__device__ __forceinline__ int v_code_at(int group, int i) {
  const int n = i / (D / 32), rest = i % (D / 32);
  return ((group * (D / 64) + rest / 2) * 16 + n) * 16 + (rest & 1) * 8;
}

// Head h of K: two 8-element pieces (c0, c1) of token t, turned.
template <typename E, int D, bool kPacked>
__device__ __forceinline__ void store_k(const StoreArgs& a, const Place& g, int h, int t, int c0,
                                        int c1, const float (&x)[8], const float (&y)[8], bool live,
                                        uint32_t* top) {
  const int page = 1 << a.c.page_shift, H = a.c.kv_heads;
  const int row = g.at + g.e0 + t;
  if constexpr (kPacked) {
    // the pieces' maxima meet in LDS: a block of 32 elements may be held by any lanes of the wave
    uint32_t mx = 0u, my = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mx = max(mx, magnitude(x[i]));
      my = max(my, magnitude(y[i]));
    }
    if (live) {
      top[c0] = mx;
      top[c1] = my;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (live && g.page >= 0) {
      uint8_t* blob = static_cast<uint8_t*>(a.K) + (int64_t)g.page * a.c.page_bytes;
      uint8_t* codes = blob + h * (page * (D / 2));
      uint8_t* scales = blob + H * page * (D / 2) + h * (page * (D / 32));
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c = p ? c1 : c0, b = c >> 2;
        const u32x4 m = *reinterpret_cast<const u32x4*>(top + 4 * b);
        const uint32_t byte = scale_byte(max(max(m.x, m.y), max(m.z, m.w)));
        const uint32_t code = byte == 255u ? 0u : code8(p ? y : x, scale_of(byte));
        *reinterpret_cast<uint32_t*>(codes + (b * page + row) * 16 + (c & 3) * 4) = code;
        if ((c & 3) == 0) scales[b * page + row] = (uint8_t)byte;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else if (live && g.page >= 0) {
    constexpr int kE = 16 / (int)sizeof(E);
    E* to = static_cast<E*>(a.K) + ((int64_t)g.page * H + h) * page * D;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int c = p ? c1 : c0;
      alignas(16) E piece[8];
      store8(piece, p ? y : x);
#pragma unroll
      for (int i = 0; i < 8 / kE; ++i)
        *reinterpret_cast<u32x4*>(to + ((int64_t)(c * (8 / kE) + i) * page + row) * kE) =
            *reinterpret_cast<const u32x4*>(piece + i * kE);
    }
  }
}

// Four neighbouring places of kBytes bytes each, those of `mask` stored in as few pieces as they make.
template <int kBytes>
__device__ __forceinline__ void put4(uint8_t* to, const uint32_t* w, uint32_t mask) {
  if (mask == 15u) {
    typedef uint32_t Four __attribute__((ext_vector_type(kBytes)));
    Four all;
#pragma unroll
    for (int i = 0; i < kBytes; ++i) {
      if constexpr (kBytes == 1) all = w[i];
      else all[i] = w[i];
    }
    *reinterpret_cast<Four*>(to) = all;
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t m = mask >> (2 * h) & 3u;
    if constexpr (kBytes == 4) {
      if (m == 3u) *reinterpret_cast<u32x2*>(to + 8 * h) = u32x2{w[2 * h], w[2 * h + 1]};
      else if (m) *reinterpret_cast<uint32_t*>(to + 8 * h + (m & 2u) * 2) = m == 1u ? w[2 * h] : w[2 * h + 1];
    } else if constexpr (kBytes == 2) {
      if (m == 3u) *reinterpret_cast<uint32_t*>(to + 4 * h) = w[h];
      else if (m) *reinterpret_cast<uint16_t*>(to + 4 * h + (m & 2u)) = (uint16_t)(m == 1u ? w[h] : w[h] >> 16);
    } else {
      const uint32_t x = w[0] >> (16 * h);
      if (m == 3u) *reinterpret_cast<uint16_t*>(to + 2 * h) = (uint16_t)x;
      else if (m) to[2 * h + (m >> 1)] = (uint8_t)(m == 1u ? x : x >> 8);
    }
  }
}
// The group's 8 places side by side (one or two bytes each).
template <int kBytes>
__device__ __forceinline__ void put8places(uint8_t* to, const uint32_t* w, uint32_t mask) {
  if (mask == 255u) {
    if constexpr (kBytes == 2) *reinterpret_cast<u32x4*>(to) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
    return;
  }
  put4<kBytes>(to, w, mask & 15u);
  put4<kBytes>(to + 4 * kBytes, w + kBytes, mask >> 4);
}

// Elements 2 i and 2 i + 1 of head h of V, all tokens of the group, by their places in it.
template <typename E, int D, bool kPacked>
__device__ __forceinline__ void store_v(const StoreArgs& a, const Place& g, int h, int i, bool live) {
  const int page = 1 << a.c.page_shift, H = a.c.kv_heads;
  const E* from = static_cast<const E*>(a.v) + ((int64_t)g.row * H + h) * D + 2 * i;
  const uint32_t mask = ((1u << g.n) - 1u) << g.e0;
  // places without a token hold a neighbour's
  const auto row = [&](int t) { return (int64_t)min(max(t - g.e0, 0), g.n - 1) * H * D; };
  if constexpr (kPacked) {
    float2 x[kGroup];
#pragma unroll
    for (int t = 0; t < kGroup; ++t) x[t] = live ? load2(from + row(t)) : make_float2(0.f, 0.f);
    uint32_t word[2] = {0u, 0u}, bytes[2] = {0u, 0u};
#pragma unroll
    for (int t = 0; t < kGroup; ++t) {
      const uint32_t byte = scale_byte(max_lanes16(max(magnitude(x[t].x), magnitude(x[t].y))));
      const float s = scale_of(byte);
      uint32_t& w = word[t >> 2];
      uint32_t old = w;
      if ((t & 3) == 0) w = code2<0>(w, x[t].x, x[t].y, s);
      if ((t & 3) == 1) w = code2<1>(w, x[t].x, x[t].y, s);
      if ((t & 3) == 2) w = code2<2>(w, x[t].x, x[t].y, s);
      if ((t & 3) == 3) w = code2<3>(w, x[t].x, x[t].y, s);
      if (byte == 255u) w = old;
      bytes[t >> 2] |= byte << (8 * (t & 3));
    }
    if (!live || g.page < 0) return;
    uint8_t* blob = static_cast<uint8_t*>(a.V) + (int64_t)g.page * a.c.page_bytes;
    put8places<1>(blob + h * (page * (D / 2)) + v_code_at<D>(g.at >> 3, i), word, mask);
    if ((i & 15) == 0)
      put8places<1>(blob + H * page * (D / 2) + h * (page * (D / 32)) + (i >> 4) * page + g.at, bytes, mask);
  } else {
    if (!live || g.page < 0) return;
    constexpr int kE = 16 / (int)sizeof(E);
    E* to = static_cast<E*>(a.V) + ((int64_t)g.page * H + h) * page * D;
    if constexpr (sizeof(E) == 2) {
      uint32_t x[kGroup], w[2][kGroup / 2];
#pragma unroll
      for (int t = 0; t < kGroup; ++t) x[t] = *reinterpret_cast<const uint32_t*>(from + row(t));
#pragma unroll
      for (int t = 0; t < kGroup / 2; ++t) {
        w[0][t] = x[2 * t] & 0xFFFFu | x[2 * t + 1] << 16;
        w[1][t] = x[2 * t] >> 16 | x[2 * t + 1] & 0xFFFF0000u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        put8places<2>(reinterpret_cast<uint8_t*>(to + ((int64_t)(g.at / kE) * D + 2 * i + e) * kE), w[e], mask);
    } else {
      u32x2 x[kGroup];
#pragma unroll
      for (int t = 0; t < kGroup; ++t) x[t] = *reinterpret_cast<const u32x2*>(from + row(t));
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int p = 0; p < kGroup / kE; ++p) {
          const uint32_t w[4] = {x[4 * p][e], x[4 * p + 1][e], x[4 * p + 2][e], x[4 * p + 3][e]};
          put4<4>(reinterpret_cast<uint8_t*>(to + ((int64_t)(g.at / kE + p) * D + 2 * i + e) * kE), w,
                  mask >> (4 * p) & 15u);
        }
    }
  }
}

constexpr int kStoreThreads = 64 * kGroup;  // a wave for each token's angles
// (registers: bf16 for three workgroups on a CU, 24.4 us against 27.4 for four with two chunks of 2048 tokens)

template <typename E, int D, bool kPacked>
__global__ __launch_bounds__(kStoreThreads, sizeof(E) == 2 ? 6 : 4) void k_cache_store(StoreArgs a) {
  constexpr int kUnits = D / 16;                           // lanes of a token of one head
  constexpr int kHeads = kUnits < 8 ? 8 / kUnits : 1;      // heads that a wave takes at once
  constexpr int kTurns = kUnits > 8 ? kUnits / 8 : 1;      // or rounds of the wave for a head
  __shared__ float2 cs[kGroup * (D / 2)];
  __shared__ __align__(16) uint32_t tops[kGroup][64 / kUnits * (D / 8)];
  const Place g = find_place<kStoreThreads>(a.c, a.N, a.offsets, a.c.t.lens);
  if (g.row < 0) return;
  const int half = a.rot / 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // The waves' rounds: first V's, which need no angles, then K's and the queries'.
  const int kv = (a.c.kv_heads + kHeads - 1) / kHeads * kTurns, qs = (a.heads + kHeads - 1) / kHeads * kTurns;
  const int stride = kGroup * (int)gridDim.y, rounds = 2 * kv + qs;
  int round = (int)blockIdx.y * kGroup + wave;
  int turned = round < kv ? round + (kv - round + stride - 1) / stride * stride : round;

  // A lane's two pieces (c0, c1) of token t of K's or a query's head.
  const int u = lane % kUnits;
  const bool turns = u < a.rot / 16, apart = !a.interleaved && turns;
  const int c0 = apart ? u : 2 * u, c1 = apart ? u + a.rot / 16 : 2 * u + 1;
  struct At {
    bool query, live;
    int h, t;
    int64_t at;
  };
  const auto place = [&](int round) {
    At p;
    p.query = round >= 2 * kv;
    const int x = (p.query ? round - 2 * kv : round - kv) % kTurns * 64 + lane;
    p.h = (p.query ? round - 2 * kv : round - kv) / kTurns * kHeads + (kHeads > 1 ? x / (8 * kUnits) : 0);
    p.t = x / kUnits % kGroup;
    const int H = p.query ? a.heads : a.c.kv_heads;
    p.live = p.h < H && p.t < g.n;
    p.at = ((int64_t)(g.row + p.t) * H + p.h) * D;
    return p;
  };
  Eight<E> next[2];
  const auto fetch = [&](int round) {
    const At p = place(round);
    if (!p.live) return;
    const E* from = static_cast<const E*>(p.query ? a.q : a.k) + p.at;
    next[0].load(from + 8 * c0);
    next[1].load(from + 8 * c1);
  };
  if (turned < rounds) fetch(turned);
  if (wave < g.n)
    for (int j = lane; j < half; j += 64) cs[wave * half + j] = cos_sin((double)(g.pos + wave) * a.freqs[j]);
  for (; round < kv; round += stride) {
    const int x = round % kTurns * 64 + lane;
    const int h = round / kTurns * kHeads + (kHeads > 1 ? x / (8 * kUnits) : 0);
    store_v<E, D, kPacked>(a, g, min(h, a.c.kv_heads - 1), kHeads > 1 ? x % (D / 2) : x, h < a.c.kv_heads);
  }
  __syncthreads();
  // a lane has the same pieces of the same token in all rounds: its angles stay in registers
  float2 w[8];
  {
    const int t = (turned % kTurns * 64 + lane) / kUnits % kGroup;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = turns && t < g.n ? cs[t * half + 8 * u + i] : make_float2(1.f, 0.f);
  }
  // a round's loads are under way while the one before is turned and stored
  for (; turned < rounds; turned += stride) {
    const At at = place(turned);
    float p[8], q[8];
    next[0].values(p);
    next[1].values(q);
    if (turned + stride < rounds) fetch(turned + stride);
    if (at.live && turns) {
      if (apart) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(p[i], q[i], w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          turn(p[2 * i], p[2 * i + 1], w[i]);
          turn(q[2 * i], q[2 * i + 1], w[4 + i]);
        }
      }
    }
    if (at.query) {
      if (at.live) {
        E* to = static_cast<E*>(a.q_out) + at.at;
        store8<true>(to + 8 * c0, p);
        store8<true>(to + 8 * c1, q);
      }
    } else {
      // lanes of one token of one head share D / 8 maxima
      store_k<E, D, kPacked>(a, g, at.h, at.t, c0, c1, p, q, at.live, tops[wave] + lane / kUnits * (D / 8));
    }
  }
}

// ---- tokens out of the pages -----------------------------------------------------------
template <int kSel>
__device__ __forceinline__ uint32_t two(uint16_t, uint32_t code, float s) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, kSel);
  return __builtin_bit_cast(uint32_t, b);
}
template <int kSel>
__device__ __forceinline__ u32x2 two(float, uint32_t code, float s) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, s, kSel);
  return __builtin_bit_cast(u32x2, b);
}
// kPairs pairs of elements, 16 bytes at a time where there are as many.  The rows are written once and are as a
// rule more than the caches hold: whole stretches of a wave's 16-byte stores pass the caches by (104 ->
// 84 us for 102,000 tokens of 8 x 2 x 128 in bf16).  Where a lane's elements take more stores than one, the
// caches have to put the lines together (binary32: 195 us against 364).
template <typename P, int kPairs>
__device__ __forceinline__ void put(void* to, const P (&x)[kPairs]) {
  constexpr int kBytes = kPairs * (int)sizeof(P);
  typedef uint32_t Word __attribute__((ext_vector_type(kBytes >= 16 ? 4 : 2)));
  union { P p[kPairs]; Word w[kBytes / (int)sizeof(Word)]; } all;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) all.p[i] = x[i];
#pragma unroll
  for (int i = 0; i < kBytes / (int)sizeof(Word); ++i) {
    if constexpr (kBytes <= 16) __builtin_nontemporal_store(all.w[i], static_cast<Word*>(to) + i);
    else static_cast<Word*>(to)[i] = all.w[i];
  }
}

// A block of values that are all NaN.
constexpr uint32_t kNoScale = 255u;
// Factors of 8 tokens' scale bytes.
__device__ __forceinline__ float factor(u32x2 bytes, int t) {
  const uint32_t b = bytes[t >> 2] >> (8 * (t & 3)) & 255u;
  return b == kNoScale ? NAN : scale_of(b);
}

// 4 x 4 words of four neighbouring lanes transposed: w[i] of lane j becomes w[j] of lane i.
__device__ __forceinline__ void transpose4(u32x4& w, int lane) {
  // first pairs of lanes, then pairs of pairs (quad_perm 1 0 3 2 and 2 3 0 1)
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t give = odd ? w[i] : w[i + 1];
    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0xB1, 0xF, 0xF, true);
    if (odd) w[i] = got;
    else w[i + 1] = got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t give = high ? w[i] : w[i + 2];
    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x4E, 0xF, 0xF, true);
    if (high) w[i] = got;
    else w[i + 2] = got;
  }
}

// What a wave reads of 8 positions: tokens t0 <= t < t1 of them have rows, the first of which is `row`;
// `at`: the first position's place in the page.
struct Part {
  int64_t row;
  int t0, t1, at, page;
};

// Heads h0 .. of K in 4 bits.  A lane's 8 elements of each token; four lanes' codes of a block of 32
// elements are loaded as 16 bytes of one token each and change places.
template <typename E, int D>
__device__ __forceinline__ void read_k4(const ReadArgs& a, const Part& g, int h0, int lane) {
  constexpr int kLanes = D / 8;  // of a head
  const int page = 1 << a.c.page_shift, H = a.c.kv_heads;
  const int c = lane % kLanes, h = h0 + lane / kLanes, hh = min(h, H - 1);
  const uint8_t* blob = static_cast<const uint8_t*>(a.K) + (int64_t)max(g.page, 0) * a.c.page_bytes;
  const uint8_t* codes = blob + hh * (page * (D / 2)) + ((c >> 2) * page + g.at + (c & 3)) * 16;
  u32x4 w[2] = {reinterpret_cast<const u32x4*>(codes)[0], reinterpret_cast<const u32x4*>(codes)[4]};
  u32x2 bytes = *reinterpret_cast<const u32x2*>(blob + H * page * (D / 2) + hh * (page * (D / 32)) +
                                                (c >> 2) * page + g.at);
  if (g.page < 0) {
    w[0] = w[1] = u32x4{0u, 0u, 0u, 0u};
    bytes = u32x2{0u, 0u};
  }
  transpose4(w[0], lane);
  transpose4(w[1], lane);
  if (h >= H) return;
  E* const out = static_cast<E*>(a.k) + ((g.row - g.t0) * H + h) * D + 8 * c;
#pragma unroll
  for (int t = 0; t < kGroup; ++t) {
    if (t < g.t0 || t >= g.t1) continue;
    const uint32_t code = w[t >> 2][t & 3];
    const float s = factor(bytes, t);
    const decltype(two<0>(E(), 0u, 0.f)) x[4] = {two<0>(E(), code, s), two<1>(E(), code, s),
                                                 two<2>(E(), code, s), two<3>(E(), code, s)};
    put(out + (int64_t)t * H * D, x);
  }
}

// Heads h0 .. h0 + 3 of V in 4 bits.  A lane's D / 16 neighbouring elements of all tokens.
template <typename E, int D>
__device__ __forceinline__ void read_v4(const ReadArgs& a, const Part& g, int h0, int lane) {
  constexpr int kRun = D / 16;  // elements
  const int page = 1 << a.c.page_shift, H = a.c.kv_heads;
  const int n = lane % 16, h = h0 + lane / 16, hh = min(h, H - 1);
  const uint8_t* blob = static_cast<const uint8_t*>(a.V) + (int64_t)max(g.page, 0) * a.c.page_bytes;
  const uint8_t* codes = blob + hh * (page * (D / 2)) + (g.at / kGroup * (D / 64) * 16 + n) * 16;
  u32x4 w[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) w[i] = reinterpret_cast<const u32x4*>(codes)[16 * i];
  u32x2 bytes = *reinterpret_cast<const u32x2*>(blob + H * page * (D / 2) + hh * (page * (D / 32)) +
                                                n * kRun / 32 * page + g.at);
  if (g.page < 0) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) w[i] = u32x4{0u, 0u, 0u, 0u};
    bytes = u32x2{0u, 0u};
  }
  if (h >= H) return;
  E* const out = static_cast<E*>(a.v) + ((g.row - g.t0) * H + h) * D + n * kRun;
#pragma unroll
  for (int t = 0; t < kGroup; ++t) {
    if (t < g.t0 || t >= g.t1) continue;
    const float s = factor(bytes, t);
    decltype(two<0>(E(), 0u, 0.f)) x[kRun / 2];
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t word = w[i][2 * e + (t >> 2)];
        auto& to = x[2 * i + e];
        if ((t & 3) == 0) to = two<0>(E(), word, s);
        if ((t & 3) == 1) to = two<1>(E(), word, s);
        if ((t & 3) == 2) to = two<2>(E(), word, s);
        if ((t & 3) == 3) to = two<3>(E(), word, s);
      }
    put(out + (int64_t)t * H * D, x);
  }
}

// A head of K, 8 elements of a token per lane and load.
template <typename E, int D>
__device__ __forceinline__ void read_k(const ReadArgs& a, const Part& g, int h, int lane) {
  constexpr int kE = 16 / (int)sizeof(E), kTurns = kGroup * (D / 8) / 64;
  const int page = 1 << a.c.page_shift, H = a.c.kv_heads;
  const E* from = static_cast<const E*>(a.K) + ((int64_t)max(g.page, 0) * H + h) * page * D;
  E* const out = static_cast<E*>(a.k) + ((g.row - g.t0) * H + h) * D;
  u32x4 w[kTurns][8 / kE];
#pragma unroll
  for (int r = 0; r < kTurns; ++r)
#pragma unroll
    for (int i = 0; i < 8 / kE; ++i) {
      const int x = 64 * r + lane, t = x / (D / 8), c = x % (D / 8);
      w[r][i] = *reinterpret_cast<const u32x4*>(from + ((int64_t)(c * (8 / kE) + i) * page + g.at + t) * kE);
    }
#pragma unroll
  for (int r = 0; r < kTurns; ++r) {
    const int x = 64 * r + lane, t = x / (D / 8), c = x % (D / 8);
    if (t < g.t0 || t >= g.t1) continue;
#pragma unroll
    for (int i = 0; i < 8 / kE; ++i)
      __builtin_nontemporal_store(g.page < 0 ? u32x4{0u, 0u, 0u, 0u} : w[r][i],
                                  reinterpret_cast<u32x4*>(out + (int64_t)t * H * D + 8 * c + i * kE));
  }
}

// A head of V: a lane takes two neighbouring elements of the tokens.
template <typename E, int D>
__device__ __forceinline__ void read_v(const ReadArgs& a, const Part& g, int h, int lane) {
  constexpr int kE = 16 / (int)sizeof(E);
  typedef E Pair __attribute__((ext_vector_type(2)));
  const int page = 1 << a.c.page_shift, H = a.c.kv_heads;
  const E* from = static_cast<const E*>(a.V) + ((int64_t)max(g.page, 0) * H + h) * page * D;
  E* const out = static_cast<E*>(a.v) + ((g.row - g.t0) * H + h) * D;
  for (int i = lane; i < D / 2; i += 64) {
    alignas(16) E x[2][kGroup];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int q = 0; q < kGroup / kE; ++q)
        *reinterpret_cast<u32x4*>(&x[e][q * kE]) =
            *reinterpret_cast<const u32x4*>(from + ((int64_t)(g.at / kE + q) * D + 2 * i + e) * kE);
#pragma unroll
    for (int t = 0; t < kGroup; ++t)
      if (t >= g.t0 && t < g.t1)
        __builtin_nontemporal_store(g.page < 0 ? Pair{(E)0, (E)0} : Pair{x[0][t], x[1][t]},
                                    reinterpret_cast<Pair*>(out + (int64_t)t * H * D + 2 * i));
  }
}

// A workgroup of 4 waves takes a group of 8 positions, whose place costs a round trip; two or four groups, so
// that more tokens share it, take longer where the states don't fit in the caches (97 -> 103 -> 109 us for
// 102,000 tokens).
template <typename E, int D, bool kPacked>
__global__ __launch_bounds__(256) void k_cache_read(ReadArgs a) {
  constexpr int kHeadsK = kPacked ? 512 / D : 1, kHeadsV = kPacked ? 4 : 1;  // that a wave takes at once
  const Place p = find_place<256>(a.c, a.N, a.offsets, a.first);
  if (p.row < 0) return;
  const Part g = {p.row, p.e0, p.e0 + p.n, p.at, p.page};
  const int H = a.c.kv_heads;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = (H + kHeadsK - 1) / kHeadsK, tasks = ks + (H + kHeadsV - 1) / kHeadsV;
  for (int task = (int)blockIdx.y * 4 + wave; task < tasks; task += 4 * (int)gridDim.y) {
    if (task < ks) {
      if constexpr (kPacked) read_k4<E, D>(a, g, task * kHeadsK, lane);
      else read_k<E, D>(a, g, task, lane);
    } else {
      if constexpr (kPacked) read_v4<E, D>(a, g, (task - ks) * kHeadsV, lane);
      else read_v<E, D>(a, g, task - ks, lane);
    }
  }
}

// Workgroups that share a group's heads: as many as the card holds (256 x 32 waves) without a second turn.
// Half and twice as many waves: 23.4 and 22.3 us against 23.4 (256 chunks of 17 tokens), 24.5 and 26.1
// against 24.5 (two chunks of 2048 tokens stored and read).
unsigned split_of(int groups, int tasks, int waves) {
  const int most = (tasks + waves - 1) / waves;
  const int want = 8192 / waves / groups;
  return (unsigned)(want < 1 ? 1 : (want < most ? want : most));
}

}  // namespace

hipError_t launch_cache_store(bool bf16, bool packed, const StoreArgs& a, hipStream_t stream) {
  TimingScope t("cache_store", stream);
  const int per = a.c.head_dim == 64 ? 2 : 1;
  const int rounds = 2 * ((a.c.kv_heads + per - 1) / per) + (a.heads + per - 1) / per;
  const int tasks = rounds * (a.c.head_dim == 256 ? 2 : 1);
  const int groups = a.N / kGroup + a.c.slots;
  const dim3 grid((unsigned)(a.N / kGroup + 3 * a.c.slots), split_of(groups, tasks, kGroup));
#define STORE(E, D, P) hipLaunchKernelGGL((k_cache_store<E, D, P>), grid, dim3(kStoreThreads), 0, stream, a)
#define STORE_DIMS(E, P)                       \
  switch (a.c.head_dim) {                      \
    case 64: STORE(E, 64, P); break;           \
    case 128: STORE(E, 128, P); break;         \
    default: STORE(E, 256, P); break;          \
  }
  if (bf16 && packed) {
    STORE_DIMS(uint16_t, true)
  } else if (bf16) {
    STORE_DIMS(uint16_t, false)
  } else if (packed) {
    STORE_DIMS(float, true)
  } else {
    STORE_DIMS(float, false)
  }
#undef STORE_DIMS
#undef STORE
  return hipGetLastError();
}

hipError_t launch_cache_read(bool bf16, bool packed, const ReadArgs& a, hipStream_t stream) {
  TimingScope t("cache_read", stream);
  const int groups = a.N / kGroup + a.c.slots;
  const int H = a.c.kv_heads;
  const int tasks = packed ? (H + 3) / 4 + (H * a.c.head_dim + 511) / 512 : 2 * H;
  const dim3 grid((unsigned)(a.N / kGroup + 3 * a.c.slots), split_of(groups, tasks, 4));
#define READ(E, D, P) hipLaunchKernelGGL((k_cache_read<E, D, P>), grid, dim3(256), 0, stream, a)
#define READ_DIMS(E, P)                       \
  switch (a.c.head_dim) {                     \
    case 64: READ(E, 64, P); break;           \
    case 128: READ(E, 128, P); break;         \
    default: READ(E, 256, P); break;          \
  }
  if (bf16 && packed) {
    READ_DIMS(uint16_t, true)
  } else if (bf16) {
    READ_DIMS(uint16_t, false)
  } else if (packed) {
    READ_DIMS(float, true)
  } else {
    READ_DIMS(float, false)
  }
#undef READ_DIMS
#undef READ
  return hipGetLastError();
}

}  // namespace dspark
