// cache.hip -- pages of a key/value cache: taking, sharing, releasing, moving and
// copying them, and writing a chunk's keys and values into them.
//
// A page holds page_size tokens of every layer.  The tables live on the device and
// every decision is taken there, from lengths that the host never sees (the
// accepted lengths of a round).  Pages are taken lowest index first: the state
// after a call depends on the calls alone, not on the order in which threads or
// atomics ran (reference counts and free bits only add up).  What is written at a
// page's place is the slot's own: a page that several slots share is copied before
// one of them writes to it (reserve names the pairs, copy_pages moves the bytes).
//
// Bookkeeping is bound by latency (one dependent memory round trip after the other):
// fork, reserve, free of 6 slots with 5 pages 4, 9 and 4 us, of 448 slots with up to 63
// pages 5, 11 and 8 us.  Copies are bound by HBM: 3,932 pages (32 KB each in K and
// V of 4 layers) 404 us, 5.1 TB/s like a large copy; the shared last pages of 448 forks of
// 64 parents 51 us, the sources from cache.
#include "device_common.h"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kBig = 1024;

__device__ __forceinline__ bool page_ok(const CacheArgs& a, int p) { return p >= 0 && p < a.pages; }

__global__ __launch_bounds__(256) void k_cache_init(CacheArgs a) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x < (int64_t)a.slots * a.max_pages) a.t.table[x] = -1;
  if (x < a.slots) {
    a.t.lens[x] = 0;
    a.t.held[x] = 0;
  }
  if (x < a.pages) a.t.refs[x] = 0;
  const int words = (a.pages + 31) / 32;
  if (x < words) {
    const int left = a.pages - (int)x * 32;
    a.t.free_bits[x] = left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u;
  }
  if (x == 0) a.t.n_free[0] = a.pages;
}

// Drops one reference of each of row's pages [from, upto) and clears the entries;
// `tid` of `n` threads.  Returns the number of pages that became free.
__device__ __forceinline__ int drop_pages(const CacheArgs& a, int32_t* row, int from, int upto,
                                          int tid, int n) {
  int freed = 0;
  for (int j = from + tid; j < upto; j += n) {
    const int p = row[j];
    row[j] = -1;
    if (!page_ok(a, p)) continue;
    if (atomicSub(&a.t.refs[p], 1) == 1) {
      atomicOr(&a.t.free_bits[p >> 5], 1u << (p & 31));
      ++freed;
    }
  }
  return freed;
}

// Sum over the workgroup's waves added to *dst by one thread per wave.
__device__ __forceinline__ void wave_add(int v, int32_t* dst) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0 && v) atomicAdd(dst, v);
}

// One workgroup per pair.  Shared are the pages that hold tokens: what src has reserved
// behind them it will write, and reserve looks for sharers in a slot's last page alone.
// A pair is refused (status 1) if an index is out of
// range, dst holds pages, an earlier pair names the same dst, or its src is any
// pair's dst: every accepted pair then reads only slots that no pair writes.
__global__ __launch_bounds__(256) void k_cache_fork(CacheArgs a, int n, const int32_t* src,
                                                    const int32_t* dst, int32_t* status) {
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  int bad = s < 0 || s >= a.slots || d < 0 || d >= a.slots;
  for (int j = threadIdx.x; j < n; j += 256) {
    const int dj = dst[j];
    bad |= (dj == d && j < i) || dj == s;
  }
  if (!bad && a.t.held[d] != 0) bad = 1;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) status[i] = bad ? 1 : 0;
  if (bad) return;
  const int len = a.t.lens[s];
  const int used = (int)(((int64_t)max(len, 0) + (1 << a.page_shift) - 1) >> a.page_shift);
  const int held = min(min(max(a.t.held[s], 0), a.max_pages), used);
  const int32_t* from = a.t.table + (int64_t)s * a.max_pages;
  int32_t* to = a.t.table + (int64_t)d * a.max_pages;
  for (int j = threadIdx.x; j < held; j += 256) {
    const int p = from[j];
    to[j] = p;
    if (page_ok(a, p)) atomicAdd(&a.t.refs[p], 1);
  }
  __syncthreads();  // every thread has read held[d] before it changes
  if (threadIdx.x == 0) {
    a.t.lens[d] = len;
    a.t.held[d] = held;
  }
}

// One workgroup per listed slot; a slot listed twice is released by its first entry.
__global__ __launch_bounds__(256) void k_cache_free(CacheArgs a, int n, const int32_t* slots) {
  const int i = blockIdx.x;
  const int s = slots[i];
  int skip = s < 0 || s >= a.slots;
  for (int j = threadIdx.x; j < i; j += 256) skip |= slots[j] == s;
  if (__syncthreads_or(skip)) return;
  const int held = min(max(a.t.held[s], 0), a.max_pages);
  const int freed = drop_pages(a, a.t.table + (int64_t)s * a.max_pages, 0, held, threadIdx.x, 256);
  wave_add(freed, a.t.n_free);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.t.lens[s] = 0;
    a.t.held[s] = 0;
  }
}

// One wave per slot: the new length, and the pages behind it released.
__global__ __launch_bounds__(64) void k_cache_commit(CacheArgs a, const int32_t* keep, int plus) {
  const int s = blockIdx.x;
  if (keep[s] == INT32_MIN) return;
  const int held = min(max(a.t.held[s], 0), a.max_pages);
  int64_t len = (int64_t)a.t.lens[s] + keep[s] + plus;
  const int64_t most = (int64_t)held << a.page_shift;
  len = len < 0 ? 0 : (len > most ? most : len);
  const int need = (int)((len + (1 << a.page_shift) - 1) >> a.page_shift);
  const int freed = drop_pages(a, a.t.table + (int64_t)s * a.max_pages, need, held, threadIdx.x, 64);
  wave_add(freed, a.t.n_free);
  if (threadIdx.x == 0) {
    a.t.lens[s] = (int)len;
    a.t.held[s] = need;
  }
}

// Exclusive prefix sum over the workgroup's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int part[kBig / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  __syncthreads();  // the previous scan's readers are done
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kBig / 64; ++w) {
    const int y = part[w];
    if (w < wave) before += y;
    all += y;
  }
  *total = all;
  return before + x - v;
}

// Index of the k-th set bit (k from 0) of a word that has more than k.
__device__ __forceinline__ int nth_bit(uint32_t w, int k) {
  int at = 0;
#pragma unroll
  for (int half = 16; half > 0; half >>= 1) {
    const int n = __popc((w >> at) & ((1u << half) - 1u));
    if (k >= n) {
      k -= n;
      at += half;
    }
  }
  return at;
}

// Place of page p among the `mask` + 1 keys, open addressing; a free place (-1) is
// taken with kTake.  There are at least as many places as slots: the search ends.
template <bool kTake>
__device__ __forceinline__ int page_place(int* keys, int mask, int p) {
  int h = (int)((uint32_t)p * 2654435761u >> 16) & mask;
  for (;;) {
    const int k = kTake ? atomicCAS(&keys[h], -1, p) : keys[h];
    if (k == p || k == -1) return h;
    h = (h + 1) & mask;
  }
}

// One workgroup.  Works out every slot's new pages and the shared page it has to
// copy, then takes the lowest free pages: page number `rank` of the call goes to
// the slot whose range of ranks holds it (both looked up by bisection, so that
// many pages for one slot go as fast as one page for many).
//
// If every slot that shares a page is about to write to it, one can keep it: the one
// with the most tokens in it (the lowest of several), which then writes behind what
// any of the others has there, also one that gets no page for its copy.  The writers
// of a page are counted in a hash table, by page: 448 slots that share 64 pages take
// 11 us less than with a search through the slots.
__global__ __launch_bounds__(kBig) void k_cache_reserve(CacheArgs a, const int32_t* add,
                                                        int32_t* status, int32_t* cow_src,
                                                        int32_t* cow_dst) {
  __shared__ int tail[kMaxCacheSlots];   // shared page that the slot would write to, or -1
  __shared__ int room[3 * kMaxCacheSlots];
  __shared__ int word_first[kBig];
  __shared__ uint32_t words[kBig];
  int* const first = room;                  // rank of the slot's first new page
  int* const info = room + kMaxCacheSlots;  // 2 * pages held before the call + (the slot copies a page)
  const int tid = threadIdx.x;
  const int page = 1 << a.page_shift;
  const int n_free = a.t.n_free[0];
  int found = 0;
  for (int s = tid; s < a.slots; s += kBig) {
    int t = -1;
    if (add[s] > 0) {
      const int len = a.t.lens[s], j = len >> a.page_shift;
      if (len > 0 && (len & (page - 1)) != 0 && j < min(a.t.held[s], a.max_pages)) {
        const int p = a.t.table[(int64_t)s * a.max_pages + j];
        if (page_ok(a, p) && a.t.refs[p] > 1) t = p;
      }
    }
    tail[s] = t;
    found |= t >= 0;
  }
  if (__syncthreads_or(found)) {
    const int places = a.slots > 1 ? 1 << (32 - __clz(a.slots - 1)) : 1;  // <= kMaxCacheSlots
    int* const keys = room;
    int* const writers = room + kMaxCacheSlots;
    int* const keeper = room + 2 * kMaxCacheSlots;  // largest (tokens in the page, -slot)
    for (int x = tid; x < places; x += kBig) {
      keys[x] = -1;
      writers[x] = 0;
      keeper[x] = 0;
    }
    __syncthreads();
    for (int s = tid; s < a.slots; s += kBig) {
      if (tail[s] < 0) continue;
      const int h = page_place<true>(keys, places - 1, tail[s]);
      atomicAdd(&writers[h], 1);
      atomicMax(&keeper[h], (a.t.lens[s] & (page - 1)) * kMaxCacheSlots + kMaxCacheSlots - 1 - s);
    }
    __syncthreads();
    for (int s = tid; s < a.slots; s += kBig) {
      const int p = tail[s];
      if (p < 0) continue;
      const int h = page_place<false>(keys, places - 1, p);
      if (writers[h] == a.t.refs[p] && (keeper[h] & (kMaxCacheSlots - 1)) == kMaxCacheSlots - 1 - s)
        tail[s] = -1;
    }
    __syncthreads();
  }
  int given = 0;  // pages given to the slots before this batch
  int wanted = 0;
  for (int base = 0; base < a.slots; base += kBig) {
    const int s = base + tid;
    int want = 0, cow = 0, held = 0, need = 0, st = 0;
    if (s < a.slots) {
      held = min(max(a.t.held[s], 0), a.max_pages);
      need = held;
      const int more = add[s];
      if (more > 0) {
        const int64_t upto = ((int64_t)a.t.lens[s] + more + page - 1) >> a.page_shift;
        if (upto > a.max_pages) st = 2;
        else need = max(held, (int)upto);
        cow = tail[s] >= 0;
        if (st == 0) want = need - held + cow;
      }
    }
    int total;
    const int upto = wanted + block_scan(want, &total) + want;
    wanted += total;
    if (st == 0 && want > 0 && upto > n_free) st = 1;
    const int got = st == 0 ? want : 0;
    // the slots that get pages are those before the first that does not fit
    int got_total;
    const int start = given + block_scan(got, &got_total);
    given += got_total;
    if (s < a.slots) {
      first[s] = start;
      status[s] = st;
      const int copy = st == 0 && cow;
      cow_src[s] = copy ? tail[s] : -1;
      cow_dst[s] = -1;
      info[s] = 2 * held + copy;
      if (st == 0) a.t.held[s] = need;
    }
  }
  __syncthreads();
  const int n_words = (a.pages + 31) / 32;
  int taken = 0;
  for (int base = 0; base < n_words && taken < given; base += kBig) {
    const int w = base + tid;
    const uint32_t bits = w < n_words ? a.t.free_bits[w] : 0u;
    int total;
    const int mine = block_scan(__popc(bits), &total);
    words[tid] = bits;
    word_first[tid] = mine;
    __syncthreads();
    const int here = min(total, given - taken);
    for (int k = tid; k < here; k += kBig) {
      int lo = 0, hi = kBig - 1;  // last word whose first rank is <= k: it holds the k-th bit
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (word_first[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      const int p = (base + lo) * 32 + nth_bit(words[lo], k - word_first[lo]);
      const int rank = taken + k;
      int s = 0, e = a.slots - 1;  // last slot whose first rank is <= rank
      while (s < e) {
        const int mid = (s + e + 1) >> 1;
        if (first[mid] <= rank) s = mid;
        else e = mid - 1;
      }
      const int held = info[s] >> 1, copy = info[s] & 1;
      const int off = rank - first[s] - copy;  // -1: the copy's place, else behind the held pages
      if (p < a.pages) {
        a.t.refs[p] = 1;
        const int at = off < 0 ? a.t.lens[s] >> a.page_shift : held + off;
        if (at < a.max_pages) a.t.table[(int64_t)s * a.max_pages + at] = p;
        if (off < 0) cow_dst[s] = p;
      }
    }
    // the word's lowest bits are gone
    const int left = min(max(given - taken - mine, 0), __popc(bits));
    if (left > 0) {
      uint32_t rest = bits;
      if (left == __popc(bits)) rest = 0u;
      else rest &= ~((1u << nth_bit(bits, left)) - 1u);
      a.t.free_bits[w] = rest;
    }
    taken += here;
    __syncthreads();
  }
  // references of the copied pages; a page nobody holds any more is free after this call
  int freed = 0;
  for (int s = tid; s < a.slots; s += kBig) {
    const int p = cow_src[s];
    if (p >= 0 && atomicSub(&a.t.refs[p], 1) == 1) {
      atomicOr(&a.t.free_bits[p >> 5], 1u << (p & 31));
      ++freed;
    }
  }
  int total_freed;
  block_scan(freed, &total_freed);
  if (tid == 0) a.t.n_free[0] = n_free - taken + total_freed;
}

// One workgroup: the used pages behind the first n_used ones, each with the free
// page among those that it moves to, both ascending.  rank[p]: the place of p.
__global__ __launch_bounds__(kBig) void k_cache_moves(CacheArgs a, int32_t* src, int32_t* dst,
                                                      int32_t* n_moves, int32_t* rank) {
  const int tid = threadIdx.x;
  const int n_used = a.pages - a.t.n_free[0];
  const int n_words = (a.pages + 31) / 32;
  int holes = 0, movers = 0;
  for (int base = 0; base < n_words; base += kBig) {
    const int w = base + tid;
    uint32_t hole = 0u, move = 0u;
    if (w < n_words) {
      const uint32_t bits = a.t.free_bits[w];
      const int low = n_used - w * 32;   // pages of the word below n_used
      const int all = a.pages - w * 32;
      const uint32_t below = low >= 32 ? 0xFFFFFFFFu : (low <= 0 ? 0u : (1u << low) - 1u);
      const uint32_t there = all >= 32 ? 0xFFFFFFFFu : (1u << all) - 1u;
      hole = bits & below;
      move = ~bits & there & ~below;
    }
    int nh, nm;
    int h = holes + block_scan(__popc(hole), &nh);
    int m = movers + block_scan(__popc(move), &nm);
    while (hole) {
      dst[h++] = w * 32 + __ffs(hole) - 1;
      hole &= hole - 1;
    }
    while (move) {
      const int p = w * 32 + __ffs(move) - 1;
      src[m] = p;
      rank[p] = m++;
      move &= move - 1;
    }
    holes += nh;
    movers += nm;
  }
  if (tid == 0) n_moves[0] = min(holes, movers);
}

// Applies the moves to the tables, one thread per table entry, page, word and
// slot, and ends the move lists with -1.  The tables written may be the ones read:
// an entry is read and written by one thread, and a moved page's count goes to a
// place whose own thread leaves it or writes the same value.
__global__ __launch_bounds__(256) void k_cache_apply(CacheArgs a, CacheTables o, int32_t* src,
                                                     int32_t* dst, const int32_t* n_moves,
                                                     const int32_t* rank) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int n_free = a.t.n_free[0];
  const int n_used = a.pages - n_free;
  const int n = n_moves[0];
  if (x < (int64_t)a.slots * a.max_pages) {
    const int s = (int)(x / a.max_pages), j = (int)(x % a.max_pages);
    int p = a.t.table[x];
    if (j >= a.t.held[s] || !page_ok(a, p)) p = -1;
    else if (p >= n_used && rank[p] >= 0 && rank[p] < n) p = dst[rank[p]];
    o.table[x] = p;
  }
  if (x < a.pages) {
    const int i = (int)x;
    const int r = a.t.refs[i];
    if (i >= n_used) {
      if (r > 0 && rank[i] >= 0 && rank[i] < n) o.refs[dst[rank[i]]] = r;
      o.refs[i] = 0;
    } else if (r > 0) {
      o.refs[i] = r;
    }
    if (i >= n) {
      src[i] = -1;
      dst[i] = -1;
    }
  }
  if (x < a.slots) {
    o.lens[x] = a.t.lens[x];
    o.held[x] = a.t.held[x];
  }
  if (x == 0) o.n_free[0] = n_free;
  const int words = (a.pages + 31) / 32;
  if (x < words) {
    const int low = n_used - (int)x * 32, all = a.pages - (int)x * 32;
    const uint32_t below = low >= 32 ? 0xFFFFFFFFu : (low <= 0 ? 0u : (1u << low) - 1u);
    const uint32_t there = all >= 32 ? 0xFFFFFFFFu : (1u << all) - 1u;
    o.free_bits[x] = there & ~below;
  }
}

// Copies whole pages of K and V in every layer.  Workgroups walk over
// (tensor, layer, pair); a pair with an index out of range is skipped.
__global__ __launch_bounds__(256) void k_cache_copy(CacheArgs a, uint8_t* K, uint8_t* V, int n,
                                                    const int32_t* src, const int32_t* dst,
                                                    const int32_t* count) {
  if (count) n = min(max(count[0], 0), n);
  const int64_t units = (int64_t)n * a.layers * 2;
  const int per = a.page_bytes / 16;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u % n);
    const int64_t kl = u / n;
    const int layer = (int)(kl >> 1);
    const int s = src[i], d = dst[i];
    if (!page_ok(a, s) || !page_ok(a, d) || s == d) continue;
    uint8_t* pool = ((kl & 1) ? V : K) + (int64_t)layer * a.pages * a.page_bytes;
    const u32x4* from = reinterpret_cast<const u32x4*>(pool + (int64_t)s * a.page_bytes);
    u32x4* to = reinterpret_cast<u32x4*>(pool + (int64_t)d * a.page_bytes);
    int x = threadIdx.x;
    for (; x + 3 * 256 < per; x += 4 * 256) {
      u32x4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = from[x + 256 * q];
#pragma unroll
      for (int q = 0; q < 4; ++q) to[x + 256 * q] = v[q];
    }
    for (; x < per; x += 256) to[x] = from[x];
  }
}

// A chunk's keys and values into the pages.  A workgroup takes one kv head of one
// group of E positions (E = 16 bytes of elements, what V stores side by side) of a
// slot; slot s's groups are numbered from offsets[s] / E + 3 s on, which leaves room
// for a group that is cut at either end.  K goes in 16-byte pieces (the first half of
// the threads); V is turned, a thread gathers one dimension of the group's tokens.
template <typename E>
__global__ __launch_bounds__(256) void k_cache_append(CacheArgs a, E* K, E* V, int N, const E* k,
                                                      const E* v, const int32_t* offsets) {
  constexpr int kE = 16 / (int)sizeof(E);
  __shared__ int found[4];
  const int w = blockIdx.x;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < a.slots; s += 256) {
    const int o0 = min(max(offsets[s], 0), N), o1 = min(max(offsets[s + 1], o0), N);
    const int first = o0 / kE + 3 * s;
    if (o0 < o1 && first <= w && w < o1 / kE + 3 * (s + 1)) {
      found[0] = s;
      found[1] = o0;
      found[2] = o1;
      found[3] = w - first;
    }
  }
  __syncthreads();
  const int s = found[0], o0 = found[1], o1 = found[2];
  if (s < 0) return;
  const int64_t len = a.t.lens[s];
  if (len < 0) return;
  const int64_t start = (len / kE + found[3]) * kE;  // of the group
  const int e0 = start < len ? (int)(len - start) : 0;
  const int64_t pos = start + e0;
  const int64_t i = o0 + (pos - len);  // first token of the group
  if (i >= o1) return;
  const int n = (int)min((int64_t)(kE - e0), o1 - i);
  const int64_t j = pos >> a.page_shift;
  if (j >= min(a.t.held[s], a.max_pages)) return;
  const int p = a.t.table[(int64_t)s * a.max_pages + j];
  if (!page_ok(a, p)) return;
  const int D = a.head_dim, H = a.kv_heads, C = D / kE, page = 1 << a.page_shift;
  const int h = blockIdx.y;
  const int t0 = (int)(pos & (page - 1));
  const int64_t base = ((int64_t)p * H + h) * page * D;
  const E* kt = k + (i * H + h) * D;
  const E* vt = v + (i * H + h) * D;
  if (threadIdx.x < 128) {
    for (int x = threadIdx.x; x < n * C; x += 128) {
      const int c = x % C, t = x / C;
      const u32x4 q = *reinterpret_cast<const u32x4*>(kt + (int64_t)t * H * D + c * kE);
      *reinterpret_cast<u32x4*>(K + base + ((int64_t)c * page + t0 + t) * kE) = q;
    }
  } else {
    for (int d = threadIdx.x - 128; d < D; d += 128) {
      E* to = V + base + ((int64_t)(t0 / kE) * D + d) * kE;
      alignas(16) E q[kE];
#pragma unroll
      for (int t = 0; t < kE; ++t) q[t] = vt[(int64_t)min(t, n - 1) * H * D + d];
      if (n == kE) {
        *reinterpret_cast<u32x4*>(to) = *reinterpret_cast<const u32x4*>(q);
      } else {
#pragma unroll
        for (int t = 0; t < kE; ++t)
          if (t < n) to[e0 + t] = q[t];
      }
    }
  }
}

unsigned blocks_for(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

hipError_t launch_cache_init(const CacheArgs& a, hipStream_t stream) {
  TimingScope t("cache_init", stream);
  int64_t n = (int64_t)a.slots * a.max_pages;
  n = n > a.pages ? n : a.pages;
  hipLaunchKernelGGL(k_cache_init, dim3(blocks_for(n, 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const CacheArgs& a, int n, const int32_t* src, const int32_t* dst,
                             int32_t* status, hipStream_t stream) {
  TimingScope t("cache_fork", stream);
  hipLaunchKernelGGL(k_cache_fork, dim3(n), dim3(256), 0, stream, a, n, src, dst, status);
  return hipGetLastError();
}

hipError_t launch_cache_free(const CacheArgs& a, int n, const int32_t* slots, hipStream_t stream) {
  TimingScope t("cache_free", stream);
  hipLaunchKernelGGL(k_cache_free, dim3(n), dim3(256), 0, stream, a, n, slots);
  return hipGetLastError();
}

hipError_t launch_cache_commit(const CacheArgs& a, const int32_t* keep, int plus,
                               hipStream_t stream) {
  TimingScope t("cache_commit", stream);
  hipLaunchKernelGGL(k_cache_commit, dim3(a.slots), dim3(64), 0, stream, a, keep, plus);
  return hipGetLastError();
}

hipError_t launch_cache_reserve(const CacheArgs& a, const int32_t* add, int32_t* status,
                                int32_t* cow_src, int32_t* cow_dst, hipStream_t stream) {
  TimingScope t("cache_reserve", stream);
  hipLaunchKernelGGL(k_cache_reserve, dim3(1), dim3(kBig), 0, stream, a, add, status, cow_src,
                     cow_dst);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CacheArgs& a, const CacheTables& out, int32_t* src,
                                int32_t* dst, int32_t* n_moves, int32_t* rank,
                                hipStream_t stream) {
  {
    TimingScope t("cache_moves", stream);
    hipLaunchKernelGGL(k_cache_moves, dim3(1), dim3(kBig), 0, stream, a, src, dst, n_moves, rank);
  }
  {
    TimingScope t("cache_apply", stream);
    int64_t n = (int64_t)a.slots * a.max_pages;
    n = n > a.pages ? n : a.pages;
    hipLaunchKernelGGL(k_cache_apply, dim3(blocks_for(n, 256)), dim3(256), 0, stream, a, out, src,
                       dst, n_moves, rank);
  }
  return hipGetLastError();
}

hipError_t launch_cache_copy(const CacheArgs& a, void* K, void* V, int n, const int32_t* src,
                             const int32_t* dst, const int32_t* count, hipStream_t stream) {
  TimingScope t("cache_copy", stream);
  const int64_t units = (int64_t)n * a.layers * 2;
  const int64_t grid = units < 2048 ? units : 2048;  // 8 workgroups per CU
  hipLaunchKernelGGL(k_cache_copy, dim3((unsigned)grid), dim3(256), 0, stream, a,
                     static_cast<uint8_t*>(K), static_cast<uint8_t*>(V), n, src, dst, count);
  return hipGetLastError();
}

hipError_t launch_cache_append(const CacheArgs& a, bool bf16, void* K, void* V, int N,
                               const void* k, const void* v, const int32_t* offsets,
                               hipStream_t stream) {
  TimingScope t("cache_append", stream);
  const dim3 grid((unsigned)(N / (bf16 ? 8 : 4) + 3 * a.slots), (unsigned)a.kv_heads);
  if (bf16)
    hipLaunchKernelGGL(k_cache_append<uint16_t>, grid, dim3(256), 0, stream, a,
                       static_cast<uint16_t*>(K), static_cast<uint16_t*>(V), N,
                       static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), offsets);
  else
    hipLaunchKernelGGL(k_cache_append<float>, grid, dim3(256), 0, stream, a,
                       static_cast<float*>(K), static_cast<float*>(V), N,
                       static_cast<const float*>(k), static_cast<const float*>(v), offsets);
  return hipGetLastError();
}

}  // namespace dspark
