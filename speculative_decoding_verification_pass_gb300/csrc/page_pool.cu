// The page pool of a paged cache on the device: who holds which page, forks
// that share pages, copies of shared pages before they are written to, and
// moves of pages within a cache or to another.
//
// The books are a count of holders per page (0: free), the page table and the
// pages mapped per sequence.  A page is taken lowest number first, by sequence
// and then by position, so that the same calls give the same tables; there is
// no free list to keep in order, and a pool's used part stays low.
//
// One CTA keeps the books of a call: its phases depend on one another through
// counts over all sequences, each phase is short, and a barrier within a CTA
// costs far less than one across the GPU.  What reads and writes the cache (the
// copies) is a kernel of its own over all SMs.  Of 4 / 64
// sequences, on the device: free and fork 4.1 / 9.4 us, the books of a reservation 3.1 /
// 5.6 us: chains of counts, lengths, entries and barriers.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace spec {
namespace {

constexpr int kT = 1024;
constexpr int kW = kT / 32;

struct Scratch {
  int32_t *writers, *keeper, *taken;  // [n_pages]
  int32_t *need, *first, *copy;       // [B]
  int32_t *src, *dst, *slots;         // moves: as many as sequences, or as half the pages
  int32_t *count;
};
__host__ __device__ inline size_t list_ints(int B, int n_pages) {
  const size_t half = static_cast<size_t>(n_pages) / 2 + 1;
  return half > static_cast<size_t>(B) ? half : static_cast<size_t>(B);
}
__host__ __device__ inline Scratch scratch_of(int32_t* s, int B, int n_pages) {
  Scratch q;
  q.count = s;
  q.writers = s + 4;
  q.keeper = q.writers + n_pages;
  q.taken = q.keeper + n_pages;
  q.need = q.taken + n_pages;
  q.first = q.need + B;
  q.copy = q.first + B;
  q.src = q.copy + B;
  q.dst = q.src + list_ints(B, n_pages);
  q.slots = q.dst + list_ints(B, n_pages);
  return q;
}

SPEC_DEVINL int pages_for(int slots) { return (slots + kPageSlots - 1) / kPageSlots; }

// Sum over the block of one value a warp (lane 0's) so far, in order of the warps: exclusive prefix, total in *all.
SPEC_DEVINL int block_prefix(int v, int* red, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  const int mine = red[lane];
  int w = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - mine, warp) + incl - v;
}

// One holder less; 1 if the page is free now.
SPEC_DEVINL int put_back(const PagesParams& p, int page) {
  const int old = atomicSub(p.ref + page, 1);
  if (old <= 0) {  // nobody held it
    atomicAdd(p.ref + page, 1);
    set_status(p.status, SPEC_DEV_BAD_PAGE);
    return 0;
  }
  return old == 1;
}

__global__ void pages_init_kernel(const PagesParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const long long n = static_cast<long long>(p.B) * p.max_pages;
  const long long i0 = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = i0; i < n; i += step) p.table[i] = -1;
  for (long long i = i0; i < p.n_pages; i += step) p.ref[i] = 0;
  for (long long i = i0; i < p.B; i += step) {
    p.mapped[i] = 0;
    p.len[i] = 0;
  }
  if (i0 == 0) *p.n_free = p.n_pages;
}

// The entries [from, to) of sequence b's row are pages of the pool (a warp).
SPEC_DEVINL bool entries_ok(const PagesParams& p, int b, int from, int to) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  for (int j = from + lane; j < to; j += 32) {
    const int pg = held_page(p.table[static_cast<long long>(b) * p.max_pages + j]);
    ok = ok && pg >= 0 && pg < p.n_pages;
  }
  return __all_sync(0xffffffffu, ok);
}

// Sequence b's entries [from, to) returned (a warp); how many pages became free.
SPEC_DEVINL int give_back(const PagesParams& p, int b, int from, int to) {
  const int lane = threadIdx.x & 31;
  int freed = 0;
  for (int j = from + lane; j < to; j += 32) {
    int32_t* e = p.table + static_cast<long long>(b) * p.max_pages + j;
    freed += put_back(p, held_page(*e));
    *e = -1;
  }
  return freed;
}

// Sequence b, of `base` pages by its length, gets no pass: its last page says so, until a reservation serves it.
SPEC_DEVINL void sit_out(const PagesParams& p, int b, int base) {
  int32_t* e = p.table + static_cast<long long>(b) * p.max_pages + base - 1;
  if (base) *e = sat_out(held_page(*e));
}

// The `want` lowest free pages, in order, to list; how many there are.
SPEC_DEVINL int lowest_free(const PagesParams& p, int want, int32_t* list, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int found = 0;
  for (long long base = 0; base < p.n_pages && found < want; base += 4 * kT) {
    unsigned m[4];
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long pg = base + warp * 128 + i * 32 + lane;
      m[i] = __ballot_sync(0xffffffffu, pg < p.n_pages && __ldcg(p.ref + pg) == 0);
      cnt += __popc(m[i]);
    }
    int all;
    int at = found + block_prefix(lane == 0 ? cnt : 0, red, &all);
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = at + __popc(m[i] & ((1u << lane) - 1u));
      if ((m[i] >> lane & 1u) && k < want) list[k] = static_cast<int32_t>(base + warp * 128 + i * 32 + lane);
      at += __popc(m[i]);
    }
    found += all;
  }
  return found < want ? found : want;
}

__global__ void __launch_bounds__(kT) pages_reserve_kernel(const PagesParams p, int n, const int32_t* d_n) {
  __shared__ int red[kW];
  __shared__ int s_freed, s_moves, s_taken;
  grid_dep_wait();
  grid_dep_launch();
  const Scratch s = scratch_of(p.scratch, p.B, p.n_pages);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_freed = s_moves = s_taken = 0;
  __syncthreads();
  // 1. pages past the lengths go back.  need[b]: pages to take, -1: the sequence is left alone
  for (int b = warp; b < p.B; b += kW) {
    const int L = p.len[b], m = p.mapped[b], want = d_n ? d_n[b] : n;
    const long long cap = static_cast<long long>(p.max_pages) * kPageSlots;
    int bad = 0;
    if (L < 0 || want < 0 || L + static_cast<long long>(want) > cap) bad = SPEC_DEV_KV_OVERFLOW;
    const int base = bad ? 0 : pages_for(L);
    if (!bad && (m < base || m > p.max_pages || !entries_ok(p, b, max(base - 1, 0), m))) bad = SPEC_DEV_BAD_PAGE;
    if (bad) {
      const int last = L > 0 && L <= cap ? pages_for(L) : 0;  // (its books may be sound: then it sits the pass out)
      const bool mark = bad == SPEC_DEV_KV_OVERFLOW && last && m >= last && m <= p.max_pages &&
                        entries_ok(p, b, last - 1, last);
      if (lane == 0) {
        set_status(p.status, bad);
        if (mark) sit_out(p, b, last);
        s.need[b] = -1;
      }
      continue;
    }
    const int freed = __reduce_add_sync(0xffffffffu, give_back(p, b, base, m));
    if (lane == 0) {
      if (freed) atomicAdd(&s_freed, freed);
      p.mapped[b] = base;
      s.need[b] = want ? pages_for(L + want) - base : 0;
      if (want && L % kPageSlots) {
        const int pg = held_page(p.table[static_cast<long long>(b) * p.max_pages + base - 1]);
        s.writers[pg] = 0;
        s.keeper[pg] = -1;
      }
    }
  }
  __syncthreads();
  // 2. who writes to a partly filled page; the longest keeps it, the lowest-numbered of equally long
  // (rows of one that gets no page now lie below what the keeper writes)
  auto partial = [&](int b, int* pg, int* key) {
    const int L = p.len[b];
    if (s.need[b] < 0 || (d_n ? d_n[b] : n) == 0 || L % kPageSlots == 0) return false;
    *pg = held_page(p.table[static_cast<long long>(b) * p.max_pages + L / kPageSlots]);
    *key = (L % kPageSlots << 16) | (65535 - b);
    return true;
  };
  for (int b = threadIdx.x; b < p.B; b += kT) {
    int pg, key;
    if (partial(b, &pg, &key)) {
      atomicAdd(s.writers + pg, 1);
      atomicMax(s.keeper + pg, key);
    }
  }
  __syncthreads();
  // 3. where each sequence's new pages start in the order of taking
  int run = 0;
  for (int b0 = 0; b0 < p.B; b0 += kT) {
    const int b = b0 + threadIdx.x;
    int c = 0, copy = 0;
    if (b < p.B && s.need[b] >= 0) {
      int pg, key;
      if (partial(b, &pg, &key))
        copy = !(__ldcg(p.ref + pg) == __ldcg(s.writers + pg) && __ldcg(s.keeper + pg) == key);
      c = s.need[b] + copy;
    }
    int all;
    const int at = run + block_prefix(c, red, &all);
    if (b < p.B) {
      s.first[b] = at;
      s.copy[b] = copy;
    }
    run += all;
    if (run > p.n_pages) run = p.n_pages + 1;  // (more than there are: no need to count on)
  }
  __syncthreads();
  const int there = lowest_free(p, min(run, p.n_pages), s.taken, red);
  __syncthreads();
  if (run > there) {  // not enough for all: in order, whoever what is left covers (a warp; first: -1 for the others)
    if (warp == 0) {
      int taken = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int c = b < p.B ? max(s.need[b], 0) + s.copy[b] : 0;
        int first = 0;
        for (int i = 0; i < 32; ++i) {
          const int ci = __shfl_sync(0xffffffffu, c, i);
          const bool fits = taken + ci <= there;
          if (lane == i) first = fits ? taken : -1;
          if (fits) taken += ci;
        }
        if (b < p.B) s.first[b] = first;
      }
    }
    __syncthreads();
  }
  // 4. the pages are put in place
  for (int b = warp; b < p.B; b += kW) {
    const int need = s.need[b];
    if (need < 0) continue;
    const int L = p.len[b], base = pages_for(L), copy = s.copy[b], at = s.first[b], c = need + copy;
    int32_t* row = p.table + static_cast<long long>(b) * p.max_pages;
    int pg, key;
    const bool writes = partial(b, &pg, &key);
    if (at < 0) {
      if (lane == 0) {
        set_status(p.status, SPEC_DEV_NO_PAGES);
        sit_out(p, b, base);
      }
      continue;
    }
    if ((d_n ? d_n[b] : n) == 0) {  // (of pages returned alone, without counts by sequence, marks stay as they are)
      if (lane == 0 && d_n) sit_out(p, b, base);
      continue;
    }
    for (int i = lane; i < need; i += 32) {
      const int q = s.taken[at + copy + i];
      row[base + i] = q;
      p.ref[q] = 1;
    }
    if (lane == 0) {
      if (base && !copy) row[base - 1] = writes ? pg : held_page(row[base - 1]);
      if (copy) {
        const int q = s.taken[at], i = atomicAdd(&s_moves, 1);
        row[base - 1] = q;
        p.ref[q] = 1;
        atomicSub(p.ref + pg, 1);
        s.src[i] = pg;
        s.dst[i] = q;
        s.slots[i] = L % kPageSlots;
      }
      p.mapped[b] = base + need;
      if (c) atomicAdd(&s_taken, c);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *s.count = s_moves;
    *p.n_free += s_freed - s_taken;
  }
}

// A sequence that is a destination twice, or a destination and a source, makes
// its pairs void: their order would decide.
__global__ void __launch_bounds__(kT) pages_fork_kernel(const PagesParams p, int n, const int32_t* src,
                                                        const int32_t* dst) {
  __shared__ int s_freed;
  grid_dep_wait();
  grid_dep_launch();
  const Scratch s = scratch_of(p.scratch, p.B, p.n_pages);
  int32_t* mark = s.need;
  constexpr int kSource = 1 << 20;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_freed = 0;
  for (int b = threadIdx.x; b < p.B; b += kT) mark[b] = 0;
  __syncthreads();
  auto inside = [&](int b) { return b >= 0 && b < p.B; };
  for (int i = threadIdx.x; i < n; i += kT) {
    const int a = src[i], b = dst[i];
    if (inside(b)) atomicAdd(mark + b, 1);
    if (inside(a)) atomicOr(mark + a, kSource);
  }
  __syncthreads();
  for (int i = warp; i < n; i += kW) {
    const int a = src[i], b = dst[i];
    if (!inside(a) || !inside(b) || __ldcg(mark + b) != 1) {
      if (lane == 0) set_status(p.status, SPEC_DEV_BAD_SEQ);
      continue;
    }
    const int L = p.len[a], ma = p.mapped[a], mb = p.mapped[b];
    const bool fits = L >= 0 && L <= static_cast<long long>(p.max_pages) * kPageSlots;
    const int base = fits ? pages_for(L) : 0;
    if (!fits || base > ma || ma > p.max_pages || mb < 0 || mb > p.max_pages || !entries_ok(p, a, 0, base) ||
        !entries_ok(p, b, 0, mb)) {
      if (lane == 0) set_status(p.status, SPEC_DEV_BAD_PAGE);
      continue;
    }
    const int freed = __reduce_add_sync(0xffffffffu, give_back(p, b, 0, mb));
    int32_t *from = p.table + static_cast<long long>(a) * p.max_pages,
            *to = p.table + static_cast<long long>(b) * p.max_pages;
    for (int j = lane; j < base; j += 32) {
      const int e = from[j], pg = held_page(e);
      atomicAdd(p.ref + pg, 1);
      // a partly filled page is shared now: not to be written to by either (several forks of one source
      // put the same word there); what sits out does so twice
      const bool out = j == base - 1 && sits_out(e), part = j == base - 1 && L % kPageSlots && !out;
      if (part) from[j] = guarded(pg);
      to[j] = out ? e : part ? guarded(pg) : pg;
    }
    if (lane == 0) {
      if (freed) atomicAdd(&s_freed, freed);
      p.len[b] = L;
      p.mapped[b] = base;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_freed) *p.n_free += s_freed;
}

__global__ void __launch_bounds__(kT) pages_free_kernel(const PagesParams p, int n, const int32_t* seq) {
  __shared__ int s_freed;
  grid_dep_wait();
  grid_dep_launch();
  const Scratch s = scratch_of(p.scratch, p.B, p.n_pages);
  int32_t* mark = s.need;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_freed = 0;
  for (int b = threadIdx.x; b < p.B; b += kT) mark[b] = 0;
  __syncthreads();
  for (int i = warp; i < n; i += kW) {
    const int b = seq[i];
    if (b < 0 || b >= p.B) {
      if (lane == 0) set_status(p.status, SPEC_DEV_BAD_SEQ);
      continue;
    }
    const int again = __shfl_sync(0xffffffffu, lane == 0 ? atomicExch(mark + b, 1) : 0, 0);
    if (again) continue;
    const int m = p.mapped[b];
    if (m < 0 || m > p.max_pages || !entries_ok(p, b, 0, m)) {
      if (lane == 0) set_status(p.status, SPEC_DEV_BAD_PAGE);
      continue;
    }
    const int freed = __reduce_add_sync(0xffffffffu, give_back(p, b, 0, m));
    if (lane == 0) {
      if (freed) atomicAdd(&s_freed, freed);
      p.len[b] = 0;
      p.mapped[b] = 0;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_freed) *p.n_free += s_freed;
}

// U pages are used: those numbered U and above move, in order, to the free ones
// below U.  (There are as many of these as of those.)
__global__ void __launch_bounds__(kT) pages_plan_kernel(const PagesParams p) {
  __shared__ int red[kW];
  grid_dep_wait();
  grid_dep_launch();
  const Scratch s = scratch_of(p.scratch, p.B, p.n_pages);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine = 0, used;
  for (long long pg = threadIdx.x; pg < p.n_pages; pg += kT) mine += p.ref[pg] != 0;
  block_prefix(mine, red, &used);
  int gaps = 0, movers = 0;
  for (long long base = 0; base < p.n_pages; base += 4 * kT) {
    unsigned m[4];
    int gap_cnt = 0, move_cnt = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long pg = base + warp * 128 + i * 32 + lane;
      const bool in = pg < p.n_pages, held = in && p.ref[pg] != 0;
      m[i] = __ballot_sync(0xffffffffu, in && held == (pg >= used));  // free below, or held above
      const unsigned low = __ballot_sync(0xffffffffu, pg < used);
      gap_cnt += __popc(m[i] & low);
      move_cnt += __popc(m[i] & ~low);
      if (in && pg >= used) s.keeper[pg] = -1;
    }
    int all_gaps, all_moves;
    int g = gaps + block_prefix(lane == 0 ? gap_cnt : 0, red, &all_gaps);
    int v = movers + block_prefix(lane == 0 ? move_cnt : 0, red, &all_moves);
    g = __shfl_sync(0xffffffffu, g, 0);
    v = __shfl_sync(0xffffffffu, v, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long pg = base + warp * 128 + i * 32 + lane;
      const unsigned low = __ballot_sync(0xffffffffu, pg < used), before = (1u << lane) - 1u;
      if (m[i] >> lane & 1u) {
        if (pg < used)
          s.dst[g + __popc(m[i] & low & before)] = static_cast<int32_t>(pg);
        else
          s.src[v + __popc(m[i] & ~low & before)] = static_cast<int32_t>(pg);
      }
      g += __popc(m[i] & low);
      v += __popc(m[i] & ~low);
    }
    gaps += all_gaps;
    movers += all_moves;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kT) {
    const int a = s.src[i], b = s.dst[i];
    s.keeper[a] = b;  // where page a goes
    p.ref[b] = p.ref[a];
    p.ref[a] = 0;
  }
  if (threadIdx.x == 0) {
    s.count[0] = movers;
    s.count[1] = used;
  }
}

// The tables after the moves (by the CTAs of the copy, before their share of it).
struct Retable {
  int32_t* table;
  const int32_t *mapped, *to, *used;
  int B, n_pages, max_pages;
};

// ------------------------------------------------------------------- moves
// A warp moves 16 slots of one KV head, k or v, of one layer at a time (1 to 4
// KB, all of it in flight before the first store), and a lane their scale.  Bound
// by memory: 200 pages of an 8B-shaped bf16 cache (3.36 GB moved) 498 us, 6.73 TB/s,
// the rate of a plain copy; 1200 pages half used, 8-bit, 300 moved (2.52 GB) 412 us
// with the books, 6.1 TB/s.  Few pages: 16 slots a warp spread 4 pages of a 1B-shaped
// cache over 4096 warps, 2.9 us.
constexpr int kCopyThreads = 256;
constexpr int kCopyWords = 8;  // 16-byte words a lane: 16 slots of at most 256 bytes

__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(const PageMoves m, const Retable t) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long warp0 = blockIdx.x * static_cast<long long>(kCopyThreads / 32) + threadIdx.x / 32;
  const long long warps = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  if (t.table && blockIdx.y == 0) {
    const int used = *t.used;
    for (long long b = warp0; b < t.B; b += warps) {
      const int n = min(max(t.mapped[b], 0), t.max_pages);
      int32_t* row = t.table + b * t.max_pages;
      for (int j = lane; j < n; j += 32) {
        const int e = row[j], pg = held_page(e);
        if (pg < used) continue;
        const int to = pg < t.n_pages ? t.to[pg] : -1;
        if (to < 0)
          set_status(m.status, SPEC_DEV_BAD_PAGE);  // a page that nobody holds by the counts
        else
          row[j] = sits_out(e) ? sat_out(to) : e < 0 ? guarded(to) : to;
      }
    }
  }
  const int n = m.count ? *m.count : m.n;
  const int l = blockIdx.y;
  constexpr int kSub = kPageSlots / SPEC_KV8_BLOCK;
  const int words = SPEC_KV8_BLOCK * m.row_bytes / 16;  // of 16 slots
  const long long units = static_cast<long long>(n) * m.Hkv * (2 * kSub);
  for (long long u = warp0; u < units; u += warps) {
    const unsigned per = static_cast<unsigned>(m.Hkv) * (2 * kSub);
    const int i = static_cast<int>(u / per);
    const unsigned r = static_cast<unsigned>(u - static_cast<long long>(i) * per);
    const int sub = r % kSub, h = r / kSub % m.Hkv;
    const bool v = r >= static_cast<unsigned>(kSub) * m.Hkv;
    const int a = m.src[i], b = m.dst[i], rows = m.rows ? m.rows[i] : kPageSlots;
    if (a < 0 || a >= m.n_pages || b < 0 || b >= m.to_n_pages) {
      if (lane == 0) set_status(m.status, SPEC_DEV_BAD_PAGE);
      continue;
    }
    const long long x = (static_cast<long long>(l) * m.n_pages + a) * m.Hkv + h;
    const long long y = (static_cast<long long>(l) * m.to_n_pages + b) * m.Hkv + h;
    if (m.ks && lane == 0) (v ? m.to_vs : m.to_ks)[y * kSub + sub] = (v ? m.vs : m.ks)[x * kSub + sub];
    const int some = min(words, (rows - sub * SPEC_KV8_BLOCK) * m.row_bytes / 16);
    const uint4* from = reinterpret_cast<const uint4*>((v ? m.v : m.k) + x * kPageSlots * m.row_bytes) + sub * words;
    uint4* to = reinterpret_cast<uint4*>((v ? m.to_v : m.to_k) + y * kPageSlots * m.row_bytes) + sub * words;
    uint4 w[kCopyWords];
#pragma unroll
    for (int q = 0; q < kCopyWords; ++q)
      if (q * 32 + lane < some) w[q] = from[q * 32 + lane];
#pragma unroll
    for (int q = 0; q < kCopyWords; ++q)
      if (q * 32 + lane < some) to[q * 32 + lane] = w[q];
  }
}

template <class... P, class... A>
cudaError_t launch_dep(void (*fn)(P...), dim3 grid, int threads, cudaStream_t stream, const A&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a...);
}

cudaError_t launch_moves(const PageMoves& m, const Retable& t, long long most, int sms, cudaStream_t stream) {
  // a layer's share of the CTAs that run at once, no more than its units need
  constexpr int kWarps = kCopyThreads / 32;
  const long long units = most * m.Hkv * (2 * kPageSlots / SPEC_KV8_BLOCK);
  const long long share = std::max(1ll, (static_cast<long long>(sms) * 8 + m.L - 1) / m.L);
  const long long x = std::max(1ll, std::min(share, (units + kWarps - 1) / kWarps));
  return launch_dep(pages_move_kernel, dim3(static_cast<unsigned>(x), m.L), kCopyThreads, stream, m, t);
}

}  // namespace

size_t pages_scratch_ints(int B, int n_pages) {
  return 4 + 3 * static_cast<size_t>(n_pages) + 3 * static_cast<size_t>(B) + 3 * list_ints(B, n_pages);
}

cudaError_t launch_pages_init(const PagesParams& p, cudaStream_t stream) {
  const long long n = std::max(static_cast<long long>(p.B) * p.max_pages, static_cast<long long>(p.n_pages));
  return launch_dep(pages_init_kernel, dim3(static_cast<unsigned>(std::min(1024ll, (n + 255) / 256))), 256, stream, p);
}

cudaError_t launch_pages_reserve(const PagesParams& p, PageMoves m, int n, const int32_t* d_n, int sms,
                                 cudaStream_t stream) {
  const cudaError_t e = launch_dep(pages_reserve_kernel, dim3(1), kT, stream, p, n, d_n);
  if (e != cudaSuccess) return e;
  if (n == 0 && !d_n) return cudaSuccess;  // nothing is written to
  const Scratch s = scratch_of(p.scratch, p.B, p.n_pages);
  m.count = s.count;
  m.src = s.src;
  m.dst = s.dst;
  m.rows = s.slots;
  return launch_moves(m, Retable{}, p.B, sms, stream);
}

cudaError_t launch_pages_fork(const PagesParams& p, int n, const int32_t* src, const int32_t* dst,
                              cudaStream_t stream) {
  return launch_dep(pages_fork_kernel, dim3(1), kT, stream, p, n, src, dst);
}

cudaError_t launch_pages_free(const PagesParams& p, int n, const int32_t* seq, cudaStream_t stream) {
  return launch_dep(pages_free_kernel, dim3(1), kT, stream, p, n, seq);
}

cudaError_t launch_pages_compact(const PagesParams& p, PageMoves m, int sms, cudaStream_t stream) {
  const cudaError_t e = launch_dep(pages_plan_kernel, dim3(1), kT, stream, p);
  if (e != cudaSuccess) return e;
  const Scratch s = scratch_of(p.scratch, p.B, p.n_pages);
  m.count = s.count;
  m.src = s.src;
  m.dst = s.dst;
  const Retable t{p.table, p.mapped, s.keeper, s.count + 1, p.B, p.n_pages, p.max_pages};
  return launch_moves(m, t, p.n_pages / 2 + 1, sms, stream);
}

cudaError_t launch_pages_copy(const PageMoves& m, int sms, cudaStream_t stream) {
  return launch_moves(m, Retable{}, m.n, sms, stream);
}

}  // namespace spec
