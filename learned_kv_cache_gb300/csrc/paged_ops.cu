// Pages of the paged cache: taking them for new tokens, sharing or copying them (fork), compacting
// a row's kept tokens into its first pages, releasing them.
//
// LKV, "LKV-H" (a budget per KV head) and How much KV cache can you prune, "Conclusion" (a copy
// into a new tensor frees nothing while the old one lives): rows hold only the pages they need.
//
// Which page a row gets must not depend on the order in which threads run, so pages are not taken
// with atomics: the needs of the rows are summed in row order, the free pages enumerated in
// ascending order (a bit per page, so 131072 pages are 16 KB), and the i-th need gets the i-th free
// page.  One CTA does that (the "plan"): it is a chain of dependent reads and two block scans, and
// the rows' and pages' numbers go straight from registers into them.  What is wide -- tokens, table
// entries, counts of the pages taken -- is left to the kernel behind it, which fills the GPU.
// References are counted with integer atomics, whose order changes nothing.
#include <cooperative_groups.h>

#include <atomic>

#include "kvp_common.cuh"
#include "kvp_launch.h"

namespace kvp {
namespace {

namespace cg = cooperative_groups;

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WORDS = 4;              // words of the free mask per thread and step

enum { PLAN_APPEND = 0, PLAN_COPY = 1, PLAN_COMPACT = 2 };

struct PlanArgs {
  // append
  const int32_t* counts;
  int n_new;
  // copy
  const int32_t* src;
  // compact
  const int32_t *idx, *count;
  int b_max, W;          // W: pages of b_max tokens
  // workspace
  int32_t* start;        // [R] append: length before; copy: tokens to copy; compact: tokens kept; -1: row left alone
  int32_t* need;         // [R] pages
  int32_t* off;          // [R] first of the row's pages in list
  int32_t* tail;         // [R] append: the shared tail page that is copied, or -1
  int32_t* list;         // the pages taken, ascending
  int32_t* owner;        // copy: the row of each page in list
  int32_t* dmap;         // compact: [R, W] the page itself, or -2 - i: the row's i-th page of list
  int32_t* used;         // [1] pages taken
  int* status;
};

__device__ __forceinline__ int pages_of(int n, const PagedView& c) { return (n + c.ps - 1) >> c.shift; }

__device__ __forceinline__ int32_t* table_row(const PagedView& c, int r) { return c.table + (size_t)r * c.max_pages; }

__device__ __forceinline__ bool page_ok(int p, const PagedView& c) { return p >= 0 && p < c.n_pages; }

// Word x of the free mask; nothing behind the last page.
__device__ __forceinline__ uint32_t mask_word(const PagedView& c, int x) {
  const int left = c.n_pages - 32 * x;
  if (left <= 0) return 0u;
  return c.free_mask[x] & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
}

// One reference less; the page is free when it was the last.
__device__ __forceinline__ void release_page(const PagedView& c, int p, int* status) {
  if (!page_ok(p, c)) {
    raise_status(status, KVP_ERR_DEVICE_CHECK);
    return;
  }
  const int old = atomicSub(c.refs + p, 1);
  if (old == 1) atomicOr(c.free_mask + (p >> 5), 1u << (p & 31));
  if (old <= 0) {                          // nobody held it: put the count back
    atomicAdd(c.refs + p, 1);
    raise_status(status, KVP_ERR_DEVICE_CHECK);
  }
}

// Releases what `pages` gives for j = first, first + step, ... < end (-1: nothing): four counts of a
// thread are under way at a time.
template <typename F>
__device__ __forceinline__ void release_pages(const PagedView& c, int first, int end, int step, int* status, F pages) {
  for (int j0 = first; j0 < end; j0 += 4 * step) {
    int p[4], old[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) p[u] = j0 + u * step < end ? pages(j0 + u * step) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) old[u] = p[u] >= 0 && p[u] < c.n_pages ? atomicSub(c.refs + p[u], 1) : 2;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (old[u] == 1) atomicOr(c.free_mask + (p[u] >> 5), 1u << (p[u] & 31));
      if (old[u] <= 0) atomicAdd(c.refs + p[u], 1);            // nobody held it: put the count back
      if (old[u] <= 0 || p[u] >= c.n_pages || p[u] < -1) raise_status(status, KVP_ERR_DEVICE_CHECK);
    }
  }
}

// What the plan finds out about a row: the pages it needs, and what the kernel behind it has to know.
struct RowPlan {
  int start, need, tail, cnt;
};

template <int MODE>
__device__ __forceinline__ RowPlan row_plan(const PagedView& c, const PlanArgs& a, int r) {
  RowPlan w{-1, 0, -1, 0};
  if (MODE == PLAN_APPEND) {
    const int n = c.lens[r];
    w.cnt = a.counts ? a.counts[r] : a.n_new;
    bool ok = n >= 0 && n <= c.cap && w.cnt >= 0 && w.cnt <= a.n_new && w.cnt <= c.cap - n;
    if (ok && w.cnt > 0) {
      int first = pages_of(n, c);
      if (n & (c.ps - 1)) {
        const int p = table_row(c, r)[n >> c.shift];
        ok = page_ok(p, c);
        if (ok && c.refs[p] > 1) {
          w.tail = p;
          first = n >> c.shift;
        }
      }
      if (ok) {
        w.start = n;
        w.need = pages_of(n + w.cnt, c) - first;
      }
    }
    if (!ok) raise_status(a.status, KVP_ERR_DEVICE_CHECK);
  } else if (MODE == PLAN_COPY) {
    const int s = a.src[r];
    if (s >= 0) {
      const bool ok = s < c.R && s != r && a.src[s] < 0 && c.lens[r] == 0;
      const int n = ok ? c.lens[s] : -1;
      if (n < 0 || n > c.cap) {
        raise_status(a.status, KVP_ERR_DEVICE_CHECK);
      } else if (n > 0) {
        w.start = n;
        w.need = pages_of(n, c);
      }
    }
  } else {                                   // compact_need_kernel has been here
    w.start = a.start[r];
    w.need = a.need[r];
  }
  return w;
}

// Looks a row over, and says which of its kept pages have to be fresh ones: those whose tokens change and
// that somebody else holds too.  One CTA per row.  A row is not touched unless every index and every page
// id in it is good.  Bound by latency.
constexpr int NEED_THREADS = 512;
constexpr int NEED_LOADS = 8;              // of a thread, under way at a time

__global__ void __launch_bounds__(NEED_THREADS) compact_need_kernel(const PagedView c, const PlanArgs a) {
  __shared__ int scan_sh[33];
  allow_next_grid();                         // the plan and the copies wait for their turn on the GPU already
  wait_prior_grid();
  const int r = blockIdx.x, tid = threadIdx.x;
  const int cnt = a.count[r], n = c.lens[r];
  const int32_t* idx = a.idx + (size_t)r * a.b_max;
  const int32_t* table = table_row(c, r);
  bool ok = n >= 0 && n <= c.cap && cnt <= n && cnt <= a.b_max;
  if (ok && cnt >= 0) {
    bool good = true;
    // ascending from 0 on and below the length: then idx[m] >= m, too
    for (int m0 = tid; m0 < cnt; m0 += NEED_LOADS * NEED_THREADS) {
      int key[NEED_LOADS], before[NEED_LOADS];
#pragma unroll
      for (int u = 0; u < NEED_LOADS; ++u) {
        const int m = m0 + u * NEED_THREADS;
        key[u] = m < cnt ? idx[m] : 0;
        before[u] = m < cnt && m > 0 ? idx[m - 1] : -1;
      }
#pragma unroll
      for (int u = 0; u < NEED_LOADS; ++u) good &= key[u] > before[u] && key[u] < n;
    }
    const int held = pages_of(n, c);
#pragma unroll 4
    for (int j = tid; j < held; j += NEED_THREADS) good &= page_ok(table[j], c);
    ok = __syncthreads_and(good);
  }
  int need = 0;
  const int pages = ok && cnt > 0 ? pages_of(cnt, c) : 0;
  for (int j0 = 0; j0 < pages; j0 += NEED_THREADS) {
    const int j = j0 + tid;
    int d = -1;
    if (j < pages) {
      const int last = min((j + 1) << c.shift, cnt) - 1;   // ascending indices: if it stays, so do all before it
      const int p = table[j];
      d = idx[last] != last && c.refs[p] > 1 ? -2 : p;
    }
    int all;
    const int before = block_exclusive_scan(d == -2, scan_sh, &all);
    if (j < pages) a.dmap[(size_t)r * a.W + j] = d == -2 ? -2 - (need + before) : d;
    need += all;
  }
  if (tid == 0) {
    if (!ok) raise_status(a.status, KVP_ERR_DEVICE_CHECK);
    a.start[r] = ok && cnt >= 0 ? cnt : -1;
    a.need[r] = need;
  }
}

// The plan.  A thread has a row (several in turn above 1024 rows) and PLAN_WORDS words of the mask.
// Bound by latency: lengths, table, counts of the tail pages 2.0 us; the mask and the list 1.3 us for
// 256 pages, 2.0 us for 5600; the rows' books 0.9 us.
template <int MODE, int PLAN_THREADS>
__device__ __forceinline__ void make_plan(const PagedView& c, const PlanArgs& a) {
  __shared__ int scan_sh[33];
  __shared__ int used_sh;
  // a word of padding per 32: below, the lanes of a warp read words 32 apart
  __shared__ uint32_t word_sh[PLAN_WORDS * PLAN_THREADS * 33 / 32];
  __shared__ int rank_sh[PLAN_WORDS * PLAN_THREADS * 33 / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int words = (c.n_pages + 31) >> 5;
  const bool one = c.R <= PLAN_THREADS;      // every row stays in its thread's registers
  // the first words are on their way while the rows are looked at
  uint32_t mask[PLAN_WORDS];
#pragma unroll
  for (int k = 0; k < PLAN_WORDS; ++k) mask[k] = mask_word(c, PLAN_WORDS * tid + k);
  if (tid == 0) used_sh = 0;

  RowPlan w{-1, 0, -1, 0};
  int off = 0, want = 0;
  for (int base = 0; base < c.R; base += PLAN_THREADS) {
    const int r = base + tid;
    w = r < c.R ? row_plan<MODE>(c, a, r) : RowPlan{-1, 0, -1, 0};
    int all;
    off = want + block_exclusive_scan(w.need, scan_sh, &all);
    want += all;
    if (r < c.R) {
      a.off[r] = off;
      if (MODE != PLAN_COMPACT && !one) {
        a.start[r] = w.start;
        a.need[r] = w.need;
        if (MODE == PLAN_APPEND) a.tail[r] = w.tail;
      }
    }
  }

  // the lowest free pages, in order, out of the mask and into the list
  int found = 0;
  for (int base = 0; base < words && found < want; base += PLAN_WORDS * PLAN_THREADS) {
    int mine = 0;
#pragma unroll
    for (int k = 0; k < PLAN_WORDS; ++k) {
      const int x = base + PLAN_WORDS * tid + k;
      if (base > 0) mask[k] = mask_word(c, x);
      mine += __popc(mask[k]);
    }
    int all;
    int at = found + block_exclusive_scan(mine, scan_sh, &all);
    // the words change hands: consecutive ones to consecutive warps, a lane per page within a warp, so
    // that a run of free pages is written by the whole CTA, in consecutive entries of the list
#pragma unroll
    for (int k = 0; k < PLAN_WORDS; ++k) {
      const int x = PLAN_WORDS * tid + k;
      word_sh[x + (x >> 5)] = mask[k];
      rank_sh[x + (x >> 5)] = at;
      at += __popc(mask[k]);
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < PLAN_WORDS; ++i) {
      const int mine_x = (i * 32 + lane) * (PLAN_THREADS / 32) + (tid >> 5);
      const uint32_t v = word_sh[mine_x + (mine_x >> 5)];
      const int to = rank_sh[mine_x + (mine_x >> 5)];
      const bool mine_taken = v != 0 && to < want;
      uint32_t some = __ballot_sync(0xffffffffu, mine_taken);
      while (some) {                         // two words at a time: their chains of shuffles overlap
        const int l0 = __ffs(some) - 1;
        some &= some - 1;
        const int l1 = some ? __ffs(some) - 1 : l0;
        some &= some - 1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int l = k == 0 ? l0 : l1;
          const uint32_t word = __shfl_sync(0xffffffffu, v, l);
          const int at_bit = __shfl_sync(0xffffffffu, to, l) + __popc(word & ((1u << lane) - 1u));
          const int x = (i * 32 + l) * (PLAN_THREADS / 32) + (tid >> 5);
          if (((word >> lane) & 1u) && at_bit < want) a.list[at_bit] = (base + x) * 32 + lane;
        }
      }
      if (mine_taken) {                      // the word without the pages taken: its lowest ones
        uint32_t rest = v;
        if (to + __popc(v) <= want) rest = 0;
        else for (int k = to; k < want; ++k) rest &= rest - 1;
        c.free_mask[base + mine_x] = rest;
      }
    }
    found += all;
  }
  found = min(found, want);

  // rows whose pages run past the free ones are left alone; the others have them
  __syncthreads();
  int used = 0;
  for (int base = 0; base < c.R; base += PLAN_THREADS) {
    const int r = base + tid;
    if (r < c.R) {
      if (!one) {
        off = a.off[r];
        w.start = a.start[r];
        w.need = a.need[r];
        if (MODE == PLAN_APPEND) {
          w.tail = a.tail[r];
          w.cnt = a.counts ? a.counts[r] : a.n_new;
        }
      }
      if (w.need > 0 && off + w.need > found) {
        w.start = -1;
        w.need = 0;
        raise_status(a.status, KVP_ERR_DEVICE_CHECK);
      }
      if (w.need > 0) used = max(used, off + w.need);
      a.start[r] = w.start;
      if (MODE == PLAN_APPEND) {
        a.tail[r] = w.tail;
        if (w.start >= 0) {
          c.lens[r] = w.start + w.cnt;
          if (w.tail >= 0) release_page(c, w.tail, a.status);   // its tokens are copied before anyone can take it
        }
      } else if (MODE == PLAN_COPY && w.start >= 0) {
        c.lens[r] = w.start;
      }
    }
    if (MODE == PLAN_COPY) {                 // the owner of each page, a warp per row
      const int mine = r < c.R ? w.need : 0;
      for (uint32_t some = __ballot_sync(0xffffffffu, mine > 0); some; some &= some - 1) {
        const int i = __ffs(some) - 1;
        const int need = __shfl_sync(0xffffffffu, mine, i), o = __shfl_sync(0xffffffffu, off, i);
        for (int k = lane; k < need; k += 32) a.owner[o + k] = base + (tid & ~31) + i;
      }
    }
  }
  used = __reduce_max_sync(0xffffffffu, used);
  if (lane == 0 && used > 0) atomicMax(&used_sh, used);
  __syncthreads();
  used = used_sh;
  if (MODE == PLAN_COPY && tid == 0) *a.used = used;
  // pages that were found for a row that was left alone go back
  for (int i = used + tid; i < found; i += PLAN_THREADS) atomicOr(c.free_mask + (a.list[i] >> 5), 1u << (a.list[i] & 31));
}

template <int MODE>
__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const PagedView c, const PlanArgs a) {
  wait_prior_grid();
  make_plan<MODE, PLAN_THREADS>(c, a);
}

// ------------------------------------------------------------------ moving tokens
// 16-byte vectors throughout: VPR of them make one token's K (or V); consecutive threads take
// consecutive vectors of a token.

// Division by a number that the launch fixes (a product with its rounded-up reciprocal: Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication"): q = (x * mul) >> (32 + shift).  mul
// exceeds the reciprocal's 2^(32 + shift) by less than `by` <= 2^(shift + 1), so q is exact for x < 2^31.
struct FastDiv {
  uint32_t mul, shift, by;
};
FastDiv fast_div(uint32_t by) {
  FastDiv d{0, 0, by};
  if (by == 1) return d;                     // handled apart: the multiplier would need 33 bits
  while ((1u << d.shift) < by) ++d.shift;    // 2^(shift-1) < by <= 2^shift
  --d.shift;
  d.mul = (uint32_t)(((1ull << (32 + d.shift)) + by - 1) / by);
  return d;
}
__device__ __forceinline__ uint32_t div_by(uint32_t x, const FastDiv& d) {
  return d.by == 1 ? x : __umulhi(x, d.mul) >> d.shift;
}

// New tokens to their slots, and the books of the pages taken for them: a page's entry and count are
// written by the thread of the first new token in it.  Bound by HBM: a thread has one vector of K and
// one of V under way, and the occupancy does the rest (56 rows x 4096..8192 tokens: 72 us, with two
// tokens per thread 72 us, with four 94 us).  Starts, tails, offsets and the list come from the plan.
template <int VPR>
__device__ __forceinline__ void append_tokens(const PagedView& c, const PagedNew& a, const int32_t* starts,
                                              const int32_t* tails, const int32_t* offs, const int32_t* list, int elt,
                                              const FastDiv& by_new, const FastDiv& by_heads, long long tokens,
                                              long long thread, long long threads) {
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  char* pk = (char*)c.k;
  char* pv = (char*)c.v;
  const int v = (int)(thread % VPR);
  for (long long x = thread / VPR; x < tokens; x += threads / VPR) {
    const int r = (int)div_by((uint32_t)x, by_new), i = (int)((uint32_t)x - (uint32_t)r * by_new.by);
    if (i >= (a.counts ? __ldg(a.counts + r) : a.n_new)) continue;
    const int b = (int)div_by((uint32_t)r, by_heads), h = r - b * a.h_kv;
    const uint4 k = ld_stream16((const char*)a.k + (b * a.ks[0] + h * a.ks[1] + i * a.ks[2]) * elt + v * 16);
    const uint4 y = ld_stream16((const char*)a.v + (b * a.vs[0] + h * a.vs[1] + i * a.vs[2]) * elt + v * 16);
    const int start = starts[r], tail = tails[r], off = offs[r];
    if (start < 0) continue;
    const int t = start + i, j = t >> c.shift, o = t & (c.ps - 1);
    const int first = tail >= 0 ? start >> c.shift : pages_of(start, c);
    const int p = j >= first ? list[off + j - first] : table_row(c, r)[j];
    if (!page_ok(p, c)) continue;            // the plan has raised the status
    const int64_t to = p * pgs + o * ts + v * 16;
    *reinterpret_cast<uint4*>(pk + to) = k;
    *reinterpret_cast<uint4*>(pv + to) = y;
    if (v == 0) {
      if (j >= first && (i == 0 || o == 0)) {
        table_row(c, r)[j] = p;
        c.refs[p] = 1;
      }
      if (c.score) c.score[(size_t)r * c.cap + t] = 0.f;
      if (c.pos) c.pos[(size_t)r * c.cap + t] = a.pos ? __ldg(a.pos + r) + i : t;
    }
  }
}

// The tokens of row r's shared tail page, to the page that replaces it; `group` threads share the row,
// UN vectors of each in flight.
template <int VPR, int UN>
__device__ __forceinline__ void copy_tail(const PagedView& c, int from, int to, int tokens, int elt, int thread, int group) {
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  char* pool[2] = {(char*)c.k, (char*)c.v};
#pragma unroll UN
  for (int e = thread; e < tokens * VPR; e += group) {
    const int64_t at = (e / VPR) * ts + (e % VPR) * 16;
    const uint4 x = ld_stream16(pool[0] + from * pgs + at), y = ld_stream16(pool[1] + from * pgs + at);
    *reinterpret_cast<uint4*>(pool[0] + to * pgs + at) = x;
    *reinterpret_cast<uint4*>(pool[1] + to * pgs + at) = y;
  }
}

template <int VPR>
__global__ void __launch_bounds__(256) append_copy_kernel(const PagedView c, const PagedNew a, const PlanArgs w,
                                                          int elt, FastDiv by_new, FastDiv by_heads, long long tokens) {
  wait_prior_grid();
  append_tokens<VPR>(c, a, w.start, w.tail, w.off, w.list, elt, by_new, by_heads, tokens,
                     (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
  for (int r = blockIdx.x; r < c.R; r += gridDim.x) {      // a CTA per row
    const int from = w.tail[r], start = w.start[r];
    if (start >= 0 && from >= 0)
      copy_tail<VPR, 1>(c, from, w.list[w.off[r]], start & (c.ps - 1), elt, threadIdx.x, 256);
  }
}

// A decode step's append in one launch and without a workspace: one cluster, whose first CTA makes the
// plan in its shared memory; the others read it there.  The plan is what a step takes long for, and a
// second launch and a workspace cost the host as much again: 56 rows x 1 token + decode + free 15.4 ->
// 14.7 us of GPU time, a call from Python 13.2 -> 6.2 us of host time.  Shared tails, which 16 SMs copy with
// a warp per row, take longer than in the wide kernels (append_is_step).
constexpr int AS_ROWS = 512;               // their numbers and the list are in static shared memory
constexpr int AS_PAGES = 1024;
constexpr int AS_CTAS = 16;                // the largest cluster: the copies have that many SMs
constexpr int AS_THREADS = 512;

template <int VPR>
__global__ void __launch_bounds__(AS_THREADS) append_step_kernel(const PagedView c, const PagedNew a, PlanArgs w,
                                                                  int elt, FastDiv by_new, FastDiv by_heads,
                                                                  int tokens) {
  __shared__ int32_t start_sh[AS_ROWS], off_sh[AS_ROWS], tail_sh[AS_ROWS], list_sh[AS_PAGES];
  allow_next_grid();                         // the step's next kernel may take its places beside this one
  wait_prior_grid();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  if (rank == 0) {
    w.start = start_sh;
    w.off = off_sh;
    w.tail = tail_sh;
    w.list = list_sh;
    make_plan<PLAN_APPEND, AS_THREADS>(c, w);
  }
  cluster.sync();
  const int32_t* starts = cluster.map_shared_rank(start_sh, 0);
  const int32_t* offs = cluster.map_shared_rank(off_sh, 0);
  const int32_t* tails = cluster.map_shared_rank(tail_sh, 0);
  const int32_t* list = cluster.map_shared_rank(list_sh, 0);
  const int thread = rank * AS_THREADS + threadIdx.x, threads = AS_CTAS * AS_THREADS;
  append_tokens<VPR>(c, a, starts, tails, offs, list, elt, by_new, by_heads, tokens, thread, threads);
  for (int r = thread >> 5; r < c.R; r += threads >> 5) {  // a warp per row
    const int from = tails[r], start = starts[r];
    if (start >= 0 && from >= 0)
      copy_tail<VPR, 4>(c, from, list[offs[r]], start & (c.ps - 1), elt, threadIdx.x & 31, 32);
  }
  cluster.sync();                            // the plan has been read
}

// Whole pages of the rows that are copied, one page per CTA at a time: the list of the pages taken is
// the list of the work, whatever the rows' lengths.
template <int VPR>
__global__ void __launch_bounds__(256) pages_copy_kernel(const PagedView c, const PlanArgs w, int elt) {
  wait_prior_grid();
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  const int used = *w.used;
  for (int i = blockIdx.x; i < used; i += gridDim.x) {
    const int r = w.owner[i], s = w.src[r], k = i - w.off[r];
    const int from = table_row(c, s)[k], to = w.list[i];
    if (threadIdx.x == 0) {
      c.table[(size_t)r * c.max_pages + k] = to;
      c.refs[to] = 1;
    }
    if (!page_ok(from, c)) {
      if (threadIdx.x == 0) raise_status(w.status, KVP_ERR_DEVICE_CHECK);
      continue;
    }
    const int n = min(c.ps, w.start[r] - (k << c.shift));
    for (int e = threadIdx.x; e < n * VPR; e += blockDim.x) {
      const int64_t at = (e / VPR) * ts + (e % VPR) * 16;
      const uint4 kx = ld_stream16((const char*)c.k + from * pgs + at);
      const uint4 vx = ld_stream16((const char*)c.v + from * pgs + at);
      *reinterpret_cast<uint4*>((char*)c.k + to * pgs + at) = kx;
      *reinterpret_cast<uint4*>((char*)c.v + to * pgs + at) = vx;
    }
    for (int o = threadIdx.x; o < n; o += blockDim.x) {
      const size_t d = (size_t)r * c.cap + (k << c.shift) + o, f = (size_t)s * c.cap + (k << c.shift) + o;
      if (c.score) c.score[d] = c.score[f];
      if (c.pos) c.pos[d] = c.pos[f];
    }
  }
}

// Kept tokens of one row, in place.  idx is ascending, so idx[m] >= m: once every load of the tokens
// up to some m has landed, the slots up to m can be written without touching a token that is still
// to be read, and the loads of later tokens may be under way at any time.  So chunks of tokens stream
// through a ring in shared memory (cp.async), written in order, one barrier per chunk: loads of
// STAGES - 1 chunks are in flight while one is stored.  Where a token lies takes two dependent reads
// (index, table); they are made for eight chunks at a time, one group ahead of the copies.  The columns
// of a token (16-byte vectors of K and of V) do not depend on each other, so a cluster of CTAs shares a
// row by columns.  At the end the cluster gives the row its new pages.  120000 -> 16384 tokens of 56
// rows run at 5.8 TB/s (bound by HBM: half reads in pieces of 256 bytes, half writes), -> 4096 at 4.4
// TB/s: of those 55 us the three launches and the first look-ups take 12.
constexpr int CP_THREADS = 512;
constexpr int CP_TOK = 128;                // tokens per chunk
constexpr int CP_GROUP = 8;                // chunks whose tokens are looked up together

template <int VPS>   // 16-byte vectors of a token per CTA
struct Cp {
  static constexpr int STAGES = VPS == 16 ? 3 : 4;
  static constexpr int STAGE = CP_TOK * VPS * 16;
  static constexpr int PLACES = 2 * CP_GROUP * CP_TOK;     // tokens whose places are kept: two groups
  static constexpr int LOOKS = CP_GROUP * CP_TOK / CP_THREADS;
  static constexpr int OFF_PLACE = STAGES * STAGE;      // [PLACES] source and target offsets
  static constexpr int OFF_INDEX = OFF_PLACE + PLACES * 16;     // int32 [PLACES] source tokens
  static constexpr int OFF_SIDE = OFF_INDEX + PLACES * 4;  // [STAGES][CP_TOK] 4 bytes
  static constexpr int SMEM = OFF_SIDE + STAGES * CP_TOK * 4;
  static_assert(STAGES <= CP_GROUP - 2, "a group's places are overwritten once its last chunk is stored");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}

template <int VPS>
__global__ void __launch_bounds__(CP_THREADS) compact_pages_kernel(const PagedView c, const PlanArgs w, int elt,
                                                                  int per_tensor) {
  using C = Cp<VPS>;
  extern __shared__ __align__(16) uint8_t smem[];
  wait_prior_grid();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
  const int r = blockIdx.x / nranks, tid = threadIdx.x;
  const int cnt = w.start[r];
  if (cnt < 0) return;                       // the whole cluster
  const int n = c.lens[r], off = w.off[r];
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  char* base = (char*)(rank < per_tensor ? c.k : c.v) + (rank % per_tensor) * VPS * 16;
  const int32_t* idx = w.idx + (size_t)r * w.b_max;
  const int32_t* dmap = w.dmap + (size_t)r * w.W;
  const int32_t* table = table_row(c, r);
  // scores move with the first CTA's columns, positions with the last one's
  char* side = rank == 0 ? (char*)c.score : rank == nranks - 1 ? (char*)c.pos : nullptr;
  if (side) side += (size_t)r * c.cap * 4;
  longlong2* places = reinterpret_cast<longlong2*>(smem + C::OFF_PLACE);   // x: source, y: target; -1: stays
  int32_t* index_sh = reinterpret_cast<int32_t*>(smem + C::OFF_INDEX);
  uint32_t* side_sh = reinterpret_cast<uint32_t*>(smem + C::OFF_SIDE);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t side_ring = ring + C::OFF_SIDE;
  const int chunks = (cnt + CP_TOK - 1) / CP_TOK;

  // A group's look-ups: what ask() loads, find() looks at some chunks later; what find() loads, place()
  // writes down some chunks after that.  Nothing is waited for where it is asked for.
  // Indices and page ids are good, compact_need_kernel has looked at all of them; the bounds here hold for
  // indices that change under the call (in memory that it writes, say): nothing outside the pools is reached.
  int key[C::LOOKS], target[C::LOOKS], page[C::LOOKS];
  const auto ask = [&](int group) {
#pragma unroll
    for (int x = 0; x < C::LOOKS; ++x) {
      const int m = group * CP_GROUP * CP_TOK + x * CP_THREADS + tid;
      key[x] = target[x] = -1;
      if (m >= cnt) continue;
      key[x] = idx[m];
      target[x] = dmap[m >> c.shift];
    }
  };
  const auto find = [&] {
#pragma unroll
    for (int x = 0; x < C::LOOKS; ++x) {
      page[x] = (uint32_t)key[x] < (uint32_t)n ? table[key[x] >> c.shift] : -1;
      if (target[x] <= -2) target[x] = w.list[off - 2 - target[x]];
    }
  };
  const auto place = [&](int group) {
#pragma unroll
    for (int x = 0; x < C::LOOKS; ++x) {
      const int m = group * CP_GROUP * CP_TOK + x * CP_THREADS + tid, at = m & (C::PLACES - 1);
      longlong2 z = make_longlong2(-1, -1);
      if (page_ok(page[x], c) && page_ok(target[x], c)) {
        z.x = page[x] * pgs + (key[x] & (c.ps - 1)) * ts;
        z.y = target[x] * pgs + (m & (c.ps - 1)) * ts;
        if (z.x == z.y) z.x = z.y = -1;
      }
      places[at] = z;
      index_sh[at] = key[x];
    }
  };

  ask(0);
  find();
  place(0);
  __syncthreads();
  for (int i = 0; i < chunks + C::STAGES - 1; ++i) {
    const int group = i / CP_GROUP + 1;
    if (i % CP_GROUP == 0) ask(group);
    if (i % CP_GROUP == CP_GROUP / 2 - 1) find();
    if (i % CP_GROUP == CP_GROUP - 2) place(group);
    if (i < chunks) {
      const int t0 = (i * CP_TOK) & (C::PLACES - 1);
      const uint32_t dst = ring + (i % C::STAGES) * C::STAGE;
#pragma unroll
      for (int e = tid; e < CP_TOK * VPS; e += CP_THREADS) {
        const long long from = places[t0 + e / VPS].x;
        if (from >= 0) cp_async16(dst + e * 16, base + from + (e % VPS) * 16);
      }
      if (side && tid < CP_TOK) {
        const int j = index_sh[t0 + tid];
        if (places[t0 + tid].x >= 0 && j != i * CP_TOK + tid)
          cp_async4(side_ring + ((i % C::STAGES) * CP_TOK + tid) * 4, side + (size_t)j * 4);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 1) : "memory");
    __syncthreads();                         // everybody's loads of the chunk below have landed
    const int d = i - (C::STAGES - 1);
    if (d >= 0) {
      const int t0 = (d * CP_TOK) & (C::PLACES - 1);
      const uint8_t* src_sh = smem + (d % C::STAGES) * C::STAGE;
#pragma unroll
      for (int e = tid; e < CP_TOK * VPS; e += CP_THREADS) {
        const long long to = places[t0 + e / VPS].y;
        if (to >= 0)
          *reinterpret_cast<uint4*>(base + to + (e % VPS) * 16) = *reinterpret_cast<const uint4*>(src_sh + e * 16);
      }
      if (side && tid < CP_TOK) {
        const int m = d * CP_TOK + tid;
        if (places[t0 + tid].y >= 0 && index_sh[t0 + tid] != m)
          *reinterpret_cast<uint32_t*>(side + (size_t)m * 4) = side_sh[(d % C::STAGES) * CP_TOK + tid];
      }
    }
  }
  cluster.sync();                            // every CTA has read the row's table and length
  const int old_pages = pages_of(n, c), new_pages = pages_of(cnt, c);
  release_pages(c, rank * CP_THREADS + tid, old_pages, nranks * CP_THREADS, w.status, [&](int j) {
    const int p = table[j];
    int d = j < new_pages ? dmap[j] : -1;
    if (p == d) return j < new_pages ? -1 : c.n_pages;         // the page stays; or no page where one should be
    if (d <= -2) {
      d = w.list[off - 2 - d];
      c.refs[d] = 1;
    }
    c.table[(size_t)r * c.max_pages + j] = d;
    return p == -1 ? c.n_pages : p;
  });
  if (rank == 0 && tid == 0) c.lens[r] = cnt;
}

// ------------------------------------------------------------------ sharing and releasing

// Row r takes the pages of row src[r]; one CTA per row.  Bound by latency: 56 forks of 1024 pages 3.9 us.  With
// scores and positions it is those that take long, 256 slots in turn: 56 forks of 1024 tokens 3.8 us, of 8192
// 13 us, of 131072 170 us (their bytes, 117 MB, would be 18 us).
__global__ void __launch_bounds__(256) fork_kernel(const PagedView c, const int32_t* __restrict__ src, int* status) {
  wait_prior_grid();
  const int r = blockIdx.x, s = src[r];
  if (s < 0) return;
  const bool ok = s < c.R && s != r && src[s] < 0 && c.lens[r] == 0;
  const int n = ok ? c.lens[s] : -1;
  if (n < 0 || n > c.cap) {
    if (threadIdx.x == 0) raise_status(status, KVP_ERR_DEVICE_CHECK);
    return;
  }
  __syncthreads();                           // every thread has seen the row empty
  for (int j = threadIdx.x; j < pages_of(n, c); j += blockDim.x) {
    const int p = table_row(c, s)[j];
    table_row(c, r)[j] = p;
    if (page_ok(p, c)) atomicAdd(c.refs + p, 1);
    else raise_status(status, KVP_ERR_DEVICE_CHECK);
  }
  for (int t = threadIdx.x; t < n; t += blockDim.x) {
    if (c.score) c.score[(size_t)r * c.cap + t] = c.score[(size_t)s * c.cap + t];
    if (c.pos) c.pos[(size_t)r * c.cap + t] = c.pos[(size_t)s * c.cap + t];
  }
  if (threadIdx.x == 0) c.lens[r] = n;
}

// Row r keeps its first keep[r] tokens; one CTA per row.  Bound by latency (28 rows of 1875 pages 4.7 us).
__global__ void __launch_bounds__(512) free_kernel(const PagedView c, const int32_t* __restrict__ keep, int* status) {
  wait_prior_grid();
  const int r = blockIdx.x;
  const int kept = keep ? keep[r] : 0;
  if (kept < 0) return;
  const int n = c.lens[r];
  if (n < 0 || n > c.cap || kept > n) {
    if (threadIdx.x == 0) raise_status(status, KVP_ERR_DEVICE_CHECK);
    return;
  }
  __syncthreads();                           // every thread has read the length
  int32_t* table = table_row(c, r);
  release_pages(c, pages_of(kept, c) + threadIdx.x, pages_of(n, c), blockDim.x, status, [&](int j) {
    const int p = table[j];
    table[j] = -1;
    return p == -1 ? c.n_pages : p;          // a live entry names a page
  });
  if (threadIdx.x == 0) c.lens[r] = kept;
}

__global__ void __launch_bounds__(256) init_kernel(const PagedView c) {
  wait_prior_grid();
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long gid = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long e = gid; e < (long long)c.R * c.max_pages; e += stride) c.table[e] = -1;
  for (long long e = gid; e < c.R; e += stride) c.lens[e] = 0;
  for (long long e = gid; e < c.n_pages; e += stride) c.refs[e] = 0;
  for (long long e = gid; e < (c.n_pages + 31) / 32; e += stride) {
    const int left = c.n_pages - (int)e * 32;
    c.free_mask[e] = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
  }
}

// ------------------------------------------------------------------ host side
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Lays the plan's arrays out in a workspace (ws null: the size alone).
size_t plan_layout(const PagedView& c, PlanArgs* a, void* ws, long long list_cap, bool owner, bool tail, long long dmap) {
  char* base = (char*)ws;
  size_t at = 0;
  const auto take = [&](long long n) {
    int32_t* p = base ? (int32_t*)(base + at) : nullptr;
    at += align256((size_t)n * 4);
    return p;
  };
  if (list_cap > c.n_pages) list_cap = c.n_pages;
  a->used = take(1);
  a->start = take(c.R);
  a->need = take(c.R);
  a->off = take(c.R);
  a->tail = tail ? take(c.R) : nullptr;
  a->list = take(list_cap);
  a->owner = owner ? take(list_cap) : nullptr;
  a->dmap = dmap ? take(dmap) : nullptr;
  return at;
}

long long append_list_cap(const PagedView& c, int n_new) { return (long long)c.R * ((n_new + c.ps - 1) / c.ps + 1); }

int compact_pages_of(const PagedView& c, int b_max) {
  const int b = b_max < c.cap ? b_max : c.cap;
  return (b + c.ps - 1) >> c.shift;
}

template <int MODE>
cudaError_t launch_plan(const PagedView& c, const PlanArgs& a, cudaStream_t st) {
  count_launches(1);
  return launch_with_pdl(paged_plan_kernel<MODE>, dim3(1), dim3(PLAN_THREADS), 0, st, c, a);
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

unsigned blocks_for(long long items, int per_sm) {
  long long b = (items + 255) / 256;
  const long long most = (long long)sm_count() * per_sm;
  if (b > most) b = most;
  return (unsigned)(b < 1 ? 1 : b);
}

template <int VPS>
cudaError_t launch_compact_pages(const PagedView& c, const PlanArgs& a, int elt, int per_tensor, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(compact_pages_kernel<VPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cp<VPS>::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.R * 2 * per_tensor));
  cfg.blockDim = dim3(CP_THREADS);
  cfg.dynamicSmemBytes = Cp<VPS>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * per_tensor;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  e = cudaLaunchKernelEx(&cfg, compact_pages_kernel<VPS>, c, a, elt, per_tensor);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_init(const PagedView& c, cudaStream_t st) {
  count_launches(1);
  init_kernel<<<blocks_for((long long)c.R * c.max_pages + c.n_pages, 8), 256, 0, st>>>(c);
  return cudaGetLastError();
}

cudaLaunchConfig_t step_config(cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(AS_CTAS);
  cfg.blockDim = dim3(AS_THREADS);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = AS_CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of 16 CTAs need 16 SMs that lie together, which a partitioned GPU may not have.  Every device is
// asked once.
bool step_clusters_fit() {
  static std::atomic<signed char> known[64];               // 1: they fit, -1: they do not
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();                      // not an error of the caller's
    return false;
  }
  if (dev < 0 || dev >= 64) return false;
  if (known[dev] == 0) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = step_config(attr, nullptr);
    int n = 0;
    const bool ok = cudaFuncSetAttribute(append_step_kernel<16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                        cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, append_step_kernel<16>, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();
    known[dev] = ok ? 1 : -1;
  }
  return known[dev] > 0;
}

// Whether an append is a step: few rows and tokens.  The rule goes by the host time of a call, and by the GPU
// time of rows with tails of their own (8 / 64 / 256 rows: 4.7 / 5.3 / 6.4 us, plan and copies apart 6.2 / 6.8 /
// 7.3).  It does not look at the tails that are shared: those are copied by 16 SMs here and by all of them
// there, which shows from pages of 256 tokens on.  GPU time, rows in pairs on the same pages, half a page to
// copy for each, in one launch / plan and copies apart: 256 rows, pages of 32 tokens 11.3 / 9.3 us, 256 29 /
// 13, 1024 92 / 32; 8 rows, 32 7.5 / 7.0, 256 15.8 / 8.9, 1024 47 / 14.
bool append_is_step(const PagedView& c, int n_new) {
  const int vpr = c.D * (c.dtype == KVP_F32 ? 4 : 2) / 16;
  return c.R <= AS_ROWS && append_list_cap(c, n_new) <= AS_PAGES &&
         (long long)n_new * c.R * vpr <= 4LL * AS_CTAS * AS_THREADS && step_clusters_fit();
}

size_t paged_append_workspace(const PagedView& c, int n_new) {
  PlanArgs a{};
  return append_is_step(c, n_new) ? 0 : plan_layout(c, &a, nullptr, append_list_cap(c, n_new), false, true, 0);
}

cudaError_t launch_paged_append(const PagedView& c, const PagedNew& n, void* ws, int* status, cudaStream_t st) {
  PlanArgs a{};
  a.counts = n.counts;
  a.n_new = n.n_new;
  a.status = status;
  const int elt = c.dtype == KVP_F32 ? 4 : 2, vpr = c.D * elt / 16;
  const long long tokens = (long long)n.n_new * c.R;
  const FastDiv by_new = fast_div((uint32_t)n.n_new), by_heads = fast_div((uint32_t)n.h_kv);
  if (append_is_step(c, n.n_new)) {
    const auto step = [&](auto kernel) {
      cudaLaunchAttribute attr[2];
      const cudaLaunchConfig_t cfg = step_config(attr, st);
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      count_launches(1);
      e = cudaLaunchKernelEx(&cfg, kernel, c, n, a, elt, by_new, by_heads, (int)tokens);
      return e != cudaSuccess ? e : cudaGetLastError();
    };
    return vpr == 8 ? step(append_step_kernel<8>) : vpr == 16 ? step(append_step_kernel<16>) : step(append_step_kernel<32>);
  }
  plan_layout(c, &a, ws, append_list_cap(c, n.n_new), false, true, 0);
  cudaError_t e = launch_plan<PLAN_APPEND>(c, a, st);
  if (e != cudaSuccess) return e;
  // a block per row at least, for the shared tails
  const dim3 grid(blocks_for(tokens * vpr > 256LL * c.R ? tokens * vpr : 256LL * c.R, 8));
  const auto go = [&](auto kernel) {
    count_launches(1);
    return launch_with_pdl(kernel, grid, dim3(256), 0, st, c, n, a, elt, by_new, by_heads, tokens);
  };
  return vpr == 8 ? go(append_copy_kernel<8>) : vpr == 16 ? go(append_copy_kernel<16>) : go(append_copy_kernel<32>);
}

size_t paged_fork_workspace(const PagedView& c, int copy) {
  PlanArgs a{};
  return copy ? plan_layout(c, &a, nullptr, (long long)c.R * c.max_pages, true, false, 0) : 0;
}

cudaError_t launch_paged_fork(const PagedView& c, const int32_t* src, int copy, void* ws, int* status,
                              cudaStream_t st) {
  if (!copy) {
    count_launches(1);
    return launch_with_pdl(fork_kernel, dim3((unsigned)c.R), dim3(256), 0, st, c, src, status);
  }
  PlanArgs a{};
  plan_layout(c, &a, ws, (long long)c.R * c.max_pages, true, false, 0);
  a.src = src;
  a.status = status;
  cudaError_t e = launch_plan<PLAN_COPY>(c, a, st);
  if (e != cudaSuccess) return e;
  const int elt = c.dtype == KVP_F32 ? 4 : 2, vpr = c.D * elt / 16;
  const dim3 grid((unsigned)sm_count() * 8);
  count_launches(1);
  switch (vpr) {
    case 8: return launch_with_pdl(pages_copy_kernel<8>, grid, dim3(256), 0, st, c, a, elt);
    case 16: return launch_with_pdl(pages_copy_kernel<16>, grid, dim3(256), 0, st, c, a, elt);
    default: return launch_with_pdl(pages_copy_kernel<32>, grid, dim3(256), 0, st, c, a, elt);
  }
}

size_t paged_compact_workspace(const PagedView& c, int b_max) {
  PlanArgs a{};
  const long long pages = (long long)c.R * compact_pages_of(c, b_max);
  return plan_layout(c, &a, nullptr, pages, false, false, pages);
}

cudaError_t launch_paged_compact(const PagedView& c, const int32_t* idx, const int32_t* count, int b_max,
                                 void* ws, int* status, cudaStream_t st) {
  PlanArgs a{};
  a.W = compact_pages_of(c, b_max);
  plan_layout(c, &a, ws, (long long)c.R * a.W, false, false, (long long)c.R * a.W);
  a.idx = idx;
  a.count = count;
  a.b_max = b_max;
  a.status = status;
  count_launches(1);
  cudaError_t e = launch_with_pdl(compact_need_kernel, dim3((unsigned)c.R), dim3(NEED_THREADS), 0, st, c, a);
  if (e != cudaSuccess) return e;
  e = launch_plan<PLAN_COMPACT>(c, a, st);
  if (e != cudaSuccess) return e;
  const int elt = c.dtype == KVP_F32 ? 4 : 2, vpr = c.D * elt / 16;
  // Bytes of a token per CTA: 256 use DRAM best (120000 -> 16384 tokens of 56 rows 166 us, with 128
  // bytes 200 us), if the rows are enough for some 100 CTAs; fewer rows are cut finer (8 rows 30000 ->
  // 4096: 41 us with 256 bytes, 30 us with 128).
  if (vpr >= 16 && (long long)c.R * (vpr / 8) >= 96) return launch_compact_pages<16>(c, a, elt, vpr / 16, st);
  if (vpr == 32 || (long long)c.R * (vpr / 4) >= 48) return launch_compact_pages<8>(c, a, elt, vpr / 8, st);
  return launch_compact_pages<4>(c, a, elt, vpr / 4, st);    // a cluster holds 8 CTAs: 4 for K, 4 for V
}

cudaError_t launch_paged_free(const PagedView& c, const int32_t* keep, int* status, cudaStream_t st) {
  count_launches(1);
  return launch_with_pdl(free_kernel, dim3((unsigned)c.R), dim3(512), 0, st, c, keep, status);
}

}  // namespace kvp
