// Pages of the paged cache: taking them for new tokens, sharing or copying them (fork), compacting
// a row's kept tokens into its first pages, releasing them.
//
// LKV, "LKV-H" (a budget per KV head) and How much KV cache can you prune, "Conclusion" (a copy
// into a new tensor frees nothing while the old one lives): rows hold only the pages they need.
//
// Which page a row gets must not depend on the order in which threads run, so pages are not taken
// with atomics: the needs of the rows are summed in row order, the free pages enumerated in
// ascending order (a bit per page, so 32768 pages are 4 KB), and the i-th need gets the i-th free
// page.  One cluster does that ("plan": needs in parallel, the two scans in its first CTA, the books
// in parallel again, cluster barriers between); the tokens then move in a kernel of their own, which
// fills the GPU.  References are counted with integer atomics, whose order changes nothing.
#include <cooperative_groups.h>

#include "kvp_common.cuh"
#include "kvp_launch.h"

namespace kvp {
namespace {

namespace cg = cooperative_groups;

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_CTAS = 8;               // the portable cluster size

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
  int32_t* dmap;         // compact: [R, W] page of each kept page
  int32_t* used;         // [1] pages taken
  int* status;
};

__device__ __forceinline__ int pages_of(int n, const PagedView& c) { return (n + c.ps - 1) >> c.shift; }

__device__ __forceinline__ int32_t* table_row(const PagedView& c, int r) { return c.table + (size_t)r * c.max_pages; }

__device__ __forceinline__ bool page_ok(int p, const PagedView& c) { return p >= 0 && p < c.n_pages; }

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

// Pages row r needs, and what the later phases have to know of it.
template <int MODE>
__device__ __forceinline__ void row_need(const PagedView& c, const PlanArgs& a, int r) {
  int start = -1, need = 0;
  if (MODE == PLAN_APPEND) {
    const int n = c.lens[r], cnt = a.counts ? a.counts[r] : a.n_new;
    int tail = -1;
    bool ok = n >= 0 && n <= c.cap && cnt >= 0 && cnt <= a.n_new && cnt <= c.cap - n;
    if (ok && cnt > 0) {
      int first = pages_of(n, c);
      if (n & (c.ps - 1)) {
        const int p = table_row(c, r)[n >> c.shift];
        ok = page_ok(p, c);
        if (ok && c.refs[p] > 1) {
          tail = p;
          first = n >> c.shift;
        }
      }
      if (ok) {
        start = n;
        need = pages_of(n + cnt, c) - first;
      }
    }
    a.tail[r] = tail;
    if (!ok) raise_status(a.status, KVP_ERR_DEVICE_CHECK);
  } else if (MODE == PLAN_COPY) {
    const int s = a.src[r];
    if (s >= 0) {
      const bool ok = s < c.R && s != r && a.src[s] < 0 && c.lens[r] == 0;
      const int n = ok ? c.lens[s] : -1;
      if (n < 0 || n > c.cap) {
        raise_status(a.status, KVP_ERR_DEVICE_CHECK);
      } else if (n > 0) {
        start = n;
        need = pages_of(n, c);
      }
    }
  }
  a.start[r] = start;
  a.need[r] = need;
}

// The kept pages of row r: -2 where a fresh page is needed (the tokens change and somebody else
// holds the page), else the page the row has there.
__device__ __forceinline__ void compact_page(const PagedView& c, const PlanArgs& a, long long e) {
  const int r = (int)(e / a.W), j = (int)(e % a.W);
  const int cnt = a.count[r];
  int d = -1;
  if (cnt > 0 && cnt <= a.b_max && cnt <= c.lens[r] && c.lens[r] <= c.cap && j < pages_of(cnt, c)) {
    const int p = table_row(c, r)[j];
    if (page_ok(p, c)) {
      const int last = min((j + 1) << c.shift, cnt) - 1;   // ascending indices: all before it moved too, or none
      d = (c.refs[p] > 1 && a.idx[(size_t)r * a.b_max + last] != last) ? -2 : p;
    } else {
      raise_status(a.status, KVP_ERR_DEVICE_CHECK);
    }
  }
  a.dmap[e] = d;
}

template <int MODE>
__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const PagedView c, const PlanArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, gid = rank * PLAN_THREADS + tid, total = nranks * PLAN_THREADS;
  const int lane = tid & 31, gwarp = gid >> 5, nwarps = total >> 5;
  __shared__ int scan_sh[33];
  __shared__ int used_sh;

  // -- needs
  if (MODE == PLAN_COMPACT) {
    const long long items = (long long)c.R * a.W;
    for (long long e = gid; e < items; e += total) compact_page(c, a, e);
    cluster.sync();
    for (int r = gwarp; r < c.R; r += nwarps) {
      const int cnt = a.count[r], n = c.lens[r];
      const bool ok = n >= 0 && n <= c.cap && cnt <= n && cnt <= a.b_max;
      int need = 0;
      if (ok && cnt > 0)
        for (int j = lane; j < pages_of(cnt, c); j += 32) need += a.dmap[(size_t)r * a.W + j] == -2;
      need = __reduce_add_sync(0xffffffffu, need);
      if (lane == 0) {
        if (!ok) raise_status(a.status, KVP_ERR_DEVICE_CHECK);
        a.start[r] = ok && cnt >= 0 ? cnt : -1;
        a.need[r] = need;
      }
    }
  } else {
    for (int r = gid; r < c.R; r += total) row_need<MODE>(c, a, r);
  }
  cluster.sync();

  // -- which pages: two scans, in the first CTA
  if (rank == 0) {
    int want = 0;
    for (int base = 0; base < c.R; base += PLAN_THREADS) {
      const int r = base + tid;
      int all;
      const int before = block_exclusive_scan(r < c.R ? a.need[r] : 0, scan_sh, &all);
      if (r < c.R) a.off[r] = want + before;
      want += all;
    }
    int found = 0;
    const int words = (c.n_pages + 31) >> 5;
    for (int base = 0; base < words && found < want; base += 4 * PLAN_THREADS) {
      uint32_t m[4];
      int mine = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int w = base + 4 * tid + k;
        m[k] = w < words ? c.free_mask[w] : 0u;
        mine += __popc(m[k]);
      }
      int all;
      int at = found + block_exclusive_scan(mine, scan_sh, &all);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        for (uint32_t v = m[k]; v && at < want; v &= v - 1, ++at)
          a.list[at] = (base + 4 * tid + k) * 32 + __ffs(v) - 1;
      found += all;
    }
    // rows whose pages run past the free ones are left alone; the pages of the others are taken
    if (tid == 0) used_sh = 0;
    __syncthreads();
    int used = 0;
    for (int r = tid; r < c.R; r += PLAN_THREADS) {
      const int need = a.need[r];
      if (need == 0) continue;
      if (a.off[r] + need <= found) {
        used = max(used, a.off[r] + need);
      } else {
        a.start[r] = -1;
        raise_status(a.status, KVP_ERR_DEVICE_CHECK);
      }
    }
    used = __reduce_max_sync(0xffffffffu, used);
    if (lane == 0 && used > 0) atomicMax(&used_sh, used);
    __syncthreads();
    if (tid == 0) *a.used = used_sh;
  }
  cluster.sync();

  // -- the books
  const int used = *reinterpret_cast<volatile int32_t*>(a.used);
  for (int i = gid; i < used; i += total) {
    const int p = a.list[i];
    c.refs[p] = 1;
    if (i == 0 || (a.list[i - 1] >> 5) != (p >> 5)) {      // the first page of its word clears the word's bits
      uint32_t m = 0;
      for (int k = i; k < used && (a.list[k] >> 5) == (p >> 5); ++k) m |= 1u << (a.list[k] & 31);
      atomicAnd(c.free_mask + (p >> 5), ~m);
    }
  }
  for (int r = gwarp; r < c.R; r += nwarps) {
    const int start = a.start[r];
    if (start < 0) continue;
    const int need = a.need[r], off = a.off[r];
    if (MODE == PLAN_APPEND) {
      const int tail = a.tail[r];
      const int first = tail >= 0 ? start >> c.shift : pages_of(start, c);
      for (int k = lane; k < need; k += 32) table_row(c, r)[first + k] = a.list[off + k];
      if (lane == 0) {
        c.lens[r] = start + (a.counts ? a.counts[r] : a.n_new);
        if (tail >= 0) release_page(c, tail, a.status);
      }
    } else if (MODE == PLAN_COPY) {
      for (int k = lane; k < need; k += 32) {
        table_row(c, r)[k] = a.list[off + k];
        a.owner[off + k] = r;
      }
      if (lane == 0) c.lens[r] = start;
    } else if (need > 0) {
      int taken = 0;
      for (int j0 = 0; j0 < pages_of(start, c); j0 += 32) {
        const int j = j0 + lane;
        int32_t* d = a.dmap + (size_t)r * a.W + j;
        const bool fresh = j < pages_of(start, c) && *d == -2;
        const uint32_t b = __ballot_sync(0xffffffffu, fresh);
        if (fresh) *d = a.list[off + taken + __popc(b & ((1u << lane) - 1u))];
        taken += __popc(b);
      }
    }
  }
}

// ------------------------------------------------------------------ moving tokens
// 16-byte vectors throughout: VPR of them make one token's K (or V); consecutive threads take
// consecutive vectors of a token.

template <int VPR>
__global__ void __launch_bounds__(256) append_copy_kernel(const PagedView c, const PagedNew a, const PlanArgs w,
                                                          int elt) {
  wait_prior_grid();
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  char* pool[2] = {(char*)c.k, (char*)c.v};
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long gid = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long items = (long long)c.R * a.n_new * VPR;
  for (long long e = gid; e < items; e += stride) {
    const int v = (int)(e % VPR);
    const long long ri = e / VPR;
    const int r = (int)(ri / a.n_new), i = (int)(ri % a.n_new);
    const int start = w.start[r];
    if (start < 0 || i >= (a.counts ? a.counts[r] : a.n_new)) continue;
    const int t = start + i, b = r / a.h_kv, h = r % a.h_kv;
    const int p = table_row(c, r)[t >> c.shift];
    if (!page_ok(p, c)) continue;
    const int64_t to = p * pgs + (t & (c.ps - 1)) * ts + v * 16;
    const uint4 k = ld_stream16((const char*)a.k + (b * a.ks[0] + h * a.ks[1] + i * a.ks[2]) * elt + v * 16);
    const uint4 x = ld_stream16((const char*)a.v + (b * a.vs[0] + h * a.vs[1] + i * a.vs[2]) * elt + v * 16);
    *reinterpret_cast<uint4*>(pool[0] + to) = k;
    *reinterpret_cast<uint4*>(pool[1] + to) = x;
    if (v == 0) {
      if (c.score) c.score[(size_t)r * c.cap + t] = 0.f;
      if (c.pos) c.pos[(size_t)r * c.cap + t] = a.pos ? a.pos[r] + i : t;
    }
  }
  // tokens of shared tail pages, to the pages that replace them
  const long long tails = (long long)c.R * c.ps * VPR;
  for (long long e = gid; e < tails; e += stride) {
    const int v = (int)(e % VPR);
    const long long ro = e / VPR;
    const int r = (int)(ro >> c.shift), o = (int)(ro & (c.ps - 1));
    const int start = w.start[r], from = w.tail[r];
    if (start < 0 || from < 0 || o >= (start & (c.ps - 1))) continue;
    const int p = table_row(c, r)[start >> c.shift];
    const int64_t at = o * ts + v * 16;
#pragma unroll
    for (int x = 0; x < 2; ++x)
      *reinterpret_cast<uint4*>(pool[x] + p * pgs + at) = *reinterpret_cast<const uint4*>(pool[x] + from * pgs + at);
  }
}

// Whole pages of the rows that are copied, one page per CTA at a time.
template <int VPR>
__global__ void __launch_bounds__(256) pages_copy_kernel(const PagedView c, const PlanArgs w, int elt) {
  wait_prior_grid();
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  const int used = *w.used;
  for (int i = blockIdx.x; i < used; i += gridDim.x) {
    const int r = w.owner[i], s = w.src[r], k = i - w.off[r];
    const int from = table_row(c, s)[k], to = w.list[i];
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

// Kept tokens of one row, in place.  idx is ascending, so idx[m] >= m: once every load of the
// tokens below some m has landed, the slots below m are written without touching a token that is
// still to be read.  A chunk of tokens is therefore read by the whole CTA, a barrier, then written;
// the columns of a token (16-byte vectors of K and of V) do not depend on each other, so a cluster
// of CTAs shares a row by columns.  At the end the cluster gives the row its new pages.
constexpr int CC_THREADS = 256;
constexpr int CC_UNROLL = 4;

template <int VPS>   // 16-byte vectors of a token per CTA
__global__ void __launch_bounds__(CC_THREADS) compact_pages_kernel(const PagedView c, const PlanArgs w, int elt,
                                                                  int per_tensor) {
  wait_prior_grid();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
  const int r = blockIdx.x / nranks, tid = threadIdx.x;
  const int cnt = w.start[r];
  if (cnt < 0) return;                       // the whole cluster
  const int n = c.lens[r];
  const int64_t ts = c.token_stride * elt, pgs = c.page_stride * elt;
  constexpr int TOK = CC_THREADS / VPS;      // tokens per pass
  char* base = (char*)(rank < per_tensor ? c.k : c.v) + (rank % per_tensor) * VPS * 16 + (tid % VPS) * 16;
  const int32_t* idx = w.idx + (size_t)r * w.b_max;
  const int32_t* dmap = w.dmap + (size_t)r * w.W;
  const int32_t* table = table_row(c, r);
  float* side = rank == 0 ? c.score : nullptr;
  int32_t* iside = rank == nranks - 1 ? c.pos : nullptr;
  bool bad = false;
  for (int m0 = 0; m0 < cnt; m0 += TOK * CC_UNROLL) {
    uint4 x[CC_UNROLL];
    char* to[CC_UNROLL];
    float sc[CC_UNROLL];
    int32_t po[CC_UNROLL];
    int at[CC_UNROLL];
#pragma unroll
    for (int u = 0; u < CC_UNROLL; ++u) {
      const int m = m0 + u * TOK + tid / VPS;
      to[u] = nullptr;
      at[u] = -1;
      if (m >= cnt) continue;
      const int j = idx[m], d = dmap[m >> c.shift];
      const int p = j >= m && j < n && (m == 0 || j > idx[m - 1]) ? table[j >> c.shift] : -1;
      // a page whose last kept token stays was planned as unchanged (it may be shared): none may move
      const int last = min(((m >> c.shift) + 1) << c.shift, cnt) - 1;
      if (!page_ok(p, c) || !page_ok(d, c) || (j != m && idx[last] == last)) {
        bad = true;
        continue;
      }
      const int64_t f = p * pgs + (j & (c.ps - 1)) * ts, t = d * pgs + (m & (c.ps - 1)) * ts;
      if (f != t) {
        x[u] = *reinterpret_cast<const uint4*>(base + f);
        to[u] = base + t;
      }
      if (tid % VPS == 0 && j != m) {
        at[u] = m;
        if (side) sc[u] = side[(size_t)r * c.cap + j];
        if (iside) po[u] = iside[(size_t)r * c.cap + j];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < CC_UNROLL; ++u) {
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
      if (at[u] >= 0 && side) side[(size_t)r * c.cap + at[u]] = sc[u];
      if (at[u] >= 0 && iside) iside[(size_t)r * c.cap + at[u]] = po[u];
    }
  }
  if (bad) raise_status(w.status, KVP_ERR_DEVICE_CHECK);
  cluster.sync();                            // every CTA has read the row's table and length
  const int old_pages = pages_of(n, c), new_pages = pages_of(cnt, c);
  for (int j = rank * CC_THREADS + tid; j < old_pages; j += nranks * CC_THREADS) {
    const int p = table[j], d = j < new_pages ? dmap[j] : -1;
    if (p == d) continue;
    c.table[(size_t)r * c.max_pages + j] = d;
    release_page(c, p, w.status);
  }
  if (rank == 0 && tid == 0) c.lens[r] = cnt;
}

// ------------------------------------------------------------------ sharing and releasing

// Row r takes the pages of row src[r]; one CTA per row.
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

// Row r keeps its first keep[r] tokens; one CTA per row.
__global__ void __launch_bounds__(256) free_kernel(const PagedView c, const int32_t* __restrict__ keep, int* status) {
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
  for (int j = pages_of(kept, c) + threadIdx.x; j < pages_of(n, c); j += blockDim.x) {
    release_page(c, table_row(c, r)[j], status);
    table_row(c, r)[j] = -1;
  }
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(PLAN_CTAS);
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PLAN_CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_plan_kernel<MODE>, c, a);
  return e != cudaSuccess ? e : cudaGetLastError();
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.R * 2 * per_tensor));
  cfg.blockDim = dim3(CC_THREADS);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, compact_pages_kernel<VPS>, c, a, elt, per_tensor);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_init(const PagedView& c, cudaStream_t st) {
  count_launches(1);
  init_kernel<<<blocks_for((long long)c.R * c.max_pages + c.n_pages, 8), 256, 0, st>>>(c);
  return cudaGetLastError();
}

size_t paged_append_workspace(const PagedView& c, int n_new) {
  PlanArgs a{};
  return plan_layout(c, &a, nullptr, append_list_cap(c, n_new), false, true, 0);
}

cudaError_t launch_paged_append(const PagedView& c, const PagedNew& n, void* ws, int* status, cudaStream_t st) {
  PlanArgs a{};
  plan_layout(c, &a, ws, append_list_cap(c, n.n_new), false, true, 0);
  a.counts = n.counts;
  a.n_new = n.n_new;
  a.status = status;
  cudaError_t e = launch_plan<PLAN_APPEND>(c, a, st);
  if (e != cudaSuccess) return e;
  const int elt = c.dtype == KVP_F32 ? 4 : 2, vpr = c.D * elt / 16;
  const long long tokens = n.n_new > c.ps ? n.n_new : c.ps;
  const dim3 grid(blocks_for(tokens * c.R * vpr, 8));
  count_launches(1);
  switch (vpr) {
    case 8: return launch_with_pdl(append_copy_kernel<8>, grid, dim3(256), 0, st, c, n, a, elt);
    case 16: return launch_with_pdl(append_copy_kernel<16>, grid, dim3(256), 0, st, c, n, a, elt);
    default: return launch_with_pdl(append_copy_kernel<32>, grid, dim3(256), 0, st, c, n, a, elt);
  }
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
  cudaError_t e = launch_plan<PLAN_COMPACT>(c, a, st);
  if (e != cudaSuccess) return e;
  const int elt = c.dtype == KVP_F32 ? 4 : 2, vpr = c.D * elt / 16;
  // 128 bytes of a token per CTA: a full line, and up to four CTAs share K (or V) of a row
  return launch_compact_pages<8>(c, a, elt, vpr / 8, st);
}

cudaError_t launch_paged_free(const PagedView& c, const int32_t* keep, int* status, cudaStream_t st) {
  count_launches(1);
  return launch_with_pdl(free_kernel, dim3((unsigned)c.R), dim3(256), 0, st, c, keep, status);
}

}  // namespace kvp
