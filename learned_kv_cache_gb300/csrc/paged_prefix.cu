// One-token decode attention for sequences that share a long prefix: the pages that rows hold in common are
// read once for all of them.
//
//   out = sum_t softmax_t(scale * q . k_t) v_t,  lse = ln sum_t exp(scale * q . k_t)
//
// over the row's tokens t, in two parts joined by their log-sum-exps: the prefix, a product of all the
// family's queries with each tile of keys, and the row's own tokens.  What is shared is seen in the tables
// (equal page ids), so a wrong `lead` costs time and no correctness.
#include <cmath>

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "paged_prefix.cuh"

namespace kvp {
namespace {

using prefix::Item;
using prefix::Params;
using prefix::Piece;
using prefix::GAP;
using prefix::TILE;

constexpr int LOOK_THREADS = 256;

// The sequence that l follows: its lead, if that follows nobody itself.
__device__ __forceinline__ int root_of(const Params& p, int l) {
  const int x = p.lead[l];
  if (x < 0 || x == l || x >= p.N) return l;
  const int y = p.lead[x];
  return y < 0 || y == x ? x : l;
}

// This thread's first page, of those from `i0` on, at which rows r and rf differ (or that is no page); each of
// the `n` threads looks at U of them.
constexpr int LOOK_U = 8;
__device__ __forceinline__ int differ(const Params& p, int r, int rf, int i0, int most, int t, int n) {
  const int32_t* a = p.c.table + (size_t)r * p.c.max_pages;
  const int32_t* b = p.c.table + (size_t)rf * p.c.max_pages;
  int x[LOOK_U], y[LOOK_U];
#pragma unroll
  for (int k = 0; k < LOOK_U; ++k) {
    const int i = i0 + k * n + t;
    x[k] = i < most ? a[i] : 0;
    y[k] = i < most ? b[i] : 0;
  }
  int at = 0x7fffffff;
#pragma unroll
  for (int k = LOOK_U - 1; k >= 0; --k) {
    const int i = i0 + k * n + t;
    if (i < most && (x[k] != y[k] || x[k] < 0 || x[k] >= p.c.n_pages)) at = i;
  }
  return at;
}
__device__ __forceinline__ void check_row(const Params& p, int r) {
  const int n = p.c.lens[r];
  if (n < 0 || n > p.c.cap || p.lead[r / p.Hkv] >= p.N) raise_status(p.status, KVP_ERR_DEVICE_CHECK);
}

// Block r: how many leading tokens row r has on pages of its root's row (whole pages, that both rows have
// filled).  The blocks of head 0 put their sequence into the families' order, by counting.
__global__ void __launch_bounds__(LOOK_THREADS) prefix_look_kernel(const Params p) {
  __shared__ int sh[LOOK_THREADS / 32][3];
  __shared__ int mismatch;
  wait_prior_grid();
  allow_next_grid();
  const int r = blockIdx.x, l = r / p.Hkv, h = r % p.Hkv, tid = threadIdx.x;
  const int f = root_of(p, l);
  if (tid == 0) {
    mismatch = 0x7fffffff;
    check_row(p, r);
  }
  if (h == 0) {
    int before = 0, rank = 0, mine = 0;        // sequences of earlier families; of this one before l; of l's own
    for (int x = tid; x < p.N; x += LOOK_THREADS) {
      const int y = root_of(p, x);
      before += y < f;
      rank += y == f && x < l;
      mine += y == f;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    rank = __reduce_add_sync(0xffffffffu, rank);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((tid & 31) == 0) {
      sh[tid >> 5][0] = before;
      sh[tid >> 5][1] = rank;
      sh[tid >> 5][2] = mine;
    }
    __syncthreads();
    if (tid == 0) {
      before = rank = mine = 0;
      for (int w = 0; w < LOOK_THREADS / 32; ++w) {
        before += sh[w][0];
        rank += sh[w][1];
        mine += sh[w][2];
      }
      p.root[l] = f;
      p.order[before + rank] = l;
      p.base[l] = before;
      p.count[l] = mine;
    }
  }
  __syncthreads();
  if (f == l) {
    if (tid == 0) p.shared[r] = 0;
    return;
  }
  const int rf = f * p.Hkv + h;
  const int most = min(prefix::row_len(p, r), prefix::row_len(p, rf)) >> p.c.shift;
  for (int i0 = 0; i0 < most; i0 += LOOK_U * LOOK_THREADS) {
    const int at = __reduce_min_sync(0xffffffffu, differ(p, r, rf, i0, most, tid, LOOK_THREADS));
    if ((tid & 31) == 0 && at != 0x7fffffff) atomicMin(&mismatch, at);
    __syncthreads();
    if (mismatch != 0x7fffffff) break;
    __syncthreads();
  }
  if (tid == 0) p.shared[r] = min(mismatch, most) << p.c.shift;
}

constexpr int PLAN_THREADS = 1024;
constexpr int CHOOSE_THREADS = 128;

// Saved tokens below which a prefix is not worth an item of its own.
constexpr int MIN_SAVED = 2 * TILE;

// Row r (a warp's); that of a family's lead chooses its prefix: of the members' shared lengths the one that
// saves most when the members that share at least so much take part.  More than 32 members offer 32 of
// theirs.
__device__ __forceinline__ void choose(const Params& p, int r) {
  const int lane = threadIdx.x & 31, l = r / p.Hkv, h = r % p.Hkv;
  const int root = p.root[l], base = p.base[l], count = p.count[l];
  if (root != l || count < 2) {
    if (lane == 0) {
      p.pre_item[r] = 0;
      if (root == l) {
        p.place[r] = -1;
        p.start[r] = 0;
      }
    }
    return;
  }
  const auto row_at = [&](int j) { return p.order[base + j] * p.Hkv + h; };
  const int pick = count <= 32 ? lane : (int)((long long)lane * count / 32);
  const int mine = pick < count ? p.shared[row_at(pick)] : 0;      // (the root's own is 0)
  int others = 0;
  for (int j0 = 0; j0 < count; j0 += 32) {
    const int s = j0 + lane < count ? p.shared[row_at(j0 + lane)] : 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) others += __shfl_sync(0xffffffffu, s, k) >= mine;
  }
  long long best = mine > 0 ? (long long)mine * others : 0;
  int tokens = mine;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const long long b = __shfl_xor_sync(0xffffffffu, best, off);
    const int t = __shfl_xor_sync(0xffffffffu, tokens, off);
    if (b > best || (b == best && t > tokens)) {
      best = b;
      tokens = t;
    }
  }
  if (best < MIN_SAVED) tokens = 0;
  int k = 0;
  for (int j0 = 0; j0 < count; j0 += 32) {
    const int j = j0 + lane, row = j < count ? row_at(j) : 0;
    const bool in = tokens > 0 && j < count && (row == r || p.shared[row] >= tokens);
    const uint32_t b = __ballot_sync(0xffffffffu, in);
    if (j < count) {
      const int at = k + __popc(b & ((1u << lane) - 1));
      p.place[row] = in ? at : -1;
      p.start[row] = in ? tokens : 0;
      if (in) p.list[(size_t)h * p.N + base + at] = row / p.Hkv;
    }
    k += __popc(b);
  }
  if (lane == 0) p.pre_item[r] = k;            // for now: participants
}
// (In the plan's one block, 8 heads' rows were one warp's: 25 us of 4 families' 35.)
__global__ void __launch_bounds__(CHOOSE_THREADS) prefix_choose_kernel(const Params p) {
  wait_prior_grid();
  allow_next_grid();
  const int r = blockIdx.x * (CHOOSE_THREADS / 32) + (threadIdx.x >> 5);
  if (r < p.c.R) choose(p, r);
}

// One block: the items in order with their places in the tile sequence, the CTAs' first items.  A warp
// has a run of the 2 R places (prefixes, then own tokens): it adds its tiles and items up, and writes them
// once the block has added up the warps'.
__device__ void make_plan(const Params& p) {
  constexpr int WARPS = PLAN_THREADS / 32, AHEAD = 4;
  __shared__ long long places_sh[WARPS];
  __shared__ int items_sh[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = p.c.R;
  const int run = (2 * R + 32 * WARPS - 1) / (32 * WARPS) * 32, begin = min(warp * run, 2 * R), end = min(begin + run, 2 * R);
  struct Place {
    int tok0, tok1, nq, n;               // tokens, queries, items
    int width, each;                     // places of a tile, of an item
  };
  const auto place = [&](int i) {
    Place x{0, 0, 0, 0, 2, GAP};
    if (i >= end) return x;
    if (i >= R) {
      x.tok0 = p.start[i - R];
      x.tok1 = prefix::row_len(p, i - R);
      x.nq = p.G;
      x.n = x.tok1 > x.tok0 ? 1 : 0;
    } else {
      const int k = p.pre_item[i], s = p.start[i];
      x.tok1 = k > 0 ? s : 0;
      x.nq = k * p.G;
      x.n = (x.nq + p.qt - 1) / p.qt;
    }
    x.width = prefix::width_of(min(x.nq, p.qt));
    x.each = prefix::tiles_of(x.tok1 - x.tok0) * x.width + GAP;
    return x;
  };
  long long sum = 0;
  int items = 0;
  for (int i0 = begin; i0 < end; i0 += 32 * AHEAD) {
    Place x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) x[k] = place(i0 + 32 * k + lane);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      sum += (long long)x[k].n * x[k].each;
      items += x[k].n;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  items = __reduce_add_sync(0xffffffffu, items);
  if (lane == 0) {
    places_sh[warp] = sum;
    items_sh[warp] = items;
  }
  __syncthreads();
  // (WARPS = 32: a lane for every warp's sum)
  const long long t = places_sh[lane];
  const int n = items_sh[lane];
  long long before = lane < warp ? t : 0;
  sum = t;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, off);
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  // places are counted in 32 bits: 2^29 are 2^28 tiles, 3 s of work (64 KB a tile of 128 16-bit values, at 6 TB/s)
  const bool fits = sum < 1LL << 29;
  if (!fits && threadIdx.x == 0) raise_status(p.status, KVP_ERR_DEVICE_CHECK);
  int at = fits ? (int)before : 0, at_n = __reduce_add_sync(0xffffffffu, lane < warp ? n : 0);
  const int total = fits ? (int)sum : 0;
  items = __reduce_add_sync(0xffffffffu, n);
  // a CTA has at least four places: a tile or more wherever it lies in an item
  const int active = min(total / 4, p.ctas);
  if (threadIdx.x == 0) *p.head = prefix::Head{total, active, total > 0 ? items : 0, 0};
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    Place x = place(i);
    if (!fits) x.n = 0;
    const int at_in = warp_inclusive_scan(x.n * x.each), n_in = warp_inclusive_scan(x.n);
    const int at0 = at + at_in - x.n * x.each, n0 = at_n + n_in - x.n;
    const bool own = i >= R;
    const int r = own ? i - R : i;
    for (int k = 0; k < x.n; ++k) {
      Item it;
      const int gap0 = at0 + k * x.each;
      it.tile0 = gap0 + GAP;
      it.row = r;
      it.tok0 = x.tok0;
      it.tok1 = x.tok1;
      it.q0 = k * p.qt;
      it.nq = min(p.qt, x.nq - k * p.qt);
      it.list = own ? -1 : (r % p.Hkv) * p.N + p.base[r / p.Hkv];
      it.width = x.width;
      p.items[n0 + k] = it;
      // the CTAs whose range begins in it or its gap
      const int hi = paged::cta_of(gap0 + x.each - 1, total, active);
      for (int c = gap0 == 0 ? 0 : paged::cta_of(gap0 - 1, total, active) + 1; c <= hi; ++c) p.cta_item[c] = n0 + k;
    }
    __syncwarp();
    if (i < end) (own ? p.own_item : p.pre_item)[r] = x.n > 0 ? n0 : -1;
    at += __shfl_sync(0xffffffffu, at_in, 31);
    at_n += __shfl_sync(0xffffffffu, n_in, 31);
  }
}

__global__ void __launch_bounds__(PLAN_THREADS) prefix_plan_kernel(const Params p) {
  wait_prior_grid();
  allow_next_grid();
  make_plan(p);
}

// All three at once for few rows of few pages: a cluster whose warps take the rows, and whose first block
// makes the plan.  It takes as long (7 us) as the three, and a host that makes small calls only 2 launches
// less, some 5 us of 27; a warp a row is slower than a block for long tables (112 rows of 1875 pages: 16 us
// for 9).
constexpr int CLUSTER = 8;
constexpr int FEW_ROWS = 128, FEW_SEQS = 128, FEW_PAGES = 256;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(PLAN_THREADS) prefix_few_kernel(const Params p) {
  __shared__ int roots[FEW_SEQS];
  wait_prior_grid();
  allow_next_grid();
  const int lane = threadIdx.x & 31, warps = CLUSTER * PLAN_THREADS / 32;
  const int warp = (threadIdx.x >> 5) * CLUSTER + blockIdx.x;    // neighbouring rows on different SMs
  for (int x = threadIdx.x; x < p.N; x += PLAN_THREADS) roots[x] = root_of(p, x);
  __syncthreads();
  for (int l = warp; l < p.N; l += warps) {
    const int f = roots[l];
    int before = 0, rank = 0, mine = 0;
    for (int x = lane; x < p.N; x += 32) {
      const int y = roots[x];
      before += y < f;
      rank += y == f && x < l;
      mine += y == f;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    rank = __reduce_add_sync(0xffffffffu, rank);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) {
      p.root[l] = f;
      p.order[before + rank] = l;
      p.base[l] = before;
      p.count[l] = mine;
    }
  }
  for (int r = warp; r < p.c.R; r += warps) {
    const int l = r / p.Hkv, f = roots[l], rf = f * p.Hkv + r % p.Hkv;
    if (lane == 0) check_row(p, r);
    const int most = f == l ? 0 : min(prefix::row_len(p, r), prefix::row_len(p, rf)) >> p.c.shift;
    int at = most;
    for (int i0 = 0; i0 < most && at == most; i0 += LOOK_U * 32)
      at = min(at, __reduce_min_sync(0xffffffffu, differ(p, r, rf, i0, most, lane, 32)));
    if (lane == 0) p.shared[r] = at << p.c.shift;
  }
  cluster_sync();
  for (int r = warp; r < p.c.R; r += warps) choose(p, r);
  cluster_sync();
  if (blockIdx.x == 0) make_plan(p);
}

// ------------------------------------------------------------------ fp32 caches
constexpr int F_THREADS = 256;
constexpr int F_QT = 32;                 // queries of an item
constexpr int F_KEYS = 64;               // keys at a time

template <int D>
struct Pf32 {
  static constexpr int ROW = D + 4;                       // padded rows
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + F_QT * ROW;
  static constexpr int OFF_V = OFF_K + F_KEYS * ROW;
  static constexpr int OFF_P = OFF_V + F_KEYS * ROW;      // [F_QT][F_KEYS + 4]
  static constexpr int OFF_M = OFF_P + F_QT * (F_KEYS + 4);   // m, l, factor
  static constexpr int SMEM = (OFF_M + 3 * F_QT) * 4;
};

constexpr int THIN = 16;                 // queries
constexpr int THIN_Q = 4;                // at a time

// A piece with few queries (a row's own tokens): warps take the keys, D / 4 lanes a key and its value, four
// queries in registers.  Every lane group keeps a state of its own, joined in shared memory when the piece
// ends.  (By the kernel below, with 32 queries' places, 1600 rows of 250 own tokens took 300 us.)
template <int D>
__device__ __forceinline__ void thin_piece(const Params& p, const Piece& a, float* sm, int cta) {
  constexpr int LANES = D / 4, KEYS = 32 / LANES, STATES = F_THREADS / LANES, U = 4;
  float* os = sm;                                          // [STATES][THIN_Q][D]
  float2* mls = reinterpret_cast<float2*>(sm + STATES * THIN_Q * D);   // [STATES][THIN_Q]
  const int tid = threadIdx.x, state = tid / LANES, d = tid % LANES * 4;
  const int begin = a.it.tok0 + a.u0 * TILE, end = min(a.it.tok1, a.it.tok0 + a.u1 * TILE);
  const int32_t* table = p.c.table + (size_t)a.it.row * p.c.max_pages;
  const auto query = [&](int i) {
    int g;
    const int r = prefix::query_row(p, a.it, i, g);
    return make_int2(r, g);
  };
  for (int c = 0; c < a.it.nq; c += THIN_Q) {
    float4 q[THIN_Q], o[THIN_Q];
    float m[THIN_Q], l[THIN_Q];
#pragma unroll
    for (int i = 0; i < THIN_Q; ++i) {
      q[i] = o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      m[i] = -INFINITY;
      l[i] = 0.f;
      if (c + i < a.it.nq && !p.zero) {
        const int2 x = query(c + i);
        q[i] = *reinterpret_cast<const float4*>((const float*)p.q + (x.x / p.Hkv) * p.q_stride +
                                                (size_t)((x.x % p.Hkv) * p.G + x.y) * D + d);
        if (p.flip) q[i] = make_float4(-q[i].x, -q[i].y, -q[i].z, -q[i].w);
      }
    }
    // (the warp's first key, so that its lanes take the same steps: the sums are the whole warp's shuffles)
    for (int t0 = begin + tid / 32 * KEYS * U; t0 < end; t0 += STATES * U) {
      float4 k[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * KEYS + tid % 32 / LANES;
        k[u] = v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < end) {
          const int page = table[t >> p.c.shift];
          if (page >= 0 && page < p.c.n_pages) {
            const int64_t at = page * p.c.page_stride + (t & (p.c.ps - 1)) * p.c.token_stride + d;
            k[u] = *reinterpret_cast<const float4*>((const float*)p.c.k + at);
            v[u] = *reinterpret_cast<const float4*>((const float*)p.c.v + at);
          } else {
            raise_status(p.status, KVP_ERR_DEVICE_CHECK);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < THIN_Q; ++i) {
        if (c + i >= a.it.nq) break;
        float s[U], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = fmaf(q[i].x, k[u].x, fmaf(q[i].y, k[u].y, fmaf(q[i].z, k[u].z, q[i].w * k[u].w)));
#pragma unroll
          for (int off = 1; off < LANES; off <<= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], off);
          s[u] = t0 + u * KEYS + tid % 32 / LANES < end ? s[u] * p.c2 : -INFINITY;
          top = fmaxf(top, s[u]);
        }
        const float up = fmaxf(m[i], top), f = paged::weight(m[i], up);
        m[i] = up;
        l[i] *= f;
        o[i] = make_float4(o[i].x * f, o[i].y * f, o[i].z * f, o[i].w * f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float w = paged::weight(s[u], up);
          l[i] += w;
          o[i].x = fmaf(w, v[u].x, o[i].x);
          o[i].y = fmaf(w, v[u].y, o[i].y);
          o[i].z = fmaf(w, v[u].z, o[i].z);
          o[i].w = fmaf(w, v[u].w, o[i].w);
        }
      }
    }
    __syncthreads();                                       // the states before have been read
#pragma unroll
    for (int i = 0; i < THIN_Q; ++i) {
      *reinterpret_cast<float4*>(os + (state * THIN_Q + i) * D + d) = o[i];
      if (d == 0) mls[state * THIN_Q + i] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    const int i = tid / LANES;
    if (i < THIN_Q && c + i < a.it.nq) {
      float M = -INFINITY, L = 0.f;
      for (int k = 0; k < STATES; ++k) M = fmaxf(M, mls[k * THIN_Q + i].x);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < STATES; ++k) {
        const float2 ml = mls[k * THIN_Q + i];
        const float w = paged::weight(ml.x, M);
        const float4 x = *reinterpret_cast<const float4*>(os + (k * THIN_Q + i) * D + d);
        L = fmaf(ml.y, w, L);
        y = make_float4(fmaf(x.x, w, y.x), fmaf(x.y, w, y.y), fmaf(x.z, w, y.z), fmaf(x.w, w, y.w));
      }
      const int2 x = query(c + i);
      const bool first = a.u0 == 0;
      const size_t at = first ? prefix::first_slot(p, a.it.list < 0, x.x, x.y) : prefix::cont_slot(p, cta, c + i);
      *reinterpret_cast<float4*>((first ? p.first_o : p.cont_o) + at * D + d) = y;
      if (d == 0) (first ? p.first_ml : p.cont_ml)[at] = make_float2(M, L);
    }
  }
  __syncthreads();
}

// The items of an fp32 cache (the tensor cores have no fp32 products): 32 queries with 64 keys at a time,
// logits and outputs by FFMA from shared memory.
template <int D>
__global__ void __launch_bounds__(F_THREADS) prefix_f32_kernel(const Params p) {
  using C = Pf32<D>;
  extern __shared__ __align__(16) float sm[];
  float *qs = sm + C::OFF_Q, *ks = sm + C::OFF_K, *vs = sm + C::OFF_V, *ps = sm + C::OFF_P;
  float *ms = sm + C::OFF_M, *ls = ms + F_QT, *fs = ls + F_QT;
  const int tid = threadIdx.x, cta = blockIdx.x;
  wait_prior_grid();
  allow_next_grid();
  prefix::Walk<true> walk(p, cta);
  Piece a;
  while (walk.step(p, a)) {
    if (a.it.nq <= THIN) {
      __syncthreads();
      thin_piece<D>(p, a, sm, cta);
      continue;
    }
    const bool own = a.it.list < 0;
    __syncthreads();
    for (int e = tid; e < F_QT * D / 4; e += F_THREADS) {
      const int i = e / (D / 4), d = e % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < a.it.nq) {
        int g;
        const int r = prefix::query_row(p, a.it, i, g);
        x = *reinterpret_cast<const float4*>((const float*)p.q + (r / p.Hkv) * p.q_stride +
                                             (size_t)((r % p.Hkv) * p.G + g) * D + d);
        if (p.zero) x = make_float4(0.f, 0.f, 0.f, 0.f);
        else if (p.flip) x = make_float4(-x.x, -x.y, -x.z, -x.w);
      }
      *reinterpret_cast<float4*>(qs + i * C::ROW + d) = x;
    }
    if (tid < F_QT) {
      ms[tid] = -INFINITY;
      ls[tid] = 0.f;
    }
    // outputs: four queries by D / 32 values of a thread
    constexpr int W = D / 32;
    float o[4][W];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) o[i][j] = 0.f;
    const int oq = tid / 32 * 4, od = tid % 32 * W;
    const int tok_end = min(a.it.tok1, a.it.tok0 + a.u1 * TILE);
    const int32_t* table = p.c.table + (size_t)a.it.row * p.c.max_pages;
    for (int t0 = a.it.tok0 + a.u0 * TILE; t0 < tok_end; t0 += F_KEYS) {
      __syncthreads();                         // the keys before have been used
      for (int e = tid; e < 2 * F_KEYS * D / 4; e += F_THREADS) {
        const int which = e / (F_KEYS * D / 4), x = e % (F_KEYS * D / 4), i = x / (D / 4), d = x % (D / 4) * 4;
        const int t = t0 + i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < tok_end) {
          const int page = table[t >> p.c.shift];
          if (page >= 0 && page < p.c.n_pages)
            v = *reinterpret_cast<const float4*>((const float*)(which ? p.c.v : p.c.k) + page * p.c.page_stride +
                                                 (t & (p.c.ps - 1)) * p.c.token_stride + d);
          else raise_status(p.status, KVP_ERR_DEVICE_CHECK);
        }
        *reinterpret_cast<float4*>((which ? vs : ks) + i * C::ROW + d) = v;
      }
      __syncthreads();
      // logits: two queries by four keys of a thread, 16 lanes side by side
      const int lq = tid / 16 * 2, lk = tid % 16;
      float s[2][4] = {};
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        const float4 q0 = *reinterpret_cast<const float4*>(qs + lq * C::ROW + d);
        const float4 q1 = *reinterpret_cast<const float4*>(qs + (lq + 1) * C::ROW + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 k = *reinterpret_cast<const float4*>(ks + (lk + 16 * j) * C::ROW + d);
          s[0][j] = fmaf(q0.x, k.x, fmaf(q0.y, k.y, fmaf(q0.z, k.z, fmaf(q0.w, k.w, s[0][j]))));
          s[1][j] = fmaf(q1.x, k.x, fmaf(q1.y, k.y, fmaf(q1.z, k.z, fmaf(q1.w, k.w, s[1][j]))));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = t0 + lk + 16 * j < tok_end ? s[i][j] * p.c2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float old = ms[lq + i], m = fmaxf(old, top);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w = s[i][j] == -INFINITY ? 0.f : fast_exp2(s[i][j] - m);
          ps[(lq + i) * (F_KEYS + 4) + lk + 16 * j] = w;
          sum += w;
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        __syncwarp();
        if (lk == 0) {
          const float f = paged::weight(old, m);
          fs[lq + i] = f;
          ls[lq + i] = fmaf(ls[lq + i], f, sum);
          ms[lq + i] = m;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = fs[oq + i];
#pragma unroll
        for (int j = 0; j < W; ++j) o[i][j] *= f;
      }
#pragma unroll 4
      for (int k = 0; k < F_KEYS; ++k) {
        float w[4], v[W];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ps[(oq + i) * (F_KEYS + 4) + k];
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = vs[k * C::ROW + od + j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < W; ++j) o[i][j] = fmaf(w[i], v[j], o[i][j]);
      }
    }
    for (int i = 0; i < 4; ++i) {
      if (oq + i >= a.it.nq) break;
      int g;
      const int r = prefix::query_row(p, a.it, oq + i, g);
      const size_t at = a.u0 == 0 ? prefix::first_slot(p, own, r, g) : prefix::cont_slot(p, cta, oq + i);
      float* to = (a.u0 == 0 ? p.first_o : p.cont_o) + at * D + od;
#pragma unroll
      for (int j = 0; j < W; ++j) to[j] = o[i][j];
      if (tid % 32 == 0) (a.u0 == 0 ? p.first_ml : p.cont_ml)[at] = make_float2(ms[oq + i], ls[oq + i]);
    }
  }
}

// ------------------------------------------------------------------ join
constexpr int JOIN_THREADS = 256;

// Results of the queries from their parts: `warps` warps of a block have a query, a lane four of its outputs.
template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) prefix_join_kernel(const Params p, int warps) {
  constexpr int LANES = D / 4;                 // of a part
  constexpr int AT_ONCE = 32 / LANES;          // parts a warp reads at once
  __shared__ float4 sum_sh[JOIN_THREADS / 32][LANES];
  // The plan may be read before the parts are there: the kernel before this one has let it go once the plan
  // was made.
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % warps;
  const long long query = (long long)blockIdx.x * (JOIN_THREADS / 32 / warps) + warp / warps;
  const bool live = query < (long long)p.c.R * p.G;
  const int r = live ? (int)(query / p.G) : 0, g = live ? (int)(query % p.G) : 0;
  const int l = r / p.Hkv, h = r % p.Hkv;
  // the parts: [0, n0) of the prefix, then [0, n1) of the row's own tokens, from CTA lo on
  int n0 = 0, n1 = 0, lo0 = 0, lo1 = 0, local = 0;
  if (live) {
    const int4 head = __ldcg((const int4*)p.head);
    const int place = __ldcg(p.place + r), root = __ldcg(p.root + l), own = __ldcg(p.own_item + r);
    int pre = -1;
    if (place >= 0) {
      // (-1: the plan had no place for the call's work, and there is no item at all)
      const int x = place * p.G + g, first = __ldcg(p.pre_item + root * p.Hkv + h);
      pre = first < 0 ? -1 : first + x / p.qt;
      local = x % p.qt;
    }
    const auto span = [&](int item, int& lo) {
      const int4 a = __ldcg((const int4*)(p.items + item)), b = __ldcg((const int4*)(p.items + item) + 1);
      // (tile0, row, tok0, tok1), (q0, nq, list, width); (places, CTAs, ...)
      const int last = a.x + (prefix::tiles_of(a.w - a.z) - 1) * b.w;
      lo = paged::cta_of(a.x, head.x, head.y);
      return paged::cta_of(last, head.x, head.y) - lo + 1;
    };
    if (pre >= 0) n0 = span(pre, lo0);
    if (own >= 0) n1 = span(own, lo1);
  }
  wait_prior_grid();
  const int all = n0 + n1;
  // where part i lies: in the pieces that begin an item, or in those that go on
  const auto at = [&](int i, bool& first) {
    const bool own = i >= n0;
    const int c = own ? i - n0 : i;
    first = c == 0;
    return first ? prefix::first_slot(p, own, r, g) : prefix::cont_slot(p, (own ? lo1 : lo0) + c, own ? g : local);
  };
  const auto ml_of = [&](int i) {
    if (i >= all) return make_float2(-INFINITY, 0.f);
    bool first;
    const size_t x = at(i, first);
    return (first ? p.first_ml : p.cont_ml)[x];
  };
  // every warp finds the maximum and the sum of all parts, and adds up its share of the outputs
  float2 ml = ml_of(lane);
  float M = ml.x;
  for (int i = lane + 32; i < all; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const int hl = lane / LANES, d = lane % LANES;
  for (int i0 = 0; i0 < all; i0 += 32) {
    if (i0 > 0) ml = ml_of(i0 + lane);
    const float w = paged::weight(ml.x, M);
    L = fmaf(ml.y, w, L);
    const int m = min(32, all - i0);
#pragma unroll 4
    for (int k = sub * AT_ONCE; k < m; k += warps * AT_ONCE) {
      const int j = k + hl;
      const float wj = __shfl_sync(0xffffffffu, w, j & 31), mj = __shfl_sync(0xffffffffu, ml.x, j & 31);
      if (j < m && mj != -INFINITY) {
        bool first;
        const size_t x = at(i0 + j, first);
        const float4 y = *reinterpret_cast<const float4*>((first ? p.first_o : p.cont_o) + x * D + 4 * d);
        o.x = fmaf(y.x, wj, o.x);
        o.y = fmaf(y.y, wj, o.y);
        o.z = fmaf(y.z, wj, o.z);
        o.w = fmaf(y.w, wj, o.w);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
#pragma unroll
  for (int off = LANES; off < 32; off <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
  }
  if (warps > 1) {
    if (lane < LANES) sum_sh[warp][lane] = o;
    __syncthreads();
    if (sub != 0) return;
    for (int k = 1; k < warps; ++k) {
      const float4 y = sum_sh[warp + k][d];
      o = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
    }
  }
  if (!live) return;
  const size_t q = (size_t)l * p.Hq + (size_t)h * p.G + g;
  if (lane < LANES) {
    // (the sum, not its reciprocal: an fp32 result keeps the division's half step)
    const float4 y = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x / L, o.y / L, o.z / L, o.w / L);
    T* out = (T*)p.out + q * D + 4 * d;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(out) = y;
    } else {
      paged::Params as{};
      as.out = p.out;
      paged::store_out4<T>(as, q * D + 4 * d, y);
    }
  }
  if (lane == 0 && p.lse) p.lse[q] = L == 0.f ? -INFINITY : (M + log2f(L)) * KVP_LN2;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

size_t layout(const PagedView& c, int G, int h_kv, Params* p, void* ws) {
  char* base = (char*)ws;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    char* x = base ? base + at : nullptr;
    at += align256(bytes);
    return x;
  };
  const size_t R = c.R, N = c.R / h_kv, D = c.D;
  const int sms = sm_count();
  p->N = (int)N;
  p->qt = c.dtype == KVP_F32 ? F_QT : 256 / G * G;
  p->ctas = c.dtype == KVP_F32 ? 2 * sms : sms;
  const size_t items = 2 * R + R * G / p->qt + 1;
  p->root = (int*)take(N * 4);
  p->order = (int*)take(N * 4);
  p->base = (int*)take(N * 4);
  p->count = (int*)take(N * 4);
  p->shared = (int*)take(R * 4);
  p->start = (int*)take(R * 4);
  p->place = (int*)take(R * 4);
  p->list = (int*)take(R * 4);
  p->pre_item = (int*)take(R * 4);
  p->own_item = (int*)take(R * 4);
  p->items = (Item*)take(items * sizeof(Item));
  p->head = (prefix::Head*)take(sizeof(prefix::Head));
  p->cta_item = (int*)take(p->ctas * 4);
  p->first_ml = (float2*)take(2 * R * G * sizeof(float2));
  p->first_o = (float*)take(2 * R * G * D * 4);
  p->cont_ml = (float2*)take((size_t)p->ctas * p->qt * sizeof(float2));
  p->cont_o = (float*)take((size_t)p->ctas * p->qt * D * 4);
  const bool keeps = c.dtype == KVP_F16 && c.cap > prefix::SEGMENT * TILE;
  p->kept = keeps ? (float*)take((size_t)p->ctas * 256 * prefix::kept_row(c.D) * 4) : nullptr;
  return at;
}

template <int D>
cudaError_t run_f32(const Params& p, cudaStream_t st) {
  const auto kern = prefix_f32_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pf32<D>::SMEM);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_with_pdl(kern, dim3((unsigned)p.ctas), dim3(F_THREADS), Pf32<D>::SMEM, st, p);
}

template <typename T, int D>
cudaError_t run(const Params& p, cudaStream_t st) {
  cudaError_t e;
  const int pages = p.c.max_pages < p.c.n_pages ? p.c.max_pages : p.c.n_pages;
  if (p.c.R <= FEW_ROWS && p.N <= FEW_SEQS && pages <= FEW_PAGES) {
    count_launches(1);
    e = launch_with_pdl(prefix_few_kernel, dim3(CLUSTER), dim3(PLAN_THREADS), 0, st, p);
  } else {
    count_launches(3);
    constexpr int PER = CHOOSE_THREADS / 32;
    e = launch_with_pdl(prefix_look_kernel, dim3((unsigned)p.c.R), dim3(LOOK_THREADS), 0, st, p);
    if (e != cudaSuccess) return e;
    e = launch_with_pdl(prefix_choose_kernel, dim3((unsigned)((p.c.R + PER - 1) / PER)), dim3(CHOOSE_THREADS), 0, st, p);
    if (e != cudaSuccess) return e;
    e = launch_with_pdl(prefix_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, p);
  }
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(T) == 2) e = launch_paged_prefix_tc(p, st);
  else e = run_f32<D>(p, st);
  if (e != cudaSuccess) return e;
  // A query can have a part or two from every CTA: as many warps for each as let the blocks (eight an SM) run
  // at once, up to eight.
  const long long queries = (long long)p.c.R * p.G;
  int warps = JOIN_THREADS / 32;
  while (warps > 1 && queries * warps > 64LL * sm_count()) warps >>= 1;
  const int per = JOIN_THREADS / 32 / warps;
  count_launches(1);
  return launch_with_pdl(prefix_join_kernel<T, D>, dim3((unsigned)((queries + per - 1) / per)), dim3(JOIN_THREADS), 0,
                         st, p, warps);
}

}  // namespace

size_t paged_prefix_workspace(const PagedView& c, int h_q, int h_kv) {
  Params p{};
  return layout(c, h_q / h_kv, h_kv, &p, nullptr);
}

cudaError_t launch_paged_prefix_decode(const PagedView& c, const PagedPrefixArgs& a, void* ws, int* status,
                                       cudaStream_t st) {
  Params p{};
  p.c = c;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.lead = a.lead;
  p.Hq = a.h_q;
  p.Hkv = a.h_kv;
  p.G = a.h_q / a.h_kv;
  p.c2 = (float)(std::fabs(a.scale) * 1.4426950408889634);
  p.flip = a.scale < 0;
  p.zero = p.c2 == 0.f;
  if (p.zero) p.c2 = 1.f;
  p.out = a.out;
  p.lse = a.lse;
  p.status = status;
  layout(c, p.G, a.h_kv, &p, ws);
  if (c.dtype == KVP_BF16) return c.D == 128 ? run<__nv_bfloat16, 128>(p, st) : run<__nv_bfloat16, 64>(p, st);
  if (c.dtype == KVP_F16) return c.D == 128 ? run<__half, 128>(p, st) : run<__half, 64>(p, st);
  return c.D == 128 ? run<float, 128>(p, st) : run<float, 64>(p, st);
}

}  // namespace kvp
