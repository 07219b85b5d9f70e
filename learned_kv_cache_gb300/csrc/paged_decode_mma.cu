// One-token decode attention over the pages of a bf16 / f16 cache.
//
//   out = sum_t softmax_t(scale * q . k_t) v_t,  lse = ln sum_t exp(scale * q . k_t)
//
// 4 G D flop per 4 D bytes of K and V: bound by HBM for every group size, so the kernel is built
// around the copies.
//
//  * Two CTAs per SM, each with an equal share of all rows' 64-key tiles (paged_decode.cuh).
//  * A producer warp looks 32 tiles ahead at a time: one lane per tile finds the tile's row (lengths
//    and a warp scan) and fetches its page ids, so that the two dependent reads cost one latency per
//    32 tiles, and they are issued while the previous tiles are still in flight.  The tiles then come
//    by TMA, one box per page, 64-column half and tensor, each issued by a lane of its own; the
//    128-byte swizzle keeps the ldmatrix reads free of bank conflicts.  The query rows ride along with
//    the first tile of a row.
//  * Four consumer warps own 16 keys of every tile.  S^T = K Q^T and O^T += V^T P^T are m16n8k16
//    products with keys or head dims in M and the group padded to N = 8 or 16.  P enters the second
//    product as a sum of 16-bit parts, two for f16 (22 bits) and three for bf16 (24 bits): with two,
//    bf16 would leave 2^-17 of every weight in an fp32 output.
//  * f16 weights are kept 2^14 above the softmax's own (the reference is the maximum minus 14): below
//    2^-14 an f16 part loses bits, and beside a sink token that is where all the others' weights lie.
//    What the two parts leave of a weight is 2^-22 of it, and never more than 2^-39 of the row's largest.
//  * The tensor cores' running sum drops bits at every step, always towards zero; over the hundreds of
//    tiles of a long row that would show, and in the logits of a sink token too.  Each step of 16 is
//    summed on its own and added in fp32; a logit keeps what its last sum and its scaling round away
//    (half a step of a sink's logit of 20 is 1e-6 of its weight).
//  * Measured: 56 rows x 120000 tokens of 128 f16 values 490 us (7.0 TB/s), x 4096 26 us with the join (6
//    us to the first tiles: lengths, page ids, K and V are three dependent reads; 3 us of join), 8 rows x
//    131072 bf16 84 us (6.4 TB/s).
//  * Slots behind a row's end may hold anything.  Their logits are replaced by -inf, and their V is
//    cleared in the fragments of the row's last tile: 0 * NaN would be NaN.
#include <type_traits>

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "mma_ptx.cuh"
#include "paged_decode.cuh"
#include "tc_ptx.cuh"

namespace kvp {
namespace {

using paged::Params;
using paged::Range;
using paged::TILE;

constexpr int PM_CWARPS = 4;
constexpr int PM_THREADS = 32 * (PM_CWARPS + 1);

template <int D, int GP>
struct Pm {
  static constexpr int HALVES = D / 64;                    // 128-byte swizzle spans per token
  static constexpr int HALF_BYTES = TILE * 128;
  static constexpr int TILE_BYTES = HALVES * HALF_BYTES;   // K (or V) of a tile
  static constexpr int Q_ROW = D * 2 + 16;                 // padded: the fragment loads hit distinct banks
  static constexpr int Q_BYTES = GP * Q_ROW;
  static constexpr int STAGES = D == 128 ? (GP == 8 ? 3 : 2) : (GP == 8 ? 5 : 4);
  static constexpr int KSTEPS = D / 16;
  static constexpr int NT = GP / 8;                        // n8 tiles of query heads
  static constexpr int OSTR = D + 4;                       // padded rows of the merge scratch
  static constexpr int OFF_Q = STAGES * 2 * TILE_BYTES;
  static constexpr int OFF_O = OFF_Q + STAGES * Q_BYTES;   // [2][GP][OSTR]
  static constexpr int OFF_ML = OFF_O + 2 * GP * OSTR * 4; // [2 rows in turn][m, l][4 warps][GP]
  static constexpr int OFF_INV = OFF_ML + 2 * 2 * PM_CWARPS * GP * 4;   // [2 rows in turn][GP]
  static constexpr int OFF_BAR = OFF_INV + 2 * GP * 4;
  static constexpr int OFF_FLAG = OFF_BAR + 16 * STAGES;
  static constexpr int OFF_SCAN = OFF_FLAG + 16;
  static constexpr int SMEM = OFF_SCAN + (36 + PM_THREADS / 2) * 4 + 1024;   // + alignment slack
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
};

// Shared address of the 16-byte chunk holding (key, d..d+7) of a swizzled tile.
__device__ __forceinline__ uint32_t swz(uint32_t tile, int key, int d) {
  return tile + (d >> 6) * (TILE * 128) + key * 128 + ((((d & 63) >> 3) ^ (key & 7)) << 4);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// The next tiles of a CTA, one per lane: row, tile within the row, the row's length, the page ids.
struct Ahead {
  int row, tile, n, count;     // count: tiles in this look (the same in every lane)
  int page[4];
};

// Looks at up to 32 tiles from (row, tile) on, and moves (row, tile) behind them.
__device__ __forceinline__ Ahead look_ahead(const Params& p, int& row, int& tile, int left) {
  const int lane = threadIdx.x & 31;
  Ahead a{};
  while (left > 0 && row < p.c.R) {
    const int n = row + lane < p.c.R ? paged::row_len(p, row + lane) : 0;
    int t = paged::tiles_of(n);
    if (lane == 0) t -= tile;
    const int upto = warp_inclusive_scan(t);
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    if (all == 0) {              // 32 rows without (further) tiles
      row += 32;
      tile = 0;
      continue;
    }
    a.count = min(min(all, left), 32);
    int j = 0;                   // rows before this lane's tile
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (__shfl_sync(0xffffffffu, upto, j + step - 1) <= lane) j += step;
    const int before = __shfl_sync(0xffffffffu, upto, j > 0 ? j - 1 : 0);
    a.n = __shfl_sync(0xffffffffu, n, j);
    a.row = row + j;
    a.tile = j > 0 ? lane - before : lane + tile;
    if (lane < a.count) {
      const int32_t* table = p.c.table + (size_t)a.row * p.c.max_pages;
      const int first = (a.tile * TILE) >> p.c.shift, held = (a.n + p.c.ps - 1) >> p.c.shift;
      const int most = p.c.ps >= TILE ? 1 : TILE >> p.c.shift;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.page[i] = -1;
        if (i < most && first + i < held) {
          a.page[i] = table[first + i];
          if (a.page[i] < 0 || a.page[i] >= p.c.n_pages) {
            raise_status(p.status, KVP_ERR_DEVICE_CHECK);
            a.page[i] = p.c.n_pages;     // outside the tensor map: zeros
          }
        }
      }
    }
    const int last = a.count - 1;
    const int lr = __shfl_sync(0xffffffffu, a.row, last), lt = __shfl_sync(0xffffffffu, a.tile, last) + 1;
    const int ln = __shfl_sync(0xffffffffu, a.n, last);
    row = lt == paged::tiles_of(ln) ? lr + 1 : lr;
    tile = lt == paged::tiles_of(ln) ? 0 : lt;
    break;
  }
  return a;
}

template <typename T, int D, int GP>
__global__ void __launch_bounds__(PM_THREADS, 2)
    paged_decode_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const T* __restrict__ q, const Params p) {
  using C = Pm<D, GP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t bar_full = sbase + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
  int* scan_sh = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 1);
      ptx::mbar_init(bar_empty + 8 * s, PM_CWARPS);
    }
    flags[0] = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  wait_prior_grid();
  const Range g = paged::find_range(p, cta, scan_sh);     // also orders the barriers' initialisation
  // the consumers have time until the first tiles land
  if (warp < PM_CWARPS) paged::empty_rows<T, D>(p, cta, PM_CWARPS * 32);
  if (cta >= g.active) return;

  if (warp == PM_CWARPS) {
    // ------------------------------------------------------------ producer
    const int box = min(p.c.ps, TILE);                     // rows of a box
    const int per_page = 2 * C::HALVES;                    // boxes of a page (or of a tile inside one)
    int row = g.row, tile = g.tile, left = g.end - g.begin, li = 0;
    bool ok = true;
    Ahead a = look_ahead(p, row, tile, left);
    while (a.count > 0 && ok) {
      left -= a.count;
      Ahead next{};
      for (int i = 0; i < a.count; ++i) {
        const int r = __shfl_sync(0xffffffffu, a.row, i), u = __shfl_sync(0xffffffffu, a.tile, i);
        const int n = __shfl_sync(0xffffffffu, a.n, i);
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) page[k] = __shfl_sync(0xffffffffu, a.page[k], i);
        const int s = li % C::STAGES, use = li / C::STAGES;
        if (use > 0) ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_empty + 8 * s, (use - 1) & 1, flags, p.status));
        if (!ok) break;
        const uint32_t bar = bar_full + 8 * s;
        const int pages = min((n - u * TILE + box - 1) / box, TILE / box);
        const bool with_q = u == 0 || li == 0;
        const int boxes = pages * per_page;
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar, boxes * box * 128 + (with_q ? p.G * D * 2 : 0));
        __syncwarp();
        if (lane < boxes) {
          const int k = lane / per_page, h = (lane >> 1) % C::HALVES, v = lane & 1;
          const int pg = k == 0 ? page[0] : k == 1 ? page[1] : k == 2 ? page[2] : page[3];
          const uint32_t dst = sbase + (2 * s + v) * C::TILE_BYTES + h * C::HALF_BYTES + k * box * 128;
          ptx::tma_load_3d(dst, v ? &tmV : &tmK, bar, 64 * h, k == 0 ? (u * TILE) & (p.c.ps - 1) : 0, pg);
        }
        if (with_q && lane >= 16 && lane - 16 < p.G)       // boxes take 16 lanes at most
          bulk_load(sbase + C::OFF_Q + s * C::Q_BYTES + (lane - 16) * C::Q_ROW,
                    q + (r / p.Hkv) * p.q_stride + (size_t)((r % p.Hkv) * p.G + lane - 16) * D, D * 2, bar);
        __syncwarp();
        ++li;
        if (i == min(C::STAGES, a.count) - 1) next = look_ahead(p, row, tile, left);
      }
      a = next;
    }
    // every copy must land before the CTA can exit
    for (int j = max(0, li - C::STAGES); j < li; ++j)
      ptx::mbar_wait_drain(bar_full + 8 * (j % C::STAGES), (j / C::STAGES) & 1, p.status);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int hg = lane >> 2, t = lane & 3;
  constexpr int SPLIT = std::is_same<T, __half>::value ? 2 : 3;   // 16-bit parts of a weight
  constexpr float ABOVE = std::is_same<T, __half>::value ? 14.f : 0.f;   // log2 of the weights' scale
  uint32_t qb[C::NT][C::KSTEPS][2];
  float m2[C::NT][2], ls[C::NT][2], lost[C::NT][2], o[C::NT][C::KSTEPS][4];   // lost: what ls rounds off
  int li = 0, turn = 0;

  // Row r, tiles [u0, u1) of its nt: merge the warps' states; the whole row's result, or a partial.
  const auto finish = [&](int r, int n, int u0, int u1, int nt) {
    float* sm_m = reinterpret_cast<float*>(smem + C::OFF_ML) + turn * 2 * PM_CWARPS * GP;
    float* sm_l = sm_m + PM_CWARPS * GP;
    float* sm_o = reinterpret_cast<float*>(smem + C::OFF_O);
    float* sm_inv = reinterpret_cast<float*>(smem + C::OFF_INV) + turn * GP;
    turn ^= 1;                   // the other half may still be read
    const bool whole = u0 == 0 && u1 == nt;
    float* part = p.part + ((size_t)cta * 2 + (u0 > 0 ? 0 : 1)) * p.pstride;
    const size_t head0 = (size_t)(r / p.Hkv) * p.Hq + (size_t)(r % p.Hkv) * p.G;
#pragma unroll
    for (int x = 0; x < C::NT; ++x) {
      float l0 = ls[x][0] + lost[x][0], l1 = ls[x][1] + lost[x][1];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
      }
      if (hg == 0) {
        sm_m[warp * GP + 8 * x + 2 * t] = m2[x][0];
        sm_m[warp * GP + 8 * x + 2 * t + 1] = m2[x][1];
        sm_l[warp * GP + 8 * x + 2 * t] = l0;
        sm_l[warp * GP + 8 * x + 2 * t + 1] = l1;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(PM_CWARPS * 32) : "memory");
    if (threadIdx.x < p.G) {     // a head's merged state, while warps 2 and 3 write below
      const int h = threadIdx.x;
      const float M = fmaxf(fmaxf(sm_m[h], sm_m[GP + h]), fmaxf(sm_m[2 * GP + h], sm_m[3 * GP + h]));
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < PM_CWARPS; ++w) L = fmaf(sm_l[w * GP + h], paged::weight(sm_m[w * GP + h], M), L);
      if (whole) {
        const float l2 = L == 0.f ? -INFINITY : M + log2f(L);
        if (p.lse) p.lse[head0 + h] = l2 * KVP_LN2;
        if (p.lse2) p.lse2[(size_t)r * GP + h] = l2;
        sm_l[h] = l2;            // only this thread reads the head's sums
      } else {
        part[h] = M;
        part[GP + h] = L;
      }
      sm_inv[h] = !whole ? 1.f : L == 0.f ? 0.f : 1.f / L;
    }
    // warps 2 and 3 hand their scaled outputs to warps 0 and 1
    float* ow = sm_o + (warp & 1) * GP * C::OSTR;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      if ((warp >= 2) == (pass == 0)) {
#pragma unroll
        for (int x = 0; x < C::NT; ++x) {
          float w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int h = 8 * x + 2 * t + i;
            const float M = fmaxf(fmaxf(sm_m[h], sm_m[GP + h]), fmaxf(sm_m[2 * GP + h], sm_m[3 * GP + h]));
            w[i] = paged::weight(m2[x][i], M);
          }
#pragma unroll
          for (int db = 0; db < C::KSTEPS; ++db)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* y = ow + (8 * x + 2 * t + (i & 1)) * C::OSTR + 16 * db + hg + (i >> 1) * 8;
              const float z = o[x][db][i] * w[i & 1];
              *y = pass == 0 ? z : *y + z;
            }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(PM_CWARPS * 32) : "memory");
    }
    for (int e = 4 * threadIdx.x; e < p.G * D; e += 4 * PM_CWARPS * 32) {
      const int h = e / D, d = e % D;
      const float4 a = *reinterpret_cast<const float4*>(sm_o + h * C::OSTR + d);
      const float4 b = *reinterpret_cast<const float4*>(sm_o + (GP + h) * C::OSTR + d);
      const float f = sm_inv[h];
      const float4 z = make_float4((a.x + b.x) * f, (a.y + b.y) * f, (a.z + b.z) * f, (a.w + b.w) * f);
      if (whole) paged::store_out4<T>(p, head0 * D + e, z);
      else *reinterpret_cast<float4*>(part + 2 * GP + e) = z;
    }
    if (p.whole && p.logits) paged::add_row_scores<GP>(p, r, threadIdx.x, n, PM_CWARPS * 32, sm_l);
  };

  int r = g.row, u0 = g.tile, n = paged::row_len(p, r);
  for (int x = g.begin; x < g.end;) {
    const int nt = paged::tiles_of(n);
    const int next_n = r + 1 < p.c.R ? paged::row_len(p, r + 1) : 0;      // in flight during this row
    const int u1 = min(nt, u0 + (g.end - x));
#pragma unroll
    for (int y = 0; y < C::NT; ++y) {
      m2[y][0] = m2[y][1] = -INFINITY;
      ls[y][0] = ls[y][1] = lost[y][0] = lost[y][1] = 0.f;
#pragma unroll
      for (int db = 0; db < C::KSTEPS; ++db) o[y][db][0] = o[y][db][1] = o[y][db][2] = o[y][db][3] = 0.f;
    }
    for (int u = u0; u < u1; ++u, ++li) {
      const int s = li % C::STAGES;
      // After a timeout every warp walks on without computing, so the barriers of finish() are still
      // reached by all four.
      if (!ptx::mbar_wait(bar_full + 8 * s, (li / C::STAGES) & 1, flags, p.status)) continue;
      if (u == u0) {
        const uint8_t* qs = smem + C::OFF_Q + s * C::Q_BYTES;
#pragma unroll
        for (int y = 0; y < C::NT; ++y) {
          const bool live = 8 * y + hg < p.G;
          const uint8_t* qr = qs + (8 * y + hg) * C::Q_ROW;
#pragma unroll
          for (int ks = 0; ks < C::KSTEPS; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qb[y][ks][i] = live ? *reinterpret_cast<const uint32_t*>(qr + (16 * ks + 8 * i + 2 * t) * 2) : 0u;
        }
      }
      const uint32_t kt = sbase + 2 * s * C::TILE_BYTES, vt = kt + C::TILE_BYTES;
      const int kw = warp * 16, key0 = u * TILE + kw + hg;
      const bool v0 = key0 < n, v1 = key0 + 8 < n;
      const int j = lane >> 3;
      if (u * TILE + kw < n) {
        // the steps of 16 in a tree, its last sum with what it rounds away
        float half[2][C::NT][4], sc[C::NT][4], low[C::NT][4];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int k2 = 0; k2 < C::KSTEPS / 4; ++k2) {
            float pair[C::NT][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int ks = z * (C::KSTEPS / 2) + 2 * k2 + k;
              uint32_t a[4];
              ldsm_x4(swz(kt, kw + (j & 1) * 8 + (lane & 7), 16 * ks + (j >> 1) * 8), a);
#pragma unroll
              for (int y = 0; y < C::NT; ++y) {
                pair[y][k][0] = pair[y][k][1] = pair[y][k][2] = pair[y][k][3] = 0.f;
                mma16816<T>(pair[y][k], a, qb[y][ks][0], qb[y][ks][1]);
              }
            }
#pragma unroll
            for (int y = 0; y < C::NT; ++y)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x = pair[y][0][i] + pair[y][1][i];
                half[z][y][i] = k2 == 0 ? x : half[z][y][i] + x;
              }
          }
        uint32_t b[C::NT][SPLIT][2];
        bool grew = false;
        float nm[C::NT][2];
#pragma unroll
        for (int y = 0; y < C::NT; ++y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[y][i] = paged::base2(p, half[0][y][i], half[1][y][i], low[y][i]);
            if (!(i < 2 ? v0 : v1)) sc[y][i] = -INFINITY;
          }
          if (p.logits) {
            float* lg = p.logits + ((size_t)r * p.c.cap + key0) * GP + 8 * y + 2 * t;
            if (v0) *reinterpret_cast<float2*>(lg) = make_float2(sc[y][0], sc[y][1]);
            if (v1) *reinterpret_cast<float2*>(lg + 8 * GP) = make_float2(sc[y][2], sc[y][3]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float z = fmaxf(sc[y][i], sc[y][i + 2]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, off));
            nm[y][i] = fmaxf(m2[y][i], z - ABOVE);
            grew |= nm[y][i] > m2[y][i];
          }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int y = 0; y < C::NT; ++y) {
            const float f0 = paged::weight(m2[y][0], nm[y][0]), f1 = paged::weight(m2[y][1], nm[y][1]);
            // nothing but NaN so far (sum NaN, maximum -inf): 0 * NaN keeps it
            ls[y][0] *= f0;
            ls[y][1] *= f1;
            lost[y][0] *= f0;
            lost[y][1] *= f1;
#pragma unroll
            for (int db = 0; db < C::KSTEPS; ++db) {
              o[y][db][0] *= f0;
              o[y][db][1] *= f1;
              o[y][db][2] *= f0;
              o[y][db][3] *= f1;
            }
            m2[y][0] = nm[y][0];
            m2[y][1] = nm[y][1];
          }
        }
#pragma unroll
        for (int y = 0; y < C::NT; ++y) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = sc[y][i] == -INFINITY ? 0.f : fast_exp2((sc[y][i] - m2[y][i & 1]) + low[y][i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float add = w[i] + w[i + 2], sum = ls[y][i] + add;
            lost[y][i] += add - (sum - ls[y][i]);
            ls[y][i] = sum;
          }
          // P^T as B fragments: movmatrix turns the [key][head] layout of the first product's result
          // into the [head][key] layout that the second one reads
#pragma unroll
          for (int k = 0; k < SPLIT; ++k) {
            float k0, k1, k2, k3;
            b[y][k][0] = movm_t(pack_split<T>(w[0], w[1], k0, k1));
            b[y][k][1] = movm_t(pack_split<T>(w[2], w[3], k2, k3));
            w[0] -= k0;
            w[1] -= k1;
            w[2] -= k2;
            w[3] -= k3;
          }
        }
        // keys 2t, 2t+1 (and 8 further) of the fragments below: clear those behind the row's end
        const int left = n - u * TILE - kw;
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (left < 16) {
          keep0 = (2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u);
          keep1 = (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int db = 0; db < C::KSTEPS; ++db) {
          uint32_t a[4];
          ldsm_x4_t(swz(vt, kw + (j >> 1) * 8 + (lane & 7), 16 * db + (j & 1) * 8), a);
          a[0] &= keep0;
          a[1] &= keep0;
          a[2] &= keep1;
          a[3] &= keep1;
#pragma unroll
          for (int y = 0; y < C::NT; ++y) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = SPLIT - 1; k >= 0; --k) mma16816<T>(sum, a, b[y][k][0], b[y][k][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[y][db][i] += sum[i];
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_empty + 8 * s);
    }
    if (x + (u1 - u0) >= g.end) allow_next_grid();   // the join kernel's CTAs may take their places
    if (u1 > u0) finish(r, n, u0, u1, nt);
    x += u1 - u0;
    ++r;
    u0 = 0;
    n = next_n;
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

bool pool_map(CUtensorMap* m, const PagedView& c, const void* base) {
  const EncodeTiledFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)c.D, (cuuint64_t)c.ps, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)c.token_stride * 2, (cuuint64_t)c.page_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(c.ps < TILE ? c.ps : TILE), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, c.dtype == KVP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int GP>
cudaError_t run(const Params& p, const void* q, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!pool_map(&tk, p.c, p.c.k) || !pool_map(&tv, p.c, p.c.v)) return cudaErrorInvalidValue;
  const auto kern = paged_decode_mma_kernel<T, D, GP>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pm<D, GP>::SMEM);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_with_pdl(kern, dim3((unsigned)p.ctas), dim3(PM_THREADS), Pm<D, GP>::SMEM, st, tk, tv, (const T*)q, p);
}

}  // namespace

cudaError_t launch_paged_decode_mma(const paged::Params& p, const void* q, cudaStream_t st) {
#define KVP_PM(TT, DD) return p.G <= 8 ? run<TT, DD, 8>(p, q, st) : run<TT, DD, 16>(p, q, st)
  if (p.c.dtype == KVP_BF16) {
    if (p.c.D == 128) KVP_PM(__nv_bfloat16, 128);
    KVP_PM(__nv_bfloat16, 64);
  }
  if (p.c.D == 128) KVP_PM(__half, 128);
  KVP_PM(__half, 64);
#undef KVP_PM
}

}  // namespace kvp
