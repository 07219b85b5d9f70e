// The items of shared-prefix decode on the tensor cores (bf16 / f16 caches).
//
//   S = Q K^T,  P = 2^(c S - m),  l = sum P,  O = P V   for up to 256 queries and 128 keys at a time
//
// 4 D flop per query and key against 4 D bytes per key: with few queries bound by HBM, with 256 by the tensor
// cores (QK^T and two parts of P V take 3700 cycles a tile of D 128, its keys and values 2790 in HBM).
// Measured: 32 rows of 32768 tokens without a family at 6.2 TB/s; 32 sequences on one prompt of 32768 tokens,
// 32 / 8 heads, with up to 1000 own tokens each in 45 us of the call's 60 (4.5 TB/s).
//
//  * One CTA per SM.  Warp 0 copies keys and values: K and V of a tile are a unit each of a ring, one TMA
//    box per page (or 128 tokens of one) and 64-column half, in the order in which the products use them.
//    Warp 1 issues the products, as a whole warp up to the elected thread's instructions: with one thread
//    walking alone, its descriptors were not known to be uniform and an instruction took 90 cycles to
//    issue, as long as it ran.  Warp 2 clears the slots behind an item's last token, warp 3 copies the
//    next piece's queries.  Sixteen warps have the softmax.
//  * Queries 0..127 and 128..255 are two groups of eight warps.  A thread has a query (a TMEM lane) and 64
//    of a tile's keys: scores come from TMEM (the second 32 again for their weights: 64 in registers spill),
//    and the weights go back in their place as the first operand of P V.  Outputs stay in TMEM until the
//    piece, or in f16 a segment of it, ends.
//  * The tensor cores' running sum drops bits at every step of 16 keys, always towards zero: 0.84 * 2^-24 of it
//    each as measured, two steps for 16 keys.  131072 tokens in one CTA lost 4e-4 (8e-4 with more than 128
//    queries): 0.8 to 1.7 of f16's half steps, 0.1 to 0.2 of bf16's.  So an f16 sum takes SEGMENT tiles, which
//    lose a tenth of a half step, and is then added to fp32 sums in memory, which L2 holds.  It costs rows of
//    that length 3 to 5 %, and by its instructions every f16 call 1 to 4 % (32 answers 61.1 -> 63.4 us; inside
//    the loop over the tiles it cost bf16 and f16 as much again), and bf16 does without.
//  * More than 128 queries: each group has its own, and both take every tile.  Up to 128: both have the
//    same, take the tiles in turn, and put their results together when the piece ends; a piece of one tile
//    is one group's, and the other goes on with the next.  Either way one group's softmax runs beside the
//    other's products.
//  * V lies [key][dim] in memory, so it is the second operand in its MN-major form; nothing is transposed.
//  * P enters the product as the sum of two 16-bit parts: 16 (bf16) or 22 (f16) bits of every weight, 1/256 or
//    1/2048 of the half step that an output is rounded by; with one part bf16 outputs would be 1.4 times as far
//    off.  The outputs come in the cache's type.
//  * f16 weights are kept 2^14 above the softmax's own (their reference is the maximum less 14): a part has
//    nothing below 2^-24, and beside a sink token that is where all the others' weights lie.  Without that the
//    tokens 17 nats below a sink lost 20 % of their sum, at 18 nats half or all of it.  (The smaller lag costs
//    prefixes with 256 queries 1.5 %: 32768 tokens, 8 heads 61.9 -> 62.7 us; the others nothing.)
//  * The running maximum may lag by a factor of 2^8 (f16: 2^1.5, as weights then reach 2^15.5 of its 2^16)
//    before the outputs are scaled again, so most tiles move nothing.
//  * Slots behind the last token of an item may hold anything: their logits become -inf, and their V is
//    cleared in shared memory (0 * NaN would be NaN).
#include <type_traits>

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "paged_prefix.cuh"
#include "tc_ptx.cuh"

namespace kvp {
namespace {

using prefix::Item;
using prefix::Params;
using prefix::Piece;
using prefix::TILE;

constexpr int X_THREADS = 640;
constexpr int ROWS = 128;                // queries of a group
constexpr int RUN = 8;                   // sequences whose queries are copied at once

// Log2 of what weights are kept above the softmax's own, and of how far the maximum may lag.  f16 parts end at
// 2^-24 and 2^16: what a pair of them leaves is 2^-22 of a weight, and never more than 2^-39 of the row's largest.
// bf16 has the range of a float.
template <typename T>
constexpr float ABOVE = std::is_same<T, __half>::value ? 14.f : 0.f;
// Whether a piece's sums are taken in segments, and of how many of a group's tiles.
template <typename T>
constexpr bool CUT = std::is_same<T, __half>::value;
using prefix::SEGMENT;

template <typename T>
constexpr float LAG = std::is_same<T, __half>::value ? 1.5f : 8.f;

template <int D>
struct Px {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = TILE * 128;            // 64 columns of 128 tokens
  static constexpr int UNIT = HALVES * HALF_BYTES;         // K or V of a tile
  static constexpr int UNITS = D == 128 ? 5 : 10;
  static constexpr int Q_HALF = 2 * ROWS * 128;            // 64 columns of 256 queries
  static constexpr int OFF_RING = HALVES * Q_HALF;
  static constexpr int OFF_X = OFF_RING + UNITS * UNIT;    // float2 [2 groups][ROWS]
  static constexpr int OFF_BAR = OFF_X + 2 * ROWS * 8;
  static constexpr int OFF_FLAG = OFF_BAR + 8 * (3 * UNITS + 10);
  static constexpr int SMEM = OFF_FLAG + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
};

// TMEM columns: scores (then weights) and outputs of the two groups.
constexpr int TM_S = 0, TM_O = 256, TM_COLS = 512;

__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t addr, uint32_t lead_bytes) {
  // 64 columns x 8 rows are an atom of 1024 bytes; the next 8 rows follow it, the next 64 columns lie
  // lead_bytes on
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lead_bytes >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Uses of r stay behind the wait for its loads.
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Lane 0's value, known to the compiler as the same in the whole warp.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void bar_sync(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void store32(float* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
               "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// A query's 16 outputs of a piece.
__device__ __forceinline__ void store_part(float* p, const uint32_t (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 8) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(x[i + j]);
    store32(p + i, f);
  }
}

// A pair of weights as 16-bit values, and what those leave of it.
__device__ __forceinline__ void split(__nv_bfloat16, uint64_t w, uint32_t& hi, uint32_t& lo) {
  float a, b;
  unpack2(w, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  unpack2(fsub2(w, pack2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u))), a, b);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void split(__half, uint64_t w, uint32_t& hi, uint32_t& lo) {
  float a, b;
  unpack2(w, a, b);
  const __half2 h = __floats2half2_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const float2 f = __half22float2(h);
  unpack2(fsub2(w, pack2(f.x, f.y)), a, b);
  const __half2 r = __floats2half2_rn(a, b);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

// The ring's units in the order in which warp 1 uses them: before a group's scores of its next tile come
// the outputs of its last one, so V of a tile follows K of the next tile or two.  next(info, both) gives
// the tiles, emit(is_v, info) takes the units; either ends the walk with false.
template <typename Info, typename Next, typename Emit>
__device__ __forceinline__ void for_units(Next&& next, Emit&& emit) {
  Info cur, held[2] = {};
  int tile[2] = {-1, -1};                // whose outputs a group has still to bring
  bool v[2] = {};                        // V of that tile has still to come
  bool both;
  for (int li = 0; next(cur, both); ++li) {
    bool k = true;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (!both && (li & 1) != g) continue;
      if (v[g]) {
        if (!emit(true, held[g])) return;
        if (tile[g ^ 1] == tile[g]) v[g ^ 1] = false;
      }
      held[g] = cur;
      tile[g] = li;
      v[g] = true;
      if (k && !emit(false, cur)) return;
      k = false;
    }
  }
  const bool a_first = tile[0] <= tile[1];
  if (!a_first && v[1] && !emit(true, held[1])) return;
  if (v[0]) {
    if (!emit(true, held[0])) return;
    if (tile[1] == tile[0]) v[1] = false;
  }
  if (a_first && v[1]) emit(true, held[1]);
}

template <typename T, int D>
__global__ void __launch_bounds__(X_THREADS, 1)
    paged_prefix_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQs,
                           const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Px<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t ring = sbase + C::OFF_RING;
  // a unit's copies have landed; it has been read; its slots behind the last token are clear
  const uint32_t bar_full = sbase + C::OFF_BAR, bar_empty = bar_full + 8 * C::UNITS, bar_clean = bar_empty + 8 * C::UNITS;
  // queries have landed, have been read; scores, weights, outputs of a group
  const uint32_t bar_q = bar_clean + 8 * C::UNITS, bar_qe = bar_q + 16;
  const uint32_t bar_s = bar_qe + 16, bar_p = bar_s + 16, bar_o = bar_p + 16;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::UNITS; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 1);
      ptx::mbar_init(bar_empty + 8 * s, 2);
      ptx::mbar_init(bar_clean + 8 * s, 1);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(bar_q + 8 * g, 1);
      ptx::mbar_init(bar_qe + 8 * g, 1);
      ptx::mbar_init(bar_s + 8 * g, 1);
      ptx::mbar_init(bar_p + 8 * g, 8);
      ptx::mbar_init(bar_o + 8 * g, 1);
    }
    flags[0] = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmQs);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  if (warp == 2) {
    ptx::tmem_alloc(ptx::smem_u32(const_cast<int*>(flags) + 1), TM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = uniform(flags[1]);

  // a warp goes on, or gives up, as a whole
  const auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, flags, p.status)) != 0;
  };

  // 128 x 64 + 512 x 104 registers, all of the 640 x 96 that the block starts with.  (Each in its own
  // branch: behind a join the compiler keeps to the smaller one.)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    wait_prior_grid();
    allow_next_grid();                   // (the join comes as SMs fall free, and may read the plan: it is done)
    prefix::Walk<true> walk(p, cta);
    Piece a;
    if (warp == 0) {
      // ------------------------------------------------------------ keys and values
      struct Pages {
        int page, boxes, y;                // a page id in each lane
      } next{};
      const int box = min(p.c.ps, TILE);
      int u = 0;
      a.u1 = 0;
      bool next_both = false;
      // the page ids are fetched a tile ahead
      const auto look = [&]() {
        if (u >= a.u1) {
          if (!walk.step(p, a)) return false;
          u = a.u0;
          next_both = a.it.nq > ROWS;
        }
        const int tok = a.it.tok0 + u * TILE, n = min(TILE, a.it.tok1 - tok);
        ++u;
        next.boxes = (n + box - 1) / box;
        next.y = tok & (p.c.ps - 1);
        next.page = 0;
        if (lane * box < n) {
          next.page = p.c.table[(size_t)a.it.row * p.c.max_pages + (tok >> p.c.shift) + lane];
          if (next.page < 0 || next.page >= p.c.n_pages) {
            raise_status(p.status, KVP_ERR_DEVICE_CHECK);
            next.page = p.c.n_pages;       // outside the tensor map: zeros
          }
        }
        return true;
      };
      const int k = lane / C::HALVES, hf = lane % C::HALVES;
      int unit = 0;
      bool more = look();
      for_units<Pages>(
          [&](Pages& x, bool& both) {
            if (!more) return false;
            x = next;
            both = next_both;
            more = look();
            return true;
          },
          [&](bool is_v, const Pages& x) {
            const int s = unit % C::UNITS, use = unit / C::UNITS;
            if (use > 0 && !wait(bar_empty + 8 * s, (use - 1) & 1)) return false;
            const int page = __shfl_sync(0xffffffffu, x.page, k);
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar_full + 8 * s, x.boxes * box * 128 * C::HALVES);
            __syncwarp();
            if (k < x.boxes)
              ptx::tma_load_3d(ring + s * C::UNIT + hf * C::HALF_BYTES + k * box * 128, is_v ? &tmV : &tmK, bar_full + 8 * s,
                               64 * hf, x.y, page);
            __syncwarp();
            ++unit;
            return true;
          });
      // every copy must land before the CTA can exit
      for (int j = max(0, unit - C::UNITS); j < unit; ++j)
        ptx::mbar_wait_drain(bar_full + 8 * (j % C::UNITS), (j / C::UNITS) & 1, p.status);
    } else if (warp == 1) {
      // ------------------------------------------------------------ products
      constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t id_s = ptx::idesc_f16(BF, ROWS, TILE);
      constexpr uint32_t id_o = ptx::idesc_f16(BF, ROWS, D) | 1u << 16;      // B (V) is MN-major
      int li = 0, unit = 0;                // tiles, units of the ring
      // of either group: the tile whose outputs it has still to bring, V's unit once that is known, whether
      // it is the first or the last of its piece; the weights it has brought
      struct Group {
        int pend = -1, v = -1;
        bool first = false, last = false;
        int uses = 1;                      // (the first are no tile's: see the softmax)
      } ga, gb;
      bool ok = wait(bar_p, 0) && wait(bar_p + 8, 0);
      const auto outputs = [&](auto which, Group& me, Group& other) {
        constexpr int g = decltype(which)::value;
        if (me.v < 0) {
          me.v = unit++;
          if (other.pend == me.pend) other.v = me.v;
        }
        const int s = me.v % C::UNITS;
        ok = ok && wait(bar_clean + 8 * s, (me.v / C::UNITS) & 1) && wait(bar_p + 8 * g, me.uses++ & 1);
        if (!ok) return;
        ptx::tc_fence_after();
        const uint32_t o = tmem + TM_O + 128 * g, w = tmem + TM_S + 128 * g;
        const uint64_t v = desc_mn_sw128(ring + s * C::UNIT, C::HALF_BYTES);
        const bool free = other.pend != me.pend;
        if (elect_one()) {
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int k = 0; k < TILE / 16; ++k)
              mma_f16_ts(o, w + 16 * k + 8 * part, v + 128 * k, id_o,
                         !(me.first && part == 1 && k == 0));
          if (me.last) ptx::mma_commit(bar_o + 8 * g);
          if (free) ptx::mma_commit(bar_empty + 8 * s);
        }
        __syncwarp();
        me.pend = me.v = -1;
      };
      int kunit = 0, qslot = 0, turn = 0, uses_q0 = 0, uses_q1 = 0;
      const auto scores = [&](auto which, Group& me, bool both, bool begin, bool end) {
        constexpr int g = decltype(which)::value;
        const int s = kunit % C::UNITS;
        if (begin && !(both && g == 1)) ok = ok && wait(bar_q + 8 * qslot, (qslot ? uses_q1++ : uses_q0++) & 1);
        if (!(both && g == 1)) ok = ok && wait(bar_full + 8 * s, (kunit / C::UNITS) & 1);
        if (!ok) return;
        ptx::tc_fence_after();
        const uint64_t q = ptx::desc_sw128(sbase + (both ? g : qslot) * (ROWS * 128));
        const uint64_t k = ptx::desc_sw128(ring + s * C::UNIT);
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            ptx::mma_f16_ss(tmem + TM_S + 128 * g, q + (((x >> 2) * C::Q_HALF + (x & 3) * 32) >> 4),
                            k + (((x >> 2) * C::HALF_BYTES + (x & 3) * 32) >> 4), id_s, x > 0);
          ptx::mma_commit(bar_s + 8 * g);
          if (!both || g == 1) {
            ptx::mma_commit(bar_empty + 8 * s);
            if (end) ptx::mma_commit(bar_qe + 8 * qslot);
            if (end && both) ptx::mma_commit(bar_qe + 8);
          }
        }
        __syncwarp();
        me.pend = li;
      };
      const std::integral_constant<int, 0> A{};
      const std::integral_constant<int, 1> B{};
      while (ok && walk.step(p, a)) {
        const bool both = uniform(a.it.nq) > ROWS;
        const int u0 = uniform(a.u0), u1 = uniform(a.u1), step = both ? 1 : 2;
        qslot = both ? 0 : turn;
        turn ^= !both;
        for (int u = u0; ok && u < u1; ++u, ++li) {
          const int at = CUT<T> ? (u - u0) & (SEGMENT * step - 1) : u - u0;
          const bool first = at < step, last = u1 - 1 - u < step || (CUT<T> && at >= (SEGMENT - 1) * step);
          const bool begin = u == u0, end = u == u1 - 1;
          if (both || !(li & 1)) {
            if (ga.pend >= 0) outputs(A, ga, gb);
            ga.first = first;
            ga.last = last;
            kunit = unit++;
            if (ok) scores(A, ga, both, begin, end);
          }
          if (ok && (both || (li & 1))) {
            if (gb.pend >= 0) outputs(B, gb, ga);
            gb.first = first;
            gb.last = last;
            if (!both) kunit = unit++;
            if (ok) scores(B, gb, both, begin, end);
          }
        }
      }
      // the older one first
      const bool a_first = ga.pend <= gb.pend;
      if (!a_first && ok && gb.pend >= 0) outputs(B, gb, ga);
      if (ok && ga.pend >= 0) outputs(A, ga, gb);
      if (a_first && ok && gb.pend >= 0) outputs(B, gb, ga);
    } else if (warp == 2) {
      // ------------------------------------------------------------ slots behind the last token
      int u = 0, unit = 0;
      a.u0 = a.u1 = 0;
      for_units<int>(
          [&](int& valid, bool& both) {
            if (u >= a.u1) {
              if (!walk.step(p, a)) return false;
              u = a.u0;
            }
            valid = a.it.tok1 - a.it.tok0 - u * TILE;
            both = a.it.nq > ROWS;
            ++u;
            return true;
          },
          [&](bool is_v, int valid) {
            const int s = unit % C::UNITS;
            if (!wait(bar_full + 8 * s, (unit / C::UNITS) & 1)) return false;
            if (is_v && valid < TILE) {
              for (int e = valid * 8 + lane; e < TILE * 8; e += 32)
#pragma unroll
                for (int hf = 0; hf < C::HALVES; ++hf)
                  *reinterpret_cast<uint4*>(smem + C::OFF_RING + s * C::UNIT + hf * C::HALF_BYTES + e * 16) =
                      make_uint4(0, 0, 0, 0);
              ptx::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(bar_clean + 8 * s);
              ptx::mbar_arrive(bar_empty + 8 * s);
            }
            __syncwarp();
            ++unit;
            return true;
          });
    } else {
      // ------------------------------------------------------------ queries, ahead of their piece
      // A box per sequence and 64-column half (some 75 cycles each, however small), or per RUN sequences
      // that follow each other.
      int turn = 0, fills0 = 0, fills1 = 0, uses0 = 0, uses1 = 0;
      bool ok = true;
      while (walk.step(p, a)) {
        const bool both = a.it.nq > ROWS;
        const int slot = both ? 0 : turn;
        turn ^= !both;
        if (slot == 0 && fills0++ > 0) ok = ok && wait(bar_qe, fills0 & 1);
        if ((both || slot == 1) && fills1++ > 0) ok = ok && wait(bar_qe + 8, fills1 & 1);
        if (!ok) break;
        const uint32_t bar = bar_q + 8 * slot, to = sbase + slot * ROWS * 128;
        const int seqs = a.it.nq / p.G, h = a.it.row % p.Hkv * p.G;
        const int* list = p.list + a.it.list + a.it.q0 / p.G;
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, a.it.nq * 128 * C::HALVES);
        __syncwarp();
        const int hf = lane % C::HALVES;
        if (a.it.list < 0) {
          if (lane < C::HALVES) ptx::tma_load_3d(to + hf * C::Q_HALF, &tmQ, bar, 64 * hf, h, a.it.row / p.Hkv);
        } else {
          for (int k0 = lane / C::HALVES * RUN; k0 < seqs; k0 += 32 / C::HALVES * RUN) {
            int n[RUN];
            bool run = true;
#pragma unroll
            for (int k = 0; k < RUN; ++k) {
              n[k] = k0 + k < seqs ? list[k0 + k] : -1;
              run = run && n[k] == n[0] + k;
            }
            const uint32_t at = to + hf * C::Q_HALF + k0 * p.G * 128;
            if (run) {
              ptx::tma_load_3d(at, &tmQs, bar, 64 * hf, h, n[0]);
            } else {
#pragma unroll
              for (int k = 0; k < RUN; ++k)
                if (k0 + k < seqs) ptx::tma_load_3d(at + k * p.G * 128, &tmQ, bar, 64 * hf, h, n[k]);
            }
          }
        }
        __syncwarp();
        uses0 += slot == 0;
        uses1 += slot == 1;
      }
      // every copy must land before the CTA can exit
      if (uses0 > 0) ptx::mbar_wait_drain(bar_q, (uses0 - 1) & 1, p.status);
      if (uses1 > 0) ptx::mbar_wait_drain(bar_q + 8, (uses1 - 1) & 1, p.status);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    prefix::Walk<false> walk;            // (registers: the item's record is read again when the piece ends)
    const int w = (warp - 4) >> 2, g = w >> 1, c = w & 1, quad = warp & 3, tid = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)quad << 21;          // this warp's TMEM lanes
    const uint32_t ts = tmem + TM_S + 128 * g + 64 * c + lanes, to = tmem + TM_O + lanes;
    const int pair = 1 + g * 4 + quad;                    // barrier of the two warps that share queries
    float2* row = reinterpret_cast<float2*>(smem + C::OFF_X) + tid;   // [g * ROWS]: what they tell each other
    constexpr int ALL = 9;                                // barrier of all sixteen
    int li0 = 0, uses_s = 0, uses_oa = 0, uses_ob = 0;
    bool ok = true;                                       // (once a wait ran out no other is begun; barriers are met)
    // The first piece is none: while the plan is still being made, a tile of whatever lies in TMEM brings
    // the instructions in (a first tile took 8000 cycles, any other 2000).
    bool dry = true;
    Piece a{Item{0, 0, 0, TILE, 0, 2 * ROWS, 0, 0}, 0, 1};
    for (; dry || walk.step(p, a);) {
      const bool both = a.it.nq > ROWS;
      const int step = both ? 1 : 2, tiles = a.u1 - a.u0;
      const int u0 = both ? a.u0 : a.u0 + ((li0 ^ g) & 1);
      const int q0 = both ? g * ROWS : 0, nq = min(ROWS, a.it.nq - q0), tokens = a.it.tok1 - a.it.tok0 - 64 * c;
      const bool busy = quad * 32 < nq;                   // (the same in both warps)
      const bool alone = both || tiles == 1;              // a group with its outputs
      int outs = g ? uses_ob : uses_oa;                   // outputs (a segment's each) that have been waited for
      if (!dry) {
        const int na = both ? tiles : (tiles + !(li0 & 1)) >> 1, nb = both ? tiles : tiles - na;   // the groups' tiles
        uses_oa += CUT<T> ? (na + SEGMENT - 1) / SEGMENT : na > 0;
        uses_ob += CUT<T> ? (nb + SEGMENT - 1) / SEGMENT : nb > 0;
        li0 += tiles;
      }
      if (u0 >= a.u1) continue;                           // the other group has the piece's only tile
      float m = -INFINITY, l = 0.f;
      // This warp's columns of the outputs, and of the sums of the segments before if there are any, to memory or
      // back into TMEM.  (The maximum that the kept sums go by lies behind them: there is no register for it.)
      const auto add_kept = [&](bool back, bool any) {
        float* kept = p.kept + ((size_t)(cta * 2 + g) * ROWS + tid) * prefix::kept_row(D);
        const float f = any ? paged::weight(kept[D + c], m) : 0.f;
        kept[D + c] = m;
#pragma unroll 1
        for (int k = c * (D / 2); k < (c + 1) * (D / 2); k += 32) {
          uint32_t o[32];
          float4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = any ? *reinterpret_cast<const float4*>(kept + k + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
          ptx::tmem_ld32(to + 128 * g + k, o);
          ptx::tmem_ld_wait();
          loaded(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i].x = fmaf(x[i].x, f, __uint_as_float(o[4 * i]));
            x[i].y = fmaf(x[i].y, f, __uint_as_float(o[4 * i + 1]));
            x[i].z = fmaf(x[i].z, f, __uint_as_float(o[4 * i + 2]));
            x[i].w = fmaf(x[i].w, f, __uint_as_float(o[4 * i + 3]));
          }
          if (back) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[4 * i] = __float_as_uint(x[i].x);
              o[4 * i + 1] = __float_as_uint(x[i].y);
              o[4 * i + 2] = __float_as_uint(x[i].z);
              o[4 * i + 3] = __float_as_uint(x[i].w);
            }
            tmem_st32(to + 128 * g + k, o);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(kept + k + 4 * i) = x[i];
          }
        }
        if (back) tmem_st_wait();
      };
      int v0 = u0;                                        // first tile of the segment
      for (;; v0 += SEGMENT * step) {
        const int v1 = CUT<T> ? min(a.u1, v0 + SEGMENT * step) : a.u1;
        for (int u = v0; u < v1; u += step) {
          if (!dry) ok = ok && wait(bar_s + 8 * g, uses_s++ & 1);
          const int valid = tokens - u * TILE;
          if (busy) {
            ptx::tc_fence_after();
            uint32_t s[32];
            float top[2] = {-INFINITY, -INFINITY};
            {
              uint32_t y[32];
              ptx::tmem_ld32(ts, s);
              ptx::tmem_ld32(ts + 32, y);
              ptx::tmem_ld_wait();
              loaded(s);
              loaded(y);
              if (p.flip || p.zero || valid < 64) {
                const float mul = p.zero ? 0.f : p.flip ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  s[i] = i < valid ? __float_as_uint(__uint_as_float(s[i]) * mul) : 0xff800000u;
                  y[i] = i + 32 < valid ? __float_as_uint(__uint_as_float(y[i]) * mul) : 0xff800000u;
                }
                tmem_st32(ts + 32, y);
                tmem_st_wait();
              }
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                top[0] = max3(top[0], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                top[1] = max3(top[1], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
              }
            }
            const float x = fmaxf(top[0], top[1]) * p.c2;
            // (lanes without a query have what was left in shared memory: no say, or results would depend on it)
            if (ptx::bar_red_or(u == v0 || (tid < nq && x > m + LAG<T>), pair, 64)) {
              (c ? row[g * ROWS].y : row[g * ROWS].x) = x;
              bar_sync(pair, 64);
              const float up = max3(m, x, c ? row[g * ROWS].x : row[g * ROWS].y);
              const float f = paged::weight(m, up);
              l *= f;
              if (u != v0) {
                // the tile before has been added up: the scores' barrier follows its products
#pragma unroll 1
                for (int k = c * (D / 2); k < (c + 1) * (D / 2); k += 8) {
                  uint32_t o[8];
                  tmem_ld8(to + 128 * g + k, o);
                  ptx::tmem_ld_wait();
                  loaded(o);
#pragma unroll
                  for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st8(to + 128 * g + k, o);
                }
              }
              m = up;
            }
            const float off = m == -INFINITY ? 0.f : ABOVE<T> - m;     // nothing but -inf so far: weights of 0
            const uint64_t c2 = pack2(p.c2, p.c2), off2 = pack2(off, off);
            uint64_t sum[2] = {0, 0};
            // 16 scores make way for 8 + 8 columns of weights; the second 32 are read again, 16 ahead (all 64 in
            // registers would spill)
            const auto weigh = [&](const uint32_t* x, int k) {
              uint32_t parts[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float w0, w1;
                unpack2(ffma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, off2), w0, w1);
                const uint64_t w = pack2(fast_exp2(w0), fast_exp2(w1));
                sum[i & 1] = fadd2(sum[i & 1], w);
                split(T(), w, parts[i], parts[8 + i]);
              }
              tmem_st16(ts + k, parts);
            };
            uint32_t y[2][16];
            weigh(s, 0);
            tmem_ld16(ts + 32, y[0]);
            weigh(s + 16, 16);
            ptx::tmem_ld_wait();
            loaded(y[0]);
            tmem_ld16(ts + 48, y[1]);
            weigh(y[0], 32);
            ptx::tmem_ld_wait();
            loaded(y[1]);
            weigh(y[1], 48);
            float a0, a1;
            unpack2(fadd2(sum[0], sum[1]), a0, a1);
            l += a0 + a1;
            tmem_st_wait();
            ptx::tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar_p + 8 * g);
        }
        if (!CUT<T> || v0 + SEGMENT * step >= a.u1) break;
        ok = ok && wait(bar_o + 8 * g, outs++ & 1);
        if (busy) {
          ptx::tc_fence_after();
          add_kept(false, v0 != u0);
        }
      }
      if (dry) {
        dry = false;
        wait_prior_grid();
        walk = prefix::Walk<false>(p, cta);
        continue;
      }
      // the piece's outputs
      size_t slot = 0;
      if (tid < nq) {
        int qg;
        const Item it = p.items[walk.item - 1];
        const int r = prefix::query_row(p, it, q0 + tid, qg);
        slot = a.u0 == 0 ? prefix::first_slot(p, it.list < 0, r, qg) : prefix::cont_slot(p, cta, q0 + tid);
      }
      float* out = (a.u0 == 0 ? p.first_o : p.cont_o) + slot * D;
      float2* ml = (a.u0 == 0 ? p.first_ml : p.cont_ml) + slot;
      ok = ok && wait(bar_o + 8 * g, outs & 1);
      ptx::tc_fence_after();
      if (CUT<T> && busy && v0 != u0) add_kept(true, true);
      if (alone) {
        if (busy) {
          (c ? row[g * ROWS].y : row[g * ROWS].x) = l;
          bar_sync(pair, 64);
          l += c ? row[g * ROWS].x : row[g * ROWS].y;
#pragma unroll
          for (int k = c * (D / 2); k < (c + 1) * (D / 2); k += 16) {
            uint32_t o[16];
            tmem_ld16(to + 128 * g + k, o);
            ptx::tmem_ld_wait();
            loaded(o);
            if (tid < nq) store_part(out + k, o);
          }
          if (tid < nq && c == 0) *ml = make_float2(m - ABOVE<T>, l);
          bar_sync(pair, 64);
        }
        ptx::tc_fence_before();
      } else {
        // (of the other group's outputs none but these can be pending: its tiles before were added up before
        // this group's last)
        ok = ok && wait(bar_o + 8 * (g ^ 1), ((g ? uses_oa : uses_ob) - 1) & 1);
        ptx::tc_fence_after();
        if (busy) {
          if (c) row[g * ROWS].y = l;
          bar_sync(pair, 64);
          if (!c) row[g * ROWS] = make_float2(m, l + row[g * ROWS].y);
        }
        ptx::tc_fence_before();
        bar_sync(ALL, 512);
        ptx::tc_fence_after();
        if (busy) {
          const float2 A = row[0], B = row[ROWS];
          const float M = fmaxf(A.x, B.x), fa = paged::weight(A.x, M), fb = paged::weight(B.x, M);
#pragma unroll
          for (int k = w * (D / 4); k < (w + 1) * (D / 4); k += 16) {
            uint32_t o[16], y[16];
            tmem_ld16(to + k, o);
            tmem_ld16(to + 128 + k, y);
            ptx::tmem_ld_wait();
            loaded(o);
            loaded(y);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), fb, __uint_as_float(o[i]) * fa));
            if (tid < nq) store_part(out + k, o);
          }
          if (tid < nq && w == 0) *ml = make_float2(M - ABOVE<T>, fmaf(A.y, fa, B.y * fb));
        }
        ptx::tc_fence_before();
        bar_sync(ALL, 512);                               // both outputs have been read
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc(tmem, TM_COLS);
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

// [z][y][D] values, the axes `z_stride` and `y_stride` elements apart; boxes of 64 values by `rows` by `runs`.
bool map_of(CUtensorMap* m, int dtype, const void* base, int D, int y, int z, int64_t y_stride, int64_t z_stride, int rows,
            int runs) {
  const EncodeTiledFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)y, (cuuint64_t)z};
  const cuuint64_t strides[2] = {(cuuint64_t)y_stride * 2, (cuuint64_t)z_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, (cuuint32_t)runs};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, dtype == KVP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t run(const Params& p, cudaStream_t st) {
  CUtensorMap tq, tqs, tk, tv;
  const int box = p.c.ps < TILE ? p.c.ps : TILE;
  if (!map_of(&tq, p.c.dtype, p.q, D, p.Hq, p.N, D, p.q_stride, p.G, 1) ||
      !map_of(&tqs, p.c.dtype, p.q, D, p.Hq, p.N, D, p.q_stride, p.G, RUN) ||
      !map_of(&tk, p.c.dtype, p.c.k, D, p.c.ps, p.c.n_pages, p.c.token_stride, p.c.page_stride, box, 1) ||
      !map_of(&tv, p.c.dtype, p.c.v, D, p.c.ps, p.c.n_pages, p.c.token_stride, p.c.page_stride, box, 1))
    return cudaErrorInvalidValue;
  const auto kern = paged_prefix_tc_kernel<T, D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Px<D>::SMEM);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_with_pdl(kern, dim3((unsigned)p.ctas), dim3(X_THREADS), Px<D>::SMEM, st, tq, tqs, tk, tv, p);
}

}  // namespace

cudaError_t launch_paged_prefix_tc(const Params& p, cudaStream_t st) {
  if (p.c.dtype == KVP_BF16) return p.c.D == 128 ? run<__nv_bfloat16, 128>(p, st) : run<__nv_bfloat16, 64>(p, st);
  return p.c.D == 128 ? run<__half, 128>(p, st) : run<__half, 64>(p, st);
}

}  // namespace kvp
