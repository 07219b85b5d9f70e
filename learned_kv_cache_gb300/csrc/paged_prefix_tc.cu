// The items of shared-prefix decode on the tensor cores (bf16 / f16 caches).
//
//   S = Q K^T,  P = 2^(c S - m),  l = sum P,  O = P V   for up to 256 queries and 128 keys at a time
//
// 4 D flop per query and key against 4 D bytes per key: with few queries bound by HBM, with 256 about as
// long on the tensor cores (QK^T and two parts of P V: 3072 cycles a tile of D 128) as in HBM (2790).
//
//  * One CTA per SM.  Warp 0 copies: per tile K and V as a unit each of a ring, one TMA box per page (or 128
//    tokens of one) and 64-column half.  Warp 1 issues the products.  Two groups of four warps have a
//    128-row block of queries each, a thread a row: scores come from TMEM, the weights go back there as
//    the first operand of P V, and the outputs stay in TMEM until the piece ends.
//  * More than 128 queries: each group has its own, and both take every tile.  Up to 128: both have the
//    same, and take the tiles in turn (a part each for the join).  Either way one group's softmax runs
//    beside the other's products.
//  * V lies [key][dim] in memory, so it is the second operand in its MN-major form; nothing is transposed.
//  * P enters the product as the sum of two 16-bit parts: 16 (bf16) or 22 (f16) bits of every weight, so
//    that an output is off by its own rounding only; with one part bf16 outputs would be 1.4 times as far
//    off.  The outputs come in the cache's type.
//  * The running maximum may lag by a factor of 2^8 before the outputs are scaled again: weights reach 2^8,
//    which f16 holds, and most tiles move nothing.
//  * Slots behind the last token of an item may hold anything: their logits become -inf, and their V is
//    cleared in shared memory (0 * NaN would be NaN).
#include <type_traits>

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "paged_prefix.cuh"
#include "tc_ptx.cuh"

namespace kvp {
namespace {

using prefix::Params;
using prefix::Piece;
using prefix::TILE;

constexpr int X_THREADS = 384;
constexpr int ROWS = 128;                // queries of a group
constexpr float LAG = 8.f;               // log2 of how far the maximum may lag

template <int D>
struct Px {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = TILE * 128;            // 64 columns of 128 tokens
  static constexpr int UNIT = HALVES * HALF_BYTES;         // K or V of a tile, or the queries of a group
  static constexpr int UNITS = D == 128 ? 5 : 10;
  static constexpr int OFF_RING = 2 * UNIT;
  static constexpr int OFF_BAR = OFF_RING + UNITS * UNIT;
  static constexpr int OFF_FLAG = OFF_BAR + 8 * (2 * UNITS + 8);
  static constexpr int SMEM = OFF_FLAG + 16 + 1024;        // + alignment slack
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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Uses of r stay behind the wait for its loads.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Packed fp32 pairs (sm_100 family): two lanes of arithmetic per instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A pair of weights as 16-bit values, and what that leaves of them.
__device__ __forceinline__ uint32_t pack_rest(__nv_bfloat16, float& a, float& b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
  a -= __uint_as_float(u << 16);
  b -= __uint_as_float(u & 0xffff0000u);
  return u;
}
__device__ __forceinline__ uint32_t pack_rest(__half, float& a, float& b) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  a -= f.x;
  b -= f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack(__nv_bfloat16, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack(__half, float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int D>
__global__ void __launch_bounds__(X_THREADS, 1)
    paged_prefix_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Px<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t ring = sbase + C::OFF_RING;
  const uint32_t bar_full = sbase + C::OFF_BAR, bar_empty = bar_full + 8 * C::UNITS;
  const uint32_t bar_q = bar_empty + 8 * C::UNITS, bar_s = bar_q + 16, bar_p = bar_s + 16, bar_o = bar_p + 16;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::UNITS; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 1);
      ptx::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(bar_q + 8 * g, 4);
      ptx::mbar_init(bar_s + 8 * g, 1);
      ptx::mbar_init(bar_p + 8 * g, 4);
      ptx::mbar_init(bar_o + 8 * g, 1);
    }
    flags[0] = 0;
    ptx::fence_mbar_init();
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
  const uint32_t tmem = flags[1];
  wait_prior_grid();

  // 128 x 80 + 256 x 208 registers, of the 384 x 168 that the block starts with
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    prefix::Walk walk(p, cta);
    Piece a;
    const int box = min(p.c.ps, TILE);
    int u = 0;
    a.u1 = 0;
    // the next tile: its tokens, and a page id in each lane
    int tok = 0, n = 0, page = 0;
    const auto look = [&]() {
      if (u >= a.u1) {
        if (!walk.step(a)) return false;
        u = a.u0;
      }
      tok = a.it.tok0 + u * TILE;
      n = min(TILE, a.it.tok1 - tok);
      ++u;
      page = 0;
      if (lane * box < n) {
        page = p.c.table[(size_t)a.it.row * p.c.max_pages + (tok >> p.c.shift) + lane];
        if (page < 0 || page >= p.c.n_pages) {
          raise_status(p.status, KVP_ERR_DEVICE_CHECK);
          page = p.c.n_pages;            // outside the tensor map: zeros
        }
      }
      return true;
    };
    int li = 0;                          // units
    bool ok = true, more = look();
    while (more && ok) {
      const int boxes = (n + box - 1) / box, y = tok & (p.c.ps - 1), held = page;
      more = look();
      const int k = lane / C::HALVES, hf = lane % C::HALVES;
      const int pg = __shfl_sync(0xffffffffu, held, k);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int s = li % C::UNITS, use = li / C::UNITS;
        if (use > 0) ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_empty + 8 * s, (use - 1) & 1, flags, p.status));
        if (!ok) break;
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_full + 8 * s, boxes * box * 128 * C::HALVES);
        __syncwarp();
        if (k < boxes)
          ptx::tma_load_3d(ring + s * C::UNIT + hf * C::HALF_BYTES + k * box * 128, v ? &tmV : &tmK, bar_full + 8 * s,
                           64 * hf, y, pg);
        __syncwarp();
        ++li;
      }
    }
    // every copy must land before the CTA can exit
    for (int j = max(0, li - C::UNITS); j < li; ++j)
      ptx::mbar_wait_drain(bar_full + 8 * (j % C::UNITS), (j / C::UNITS) & 1, p.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t id_s = ptx::idesc_f16(BF, ROWS, TILE);
      constexpr uint32_t id_o = ptx::idesc_f16(BF, ROWS, D) | 1u << 16;      // B (V) is MN-major
      prefix::Walk walk(p, cta);
      Piece a;
      int li = 0;                        // tiles
      // of either group: the tile whose weights it has still to bring, and whether that is the first or
      // the last of its piece; the weights and queries it has brought
      struct Group {
        int pend = -1;
        bool first = false, last = false;
        int uses_q = 0, uses_p = 0;
      } ga, gb;
      bool ok = true;
      const auto outputs = [&](auto which, Group& me, const Group& other) {
        constexpr int g = decltype(which)::value;
        const int unit = 2 * me.pend + 1, s = unit % C::UNITS;
        ok = ok && ptx::mbar_wait(bar_p + 8 * g, me.uses_p++ & 1, flags, p.status) &&
             ptx::mbar_wait(bar_full + 8 * s, (unit / C::UNITS) & 1, flags, p.status);
        if (!ok) return;
        ptx::tc_fence_after();
        const uint32_t v = ring + s * C::UNIT, o = tmem + TM_O + 128 * g, w = tmem + TM_S + 128 * g;
#pragma unroll
        for (int part = 1; part >= 0; --part)
#pragma unroll
          for (int k = 0; k < TILE / 16; ++k)
            mma_f16_ts(o, w + 32 * (k >> 1) + 16 * part + 8 * (k & 1), desc_mn_sw128(v + 2048 * k, C::HALF_BYTES), id_o,
                       !(me.first && part == 1 && k == 0));
        if (me.last) ptx::mma_commit(bar_o + 8 * g);
        if (other.pend != me.pend) ptx::mma_commit(bar_empty + 8 * s);
        me.pend = -1;
      };
      const auto scores = [&](auto which, Group& me, bool both) {
        constexpr int g = decltype(which)::value;
        const int unit = 2 * li, s = unit % C::UNITS;
        if (me.first) ok = ok && ptx::mbar_wait(bar_q + 8 * g, me.uses_q++ & 1, flags, p.status);
        ok = ok && ptx::mbar_wait(bar_full + 8 * s, (unit / C::UNITS) & 1, flags, p.status);
        if (!ok) return;
        ptx::tc_fence_after();
        const uint32_t q = sbase + g * C::UNIT, k = ring + s * C::UNIT;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t at = (x >> 2) * C::HALF_BYTES + (x & 3) * 32;
          ptx::mma_f16_ss(tmem + TM_S + 128 * g, ptx::desc_sw128(q + at), ptx::desc_sw128(k + at), id_s, x > 0);
        }
        ptx::mma_commit(bar_s + 8 * g);
        if (!both || g == 1) ptx::mma_commit(bar_empty + 8 * s);
        me.pend = li;
      };
      const std::integral_constant<int, 0> A{};
      const std::integral_constant<int, 1> B{};
      while (ok && walk.step(a)) {
        const bool both = a.it.nq > ROWS;
        const int step = both ? 1 : 2;
        for (int u = a.u0; ok && u < a.u1; ++u, ++li) {
          const bool first = u - a.u0 < step, last = a.u1 - 1 - u < step;
          if (both || !(li & 1)) {
            if (ga.pend >= 0) outputs(A, ga, gb);
            ga.first = first;
            ga.last = last;
            if (ok) scores(A, ga, both);
          }
          if (ok && (both || (li & 1))) {
            if (gb.pend >= 0) outputs(B, gb, ga);
            gb.first = first;
            gb.last = last;
            if (ok) scores(B, gb, both);
          }
        }
      }
      // the older one first
      const bool second = ga.pend >= 0 && (gb.pend < 0 || ga.pend <= gb.pend);
      if (!second && ok && gb.pend >= 0) outputs(B, gb, ga);
      if (ok && ga.pend >= 0) outputs(A, ga, gb);
      if (second && ok && gb.pend >= 0) outputs(B, gb, ga);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int g = (warp - 4) >> 2, quad = warp & 3, tid = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)quad << 21;          // this warp's TMEM lanes
    const uint32_t ts = tmem + TM_S + 128 * g + lanes, to = tmem + TM_O + 128 * g + lanes;
    prefix::Walk walk(p, cta);
    Piece a;
    int li0 = 0, uses_s = 0, uses_o = 0;
    bool ok = true;
    const auto wait = [&](uint32_t bar, uint32_t parity) {   // a warp goes on, or gives up, as a whole
      return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, flags, p.status)) != 0;
    };
    while (walk.step(a)) {
      const bool own = a.it.list < 0, both = a.it.nq > ROWS;
      const int step = both ? 1 : 2, tiles = a.u1 - a.u0;
      const int u0 = both ? a.u0 : a.u0 + ((li0 ^ g) & 1);
      const int q0 = both ? g * ROWS : 0, nq = min(ROWS, a.it.nq - q0);
      const bool busy = quad * 32 < nq;                   // (the same in a warp)
      const int li_piece = li0;
      li0 += tiles;
      // this thread's query, and where its part goes
      size_t slot = 0;
      if (tid < nq) {
        int qg;
        const int r = prefix::query_row(p, a.it, q0 + tid, qg);
        slot = a.u0 == 0 ? prefix::first_slot(p, own, r, qg, both ? 0 : g)
                         : prefix::cont_slot(p, cta, g * ROWS + tid);
      }
      float2* ml = (a.u0 == 0 ? p.first_ml : p.cont_ml) + slot;
      if (u0 >= a.u1) {                                   // the other group has the piece's only tile
        if (tid < nq) *ml = make_float2(-INFINITY, 0.f);
        continue;
      }
      // the queries, a lane per 16 bytes of a row
      {
        constexpr int CH = D / 8;
        const uint32_t keep = p.zero ? 0u : 0xffffffffu, sign = p.flip ? 0x80008000u : 0u;
        for (int e = tid; e < nq * CH; e += ROWS) {
          const int i = e / CH, ch = e % CH;
          int qg;
          const int r = prefix::query_row(p, a.it, q0 + i, qg);
          uint4 x = *reinterpret_cast<const uint4*>((const T*)p.q + (r / p.Hkv) * p.q_stride +
                                                    (size_t)((r % p.Hkv) * p.G + qg) * D + ch * 8);
          x.x = (x.x & keep) ^ sign;
          x.y = (x.y & keep) ^ sign;
          x.z = (x.z & keep) ^ sign;
          x.w = (x.w & keep) ^ sign;
          *reinterpret_cast<uint4*>(smem + g * C::UNIT + (ch >> 3) * C::HALF_BYTES + i * 128 +
                                    (((ch & 7) ^ (i & 7)) << 4)) = x;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_q + 8 * g);
      }
      float m = -INFINITY, l = 0.f;
      for (int u = u0; ok && u < a.u1; u += step) {
        ok = wait(bar_s + 8 * g, uses_s++ & 1);
        if (!ok) break;
        const int valid = a.it.tok1 - a.it.tok0 - u * TILE;
        if (busy) {
          ptx::tc_fence_after();
          // the largest score, then the weights chunk by chunk: 32 scores make way for 16 + 16 columns of weights
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < TILE; k += 32) {
            uint32_t s[32];
            ptx::tmem_ld32(ts + k, s);
            ptx::tmem_ld_wait();
            loaded(s);
            if (valid < TILE) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (k + i >= valid) s[i] = 0xff800000u;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) top = max3(top, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          }
          const float x = top * p.c2;
          if (u == u0) {
            m = x;
          } else if (__any_sync(0xffffffffu, x > m + LAG)) {
            const float up = fmaxf(m, x), f = paged::weight(m, up);
            m = up;
            l *= f;
            // the tile before has been added up: the scores' barrier follows its products
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              uint32_t o[32], w[2][16];
              ptx::tmem_ld32(to + k, o);
              ptx::tmem_ld_wait();
              loaded(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i >> 4][i & 15] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(to + k, w[0]);
              tmem_st16(to + k + 16, w[1]);
            }
          }
          const float off = m == -INFINITY ? 0.f : -m;     // nothing but -inf so far: weights of 0
          const uint64_t c2 = pack2(p.c2, p.c2), off2 = pack2(off, off);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < TILE; k += 32) {
            uint32_t s[32], hi[16], lo[16];
            ptx::tmem_ld32(ts + k, s);
            ptx::tmem_ld_wait();
            loaded(s);
            if (valid < TILE) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (k + i >= valid) s[i] = 0xff800000u;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float w0, w1;
              unpack2(ffma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, off2), w0, w1);
              w0 = fast_exp2(w0);
              w1 = fast_exp2(w1);
              sum[i & 1] = fadd2(sum[i & 1], pack2(w0, w1));
              hi[i] = pack_rest(T(), w0, w1);
              lo[i] = pack(T(), w0, w1);
            }
            tmem_st16(ts + k, hi);
            tmem_st16(ts + k + 16, lo);
          }
          float a0, a1, b0, b1;
          unpack2(sum[0], a0, a1);
          unpack2(sum[1], b0, b1);
          l += (a0 + a1) + (b0 + b1);
          tmem_st_wait();
          ptx::tc_fence_before();
        }
        if (valid < TILE) {
          const int unit = 2 * (li_piece + u - a.u0) + 1, sl = unit % C::UNITS;
          ok = wait(bar_full + 8 * sl, (unit / C::UNITS) & 1);
          for (int e = valid * 8 + tid; e < TILE * 8; e += ROWS)
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf)
              *reinterpret_cast<uint4*>(smem + C::OFF_RING + sl * C::UNIT + hf * C::HALF_BYTES + e * 16) = make_uint4(0, 0, 0, 0);
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_p + 8 * g);
      }
      if (!ok) break;
      ok = wait(bar_o + 8 * g, uses_o++ & 1);
      if (!ok) break;
      if (busy) {
        ptx::tc_fence_after();
        float* out = (a.u0 == 0 ? p.first_o : p.cont_o) + slot * D;
#pragma unroll
        for (int k = 0; k < D; k += 32) {
          uint32_t o[32];
          ptx::tmem_ld32(to + k, o);
          ptx::tmem_ld_wait();
          loaded(o);
          if (tid < nq) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(out + k + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        ptx::tc_fence_before();
        if (tid < nq) *ml = make_float2(m, l);
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

template <typename T, int D>
cudaError_t run(const Params& p, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!pool_map(&tk, p.c, p.c.k) || !pool_map(&tv, p.c, p.c.v)) return cudaErrorInvalidValue;
  const auto kern = paged_prefix_tc_kernel<T, D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Px<D>::SMEM);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_with_pdl(kern, dim3((unsigned)p.ctas), dim3(X_THREADS), Px<D>::SMEM, st, tk, tv, p);
}

}  // namespace

cudaError_t launch_paged_prefix_tc(const Params& p, cudaStream_t st) {
  if (p.c.dtype == KVP_BF16) return p.c.D == 128 ? run<__nv_bfloat16, 128>(p, st) : run<__nv_bfloat16, 64>(p, st);
  return p.c.D == 128 ? run<__half, 128>(p, st) : run<__half, 64>(p, st);
}

}  // namespace kvp
