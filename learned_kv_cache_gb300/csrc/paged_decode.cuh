// What the paged decode kernels share: how the rows' key tiles are dealt to the CTAs, and the
// layout of the partial results that the join kernel puts together.
//
// The rows' lengths are known on the device only, differ by an order of magnitude under head-wise
// budgets, and say nothing of the table's width.  So the host fixes the number of CTAs and the
// device the split: the tiles of TILE keys of all rows form one sequence, and CTA c of the P active
// ones takes [c * total / P, (c + 1) * total / P) of it.  A row that lies inside one CTA's range is
// finished there; of a longer one every CTA leaves a partial (maximum, sum, output) that the join
// kernel merges in CTA order, so results do not depend on timing.  Short rows are not cut (whole_tiles).
#pragma once

#include <type_traits>

#include "kvp_common.cuh"
#include "kvp_launch.h"

namespace kvp {
namespace paged {

constexpr int TILE = 64;                 // keys per tile
constexpr int MAX_CTAS = 512;            // (two per SM)
// Tiles per CTA below which fewer CTAs are active.  GPU time of a call at 4 / 2 / 1 (f16, 12 query
// heads on 2 KV heads, 28 layers, in tables wide enough to be cut): 64 tokens a row 12.3 / 9.0 / 7.4 us,
// 512 tokens 10.9 / 10.4 / 11.6 us (more parts to join), longer rows the same.
constexpr int MIN_TILES = 2;

// Rows whose table holds no more tiles than this are not cut: a CTA takes whole rows, an equal number each,
// so that nothing is left to join or to score, and nobody has to know the lengths of all rows.  GPU time
// of a call without / with the rule, 6 query heads on a KV head, D 128:
//   bf16, 56 rows: 64 tokens 8.0 / 4.9 us, 256 9.3 / 6.8, 512 9.7 / 8.9; 900 rows: 64 12.0 / 9.7, 512 46.9 / 40.1
//   fp32, 56 rows: 64 tokens 12.4 / 6.4 us, 128 10.6 / 9.2, 256 13.7 / 15.1; 900 rows: 64 24.8 / 23.1
//   with scores: bf16, 56 rows: 64 tokens 9.5 / 5.3 us, 512 11.2 / 10.6; 300 rows: 512 20.9 / 13.7
// A CTA of the fp32 kernel takes three times as long over a tile, and so gains less by the wait it saves.
// It is the table's width that says so, as the host does not know the lengths: 56 f16 rows of 64 tokens in a
// table for 131072 take 8.1 us (with scores 11.8), of 512 tokens 9.8 us (17.4).
constexpr int whole_tiles(int dtype) { return dtype == KVP_F32 ? 3 : 9; }
// Rows per CTA up to which that holds.  More rows gain 8 % by it (16384 of ~64 tokens 152 / 140 us), but where
// the long ones lie side by side an equal number of rows is no equal share.
constexpr int WHOLE_ROWS = 4;

// Range of one CTA in the tile sequence, kept for the join kernel.
struct Range {
  int begin, end;        // tiles
  int row, tile;         // row and tile within the row at `begin`
  int total, active;     // tiles of all rows; CTAs that take part
  int lo, hi;            // CTAs that share `row`
};

struct Params {
  PagedView c;
  int G, Hq, Hkv;
  int gpad;              // G padded to 8 or 16: the GP of the layouts below
  int64_t q_stride;
  float c2, c2_low;      // scale * log2 e, and what the float leaves of it
  int ctas;              // launched
  int whole;             // 1: rows are not cut (part and range are not used)
  float* part;           // [ctas][2][pstride]: m[GP], l[GP], o[GP][D]; slot 0: the row began in an
  int pstride;           //   earlier CTA, slot 1: it goes on in the next one
  Range* range;          // [ctas]
  float* lse2;           // [R][GP] base-2 LSE of the rows finished in one CTA (scores only)
  float* logits;         // [R * cap][GP] base-2 logits (scores only)
  void* out;
  int out_f32;
  float* lse;
  int* status;
};

__device__ __forceinline__ int clamp_len(const Params& p, int n) { return n < 0 ? 0 : (n > p.c.cap ? p.c.cap : n); }
__device__ __forceinline__ int row_len(const Params& p, int r) { return clamp_len(p, p.c.lens[r]); }
// Base-2 logit of the dot product a + b, and in `low` what is left of it (a two-term sum and product:
// what a + b and the product with c2 round off, and c2's own remainder).
__device__ __forceinline__ float base2(const Params& p, float a, float b, float& low) {
  const float s = a + b, t = s - a, left = (a - (s - t)) + (b - t);
  const float x = s * p.c2;
  low = fmaf(s, p.c2, -x) + fmaf(s, p.c2_low, left * p.c2);
  return x;
}
__device__ __forceinline__ int tiles_of(int n) { return (n + TILE - 1) / TILE; }

// 32-bit divisions where the products fit (a 64-bit one is a subroutine of some hundred cycles, and
// nothing is copied yet while a CTA looks for its range).
__device__ __forceinline__ int cta_begin(int c, int total, int active) {
  if (total < (1 << 22)) return (int)((uint32_t)c * (uint32_t)total / (uint32_t)active);   // c, active <= MAX_CTAS
  return (int)((long long)c * total / active);
}
// CTA that owns tile x.
__device__ __forceinline__ int cta_of(int x, int total, int active) {
  if (total < (1 << 22)) return (int)((((uint32_t)x + 1) * (uint32_t)active - 1) / (uint32_t)total);
  return (int)((((long long)x + 1) * active - 1) / total);
}

__device__ __forceinline__ int active_ctas(const Params& p, int total) {
  return min((total + MIN_TILES - 1) / MIN_TILES, p.ctas);
}

// This CTA's range.  Every thread of the block calls it; `sh` holds 36 + blockDim.x / 2 ints.  Each thread
// has a run of consecutive rows, and a block scan gives every run its place in the sequence.  Up to
// blockDim.x rows a run is one row, and the thread whose row the CTA's first tile lies in says so.  Of
// more rows a warp finds it: the run, then 32 rows at a time (16384 rows of ~64 tokens: 168 -> 152 us of
// the whole call; for few rows it would be one barrier and 0.3 us more).
__device__ __forceinline__ Range find_range(const Params& p, int cta, int* sh) {
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31;
  if (p.whole) {                             // an equal number of rows each
    Range g{};
    const int end = (int)((long long)(cta + 1) * p.c.R / p.ctas);
    g.row = (int)((long long)cta * p.c.R / p.ctas);
    for (int r = g.row; r < end; ++r) g.end += tiles_of(row_len(p, r));
    g.active = g.end > 0 ? p.ctas : 0;
    __syncthreads();                         // as on the other way, for the caller's shared memory
    return g;
  }
  const bool one = p.c.R <= nt;
  const int per = one ? 1 : ((p.c.R + nt - 1) / nt + 3) & ~3, r0 = min(tid * per, p.c.R), r1 = min(r0 + per, p.c.R);
  int mine = 0;
  if (!one && ((size_t)p.c.lens & 15) == 0) {              // four rows at a time
#pragma unroll 4
    for (int r = r0; r < r1; r += 4) {
      if (r + 4 <= p.c.R) {
        const int4 n = *reinterpret_cast<const int4*>(p.c.lens + r);
        mine += tiles_of(clamp_len(p, n.x)) + tiles_of(clamp_len(p, n.y)) + tiles_of(clamp_len(p, n.z)) +
                tiles_of(clamp_len(p, n.w));
      } else {
        for (int x = r; x < r1; ++x) mine += tiles_of(row_len(p, x));
      }
    }
  } else {
#pragma unroll 8
    for (int r = r0; r < r1; ++r) mine += tiles_of(row_len(p, r));
  }
  int total;
  const int before = block_exclusive_scan(mine, sh, &total);
  const int active = active_ctas(p, total);
  Range g{};
  g.total = total;
  g.active = active;
  if (cta < active) {
    g.begin = cta_begin(cta, total, active);
    g.end = cta_begin(cta + 1, total, active);
  }
  if (one) {
    if (cta < active && g.begin >= before && g.begin < before + mine) {
      sh[33] = tid;
      sh[34] = g.begin - before;
      sh[35] = mine;
    }
  } else {
    int* run_sh = sh + 36;                   // places of every second thread's run
    if ((tid & 1) == 0) run_sh[tid >> 1] = before;
    __syncthreads();
    if (tid < 32 && cta < active) {
      int run = -1;                          // the last run that starts at or before the range
      for (int t0 = 0; t0 < nt / 2; t0 += 32)
        run += __popc(__ballot_sync(0xffffffffu, t0 + lane < nt / 2 && run_sh[min(t0 + lane, nt / 2 - 1)] <= g.begin));
      int at = run_sh[run];
      for (int x0 = run * 2 * per; x0 < p.c.R; x0 += 32) {
        const int t = x0 + lane < p.c.R ? tiles_of(row_len(p, x0 + lane)) : 0;
        const int upto = at + warp_inclusive_scan(t);
        const uint32_t b = __ballot_sync(0xffffffffu, upto > g.begin);
        if (b) {
          if (lane == __ffs(b) - 1) {
            sh[33] = x0 + lane;
            sh[34] = g.begin - (upto - t);
            sh[35] = t;
          }
          break;
        }
        at = __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  __syncthreads();
  if (cta < active) {
    g.row = sh[33];
    g.tile = sh[34];
    g.lo = cta_of(g.begin - g.tile, total, active);
    g.hi = cta_of(g.begin - g.tile + sh[35] - 1, total, active);
  }
  if (tid == 0) p.range[cta] = g;
  return g;
}

// Weight of a state whose maximum is m in a merge whose maximum is M.  A state that has seen no finite
// logit weighs 0 (its sum is 0, or NaN, which 0 * NaN carries on).
__device__ __forceinline__ float weight(float m, float M) { return m == -INFINITY ? 0.f : fast_exp2(m - M); }

// Four outputs from i on (a multiple of 4; the output is 16-byte aligned), with the one rounding of the
// result: to the type the model goes on with, when the caller asks for it.
template <typename T>
__device__ __forceinline__ void store_out4(const Params& p, size_t i, float4 x) {
  if (p.out_f32 || sizeof(T) == 4) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + i) = x;
  } else if constexpr (std::is_same<T, __half>::value) {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(p.out) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// Adds the probabilities of tokens [m0, hi) of row r, `step` apart, to their scores; lse: base 2, of the
// group's heads.
template <int GP>
__device__ __forceinline__ void add_row_scores(const Params& p, int r, int m0, int hi, int step, const float* lse_sh) {
  float lse[GP];
#pragma unroll
  for (int h = 0; h < GP; ++h) lse[h] = h < p.G ? lse_sh[h] : 0.f;
  for (int m = m0; m < hi; m += step) {
    const float4* lg = reinterpret_cast<const float4*>(p.logits + ((size_t)r * p.c.cap + m) * GP);
    float* score = p.c.score + (size_t)r * p.c.cap + m;
    const float before = *score;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < GP / 4; ++k) {
      const float4 w = lg[k];
      const float z[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * k + i < p.G && z[i] != -INFINITY) s += fast_exp2(z[i] - lse[4 * k + i]);
    }
    *score = before + s;
  }
}

// Rows without tokens have no tile: the CTAs share them out by index, a lane looks at a row and a warp
// clears its outputs.  `threads` of the CTA take part.
template <typename T, int D>
__device__ __forceinline__ void empty_rows(const Params& p, int cta, int threads) {
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x - lane; (long long)i * p.ctas + cta < p.c.R; i += threads) {
    const long long x = (long long)(i + lane) * p.ctas + cta;
    const int n = x < p.c.R ? p.c.lens[x] : 1;
    if (n < 0 || n > p.c.cap) raise_status(p.status, KVP_ERR_DEVICE_CHECK);
    for (uint32_t b = __ballot_sync(0xffffffffu, n <= 0); b; b &= b - 1) {
      const int r = (i + __ffs(b) - 1) * p.ctas + cta;
      const size_t head = (size_t)(r / p.Hkv) * p.Hq + (size_t)(r % p.Hkv) * p.G;
      for (int e = 4 * lane; e < p.G * D; e += 128) store_out4<T>(p, head * D + e, make_float4(0.f, 0.f, 0.f, 0.f));
      if (p.lse)
        for (int g = lane; g < p.G; g += 32) p.lse[head + g] = -INFINITY;
    }
  }
}

}  // namespace paged

// The tensor-core path of bf16 / f16 caches (paged_decode_mma.cu).
cudaError_t launch_paged_decode_mma(const paged::Params& p, const void* q, cudaStream_t st);

}  // namespace kvp
