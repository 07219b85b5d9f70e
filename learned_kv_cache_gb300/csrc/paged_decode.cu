// One-token decode attention over the paged cache.
//
// How much KV cache can you prune, "What we did" / "Bounded windows" (one-token attention over the
// retained entries) over rows of pages:
//   out = sum_t softmax_t(scale * q . k_t) v_t,  lse = ln sum_t exp(scale * q . k_t).
// Base-2 online softmax; the state (maximum, sum, output) stays in fp32 registers.  The split is
// described in paged_decode.cuh.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "paged_decode.cuh"

namespace kvp {
namespace {

using paged::MAX_CTAS;
using paged::Params;
using paged::Range;
using paged::TILE;

// The kernel of fp32 caches (the tensor cores have no fp32 products).  4 G D FMAs per 8 D bytes: bound
// by HBM up to some four query heads; above, by what the two warps per scheduler that 2 D GP registers of
// queries and outputs leave room for can issue, so what surrounds the FMAs is kept small.  A group of
// LPK lanes reads KB keys at a time, 16 bytes of each per lane.  Summing the
// KB * GP partial dot products over the lanes one by one would take log2(LPK) shuffles each; halving
// exchanges (a lane passes on the half of its values that its partner keeps) take one each, and leave
// every lane with the logit of one (key, head), so that the softmax is computed once and not LPK times.
// The weights come back to all lanes through shared memory.
// Few warps have few loads in flight: from five heads on, K and V come through a ring in shared memory,
// in which a lane reads what it has copied itself.  64 rows x 8192 tokens, D 128, with the loads where
// they are used / one step ahead in registers / the ring / and the weighted sums two at a time: 8 heads
// 138 / 135 / 109 / 104 us, 16 heads 252 / 237 / 190 / 187 us (4 heads 84 us, 6.4 TB/s).  Six warps per
// CTA, with three stages: 113 us.
template <int D, int GP>
struct Pf {
  static constexpr int LPK = D / 4;                        // lanes per key
  static constexpr int SUBS = 32 / LPK;                    // groups of lanes in a warp, each with its own keys
  static constexpr int KB = GP <= 4 ? 8 : 32 / GP;         // keys at a time: never across a page (16 slots)
  static constexpr int V = KB * GP;                        // logits of a group at a time
  static constexpr int WARPS = GP <= 4 ? 8 : 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int STATES = WARPS * SUBS;
  static constexpr int STAGES = GP <= 4 ? 1 : 16 / KB;     // steps of a warp under way
  static constexpr int STAGE_BYTES = 2 * KB * 512;         // K, then V
  static constexpr int SMEM = STAGES > 1 ? WARPS * STAGES * STAGE_BYTES : 0;
  static constexpr int HAVE = V > LPK ? V / LPK : 1;       // logits a lane ends up with
  static constexpr int SAME = LPK > V ? LPK / V : 1;       // lanes that end up with the same one
};

// Sums v[0, V) over the LPK lanes of a group; lane l is left with the sums of values
// [l * HAVE / SAME, ...) in v[0, HAVE).
template <int V, int LPK>
__device__ __forceinline__ void sum_scatter(float (&v)[V]) {
  const int lane = threadIdx.x & 31;
  int n = V;
#pragma unroll
  for (int s = LPK / 2; s > 0; s >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (i < n) {
          const float keep = (lane & s) ? v[i + n] : v[i], pass = (lane & s) ? v[i] : v[i + n];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, pass, s);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
    }
  }
}

__device__ __forceinline__ float4 stream_float4(const float* p) {
  const uint4 u = ld_stream16(p);
  return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
}

// Two products and sums in one instruction, each rounded as by fmaf.  (The dot products gain nothing by
// it: their halves still have to be added.)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
               "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, int GP>
__global__ void __launch_bounds__(Pf<D, GP>::THREADS, GP <= 8 ? 2 : 1)
    paged_decode_f32_kernel(const float* __restrict__ q, const Params p) {
  using C = Pf<D, GP>;
  __shared__ int scan_sh[36 + C::THREADS / 2];
  __shared__ float st_m[C::STATES][GP], st_l[C::STATES][GP];
  __shared__ __align__(16) float st_o[C::STATES][GP][D];
  __shared__ __align__(16) float weight_sh[C::STATES][C::V];
  __shared__ float factor_sh[C::STATES][GP];
  extern __shared__ __align__(16) uint8_t ring_raw[];      // per warp: STAGES of K and V
  wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dl = lane % C::LPK;
  const int state = warp * C::SUBS + lane / C::LPK;
  const int first_value = dl * C::HAVE / C::SAME;          // of this lane's logits
  const int key_of = first_value / GP, head_of = first_value % GP;
  const bool counts = dl % C::SAME == 0;                   // one of the lanes that have the same logit
  const int cta = blockIdx.x;
  // a lane reads what it has copied itself, so that nobody has to be waited for
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_raw) + warp * C::STAGES * C::STAGE_BYTES + lane * 16;
  const Range g = paged::find_range(p, cta, scan_sh);
  paged::empty_rows<float, D>(p, cta, C::THREADS);
  if (cta >= g.active) return;
  const PagedView& c = p.c;
  const float* kp = (const float*)c.k + dl * 4;
  const float* vp = (const float*)c.v + dl * 4;

  int r = g.row, u = g.tile;
  for (int x = g.begin; x < g.end;) {
    const int n = paged::row_len(p, r), nt = paged::tiles_of(n);
    if (nt == 0) {
      ++r;
      u = 0;
      continue;
    }
    const int u1 = min(nt, u + (g.end - x));
    const int lo = u * TILE, hi = min(n, u1 * TILE);
    const int l = r / p.Hkv, hk = r % p.Hkv;
    float4 qf[GP], o[GP];
    float mx[C::HAVE], sum[C::HAVE], lost[C::HAVE];        // of this lane's heads; lost: what sum rounds off
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      qf[h] = o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (h < p.G) qf[h] = *reinterpret_cast<const float4*>(q + l * p.q_stride + (size_t)(hk * p.G + h) * D + dl * 4);
    }
#pragma unroll
    for (int i = 0; i < C::HAVE; ++i) {
      mx[i] = -INFINITY;
      sum[i] = lost[i] = 0.f;
    }
    const int32_t* table = c.table + (size_t)r * c.max_pages;
    constexpr int STEP = C::STATES * C::KB;
    int m = lo + state * C::KB;
    const auto page_of = [&](int t) { return t < hi ? table[t >> c.shift] : 0; };
    const auto page_good = [&](int t, int page) {
      const bool good = page >= 0 && page < c.n_pages;
      if (t < hi && !good) raise_status(p.status, KVP_ERR_DEVICE_CHECK);
      return good;
    };
    // slots behind the row's end are not read, but cleared
    const auto fetch = [&](float4 (&x)[C::KB], const float* pool, int t, int page, bool good) {
      const float* at = pool + page * c.page_stride + (t & (c.ps - 1)) * c.token_stride;
#pragma unroll
      for (int i = 0; i < C::KB; ++i) {
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (good && t + i < hi) x[i] = stream_float4(at + i * c.token_stride);
      }
    };
    uint32_t goods = 0;                      // a bit per stage
    const auto issue = [&](int t, int page, int stage) {
      const bool good = page_good(t, page);
      goods = good ? goods | 1u << stage : goods & ~(1u << stage);
      const int64_t at = page * c.page_stride + (t & (c.ps - 1)) * c.token_stride;
#pragma unroll
      for (int i = 0; i < C::KB; ++i) {
        const bool live = good && t + i < hi;
        const uint32_t to = ring + stage * C::STAGE_BYTES + i * 512;
        cp_async16_zfill(to, live ? kp + at + i * c.token_stride : kp, live);
        cp_async16_zfill(to + C::KB * 512, live ? vp + at + i * c.token_stride : vp, live);
      }
    };
    const auto staged = [&](int stage, int i) {
      return *reinterpret_cast<const float4*>(ring_raw + warp * C::STAGES * C::STAGE_BYTES + stage * C::STAGE_BYTES +
                                              i * 512 + lane * 16);
    };
    int page = page_of(m), stage = 0;
    if constexpr (C::STAGES > 1) {
      int pages[C::STAGES];
#pragma unroll
      for (int i = 0; i < C::STAGES; ++i) pages[i] = page_of(m + i * STEP);
#pragma unroll
      for (int i = 0; i < C::STAGES - 1; ++i) {
        if (lo + i * STEP < hi) issue(m + i * STEP, pages[i], i);
        cp_async_commit();
      }
      page = pages[C::STAGES - 1];
    }
    for (int m0 = lo; m0 < hi; m0 += STEP, m += STEP) {
      float4 k[C::KB], v[C::KB];
      bool good;
      if constexpr (C::STAGES > 1) {
        // the stage before this one has been read: its place is the next one's
        const int next = page_of(m + C::STAGES * STEP);
        if (m0 + (C::STAGES - 1) * STEP < hi)
          issue(m + (C::STAGES - 1) * STEP, page, stage == 0 ? C::STAGES - 1 : stage - 1);
        cp_async_commit();
        page = next;
        cp_async_wait<C::STAGES - 1>();
        good = goods >> stage & 1;
#pragma unroll
        for (int i = 0; i < C::KB; ++i) k[i] = staged(stage, i);
      } else {
        const int next = page_of(m + STEP);
        good = page_good(m, page);
        fetch(k, kp, m, page, good);
        fetch(v, vp, m, page, good);
        page = next;
      }
      float s[C::V];
#pragma unroll
      for (int i = 0; i < C::KB; ++i)
#pragma unroll
        for (int h = 0; h < GP; ++h)
          s[i * GP + h] = fmaf(qf[h].x, k[i].x, fmaf(qf[h].y, k[i].y, fmaf(qf[h].z, k[i].z, qf[h].w * k[i].w)));
      sum_scatter<C::V, C::LPK>(s);
      // this lane's logits, the new maxima of their heads (over the group's keys), the weights
      float w[C::HAVE], top[C::HAVE];
      bool grew = false;
#pragma unroll
      for (int i = 0; i < C::HAVE; ++i) {
        w[i] = good && m + key_of < hi ? fmaf(s[i], p.c2, s[i] * p.c2_low) : -INFINITY;
        if (p.logits && counts && good && m + key_of < hi && head_of + i < p.G)
          p.logits[((size_t)r * c.cap + m + key_of) * p.gpad + head_of + i] = w[i];
        top[i] = w[i];
      }
#pragma unroll
      for (int b = C::SAME * GP / C::HAVE; b < C::LPK; b <<= 1)
#pragma unroll
        for (int i = 0; i < C::HAVE; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], b));
#pragma unroll
      for (int i = 0; i < C::HAVE; ++i) {
        top[i] = fmaxf(top[i], mx[i]);
        grew |= top[i] > mx[i];
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < C::HAVE; ++i) {
          const float f = paged::weight(mx[i], top[i]);
          sum[i] *= f;
          lost[i] *= f;
          mx[i] = top[i];
          if (counts && key_of == 0) factor_sh[state][head_of + i] = f;
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float f = factor_sh[state][h];
          o[h].x *= f;
          o[h].y *= f;
          o[h].z *= f;
          o[h].w *= f;
        }
      }
#pragma unroll
      for (int i = 0; i < C::HAVE; ++i) {
        w[i] = w[i] == -INFINITY ? 0.f : fast_exp2(w[i] - mx[i]);
        const float to = sum[i] + w[i];
        lost[i] += w[i] - (to - sum[i]);
        sum[i] = to;
        if (counts) weight_sh[state][first_value + i] = w[i];
      }
      if constexpr (C::STAGES > 1) {
#pragma unroll
        for (int i = 0; i < C::KB; ++i) v[i] = staged(stage, C::KB + i);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < C::KB; ++i)
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float w1 = weight_sh[state][i * GP + h];
          const float2 f = make_float2(w1, w1);
          const float2 a = fma2(f, make_float2(v[i].x, v[i].y), make_float2(o[h].x, o[h].y));
          const float2 b = fma2(f, make_float2(v[i].z, v[i].w), make_float2(o[h].z, o[h].w));
          o[h] = make_float4(a.x, a.y, b.x, b.y);
        }
      if constexpr (C::STAGES > 1) stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      __syncwarp();                          // the weights are read
    }
    // the sums of the lanes that share a head, then the states of the CTA
#pragma unroll
    for (int i = 0; i < C::HAVE; ++i) {
      float t = sum[i] + lost[i];
#pragma unroll
      for (int b = C::SAME * GP / C::HAVE; b < C::LPK; b <<= 1) t += __shfl_xor_sync(0xffffffffu, t, b);
      if (counts && key_of == 0) {
        st_m[state][head_of + i] = mx[i];
        st_l[state][head_of + i] = t;
      }
    }
#pragma unroll
    for (int h = 0; h < GP; ++h)
      if (h < p.G) *reinterpret_cast<float4*>(&st_o[state][h][dl * 4]) = o[h];
    __syncthreads();
    const bool whole = u == 0 && u1 == nt;
    float* part = p.part + ((size_t)cta * 2 + (u > 0 ? 0 : 1)) * p.pstride;
    for (int e = tid; e < p.G * D; e += C::THREADS) {
      const int h = e / D, d = e % D;
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < C::STATES; ++w) M = fmaxf(M, st_m[w][h]);
#pragma unroll
      for (int w = 0; w < C::STATES; ++w) {
        const float f = paged::weight(st_m[w][h], M);
        L = fmaf(st_l[w][h], f, L);
        O = fmaf(st_o[w][h][d], f, O);
      }
      if (whole) {
        const size_t head = (size_t)l * p.Hq + hk * p.G + h;
        reinterpret_cast<float*>(p.out)[head * D + d] = L == 0.f ? 0.f : O / L;
        if (d == 0) {
          const float l2 = L == 0.f ? -INFINITY : M + log2f(L);
          if (p.lse) p.lse[head] = l2 * KVP_LN2;
          if (p.lse2) p.lse2[(size_t)r * p.gpad + h] = l2;
          factor_sh[0][h] = l2;              // (the factors are not in use here)
        }
      } else {
        part[2 * p.gpad + e] = O;
        if (d == 0) {
          part[h] = M;
          part[p.gpad + h] = L;
        }
      }
    }
    __syncthreads();
    if (p.whole && p.logits) {
      constexpr int PAD = GP <= 8 ? 8 : 16;
      paged::add_row_scores<PAD>(p, r, tid, n, C::THREADS, factor_sh[0]);
      __syncthreads();
    }
    x += u1 - u;
    ++r;
    u = 0;
  }
}

template <int D>
cudaError_t run_f32(const Params& p, const void* q, cudaStream_t st) {
  const auto go = [&](auto kernel, int threads, int smem) {
    if (smem > 0) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
    count_launches(1);
    return launch_with_pdl(kernel, dim3((unsigned)p.ctas), dim3((unsigned)threads), (size_t)smem, st, (const float*)q, p);
  };
  if (p.G == 1) return go(paged_decode_f32_kernel<D, 1>, Pf<D, 1>::THREADS, Pf<D, 1>::SMEM);
  if (p.G == 2) return go(paged_decode_f32_kernel<D, 2>, Pf<D, 2>::THREADS, Pf<D, 2>::SMEM);
  if (p.G <= 4) return go(paged_decode_f32_kernel<D, 4>, Pf<D, 4>::THREADS, Pf<D, 4>::SMEM);
  if (p.G <= 8) return go(paged_decode_f32_kernel<D, 8>, Pf<D, 8>::THREADS, Pf<D, 8>::SMEM);
  return go(paged_decode_f32_kernel<D, 16>, Pf<D, 16>::THREADS, Pf<D, 16>::SMEM);
}

// Merges the partials of the rows that several CTAs share, and adds the tokens' probabilities to the
// scores once the rows' log-sum-exps are known.  Block (c, y) belongs to CTA c of the decode kernel:
// it merges the row that continues from CTA c - 1 if that CTA held its first tiles, and scores c's
// own keys; y shares out the outputs and the tiles.
constexpr int JOIN_THREADS = 256;

// Base-2 log-sum-exp of every head of a row whose parts CTAs [lo, hi] hold, and (weights not null) what
// each part weighs in it: a warp per head, a lane per part, the reads of all parts in flight at once.
// Ends with a barrier.
template <int GP>
__device__ __forceinline__ void join_states(const Params& p, int lo, int hi, float* lse_sh, float* weights) {
  const int lane = threadIdx.x & 31, n = hi - lo + 1;
  // part i of the row: CTA lo has it in slot 1, the others in slot 0
  const auto at = [&](int i) { return p.part + ((size_t)(lo + i) * 2 + (i == 0 ? 1 : 0)) * p.pstride; };
  for (int h = threadIdx.x >> 5; h < p.G; h += JOIN_THREADS / 32) {
    constexpr int K = 4;                     // parts per lane and step
    float M = -INFINITY, L = 0.f, m[K], l[K];
    for (int i0 = 0; i0 < n; i0 += 32 * K) {
      float top = M;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = i0 + 32 * k + lane;
        m[k] = i < n ? at(i)[h] : -INFINITY;
        l[k] = i < n ? at(i)[GP + h] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) top = fmaxf(top, m[k]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) s = fmaf(l[k], paged::weight(m[k], top), s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      L = fmaf(L, paged::weight(M, top), s);
      M = top;
    }
    if (lane == 0) lse_sh[h] = L == 0.f ? -INFINITY : M + log2f(L);
    if (weights)
      for (int i = lane, k = 0; i < n; i += 32, ++k) {
        const float mi = n <= 32 ? m[0] : at(i)[h];
        weights[i * GP + h] = L == 0.f ? 0.f : paged::weight(mi, M) / L;
      }
  }
  __syncthreads();
}

template <typename T, int D, int GP>
__global__ void __launch_bounds__(JOIN_THREADS) paged_join_kernel(const Params p, int add_scores) {
  extern __shared__ float weights[];         // [ctas][GP]
  __shared__ float lse_sh[GP];
  __shared__ float4 sum_sh[JOIN_THREADS];
  wait_prior_grid();
  allow_next_grid();                         // few, short blocks: the next kernel may take its places beside them
  const int cta = blockIdx.x, y = blockIdx.y, ny = gridDim.y, tid = threadIdx.x;
  const Range g = p.range[cta];
  if (cta >= g.active) return;
  if (g.tile > 0 && g.lo == cta - 1) {
    const int lo = g.lo, hi = g.hi;
    const size_t head0 = (size_t)(g.row / p.Hkv) * p.Hq + (size_t)(g.row % p.Hkv) * p.G;
    // a thread per quad of outputs and eight parts; with more parts, several threads per quad
    int lanes = JOIN_THREADS;                // quads per block
    while (lanes > 32 && (hi - lo + 1) > 8 * (JOIN_THREADS / lanes)) lanes >>= 1;
    const int split = JOIN_THREADS / lanes, grp = tid / lanes, quads = p.G * D / 4;
    bool ready = false;
    for (int q0 = y * lanes; q0 < quads; q0 += ny * lanes) {
      const int e = 4 * (q0 + tid % lanes), h = e / D;
      const bool mine = e < p.G * D;
      const auto out_of = [&](int i) {
        return *reinterpret_cast<const float4*>(p.part + ((size_t)(lo + i) * 2 + (i == 0 ? 1 : 0)) * p.pstride +
                                                2 * GP + e);
      };
      // the first outputs are fetched beside the states that weigh them
      float4 early[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        early[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine && grp + k * split <= hi - lo) early[k] = out_of(grp + k * split);
      }
      if (!ready) join_states<GP>(p, lo, hi, lse_sh, weights);
      ready = true;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      const auto add = [&](const float4& x, float f) {
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
      };
      if (mine) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (grp + k * split <= hi - lo) add(early[k], weights[(grp + k * split) * GP + h]);
#pragma unroll 8
        for (int i = grp + 8 * split; i <= hi - lo; i += split) add(out_of(i), weights[i * GP + h]);
      }
      if (split > 1) {
        __syncthreads();                     // the quads before have been summed
        sum_sh[tid] = o;
        __syncthreads();
        if (grp == 0)
          for (int k = 1; k < split; ++k) add(sum_sh[k * lanes + tid], 1.f);
      }
      if (grp == 0 && mine) {
        paged::store_out4<T>(p, head0 * D + e, o);
        if (p.lse && e % D == 0) p.lse[head0 + h] = lse_sh[h] * KVP_LN2;
      }
    }
  }
  if (!add_scores) return;
  int r = g.row, u = g.tile;
  for (int x = g.begin; x < g.end;) {
    const int n = paged::row_len(p, r), nt = paged::tiles_of(n);
    if (nt == 0) {
      ++r;
      u = 0;
      continue;
    }
    const int u1 = min(nt, u + (g.end - x));
    __syncthreads();                         // the row before is done with lse_sh
    if (u == 0 && u1 == nt) {
      if (tid < p.G) lse_sh[tid] = p.lse2[(size_t)r * GP + tid];
      __syncthreads();
    } else {
      join_states<GP>(p, paged::cta_of(x - u, g.total, g.active), paged::cta_of(x - u + nt - 1, g.total, g.active),
                      lse_sh, nullptr);
    }
    paged::add_row_scores<GP>(p, r, u * TILE + y * JOIN_THREADS + tid, min(n, u1 * TILE), ny * JOIN_THREADS, lse_sh);
    x += u1 - u;
    ++r;
    u = 0;
  }
}

// The same of few rows, which have many parts each, when no scores are asked for: a block joins JOIN_LANES
// quads of outputs of one head.  It finds the row's parts from the lengths, so that there is a block per
// result and not per CTA of the decode kernel, and reads all its states and outputs in one go.
constexpr int JOIN_LANES = 8;
// Parts a row can have for that.  GPU time of a call with the other kernel / this one, rows of 8192 tokens,
// D 128: 1 row of 8 query heads on a KV head 11.9 / 8.6 us, 8 rows 15.2 / 12.2, 16 rows 15.6 / 15.7, 24 rows
// 19.7 / 21.4; 16 heads 18.4 / 10.6, 24.5 / 17.3, 25.6 / 24.3, 32.4 / 33.4; 1 row of 131072 tokens 25.5 / 14.7.
constexpr int FEW_PARTS = 16;

template <typename T, int D, int GP>
__global__ void __launch_bounds__(JOIN_THREADS) paged_join_few_kernel(const Params p) {
  constexpr int GROUPS = JOIN_THREADS / JOIN_LANES, WARPS = JOIN_THREADS / 32;
  constexpr int K = MAX_CTAS / GROUPS, KS = MAX_CTAS / JOIN_THREADS;
  __shared__ float weights[MAX_CTAS], red[2][WARPS];
  __shared__ float4 sum_sh[WARPS * JOIN_LANES];
  wait_prior_grid();
  allow_next_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / p.G, h = blockIdx.x % p.G;
  int before = 0, mine = 0, total = 0;
  for (int x = lane; x < p.c.R; x += 32) {
    const int t = paged::tiles_of(paged::row_len(p, x));
    total += t;
    if (x < r) before += t;
    if (x == r) mine = t;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  before = __reduce_add_sync(0xffffffffu, before);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (mine == 0) return;
  const int active = paged::active_ctas(p, total);
  const int lo = paged::cta_of(before, total, active), n = paged::cta_of(before + mine - 1, total, active) - lo + 1;
  if (n == 1) return;                        // finished where it was read
  const auto at = [&](int i) { return p.part + ((size_t)(lo + i) * 2 + (i == 0 ? 1 : 0)) * p.pstride; };
  const int e = 4 * (blockIdx.y * JOIN_LANES + tid % JOIN_LANES), grp = tid / JOIN_LANES;
  float m[KS], l[KS];
  float4 x[K];
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int i = tid + k * JOIN_THREADS;
    m[k] = i < n ? at(i)[h] : -INFINITY;
    l[k] = i < n ? at(i)[GP + h] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp + k * GROUPS < n) x[k] = *reinterpret_cast<const float4*>(at(grp + k * GROUPS) + 2 * GP + h * D + e);
  }
  float M = m[0];
#pragma unroll
  for (int k = 1; k < KS; ++k) M = fmaxf(M, m[k]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = fmaxf(M, red[0][w]);
  float L = 0.f;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const float f = paged::weight(m[k], M);
    weights[tid + k * JOIN_THREADS] = f;
    L = fmaf(l[k], f, L);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  L = red[1][0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) L += red[1][w];
  const float inv = L == 0.f ? 0.f : 1.f / L;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](const float4& a, float f) {
    o.x = fmaf(a.x, f, o.x);
    o.y = fmaf(a.y, f, o.y);
    o.z = fmaf(a.z, f, o.z);
    o.w = fmaf(a.w, f, o.w);
  };
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (grp + k * GROUPS < n) add(x[k], weights[grp + k * GROUPS] * inv);
  // the groups' sums: those of a warp by shuffles, then the warps'
#pragma unroll
  for (int off = JOIN_LANES; off < 32; off <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
  }
  if (lane < JOIN_LANES) sum_sh[warp * JOIN_LANES + lane] = o;
  __syncthreads();
  if (tid >= JOIN_LANES) return;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) add(sum_sh[w * JOIN_LANES + tid], 1.f);
  const size_t head = (size_t)(r / p.Hkv) * p.Hq + (size_t)(r % p.Hkv) * p.G + h;
  paged::store_out4<T>(p, head * D + e, o);
  if (p.lse && e == 0) p.lse[head] = L == 0.f ? -INFINITY : (M + log2f(L)) * KVP_LN2;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int decode_ctas() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return 2 * sms < paged::MAX_CTAS ? 2 * sms : paged::MAX_CTAS;
}

int padded_group(int G) { return G <= 8 ? 8 : 16; }

size_t layout(const PagedView& c, int G, int add_scores, Params* p, void* ws) {
  const int GP = padded_group(G), ctas = decode_ctas();
  char* base = (char*)ws;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    char* x = base ? base + at : nullptr;
    at += align256(bytes);
    return x;
  };
  p->ctas = ctas;
  p->gpad = GP;
  p->logits = add_scores ? (float*)take((size_t)c.R * c.cap * GP * 4) : nullptr;
  p->whole = (c.cap + TILE - 1) / TILE <= paged::whole_tiles(c.dtype) &&
             c.R <= paged::WHOLE_ROWS * ctas;
  if (p->whole) {
    if (p->ctas > c.R) p->ctas = c.R;
    return at;
  }
  p->pstride = 2 * GP + GP * c.D;
  p->part = (float*)take((size_t)ctas * 2 * p->pstride * 4);
  p->range = (Range*)take((size_t)ctas * sizeof(Range));
  p->lse2 = add_scores ? (float*)take((size_t)c.R * GP * 4) : nullptr;
  return at;
}

template <typename T, int D, int GP>
cudaError_t run(const Params& p, const PagedDecodeArgs& a, cudaStream_t st) {
  cudaError_t e;
  if constexpr (sizeof(T) == 2) e = launch_paged_decode_mma(p, a.q, st);
  else e = run_f32<D>(p, a.q, st);
  if (e != cudaSuccess) return e;
  if (p.whole) return cudaSuccess;           // every row has been finished, and scored, where it was read
  if (!a.add_scores && (long long)FEW_PARTS * p.c.R < p.ctas) {
    count_launches(1);
    return launch_with_pdl(paged_join_few_kernel<T, D, GP>, dim3((unsigned)(p.c.R * p.G), D / (4 * JOIN_LANES)),
                           dim3(JOIN_THREADS), 0, st, p);
  }
  // Blocks per CTA of the decode kernel.  Rows of which there are many have few parts each (one block
  // joins 1024 outputs of up to 8 parts in one go); of a few long rows the outputs are dealt out
  // further, and so are the scores of long ranges.
  int slices = (p.G * D + 1023) / 1024;
  if (8LL * p.c.R < p.ctas) slices = (p.G * D + 127) / 128;
  if (a.add_scores) {
    const long long keys = (long long)p.c.R * p.c.cap / p.ctas;
    while (slices < 8 && keys > 4LL * JOIN_THREADS * slices) slices *= 2;
  }
  count_launches(1);
  return launch_with_pdl(paged_join_kernel<T, D, GP>, dim3((unsigned)p.ctas, (unsigned)slices), dim3(JOIN_THREADS),
                         (size_t)p.ctas * GP * sizeof(float), st, p, a.add_scores);
}

}  // namespace

size_t paged_decode_workspace(const PagedView& c, int h_q, int h_kv, int add_scores) {
  Params p{};
  return layout(c, h_q / h_kv, add_scores, &p, nullptr);
}

cudaError_t launch_paged_decode(const PagedView& c, const PagedDecodeArgs& a, void* ws, int* status,
                                cudaStream_t st) {
  Params p{};
  p.c = c;
  p.Hq = a.h_q;
  p.Hkv = a.h_kv;
  p.G = a.h_q / a.h_kv;
  p.q_stride = a.q_stride;
  const double c2 = a.scale * 1.4426950408889634;
  p.c2 = (float)c2;
  // The fp32 kernel's logit is s * c2 + s * c2_low, which for an infinite s has to be infinite too: c2_low
  // gets c2's sign and is 0 only with it.  (A test in the kernel costs 3 % with 4 query heads a group, 5 % with 16.)
  if (c.dtype == KVP_F32 && std::fabs((double)p.c2) > std::fabs(c2)) p.c2 = std::nextafter(p.c2, 0.f);
  p.c2_low = (float)(c2 - (double)p.c2);
  if (c.dtype == KVP_F32 && p.c2 != 0.f && p.c2_low == 0.f) p.c2_low = std::copysign(FLT_MIN, p.c2);
  p.out = a.out;
  p.out_f32 = a.out_f32;
  p.lse = a.lse;
  p.status = status;
  layout(c, p.G, a.add_scores, &p, ws);
#define KVP_PD(TT, DD) \
  return p.G <= 8 ? run<TT, DD, 8>(p, a, st) : run<TT, DD, 16>(p, a, st)
  if (c.dtype == KVP_BF16) {
    if (c.D == 128) KVP_PD(__nv_bfloat16, 128);
    KVP_PD(__nv_bfloat16, 64);
  }
  if (c.dtype == KVP_F16) {
    if (c.D == 128) KVP_PD(__half, 128);
    KVP_PD(__half, 64);
  }
  if (c.D == 128) KVP_PD(float, 128);
  KVP_PD(float, 64);
#undef KVP_PD
}

}  // namespace kvp
