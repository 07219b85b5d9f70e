// One-token decode attention over the paged cache.
//
// How much KV cache can you prune, "What we did" / "Bounded windows" (one-token attention over the
// retained entries) over rows of pages:
//   out = sum_t softmax_t(scale * q . k_t) v_t,  lse = ln sum_t exp(scale * q . k_t).
// Base-2 online softmax; the state (maximum, sum, output) stays in fp32 registers.  The split is
// described in paged_decode.cuh.
#include <type_traits>

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "paged_decode.cuh"

namespace kvp {
namespace {

using paged::Params;
using paged::Range;
using paged::TILE;

constexpr int PD_WARPS = 4;

// Each warp takes every fourth step of keys; a key's row is read by a group of lanes with 16-byte
// loads, the partial dot products are summed across the group.
template <typename T, int D, int GP>
__global__ void __launch_bounds__(PD_WARPS * 32) paged_decode_kernel(const T* __restrict__ q, const Params p) {
  constexpr int EV = 16 / sizeof(T), LPK = D / EV, KPW = 32 / LPK, UN = 4;
  __shared__ int scan_sh[41];
  __shared__ float st_m[PD_WARPS][GP], st_l[PD_WARPS][GP];
  __shared__ float st_o[PD_WARPS][GP][D];
  wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane / LPK, dl = lane % LPK;
  const int cta = blockIdx.x;
  const Range g = paged::find_range(p, cta, scan_sh);
  paged::empty_rows<T, D>(p, cta);
  if (cta >= g.active) return;
  const PagedView& c = p.c;
  const T* kp = (const T*)c.k + dl * EV;
  const T* vp = (const T*)c.v + dl * EV;

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
    float qf[GP][EV], mx[GP], sm[GP], o[GP][EV];
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      mx[h] = -INFINITY;
      sm[h] = 0.f;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (h < p.G) w = *reinterpret_cast<const uint4*>(q + l * p.q_stride + (size_t)(hk * p.G + h) * D + dl * EV);
      Vec16<T>::unpack(w, qf[h]);
#pragma unroll
      for (int t = 0; t < EV; ++t) o[h][t] = 0.f;
    }
    const int32_t* table = c.table + (size_t)r * c.max_pages;
    for (int m0 = lo; m0 < hi; m0 += PD_WARPS * KPW * UN) {
      uint4 ku[UN], vu[UN];
      bool ok[UN];
#pragma unroll
      for (int s = 0; s < UN; ++s) {
        const int m = m0 + (s * PD_WARPS + warp) * KPW + sub;
        ok[s] = m < hi;
        ku[s] = vu[s] = make_uint4(0, 0, 0, 0);
        if (ok[s]) {
          const int pg = table[m >> c.shift];
          ok[s] = pg >= 0 && pg < c.n_pages;
          if (ok[s]) {
            const int64_t at = pg * c.page_stride + (m & (c.ps - 1)) * c.token_stride;
            ku[s] = ld_stream16(kp + at);
            vu[s] = ld_stream16(vp + at);
          } else {
            raise_status(p.status, KVP_ERR_DEVICE_CHECK);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < UN; ++s) {
        const int m = m0 + (s * PD_WARPS + warp) * KPW + sub;
        float kf[EV], vf[EV];
        Vec16<T>::unpack(ku[s], kf);
        Vec16<T>::unpack(vu[s], vf);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          if (h >= p.G) break;
          float a = 0.f;
#pragma unroll
          for (int t = 0; t < EV; ++t) a = fmaf(qf[h][t], kf[t], a);
#pragma unroll
          for (int off = LPK / 2; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
          a = paged::base2(p, a);
          if (!ok[s]) continue;
          if (p.logits && dl == 0) p.logits[((size_t)r * c.cap + m) * GP + h] = a;
          if (a > mx[h]) {
            const float f = fast_exp2(mx[h] - a);
            sm[h] *= f;
#pragma unroll
            for (int t = 0; t < EV; ++t) o[h][t] *= f;
            mx[h] = a;
          }
          const float w = a == -INFINITY ? 0.f : fast_exp2(a - mx[h]);
          sm[h] += w;
#pragma unroll
          for (int t = 0; t < EV; ++t) o[h][t] = fmaf(w, vf[t], o[h][t]);
        }
      }
    }
    // the lane groups of a warp, then the warps
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      if (h >= p.G) break;
      float M = mx[h];
#pragma unroll
      for (int off = LPK; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      const float f = paged::weight(mx[h], M);
      float s = sm[h] * f;
#pragma unroll
      for (int off = LPK; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (lane == 0) {
        st_m[warp][h] = M;
        st_l[warp][h] = s;
      }
#pragma unroll
      for (int t = 0; t < EV; ++t) {
        float y = o[h][t] * f;
#pragma unroll
        for (int off = LPK; off < 32; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (sub == 0) st_o[warp][h][dl * EV + t] = y;
      }
    }
    __syncthreads();
    const bool whole = u == 0 && u1 == nt;
    float* part = p.part + ((size_t)cta * 2 + (u > 0 ? 0 : 1)) * p.pstride;
    for (int e = tid; e < p.G * D; e += PD_WARPS * 32) {
      const int h = e / D, d = e % D;
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < PD_WARPS; ++w) M = fmaxf(M, st_m[w][h]);
#pragma unroll
      for (int w = 0; w < PD_WARPS; ++w) {
        const float f = paged::weight(st_m[w][h], M);
        L = fmaf(st_l[w][h], f, L);
        O = fmaf(st_o[w][h][d], f, O);
      }
      if (whole) {
        const size_t head = (size_t)l * p.Hq + hk * p.G + h;
        paged::store_out<T>(p, head * D + d, L == 0.f ? 0.f : O / L);
        if (d == 0) {
          const float l2 = L == 0.f ? -INFINITY : M + log2f(L);
          if (p.lse) p.lse[head] = l2 * KVP_LN2;
          if (p.lse2) p.lse2[(size_t)r * GP + h] = l2;
        }
      } else {
        part[2 * GP + e] = O;
        if (d == 0) {
          part[h] = M;
          part[GP + h] = L;
        }
      }
    }
    __syncthreads();
    x += u1 - u;
    ++r;
    u = 0;
  }
}

// Merges the partials of the rows that several CTAs share, and adds the tokens' probabilities to the
// scores once the rows' log-sum-exps are known.  Block (c, y) belongs to CTA c of the decode kernel:
// it merges the row that continues from CTA c - 1 if that CTA held its first tiles, and scores c's
// own keys; y shares out the outputs and the tiles.
constexpr int JOIN_THREADS = 128;

template <typename T, int D, int GP>
__global__ void __launch_bounds__(JOIN_THREADS) paged_join_kernel(const Params p, int add_scores) {
  wait_prior_grid();
  const int cta = blockIdx.x, y = blockIdx.y, ny = gridDim.y, tid = threadIdx.x;
  __shared__ float lse_sh[GP];
  const Range g = p.range[cta];
  if (cta >= g.active) return;
  const PagedView& c = p.c;
  const auto part = [&](int i, int first) {   // partial of CTA i of a row whose first tiles CTA `first` has
    return p.part + ((size_t)i * 2 + (i == first ? 1 : 0)) * p.pstride;
  };
  if (g.tile > 0) {
    const int x0 = g.begin - g.tile, c_lo = paged::cta_of(x0, g.total, g.active);
    if (c_lo == cta - 1) {
      const int nt = paged::tiles_of(paged::row_len(p, g.row));
      const int c_hi = paged::cta_of(x0 + nt - 1, g.total, g.active);
      const size_t head0 = (size_t)(g.row / p.Hkv) * p.Hq + (size_t)(g.row % p.Hkv) * p.G;
      for (int e = y * JOIN_THREADS + tid; e < p.G * D; e += ny * JOIN_THREADS) {
        const int h = e / D;
        float M = -INFINITY;
        for (int i = c_lo; i <= c_hi; ++i) M = fmaxf(M, part(i, c_lo)[h]);
        float L = 0.f, O = 0.f;
        for (int i = c_lo; i <= c_hi; ++i) {
          const float* q = part(i, c_lo);
          const float f = paged::weight(q[h], M);
          L = fmaf(q[GP + h], f, L);
          O = fmaf(q[2 * GP + e], f, O);
        }
        paged::store_out<T>(p, head0 * D + e, L == 0.f ? 0.f : O / L);
        if (p.lse && e % D == 0) p.lse[head0 + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * KVP_LN2;
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
    const bool whole = u == 0 && u1 == nt;
    __syncthreads();
    if (tid < p.G) {
      if (whole) {
        lse_sh[tid] = p.lse2[(size_t)r * GP + tid];
      } else {
        const int x0 = x - u;
        const int c_lo = paged::cta_of(x0, g.total, g.active), c_hi = paged::cta_of(x0 + nt - 1, g.total, g.active);
        float M = -INFINITY, L = 0.f;
        for (int i = c_lo; i <= c_hi; ++i) M = fmaxf(M, part(i, c_lo)[tid]);
        for (int i = c_lo; i <= c_hi; ++i) {
          const float* q = part(i, c_lo);
          L = fmaf(q[GP + tid], paged::weight(q[tid], M), L);
        }
        lse_sh[tid] = L == 0.f ? -INFINITY : M + log2f(L);
      }
    }
    __syncthreads();
    const int hi = min(n, u1 * TILE);
    for (int m = u * TILE + y * JOIN_THREADS + tid; m < hi; m += ny * JOIN_THREADS) {
      const float* lg = p.logits + ((size_t)r * c.cap + m) * GP;
      float s = 0.f;
#pragma unroll
      for (int h = 0; h < GP; ++h)
        if (h < p.G && lg[h] != -INFINITY) s += fast_exp2(lg[h] - lse_sh[h]);
      c.score[(size_t)r * c.cap + m] += s;
    }
    x += u1 - u;
    ++r;
    u = 0;
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int decode_ctas() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return 2 * sms;
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
  p->pstride = 2 * GP + GP * c.D;
  p->part = (float*)take((size_t)ctas * 2 * p->pstride * 4);
  p->range = (Range*)take((size_t)ctas * sizeof(Range));
  p->lse2 = add_scores ? (float*)take((size_t)c.R * GP * 4) : nullptr;
  p->logits = add_scores ? (float*)take((size_t)c.R * c.cap * GP * 4) : nullptr;
  return at;
}

template <typename T, int D, int GP>
cudaError_t run(const Params& p, const PagedDecodeArgs& a, cudaStream_t st) {
  cudaError_t e;
  if constexpr (sizeof(T) == 2) {
    e = launch_paged_decode_mma(p, a.q, st);
  } else {
    count_launches(1);
    e = launch_with_pdl(paged_decode_kernel<T, D, GP>, dim3((unsigned)p.ctas), dim3(PD_WARPS * 32), 0, st,
                        (const T*)a.q, p);
  }
  if (e != cudaSuccess) return e;
  // a row of one tile is never shared, and without scores nothing is left to do
  if (!a.add_scores && p.c.cap <= TILE) return cudaSuccess;
  const int slices = (p.G * D + JOIN_THREADS - 1) / JOIN_THREADS;
  count_launches(1);
  return launch_with_pdl(paged_join_kernel<T, D, GP>, dim3((unsigned)p.ctas, (unsigned)slices), dim3(JOIN_THREADS), 0,
                         st, p, a.add_scores);
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
  p.c2_low = (float)(c2 - (double)p.c2);
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
