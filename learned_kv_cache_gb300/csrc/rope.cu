// Rotary positions, and the norms of queries and keys with the rotation in the same pass (and their
// gradients).
//
//   n = x / sqrt(mean(x^2) + eps),  z = w n,  y = R(pos) z,
//   R(pos): pairs (a, b) of the head's first rotary_dim values -> gain (a cos t - b sin t, a sin t + b cos t),
//   t = pos * inv_freq of the pair; the values behind rotary_dim pass.
//   dz = R^T dy,  dw = sum dz n,  dx = (w dz - n mean(w dz n)) / sqrt(mean(x^2) + eps)
//
// A few operations per value: bound by HBM (every input read once, every output written once).
//
//  * Angles.  pos * inv_freq reaches 1e5 radians, of which a float keeps 1e-2.  The host gives each pair's
//    frequency in turns as a fraction of 2^64, so that the angle is one 64-bit product whose overflow drops
//    the whole turns: exact up to 2^-64 of a turn per position, for every 32-bit position.  Its upper 32
//    bits, less the nearest quarter turn, are exact to 2^-25 of an eighth of a turn as a float.
//  * The unit of work is a token with some of a tensor's heads, and D / 16 lanes have one: they compute its
//    cosines and sines (8 pairs a lane, while the first rows are on their way) and walk over the heads, the
//    next rows' loads always ahead of the arithmetic.  Nothing is shared, so no warp waits for another (with
//    the angles in shared memory and a few tokens a block, 8192 tokens of 32 + 8 heads took 52 us).
//  * A lane owns 8 pairs of a row: two vectors of 8 values that lie rotary_dim / 2 apart (halves) or side
//    by side (interleaved), so pairs never cross lanes and sums over a row are 2 or 3 shuffles.
//  * Lane groups side by side have tokens side by side: in a tensor laid out by heads their rows touch.
#include <cmath>

#include "kvp_common.cuh"
#include "kvp_launch.h"

namespace kvp {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 64;
constexpr int FORWARD_BLOCKS = 2, BACK_BLOCKS = 1;          // per SM

struct Freqs {
  uint64_t step[MAX_PAIRS];   // turns per position, times 2^64
};

// Eight consecutive values as they lie in memory.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) Vec16<T>::unpack(v[i], f + i * Vec16<T>::N);
  }
};
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ void store8(__half* p, const float* f) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}

// Cosine and sine of pos * step turns.
__device__ __forceinline__ float2 turn_of(int pos, uint64_t step) {
  const uint32_t t = (uint32_t)(((uint64_t)(int64_t)pos * step) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const int rest = (int)(t - (quarter << 30));              // within an eighth of a turn of it
  float s, c;
  sincospif((float)rest * 0x1p-31f, &s, &c);
  switch (quarter & 3) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

// The lane's place in a row.
template <int D, bool INTERLEAVED>
struct Lane {
  static constexpr int PER_ROW = D / 16;
  static constexpr int GROUPS = THREADS / PER_ROW;
  int u, at0, at1;        // unit; first values of its two vectors
  bool turns;
  __device__ __forceinline__ Lane(int rotary_dim) {
    u = threadIdx.x % PER_ROW;
    turns = 16 * u < rotary_dim;
    at0 = INTERLEAVED || !turns ? 16 * u : 8 * u;
    at1 = INTERLEAVED || !turns ? 16 * u + 8 : 8 * u + (rotary_dim >> 1);
  }
};
template <int PER_ROW>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < PER_ROW; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The pairs (a, b) of a lane turned by cs.  dir = 1: by the angle; -1: back.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&x)[2][8], const float2 (&cs)[8], float dir) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = INTERLEAVED ? x[i >> 2][2 * (i & 3)] : x[0][i];
    float& b = INTERLEAVED ? x[i >> 2][2 * (i & 3) + 1] : x[1][i];
    const float c = cs[i].x, s = cs[i].y * dir, y = a * c - b * s;
    b = b * c + a * s;
    a = y;
  }
}

// Units of a tensor: token by token for the first `chunk` heads, then for the next.
struct Split {
  uint32_t n_tokens;
  int chunk;
  uint32_t units[2];     // of either tensor
};
// A unit: rows [h0, h0 + n) of a tensor's heads at a token (none: n = 0).
struct Unit {
  int b, s, h0, n;
  __device__ __forceinline__ Unit(const RopeArgs& a, const Split& split, int heads, uint32_t u, bool live) {
    const uint32_t part = live ? u / split.n_tokens : 0, t = live ? u - part * split.n_tokens : 0;
    b = (int)(t / (uint32_t)a.seq_len);
    s = (int)(t - (uint32_t)b * a.seq_len);
    h0 = part * split.chunk;
    n = live ? min(split.chunk, heads - h0) : 0;
  }
};

// What every block has in shared memory.
template <int D>
struct Tables {
  uint64_t step[MAX_PAIRS];
  float w[2][D];         // weights (1 without any)
};
template <typename T, int D, bool NORM>
__device__ __forceinline__ void fill_tables(Tables<D>& sh, const RopeArgs& a, const Freqs& f) {
  if (threadIdx.x < MAX_PAIRS) sh.step[threadIdx.x] = f.step[threadIdx.x];
  wait_prior_grid();
  allow_next_grid();
  if (NORM && threadIdx.x < 2 * D) {
    const int j = threadIdx.x / D, i = threadIdx.x % D;
    const void* w = j ? a.t[1].w : a.t[0].w;
    sh.w[j][i] = !w ? 1.f : a.w_f32 ? ((const float*)w)[i] : to_f32<T>(((const T*)w)[i]);
  }
  __syncthreads();
}
__device__ __forceinline__ int position(const RopeArgs& a, const Unit& u) {
  return a.positions ? a.positions[u.b * a.position_stride + u.s] : a.start + u.s;
}
// Cosines and sines (times gain) of the lane's pairs.
__device__ __forceinline__ void turns(const RopeArgs& a, const uint64_t* step, int pos, bool rotates, float2 (&cs)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 v = make_float2(1.f, 0.f);
    if (rotates) {
      v = turn_of(pos, step[i]);
      v.x *= a.gain;
      v.y *= a.inverse ? -a.gain : a.gain;
    }
    cs[i] = v;
  }
}
__device__ __forceinline__ void load_w(const float* w, int at0, int at1, float (&out)[2][8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(&out[0][i]) = *reinterpret_cast<const float4*>(w + at0 + i);
    *reinterpret_cast<float4*>(&out[1][i]) = *reinterpret_cast<const float4*>(w + at1 + i);
  }
}

template <typename T, int D, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, FORWARD_BLOCKS)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Freqs f, const Split split) {
  using L = Lane<D, INTERLEAVED>;
  // rows at a time: twice these in registers (four with norms spill: 457 us for 434)
  constexpr int U = sizeof(T) == 4 ? 2 : NORM ? 3 : 4;
  __shared__ __align__(16) Tables<D> sh;
  const L lane(a.rotary_dim);
  fill_tables<T, D, NORM>(sh, a, f);
  const uint32_t all = split.units[0] + split.units[1];
  const uint32_t first = blockIdx.x * L::GROUPS + threadIdx.x / 32 * (32 / L::PER_ROW);   // the warp's
  for (uint32_t u0 = first; u0 < all; u0 += gridDim.x * L::GROUPS) {
    const uint32_t id = u0 + (threadIdx.x & 31) / L::PER_ROW;
    const bool second = id >= split.units[0];
    const RopeTensor& z = second ? a.t[1] : a.t[0];
    const Unit u(a, split, z.heads, second ? id - split.units[0] : id, id < all);
    const int64_t xs = z.xs[1], ys = z.ys[1];
    const T* in = (const T*)z.x + u.b * z.xs[0] + u.s * z.xs[2] + u.h0 * xs;
    T* out = (T*)z.y + u.b * z.ys[0] + u.s * z.ys[2] + u.h0 * ys;
    const auto load = [&](Raw<T> (&raw)[U][2], int h) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (h + k < u.n) {
          raw[k][0].load(in + (h + k) * xs + lane.at0);
          raw[k][1].load(in + (h + k) * xs + lane.at1);
        }
    };
    float2 cs[8];
    const auto rows = [&](const Raw<T> (&raw)[U][2], int h) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float v[2][8];
        raw[k][0].get(v[0]);
        raw[k][1].get(v[1]);
        if (NORM) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[0][i], v[0][i], fmaf(v[1][i], v[1][i], ss));
          const float r = __frsqrt_rn(row_sum<L::PER_ROW>(ss) * (1.f / D) + a.eps);
          float w[2][8];
          load_w(sh.w[second], lane.at0, lane.at1, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[0][i] = v[0][i] * r * w[0][i];
            v[1][i] = v[1][i] * r * w[1][i];
          }
        }
        if (lane.turns) turn<INTERLEAVED>(v, cs, 1.f);
        if (h + k < u.n) {
          store8(out + (h + k) * ys + lane.at0, v[0]);
          store8(out + (h + k) * ys + lane.at1, v[1]);
        }
      }
    };
    // every lane of the warp takes as many steps as any: sums over a row are the whole warp's shuffles
    const int most = __reduce_max_sync(0xffffffffu, u.n);
    Raw<T> even[U][2], odd[U][2];
    const int pos = position(a, u);
    load(even, 0);
    turns(a, sh.step + 8 * lane.u, pos, lane.turns, cs);
    for (int h = 0; h < most; h += 2 * U) {
      load(odd, h + U);
      rows(even, h);
      if (h + U >= most) break;
      load(even, h + 2 * U);
      rows(odd, h + U);
    }
  }
}

// Gradients: blocks [0, split_at) have the first tensor's units, the rest the second's.  A lane sums its 16
// values' weight gradients over all its rows in registers; the block's groups are added at the end, and the
// blocks' sums by rope_weight_kernel in a fixed order.
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, BACK_BLOCKS)
    norm_rope_backward_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Freqs f, const Split split,
                              int split_at, float* __restrict__ part) {
  using L = Lane<D, INTERLEAVED>;
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  __shared__ __align__(16) Tables<D> sh;
  __shared__ float sum_sh[THREADS / 32][D];
  const L lane(a.rotary_dim);
  fill_tables<T, D, true>(sh, a, f);
  const bool second = (int)blockIdx.x >= split_at;
  const uint32_t block = second ? blockIdx.x - split_at : blockIdx.x, blocks = second ? gridDim.x - split_at : split_at;
  const RopeTensor& z = second ? a.t[1] : a.t[0];
  const uint32_t all = split.units[second];
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  const uint32_t first = block * L::GROUPS + threadIdx.x / 32 * (32 / L::PER_ROW);
  for (uint32_t u0 = first; u0 < all; u0 += blocks * L::GROUPS) {
    const uint32_t id = u0 + (threadIdx.x & 31) / L::PER_ROW;
    const Unit u(a, split, z.heads, id, id < all);
    const int64_t xs = z.xs[1], ds = z.dys[1], ys = z.ys[1];
    const T* in = (const T*)z.x + u.b * z.xs[0] + u.s * z.xs[2] + u.h0 * xs;
    const T* dy = (const T*)z.dy + u.b * z.dys[0] + u.s * z.dys[2] + u.h0 * ds;
    T* out = (T*)z.y + u.b * z.ys[0] + u.s * z.ys[2] + u.h0 * ys;
    const auto load = [&](Raw<T> (&raw)[U][4], int h) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (h + k < u.n) {
          raw[k][0].load(in + (h + k) * xs + lane.at0);
          raw[k][1].load(in + (h + k) * xs + lane.at1);
          raw[k][2].load(dy + (h + k) * ds + lane.at0);
          raw[k][3].load(dy + (h + k) * ds + lane.at1);
        }
    };
    float2 cs[8];
    const auto rows = [&](const Raw<T> (&raw)[U][4], int h) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float v[2][8], g[2][8], w[2][8];
        raw[k][0].get(v[0]);
        raw[k][1].get(v[1]);
        raw[k][2].get(g[0]);
        raw[k][3].get(g[1]);
        if (lane.turns) turn<INTERLEAVED>(g, cs, -1.f);
        load_w(sh.w[second], lane.at0, lane.at1, w);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(v[0][i], v[0][i], fmaf(v[1][i], v[1][i], ss));
          dot = fmaf(g[0][i] * w[0][i], v[0][i], fmaf(g[1][i] * w[1][i], v[1][i], dot));
        }
        const float r = __frsqrt_rn(row_sum<L::PER_ROW>(ss) * (1.f / D) + a.eps);
        const float mean = row_sum<L::PER_ROW>(dot) * r * (1.f / D);
        if (h + k < u.n) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float n = v[m][i] * r;
              dw[m][i] = fmaf(g[m][i], n, dw[m][i]);
              v[m][i] = r * (g[m][i] * w[m][i] - n * mean);
            }
          store8(out + (h + k) * ys + lane.at0, v[0]);
          store8(out + (h + k) * ys + lane.at1, v[1]);
        }
      }
    };
    const int most = __reduce_max_sync(0xffffffffu, u.n);
    Raw<T> even[U][4], odd[U][4];
    const int pos = position(a, u);
    load(even, 0);
    turns(a, sh.step + 8 * lane.u, pos, lane.turns, cs);
    for (int h = 0; h < most; h += 2 * U) {
      load(odd, h + U);
      rows(even, h);
      if (h + U >= most) break;
      load(even, h + 2 * U);
      rows(odd, h + U);
    }
  }
  // the groups of a warp, then the warps
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = L::PER_ROW; o < 32; o <<= 1) dw[m][i] += __shfl_xor_sync(0xffffffffu, dw[m][i], o);
      if ((threadIdx.x & 31) < L::PER_ROW) sum_sh[threadIdx.x >> 5][(m ? lane.at1 : lane.at0) + i] = dw[m][i];
    }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) sum += sum_sh[k][threadIdx.x];
    part[(size_t)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// dw of both tensors from the blocks' sums: a block per 8 columns of a tensor, its warps' lanes over the rows.
template <int D>
__global__ void __launch_bounds__(THREADS) rope_weight_kernel(const float* __restrict__ part, int split, int blocks,
                                                              float* dw0, float* dw1) {
  __shared__ float sum_sh[THREADS / 8][8];
  wait_prior_grid();
  const int j = blockIdx.y, col = threadIdx.x & 7, row = threadIdx.x >> 3;
  float* out = j == 0 ? dw0 : dw1;
  if (!out) return;
  float s = 0.f;
  for (int i = (j == 0 ? 0 : split) + row; i < (j == 0 ? split : blocks); i += THREADS / 8)
    s += part[(size_t)i * D + blockIdx.x * 8 + col];
  sum_sh[row][col] = s;
  __syncthreads();
  if (row == 0) {
    for (int k = 1; k < THREADS / 8; ++k) s += sum_sh[k][col];
    out[blockIdx.x * 8 + col] = s;
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Turns per position as a fraction of 2^64.  1 / 2 pi in two doubles: with one, a position of 2^20 would
// be off by 2^-33 of a turn times the whole turns.
uint64_t turns_per_position(double inv_freq) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  const double p = inv_freq * hi, e = std::fma(inv_freq, hi, -p) + inv_freq * lo;
  const double frac = p - std::floor(p);                    // exact
  return (uint64_t)(frac * 0x1p64) + (uint64_t)(int64_t)(e * 0x1p64);
}

Freqs freqs_of(const RopeArgs& a) {
  Freqs f;
  for (int i = 0; i < MAX_PAIRS; ++i) f.step[i] = 2 * i < a.rotary_dim ? turns_per_position(a.inv_freq[i]) : 0;
  return f;
}

// Heads of a unit, for `slots` lane groups at once: all of them when there are units enough to even out, else
// fewer, down to the rows of two steps, as long as that gives every group more than one.
Split split_of(const RopeArgs& a, int slots, int step) {
  Split s{};
  s.n_tokens = (uint32_t)a.n_batch * (uint32_t)a.seq_len;
  const int most = a.n_tensors > 1 && a.t[1].heads > a.t[0].heads ? a.t[1].heads : a.t[0].heads;
  int parts = 1;
  while ((most + parts - 1) / parts > step && (unsigned long long)s.n_tokens * parts < 3ULL * slots) parts <<= 1;
  s.chunk = (most + parts - 1) / parts;
  for (int j = 0; j < a.n_tensors; ++j) s.units[j] = s.n_tokens * (uint32_t)((a.t[j].heads + s.chunk - 1) / s.chunk);
  return s;
}

template <typename T, int D, bool NORM>
cudaError_t run(const RopeArgs& a, cudaStream_t st) {
  const int groups = THREADS / (D / 16), most = FORWARD_BLOCKS * sm_count();
  const Split split = split_of(a, most * groups, sizeof(T) == 2 ? 8 : 4);
  const long long blocks = ((long long)split.units[0] + split.units[1] + groups - 1) / groups;
  const auto kern = a.interleaved ? rope_kernel<T, D, NORM, true> : rope_kernel<T, D, NORM, false>;
  count_launches(1);
  return launch_with_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(THREADS), 0, st, a, freqs_of(a), split);
}

// Blocks of the gradient kernel, and the first of the second tensor's: shared out by heads.
Split back_split(const RopeArgs& a, int D, int* blocks, int* split_at) {
  const int groups = THREADS / (D / 16), most = BACK_BLOCKS * sm_count();
  const Split s = split_of(a, most * groups, 4);
  int b[2];
  for (int j = 0; j < 2; ++j) {
    const long long need = ((long long)s.units[j] + groups - 1) / groups;
    const long long share = ((long long)most * a.t[j].heads) / (a.t[0].heads + a.t[1].heads);
    b[j] = (int)(need < share ? need : share > 0 ? share : 1);
  }
  *split_at = b[0];
  *blocks = b[0] + b[1];
  return s;
}

template <typename T, int D>
cudaError_t run_backward(const RopeArgs& a, float* dw0, float* dw1, void* ws, cudaStream_t st) {
  int blocks, split_at;
  const Split split = back_split(a, D, &blocks, &split_at);
  const auto kern = a.interleaved ? norm_rope_backward_kernel<T, D, true> : norm_rope_backward_kernel<T, D, false>;
  count_launches(1);
  const cudaError_t e = launch_with_pdl(kern, dim3((unsigned)blocks), dim3(THREADS), 0, st, a, freqs_of(a), split, split_at,
                                        (float*)ws);
  if (e != cudaSuccess || (!dw0 && !dw1)) return e;
  count_launches(1);
  return launch_with_pdl(rope_weight_kernel<D>, dim3(D / 8, 2), dim3(THREADS), 0, st, (const float*)ws, split_at, blocks,
                         dw0, dw1);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, int head_dim, int norm, cudaStream_t st) {
#define KVP_RP(TT, DD) return norm ? run<TT, DD, true>(a, st) : run<TT, DD, false>(a, st)
  if (dtype == KVP_BF16) {
    if (head_dim == 128) KVP_RP(__nv_bfloat16, 128);
    KVP_RP(__nv_bfloat16, 64);
  }
  if (dtype == KVP_F16) {
    if (head_dim == 128) KVP_RP(__half, 128);
    KVP_RP(__half, 64);
  }
  if (head_dim == 128) KVP_RP(float, 128);
  KVP_RP(float, 64);
#undef KVP_RP
}

size_t norm_rope_backward_workspace(const RopeArgs& a, int head_dim) {
  int blocks, split_at;
  back_split(a, head_dim, &blocks, &split_at);
  return (size_t)blocks * head_dim * sizeof(float);
}

cudaError_t launch_norm_rope_backward(const RopeArgs& a, int dtype, int head_dim, float* dw0, float* dw1, void* ws,
                                      cudaStream_t st) {
#define KVP_RB(TT) return head_dim == 128 ? run_backward<TT, 128>(a, dw0, dw1, ws, st) : run_backward<TT, 64>(a, dw0, dw1, ws, st)
  if (dtype == KVP_BF16) KVP_RB(__nv_bfloat16);
  if (dtype == KVP_F16) KVP_RB(__half);
  KVP_RB(float);
#undef KVP_RB
}

}  // namespace kvp
