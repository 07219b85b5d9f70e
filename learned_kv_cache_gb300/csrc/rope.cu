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
//  * A block takes TOK tokens and all their heads; its threads compute the tokens' cosines and sines once
//    (64 pairs x 4 tokens: one each), and a group of D / 16 lanes then walks over heads of one token with
//    its 8 pairs' values in registers.
//  * A lane owns 8 pairs of a row: two vectors of 8 values that lie rotary_dim / 2 apart (halves) or side
//    by side (interleaved), so pairs never cross lanes and sums over a row are 2 or 3 shuffles.
//  * Rows are taken a few at a time, all their loads before the first is used.
#include <cmath>

#include "kvp_common.cuh"
#include "kvp_launch.h"

namespace kvp {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 64;
constexpr int MAX_TOK = 32;

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

// Fills cs[tok][pair] for tokens [t0, t0 + TOK) of the n_tokens.
__device__ __forceinline__ void block_turns(const RopeArgs& a, const Freqs& f, long long t0, int tok, long long n_tokens,
                                            float2* cs, int pairs_stride) {
  const int pairs = a.rotary_dim >> 1;
  for (int i = threadIdx.x; i < tok * pairs; i += THREADS) {
    const int x = i / pairs, pair = i - x * pairs;
    const long long t = t0 + x;
    if (t >= n_tokens) break;
    const int b = (int)(t / a.seq_len), s = (int)(t - (long long)b * a.seq_len);
    const int pos = a.positions ? a.positions[b * a.position_stride + s] : a.start + s;
    float2 v = turn_of(pos, f.step[pair]);
    v.x *= a.gain;
    v.y *= a.gain;
    if (a.inverse) v.y = -v.y;
    cs[x * pairs_stride + pair] = v;
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

// This lane's weights (1 without any).
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, int f32, int at0, int at1, float (&out)[2][8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = (k ? at1 : at0) + i;
      out[k][i] = !w ? 1.f : f32 ? ((const float*)w)[at] : to_f32<T>(((const T*)w)[at]);
    }
}

template <typename T, int D, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, 2)
    rope_kernel(const RopeArgs a, const __grid_constant__ Freqs f, int tok, long long n_tokens) {
  using L = Lane<D, INTERLEAVED>;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;               // rows at a time
  __shared__ float2 cs_sh[MAX_TOK * (D / 2)];
  const L lane(a.rotary_dim);
  wait_prior_grid();
  allow_next_grid();
  const long long t0 = (long long)blockIdx.x * tok;
  block_turns(a, f, t0, tok, n_tokens, cs_sh, D / 2);
  __syncthreads();
  const int group = threadIdx.x / L::PER_ROW, x = group % tok, stride = L::GROUPS / tok;
  const long long t = t0 + x;
  const bool live = t < n_tokens;                         // the lanes of a row agree
  const int b = live ? (int)(t / a.seq_len) : 0, s = live ? (int)(t - (long long)b * a.seq_len) : 0;
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = lane.turns && live ? cs_sh[x * (D / 2) + 8 * lane.u + i] : make_float2(1.f, 0.f);
#pragma unroll 1
  for (int j = 0; j < a.n_tensors; ++j) {
    const RopeTensor& z = a.t[j];
    const T* in = (const T*)z.x + b * z.xs[0] + s * z.xs[2];
    T* out = (T*)z.y + b * z.ys[0] + s * z.ys[2];
    float w[2][8];
    if (NORM) load_weights<T>(z.w, a.w_f32, lane.at0, lane.at1, w);
    // the same number of steps for every lane of a warp: the sums are warp-wide shuffles
    for (int h0 = 0; h0 < z.heads; h0 += U * stride) {
      const int h = h0 + group / tok;
      Raw<T> raw[U][2];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (live && h + k * stride < z.heads) {
          raw[k][0].load(in + (h + k * stride) * z.xs[1] + lane.at0);
          raw[k][1].load(in + (h + k * stride) * z.xs[1] + lane.at1);
        }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (h0 + k * stride >= z.heads) break;            // none of the block's
        const bool mine = live && h + k * stride < z.heads;
        float v[2][8];
        raw[k][0].get(v[0]);
        raw[k][1].get(v[1]);
        if (NORM) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[0][i], v[0][i], fmaf(v[1][i], v[1][i], ss));
          const float r = __frsqrt_rn(row_sum<L::PER_ROW>(ss) * (1.f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[0][i] = v[0][i] * r * w[0][i];
            v[1][i] = v[1][i] * r * w[1][i];
          }
        }
        if (lane.turns) turn<INTERLEAVED>(v, cs, 1.f);
        if (mine) {
          store8(out + (h + k * stride) * z.ys[1] + lane.at0, v[0]);
          store8(out + (h + k * stride) * z.ys[1] + lane.at1, v[1]);
        }
      }
    }
  }
}

// Gradients of one tensor: blocks [first, first + blocks) walk over its tokens.  A lane sums its 16 values'
// weight gradients over all its rows in registers; the block's groups are added at the end, and the blocks'
// sums by rope_weight_kernel in a fixed order.
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, 2)
    norm_rope_backward_kernel(const RopeArgs a, const __grid_constant__ Freqs f, long long n_tokens, int split,
                              int tok0, int tok1, float* __restrict__ part) {
  using L = Lane<D, INTERLEAVED>;
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  __shared__ float2 cs_sh[MAX_TOK * (D / 2)];
  __shared__ float sum_sh[THREADS / 32][D];
  const L lane(a.rotary_dim);
  const int j = (int)blockIdx.x < split ? 0 : 1, tok = j == 0 ? tok0 : tok1;
  const int block = j == 0 ? blockIdx.x : blockIdx.x - split, blocks = j == 0 ? split : gridDim.x - split;
  const RopeTensor& z = a.t[j];
  wait_prior_grid();
  allow_next_grid();
  const int group = threadIdx.x / L::PER_ROW, x = group % tok, stride = L::GROUPS / tok;
  float w[2][8], dw[2][8];
  load_weights<T>(z.w, a.w_f32, lane.at0, lane.at1, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  for (long long t0 = (long long)block * tok; t0 < n_tokens; t0 += (long long)blocks * tok) {
    __syncthreads();                                      // the last tokens' values are read
    block_turns(a, f, t0, tok, n_tokens, cs_sh, D / 2);
    __syncthreads();
    const long long t = t0 + x;
    const bool live = t < n_tokens;
    const int b = live ? (int)(t / a.seq_len) : 0, s = live ? (int)(t - (long long)b * a.seq_len) : 0;
    const T* in = (const T*)z.x + b * z.xs[0] + s * z.xs[2];
    const T* dy = (const T*)z.dy + b * z.dys[0] + s * z.dys[2];
    T* out = (T*)z.y + b * z.ys[0] + s * z.ys[2];
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = lane.turns && live ? cs_sh[x * (D / 2) + 8 * lane.u + i] : make_float2(1.f, 0.f);
    for (int h0 = 0; h0 < z.heads; h0 += U * stride) {
      const int h = h0 + group / tok;
      Raw<T> raw[U][2], back[U][2];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (live && h + k * stride < z.heads) {
          raw[k][0].load(in + (h + k * stride) * z.xs[1] + lane.at0);
          raw[k][1].load(in + (h + k * stride) * z.xs[1] + lane.at1);
          back[k][0].load(dy + (h + k * stride) * z.dys[1] + lane.at0);
          back[k][1].load(dy + (h + k * stride) * z.dys[1] + lane.at1);
        }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (h0 + k * stride >= z.heads) break;
        const bool mine = live && h + k * stride < z.heads;
        float v[2][8], g[2][8];
        raw[k][0].get(v[0]);
        raw[k][1].get(v[1]);
        back[k][0].get(g[0]);
        back[k][1].get(g[1]);
        if (lane.turns) turn<INTERLEAVED>(g, cs, -1.f);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(v[0][i], v[0][i], fmaf(v[1][i], v[1][i], ss));
          dot = fmaf(g[0][i] * w[0][i], v[0][i], fmaf(g[1][i] * w[1][i], v[1][i], dot));
        }
        const float r = __frsqrt_rn(row_sum<L::PER_ROW>(ss) * (1.f / D) + a.eps);
        const float mean = row_sum<L::PER_ROW>(dot) * r * (1.f / D);
        if (mine) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float n = v[m][i] * r;
              dw[m][i] = fmaf(g[m][i], n, dw[m][i]);
              v[m][i] = r * (g[m][i] * w[m][i] - n * mean);
            }
          store8(out + (h + k * stride) * z.ys[1] + lane.at0, v[0]);
          store8(out + (h + k * stride) * z.ys[1] + lane.at1, v[1]);
        }
      }
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

template <typename T, int D, bool NORM>
cudaError_t run(const RopeArgs& a, cudaStream_t st) {
  const long long n = (long long)a.n_batch * a.seq_len;
  // Tokens of a block: as many as give every thread one cosine and sine (4 at 64 pairs), fewer while that
  // leaves SMs without a block.
  int tok = D == 128 ? 4 : 8;
  const int sms = sm_count();
  while (tok > 1 && (n + tok - 1) / tok < 2LL * sms) tok >>= 1;
  const auto kern = a.interleaved ? rope_kernel<T, D, NORM, true> : rope_kernel<T, D, NORM, false>;
  count_launches(1);
  return launch_with_pdl(kern, dim3((unsigned)((n + tok - 1) / tok)), dim3(THREADS), 0, st, a, freqs_of(a), tok, n);
}

constexpr int BACK_BLOCKS = 2;                              // per SM

// Blocks of the gradient kernel, and the first of the second tensor's: shared out by heads.
void back_blocks(const RopeArgs& a, int D, int* blocks, int* split, int* tok) {
  const long long n = (long long)a.n_batch * a.seq_len;
  const int sms = sm_count(), groups = THREADS / (D / 16), all = a.t[0].heads + a.t[1].heads;
  int b[2];
  for (int j = 0; j < 2; ++j) {
    tok[j] = 1;
    // tokens until every group has two rows
    while (tok[j] < MAX_TOK && tok[j] < groups && tok[j] * a.t[j].heads < 2 * groups) tok[j] <<= 1;
    const long long most = (n + tok[j] - 1) / tok[j];
    b[j] = (int)(((long long)BACK_BLOCKS * sms * a.t[j].heads + all - 1) / all);
    if (b[j] > most) b[j] = (int)most;
  }
  *split = b[0];
  *blocks = b[0] + b[1];
}

template <typename T, int D>
cudaError_t run_backward(const RopeArgs& a, float* dw0, float* dw1, void* ws, cudaStream_t st) {
  int blocks, split, tok[2];
  back_blocks(a, D, &blocks, &split, tok);
  const auto kern = a.interleaved ? norm_rope_backward_kernel<T, D, true> : norm_rope_backward_kernel<T, D, false>;
  const long long n = (long long)a.n_batch * a.seq_len;
  count_launches(1);
  const cudaError_t e = launch_with_pdl(kern, dim3((unsigned)blocks), dim3(THREADS), 0, st, a, freqs_of(a), n, split,
                                        tok[0], tok[1], (float*)ws);
  if (e != cudaSuccess || (!dw0 && !dw1)) return e;
  count_launches(1);
  return launch_with_pdl(rope_weight_kernel<D>, dim3(D / 8, 2), dim3(THREADS), 0, st, (const float*)ws, split, blocks,
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
  int blocks, split, tok[2];
  back_blocks(a, head_dim, &blocks, &split, tok);
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
