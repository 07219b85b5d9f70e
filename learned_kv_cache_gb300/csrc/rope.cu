// Rotary positions, and the norms of queries and keys with the rotation in the same pass (and their
// gradients).
//
//   n = x / sqrt(mean(x^2) + eps),  z = w n,  y = R(pos) z,
//   R(pos): pairs (a, b) of the head's first rotary_dim values -> gain (a cos t - b sin t, a sin t + b cos t),
//   t = pos * inv_freq of the pair; the values behind rotary_dim pass.
//   dz = R^T dy,  dw = sum dz n,  dx = (w dz - n mean(w dz n)) / sqrt(mean(x^2) + eps)
//
// A few operations per value: bound by HBM (every input read once, every output written once).  Measured,
// 32 + 8 heads of 128 in bf16, norms and rotation: 131072 tokens 425 us (6.3 TB/s), 8192 tokens 33.5 us, their
// gradients 49 us (5.1 TB/s); rotation alone of 32768 tokens 112 us (6.0 TB/s).
//
//  * Angles.  pos * inv_freq reaches 1e5 radians, of which a float keeps 1e-2.  The host gives each pair's
//    frequency in turns as a fraction of 2^64, so that the angle is one 64-bit product whose overflow drops
//    the whole turns: exact up to 2^-64 of a turn per position, for every 32-bit position.  Its upper 32
//    bits, less the nearest quarter turn, are exact to 2^-25 of an eighth of a turn as a float.
//  * The unit of work is a token with some of a tensor's heads, and D / 16 lanes have one: they compute its
//    cosines and sines (8 pairs a lane) and walk over the heads.  Nothing is shared between lanes but sums
//    over a row, so no warp waits for another (with the angles in shared memory and a few tokens a block,
//    8192 tokens of 32 + 8 heads took 52 us).
//  * What keeps HBM busy is bytes on their way.  The forward kernels have the next rows in registers; the
//    gradients, with two sources, copy theirs into a ring of every lane's own in shared memory (cp.async) some
//    steps before they use them, beyond the end of a unit: as many in registers spill, or leave an SM too few
//    warps (58 us).  For the forward kernels the ring was slower (485 us of 131072 tokens for 425).
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
constexpr int FORWARD_BLOCKS = 2, BACK_BLOCKS = 2;          // per SM

struct Freqs {
  uint64_t step[MAX_PAIRS];   // turns per position, times 2^64
};

// Eight values as four pairs, from memory and back.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 (&x)[sizeof(T) / 2], uint64_t* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = (uint64_t)x[0].y << 32 | x[0].x;
    v[1] = (uint64_t)x[0].w << 32 | x[0].z;
    v[2] = (uint64_t)x[1].y << 32 | x[1].x;
    v[3] = (uint64_t)x[1].w << 32 | x[1].z;
  } else {
    float f[8];
    Vec16<T>::unpack(x[0], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
}
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(uint64_t* f) const { unpack8<T>(v, f); }
};
__device__ __forceinline__ void store8(float* p, const uint64_t* v) {
  reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(v[0], v[1]);
  reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(v[2], v[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint64_t* v) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(v[i], a, b);
    h[i] = __floats2bfloat162_rn(a, b);
  }
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ void store8(__half* p, const uint64_t* v) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(v[i], a, b);
    h[i] = __floats2half2_rn(a, b);
  }
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}

// Cosine and sine of pos * step turns.  Within an eighth of a turn of the nearest quarter the Taylor series
// up to t^10 leave 1.8e-9 (t^11 / 11! at pi / 4); no branches, as the quarters differ from lane to lane (the
// library's function and a switch took 3 times the instructions, half of all).
__device__ __forceinline__ float2 turn_of(int pos, uint64_t step) {
  const uint32_t t = (uint32_t)(((uint64_t)(int64_t)pos * step) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float x = (float)(int)(t - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), xx = x * x;
  float c = fmaf(xx, fmaf(xx, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f);
  c = fmaf(xx, fmaf(xx, fmaf(xx, c, 1.f / 24.f), -0.5f), 1.f);
  const float s = fmaf(x * xx, fmaf(xx, fmaf(xx, fmaf(xx, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  // a quarter turn on: (c, s) -> (-s, c)
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(a) ^ ((quarter + 1) << 30 & 0x80000000u)),
                     __uint_as_float(__float_as_uint(b) ^ (quarter << 30 & 0x80000000u)));
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

// Cosines and sines (times gain) of the lane's eight pairs, two to a register pair.
struct Turns {
  uint64_t c[4], s[4], minus[4];         // (minus the sines: packed arithmetic has no signs)
  template <bool INTERLEAVED>
  __device__ __forceinline__ void fill(const RopeArgs& a, const uint64_t* step, int pos, bool rotates) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 x = make_float2(1.f, 0.f), y = x;
      if (rotates) {
        const float up = a.inverse ? -a.gain : a.gain;
        x = turn_of(pos, step[2 * i]);
        y = turn_of(pos, step[2 * i + 1]);
        x.x *= a.gain;
        y.x *= a.gain;
        x.y *= up;
        y.y *= up;
      }
      c[i] = pack2(x.x, y.x);
      s[i] = pack2(x.y, y.y);
      if (!INTERLEAVED) minus[i] = pack2(-x.y, -y.y);
    }
  }
};
// The pairs (a, b) of a lane turned, or turned back.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(uint64_t (&v)[8], const Turns& t, bool back) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float c[2], s[2], a, b;
      unpack2(t.c[i >> 1], c[0], c[1]);
      unpack2(t.s[i >> 1], s[0], s[1]);
      unpack2(v[i], a, b);
      const float ci = c[i & 1], si = back ? -s[i & 1] : s[i & 1];
      v[i] = pack2(a * ci - b * si, b * ci + a * si);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = v[i], b = v[4 + i], s = back ? t.minus[i] : t.s[i], minus = back ? t.s[i] : t.minus[i];
      v[i] = ffma2(b, minus, fmul2(a, t.c[i]));
      v[4 + i] = ffma2(a, s, fmul2(b, t.c[i]));
    }
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
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// The rows of a warp's units, one step of every lane group after the other, copied STEPS - 1 steps ahead (of
// 64 or, in fp32, 128 bytes a lane: 70 or 101 KB a block).  The sources are x and dy.
template <typename T>
struct Rows {
  static constexpr int SOURCES = 2;
  static constexpr int PARTS = 16 * sizeof(T) / 16;        // 16-byte parts of a lane's 16 values
  static constexpr int STEPS = PARTS * SOURCES > 4 ? 3 : 4;
  static constexpr int SMEM = STEPS * (PARTS * SOURCES * 16 + 4) * THREADS;
  // [step][part][thread], then the tokens' positions
  uint4* ring;
  int* ring_pos;
  const RopeArgs& a;
  const Split& split;
  int at0, at1;
  uint32_t u0, stride, all, begin;   // the warp's first unit, from step to step, the last; the lane's within the warp
  int tensor;
  // the unit that is being copied
  int h, most, n, slot;
  const T* src[SOURCES];
  int64_t hs[SOURCES];
  const int32_t* pos;

  __device__ __forceinline__ Rows(const RopeArgs& a_, const Split& split_, uint4* smem, int at0_, int at1_)
      : a(a_), split(split_), at0(at0_), at1(at1_) {
    ring = smem + threadIdx.x;
    ring_pos = reinterpret_cast<int*>(smem + STEPS * PARTS * SOURCES * THREADS) + threadIdx.x;
  }
  // This lane's unit of the warp's step u.
  __device__ __forceinline__ Unit unit(uint32_t u) const {
    return Unit(a, split, tensor ? a.t[1].heads : a.t[0].heads, u + begin, u + begin < all);
  }
  __device__ __forceinline__ void enter() {
    const Unit x = unit(u0);
    const RopeTensor& z = tensor ? a.t[1] : a.t[0];
    hs[0] = z.xs[1];
    src[0] = (const T*)z.x + x.b * z.xs[0] + x.s * z.xs[2] + x.h0 * hs[0];
    hs[1] = z.dys[1];
    src[1] = (const T*)z.dy + x.b * z.dys[0] + x.s * z.dys[2] + x.h0 * hs[1];
    pos = a.positions ? a.positions + x.b * a.position_stride + x.s : nullptr;
    n = x.n;
    most = __reduce_max_sync(0xffffffffu, n);
    h = 0;
  }
  // Copies the next step's rows.
  __device__ __forceinline__ void copy() {
    if (u0 < all) {
      if (h < n) {
#pragma unroll
        for (int k = 0; k < SOURCES; ++k)
#pragma unroll
          for (int i = 0; i < PARTS; ++i)
            copy16(ring + ((slot * SOURCES + k) * PARTS + i) * THREADS,
                   src[k] + (i < PARTS / 2 ? at0 + i * (8 / (PARTS / 2)) : at1 + (i - PARTS / 2) * (8 / (PARTS / 2))));
        if (h == 0 && pos) copy4(ring_pos + slot * THREADS, pos);
#pragma unroll
        for (int k = 0; k < SOURCES; ++k) src[k] += hs[k];
      }
      if (++h == most) {
        u0 += stride;
        if (u0 < all) enter();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    slot = slot + 1 == STEPS ? 0 : slot + 1;
  }
  __device__ __forceinline__ void start(uint32_t first, uint32_t stride_, uint32_t all_, uint32_t begin_, int tensor_) {
    u0 = first;
    stride = stride_;
    all = all_;
    begin = begin_;
    tensor = tensor_;
    slot = 0;
    if (u0 < all) enter();
#pragma unroll 1
    for (int i = 0; i < STEPS - 1; ++i) copy();
  }
  __device__ __forceinline__ void landed() { asm volatile("cp.async.wait_group %0;" ::"n"(STEPS - 2) : "memory"); }
  // The 16 values of source k in the ring's place s.
  __device__ __forceinline__ void get(int s, int k, uint64_t (&v)[8]) const {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint4 x[PARTS / 2];
#pragma unroll
      for (int i = 0; i < PARTS / 2; ++i) x[i] = ring[((s * SOURCES + k) * PARTS + m * (PARTS / 2) + i) * THREADS];
      unpack8<T>(x, v + 4 * m);
    }
  }
};

template <typename T, int D, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, FORWARD_BLOCKS)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Freqs f, const __grid_constant__ Split split) {
  using L = Lane<D, INTERLEAVED>;
  // Rows at a time: twice these in registers.  (Norms of 16-bit rows with four: 457 us of 131072 tokens for 434.
  // With three and two, the norms of pairs of halves spill 12 bytes in 16 bits and 108 in fp32, interleaved 0 and 28.)
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
    Turns t;
    const auto rows = [&](const Raw<T> (&raw)[U][2], int h) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        uint64_t v[8];
        raw[k][0].get(v);
        raw[k][1].get(v + 4);
        if (NORM) {
          uint64_t ss[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i) ss[i & 1] = ffma2(v[i], v[i], ss[i & 1]);
          const float r = __frsqrt_rn(row_sum<L::PER_ROW>(sum2(fadd2(ss[0], ss[1]))) * (1.f / D) + a.eps);
          const uint64_t r2 = pack2(r, r);
          const float* w = sh.w[second];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + (i < 4 ? lane.at0 : lane.at1 - 8) + 2 * i);
            v[i] = fmul2(fmul2(v[i], r2), x.x);
            v[i + 1] = fmul2(fmul2(v[i + 1], r2), x.y);
          }
        }
        if (lane.turns) turn<INTERLEAVED>(v, t, false);
        if (h + k < u.n) {
          store8(out + (h + k) * ys + lane.at0, v);
          store8(out + (h + k) * ys + lane.at1, v + 4);
        }
      }
    };
    // every lane of the warp takes as many steps as any: sums over a row are the whole warp's shuffles
    const int most = __reduce_max_sync(0xffffffffu, u.n);
    Raw<T> even[U][2], odd[U][2];
    const int pos = a.positions ? a.positions[u.b * a.position_stride + u.s] : a.start + u.s;
    load(even, 0);
    t.fill<INTERLEAVED>(a, sh.step + 8 * lane.u, pos, lane.turns);
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
    norm_rope_backward_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Freqs f,
                              const __grid_constant__ Split split, int split_at, float* __restrict__ part) {
  using L = Lane<D, INTERLEAVED>;
  using R = Rows<T>;
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) Tables<D> sh;
  __shared__ float sum_sh[THREADS / 32][D];
  const L lane(a.rotary_dim);
  fill_tables<T, D, true>(sh, a, f);
  const int j = (int)blockIdx.x >= split_at;
  const uint32_t block = j ? blockIdx.x - split_at : blockIdx.x, blocks = j ? gridDim.x - split_at : split_at;
  const RopeTensor& z = j ? a.t[1] : a.t[0];
  const uint32_t all = split.units[j], stride = blocks * L::GROUPS;
  R rows(a, split, ring, lane.at0, lane.at1);
  uint32_t u0 = block * L::GROUPS + threadIdx.x / 32 * (32 / L::PER_ROW);
  rows.start(u0, stride, all, (threadIdx.x & 31) / L::PER_ROW, j);
  uint64_t dw[8] = {};
  int slot = 0;
  for (; u0 < all; u0 += stride) {
    const Unit u = rows.unit(u0);
    const int64_t ys = z.ys[1];
    T* out = (T*)z.y + u.b * z.ys[0] + u.s * z.ys[2] + u.h0 * ys;
    // every lane of the warp takes as many steps as any: sums over a row are the whole warp's shuffles
    const int most = __reduce_max_sync(0xffffffffu, u.n);
    Turns t;
    for (int h = 0; h < most; ++h) {
      rows.landed();
      if (h == 0)
        t.fill<INTERLEAVED>(a, sh.step + 8 * lane.u, a.positions ? rows.ring_pos[slot * THREADS] : a.start + u.s, lane.turns);
      uint64_t v[8], g[8], gw[8];
      rows.get(slot, 0, v);
      rows.get(slot, 1, g);
      rows.copy();                     // into the place before this one
      slot = slot + 1 == R::STEPS ? 0 : slot + 1;
      if (lane.turns) turn<INTERLEAVED>(g, t, true);
      const float* w = sh.w[j];
      uint64_t ss[2] = {0, 0}, dot[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + (i < 4 ? lane.at0 : lane.at1 - 8) + 2 * i);
        gw[i] = fmul2(g[i], x.x);
        gw[i + 1] = fmul2(g[i + 1], x.y);
        ss[0] = ffma2(v[i], v[i], ss[0]);
        ss[1] = ffma2(v[i + 1], v[i + 1], ss[1]);
        dot[0] = ffma2(gw[i], v[i], dot[0]);
        dot[1] = ffma2(gw[i + 1], v[i + 1], dot[1]);
      }
      const float r = __frsqrt_rn(row_sum<L::PER_ROW>(sum2(fadd2(ss[0], ss[1]))) * (1.f / D) + a.eps);
      const float mean = row_sum<L::PER_ROW>(sum2(fadd2(dot[0], dot[1]))) * r * (1.f / D);
      if (h < u.n) {
        const uint64_t r2 = pack2(r, r), m2 = pack2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t n = fmul2(v[i], r2);
          dw[i] = ffma2(g[i], n, dw[i]);
          v[i] = fmul2(r2, ffma2(n, m2, gw[i]));
        }
        store8(out + lane.at0, v);
        store8(out + lane.at1, v + 4);
        out += ys;
      }
    }
  }
  // the groups of a warp, then the warps
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x[2];
    unpack2(dw[i], x[0], x[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int o = L::PER_ROW; o < 32; o <<= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
      if ((threadIdx.x & 31) < L::PER_ROW) sum_sh[threadIdx.x >> 5][(i < 4 ? lane.at0 : lane.at1 - 8) + 2 * i + k] = x[k];
    }
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

// Blocks of the gradient kernel, and the first of the second tensor's: shared out by rows, a unit's beginning
// (its cosines and sines) counting as two (27162 tokens of 32 + 4 heads: 135 us by rows alone, 122 us).
Split back_split(const RopeArgs& a, int D, int* blocks, int* split_at) {
  const int groups = THREADS / (D / 16), most = BACK_BLOCKS * sm_count();
  const Split s = split_of(a, most * groups, 4);
  int b[2];
  double work[2];
  for (int j = 0; j < 2; ++j) work[j] = (double)s.n_tokens * a.t[j].heads + 2.0 * s.units[j];
  for (int j = 0; j < 2; ++j) {
    const long long need = ((long long)s.units[j] + groups - 1) / groups;
    const long long share = (long long)(most * (work[j] / (work[0] + work[1])));
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
  constexpr int SMEM = Rows<T>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  count_launches(1);
  e = launch_with_pdl(kern, dim3((unsigned)blocks), dim3(THREADS), SMEM, st, a, freqs_of(a), split, split_at, (float*)ws);
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
