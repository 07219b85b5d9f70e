// What the kernels of shared-prefix decode share: the plan that the device makes of a call's work, and the
// layout of the partial results that the join puts together.
//
// Work comes in items: the shared prefix of a family and KV head with up to `qt` of the family's queries,
// or one row's own tokens (behind the prefix it takes part in) with its G queries.  The tiles of TILE keys
// of all items form one sequence, of which every CTA takes an equal range; a CTA's share of an item is a
// piece.  The sequence has two places for a tile, three for one that meets more than 128 queries (bound by
// the tensor cores), and before every item GAP places, about what it costs to begin and end one: without
// those, the CTAs that had the short items at the end took 1.4 times as long as the rest.
//
// A piece that begins an item leaves its partial results (maximum, sum, unnormalised output) at the queries'
// own places, one that goes on from the CTA before at the CTA's, and the join adds a query's parts in the
// order of the tiles, so results do not depend on timing.
#pragma once

#include "kvp_common.cuh"
#include "kvp_launch.h"
#include "paged_decode.cuh"

namespace kvp {
namespace prefix {

constexpr int TILE = 128;                // keys
constexpr int GAP = 4;
constexpr int SEGMENT = 64;              // of a group's f16 tiles that the tensor cores add up (a power of two)
// Values of a query's kept sums (two groups of 128 queries a CTA): the outputs', and the maximum that they go by.
__host__ __device__ constexpr int kept_row(int D) { return D + 8; }

// A prefix with some of its queries, or a row's own tokens.
struct __align__(16) Item {
  int tile0;             // place of its first tile
  int row;               // row whose pages hold the tokens
  int tok0, tok1;        // tokens
  int q0, nq;            // queries, counted in the family's list (own tokens: 0, G)
  int list;              // prefix: where the head's list of participants begins; own tokens: -1
  int width;             // places of a tile
};

struct __align__(16) Head {
  int total, active, n_items, pad;       // places, CTAs that have any
};

struct Params {
  PagedView c;
  const void* q;
  int64_t q_stride;
  const int32_t* lead;
  int N, G, Hq, Hkv;     // sequences; queries of a row
  float c2;              // |scale| * log2 e
  int flip;              // scale < 0: the queries' signs change
  int zero;              // scale = 0: c2 is 1, and the queries count as 0 (-inf stays the logit of no token)
  int ctas;              // launched
  int qt;                // queries of an item: whole sequences'
  // the plan
  int* root;             // [N] sequence a sequence follows (itself)
  int* order;            // [N] sequences by family
  int* base;             // [N] where a root's family begins in it
  int* count;            // [N] members of a root's family
  int* shared;           // [R] leading tokens on pages of the root's row
  int* start;            // [R] first own token
  int* place;            // [R] place in the list of participants, -1: reads everything itself
  int* list;             // [Hkv][N] participants (sequences) of the heads' prefixes, at the families' places
  int* pre_item;         // [R] a root row's first prefix item, -1: none
  int* own_item;         // [R]
  Item* items;
  Head* head;
  int* cta_item;         // [ctas] first item with a tile in a CTA's range
  // partial results
  float2* first_ml;      // [2 kinds][R * G]
  float* first_o;        // [...][D]
  float2* cont_ml;       // [ctas][qt]
  float* cont_o;
  float* kept;           // [ctas][2][128][kept_row] sums of the segments before (f16 caches whose rows may have any)
  void* out;
  float* lse;
  int* status;
};

__device__ __forceinline__ int tiles_of(int n) { return (n + TILE - 1) / TILE; }
__device__ __forceinline__ int width_of(int nq) { return nq > 128 ? 3 : 2; }
__device__ __forceinline__ int row_len(const Params& p, int r) {
  const int n = p.c.lens[r];
  return n < 0 ? 0 : (n > p.c.cap ? p.c.cap : n);
}

// One piece: tiles [u0, u1) of an item.
struct Piece {
  Item it;
  int u0, u1;
};

// Walks over a CTA's pieces; with AHEAD the next item's record is fetched one ahead.
template <bool AHEAD>
struct Walk {
  int item, n_items, x, end;
  Item next;
  __device__ __forceinline__ Walk() {}
  __device__ __forceinline__ Walk(const Params& p, int cta) {
    const Head h = *p.head;
    const int first = p.cta_item[cta];
    n_items = h.n_items;
    x = end = 0;
    if (cta >= h.active) return;
    x = paged::cta_begin(cta, h.total, h.active);
    end = paged::cta_begin(cta + 1, h.total, h.active);
    item = first;
    if (AHEAD) next = p.items[item];
  }
  __device__ __forceinline__ bool step(const Params& p, Piece& a) {
    while (x < end) {
      a.it = AHEAD ? next : p.items[item];
      if (a.it.tile0 >= end) break;
      const int w = a.it.width, past = max(0, x - a.it.tile0);
      a.u0 = (past + w - 1) / w;
      a.u1 = min(tiles_of(a.it.tok1 - a.it.tok0), (end - a.it.tile0 + w - 1) / w);
      x = a.it.tile0 + a.u1 * w;
      if (++item >= n_items) x = end;
      else if (AHEAD && x < end) next = p.items[item];
      if (a.u0 < a.u1) return true;
    }
    return false;
  }
};

// Sequence and row of query i (of the item's) and, in g, its place in the row's group.
__device__ __forceinline__ int query_row(const Params& p, const Item& it, int i, int& g) {
  if (it.list < 0) {
    g = i;
    return it.row;
  }
  const int x = it.q0 + i, k = x / p.G;
  g = x - k * p.G;
  return p.list[it.list + k] * p.Hkv + it.row % p.Hkv;
}

// Where a piece's partial result of a query goes: of a piece that begins an item, and of one that goes on
// (the item's query `local`).
__device__ __forceinline__ size_t first_slot(const Params& p, bool own, int row, int g) {
  return ((size_t)own * p.c.R + row) * p.G + g;
}
__device__ __forceinline__ size_t cont_slot(const Params& p, int cta, int local) { return (size_t)cta * p.qt + local; }

}  // namespace prefix

// The tensor-core kernel of bf16 / f16 caches (paged_prefix_tc.cu).
cudaError_t launch_paged_prefix_tc(const prefix::Params& p, cudaStream_t st);

}  // namespace kvp
