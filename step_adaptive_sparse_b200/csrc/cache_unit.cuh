// How the tensor-core kernels cut a launch into work units: two row tiles of a
// group (fp32: one) and a split of the list of keys that they see, in tiles of
// KT keys.  Integer arithmetic alone, also compiled for the host and checked
// there.
#pragma once

#include "cache.cuh"

namespace area {

struct Unit {
  int valid;
  int g, sp;               // row group, split
  int kvh, ph;             // (sequence, key head) of the own keys, key head of the prefix
  int r0[2];               // first row of each row tile (RG: the tile has none)
  int t0, nt;              // this split's first list tile and its tiles
  int tp, ts;              // list tiles of the prefix, of the sinks
  KeyList kl;
  int hi;                  // end of the own keys in the list
  int safe_lo, safe_hi;    // own rows that some query of the sequence sees, or zero fill
  // tiles [0, lead) and [oa, ob) of this split are the row tile's
  int lead[2], oa[2], ob[2];
};
static_assert(sizeof(Unit) <= 160, "unit record");

struct UnitParams {
  CacheArgs a;
  CacheRows rm;
  CacheOut out;
  int nrb;                 // units that a group's rows make
  int tile_rows;           // rows of a row tile
  int tiles;               // row tiles of a unit
  int units;
  int heavy_first;         // row tiles from the last to the first, over all groups
  int halved;              // the last units come as two, of one row tile each
};

// A key tile of a unit.
struct Tile {
  int kind;                // 0 prefix, 1 own
  int j0, n;               // first key, keys
  bool copy;               // copied row by row
};
template <int KT>
__host__ __device__ __forceinline__ Tile tile_of(const Unit& u, int j) {
  Tile t;
  int i = u.t0 + j;
  if (i < u.tp) {
    t.kind = 0;
    t.j0 = i * KT;
    t.n = min(KT, u.kl.np - t.j0);
    t.copy = false;                        // its map ends with the prefix
    return t;
  }
  i -= u.tp;
  t.kind = 1;
  if (i < u.ts) {
    t.j0 = i * KT;
    t.n = min(KT, u.kl.ns - t.j0);
  } else {
    t.j0 = u.kl.lo + (i - u.ts) * KT;
    t.n = min(KT, u.hi - t.j0);
  }
  t.copy = t.n < KT && !(t.j0 >= u.safe_lo && t.j0 + KT <= u.safe_hi);
  return t;
}
__host__ __device__ __forceinline__ bool is_active(const Unit& u, int t, int j) {
  return j < u.lead[t] || (j >= u.oa[t] && j < u.ob[t]);
}
// First and last tile of a row tile; last < 0: it has none.
__host__ __device__ __forceinline__ int first_tile(const Unit& u, int t) {
  return u.lead[t] > 0 ? 0 : u.oa[t];
}
__host__ __device__ __forceinline__ int last_tile(const Unit& u, int t) {
  return u.ob[t] > u.oa[t] ? u.ob[t] - 1 : u.lead[t] - 1;
}

// The tile after j of a row tile's tiles, first_tile() to last_tile().
__host__ __device__ __forceinline__ int next_tile(int j, int lead, int oa) {
  return j + 1 == lead ? oa : j + 1;
}

// The tiles of a row tile, in registers.
struct TileRange {
  int lead, oa, ob, first, last;
  __host__ __device__ __forceinline__ bool has(int j) const {
    return j < lead || (j >= oa && j < ob);
  }
};
__host__ __device__ __forceinline__ TileRange tile_range(const Unit& u, int t) {
  return TileRange{u.lead[t], u.oa[t], u.ob[t], first_tile(u, t), last_tile(u, t)};
}

// The k-th unit of a block: the blocks take units in turn, there and back, so
// that units in the order of their cost come out even.
__device__ __forceinline__ int unit_index(uint32_t k) {
  return (int)(k * gridDim.x + (k & 1u ? gridDim.x - 1 - blockIdx.x : blockIdx.x));
}

// Unit idx of a launch; false behind the last one.
template <int KT>
__host__ __device__ inline bool decode_unit(int idx, const UnitParams& p, Unit& u) {
  const CacheArgs& a = p.a;
  const CacheRows& rm = p.rm;
  if (idx >= p.units) return false;
  const int in_halves = idx - (p.units - 2 * p.halved), half = in_halves & 1;
  if (in_halves >= 0) idx -= in_halves - in_halves / 2;
  u.sp = idx % p.out.nsplit;
  const int rest = idx / p.out.nsplit;
  int rb;
  if (p.heavy_first) {
    u.g = rest % rm.groups;
    rb = p.nrb - 1 - rest / rm.groups;
  } else {
    rb = rest % p.nrb;
    u.g = rest / p.nrb;
  }
  u.r0[0] = rb * p.tiles * p.tile_rows;
  int r1 = min(u.r0[0] + p.tiles * p.tile_rows, rm.RG);
  const int k0 = u.r0[0], k1 = r1;               // a half has its unit's list, cut as its unit's
  if (in_halves >= 0) {
    u.r0[0] = min(u.r0[0] + half * p.tile_rows, rm.RG);
    r1 = min(u.r0[0] + p.tile_rows, rm.RG);
  }
  u.r0[1] = in_halves >= 0 ? rm.RG : min(u.r0[0] + p.tile_rows, rm.RG);
  u.kvh = rm.pool_rows ? 0 : u.g / rm.kv_div;
  u.ph = rm.pool_rows ? u.g : u.kvh % a.Hk;
  const int b = rm.pool_rows ? 0 : u.kvh / a.Hk;
  u.kl = key_list(a, rm, b, k0, k1);
  u.hi = u.kl.lo + (u.kl.total - u.kl.np - u.kl.ns);
  u.tp = (u.kl.np + KT - 1) / KT;
  u.ts = (u.kl.ns + KT - 1) / KT;
  const int to = (u.hi - u.kl.lo + KT - 1) / KT;
  const int ntile = u.tp + u.ts + to;
  u.t0 = (int)((int64_t)ntile * u.sp / p.out.nsplit);
  const int t1 = (int)((int64_t)ntile * (u.sp + 1) / p.out.nsplit);
  u.nt = u.r0[0] < r1 ? t1 - u.t0 : 0;           // 0: the second half of a unit with one row tile
  u.safe_lo = u.safe_hi = 0;
  if (!rm.pool_rows && rm.use_own) {
    const int len = cache_len(a, b);
    const int lo = key_span(a, len, 0).lo;
    u.safe_lo = a.sinks >= lo ? 0 : lo;
    u.safe_hi = len == a.S ? INT_MAX : len;      // the map fills with zeros from S on
  }
  for (int t = 0; t < 2; ++t) {
    u.lead[t] = u.oa[t] = u.ob[t] = 0;
    const int ra = u.r0[t], rz = t == 0 ? min(u.r0[1], r1) : r1;
    if (ra >= rz) continue;                      // no rows
    u.lead[t] = u.oa[t] = u.ob[t] = max(0, min(u.nt, u.tp + u.ts - u.t0));
    if (to == 0) continue;
    int i0, i1;
    query_range(a, ra, rz, i0, i1);
    const int len = cache_len(a, b);
    int lo = key_span(a, len, i0).lo;
    const int hi = key_span(a, len, i1).hi;
    if (hi <= lo) {                              // padding rows alone: nothing to see
      u.lead[t] = u.oa[t] = u.ob[t] = 0;
      continue;
    }
    if (a.sinks > u.kl.lo) lo = u.kl.lo;         // sinks among the first own tiles
    const int base = u.tp + u.ts - u.t0;         // the first own tile, in this split's count
    u.oa[t] = max(0, min(u.nt, base + (lo - u.kl.lo) / KT));
    u.ob[t] = max(u.oa[t], min(u.nt, base + (hi - u.kl.lo + KT - 1) / KT));
  }
  return true;
}

#ifdef __CUDACC__
// A row's weights are 2^(s mul + add), one fused step: mul is the scale in base 2, add
// minus the rounded product of it and the reference.  They share a factor 2^c,
// |c| <= 2^-24 |add|, which the division cancels, but which leaves the number range
// once the product passes 2^31.  A reference with a product m beyond kFar takes mul
// down until it is kFar: |c| is then 2^6 at most, and scores that differ at all are
// 2^6 apart still, so that those below the largest have no weight, as they should.
// (Kept over the tiles: where the reference stays, nothing is computed.  Prompt of 8192
// tokens, window 2048: 250 us, taking -m anew in every tile 253; four images 887, 895;
// units of few tiles, 24 heads' 256 queries on 3515 tokens: 32.8, 32.0.)
struct RowRef {
  float mul, add;
};
constexpr float kFar = 1073741824.f;         // 2^30
__device__ __forceinline__ RowRef row_ref(float top, float m, float sl2) {
  RowRef r{sl2, -m};
  if (__builtin_expect(fabsf(m) > kFar, 0)) {
    r.mul = __fdividef(0.25f * kFar, 0.25f * fabsf(top));   // (0 from 2^126 on)
    r.add = -(top * r.mul);
  }
  return r;
}
#endif

}  // namespace area
