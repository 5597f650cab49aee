// Host-only check of how the tensor-core kernel for key/value caches cuts its
// work (cache_unit.cuh): over many problems, every row meets every key that it
// sees in exactly one tile that its row tile takes, no tile starts outside its
// tensor, and a tile loaded whole holds no row that nobody sees.  Exit code 0
// when every check holds.  Built and run by a CPU test.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "cache_unit.cuh"

using namespace area;

template <int KT, int TILES>
static int check(const CacheArgs& a, const CacheRows& rm, int nsplit) {
  UnitParams p{a, rm, CacheOut{}, 0, TILES == 2 ? tc_tile_rows(rm) : 128, TILES, 0, 0};
  p.out.nsplit = nsplit;
  const int unit_rows = TILES * p.tile_rows;
  p.nrb = (rm.RG + unit_rows - 1) / unit_rows;
  p.units = rm.groups * p.nrb * nsplit;
  const int whole = p.units;
  // in either order, with no unit, the last two and every unit in halves
  for (int turn = 0; turn < (TILES == 2 ? 6 : 2); ++turn) {
    p.heavy_first = turn % 2;
    p.halved = turn / 2 == 0 ? 0 : turn / 2 == 1 ? std::min(whole, 2) : whole;
    p.units = whole + p.halved;
    // per row of q: how often each key was met (prefix, then own)
    const int rows = a.B * a.H * a.Nq, keys = a.P + a.S;
    std::vector<unsigned char> met((size_t)rows * keys, 0), touched(rows, 0);
    Unit u;
    for (int idx = 0; idx < p.units; ++idx) {
      if (!decode_unit<KT>(idx, p, u)) return printf("unit %d missing\n", idx), 1;
      for (int j = 0; j < u.nt; ++j) {
        const Tile t = tile_of<KT>(u, j);
        if (t.n < 1 || t.n > KT || t.j0 < 0) return printf("tile of %d keys at %d\n", t.n, t.j0), 1;
        if (t.j0 + t.n > (t.kind ? a.S : a.P)) return printf("tile past its tensor\n"), 1;
        if (t.kind && !t.copy) {
          const int b = u.kvh / a.Hk, len = cache_len(a, b);
          const int lo = key_span(a, len, 0).lo;
          for (int key = t.j0; key < std::min(t.j0 + KT, a.S); ++key)
            if (key >= len || (key < lo && key >= a.sinks)) return printf("row %d loaded\n", key), 1;
        }
      }
      for (int t = 0; t < TILES; ++t) {
        const int first = first_tile(u, t), last = last_tile(u, t);
        int n = 0;
        for (int j = 0; j < u.nt; ++j) {
          if (!is_active(u, t, j)) continue;
          if (n++ == 0 && j != first) return printf("first tile\n"), 1;
          if (j > last) return printf("last tile\n"), 1;
        }
        // the softmax warps' walk takes exactly these tiles, in order
        int m = 0;
        for (int j = first, before = -1; j <= last; j = next_tile(j, u.lead[t], u.oa[t]), ++m)
          if (j <= before || !is_active(u, t, j)) return printf("walk takes tile %d\n", j), 1;
          else before = j;
        if (m != n) return printf("walk of %d tiles, not %d\n", m, n), 1;
        if ((n == 0) != (last < 0)) return printf("no tile, last %d\n", last), 1;
        if (n && !is_active(u, t, last)) return printf("last tile inactive\n"), 1;
        for (int r = u.r0[t]; r < std::min(u.r0[t] + p.tile_rows, rm.RG); ++r) {
          const CacheRow cr = cache_row(a, rm, u.g, r);
          if (cr.row < 0 || cr.row >= rows) return printf("row out of range\n"), 1;
          if (touched[cr.row]++ >= nsplit) return printf("row twice\n"), 1;
          const KeySpan sp = key_span(a, cache_len(a, cr.b), cr.i);
          for (int j = 0; j < u.nt; ++j) {
            if (!is_active(u, t, j)) continue;
            const Tile tl = tile_of<KT>(u, j);
            for (int x = 0; x < tl.n; ++x) {
              const int key = tl.j0 + x;
              // the limits that the kernel applies to a row's scores
              const bool in = tl.kind == 0 ? sees_prefix(a, sp)
                                           : key < sp.hi && (key >= sp.lo || key < a.sinks);
              if (in) ++met[(size_t)cr.row * keys + (tl.kind ? a.P + key : key)];
            }
          }
        }
      }
    }
    if (decode_unit<KT>(p.units, p, u)) return printf("a unit too many\n"), 1;
    for (int row = 0; row < rows; ++row) {
      if (touched[row] != nsplit) return printf("row %d in %d splits\n", row, touched[row]), 1;
      const int b = row / (a.H * a.Nq), i = row % a.Nq, len = cache_len(a, b);
      const int pos = len - a.Nq + i;
      for (int key = 0; key < keys; ++key) {
        const int j = key - a.P;
        bool sees;
        if (j < 0)
          sees = rm.use_prefix && (!a.causal || pos >= 0);
        else
          sees = rm.use_own && (a.causal ? j <= pos : j < len) &&
                 (!a.causal || (int64_t)j > (int64_t)pos - a.window || j < a.sinks);
        if (met[(size_t)row * keys + key] != (sees ? 1 : 0))
          return printf("row %d meets key %d %d times, sees it: %d\n", row, j,
                        met[(size_t)row * keys + key], sees), 1;
      }
    }
  }
  return 0;
}

int main() {
  unsigned seed = 1;
  auto rnd = [&](int n) {
    seed = seed * 1664525u + 1013904223u;
    return (int)((seed >> 8) % (unsigned)n);
  };
  int cases = 0;
  for (int it = 0; it < 700; ++it) {
    const int Hk = 1 + rnd(2), G = 1 + rnd(4), B = 1 + rnd(3);
    const int Nq = it % 3 == 0 ? 1 + rnd(40) : 1 + rnd(600);
    const int S = Nq + (rnd(2) ? rnd(700) : 0);
    const int mode = rnd(3);            // window, causal with a prefix, all keys with a prefix
    std::vector<int> lens(B);
    for (int& n : lens) n = rnd(4) == 0 ? rnd(S + 1) : rnd(3) ? S : S - rnd(S / 2 + 1);
    CacheArgs a{};
    a.lens = rnd(5) ? lens.data() : nullptr;
    a.B = B, a.H = G * Hk, a.Hk = Hk, a.Nq = Nq, a.S = S, a.D = 64;
    a.P = mode ? rnd(400) : 0;
    a.causal = mode < 2;
    a.window = mode ? INT_MAX : rnd(6) ? 1 + rnd(S) : 1 + rnd(130);
    a.sinks = mode ? 0 : rnd(3) ? rnd(8) : rnd(700);
    const int R = G * Nq;
    const bool per_head = rnd(2);
    const int nsplit = 1 + (rnd(2) ? rnd(6) : 0);
    const CacheRows own{per_head ? Nq : R, per_head ? B * G * Hk : B * Hk, per_head ? G : 1, 0,
                        a.P > 0, 1};
    if (check<128, 2>(a, own, nsplit) || check<64, 1>(a, own, nsplit))
      return printf("B=%d Hk=%d G=%d Nq=%d P=%d S=%d window=%d sinks=%d per_head=%d\n", B, Hk, G, Nq,
                    a.P, S, a.window, a.sinks, per_head), 1;
    ++cases;
    if (a.P > 0 && R < 64) {
      const CacheRows pooled{B * R, Hk, 1, R, 1, 0};
      if (check<128, 2>(a, pooled, nsplit) || check<64, 1>(a, pooled, nsplit)) return printf("pooled B=%d R=%d P=%d\n", B, R, a.P), 1;
      ++cases;
    }
  }
  printf("%d problems checked\n", cases);
  return 0;
}
