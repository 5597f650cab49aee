// extern "C" entry points of the key/value cache: argument validation, the
// launches of a call and the layout of its workspace.
#include <math.h>

#include "cache.cuh"

namespace area {
namespace {

constexpr int64_t kSms = 148;        // B200; the workspace's size may not hang on the device

// Most keys of a unit of the kernels for many rows: a role may wait for another through
// a whole unit, 0.4 s with as many (fp32, D = 128), and waits end after 2 s.
constexpr int64_t kUnitKeys = 1 << 23;
constexpr double kPoolBytes = 32 << 20;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t ceil256(int64_t n) { return (n + 255) & ~int64_t(255); }

// Rows that one work item of a kernel takes.
int rows_per_block(int kernel, int dtype, const CacheRows& rm) {
  switch (kernel) {
    case CACHE_TC: return dtype == AREA_DTYPE_BF16 ? 2 * tc_tile_rows(rm) : 128;
    default:
      if (dtype == AREA_DTYPE_BF16) return 8;
      return rm.RG <= 2 ? 2 : rm.RG <= 4 ? 4 : 8;
  }
}

// What a launch of `units` that need `keys` keys each takes when those are split
// n ways, in us: waves of `slots` units at once, a unit `fixed` and `per_key` a key.
// A last wave that is not full goes faster, down to `alone` of that.  Splits
// cost the join: 3 us, and their outputs written and read again.
struct SplitCost {
  int64_t units, keys, slots, rows;
  int D;
  double fixed, per_key, alone;
  double operator()(int64_t n) const {
    const int64_t all = units * n, waves = all / slots, rest = all % slots;
    const double k = per_key * (double)cdiv(keys, n);
    double t = (double)waves * (fixed + k);
    if (rest) t += fixed + k * std::max(alone, alone + (1 - alone) * (1.5 * rest / slots - 0.5));
    return n > 1 ? t + 3.0 + (double)rows * n * D * 8 / 5.0e6 : t;
  }
};
// The best of no split and those that fill one to five waves; `most` at most.
// (More waves even out sequences of different lengths, but each costs.)
int64_t best_split(const SplitCost& c, int64_t most) {
  int64_t best = 1;
  double least = c(1);
  for (int w = 1; w <= 5; ++w) {
    const int64_t n = std::min(w * c.slots / c.units, most);
    if (n <= best) continue;
    const double t = c(n);
    if (t < least) {
      least = t;
      best = n;
    }
    if (n == most) break;
  }
  return best;
}

// What the kernels for few and for many rows take, in us, for a launch of `groups`
// groups of RG rows: a start, a further wave, and a block's or unit's keys; with
// weights, the scores that few rows leave are read per row, those of many rows are
// computed twice.  From runs of 2 to 256 groups of 12 to 64 rows and 50 to 8000 keys,
// bf16 at D = 128 for example (few rows / many): 16 groups of 32 rows, 200 keys: 8.5 /
// 10.8 us, 1000: 13.8 / 13.0, 8000: 38 / 22; 2 groups of 16, 1000 keys: 7.4 / 11.7;
// 64 of 64, 200 keys: 20 / 15; with weights, 64 of 16, 500 keys: 24 / 21, 8000: 100 /
// 119.
struct KernelCost {
  double few, few_row, few_key, many, many_key;
};
constexpr KernelCost kCost[2][2][2] = {                      // weights, fp32, D = 128
    {{{5, 0, 3.1e-5, 8, 8.2e-5}, {5, 0, 6.0e-5, 8, 9.7e-5}},
     {{7, 0, 9.4e-5, 12, 1.84e-4}, {8, 0, 1.7e-4, 15, 3.0e-4}}},
    {{{8, 0.55, 5.8e-5, 13, 1.76e-4}, {8, 0.55, 8.6e-5, 13, 2.0e-4}},
     {{10, 0.5, 1.1e-4, 14, 3.37e-4}, {10, 0.5, 1.95e-4, 18, 6.8e-4}}}};

// Blocks of the kernel for few rows that run at once on an SM.
int few_per_sm(int dtype, int D) {
  return dtype == AREA_DTYPE_BF16 ? (D == 64 ? 4 : 3) : (D == 64 ? 3 : 2);
}

// Whether the rows of query heads that share a key head go apart (a row tile ends with
// its head) or one after the other.  Apart, tiles leave out what a window or the causal
// order hides from all their rows; together, fewer tiles end early.  Compared is what
// the units of a key head cost either way, a unit with one row tile of its two 0.63
// (bf16, apart / together: 16 heads' 300 queries on 20000 keys 90 / 60 us, 2500 on
// 2500 46 / 90; 400 on a window of 500 22 / 24).
bool heads_apart(int G, int Nq, int P, int S, int64_t window, int64_t sinks, int dtype) {
  if (Nq < 128) return false;
  if (sinks + window < S) return true;
  auto units = [&](int64_t rows) {
    const int64_t t = cdiv(rows, 128);
    return dtype == AREA_DTYPE_BF16 ? (double)(t / 2) + 0.63 * (double)(t % 2) : (double)t;
  };
  const double together = (double)S + P, apart = together - 0.5 * std::min(Nq, S);
  return G * units(Nq) * apart <= units((int64_t)G * Nq) * together;
}

int choose_kernel(const CacheRows& rm, int op, int dtype, int64_t few_keys, int64_t many_keys, int D) {
  const bool weights = op == CACHE_OP_WEIGHTS, f32 = dtype == AREA_DTYPE_F32;
  // one block's rows: a row tile of 128 would be nearly empty
  if (rm.RG <= 8) return CACHE_DEC;
  if (weights && rm.RG > kCacheFewWeights) return CACHE_TC;
  const KernelCost& c = kCost[weights][f32][D == 128];
  const int64_t blocks = rm.groups * cdiv(rm.RG, rows_per_block(CACHE_DEC, dtype, rm));
  const int64_t units = rm.groups * cdiv(rm.RG, rows_per_block(CACHE_TC, dtype, rm));
  const double few = c.few + c.few_row * rm.RG + 5.0 * ((blocks - 1) / (few_per_sm(dtype, D) * kSms)) +
                     c.few_key * (double)blocks * (double)few_keys;
  const double many = c.many + 4.0 * ((units - 1) / kSms) + c.many_key * (double)units * (double)many_keys;
  return few <= many ? CACHE_DEC : CACHE_TC;
}

// Chooses a launch's kernel, and splits its keys: at most few_keys or many_keys of
// them, for a block of either kernel.  even: most sequences have as many.
void cut(CacheLaunch& l, int op, int dtype, int64_t few_keys, int64_t many_keys, int64_t rows, int D,
         bool even) {
  const int RG = l.rows.RG;
  l.used = true;
  l.cluster = 1;
  l.warps = 4;
  l.kernel = choose_kernel(l.rows, op, dtype, few_keys, many_keys, D);
  const int64_t keys = l.kernel == CACHE_DEC ? few_keys : many_keys;
  const int64_t blocks = l.rows.groups * cdiv(RG, rows_per_block(l.kernel, dtype, l.rows));
  int64_t n;
  if (l.kernel == CACHE_TC) {
    // measured per unit: 4 us, and 2.1 us for 128 keys (bf16, 256 rows), 3.2 or
    // 5.6 us (fp32, 128 rows, D = 64 or 128)
    const double tile = dtype == AREA_DTYPE_BF16 ? 2.1 : D == 64 ? 3.2 : 5.6;
    n = best_split({blocks, keys, kSms, rows, D, 4.0, tile / 128, 1.0}, cdiv(keys, 256));
    n = std::max(n, cdiv(keys, kUnitKeys));
  } else {
    const int64_t slots = few_per_sm(dtype, D) * kSms;
    if (blocks * 8 <= slots && (keys <= 4096 || blocks * 8 >= 2 * kSms)) {
      // All blocks run at once: a cluster of up to 8 joins its splits itself
      // (4 heads of 500 keys: 6.0 us, with a join launch 7.1).  In larger grids
      // the blocks of a cluster wait for room together (512 heads of 4100 keys in
      // 8 splits: 214 us, without clusters 186).
      while (l.cluster < 8 && l.cluster * 128 < keys) l.cluster *= 2;
      n = l.cluster;
      // Eight warps, fewer steps each, where every SM has one block at most (8 heads of
      // 4000 keys, bf16: 12.9 -> 10.7 us, fp32 15.3 -> 13.5).  One block fills an SM's
      // registers (bf16 with D = 64: half), so that more than 12 clusters of 8 may find no room
      // in their part of the GPU (16 clusters: 14.6 -> 20.6 us).
      const bool half = dtype == AREA_DTYPE_BF16 && D == 64;
      if (blocks * n <= (half ? kSms : 96) && keys > 64 * n) l.warps = 8;
    } else {
      // all slots together read 6.3 TB/s (64 heads of 8000 keys in 6 splits, 0.86
      // waves: 51 us, in 8, 1.15 waves: 68)
      const double key = (dtype == AREA_DTYPE_BF16 ? 4.0 : 8.0) * D * (double)slots / 6.3e6;
      n = best_split({blocks, keys, slots, rows, D, 3.0, key, 0.64}, cdiv(keys, 128));
      // More blocks than run at once: those of the longest sequences first (100
      // heads' sequences of 10 to 9000 tokens: 345 -> 273 us; 32 of 2000 to 8192 with
      // weights 144 -> 132).  It costs 2 to 5 us: not where a window evens them out.
      l.rows.by_length = even ? 0 : blocks * n > slots && !l.rows.pool_rows && l.rows.kv_div == 1;
    }
  }
  l.nsplit = (int)std::max<int64_t>(n, 1);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Buf {               // null: none
  const void* p;
  int64_t n;
};
bool overlap(const Buf& a, const Buf& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + (uintptr_t)b.n && y < x + (uintptr_t)a.n;
}

}  // namespace

int cache_plan(int op, int B, int H, int Hk, int Nq, int P, int S, int D, int window, int sinks,
               int dtype, CachePlan* p) {
  if (dtype != AREA_DTYPE_F32 && dtype != AREA_DTYPE_BF16) return AREA_EUNSUPPORTED;
  if (B < 1 || H < 1 || Hk < 1 || Nq < 1 || P < 0 || S < 0) return AREA_EINVAL;
  if (H % Hk || window < 1 || sinks < 0) return AREA_EINVAL;
  if (S < 1 && P < 1) return AREA_EINVAL;
  if (D != 64 && D != 128) return AREA_EUNSUPPORTED;
  // row and key indexes are 32-bit, also rounded up to a block; a key list may hold
  // prefix and cache
  if ((int64_t)P + S > INT_MAX - 256) return AREA_EUNSUPPORTED;
  if ((int64_t)B * H > INT_MAX) return AREA_EUNSUPPORTED;
  p->rows = (int64_t)B * H * Nq;
  if (p->rows > INT_MAX - 256) return AREA_EUNSUPPORTED;
  const int R = H / Hk * Nq;
  // Few rows of a sequence: the prefix against the rows of all sequences, once
  // it is so large that reading it from L2 for each costs more than the second
  // launch and the join.  Pooled / not, us, by the bytes that all sequences would read,
  // bf16: 6 MB 15.1 / 11.5; 31 MB 15.5 / 16.6 and 15.1 / 13.8; 62 MB 22.6 / 19.0 and
  // 22.9 / 27.4; 125 MB 23.4 / 39.6 and 26.0 / 26.5; 938 MB 43 / 188.  fp32: 31 MB 23 /
  // 18, 62 MB 25 / 17 to 33 / 42, 250 MB 39 / 47, 938 MB and more 95 / 533.  (30000
  // keys, 64 sequences, bf16, by the rows: 32: 56 / 190; 48: 78 / 192.  Of 64 rows on
  // two sequences fill a row tile, or one: 64: 80 / 194, 128: 140 / 201, but with 8
  // sequences 40 / 38 and 43 / 40, with two 28 / 27 and 38 / 29; fp32 335 / 615 and
  // 666 / 658.  The limit is on the safe side for small batches; large ones would gain.)
  const double pre = (double)B * Hk * P * D * (dtype == AREA_DTYPE_BF16 ? 4 : 8);
  const bool pool = op == CACHE_OP_PREFIX && P > 0 && B > 1 && R < 64 && pre > kPoolBytes;
  p->pooled = CacheLaunch{};
  CacheLaunch& m = p->main;
  m = CacheLaunch{};
  const bool per_head = heads_apart(H / Hk, Nq, P, S, window, sinks, dtype);
  m.rows = CacheRows{per_head ? Nq : R, per_head ? B * H : B * Hk, per_head ? H / Hk : 1, 0,
                     P > 0 && !pool, S > 0, 0};
  // keys that a block of n rows can see at most
  auto own = [&](int64_t n) {
    return std::min<int64_t>(S, (int64_t)sinks + window + std::min<int64_t>(n, Nq));
  };
  const int64_t pk = m.rows.use_prefix ? P : 0;
  if (!pool || S > 0) cut(m, op, dtype, own(per_head ? 8 : Nq) + pk, own(256) + pk, p->rows, D, own(256) < S);
  p->slots = m.used ? m.nsplit / m.cluster : 0;
  if (pool) {
    p->pooled.rows = CacheRows{B * R, Hk, 1, R, 1, 0, 0};
    cut(p->pooled, op, dtype, P, P, p->rows, D, true);
    p->slots += p->pooled.nsplit / p->pooled.cluster;
  }
  // The weights need a row's whole sum: the kernel for few rows has it when one
  // block or cluster has all of a key head's rows and splits, and adds them up
  // from its scores; the others leave the sums for a launch of its own.
  const bool weights = op == CACHE_OP_WEIGHTS, few = m.kernel == CACHE_DEC;
  const bool whole = !weights || !few || m.rows.RG <= rows_per_block(CACHE_DEC, dtype, m.rows);
  if (p->slots == 1 && whole) p->slots = 0;
  p->off_ml = 0;
  p->off_o = p->off_ml + ceil256(p->slots * p->rows * 8);
  p->off_lse = p->off_o + ceil256(p->slots * p->rows * D * 4);
  p->off_logits = p->off_lse + (weights && !few ? ceil256(p->rows * 4) : 0);
  if (p->rows > (int64_t(1) << 58) / (S + 1)) return AREA_EUNSUPPORTED;
  p->bytes = p->off_logits + (weights && few ? ceil256(p->rows * S * 4) : 0);
  auto blocks = [&](const CacheLaunch& l) {
    return l.used ? cdiv(l.rows.RG, rows_per_block(l.kernel, dtype, l.rows)) * l.rows.groups * l.nsplit : 0;
  };
  if (blocks(m) > INT_MAX - 1024 || blocks(p->pooled) > INT_MAX - 1024 || cdiv(S, 128) * B * Hk > INT_MAX ||
      (weights && few && p->rows + cdiv(S, 512) * B * Hk > INT_MAX))
    return AREA_EUNSUPPORTED;
  return AREA_OK;
}

namespace {

int finish(cudaError_t e) { return e == cudaSuccess ? AREA_OK : fail_cuda(e); }

int cache_call(int op, CacheArgs& a, float scale, const float* acc, float* acco, void* ws,
               size_t ws_bytes, int dtype, cudaStream_t s) {
  if (!a.q || !a.o) return AREA_EINVAL;
  CachePlan p;
  const int st = cache_plan(op, a.B, a.H, a.Hk, a.Nq, a.P, a.S, a.D, a.window, a.sinks, dtype, &p);
  if (st != AREA_OK) return st;
  if ((a.S > 0 && (!a.k || !a.v)) || (a.P > 0 && (!a.kp || !a.vp))) return AREA_EINVAL;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || !isfinite(a.scale_log2)) return AREA_EINVAL;
  if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.kp, 16) ||
      !aligned(a.vp, 16) || !aligned(a.o, 32) || !aligned(a.lens, 4))
    return AREA_EINVAL;
  if (ws_bytes < (size_t)p.bytes) return AREA_ENOSPACE;
  if ((p.bytes > 0 && !ws) || !aligned(ws, 32)) return AREA_EINVAL;
  // what a call writes touches neither its inputs nor itself, except acco = acc
  const int64_t e2 = dtype == AREA_DTYPE_F32 ? 4 : 2, most = int64_t(1) << 50;
  const int64_t kv = std::min((int64_t)a.B * a.Hk * a.S, most), pre = std::min((int64_t)a.Hk * a.P, most);
  const int64_t no = p.rows * a.D * e2, nkv = kv * a.D * e2, npre = pre * a.D * e2;
  const Buf in[7] = {{a.q, no},     {a.k, nkv},   {a.v, nkv}, {a.kp, npre},
                     {a.vp, npre}, {a.lens, a.B * 4ll}, {acc, kv * 4}};
  const Buf to[3] = {{a.o, no}, {acco, kv * 4}, {ws, p.bytes}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 7; ++j)
      if (!(i == 1 && j == 6 && acc == acco) && overlap(to[i], in[j])) return AREA_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(to[i], to[j])) return AREA_EINVAL;
  }
  char* w = static_cast<char*>(ws);
  CacheOut out{};
  out.direct = p.slots == 0;
  out.rows = p.rows;
  if (p.slots) {
    out.part_ml = reinterpret_cast<float2*>(w + p.off_ml);
    out.part_o = reinterpret_cast<float*>(w + p.off_o);
  }
  const bool weights = op == CACHE_OP_WEIGHTS, few = p.main.kernel == CACHE_DEC;
  float* lse = weights && !few ? reinterpret_cast<float*>(w + p.off_lse) : nullptr;
  if (weights && few) {
    out.logits = reinterpret_cast<float*>(w + p.off_logits);
    out.acc = acc;
    out.acco = acco;
  } else if (out.direct) {
    out.lse = lse;
  }
  cudaError_t e;
  const CacheLaunch* ls[2] = {&p.main, &p.pooled};
  for (const CacheLaunch* l : ls) {
    if (!l->used) continue;
    out.nsplit = l->nsplit;
    out.cluster = l->cluster;
    out.warps = l->warps;
    switch (l->kernel) {
      case CACHE_TC:
        e = dtype == AREA_DTYPE_BF16 ? launch_cache_tc(a, l->rows, out, s)
                                     : launch_cache_tc32(a, l->rows, out, s);
        break;
      default:
        e = dtype == AREA_DTYPE_BF16 ? launch_cache_dec_bf16(a, l->rows, out, s)
                                     : launch_cache_dec_f32(a, l->rows, out, s);
    }
    if (e != cudaSuccess) return fail_cuda(e);
    out.slot0 += l->nsplit / l->cluster;
    out.early = 1;         // launches for other keys do not read one another's results
  }
  if (p.slots) {
    e = weights && few ? launch_cache_join_weights(a, out, p.slots, dtype, s)
                       : launch_cache_join(a, out.part_o, out.part_ml, p.slots, p.rows, lse, dtype, s);
    if (e != cudaSuccess) return fail_cuda(e);
  }
  return lse ? finish(launch_cache_weights_tc(a, lse, acc, acco, dtype, s)) : AREA_OK;
}

int ws_bytes_of(int op, int B, int H, int Hk, int Nq, int P, int S, int D, int window, int sinks,
                int dtype, size_t* ws_bytes) {
  if (!ws_bytes) return AREA_EINVAL;
  CachePlan p;
  const int st = cache_plan(op, B, H, Hk, Nq, P, S, D, window, sinks, dtype, &p);
  if (st == AREA_OK) *ws_bytes = (size_t)p.bytes;
  return st;
}

}  // namespace
}  // namespace area

extern "C" {

int area_sink_attn_ws_bytes(int B, int H, int Hk, int Nq, int S, int D, int window, int sinks,
                            int dtype, size_t* ws_bytes) {
  if (S < 1) return AREA_EINVAL;
  return area::ws_bytes_of(area::CACHE_OP_SINK, B, H, Hk, Nq, 0, S, D, window, sinks, dtype,
                           ws_bytes);
}

int area_sink_attn(const void* q, const void* k, const void* v, const int* lens, void* o, void* ws,
                   size_t ws_bytes, int B, int H, int Hk, int Nq, int S, int D, int window,
                   int sinks, float scale, int dtype, cudaStream_t stream) {
  if (S < 1) return AREA_EINVAL;
  area::CacheArgs a{q, k, v, nullptr, nullptr, lens, o, B, H, Hk, Nq, 0, S, D, window, sinks, 1, 0.f};
  return area::cache_call(area::CACHE_OP_SINK, a, scale, nullptr, nullptr, ws, ws_bytes, dtype,
                          stream);
}

int area_prefix_attn_ws_bytes(int B, int H, int Hk, int Nq, int P, int S, int D, int dtype,
                              size_t* ws_bytes) {
  return area::ws_bytes_of(area::CACHE_OP_PREFIX, B, H, Hk, Nq, P, S, D, INT_MAX, 0, dtype,
                           ws_bytes);
}

int area_prefix_attn(const void* q, const void* kp, const void* vp, const void* k, const void* v,
                     const int* lens, void* o, void* ws, size_t ws_bytes, int B, int H, int Hk,
                     int Nq, int P, int S, int D, int causal, float scale, int dtype,
                     cudaStream_t stream) {
  if (causal != 0 && causal != 1) return AREA_EINVAL;
  if (S == 0) lens = nullptr;              // not read: every sequence has no tokens of its own
  area::CacheArgs a{q, k, v, kp, vp, lens, o, B, H, Hk, Nq, P, S, D, INT_MAX, 0, causal, 0.f};
  return area::cache_call(area::CACHE_OP_PREFIX, a, scale, nullptr, nullptr, ws, ws_bytes, dtype,
                          stream);
}

int area_cache_attn_ws_bytes(int B, int H, int Hk, int Nq, int S, int D, int dtype,
                             size_t* ws_bytes) {
  if (S < 1) return AREA_EINVAL;
  return area::ws_bytes_of(area::CACHE_OP_WEIGHTS, B, H, Hk, Nq, 0, S, D, INT_MAX, 0, dtype,
                           ws_bytes);
}

int area_cache_attn(const void* q, const void* k, const void* v, const int* lens, const float* acc,
                    void* o, float* acco, void* ws, size_t ws_bytes, int B, int H, int Hk, int Nq,
                    int S, int D, float scale, int dtype, cudaStream_t stream) {
  if (S < 1 || !acco || !area::aligned(acco, 4) || !area::aligned(acc, 4)) return AREA_EINVAL;
  area::CacheArgs a{q, k, v, nullptr, nullptr, lens, o, B, H, Hk, Nq, 0, S, D, INT_MAX, 0, 1, 0.f};
  return area::cache_call(area::CACHE_OP_WEIGHTS, a, scale, acc, acco, ws, ws_bytes, dtype, stream);
}

int area_cache_evict(const void* k, const void* v, const float* acc, const int* lens, void* ko,
                     void* vo, float* acco, int* lenso, int* idx, int B, int Hk, int S, int So,
                     int D, int budget, int sinks, int recent, int dtype, cudaStream_t stream) {
  using area::aligned;
  using area::overlap;
  if (!k || !v || !acc || !ko || !vo || !acco || !lenso || !idx) return AREA_EINVAL;
  if (B < 1 || Hk < 1 || S < 1 || So < 1) return AREA_EINVAL;
  if (budget < 1 || budget > So || sinks < 0 || recent < 0 ||
      (int64_t)sinks + recent > budget)
    return AREA_EINVAL;
  if (dtype != AREA_DTYPE_F32 && dtype != AREA_DTYPE_BF16) return AREA_EUNSUPPORTED;
  if (D != 64 && D != 128) return AREA_EUNSUPPORTED;
  if (S > INT_MAX - 4096 || So > INT_MAX - 4096) return AREA_EUNSUPPORTED;   // 32-bit indexes
  const int64_t heads = (int64_t)B * Hk, elem = dtype == AREA_DTYPE_F32 ? 4 : 2;
  if (heads > INT_MAX || heads * std::max<int64_t>(2 * D * elem / 64 + 1, 8) > INT_MAX ||
      heads * area::cdiv(budget, 512 / (D * elem / 16)) > INT_MAX)
    return AREA_EUNSUPPORTED;                                                // grid sizes
  for (const void* p : {k, v, (const void*)ko, (const void*)vo})
    if (!aligned(p, 16)) return AREA_EINVAL;
  for (const void* p : {(const void*)acc, (const void*)lens, (const void*)acco,
                        (const void*)lenso, (const void*)idx})
    if (!aligned(p, 4)) return AREA_EINVAL;
  // in place: all three of k, v and acc; otherwise no output may touch an input
  const bool in_place = k == ko || v == vo || acc == acco;
  if (in_place && (k != ko || v != vo || acc != acco || S != So)) return AREA_EINVAL;
  const int64_t nin = heads * S, nout = heads * So;
  using area::Buf;
  const Buf in[4] = {{k, nin * D * elem}, {v, nin * D * elem}, {acc, nin * 4}, {lens, lens ? B * 4ll : 0}};
  const Buf to[5] = {{lenso, B * 4ll}, {idx, nout * 4}, {ko, nout * D * elem},
                     {vo, nout * D * elem}, {acco, nout * 4}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 4; ++j)
      if (!(in_place && i >= 2 && j == i - 2) && overlap(to[i], in[j]))
        return AREA_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(to[i], to[j])) return AREA_EINVAL;
  }
  const area::EvictArgs e{k, v, acc, lens, ko, vo, acco, lenso, idx, B, Hk, S, So, D,
                          budget, sinks, recent, (int)elem};
  return area::finish(area::launch_cache_evict(e, stream));
}

}  // extern "C"
