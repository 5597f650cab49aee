// Attention over a key/value cache: what the translation units of
// area_sink_attn, area_prefix_attn and area_cache_attn share.
//
// All three are one problem.  Query head h reads key head h / (H / Hk).  A
// sequence's Nq queries are its last tokens: query i sits at position
// p = len - Nq + i and sees
//   * the P shared prefix keys (prefix call), unless it is causal and p < 0;
//   * of the sequence's own keys, j <= p (causal) or j < len, and with a
//     window only j > p - window or j < sinks.
// A split of the keys over several CTAs leaves per split and row the running
// maximum m (log2 units), the sum l and the unnormalised output; cache_join.cu
// adds them up.
#pragma once

#include <limits.h>

#include <algorithm>

#include "area_internal.cuh"

namespace area {

struct CacheArgs {
  const void *q, *k, *v;     // [B, H, Nq, D], [B, Hk, S, D]
  const void *kp, *vp;       // [Hk, P, D] or null
  const int* lens;           // [B] or null: every sequence has S tokens
  void* o;                   // [B, H, Nq, D]
  int B, H, Hk, Nq, P, S, D;
  int window, sinks;         // window: INT_MAX without one
  int causal;
  float scale_log2;          // softmax scale times log2(e)
};

// How one launch cuts rows and keys.  A row group is RG rows that follow one
// another in q and read the same keys: the G * Nq rows of a key head, or the
// Nq rows of a query head; group g reads key head g / kv_div of B * Hk.  In a
// pooled launch group g is key head g of the prefix and has the rows of all B
// sequences, pool_rows of each.
struct CacheRows {
  int RG;          // rows of a group
  int groups;
  int kv_div;
  int pool_rows;   // 0: not pooled
  int use_prefix;  // the launch covers the prefix keys
  int use_own;     // the launch covers the sequences' own keys
  int by_length;   // kernels for few rows: the longest sequences' blocks first
};

// Where a launch leaves its results.
struct CacheOut {
  int nsplit;        // splits of this launch
  int cluster;       // splits that one cluster joins; the others' slots hold one split
  int slot0;         // its first slot in part_o / part_ml
  int warps;         // of a block of the kernels for few rows
  int early;         // the launch may start before the call's last one is done
  int direct;        // 1: one split in all, the output is written to o
  float* part_o;     // [slots][rows][D]
  float2* part_ml;   // [slots][rows] (m, l)
  float* logits;     // [rows][S] scores in log2 units, or null (kernels for few rows)
  float* lse;        // [rows] log2-sums, +inf without a key, or null (kernels for many
                     // rows, when direct)
  int64_t rows;      // B * H * Nq
  const float* acc;  // with a direct launch that has scores: the weights' sums
  float* acco;
};

__host__ __device__ __forceinline__ int cache_len(const CacheArgs& a, int b) {
  if (!a.lens || a.S == 0) return a.S;       // without room for tokens lengths are not read
  const int n = a.lens[b];
  return n < 0 ? 0 : n > a.S ? a.S : n;      // a length outside the cache is cut to it
}

// Own keys that query i of a sequence of len tokens sees: [lo, hi) and, below
// lo, the first `sinks`.  hi = 0: a causal query before the first token, which
// sees nothing, the prefix included.
struct KeySpan {
  int lo, hi;
};
__host__ __device__ __forceinline__ KeySpan key_span(const CacheArgs& a, int len, int i) {
  KeySpan s;
  s.hi = a.causal ? len - a.Nq + 1 + i : len;
  if (s.hi < 0) s.hi = 0;
  s.lo = s.hi > a.window ? s.hi - a.window : 0;
  return s;
}
__host__ __device__ __forceinline__ bool sees_prefix(const CacheArgs& a, KeySpan s) {
  return !a.causal || s.hi > 0;
}
__host__ __device__ __forceinline__ bool sees_own(const CacheArgs& a, KeySpan s, int j) {
  return j < s.hi && (j >= s.lo || j < a.sinks);
}

// Row r of group g: its row in q, o and the partial results, its sequence and
// its index among the sequence's queries.
struct CacheRow {
  int64_t row;
  int b, i;
};
__host__ __device__ __forceinline__ CacheRow cache_row(const CacheArgs& a, const CacheRows& rm, int g,
                                              int r) {
  CacheRow c;
  if (rm.pool_rows) {
    c.b = r / rm.pool_rows;
    const int rr = r - c.b * rm.pool_rows;
    c.row = ((int64_t)c.b * a.Hk + g) * rm.pool_rows + rr;
    c.i = rr % a.Nq;
  } else {
    c.b = g / rm.kv_div / a.Hk;
    c.row = (int64_t)g * rm.RG + r;
    c.i = r % a.Nq;
  }
  return c;
}

// The indexes of the queries of rows [r0, r1) run over [i0, i1], or over all
// where the rows pass from one head to the next.
__host__ __device__ __forceinline__ void query_range(const CacheArgs& a, int r0, int r1, int& i0,
                                                     int& i1) {
  i0 = r0 % a.Nq;
  i1 = (r1 - 1) % a.Nq;
  if (r1 - r0 >= a.Nq || i1 < i0) {
    i0 = 0;
    i1 = a.Nq - 1;
  }
}

// The keys that rows [r0, r1) of a group see between them, as one list: the
// prefix, the sinks below the windows, the windows' union.
struct KeyList {
  int np;       // prefix keys
  int ns;       // sinks before lo
  int lo;       // first key of the windows' union
  int total;    // keys in all
};
__host__ __device__ __forceinline__ KeyList key_list(const CacheArgs& a, const CacheRows& rm, int b,
                                                     int r0, int r1) {
  KeyList l;
  l.np = rm.use_prefix ? a.P : 0;
  l.ns = l.lo = 0;
  l.total = l.np;
  if (rm.pool_rows || !rm.use_own) return l;
  int i0, i1;
  query_range(a, r0, r1, i0, i1);
  const int len = cache_len(a, b);
  const KeySpan first = key_span(a, len, i0), last = key_span(a, len, i1);
  if (!sees_prefix(a, last)) {       // every row before the first token
    l.np = l.total = 0;
    return l;
  }
  l.lo = first.lo;
  l.ns = a.sinks < first.lo ? a.sinks : first.lo;
  l.total = l.np + l.ns + (last.hi - first.lo);
  return l;
}

// A call's launches follow one another closely: a block of the next may start once
// every block of this one has called let_next_start() or ended, and what it reads of
// earlier launches it reads after wait_for_last(), which returns when those are
// done.  Every launch that may start early waits before it ends, so that the end
// of a call's last launch is the end of all.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_last() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- host side ------------------------------------------------------------
// Launches a kernel in clusters of `cluster` blocks; early: before the last launch of
// the call is done (see let_next_start).
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), int64_t grid, int threads, size_t smem, int cluster,
                          bool early, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (early) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

enum { CACHE_OP_SINK, CACHE_OP_PREFIX, CACHE_OP_WEIGHTS };

// The kernels: for few rows, for many rows.
enum { CACHE_DEC, CACHE_TC };
// Most rows of a key head whose scores the kernel for few rows leaves for the weights.
constexpr int kCacheFewWeights = 24;
// A launch of a call: the kernel, the rows and the splits of their keys.
struct CacheLaunch {
  bool used;
  int kernel;
  CacheRows rows;
  int nsplit;
  int cluster;
  int warps;       // of a block of the kernels for few rows
};
// The launches of a call and the layout of its workspace; cache_plan computes
// them from the sizes alone.
struct CachePlan {
  CacheLaunch main, pooled;   // pooled: the prefix against the rows of all sequences
  int slots;                  // partial results per row (0: the one launch writes o)
  int64_t rows;               // B * H * Nq
  int64_t off_ml, off_o, off_lse, off_logits, bytes;
};
int cache_plan(int op, int B, int H, int Hk, int Nq, int P, int S, int D, int window, int sinks,
               int dtype, CachePlan* p);

cudaError_t launch_cache_dec_bf16(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                                  cudaStream_t s);
cudaError_t launch_cache_dec_f32(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                                 cudaStream_t s);
// Joins `slots` partial results per row into o, and their log2-sum-exp into
// lse when that is given.
cudaError_t launch_cache_join(const CacheArgs& a, const float* part_o, const float2* part_ml,
                              int slots, int64_t rows, float* lse, int dtype, cudaStream_t s);
// The same for the kernels for few rows when they have left scores, and then
// acco[b, hk, j] = acc[b, hk, j] + sum over the rows that see j of
// 2^(logits[row][j] - log2-sum of the row).
cudaError_t launch_cache_join_weights(const CacheArgs& a, const CacheOut& out, int slots, int dtype,
                                      cudaStream_t s);

// Rows of a row tile of the bf16 tensor-core kernel: 128, or in a pooled launch as
// many whole sequences' rows as fit.
inline int tc_tile_rows(const CacheRows& rm) {
  return rm.pool_rows ? 128 / rm.pool_rows * rm.pool_rows : 128;
}
cudaError_t launch_cache_tc(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                            cudaStream_t s);
cudaError_t launch_cache_tc32(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                              cudaStream_t s);
cudaError_t read_and_clear_cache_tc_error(int* code);
cudaError_t read_and_clear_cache_tc32_error(int* code);
// The same sums for many rows of a key head: the scores are computed once more
// instead of read.
cudaError_t launch_cache_weights_tc(const CacheArgs& a, const float* lse, const float* acc,
                                    float* acco, int dtype, cudaStream_t s);
cudaError_t read_and_clear_cache_weights_error(int* code);

struct EvictArgs {
  const void *k, *v;
  const float* acc;
  const int* lens;
  void *ko, *vo;
  float* acco;
  int *lenso, *idx;
  int B, Hk, S, So, D, budget, sinks, recent, elem;   // elem: bytes of a value
};
// Where part `part` of n things begins when `parts` parts share them evenly.  (Parts
// are walked from here to the next one's, which no 32-bit index leaves: S and So end
// 4096 before the largest.)
__host__ __device__ __forceinline__ int share_of(int n, int part, int parts) {
  return (int)((int64_t)n * part / parts);
}
cudaError_t launch_cache_evict(const EvictArgs& e, cudaStream_t s);

}  // namespace area
