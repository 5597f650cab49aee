// What the kernels for few query rows share: how the results of a block's
// warps, and of the blocks of a cluster, become one.
#pragma once

#include <cooperative_groups.h>

#include "cache.cuh"

namespace area {
namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&f)[4]) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]), y = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                            *reinterpret_cast<const uint32_t*>(&y));
}

constexpr int kDecOrder = 128;            // sequences that a block can order

// The rows of a block and its warps' results.
template <int D, int ROWS, int WARPS>
struct DecSmem {
  int64_t row[ROWS];                     // -1: none
  KeySpan span[ROWS];
  float m[WARPS][ROWS], l[WARPS][ROWS];
  float bm[ROWS], bl[ROWS];              // of the whole block
  float lse[ROWS];
  __align__(16) float o[WARPS][ROWS][D];   // the block's in [0] in the end
};

// The group of a block whose place in the order is g: as it is, or the sequences
// from the longest to the shortest, so that the last blocks to start are short
// (up to kDecOrder sequences, as many as a block has threads).
__device__ __forceinline__ int dec_group(const CacheArgs& a, const CacheRows& rm, int g) {
  if (!rm.by_length || !a.lens || a.B == 1 || a.B > kDecOrder) return g;
  __shared__ int s_len[kDecOrder], s_b;
  const int i = threadIdx.x, hk = g % a.Hk, want = g / a.Hk;
  if (i < a.B) s_len[i] = cache_len(a, i);
  __syncthreads();
  if (i < a.B) {
    const int n = s_len[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < a.B; ++j) rank += s_len[j] > n || (s_len[j] == n && j < i);
    if (rank == want) s_b = i;
  }
  __syncthreads();
  return s_b * a.Hk + hk;
}

template <int D, int ROWS, int WARPS>
__device__ __forceinline__ void dec_rows(DecSmem<D, ROWS, WARPS>& sm, const CacheArgs& a,
                                         const CacheRows& rm, int g, int r0) {
  if (threadIdx.x < ROWS) {
    KeySpan s{0, 0};
    int64_t row = -1;
    if (r0 + (int)threadIdx.x < rm.RG) {
      const CacheRow cr = cache_row(a, rm, g, r0 + threadIdx.x);
      row = cr.row;
      s = key_span(a, cache_len(a, cr.b), cr.i);
    }
    sm.row[threadIdx.x] = row;
    sm.span[threadIdx.x] = s;
  }
  __syncthreads();
}

// The warps' results are in sm.m, sm.l, sm.o.  They are added up for the block
// in the warps' order; then the splits of a cluster, which sit in its blocks'
// shared memory, in the order of the ranks, each block a share of the outputs.
// The sums go to o when the cluster has all splits (out.direct), else to slot
// slot0 + sp / cluster size.  With out.acco the direct form then adds up the
// weights of the block's own keys [j0, j1), whose scores it has left in
// out.logits, and copies its share of the sums behind the last token.
template <typename T, int D, int ROWS, int WARPS>
__device__ __forceinline__ void dec_finish(DecSmem<D, ROWS, WARPS>& sm, const CacheArgs& a,
                                           const CacheOut& out, int sp, int kvh, int j0, int j1) {
  constexpr int kThreads = WARPS * 32, kVecs = ROWS * (D / 4);
  const auto cluster = cooperative_groups::this_cluster();
  const int cs = out.cluster, rank = sp % cs, tid = threadIdx.x;
  __syncthreads();
  for (int e = tid; e < kVecs; e += kThreads) {
    const int r = e / (D / 4), d = e % (D / 4) * 4;
    float mm = sm.m[0][r];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) mm = fmaxf(mm, sm.m[w][r]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, f[4] = {};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float al = ex2(sm.m[w][r] - ref);
      ll = fmaf(al, sm.l[w][r], ll);
      const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][d]);
      f[0] = fmaf(al, x.x, f[0]), f[1] = fmaf(al, x.y, f[1]);
      f[2] = fmaf(al, x.z, f[2]), f[3] = fmaf(al, x.w, f[3]);
    }
    store4(&sm.o[0][r][d], f);
    if (d == 0) sm.bm[r] = mm, sm.bl[r] = ll;
  }
  if (cs > 1) cluster.sync(); else __syncthreads();
  for (int e = rank * kThreads + tid; e < kVecs; e += cs * kThreads) {
    const int r = e / (D / 4), d = e % (D / 4) * 4;
    const int64_t row = sm.row[r];
    if (row < 0) continue;
    float mm = -INFINITY, ll = 0.f, f[4] = {};
    for (int i = 0; i < cs; ++i) mm = fmaxf(mm, *cluster.map_shared_rank(&sm.bm[r], i));
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
    for (int i = 0; i < cs; ++i) {
      const float al = ex2(*cluster.map_shared_rank(&sm.bm[r], i) - ref);
      ll = fmaf(al, *cluster.map_shared_rank(&sm.bl[r], i), ll);
      const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sm.o[0][r][d], i));
      f[0] = fmaf(al, x.x, f[0]), f[1] = fmaf(al, x.y, f[1]);
      f[2] = fmaf(al, x.z, f[2]), f[3] = fmaf(al, x.w, f[3]);
    }
    if (out.direct) {
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = ll == 0.f ? 0.f : f[i] * inv;
      store4(static_cast<T*>(a.o) + row * D + d, f);
    } else {
      const int64_t at = (int64_t)(out.slot0 + sp / cs) * out.rows + row;
      if (d == 0) out.part_ml[at] = make_float2(mm, ll);
      if (ll != 0.f) store4(out.part_o + at * D + d, f);
    }
  }
  if (out.direct && out.acco) {
    if (tid < ROWS) {
      float mm = -INFINITY, ll = 0.f;
      for (int i = 0; i < cs; ++i) mm = fmaxf(mm, *cluster.map_shared_rank(&sm.bm[tid], i));
      const float ref = mm == -INFINITY ? 0.f : mm;
      for (int i = 0; i < cs; ++i)
        ll = fmaf(ex2(*cluster.map_shared_rank(&sm.bm[tid], i) - ref),
                  *cluster.map_shared_rank(&sm.bl[tid], i), ll);
      // a row without a weight: +inf, so that 2^(x - lse) is 0 for every key
      sm.lse[tid] = ll == 0.f ? INFINITY : ref + log2f(ll);
    }
    __syncthreads();
    const int64_t at = (int64_t)kvh * a.S;
    for (int j = j0 + tid; j < j1; j += kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (j < sm.span[r].hi) sum += ex2(out.logits[sm.row[r] * a.S + j] - sm.lse[r]);
      out.acco[at + j] = (out.acc ? out.acc[at + j] : 0.f) + sum;
    }
    const int len = cache_len(a, kvh / a.Hk), behind = a.S - len;
    const int e1 = len + (int)((int64_t)behind * (sp + 1) / out.nsplit);
    for (int j = len + (int)((int64_t)behind * sp / out.nsplit) + tid; j < e1; j += kThreads)
      out.acco[at + j] = out.acc ? out.acc[at + j] : 0.f;
  }
  if (cs > 1) cluster.sync();            // the others have read this block's sums
  if (out.early) wait_for_last();
}

template <typename K>
cudaError_t launch_dec(K kernel, int64_t grid, const CacheArgs& a, const CacheRows& rm,
                       const CacheOut& out, int nrb, cudaStream_t s) {
  return launch_kernel(kernel, grid, out.warps * 32, 0, out.cluster, out.early, s, a, rm, out, nrb);
}

}  // namespace
}  // namespace area
