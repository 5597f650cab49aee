// Eviction from a key/value cache by accumulated attention weight.
//
// Of a sequence of n > budget tokens each key head keeps the first `sinks`,
// the last `recent` and, of the tokens between, the budget - sinks - recent
// with the largest accumulated weight (ties: the lowest index), in their
// order.  One launch chooses, and copies where the cache is short; in long caches a second
// one copies, in place a second one moves the rows.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace area {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 4, kTile = kThreads * kPer;     // candidates of a thread, of a block's step

// An integer that orders as the weight does; -0 as 0, a NaN as -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  if (w == 0.f) w = 0.f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const EvictArgs& e, int b) {
  if (!e.lens) return e.S;
  const int n = e.lens[b];
  return n < 0 ? 0 : n > e.S ? e.S : n;
}

// A thread's share of a block's copy: rows i0, i0 + step, ... < n of K and V, 16
// bytes of each per load, two rows in flight.  from(i): row i's old and new place.
template <typename F>
__device__ __forceinline__ void copy_rows(const EvictArgs& e, int64_t g, int n, F from) {
  const int chunks = e.D * e.elem / 16;                  // 16-byte pieces of a row: 8, 16 or 32
  const int per = kThreads / chunks, c = threadIdx.x % chunks;
  const uint4 *k = static_cast<const uint4*>(e.k) + g * e.S * chunks + c;
  const uint4 *v = static_cast<const uint4*>(e.v) + g * e.S * chunks + c;
  uint4 *ko = static_cast<uint4*>(e.ko) + g * e.So * chunks + c;
  uint4 *vo = static_cast<uint4*>(e.vo) + g * e.So * chunks + c;
  for (int i = threadIdx.x / chunks; i < n; i += 2 * per) {
    const int2 a = from(i), b = from(min(i + per, n - 1));
    const uint4 ka = __ldcs(k + (int64_t)a.x * chunks), va = __ldcs(v + (int64_t)a.x * chunks);
    const uint4 kb = __ldcs(k + (int64_t)b.x * chunks), vb = __ldcs(v + (int64_t)b.x * chunks);
    __stcs(ko + (int64_t)a.y * chunks, ka);
    __stcs(vo + (int64_t)a.y * chunks, va);
    if (i + per < n) {
      __stcs(ko + (int64_t)b.y * chunks, kb);
      __stcs(vo + (int64_t)b.y * chunks, vb);
    }
  }
}

// A cluster per (sequence, key head), each block a contiguous share of the
// candidates.  Radix selection of the smallest kept key from the top byte down:
// a block counts its share, the counts are added up over the cluster's shared
// memory; the lower ranks' counts also give a block the place of its first kept
// token.  Then every block writes its share's indexes in order and, with COPY,
// copies their rows.  Counts are integers: their order does not matter.  Without COPY,
// which serves long caches, candidates stay in registers over the passes (256 heads of
// 8192 tokens: 3 us less; caches of one step lose 1.5 us to the longer code).
template <bool COPY>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs e, int cs) {
  __shared__ int s_hist[4][256];
  __shared__ int s_tot[256];
  __shared__ int s_bin, s_above, s_gt, s_eq;   // kept keys above the threshold, equal to it, in lower ranks
  __shared__ int s_wgt[kWarps], s_weq[kWarps];
  __shared__ int s_list[kTile];
  let_next_start();
  const auto cluster = cooperative_groups::this_cluster();
  const int64_t g = blockIdx.x / cs;
  const int rank = blockIdx.x % cs, b = (int)(g / e.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = evict_len(e, b);
  const int kept = min(n, e.budget);
  const float* acc = e.acc + g * e.S;
  int* idx = e.idx + g * e.So;
  float* acco = e.acco + g * e.So;
  auto share = [&](int of, int r) { return share_of(of, r, cs); };
  if (g % e.Hk == 0 && rank == 0 && tid == 0) e.lenso[b] = kept;
  for (int j = kept + share(e.So - kept, rank) + tid; j < kept + share(e.So - kept, rank + 1);
       j += kThreads) {
    idx[j] = -1;
    if (COPY) acco[j] = 0.f;
  }
  // what is kept in any case: all, or the sinks and the last tokens
  const bool all = n <= e.budget;
  const int want = all ? 0 : e.budget - e.sinks - e.recent;      // to be chosen
  const int first = all ? n : e.sinks, fixed = all ? n : e.sinks + e.recent;
  const int f0 = share(fixed, rank), nf = share(fixed, rank + 1) - f0;
  auto always = [&](int i) {
    const int f = f0 + i;
    return f < first ? make_int2(f, f) : make_int2(n - fixed + f, want + f);
  };
  for (int i = tid; i < nf; i += kThreads) {
    const int2 m = always(i);
    idx[m.y] = m.x;
    if (COPY) acco[m.y] = acc[m.x];
  }
  if (COPY) copy_rows(e, g, nf, always);
  if (want == 0) return;                                 // the whole cluster does

  acc += e.sinks;
  const int cand = n - e.sinks - e.recent;               // tokens to choose from, > want
  const int c0 = share(cand, rank), c1 = share(cand, rank + 1);
#pragma unroll
  for (int p = 0; p < 4; ++p) s_hist[p][tid] = 0;
  if (tid == 0) s_gt = s_eq = 0;
  __syncthreads();
  constexpr int kHeld = COPY ? 0 : 16;                   // steps of kThreads
  uint32_t held[kHeld + 1];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = c0 + tid + i * kThreads;
    held[i] = j < c1 ? weight_key(acc[j]) : 0;
  }
  uint32_t prefix = 0;           // the bytes of the threshold found so far
  int left = want;               // kept keys among those that share them
#pragma unroll 1
  for (int p = 0; p < 4; ++p) {
    const int shift = 24 - 8 * p;
    auto count = [&](uint32_t key) {
      if (p == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&s_hist[p][key >> shift & 255], 1);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (c0 + tid + i * kThreads < c1) count(held[i]);
#pragma unroll 4
    for (int j = c0 + kHeld * kThreads + tid; j < c1; j += kThreads) count(weight_key(acc[j]));
    cluster.sync();
    int total = 0, lower = 0;                            // of bin tid
    for (int r = 0; r < cs; ++r) {
      const int x = *cluster.map_shared_rank(&s_hist[p][tid], r);
      total += x;
      if (r < rank) lower += x;
    }
    s_tot[tid] = total;
    __syncthreads();
    if (warp == 0) {
      // lane 0 holds the eight highest bins; `above` = keys in higher bins
      int h[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += h[i] = s_tot[255 - (lane * 8 + i)];
      int incl = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += t;
      }
      int above = incl - sum;
      if (above < left && incl >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < left && above + h[i] >= left) {
            s_bin = 255 - (lane * 8 + i);
            s_above = above;
          }
          above += h[i];
        }
      }
    }
    __syncthreads();
    if (tid > s_bin && lower) atomicAdd(&s_gt, lower);
    if (p == 3 && tid == s_bin) s_eq = lower;
    prefix |= (uint32_t)s_bin << shift;
    left -= s_above;
    __syncthreads();
  }
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  // keys above the threshold are kept, and the first `left` of those equal to it
  int gt0 = s_gt, eq0 = s_eq;    // found so far
  if constexpr (kHeld > 0) {
    // those in registers: every warp's counts of every step, their sums before it
    __shared__ int s_cnt[kHeld * kWarps], s_sum;         // above in the low half, equal in the high
    const unsigned below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const bool in = c0 + tid + i * kThreads < c1;
      const unsigned gt = __ballot_sync(0xffffffffu, in && held[i] > prefix);
      const unsigned eq = __ballot_sync(0xffffffffu, in && held[i] == prefix);
      if (lane == 0) s_cnt[i * kWarps + warp] = __popc(gt) | __popc(eq) << 16;
    }
    __syncthreads();
    if (warp == 0) {
      constexpr int kOwn = kHeld * kWarps / 32;
      int c[kOwn], sum = 0;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) c[i] = s_cnt[lane * kOwn + i], sum += c[i];
      int incl = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += t;
      }
      int before = incl - sum;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        s_cnt[lane * kOwn + i] = before;
        before += c[i];
      }
      if (lane == 31) s_sum = incl;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int j = c0 + tid + i * kThreads;
      const bool is_gt = j < c1 && held[i] > prefix, is_eq = j < c1 && held[i] == prefix;
      const unsigned gt = __ballot_sync(0xffffffffu, is_gt), eq = __ballot_sync(0xffffffffu, is_eq);
      const int base = s_cnt[i * kWarps + warp];
      const int gtb = gt0 + (base & 0xffff) + __popc(gt & below);
      const int eqb = eq0 + (base >> 16) + __popc(eq & below);
      if (is_gt || (is_eq && eqb < left)) idx[e.sinks + gtb + min(eqb, left)] = e.sinks + j;
    }
    gt0 += s_sum & 0xffff, eq0 += s_sum >> 16;
  }
  for (int j0 = c0 + kHeld * kThreads; j0 < c1; j0 += kTile) {
    const int j = j0 + tid * kPer;
    float w[kPer];
    uint32_t gt = 0, eq = 0;     // one bit per candidate of the thread
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      w[i] = j + i < c1 ? acc[j + i] : 0.f;
      const uint32_t key = weight_key(w[i]);
      if (j + i < c1 && key > prefix) gt |= 1u << i;
      if (j + i < c1 && key == prefix) eq |= 1u << i;
    }
    int igt = __popc(gt), ieq = __popc(eq);              // including this thread's
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int tg = __shfl_up_sync(0xffffffffu, igt, x), te = __shfl_up_sync(0xffffffffu, ieq, x);
      if (lane >= x) igt += tg, ieq += te;
    }
    if (lane == 31) s_wgt[warp] = igt, s_weq[warp] = ieq;
    __syncthreads();
    const int start = gt0 + min(eq0, left);              // kept tokens before this step
    int gtb = gt0 + igt - __popc(gt), eqb = eq0 + ieq - __popc(eq);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const int tg = s_wgt[x], te = s_weq[x];
      if (x < warp) gtb += tg, eqb += te;
      gt0 += tg, eq0 += te;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if ((gt >> i & 1u) || ((eq >> i & 1u) && eqb < left)) {
        const int at = gtb + min(eqb, left);
        idx[e.sinks + at] = e.sinks + j + i;
        if (COPY) {
          acco[e.sinks + at] = w[i];
          s_list[at - start] = e.sinks + j + i;
        }
      }
      gtb += gt >> i & 1u, eqb += eq >> i & 1u;
    }
    __syncthreads();
    if (COPY) {
      copy_rows(e, g, gt0 + min(eq0, left) - start,
                [&](int i) { return make_int2(s_list[i], e.sinks + start + i); });
      __syncthreads();
    }
  }
  // the others have read this block's counts
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// The copy of the kept rows on its own: blocks_per_head blocks take the rows of a
// head in equal shares, two to a thread (256 heads of 8192 tokens to 4096: 160 us, all
// of copy bandwidth).
__global__ void __launch_bounds__(kThreads) evict_copy_kernel(const EvictArgs e,
                                                              int blocks_per_head) {
  wait_for_last();
  const int64_t g = blockIdx.x / blocks_per_head;
  const int blk = blockIdx.x % blocks_per_head;
  const int m = min(evict_len(e, (int)(g / e.Hk)), e.budget);
  const int* idx = e.idx + g * e.So;
  const int r0 = share_of(m, blk, blocks_per_head), r1 = share_of(m, blk + 1, blocks_per_head);
  copy_rows(e, g, r1 - r0, [&](int i) { return make_int2(idx[r0 + i], r0 + i); });
  const int j1 = share_of(e.So, blk + 1, blocks_per_head);
  for (int j = share_of(e.So, blk, blocks_per_head) + threadIdx.x; j < j1; j += kThreads)
    e.acco[g * e.So + j] = j < m ? e.acc[g * e.S + idx[j]] : 0.f;
}

// The copy within the cache itself.  A kept row moves to an index not above
// its own, so a block that moves rows in ascending order, all of a step read
// before any is written, never writes a row that is still to be read.  A block
// has one 64-byte column of K or V, or the weights, of a key head.  The steps of a block
// follow one another, which bounds the call where heads are few: 8 heads of 40000
// tokens to 20000 take 245 us in bf16 (copied: 47) and 265 in fp32 (72); 256 heads of
// 8192 to 4096 in bf16 220 (186), 128 in fp32 213 (180).
constexpr int kMoveRows = 4;                             // rows of a thread and step
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs e, int cols) {
  wait_for_last();
  const int g = blockIdx.x / (2 * cols + 1), part = blockIdx.x % (2 * cols + 1);
  const int n = evict_len(e, g / e.Hk), m = min(n, e.budget);
  const int* idx = e.idx + (int64_t)g * e.So;
  if (part == 2 * cols) {
    float* acc = e.acco + (int64_t)g * e.So;
    for (int j0 = 0; j0 < e.So; j0 += 256 * kMoveRows) {
      float f[kMoveRows];
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const int j = j0 + i * 256 + threadIdx.x;
        f[i] = j < m ? acc[idx[j]] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const int j = j0 + i * 256 + threadIdx.x;
        if (j < e.So) acc[j] = f[i];
      }
      __syncthreads();
    }
    return;
  }
  if (n <= e.budget) return;                             // nothing moves
  const int chunks = e.D * e.elem / 16;
  uint4* x = static_cast<uint4*>(part < cols ? e.ko : e.vo) + (int64_t)g * e.So * chunks +
             part % cols * 4 + threadIdx.x % 4;
  for (int j0 = e.sinks; j0 < m; j0 += 64 * kMoveRows) {
    uint4 t[kMoveRows];
    int from[kMoveRows];
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
      const int j = j0 + i * 64 + threadIdx.x / 4;
      from[i] = j < m ? idx[j] : j;
      if (from[i] != j) t[i] = x[(int64_t)from[i] * chunks];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
      const int j = j0 + i * 64 + threadIdx.x / 4;
      if (from[i] != j) x[(int64_t)j * chunks] = t[i];
    }
    __syncthreads();
  }
}

// Blocks of a cluster: a share of `least` candidates at least, and four blocks to an
// SM at most (256 heads of 8192 tokens: 2 blocks 183 us, 8 blocks 217; 8 heads of
// 40000 to 10000: 8 blocks 31 us, 2 blocks 56; 2048 heads of 500: one block 73, 2 blocks 100).
int evict_cluster(int heads, int S, int least, int most) {
  int cs = 1;
  while (cs < most && S > least * cs && (int64_t)heads * cs * 2 <= 4 * 148) cs *= 2;
  return cs;
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& e, cudaStream_t s) {
  // Short caches: the blocks that choose also copy (2 heads of 600 tokens: 9.1 us, with
  // a launch for the copy 11.6; 2048 heads of 500: 73 and 80).  Long ones: more blocks
  // copy than choose (8 heads of 40000 to 10000: 31 us, in one launch 51; 256 of 8192: 183, 196).
  const int heads = e.B * e.Hk;
  const bool in_place = e.k == e.ko, one = !in_place && e.S <= kTile;
  const int cs = one ? evict_cluster(heads, e.S, 256, 4) : evict_cluster(heads, e.S, 1024, 8);
  cudaError_t st = launch_kernel(one ? evict_kernel<true> : evict_kernel<false>, (int64_t)heads * cs,
                                 kThreads, 0, cs, false, s, e, cs);
  if (st != cudaSuccess || one) return st;
  if (in_place) {
    const int cols = e.D * e.elem / 64;
    return launch_kernel(evict_move_kernel, (int64_t)heads * (2 * cols + 1), 256, 0, 1, true, s, e,
                         cols);
  }
  const int per = kThreads / (e.D * e.elem / 16) * 2;    // rows of a block: two of each thread
  const int nb = (e.budget + per - 1) / per;
  return launch_kernel(evict_copy_kernel, (int64_t)heads * nb, kThreads, 0, 1, true, s, e, nb);
}

}  // namespace area
