// Eviction from a key/value cache by accumulated attention weight.
//
// Of a sequence of n > budget tokens each key head keeps the first `sinks`,
// the last `recent` and, of the tokens between, the budget - sinks - recent
// with the largest accumulated weight (ties: the lowest index), in their
// order.  Two launches: the choice, which leaves the kept tokens' indexes, and
// the copy of their rows.
#include "cache.cuh"

namespace area {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

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

// One block per (sequence, key head).  Radix selection of the smallest kept
// key from the top byte down, then one ordered pass that writes the indexes.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs e) {
  __shared__ int s_hist[256];
  __shared__ int s_bin, s_above;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  const int g = blockIdx.x, b = g / e.Hk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = evict_len(e, b);
  int* idx = e.idx + (int64_t)g * e.So;
  const int kept = min(n, e.budget);
  if (g % e.Hk == 0 && tid == 0) e.lenso[b] = kept;
  for (int j = kept + tid; j < e.So; j += kSelThreads) idx[j] = -1;
  if (n <= e.budget) {
    for (int j = tid; j < n; j += kSelThreads) idx[j] = j;
    return;
  }
  const float* acc = e.acc + (int64_t)g * e.S + e.sinks;
  const int cand = n - e.sinks - e.recent;               // tokens to choose from
  const int want = e.budget - e.sinks - e.recent;        // < cand
  for (int j = tid; j < e.sinks; j += kSelThreads) idx[j] = j;
  for (int j = tid; j < e.recent; j += kSelThreads) idx[e.sinks + want + j] = n - e.recent + j;
  if (want == 0) return;

  uint32_t prefix = 0;           // the bytes of the threshold found so far
  int left = want;               // kept keys among those that share them
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < cand; j += kSelThreads) {
      const uint32_t key = weight_key(acc[j]);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&s_hist[key >> shift & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane 0 holds the eight highest bins; `before` = keys in higher lanes' bins
      int h[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += h[i] = s_hist[255 - (lane * 8 + i)];
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
    prefix |= (uint32_t)s_bin << shift;
    left -= s_above;
    __syncthreads();
  }
  // keys above the threshold are kept, and the first `left` of those equal to it
  int gt0 = 0, eq0 = 0;          // found in earlier tiles
  for (int j0 = 0; j0 < cand; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t key = j < cand ? weight_key(acc[j]) : 0;
    const unsigned gt = __ballot_sync(0xffffffffu, j < cand && key > prefix);
    const unsigned eq = __ballot_sync(0xffffffffu, j < cand && key == prefix);
    if (lane == 0) {
      s_gt[warp] = __popc(gt);
      s_eq[warp] = __popc(eq);
    }
    __syncthreads();
    int gtb = gt0, eqb = eq0;
    for (int w = 0; w < kSelWarps; ++w) {
      const int x = s_gt[w], y = s_eq[w];
      if (w < warp) {
        gtb += x;
        eqb += y;
      }
      gt0 += x;
      eq0 += y;
    }
    const unsigned below = (1u << lane) - 1;
    gtb += __popc(gt & below);
    eqb += __popc(eq & below);
    const bool mine_eq = eq >> lane & 1;
    if ((gt >> lane & 1) || (mine_eq && eqb < left))
      idx[e.sinks + gtb + min(eqb, left)] = e.sinks + j;
    __syncthreads();
  }
}

// Copies the kept rows: 16 bytes of K and of V per thread and step.
__global__ void __launch_bounds__(256) evict_copy_kernel(const EvictArgs e, int blocks_per_head) {
  const int g = blockIdx.x / blocks_per_head, blk = blockIdx.x % blocks_per_head;
  const int m = min(evict_len(e, g / e.Hk), e.budget);
  const int* idx = e.idx + (int64_t)g * e.So;
  const int chunks = e.D * e.elem / 16;                  // 16-byte pieces of a row
  const int64_t src0 = (int64_t)g * e.S * chunks, dst0 = (int64_t)g * e.So * chunks;
  const uint4 *k = static_cast<const uint4*>(e.k), *v = static_cast<const uint4*>(e.v);
  uint4 *ko = static_cast<uint4*>(e.ko), *vo = static_cast<uint4*>(e.vo);
  const int per = 256 / chunks;                          // rows of a step
  const int c = threadIdx.x % chunks;
  for (int j = blk * per + threadIdx.x / chunks; j < m; j += blocks_per_head * per) {
    const int64_t src = src0 + (int64_t)idx[j] * chunks + c, dst = dst0 + (int64_t)j * chunks + c;
    const uint4 x = k[src], y = v[src];
    ko[dst] = x;
    vo[dst] = y;
  }
  for (int j = blk * 256 + threadIdx.x; j < e.So; j += blocks_per_head * 256)
    e.acco[(int64_t)g * e.So + j] = j < m ? e.acc[(int64_t)g * e.S + idx[j]] : 0.f;
}

// The copy within the cache itself.  A kept row moves to an index not above
// its own, so a block that moves rows in ascending order, all of a step read
// before any is written, never writes a row that is still to be read.  A block
// has one 64-byte column of K or V, or the weights, of a key head.
constexpr int kMoveRows = 4;                             // rows of a thread and step
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs e, int cols) {
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

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& e, cudaStream_t s) {
  const int heads = e.B * e.Hk;
  evict_select_kernel<<<(unsigned)heads, kSelThreads, 0, s>>>(e);
  cudaError_t st = cudaGetLastError();
  if (st != cudaSuccess) return st;
  const int chunks = e.D * e.elem / 16;
  if (e.k == e.ko) {
    const int cols = chunks / 4;
    evict_move_kernel<<<(unsigned)(heads * (2 * cols + 1)), 256, 0, s>>>(e, cols);
  } else {
    const int per = 256 / chunks * 8;                    // rows of a block: eight steps
    const int nb = (e.budget + per - 1) / per;
    evict_copy_kernel<<<(unsigned)((int64_t)heads * nb), 256, 0, s>>>(e, nb);
  }
  return cudaGetLastError();
}

}  // namespace area
