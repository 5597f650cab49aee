// Joining the splits of an attention over a key/value cache, and adding up
// the weights of its keys.
#include "cache.cuh"

namespace area {
namespace {

// The row's output is
//   sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s,   m = max_s m_s.
// WARPS warps to a row take the slots in turn, four at once, and add up in shared
// memory in a fixed order; a block of NW warps has NW / WARPS rows, from row0 on.  A slot without a key has l = 0 and its output, which nobody wrote,
// counts as zeros.  A row without a weight has a log-sum of +inf, so that
// 2^(x - lse) is 0 for every key.  (No __restrict__: nothing may be read before
// wait_for_last.)
template <typename T, int D, int WARPS, int NW>
__device__ __forceinline__ void join_rows(const float* part_o,
                                         const float2* part_ml, int slots,
                                         int64_t rows, int64_t row0, T* o, float* lse) {
  constexpr int kPer = D / 32;                             // columns of a lane
  __shared__ float s_o[WARPS > 1 ? NW : 1][D], s_l[NW];
  const int wid = threadIdx.x >> 5, warp = wid % WARPS, lane = threadIdx.x & 31;
  const int64_t mine = row0 + wid / WARPS;
  const int64_t row = mine < rows ? mine : rows - 1;       // behind the last: not written
  float m = -INFINITY;
  for (int s = lane; s < slots; s += 32) m = fmaxf(m, part_ml[s * rows + row].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == -INFINITY ? 0.f : m;
  float acc[kPer] = {}, l = 0.f;
  for (int s0 = warp; s0 < slots; s0 += 4 * WARPS) {
    float x[4][kPer];
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + i * WARPS;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[i][j] = 0.f;
      if (s >= slots) continue;
      ml[i] = part_ml[s * rows + row];
      const float* src = part_o + (s * rows + row) * D + lane * kPer;
      if constexpr (kPer == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        x[i][0] = f.x, x[i][1] = f.y, x[i][2] = f.z, x[i][3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        x[i][0] = f.x, x[i][1] = f.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool any = ml[i].y != 0.f;
      const float w = any ? exp2f(ml[i].x - ref) : 0.f;
      l = fmaf(w, ml[i].y, l);
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] = fmaf(w, any ? x[i][j] : 0.f, acc[j]);
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s_o[wid][lane * kPer + j] = acc[j];
    if (lane == 0) s_l[wid] = l;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      l += s_l[wid + w];
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] += s_o[wid + w][lane * kPer + j];
    }
  }
  if (mine >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int j = 0; j < kPer; ++j) acc[j] = l == 0.f ? 0.f : acc[j] * inv;
  T* dst = o + row * D + lane * kPer;
  if constexpr (sizeof(T) == 4) {
    if constexpr (kPer == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else
      *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; j += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + j) = __floats2bfloat162_rn(acc[j], acc[j + 1]);
  }
  if (lse && lane == 0) lse[row] = l == 0.f ? INFINITY : ref + log2f(l);
}

constexpr int kJoinWarps = 8;
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(kJoinWarps * 32)
cache_join_kernel(const float* part_o, const float2* part_ml, int slots,
                  int64_t rows, T* o, float* lse) {
  wait_for_last();
  join_rows<T, D, WARPS, kJoinWarps>(part_o, part_ml, slots, rows,
                                     (int64_t)blockIdx.x * (kJoinWarps / WARPS), o, lse);
}

// The join for few rows of a key head, and the weights of its keys from the scores:
// a grid's first blocks join a row each; the others have kWKeys keys of a key head
// to a thread, a block apart, work out the rows' log-sums for themselves and add a
// key's weights in the rows' order.  One launch instead of two, neither of which
// fills the GPU (32 sequences of 8192 tokens, 8 key heads of 4 rows: 144 us in all,
// with two launches 150).
constexpr int kWThreads = 128, kWKeys = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kWThreads)
cache_join_weights_kernel(const CacheArgs a, const float* part_o,
                          const float2* part_ml, int slots, int64_t rows,
                          const float* logits, const float* acc, float* acco,
                          int chunks) {
  wait_for_last();
  if (blockIdx.x < rows) {
    join_rows<T, D, kWThreads / 32, kWThreads / 32>(part_o, part_ml, slots, rows, blockIdx.x,
                                                    static_cast<T*>(a.o), nullptr);
    return;
  }
  __shared__ float s_lse[kCacheFewWeights];
  const int block = (int)(blockIdx.x - rows);
  const int kvh = block / chunks;                            // (b, key head)
  const int j0 = block % chunks * (kWThreads * kWKeys) + threadIdx.x;
  const int len = cache_len(a, kvh / a.Hk);
  const int R = a.H / a.Hk * a.Nq;
  const int64_t row0 = (int64_t)kvh * R, at = (int64_t)kvh * a.S;
  float sum[kWKeys] = {}, old[kWKeys];
#pragma unroll
  for (int x = 0; x < kWKeys; ++x) {
    const int j = j0 + x * kWThreads;
    old[x] = acc && j < a.S ? acc[at + j] : 0.f;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < R; r += kWThreads / 32) {
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < slots; s += 32) m = fmaxf(m, part_ml[s * rows + row0 + r].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int s = lane; s < slots; s += 32) {
      const float2 ml = part_ml[s * rows + row0 + r];
      if (ml.y != 0.f) l = fmaf(exp2f(ml.x - ref), ml.y, l);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (lane == 0) s_lse[r] = l == 0.f ? INFINITY : ref + log2f(l);
  }
  __syncthreads();
  int i = 0;
#pragma unroll 4
  for (int r = 0; r < R; ++r) {
    const int end = len - a.Nq + 1 + i;                      // the row sees keys below it
    const float z = s_lse[r];
    const float* src = logits + (row0 + r) * a.S + j0;
#pragma unroll
    for (int x = 0; x < kWKeys; ++x)
      if (j0 + x * kWThreads < end) sum[x] += exp2f(src[x * kWThreads] - z);
    if (++i == a.Nq) i = 0;
  }
#pragma unroll
  for (int x = 0; x < kWKeys; ++x) {
    const int j = j0 + x * kWThreads;
    if (j < a.S) acco[at + j] = old[x] + sum[x];
  }
}

template <typename T, int D>
cudaError_t join(const CacheArgs& a, const float* part_o, const float2* part_ml, int slots,
                 int64_t rows, float* lse, cudaStream_t s) {
  // four slots to a warp (calls with 6144 rows of 6: 41.6 us, with eight warps to a row 48;
  // 128 rows of 7: 92.7, with one warp 100)
  auto launch = [&](auto fn, int warps) {
    const int64_t per = kJoinWarps / warps;
    return launch_kernel(fn, (rows + per - 1) / per, kJoinWarps * 32, 0, 1, true, s, part_o, part_ml,
                         slots, rows, static_cast<T*>(a.o), lse);
  };
  const int w = slots <= 4 ? 1 : slots <= 8 ? 2 : slots <= 16 ? 4 : 8;
  if (w == 1) return launch(cache_join_kernel<T, D, 1>, 1);
  if (w == 2) return launch(cache_join_kernel<T, D, 2>, 2);
  if (w == 4) return launch(cache_join_kernel<T, D, 4>, 4);
  return launch(cache_join_kernel<T, D, 8>, 8);
}

}  // namespace

cudaError_t launch_cache_join(const CacheArgs& a, const float* part_o, const float2* part_ml,
                              int slots, int64_t rows, float* lse, int dtype, cudaStream_t s) {
  auto fn = dtype == AREA_DTYPE_F32 ? (a.D == 64 ? join<float, 64> : join<float, 128>)
                                    : (a.D == 64 ? join<__nv_bfloat16, 64> : join<__nv_bfloat16, 128>);
  return fn(a, part_o, part_ml, slots, rows, lse, s);
}

cudaError_t launch_cache_join_weights(const CacheArgs& a, const CacheOut& out, int slots, int dtype,
                                      cudaStream_t s) {
  if (a.H / a.Hk * a.Nq > kCacheFewWeights) return cudaErrorInvalidValue;
  const int per = kWThreads * kWKeys, chunks = (a.S + per - 1) / per;
  auto fn = dtype == AREA_DTYPE_F32
                ? (a.D == 64 ? cache_join_weights_kernel<float, 64> : cache_join_weights_kernel<float, 128>)
                : (a.D == 64 ? cache_join_weights_kernel<__nv_bfloat16, 64>
                             : cache_join_weights_kernel<__nv_bfloat16, 128>);
  return launch_kernel(fn, out.rows + (int64_t)a.B * a.Hk * chunks, kWThreads, 0, 1, true, s, a,
                       out.part_o, out.part_ml, slots, out.rows, out.logits, out.acc, out.acco,
                       chunks);
}

}  // namespace area
