// Joining the splits of an attention over a key/value cache, and adding up
// the weights of its keys.
#include "cache.cuh"

namespace area {
namespace {

// One block of four warps per row.  The row's output is
//   sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s,   m = max_s m_s;
// the warps take the slots in turn and add up in shared memory in a fixed
// order.  A slot without a key has l = 0 and its output is not read.
template <typename T, int D>
__global__ void __launch_bounds__(128) cache_join_kernel(const float* __restrict__ part_o,
                                                         const float2* __restrict__ part_ml,
                                                         int slots, int64_t rows, T* o,
                                                         float* lse) {
  constexpr int kPer = D / 32;
  __shared__ float s_o[4][D], s_l[4];
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int s = lane; s < slots; s += 32) m = fmaxf(m, part_ml[s * rows + row].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ref = m == -INFINITY ? 0.f : m;
  float acc[kPer] = {}, l = 0.f;
  for (int s = warp; s < slots; s += 4) {
    const float2 ml = part_ml[s * rows + row];
    if (ml.y == 0.f) continue;
    const float w = exp2f(ml.x - ref);
    l += w * ml.y;
    const float* src = part_o + (s * rows + row) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, src[i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_o[warp][lane * kPer + i] = acc[i];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  const float total = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  for (int d = threadIdx.x; d < D; d += 128) {
    const float v = (s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d]);
    store_from_float(o, row * D + d, total == 0.f ? 0.f : v / total);
  }
  // a row without a weight: +inf, so that 2^(x - lse) is 0 for every key
  if (lse && threadIdx.x == 0) lse[row] = total == 0.f ? INFINITY : ref + log2f(total);
}

// kWKeys keys of a key head to a thread, a block apart; a key's rows' weights
// are added in order.
constexpr int kWThreads = 128, kWKeys = 4;
__global__ void __launch_bounds__(kWThreads) cache_weights_kernel(const CacheArgs a,
                                                                  const float* __restrict__ logits,
                                                                  const float* __restrict__ lse,
                                                                  const float* acc, float* acco,
                                                                  int chunks) {
  const int kvh = blockIdx.x / chunks;                       // (b, key head)
  const int j0 = blockIdx.x % chunks * (kWThreads * kWKeys) + threadIdx.x;
  const int len = cache_len(a, kvh / a.Hk);
  const int R = a.H / a.Hk * a.Nq;
  const int64_t row0 = (int64_t)kvh * R, at = (int64_t)kvh * a.S;
  float sum[kWKeys] = {}, old[kWKeys];
#pragma unroll
  for (int x = 0; x < kWKeys; ++x) {
    const int j = j0 + x * kWThreads;
    old[x] = acc && j < a.S ? acc[at + j] : 0.f;
  }
  int i = 0;
#pragma unroll 4
  for (int r = 0; r < R; ++r) {
    const int end = len - a.Nq + 1 + i;                      // the row sees keys below it
    const float z = lse[row0 + r];
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

}  // namespace

cudaError_t launch_cache_join(const CacheArgs& a, const float* part_o, const float2* part_ml,
                              int slots, int64_t rows, float* lse, int dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)rows;
  if (dtype == AREA_DTYPE_F32) {
    float* o = static_cast<float*>(a.o);
    if (a.D == 64) cache_join_kernel<float, 64><<<grid, 128, 0, s>>>(part_o, part_ml, slots, rows, o, lse);
    else cache_join_kernel<float, 128><<<grid, 128, 0, s>>>(part_o, part_ml, slots, rows, o, lse);
  } else {
    auto* o = static_cast<__nv_bfloat16*>(a.o);
    if (a.D == 64) cache_join_kernel<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(part_o, part_ml, slots, rows, o, lse);
    else cache_join_kernel<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(part_o, part_ml, slots, rows, o, lse);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_weights(const CacheArgs& a, const float* logits, const float* lse,
                                 const float* acc, float* acco, cudaStream_t s) {
  const int per = kWThreads * kWKeys, chunks = (a.S + per - 1) / per;
  cache_weights_kernel<<<(unsigned)((int64_t)a.B * a.Hk * chunks), kWThreads, 0, s>>>(
      a, logits, lse, acc, acco, chunks);
  return cudaGetLastError();
}

}  // namespace area
