// How much weight every key of a cache has received, when a key head has many
// query rows: the scores once more, now with each row's log-sum known.
//
// A block has 128 keys of a key head; the products are taken transposed,
// S^T (128 keys x rows) = K Q^T, so that a thread has one key in its TMEM lane
// and adds up 2^(s - lse) over the columns, in order: no sums across threads,
// no atomics, and the scores never leave the SM (written out they would be
// B H Nq S values: 16 heads' 256 queries on 60000 tokens are 1 GB).
// Few keys: a cluster of blocks shares the rows of 128 keys, and its first block
// adds their sums up in order (2 key heads of 1519 keys, 1024 rows, fp32: the call
// 65 -> 43 us).
// Tiles of rows that end before the block's keys are left out.  Keys that no
// query sees may hold anything: a key's value stays in its own lane, which the
// mask drops.
#include <cooperative_groups.h>

#include "cache.cuh"
#include "cut3.cuh"
#include "tc_common.cuh"

namespace area {
namespace {

struct WParams {
  CacheArgs a;
  const float* lse;        // [B * H * Nq] log2-sums
  const float* acc;        // [B, Hk, S] or null
  float* acco;
  int R;                   // rows of a key head
  int chunks;              // clusters of a key head
  int cs;                  // blocks of a cluster
};

// A tile of KR rows: those of [r0, r0 + n) see keys below hi0 at least and
// below hi1 at most.
struct RowTile {
  int n, hi0, hi1;
};
template <int KR>
__device__ __forceinline__ RowTile row_tile(const CacheArgs& a, int R, int len, int t) {
  const int r0 = t * KR, r1 = min(r0 + KR, R);
  int i0, i1;
  query_range(a, r0, r1, i0, i1);
  return RowTile{r1 - r0, key_span(a, len, i0).hi, key_span(a, len, i1).hi};
}

// Loads a tile's log-sums and ends, thread th's row; rows behind the last end
// at 0.  The group's barrier follows.
template <int KR>
__device__ __forceinline__ void load_rows(const WParams& p, int64_t row0, int len, int t,
                                          float* s_lse, int* s_hi, int th, int bar_id) {
  if (th < KR) {
    const int r = t * KR + th;
    const bool in = r < p.R;
    s_lse[th] = in ? p.lse[row0 + r] : INFINITY;
    s_hi[th] = in ? key_span(p.a, len, r % p.a.Nq).hi : 0;
  }
  asm volatile("bar.sync %0, 128;" ::"r"(bar_id) : "memory");
}

// What a thread, one key of 128, adds up over a tile of scores; the rows'
// log-sums and ends lie in shared memory.
__device__ __forceinline__ float add_tile(const WParams& p, RowTile rt, int j0, uint32_t tS,
                                          const float* s_lse, const int* s_hi, int th) {
  float sum = 0.f;
  const int j = j0 + th;
  const bool masked = rt.hi0 < j0 + 128;
#pragma unroll 1
  for (int c = 0; c < rt.n; c += 32) {
    uint32_t s[32];
    tmem_ld32(tS + c, s);
    if (masked || c + 32 > rt.n) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (j < s_hi[c + i])
          sum += fast_exp2(fmaf(__uint_as_float(s[i]), p.a.scale_log2, -s_lse[c + i]));
    } else {
      float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 z = *reinterpret_cast<const float4*>(&s_lse[c + i]);
        sum += fast_exp2(fmaf(__uint_as_float(s[i]), p.a.scale_log2, -z.x));
        s1 += fast_exp2(fmaf(__uint_as_float(s[i + 1]), p.a.scale_log2, -z.y));
        s2 += fast_exp2(fmaf(__uint_as_float(s[i + 2]), p.a.scale_log2, -z.z));
        s3 += fast_exp2(fmaf(__uint_as_float(s[i + 3]), p.a.scale_log2, -z.w));
      }
      sum += (s1 + s2) + s3;
    }
  }
  return sum;
}
// The cluster's sums, in the ranks' order, for the first block to write: own is this
// block's for thread th's key.
__device__ __forceinline__ void write_sums(const WParams& p, float own, float* s_part, int kvh, int j0,
                                           int th, bool mine) {
  const auto cluster = cooperative_groups::this_cluster();
  const int rank = blockIdx.x % p.cs;
  if (p.cs > 1) {
    if (mine) s_part[th] = own;
    cluster.sync();
  }
  const int j = j0 + th;
  if (mine && rank == 0 && j < p.a.S) {
    for (int r = 1; r < p.cs; ++r) own += *cluster.map_shared_rank(&s_part[th], r);
    const int64_t at = (int64_t)kvh * p.a.S + j;
    p.acco[at] = (p.acc ? p.acc[at] : 0.f) + own;
  }
  if (p.cs > 1) cluster.sync();          // the first block has read the others' sums
}

// ---- bf16: keys and rows by TMA -------------------------------------------
constexpr int kThreads = 384;              // TMA, products, two groups of 128 keys' threads
template <int D>
struct Geo {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kSmemQ = kTileBytes;                     // after the key tile
  static constexpr int kSmemBar = kSmemQ + 2 * kTileBytes;
  static constexpr int kSmemBytes = kSmemBar + 128 + 1024;
};
enum { W_K_FULL = 0, W_Q_FULL, W_Q_EMPTY = W_Q_FULL + 2, W_S_FULL = W_Q_EMPTY + 2,
       W_S_EMPTY = W_S_FULL + 2, W_DRAIN = W_S_EMPTY + 2, W_COUNT };
static_assert(W_COUNT * 8 <= 128, "barrier area");

struct WMaps {
  CUtensorMap q, k;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
cache_weights_tc_kernel(const __grid_constant__ WMaps tm, const __grid_constant__ WParams p) {
  using G = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + G::kSmemBar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ __align__(16) float s_lse[2][128];
  __shared__ int s_hi[2][128];
  __shared__ float s_sum[128], s_part[128];
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x / p.cs, rank = blockIdx.x % p.cs;
  const int kvh = block / p.chunks, j0 = block % p.chunks * 128;
  const int len = cache_len(p.a, kvh / p.a.Hk);
  // this block's row tiles
  const int all = j0 < len ? (p.R + 127) / 128 : 0;
  const int rt0 = all * rank / p.cs, nrt = all * (rank + 1) / p.cs;

  if (threadIdx.x == 0) {
    s_abort = 0;
    mbar_init(bar(W_K_FULL), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(W_Q_FULL + b), 1);
      mbar_init(bar(W_Q_EMPTY + b), 1);
      mbar_init(bar(W_S_FULL + b), 1);
      mbar_init(bar(W_S_EMPTY + b), 128);
    }
    mbar_init(bar(W_DRAIN), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_last();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(
                     smem_u32(&s_tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  int* abort_flag = &s_abort;
  float sum = 0.f;

  if (warp == 0) {
    if (lane == 0 && nrt > rt0) {
      uint32_t it = 0;
      mbar_arrive_tx(bar(W_K_FULL), G::kTileBytes);
      for (int hf = 0; hf < G::kHalves; ++hf)
        tma_load_3d(sbase + hf * kHalfBytes, &tm.k, bar(W_K_FULL), hf * 64, j0, kvh);
      for (int t = rt0; t < nrt; ++t) {
        if (row_tile<128>(p.a, p.R, len, t).hi1 <= j0) continue;
        const uint32_t b = it & 1u;
        if (!mbar_wait(bar(W_Q_EMPTY + b), ((it >> 1) & 1u) ^ 1u, abort_flag)) break;
        mbar_arrive_tx(bar(W_Q_FULL + b), G::kTileBytes);
        for (int hf = 0; hf < G::kHalves; ++hf)
          tma_load_3d(sbase + G::kSmemQ + b * G::kTileBytes + hf * kHalfBytes, &tm.q,
                      bar(W_Q_FULL + b), hf * 64, t * 128, kvh);
        ++it;
      }
      // no copy is in flight when the block ends
      int drain_abort = 0;
      mbar_wait(bar(W_K_FULL), 0, &drain_abort);
      for (uint32_t x = it > 2 ? it - 2 : 0; x < it; ++x)
        mbar_wait(bar(W_Q_FULL + (x & 1u)), (x >> 1) & 1u, &drain_abort);
    }
  } else if (warp == 1) {
    {
      uint32_t it = 0;
      const uint64_t dk = sdesc(sbase, 16, 1024), dq = sdesc(sbase + G::kSmemQ, 16, 1024);
      bool ok = nrt == rt0 || warp_wait_all(bar(W_K_FULL), 0, abort_flag);
      for (int t = rt0; t < nrt && ok; ++t) {
        if (row_tile<128>(p.a, p.R, len, t).hi1 <= j0) continue;
        const uint32_t b = it & 1u, ph = (it >> 1) & 1u;
        if (!(ok = warp_wait_all(bar(W_Q_FULL + b), ph, abort_flag))) break;
        if (!(ok = warp_wait_all(bar(W_S_EMPTY + b), ph ^ 1u, abort_flag))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
            mma_ss(tmem + b * 128, sdesc_at(dk, off), sdesc_at(dq, b * G::kTileBytes + off),
                     kIdescQK, kk > 0);
          }
          mma_commit(bar(W_S_FULL + b));
          mma_commit(bar(W_Q_EMPTY + b));
        }
        __syncwarp();
        ++it;
      }
      int drain_abort = 0;
      if (elect_one()) mma_commit(bar(W_DRAIN));
      __syncwarp();
      warp_wait_all(bar(W_DRAIN), 0, &drain_abort);
    }
  } else if (warp >= 4) {
    // group grp takes every second tile
    const uint32_t grp = (uint32_t)(warp - 4) >> 2;
    const int th = ((warp & 3) << 5) + lane;         // TMEM lane = key of the block
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) << 5) << 16) + grp * 128;
    const int64_t row0 = (int64_t)kvh * p.R;
    uint32_t it = 0;
    for (int t = rt0; t < nrt; ++t) {
      const RowTile rt = row_tile<128>(p.a, p.R, len, t);
      if (rt.hi1 <= j0) continue;
      const uint32_t ph = (it >> 1) & 1u;
      if ((it++ & 1u) != grp) continue;
      load_rows<128>(p, row0, len, t, s_lse[grp], s_hi[grp], th, 1 + (int)grp);
      const bool ok = warp_wait_all(bar(W_S_FULL + grp), ph, abort_flag);
      tc_fence_after();
      // (an expired wait still takes part in the group's barriers)
      if (ok)
        sum += add_tile(p, rt, j0, tS, s_lse[grp], s_hi[grp], th);
      tc_fence_before();
      mbar_arrive(bar(W_S_EMPTY + grp));
      asm volatile("bar.sync %0, 128;" ::"r"(1 + (int)grp) : "memory");
    }
    if (grp == 1) s_sum[th] = sum;
  }
  tc_fence_before();
  __syncthreads();
  {
    const bool mine = warp >= 4 && warp < 8;
    const int th = mine ? threadIdx.x - 128 : 0;
    write_sums(p, mine ? sum + s_sum[th] : 0.f, s_part, kvh, j0, th, mine);
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem) : "memory");
  }
}

// ---- fp32: keys and rows cut into three bf16 parts, six products ------------
constexpr int kKR32 = 64;                  // rows of a tile
template <int D>
struct Geo32 {
  static constexpr int kHalves = D / 64;
  static constexpr int kKHalf = 128 * 128, kQHalf = kKR32 * 128;   // bytes of 64 columns
  static constexpr int kKTerm = kHalves * kKHalf, kQTerm = kHalves * kQHalf;
  static constexpr int kSmemQ = 3 * kKTerm;
  static constexpr int kSmemBar = kSmemQ + 2 * 3 * kQTerm;
  static constexpr int kSmemBytes = kSmemBar + 128 + 1024;
  static_assert(kSmemBytes + 2048 <= 227 * 1024, "shared memory of one CTA");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_weights_tc32_kernel(const __grid_constant__ WParams p) {
  using G = Geo32<D>;
  constexpr int kChunks = D / 8, kPer = kKR32 * kChunks / 128, kRowStep = 128 / kChunks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + G::kSmemBar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ __align__(16) float s_lse[kKR32];
  __shared__ int s_hi[kKR32];
  __shared__ float s_part[128];
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x / p.cs, rank = blockIdx.x % p.cs;
  const int kvh = block / p.chunks, j0 = block % p.chunks * 128;
  const int len = cache_len(p.a, kvh / p.a.Hk);
  const int all = j0 < len ? (p.R + kKR32 - 1) / kKR32 : 0;
  const int rt0 = all * rank / p.cs, nrt = all * (rank + 1) / p.cs;

  if (threadIdx.x == 0) {
    s_abort = 0;
    mbar_init(bar(W_K_FULL), 128);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(W_Q_FULL + b), 128);
      mbar_init(bar(W_Q_EMPTY + b), 1);
      mbar_init(bar(W_S_FULL + b), 1);
      mbar_init(bar(W_S_EMPTY + b), 128);
    }
    mbar_init(bar(W_DRAIN), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_last();
  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(
                     smem_u32(&s_tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  int* abort_flag = &s_abort;
  float sum = 0.f;

  if (warp < 4) {
    if (nrt > rt0) {
      const int tid = threadIdx.x, ch = tid % kChunks, row0 = tid / kChunks;
      // 64 rows of a tensor from base on, n of them there, into registers and on
      // into an operand tile at `at`
      float f[kPer][8];
      auto load = [&](const float* base, int n) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = row0 + i * kRowStep;
          get8(base + (int64_t)r * D + ch * 8, r < n, f[i]);
        }
      };
      auto put = [&](uint32_t at, int half, int term) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = row0 + i * kRowStep;
          put8(at + (ch >> 3) * half + r * 128 + (((ch & 7) ^ (r & 7)) << 4), term, f[i]);
        }
        fence_proxy_async();
      };
      const float* kb = static_cast<const float*>(p.a.k) + ((int64_t)kvh * p.a.S + j0) * D;
      const float* qb = static_cast<const float*>(p.a.q) + (int64_t)kvh * p.R * D;
      const int nk = min(128, len - j0);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        load(kb + (int64_t)h * 64 * D, nk - h * 64);
        put(sbase + h * 64 * 128, G::kKHalf, G::kKTerm);
      }
      mbar_arrive(bar(W_K_FULL));
      uint32_t it = 0;
      for (int t = rt0; t < nrt; ++t) {
        const RowTile rt = row_tile<kKR32>(p.a, p.R, len, t);
        if (rt.hi1 <= j0) continue;
        const uint32_t b = it & 1u;
        load(qb + (int64_t)t * kKR32 * D, rt.n);
        if (!warp_wait_all(bar(W_Q_EMPTY + b), ((it >> 1) & 1u) ^ 1u, abort_flag)) break;
        put(sbase + G::kSmemQ + b * 3 * G::kQTerm, G::kQHalf, G::kQTerm);
        mbar_arrive(bar(W_Q_FULL + b));
        ++it;
      }
    }
  } else if (warp == 4) {
    {
      uint32_t it = 0;
      const uint64_t dk = sdesc(sbase, 16, 1024), dq = sdesc(sbase + G::kSmemQ, 16, 1024);
      bool ok = nrt == rt0 || warp_wait_all(bar(W_K_FULL), 0, abort_flag);
      for (int t = rt0; t < nrt && ok; ++t) {
        if (row_tile<kKR32>(p.a, p.R, len, t).hi1 <= j0) continue;
        const uint32_t b = it & 1u, ph = (it >> 1) & 1u;
        if (!(ok = warp_wait_all(bar(W_Q_FULL + b), ph, abort_flag))) break;
        if (!(ok = warp_wait_all(bar(W_S_EMPTY + b), ph ^ 1u, abort_flag))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < 6; ++x) {
            const uint32_t ks = part_a(x) * G::kKTerm, qs = (b * 3 + part_b(x)) * G::kQTerm;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + b * kKR32, sdesc_at(dk, ks + (kk >> 2) * G::kKHalf + (kk & 3) * 32),
                       sdesc_at(dq, qs + (kk >> 2) * G::kQHalf + (kk & 3) * 32), idesc(kKR32, false),
                       (x > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar(W_S_FULL + b));
          mma_commit(bar(W_Q_EMPTY + b));
        }
        __syncwarp();
        ++it;
      }
      int drain_abort = 0;
      if (elect_one()) mma_commit(bar(W_DRAIN));
      __syncwarp();
      warp_wait_all(bar(W_DRAIN), 0, &drain_abort);
    }
  } else if (warp >= 8) {
    const int th = ((warp & 3) << 5) + lane;         // TMEM lane = key of the block
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) << 5) << 16);
    const int64_t row0 = (int64_t)kvh * p.R;
    uint32_t it = 0;
    for (int t = rt0; t < nrt; ++t) {
      const RowTile rt = row_tile<kKR32>(p.a, p.R, len, t);
      if (rt.hi1 <= j0) continue;
      const uint32_t b = it & 1u, ph = (it >> 1) & 1u;
      ++it;
      load_rows<kKR32>(p, row0, len, t, s_lse, s_hi, th, 1);
      const bool ok = warp_wait_all(bar(W_S_FULL + b), ph, abort_flag);
      tc_fence_after();
      if (ok) sum += add_tile(p, rt, j0, tS + b * kKR32, s_lse, s_hi, th);
      tc_fence_before();
      mbar_arrive(bar(W_S_EMPTY + b));
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  {
    const bool mine = warp >= 8;
    write_sums(p, sum, s_part, kvh, j0, mine ? (int)threadIdx.x - 256 : 0, mine);
  }
  if (warp == 4) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
  }
}

template <int D>
cudaError_t launch_bf16(const WParams& p, int64_t grid, cudaStream_t s) {
  const CacheArgs& a = p.a;
  WMaps m;
  cudaError_t e = make_map3(&m.q, a.q, (int64_t)a.B * a.Hk, p.R, D, 128, 1);
  if (e == cudaSuccess) e = make_map3(&m.k, a.k, (int64_t)a.B * a.Hk, a.S, D, 128, 1);
  if (e != cudaSuccess) return e;
  auto fn = cache_weights_tc_kernel<D>;
  constexpr int kSmem = Geo<D>::kSmemBytes;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(fn, grid * p.cs, kThreads, kSmem, p.cs, true, s, m, p);
}
template <int D>
cudaError_t launch_f32(const WParams& p, int64_t grid, cudaStream_t s) {
  auto fn = cache_weights_tc32_kernel<D>;
  constexpr int kSmem = Geo32<D>::kSmemBytes;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(fn, grid * p.cs, kThreads, kSmem, p.cs, true, s, p);
}

}  // namespace

cudaError_t read_and_clear_cache_weights_error(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(code, g_tc_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_tc_error, &zero, sizeof(int));
}

cudaError_t launch_cache_weights_tc(const CacheArgs& a, const float* lse, const float* acc,
                                    float* acco, int dtype, cudaStream_t s) {
  WParams p{a, lse, acc, acco, a.H / a.Hk * a.Nq, (a.S + 127) / 128, 1};
  const int64_t grid = (int64_t)a.B * a.Hk * p.chunks;
  // as many blocks as run at once, two row tiles to a block
  const int tile = dtype == AREA_DTYPE_BF16 ? 128 : kKR32;
  const int64_t most = dtype == AREA_DTYPE_BF16 ? 2 * num_sms() : num_sms();
  while (p.cs < 8 && grid * p.cs * 2 <= most && p.R >= 4 * p.cs * tile) p.cs *= 2;
  if (dtype == AREA_DTYPE_BF16)
    return a.D == 64 ? launch_bf16<64>(p, grid, s) : launch_bf16<128>(p, grid, s);
  return a.D == 64 ? launch_f32<64>(p, grid, s) : launch_f32<128>(p, grid, s);
}

}  // namespace area
