// Attention over a key/value cache for few query rows (fp32): one pass over
// the keys on the CUDA cores.
//
// A block has ROWS rows of a group and four warps (eight where the blocks do not
// fill the GPU), which take the keys 16 at a time in turn, straight from global memory into registers:
//   scores  eight lanes to a key and four keys to a lane: a lane multiplies
//           its 16-byte pieces of the keys with those of the rows (shared
//           memory, one broadcast read per piece and four keys), and the
//           eight lanes' sums are exchanged by halves, so that each lane ends
//           with ROWS / 2 whole scores;
//   values  D / 32 columns to a lane: every key's weights come back through
//           shared memory and meet the lane's piece of the value row.
// A buffer is loaded again as soon as it has been used, so that a warp keeps 16
// keys and values in flight (16 KB at D = 128).  As in the bf16 kernel one
// reference per row serves until a score exceeds it by more than 2^8.
// Eight rows take about 1000 fp32 instructions per 16 keys and warp, less time
// than the keys need to arrive; 32-bit inputs leave no narrower products.
#include "cache_dec.cuh"

namespace area {
namespace {

constexpr int kStep = 16;                    // keys of a warp and step
constexpr float kSlack = 8.f;                // log2 units

// Keys and values are read once: they need no place in L1.
__device__ __forceinline__ float4 load16(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}
template <int W>
__device__ __forceinline__ void load_cols(const float* p, float (&f)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                 : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.v2.f32 {%0, %1}, [%2];"
                 : "=f"(f[0]), "=f"(f[1])
                 : "l"(p));
}

// Adds up v[0 .. N) over the lanes that differ in bits BIT, BIT / 2, ..., 1:
// afterwards v[0 .. N / (2 BIT)) are the sums of the lane's part.
template <int N, int BIT>
__device__ __forceinline__ void reduce_halves(float* v, int lane) {
  const bool up = lane & BIT;
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    const float keep = up ? v[k + N / 2] : v[k], give = up ? v[k] : v[k + N / 2];
    v[k] = keep + __shfl_xor_sync(0xffffffffu, give, BIT);
  }
  if constexpr (BIT > 1) reduce_halves<N / 2, BIT / 2>(v, lane);
}

template <int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 1 : 2)
cache_dec32_kernel(const CacheArgs a, const CacheRows rm, const CacheOut out, int nrb) {
  constexpr int kTile = WARPS * kStep;       // keys of a block and step
  constexpr int kU = D / 32;                 // 16-byte pieces of a lane per key
  constexpr int kW = D / 32;                 // value columns of a lane
  constexpr int kOwn = ROWS / 2;             // scores of a lane after the exchange
  __shared__ DecSmem<D, ROWS, WARPS> sm;
  __shared__ __align__(16) float s_q[ROWS][D], s_p[WARPS][kStep][ROWS];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 3, c = lane & 7;   // keys 4 grp .. + 3 of a step
  const int sp = blockIdx.x % out.nsplit;
  const int rb = blockIdx.x / out.nsplit % nrb;
  let_next_start();
  const int g = dec_group(a, rm, blockIdx.x / out.nsplit / nrb);
  const int r0 = rb * ROWS, r1 = min(r0 + ROWS, rm.RG);
  const int kvh = rm.pool_rows ? 0 : g / rm.kv_div;           // (b, key head)
  const KeyList kl = key_list(a, rm, rm.pool_rows ? 0 : kvh / a.Hk, r0, r1);
  const float* kb = static_cast<const float*>(a.k) + (int64_t)kvh * a.S * D;
  const float* vb = static_cast<const float*>(a.v) + (int64_t)kvh * a.S * D;
  const int64_t pbase = (int64_t)(rm.pool_rows ? g : kvh % a.Hk) * a.P * D;
  const float* kpb = static_cast<const float*>(a.kp) + pbase;
  const float* vpb = static_cast<const float*>(a.vp) + pbase;

  // this split's tiles of kTile keys
  const int ntile = (kl.total + kTile - 1) / kTile;
  const int t0 = (int)((int64_t)ntile * sp / out.nsplit);
  const int t1 = (int)((int64_t)ntile * (sp + 1) / out.nsplit);
  const int uend = min(t1 * kTile, kl.total);
  int u0 = t0 * kTile + warp * kStep;

  // the base address of key u of the list (past its end: the last key's, whose
  // weight is zero there)
  auto key_at = [&](int u, const float* own, const float* pre) {
    u = min(u, kl.total - 1);
    if (u < kl.np) return pre + (int64_t)u * D;
    const int w = u - kl.np;
    return own + (int64_t)(w < kl.ns ? w : kl.lo + (w - kl.ns)) * D;
  };
  float4 kf[4][kU];
  float vf[kStep][kW];
  auto load_k = [&](int u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* p = key_at(u + grp * 4 + i, kb, kpb) + 4 * c;
#pragma unroll
      for (int x = 0; x < kU; ++x) kf[i][x] = load16(p + 32 * x);
    }
  };
  auto load_v = [&](int u) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) load_cols<kW>(key_at(u + i, vb, vpb) + kW * lane, vf[i]);
  };
  if (u0 < uend) {
    load_k(u0);
    load_v(u0);
  }
  dec_rows(sm, a, rm, g, r0);
  for (int e = threadIdx.x; e < ROWS * (D / 4); e += WARPS * 32) {
    const int r = e / (D / 4), d = e % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sm.row[r] >= 0)
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + sm.row[r] * D + d);
    const float sc = a.scale_log2;
    *reinterpret_cast<float4*>(&s_q[r][d]) = make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
  }
  __syncthreads();

  // after the exchange a lane holds scores own = c * kOwn .. of row own / 4,
  // key own % 4 of its four
  const int row = c * kOwn / 4, key0 = c * kOwn % 4;
  const KeySpan span = sm.span[row];
  const bool valid = sm.row[row] >= 0, pre = valid && sees_prefix(a, span);
  float* const score = out.logits && valid ? out.logits + sm.row[row] * a.S : nullptr;
  float o[ROWS][kW], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int x = 0; x < kW; ++x) o[r][x] = 0.f;

  for (; u0 < uend; u0 += kTile) {
    float s[ROWS * 4];
#pragma unroll
    for (int i = 0; i < ROWS * 4; ++i) s[i] = 0.f;
#pragma unroll
    for (int x = 0; x < kU; ++x)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(&s_q[r][32 * x + 4 * c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& t = s[r * 4 + i];
          t = fmaf(q.x, kf[i][x].x, t);
          t = fmaf(q.y, kf[i][x].y, t);
          t = fmaf(q.z, kf[i][x].z, t);
          t = fmaf(q.w, kf[i][x].w, t);
        }
      }
    if (u0 + kTile < uend) load_k(u0 + kTile);
    reduce_halves<ROWS * 4, 4>(s, lane);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int u = u0 + grp * 4 + key0 + i, w = u - kl.np;
      const int key = w < kl.ns ? w : kl.lo + (w - kl.ns);
      const bool in = valid && u < uend && (u < kl.np ? pre : sees_own(a, span, key));
      if (score && in) score[key] = s[i];
      if (!in) s[i] = -INFINITY;
      top = fmaxf(top, s[i]);
    }
    if (__any_sync(0xffffffffu, top > m + kSlack)) {
      // the row's maximum, over the groups and the lanes that share the row
#pragma unroll
      for (int x = 8; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
#pragma unroll
      for (int x = 1; x < 8 / ROWS; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m, top);
      const float alpha = ex2(m - (mn == -INFINITY ? 0.f : mn));
      m = mn;
      l *= alpha;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float al = __shfl_sync(0xffffffffu, alpha, r * (8 / ROWS));
#pragma unroll
        for (int x = 0; x < kW; ++x) o[r][x] *= al;
      }
    }
    const float ref = m == -INFINITY ? 0.f : m;      // nothing seen so far: every weight is 0
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      s[i] = ex2(s[i] - ref);
      l += s[i];
      s_p[warp][grp * 4 + key0 + i][row] = s[i];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float p[ROWS];
      if constexpr (ROWS == 2) {
        const float2 t = *reinterpret_cast<const float2*>(s_p[warp][k]);
        p[0] = t.x, p[1] = t.y;
      } else {
#pragma unroll
        for (int r = 0; r < ROWS; r += 4) {
          const float4 t = *reinterpret_cast<const float4*>(&s_p[warp][k][r]);
          p[r] = t.x, p[r + 1] = t.y, p[r + 2] = t.z, p[r + 3] = t.w;
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int x = 0; x < kW; ++x) o[r][x] = fmaf(p[r], vf[k][x], o[r][x]);
    }
    if (u0 + kTile < uend) load_v(u0 + kTile);
    __syncwarp();                          // the weights are read before the next are written
  }

  // the row's sum over the lanes that hold its scores
#pragma unroll
  for (int x = 8; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
  for (int x = 1; x < 8 / ROWS; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if (grp == 0 && key0 == 0) {
    sm.m[warp][row] = m;
    sm.l[warp][row] = l;
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int x = 0; x < kW; ++x) sm.o[warp][r][kW * lane + x] = o[r][x];
  dec_finish<float>(sm, a, out, sp, kvh, t0 * kTile, uend);
}

template <int D, int ROWS>
cudaError_t launch(const CacheArgs& a, const CacheRows& rm, const CacheOut& out, cudaStream_t s) {
  const int nrb = (rm.RG + ROWS - 1) / ROWS;
  return launch_dec(out.warps == 8 ? cache_dec32_kernel<D, ROWS, 8> : cache_dec32_kernel<D, ROWS, 4>,
                    (int64_t)rm.groups * nrb * out.nsplit, a, rm, out, nrb, s);
}

template <int D>
cudaError_t launch_d(const CacheArgs& a, const CacheRows& rm, const CacheOut& out, cudaStream_t s) {
  if (rm.RG <= 2) return launch<D, 2>(a, rm, out, s);
  if (rm.RG <= 4) return launch<D, 4>(a, rm, out, s);
  return launch<D, 8>(a, rm, out, s);
}

}  // namespace

cudaError_t launch_cache_dec_f32(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                                 cudaStream_t s) {
  return a.D == 64 ? launch_d<64>(a, rm, out, s) : launch_d<128>(a, rm, out, s);
}

}  // namespace area
