// Attention over a key/value cache on the CUDA cores: M query rows against
// tiles of 64 keys staged in shared memory as fp32, one pass over the keys
// with the running maximum and sum of the softmax (see cache.cuh for which
// keys a row sees).
//
// A block of M = 16 or 64 rows; each thread owns 4 rows x 64 / TPR scores and
// the same 4 rows x D / TPR output columns, TPR threads to a row.
#include "cache.cuh"

namespace area {
namespace {

constexpr int kKeys = 64;       // keys of a tile
constexpr int kRowsPer = 4;     // rows of a thread

template <int D, int M>
struct Simt {
  static constexpr int kTPR = M == 64 ? 16 : 32;          // threads of a row
  static constexpr int kThreads = M / kRowsPer * kTPR;
  static constexpr int kKPT = kKeys / kTPR;               // scores of a thread and row
  static constexpr int kDPT = D / kTPR;                   // output columns of a thread
  static constexpr int kVec = kDPT < 4 ? kDPT : 4;        // ... in vectors of this width
  static constexpr int kKStride = D + 4;                  // eight key rows touch all 32 banks
  static constexpr int kPStride = kKeys + 4;
  static constexpr int kFloats = M * D + kKeys * kKStride + kKeys * D + M * kPStride;
};

// 16 bytes of T as floats.
__device__ __forceinline__ void load_vec(const float* p, float (&f)[4]) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w;
}
template <int W>
__device__ __forceinline__ void lds(const float* p, float (&f)[W]) {
  if constexpr (W == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(p);
    f[0] = t.x, f[1] = t.y;
  }
}

template <typename T, int D, int M>
__global__ void __launch_bounds__(Simt<D, M>::kThreads)
cache_simt_kernel(const CacheArgs a, const CacheRows rm, const CacheOut out, int nrb) {
  using C = Simt<D, M>;
  extern __shared__ float smem[];
  float* Qs = smem;                             // [M][D], times scale * log2(e)
  float* Ks = Qs + M * D;                       // [kKeys][kKStride]
  float* Vs = Ks + kKeys * C::kKStride;         // [kKeys][D]
  float* Ps = Vs + kKeys * D;                   // [M][kPStride]
  __shared__ int64_t s_row[M];
  __shared__ KeySpan s_span[M];

  const int tid = threadIdx.x;
  const int sp = blockIdx.x % out.nsplit;
  const int rb = blockIdx.x / out.nsplit % nrb;
  const int g = blockIdx.x / out.nsplit / nrb;
  const int r0 = rb * M, r1 = min(r0 + M, rm.RG);
  const int kvh = rm.pool_rows ? 0 : g / rm.kv_div;           // (b, key head)
  const KeyList kl = key_list(a, rm, rm.pool_rows ? 0 : kvh / a.Hk, r0, r1);
  const T* kb = static_cast<const T*>(a.k) + (int64_t)kvh * a.S * D;
  const T* vb = static_cast<const T*>(a.v) + (int64_t)kvh * a.S * D;
  const int64_t pbase = (int64_t)(rm.pool_rows ? g : kvh % a.Hk) * a.P * D;
  const T* kpb = static_cast<const T*>(a.kp) + pbase;
  const T* vpb = static_cast<const T*>(a.vp) + pbase;

  for (int r = tid; r < M; r += C::kThreads) {
    KeySpan s{0, 0};
    int64_t row = -1;
    if (r0 + r < r1) {
      const CacheRow cr = cache_row(a, rm, g, r0 + r);
      row = cr.row;
      s = key_span(a, cache_len(a, cr.b), cr.i);
    }
    s_row[r] = row;
    s_span[r] = s;
  }
  __syncthreads();
  constexpr int kW = 16 / sizeof(T);            // values of one 16-byte load
  for (int e = tid; e < M * (D / kW); e += C::kThreads) {
    const int r = e / (D / kW), d = e % (D / kW) * kW;
    float f[kW] = {};
    if (s_row[r] >= 0) load_vec(static_cast<const T*>(a.q) + s_row[r] * D + d, f);
#pragma unroll
    for (int i = 0; i < kW; ++i) Qs[r * D + d + i] = f[i] * a.scale_log2;
  }

  const int ty = tid / C::kTPR, tx = tid % C::kTPR;
  float acc[kRowsPer][C::kDPT], m[kRowsPer], l[kRowsPer];
  KeySpan span[kRowsPer];
  bool pre[kRowsPer];
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    span[i] = s_span[ty * kRowsPer + i];
    pre[i] = s_row[ty * kRowsPer + i] >= 0 && sees_prefix(a, span[i]);
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < C::kDPT; ++d) acc[i][d] = 0.f;
  }

  // this split's tiles: an even share of the tiles that these rows need
  const int ntile = (kl.total + kKeys - 1) / kKeys;
  const int t0 = (int)((int64_t)ntile * sp / out.nsplit);
  const int t1 = (int)((int64_t)ntile * (sp + 1) / out.nsplit);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    for (int e = tid; e < kKeys * (D / kW); e += C::kThreads) {
      const int key = e / (D / kW), d = e % (D / kW) * kW;
      const int u = t * kKeys + key;
      float fk[kW] = {}, fv[kW] = {};             // past the list: zeros, never memory
      if (u < kl.total) {
        const bool p = u < kl.np;
        const int w = u - kl.np;
        const int64_t j = p ? u : w < kl.ns ? w : kl.lo + (w - kl.ns);
        load_vec((p ? kpb : kb) + j * D + d, fk);
        load_vec((p ? vpb : vb) + j * D + d, fv);
      }
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        Ks[key * C::kKStride + d + i] = fk[i];
        Vs[key * D + d + i] = fv[i];
      }
    }
    __syncthreads();
    float s[kRowsPer][C::kKPT];
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
      for (int j = 0; j < C::kKPT; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float qf[kRowsPer][4], kf[C::kKPT][4];
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) lds<4>(Qs + (ty * kRowsPer + i) * D + d, qf[i]);
#pragma unroll
      for (int j = 0; j < C::kKPT; ++j) lds<4>(Ks + (tx + C::kTPR * j) * C::kKStride + d, kf[j]);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
          for (int j = 0; j < C::kKPT; ++j) s[i][j] = fmaf(qf[i][c], kf[j][c], s[i][j]);
    }
#pragma unroll
    for (int j = 0; j < C::kKPT; ++j) {
      const int u = t * kKeys + tx + C::kTPR * j;
      const int w = u - kl.np;
      const int key = w < kl.ns ? w : kl.lo + (w - kl.ns);
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) {
        const bool in = u < kl.total && (u < kl.np ? pre[i] : sees_own(a, span[i], key));
        if (out.logits && in && s_row[ty * kRowsPer + i] >= 0)
          out.logits[s_row[ty * kRowsPer + i] * a.S + key] = s[i][j];
        if (!in) s[i][j] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      float mx = s[i][0];
#pragma unroll
      for (int j = 1; j < C::kKPT; ++j) mx = fmaxf(mx, s[i][j]);
#pragma unroll
      for (int x = 1; x < C::kTPR; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;     // nothing seen so far: every weight is 0
      const float alpha = exp2f(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < C::kKPT; ++j) {
        const float p = exp2f(s[i][j] - ref);
        sum += p;
        Ps[(ty * kRowsPer + i) * C::kPStride + tx + C::kTPR * j] = p;
      }
      l[i] = l[i] * alpha + sum;                        // this thread's keys only
      m[i] = mn;
#pragma unroll
      for (int d = 0; d < C::kDPT; ++d) acc[i][d] *= alpha;
    }
    __syncwarp();        // a row's weights are written and read by one warp
    const int kn = min(kKeys, kl.total - t * kKeys);
#pragma unroll 2
    for (int k = 0; k < kn; k += 4) {                  // rows past kn are zeros
      float pf[kRowsPer][4];
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) lds<4>(Ps + (ty * kRowsPer + i) * C::kPStride + k, pf[i]);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int x = 0; x < C::kDPT / C::kVec; ++x) {
          float vf[C::kVec];
          lds<C::kVec>(Vs + (k + c) * D + (x * C::kTPR + tx) * C::kVec, vf);
#pragma unroll
          for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
            for (int y = 0; y < C::kVec; ++y)
              acc[i][x * C::kVec + y] = fmaf(pf[i][c], vf[y], acc[i][x * C::kVec + y]);
        }
    }
  }

#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
#pragma unroll
    for (int x = 1; x < C::kTPR; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    const int64_t row = s_row[ty * kRowsPer + i];
    if (row < 0) continue;
    if (out.direct) {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      T* dst = static_cast<T*>(a.o) + row * D;
#pragma unroll
      for (int x = 0; x < C::kDPT / C::kVec; ++x)
#pragma unroll
        for (int y = 0; y < C::kVec; ++y)
          store_from_float(dst, (x * C::kTPR + tx) * C::kVec + y,
                           l[i] == 0.f ? 0.f : acc[i][x * C::kVec + y] * inv);
    } else {
      const int64_t at = (int64_t)(out.slot0 + sp) * out.rows + row;
      if (tx == 0) out.part_ml[at] = make_float2(m[i], l[i]);
      float* dst = out.part_o + at * D;
#pragma unroll
      for (int x = 0; x < C::kDPT / C::kVec; ++x)
#pragma unroll
        for (int y = 0; y < C::kVec; ++y)
          dst[(x * C::kTPR + tx) * C::kVec + y] = acc[i][x * C::kVec + y];
    }
  }
}

template <typename T, int D, int M>
cudaError_t launch(const CacheArgs& a, const CacheRows& rm, const CacheOut& out, cudaStream_t s) {
  using C = Simt<D, M>;
  const int smem = C::kFloats * (int)sizeof(float);
  auto fn = cache_simt_kernel<T, D, M>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int nrb = (rm.RG + M - 1) / M;
  const int64_t grid = (int64_t)rm.groups * nrb * out.nsplit;
  fn<<<(unsigned)grid, C::kThreads, smem, s>>>(a, rm, out, nrb);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_simt(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                              cudaStream_t s) {
  return a.D == 64 ? launch<float, 64, 64>(a, rm, out, s) : launch<float, 128, 64>(a, rm, out, s);
}

}  // namespace area
