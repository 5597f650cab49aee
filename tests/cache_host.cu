// The host side of the key/value cache's calls without a GPU: their entry points
// (cache_api.cu) over launches that only count themselves, and the index
// arithmetic that kernels share with the host.  Built as a shared library and
// called by CPU tests; no kernel is in it, so that a call that passes validation
// touches no memory.
#include "cache_api.cu"

extern "C" {
int host_cache_len(const int* lens, int S, int b) {
  area::CacheArgs a{};
  a.lens = lens;
  a.S = S;
  return area::cache_len(a, b);
}
// 1: the prefix goes against the rows of all sequences in a launch of its own.
int host_pools(int B, int H, int Hk, int Nq, int P, int S, int D, int dtype) {
  area::CachePlan p;
  if (area::cache_plan(area::CACHE_OP_PREFIX, B, H, Hk, Nq, P, S, D, INT_MAX, 0, dtype, &p) != AREA_OK) return -1;
  return p.pooled.used;
}
// Most keys of a unit of the kernels for many rows (0: the call has none); -1: refused.
int64_t host_unit_keys(int op, int B, int H, int Hk, int Nq, int P, int S, int D, int dtype) {
  area::CachePlan p;
  if (area::cache_plan(op, B, H, Hk, Nq, P, S, D, INT_MAX, 0, dtype, &p) != AREA_OK) return -1;
  int64_t most = 0;
  for (const area::CacheLaunch* l : {&p.main, &p.pooled})
    if (l->used && l->kernel == area::CACHE_TC) {
      const int64_t keys = (l->rows.use_prefix ? (int64_t)P : 0) + (l->rows.use_own ? S : 0);
      most = std::max(most, (keys + l->nsplit - 1) / l->nsplit);
    }
  return most;
}
int host_share_of(int n, int part, int parts) { return area::share_of(n, part, parts); }
}

namespace {
int g_launches = 0;
cudaError_t counted() {
  ++g_launches;
  return cudaSuccess;
}
}  // namespace

extern "C" int host_launches(void) {        // since the last look
  const int n = g_launches;
  g_launches = 0;
  return n;
}

namespace area {
int fail_cuda(cudaError_t) { return AREA_ECUDA; }
cudaError_t launch_cache_dec_bf16(const CacheArgs&, const CacheRows&, const CacheOut&, cudaStream_t) { return counted(); }
cudaError_t launch_cache_dec_f32(const CacheArgs&, const CacheRows&, const CacheOut&, cudaStream_t) { return counted(); }
cudaError_t launch_cache_tc(const CacheArgs&, const CacheRows&, const CacheOut&, cudaStream_t) { return counted(); }
cudaError_t launch_cache_tc32(const CacheArgs&, const CacheRows&, const CacheOut&, cudaStream_t) { return counted(); }
cudaError_t launch_cache_join(const CacheArgs&, const float*, const float2*, int, int64_t, float*, int,
                              cudaStream_t) { return counted(); }
cudaError_t launch_cache_join_weights(const CacheArgs&, const CacheOut&, int, int, cudaStream_t) { return counted(); }
cudaError_t launch_cache_weights_tc(const CacheArgs&, const float*, const float*, float*, int, cudaStream_t) {
  return counted();
}
cudaError_t launch_cache_evict(const EvictArgs&, cudaStream_t) { return counted(); }
}  // namespace area
