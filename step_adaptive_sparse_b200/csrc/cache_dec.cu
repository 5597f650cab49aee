// Attention over a key/value cache for few query rows (bf16): one pass over
// the keys, which is what bounds it.
//
// A block has up to 8 rows of a group and four warps (eight where the blocks do not
// fill the GPU), which take the keys 16 at a time in turn.  The products are taken transposed, so that 8 rows
// fill a whole mma.m16n8k16 and no row is padded beyond that:
//   S^T (16 keys x 8 rows)    = K (16 x D)    Q^T (D x 8)
//   O^T (D x 8 rows)          = V^T (D x 16)  P^T (16 x 8)
// Keys and values go from global memory into the fragments without passing
// through shared memory: a fragment's order of the summed index is free as
// long as both operands agree, so a thread takes 16 contiguous bytes of a key
// row as the fragments of two k-steps, and 16 bytes of each of four value rows,
// interleaved pairwise, as those of four 16 x 16 blocks of V^T.  Each buffer
// is loaded again as soon as the products have read it, so that a warp keeps
// 16 keys and values (8 KB at D = 128) in flight.
// The softmax keeps one reference per row and rescales only when a score
// exceeds it by more than 2^8 (numerator and denominator use the same one, so
// the result is exact).  The weights are rounded once, to bf16: an mma takes both its
// factors in one type, and the values have that one.  It costs a row 2^-8 of its
// weighted values at most (measured: outputs off by 2.3e-3 rms of their size on long
// caches, 1.7e-3 with weights of 32 bits, which is the output's own rounding).
// mma.sync is enough here: at 8 rows the products take a fifth of
// the time that the keys take to arrive.
#include "cache_dec.cuh"

namespace area {
namespace {

constexpr int kRows = 8;                     // rows of a block
constexpr int kStep = 16;                    // keys of a warp and step
constexpr float kSlack = 8.f;                // log2 units

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Keys and values are read once: they need no place in L1.
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 1 : D == 64 ? 4 : 3)
cache_dec_kernel(const CacheArgs a, const CacheRows rm, const CacheOut out, int nrb) {
  constexpr int kTile = WARPS * kStep;       // keys of a block and step
  constexpr int kU = D / 32;                 // 16-byte loads of a thread per key row
  constexpr int kG = D / 64;                 // 16-byte loads of a thread per value row
  __shared__ DecSmem<D, kRows, WARPS> sm;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = lane >> 2, c = lane & 3;
  const int sp = blockIdx.x % out.nsplit;
  const int rb = blockIdx.x / out.nsplit % nrb;
  let_next_start();
  const int g = dec_group(a, rm, blockIdx.x / out.nsplit / nrb);
  const int r0 = rb * kRows, r1 = min(r0 + kRows, rm.RG);
  const int kvh = rm.pool_rows ? 0 : g / rm.kv_div;           // (b, key head)
  const KeyList kl = key_list(a, rm, rm.pool_rows ? 0 : kvh / a.Hk, r0, r1);
  const auto* kb = static_cast<const __nv_bfloat16*>(a.k) + (int64_t)kvh * a.S * D;
  const auto* vb = static_cast<const __nv_bfloat16*>(a.v) + (int64_t)kvh * a.S * D;
  const int64_t pbase = (int64_t)(rm.pool_rows ? g : kvh % a.Hk) * a.P * D;
  const auto* kpb = static_cast<const __nv_bfloat16*>(a.kp) + pbase;
  const auto* vpb = static_cast<const __nv_bfloat16*>(a.vp) + pbase;

  dec_rows(sm, a, rm, g, r0);

  // this split's tiles of kTile keys
  const int ntile = (kl.total + kTile - 1) / kTile;
  const int t0 = (int)((int64_t)ntile * sp / out.nsplit);
  const int t1 = (int)((int64_t)ntile * (sp + 1) / out.nsplit);

  // the base address of key u of the list (past its end: the last key's)
  auto key_at = [&](int u, const __nv_bfloat16* own, const __nv_bfloat16* pre) {
    u = min(u, kl.total - 1);
    if (u < kl.np) return pre + (int64_t)u * D;
    const int w = u - kl.np;
    return own + (int64_t)(w < kl.ns ? w : kl.lo + (w - kl.ns)) * D;
  };
  uint4 kf[2][kU], vf[4][kG];
  auto load_k = [&](int u0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat16* p = key_at(u0 + n + 8 * h, kb, kpb) + 8 * c;
#pragma unroll
      for (int u = 0; u < kU; ++u) kf[h][u] = load16(p + 32 * u);
    }
  };
  auto load_v = [&](int u0) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int u = u0 + 2 * c + (h & 1) + 8 * (h >> 1);
      const __nv_bfloat16* p = key_at(u, vb, vpb) + 8 * n;
#pragma unroll
      for (int q = 0; q < kG; ++q) {
        vf[h][q] = load16(p + 64 * q);
        // past the list: zeros, so that a weight of zero meets no other value
        if (u >= kl.total) vf[h][q] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  int u0 = t0 * kTile + warp * kStep;
  const int uend = min(t1 * kTile, kl.total);
  if (u0 < uend) {
    load_k(u0);
    load_v(u0);
  }

  // queries: row n, in the order of the key fragments
  uint32_t qf[kU][4];
  const int64_t row = sm.row[n];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row >= 0)
      x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + row * D +
                                          32 * u + 8 * c);
    qf[u][0] = x.x, qf[u][1] = x.y, qf[u][2] = x.z, qf[u][3] = x.w;
  }
  // a thread's scores are those of rows 2c and 2c + 1
  KeySpan span[2];
  bool pre[2], all = true;        // all: every row of the block sees the whole list
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = 2 * c + x;
    span[x] = sm.span[r];
    pre[x] = sm.row[r] >= 0 && sees_prefix(a, span[x]);
    if (sm.row[r] >= 0)
      all = all && (kl.np == 0 || pre[x]) &&
            (kl.total == kl.np ||
             (span[x].hi - kl.lo == kl.total - kl.np - kl.ns && span[x].lo == kl.lo));
  }
  all = __all_sync(0xffffffffu, all);
  float* score[2];               // where key 0's scores of these rows go
#pragma unroll
  for (int x = 0; x < 2; ++x)
    score[x] = out.logits && sm.row[2 * c + x] >= 0 ? out.logits + sm.row[2 * c + x] * a.S : nullptr;

  float o[kG * 4][4], m[2], l[2];
#pragma unroll
  for (int i = 0; i < kG * 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  m[0] = m[1] = -INFINITY;
  l[0] = l[1] = 0.f;

  for (; u0 < uend; u0 += kTile) {
    float s[4] = {};
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      mma_bf16(s, kf[0][u].x, kf[1][u].x, kf[0][u].y, kf[1][u].y, qf[u][0], qf[u][1]);
      mma_bf16(s, kf[0][u].z, kf[1][u].z, kf[0][u].w, kf[1][u].w, qf[u][2], qf[u][3]);
    }
    if (u0 + kTile < uend) load_k(u0 + kTile);
    // s[0..3]: key n of rows 2c, 2c + 1, then key n + 8
    const bool whole = all && u0 + kStep <= uend;
    bool grow = false;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[x] *= a.scale_log2;
      if (whole) {
        // (with scores the list is the cache's first keys)
        if (score[x & 1]) score[x & 1][u0 + n + 8 * (x >> 1)] = s[x];
      } else {
        const int u = u0 + n + 8 * (x >> 1), w = u - kl.np;
        const int key = w < kl.ns ? w : kl.lo + (w - kl.ns);
        const bool in = u < uend && (u < kl.np ? pre[x & 1] : sees_own(a, span[x & 1], key));
        if (score[x & 1] && in) score[x & 1][key] = s[x];
        if (!in) s[x] = -INFINITY;
      }
      grow = grow || s[x] > m[x & 1] + kSlack;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = fmaxf(s[x], s[x + 2]);
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        const float mn = fmaxf(m[x], mx);
        const float alpha = ex2(m[x] - (mn == -INFINITY ? 0.f : mn));
        m[x] = mn;
        l[x] *= alpha;
#pragma unroll
        for (int i = 0; i < kG * 4; ++i) {
          o[i][x] *= alpha;
          o[i][x + 2] *= alpha;
        }
      }
    }
    uint32_t pf[2];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      // nothing seen so far: every weight is 0
      const float ref = m[x & 1] == -INFINITY ? 0.f : m[x & 1];
      s[x] = ex2(s[x] - ref);
      l[x & 1] += s[x];
    }
    pf[0] = transpose8x8(pack2(s[0], s[1]));
    pf[1] = transpose8x8(pack2(s[2], s[3]));
#pragma unroll
    for (int q = 0; q < kG; ++q) {
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&vf[0][q]);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&vf[1][q]);
      const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&vf[2][q]);
      const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&vf[3][q]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = __byte_perm(w0[w], w1[w], 0x5410), a1 = __byte_perm(w0[w], w1[w], 0x7632);
        const uint32_t a2 = __byte_perm(w2[w], w3[w], 0x5410), a3 = __byte_perm(w2[w], w3[w], 0x7632);
        mma_bf16(o[q * 4 + w], a0, a1, a2, a3, pf[0], pf[1]);
      }
    }
    if (u0 + kTile < uend) load_v(u0 + kTile);
  }

  // the warps' results: rows 2c, 2c + 1 and dims 64 q + 8 n + 2 w, + 1
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = 2 * c + x;
#pragma unroll
    for (int y = 4; y < 32; y <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], y);
    if (n == 0) {
      sm.m[warp][r] = m[x];
      sm.l[warp][r] = l[x];
    }
#pragma unroll
    for (int i = 0; i < kG * 4; ++i)
      *reinterpret_cast<float2*>(&sm.o[warp][r][64 * (i >> 2) + 8 * n + 2 * (i & 3)]) =
          make_float2(o[i][x], o[i][x + 2]);
  }
  dec_finish<__nv_bfloat16>(sm, a, out, sp, kvh, t0 * kTile, uend);
}

template <int D>
cudaError_t launch(const CacheArgs& a, const CacheRows& rm, const CacheOut& out, cudaStream_t s) {
  const int nrb = (rm.RG + kRows - 1) / kRows;
  const int64_t grid = (int64_t)rm.groups * nrb * out.nsplit;
  return launch_dec(out.warps == 8 ? cache_dec_kernel<D, 8> : cache_dec_kernel<D, 4>, grid, a, rm, out, nrb, s);
}

}  // namespace

cudaError_t launch_cache_dec_bf16(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                                  cudaStream_t s) {
  return a.D == 64 ? launch<64>(a, rm, out, s) : launch<128>(a, rm, out, s);
}

}  // namespace area
