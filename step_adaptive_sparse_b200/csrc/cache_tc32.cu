// Attention over a key/value cache for many query rows (fp32) on the tensor
// cores, without giving up fp32's precision.
//
// Every fp32 value is the exact sum of three bf16 values: its top 8 significand
// bits, the next 8 and the last 8 (x = x0 + x1 + x2, cut off, not rounded, so
// that no value overflows).  A product of two values is taken as the six terms
//   x1 y1, x0 y2, x2 y0, x0 y1, x1 y0, x0 y0,
// the small ones first; what is left out is below 2^-22 of it, and about 2^-25
// on average.  That is six bf16 products for one of fp32, still four times
// the rate of the CUDA cores (1643 / 6 against 64 TFLOP/s measured).
// The accumulator of a chain of products loses up to a bit in each addition, so
// a chain is kept short: one tile's scores, or one tile's 64 keys times their
// values, whose sum is added in registers with the running output.
//
// A persistent CTA per SM of 512 threads: warps 0-7 read keys and values, cut
// them into their parts and write these as swizzled operand tiles (rows past
// the list as zeros, so that nothing outside it is read), two buffers each;
// warp 8 issues the products, warp 9 decodes work units; warps 12-15 hold one tile of 128 query rows, one
// row to a thread: they cut the queries, do the softmax and hold the output.
// Both products take their first factor from TMEM, so that shared memory, which
// also takes the parts' writes, feeds the tensor cores with the second alone
// (queries in shared memory: 7000 cycles a tile at D = 128).  TMEM: S0 | S1 (64
// columns each; the weights' first two parts replace a tile's scores) | X0 | X1
// (32 each, the third part) | Q (three parts of D / 2) | O (one tile's output).
// Products are issued as QK(j + 1), PV(j), so that a tile's softmax and the
// reading of its output run under the other products.
// Work units and the keys of a row are as in the bf16 kernel, with one row tile
// and key tiles of 64.  Every mbarrier wait is bounded.
#include "cache_unit.cuh"
#include "cut3.cuh"
#include "tc_common.cuh"

namespace area {
namespace {

constexpr int kThreads = 512, kReadWarps = 8, kReadThreads = 32 * kReadWarps;
constexpr int kKT = 64;                    // keys of a tile
constexpr int kRecSlots = 3;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// The softmax warpgroup gets what the others give up; the sum is exactly the
// allocation of a 128-register launch (checked before it).
constexpr int kRegsRead = 96, kRegsMma = 72, kRegsSoft = 248;
static_assert(2 * kRegsRead + kRegsMma + kRegsSoft == 4 * 128, "register split");

template <int D>
struct Geo {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kKT * 128;                        // bytes of 64 columns
  static constexpr int kTerm = kHalves * kHalf, kTile = 3 * kTerm;
  static constexpr int kSmemV = 2 * kTile, kSmemBar = kSmemV + 2 * kTile;
  static constexpr int kSmemBytes = kSmemBar + 256 + 1024;       // barriers + alignment slack
  static_assert(kSmemBytes + 2048 <= 227 * 1024, "shared memory of one CTA");
  static constexpr uint32_t kColX = 128, kColQ = 192, kColO = kColQ + 3 * D / 2;
  static_assert(kColO + D <= 512, "TMEM");
};

enum {
  BAR_Q_FULL = 0, BAR_O_FULL, BAR_O_EMPTY,
  BAR_K_FULL, BAR_K_EMPTY = BAR_K_FULL + 2,
  BAR_V_FULL = BAR_K_EMPTY + 2, BAR_V_EMPTY = BAR_V_FULL + 2,
  BAR_S_FULL = BAR_V_EMPTY + 2, BAR_P_FULL = BAR_S_FULL + 2,
  BAR_REC_FULL = BAR_P_FULL + 2,
  BAR_REC_EMPTY = BAR_REC_FULL + kRecSlots,
  BAR_DRAIN = BAR_REC_EMPTY + kRecSlots,
  BAR_COUNT
};
static_assert(BAR_COUNT * 8 <= 256, "barrier area");

// The bits below n of a word.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_tc32_kernel(const __grid_constant__ UnitParams prm) {
  using G = Geo<D>;
  constexpr uint32_t kIdescS = idesc(kKT, false), kIdescO = idesc(D, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + G::kSmemBar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ __align__(16) Unit s_rec[kRecSlots];
  __shared__ KeySpan s_span[128];          // of the softmax threads' rows
  auto bar = [&](uint32_t i) { return bar0 + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s_abort = 0;
    mbar_init(bar(BAR_Q_FULL), 128);
    mbar_init(bar(BAR_O_FULL), 1);
    mbar_init(bar(BAR_O_EMPTY), 128);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_K_FULL + t), kReadThreads);
      mbar_init(bar(BAR_K_EMPTY + t), 1);
      mbar_init(bar(BAR_V_FULL + t), kReadThreads);
      mbar_init(bar(BAR_V_EMPTY + t), 1);
      mbar_init(bar(BAR_S_FULL + t), 1);
      mbar_init(bar(BAR_P_FULL + t), 128);
    }
    for (int s = 0; s < kRecSlots; ++s) {
      mbar_init(bar(BAR_REC_FULL + s), 1);
      // the reading warps, the product warp, four softmax warps
      mbar_init(bar(BAR_REC_EMPTY + s), kReadWarps + 5);
    }
    mbar_init(bar(BAR_DRAIN), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kReadWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&s_tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  int* abort_flag = &s_abort;

  // the paths must not meet again before the end (see the bf16 kernel)
  if (warp < kReadWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRead) : "memory");
    // ---------------------------------------------- reading and cutting up
    constexpr int kPieces = D / 4;                  // 16-byte pieces of a row
    constexpr int kRowStep = kReadThreads / kPieces, kPer = kKT / kRowStep;
    const int piece = threadIdx.x % kPieces, row0 = threadIdx.x / kPieces;
    uint32_t k_it = 0, v_it = 0, unit_count = 0;
    bool ok = true;
    while (ok) {
      const uint32_t slot = unit_count % kRecSlots;
      if (!(ok = warp_wait_all(bar(BAR_REC_FULL + slot), (unit_count / kRecSlots) & 1u,
                               abort_flag)))
        break;
      const Unit& u = s_rec[slot];
      if (!u.valid) break;
      const int nt = u.nt;
      float kf[kPer][4], vf[kPer][4];
      auto load = [&](float (&f)[kPer][4], int j, bool val) {
        const Tile t = tile_of<kKT>(u, j);
        const float* p = static_cast<const float*>(t.kind ? (val ? prm.a.v : prm.a.k)
                                                          : (val ? prm.a.vp : prm.a.kp)) +
                         ((int64_t)(t.kind ? u.kvh : u.ph) * (t.kind ? prm.a.S : prm.a.P) + t.j0 +
                          row0) * D + piece * 4;
#pragma unroll
        for (int i = 0; i < kPer; ++i) get4(p + i * kRowStep * D, row0 + i * kRowStep < t.n, f[i]);
      };
      auto put = [&](float (&f)[kPer][4], uint32_t at) {
        at += sbase + (piece >> 4) * G::kHalf + (piece & 1) * 8;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = row0 + i * kRowStep;
          put4(at + r * 128 + ((((piece >> 1) & 7) ^ (r & 7)) << 4), G::kTerm, f[i]);
        }
        fence_proxy_async();
      };
      if (nt > 0) load(kf, 0, false);
      // K(j + 1) before V(j): the order in which their buffers become free
      for (int j = -1; j < nt; ++j) {
        if (j + 1 < nt) {
          const uint32_t b = k_it & 1u;
          if (!(ok = warp_wait_all(bar(BAR_K_EMPTY + b), ((k_it >> 1) & 1u) ^ 1u, abort_flag)))
            break;
          put(kf, b * G::kTile);
          mbar_arrive(bar(BAR_K_FULL + b));
          ++k_it;
          if (j + 2 < nt) load(kf, j + 2, false);
        }
        if (j >= 0) {
          const uint32_t b = v_it & 1u;
          if (!(ok = warp_wait_all(bar(BAR_V_EMPTY + b), ((v_it >> 1) & 1u) ^ 1u, abort_flag)))
            break;
          put(vf, G::kSmemV + b * G::kTile);
          mbar_arrive(bar(BAR_V_FULL + b));
          ++v_it;
        }
        if (j + 1 < nt) load(vf, j + 1, true);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(bar(BAR_REC_EMPTY + slot));
      ++unit_count;
    }
  } else if (warp < kReadWarps + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma) : "memory");
    // -------------------------------------------------------------- products
    if (warp == kReadWarps) {
      uint32_t unit_count = 0, q_count = 0;
      uint32_t s_it = 0, p_it = 0;     // tiles whose scores, whose outputs have been issued
      bool ok = true;
      const uint64_t dk = sdesc(sbase, 16, 1024), dv = sdesc(sbase + G::kSmemV, G::kHalf, 1024);
      auto qk = [&]() -> bool {
        const uint32_t b = s_it & 1u;
        if (!warp_wait_all(bar(BAR_K_FULL + b), (s_it >> 1) & 1u, abort_flag)) return false;
        tc_fence_after();
        const uint32_t d = tmem + b * 64;
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < 6; ++t) {
            const uint32_t tq = tmem + G::kColQ + part_a(t) * (D / 2);
            const uint64_t tk = opaque(sdesc_at(dk, b * G::kTile + part_b(t) * G::kTerm));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ts(d, tq + kk * 8, sdesc_at(tk, (kk >> 2) * G::kHalf + (kk & 3) * 32), kIdescS,
                       (t > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar(BAR_S_FULL + b));
          mma_commit(bar(BAR_K_EMPTY + b));
        }
        __syncwarp();
        ++s_it;
        return true;
      };
      auto pv = [&]() -> bool {
        const uint32_t b = p_it & 1u, ph = (p_it >> 1) & 1u;
        if (!warp_wait_all(bar(BAR_V_FULL + b), ph, abort_flag)) return false;
        if (!warp_wait_all(bar(BAR_P_FULL + b), ph, abort_flag)) return false;
        if (!warp_wait_all(bar(BAR_O_EMPTY), (p_it & 1u) ^ 1u, abort_flag)) return false;
        tc_fence_after();
        const uint32_t d = tmem + G::kColO;
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < 6; ++t) {
            const uint32_t pa = part_a(t);
            const uint32_t p = tmem + (pa < 2 ? b * 64 + pa * 32 : G::kColX + b * 32);
            const uint64_t tv = opaque(sdesc_at(dv, b * G::kTile + part_b(t) * G::kTerm));
#pragma unroll
            for (int kk = 0; kk < kKT / 16; ++kk)
              mma_ts(d, p + kk * 8, sdesc_at(tv, kk * 2048), kIdescO, (t > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar(BAR_O_FULL));
          mma_commit(bar(BAR_V_EMPTY + b));
        }
        __syncwarp();
        ++p_it;
        return true;
      };
      while (ok) {
        const uint32_t slot = unit_count % kRecSlots;
        if (!(ok = warp_wait_all(bar(BAR_REC_FULL + slot), (unit_count / kRecSlots) & 1u,
                                 abort_flag)))
          break;
        const int valid = __shfl_sync(0xffffffffu, s_rec[slot].valid, 0);
        const int nt = __shfl_sync(0xffffffffu, s_rec[slot].nt, 0);
        if (lane == 0) mbar_arrive(bar(BAR_REC_EMPTY + slot));
        __syncwarp();
        if (!valid) break;
        ++unit_count;
        // Units without a tile have no queries.  Those of the next unit that has
        // some are written after the scores of the last one's tiles, which follow
        // this wait, so that no phase of the barrier passes unseen.
        if (nt == 0) continue;
        if (!(ok = warp_wait_all(bar(BAR_Q_FULL), q_count++ & 1u, abort_flag))) break;
        for (int j = 0; j < nt; ++j) {
          if (j == 0 && !(ok = qk())) break;
          if (j + 1 < nt && !(ok = qk())) break;
          if (!(ok = pv())) break;
        }
      }
      int drain_abort = 0;
      if (elect_one()) mma_commit(bar(BAR_DRAIN));
      __syncwarp();
      warp_wait_all(bar(BAR_DRAIN), 0, &drain_abort);
    } else if (warp == kReadWarps + 1) {
      // the units' records, up to kRecSlots ahead; the first that is not valid
      // ends every role
      for (uint32_t k = 0;; ++k) {
        const uint32_t slot = k % kRecSlots;
        if (!warp_wait0(bar(BAR_REC_EMPTY + slot), ((k / kRecSlots) & 1u) ^ 1u, abort_flag)) break;
        int valid = 0;
        if (lane == 0) {
          Unit u;
          valid = u.valid = decode_unit<kKT>(unit_index(k), prm, u) ? 1 : 0;
          s_rec[slot] = u;
          mbar_arrive(bar(BAR_REC_FULL + slot));
        }
        if (!__shfl_sync(0xffffffffu, valid, 0)) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft) : "memory");
    // ------------------------------------------------------ softmax / output
    const int trow = ((warp & 3) << 5) + lane;       // TMEM lane = row of the tile
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) << 5) << 16);
    uint32_t it = 0, unit_count = 0;                 // tiles so far, over all units
    const float sl2 = prm.a.scale_log2;
    bool ok = true;
    while (ok) {
      const uint32_t slot = unit_count % kRecSlots;
      if (!(ok = warp_wait_all(bar(BAR_REC_FULL + slot), (unit_count / kRecSlots) & 1u,
                               abort_flag)))
        break;
      const Unit& u = s_rec[slot];
      if (!u.valid) break;
      // this thread's row and what it sees; rows that do not exist see all
      const int r = u.r0[0] + trow;
      const bool rvalid = r < prm.rm.RG;
      const int nt = u.nt;
      // The query's parts, once the last unit's scores are done with the old ones
      // (the last of them was waited for).  The span is kept in shared memory:
      // the output and a score row fill the registers.
      if (nt > 0) {
        KeySpan sp{0, INT_MAX};
        const float* q = nullptr;
        if (rvalid) {
          const CacheRow cr = cache_row(prm.a, prm.rm, u.g, r);
          sp = key_span(prm.a, cache_len(prm.a, cr.b), cr.i);
          q = static_cast<const float*>(prm.a.q) + cr.row * D;
        }
        s_span[trow] = sp;
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          float f[16][4];
#pragma unroll
          for (int i = 0; i < 16; ++i) get4(q + c + 4 * i, rvalid, f[i]);
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            uint32_t p[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) p[i] = cut2(f[i / 2][i % 2 * 2], f[i / 2][i % 2 * 2 + 1]);
            tmem_st32(tl + G::kColQ + part * (D / 2) + c / 2, p);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(BAR_Q_FULL));
      }
      float m = -INFINITY, l = 0.f, o[D];
      RowRef ref{sl2, 0.f};                // nothing seen so far: all weights 0
#pragma unroll
      for (int i = 0; i < D; ++i) o[i] = 0.f;
      // adds tile k's output
      auto add_output = [&](uint32_t k) -> bool {
        if (!warp_wait_all(bar(BAR_O_FULL), k & 1u, abort_flag)) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t t[32];
          tmem_ld32(tl + G::kColO + c * 32, t);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[c * 32 + i] += __uint_as_float(t[i]);
        }
        tc_fence_before();
        mbar_arrive(bar(BAR_O_EMPTY));
        return true;
      };
      for (int j = 0; j < nt; ++j, ++it) {
        const Tile t = tile_of<kKT>(u, j);
        // the tile's keys that this row sees, one bit each
        uint32_t sees0, sees1;
        {
          const KeySpan sp = s_span[trow];
          int ka = 0, kb, kc = 0;
          if (t.kind == 0) {
            kb = sees_prefix(prm.a, sp) ? t.n : 0;
          } else {
            ka = sp.lo - t.j0;
            kb = min(sp.hi - t.j0, t.n);
            kc = min(prm.a.sinks - t.j0, kb);
          }
          sees0 = (bits_below(kb) & ~bits_below(ka)) | bits_below(kc);
          sees1 = (bits_below(kb - 32) & ~bits_below(ka - 32)) | bits_below(kc - 32);
        }
        if (!(ok = warp_wait_all(bar(BAR_S_FULL + (it & 1u)), (it >> 1) & 1u, abort_flag))) break;
        tc_fence_after();
        const uint32_t tS = tl + (it & 1u) * 64, tX = tl + G::kColX + (it & 1u) * 32;
        float s[kKT];
        tmem_ld32(tS, reinterpret_cast<uint32_t(&)[32]>(s[0]));
        tmem_ld32(tS + 32, reinterpret_cast<uint32_t(&)[32]>(s[32]));
        if (__any_sync(0xffffffffu, (sees0 & sees1) != 0xffffffffu)) {
#pragma unroll
          for (int i = 0; i < kKT; ++i)
            if (!((i < 32 ? sees0 : sees1) >> (i & 31) & 1u)) s[i] = -INFINITY;   // no weight
        }
        float pm[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kKT; i += 2) pm[(i >> 1) & 3] = max3(pm[(i >> 1) & 3], s[i], s[i + 1]);
        const float top = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
        const float mnew = fmaxf(top * sl2, m);
        const bool rescale = __any_sync(0xffffffffu, mnew > m + kRescaleThreshold);
        const float alpha = rescale ? (m == -INFINITY ? 0.f : fast_exp2(m - mnew)) : 1.f;
        if (rescale) {
          if (mnew > m) ref = row_ref(top, mnew, sl2);
          m = mnew;
        }
        l *= alpha;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kKT; i += 2) {
          float x0, x1;
          fma2(x0, x1, s[i], s[i + 1], ref.mul, ref.add);
          s[i] = fast_exp2(x0);
          s[i + 1] = fast_exp2(x1);
          if ((i >> 1) & 1) add2(ls[2], ls[3], s[i], s[i + 1]); else add2(ls[0], ls[1], s[i], s[i + 1]);
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        // the weights' parts, one after the other: what is left takes their place
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) p[i] = cut2(s[2 * i], s[2 * i + 1]);
          tmem_st32(part < 2 ? tS + part * 32 : tX, p);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(BAR_P_FULL + (it & 1u)));
        if (j > 0 && !(ok = add_output(it - 1))) break;
        if (rescale) {
#pragma unroll
          for (int i = 0; i < D; ++i) o[i] *= alpha;
        }
      }
      if (!ok) break;
      if (nt > 0 && !(ok = add_output(it - 1))) break;
      // ---- epilogue
      if (rvalid) {
        const int64_t row = cache_row(prm.a, prm.rm, u.g, r).row;
        const int64_t at = (int64_t)(prm.out.slot0 + u.sp) * prm.out.rows + row;
        if (!prm.out.direct) prm.out.part_ml[at] = make_float2(m, l);
        if (prm.out.lse) prm.out.lse[row] = l == 0.f ? INFINITY : m + log2f(l);
        const float mul = !prm.out.direct ? 1.f : l == 0.f ? 0.f : 1.f / l;
        float* dst = prm.out.direct ? static_cast<float*>(prm.a.o) + row * D
                                    : prm.out.part_o + at * D;
        if (prm.out.direct || l != 0.f) {
#pragma unroll
          for (int c = 0; c < D; c += 8) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = o[c + i] * mul;
            st_global_v8f(dst + c, f);
          }
        }
      }
      if (lane == 0) mbar_arrive(bar(BAR_REC_EMPTY + slot));
      ++unit_count;
    }
  }
  let_next_start();
  if (prm.out.early) wait_for_last();
  tc_fence_before();
  __syncthreads();
  if (warp == kReadWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D>
cudaError_t launch(const UnitParams& prm, cudaStream_t s) {
  auto fn = cache_tc32_kernel<D>;
  constexpr int kSmem = Geo<D>::kSmemBytes;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, fn);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc waits until the registers it asks for are free, so the split
  // must fit in what the launch allocates
  if (fa.numRegs != 128) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(fn, std::min(prm.units, num_sms()), kThreads, kSmem, 1, prm.out.early, s, prm);
}

}  // namespace

cudaError_t read_and_clear_cache_tc32_error(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(code, g_tc_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_tc_error, &zero, sizeof(int));
}

cudaError_t launch_cache_tc32(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                              cudaStream_t s) {
  UnitParams p{a, rm, out, (rm.RG + 127) / 128, 128, 1, 0, 0};
  p.units = (int)((int64_t)rm.groups * p.nrb * out.nsplit);
  p.heavy_first = a.causal && !rm.pool_rows;
  return a.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

}  // namespace area
