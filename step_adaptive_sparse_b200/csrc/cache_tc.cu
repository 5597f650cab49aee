// Attention over a key/value cache for many query rows (bf16): tcgen05 flash
// attention with causal order, a sliding window, sinks, a shared prefix and a
// split of the keys.
//
// A persistent CTA per SM of 384 threads: warp 0 decodes work units and loads
// (TMA), warp 1 issues the products, warps 4-7 and 8-11 do the softmax of the
// unit's two tiles of 128 query rows, one row to a thread (warps 2 and 3 are
// there so that the register split can take from whole warpgroups).  TMEM: S0 | S1 |
// O0 | O1, 128 fp32 columns each; P (bf16) replaces S and feeds the second
// product from TMEM, handed over in two halves.  P is bf16 because a product has both
// factors in one type, and the values' is that one; products with P's lower parts would be
// half as many again.  It costs a row 2^-8 of its weighted values at most (measured:
// outputs off by 2.3e-3 rms of their size, of which their own rounding is 1.7e-3).  The output is rescaled only
// when a row's maximum grows by more than 2^8.
//
// A unit is two row tiles of a group and a split of the list of keys that
// they see (key_list): tiles of 128 prefix keys, of sinks, of the windows'
// union.  Both row tiles read the same key tiles, but each skips those
// outside its own windows, so that at a window of W keys a row tile computes
// W / 128 + 1 tiles.  A row's own limits are applied to the scores of tiles
// that cross them only.
// Tiles come by TMA from [head, token, D] maps, whose end fills with zeros.
// Rows that no query of the sequence sees (behind its last token, between the
// sinks and its first window) may hold anything, also NaN, which a weight of
// zero would not stop: a tile that holds such rows is copied row by row
// instead, with zeros in their place.  That is one or two tiles of a unit.
// Every mbarrier wait is bounded; on expiry the kernel records an error, stops
// issuing work and releases its TMEM.
#include "cache_unit.cuh"
#include "tc_common.cuh"

namespace area {
namespace {

constexpr int kThreads = 384;
constexpr int kSoftWarp0 = 4;
// Warpgroup 0 gives up registers for the two softmax warpgroups; the split uses
// exactly the allocation of a 168-register launch (checked before it).
constexpr int kRegsLow = 136, kRegsHigh = 184;
static_assert(128 * kRegsLow + 256 * kRegsHigh == kThreads * 168, "register split");
constexpr int kStages = 4;                 // K/V ring, one tile of 128 keys each
constexpr int kRecSlots = 3;               // unit records in flight
constexpr int kPParts = 2;
constexpr int kMaxChains = 8;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D>
struct Geo {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kSmemKV = 2 * kTileBytes;                // after the two query tiles
  static constexpr int kSmemBar = kSmemKV + kStages * kTileBytes;
  static constexpr int kSmemBytes = kSmemBar + 256 + 1024;      // barriers + alignment slack
  static_assert(kSmemBytes + 1024 <= 227 * 1024, "shared memory of one CTA");
};

enum {
  BAR_Q_FULL = 0, BAR_Q_EMPTY,
  BAR_S_FULL0, BAR_S_FULL1,
  BAR_P_FULL0, BAR_P_FULL1,
  BAR_O_FULL0, BAR_O_FULL1,
  BAR_P_PART0, BAR_P_PART1,
  BAR_KV_FULL,
  BAR_KV_EMPTY = BAR_KV_FULL + kStages,
  BAR_REC_FULL = BAR_KV_EMPTY + kStages,
  BAR_REC_EMPTY = BAR_REC_FULL + kRecSlots,
  BAR_DRAIN = BAR_REC_EMPTY + kRecSlots,
  BAR_COUNT
};
static_assert(BAR_COUNT * 8 <= 256, "barrier area");

struct Maps {
  CUtensorMap q, k, v, kp, vp;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache_tc_kernel(const __grid_constant__ Maps tm, const __grid_constant__ UnitParams prm) {
  using G = Geo<D>;
  constexpr uint32_t kIdescPV = idesc(D, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + G::kSmemBar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ __align__(16) Unit s_rec[kRecSlots];
  __shared__ KeySpan s_span[256];          // of the softmax threads' rows
  __shared__ int s_copied[kStages];        // the stage's tile came by cp.async
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s_abort = 0;
    mbar_init(bar(BAR_Q_FULL), 1);
    mbar_init(bar(BAR_Q_EMPTY), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_S_FULL0 + t), 1);
      mbar_init(bar(BAR_P_FULL0 + t), 128);
      mbar_init(bar(BAR_P_PART0 + t), 128);
      mbar_init(bar(BAR_O_FULL0 + t), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(BAR_KV_FULL + s), 1);
      mbar_init(bar(BAR_KV_EMPTY + s), 1);
    }
    for (int s = 0; s < kRecSlots; ++s) {
      mbar_init(bar(BAR_REC_FULL + s), 1);
      mbar_init(bar(BAR_REC_EMPTY + s), 9);   // the MMA thread and the 8 softmax warps
    }
    mbar_init(bar(BAR_DRAIN), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
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

  // The paths must not meet between the split and the roles: the compiler then
  // holds the softmax to the smaller share and spills.
  if (warp < kSoftWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow) : "memory");
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      uint32_t kv_it = 0, unit_count = 0;
      bool ok = true;
      auto publish = [&](uint32_t k) -> bool {
        const uint32_t slot = k % kRecSlots;
        if (!warp_wait0(bar(BAR_REC_EMPTY + slot), ((k / kRecSlots) & 1u) ^ 1u, abort_flag))
          return false;
        if (lane == 0) {
          Unit u;
          u.valid = decode_unit<128>(unit_index(k), prm, u) ? 1 : 0;
          s_rec[slot] = u;
          mbar_arrive(bar(BAR_REC_FULL + slot));
        }
        __syncwarp();
        return true;
      };
      ok = publish(0);
      while (ok) {
        const Unit& u = s_rec[unit_count % kRecSlots];
        if (!u.valid) break;
        if (!(ok = warp_wait0(bar(BAR_Q_EMPTY), (unit_count & 1u) ^ 1u, abort_flag))) break;
        if (lane == 0) {
          const int nq = u.r0[1] < prm.rm.RG ? 2 : 1;
          const uint32_t box = (uint32_t)prm.tile_rows * 128u;    // bytes of a box (64 columns)
          mbar_arrive_tx(bar(BAR_Q_FULL), nq * G::kHalves * box);
          for (int t = 0; t < nq; ++t)
            for (int hf = 0; hf < G::kHalves; ++hf) {
              const uint32_t dst = sbase + t * G::kTileBytes + hf * kHalfBytes;
              if (prm.rm.pool_rows)
                tma_load_3d(dst, &tm.q, bar(BAR_Q_FULL), hf * 64, u.g * prm.rm.pool_rows,
                            u.r0[t] / prm.rm.pool_rows);
              else
                tma_load_3d(dst, &tm.q, bar(BAR_Q_FULL), hf * 64, u.r0[t], u.g);
            }
        }
        __syncwarp();
        const int nt = u.nt;
        const int jn = nt < 2 ? nt : 2;         // the next record is published before tile jn
        bool published = false;
        for (int j = 0; j < nt && ok; ++j) {
          if (j == jn) {
            published = true;
            if (!(ok = publish(unit_count + 1))) break;
          }
          const Tile t = tile_of<128>(u, j);
          for (int kv = 0; kv < 2; ++kv) {       // K then V
            const int s = (int)(kv_it % kStages);
            if (!warp_wait0(bar(BAR_KV_EMPTY + s), ((kv_it / kStages) & 1u) ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t dst = sbase + G::kSmemKV + s * G::kTileBytes;
            const uint32_t full = bar(BAR_KV_FULL + s);
            if (lane == 0) s_copied[s] = t.copy;     // read after the stage's barrier
            if (t.copy) {
              // rows past t.n become zeros and are not read
              const auto* base = static_cast<const __nv_bfloat16*>(kv ? prm.a.v : prm.a.k) +
                                 ((int64_t)u.kvh * prm.a.S + t.j0) * D;
              constexpr int kChunks = D / 8;              // 16-byte pieces of a row
              const int q = lane % kChunks;
  #pragma unroll 8
              for (int r = lane / kChunks; r < 128; r += 32 / kChunks) {
                const uint32_t at = dst + (uint32_t)((q >> 3) * kHalfBytes + r * 128 +
                                                     (((q & 7) ^ (r & 7)) << 4));
                const int rr = r < t.n ? r : 0;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at),
                             "l"(base + (int64_t)rr * D + q * 8), "r"(r < t.n ? 16 : 0)
                             : "memory");
              }
              cp_async_arrive(full);
              __syncwarp();
              if (lane == 0) mbar_arrive(full);
            } else if (lane == 0) {
              mbar_arrive_tx(full, G::kTileBytes);
              const CUtensorMap* map = t.kind ? (kv ? &tm.v : &tm.k) : (kv ? &tm.vp : &tm.kp);
              for (int hf = 0; hf < G::kHalves; ++hf)
                tma_load_3d(dst + hf * kHalfBytes, map, full, hf * 64, t.j0, t.kind ? u.kvh : u.ph);
            }
            __syncwarp();
            ++kv_it;
          }
        }
        if (!ok) break;
        if (!published && !(ok = publish(unit_count + 1))) break;
        ++unit_count;
      }
      // drain: the last load of every stage has landed, no copy is in flight
      int drain_abort = 0;
      for (uint32_t k = 0; k < kStages && k < kv_it; ++k) {
        const uint32_t it = kv_it - 1 - k;
        warp_wait0(bar(BAR_KV_FULL + it % kStages), (it / kStages) & 1u, &drain_abort);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      uint32_t kv_it = 0, unit_count = 0;
      uint32_t p_cnt[2] = {0, 0};
      bool ok = true;
      const uint64_t dq = sdesc(sbase, 16, 1024), dk = sdesc(sbase + G::kSmemKV, 16, 1024);
      const uint64_t dv = sdesc(sbase + G::kSmemKV, kHalfBytes, 1024);
      auto wait_kv = [&](uint32_t it) {
        if (!warp_wait_all(bar(BAR_KV_FULL + it % kStages), (it / kStages) & 1u, abort_flag))
          return false;
        if (s_copied[it % kStages]) fence_proxy_async();
        tc_fence_after();
        return true;
      };
      auto commit = [&](uint32_t b) {
        if (elect_one()) mma_commit(b);
        __syncwarp();
      };
      auto qk = [&](int t, uint32_t it) {
        const uint32_t d = tmem + t * 128, ks = it % kStages * G::kTileBytes;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
            mma_ss(d, sdesc_at(dq, t * G::kTileBytes + off), sdesc_at(dk, ks + off), kIdescQK,
                   kk > 0);
          }
          mma_commit(bar(BAR_S_FULL0 + t));
        }
        __syncwarp();
      };
      auto pv = [&](int t, uint32_t it, bool first, bool last) -> bool {
        const uint32_t d = tmem + 256 + t * 128, p = tmem + t * 128;
        const uint32_t vs = it % kStages * G::kTileBytes;
        constexpr int kPer = 8 / kPParts;
#pragma unroll
        for (int h = 0; h < kPParts; ++h) {
          if (!warp_wait_all(bar((h + 1 < kPParts ? BAR_P_PART0 : BAR_P_FULL0) + t), p_cnt[t] & 1u,
                             abort_flag))
            return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = kPer * h; kk < kPer * h + kPer; ++kk)
              mma_ts(d, p + kk * 8, sdesc_at(dv, vs + kk * 2048), kIdescPV,
                     (first && kk == 0) ? 0u : 1u);
            if (last && h + 1 == kPParts) mma_commit(bar(BAR_O_FULL0 + t));
          }
          __syncwarp();
        }
        ++p_cnt[t];
        return true;
      };
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      while (ok) {
        const uint32_t slot = unit_count % kRecSlots;
        if (!(ok = warp_wait_all(bar(BAR_REC_FULL + slot), (unit_count / kRecSlots) & 1u,
                                 abort_flag)))
          break;
        const Unit& u = s_rec[slot];
        if (!uniform(u.valid)) break;
        const int nt = uniform(u.nt);
        TileRange ar[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const TileRange x = tile_range(u, t);
          ar[t] = TileRange{uniform(x.lead), uniform(x.oa), uniform(x.ob), uniform(x.first),
                            uniform(x.last)};
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_REC_EMPTY + slot));
        __syncwarp();
        if (!(ok = warp_wait_all(bar(BAR_Q_FULL), unit_count & 1u, abort_flag))) break;
        if (nt == 0) commit(bar(BAR_Q_EMPTY));
        if (nt > 0) {
          if (!(ok = wait_kv(kv_it))) break;
          if (ar[0].has(0)) qk(0, kv_it);
          if (ar[1].has(0)) qk(1, kv_it);
          commit(bar(BAR_KV_EMPTY + kv_it % kStages));
          if (nt == 1) commit(bar(BAR_Q_EMPTY));
        }
        // the tiles of the next step are waited for before this step's weights
        // are: their loads are long done, so that no wait comes between a tile's
        // products
        if (nt > 0 && !(ok = wait_kv(kv_it + 1))) break;
        for (int j = 0; j < nt; ++j) {
          const uint32_t vi = kv_it + 2 * j + 1, kn = vi + 1;
          const bool next = j + 1 < nt;
          if (next && !(ok = wait_kv(kn))) break;
          if (ar[0].has(j) && !(ok = pv(0, vi, j == ar[0].first, j == ar[0].last))) break;
          if (next && ar[0].has(j + 1)) qk(0, kn);
          if (ar[1].has(j) && !(ok = pv(1, vi, j == ar[1].first, j == ar[1].last))) break;
          if (next && ar[1].has(j + 1)) qk(1, kn);
          commit(bar(BAR_KV_EMPTY + vi % kStages));
          if (next) {
            commit(bar(BAR_KV_EMPTY + kn % kStages));
            if (j + 2 == nt) commit(bar(BAR_Q_EMPTY));
            if (!(ok = wait_kv(kn + 1))) break;
          }
        }
        kv_it += 2 * nt;
        ++unit_count;
      }
      int drain_abort = 0;
      commit(bar(BAR_DRAIN));
      warp_wait_all(bar(BAR_DRAIN), 0, &drain_abort);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh) : "memory");
    // ------------------------------------------------------ softmax / epilogue
    const int qt = (warp - kSoftWarp0) >> 2;
    const int trow = ((warp & 3) << 5) + lane;       // TMEM lane = row of the tile
    const uint32_t lane_off = (uint32_t)((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + (qt ? 128u : 0u);
    const uint32_t tO = tmem + lane_off + (qt ? 384u : 256u);
    uint32_t s_cnt = 0, o_cnt = 0, unit_count = 0;
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
      const int r = u.r0[qt] + trow;
      const bool rvalid = trow < prm.tile_rows && r < prm.rm.RG;
      // (kept in shared memory: registers are short while a score row is held)
      {
        KeySpan sp{0, INT_MAX};
        if (rvalid) {
          const CacheRow cr = cache_row(prm.a, prm.rm, u.g, r);
          sp = key_span(prm.a, cache_len(prm.a, cr.b), cr.i);
        }
        s_span[qt * 128 + trow] = sp;
      }
      // tiles that every row of the warp sees whole: keys [max lo, min hi)
      const int wlo = __reduce_max_sync(0xffffffffu, s_span[qt * 128 + trow].lo);
      const int whi = __reduce_min_sync(0xffffffffu, s_span[qt * 128 + trow].hi);
      const int first = first_tile(u, qt), last = last_tile(u, qt), lead = u.lead[qt];
      uint32_t whole = 0;                      // of 32 tiles, one bit each
      int at32 = INT_MIN / 2;                  // the first of them
      float m = -INFINITY, l = 0.f;
      RowRef ref{sl2, 0.f};                    // nothing seen so far: all weights 0
      for (int j = first; j <= last;) {
        if (j - at32 >= 32) {
          at32 = j;
          const Tile t = tile_of<128>(u, min(j + lane, u.nt - 1));
          whole = __ballot_sync(0xffffffffu, t.n == 128 && (t.kind == 0 ? !prm.a.causal || whi > 0
                                                                        : whi >= t.j0 + 128 &&
                                             (wlo <= t.j0 || prm.a.sinks >= t.j0 + 128)));
        }
        const bool masked = !(whole >> (j - at32) & 1u);
        if (!(ok = warp_wait_all(bar(BAR_S_FULL0 + qt), s_cnt & 1u, abort_flag))) break;
        ++s_cnt;
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld128(tS, sr);
        if (masked) {
          // keys [ka, kb) and [0, kc) of the tile are this row's
          const Tile t = tile_of<128>(u, j);
          const KeySpan sp = s_span[qt * 128 + trow];
          int ka = 0, kb, kc = 0;
          if (t.kind == 0) {
            kb = sees_prefix(prm.a, sp) ? t.n : 0;
          } else {
            ka = max(sp.lo - t.j0, 0);
            kb = min(sp.hi - t.j0, t.n);
            kc = min(prm.a.sinks - t.j0, kb);
          }
          const unsigned width = kb > ka ? (unsigned)(kb - ka) : 0u;
          if (__any_sync(0xffffffffu, kc > 0)) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if ((unsigned)(i - ka) >= width && i >= kc) sr[i] = 0xff800000u;
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if ((unsigned)(i - ka) >= width) sr[i] = 0xff800000u;        // -inf: no weight
          }
        }
        float pm[kMaxChains];
#pragma unroll
        for (int t = 0; t < kMaxChains; ++t) pm[t] = __uint_as_float(sr[t]);
#pragma unroll
        for (int i = kMaxChains; i < 128; i += 2)
          pm[(i >> 1) % kMaxChains] = max3(pm[(i >> 1) % kMaxChains],
                                           __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
#pragma unroll
        for (int t = kMaxChains / 2; t > 0; t >>= 1)
#pragma unroll
          for (int q = 0; q < t; ++q) pm[q] = fmaxf(pm[q], pm[q + t]);
        const float mnew = fmaxf(pm[0] * sl2, m);
        // rows that do not exist hold what the tile last held: they have no say, or
        // the real rows' rounding would hang on it
        const bool rescale =
            j > first && __any_sync(0xffffffffu, rvalid && mnew > m + kRescaleThreshold);
        const float alpha = rescale ? (m == -INFINITY ? 0.f : fast_exp2(m - mnew)) : 1.f;
        if (j == first || rescale) {
          if (mnew > m) ref = row_ref(pm[0], mnew, sl2);
          m = mnew;
        }
        l *= alpha;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < kPParts; ++h) {
          constexpr int kKeys = 128 / kPParts;
#pragma unroll
          for (int i = kKeys * h; i < kKeys * h + kKeys; i += 2) {
            float x0, x1;
            fma2(x0, x1, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]), ref.mul, ref.add);
            const float p0 = fast_exp2(x0);
            const float p1 = fast_exp2(x1);
            if ((i >> 1) & 1) add2(ls[2], ls[3], p0, p1); else add2(ls[0], ls[1], p0, p1);
            sr[i >> 1] = pack_bf16(p0, p1);
          }
          if (h == 0 && rescale) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t orr[32];
              tmem_ld32(tO + c * 32, orr);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
              tmem_st32(tO + c * 32, orr);
            }
          }
          tmem_st32(tS + 32 * h, *reinterpret_cast<const uint32_t(*)[32]>(&sr[32 * h]));
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar((h + 1 < kPParts ? BAR_P_PART0 : BAR_P_FULL0) + qt));
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        j = next_tile(j, lead, u.oa[qt]);
      }
      if (!ok) break;
      // ---- epilogue
      const int64_t row = rvalid ? cache_row(prm.a, prm.rm, u.g, r).row : 0;
      const int64_t at = (int64_t)(prm.out.slot0 + u.sp) * prm.out.rows + row;
      if (last >= 0) {
        if (!(ok = warp_wait_all(bar(BAR_O_FULL0 + qt), o_cnt & 1u, abort_flag))) break;
        ++o_cnt;
        tc_fence_after();
      }
      if (!prm.out.direct && rvalid) prm.out.part_ml[at] = make_float2(m, l);
      if (prm.out.lse && rvalid) prm.out.lse[row] = l == 0.f ? INFINITY : m + log2f(l);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (prm.out.direct || last >= 0) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orr[32];
          if (last >= 0) {
            tmem_ld32(tO + c * 32, orr);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) orr[i] = 0;
          }
          if (!rvalid) continue;
          if (prm.out.direct) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(prm.a.o) + row * D + c * 32;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                w[i] = l == 0.f ? 0u
                                : pack_bf16(__uint_as_float(orr[16 * h + 2 * i]) * inv,
                                            __uint_as_float(orr[16 * h + 2 * i + 1]) * inv);
              st_global_v8(dst + h * 16, w);
            }
          } else {
            float* dst = prm.out.part_o + at * D + c * 32;
#pragma unroll
            for (int h = 0; h < 4; ++h)
              st_global_v8f(dst + 8 * h, reinterpret_cast<const float*>(orr) + 8 * h);
          }
        }
      }
      tc_fence_before();
      if (lane == 0) mbar_arrive(bar(BAR_REC_EMPTY + slot));
      ++unit_count;
    }
  }
  let_next_start();
  if (prm.out.early) wait_for_last();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D>
cudaError_t launch(const Maps& maps, const UnitParams& prm, cudaStream_t s) {
  auto fn = cache_tc_kernel<D>;
  constexpr int kSmem = Geo<D>::kSmemBytes;
  // setmaxnreg.inc waits until the registers it asks for are free, so the split
  // must fit in what the launch allocates
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, fn);
  if (e != cudaSuccess) return e;
  if (kThreads * (fa.numRegs / 8 * 8) < 128 * kRegsLow + 256 * kRegsHigh)
    return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(prm.units, num_sms());
  return launch_kernel(fn, grid, kThreads, kSmem, 1, prm.out.early, s, maps, prm);
}

}  // namespace

cudaError_t read_and_clear_cache_tc_error(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(code, g_tc_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_tc_error, &zero, sizeof(int));
}

cudaError_t launch_cache_tc(const CacheArgs& a, const CacheRows& rm, const CacheOut& out,
                            cudaStream_t s) {
  Maps m;
  cudaError_t e;
  UnitParams p{a, rm, out, 0, tc_tile_rows(rm), 2, 0, 0};
  if (rm.pool_rows)
    e = make_map3(&m.q, a.q, a.B, (int64_t)a.Hk * rm.pool_rows, a.D, rm.pool_rows,
                  p.tile_rows / rm.pool_rows);
  else
    e = make_map3(&m.q, a.q, rm.groups, rm.RG, a.D, 128, 1);
  if (e != cudaSuccess) return e;
  if (rm.use_own && a.S > 0) {
    if ((e = make_map3(&m.k, a.k, (int64_t)a.B * a.Hk, a.S, a.D, 128, 1)) != cudaSuccess) return e;
    if ((e = make_map3(&m.v, a.v, (int64_t)a.B * a.Hk, a.S, a.D, 128, 1)) != cudaSuccess) return e;
  } else {
    m.k = m.v = m.q;      // never read
  }
  if (rm.use_prefix) {
    if ((e = make_map3(&m.kp, a.kp, a.Hk, a.P, a.D, 128, 1)) != cudaSuccess) return e;
    if ((e = make_map3(&m.vp, a.vp, a.Hk, a.P, a.D, 128, 1)) != cudaSuccess) return e;
  } else {
    m.kp = m.vp = m.q;    // never read
  }
  p.nrb = (rm.RG + 2 * p.tile_rows - 1) / (2 * p.tile_rows);
  p.units = (int)((int64_t)rm.groups * p.nrb * out.nsplit);
  // Causal units cost what they see: the last row tiles go first, over all groups,
  // so that the blocks come out even (a prompt of 8192 tokens, window 2048, 5.2
  // units to a block: 214 us in short runs, group by group 260).  The units at work have as many
  // keys between them either way: 96 groups of 16384 tokens 1.77-1.85 ms, group by
  // group 1.63-1.89.  Other units cost the same; a group's row tiles follow one
  // another.
  p.heavy_first = a.causal && !rm.pool_rows;
  // A last round that would leave half the SMs or more idle: its units one row tile at
  // a time, two thirds of the time (24 heads of 512 tokens: 19.5 -> 16.5 us; where half
  // the SMs do not suffice, 8 heads of 2048: 37 -> 49).  Causal units end with the
  // lightest anyway.
  const int sms = num_sms(), rest = p.units % sms;
  if (rm.RG > p.tile_rows && 2 * rest <= sms && (!p.heavy_first || p.units < sms)) {
    p.halved = rest;
    p.units += rest;
  }
  if (a.D == 64) return launch<64>(m, p, s);
  return launch<128>(m, p, s);
}

}  // namespace area
