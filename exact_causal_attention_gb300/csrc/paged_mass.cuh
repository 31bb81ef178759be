// Attention weight that every cached token received from a ragged chunk:
//   mass[b, kvh, j] (+)= sum over rows r of b and heads h of kvh of e^(s(r, h, j) - lse[r, h]).
//
// The sum runs over the rows, so the product is taken the other way round: S^T = K Q^T with a tile of
// 128 keys as the rows (a key is a TMEM lane, one thread sums its row without shuffles or atomics) and
// a step of up to 128 (row, head) pairs as the columns.  K is read once, V not at all.
// For one decode step a key tile meets one step of g columns and the kernel is bound by reading K;
// for a chunk it is bound by the exponentials, one per (pair, key).
//
// A CTA takes an equal part of the line of units (paged_plan.cuh): two consecutive key tiles of one
// (request, head), one per slot, with the heads of a pair of tiles side by side, as they lie in
// memory (a token's heads are contiguous): 16-token pages then cost a decode step at 32K 90 us, 64-token
// pages 85, the floor of reading K once being 71.  The queries' steps stream through a ring that both slots share.
// Warps: 4 per slot that sum (8 where a step has more than 64 columns: the first four then take
// columns 0-63, the others 64-127), and four more: one produces key tiles from their pages, one issues
// the MMAs, one loads Q, one the columns' log-sum-exps (and slopes and positions).  With 4 per slot the
// sums wait for latencies, two warps per scheduler keeping the exponential unit at half its rate (500
// tokens, 12000 keys, one capped request: 102 us, with 8 warps 86); where a step has few columns more warps only take
// issue slots from the producer (a decode step at 32K: 90 us, with 8 warps 100).  S^T is double-buffered
// per slot, so the next product does not wait for the sums.
//
// e^(s - lse) is taken as 2^(log2e (s - lse)) with the difference formed first in natural units: where
// the weight matters s is near lse, so the one rounding of the difference is small.  (In base 2 from the
// start the rounding of lse and of the cap would each cost 1e-6 of the weights.)
#pragma once
#include <cuda.h>

#include "attn_fwd_kernel.cuh"
#include "paged_form.cuh"
#include "paged_plan.cuh"

namespace eca {

template <int kParts>
constexpr int kMsThreads = 32 * (8 * kParts + 4);
constexpr int kMsTile = 128;       // keys per tile
constexpr int kMsCols = 128;       // most columns of a step
constexpr int kMsPairCost = 2;     // a pair of key tiles' own cost, in steps
constexpr int kMsQueue = 4;
constexpr int kMsColStages = 4;    // ring of the columns' values
// Per key tile, which of its pages have a bad id.  The sums may trail the products by two steps
// (four tiles), and the producer runs ahead of those by the ring.
constexpr int kMsBadRing = 32;

struct MassParams {
  ChunkShape s;
  ScoreForm f;
  const float* lse;   // [total, Hq]
  float* mass;        // [B, Hkv, max_pages * page_size]
  int accumulate;
  int Hq;
  int hc, chunks;     // query heads per step, and chunks of the group
  int tq;             // tokens per step
  int small_plan;     // the line is laid out by one warp
  uint32_t idesc;     // of the MMA: 128 x (hc tq rounded up to 16)
  FastDiv by_hc, by_tq;
  unsigned long long wait_limit_ns;
  int timeout_code;
};

template <int D>
struct MassSmem {
  static constexpr int kSub = D / 64;
  static constexpr int kTileBytes = kSub * kSubTileBytes;
  static constexpr int kKStages = D == 128 ? 4 : 6;
  static constexpr int kQStages = D == 128 ? 2 : 4;
  static constexpr int kKOff = 0;
  static constexpr int kQOff = kKStages * kTileBytes;
  static constexpr int kColOff = kQOff + kQStages * kTileBytes;  // fp32 [stages][3][128]: - lse, slope, position
  static constexpr int kColBytes = 3 * kMsCols * 4;
  static constexpr int kBarOff = kColOff + kMsColStages * kColBytes;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kKStages;
  static constexpr int kBarQFull = kBarKEmpty + kKStages;
  static constexpr int kBarQEmpty = kBarQFull + kQStages;
  static constexpr int kBarColFull = kBarQEmpty + kQStages;
  static constexpr int kBarColEmpty = kBarColFull + kMsColStages;
  static constexpr int kBarS = kBarColEmpty + kMsColStages;  // + 2 slot + buffer
  static constexpr int kBarSFree = kBarS + 4;                // + 2 slot + buffer
  static constexpr int kBarUnitFull = kBarSFree + 4;
  static constexpr int kBarUnitFree = kBarUnitFull + kMsQueue;
  static constexpr int kBarDrain = kBarUnitFree + kMsQueue;
  static constexpr int kBarSumFull = kBarDrain + 1;    // + 2 slot + unit parity: the second half's sums
  static constexpr int kBarSumFree = kBarSumFull + 4;  // + 2 slot + unit parity
  static constexpr int kNumBars = kBarSumFree + 4;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kBadOff = kMiscOff + 8;
  static constexpr int kQueueOff = (kBadOff + 4 * kMsBadRing + 15) & ~15;
  static constexpr int kEntryInts = 16;
  static constexpr int kScanOff = kQueueOff + kMsQueue * kEntryInts * 4;
  static constexpr int kSumOff = kScanOff + 24 * 8;  // fp32 [slot][unit parity][128]
  static constexpr int kBytes = kSumOff + 4 * kMsTile * 4;
  static constexpr int kDynamicBytes = kBytes + 1024;
  static_assert(kLineTableBytes <= kColOff, "the plan's tables fit over the rings");
  static_assert(kDynamicBytes <= 227 * 1024, "shared memory exceeds the per-block limit");
};

// Steps (query tiles of tq tokens) that see a key of tile kt: q0 .. q1 - 1.
struct TileSteps {
  int q0, q1;
};
__device__ __forceinline__ TileSteps tile_steps(const MassParams& p, int n, int pos0, int prefix, int len, int kt) {
  const int kb = kt * kMsTile;
  if (kb >= len || n == 0) return TileSteps{0, 0};
  if (kb < prefix) return TileSteps{0, fast_div(n - 1, p.by_tq) + 1};
  const int lo = max(0, kb - pos0);
  const int hi = p.f.window > 0 ? static_cast<int>(min(static_cast<long long>(n),
                                                       static_cast<long long>(kb) + kMsTile - 1 + p.f.window - pos0))
                                : n;
  if (lo >= hi) return TileSteps{0, 0};
  return TileSteps{fast_div(lo, p.by_tq), fast_div(hi - 1, p.by_tq) + 1};
}

// Two key tiles (or one) of one (request, head).
struct MassUnit {
  int steps;     // query tiles per chunk of heads; -1 past the last unit
  int q0;        // first of them
  int kt;        // key tile of slot 0; slot 1 has the next one
  int two;       // slot 1 has one
  int row0, n, pos0, len, prefix;
  int kvh, b;
};

// kParts: the warp groups that share a step's columns.
template <int D, bool BF16, int FORM, int kParts>
__global__ void __launch_bounds__(kMsThreads<kParts>, 1)
    paged_mass_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_cache,
                      const MassParams p) {
  using L = MassSmem<D>;
  constexpr int kProducer = 8 * kParts, kIssuer = kProducer + 1, kQLoader = kProducer + 2, kColumns = kProducer + 3;
  constexpr int kReaders = kProducer + 3;  // of a unit: every warp but the producer
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_base);
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBarOff + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile uint32_t* bad_pages = reinterpret_cast<volatile uint32_t*>(smem + L::kBadOff);
  volatile int* queue = reinterpret_cast<volatile int*>(smem + L::kQueueOff);
  float* cols_s = reinterpret_cast<float*>(smem + L::kColOff);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bar(L::kBarKFull + s), 1);
      mbar_init(bar(L::kBarKEmpty + s), 1);
    }
    for (int s = 0; s < L::kQStages; ++s) {
      mbar_init(bar(L::kBarQFull + s), 1);
      mbar_init(bar(L::kBarQEmpty + s), 1);
    }
    for (int s = 0; s < kMsColStages; ++s) {
      mbar_init(bar(L::kBarColFull + s), 1);
      mbar_init(bar(L::kBarColEmpty + s), 8 * kParts);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(L::kBarS + s), 1);
      mbar_init(bar(L::kBarSFree + s), 4 * kParts);
      mbar_init(bar(L::kBarSumFull + s), 4);
      mbar_init(bar(L::kBarSumFree + s), 4);
    }
    for (int q = 0; q < kMsQueue; ++q) {
      mbar_init(bar(L::kBarUnitFull + q), 1);
      mbar_init(bar(L::kBarUnitFree + q), kReaders);
    }
    mbar_init(bar(L::kBarDrain), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) tma_prefetch_map(&tm_cache);
  if (warp == kQLoader && lane == 0) tma_prefetch_map(&tm_q);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_launch_dependents();
  grid_dependency_wait();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Watchdog wd{abort_flag, p.s.status, p.wait_limit_ns, p.timeout_code};

  // ------------------------------------------------------------------------ plan
  const int B = p.s.B;
  const int most = p.s.max_pages * p.s.page_size;
  const LineTables line = line_tables(smem, reinterpret_cast<long long*>(smem + L::kScanOff));
  // Items are pairs of key tiles; written in full, a pair that no row sees is one too.
  auto items_of = [&](int n, int len) {
    return ((p.accumulate ? (n > 0 ? len : 0) : most) + 2 * kMsTile - 1) / (2 * kMsTile);
  };
  auto items = [&](const int4& r) { return items_of(r.x, r.w); };
  auto steps_of = [&](int n, int pos0, int prefix, int len, int pair) -> TileSteps {
    const TileSteps a = tile_steps(p, n, pos0, prefix, len, 2 * pair), b = tile_steps(p, n, pos0, prefix, len, 2 * pair + 1);
    if (a.q1 == 0) return b;
    if (b.q1 == 0) return a;
    return TileSteps{min(a.q0, b.q0), max(a.q1, b.q1)};
  };
  auto cost = [&](const int4& r, int i) {
    const TileSteps t = steps_of(r.x, r.y, r.z, r.w, i);
    return t.q1 > t.q0 ? kMsPairCost + (t.q1 - t.q0) * p.chunks : 1;
  };
  // Only the producer needs the plan; a long one is laid out by the whole block.
  long long W = 0;
  if (!p.small_plan) {
    W = line_build<kMsThreads<kParts>>(line, p.s, p.f, p.s.Hkv, items, cost);
  } else if (warp == kProducer) {
    W = line_build_warp(line, p.s, p.f, p.s.Hkv, items, cost);
  }
  const int cta = static_cast<int>(blockIdx.x), G = static_cast<int>(gridDim.x);
  struct Place {
    int b, pair, head;
  };
  // Whole units: a place past a unit's middle cuts behind it.
  auto locate = [&](long long x) -> Place {
    const LinePlace at = line_locate<true>(line, B, p.s.Hkv, W, x, cost);
    Place r{at.b, at.item, at.head + (2 * at.in >= at.cost ? 1 : 0)};
    if (r.head == p.s.Hkv) {  // (the pair may then be one past the request's last)
      r.head = 0;
      ++r.pair;
    }
    return r;
  };
  Place from = {B, 0, 0}, to = {B, 0, 0};
  if (warp == kProducer && W > 0) {
    from = locate(line_cut(W, G, cta));
    if (cta + 1 < G) to = locate(line_cut(W, G, cta + 1));
  }
  // The plan's reads and writes come before the rings' copies and the columns' values.
  fence_proxy_async_smem();
  __syncthreads();

  int units_read = 0;
  auto next_unit = [&](MassUnit& w, bool whole_warp) -> bool {
    const int q = units_read % kMsQueue;
    bool got = wd.wait(bar(L::kBarUnitFull + q), parity(units_read / kMsQueue));
    if (whole_warp) got = __all_sync(0xffffffffu, got) != 0;
    if (!got) return false;
    volatile int* e = queue + q * L::kEntryInts;
    int v[11];
#pragma unroll
    for (int i = 0; i < 11; ++i) v[i] = e[i];
    if (whole_warp) {
#pragma unroll
      for (int i = 0; i < 11; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
    }
    w = MassUnit{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10]};
    if (lane == 0) mbar_arrive(bar(L::kBarUnitFree + q));
    ++units_read;
    return true;
  };

  if (warp == kProducer) {
    // ------------------------------------------------------------ key tiles, from pages
    const int T = p.s.page_size;
    const int log2T = 31 - __clz(T);
    const int pages = kMsTile >> log2T;
    // A key tile meets all its queries in one unit, so K is read once.
    const uint64_t pol = policy_evict_first();
    int it = 0, pushed = 0;
    bool ok = true;
    PageWalk walk;
    walk.step = 1;
    walk.log2T = log2T;
    walk.num_pages = p.s.num_pages;
    int b = from.b, pair = from.pair, head = from.head;
    while (ok && b < B && b <= to.b) {
      const Request r = load_request(p.s, &p.f, b);
      const int n_items = items_of(r.n, r.len);
      // The window reaches down to the first token's.
      walk.from0 = p.f.window > 0 ? max(0, r.pos0 - p.f.window + 1) : 0;
      walk.to0 = r.len;
      walk.prefix = r.prefix;
      if (pair < n_items) walk.start(p.s.block_table + static_cast<size_t>(b) * p.s.max_pages, 2 * pair * pages >> 5);
      for (; ok && pair < n_items; ++pair, head = 0) {
        const bool last = b == to.b && pair == to.pair;
        const int stop = last ? to.head : p.s.Hkv;
        const TileSteps t = steps_of(r.n, r.pos0, r.prefix, r.len, pair);
        const bool seen = t.q1 > t.q0;
        // A slot without keys in the context takes no part.
        const bool two = (2 * pair + 1) * kMsTile < (seen ? r.len : most);
        for (; ok && head < stop; ++head) {
          const int q = pushed % kMsQueue;
          if (!__all_sync(0xffffffffu, wd.wait(bar(L::kBarUnitFree + q), parity(pushed / kMsQueue) ^ 1u))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            volatile int* e = queue + q * L::kEntryInts;
            e[0] = seen ? t.q1 - t.q0 : 0;
            e[1] = t.q0;
            e[2] = 2 * pair;
            e[3] = two;
            e[4] = r.row0;
            e[5] = r.n;
            e[6] = r.pos0;
            e[7] = r.len;
            e[8] = r.prefix;
            e[9] = head;
            e[10] = b;
            mbar_arrive(bar(L::kBarUnitFull + q));
          }
          ++pushed;
          for (int x = 0; seen && x < (two ? 2 : 1); ++x) {
            const int at = walk.hold((2 * pair + x) * pages, p.s.status, p.s.bad_index_code);
            const int slot = it % L::kKStages;
            if (!__all_sync(0xffffffffu, wd.wait(bar(L::kBarKEmpty + slot), parity(it / L::kKStages) ^ 1u))) {
              ok = false;
              break;
            }
            const uint32_t full = bar(L::kBarKFull + slot);
            if (lane == 0) {
              bad_pages[it % kMsBadRing] = (walk.bad >> at) & ((1u << pages) - 1u);
              mbar_arrive_expect_tx(full, L::kTileBytes);
            }
            __syncwarp();
            uint32_t dst = sbase + L::kKOff + slot * L::kTileBytes;
#pragma unroll 2
            for (int i = 0; i < pages; ++i, dst += T * 2 * D) {
              tma_load_page(dst, &tm_cache, full, __shfl_sync(0xffffffffu, walk.z, at + i), head, pol);
            }
            ++it;
          }
        }
        if (last) {
          b = B;  // done
          break;
        }
      }
      ++b;
      pair = head = 0;
    }
    if (ok) {
      const int q = pushed % kMsQueue;
      if (__all_sync(0xffffffffu, wd.wait(bar(L::kBarUnitFree + q), parity(pushed / kMsQueue) ^ 1u)) && lane == 0) {
        queue[q * L::kEntryInts] = -1;
        mbar_arrive(bar(L::kBarUnitFull + q));
      }
    }
    for (int x = (it > L::kKStages ? it - L::kKStages : 0); x < it; ++x) {
      wd.drain(bar(L::kBarKFull + x % L::kKStages), parity(x / L::kKStages));
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------------ MMA issuer
    const uint64_t k_desc = TileLayout<D>::k_desc(sbase + L::kKOff);
    const uint64_t q_desc = smem_desc_sw128(sbase + L::kQOff, 16, 1024);
    auto warp_wait = [&](uint32_t b, uint32_t ph) -> bool { return __all_sync(0xffffffffu, wd.wait(b, ph)) != 0; };
    int it = 0, step = 0;
    int uses[2] = {0, 0};  // steps of each slot so far
    bool ok = true;
    MassUnit w;
    while (ok) {
      if (!next_unit(w, true) || w.steps < 0) break;
      if (w.steps == 0) continue;
      const int tiles = 1 + w.two;
      for (int x = 0; ok && x < tiles; ++x) {
        const int item = it + x;
        ok = warp_wait(bar(L::kBarKFull + item % L::kKStages), parity(item / L::kKStages));
      }
      if (!ok) break;
      const int n = w.steps * p.chunks;
      for (int i = 0; i < n; ++i, ++step) {
        const int qs = step % L::kQStages;
        if (!warp_wait(bar(L::kBarQFull + qs), parity(step / L::kQStages))) {
          ok = false;
          break;
        }
        for (int x = 0; x < tiles; ++x) {
          const int buf = uses[x] & 1;
          if (!warp_wait(bar(L::kBarSFree + 2 * x + buf), parity(uses[x] / 2) ^ 1u)) {
            ok = false;
            break;
          }
          ++uses[x];
          tc_fence_after_sync();
          const uint64_t a = k_desc + static_cast<uint64_t>(((it + x) % L::kKStages) * (L::kTileBytes >> 4));
          const uint64_t bq = q_desc + static_cast<uint64_t>(qs * (L::kTileBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            mma_ss_warp(tmem + 256u * x + 128u * buf, a + TileLayout<D>::k_step(kk),
                        bq + static_cast<uint64_t>((kk / 4) * (kSubTileBytes >> 4) + (kk % 4) * 2), p.idesc,
                        kk > 0 ? 1u : 0u);
          }
          tc_commit_warp(bar(L::kBarS + 2 * x + buf));
        }
        if (!ok) break;
        tc_commit_warp(bar(L::kBarQEmpty + qs));
      }
      for (int x = 0; ok && x < tiles; ++x) tc_commit_warp(bar(L::kBarKEmpty + (it + x) % L::kKStages));
      it += tiles;
    }
    tc_commit_warp(bar(L::kBarDrain));
    wd.drain(bar(L::kBarDrain), 0);
  } else if (warp == kQLoader) {
    // --------------------------------------------------------------------- Q loader
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();  // every key tile of the request meets these rows
      const uint32_t bytes = static_cast<uint32_t>(L::kSub * p.hc * p.tq * 128);
      int step = 0;
      bool ok = true;
      MassUnit w;
      while (ok && next_unit(w, false) && w.steps >= 0) {
        for (int i = 0; i < w.steps * p.chunks; ++i, ++step) {
          const int qs = step % L::kQStages;
          if (!wd.wait(bar(L::kBarQEmpty + qs), parity(step / L::kQStages) ^ 1u)) {
            ok = false;
            break;
          }
          const int chunk = i / w.steps, qt = w.q0 + i % w.steps;
          mbar_arrive_expect_tx(bar(L::kBarQFull + qs), bytes);
          for (int s = 0; s < L::kSub; ++s) {
            tma_load_3d(sbase + L::kQOff + qs * L::kTileBytes + s * kSubTileBytes, &tm_q, bar(L::kBarQFull + qs), 64 * s,
                        (w.kvh * p.chunks + chunk) * p.hc, w.row0 + qt * p.tq, pol);
          }
        }
      }
      for (int x = (step > L::kQStages ? step - L::kQStages : 0); x < step; ++x) {
        wd.drain(bar(L::kBarQFull + x % L::kQStages), parity(x / L::kQStages));
      }
    }
  } else if (warp == kColumns) {
    // ------------------------------------------------- the columns' values, lane by column
    // (times the power of two that capped scores come with)
    const float big = form_caps(FORM) ? cap_scale(p.f.scale, p.f.softcap, 1.f).big : 1.f;
    int tok[4], head[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tok[i] = fast_div(lane + 32 * i, p.by_hc);
      head[i] = lane + 32 * i - tok[i] * p.hc;
    }
    int step = 0;
    bool ok = true;
    MassUnit w;
    while (ok && next_unit(w, true) && w.steps >= 0) {
      const int n = w.steps * p.chunks;
      float next[4];
      // Minus the log-sum-exp; minus infinity (no weight) for a column of no row and for a row that saw no key.
      auto load = [&](int i) {
        const int chunk = i / w.steps, t0 = (w.q0 + i % w.steps) * p.tq;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          next[c] = -INFINITY;
          if (tok[c] < p.tq && t0 + tok[c] < w.n) {
            const float z = p.lse[static_cast<size_t>(w.row0 + t0 + tok[c]) * p.Hq + (w.kvh * p.chunks + chunk) * p.hc + head[c]];
            next[c] = z == -INFINITY ? z : -z * big;
          }
        }
      };
      if (n > 0) load(0);
      for (int i = 0; i < n; ++i, ++step) {
        const int cs = step % kMsColStages;
        float now[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) now[c] = next[c];
        const int chunk = i / w.steps, t0 = (w.q0 + i % w.steps) * p.tq;
        if (i + 1 < n) load(i + 1);
        if (!__all_sync(0xffffffffu, wd.wait(bar(L::kBarColEmpty + cs), parity(step / kMsColStages) ^ 1u))) {
          ok = false;
          break;
        }
        float* dst = cols_s + cs * 3 * kMsCols;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          dst[lane + 32 * c] = now[c];
          if constexpr (form_biases(FORM)) {
            dst[kMsCols + lane + 32 * c] = big * p.f.slopes[(w.kvh * p.chunks + chunk) * p.hc + head[c]];
            dst[2 * kMsCols + lane + 32 * c] = static_cast<float>(w.pos0 + t0 + tok[c]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarColFull + cs));
      }
    }
  } else {
    // -------------------------------------------------------------------------- sums
    const int x = warp / (4 * kParts);     // slot
    const int half = (warp / 4) % kParts;  // columns 64 half .. of every step
    const int r_local = (warp % 4) * 32 + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16) + 256u * x;
    const int log2T = 31 - __clz(p.s.page_size);
    auto warp_wait = [&](uint32_t b, uint32_t ph) -> bool { return __all_sync(0xffffffffu, wd.wait(b, ph)) != 0; };
    const CapScale cap = cap_scale(p.f.scale, p.f.softcap, 1.f);
    const float to_base2 = form_caps(FORM) ? kLog2e * cap.inv_big : kLog2e;
    float* sums_s = reinterpret_cast<float*>(smem + L::kSumOff) + 2 * x * kMsTile;
    int it = 0, step = 0, uses = 0;
    int joined = 0;  // units of this slot whose halves were joined
    bool ok = true;
    MassUnit w;
    while (ok) {
      if (!next_unit(w, true) || w.steps < 0) break;
      const int n = w.steps * p.chunks;
      const int item = it + x;
      if (n > 0) it += 1 + w.two;
      const int key = (w.kt + x) * kMsTile + r_local;
      if (x > w.two) {
        // No tile for this slot: it still hands the steps' columns back.
        for (int i = 0; i < n; ++i, ++step) {
          const int cs = step % kMsColStages;
          if (!warp_wait(bar(L::kBarColFull + cs), parity(step / kMsColStages))) {
            ok = false;
            break;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kBarColEmpty + cs));
        }
        if (ok && !p.accumulate && half == 0 && key < most) {
          p.mass[(static_cast<size_t>(w.b) * p.s.Hkv + w.kvh) * most + key] = 0.f;  // past the context
        }
        continue;
      }
      const float key_f = static_cast<float>(key);
      // Tokens that see this key: from .. upto - 1 of the request.
      int from_tok = max(0, key - w.pos0), upto = w.n;
      if (key < w.prefix) {
        from_tok = 0;
      } else if (key >= w.len) {
        upto = 0;
      } else if (p.f.window > 0) {
        upto = static_cast<int>(min(static_cast<long long>(w.n), static_cast<long long>(key) + p.f.window - w.pos0));
      }
      float2 acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.f, 0.f);
      uint32_t bad = 0;
      for (int i = 0; i < n; ++i, ++step) {
        const int t0 = (w.q0 + (p.chunks == 1 ? i : i % w.steps)) * p.tq;
        const int cols = min(p.tq, w.n - t0) * p.hc;
        // Columns of this step that see this key.
        const int lo = (max(from_tok, t0) - t0) * p.hc, hi = min(cols, (min(upto, t0 + p.tq) - t0) * p.hc);
        const int buf = uses & 1;
        const uint32_t t_b = t_s + 128u * buf;
        if (!warp_wait(bar(L::kBarS + 2 * x + buf), parity(uses / 2))) {
          ok = false;
          break;
        }
        ++uses;
        tc_fence_after_sync();
        if (i == 0) bad = bad_pages[item % kMsBadRing];
        const int cs = step % kMsColStages;
        if (!warp_wait(bar(L::kBarColFull + cs), parity(step / kMsColStages))) {
          ok = false;
          break;
        }
        const float* col = cols_s + cs * 3 * kMsCols;
        // Sums 32 columns: 2^(log2e (form(s) - lse)).
        auto add = [&](uint32_t (&v)[32], int q) {
          if constexpr (form_caps(FORM)) cap_scores<true, true>(v, cap, col + 32 * q);
          const float2 c2 = make_float2(p.f.scale, p.f.scale), k2 = make_float2(to_base2, to_base2);
          const bool all = __all_sync(0xffffffffu, lo <= 32 * q && hi >= 32 * q + 32) != 0;
          auto low = [](int m) -> uint32_t { return m <= 0 ? 0u : (m >= 32 ? ~0u : (1u << m) - 1u); };
          const uint32_t seen = low(hi - 32 * q) & ~low(lo - 32 * q);
#pragma unroll
          for (int i4 = 0; i4 < 32; i4 += 4) {
            float2 y0 = make_float2(__uint_as_float(v[i4]), __uint_as_float(v[i4 + 1]));
            float2 y1 = make_float2(__uint_as_float(v[i4 + 2]), __uint_as_float(v[i4 + 3]));
            if constexpr (!form_caps(FORM)) {
              const float4 z = *reinterpret_cast<const float4*>(col + 32 * q + i4);  // - lse
              y0 = __ffma2_rn(y0, c2, make_float2(z.x, z.y));
              y1 = __ffma2_rn(y1, c2, make_float2(z.z, z.w));
            }
            if constexpr (form_biases(FORM)) {
              const float4 sl = *reinterpret_cast<const float4*>(col + kMsCols + 32 * q + i4);
              const float4 ps = *reinterpret_cast<const float4*>(col + 2 * kMsCols + 32 * q + i4);
              y0.x = fmaf(-sl.x, fabsf(ps.x - key_f), y0.x);
              y0.y = fmaf(-sl.y, fabsf(ps.y - key_f), y0.y);
              y1.x = fmaf(-sl.z, fabsf(ps.z - key_f), y1.x);
              y1.y = fmaf(-sl.w, fabsf(ps.w - key_f), y1.y);
            }
            y0 = __fmul2_rn(y0, k2);
            y1 = __fmul2_rn(y1, k2);
            v[i4] = __float_as_uint(ex2(y0.x));
            v[i4 + 1] = __float_as_uint(ex2(y0.y));
            v[i4 + 2] = __float_as_uint(ex2(y1.x));
            v[i4 + 3] = __float_as_uint(ex2(y1.y));
          }
          if (!all) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(seen & (1u << e))) v[e] = 0u;
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            acc[(e / 2) % 4] = __fadd2_rn(acc[(e / 2) % 4], make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
          }
        };
        // S is free for the next product but one once this part's columns are in registers.
        constexpr int kQuarters = 2;  // (one part has 64 columns at most)
#pragma unroll 1
        for (int q = kQuarters * half; q < kQuarters * (half + 1); ++q) {
          uint32_t s[32];
          if (32 * q < cols) {
            tmem_ld_x32(t_b + 32u * q, s);
            tmem_wait_ld_x32(s);
          }
          if (q == kQuarters * (half + 1) - 1) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kBarSFree + 2 * x + buf));
          }
          if (32 * q < cols) add(s, q);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarColEmpty + cs));
      }
      if (!ok) break;
      const float2 both = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      float sum = both.x + both.y;
      if (kParts == 2 && n > 0) {
        // The second half hands its sums to the first, in one of two buffers.
        const int j = joined % 2;
        const uint32_t full = bar(L::kBarSumFull + 2 * x + j), free = bar(L::kBarSumFree + 2 * x + j);
        if (half == 1) {
          if (!warp_wait(free, parity(joined / 2) ^ 1u)) break;
          sums_s[j * kMsTile + r_local] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        } else {
          if (!warp_wait(full, parity(joined / 2))) break;
          sum += sums_s[j * kMsTile + r_local];
          __syncwarp();
          if (lane == 0) mbar_arrive(free);
        }
        ++joined;
      }
      if (half == 0 && key < most && (n > 0 || !p.accumulate)) {
        if (((bad >> (r_local >> log2T)) & 1u) != 0) sum = 0.f;
        float* dst = p.mass + (static_cast<size_t>(w.b) * p.s.Hkv + w.kvh) * most + key;
        *dst = p.accumulate ? *dst + sum : sum;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace eca
