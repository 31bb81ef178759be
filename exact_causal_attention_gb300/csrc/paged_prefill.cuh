// Attention of a ragged chunk of new tokens over a paged cache, with the score forms of
// include/attn_cache.h, on the tensor cores.
//
//   S = Q K^T,  s = form(S),  online softmax (running max m, sum l, output o rescaled by
//   2^(m_old - m_new)),  O += P V,  lse = ln sum e^s.
//
// Work.  A query tile is 128 rows of one key/value head: up to TQ = floor(128 / hc) consecutive
// tokens of a request times the hc query heads that share the key/value head (head fastest), so
// that one K/V tile serves the whole group and a chunk of a few tokens still fills rows.  A unit is
// two consecutive query tiles of one (request, key/value head) against that head's visible key
// tiles of 128; the CTA holds both tiles, so a K/V tile that is fetched once serves 256 rows.
//
// Who does what.  Lengths live on the device, so the plan is made there, by every CTA for
// itself: it lists what each unit costs (its key tiles plus a fixed share for starting and
// ending it), cuts the whole line of units into equal parts, one per CTA, and takes its part, which
// may start or end inside a unit.  Such parts of a unit leave a normalised fp32 partial output and its
// log-sum-exp in the workspace, and paged_prefill_combine joins them (lse = log sum of the parts'
// sums, O weighted by them).  Every CTA is then done at about the same time whatever the requests'
// sizes; nothing is counted or waited for across CTAs, and the same call gives the same bits.
//
// Inside a CTA (384 threads), as in the dense kernel: warps 0-3 and 4-7 softmax of query tiles 0 and
// 1 (one row per thread = one TMEM lane), warp 8 producer (page ids, TMA of K and V), warps 9 and 10
// one MMA issuer per query tile, passing a turn token, warp 11 TMA loads of Q.  K and V tiles alternate
// in one ring of shared memory, each assembled from the tile's pages, one copy per page (TileLayout).  TMEM: S_t at column 128 t, O_t at 256 + D t, P_t over S_t.
//
// Masks.  Key tiles that no row of the unit sees are skipped (a window leaves a gap between the
// prefix and the window).  In a tile that some row sees in part, hidden scores become -inf before
// the maximum.  Pages that nobody needs, or whose id is out of range, are loaded from outside the
// tensor, where TMA writes zeros: a hidden V row must be a number, as 0 x NaN would reach every row of the
// tile; rows behind the context's last token on its last page are zeroed by the softmax warps.
//
// Bounds and figures (32 query, 8 key/value heads, D = 128, pages of 16).  Plain scores, 4096 tokens at
// 32768, fp16: 1460 to 1480 us, 1.4 PFLOP/s, bound by the tensor pipe (69% in a capture) and power.  With a cap
// and a window, eight requests of up to 700 tokens, bf16: 209 us, bound by the softmax warps, which pass over
// S twice with the cap's polynomial (tensor 28%, issue 42%).  Sixteen tokens each after 1000, four requests: 17 us,
// latency.  The linear bias in the plain form's single pass took whole prompts (D = 64) from 56 us to 51.
// Two warp groups per query tile, for more latency hidden, took the capped case from 226 us to 325.
#pragma once
#include <cuda.h>

#include "attn_fwd_kernel.cuh"
#include "paged_form.cuh"
#include "paged_plan.cuh"

namespace eca {

constexpr int kPfThreads = 384;
constexpr int kPfTile = 128;          // keys per tile, and rows per query tile
// What starting and ending a unit costs, in key tiles, and the least work a part of
// the line is cut to.
constexpr int kPfUnitCost = 3;
constexpr int kPfMinCost = 3;
constexpr int kPfMinPart = 2;         // a unit is not cut within so many tiles of its ends
constexpr int kPfQueue = 4;
constexpr int kPfReaders = 11;
// Per key tile, which of its pages have a bad id.  A softmax warp reads tile j's entry
// before it hands P_j over, so before V_j's place in the ring is free: the producer is
// then at most 10 places (5 tiles) further.
constexpr int kPfBadRing = 8;

struct PrefillParams {
  ChunkShape s;
  ScoreForm f;
  void* out;          // [total, Hq, D] 16-bit
  float* lse;         // [total, Hq] or null
  float* part_o;      // [2 gridDim][D / 4][256][4] fp32
  float* part_lse;    // [2 gridDim][256], base 2
  int* split;         // [gridDim][kPfSplitWords]: the unit that starts in a CTA's part and ends in a later one
  int Hq;
  int hc;             // query heads per query tile
  int chunks;         // of the group: Hq / Hkv / hc
  int tq;             // tokens per query tile
  FastDiv by_hc;
  int small_plan;     // the line is laid out by one warp
  float scale_log2e;
  unsigned long long wait_limit_ns;
  int timeout_code;
};
constexpr int kPfSplitWords = 8;  // parts, first packed row, tokens, first head

template <int D>
struct PrefillSmem {
  static constexpr int kSub = D / 64;
  static constexpr int kTileBytes = kSub * kSubTileBytes;
  static constexpr int kStages = D == 128 ? 5 : 10;  // K or V tiles
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
  static constexpr int kBarQFull = 0;              // + t
  static constexpr int kBarQFree = 2;              // + t
  static constexpr int kBarS = 4;                  // + t: S_t computed
  static constexpr int kBarPa = 6;                 // + t: P_t of keys 0-63 written
  static constexpr int kBarPb = 8;                 // + t: of keys 64-127
  static constexpr int kBarO = 10;                 // + t: last P V of the unit done
  static constexpr int kBarOFree = 12;             // + t: epilogue has read O_t
  static constexpr int kBarDrain = 14;             // + t
  static constexpr int kBarTurn = 16;              // + t
  static constexpr int kBarUnitFull = 18;          // + slot
  static constexpr int kBarUnitFree = kBarUnitFull + kPfQueue;
  static constexpr int kBarFull = kBarUnitFree + kPfQueue;  // + stage
  static constexpr int kBarEmpty = kBarFull + kStages;      // + stage: both issuers
  static constexpr int kNumBars = kBarEmpty + kStages;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // TMEM base, abort flag
  static constexpr int kBadOff = kMiscOff + 8;             // uint32 [kPfBadRing]
  static constexpr int kQueueOff = (kBadOff + 4 * kPfBadRing + 15) & ~15;
  static constexpr int kEntryInts = 16;
  static constexpr int kScanOff = kQueueOff + kPfQueue * kEntryInts * 4;  // 12 warps' sums, 64-bit
  static constexpr int kBytes = kScanOff + 16 * 8;
  static constexpr int kDynamicBytes = kBytes + 1024;
  // The plan's tables lie over the ring.
  static_assert(kLineTableBytes <= kStages * kTileBytes, "the plan's tables fit over the ring");
  static_assert(kDynamicBytes <= 227 * 1024, "shared memory exceeds the per-block limit");
};

// One unit's key tiles: virtual tiles 0 .. k - 1 are logical tiles 0 .. pre - 1 (the prefix)
// and from pre + gap on; end[t] is the end for query tile t alone.
struct PairTiles {
  int tok0;       // first token of the pair, within the request
  int n0, n1;     // tokens of its query tiles
  int pos;        // position of tok0
  int w0;         // first key of the window of tok0
  int hi;         // one past the last token's position
  int pre, gap, k, end0, end1;
};

__device__ __forceinline__ PairTiles pair_tiles(const PrefillParams& p, int n, int pos0, int prefix, int pair) {
  PairTiles u;
  u.tok0 = pair * 2 * p.tq;
  u.n0 = min(p.tq, n - u.tok0);
  u.n1 = max(0, min(p.tq, n - u.tok0 - p.tq));
  u.pos = pos0 + u.tok0;
  u.w0 = p.f.window > 0 ? max(0, u.pos - p.f.window + 1) : 0;
  const int hi0 = max(0, u.pos + u.n0), hi1 = max(0, u.pos + u.n0 + u.n1);
  u.hi = hi1;
  u.pre = (prefix + kPfTile - 1) / kPfTile;
  u.gap = max(0, u.w0 / kPfTile - u.pre);
  u.end0 = max(u.pre, (hi0 + kPfTile - 1) / kPfTile - u.gap);
  u.end1 = u.n1 > 0 ? max(u.pre, (hi1 + kPfTile - 1) / kPfTile - u.gap) : 0;
  u.k = max(u.end0, u.end1);
  return u;
}

// Where a place y on a unit's own line (its cost is k + kPfUnitCost, shared by its tiles)
// cuts it: before key tile 0 .. k.
__device__ __forceinline__ int cut_tile(long long y, int k) {
  const long long cost = k + kPfUnitCost;
  const long long t = y < (1 << 15) && k < (1 << 15)
                          ? static_cast<long long>((static_cast<uint32_t>(y) * static_cast<uint32_t>(k) +
                                                    static_cast<uint32_t>(cost) / 2) / static_cast<uint32_t>(cost))
                          : (y * k + cost / 2) / cost;
  if (t < kPfMinPart) return 0;
  if (t > k - kPfMinPart) return k;
  return static_cast<int>(t);
}

// A fragment of a unit as the producer hands it to the other warps.
struct Fragment {
  int n_max;        // key tiles; -1 past the last fragment
  int n0, n1;       // of them for query tiles 0, 1
  int row;          // packed row of the pair's first token
  int toks0, toks1; // tokens of the query tiles
  int head;         // first query head
  int pos;          // position of the first token
  int prefix, len;
  int pre, gap, kv; // its tiles are kv .. kv + n_max - 1, taken from the last down; v < pre ? v : v + gap
  int part;         // partial slot, or -1: the whole unit
};

template <int D, bool BF16, int FORM>
__global__ void __launch_bounds__(kPfThreads, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_cache,
                         const PrefillParams p) {
  using L = PrefillSmem<D>;
  using Tile = TileLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_base);
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBarOff + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  volatile uint32_t* bad_pages = reinterpret_cast<volatile uint32_t*>(smem + L::kBadOff);
  volatile int* queue = reinterpret_cast<volatile int*>(smem + L::kQueueOff);
  long long* scan_s = reinterpret_cast<long long*>(smem + L::kScanOff);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int lane = threadIdx.x % 32;
  const int tid = threadIdx.x;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::kBarQFull + t), 1);
      mbar_init(bar(L::kBarQFree + t), 1);
      mbar_init(bar(L::kBarS + t), 1);
      mbar_init(bar(L::kBarPa + t), 4);
      mbar_init(bar(L::kBarPb + t), 4);
      mbar_init(bar(L::kBarO + t), 1);
      mbar_init(bar(L::kBarOFree + t), 4);
      mbar_init(bar(L::kBarDrain + t), 1);
      mbar_init(bar(L::kBarTurn + t), 1);
    }
    for (int q = 0; q < kPfQueue; ++q) {
      mbar_init(bar(L::kBarUnitFull + q), 1);
      mbar_init(bar(L::kBarUnitFree + q), kPfReaders);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarFull + s), 1);
      mbar_init(bar(L::kBarEmpty + s), 2);
    }
    mbar_arrive(bar(L::kBarTurn + 0));  // issuer 0 takes the first turn
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) tma_prefetch_map(&tm_cache);
  if (warp == 11 && lane == 0) tma_prefetch_map(&tm_q);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_launch_dependents();
  grid_dependency_wait();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Watchdog wd{abort_flag, p.s.status, p.wait_limit_ns, p.timeout_code};

  // ------------------------------------------------------------------------ plan
  const int B = p.s.B;
  const int heads = p.s.Hkv * p.chunks;  // units of a pair
  const int per_pair = 2 * p.tq;
  const LineTables line = line_tables(smem + L::kRingOff, scan_s);
  auto items = [&](const int4& r) { return (r.x + per_pair - 1) / per_pair; };
  auto cost = [&](const int4& r, int i) { return pair_tiles(p, r.x, r.y, r.z, i).k + kPfUnitCost; };
  const int grid = static_cast<int>(gridDim.x);
  const int cta = static_cast<int>(blockIdx.x);
  // Only the producer needs the plan; a long one is laid out by the whole block.
  long long W = 0;
  if (!p.small_plan) {
    W = line_build<kPfThreads>(line, p.s, p.f, heads, items, cost);
  } else if (warp == 8) {
    W = line_build_warp(line, p.s, p.f, heads, items, cost);
  }
  const long long most = W / kPfMinCost;
  const int G = most < 1 ? 1 : (most < grid ? static_cast<int>(most) : grid);

  // A place on the line: the unit that holds it, and the key tile before which it cuts it.
  struct Place {
    int b, head, pair, tile, k;
    long long start;  // of the unit, on the line
  };
  auto locate = [&](long long x) -> Place {
    const LinePlace at = line_locate<false>(line, B, heads, W, x, cost);
    const int k = at.cost - kPfUnitCost;
    return Place{at.b, at.head, at.item, cut_tile(at.in, k), k, at.start};
  };
  Place from = {}, to = {};
  const bool has_work = cta < G && W > 0;
  if (warp == 8 && has_work) {
    from = locate(line_cut(W, G, cta));
    if (cta + 1 < G) {
      to = locate(line_cut(W, G, cta + 1));
    } else {
      to.b = B;
    }
  }
  // The first request's sizes, before the ring's copies overwrite the tables.
  int4 first_req = make_int4(0, 0, 0, 0);
  if (warp == 8 && has_work) first_req = line.req[from.b];
  // The plan's reads and writes come before the ring's copies (which this warp issues).
  fence_proxy_async_smem();
  if (!p.small_plan) {
    __syncthreads();
  } else {
    __syncwarp();
  }
  // --------------------------------------------------------------------- the roles
  int frags_read = 0;
  // Next fragment for a role (a whole warp, or lane 0 alone): false when a wait gave up.
  auto next_fragment = [&](Fragment& w, bool whole_warp) -> bool {
    const int q = frags_read % kPfQueue;
    bool got = wd.wait(bar(L::kBarUnitFull + q), parity(frags_read / kPfQueue));
    if (whole_warp) got = __all_sync(0xffffffffu, got) != 0;
    if (!got) return false;
    volatile int* e = queue + q * L::kEntryInts;
    int v[14];
#pragma unroll
    for (int i = 0; i < 14; ++i) v[i] = e[i];
    if (whole_warp) {
#pragma unroll
      for (int i = 0; i < 14; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
    }
    w = Fragment{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10], v[11], v[12], v[13]};
    if (lane == 0) mbar_arrive(bar(L::kBarUnitFree + q));
    ++frags_read;
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kRegsControl>();
    if (warp == 8) {
      // ---------------------------------------------------------------- producer
      const int T = p.s.page_size;
      const int log2T = 31 - __clz(T);
      const int pages = kPfTile >> log2T;
      int it = 0, pushed = 0;
      bool ok = true;
      Request r = {};
      int b = from.b, head = from.head, pair = from.pair, tile = from.tile;
      int loaded = -1;  // request that r describes
      PageWalk walk;
      walk.step = -1;
      walk.log2T = log2T;
      walk.num_pages = p.s.num_pages;
      const int end_b = has_work ? to.b : -1;
      auto push = [&](const Fragment& w) -> bool {
        const int q = pushed % kPfQueue;
        const bool free = __all_sync(0xffffffffu, wd.wait(bar(L::kBarUnitFree + q), parity(pushed / kPfQueue) ^ 1u)) != 0;
        if (!free) return false;
        if (lane == 0) {
          volatile int* e = queue + q * L::kEntryInts;
          e[0] = w.n_max;
          e[1] = w.n0;
          e[2] = w.n1;
          e[3] = w.row;
          e[4] = w.toks0;
          e[5] = w.toks1;
          e[6] = w.head;
          e[7] = w.pos;
          e[8] = w.prefix;
          e[9] = w.len;
          e[10] = w.pre;
          e[11] = w.gap;
          e[12] = w.kv;
          e[13] = w.part;
          mbar_arrive(bar(L::kBarUnitFull + q));
        }
        ++pushed;
        return true;
      };
      while (ok && has_work && b <= end_b && b < B) {
        if (loaded != b) {
          if (loaded < 0) {
            r = Request{p.s.q_offsets[b], first_req.x, first_req.w, first_req.y, first_req.z};
          } else {
            r = load_request(p.s, &p.f, b);
          }
          loaded = b;
        }
        const bool last = b == end_b && head == to.head && pair == to.pair;  // the unit the part ends in
        if (r.n == 0) {
          ++b;
          head = pair = tile = 0;
          continue;
        }
        const PairTiles u = pair_tiles(p, r.n, r.pos0, r.prefix, pair);
        const int stop = last ? to.tile : u.k;
        if (stop > tile || (u.k == 0 && !last)) {
          Fragment w;
          w.n_max = stop - tile;
          w.n0 = max(0, min(stop, u.end0) - tile);
          w.n1 = max(0, min(stop, u.end1) - tile);
          w.row = r.row0 + u.tok0;
          w.toks0 = u.n0;
          w.toks1 = u.n1;
          w.head = head * p.hc;
          w.pos = u.pos;
          w.prefix = r.prefix;
          w.len = r.len;
          w.pre = u.pre;
          w.gap = u.gap;
          w.kv = tile;
          w.part = tile > 0 ? 2 * cta : (stop < u.k ? 2 * cta + 1 : -1);
          auto first_page = [&](int j) -> int {  // of the j-th tile
            const int v = tile + w.n_max - 1 - j;
            return (v < u.pre ? v : v + u.gap) * pages;
          };
          // The first page ids are on their way while the fragment is handed out.
          walk.from0 = u.w0;
          walk.to0 = u.hi;
          walk.prefix = r.prefix;
          if (w.n_max > 0) {
            walk.start(p.s.block_table + static_cast<size_t>(b) * p.s.max_pages, first_page(0) >> 5);
          }
          if (!push(w)) {
            ok = false;
            break;
          }
          // K and V tiles of the fragment, alternating.
          const int kvh = head / p.chunks;
          // K/V that several units read stays in L2; a lone pair's is read once.
          const uint64_t pol = r.n > per_pair ? policy_evict_last() : policy_evict_first();
          for (int j = 0; ok && j < w.n_max; ++j) {
            const int at = walk.hold(first_page(j), p.s.status, p.s.bad_index_code);
            for (int kind = 0; kind < 2; ++kind) {
              const int slot = it % L::kStages;
              if (!__all_sync(0xffffffffu, wd.wait(bar(L::kBarEmpty + slot), parity(it / L::kStages) ^ 1u))) {
                ok = false;
                break;
              }
              const uint32_t full = bar(L::kBarFull + slot);
              if (lane == 0) {
                if (kind == 0) bad_pages[it / 2 % kPfBadRing] = (walk.bad >> at) & ((1u << pages) - 1u);
                mbar_arrive_expect_tx(full, L::kTileBytes);
              }
              __syncwarp();
              uint32_t dst = sbase + L::kRingOff + slot * L::kTileBytes;
#pragma unroll 2
              for (int i = 0; i < pages; ++i, dst += T * 2 * D) {
                const int z = __shfl_sync(0xffffffffu, walk.z, at + i) + kind * (T >> 3);
                tma_load_page(dst, &tm_cache, full, z, kvh, pol);
              }
              ++it;
            }
          }
        }
        if (last) break;
        tile = 0;
        if (++pair * per_pair >= r.n) {
          pair = 0;
          if (++head == heads) {
            head = 0;
            ++b;
          }
        }
      }
      if (ok) {
        Fragment w = {};
        w.n_max = -1;
        push(w);
      }
      // The unit that starts here and ends in a later CTA: for the combine kernel.
      if (lane == 0) {
        int parts = 0;
        int* split = p.split + cta * kPfSplitWords;
        if (has_work && to.b < B && to.tile > 0 && to.tile < to.k) {
          const bool started_before = from.b == to.b && from.head == to.head && from.pair == to.pair && from.tile > 0;
          if (!started_before) {
            parts = 2;
            for (int c = cta + 2; c < G; ++c) {
              const long long y = line_cut(W, G, c) - to.start;
              if (y >= to.k + kPfUnitCost || cut_tile(y, to.k) >= to.k) break;
              ++parts;
            }
            const Request r = load_request(p.s, &p.f, to.b);
            const PairTiles u = pair_tiles(p, r.n, r.pos0, r.prefix, to.pair);
            split[1] = r.row0 + u.tok0;
            split[2] = u.n0 + u.n1;
            split[3] = to.head * p.hc;
          }
        }
        split[0] = parts;
      }
      // Let every copy this warp started land before the block can exit.
      for (int x = (it > L::kStages ? it - L::kStages : 0); x < it; ++x) {
        wd.drain(bar(L::kBarFull + x % L::kStages), parity(x / L::kStages));
      }
    } else if (warp == 11) {
      // ----------------------------------------------------------------- Q loader
      if (lane == 0) {
        const uint64_t pol_q = policy_evict_first();
        const uint32_t bytes = static_cast<uint32_t>(L::kSub * p.hc * p.tq * 128);
        int loads[2] = {0, 0};
        bool ok = true;
        Fragment w;
        while (ok && next_fragment(w, false) && w.n_max >= 0) {
          for (int t = 0; t < 2; ++t) {
            if ((t ? w.n1 : w.n0) == 0) continue;
            if (loads[t] > 0 && !wd.wait(bar(L::kBarQFree + t), parity(loads[t] - 1))) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar(L::kBarQFull + t), bytes);
            for (int s = 0; s < L::kSub; ++s) {
              tma_load_3d(sbase + L::kQOff + t * L::kTileBytes + s * kSubTileBytes, &tm_q, bar(L::kBarQFull + t), 64 * s,
                          w.head, w.row + t * p.tq, pol_q);
            }
            ++loads[t];
          }
        }
        for (int t = 0; t < 2; ++t) {
          if (loads[t] > 0) wd.drain(bar(L::kBarQFull + t), parity(loads[t] - 1));
        }
      }
    } else {
      // ------------------------------------------------- MMA issuer of query tile t
      const int t = warp - 9;
      const uint32_t s_tmem = tmem + 128u * t;
      const uint32_t o_tmem = tmem + 256u + static_cast<uint32_t>(D) * t;
      const uint64_t q_desc = smem_desc_sw128(sbase + L::kQOff + t * L::kTileBytes, 16, 1024);
      const uint64_t k_desc = Tile::k_desc(sbase + L::kRingOff);
      const uint64_t v_desc = Tile::v_desc(sbase + L::kRingOff);
      auto stage_off = [&](int item) { return static_cast<uint64_t>((item % L::kStages) * (L::kTileBytes >> 4)); };
      // S_t = Q K^T, and O_t (+)= P V of keys 16 k0 .. 16 k1 - 1.
      auto qk = [&](int item) {
        constexpr uint32_t idesc = idesc_f16_f32acc(kBlockM, kBlockN, BF16, false);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma_ss_warp(s_tmem, q_desc + static_cast<uint64_t>((kk / 4) * (kSubTileBytes >> 4) + (kk % 4) * 2),
                      k_desc + stage_off(item) + Tile::k_step(kk), idesc, kk > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](int item, bool accumulate, int k0, int k1) {
        constexpr uint32_t idesc = idesc_f16_f32acc(kBlockM, D, BF16, true);
#pragma unroll
        for (int kk = k0; kk < k1; ++kk) {
          mma_ts_warp(o_tmem, s_tmem + kk * 8, v_desc + stage_off(item) + Tile::v_step(kk), idesc,
                      (accumulate || kk > 0) ? 1u : 0u);
        }
      };
      auto warp_wait = [&](uint32_t b, uint32_t ph) -> bool { return __all_sync(0xffffffffu, wd.wait(b, ph)) != 0; };
      auto item_wait = [&](int x) -> bool { return warp_wait(bar(L::kBarFull + x % L::kStages), parity(x / L::kStages)); };
      int turns = 0;
      auto take_turn = [&]() -> bool { return warp_wait(bar(L::kBarTurn + t), parity(turns++)); };
      auto pass_turn = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarTurn + (1 - t)));
      };
      int it = 0;       // ring items of the fragments done so far
      int p_waits = 0;  // P_t handshakes consumed
      int used = 0;     // earlier fragments with keys for tile t
      bool ok = true;
      Fragment w;
      while (ok) {
        if (!next_fragment(w, true) || w.n_max < 0) break;
        if (w.n_max == 0) continue;
        const int n_kv = t ? w.n1 : w.n0;
        const int first = w.n_max - n_kv;  // tiles that this query tile does not look at
        // Items of the fragment: K_j at it + 2 j, V_j behind it.  Every item is waited for and released
        // by both issuers.
        if ((n_kv > 0 && !warp_wait(bar(L::kBarQFull + t), parity(used))) || !item_wait(it)) break;
        tc_fence_after_sync();
        if (!take_turn()) break;
        if (first == 0) qk(it);
        pass_turn();
        if (first == 0) {
          tc_commit_warp(bar(L::kBarS + t));
          if (w.n_max == 1) tc_commit_warp(bar(L::kBarQFree + t));
        }
        tc_commit_warp(bar(L::kBarEmpty + it % L::kStages));
        for (int j = 0; j < w.n_max; ++j) {
          const int xv = it + 2 * j + 1, xk = xv + 1;
          if (!item_wait(xv)) {
            ok = false;
            break;
          }
          if (j >= first) {
            // O_t is overwritten by a unit's first P V: the epilogue before must have read it.
            if (j == first && used > 0 && !warp_wait(bar(L::kBarOFree + t), parity(used - 1))) {
              ok = false;
              break;
            }
            if (!warp_wait(bar(L::kBarPa + t), parity(p_waits))) {
              ok = false;
              break;
            }
            ++p_waits;
            tc_fence_after_sync();
          }
          if (!take_turn()) {
            ok = false;
            break;
          }
          if (j >= first) {
            pv(xv, j > first, 0, 4);
            if (!warp_wait(bar(L::kBarPb + t), parity(p_waits - 1))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            pv(xv, true, 4, 8);
          }
          if (j + 1 < w.n_max) {
            if (!item_wait(xk)) {
              ok = false;
              break;
            }
            if (j + 1 >= first) {
              tc_fence_after_sync();
              qk(xk);
            }
          }
          pass_turn();
          if (j + 1 < w.n_max) {
            if (j + 1 >= first) {
              tc_commit_warp(bar(L::kBarS + t));
              if (j + 2 == w.n_max) tc_commit_warp(bar(L::kBarQFree + t));
            }
          } else if (n_kv > 0) {
            tc_commit_warp(bar(L::kBarO + t));
          }
          tc_commit_warp(bar(L::kBarEmpty + xv % L::kStages));
          if (j + 1 < w.n_max) tc_commit_warp(bar(L::kBarEmpty + xk % L::kStages));
        }
        it += 2 * w.n_max;
        used += n_kv > 0 ? 1 : 0;
      }
      // Every MMA issued above must finish before TMEM is released.
      tc_commit_warp(bar(L::kBarDrain + t));
      wd.drain(bar(L::kBarDrain + t), 0);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax
    const int t = warp / 4;
    const int wq = warp % 4;
    const int r_local = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_base + 128u * t;
    const uint32_t t_o = tmem + lane_base + 256u + static_cast<uint32_t>(D) * t;
    // Scores arrive as q . k; the form's pass leaves them in the base-2 domain but for a factor c.
    const CapScale cap = cap_scale(p.f.scale, p.f.softcap, kLog2e);
    const float c = FORM == kFormPlain ? p.scale_log2e : (FORM == kFormCap ? cap.inv_big : 1.f);
    const int row_tok = fast_div(r_local, p.by_hc);  // this row's token and head within the tile
    const int row_head = r_local - row_tok * p.hc;
    const int T = p.s.page_size;
    const int log2T = 31 - __clz(T);
    auto warp_wait = [&](uint32_t b, uint32_t ph) -> bool {
      const bool got = wd.wait(b, ph);
      return __all_sync(0xffffffffu, got) != 0;
    };
    int s_waits = 0, o_waits = 0;
    int it = 0;
    bool ok = true;
    Fragment w;
    while (ok) {
      if (!next_fragment(w, true) || w.n_max < 0) break;
      const int n_kv = t ? w.n1 : w.n0;
      const int toks = t ? w.toks1 : w.toks0;
      const int it0 = it;
      it += 2 * w.n_max;
      if (toks == 0) continue;
      const bool row_ok = row_tok < toks;  // (also false for rows past tq hc)
      const int tok = t * p.tq + row_tok;
      const int pos = w.pos + tok;
      float slope2 = 0.f;
      if (form_biases(FORM) && row_ok) slope2 = p.f.slopes[w.head + row_head] * kLog2e;
      float m_ref = -INFINITY;
      float l = 0.f;
      const int first = w.n_max - n_kv;
      for (int j = first; j < w.n_max; ++j) {
        const int v = w.kv + w.n_max - 1 - j;
        const int kb = (v < w.pre ? v : v + w.gap) * kPfTile;  // position of the tile's first key
        // Columns this row sees: [0, pe) and [ws, ce).
        const int pe = w.prefix - kb, ce = pos + 1 - kb;
        const int ws = p.f.window > 0 ? ce - p.f.window : 0;
        if (!warp_wait(bar(L::kBarS + t), parity(s_waits))) {
          ok = false;
          break;
        }
        ++s_waits;
        tc_fence_after_sync();
        const uint32_t bad = bad_pages[(it0 / 2 + j) % kPfBadRing];
        const bool tail = w.len - kb < kPfTile && (w.len & (T - 1)) != 0;  // the context ends inside one of its pages
        const bool full = pe >= kPfTile || (ws <= 0 && ce >= kPfTile) || !row_ok;
        const bool masked = __any_sync(0xffffffffu, !full) || bad != 0 || tail;
        // Rows of V behind the context's last token, on its last page, may hold anything: zeros,
        // before P is handed over.
        auto zero_tail = [&]() -> bool {
          const int x = it0 + 2 * j + 1;
          if (!warp_wait(bar(L::kBarFull + x % L::kStages), parity(x / L::kStages))) return false;
          const int z0 = max(0, w.len - kb), z1 = min(kPfTile, (((w.len + T - 1) >> log2T) << log2T) - kb);
          const uint32_t base = sbase + L::kRingOff + (x % L::kStages) * L::kTileBytes;
          for (int i = r_local; i < (z1 - z0) * L::kSub * 8; i += 128) {
            const int row = z0 + i / (L::kSub * 8), at = i % (L::kSub * 8);
            st_shared_v4(base + Tile::row(row, at / 8) + (at % 8) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          return true;
        };
        // Columns of quarter q that this row sees, as bits.
        auto seen_bits = [&](int q) -> uint32_t {
          auto low = [](int n) -> uint32_t { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); };
          uint32_t seen = low(pe - 32 * q) | (low(ce - 32 * q) & ~low(ws - 32 * q));
          if (bad != 0) {
#pragma unroll 1
            for (int i = 0; i < 32; i += 8) {  // a page holds 8 tokens at least
              if ((bad >> ((32 * q + i) >> log2T)) & 1u) seen &= ~(0xffu << i);
            }
          }
          return seen;
        };
        // O rescaled in TMEM (P V of the tile before is complete: S was committed after it).
        auto rescale_o = [&](float alpha) {
          const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld_x32(t_o + c0, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = __fmul2_rn(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), al2);
              o[i] = __float_as_uint(x.x);
              o[i + 1] = __float_as_uint(x.y);
            }
            tmem_st_x32(t_o + c0, o);
          }
        };
        auto row_total = [](const float2 (&acc)[8]) -> float {
          const float2 a = __fadd2_rn(__fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3])),
                                      __fadd2_rn(__fadd2_rn(acc[4], acc[5]), __fadd2_rn(acc[6], acc[7])));
          return a.x + a.y;
        };
        // P's half h is in its place in TMEM: hand it to the issuer.
        auto hand_over = [&](int b) {
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(b + t));
        };
        bool move = j == first;  // take the row's max as the reference
        // Before every row's position a distance bias is linear in the key: slope (key - position).
        const bool linear = FORM != kFormBias || __all_sync(0xffffffffu, ce >= kPfTile || !row_ok) != 0;
        if ((FORM == kFormPlain || FORM == kFormBias) && j > first && !masked && linear) {
          // One pass against the reference as it stands.  Keys 64-127 load while keys 0-63 are
          // exponentiated; the checks that let a stale reference stand are those of the dense kernel.
          uint32_t s[4][32];
          uint32_t pk[2][32];
          // What is added to a score of the tile's key 0: the reference, and its bias.
          const float neg_at0 = FORM == kFormBias ? fmaf(-slope2, static_cast<float>(pos - kb), -m_ref) : -m_ref;
          auto exp_quarters = [&](int q0, int q1) -> float {
            float2 acc[8];
#pragma unroll
            for (int a = 0; a < 8; ++a) acc[a] = make_float2(0.f, 0.f);
            const float2 c2 = make_float2(p.scale_log2e, p.scale_log2e);
            const float2 sl2 = make_float2(slope2, slope2);
            const float2 at0 = make_float2(neg_at0, neg_at0);
#pragma unroll
            for (int q = q0; q < q1; ++q) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 key = make_float2(static_cast<float>(32 * q + i), static_cast<float>(32 * q + i + 1));
                const float2 nm2 = FORM == kFormBias ? __ffma2_rn(sl2, key, at0) : at0;
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), c2, nm2);
                const float2 e = make_float2(ex2(x.x), ex2(x.y));
                acc[(i / 2) % 8] = __fadd2_rn(acc[(i / 2) % 8], e);
                pk[q / 2][(q % 2) * 16 + i / 2] = pack2<BF16>(e.x, e.y);
              }
            }
            return row_total(acc);
          };
          tmem_ld_x32(t_s, s[0]);
          tmem_ld_x32(t_s + 32u, s[1]);
          tmem_wait_ld_x32(s[0]);
          tmem_wait_ld_x32(s[1]);
          tmem_ld_x32(t_s + 64u, s[2]);
          tmem_ld_x32(t_s + 96u, s[3]);
          const float sum_a = exp_quarters(0, 2);
          tmem_wait_ld_x32(s[2]);
          tmem_wait_ld_x32(s[3]);
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            mx[0] = fmax3(mx[0], __uint_as_float(s[2][i]), __uint_as_float(s[2][i + 1]));
            mx[1] = fmax3(mx[1], __uint_as_float(s[3][i]), __uint_as_float(s[3][i + 1]));
          }
          // (with a bias, at most that of key 127, or 64 should the slope be negative)
          const float top_b = fmaf(fmaxf(mx[0], mx[1]), p.scale_log2e,
                                   FORM == kFormBias ? fmaf(slope2, slope2 >= 0.f ? 127.f : 64.f, neg_at0) : -m_ref);
          const bool fast = !row_ok || (sum_a <= max_row_sum<BF16>() && top_b <= max_lead<BF16>());
          if (__all_sync(0xffffffffu, fast)) {
            tmem_st_x32(t_s, pk[0]);
            hand_over(L::kBarPa);
            const float sum_b = exp_quarters(2, 4);
            tmem_st_x32(t_s + 32u, pk[1]);
            hand_over(L::kBarPb);
            l += sum_a + sum_b;
            continue;
          }
          move = !fast;  // S is still intact in TMEM: P has not been stored yet
        }
        // Two passes: the first applies the form and the mask, takes the row's max and writes the scores
        // back, the second exponentiates them against a reference that is known to hold.  (The first
        // is a loop: with the form's code inlined four times and more the softmax warps waited for
        // instructions.)
        float top = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t s[32];
          tmem_ld_x32(t_s + 32u * q, s);
          tmem_wait_ld_x32(s);
          if constexpr (form_caps(FORM)) cap_scores<false, false>(s, cap, nullptr);
          if constexpr (form_biases(FORM)) {
            const float away = static_cast<float>(pos - kb - 32 * q);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = __uint_as_float(s[i]) * (FORM == kFormBias ? p.scale_log2e : cap.inv_big);
              s[i] = __float_as_uint(fmaf(-slope2, fabsf(away - static_cast<float>(i)), x));
            }
          }
          if (masked) {
            const uint32_t seen = seen_bits(q);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (!(seen & (1u << i))) s[i] = __float_as_uint(-INFINITY);
            }
          }
          float t4[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            t4[i / 2 % 4] = fmax3(t4[i / 2 % 4], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          }
          top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          if (FORM != kFormPlain || masked) tmem_st_x32(t_s + 32u * q, s);
        }
        top *= c;
        // The reference moves on the first tile, and when a p could leave the 16-bit range.
        float alpha = 1.f;
        if (move || top > m_ref + max_lead<BF16>()) {
          const float m_new = j == first ? top : fmaxf(m_ref, top);
          alpha = (j == first || m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_new);
          m_ref = m_new;
        }
        l *= alpha;
        if (j > first && __any_sync(0xffffffffu, alpha != 1.f)) rescale_o(alpha);
        if (tail && !zero_tail()) {
          ok = false;
          break;
        }
        tmem_wait_st();
        const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
        const float2 c2 = make_float2(c, c);
        const float2 nm2 = make_float2(neg_m, neg_m);
        float2 acc[8];
#pragma unroll
        for (int a = 0; a < 8; ++a) acc[a] = make_float2(0.f, 0.f);
        uint32_t s[2][32];
        tmem_ld_x32(t_s, s[0]);
        tmem_ld_x32(t_s + 32u, s[1]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tmem_wait_ld_x32(s[0]);
          tmem_tie_x32(s[1]);
          uint32_t pk[32];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), c2, nm2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              acc[(i / 2) % 8] = __fadd2_rn(acc[(i / 2) % 8], e);
              pk[q * 16 + i / 2] = pack2<BF16>(e.x, e.y);
            }
          }
          tmem_st_x32(t_s + 32u * half, pk);
          if (half == 0) {
            tmem_ld_x32(t_s + 64u, s[0]);
            tmem_ld_x32(t_s + 96u, s[1]);
          }
          hand_over(half == 0 ? L::kBarPa : L::kBarPb);
        }
        l += row_total(acc);
      }
      if (!ok) break;
      if (n_kv > 0) {
        if (!warp_wait(bar(L::kBarO + t), parity(o_waits))) break;
        ++o_waits;
        tc_fence_after_sync();
      }
      // Epilogue: the whole unit's O and lse, or a part's in fp32.
      const bool any = l > 0.f;
      const float inv_l = any ? 1.f / l : 0.f;
      const float lse2 = any ? m_ref + log2f(l) : -INFINITY;
      const size_t out_row = static_cast<size_t>(w.row + tok) * p.Hq + w.head + row_head;
      if (w.part >= 0) {
        float4* dst = reinterpret_cast<float4*>(p.part_o) + (static_cast<size_t>(w.part) * (D / 4)) * 256 + t * 128 + r_local;
        if (n_kv > 0) {
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld_x32(t_o + c0, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (row_ok) {
                dst[static_cast<size_t>(c0 / 4 + i) * 256] =
                    make_float4(__uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                                __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
              }
            }
          }
        }
        p.part_lse[static_cast<size_t>(w.part) * 256 + t * 128 + r_local] = row_ok ? lse2 : -INFINITY;
      } else {
        // 32 columns at a time.  Four lanes exchange 16-byte chunks, so that each then writes a
        // quarter of 64 bytes of one row: a store touches 8 rows instead of 32 (which took 4 times as long).
        const int q0 = lane & ~3, qj = lane & 3;
        uint16_t* dst[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = wq * 32 + q0 + i;
          const int rt = fast_div(r, p.by_hc);
          dst[i] = rt < toks ? static_cast<uint16_t*>(p.out) +
                                   (static_cast<size_t>(w.row + t * p.tq + rt) * p.Hq + w.head + r - rt * p.hc) * D + 8 * qj
                             : nullptr;
        }
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          if (n_kv > 0) {
            tmem_ld_x32(t_o + c0, o);
            tmem_wait_ld_x32(o);
          }
          uint32_t h[4][4];  // [chunk][word]
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            h[i / 4][i % 4] = any ? pack2<BF16>(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l) : 0u;
          }
          // Transpose of 4 lanes x 4 chunks: first between neighbours, then between pairs.
#pragma unroll
          for (int d = 1; d < 4; d *= 2) {
            const bool upper = (qj & d) != 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (x & d) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t give = upper ? h[x][k] : h[x | d][k];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, d);
                if (upper) {
                  h[x][k] = got;
                } else {
                  h[x | d][k] = got;
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (dst[i] != nullptr) {
              *reinterpret_cast<uint4*>(dst[i] + c0) = make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
            }
          }
        }
        if (p.lse != nullptr && row_ok) p.lse[out_row] = lse2 * kLn2;
      }
      if (n_kv > 0) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarOFree + t));
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of a unit that several CTAs of the kernel above shared: with
// L = log2 sum_s 2^(lse_s), O = sum_s 2^(lse_s - L) O_s.  Block (c, rows): the unit that starts in CTA c,
// 32 of its 256 rows; a thread takes one row and 16 columns.
template <int D, bool BF16>
__global__ void __launch_bounds__(2 * D) paged_prefill_combine(const PrefillParams p, int part_rows) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int cta = blockIdx.x / (256 / part_rows);
  const int row0 = blockIdx.x % (256 / part_rows) * part_rows;
  const int* split = p.split + cta * kPfSplitWords;
  const int parts = split[0];
  if (parts == 0) return;
  const int t = threadIdx.x % 32 + row0, c16 = threadIdx.x / 32;
  const int tile = t / 128, r = t % 128;
  const int tok = fast_div(r, p.by_hc);
  const int head = r - tok * p.hc;
  if (tok >= p.tq || tile * p.tq + tok >= split[2]) return;
  // CTA c left its part in its second slot, the following ones in their first.
  auto slot = [&](int i) -> size_t { return i == 0 ? 2 * cta + 1 : 2 * (cta + i); };
  // Three parts' sums and outputs at a time in one round trip, folded in with the online law.
  float top = -INFINITY;
  float sum = 0.f;
  float4 acc[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < parts; i0 += 3) {
    float ls[3];
    float4 x[3][4];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      ls[i] = -INFINITY;
      if (i0 + i < parts) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o) + (slot(i0 + i) * (D / 4) + c16 * 4) * 256 + t;
        ls[i] = p.part_lse[slot(i0 + i) * 256 + t];
#pragma unroll
        for (int v = 0; v < 4; ++v) x[i][v] = src[v * 256];
      }
    }
    const float now = fmaxf(fmaxf(top, ls[0]), fmaxf(ls[1], ls[2]));
    if (now == -INFINITY) continue;
    const float keep = top == -INFINITY ? 0.f : exp2f(top - now);
    top = now;
    sum *= keep;
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = make_float4(acc[v].x * keep, acc[v].y * keep, acc[v].z * keep, acc[v].w * keep);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float w = exp2f(ls[i] - now);
      if (w == 0.f) continue;  // (a part without keys for this row has written no output)
      sum += w;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        acc[v].x += w * x[i][v].x;
        acc[v].y += w * x[i][v].y;
        acc[v].z += w * x[i][v].z;
        acc[v].w += w * x[i][v].w;
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const size_t row = static_cast<size_t>(split[1] + tile * p.tq + tok) * p.Hq + split[3] + head;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + c16 * 16);
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float4 a = acc[2 * v], b = acc[2 * v + 1];
    dst[v] = make_uint4(pack2<BF16>(a.x * inv, a.y * inv), pack2<BF16>(a.z * inv, a.w * inv),
                        pack2<BF16>(b.x * inv, b.y * inv), pack2<BF16>(b.z * inv, b.w * inv));
  }
  if (p.lse != nullptr && c16 == 0) p.lse[row] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

}  // namespace eca
