// Eviction from the paged cache by accumulated attention weight.  For every request b
// with more than `budget` tokens and every key/value head: the last `recent` tokens are
// kept, and of the others the budget - recent with the largest mass (equal masses: the
// lowest position first); the kept rows move in order to positions 0 .. budget - 1.
//
// Two kernels.  paged_evict_select: one block per (request, head) finds the mass of
// the last token that is kept by a radix select on the masses' bit patterns (three
// digits of 11, 11 and 10 bits; a histogram of the tokens that share the digits
// fixed so far, in shared memory), then walks the tokens in order with a block scan that
// gives every kept token its new position.  paged_evict_move: the rows move in
// place.  A kept token's new position never exceeds its old one and both grow
// together, so a block that walks its rows in order, reading a batch before it writes one,
// never overwrites a row that it has yet to read; blocks split a row's columns
// (and K from V), not the rows, so they do not meet.
#pragma once
#include "paged_common.cuh"

namespace eca {

struct EvictParams {
  ChunkShape s;  // q_offsets unused
  void* cache;
  const float* mass;   // [B, Hkv, max_pages * page_size]
  int* kept;           // [B, Hkv, budget]
  int* new_lengths;    // [B]
  float* mass_out;     // like mass, or null
  int budget, recent;
};

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;

// Order of masses as unsigned integers: larger mass, larger key; -0 equals +0; NaN
// below every number.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive sum over the block's threads in order; `ws` holds one value per warp.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* ws, uint32_t* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += up;
  }
  __syncthreads();  // ws may still be read from an earlier call
  if (lane == 31) ws[warp] = v;
  __syncthreads();
  uint32_t w = ws[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += up;
  }
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp) - ws[warp];
  *total = __shfl_sync(0xffffffffu, w, 31);
  return before + v;
}

__global__ void __launch_bounds__(kSelThreads) paged_evict_select_kernel(const EvictParams p) {
  static_assert(kSelThreads == 1024, "block_scan reads one sum per warp of a full block");
  __shared__ uint32_t hist[kSelBins];
  __shared__ uint32_t ws[32];
  __shared__ uint32_t chosen[2];  // digit, candidates above it
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.x / p.s.Hkv;
  const int most = p.s.max_pages * p.s.page_size;
  int len = p.s.lengths[b];
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) atomicExch(p.s.status, p.s.bad_index_code);
    len = len < 0 ? 0 : most;
  }
  const float* mass = p.mass + static_cast<size_t>(blockIdx.x) * most;
  float* mass_out = p.mass_out == nullptr ? nullptr : p.mass_out + static_cast<size_t>(blockIdx.x) * most;
  int* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.budget;
  const int n_new = min(len, p.budget);
  const int tail = min(p.recent, n_new);
  const int cand = len - tail;        // tokens that compete: 0 .. cand - 1
  uint32_t want = n_new - tail;       // that many of them are kept
  // Keys above `floor_key` are kept, and the first `ties` of those equal to it.
  uint32_t floor_key = 0, ties = 0;
  if (want == static_cast<uint32_t>(cand)) {
    ties = static_cast<uint32_t>(cand);  // everything stays: nothing ranks below 0
  } else if (want == 0) {
    floor_key = 0xffffffffu;
  } else {
    uint32_t mask = 0;
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0);
      const uint32_t digits = round == 2 ? 0x3ffu : 0x7ffu;
      for (int i = threadIdx.x; i < kSelBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < cand; i += kSelThreads) {
        const uint32_t key = mass_key(mass[i]);
        if ((key & mask) == floor_key) atomicAdd(&hist[(key >> shift) & digits], 1u);
      }
      __syncthreads();
      // Bins from the largest digit down: thread t takes digits top - 2 t and the next.
      const int d0 = kSelBins - 1 - 2 * threadIdx.x;
      const uint32_t h0 = hist[d0], h1 = hist[d0 - 1];
      uint32_t total;
      const uint32_t upto = block_scan(h0 + h1, ws, &total);
      const uint32_t above = upto - h0 - h1;
      if (above < want && want <= above + h0) {
        chosen[0] = d0;
        chosen[1] = above;
      } else if (above + h0 < want && want <= upto) {
        chosen[0] = d0 - 1;
        chosen[1] = above + h0;
      }
      __syncthreads();
      floor_key |= chosen[0] << shift;
      mask |= digits << shift;
      want -= chosen[1];
      __syncthreads();
    }
    ties = want;
  }
  // Tokens in order, one per thread and pass; a pass reads before it writes, and
  // writes only places up to those it read (mass_out may be mass).
  uint32_t kept_before = 0, ties_before = 0;
  for (int base = 0; base < len; base += kSelThreads) {
    const int i = base + threadIdx.x;
    float m = 0.f;
    bool above = false, equal = false;
    if (i < len) {
      m = mass[i];
      const uint32_t key = mass_key(m);
      above = i >= cand || key > floor_key;
      equal = i < cand && key == floor_key;
    }
    uint32_t total;
    const uint32_t scan = block_scan((above ? 1u << 16 : 0u) + (equal ? 1u : 0u), ws, &total);
    // Ties before this token, and the tokens kept before it.
    const uint32_t t_incl = ties_before + (scan & 0xffffu);
    const uint32_t t_excl = t_incl - (equal ? 1u : 0u);
    const bool keep = above || (equal && t_excl < ties);
    const uint32_t slot = kept_before + (scan >> 16) - (above ? 1u : 0u) + min(t_excl, ties) - min(ties_before, ties);
    if (keep) {
      kept[slot] = i;
      if (mass_out != nullptr) mass_out[slot] = m;
    }
    kept_before += (total >> 16) + min(ties_before + (total & 0xffffu), ties) - min(ties_before, ties);
    ties_before += total & 0xffffu;
  }
  __syncthreads();
  for (int i = n_new + threadIdx.x; i < p.budget; i += kSelThreads) kept[i] = -1;
  if (mass_out != nullptr) {
    for (int i = n_new + threadIdx.x; i < most; i += kSelThreads) mass_out[i] = 0.f;
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveSlice = 4;  // 16-byte vectors of a row that one block moves
constexpr int kMoveBatch = 4;  // of them per thread and pass

__global__ void __launch_bounds__(kMoveThreads) paged_evict_move_kernel(const EvictParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int slices = p.s.D / (8 * kMoveSlice);
  int u = blockIdx.x;
  const int slice = u % slices;
  u /= slices;
  const int kind = u % 2;
  u /= 2;
  const int h = u % p.s.Hkv, b = u / p.s.Hkv;
  const int most = p.s.max_pages * p.s.page_size;
  const int n_new = min(min(max(p.s.lengths[b], 0), most), p.budget);
  if (h == 0 && kind == 0 && slice == 0 && threadIdx.x == 0) p.new_lengths[b] = n_new;
  const int* kept = p.kept + (static_cast<size_t>(b) * p.s.Hkv + h) * p.budget;
  const int* table = p.s.block_table + static_cast<size_t>(b) * p.s.max_pages;
  const int log2T = 31 - __clz(p.s.page_size);
  uint4* cache = static_cast<uint4*>(p.cache);
  // The slice's vector of token position t, or -1 on a page out of range.
  auto place = [&](int t) -> long long {
    const int page = table[t >> log2T];
    if (page < 0 || page >= p.s.num_pages) {
      atomicExch(p.s.status, p.s.bad_index_code);
      return -1;
    }
    const size_t row = (static_cast<size_t>(page) * 2 + kind) * p.s.page_size + (t & (p.s.page_size - 1));
    return static_cast<long long>((row * p.s.Hkv + h) * (p.s.D / 8) + slice * kMoveSlice + threadIdx.x % kMoveSlice);
  };
  constexpr int kRows = kMoveThreads / kMoveSlice;
  for (int d0 = 0; d0 < n_new; d0 += kRows * kMoveBatch) {
    uint4 v[kMoveBatch];
    long long to[kMoveBatch];
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      const int d = d0 + i * kRows + threadIdx.x / kMoveSlice;
      to[i] = -1;
      if (d >= n_new) continue;
      const int from = kept[d];
      if (from == d) continue;
      const long long src = place(from);
      to[i] = src < 0 ? -1 : place(d);
      if (to[i] >= 0) v[i] = cache[src];
    }
    __syncthreads();  // the batch is read: its rows, and any behind them, may be overwritten
#pragma unroll
    for (int i = 0; i < kMoveBatch; ++i) {
      if (to[i] >= 0) cache[to[i]] = v[i];
    }
  }
}

}  // namespace eca
