// Eviction from the paged cache by accumulated attention weight.  For every request b
// with more than `budget` tokens and every key/value head: the last `recent` tokens are
// kept, and of the others the budget - recent with the largest mass (equal masses: the
// lowest position first); the kept rows move in order to positions 0 .. budget - 1.
//
// Two kernels.  paged_evict_select: a cluster of 1 to 4 blocks per (request, head), each with a run of
// its tokens, finds the mass of the last token that is kept by a radix select on the masses' bit
// patterns (three digits of 11, 11 and 10 bits; a histogram of the tokens that share the digits
// fixed so far, summed over the cluster through its shared memory), then walks the tokens in
// order and gives every kept one its new position.  The masses are read once and kept in shared
// memory as keys.  Bound by instructions (some 40 per token), so few heads are spread over more blocks.
// (8 requests x 8 heads, 8192 tokens to 2048: 42 us in all, of which the move of 68 MB each way 26.)
// paged_evict_move: the rows move in place.  A kept token's new position never exceeds its old
// one and both grow together, so a batch of rows in order may be written once it has been
// read, and never touches a row of a later batch.  A cluster of 8 blocks takes one head's K or V: they
// read a batch together, meet at the cluster's barrier, and write it.  Bound by HBM for many heads
// and by the chain position -> page -> row for few.
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

__device__ __forceinline__ float key_mass(uint32_t k) {
  return k == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
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

constexpr int kSelCopies = 4;          // of the histogram: lanes of a warp often meet in one bin
constexpr int kSelSmemTokens = 32768;  // most tokens of a block whose keys are kept in shared memory
constexpr int kSelMaxCluster = 4;

__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n"
      "barrier.cluster.wait.acquire.aligned;\n" ::
          : "memory");
}

// A word of the shared memory of the cluster's block `rank`.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, int rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// kKeep: every block's keys fit in (dynamic) shared memory, 4 bytes a token; otherwise
// launched without a cluster, and the masses are read again for every digit.
template <bool kKeep>
__global__ void __launch_bounds__(kSelThreads) paged_evict_select_kernel(const EvictParams p, int cluster) {
  static_assert(kSelThreads == 1024, "block_scan reads one sum per warp of a full block");
  __shared__ uint32_t hist[kSelCopies][kSelBins];
  __shared__ uint32_t merged[kKeep ? 3 : 1][kSelBins];  // this block's counts, one array per digit
  __shared__ uint32_t ws[32];
  __shared__ uint32_t chosen[2];  // digit, candidates above it
  __shared__ uint32_t totals[2];  // this block's kept and tied tokens
  extern __shared__ uint32_t keys[];
  grid_launch_dependents();
  for (int i = threadIdx.x; i < kSelCopies * kSelBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  grid_dependency_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int rank = blockIdx.x % cluster, unit = blockIdx.x / cluster;  // unit: (b, head)
  const int b = unit / p.s.Hkv;
  const int most = p.s.max_pages * p.s.page_size;
  int len = p.s.lengths[b];
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) atomicExch(p.s.status, p.s.bad_index_code);
    len = len < 0 ? 0 : most;
  }
  const float* mass = p.mass + static_cast<size_t>(unit) * most;
  float* mass_out = p.mass_out == nullptr ? nullptr : p.mass_out + static_cast<size_t>(unit) * most;
  int* kept = p.kept + static_cast<size_t>(unit) * p.budget;
  const int n_new = min(len, p.budget);
  const int tail = min(p.recent, n_new);
  const int cand = len - tail;        // tokens that compete: 0 .. cand - 1
  uint32_t want = n_new - tail;       // that many of them are kept
  // Each block takes a run of tokens, and each of its warps a run of those.
  const int share = ((len + 32 * cluster - 1) / (32 * cluster)) * 32;
  const int run = ((share + 1023) / 1024) * 32;
  const int first = rank * share, past = min(len, first + share);
  const int begin = min(past, first + warp * run), end = min(past, begin + run);
  __syncthreads();
  if constexpr (kKeep) {
#pragma unroll 8
    for (int i = begin + lane; i < end; i += 32) keys[i - first] = mass_key(mass[i]);
    __syncwarp();
  }
  auto key_at = [&](int i) -> uint32_t { return kKeep ? keys[i - first] : mass_key(mass[i]); };
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
      const int stop = min(end, cand);
#pragma unroll 8
      for (int i = begin + lane; i < stop; i += 32) {
        const uint32_t key = key_at(i);
        if ((key & mask) == floor_key) atomicAdd(&hist[lane % kSelCopies][(key >> shift) & digits], 1u);
      }
      __syncthreads();
      // Bins from the largest digit down: thread t takes digits top - 2 t and the next.
      const int d0 = kSelBins - 1 - 2 * threadIdx.x;
      uint32_t h0 = 0, h1 = 0;
#pragma unroll
      for (int c = 0; c < kSelCopies; ++c) {
        h0 += hist[c][d0];
        h1 += hist[c][d0 - 1];
        hist[c][d0] = hist[c][d0 - 1] = 0;
      }
      if (kKeep && cluster > 1) {
        merged[kKeep ? round : 0][d0] = h0;
        merged[kKeep ? round : 0][d0 - 1] = h1;
        cluster_barrier();
        h0 = h1 = 0;
#pragma unroll
        for (int c = 0; c < kSelMaxCluster; ++c) {
          if (c < cluster) {
            h0 += cluster_load(&merged[kKeep ? round : 0][d0], c);
            h1 += cluster_load(&merged[kKeep ? round : 0][d0 - 1], c);
          }
        }
      }
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
  if constexpr (kKeep) {
    // Every warp counts its run, learns what the runs before hold, and writes its kept tokens.
    uint32_t n_above = 0, n_equal = 0;
#pragma unroll 8
    for (int i = begin + lane; i < end; i += 32) {
      const uint32_t key = keys[i - first];
      n_above += (i >= cand || key > floor_key) ? 1u : 0u;
      n_equal += (i < cand && key == floor_key) ? 1u : 0u;
    }
    n_above = __reduce_add_sync(0xffffffffu, n_above);
    n_equal = __reduce_add_sync(0xffffffffu, n_equal);
    __syncthreads();
    // (16 bits hold either count: 32768 tokens at most)
    if (lane == 0) ws[warp] = n_above << 16 | (n_equal & 0xffffu);
    __syncthreads();
    uint32_t a = 0, e = 0;
    for (int w = 0; w < warp; ++w) {
      a += ws[w] >> 16;
      e += ws[w] & 0xffffu;
    }
    if (cluster > 1) {
      if (threadIdx.x == kSelThreads - 32) {
        totals[0] = a + n_above;
        totals[1] = e + n_equal;
      }
      cluster_barrier();
      for (int c = 0; c < rank; ++c) {
        a += cluster_load(&totals[0], c);
        e += cluster_load(&totals[1], c);
      }
    }
    const uint32_t before_me = (1u << lane) - 1u;
    constexpr int kGroups = 4;  // of 32 tokens at a time, so that their votes overlap
    for (int i0 = begin; i0 < end; i0 += 32 * kGroups) {
      uint32_t key[kGroups], ab[kGroups], eb[kGroups];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int i = i0 + 32 * g + lane;
        key[g] = i < end ? keys[i - first] : 0u;
        ab[g] = __ballot_sync(0xffffffffu, i < end && (i >= cand || key[g] > floor_key));
        eb[g] = __ballot_sync(0xffffffffu, i < end && i < cand && key[g] == floor_key);
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const uint32_t my_a = a + __popc(ab[g] & before_me), my_e = e + __popc(eb[g] & before_me);
        const bool above = (ab[g] >> lane) & 1u, equal = (eb[g] >> lane) & 1u;
        if (above || (equal && my_e < ties)) {
          const uint32_t slot = my_a + min(my_e, ties);
          kept[slot] = i0 + 32 * g + lane;
          if (mass_out != nullptr) mass_out[slot] = key_mass(key[g]);
        }
        a += __popc(ab[g]);
        e += __popc(eb[g]);
      }
    }
  } else {
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
      const uint32_t t_excl = ties_before + (scan & 0xffffu) - (equal ? 1u : 0u);
      if (above || (equal && t_excl < ties)) {
        const uint32_t slot =
            kept_before + (scan >> 16) - (above ? 1u : 0u) + min(t_excl, ties) - min(ties_before, ties);
        kept[slot] = i;
        if (mass_out != nullptr) mass_out[slot] = m;
      }
      kept_before += (total >> 16) + min(ties_before + (total & 0xffffu), ties) - min(ties_before, ties);
      ties_before += total & 0xffffu;
    }
  }
  for (int i = n_new + rank * kSelThreads + threadIdx.x; i < p.budget; i += kSelThreads * cluster) kept[i] = -1;
  if (kKeep && cluster > 1) cluster_barrier();  // no block leaves while another may read its counts
}

constexpr int kMoveThreads = 256;
constexpr int kMoveCluster = 8;          // blocks that move one head's K or V
constexpr int kMoveBytes = 64 * 1024;    // rows a block reads before it writes them, in shared memory

template <int D>
__global__ void __cluster_dims__(kMoveCluster, 1, 1) __launch_bounds__(kMoveThreads)
    paged_evict_move_kernel(const EvictParams p) {
  constexpr int kVecs = D / 8;                   // 16-byte vectors of a row
  constexpr int kRows = kMoveBytes / (D * 2);    // rows of a block's batch
  constexpr int kItems = kMoveBytes / 16 / kMoveThreads;
  extern __shared__ uint4 staged[];
  __shared__ int2 rows[2][kRows];                // old and new token row in the cache, or -1
  grid_launch_dependents();
  grid_dependency_wait();
  const int rank = blockIdx.x % kMoveCluster;
  int u = blockIdx.x / kMoveCluster;
  const int kind = u % 2;
  u /= 2;
  const int h = u % p.s.Hkv, b = u / p.s.Hkv;
  const int most = p.s.max_pages * p.s.page_size;
  const int n_new = min(min(max(p.s.lengths[b], 0), most), p.budget);
  if (h == 0 && kind == 0 && rank == 0 && threadIdx.x == 0) p.new_lengths[b] = n_new;
  const size_t head = static_cast<size_t>(b) * p.s.Hkv + h;
  const int* kept = p.kept + head * p.budget;
  const int* table = p.s.block_table + static_cast<size_t>(b) * p.s.max_pages;
  const int log2T = 31 - __clz(p.s.page_size);
  uint4* cache = static_cast<uint4*>(p.cache);
  // Where the rows of the batch at d0 come from and go to.
  auto look_up = [&](int d0, int2* out) {
    for (int r = threadIdx.x; r < kRows; r += kMoveThreads) {
      const int d = d0 + rank * kRows + r;
      int2 move = make_int2(-1, -1);
      const int from = d < n_new ? kept[d] : d;
      if (from != d) {
        const int page_from = table[from >> log2T], page_to = table[d >> log2T];
        if (page_from < 0 || page_from >= p.s.num_pages || page_to < 0 || page_to >= p.s.num_pages) {
          atomicExch(p.s.status, p.s.bad_index_code);
        } else {
          const int in = p.s.page_size - 1;
          move = make_int2(((page_from * 2 + kind) << log2T) + (from & in), ((page_to * 2 + kind) << log2T) + (d & in));
        }
      }
      out[r] = move;
    }
  };
  auto place = [&](int row, int vec) -> size_t { return (static_cast<size_t>(row) * p.s.Hkv + h) * kVecs + vec; };
  look_up(0, rows[0]);
  __syncthreads();
  int buf = 0;
  for (int d0 = 0; d0 < n_new; d0 += kRows * kMoveCluster, buf ^= 1) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = i * kMoveThreads + threadIdx.x;
      const int from = rows[buf][x / kVecs].x;
      if (from >= 0) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(staged + x)),
                     "l"(cache + place(from, x % kVecs))
                     : "memory");
      }
    }
    // The next batch's places are looked up while this one's rows are on their way.
    look_up(d0 + kRows * kMoveCluster, rows[buf ^ 1]);
    asm volatile("cp.async.wait_all;" ::: "memory");
    cluster_barrier();  // the batch is read: its rows, and any behind them, may be overwritten
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int x = i * kMoveThreads + threadIdx.x;
      const int to = rows[buf][x / kVecs].y;
      if (to >= 0) cache[place(to, x % kVecs)] = staged[x];
    }
    __syncthreads();  // rows[buf] is written again in the next round
  }
  if (kind == 0 && p.mass_out != nullptr) {  // no token is left there
    float* mass_out = p.mass_out + head * most;
    for (int i = n_new + rank * kMoveThreads + threadIdx.x; i < most; i += kMoveThreads * kMoveCluster) mass_out[i] = 0.f;
  }
}

}  // namespace eca
