// What the kernels over a paged cache and a ragged chunk of new tokens share: the
// request's sizes with their checks, and the score forms.
#pragma once
#include <cuda.h>
#include <cstdint>

#include "ptx.cuh"

namespace eca {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t h) {
  if constexpr (BF16) {
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  } else {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
    return f;
  }
}

template <bool BF16>
__device__ __forceinline__ float2 to_f32x2(uint32_t w) {
  return make_float2(to_f32<BF16>(static_cast<uint16_t>(w & 0xffffu)), to_f32<BF16>(static_cast<uint16_t>(w >> 16)));
}

// Sizes of the paged cache and the ragged chunk, the same for every kernel.
struct ChunkShape {
  const int* block_table;  // [B, max_pages]
  const int* lengths;      // [B]
  const int* q_offsets;    // [B + 1], or null: one row a request
  int* status;
  int total;               // packed rows
  int B, Hkv, D, page_size, max_pages, num_pages;
  int bad_index_code;
};

// Score forms (include/attn_cache.h).
struct ScoreForm {
  float scale;
  float softcap;        // 0: none
  const float* slopes;  // [Hq] or null
  const int* prefix;    // [B] or null
  int window;           // 0: none
};

// One request of the chunk: rows row0 .. row0 + n - 1 at positions pos0, pos0 + 1, ...
// of a context of len tokens, the first `prefix` of them visible to every row.
struct Request {
  int row0, n, len, pos0, prefix;
};

// Reads and checks request b (below B); what is out of range is reported, offsets that
// make no sense leave the request without rows, and a length out of range is taken at
// the nearest end.
__device__ __forceinline__ Request load_request(const ChunkShape& s, const ScoreForm* form, int b) {
  Request r;
  int end = b + 1;
  r.row0 = b;
  if (s.q_offsets != nullptr) {
    r.row0 = s.q_offsets[b];
    end = s.q_offsets[b + 1];
  }
  bool bad = false;
  if (r.row0 < 0 || end < r.row0 || end > s.total) {
    bad = true;
    r.row0 = end = 0;
  }
  r.n = end - r.row0;
  r.len = s.lengths[b];
  const int most = s.max_pages * s.page_size;
  if (r.len < 0 || r.len > most) {
    bad = true;
    r.len = r.len < 0 ? 0 : most;
  }
  if (s.q_offsets == nullptr && r.len == 0) r.n = 0;  // a decode step's request without tokens
  r.pos0 = r.len - r.n;
  if (r.pos0 < 0) bad = true;
  if (bad) atomicExch(s.status, s.bad_index_code);
  r.prefix = 0;
  if (form != nullptr && form->prefix != nullptr) r.prefix = min(max(form->prefix[b], 0), r.len);
  return r;
}

// Request that owns packed row t, or -1 when none does: the last b with
// q_offsets[b] <= t, provided t lies below q_offsets[b + 1].
__device__ __forceinline__ int request_of_row(const ChunkShape& s, int t) {
  int lo = 0, hi = s.B;  // q_offsets[lo] <= t < q_offsets[hi], where the offsets are in order
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (s.q_offsets[mid] <= t) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return s.q_offsets[lo] <= t && t < s.q_offsets[lo + 1] ? lo : -1;
}

// A tile of K or V in shared memory: groups of 8 tokens, each D / 64 blocks of 64 columns, each 8 rows
// of 128 bytes with the 128-byte swizzle.  A page is then one contiguous copy whatever its
// size (cache_group_map on the host), and for the tensor core the groups of a whole tile lie at one
// stride: as a K-major operand (K) and as an MN-major one (V).
template <int D>
struct TileLayout {
  static constexpr int kGroupBytes = D / 64 * 1024;
  // Byte offset of row r's part in column block h.
  static __device__ __forceinline__ uint32_t row(int r, int h) { return r / 8 * kGroupBytes + h * 1024 + r % 8 * 128; }
  static __device__ __forceinline__ uint64_t k_desc(uint32_t base) { return smem_desc_sw128(base, 16, kGroupBytes); }
  static __device__ __forceinline__ uint64_t v_desc(uint32_t base) { return smem_desc_sw128(base, 1024, kGroupBytes); }
  // Steps of a descriptor (in its 16-byte units) to columns 16 kk .. of K, and to rows 16 kk .. of V.
  static __device__ __forceinline__ constexpr uint64_t k_step(int kk) { return (kk / 4) * (1024 >> 4) + (kk % 4) * 2; }
  static __device__ __forceinline__ constexpr uint64_t v_step(int kk) { return kk * (2 * kGroupBytes >> 4); }
};

// One page of K or V: its page_size / 8 groups.  The whole warp, with warp-uniform
// operands; one elected lane issues it.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, uint32_t bar, int group, int head,
                                              uint64_t cache_policy) {
  asm volatile(
      "{\n"
      "  .reg .pred e;\n"
      "  elect.sync _|e, 0xffffffff;\n"
      "  @e cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %3, %3, %4, %5}], [%2], %6;\n"
      "}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(group), "r"(head), "l"(cache_policy)
      : "memory");
}

// A request's pages as a producer warp walks them, up or down: lane i holds the i-th
// of 32 consecutive block-table entries, and the next 32 are on their way.  Pages that
// nobody needs, and those with an id out of range (reported), get the place behind the
// tensor's last group, where TMA reads zeros.
struct PageWalk {
  const int* table;
  int step;          // +1 or -1: the direction
  int log2T;
  int from0, to0;    // needed: tokens in [from0, to0) or [0, prefix)
  int prefix;
  int num_pages;
  int group;         // of the entries held: pages 32 group .. + 31
  int z;             // this lane's page: its first group of 8 tokens in the tensor (of K; V's follow)
  uint32_t bad;      // entries with an id out of range
  int next_group, next_id;
  bool next_need;

  __device__ __forceinline__ void fetch(int g) {
    const int page = g * 32 + static_cast<int>(threadIdx.x % 32);
    // (positions stay below 2^31: a page that starts past the range is not needed)
    const long long tok = static_cast<long long>(page) << log2T;
    next_group = g;
    next_need = g >= 0 && (tok < prefix || (tok + (1 << log2T) > from0 && tok < to0));
    next_id = next_need ? table[page] : 0;
  }
  __device__ __forceinline__ void start(const int* row, int first_group) {
    table = row;
    group = -2;
    fetch(first_group);
  }
  // Holds the entries of `page`; returns its lane.
  __device__ __forceinline__ int hold(int page, int* status, int code) {
    const int g = page >> 5;
    if (g != group) {
      if (g != next_group) fetch(g);
      const bool good = next_need && next_id >= 0 && next_id < num_pages;
      bad = __ballot_sync(0xffffffffu, next_need && !good);
      if (next_need && !good) atomicExch(status, code);
      z = (good ? next_id : num_pages) << (log2T - 2);
      group = g;
      fetch(g + step);
    }
    return page & 31;
  }
};

}  // namespace eca
