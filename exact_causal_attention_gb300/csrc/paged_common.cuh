// What the kernels over a paged cache and a ragged chunk of new tokens share: the
// request's sizes with their checks, and the score forms.
#pragma once
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

}  // namespace eca
