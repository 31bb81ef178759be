// Host-side pieces of the paged cache's operators (include/attn_cache.h): the shared
// argument checks and what every launch fills in.
#pragma once
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_cache.h"
#include "attn_fwd_kernel.cuh"
#include "host_common.h"
#include "paged_common.cuh"

namespace eca_host {

inline eca::ChunkShape chunk_shape(const int* block_table, const int* lengths, const int* q_offsets, int total, int B,
                            int Hkv, int D, int page_size, int max_pages, int num_pages, int* status) {
  eca::ChunkShape s;
  s.block_table = block_table;
  s.lengths = lengths;
  s.q_offsets = q_offsets;
  s.status = status;
  s.total = total;
  s.B = B;
  s.Hkv = Hkv;
  s.D = D;
  s.page_size = page_size;
  s.max_pages = max_pages;
  s.num_pages = num_pages;
  s.bad_index_code = ATTN_ERR_BAD_INDEX;
  return s;
}

inline uint64_t cache_bytes(int Hkv, int D, int page_size, int num_pages) {
  return static_cast<uint64_t>(num_pages) * 2 * page_size * Hkv * D * 2;
}

// Positions are counted up to two key tiles past the longest context in an int.
inline int check_positions(int page_size, int max_pages) {
  return static_cast<uint64_t>(max_pages) * page_size > 0x7fffffffull - 512 ? ATTN_ERR_INVALID_ARG : ATTN_OK;
}

// Query-side arguments of the chunk operators.
inline int check_chunk_args(const void* q, int total, int Hq, int Hkv, int D, float scale, float softcap, int window,
                     const float* slopes, const int* prefix) {
  if (total < 0 || Hq < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!q && total > 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(softcap) || softcap < 0.f || window < 0) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || (slopes && !aligned(slopes, 4)) || (prefix && !aligned(prefix, 4))) return ATTN_ERR_UNALIGNED;
  // Packed (row, head) pairs are counted in an int.
  if (static_cast<uint64_t>(total) * Hq > 0x7fffffffull) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// A window that reaches past every context is none.
inline eca::ScoreForm score_form(float scale, float softcap, int window, const float* slopes, const int* prefix, int most) {
  return eca::ScoreForm{scale, softcap, slopes, prefix, window >= most ? 0 : window};
}

inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  cudaGetLastError();  // clear the error the failed launch recorded
  return ATTN_ERR_LAUNCH;
}

// Shared memory and register checks of a kernel, once per device and instance.
template <typename Kernel>
int configure(Kernel kernel, const Device& dev, std::atomic<uint64_t>* done, int smem, int min_regs) {
  const uint64_t bit = 1ull << dev.index;  // fewer than 64 devices
  if (done->load(std::memory_order_acquire) & bit) return ATTN_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return ATTN_ERR_CUDA;
  if (fa.numRegs < min_regs) return ATTN_ERR_LAUNCH;
  done->fetch_or(bit, std::memory_order_release);
  return ATTN_OK;
}

// Heads of a key/value group that share a query tile: the largest divisor of the
// group's size that fits its 128 rows.
inline int heads_per_tile(int group) {
  int hc = group < eca::kBlockM ? group : eca::kBlockM;
  while (group % hc != 0) --hc;
  return hc;
}

}  // namespace eca_host
