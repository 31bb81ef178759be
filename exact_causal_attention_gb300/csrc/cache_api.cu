// Host side of include/attn_cache.h: argument checks and launches of the paged cache's
// operators.  The one-token decode with score forms is in attn_api.cu, beside
// attn_decode_paged.
#include <cmath>
#include <cstdint>

#include "attn_cache.h"
#include "host_common.h"
#include "paged_append_chunk.cuh"
#include "paged_evict.cuh"
#include "paged_mass.cuh"
#include "paged_prefill.cuh"

namespace {

using namespace eca_host;

eca::ChunkShape chunk_shape(const int* block_table, const int* lengths, const int* q_offsets, int total, int B,
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

uint64_t cache_bytes(int Hkv, int D, int page_size, int num_pages) {
  return static_cast<uint64_t>(num_pages) * 2 * page_size * Hkv * D * 2;
}

// Query-side arguments of the chunk operators.
int check_chunk_args(const void* q, int total, int Hq, int Hkv, int D, float scale, float softcap, int window,
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

int launched(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  cudaGetLastError();  // clear the error the failed launch recorded
  return ATTN_ERR_LAUNCH;
}

template <int D, bool BF16>
int launch_prefill(const eca::PrefillParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.s.total) * p.Hq + 3) / 4);
  return launched(launch_pdl(eca::paged_prefill_kernel<D, BF16>, grid, 128, 0, stream, p));
}

int prefill_impl(bool bf16, const void* q, const void* cache, const int* block_table, const int* lengths,
                 const int* q_offsets, void* out, float* lse, int total_q, int B, int Hq, int Hkv, int D,
                 int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
                 const float* alibi_slopes, const int* prefix_lens, void* workspace, size_t workspace_bytes,
                 attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc == ATTN_OK) rc = check_chunk_args(q, total_q, Hq, Hkv, D, scale, softcap, window, alibi_slopes, prefix_lens);
  if (rc != ATTN_OK) return rc;
  if (!q_offsets || (!out && total_q > 0)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q_offsets, 4) || (lse && !aligned(lse, 4))) return ATTN_ERR_UNALIGNED;
  if (total_q == 0) return ATTN_OK;
  const uint64_t qbytes = static_cast<uint64_t>(total_q) * Hq * D * 2;
  if (overlaps(out, qbytes, q, qbytes) ||
      overlaps(out, qbytes, cache, cache_bytes(Hkv, D, page_size, num_pages))) {
    return ATTN_ERR_INVALID_ARG;
  }
  const uint64_t need = attn_prefill_workspace_bytes(total_q, B, Hq, Hkv, D, page_size, max_pages);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return ATTN_ERR_UNALIGNED;
    if (overlaps(workspace, need, q, qbytes) || overlaps(workspace, need, out, qbytes)) return ATTN_ERR_INVALID_ARG;
  }
  Device dev;
  rc = current_device(&dev);
  if (rc != ATTN_OK) return rc;
  eca::PrefillParams p;
  p.s = chunk_shape(block_table, lengths, q_offsets, total_q, B, Hkv, D, page_size, max_pages, num_pages, dev.status);
  p.f = eca::ScoreForm{scale, softcap, alibi_slopes, prefix_lens, window};
  p.q = q;
  p.cache = cache;
  p.out = out;
  p.lse = lse;
  p.Hq = Hq;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) return bf16 ? launch_prefill<128, true>(p, s) : launch_prefill<128, false>(p, s);
  return bf16 ? launch_prefill<64, true>(p, s) : launch_prefill<64, false>(p, s);
}

template <int D, bool BF16>
int launch_mass(const eca::MassParams& p, cudaStream_t stream) {
  const long long warps = static_cast<long long>(p.s.B) * p.s.Hkv * p.s.max_pages * p.s.page_size;
  return launched(
      launch_pdl(eca::paged_mass_kernel<D, BF16>, static_cast<unsigned>((warps + 3) / 4), 128, 0, stream, p));
}

int mass_impl(bool bf16, const void* q, const float* lse, const void* cache, const int* block_table,
              const int* lengths, const int* q_offsets, float* mass, int accumulate, int total_q, int B, int Hq,
              int Hkv, int D, int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
              const float* alibi_slopes, const int* prefix_lens, attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc == ATTN_OK) rc = check_chunk_args(q, total_q, Hq, Hkv, D, scale, softcap, window, alibi_slopes, prefix_lens);
  if (rc != ATTN_OK) return rc;
  if (!mass || (!lse && total_q > 0) || (!q_offsets && total_q != B)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(mass, 4) || !aligned(lse, 4) || (q_offsets && !aligned(q_offsets, 4))) return ATTN_ERR_UNALIGNED;
  const uint64_t cells = static_cast<uint64_t>(B) * Hkv * max_pages * page_size;
  if (cells > (1ull << 33)) return ATTN_ERR_INVALID_ARG;
  if (overlaps(mass, cells * 4, q, static_cast<uint64_t>(total_q) * Hq * D * 2) ||
      overlaps(mass, cells * 4, lse, static_cast<uint64_t>(total_q) * Hq * 4) ||
      overlaps(mass, cells * 4, cache, cache_bytes(Hkv, D, page_size, num_pages))) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (total_q == 0 && accumulate) return ATTN_OK;
  Device dev;
  rc = current_device(&dev);
  if (rc != ATTN_OK) return rc;
  eca::MassParams p;
  p.s = chunk_shape(block_table, lengths, q_offsets, total_q, B, Hkv, D, page_size, max_pages, num_pages, dev.status);
  p.f = eca::ScoreForm{scale, softcap, alibi_slopes, prefix_lens, window};
  p.q = q;
  p.cache = cache;
  p.lse = lse;
  p.mass = mass;
  p.accumulate = accumulate;
  p.Hq = Hq;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) return bf16 ? launch_mass<128, true>(p, s) : launch_mass<128, false>(p, s);
  return bf16 ? launch_mass<64, true>(p, s) : launch_mass<64, false>(p, s);
}

}  // namespace

extern "C" {

int attn_prefill_paged(const void* q, const void* cache, const int* block_table, const int* lengths,
                       const int* q_offsets, void* out, float* lse, int total_q, int B, int Hq, int Hkv, int D,
                       int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
                       const float* alibi_slopes, const int* prefix_lens, void* workspace, size_t workspace_bytes,
                       attn_stream_t stream) {
  return prefill_impl(false, q, cache, block_table, lengths, q_offsets, out, lse, total_q, B, Hq, Hkv, D, page_size,
                      max_pages, num_pages, scale, softcap, window, alibi_slopes, prefix_lens, workspace,
                      workspace_bytes, stream);
}

int attn_prefill_paged_bf16(const void* q, const void* cache, const int* block_table, const int* lengths,
                            const int* q_offsets, void* out, float* lse, int total_q, int B, int Hq, int Hkv, int D,
                            int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
                            const float* alibi_slopes, const int* prefix_lens, void* workspace,
                            size_t workspace_bytes, attn_stream_t stream) {
  return prefill_impl(true, q, cache, block_table, lengths, q_offsets, out, lse, total_q, B, Hq, Hkv, D, page_size,
                      max_pages, num_pages, scale, softcap, window, alibi_slopes, prefix_lens, workspace,
                      workspace_bytes, stream);
}

size_t attn_prefill_workspace_bytes(int total_q, int B, int Hq, int Hkv, int D, int page_size, int max_pages) {
  (void)total_q, (void)B, (void)Hq, (void)Hkv, (void)D, (void)page_size, (void)max_pages;
  return 0;
}

int attn_paged_append_chunk(const void* new_kv, void* cache, const int* block_table, const int* lengths,
                            const int* q_offsets, int total, int B, int Hkv, int D, int page_size, int max_pages,
                            int num_pages, attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc != ATTN_OK) return rc;
  if (total < 0 || !q_offsets || (!new_kv && total > 0)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(new_kv, 16) || !aligned(q_offsets, 4)) return ATTN_ERR_UNALIGNED;
  if (overlaps(new_kv, static_cast<uint64_t>(total) * 2 * Hkv * D * 2, cache,
               cache_bytes(Hkv, D, page_size, num_pages))) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (total == 0) return ATTN_OK;
  Device dev;
  rc = current_device(&dev);
  if (rc != ATTN_OK) return rc;
  const eca::ChunkShape s =
      chunk_shape(block_table, lengths, q_offsets, total, B, Hkv, D, page_size, max_pages, num_pages, dev.status);
  const long long vecs = static_cast<long long>(total) * 2 * Hkv * D / 8;
  const long long want = (vecs + eca::kAppendThreads - 1) / eca::kAppendThreads, cap = dev.sm_count * 8LL;
  return launched(launch_pdl(eca::paged_append_chunk_kernel, static_cast<unsigned>(want < cap ? want : cap),
                             eca::kAppendThreads, 0, reinterpret_cast<cudaStream_t>(stream),
                             static_cast<const uint4*>(new_kv), static_cast<uint4*>(cache), s));
}

int attn_paged_mass(const void* q, const float* lse, const void* cache, const int* block_table, const int* lengths,
                    const int* q_offsets, float* mass, int accumulate, int total_q, int B, int Hq, int Hkv, int D,
                    int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
                    const float* alibi_slopes, const int* prefix_lens, attn_stream_t stream) {
  return mass_impl(false, q, lse, cache, block_table, lengths, q_offsets, mass, accumulate, total_q, B, Hq, Hkv, D,
                   page_size, max_pages, num_pages, scale, softcap, window, alibi_slopes, prefix_lens, stream);
}

int attn_paged_mass_bf16(const void* q, const float* lse, const void* cache, const int* block_table,
                         const int* lengths, const int* q_offsets, float* mass, int accumulate, int total_q, int B,
                         int Hq, int Hkv, int D, int page_size, int max_pages, int num_pages, float scale,
                         float softcap, int window, const float* alibi_slopes, const int* prefix_lens,
                         attn_stream_t stream) {
  return mass_impl(true, q, lse, cache, block_table, lengths, q_offsets, mass, accumulate, total_q, B, Hq, Hkv, D,
                   page_size, max_pages, num_pages, scale, softcap, window, alibi_slopes, prefix_lens, stream);
}

int attn_paged_evict(void* cache, const int* block_table, const int* lengths, const float* mass, int* kept,
                     int* new_lengths, float* mass_out, int B, int Hkv, int D, int page_size, int max_pages,
                     int num_pages, int budget, int recent, attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc != ATTN_OK) return rc;
  if (!mass || !kept || !new_lengths) return ATTN_ERR_INVALID_ARG;
  if (budget < 1 || budget > max_pages * page_size || recent < 0 || recent > budget) return ATTN_ERR_INVALID_ARG;
  if (!aligned(mass, 4) || !aligned(kept, 4) || !aligned(new_lengths, 4) || (mass_out && !aligned(mass_out, 4))) {
    return ATTN_ERR_UNALIGNED;
  }
  const uint64_t heads = static_cast<uint64_t>(B) * Hkv;
  const uint64_t mass_bytes = heads * max_pages * page_size * 4, kept_bytes = heads * budget * 4;
  const int parts = 2 * (D / (8 * eca::kMoveSlice));
  if (heads * parts > 0x7fffffffull || mass_bytes > (1ull << 40)) return ATTN_ERR_INVALID_ARG;
  const uint64_t c_bytes = cache_bytes(Hkv, D, page_size, num_pages);
  if (overlaps(kept, kept_bytes, mass, mass_bytes) || overlaps(kept, kept_bytes, cache, c_bytes) ||
      overlaps(mass, mass_bytes, cache, c_bytes)) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (mass_out != nullptr &&
      ((mass_out != mass && overlaps(mass_out, mass_bytes, mass, mass_bytes)) ||
       overlaps(mass_out, mass_bytes, cache, c_bytes) || overlaps(mass_out, mass_bytes, kept, kept_bytes))) {
    return ATTN_ERR_INVALID_ARG;
  }
  Device dev;
  rc = current_device(&dev);
  if (rc != ATTN_OK) return rc;
  eca::EvictParams p;
  p.s = chunk_shape(block_table, lengths, nullptr, 0, B, Hkv, D, page_size, max_pages, num_pages, dev.status);
  p.cache = cache;
  p.mass = mass;
  p.kept = kept;
  p.new_lengths = new_lengths;
  p.mass_out = mass_out;
  p.budget = budget;
  p.recent = recent;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rc = launched(launch_pdl(eca::paged_evict_select_kernel, static_cast<unsigned>(heads), eca::kSelThreads, 0, s, p));
  if (rc != ATTN_OK) return rc;
  return launched(
      launch_pdl(eca::paged_evict_move_kernel, static_cast<unsigned>(heads * parts), eca::kMoveThreads, 0, s, p));
}

}  // extern "C"
