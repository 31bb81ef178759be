// Host side of the append of a chunk and the eviction (include/attn_cache.h).
#include "cache_host.h"
#include "paged_append_chunk.cuh"
#include "paged_evict.cuh"

using namespace eca_host;

extern "C" {

int attn_paged_append_chunk(const void* new_kv, void* cache, const int* block_table, const int* lengths,
                            const int* q_offsets, int total, int B, int Hkv, int D, int page_size, int max_pages,
                            int num_pages, attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc == ATTN_OK) rc = check_positions(page_size, max_pages);
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
  // A few tokens a block where that still fills the GPU.
  const int tokens = total >= 2 * dev.sm_count * eca::kAppendTokens ? eca::kAppendTokens : 1;
  const long long want = (total + tokens - 1LL) / tokens, cap = dev.sm_count * 8LL;
  return launched(launch_pdl(eca::paged_append_chunk_kernel, static_cast<unsigned>(want < cap ? want : cap),
                             eca::kAppendThreads, 0, reinterpret_cast<cudaStream_t>(stream),
                             static_cast<const uint4*>(new_kv), static_cast<uint4*>(cache), s,
                             eca::make_fast_div(Hkv * D / 8), tokens));
}

int attn_paged_evict(void* cache, const int* block_table, const int* lengths, const float* mass, int* kept,
                     int* new_lengths, float* mass_out, int B, int Hkv, int D, int page_size, int max_pages,
                     int num_pages, int budget, int recent, attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc == ATTN_OK) rc = check_positions(page_size, max_pages);
  if (rc != ATTN_OK) return rc;
  if (!mass || !kept || !new_lengths) return ATTN_ERR_INVALID_ARG;
  if (budget < 1 || budget > max_pages * page_size || recent < 0 || recent > budget) return ATTN_ERR_INVALID_ARG;
  if (!aligned(mass, 4) || !aligned(kept, 4) || !aligned(new_lengths, 4) || (mass_out && !aligned(mass_out, 4))) {
    return ATTN_ERR_UNALIGNED;
  }
  const uint64_t heads = static_cast<uint64_t>(B) * Hkv;
  const uint64_t mass_bytes = heads * max_pages * page_size * 4, kept_bytes = heads * budget * 4;
  const uint64_t movers = heads * 2 * eca::kMoveCluster;
  if (movers > 0x7fffffffull || mass_bytes > (1ull << 40)) return ATTN_ERR_INVALID_ARG;
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
  // Few heads with long contexts are spread over clusters of blocks, 8192 tokens a block (32768 tokens
  // of 8 heads: 30 us with one block a head, 26 with two, 25 with four; 8192 tokens of 64 heads: 39 with one,
  // 40 with two).  Keys go to shared memory where every block's fit.
  const int most = max_pages * page_size;
  int cluster = 1;
  while (cluster < eca::kSelMaxCluster && heads * cluster * 2 <= static_cast<uint64_t>(dev.sm_count) &&
         most / cluster > 8192) {
    cluster *= 2;
  }
  const int share = static_cast<int>((most + 32LL * cluster - 1) / (32LL * cluster) * 32);
  if (share <= eca::kSelSmemTokens) {
    static std::atomic<uint64_t> done{0};
    rc = configure(eca::paged_evict_select_kernel<true>, dev, &done, eca::kSelSmemTokens * 4, 0);
    if (rc != ATTN_OK) return rc;
    rc = launched(launch_pdl_cluster(eca::paged_evict_select_kernel<true>, static_cast<unsigned>(heads * cluster),
                                     eca::kSelThreads, static_cast<size_t>(share) * 4, static_cast<unsigned>(cluster), s,
                                     p, cluster));
  } else {
    rc = launched(
        launch_pdl(eca::paged_evict_select_kernel<false>, static_cast<unsigned>(heads), eca::kSelThreads, 0, s, p, 1));
  }
  if (rc != ATTN_OK) return rc;
  auto move = [&](auto kernel, std::atomic<uint64_t>* done) -> int {
    const int r = configure(kernel, dev, done, eca::kMoveBytes, 0);
    if (r != ATTN_OK) return r;
    return launched(
        launch_pdl(kernel, static_cast<unsigned>(movers), eca::kMoveThreads, static_cast<size_t>(eca::kMoveBytes), s, p));
  };
  static std::atomic<uint64_t> done128{0}, done64{0};
  return D == 128 ? move(eca::paged_evict_move_kernel<128>, &done128) : move(eca::paged_evict_move_kernel<64>, &done64);
}

}  // extern "C"
