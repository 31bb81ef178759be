// Host side of the attention weights (include/attn_cache.h).
#include "cache_host.h"
#include "paged_mass.cuh"

namespace {

using namespace eca_host;

template <int D, bool BF16, int FORM, int kParts>
int launch_mass_parts(const CUtensorMap& tm_q, const CUtensorMap& tm_cache, const eca::MassParams& p, int grid,
                const Device& dev, cudaStream_t stream) {
  using L = eca::MassSmem<D>;
  static std::atomic<uint64_t> done{0};
  const int rc = configure(eca::paged_mass_kernel<D, BF16, FORM, kParts>, dev, &done, L::kDynamicBytes, 0);
  if (rc != ATTN_OK) return rc;
  return launched(launch_pdl(eca::paged_mass_kernel<D, BF16, FORM, kParts>, static_cast<unsigned>(grid),
                             eca::kMsThreads<kParts>, L::kDynamicBytes, stream, tm_q, tm_cache, p));
}

template <int D, bool BF16, int FORM>
int launch_mass(const CUtensorMap& tm_q, const CUtensorMap& tm_cache, const eca::MassParams& p, int grid,
                const Device& dev, cudaStream_t stream) {
  return p.hc * p.tq > 64 ? launch_mass_parts<D, BF16, FORM, 2>(tm_q, tm_cache, p, grid, dev, stream)
                          : launch_mass_parts<D, BF16, FORM, 1>(tm_q, tm_cache, p, grid, dev, stream);
}

template <int D, bool BF16>
int launch_mass_form(const CUtensorMap& tm_q, const CUtensorMap& tm_cache, const eca::MassParams& p, int grid,
                     const Device& dev, cudaStream_t stream) {
  if (p.f.softcap > 0.f && p.f.slopes != nullptr) {
    return launch_mass<D, BF16, eca::kFormBoth>(tm_q, tm_cache, p, grid, dev, stream);
  }
  if (p.f.softcap > 0.f) return launch_mass<D, BF16, eca::kFormCap>(tm_q, tm_cache, p, grid, dev, stream);
  if (p.f.slopes != nullptr) return launch_mass<D, BF16, eca::kFormBias>(tm_q, tm_cache, p, grid, dev, stream);
  return launch_mass<D, BF16, eca::kFormPlain>(tm_q, tm_cache, p, grid, dev, stream);
}

int mass_impl(bool bf16, const void* q, const float* lse, const void* cache, const int* block_table,
              const int* lengths, const int* q_offsets, float* mass, int accumulate, int total_q, int B, int Hq,
              int Hkv, int D, int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
              const float* alibi_slopes, const int* prefix_lens, attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc == ATTN_OK) rc = check_positions(page_size, max_pages);
  if (rc == ATTN_OK) rc = check_chunk_args(q, total_q, Hq, Hkv, D, scale, softcap, window, alibi_slopes, prefix_lens);
  if (rc != ATTN_OK) return rc;
  if (!mass || (!lse && total_q > 0) || (!q_offsets && total_q != B)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(mass, 4) || !aligned(lse, 4) || (q_offsets && !aligned(q_offsets, 4))) return ATTN_ERR_UNALIGNED;
  if (B > eca::kPlanMaxRequests) return ATTN_ERR_INVALID_ARG;
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
  p.f = score_form(scale, softcap, window, alibi_slopes, prefix_lens, max_pages * page_size);
  p.lse = lse;
  p.mass = mass;
  p.accumulate = accumulate != 0;
  p.Hq = Hq;
  p.hc = heads_per_tile(Hq / Hkv);
  p.chunks = Hq / Hkv / p.hc;
  // A step's tokens: what fits its columns, but no more than the requests have on average,
  // so that a decode step does not load its neighbours' rows.
  const int mean = total_q / B + (total_q % B != 0);
  p.tq = eca::kMsCols / p.hc;
  if (p.tq > mean) p.tq = mean > 0 ? mean : 1;
  p.idesc = eca::idesc_f16_f32acc(eca::kMsTile, (p.hc * p.tq + 15) / 16 * 16, bf16, false);
  p.small_plan = eca::line_is_small(
      B, static_cast<double>(B) * ((static_cast<double>(max_pages) * page_size) / (2 * eca::kMsTile) + 1));
  p.by_hc = eca::make_fast_div(p.hc);
  p.by_tq = eca::make_fast_div(p.tq);
  p.wait_limit_ns = kWaitLimitNs;
  p.timeout_code = ATTN_ERR_TIMEOUT;
  CUtensorMap tm_q, tm_cache;
  // Without rows nothing reads the queries' map.
  rc = head_rows_map(&tm_q, total_q > 0 ? q : cache, bf16, D, Hq, total_q > 0 ? total_q : 1,
                     static_cast<unsigned>(p.hc), static_cast<unsigned>(p.tq));
  if (rc == ATTN_OK) rc = cache_group_map(&tm_cache, cache, bf16, D, Hkv, page_size, num_pages);
  if (rc != ATTN_OK) return rc;
  const uint64_t tiles = static_cast<uint64_t>(B) * Hkv *
                         ((static_cast<uint64_t>(max_pages) * page_size + eca::kMsTile - 1) / eca::kMsTile);
  const int grid = tiles < static_cast<uint64_t>(dev.sm_count) ? static_cast<int>(tiles) : dev.sm_count;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) {
    return bf16 ? launch_mass_form<128, true>(tm_q, tm_cache, p, grid, dev, s)
                : launch_mass_form<128, false>(tm_q, tm_cache, p, grid, dev, s);
  }
  return bf16 ? launch_mass_form<64, true>(tm_q, tm_cache, p, grid, dev, s)
              : launch_mass_form<64, false>(tm_q, tm_cache, p, grid, dev, s);
}

}  // namespace

extern "C" {

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

}  // extern "C"
