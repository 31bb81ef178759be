// Host side of the chunk attention (include/attn_cache.h).
#include "cache_host.h"
#include "paged_prefill.cuh"

namespace {

using namespace eca_host;

struct PrefillShape {
  int hc, chunks, tq;
  int grid;             // CTAs: no more than there can be work for
  uint64_t o_bytes, lse_bytes, bytes;
};

constexpr int kPrefillMaxCtas = 160;

PrefillShape prefill_shape(int total_q, int B, int Hq, int Hkv, int D, int page_size, int max_pages) {
  PrefillShape sh;
  const int group = Hq / Hkv;
  sh.hc = heads_per_tile(group);
  sh.chunks = group / sh.hc;
  sh.tq = eca::kPfTile / sh.hc;
  // At most so many units (pairs of query tiles per key/value head and chunk) of at most so many key tiles.
  const double pairs = static_cast<double>(total_q) / (2 * sh.tq) + (total_q < B ? total_q : B);
  const double tiles = (static_cast<double>(max_pages) * page_size + eca::kPfTile - 1) / eca::kPfTile;
  const double most = pairs * Hkv * sh.chunks * (tiles + eca::kPfUnitCost) / eca::kPfMinCost + 1;
  sh.grid = most < kPrefillMaxCtas ? static_cast<int>(most) : kPrefillMaxCtas;
  sh.o_bytes = align256(2ull * sh.grid * 256 * D * 4);
  sh.lse_bytes = align256(2ull * sh.grid * 256 * 4);
  sh.bytes = sh.o_bytes + sh.lse_bytes + align256(4ull * sh.grid * eca::kPfSplitWords);
  return sh;
}

template <int D, bool BF16, int FORM>
int launch_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_cache, const eca::PrefillParams& p, int grid,
                   const Device& dev, cudaStream_t stream) {
  using L = eca::PrefillSmem<D>;
  static std::atomic<uint64_t> done{0};
  const int rc = configure(eca::paged_prefill_kernel<D, BF16, FORM>, dev, &done, L::kDynamicBytes,
                           (256 * eca::kRegsSoftmax + 128 * eca::kRegsControl + eca::kPfThreads - 1) / eca::kPfThreads);
  if (rc != ATTN_OK) return rc;
  const int r = launched(launch_pdl(eca::paged_prefill_kernel<D, BF16, FORM>, static_cast<unsigned>(grid),
                                    eca::kPfThreads, L::kDynamicBytes, stream, tm_q, tm_cache, p));
  if (r != ATTN_OK) return r;
  constexpr int kRows = 32;
  return launched(launch_pdl(eca::paged_prefill_combine<D, BF16>, static_cast<unsigned>(grid * (256 / kRows)), 2 * D, 0,
                             stream, p, kRows));
}

template <int D, bool BF16>
int launch_prefill_form(const CUtensorMap& tm_q, const CUtensorMap& tm_cache, const eca::PrefillParams& p, int grid,
                        const Device& dev, cudaStream_t stream) {
  if (p.f.softcap > 0.f && p.f.slopes != nullptr) {
    return launch_prefill<D, BF16, eca::kFormBoth>(tm_q, tm_cache, p, grid, dev, stream);
  }
  if (p.f.softcap > 0.f) return launch_prefill<D, BF16, eca::kFormCap>(tm_q, tm_cache, p, grid, dev, stream);
  if (p.f.slopes != nullptr) return launch_prefill<D, BF16, eca::kFormBias>(tm_q, tm_cache, p, grid, dev, stream);
  return launch_prefill<D, BF16, eca::kFormPlain>(tm_q, tm_cache, p, grid, dev, stream);
}

int prefill_impl(bool bf16, const void* q, const void* cache, const int* block_table, const int* lengths,
                 const int* q_offsets, void* out, float* lse, int total_q, int B, int Hq, int Hkv, int D,
                 int page_size, int max_pages, int num_pages, float scale, float softcap, int window,
                 const float* alibi_slopes, const int* prefix_lens, void* workspace, size_t workspace_bytes,
                 attn_stream_t stream) {
  int rc = check_paged_args(cache, block_table, lengths, B, Hkv, D, page_size, max_pages, num_pages);
  if (rc == ATTN_OK) rc = check_positions(page_size, max_pages);
  if (rc == ATTN_OK) rc = check_chunk_args(q, total_q, Hq, Hkv, D, scale, softcap, window, alibi_slopes, prefix_lens);
  if (rc != ATTN_OK) return rc;
  if (!q_offsets || (!out && total_q > 0) || B > eca::kPlanMaxRequests) return ATTN_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q_offsets, 4) || (lse && !aligned(lse, 4))) return ATTN_ERR_UNALIGNED;
  if (total_q == 0) return ATTN_OK;
  const uint64_t qbytes = static_cast<uint64_t>(total_q) * Hq * D * 2;
  if (overlaps(out, qbytes, q, qbytes) ||
      overlaps(out, qbytes, cache, cache_bytes(Hkv, D, page_size, num_pages))) {
    return ATTN_ERR_INVALID_ARG;
  }
  const PrefillShape sh = prefill_shape(total_q, B, Hq, Hkv, D, page_size, max_pages);
  if (!workspace || workspace_bytes < sh.bytes) return ATTN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return ATTN_ERR_UNALIGNED;
  if (overlaps(workspace, sh.bytes, q, qbytes) || overlaps(workspace, sh.bytes, out, qbytes) ||
      overlaps(workspace, sh.bytes, cache, cache_bytes(Hkv, D, page_size, num_pages))) {
    return ATTN_ERR_INVALID_ARG;
  }
  Device dev;
  rc = current_device(&dev);
  if (rc != ATTN_OK) return rc;
  eca::PrefillParams p;
  p.s = chunk_shape(block_table, lengths, q_offsets, total_q, B, Hkv, D, page_size, max_pages, num_pages, dev.status);
  p.f = score_form(scale, softcap, window, alibi_slopes, prefix_lens, max_pages * page_size);
  p.out = out;
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sh.o_bytes);
  p.split = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + sh.o_bytes + sh.lse_bytes);
  p.Hq = Hq;
  p.hc = sh.hc;
  p.chunks = sh.chunks;
  p.tq = sh.tq;
  p.by_hc = eca::make_fast_div(sh.hc);
  p.small_plan = eca::line_is_small(B, static_cast<double>(total_q) / (2 * sh.tq) + B);
  p.scale_log2e = scale * eca::kLog2e;
  p.wait_limit_ns = kWaitLimitNs;
  p.timeout_code = ATTN_ERR_TIMEOUT;
  CUtensorMap tm_q, tm_cache;
  rc = head_rows_map(&tm_q, q, bf16, D, Hq, total_q, static_cast<unsigned>(sh.hc), static_cast<unsigned>(sh.tq));
  if (rc == ATTN_OK) rc = cache_group_map(&tm_cache, cache, bf16, D, Hkv, page_size, num_pages);
  if (rc != ATTN_OK) return rc;
  const int grid = sh.grid < dev.sm_count ? sh.grid : dev.sm_count;  // one CTA per SM
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) {
    return bf16 ? launch_prefill_form<128, true>(tm_q, tm_cache, p, grid, dev, s)
                : launch_prefill_form<128, false>(tm_q, tm_cache, p, grid, dev, s);
  }
  return bf16 ? launch_prefill_form<64, true>(tm_q, tm_cache, p, grid, dev, s)
              : launch_prefill_form<64, false>(tm_q, tm_cache, p, grid, dev, s);
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
  if (total_q < 1 || B < 1 || B > eca::kPlanMaxRequests || Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return 0;
  if ((D != 64 && D != 128) || max_pages < 1 || page_size < 8 || page_size > 64) return 0;
  return static_cast<size_t>(prefill_shape(total_q, B, Hq, Hkv, D, page_size, max_pages).bytes);
}

}  // extern "C"
