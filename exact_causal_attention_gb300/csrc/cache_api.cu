// Host side of include/attn_cache.h: argument checks and launches of the paged cache's
// operators.  The one-token decode with score forms is in attn_api.cu, beside
// attn_decode_paged.
#include <atomic>
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

// A window that reaches past every context is none.
eca::ScoreForm score_form(float scale, float softcap, int window, const float* slopes, const int* prefix, int most) {
  return eca::ScoreForm{scale, softcap, slopes, prefix, window >= most ? 0 : window};
}

int launched(cudaError_t e) {
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
int heads_per_tile(int group) {
  int hc = group < eca::kPfTile ? group : eca::kPfTile;
  while (group % hc != 0) --hc;
  return hc;
}

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
  if (rc == ATTN_OK) rc = check_chunk_args(q, total_q, Hq, Hkv, D, scale, softcap, window, alibi_slopes, prefix_lens);
  if (rc != ATTN_OK) return rc;
  if (!q_offsets || (!out && total_q > 0) || B > eca::kPfMaxRequests) return ATTN_ERR_INVALID_ARG;
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
  p.scale_log2e = scale * eca::kLog2e;
  p.wait_limit_ns = kWaitLimitNs;
  p.timeout_code = ATTN_ERR_TIMEOUT;
  CUtensorMap tm_q, tm_cache;
  rc = head_rows_map(&tm_q, q, bf16, D, Hq, total_q, static_cast<unsigned>(sh.hc), static_cast<unsigned>(sh.tq));
  if (rc == ATTN_OK) rc = paged_cache_map(&tm_cache, cache, bf16, D, Hkv, page_size, num_pages);
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
  p.f = score_form(scale, softcap, window, alibi_slopes, prefix_lens, max_pages * page_size);
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
  if (total_q < 1 || B < 1 || B > eca::kPfMaxRequests || Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return 0;
  if ((D != 64 && D != 128) || max_pages < 1 || page_size < 8 || page_size > 64) return 0;
  return static_cast<size_t>(prefill_shape(total_q, B, Hq, Hkv, D, page_size, max_pages).bytes);
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
