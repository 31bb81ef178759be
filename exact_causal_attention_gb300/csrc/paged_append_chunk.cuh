// Append of a ragged chunk of new tokens to the paged cache: token i of request b goes
// to position t = lengths[b] - n_b + i, page block_table[b, t / T], offset t % T.
//
// A copy, bound by HBM (4 Hkv D bytes read and written per token) and, for a few
// tokens, by the launch.  A token's K and its V are each one contiguous run of
// Hkv x D values on both sides, so a token is copied by consecutive threads in 16-byte
// vectors, and the request and page of a token are looked up once per thread that
// copies a part of it (the offsets and the table stay in L1).
#pragma once
#include "paged_common.cuh"

namespace eca {

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) paged_append_chunk_kernel(const uint4* new_kv, uint4* cache,
                                                                            const ChunkShape s) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int half = s.Hkv * s.D / 8;  // 16-byte vectors of a token's K (and of its V)
  const long long vecs = static_cast<long long>(s.total) * 2 * half;
  const int log2T = 31 - __clz(s.page_size);
  const long long step = static_cast<long long>(gridDim.x) * kAppendThreads;
  for (long long v = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x; v < vecs; v += step) {
    const int t = static_cast<int>(v / (2 * half));
    const int in = static_cast<int>(v - static_cast<long long>(t) * (2 * half));
    const int b = request_of_row(s, t);
    if (b < 0) continue;
    const Request r = load_request(s, nullptr, b);
    const int pos = r.pos0 + t - r.row0;
    if (r.n == 0 || pos < 0) continue;
    const int page = s.block_table[static_cast<size_t>(b) * s.max_pages + (pos >> log2T)];
    if (page < 0 || page >= s.num_pages) {
      atomicExch(s.status, s.bad_index_code);
      continue;
    }
    const int kind = in >= half;
    const size_t row = (static_cast<size_t>(page) * 2 + kind) * s.page_size + (pos & (s.page_size - 1));
    cache[row * half + (in - kind * half)] = new_kv[v];
  }
}

}  // namespace eca
