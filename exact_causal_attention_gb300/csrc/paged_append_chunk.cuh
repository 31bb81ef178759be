// Append of a ragged chunk of new tokens to the paged cache: token i of request b goes
// to position t = lengths[b] - n_b + i, page block_table[b, t / T], offset t % T.
//
// A copy, bound by HBM (4 Hkv D bytes read and as many written per token) and, for a few
// tokens, by the launch.  A token's K and its V are each one contiguous run of Hkv x D values on both
// sides.  A block takes a few consecutive tokens: one thread per token finds its request and page, then all
// threads copy 16-byte vectors, several in flight each.  (With every thread looking up its own
// vectors' tokens the copy of 3500-token prompts was bound by instructions: 12.1 us, now 8.1.)
#pragma once
#include "attn_fwd_kernel.cuh"
#include "paged_common.cuh"

namespace eca {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 4;  // most tokens of a block at a time

__global__ void __launch_bounds__(kAppendThreads) paged_append_chunk_kernel(const uint4* new_kv, uint4* cache,
                                                                            const ChunkShape s, const FastDiv by_half,
                                                                            int tokens) {
  __shared__ long long to[2 * kAppendTokens];  // where each token's K and V start in the cache, or -1
  grid_launch_dependents();
  grid_dependency_wait();
  const int half = by_half.d;  // 16-byte vectors of a token's K (and of its V)
  const int log2T = 31 - __clz(s.page_size);
  for (long long first = static_cast<long long>(blockIdx.x) * tokens; first < s.total;
       first += static_cast<long long>(gridDim.x) * tokens) {
    const int count = static_cast<int>(min(static_cast<long long>(tokens), s.total - first));
    if (threadIdx.x < static_cast<unsigned>(count)) {
      const int t = static_cast<int>(first) + threadIdx.x;
      long long k = -1, v = -1;
      const int b = request_of_row(s, t);
      if (b >= 0) {
        const Request r = load_request(s, nullptr, b);
        const int pos = r.pos0 + t - r.row0;
        if (r.n > 0 && pos >= 0) {
          const int page = s.block_table[static_cast<size_t>(b) * s.max_pages + (pos >> log2T)];
          if (page < 0 || page >= s.num_pages) {
            atomicExch(s.status, s.bad_index_code);
          } else {
            k = ((static_cast<long long>(page) * 2 << log2T) + (pos & (s.page_size - 1))) * half;
            v = k + (static_cast<long long>(half) << log2T);
          }
        }
      }
      to[2 * threadIdx.x] = k;
      to[2 * threadIdx.x + 1] = v;
    }
    __syncthreads();
    const uint4* src = new_kv + first * 2 * half;
    const int vecs = count * 2 * half;
    constexpr int kFlight = 4;
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kFlight * kAppendThreads) {
      uint4 x[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int i = i0 + f * kAppendThreads;
        if (i < vecs) x[f] = src[i];
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int i = i0 + f * kAppendThreads;
        if (i < vecs) {
          const int part = fast_div(i, by_half);
          if (to[part] >= 0) cache[to[part] + (i - part * half)] = x[f];
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace eca
