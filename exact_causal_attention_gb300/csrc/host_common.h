// Host-side pieces that every translation unit of the library shares: the device's
// state, argument checks, the paged cache's tensor map and the launch call.  Their
// definitions are in attn_api.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "attn.h"

namespace eca_host {

constexpr unsigned long long kWaitLimitNs = 2000000000ull;  // 2 s per single wait

struct Device {
  int index;     // CUDA device ordinal
  int sm_count;
  int* status;   // device status word
};

// The current device, probed on first use.  ATTN_OK, or a negative status.
int current_device(Device* out);

bool aligned(const void* p, uintptr_t a);

// Do [a, a + na) and [b, b + nb) intersect?
bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb);

uint64_t align256(uint64_t x);

// Pointers, sizes and limits of a paged cache; needs no GPU.
int check_paged_args(const void* cache, const int* block_table, const int* lengths, int B, int Hkv, int D,
                     int page_size, int max_pages, int num_pages);

// Paged cache [P, 2, T, Hkv, D] in groups of 8 tokens, as a rank-5 map (64 columns, 8 tokens,
// D/64 column blocks, P*2*T/8 groups, Hkv): one box is one head's K or V of one page, 128-byte
// swizzle, in shared memory group by group, column block by column block.
int cache_group_map(CUtensorMap* map, const void* cache, bool bf16, int D, int Hkv, int T, int P);

// Rows [R, H, D] of 16-bit elements (D contiguous) as a rank-3 map (D, H, R): one box
// is 64 columns of box_h heads of box_r rows, 128-byte swizzle; heads fastest in
// shared memory; what lies outside reads as zero.
int head_rows_map(CUtensorMap* map, const void* ptr, bool bf16, int D, int H, int R, unsigned box_h, unsigned box_r);

bool programmatic_launch_enabled();

// Launch with programmatic stream serialisation: the grid may be scheduled before
// the grid ahead of it on the stream has finished.  Only kernels that call
// grid_dependency_wait before touching global memory are launched this way.
// Between two back-to-back attention launches the second then starts as soon as
// the first completes, instead of after the full stream-ordered launch latency.
// ECA_PDL=0 in the environment (read once per process) launches in plain stream
// order instead, with the same results; it exists to measure the difference.
// launch_pdl_cluster launches clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                               cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (programmatic_launch_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  return launch_pdl_cluster(kernel, grid, block, smem, 1, stream, std::forward<Args>(args)...);
}

}  // namespace eca_host
