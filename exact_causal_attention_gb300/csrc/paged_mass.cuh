// Attention weight that every cached token received from a ragged chunk.  One warp per
// (request, key/value head, token), walking the chunk's rows and heads in order.
#pragma once
#include "paged_common.cuh"

namespace eca {

struct MassParams {
  ChunkShape s;
  ScoreForm f;
  const void* q;      // [total, Hq, D] 16-bit
  const void* cache;
  const float* lse;   // [total, Hq]
  float* mass;        // [B, Hkv, max_pages * page_size]
  int accumulate;
  int Hq;
};

// Score of one key from q . k (natural units).
__device__ __forceinline__ float form_score(const ScoreForm& f, float dot, float slope, int away) {
  float x = dot * f.scale;
  if (f.softcap > 0.f) x = f.softcap * tanhf(x / f.softcap);
  return x - slope * fabsf(static_cast<float>(away));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) paged_mass_kernel(const MassParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int most = p.s.max_pages * p.s.page_size;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (w >= static_cast<long long>(p.s.B) * p.s.Hkv * most) return;
  const int j = static_cast<int>(w % most);
  const int kvh = static_cast<int>(w / most % p.s.Hkv), b = static_cast<int>(w / most / p.s.Hkv);
  const Request r = load_request(p.s, &p.f, b);
  float sum = 0.f;
  if (j < r.len) {
    const int log2T = 31 - __clz(p.s.page_size), group = p.Hq / p.s.Hkv;
    bool seen = false;
    int page = -1;
    float2 kv[D / 64];
    for (int i = 0; i < r.n; ++i) {
      const int pos = r.pos0 + i;
      if (!((j <= pos && (p.f.window == 0 || j > pos - p.f.window)) || j < r.prefix)) continue;
      if (!seen) {
        seen = true;
        page = p.s.block_table[static_cast<size_t>(b) * p.s.max_pages + (j >> log2T)];
        if (page < 0 || page >= p.s.num_pages) {
          if (lane == 0) atomicExch(p.s.status, p.s.bad_index_code);
          page = -1;
        } else {
          const size_t krow =
              (static_cast<size_t>(page) * 2 * p.s.page_size + (j & (p.s.page_size - 1))) * p.s.Hkv + kvh;
          const uint32_t* k = reinterpret_cast<const uint32_t*>(p.cache) + krow * (D / 2);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) kv[x] = to_f32x2<BF16>(k[lane + 32 * x]);
        }
      }
      if (page < 0) break;
      for (int h = kvh * group; h < (kvh + 1) * group; ++h) {
        const size_t row = static_cast<size_t>(r.row0 + i) * p.Hq + h;
        const float lse = p.lse[row];
        if (lse == -INFINITY) continue;
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q) + row * (D / 2);
        float dot = 0.f;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          const float2 qv = to_f32x2<BF16>(q[lane + 32 * x]);
          dot += qv.x * kv[x].x + qv.y * kv[x].y;
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        sum += expf(form_score(p.f, dot, p.f.slopes != nullptr ? p.f.slopes[h] : 0.f, pos - j) - lse);
      }
    }
    if (p.accumulate && !seen) return;
  } else if (p.accumulate) {
    return;
  }
  if (lane == 0) p.mass[w] = p.accumulate ? p.mass[w] + sum : sum;
}

}  // namespace eca
