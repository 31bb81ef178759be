// Attention of a ragged chunk of new tokens over a paged cache, with the score forms.
// One warp per (row, query head), walking the visible keys in order with the
// online-softmax recurrence.
#pragma once
#include "paged_common.cuh"

namespace eca {

struct PrefillParams {
  ChunkShape s;
  ScoreForm f;
  const void* q;      // [total, Hq, D] 16-bit
  const void* cache;
  void* out;
  float* lse;         // [total, Hq] or null
  int Hq;
};

// Score of one key from q . k (natural units).
__device__ __forceinline__ float form_score(const ScoreForm& f, float dot, float slope, int away) {
  float x = dot * f.scale;
  if (f.softcap > 0.f) x = f.softcap * tanhf(x / f.softcap);
  return x - slope * fabsf(static_cast<float>(away));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) paged_prefill_kernel(const PrefillParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const long long w = static_cast<long long>(blockIdx.x) * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (w >= static_cast<long long>(p.s.total) * p.Hq) return;
  const int t = static_cast<int>(w / p.Hq), h = static_cast<int>(w % p.Hq);
  const int b = request_of_row(p.s, t);
  if (b < 0) return;
  const Request r = load_request(p.s, &p.f, b);
  if (r.n == 0) return;
  const int pos = r.pos0 + t - r.row0;
  const int kvh = h / (p.Hq / p.s.Hkv);
  const int log2T = 31 - __clz(p.s.page_size);
  const float slope = p.f.slopes != nullptr ? p.f.slopes[h] : 0.f;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q) + w * (D / 2);
  float2 qv[D / 64];
  float2 o[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    qv[i] = to_f32x2<BF16>(q[lane + 32 * i]);
    o[i] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < r.len; ++j) {
    if (!((j <= pos && (p.f.window == 0 || j > pos - p.f.window)) || j < r.prefix)) continue;
    const int page = p.s.block_table[static_cast<size_t>(b) * p.s.max_pages + (j >> log2T)];
    if (page < 0 || page >= p.s.num_pages) {
      if (lane == 0) atomicExch(p.s.status, p.s.bad_index_code);
      continue;
    }
    const size_t krow =
        (static_cast<size_t>(page) * 2 * p.s.page_size + (j & (p.s.page_size - 1))) * p.s.Hkv + kvh;
    const uint32_t* k = reinterpret_cast<const uint32_t*>(p.cache) + krow * (D / 2);
    const uint32_t* v = k + static_cast<size_t>(p.s.page_size) * p.s.Hkv * (D / 2);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 kv = to_f32x2<BF16>(k[lane + 32 * i]);
      dot += qv[i].x * kv.x + qv[i].y * kv.y;
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    const float x = form_score(p.f, dot, slope, pos - j);
    const float mn = fmaxf(m, x);
    const float a = m == -INFINITY ? 0.f : expf(m - mn), e = expf(x - mn);
    l = l * a + e;
    m = mn;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 vv = to_f32x2<BF16>(v[lane + 32 * i]);
      o[i].x = o[i].x * a + e * vv.x;
      o[i].y = o[i].y * a + e * vv.y;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* out = static_cast<uint32_t*>(p.out) + w * (D / 2);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) out[lane + 32 * i] = pack2<BF16>(o[i].x * inv, o[i].y * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[w] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace eca
