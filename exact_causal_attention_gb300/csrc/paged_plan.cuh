// Sharing out work whose sizes live on the device.  Every request has items (pairs of query
// tiles, pairs of key tiles) that cost something, each once per head.  Laid end to end
// (request, head, item, or request, item, head) they form a line; every CTA lays it out for itself and takes its
// equal part, so that nothing is counted or waited for across CTAs and the parts
// are the same whenever the sizes are.
#pragma once
#include "paged_common.cuh"

namespace eca {

constexpr int kPlanMaxRequests = 4096;

// Shared-memory tables of the line, free again once the CTA knows its part.
struct LineTables {
  int4* req;                 // [B]: n, pos0, prefix, len
  unsigned long long* cost;  // [B]: of one head
  long long* base;           // [B + 1]: where the request starts on the line
  int* first;                // [B + 1]: items of the requests before
  long long* warp_sums;      // [warps]
};
constexpr int kLineTableBytes = 16 * kPlanMaxRequests + 8 * kPlanMaxRequests + 8 * (kPlanMaxRequests + 2) +
                                4 * (kPlanMaxRequests + 4);

__device__ __forceinline__ LineTables line_tables(uint8_t* smem, long long* warp_sums) {
  LineTables t;
  t.req = reinterpret_cast<int4*>(smem);
  t.cost = reinterpret_cast<unsigned long long*>(smem + 16 * kPlanMaxRequests);
  t.base = reinterpret_cast<long long*>(smem + 24 * kPlanMaxRequests);
  t.first = reinterpret_cast<int*>(smem + 32 * kPlanMaxRequests + 16);
  t.warp_sums = warp_sums;
  return t;
}

// The last i in [0, n) with a[i] <= x, for a[0] <= x and a in order.
template <typename T, typename X>
__device__ __forceinline__ int last_at_most(const T* a, int n, X x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a[mid] <= x) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// Inclusive sum over the block in thread order.
template <int kThreads>
__device__ __forceinline__ long long line_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += up;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + v;
}

// Lays the line out; called by the whole block.  items(req) and cost(req, item) of a
// request's int4.  Returns the line's length.
template <int kThreads, typename Items, typename Cost>
__device__ __forceinline__ long long line_build(const LineTables& t, const ChunkShape& s, const ScoreForm& f, int heads,
                                                Items items, Cost cost) {
  const int B = s.B, tid = threadIdx.x;
  int count = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    int mine = 0;
    if (b < B) {
      const Request r = load_request(s, &f, b);
      t.req[b] = make_int4(r.n, r.pos0, r.prefix, r.len);
      t.cost[b] = 0;
      mine = items(t.req[b]);
    }
    long long all;
    const long long upto = line_scan<kThreads>(mine, t.warp_sums, &all);
    if (b < B) t.first[b] = count + static_cast<int>(upto) - mine;
    count += static_cast<int>(all);
  }
  if (tid == 0) t.first[B] = count;
  __syncthreads();
  for (int i = tid; i < count; i += kThreads) {
    const int b = last_at_most(t.first, B, i);
    atomicAdd(t.cost + b, static_cast<unsigned long long>(cost(t.req[b], i - t.first[b])));
  }
  __syncthreads();
  long long length = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    const long long mine = b < B ? static_cast<long long>(t.cost[b]) * heads : 0;
    long long all;
    const long long upto = line_scan<kThreads>(mine, t.warp_sums, &all);
    if (b < B) t.base[b] = length + upto - mine;
    length += all;
  }
  if (tid == 0) t.base[B] = length;
  __syncthreads();
  return length;
}

// The same by one warp, without the block's barriers, for at most 32 requests and few
// enough items that 32 lanes get through them as fast (line_is_small).
template <typename Items, typename Cost>
__device__ __forceinline__ long long line_build_warp(const LineTables& t, const ChunkShape& s, const ScoreForm& f,
                                                     int heads, Items items, Cost cost) {
  const int B = s.B, b = threadIdx.x % 32;
  int4 req = make_int4(0, 0, 0, 0);
  int mine = 0;
  if (b < B) {
    const Request r = load_request(s, &f, b);
    req = make_int4(r.n, r.pos0, r.prefix, r.len);
    mine = items(req);
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, upto, d);
    if (b >= d) upto += up;
  }
  long long sum = 0;
  const int longest = __reduce_max_sync(0xffffffffu, mine);
  if (longest <= 8) {  // every lane its own request's
    for (int i = 0; i < longest; ++i) sum += i < mine ? cost(req, i) : 0;
  }
  for (int r = 0; longest > 8 && r < B; ++r) {
    const int4 q = make_int4(__shfl_sync(0xffffffffu, req.x, r), __shfl_sync(0xffffffffu, req.y, r),
                             __shfl_sync(0xffffffffu, req.z, r), __shfl_sync(0xffffffffu, req.w, r));
    const int n = __shfl_sync(0xffffffffu, mine, r);
    for (int i0 = 0; i0 < n; i0 += 32) {
      // A cost is below 2^25 (key tiles of a context below 2^31 tokens), so 32 of them fit.
      const int c = __reduce_add_sync(0xffffffffu, i0 + b < n ? cost(q, i0 + b) : 0);
      if (b == r) sum += c;
    }
  }
  long long end = sum * heads;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, end, d);
    if (b >= d) end += up;
  }
  if (b < B) {
    t.req[b] = req;
    t.cost[b] = static_cast<unsigned long long>(sum);
    t.base[b] = end - sum * heads;
    t.first[b] = upto - mine;
    if (b == B - 1) {
      t.base[B] = end;
      t.first[B] = upto;
    }
  }
  __syncwarp();
  return __shfl_sync(0xffffffffu, end, B - 1);
}

// Is a line of B requests and at most `total` items short enough for line_build_warp?
__host__ inline bool line_is_small(int B, double total) { return B <= 32 && total / 32 + B <= 64; }

// Where the c-th of G equal parts of a line of length W starts.
__device__ __forceinline__ long long line_cut(long long W, int G, int c) {
  if (W < (1ll << 32)) {  // 32-bit divisions take a fraction of the time
    const uint32_t w = static_cast<uint32_t>(W), g = static_cast<uint32_t>(G);
    return static_cast<long long>(w / g) * c + (w % g) * static_cast<uint32_t>(c) / g;
  }
  return W / G * c + W % G * c / G;
}

// The item that holds place x of the line.
struct LinePlace {
  int b, head, item;
  int in;           // x, from the item's start
  int cost;         // the item's
  long long start;  // of the item, on the line
};

// Called by a whole warp; x below the line's length.  kHeadsInside: a request's items
// in order, each with all its heads; else its heads in order, each with all items.
// Int: a type that holds the line's length (64-bit arithmetic takes several times longer).
template <bool kHeadsInside, typename Int, typename Cost>
__device__ __forceinline__ LinePlace line_locate_as(const LineTables& t, int B, int heads, Int x, Cost cost) {
  const int lane = threadIdx.x % 32;
  LinePlace r;
  // Requests without items share their base with the next: the last such one has items.
  if (B <= 32) {
    r.b = __popc(__ballot_sync(0xffffffffu, lane < B && static_cast<Int>(t.base[min(lane, B - 1)]) <= x)) - 1;
  } else {
    r.b = last_at_most(t.base, B, static_cast<long long>(x));
  }
  const Int sum = static_cast<Int>(t.cost[r.b]);
  Int rest = x - static_cast<Int>(t.base[r.b]);
  Int start = static_cast<Int>(t.base[r.b]);
  r.head = 0;
  if constexpr (!kHeadsInside) {
    r.head = static_cast<int>(rest / sum);
    start += static_cast<Int>(r.head) * sum;
    rest -= static_cast<Int>(r.head) * sum;
  }
  const int4 q = t.req[r.b];
  const int n = t.first[r.b + 1] - t.first[r.b];
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int one = i < n ? cost(q, i) : 0;
    const Int mine = kHeadsInside ? static_cast<Int>(one) * heads : one;
    Int c = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const Int up = __shfl_up_sync(0xffffffffu, c, d);
      if (lane >= d) c += up;
    }
    const unsigned here = __ballot_sync(0xffffffffu, i < n && rest < c);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      const Int before = __shfl_sync(0xffffffffu, c - mine, src);
      r.item = i0 + src;
      r.cost = __shfl_sync(0xffffffffu, one, src);
      Int at = rest - before;
      start += before;
      if constexpr (kHeadsInside) {
        r.head = static_cast<int>(at / r.cost);
        at -= static_cast<Int>(r.head) * r.cost;
        start += static_cast<Int>(r.head) * r.cost;
      }
      r.in = static_cast<int>(at);
      r.start = static_cast<long long>(start);
      return r;
    }
    const Int all = __shfl_sync(0xffffffffu, c, 31);
    rest -= all;
    start += all;
  }
  r.item = n;  // not reached: a request's items cover its stretch
  r.cost = r.in = 0;
  r.start = static_cast<long long>(start);
  return r;
}

template <bool kHeadsInside, typename Cost>
__device__ __forceinline__ LinePlace line_locate(const LineTables& t, int B, int heads, long long length, long long x,
                                                 Cost cost) {
  if (length < (1ll << 31)) {
    return line_locate_as<kHeadsInside, uint32_t>(t, B, heads, static_cast<uint32_t>(x), cost);
  }
  return line_locate_as<kHeadsInside, unsigned long long>(t, B, heads, static_cast<unsigned long long>(x), cost);
}

}  // namespace eca
