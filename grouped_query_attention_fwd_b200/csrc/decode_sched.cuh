// How decode work is cut into CTA ranges, shared by the decode kernels over
// 16-bit and over 4-bit caches: all units (128-key tiles) of a launch lie end
// to end, one contiguous range per CTA.
#pragma once

#include <stdint.h>

#include "kernels.h"

namespace gqa {

__host__ __device__ inline int range_start(int c, int T, int P) {
  // floor(c T / P) = c q + floor(c r / P) with T = q P + r: 32-bit operations
  // only (c <= P, so c r < P^2), on every CTA's path to its first copy.
  const int q = T / P, r = T - q * P;
  return c * q + (c * r) / P;
}

// The CTA whose range [range_start(c), range_start(c + 1)) holds unit u:
// the largest c with floor(c T / P) <= u, i.e. ceil((u + 1) P / T) - 1.
__host__ __device__ inline int cta_of_unit(int u, int T, int P) {
  return static_cast<int>(((static_cast<int64_t>(u) + 1) * P + T - 1) / T) - 1;
}

// Unit layout of one launch.  Units run over batch entries, then kv heads,
// then head passes, then key tiles; every group (one kv head and pass of one
// batch entry) of entry b has the same number of tiles, so the units of b
// start at pre[b] (ragged) or b * per_b.
struct Sched {
  const int* pre;  // ragged: B + 1 prefix sums (shared memory), else nullptr
  const int* len;  // ragged: cache length per entry (shared memory), else nullptr
  int per_b;       // uniform: units per batch entry
  int gpb;         // groups per batch entry = Hkv * passes
  int B;
  int total;       // units of the launch (< 2^31, checked by the planner)
  int P;           // CTAs that get units: min(grid, total)

  __device__ int batch_of(int u) const {
    if (pre == nullptr) return u / per_b;
    int lo = 0, hi = B - 1;  // largest b with pre[b] <= u (pre is strictly increasing)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
  __device__ int start_of(int b) const { return pre ? pre[b] : b * per_b; }
};

// Batch entry of the unit last looked up, with its key range.
struct Cursor {
  int b = -1;
  int beg = 0, end = 0;  // units [beg, end) belong to entry b
  KeyRange kr{};
};

__device__ __forceinline__ void seek(Cursor& c, int u, const Sched& sc, const DecodeArgs& a) {
  if (c.b >= 0 && u >= c.beg && u < c.end) return;
  c.b = sc.batch_of(u);
  c.beg = sc.start_of(c.b);
  c.kr = decode_key_range(sc.len ? sc.len[c.b] : a.Sk, a.Sk, a.Sq, a.causal, a.causal_offset,
                          a.window);
  c.end = c.beg + sc.gpb * c.kr.tiles;
}

// Group of unit u (its index over the whole launch).
__device__ __forceinline__ int group_of(int u, const Sched& sc, const DecodeArgs& a) {
  Cursor c;
  seek(c, u, sc, a);
  return c.b * sc.gpb + (u - c.beg) / c.kr.tiles;
}

}  // namespace gqa
