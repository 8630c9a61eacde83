// tree_sched.cuh -- the division of tree attention's work over the blocks of a
// launch, computed on the device from the elements' lengths (so that one
// captured graph serves every length up to the cache's capacity).
//
// A group is one (element b, KV head g, block mb of its G * t_len[b] query
// rows); it has nt(b) = ceil(n[b] / tile rows) tiles of the cache.  The tiles of all groups, in order, are cut into `grid`
// equal runs, one for each CTA (with fewer tiles than CTAs, the CTAs past the
// last tile have none: a CTA inside a cut group always has a slot).  A run holds whole groups, whose outputs its
// CTA writes, and at most two cut ones: the end of a group begun by an earlier
// CTA (partial slot 2c) and the start of one that a later CTA goes on with
// (slot 2c + 1).  The combine launch merges a cut group's slots.
#pragma once
#include <stdint.h>

#include "serve_plan.h"

namespace lyc {

struct TreeElem {
  int n, cnt;  // rows, drafted tokens; cnt == 0: nothing to do
};

__device__ __forceinline__ TreeElem tree_elem(const TreeParams& p, int b, bool* bad) {
  TreeElem e;
  e.n = p.n[b];
  e.cnt = p.t_len ? p.t_len[b] : p.T;
  if (e.cnt < 0 || e.cnt > p.T || e.n < e.cnt || e.n > p.cache.cap) {
    *bad = true;
    e.n = e.cnt = 0;
  }
  return e;
}

// Called by whole warps; every lane gets the result.
template <int TR, int ROWS>
struct TreeSched {
  const TreeParams& p;
  int64_t total;
  int grid;  // CTAs that have tiles

  __device__ __forceinline__ int64_t elem_tiles(int b) const {
    if (b >= p.B) return 0;
    bool bad = false;
    const TreeElem e = tree_elem(p, b, &bad);
    return static_cast<int64_t>((e.n + TR - 1) / TR) * p.Hkv * blocks(e);
  }
  // blocks of query rows of a KV head
  __device__ __forceinline__ int blocks(const TreeElem& e) const { return (e.cnt * p.G + ROWS - 1) / ROWS; }
  __device__ __forceinline__ explicit TreeSched(const TreeParams& prm) : p(prm) {
    int64_t s = 0;
    const int lane = threadIdx.x & 31;
    for (int b0 = 0; b0 < p.B; b0 += 32) s += elem_tiles(b0 + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    total = s;
    grid = static_cast<int>(min(static_cast<int64_t>(p.grid), s));
  }
  __device__ __forceinline__ int64_t begin(int cta) const { return cta >= grid ? total : total * cta / grid; }
  // the CTA whose run holds tile x
  __device__ __forceinline__ int owner(int64_t x) const {
    int c = static_cast<int>(x * grid / total);
    while (c + 1 < grid && begin(c + 1) <= x) ++c;
    while (c > 0 && begin(c) > x) --c;
    return c;
  }
  // the element that tile x belongs to, and its first tile
  __device__ __forceinline__ void locate(int64_t x, int* b, int64_t* first) const {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    *b = 0;
    *first = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int64_t mine = elem_tiles(b0 + lane);
      int64_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x < base + inc);
      if (hit) {
        const int src = __ffs(hit) - 1;
        *b = b0 + src;
        *first = __shfl_sync(0xffffffffu, base + inc - mine, src);
        return;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  // the first tile of element b
  __device__ __forceinline__ int64_t first_tile(int b) const {
    const int lane = threadIdx.x & 31;
    int64_t s = 0;
    for (int b0 = 0; b0 < b; b0 += 32)
      if (b0 + lane < b) s += elem_tiles(b0 + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
};

// Does query t of element b see drafted node j (both below its count)?
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int j) {
  if (!p.mask) return j <= t;
  const unsigned long long w = p.mask[(static_cast<int64_t>(b) * p.T + t) * p.W + (j >> 6)];
  return (w >> (j & 63)) & 1ull;
}

}  // namespace lyc
