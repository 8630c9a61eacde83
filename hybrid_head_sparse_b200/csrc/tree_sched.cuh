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

// Called by whole warps; every lane gets the result.  Lane j keeps element
// j's lengths (of the first 32; a larger batch is read again, 32 at a time).
// The host refuses calls that could have 2^31 tiles, so 32 bits do.
template <int TR, int ROWS>
struct TreeSched {
  const TreeParams& p;
  TreeElem mine;         // of element `lane`
  uint32_t tiles, upto;  // its tiles; the tiles of elements 0 .. lane
  uint32_t total;
  uint32_t grid;         // CTAs that have tiles
  uint32_t share, more;  // the first `more` CTAs have share + 1 tiles, the others share
  uint32_t per, nt1;     // groups of one length (one element): CTAs and tiles of each; per 0: as above

  // blocks of query rows of a KV head
  __device__ __forceinline__ int blocks(const TreeElem& e) const { return (e.cnt * p.G + ROWS - 1) / ROWS; }
  __device__ __forceinline__ TreeElem elem_of_lane(int b0) const {
    const int b = b0 + static_cast<int>(threadIdx.x & 31);
    bool bad = false;
    return b < p.B ? tree_elem(p, b, &bad) : TreeElem{0, 0};
  }
  __device__ __forceinline__ uint32_t tiles_of(const TreeElem& e) const {
    return static_cast<uint32_t>((e.n + TR - 1) / TR) * static_cast<uint32_t>(p.Hkv * blocks(e));
  }
  static __device__ __forceinline__ uint32_t scan(uint32_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
  __device__ __forceinline__ explicit TreeSched(const TreeParams& prm) : p(prm) {
    mine = elem_of_lane(0);
    tiles = tiles_of(mine);
    upto = scan(tiles);
    total = __shfl_sync(0xffffffffu, upto, 31);
    for (int b0 = 32; b0 < p.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, tiles_of(elem_of_lane(b0)));
    grid = min(static_cast<uint32_t>(p.grid), max(total, 1u));
    per = 0;
    if (p.B == 1) {
      // as many CTAs for each group, so that no run spans two groups (a second
      // start and merge in one CTA costs more than the few CTAs left over: one
      // token at 4097 rows, 144 CTAs against 148)
      const TreeElem e = elem(0);
      const uint32_t groups = static_cast<uint32_t>(p.Hkv * blocks(e));
      nt1 = static_cast<uint32_t>((e.n + TR - 1) / TR);
      if (groups > 0 && grid >= groups) {
        per = min(grid / groups, nt1);
        grid = groups * per;
      }
    }
    share = total / grid;
    more = total - share * grid;
  }
  __device__ __forceinline__ TreeElem elem(int b) const {
    TreeElem e;
    if (b < 32) {
      e.n = __shfl_sync(0xffffffffu, mine.n, b);
      e.cnt = __shfl_sync(0xffffffffu, mine.cnt, b);
    } else {
      bool bad = false;
      e = tree_elem(p, b, &bad);
    }
    return e;
  }
  // (a group has at most 2^23 tiles of 128 rows, and `per` is at most the SMs)
  __device__ __forceinline__ uint32_t begin(uint32_t cta) const {
    if (cta >= grid) return total;
    if (per == 0) return cta * share + min(cta, more);
    const uint32_t g = cta / per;
    return g * nt1 + nt1 * (cta - g * per) / per;
  }
  // the CTA whose run holds tile x
  __device__ __forceinline__ uint32_t owner(uint32_t x) const {
    if (per == 0) {
      const uint32_t big = more * (share + 1);
      return x < big ? x / (share + 1) : more + (x - big) / share;
    }
    const uint32_t g = x / nt1, r = x - g * nt1;
    uint32_t j = r * per / nt1;  // run j starts at nt1 j / per, rounded down
    if (j + 1 < per && nt1 * (j + 1) / per <= r) ++j;
    return g * per + j;
  }
  // the element that tile x belongs to, and its first tile
  __device__ __forceinline__ void locate(uint32_t x, int* b, uint32_t* first) const {
    unsigned hit = __ballot_sync(0xffffffffu, x < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      *b = src;
      *first = __shfl_sync(0xffffffffu, upto - tiles, src);
      return;
    }
    uint32_t base = __shfl_sync(0xffffffffu, upto, 31);
    *b = 0;
    *first = 0;
    for (int b0 = 32; b0 < p.B; b0 += 32) {
      const uint32_t tl = tiles_of(elem_of_lane(b0)), up = scan(tl);
      hit = __ballot_sync(0xffffffffu, x < base + up);
      if (hit) {
        const int src = __ffs(hit) - 1;
        *b = b0 + src;
        *first = __shfl_sync(0xffffffffu, base + up - tl, src);
        return;
      }
      base += __shfl_sync(0xffffffffu, up, 31);
    }
  }
  // the first tile of element b
  __device__ __forceinline__ uint32_t first_tile(int b) const {
    if (b < 32) return __shfl_sync(0xffffffffu, upto - tiles, b);
    uint32_t base = __shfl_sync(0xffffffffu, upto, 31);
    for (int b0 = 32; b0 < b; b0 += 32) {
      const uint32_t tl = tiles_of(elem_of_lane(b0));
      base += __reduce_add_sync(0xffffffffu, b0 + static_cast<int>(threadIdx.x & 31) < b ? tl : 0u);
    }
    return base;
  }
};

// A run's part of one group: tiles [t0, t1) of its nt.
struct TreePiece {
  int b, g, mb, t0, t1, nt;
  TreeElem e;
};

// The piece that holds tile x of a run that ends at xend.
template <int TR, int ROWS>
__device__ __forceinline__ TreePiece piece_at(const TreeSched<TR, ROWS>& sched, uint32_t x, uint32_t xend) {
  TreePiece pc;
  uint32_t first;
  sched.locate(x, &pc.b, &first);
  pc.e = sched.elem(pc.b);
  pc.nt = (pc.e.n + TR - 1) / TR;
  const uint32_t rel = x - first, nt = static_cast<uint32_t>(pc.nt);
  const int grp = static_cast<int>(rel / nt);
  const int mbs = sched.blocks(pc.e);
  pc.g = mbs == 1 ? grp : grp / mbs;
  pc.mb = grp - pc.g * mbs;
  pc.t0 = static_cast<int>(rel - static_cast<uint32_t>(grp) * nt);
  pc.t1 = static_cast<int>(min(nt, pc.t0 + (xend - x)));
  return pc;
}

// As calls, not inlined: each role of the tcgen05 kernel walks the run, and with
// the walk in each of them its loops lie far apart in the instruction caches.
template <int TR, int ROWS>
__device__ __noinline__ TreePiece tree_piece(const TreeParams& p, uint32_t x) {
  const TreeSched<TR, ROWS> sched(p);
  return piece_at(sched, x, sched.begin(blockIdx.x + 1));
}
template <int TR, int ROWS>
__device__ __noinline__ uint2 tree_run(const TreeParams& p) {
  const TreeSched<TR, ROWS> sched(p);
  return make_uint2(sched.begin(blockIdx.x), sched.begin(blockIdx.x + 1));
}

// The pieces of this CTA's run in order.
template <int TR, int ROWS>
struct TreeWalk {
  const TreeParams& p;
  uint32_t x, xend;
  __device__ __forceinline__ explicit TreeWalk(const TreeParams& prm) : p(prm) {
    const uint2 run = tree_run<TR, ROWS>(prm);
    x = run.x;
    xend = run.y;
  }
  // tiles of the run; before the first next()
  __device__ __forceinline__ uint32_t run_tiles() const { return xend - x; }
  __device__ __forceinline__ bool next(TreePiece* pc) {
    if (x >= xend) return false;
    *pc = tree_piece<TR, ROWS>(p, x);
    x += pc->t1 - pc->t0;
    return true;
  }
};

// How often the tcgen05 kernel's 128 lanes hold the rows of a block.
__device__ __forceinline__ int tree_copies(int rows) { return rows <= 64 ? 2 : 1; }

// Does query t of element b see drafted node j (both below its count)?
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int j) {
  if (!p.mask) return j <= t;
  const unsigned long long w = p.mask[(static_cast<int64_t>(b) * p.T + t) * p.W + (j >> 6)];
  return (w >> (j & 63)) & 1ull;
}

}  // namespace lyc
