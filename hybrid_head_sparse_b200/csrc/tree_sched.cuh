// tree_sched.cuh -- the division of tree attention's work over the blocks of a
// launch, computed on the device from the elements' lengths (so that one
// captured graph serves every length up to the cache's capacity).
//
// A group is one (element b, KV head g, block mb of its G * t_len[b] query
// rows); it has nt(b) = ceil(n[b] / tile rows) tiles of the cache.  The tiles of
// all groups, in order, are cut into `grid` equal runs, one for each CTA (with
// fewer tiles than CTAs, the CTAs past the last tile have none: a CTA inside a cut
// group always has a slot).  A run holds whole groups, whose outputs its CTA
// writes, and at most two cut ones: the end of a group begun by an earlier CTA
// (partial slot 2c) and the start of one that a later CTA goes on with (slot 2c +
// 1).  The combine launch merges a cut group's slots.
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

// Tiles of 32 elements, a window of the batch: lane j keeps element b0 + j's
// lengths.  Called by whole warps; every lane gets the result.  The host refuses
// calls that could have 2^31 tiles, so 32 bits do.
template <int TR, int ROWS>
struct TreeLens {
  const TreeParams& p;
  TreeElem mine;         // of element b0 + lane
  uint32_t tiles, upto;  // its tiles; the tiles of all elements up to it
  int b0;
  uint32_t base;  // the tiles of the elements before the window

  // blocks of query rows of a KV head
  __device__ __forceinline__ int blocks(const TreeElem& e) const { return (e.cnt * p.G + ROWS - 1) / ROWS; }
  __device__ __forceinline__ TreeElem elem_of_lane(int first) const {
    const int b = first + static_cast<int>(threadIdx.x & 31);
    bool bad = false;
    return b < p.B ? tree_elem(p, b, &bad) : TreeElem{0, 0};
  }
  __device__ __forceinline__ uint32_t tiles_of(const TreeElem& e) const {
    return static_cast<uint32_t>((e.n + TR - 1) / TR) * static_cast<uint32_t>(p.Hkv * blocks(e));
  }
  __device__ __forceinline__ void window(int first, uint32_t before) {
    b0 = first;
    base = before;
    mine = elem_of_lane(first);
    tiles = tiles_of(mine);
    upto = tiles;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    upto += before;
  }
  __device__ __forceinline__ TreeLens(const TreeParams& prm, int first, uint32_t before) : p(prm) { window(first, before); }
  // element b of the window
  __device__ __forceinline__ TreeElem elem(int b) const {
    TreeElem e;
    e.n = __shfl_sync(0xffffffffu, mine.n, b - b0);
    e.cnt = __shfl_sync(0xffffffffu, mine.cnt, b - b0);
    return e;
  }
  // the element that tile x belongs to, and its first tile; x is not before the
  // window, which moves on to it
  __device__ __forceinline__ void locate(uint32_t x, int* b, uint32_t* first) {
    unsigned hit = __ballot_sync(0xffffffffu, x < upto);
    while (!hit && b0 + 32 < p.B) {
      window(b0 + 32, __shfl_sync(0xffffffffu, upto, 31));
      hit = __ballot_sync(0xffffffffu, x < upto);
    }
    const int src = hit ? __ffs(hit) - 1 : 0;
    *b = b0 + src;
    *first = __shfl_sync(0xffffffffu, upto - tiles, src);
  }
};

template <int TR, int ROWS>
struct TreeSched : TreeLens<TR, ROWS> {
  uint32_t total;
  uint32_t grid;         // CTAs that have tiles
  uint32_t share, more;  // the first `more` CTAs have share + 1 tiles, the others share
  uint32_t per, nt1;     // one element's groups: CTAs and tiles of each; per 0: as above

  __device__ __forceinline__ explicit TreeSched(const TreeParams& prm) : TreeLens<TR, ROWS>(prm, 0, 0u) {
    total = __shfl_sync(0xffffffffu, this->upto, 31);
    if (prm.B > 32) {
      uint32_t mine = 0u;
#pragma unroll 4
      for (int b = 32; b < prm.B; b += 32) mine += this->tiles_of(this->elem_of_lane(b));
      total += __reduce_add_sync(0xffffffffu, mine);
    }
    grid = min(static_cast<uint32_t>(prm.grid), max(total, 1u));
    per = 0;
    nt1 = 1;
    if (prm.B == 1) {
      // as many CTAs for each group, so that no run spans two groups, where that
      // leaves at most a sixteenth of them over.  In us against equal runs, one
      // token over 4 h / h heads of 128:
      //   few left over: h 8, 4097 rows bf16 10.0, 12.2; 65536 bf16 47.6, 48.4, e4m3 36.2, 39.0
      //   many: h 40, 65536 rows e4m3 151, 126; h 64 bf16 332, 320, e4m3 222, 192
      // and 160 nodes over 32768 rows, 64 / 8 heads (80 groups) bf16 350, 225, e4m3 485, 322
      const TreeElem e = this->elem(0);
      const uint32_t groups = static_cast<uint32_t>(prm.Hkv * this->blocks(e));
      nt1 = static_cast<uint32_t>((e.n + TR - 1) / TR);
      if (groups > 0 && grid >= groups) {
        const uint32_t each = min(grid / groups, nt1);
        if ((grid - groups * each) * 16u <= grid) {
          per = each;
          grid = groups * each;
        }
      }
    }
    share = total / grid;
    more = total - share * grid;
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
};

// A run's part of one group: tiles [t0, t1) of its nt.
struct TreePiece {
  int b, g, mb, t0, t1, nt;
  TreeElem e;
  int b0;  // the window that it was found in
  uint32_t base;
};

// The piece that holds tile x of a run that ends at xend.
template <int TR, int ROWS>
__device__ __forceinline__ TreePiece piece_at(TreeLens<TR, ROWS>& lens, uint32_t x, uint32_t xend) {
  TreePiece pc;
  uint32_t first;
  lens.locate(x, &pc.b, &first);
  pc.e = lens.elem(pc.b);
  pc.b0 = lens.b0;
  pc.base = lens.base;
  pc.nt = (pc.e.n + TR - 1) / TR;
  const uint32_t rel = x - first, nt = static_cast<uint32_t>(pc.nt);
  const int grp = static_cast<int>(rel / nt);
  const int mbs = lens.blocks(pc.e);
  pc.g = mbs == 1 ? grp : grp / mbs;
  pc.mb = grp - pc.g * mbs;
  pc.t0 = static_cast<int>(rel - static_cast<uint32_t>(grp) * nt);
  pc.t1 = static_cast<int>(min(nt, pc.t0 + (xend - x)));
  return pc;
}

// As calls, not inlined: each role of the tcgen05 kernel walks the run, and with
// the walk in each of them its loops lie far apart in the instruction caches.
template <int TR, int ROWS>
__device__ __noinline__ TreePiece tree_piece(const TreeParams& p, uint32_t x, uint32_t xend, int b0, uint32_t base) {
  TreeLens<TR, ROWS> lens(p, b0, base);
  return piece_at(lens, x, xend);
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
  int b0 = 0;
  uint32_t base = 0;
  __device__ __forceinline__ explicit TreeWalk(const TreeParams& prm) : p(prm) {
    const uint2 run = tree_run<TR, ROWS>(prm);
    x = run.x;
    xend = run.y;
  }
  __device__ __forceinline__ bool next(TreePiece* pc) {
    if (x >= xend) return false;
    *pc = tree_piece<TR, ROWS>(p, x, xend, b0, base);
    x += pc->t1 - pc->t0;
    b0 = pc->b0;
    base = pc->base;
    return true;
  }
};

// How often the tcgen05 kernel's 128 lanes hold the rows of a block.
__device__ __forceinline__ int tree_copies(int rows) { return rows <= 64 ? 2 : 1; }

// What a p' of a row with this scale byte of V is multiplied by for the sum:
// 2^-e kSumUnitE4m3 = 2^(111 - byte).
__device__ __forceinline__ float tree_sum_factor(uint32_t byte) {
  return __uint_as_float(byte < 238u ? (238u - byte) << 23 : 1u << (260u - byte));
}

// Does query t of element b see drafted node j (both below its count)?
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int j) {
  if (!p.mask) return j <= t;
  const unsigned long long w = p.mask[(static_cast<int64_t>(b) * p.T + t) * p.W + (j >> 6)];
  return (w >> (j & 63)) & 1ull;
}

}  // namespace lyc
