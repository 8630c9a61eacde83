// tree_tc_kernel.cu -- attention of many query rows over the cache
// (lyc_tree_attention), head_dim 128, on the 5th-generation tensor cores.
//
// The same sums as tree_mma_kernel.cu for blocks of up to 128 of a KV head's
// G * T query rows (row i = node i / G, head g * G + i % G), the M side of the
// MMAs, over tiles of 128 cached rows:
//   S[128 q x 128 keys] = Q K^T, O[128 q x 128 d] += P V, both in tensor memory.
//
// Warps 0-7 are the softmax warps: warp w owns query rows 32 (w % 4) .. + 31
// (their tensor-memory lanes) and key half w / 4 of every tile, with a running
// maximum, sum and O accumulator of its own; the two halves are merged at the
// end of a run.  P overwrites S in tensor memory (16-bit, half the columns)
// and is the A operand from there, so it costs no shared memory and no shared
// memory bandwidth, and the ring of K/V tiles is as deep as the SM allows.
// Warp 8 issues the MMAs (one thread), for bf16 rows warp 9 the TMA copies; two
// S buffers let the QK of tile t+1 run beside the softmax of tile t.  A warp none of
// whose rows is a query does nothing but keep the barriers going.
//
// A block of 64 query rows or fewer has them twice over in the 128 lanes, and each
// copy takes half of a key half (its P is zero elsewhere), so the exponentials are
// spread over all the schedulers instead of staying with the warps of the first
// rows.  The copies are parts like those of other CTAs, merged with them, or in the
// CTA for a whole group, which has them only where it is long.
//
// bf16 rows: K and V tiles are read by the tensor core where TMA puts them.
// Masked rows have P = 0, and 0 * NaN would reach every row, so in the tiles
// that hold drafted rows or end an element the softmax warps clear rows past
// the end, and take a drafted row's NaNs and infinities out of V; the nodes
// that see such a row get them added at the end.
//
// e4m3 rows become f16 tiles on their way: code * 2^(e - E), E the largest e of the
// tile's rows, so the products run in f16.  2^E of K is a factor of the tile's
// logits; V's goes into the exponent, p' = 2^(z + E - m'), m' the running maximum of
// z + E, and the sum takes p' 2^-E (kSumUnitE4m3).  That is exact while the tile's e
// are within 14 of each other, and V's are held within 6, so that p' of a row far
// below E does not fall out of f16's range (at 14, a tail of 65536 rows 2^-18 below
// the top one was lost beside a row of negligible probability 2^14 larger).  Where
// they are not (a row of zeros; a drafted row that nobody has written or sees), the
// tile is the codes alone and the softmax warps apply each row's scales.  A query row
// becomes f16 as in tree_mma_kernel.cu.  Three warps find the rows of coming tiles
// and their scales; eight producer warps copy the codes in, convert them (two
// instructions for two codes) and store them.
//
// Device times, 32 query and 8 KV heads.  32 nodes over 131072 bf16 rows: 96 to
// 101 us by the box, 5.3 to 5.6 TB/s, 0.81 to 0.85 of the copy rate: HBM, and the
// exponentials (1024 cycles a tile at 16 a cycle).  4 x 16 nodes over up to 65536
// e4m3 rows each: 165 us, 0.37 of the floor; 2 x 64 nodes over up to 32768 rows: 114 to 135.
// There a tile's share is 2.0 us, its bytes' 0.75; counted, it needs 1000 cycles of
// the tensor cores and 1800 of shared memory (128 bytes a cycle), each of them less
// than half of that, and the issue slots are half busy: what bounds it is the softmax
// warps' chain of latencies among twenty warps.  Slower were: bf16 tiles, codes
// converted by bit moves (175); each row's own scale in the softmax, K's codes as an
// e4m3 operand (212); codes brought by TMA (205); four or sixteen producers (190,
// 203); a fourth finder (200: the schedulers' warps are no longer the same); one pass
// over the logits (185).  Leaving out the check of the scales' spread gained 4.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "lyc_device.cuh"
#include "serve_plan.h"
#include "tc_ptx.cuh"
#include "tree_sched.cuh"

namespace lyc {

namespace {

constexpr int kRows = 128;  // query rows of a block, cached rows of a tile
constexpr int kD = 128;
constexpr int kSoft = 256;  // softmax threads
constexpr int kOkRing = 16;
constexpr int kRawRing = 3;    // e4m3: groups of units on their way to a producer warp
constexpr int kInfoRing = 8;   // e4m3: tiles whose rows are known
constexpr int kProducers = 8;  // warps, half of them for K, half for V
constexpr int kFinders = 3;    // warps that find rows, every third tile each
constexpr int kUnits = 4;      // 4-row units that a producer warp converts at a time
constexpr int kSide = kProducers / 2;
constexpr int kGroups = 32 / (kSide * kUnits);  // of a warp's units of a tile

// How far z may grow (log2 units) before the running maximum moves, and where a
// probability at the maximum lies.  f16 (e4m3 rows) is used from the top, 2^15.9 of
// 65504; it ends at 2^-24, so a probability is off by at most 2^-36 of the tile's
// largest times its largest scale of V.  Rows of up to kApartV octaves share a tile's
// scale: that is 2^-30 of the largest probability * scale of a row.  Beyond that they
// keep their own.  (4 x 16 nodes over up to 65536 rows: 164.8 us, as with a range of 8 and
// an apartness of 14; a range of 4 took 168.5, an apartness of 5, which ordinary rows
// of V reach, 4 us more over 512 rows.  Where every tile's rows are further apart, 355.)
template <bool F8>
struct TcRange {
  static constexpr float kLag = F8 ? 4.9f : 8.f;
  static constexpr float kTop = F8 ? 11.f : 0.f;
};
constexpr uint32_t kApartK = 14;  // every factor of a row is a normal f16, and codes (multiples of 2^-9) times it exact
constexpr uint32_t kApartV = 6;

template <bool F8_>
struct TcCfg {
  static constexpr bool F8 = F8_;
  static constexpr int SK = F8 ? 2 : 3;              // K tiles
  static constexpr int SV = F8 ? 2 : 3;              // V tiles
  static constexpr int TILEB = 32768;                // a K or V tile of bf16
  static constexpr int THREADS = 9 * 32 + (F8 ? (kFinders + kProducers) * 32 : 32);
  static constexpr int MMA_WARP = 8, LOAD_WARP = 9;  // F8: finders from LOAD_WARP on
  static constexpr int PROD_WARP = LOAD_WARP + kFinders;
  static constexpr int FULL = F8 ? kProducers / 2 : 1;  // arrivals that fill a tile
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 32768;
  static constexpr int OFF_V = OFF_K + SK * TILEB;
  static constexpr int OFF_RAW = OFF_V + SV * TILEB;  // F8: codes, [producer][kRawRing][unit][lane] of 16 bytes
  static constexpr int OFF_INFO = OFF_RAW + (F8 ? kRawRing * kProducers * kUnits * 512 : 0);  // F8: [kInfoRing][128] rows
  static constexpr int OFF_BAR = OFF_INFO + (F8 ? kInfoRing * kRows * 16 : 0);
  // kfull, kempty [SK]; vfull, vempty [SV]; s_ready, p_ready, pv_done [2];
  // q_ready, o_free, ml_ready, idle; F8: info_full, info_empty [kInfoRing]
  static constexpr int NBAR = 2 * SK + 2 * SV + 6 + 4 + (F8 ? 2 * kInfoRing : 0);
  // abort, tmem, odd rows [2][8], ok [kOkRing][4], F8: scale bytes [kOkRing][2]
  static constexpr int OFF_FLAGS = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_FLAGS + 8 + 64 + 16 * kOkRing + (F8 ? 8 * kOkRing : 0) + 1024;  // + alignment
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

template <class C>
struct TcBars {
  uint64_t *kfull, *kempty, *vfull, *vempty, *s_ready, *p_ready, *pv_done, *q_ready, *o_free, *ml_ready, *idle,
      *info_full, *info_empty;
  __device__ explicit TcBars(unsigned char* smem) {
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    kfull = b;
    kempty = kfull + C::SK;
    vfull = kempty + C::SK;
    vempty = vfull + C::SV;
    s_ready = vempty + C::SV;
    p_ready = s_ready + 2;
    pv_done = p_ready + 2;
    q_ready = pv_done + 2;
    o_free = q_ready + 1;
    ml_ready = o_free + 1;
    idle = ml_ready + 1;
    info_full = idle + 1;
    info_empty = info_full + kInfoRing;
  }
};

constexpr uint32_t kOwn = 0x100u;

struct TcShared {
  int* abort;
  uint32_t* tmem;
  uint32_t* odd;  // [2] by piece: drafted rows with a NaN or an infinity in V, by node
  uint32_t* ok;   // ring of the tiles' rows that were found (paged), 4 words each
  uint32_t* top;  // F8: ring of the tiles' largest scale bytes of K (kOwn: rows have their own) and of V
};
template <class C>
__device__ __forceinline__ TcShared shared_of(unsigned char* smem) {
  TcShared s;
  s.abort = reinterpret_cast<int*>(smem + C::OFF_FLAGS);
  s.tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAGS + 4);
  s.odd = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAGS + 8);
  s.ok = s.odd + 16;
  s.top = s.ok + 4 * kOkRing;
  return s;
}

// Wait for a phase of `bar`; false once the CTA has given up (a wait above
// kWaitLimitNs).  heed: also give up where another warp has.
__device__ __noinline__ bool tc_wait_on(uint32_t bar, uint32_t parity, int* abort_flag, uint32_t* status, bool heed) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 1023u) == 0) {
      if (heed && *reinterpret_cast<volatile int*>(abort_flag)) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        *reinterpret_cast<volatile int*>(abort_flag) = 1;
        if (status) atomicOr(status, LYC_OP_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t* status,
                                        bool heed = true) {
  if (mbar_try_wait(bar, parity)) return true;
  return tc_wait_on(smem_u32(bar), parity, abort_flag, status, heed);
}

// One arrival for a warp, after all its lanes' earlier accesses.  (Arrivals of 32
// lanes on one barrier are taken one after another.)
__device__ __forceinline__ void tc_arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t* status) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag, status));
}

// byte offset of 16-byte piece ch of row r of a 256-byte-row tile: two halves
// of 128-byte rows with the 128-byte swizzle
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  return static_cast<uint32_t>((ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                       uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ float tc_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t tc_pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tc_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// The loads of N registers are done: naming them here keeps the compiler from
// using one before the wait.
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t (*r)[16]) {
#pragma unroll
  for (int c = 0; c < N; ++c)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[c][0]), "+r"(r[c][1]), "+r"(r[c][2]), "+r"(r[c][3]), "+r"(r[c][4]), "+r"(r[c][5]),
                   "+r"(r[c][6]), "+r"(r[c][7]), "+r"(r[c][8]), "+r"(r[c][9]), "+r"(r[c][10]), "+r"(r[c][11]),
                   "+r"(r[c][12]), "+r"(r[c][13]), "+r"(r[c][14]), "+r"(r[c][15])::"memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations an instruction (sm_100's packed forms).
typedef unsigned long long f2_t;
__device__ __forceinline__ f2_t f2(float a, float b) {
  f2_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(f2_t r, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(r));
}
__device__ __forceinline__ f2_t f2_fma(f2_t a, f2_t b, f2_t c) {
  f2_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2_t f2_add(f2_t a, f2_t b) {
  f2_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Both operands bf16, or both f16 (format 0).
__device__ __forceinline__ constexpr uint32_t tc_idesc(bool f16, int b_mn_major) {
  return tc::idesc_bf16(128, 128, 0, b_mn_major) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}
// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

typedef TreeWalk<kRows, kRows> TcWalk;

// ---------------------------------------------------------------- loads (bf16)
// The whole warp: lane j looks up and copies box j of a tile (one box of 128
// rows where the cache is contiguous, else box_rows rows of a page).
template <class C>
__device__ __forceinline__ void tc_loads(const TreeTcParams& P, unsigned char* smem) {
  const TreeParams& p = P.t;
  const int lane = threadIdx.x & 31;
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  // a cache that several blocks of query rows read stays in L2
  const uint64_t pol = p.G * p.T > kRows ? l2_policy_evict_normal() : l2_policy_evict_first();
  const bool paged = p.cache.bt != nullptr;
  const int nbox = kRows / p.box_rows;
  const uint32_t boxb = static_cast<uint32_t>(C::TILEB) / nbox;  // bytes of a box
  TcWalk walk(p);
  TreePiece pc;
  int t = 0;
  int asked[2] = {0, 0};  // tiles of K and of V whose copies went out
  bool ok = true;
  while (ok && walk.next(&pc)) {
    for (int tile = pc.t0; ok && tile < pc.t1; ++tile, ++t) {
      const int row0 = tile * kRows + lane * p.box_rows;
      bool have = lane < nbox && row0 < pc.e.n;
      int c1 = row0, c2 = pc.g, c3 = pc.b;
      if (paged && have) {
        const int blk = page_of(p.cache, row0);
        const int32_t page = p.cache.bt[static_cast<int64_t>(pc.b) * p.cache.max_blocks + blk];
        have = page >= 0 && page < p.cache.num_pages;
        if (!have && p.status) atomicOr(p.status, LYC_OP_BAD_PAGE);
        c1 = pc.g;
        c2 = row0 - blk * p.cache.page_rows;
        c3 = page;
      }
      const uint32_t found = __ballot_sync(0xffffffffu, have);
      const uint32_t bytes = static_cast<uint32_t>(__popc(found)) * boxb;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int S = kv ? C::SV : C::SK;
        const int stage = t % S;
        uint64_t* full = (kv ? br.vfull : br.kfull) + stage;
        uint64_t* empty = (kv ? br.vempty : br.kempty) + stage;
        if (t >= S && !tc_wait_warp(empty, ((t / S) - 1) & 1, sh.abort, p.status)) {
          ok = false;
          break;
        }
        if (kv == 0 && paged && lane < 4) {
          uint32_t rows = 0;  // rows 32 lane .. + 31 by their boxes (of 8 rows or more)
          for (int x = 0; x < 32; x += 8)
            if ((found >> ((lane * 32 + x) / p.box_rows)) & 1u) rows |= 0xffu << x;
          sh.ok[(t % kOkRing) * 4 + lane] = rows;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (have) {
          unsigned char* dst = smem + (kv ? C::OFF_V : C::OFF_K) + stage * C::TILEB + lane * p.box_rows * 128;
          const CUtensorMap* map = kv ? &P.tmv : &P.tmk;
          tma_4d(dst, map, 0, c1, c2, c3, full, pol);
          tma_4d(dst + 16384, map, 64, c1, c2, c3, full, pol);
        }
        asked[kv] = t + 1;
        __syncwarp();
      }
      if (!ok) break;
    }
  }
  if (!ok) {
    // given up: wait for the copies in flight before the CTA's memory goes
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const int S = kv ? C::SV : C::SK;
      for (int x = max(0, asked[kv] - S); x < asked[kv]; ++x)
        tc_wait((kv ? br.vfull : br.kfull) + x % S, (x / S) & 1, sh.abort, p.status, false);
    }
  }
}

// ---------------------------------------------------------------- producers (e4m3)
// Four e4m3 codes as f16, exactly: codes 0 and 1, codes 2 and 3.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t* h01, uint32_t* h23) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*h01), "=r"(*h23)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// What is known of a row of a tile.
struct RowInfo {
  long long off;    // of its codes in K and in V; odd: no such row, zeros
  uint32_t factor;  // its scales over the tile's largest, as f16, K's and V's << 16
  uint32_t own;     // its scale bytes, V's << 8
};

// A finder warp finds the rows of every third tile of the run, lane j rows j + 32 k:
// pages are asked for a turn ahead, and a tile's scales arrive while the next
// one's rows are found.  A turn is a chain of dependent loads that is longer than a
// tile, so one warp was what a tile took.  (In the producers, a row a lane, it held
// them up: their waits for shared memory are also waits for the loads that share a
// counter.)
template <class C>
__device__ __forceinline__ void tc_rows(const TreeTcParams& P, unsigned char* smem) {
  const TreeParams& p = P.t;
  const int lane = threadIdx.x & 31;
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  RowInfo* info = reinterpret_cast<RowInfo*>(smem + C::OFF_INFO) + lane;
  const bool paged = p.cache.bt != nullptr;
  const int first = (threadIdx.x >> 5) - C::LOAD_WARP;
  TcWalk walk(p);
  TreePiece pc;
  bool more = walk.next(&pc);
  int tile = more ? pc.t0 : 0;
  auto skip = [&](int n) {  // n tiles on
    tile += n;
    while (more && tile >= pc.t1) {
      const int over = tile - pc.t1;
      more = walk.next(&pc);
      tile = pc.t0 + over;
    }
  };
  skip(first);
  int32_t page[4] = {0, 0, 0, 0};
  uint32_t kb[4], vb[4];
  long long off[4];
  auto ask = [&]() {  // pages of tile `tile`
    if (!paged || !more) return;
    const int64_t row_of = static_cast<int64_t>(pc.b) * p.cache.max_blocks;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = tile * kRows + lane + 32 * k;
      page[k] = p.cache.bt[row_of + page_of(p.cache, min(row, pc.e.n - 1))];
    }
  };
  auto put = [&](int t) {
    // the tile's largest scales, as byte + 1, so that NaN rows' and those of rows that
    // are not there count as 0
    uint32_t kk[4], vv[4], kt = 0u, vt = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t have = (off[k] & 1) ? 0u : 255u;
      vb[k] = max(vb[k], kMinScaleV);  // (here, not at the load: that would wait for it)
      kk[k] = (kb[k] + 1u) & have;
      vv[k] = (vb[k] + 1u) & have;
      kt = max(kt, kk[k]);
      vt = max(vt, vv[k]);
    }
    kt = __reduce_max_sync(0xffffffffu, kt);
    vt = __reduce_max_sync(0xffffffffu, vt);
    bool apart = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) apart |= (kk[k] && kk[k] + kApartK < kt) || (vv[k] && vv[k] + kApartV < vt);
    const bool own = __any_sync(0xffffffffu, apart);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t kf = own || kk[k] == 0u ? 15u << 10 : (15u + kk[k] - kt) << 10;
      uint32_t vf = own || vv[k] == 0u ? 15u << 10 : (15u + vv[k] - vt) << 10;
      if (kb[k] == 255u) kf = 0x7fffu;  // NaN (harmless where the row is not there: it is not seen, and V's is cleared)
      if (vb[k] == 255u) vf = 0x7fffu;
      *reinterpret_cast<uint4*>(&info[(t % kInfoRing) * kRows + 32 * k]) =
          make_uint4(static_cast<uint32_t>(off[k]), static_cast<uint32_t>(off[k] >> 32), kf | (vf << 16), kb[k] | (vb[k] << 8));
    }
    if (lane == 0)
      *reinterpret_cast<uint2*>(sh.top + (t % kOkRing) * 2) =
          own ? make_uint2(127u | kOwn, 127u) : make_uint2(max(kt, 1u) - 1u, max(vt, 1u) - 1u);
    tc_arrive_warp(&br.info_full[t % kInfoRing]);
  };
  ask();
  int t = first;
#pragma unroll 1
  for (; more; t += kFinders) {
    if (t >= kFinders) put(t - kFinders);
    if (t >= kInfoRing && !tc_wait_warp(&br.info_empty[t % kInfoRing], ((t / kInfoRing) - 1) & 1, sh.abort, p.status))
      return;
    const int64_t kv0 = pc.g * p.cache.s_head + (paged ? 0 : pc.b * p.cache.s_batch);
    const int64_t sc0 = pc.g * p.cache.ss_head + (paged ? 0 : pc.b * p.cache.ss_batch);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = tile * kRows + lane + 32 * k;
      bool have = row < pc.e.n;
      int r = row;
      int64_t at = sc0;
      off[k] = kv0;
      if (paged) {
        r = row - page_of(p.cache, row) * p.cache.page_rows;
        const bool in = page[k] >= 0 && page[k] < p.cache.num_pages;
        if (have && !in && p.status) atomicOr(p.status, LYC_OP_BAD_PAGE);
        have = have && in;
        off[k] += page[k] * p.cache.s_page;
        at += page[k] * p.cache.ss_page;
        const uint32_t found = __ballot_sync(0xffffffffu, have);
        if (lane == k) sh.ok[(t % kOkRing) * 4 + k] = found;
      }
      off[k] = have ? off[k] + r * p.cache.s_token : 1;
      at = have ? at + r * p.cache.ss_token : 0;
      kb[k] = p.cache.ks[at];  // some row's where there is none
      vb[k] = p.cache.vs[at];
    }
    skip(kFinders);
    ask();
  }
  if (t >= kFinders) put(t - kFinders);
}

// Half of the producer warps have K, half V; a warp has every kSide-th 4-row unit
// of a tile, eight lanes a row.  A lane copies its 16 codes of a unit to shared
// memory kRawRing groups ahead and converts what it copied itself, so a warp waits for
// nobody's copies but its own.  (With the codes kept in registers instead, the
// loops had to be unrolled over them and, with the softmax's, were larger than the
// SM's instruction cache: more than twice the time.)
template <class C>
__device__ __forceinline__ void tc_produce(const TreeTcParams& P, unsigned char* smem) {
  const TreeParams& p = P.t;
  const int pw = (threadIdx.x >> 5) - C::PROD_WARP, lane = threadIdx.x & 31;
  const int w = pw % kSide, kv = pw / kSide;
  // eight adjacent lanes store half a row each of an even and an odd row: with
  // the swizzle, eight different banks
  const int c = (lane & 3) | (((lane >> 3) & 1) << 2);
  const int r0 = w * 4 + (((lane >> 4) << 1) | ((lane >> 2) & 1));  // the first unit's row; + 4 kSide for each unit
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  uint64_t* const full = kv ? br.vfull : br.kfull;
  uint64_t* const empty = kv ? br.vempty : br.kempty;
  const int S = kv ? C::SV : C::SK;
  unsigned char* const tiles = smem + (kv ? C::OFF_V : C::OFF_K);
  const unsigned char* const base = (kv ? p.cache.v : p.cache.k) + c * 16;
  const uint32_t sel = kv ? 0x3232u : 0x1010u;
  const uint32_t st0 = tile_off(r0, 2 * c), st1 = tile_off(r0, 2 * c + 1);
  unsigned char* const raw = smem + C::OFF_RAW + pw * (kRawRing * kUnits * 512) + lane * 16;
  const RowInfo* const info = reinterpret_cast<const RowInfo*>(smem + C::OFF_INFO) + r0;
  const uint2 run = tree_run<kRows, kRows>(p);
  const int groups = kGroups * static_cast<int>(run.y - run.x);
#pragma unroll 1
  for (int h = -kRawRing; h < groups; ++h) {  // group h is converted, h + kRawRing copied
    if (h >= 0) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRawRing - 1) : "memory");
      const int t = h / kGroups, g = h % kGroups, stage = t % S;
      if (g == 0 && t >= S && !tc_wait_warp(empty + stage, ((t / S) - 1) & 1, sh.abort, p.status)) break;
      const unsigned char* src = raw + (h % kRawRing) * (kUnits * 512);
      const RowInfo* rows = info + (t % kInfoRing) * kRows + g * (kRows / kGroups);
      unsigned char* dst = tiles + stage * C::TILEB + g * (kRows / kGroups) * 128;
      // (all loads before the first store: the compiler cannot tell them apart, and
      // would take one unit after another)
      uint4 codes[kUnits];
      uint32_t factor[kUnits];
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        codes[j] = *reinterpret_cast<const uint4*>(src + j * 512);
        factor[j] = rows[4 * kSide * j].factor;
      }
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const uint4 u = codes[j];
        const uint32_t f = __byte_perm(factor[j], 0, sel);
        uint32_t x[8];
        codes_f16(u.x, &x[0], &x[1]);
        codes_f16(u.y, &x[2], &x[3]);
        codes_f16(u.z, &x[4], &x[5]);
        codes_f16(u.w, &x[6], &x[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = mul_f16x2(x[k], f);
        *reinterpret_cast<uint4*>(dst + st0 + j * (kSide * 512)) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4*>(dst + st1 + j * (kSide * 512)) = make_uint4(x[4], x[5], x[6], x[7]);
      }
      if (g == kGroups - 1) {
        tc::fence_async_smem();
        tc_arrive_warp(full + stage);
        if (lane == 0) mbar_arrive(&br.info_empty[t % kInfoRing]);
      }
    }
    const int hn = h + kRawRing;
    if (hn < groups) {
      const int t = hn / kGroups, g = hn % kGroups;
      if (g == 0 && !tc_wait_warp(&br.info_full[t % kInfoRing], (t / kInfoRing) & 1, sh.abort, p.status)) break;
      const RowInfo* rows = info + (t % kInfoRing) * kRows + g * (kRows / kGroups);
      const uint32_t dst = smem_u32(raw + (hn % kRawRing) * (kUnits * 512));
      long long off[kUnits];
#pragma unroll
      for (int j = 0; j < kUnits; ++j) off[j] = rows[4 * kSide * j].off;
#pragma unroll
      for (int j = 0; j < kUnits; ++j)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + j * 512), "l"(base + (off[j] & ~1ll)),
                     "r"((off[j] & 1) ? 0 : 16)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------- MMA warp
// QK of tile t+1 goes out before the PV of tile t, within a piece (the next
// piece's queries are written only after this one's last PV), and once the PV
// of tile t-1, whose P lies in the same columns, is done.
// (The whole warp waits and keeps the counts, so that the descriptors are uniform
// values; one elected lane issues.)
__device__ __forceinline__ bool tc_elect() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

template <class C>
__device__ __forceinline__ void tc_mma(const TreeTcParams& P, unsigned char* smem, uint32_t tmem) {
  const TreeParams& p = P.t;
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  const uint64_t qd = tc::smem_desc(smem_u32(smem + C::OFF_Q), 16, 1024, 2);
  const uint64_t kd = tc::smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
  const uint64_t vd = tc::smem_desc(smem_u32(smem + C::OFF_V), 16384, 1024, 2);
  TcWalk walk(p);
  TreePiece pc;
  int t = 0, piece = 0;
  bool ok = true;

  auto issue_qk = [&](int tt, bool first) -> bool {
    const int stage = tt % C::SK, b = tt & 1;
    if (first && !tc_wait_warp(br.q_ready, piece & 1, sh.abort, p.status)) return false;
    if (tt >= 2 && !tc_wait_warp(&br.pv_done[b], ((tt - 2) >> 1) & 1, sh.abort, p.status)) return false;
    if (!tc_wait_warp(&br.kfull[stage], (tt / C::SK) & 1, sh.abort, p.status)) return false;
    tc::fence_after_sync();
    const uint64_t ks = kd + static_cast<uint32_t>(stage * (C::TILEB >> 4));
    if (tc_elect()) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
        tc::mma_bf16_ss(tmem + b * 128, qd + off, ks + off, tc_idesc(C::F8, 0), kk > 0 ? 1u : 0u);
      }
      tc::commit(&br.kempty[stage]);
      tc::commit(&br.s_ready[b]);
    }
    __syncwarp();
    return true;
  };

  while (ok && walk.next(&pc)) {
    const int cnt = pc.t1 - pc.t0;
#pragma unroll 1
    for (int u = -1; ok && u < cnt; ++u) {
      // the next tile's QK (the first time the piece's first), then this tile's PV
      if (u + 1 < cnt) ok = issue_qk(t + (u < 0 ? 0 : 1), u < 0);
      if (!ok || u < 0) continue;
      const int b = t & 1, vs = t % C::SV;
      ok = tc_wait_warp(&br.p_ready[b], (t >> 1) & 1, sh.abort, p.status) &&
           tc_wait_warp(&br.vfull[vs], (t / C::SV) & 1, sh.abort, p.status) &&
           (u > 0 || piece == 0 || tc_wait_warp(br.o_free, (piece - 1) & 1, sh.abort, p.status));
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t vst = vd + static_cast<uint32_t>(vs * (C::TILEB >> 4));
      if (tc_elect()) {
#pragma unroll
        for (int kt = 0; kt < 8; ++kt) {
          // keys 0-63 into O_a (column 256), 64-127 into O_b (384); P's half at its S half
          const uint32_t a = tmem + b * 128 + (kt >> 2) * 64 + (kt & 3) * 8;
          mma_ts(tmem + 256 + (kt >> 2) * 128, a, vst + kt * 128, tc_idesc(C::F8, 1),
                 ((kt & 3) > 0 || u > 0) ? 1u : 0u);
        }
        tc::commit(&br.vempty[vs]);
        tc::commit(&br.pv_done[b]);
        if (C::F8) tc::commit(&br.info_empty[t % kInfoRing]);  // the softmax is done with the tile's rows, too
      }
      __syncwarp();
      ++t;
    }
    ++piece;
  }
  // every MMA has completed before the tensor memory is given back
  if (tc_elect()) tc::commit(br.idle);
  __syncwarp();
  tc_wait(br.idle, 0, sh.abort, p.status, false);
  __syncwarp();
}

// ---------------------------------------------------------------- softmax warps
// Bits x of the result: row kb + x (x < 64) is seen by node t.
__device__ __noinline__ unsigned long long seen_bits(const TreeParams& p, const TreePiece& pc, int t, int kb) {
  const int first = pc.e.n - pc.e.cnt;
  const int node0 = kb - first;  // node of bit 0 (negative: rows before the draft)
  auto word = [&](int w) -> unsigned long long {
    if (w < 0 || 64 * w >= pc.e.cnt) return 0ull;
    unsigned long long m;
    if (p.mask)
      m = p.mask[(static_cast<int64_t>(pc.b) * p.T + t) * p.W + w];
    else
      m = t - 64 * w >= 63 ? ~0ull : t < 64 * w ? 0ull : (2ull << (t - 64 * w)) - 1ull;
    const int left = pc.e.cnt - 64 * w;  // nodes of the word
    return left >= 64 ? m : m & ((1ull << left) - 1ull);
  };
  unsigned long long v;
  if (node0 <= -64) {
    v = ~0ull;
  } else if (node0 < 0) {
    v = (word(0) << (-node0)) | ((1ull << (-node0)) - 1ull);
  } else {
    const int w = node0 >> 6, s = node0 & 63;
    v = word(w) >> s;
    if (s) v |= word(w + 1) << (64 - s);
  }
  return v;
}

// Half h of row r of a V tile: zeros where the row is gone; in drafted rows
// (node >= 0) NaNs and infinities become zeros, and the node is marked.
template <bool F8>
__device__ __noinline__ void clean_row(unsigned char* v, int r, int h, bool gone, int node, uint32_t* odd_rows) {
  if (!gone && node < 0) return;
  bool odd = false;
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint4* at = reinterpret_cast<uint4*>(v + tile_off(r, h * 8 + c));
    const uint4 x = *at;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool here = gone;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      constexpr uint32_t kExp = F8 ? 0x7c00u : 0x7f80u;  // of f16, bf16
      const bool lo = (w[k] & kExp) == kExp, hi = (w[k] & (kExp << 16)) == kExp << 16;
      here |= lo | hi;
      if (gone || lo) w[k] &= 0xffff0000u;
      if (gone || hi) w[k] &= 0xffffu;
    }
    if (here) *at = make_uint4(w[0], w[1], w[2], w[3]);
    odd |= here;
  }
  if (odd && !gone) atomicOr(&odd_rows[node >> 5], 1u << (node & 31));
}

// Adds the NaNs and infinities of the marked drafted rows that `node` sees to its
// row's 64 columns from col0 on, written before by this thread.
template <bool F8>
__device__ __noinline__ void add_odd(const TreeParams& p, const TreePiece& pc, int node, int col0, const uint32_t* odd_rows,
                                     uint16_t* out, float* part) {
#pragma unroll 1
  for (int x = 0; x < pc.e.cnt; ++x) {
    if (!((odd_rows[x >> 5] >> (x & 31)) & 1u) || !tree_sees(p, pc.b, node, x)) continue;
    RowAt at;
    if (!cache_row(p.cache, pc.b, pc.e.n - pc.e.cnt + x, &at)) continue;
    const int64_t v = at.kv + pc.g * p.cache.s_head + col0;
#pragma unroll 1
    for (int j = 0; j < 64; ++j) {
      float y;
      if (F8) {  // a NaN row (or a code that no writer makes)
        const bool nan = p.cache.vs[at.sc + pc.g * p.cache.ss_head] == 255 || (p.cache.v[v + j] & 0x7f) == 0x7f;
        y = nan ? __uint_as_float(0x7fffffffu) : 0.f;
      } else {
        y = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.cache.v)[v + j]) << 16);
      }
      if (fabsf(y) < INFINITY) continue;
      if (part)
        part[j] += y;
      else
        out[j] = static_cast<uint16_t>(tc_pack(__uint_as_float(static_cast<uint32_t>(out[j]) << 16) + y, 0.f));
    }
  }
}

// The copies of a whole group's rows merged into its output, by all softmax warps
// (half hf has columns 64 hf .. + 63), 32 columns a turn through the query
// buffer.  (M, L) is the copy's state, fa and fb its key halves' factors.
struct CopyMerge {
  uint32_t tl;  // this warp's lanes of the tensor memory
  int hf, copy, copies, li, span;
  bool live;
  float M, L, fa, fb;
  unsigned char* qbuf;
  uint64_t* bar;  // all softmax warps'
  int* abort;
  uint32_t* status;
  unsigned char* dst;
};
template <class C>
__device__ __noinline__ bool merge_copies(const CopyMerge& m, uint32_t phase) {
  float2* cm = reinterpret_cast<float2*>(m.qbuf + 24576);
  auto together = [&]() {
    tc_arrive_warp(m.bar);
    return tc_wait_warp(m.bar, phase++ & 1, m.abort, m.status);
  };
  if (!together()) return false;  // the halves' states have been read
  if (m.hf == 0) cm[m.copy * m.span + m.li] = make_float2(m.M, m.L);
#pragma unroll 1
  for (int step = 0; step < 2; ++step) {
    uint32_t a[2][16], b[2][16];
    const uint32_t col = m.tl + 256 + m.hf * 64 + step * 32;
    tc::ld_32x32b_x16(col, a[0]);
    tc::ld_32x32b_x16(col + 16, a[1]);
    tc::ld_32x32b_x16(col + 128, b[0]);
    tc::ld_32x32b_x16(col + 144, b[1]);
    tc_wait_ld<2>(a);
    tc_wait_ld<2>(b);
    float o[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      o[j] = fmaf(__uint_as_float(a[j >> 4][j & 15]), m.fa, __uint_as_float(b[j >> 4][j & 15]) * m.fb);
    }
    unsigned char* mine = m.qbuf + m.li * 256 + m.hf * 128;
    if (m.copy > 0)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<float4*>(mine + (m.copy - 1) * m.span * 256 + ((q ^ (m.li & 7)) << 4)) =
            make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    if (!together()) return false;
    if (m.copy == 0 && m.live) {
      float M = m.M;
      for (int k = 1; k < m.copies; ++k) M = fmaxf(M, cm[k * m.span + m.li].x);
      const float f0 = m.M == -INFINITY ? 1.f : tc_ex2(m.M - M);  // 1: the state is zero, or NaN
      float L = m.L * f0;
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] *= f0;
#pragma unroll 1
      for (int k = 1; k < m.copies; ++k) {
        const float2 s = cm[k * m.span + m.li];
        const float f = s.x == -INFINITY ? 1.f : tc_ex2(s.x - M);
        L = fmaf(s.y, f, L);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 u = *reinterpret_cast<const float4*>(mine + (k - 1) * m.span * 256 + ((q ^ (m.li & 7)) << 4));
          o[4 * q] = fmaf(u.x, f, o[4 * q]);
          o[4 * q + 1] = fmaf(u.y, f, o[4 * q + 1]);
          o[4 * q + 2] = fmaf(u.z, f, o[4 * q + 2]);
          o[4 * q + 3] = fmaf(u.w, f, o[4 * q + 3]);
        }
      }
      const float inv = L == 0.f ? 0.f : (C::F8 ? kSumUnitE4m3 : 1.f) / L;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(m.dst + step * 64 + q * 16) =
            make_uint4(tc_pack(o[8 * q] * inv, o[8 * q + 1] * inv), tc_pack(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                       tc_pack(o[8 * q + 4] * inv, o[8 * q + 5] * inv), tc_pack(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
    }
    if (!together()) return false;
  }
  return true;
}
constexpr uint32_t kMergeWaits = 5;
// Of a whole group: fewer are not worth the merge (12 nodes over 512 rows, 64
// elements: 78 us with it, 56 without; e4m3 111 and 84).
constexpr int kMergeTiles = 16;

// A tile whose rows have their own scales: n columns of logits from `col` on become
// z + e in log2 units (e of V), -inf where `vis` is not set.
__device__ __noinline__ void own_logits(uint32_t col, int n, const RowInfo* own, float per_s, unsigned long long vis) {
#pragma unroll 1
  for (int c = 0; c < n; c += 16) {
    uint32_t r[1][16];
    tc::ld_32x32b_x16(col + c, r[0]);
    tc_wait_ld<1>(r);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t k = own[c + j].own & 255u, v = own[c + j].own >> 8;
      const float kf = k == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(max(k, 1u) << 23);
      const float ev = v == 255u ? 0.f : static_cast<float>(static_cast<int>(v) - 127);  // (its V row is NaN itself)
      const float x = fmaf(__uint_as_float(r[0][j]) * per_s, kf, ev);
      r[0][j] = (vis >> (c + j)) & 1ull ? __float_as_uint(x) : __float_as_uint(-INFINITY);
    }
    tc_st_x16(col + c, r[0]);
  }
  tc_wait_st();
}
// ... and the sum of 2^(z + neg) over them, in units of 2^16 (kSumUnitE4m3).
__device__ __noinline__ float own_sum(uint32_t col, int n, const RowInfo* own, float neg) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < n; c += 16) {
    uint32_t r[1][16];
    tc::ld_32x32b_x16(col + c, r[0]);
    tc_wait_ld<1>(r);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t v = own[c + j].own >> 8;
      const float ev = v == 255u ? 0.f : static_cast<float>(static_cast<int>(v) - 127);
      sum += tc_ex2(__uint_as_float(r[0][j]) - ev + (neg - 16.f));
    }
  }
  return sum;
}

template <class C>
__device__ __forceinline__ void tc_softmax(const TreeTcParams& P, unsigned char* smem, uint32_t tmem) {
  const TreeParams& p = P.t;
  constexpr unsigned FULL = 0xffffffffu;
  const float NEG = -INFINITY;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, hf = warp >> 2;
  const int i = quarter * 32 + lane;
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t tl_o = tl + 256 + hf * 128;
  unsigned char* qbuf = smem + C::OFF_Q;
  // where half x of this row finds the other half's (m, l) at the end of a
  // piece: in the part of the query row that x itself writes next
  auto ml_of = [&](int x) {
    return reinterpret_cast<float2*>(qbuf + tile_off(i, x * 8));
  };
  TcWalk walk(p);
  TreePiece pc;
  int t = 0, piece = 0;
  uint32_t together = 0;  // times that all softmax warps have waited for one another
  while (walk.next(&pc)) {
    const bool whole = pc.t0 == 0 && pc.t1 == pc.nt;
    const int copies = whole && pc.nt < kMergeTiles ? 1 : tree_copies(pc.e.cnt * p.G - pc.mb * kRows), span = kRows / copies;
    const int copy = i / span;
    const int row = pc.mb * kRows + i - copy * span;
    const int node = row / p.G, head = pc.g * p.G + row % p.G;
    const bool live = node < pc.e.cnt;
    const bool warp_live = (pc.mb * kRows + (quarter * 32) % span) / p.G < pc.e.cnt;
    const int k0 = copy * (64 / copies);  // the copy's keys of the half: k0 .. k0 + 64 / copies - 1
    const int first_draft = pc.e.n - pc.e.cnt;
    float row_log2 = p.scale_log2;  // F8: with the row's power of two
    if (warp_live) {
      const unsigned char* src = p.q + 2 * (pc.b * p.q_batch + node * p.q_token + head * p.q_head);
      uint4 mine[8];
#pragma unroll
      for (int c8 = 0; c8 < 8; ++c8) {
        mine[c8] = make_uint4(0u, 0u, 0u, 0u);
        if (live) mine[c8] = *reinterpret_cast<const uint4*>(src + (hf * 8 + c8) * 16);
      }
      float f1 = 1.f, f2 = 1.f;
      if (C::F8) {
        // as f16, scaled by a power of two to below 2 (exact for elements down to 2^-17
        // of the row's largest: bf16's 8 bits end at f16's 2^-24; half of that off below)
        uint32_t mx = 0u;
        auto most = [&](const uint4& v) {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        };
        uint4 other[8];  // all of the row is asked for at once
#pragma unroll
        for (int c8 = 0; c8 < 8; ++c8) {
          other[c8] = make_uint4(0u, 0u, 0u, 0u);
          if (live) other[c8] = *reinterpret_cast<const uint4*>(src + ((1 - hf) * 8 + c8) * 16);
        }
#pragma unroll
        for (int c8 = 0; c8 < 8; ++c8) {
          most(mine[c8]);
          most(other[c8]);
        }
        int ex = static_cast<int>(mx >> 7);  // biased exponent of the row's largest element
        if (ex == 0 || ex == 255) ex = 127;
        // it comes off in two factors: 2^-(ex - 127) may be out of fp32's range
        const int e1 = (ex - 127) / 2, e2 = ex - 127 - e1;
        f1 = __uint_as_float(static_cast<uint32_t>(127 - e1) << 23);
        f2 = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
        row_log2 *= __uint_as_float(static_cast<uint32_t>(ex) << 23);
      }
#pragma unroll
      for (int c8 = 0; c8 < 8; ++c8) {
        const int ch = hf * 8 + c8;
        uint4 v = mine[c8];
        if (C::F8) {
          v.x = tc_pack_f16(bf16lo(v.x) * f1 * f2, bf16hi(v.x) * f1 * f2);
          v.y = tc_pack_f16(bf16lo(v.y) * f1 * f2, bf16hi(v.y) * f1 * f2);
          v.z = tc_pack_f16(bf16lo(v.z) * f1 * f2, bf16hi(v.z) * f1 * f2);
          v.w = tc_pack_f16(bf16lo(v.w) * f1 * f2, bf16hi(v.w) * f1 * f2);
        }
        *reinterpret_cast<uint4*>(qbuf + tile_off(i, ch)) = v;
      }
      tc::fence_async_smem();
    }
    uint32_t* odd_rows = sh.odd + (piece & 1) * 8;  // last read two pieces ago
    if (threadIdx.x < 8) odd_rows[threadIdx.x] = 0u;
    tc_arrive_warp(br.q_ready);

    float m_used = NEG, lsum = 0.f;
    for (int u = pc.t0; u < pc.t1; ++u, ++t) {
      const int b = t & 1;
      if (!tc_wait_warp(&br.s_ready[b], (t >> 1) & 1, sh.abort, p.status)) return;
      const int tile_row = u * kRows;
      const int kb = tile_row + hf * 64;
      uint2 top = make_uint2(127u, 127u);
      if (C::F8) top = *reinterpret_cast<const uint2*>(sh.top + (t % kOkRing) * 2);
      bool found_all = true;
      const volatile uint32_t* okw = sh.ok + (t % kOkRing) * 4;
      if (p.cache.bt)  // written before the tile's rows were asked for; ten tiles on, this one's PV is done
        found_all = (okw[0] & okw[1] & okw[2] & okw[3]) == 0xffffffffu;
      const bool special = !found_all || tile_row + kRows > first_draft;
      tc::fence_after_sync();
      unsigned long long vis = ~0ull, there = ~0ull;
      if (__builtin_expect(special, 0)) {
        if (!found_all) there = okw[2 * hf] | (static_cast<unsigned long long>(okw[2 * hf + 1]) << 32);
        vis = live ? seen_bits(p, pc, node, kb) & there : 0ull;
      }
      // F8: the tile's K scale is the logit's, its V scale is taken into the exponent
      // (p' = 2^(z + e - m'), and the sum takes p' 2^-e)
      float per_s = p.scale_log2, v_exp = 0.f, v_inv = 1.f;
      if (C::F8) {
        per_s = fminf(fmaxf(row_log2 * __uint_as_float(max(top.x & 255u, 1u) << 23), 1.17549435e-38f), 3.4e38f);
        v_exp = static_cast<float>(static_cast<int>(top.y) - 127);
        v_inv = tree_sum_factor(top.y);
      }
      if (warp_live) {
        // both passes read the logits from tensor memory, 32 columns a turn: the
        // loops stay small (all 64 in registers made the kernel's loops together
        // larger than the SM's instruction cache); a quarter's 16 stay in registers
        const uint32_t ts = tl + b * 128 + hf * 64;
        const bool own = C::F8 && (top.x & kOwn) != 0u;
        const RowInfo* own_row = reinterpret_cast<const RowInfo*>(smem + C::OFF_INFO) + (t % kInfoRing) * kRows + hf * 64 + k0;
        if (__builtin_expect(own, 0)) {
          own_logits(ts + k0, 64 / copies, own_row, row_log2, vis >> k0);
          per_s = 1.f;
          v_inv = 0.f;  // the sum is own_sum's
        }
        float mraw = NEG;
        uint32_t few[2][16];
        if (copies == 2) {
          tc::ld_32x32b_x16(ts + k0, few[0]);
          tc::ld_32x32b_x16(ts + k0 + 16, few[1]);
          tc_wait_ld<2>(few);
          if (__builtin_expect(special, 0)) {
            const uint32_t v = static_cast<uint32_t>(vis >> k0);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((v >> j) & 1u)) few[j >> 4][j & 15] = __float_as_uint(NEG);
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            mraw = fmaxf(mraw, fmaxf(__uint_as_float(few[j >> 4][j & 15]), __uint_as_float(few[j >> 4][(j + 1) & 15])));
        } else {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t r[2][16];
            tc::ld_32x32b_x16(ts + c, r[0]);
            tc::ld_32x32b_x16(ts + c + 16, r[1]);
            tc_wait_ld<2>(r);
            if (__builtin_expect(special, 0)) {
              const uint32_t v = static_cast<uint32_t>(vis >> c);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((v >> j) & 1u)) r[j >> 4][j & 15] = __float_as_uint(NEG);
              tc_st_x16(ts + c, r[0]);
              tc_st_x16(ts + c + 16, r[1]);
              tc_wait_st();
            }
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              mraw = fmaxf(mraw, fmaxf(__uint_as_float(r[j >> 4][j & 15]), __uint_as_float(r[j >> 4][(j + 1) & 15])));
          }
        }
        const float mx = fmaf(mraw, per_s, v_exp);
        const bool grow = mx > m_used + TcRange<C::F8>::kLag;
        const bool rescale = grow && m_used != NEG;
        if (__any_sync(FULL, rescale)) {
          if (!tc_wait_warp(&br.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, sh.abort, p.status)) return;
          tc::fence_after_sync();
          const float f = rescale ? tc_ex2(m_used - mx) : 1.f;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[1][16];
            tc::ld_32x32b_x16(tl_o + c * 16, o[0]);
            tc_wait_ld<1>(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[0][j] = __float_as_uint(__uint_as_float(o[0][j]) * f);
            tc_st_x16(tl_o + c * 16, o[0]);
          }
          lsum *= f;
        }
        if (grow) m_used = mx;
        const float neg = (m_used == NEG ? 0.f : -m_used) + (C::F8 ? v_exp + TcRange<true>::kTop : 0.f);
        if (__builtin_expect(own, 0)) lsum += own_sum(ts + k0, 64 / copies, own_row, neg);
        const f2_t neg2 = f2(neg, neg), sl2 = f2(per_s, per_s);
        f2_t sum2 = f2(0.f, 0.f);
        auto prob = [&](const uint32_t* x) -> uint32_t {  // two columns' probabilities, packed
          float p0, p1;
          f2_split(f2_fma(f2(__uint_as_float(x[0]), __uint_as_float(x[1])), sl2, neg2), &p0, &p1);
          p0 = tc_ex2(p0);
          p1 = tc_ex2(p1);
          sum2 = f2_add(f2(p0, p1), sum2);
          return C::F8 ? tc_pack_f16(p0, p1) : tc_pack(p0, p1);
        };
        // P's columns (two keys each) take the place of logits that were read
        uint32_t w[16];
        if (copies == 2) {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = prob(&few[e >> 3][(2 * e) & 15]);
          tc_st_x16(ts + k0 / 2, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0u;
          tc_st_x16(ts + 16 * (1 - copy), w);
        } else {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t r[2][16];
            tc::ld_32x32b_x16(ts + c, r[0]);
            tc::ld_32x32b_x16(ts + c + 16, r[1]);
            tc_wait_ld<2>(r);
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = prob(&r[e >> 3][(2 * e) & 15]);
            tc_st_x16(ts + c / 2, w);
          }
        }
        {
          float s0, s1;
          f2_split(sum2, &s0, &s1);
          lsum = fmaf(s0 + s1, v_inv, lsum);
        }
        tc_wait_st();
      }
      if (special) {
        // V's rows that the tensor core must not meet as they are
        const int stage = t % C::SV;
        if (!tc_wait_warp(&br.vfull[stage], (t / C::SV) & 1, sh.abort, p.status)) return;
        const int r = threadIdx.x >> 1;  // two threads a row
        const bool gone = tile_row + r >= pc.e.n || (!found_all && !((okw[r >> 5] >> (r & 31)) & 1u));
        clean_row<C::F8>(smem + C::OFF_V + stage * C::TILEB, r, threadIdx.x & 1, gone, tile_row + r - first_draft, odd_rows);
        tc::fence_async_smem();
      }
      tc::fence_before_sync();
      tc_arrive_warp(&br.p_ready[b]);
    }

    // the piece's state: both halves' outputs under one maximum
    const int last = t - 1;
    if (!tc_wait_warp(&br.pv_done[last & 1], (last >> 1) & 1, sh.abort, p.status)) return;
    tc::fence_after_sync();
    *ml_of(1 - hf) = make_float2(m_used, lsum);
    tc_arrive_warp(br.ml_ready);
    if (!tc_wait_warp(br.ml_ready, together++ & 1, sh.abort, p.status)) return;
    const bool merge = whole && copies > 1;
    if (warp_live || merge) {
      const float2 own = make_float2(m_used, lsum), other = *ml_of(hf);
      const float2 sa = hf ? other : own, sb = hf ? own : other;
      const float M = fmaxf(sa.x, sb.x);
      const float fa = sa.x == NEG ? 1.f : tc_ex2(sa.x - M);  // 1: the state is zero, or NaN
      const float fb = sb.x == NEG ? 1.f : tc_ex2(sb.x - M);
      const float L = fmaf(sa.y, fa, sb.y * fb);
      const float unit = whole ? (L == 0.f ? 0.f : p.sum_unit / L) : 1.f;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (pc.t0 == 0 ? 1 : 0);
      float* part = p.part_o + (slot * kRows + i) * kD + hf * 64;
      unsigned char* dst = p.out + 2 * (pc.b * p.o_batch + node * p.o_token + head * p.o_head + hf * 64);
      bool odd = false;
      for (int w = 0; w < 8; ++w) odd |= odd_rows[w] != 0u;
      if (merge) {
        const CopyMerge cm{tl, hf, copy, copies, i - copy * span, span, live, M, L, fa, fb, qbuf, br.ml_ready, sh.abort, p.status, dst};
        if (!merge_copies<C>(cm, together)) return;
        together += kMergeWaits;
      } else
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t ab[2][16];
        tc::ld_32x32b_x16(tl + 256 + hf * 64 + c * 16, ab[0]);
        tc::ld_32x32b_x16(tl + 384 + hf * 64 + c * 16, ab[1]);
        tc_wait_ld<2>(ab);
        float o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j] = fmaf(__uint_as_float(ab[0][j]), fa, __uint_as_float(ab[1][j]) * fb) * unit;
        }
        if (live) {
          if (whole) {
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              *reinterpret_cast<uint4*>(dst + 2 * (c * 16 + j)) =
                  make_uint4(tc_pack(o[j], o[j + 1]), tc_pack(o[j + 2], o[j + 3]),
                             tc_pack(o[j + 4], o[j + 5]), tc_pack(o[j + 6], o[j + 7]));
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              *reinterpret_cast<float4*>(part + c * 16 + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
      }
      if (__builtin_expect(odd, 0) && live && copy == 0)
        add_odd<C::F8>(p, pc, node, hf * 64, odd_rows, reinterpret_cast<uint16_t*>(dst), whole ? nullptr : part);
      if (!whole && live && hf == 0) p.part_ml[slot * kRows + i] = make_float2(M, L);
    }
    tc::fence_before_sync();
    tc_arrive_warp(br.o_free);
    ++piece;
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tree_tc_kernel(const __grid_constant__ TreeTcParams P) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const TcShared sh = shared_of<C>(smem);
  if (threadIdx.x == 0) {
    TcBars<C> br(smem);
    for (int s = 0; s < C::SK; ++s) {
      mbar_init(&br.kfull[s], C::FULL);
      mbar_init(&br.kempty[s], 1);
    }
    for (int s = 0; s < C::SV; ++s) {
      mbar_init(&br.vfull[s], C::FULL);
      mbar_init(&br.vempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&br.s_ready[b], 1);
      mbar_init(&br.p_ready[b], kSoft / 32);
      mbar_init(&br.pv_done[b], 1);
    }
    mbar_init(br.q_ready, kSoft / 32);
    mbar_init(br.o_free, kSoft / 32);
    mbar_init(br.ml_ready, kSoft / 32);
    mbar_init(br.idle, 1);
    if (C::F8)
      for (int s = 0; s < kInfoRing; ++s) {
        mbar_init(&br.info_full[s], 1);
        mbar_init(&br.info_empty[s], kProducers + 1);
      }
    *sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) {
    tc::tmem_alloc(sh.tmem, 512);
    tc::tmem_relinquish();
  }
  if (!C::F8 && threadIdx.x == C::LOAD_WARP * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmv)) : "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *sh.tmem;
  pdl_wait();
  pdl_launch_dependents();
  if (warp < 8) {
    if (blockIdx.x == 0 && P.t.status)
      for (int b = threadIdx.x; b < P.t.B; b += kSoft) {
        bool bad = false;
        tree_elem(P.t, b, &bad);
        if (bad) atomicOr(P.t.status, LYC_OP_BAD_LENGTH);
      }
    __syncwarp();
    tc_softmax<C>(P, smem, tmem);
  } else if (warp == C::MMA_WARP) {
    tc_mma<C>(P, smem, tmem);
  } else if (!C::F8) {
    tc_loads<C>(P, smem);
  } else if (warp < C::PROD_WARP) {
    tc_rows<C>(P, smem);
  } else {
    tc_produce<C>(P, smem);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == C::MMA_WARP) tc::tmem_dealloc(tmem, 512);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<EncodeTiledFn>(ptr);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

// 4-D map of a bf16 K or V: (d, row, head, element), or paged (d, head, row, page).
bool encode(CUtensorMap* map, void* base, const CacheView& c, int heads, int batch, int box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int64_t es = 2;
  const bool paged = c.bt != nullptr;
  cuuint64_t dims[4] = {kD, static_cast<cuuint64_t>(paged ? heads : c.cap), static_cast<cuuint64_t>(paged ? c.page_rows : heads),
                        static_cast<cuuint64_t>(paged ? c.num_pages : batch)};
  int64_t st[3] = {(paged ? c.s_head : c.s_token) * es, (paged ? c.s_token : c.s_head) * es,
                   (paged ? c.s_page : c.s_batch) * es};
  // a dimension of one entry is only read at coordinate 0: any stride will do
  for (int k = 0; k < 3; ++k)
    if (dims[k + 1] == 1) st[k] = kD * es;
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st[0]), static_cast<cuuint64_t>(st[1]),
                                 static_cast<cuuint64_t>(st[2])};
  cuuint32_t box[4] = {64, 1, 1, 1};
  box[paged ? 2 : 1] = static_cast<cuuint32_t>(box_rows);
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_tc(const TreeTcParams* P, int device, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // per device; setting the attribute twice does no harm
  if (device >= 64 || !configured[device].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (device < 64) configured[device].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(P->t.grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_tc_kernel<C>, *P);
}

}  // namespace

// Rows of a box: a whole tile of a contiguous cache, else the largest power of
// two that divides a page (a tile is then made of whole boxes); 0 where that
// is below the eight rows that the shared-memory layout swizzles together.
int tree_tc_box_rows(const CacheView& c) {
  if (!c.bt) return kRows;
  const int low = c.page_rows & -c.page_rows;
  return low < 8 ? 0 : low < kRows ? low : kRows;
}

bool tree_tc_maps(TreeTcParams* P) {
  const CacheView& c = P->t.cache;
  return encode(&P->tmk, c.k, c, P->t.Hkv, P->t.B, P->t.box_rows) &&
         encode(&P->tmv, c.v, c, P->t.Hkv, P->t.B, P->t.box_rows);
}

cudaError_t tree_tc_launch(const TreeTcParams* P, int cache_type, int device, cudaStream_t stream) {
  return cache_type == LYC_CACHE_E4M3 ? launch_tc<TcCfg<true>>(P, device, stream)
                                      : launch_tc<TcCfg<false>>(P, device, stream);
}

}  // namespace lyc
