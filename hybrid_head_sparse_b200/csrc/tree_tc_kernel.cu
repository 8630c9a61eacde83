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
// Warp 8 issues the MMAs (one thread), warp 9 the TMA copies; two S buffers
// let the QK of tile t+1 run beside the softmax of tile t.  A warp none of
// whose rows is a query does nothing but keep the barriers going.
//
// bf16 rows: K and V tiles are read by the tensor core where TMA puts them.
// Masked rows have P = 0, and 0 * NaN would reach every row, so in the tiles
// that hold drafted rows or end an element the softmax warps clear rows past
// the end, and take a drafted row's NaNs and infinities out of V; the nodes
// that see such a row get them added at the end.
//
// e4m3 rows: K's codes are the B operand as they are (kind::f8f6f4), against
// the query row in two e4m3 terms, high and low (four significant bits each,
// a bf16 query's eight; what is below 2^-17 of the row's largest element is
// rounded there).  V's codes become f16 on their way through four converter
// warps (value * 2^-8, exact), P is f16.  V's scales go into the exponent and
// K's into the logit, as in tree_mma_kernel.cu.
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
constexpr int kOkRing = 8;

template <bool F8_>
struct TcCfg {
  static constexpr bool F8 = F8_;
  static constexpr int SK = F8 ? 4 : 3;              // K tiles in flight
  static constexpr int SV = F8 ? 3 : 3;              // V tiles in flight
  static constexpr int SC = 2;                       // converted V tiles (F8)
  static constexpr int NS = 4;                       // tiles of scales (F8)
  static constexpr int TILEB = F8 ? 16384 : 32768;   // a K or V tile as it lies in the cache
  static constexpr int CONV = F8 ? 128 : 0;          // converter threads
  static constexpr int THREADS = kSoft + 64 + CONV;
  static constexpr int MMA_WARP = 8, LOAD_WARP = 9, CONV_WARP = 10;
  static constexpr int OFF_Q = 0;                    // bf16 32 KiB; F8: high terms, low terms
  static constexpr int OFF_K = 32768;
  static constexpr int OFF_V = OFF_K + SK * TILEB;
  static constexpr int OFF_VC = OFF_V + SV * TILEB;
  static constexpr int OFF_SCALE = OFF_VC + (F8 ? SC * 32768 : 0);  // [NS][3][128] floats
  static constexpr int OFF_BAR = OFF_SCALE + (F8 ? NS * 3 * 512 : 0);
  // kfull, kempty [SK]; vfull, vempty [SV]; s_ready, p_ready, pv_done [2];
  // q_ready, o_free, ml_ready, idle; F8: vc_full, vc_empty [SC], sc_full [NS]
  static constexpr int NBAR = 2 * SK + 2 * SV + 6 + 4 + (F8 ? 2 * SC + NS : 0);
  static constexpr int OFF_FLAGS = OFF_BAR + NBAR * 8;  // abort, tmem, odd rows [2][8], ok [kOkRing]
  static constexpr int SMEM = OFF_FLAGS + 8 + 64 + 4 * kOkRing + 1024;  // + alignment
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

template <class C>
struct TcBars {
  uint64_t *kfull, *kempty, *vfull, *vempty, *s_ready, *p_ready, *pv_done, *q_ready, *o_free, *ml_ready, *idle,
      *vc_full, *vc_empty, *sc_full;
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
    vc_full = idle + 1;
    vc_empty = vc_full + (C::F8 ? C::SC : 0);
    sc_full = vc_empty + (C::F8 ? C::SC : 0);
  }
};

struct TcShared {
  int* abort;
  uint32_t* tmem;
  uint32_t* odd;  // [2] by piece: drafted rows with a NaN or an infinity in V, by node
  uint32_t* ok;   // ring of the tiles' boxes that were found
};
template <class C>
__device__ __forceinline__ TcShared shared_of(unsigned char* smem) {
  TcShared s;
  s.abort = reinterpret_cast<int*>(smem + C::OFF_FLAGS);
  s.tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAGS + 4);
  s.odd = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAGS + 8);
  s.ok = s.odd + 16;
  return s;
}

// Wait for a phase of `bar`; false once the CTA has given up (a wait above
// kWaitLimitNs).  heed: also give up where another warp has.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t* status,
                                        bool heed = true) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
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
template <bool F16>
__device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
  uint32_t r;
  if (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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

// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem], e4m3 operands, K = 32
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// fp32 sums, M = N = 128; bits 7-9 and 10-12 the types of A and B (f16 0, bf16 1; e4m3 0)
__host__ __device__ constexpr uint32_t idesc128(uint32_t type, int b_mn_major) {
  return (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(b_mn_major) << 16) | ((128u >> 3) << 17) |
         ((128u >> 4) << 24);
}

typedef TreeWalk<kRows, kRows> TcWalk;

// ---------------------------------------------------------------- loads
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
  const int nbox = kRows / P.t.box_rows;
  const uint32_t boxb = static_cast<uint32_t>(C::TILEB) / nbox;  // bytes of a box
  TcWalk walk(p);
  TreePiece pc;
  int t = 0;
  int asked[2] = {0, 0};  // tiles of K and of V whose copies went out
  bool ok = true;
  while (ok && walk.next(&pc)) {
    for (int tile = pc.t0; ok && tile < pc.t1; ++tile, ++t) {
      const int row0 = tile * kRows + lane * P.t.box_rows;
      bool have = lane < nbox && row0 < pc.e.n;
      int c1 = row0, c2 = pc.g, c3 = pc.b;
      if (paged && have) {
        const int blk = row0 / p.cache.page_rows;
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
        if (lane == 0) {
          if (kv == 0) sh.ok[t % kOkRing] = found;
          mbar_arrive_expect_tx(full, bytes);
        }
        __syncwarp();
        if (have) {
          unsigned char* dst = smem + (kv ? C::OFF_V : C::OFF_K) + stage * C::TILEB + lane * P.t.box_rows * 128;
          const CUtensorMap* map = kv ? &P.tmv : &P.tmk;
          tma_4d(dst, map, 0, c1, c2, c3, full, pol);
          if (!C::F8) tma_4d(dst + 16384, map, 64, c1, c2, c3, full, pol);
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

// ---------------------------------------------------------------- MMA warp
// QK of tile t+1 goes out before the PV of tile t, within a piece (the next
// piece's queries are written only after this one's last PV), and once the PV
// of tile t-1, whose P lies in the same columns, is done.
template <class C>
__device__ __forceinline__ void tc_mma(const TreeTcParams& P, unsigned char* smem, uint32_t tmem) {
  const TreeParams& p = P.t;
  const int lane = threadIdx.x & 31;
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  const uint32_t qbase = smem_u32(smem + C::OFF_Q);
  const uint32_t kbase = smem_u32(smem + C::OFF_K);
  const uint32_t vbase = smem_u32(smem + (C::F8 ? C::OFF_VC : C::OFF_V));
  TcWalk walk(p);
  TreePiece pc;
  int t = 0, piece = 0;
  bool ok = true;

  auto issue_qk = [&](int tt, bool first) -> bool {
    const int stage = tt % C::SK, b = tt & 1;
    bool go = true;
    if (lane == 0) {
      go = (!first || tc_wait(br.q_ready, piece & 1, sh.abort, p.status)) &&
           (tt < 2 || tc_wait(&br.pv_done[b], ((tt - 2) >> 1) & 1, sh.abort, p.status)) &&
           tc_wait(&br.kfull[stage], (tt / C::SK) & 1, sh.abort, p.status);
      if (go) {
        tc::fence_after_sync();
        const uint32_t kb = kbase + stage * C::TILEB;
        if (C::F8) {
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8_ss(tmem + b * 128, tc::smem_desc(qbase + term * 16384 + kk * 32, 16, 1024, 2),
                        tc::smem_desc(kb + kk * 32, 16, 1024, 2), idesc128(0, 0), term + kk > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            tc::mma_bf16_ss(tmem + b * 128, tc::smem_desc(qbase + off, 16, 1024, 2),
                            tc::smem_desc(kb + off, 16, 1024, 2), idesc128(1, 0), kk > 0 ? 1u : 0u);
          }
        }
        tc::commit(&br.kempty[stage]);
        tc::commit(&br.s_ready[b]);
      }
    }
    return __shfl_sync(0xffffffffu, go ? 1 : 0, 0) != 0;
  };

  while (ok && walk.next(&pc)) {
    const int cnt = pc.t1 - pc.t0;
    ok = issue_qk(t, true);
    for (int u = 0; ok && u < cnt; ++u, ++t) {
      if (u + 1 < cnt) ok = issue_qk(t + 1, false);
      if (!ok) break;
      const int b = t & 1;
      bool go = true;
      if (lane == 0) {
        const int vs = C::F8 ? t % C::SC : t % C::SV;
        go = tc_wait(&br.p_ready[b], (t >> 1) & 1, sh.abort, p.status) &&
             tc_wait(C::F8 ? &br.vc_full[vs] : &br.vfull[vs], C::F8 ? (t / C::SC) & 1 : (t / C::SV) & 1, sh.abort,
                     p.status) &&
             (u > 0 || piece == 0 || tc_wait(br.o_free, (piece - 1) & 1, sh.abort, p.status));
        if (go) {
          tc::fence_after_sync();
#pragma unroll
          for (int kt = 0; kt < 8; ++kt) {
            // keys 0-63 into O_a (column 256), 64-127 into O_b (384); P's half at its S half
            const uint32_t a = tmem + b * 128 + (kt >> 2) * 64 + (kt & 3) * 8;
            mma_ts(tmem + 256 + (kt >> 2) * 128, a, tc::smem_desc(vbase + vs * 32768 + kt * 2048, 16384, 1024, 2),
                   idesc128(C::F8 ? 0 : 1, 1), ((kt & 3) > 0 || u > 0) ? 1u : 0u);
          }
          tc::commit(C::F8 ? &br.vc_empty[vs] : &br.vempty[vs]);
          tc::commit(&br.pv_done[b]);
        }
      }
      ok = __shfl_sync(0xffffffffu, go ? 1 : 0, 0) != 0;
    }
    ++piece;
  }
  // every MMA has completed before the tensor memory is given back
  if (lane == 0) {
    tc::commit(br.idle);
    tc_wait(br.idle, 0, sh.abort, p.status, false);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- converters (e4m3)
// 128 threads.  Thread i reads the scales of row i of a tile one tile ahead,
// and turns eight 16-byte pieces of V's codes into f16.  The two 16-bit words
// of four codes hold codes (0, 2) and (1, 3): V's columns 4w + {1, 2} change
// places, and O's with them.
template <class C>
__device__ __forceinline__ void tc_convert(const TreeTcParams& P, unsigned char* smem) {
  const TreeParams& p = P.t;
  const int i = threadIdx.x - C::CONV_WARP * 32;
  TcBars<C> br(smem);
  const TcShared sh = shared_of<C>(smem);
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE);
  TcWalk walk(p), ahead(p);
  TreePiece pc, apc;
  int at = 0;  // the next tile of apc whose scales are read
  bool amore = ahead.next(&apc);
  if (amore) at = apc.t0;
  int kb = 127, vb = 127;
  auto fetch = [&]() {
    kb = vb = 127;
    if (!amore) return;
    const int row = at * kRows + i;
    RowAt ra;
    if (row < apc.e.n && cache_row(p.cache, apc.b, row, &ra)) {
      kb = p.cache.ks[ra.sc + apc.g * p.cache.ss_head];
      vb = p.cache.vs[ra.sc + apc.g * p.cache.ss_head];
    }
    if (++at >= apc.t1) {
      amore = ahead.next(&apc);
      if (amore) at = apc.t0;
    }
  };
  auto put = [&](int tt) {
    float* s = scales + (tt % C::NS) * 384 + i;
    const float nan = __uint_as_float(0x7fffffffu);
    s[0] = kb == 255 ? nan : __uint_as_float(static_cast<uint32_t>(kb) << 23);
    s[128] = vb == 255 ? nan : static_cast<float>(vb - 127);
    // finite for a NaN row too: its exponent makes p NaN where it is seen, and 0 * NaN is not 0 where not
    s[256] = vb == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(max(254 - vb, 1)) << 23);
    mbar_arrive(&br.sc_full[tt % C::NS]);
  };
  bool more = amore;
  if (more) {
    fetch();
    put(0);
  }
  int t = 0;
  while (walk.next(&pc)) {
    for (int tile = pc.t0; tile < pc.t1; ++tile, ++t) {
      const bool next = amore;
      fetch();
      const int stage = t % C::SV, cs = t % C::SC;
      if (!tc_wait_warp(&br.vfull[stage], (t / C::SV) & 1, sh.abort, p.status)) return;
      if (t >= C::SC && !tc_wait_warp(&br.vc_empty[cs], ((t / C::SC) - 1) & 1, sh.abort, p.status)) return;
      const unsigned char* src = smem + C::OFF_V + stage * C::TILEB;
      unsigned char* dst = smem + C::OFF_VC + cs * 32768;
      const int c = i & 7, r0 = i >> 3;
      uint4 u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = *reinterpret_cast<const uint4*>(src + (r0 + 16 * k) * 128 + c * 16);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + 16 * k;
        const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = w[j] << 8;
          h[2 * j] = (x & 0x80008000u) | ((x >> 1) & 0x3f803f80u);
          h[2 * j + 1] = (w[j] & 0x80008000u) | ((w[j] >> 1) & 0x3f803f80u);
        }
        // lanes of the two column halves store their pieces in turn, so that the
        // eight lanes of a row write eight different banks
        const int ch = 2 * c;
        const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
        const int sw = c >> 2;
        *reinterpret_cast<uint4*>(dst + tile_off(r, ch + sw)) = sw ? hi : lo;
        *reinterpret_cast<uint4*>(dst + tile_off(r, ch + 1 - sw)) = sw ? lo : hi;
      }
      tc::fence_async_smem();
      mbar_arrive(&br.vc_full[cs]);
      // only now: given back right after the loads, the last of them was seen to
      // bring the next tile's codes
      mbar_arrive(&br.vempty[stage]);
      // the scales' buffer was last read by the softmax of tile t + 1 - NS, whose PV
      // is behind the one that vc_empty stood for
      if (next) put(t + 1);
    }
  }
}

// ---------------------------------------------------------------- softmax warps
// Bits x of the result: row kb + x (x < 64) is seen by node t.
__device__ __forceinline__ unsigned long long seen_bits(const TreeParams& p, const TreePiece& pc, int t, int kb,
                                                        uint32_t okbox, int box_rows) {
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
  if (okbox != 0xffffffffu) {
    const int r0 = kb & (kRows - 1);
    for (int x = 0; x < 64; x += 8)  // boxes hold 8 rows or more
      if (!((okbox >> ((r0 + x) / box_rows)) & 1u)) v &= ~(0xffull << x);
  }
  return v;
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
  const int nbox = kRows / P.t.box_rows;
  const uint32_t all_boxes = nbox == 32 ? 0xffffffffu : (1u << nbox) - 1u;
  unsigned char* qbuf = smem + C::OFF_Q;
  // where half x of this row finds the other half's (m, l) at the end of a
  // piece: in the part of the query row that x itself writes next
  auto ml_of = [&](int x) {
    return reinterpret_cast<float2*>(qbuf + (C::F8 ? i * 128 + (((x * 4) ^ (i & 7)) << 4) : tile_off(i, x * 8)));
  };
  TcWalk walk(p);
  TreePiece pc;
  int t = 0, piece = 0;
  while (walk.next(&pc)) {
    const int row = pc.mb * kRows + i;
    const int node = row / p.G, head = pc.g * p.G + row % p.G;
    const bool live = node < pc.e.cnt;
    const bool warp_live = (pc.mb * kRows + quarter * 32) / p.G < pc.e.cnt;
    const int first_draft = pc.e.n - pc.e.cnt;
    float rowf = p.scale_log2;
    if (warp_live) {
      const unsigned char* src = p.q + 2 * (pc.b * p.q_batch + node * p.q_token + head * p.q_head);
      if (!C::F8) {
#pragma unroll
        for (int c8 = 0; c8 < 8; ++c8) {
          const int ch = hf * 8 + c8;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live) v = *reinterpret_cast<const uint4*>(src + ch * 16);
          *reinterpret_cast<uint4*>(qbuf + tile_off(i, ch)) = v;
        }
      } else {
        uint32_t mx = 0;
        uint4 mine[8];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live) v = *reinterpret_cast<const uint4*>(src + (c ^ (hf * 8)) * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
          if (c < 8) mine[c] = v;
        }
        int ex = static_cast<int>(mx >> 7);  // biased exponent of the row's largest element
        const bool odd_q = ex == 255;        // a NaN or an infinity: the row's result is NaN
        if (ex == 0 || odd_q) ex = 127;
        // q * 2^-(ex - 134): the largest in [128, 256); in two factors, for the range of fp32
        const int e1 = (ex - 134) / 2, e2 = ex - 134 - e1;
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 - e1) << 23);
        const float f2 = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
        rowf = odd_q ? __uint_as_float(0x7fffffffu)
                     : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(ex) << 23) * 0.0078125f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 elements: one piece of each term
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = mine[2 * c + (k >> 1)];
            const uint32_t w0 = (k & 1) ? v.z : v.x, w1 = (k & 1) ? v.w : v.y;
            const float a[4] = {bf16lo(w0) * f1 * f2, bf16hi(w0) * f1 * f2, bf16lo(w1) * f1 * f2, bf16hi(w1) * f1 * f2};
            hi[k] = lo[k] = 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint16_t hc, lc;
              uint32_t hh;
              float x0, x1;
              asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hc) : "f"(a[2 * e + 1]), "f"(a[2 * e]));
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"(hc));
              asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                  : "=f"(x0), "=f"(x1)
                  : "r"(hh));
              asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lc) : "f"(a[2 * e + 1] - x1), "f"(a[2 * e] - x0));
              hi[k] |= static_cast<uint32_t>(hc) << (16 * e);
              lo[k] |= static_cast<uint32_t>(lc) << (16 * e);
            }
          }
          const int ch = hf * 4 + c;
          const uint32_t off = i * 128 + ((ch ^ (i & 7)) << 4);
          *reinterpret_cast<uint4*>(qbuf + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(qbuf + 16384 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      tc::fence_async_smem();
    }
    uint32_t* odd_rows = sh.odd + (piece & 1) * 8;  // last read two pieces ago
    if (!C::F8 && threadIdx.x < 8) odd_rows[threadIdx.x] = 0u;
    mbar_arrive(br.q_ready);

    float m_used = NEG, lsum = 0.f;
    for (int u = pc.t0; u < pc.t1; ++u, ++t) {
      const int b = t & 1;
      if (!tc_wait_warp(&br.s_ready[b], (t >> 1) & 1, sh.abort, p.status)) return;
      const int tile_row = u * kRows;
      const int kb = tile_row + hf * 64;
      uint32_t okbox = all_boxes;
      // written before the tile's copies were asked for; eight tiles on, this one's PV is done
      if (p.cache.bt) okbox = *reinterpret_cast<volatile uint32_t*>(&sh.ok[t % kOkRing]);
      const bool special = okbox != all_boxes || tile_row + kRows > first_draft;
      tc::fence_after_sync();
      if (warp_live) {
        uint32_t r[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld_32x32b_x16(tl + b * 128 + hf * 64 + c * 16, r[c]);
        tc_wait_ld<4>(r);
        const float* sc = nullptr;
        if (C::F8) {
          if (!tc_wait_warp(&br.sc_full[t % C::NS], (t / C::NS) & 1, sh.abort, p.status)) return;
          sc = reinterpret_cast<const float*>(smem + C::OFF_SCALE) + (t % C::NS) * 384 + hf * 64;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 kf = *reinterpret_cast<const float4*>(sc + c * 16 + j);
              const float4 ev = *reinterpret_cast<const float4*>(sc + 128 + c * 16 + j);
              r[c][j] = __float_as_uint(fmaf(__uint_as_float(r[c][j]) * rowf, kf.x, ev.x));
              r[c][j + 1] = __float_as_uint(fmaf(__uint_as_float(r[c][j + 1]) * rowf, kf.y, ev.y));
              r[c][j + 2] = __float_as_uint(fmaf(__uint_as_float(r[c][j + 2]) * rowf, kf.z, ev.z));
              r[c][j + 3] = __float_as_uint(fmaf(__uint_as_float(r[c][j + 3]) * rowf, kf.w, ev.w));
            }
        }
        if (special) {
          const unsigned long long vis =
              live ? seen_bits(p, pc, node, kb, okbox == all_boxes ? 0xffffffffu : okbox, P.t.box_rows) : 0ull;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!((vis >> (c * 16 + j)) & 1ull)) r[c][j] = __float_as_uint(NEG);
        }
        float mraw = NEG;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 16; ++j) mraw = fmaxf(mraw, __uint_as_float(r[c][j]));
        const float mx = C::F8 ? mraw : mraw * rowf;
        const bool grow = mx > m_used + 8.f;
        const bool rescale = grow && m_used != NEG;
        if (__any_sync(FULL, rescale)) {
          if (!tc_wait_warp(&br.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, sh.abort, p.status)) return;
          tc::fence_after_sync();
          const float f = rescale ? tc_ex2(m_used - mx) : 1.f;
#pragma unroll
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
        // f16's range is used from the top: p up to 2^(8 + 6)
        const float neg = (m_used == NEG ? 0.f : -m_used) + (C::F8 ? 6.f : 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x0 = __uint_as_float(r[2 * c + (e >> 3)][(2 * e) & 15]);
            const float x1 = __uint_as_float(r[2 * c + (e >> 3)][(2 * e + 1) & 15]);
            const float p0 = tc_ex2(C::F8 ? x0 + neg : fmaf(x0, rowf, neg));
            const float p1 = tc_ex2(C::F8 ? x1 + neg : fmaf(x1, rowf, neg));
            w[e] = tc_pack<C::F8>(p0, p1);
            if (C::F8) {
              const float2 iv = *reinterpret_cast<const float2*>(sc + 256 + c * 32 + 2 * e);
              lsum = fmaf(p0, iv.x, fmaf(p1, iv.y, lsum));
            } else {
              lsum += p0 + p1;
            }
          }
          tc_st_x16(tl + b * 128 + hf * 64 + c * 16, w);
        }
        tc_wait_st();
      }
      if (!C::F8 && special) {
        // V's rows that the tensor core must not meet as they are
        const int stage = t % C::SV;
        if (!tc_wait_warp(&br.vfull[stage], (t / C::SV) & 1, sh.abort, p.status)) return;
        unsigned char* v = smem + C::OFF_V + stage * C::TILEB;
        const int r = threadIdx.x >> 1, h = threadIdx.x & 1;  // a row's half
        const int krow = tile_row + r;
        if (krow >= pc.e.n || !((okbox >> (r / P.t.box_rows)) & 1u)) {
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(v + tile_off(r, h * 8 + c)) = make_uint4(0u, 0u, 0u, 0u);
        } else if (krow >= first_draft) {
          bool odd = false;
          for (int c = 0; c < 8; ++c) {
            uint4* at = reinterpret_cast<uint4*>(v + tile_off(r, h * 8 + c));
            const uint4 x = *at;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            bool here = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((w[k] & 0x7f80u) == 0x7f80u) {
                w[k] &= 0xffff0000u;
                here = true;
              }
              if ((w[k] & 0x7f800000u) == 0x7f800000u) {
                w[k] &= 0xffffu;
                here = true;
              }
            }
            if (here) *at = make_uint4(w[0], w[1], w[2], w[3]);
            odd |= here;
          }
          if (odd) atomicOr(&odd_rows[(krow - first_draft) >> 5], 1u << ((krow - first_draft) & 31));
        }
        tc::fence_async_smem();
      }
      tc::fence_before_sync();
      mbar_arrive(&br.p_ready[b]);
    }

    // the piece's state: both halves' outputs under one maximum
    const int last = t - 1;
    if (!tc_wait_warp(&br.pv_done[last & 1], (last >> 1) & 1, sh.abort, p.status)) return;
    tc::fence_after_sync();
    *ml_of(1 - hf) = make_float2(m_used, lsum);
    mbar_arrive(br.ml_ready);
    if (!tc_wait_warp(br.ml_ready, piece & 1, sh.abort, p.status)) return;
    if (warp_live) {
      const float2 own = make_float2(m_used, lsum), other = *ml_of(hf);
      const float2 sa = hf ? other : own, sb = hf ? own : other;
      const float M = fmaxf(sa.x, sb.x);
      const float fa = sa.x == NEG ? 1.f : tc_ex2(sa.x - M);  // 1: the state is zero, or NaN
      const float fb = sb.x == NEG ? 1.f : tc_ex2(sb.x - M);
      const float L = fmaf(sa.y, fa, sb.y * fb);
      const bool whole = pc.t0 == 0 && pc.t1 == pc.nt;
      const float unit = (C::F8 ? 256.f : 1.f) * (whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f);
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (pc.t0 == 0 ? 1 : 0);
      float* part = p.part_o + (slot * kRows + i) * kD + hf * 64;
      unsigned char* dst = p.out + 2 * (pc.b * p.o_batch + node * p.o_token + head * p.o_head + hf * 64);
      bool odd = false;
      if (!C::F8)
        for (int w = 0; w < 8; ++w) odd |= odd_rows[w] != 0u;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t ab[2][16];
        tc::ld_32x32b_x16(tl + 256 + hf * 64 + c * 16, ab[0]);
        tc::ld_32x32b_x16(tl + 384 + hf * 64 + c * 16, ab[1]);
        tc_wait_ld<2>(ab);
        float o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int col = C::F8 ? (j & ~3) | ((j & 1) << 1) | ((j >> 1) & 1) : j;  // the converter's order
          o[col] = fmaf(__uint_as_float(ab[0][j]), fa, __uint_as_float(ab[1][j]) * fb) * unit;
        }
        if (odd && live) {
          for (int x = 0; x < pc.e.cnt; ++x) {
            if (!((odd_rows[x >> 5] >> (x & 31)) & 1u) || !tree_sees(p, pc.b, node, x)) continue;
            RowAt at;
            if (!cache_row(p.cache, pc.b, first_draft + x, &at)) continue;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(p.cache.v) + at.kv + pc.g * p.cache.s_head + hf * 64 + c * 16;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if ((v[j] & 0x7f80u) == 0x7f80u) o[j] += __uint_as_float(static_cast<uint32_t>(v[j]) << 16);
          }
        }
        if (live) {
          if (whole) {
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              *reinterpret_cast<uint4*>(dst + 2 * (c * 16 + j)) =
                  make_uint4(tc_pack<false>(o[j], o[j + 1]), tc_pack<false>(o[j + 2], o[j + 3]),
                             tc_pack<false>(o[j + 4], o[j + 5]), tc_pack<false>(o[j + 6], o[j + 7]));
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              *reinterpret_cast<float4*>(part + c * 16 + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
      }
      if (!whole && live && hf == 0) p.part_ml[slot * kRows + i] = make_float2(M, L);
    }
    tc::fence_before_sync();
    mbar_arrive(br.o_free);
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
      mbar_init(&br.kfull[s], 1);
      mbar_init(&br.kempty[s], 1);
    }
    for (int s = 0; s < C::SV; ++s) {
      mbar_init(&br.vfull[s], 1);
      mbar_init(&br.vempty[s], C::F8 ? C::CONV : 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&br.s_ready[b], 1);
      mbar_init(&br.p_ready[b], kSoft);
      mbar_init(&br.pv_done[b], 1);
    }
    mbar_init(br.q_ready, kSoft);
    mbar_init(br.o_free, kSoft);
    mbar_init(br.ml_ready, kSoft);
    mbar_init(br.idle, 1);
    if (C::F8) {
      for (int s = 0; s < C::SC; ++s) {
        mbar_init(&br.vc_full[s], C::CONV);
        mbar_init(&br.vc_empty[s], 1);
      }
      for (int s = 0; s < C::NS; ++s) mbar_init(&br.sc_full[s], C::CONV);
    }
    *sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) {
    tc::tmem_alloc(sh.tmem, 512);
    tc::tmem_relinquish();
  }
  if (threadIdx.x == C::LOAD_WARP * 32) {
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
  } else if (warp == C::LOAD_WARP) {
    tc_loads<C>(P, smem);
  } else {
    tc_convert<C>(P, smem);
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

// 4-D map of K or V: (d, row, head, element), or paged (d, head, row, page).
bool encode(CUtensorMap* map, void* base, const CacheView& c, int heads, int batch, bool f8, bool swizzle,
            int box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int64_t es = f8 ? 1 : 2;
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
  cuuint32_t box[4] = {static_cast<cuuint32_t>(f8 ? 128 : 64), 1, 1, 1};
  box[paged ? 2 : 1] = static_cast<cuuint32_t>(box_rows);
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
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

bool tree_tc_maps(TreeTcParams* P, int cache_type) {
  const CacheView& c = P->t.cache;
  const bool f8 = cache_type == LYC_CACHE_E4M3;
  return encode(&P->tmk, c.k, c, P->t.Hkv, P->t.B, f8, true, P->t.box_rows) &&
         encode(&P->tmv, c.v, c, P->t.Hkv, P->t.B, f8, !f8, P->t.box_rows);
}

cudaError_t tree_tc_launch(const TreeTcParams* P, int cache_type, int device, cudaStream_t stream) {
  return cache_type == LYC_CACHE_E4M3 ? launch_tc<TcCfg<true>>(P, device, stream)
                                      : launch_tc<TcCfg<false>>(P, device, stream);
}

}  // namespace lyc
