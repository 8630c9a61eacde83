// tree_mma_kernel.cu -- attention of a few query rows over the cache
// (lyc_tree_attention), bf16 or e4m3 rows, on mma.sync.
//
// For every element, KV head and block of up to 16 or 32 of its G * T query
// rows (row i = node i / G, head g * G + i % G):
//   z[i][j] = scale log2(e) q_i . k_j  (-inf where node i does not see row j)
//   o_i = sum_j 2^(z[i][j] - m_i) v_j / sum_j 2^(z[i][j] - m_i)
// in one pass with a running maximum m and sum per row.
//
// With few query rows a call reads every cached byte once and does 4 G T flop
// for each element of K: HBM bounds it, and what counts is bytes in flight.
// Eight warps a CTA, one CTA an SM; each warp takes its own 4 KiB of K and of
// V rows out of every tile through a ring of stages that only it uses, filled
// with 16-byte cp.async, so no warp waits for another until the end of the
// CTA's run of tiles, where the eight states are merged in shared memory.
// Device times, 32/8 heads of 128, one token: 131072 bf16 rows 85 us (0.97 of the
// floor at the copy rate), 4 x 8192 rows 30 (0.68), 4097 rows 9.6 with the merge
// (2.6 of bytes; the rest is the chain length, page, rows, states, merge).
//
// 8-bit rows: codes become f16, exactly, so both products run in f16 with fp32
// sums.  Which elements share a register is
// free in a sum over the head's dimensions, so K's codes are read 16 bytes at
// a time in an order that needs no shuffling and Q is laid out to match.  A
// query row is scaled by a power of two to below 2 before it becomes f16
// (exact for elements down to 2^-17 of the row's largest).  V's scales 2^e_j
// go into the exponent: p'_j = 2^(z_j + e_j - m'), m' the running maximum of
// z_j + e_j, so p' stays in f16's range whatever the scales are, and the sum
// takes p'_j 2^-e_j (kSumUnitE4m3).  One token over 131072 such rows: 63 us, 0.66 of
// the floor (8192 x 4: 24, 0.42; head_dim 64: 49, 0.42), bound by chains of
// instructions (the issue slots are busy for 0.4 of the time): codes converted by bit
// moves took 74, 16 rows at a time 66 (32 at a time cost a cache of 300 rows 1 us of
// 18), 12 warps of half the chunk no less.  32 query rows: 122 us, 0.34; the 255
// registers a thread do not hold the queries and the output, and some spill.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "lyc_device.cuh"
#include "serve_plan.h"
#include "tree_sched.cuh"

namespace lyc {

namespace {

template <int D_, bool F8_, int MT_>
struct TmCfg {
  static constexpr int D = D_;
  static constexpr bool F8 = F8_;
  static constexpr int MT = MT_;                // 16-row blocks of queries
  static constexpr int ROWS = 16 * MT;
  static constexpr int NW = 8;
  static constexpr int THREADS = NW * 32;
  static constexpr int ROWB = D * (F8 ? 1 : 2);
  static constexpr int KC = 4096 / ROWB;        // rows of a warp's chunk
  static constexpr int TR = NW * KC;            // rows of a tile
  static constexpr int SUB = F8 && MT == 1 ? 32 : 16;  // rows a warp takes at a time
  static constexpr int KT = SUB / 8;
  static constexpr int LPR = ROWB / 16;         // 16-byte pieces of a row
  static constexpr int RPI = 32 / LPR;          // rows of one warp-wide copy
  static constexpr int KPL = (KC + 31) / 32;    // rows a lane looks up
  static constexpr int ST = 3;                  // stages
  static constexpr int WARPB = ST * 8192;       // a warp's ring
  static constexpr int OFF_SC = NW * WARPB;     // per warp and stage: K factor, V exponent, factor of the sum
  static constexpr int SCB = F8 ? KC * 12 : 0;
  static constexpr int OFF_OK = OFF_SC + NW * ST * SCB;  // per warp and stage: rows that exist
  static constexpr int OFF_ML = OFF_OK + NW * ST * 8;    // per warp and row: (m, l)
  static constexpr int SMEM = OFF_ML + NW * ROWS * 8;
  static_assert(ROWS * D * 4 <= WARPB, "a warp's output fits its ring");
};

// byte offset of 16-byte piece ch of row r in a chunk
template <class C>
__device__ __forceinline__ int k_off(int r, int ch) {
  if (!C::F8) return (ch >> 3) * (C::KC * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  if (C::D == 128) return r * 128 + ((ch ^ ((r & 1) << 2)) << 4);
  return r * 64 + (ch << 4);
}
template <class C>
__device__ __forceinline__ int v_off(int r, int ch) {
  if (!C::F8) return (ch >> 3) * (C::KC * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  if (C::D == 128) return r * 128 + ((ch ^ (r & 7)) << 4);
  return (r >> 1) * 128 + ((((r & 1) << 2) + (ch ^ ((r >> 1) & 3))) << 4);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F8>
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (F8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool F8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (F8)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four e4m3 codes as f16, exactly: codes 0 and 1, codes 2 and 3.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t* h01, uint32_t* h23) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*h01), "=r"(*h23)
      : "r"(w));
}

__device__ __forceinline__ uint16_t bf16_bits(const unsigned char* p) { return *reinterpret_cast<const uint16_t*>(p); }

// The loads of one warp's chunks: where the rows lie is looked up one chunk
// ahead of its copies, their scale bytes are kept in registers for one chunk
// before they go to shared memory.  Where a chunk never spans two pages, it is
// looked up as a whole and its rows are a stride apart; else each row is.
template <class C>
struct TmLoader {
  const TreeParams& p;
  const TreePiece& pc;
  unsigned char* ring;
  float* scales;
  unsigned long long* okw;
  int warp, lane, nchunks;
  RowAt at[C::KPL];
  unsigned long long ok;  // rows of the looked-up chunk that exist
  int kb[C::KPL], vb[C::KPL];  // scale bytes waiting for shared memory
  int pending;                 // their stage, or -1
  const bool whole;            // a chunk is within one page

  __device__ __forceinline__ TmLoader(const TreeParams& prm, const TreePiece& piece, unsigned char* smem, int w, int l)
      : p(prm), pc(piece), ring(smem + w * C::WARPB),
        scales(reinterpret_cast<float*>(smem + C::OFF_SC + w * C::ST * C::SCB)),
        okw(reinterpret_cast<unsigned long long*>(smem + C::OFF_OK) + w * C::ST), warp(w), lane(l),
        nchunks(piece.t1 - piece.t0), pending(-1), whole(!prm.cache.bt || prm.cache.page_rows % C::KC == 0) {}

  __device__ __forceinline__ int first_row(int i) const { return (pc.t0 + i) * C::TR + warp * C::KC; }

  __device__ __forceinline__ void look_up(int i) {
    ok = 0;
    if (i >= nchunks) return;
    const int base = first_row(i);
    if (whole) {
      const int rows = min(C::KC, pc.e.n - base);
      if (rows <= 0) return;
      if (cache_row(p.cache, pc.b, base, &at[0]))
        ok = ~0ull >> (64 - rows);
      else if (lane == 0 && p.status)
        atomicOr(p.status, LYC_OP_BAD_PAGE);
      return;
    }
#pragma unroll
    for (int k = 0; k < C::KPL; ++k) {
      const int r = k * 32 + lane;
      const bool in = r < C::KC && base + r < pc.e.n;
      bool found = false;
      at[k] = RowAt{0, 0};
      if (in) {
        found = cache_row(p.cache, pc.b, base + r, &at[k]);
        if (!found) at[k] = RowAt{0, 0};
      }
      if (in && !found && p.status) atomicOr(p.status, LYC_OP_BAD_PAGE);
      const unsigned long long m = __ballot_sync(0xffffffffu, found);
      ok |= m << (32 * k);
    }
  }
  __device__ __forceinline__ void flush_scales() {
    if (!C::F8 || pending < 0) return;
    float* s = scales + pending * (C::KC * 3);
#pragma unroll
    for (int k = 0; k < C::KPL; ++k) {
      const int r = k * 32 + lane;
      if (r < C::KC) {
        const float nan = __uint_as_float(0x7fffffffu);
        s[r] = kb[k] == 255 ? nan : __uint_as_float(static_cast<uint32_t>(max(kb[k], 1)) << 23);
        const int v = max(vb[k], static_cast<int>(kMinScaleV));  // (at the load it would wait for that)
        s[C::KC + r] = v == 255 ? nan : static_cast<float>(v - 127);
        // finite for a NaN row too: its exponent makes p NaN where it is seen, and 0 * NaN is not 0 where not
        s[2 * C::KC + r] = v == 255 ? 1.f : tree_sum_factor(static_cast<uint32_t>(v));
      }
    }
    pending = -1;
  }
  // copies of chunk i (looked up before) into its stage
  __device__ __forceinline__ void issue(int i) {
    if (i < nchunks) {
      const int stage = i % C::ST;
      unsigned char* k = ring + stage * 8192;
      const int ch = lane % C::LPR;
      const unsigned char* kg = p.cache.k + pc.g * p.cache.s_head * (C::F8 ? 1 : 2) + ch * 16;
      const unsigned char* vg = p.cache.v + pc.g * p.cache.s_head * (C::F8 ? 1 : 2) + ch * 16;
      if (whole) {
        const int64_t step = p.cache.s_token * (C::F8 ? C::RPI : 2 * C::RPI);
        int64_t off = ok ? at[0].kv * (C::F8 ? 1 : 2) + (lane / C::LPR) * (step / C::RPI) : 0;
        const int rows = __popcll(ok) - lane / C::LPR;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int r = s * C::RPI + lane / C::LPR;
          const bool have = s * C::RPI < rows;
          const int64_t o = have ? off : 0;
          cp16(smem_u32(k + k_off<C>(r, ch)), kg + o, have ? 16 : 0);
          cp16(smem_u32(k + 4096 + v_off<C>(r, ch)), vg + o, have ? 16 : 0);
          off += step;
        }
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int r = s * C::RPI + lane / C::LPR;
          const int64_t kv = __shfl_sync(0xffffffffu, at[(s * C::RPI) / 32].kv, r & 31);
          const bool have = (ok >> r) & 1ull;
          const int64_t off = have ? kv * (C::F8 ? 1 : 2) : 0;
          cp16(smem_u32(k + k_off<C>(r, ch)), kg + off, have ? 16 : 0);
          cp16(smem_u32(k + 4096 + v_off<C>(r, ch)), vg + off, have ? 16 : 0);
        }
      }
      if (lane == 0) okw[stage] = ok;
      if (C::F8) {
#pragma unroll
        for (int j = 0; j < C::KPL; ++j) {
          const int r = j * 32 + lane;
          kb[j] = vb[j] = 127;
          if (r < C::KC && ((ok >> r) & 1ull)) {
            const int64_t sc = (whole ? at[0].sc + r * p.cache.ss_token : at[j].sc) + pc.g * p.cache.ss_head;
            kb[j] = p.cache.ks[sc];
            vb[j] = p.cache.vs[sc];
          }
        }
        pending = stage;
      }
    }
    cp_commit();
  }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tree_mma_kernel(const __grid_constant__ TreeParams p) {
  constexpr int D = C::D, MT = C::MT, KS = D / 16, NT = D / 8;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g4 = lane >> 2, j4 = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && p.status)
    for (int b = threadIdx.x; b < p.B; b += C::THREADS) {
      bool bad = false;
      tree_elem(p, b, &bad);
      if (bad) atomicOr(p.status, LYC_OP_BAD_LENGTH);
    }
  TreeSched<C::TR, C::ROWS> sched(p);
  const int cta = blockIdx.x;
  const float NEG = -INFINITY;
  const uint32_t xend = sched.begin(cta + 1);

  for (uint32_t x = sched.begin(cta); x < xend;) {
    const TreePiece pc = piece_at<C::TR, C::ROWS>(sched, x, xend);
    x += pc.t1 - pc.t0;
    const int first_draft = pc.e.n - pc.e.cnt;
    TmLoader<C> ld(p, pc, smem, warp, lane);
    ld.look_up(0);
#pragma unroll
    for (int i = 0; i < C::ST - 1; ++i) {
      ld.flush_scales();
      ld.issue(i);
      ld.look_up(i + 1);
    }

    // the queries: rows g4 and g4 + 8 of each 16-row block
    uint32_t qa[MT][KS][4];
    float rowf[MT][2];  // logits factor of the row (F8: with the row's power of two)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int i = pc.mb * C::ROWS + mt * 16 + hf * 8 + g4;
        const int t = i / p.G, h = pc.g * p.G + i % p.G;
        const bool live = t < pc.e.cnt;
        const unsigned char* src = p.q + 2 * (pc.b * p.q_batch + t * p.q_token + h * p.q_head);
        rowf[mt][hf] = p.scale_log2;
        if (!C::F8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              qa[mt][ks][hf + 2 * e] =
                  live ? *reinterpret_cast<const uint32_t*>(src + 2 * (ks * 16 + e * 8 + j4 * 2)) : 0u;
        } else {
          // dims 64 blk + 16 j4 + 4 s + {0, 1} and {2, 3} of step 4 blk + s
          uint32_t raw[D / 64][8];
          uint32_t mx = 0;
#pragma unroll
          for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint4 u = make_uint4(0u, 0u, 0u, 0u);
              if (live) u = *reinterpret_cast<const uint4*>(src + 2 * (blk * 64 + j4 * 16 + v * 8));
              raw[blk][4 * v] = u.x;
              raw[blk][4 * v + 1] = u.y;
              raw[blk][4 * v + 2] = u.z;
              raw[blk][4 * v + 3] = u.w;
            }
#pragma unroll
          for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mx = max(mx, max(raw[blk][k] & 0x7fffu, (raw[blk][k] >> 16) & 0x7fffu));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
          mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
          int ex = static_cast<int>(mx >> 7);  // biased exponent of the row's largest element
          if (ex == 0 || ex == 255) ex = 127;
          // the power of two comes off in two factors: 2^-(ex - 127) may be out of fp32's range
          const int e1 = (ex - 127) / 2, e2 = ex - 127 - e1;
          const float f1 = __uint_as_float(static_cast<uint32_t>(127 - e1) << 23);
          const float f2 = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
          rowf[mt][hf] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll
          for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint32_t w0 = raw[blk][2 * s], w1 = raw[blk][2 * s + 1];
              qa[mt][blk * 4 + s][hf] = pack16<true>(bf16lo(w0) * f1 * f2, bf16hi(w0) * f1 * f2);
              qa[mt][blk * 4 + s][hf + 2] = pack16<true>(bf16lo(w1) * f1 * f2, bf16hi(w1) * f1 * f2);
            }
        }
      }

    float o[MT][NT][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[mt][n][c] = 0.f;
      m[mt][0] = m[mt][1] = NEG;
      l[mt][0] = l[mt][1] = 0.f;
    }

    for (int i = 0; i < ld.nchunks; ++i) {
      ld.flush_scales();
      cp_wait<C::ST - 2>();
      __syncwarp();
      ld.issue(i + C::ST - 1);
      ld.look_up(i + C::ST);
      const int base = ld.first_row(i);
      if (base >= pc.e.n) continue;
      const int stage = i % C::ST;
      unsigned char* kbuf = ld.ring + stage * 8192;
      unsigned char* vbuf = kbuf + 4096;
      const unsigned long long ok = ld.okw[stage];
      const float* sc = ld.scales + stage * (C::KC * 3);

#pragma unroll 1
      for (int sub = 0; sub < C::KC / C::SUB; ++sub) {
        const int key0 = base + sub * C::SUB;
        if (key0 >= pc.e.n) break;
        float s[MT][C::KT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int t = 0; t < C::KT; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[mt][t][c] = 0.f;
        if (!C::F8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t kf[4];
            ldsm4(kf, smem_u32(kbuf + k_off<C>(sub * 16 + ((lane >> 4) << 3) + (lane & 7), ks * 2 + ((lane >> 3) & 1))));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16<false>(s[mt][0], qa[mt][ks], kf[0], kf[1]);
              mma16<false>(s[mt][1], qa[mt][ks], kf[2], kf[3]);
            }
          }
        } else {
#pragma unroll
          for (int t = 0; t < C::KT; ++t)
#pragma unroll
            for (int blk = 0; blk < D / 64; ++blk) {
              const uint4 u = *reinterpret_cast<const uint4*>(kbuf + k_off<C>(sub * C::SUB + t * 8 + g4, blk * 4 + j4));
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int st = 0; st < 4; ++st) {
                uint32_t b0, b1;
                codes_f16(w[st], &b0, &b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma16<true>(s[mt][t], qa[mt][blk * 4 + st], b0, b1);
              }
            }
        }
        // log2-unit logits, with V's exponent where rows are scaled
        float isv[C::KT][2];
#pragma unroll
        for (int t = 0; t < C::KT; ++t) {
          if (C::F8) {
            const int k = sub * C::SUB + t * 8 + 2 * j4;
            const float2 kf = *reinterpret_cast<const float2*>(sc + k);
            const float2 ev = *reinterpret_cast<const float2*>(sc + C::KC + k);
            const float2 iv = *reinterpret_cast<const float2*>(sc + 2 * C::KC + k);
            isv[t][0] = iv.x;
            isv[t][1] = iv.y;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                s[mt][t][c] = fmaf(s[mt][t][c] * rowf[mt][c >> 1], (c & 1) ? kf.y : kf.x, (c & 1) ? ev.y : ev.x);
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int c = 0; c < 4; ++c) s[mt][t][c] *= rowf[mt][c >> 1];
          }
        }
        constexpr uint32_t kAll = 0xffffffffu >> (32 - C::SUB);
        const uint32_t okh = static_cast<uint32_t>(ok >> (sub * C::SUB)) & kAll;
        const bool masked = okh != kAll || key0 + C::SUB > first_draft;
        if (masked) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int t = (pc.mb * C::ROWS + mt * 16 + (c >> 1) * 8 + g4) / p.G;
#pragma unroll
              for (int tl = 0; tl < C::KT; ++tl) {
                const int kk = tl * 8 + 2 * j4 + (c & 1);
                const int node = key0 + kk - first_draft;
                const bool sees = ((okh >> kk) & 1u) &&
                                  (node < 0 || (t < pc.e.cnt && node < pc.e.cnt && tree_sees(p, pc.b, t, node)));
                if (!sees) s[mt][tl][c] = NEG;
              }
            }
        }
        // the running maxima move only when some row's grows by more than 2^8
        bool grow = false;
        float mx[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            mx[mt][hf] = fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]);
#pragma unroll
            for (int t = 1; t < C::KT; ++t)
              mx[mt][hf] = fmaxf(mx[mt][hf], fmaxf(s[mt][t][2 * hf], s[mt][t][2 * hf + 1]));
            grow |= mx[mt][hf] > m[mt][hf] + 8.f;
          }
        if (__any_sync(FULL, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float r = mx[mt][hf];
              r = fmaxf(r, __shfl_xor_sync(FULL, r, 1));
              r = fmaxf(r, __shfl_xor_sync(FULL, r, 2));
              if (r > m[mt][hf] + 8.f) {
                const float f = m[mt][hf] == NEG ? 1.f : ex2(m[mt][hf] - r);  // 1: the state is zero, or NaN
                m[mt][hf] = r;
                l[mt][hf] *= f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  o[mt][n][2 * hf] *= f;
                  o[mt][n][2 * hf + 1] *= f;
                }
              }
            }
        }
        uint32_t pa[MT][C::SUB / 16][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            // f16's range is used from the top: p' up to 2^(8 + 6)
            const float neg = (m[mt][hf] == NEG ? 0.f : -m[mt][hf]) + (C::F8 ? 6.f : 0.f);
#pragma unroll
            for (int t = 0; t < C::KT; ++t) {
              const float p0 = ex2(s[mt][t][2 * hf] + neg), p1 = ex2(s[mt][t][2 * hf + 1] + neg);
              if (C::F8)
                l[mt][hf] = fmaf(p0, isv[t][0], fmaf(p1, isv[t][1], l[mt][hf]));
              else
                l[mt][hf] += p0 + p1;
              pa[mt][t >> 1][hf + 2 * (t & 1)] = pack16<C::F8>(p0, p1);
            }
          }
        if (!C::F8 && key0 + 16 > first_draft) {
          // drafted rows that some queries do not see: a NaN or an infinity in V
          // would reach every row through the product (0 * NaN), so it is added
          // to the rows that see it and taken out of the tile
          bool odd = false;
          for (int e = lane; e < 16 * (D / 8); e += 32) {
            const int r = e / (D / 8), ch = e % (D / 8);
            const uint4 u = *reinterpret_cast<const uint4*>(vbuf + v_off<C>(sub * 16 + r, ch));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              odd |= (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
          }
          if (__any_sync(FULL, odd)) {
            for (int kk = 0; kk < 16; ++kk) {
              const int node = key0 + kk - first_draft;
              if (!((okh >> kk) & 1u)) continue;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  const int t = (pc.mb * C::ROWS + mt * 16 + hf * 8 + g4) / p.G;
                  const bool sees = node < 0 || (t < pc.e.cnt && node < pc.e.cnt && tree_sees(p, pc.b, t, node));
                  if (!sees) continue;
#pragma unroll
                  for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                      const uint32_t v = bf16_bits(vbuf + v_off<C>(sub * 16 + kk, n) + (2 * j4 + c) * 2);
                      if ((v & 0x7f80u) == 0x7f80u) o[mt][n][2 * hf + c] += __uint_as_float(v << 16);
                    }
                }
            }
            __syncwarp();
            for (int e = lane; e < 16 * D; e += 32) {
              unsigned char* q = vbuf + v_off<C>(sub * 16 + e / D, (e % D) / 8) + (e % 8) * 2;
              if ((bf16_bits(q) & 0x7f80u) == 0x7f80u) *reinterpret_cast<uint16_t*>(q) = 0;
            }
            __syncwarp();
          }
        }
        if (C::F8 && key0 + C::SUB > first_draft) {
          // a drafted row that some queries do not see and nobody has written yet may
          // hold any byte: the NaN codes, which a written row never has, become zeros
          for (int e = lane; e < C::SUB * (D / 16); e += 32) {
            uint4* at = reinterpret_cast<uint4*>(vbuf + v_off<C>(sub * C::SUB + e / (D / 16), e % (D / 16)));
            const uint4 u = *at;
            uint32_t w[4] = {u.x, u.y, u.z, u.w}, any = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t nan = (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in such a byte
              any |= nan;
              w[k] &= ~(nan * 255u);
            }
            if (any) *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
        }
        if (!C::F8) {
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            uint32_t vf[4];
            ldsm4t(vf, smem_u32(vbuf + v_off<C>(sub * 16 + (lane & 15), dt * 2 + (lane >> 4))));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16<false>(o[mt][2 * dt], pa[mt][0], vf[0], vf[1]);
              mma16<false>(o[mt][2 * dt + 1], pa[mt][0], vf[2], vf[3]);
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < C::SUB / 16; ++ks)
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt) {
            uint32_t vf[4];
            ldsm4t(vf, smem_u32(vbuf + v_off<C>(sub * C::SUB + ks * 16 + (lane & 15), dt * 2 + (lane >> 4))));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // two keys' codes of an even and an odd dim lie alternately
              uint32_t e0, e1, o0, o1;
              codes_f16(__byte_perm(vf[2 * half], 0u, 0x3120), &e0, &o0);
              codes_f16(__byte_perm(vf[2 * half + 1], 0u, 0x3120), &e1, &o1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16<true>(o[mt][4 * dt + 2 * half], pa[mt][ks], e0, e1);
                mma16<true>(o[mt][4 * dt + 2 * half + 1], pa[mt][ks], o0, o1);
              }
            }
          }
        }
      }
      __syncwarp();
    }
    cp_wait<0>();

    // merge the eight warps' states of the rows that are queries; each warp's
    // output goes into its ring
    const int rows = min(C::ROWS, pc.e.cnt * p.G - pc.mb * C::ROWS);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    float* ow = reinterpret_cast<float*>(ld.ring);
    __syncwarp();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (mt * 16 + hf * 8 >= rows) continue;
        const int row = mt * 16 + hf * 8 + g4;
        float ls = l[mt][hf];
        ls += __shfl_xor_sync(FULL, ls, 1);
        ls += __shfl_xor_sync(FULL, ls, 2);
        if (j4 == 0) ml[warp * C::ROWS + row] = make_float2(m[mt][hf], ls);
        if (row >= rows) continue;
        if (!C::F8) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(ow + row * D + n * 8 + 2 * j4) =
                make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
        } else {
          // tiles 2c and 2c + 1 hold the even and odd dims
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            *reinterpret_cast<float4*>(ow + row * D + c * 16 + 4 * j4) =
                make_float4(o[mt][2 * c][2 * hf], o[mt][2 * c + 1][2 * hf], o[mt][2 * c][2 * hf + 1],
                            o[mt][2 * c + 1][2 * hf + 1]);
        }
      }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (D / 4); x += C::THREADS) {
      const int row = x / (D / 4), d0 = x % (D / 4) * 4;
      float M = NEG, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::NW; ++w) M = fmaxf(M, ml[w * C::ROWS + row].x);
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        const float2 s = ml[w * C::ROWS + row];
        const float f = s.x == NEG ? 1.f : ex2(s.x - M);  // 1: the state is zero, or NaN
        L = fmaf(s.y, f, L);
        const float4 u = *reinterpret_cast<const float4*>(smem + w * C::WARPB + (row * D + d0) * 4);
        acc.x = fmaf(u.x, f, acc.x);
        acc.y = fmaf(u.y, f, acc.y);
        acc.z = fmaf(u.z, f, acc.z);
        acc.w = fmaf(u.w, f, acc.w);
      }
      const int i = pc.mb * C::ROWS + row;
      const int t = i / p.G, h = pc.g * p.G + i % p.G;
      if (pc.t0 == 0 && pc.t1 == pc.nt) {
        const float inv = L == 0.f ? 0.f : p.sum_unit / L;
        *reinterpret_cast<uint2*>(p.out + 2 * (pc.b * p.o_batch + t * p.o_token + h * p.o_head + d0)) =
            make_uint2(pack16<false>(acc.x * inv, acc.y * inv), pack16<false>(acc.z * inv, acc.w * inv));
      } else {
        const int64_t slot = 2 * static_cast<int64_t>(cta) + (pc.t0 == 0 ? 1 : 0);
        *reinterpret_cast<float4*>(p.part_o + (slot * C::ROWS + row) * D + d0) = acc;
        if (d0 == 0) p.part_ml[slot * C::ROWS + row] = make_float2(M, L);
      }
    }
    __syncthreads();
  }
}

// A warp for a query row (4 y + warp of its block of rows) of each group that may have
// been cut: merges the states of the CTAs among which it was, in their order.
// Blocks x are the groups, or where those are more than the CTAs (of which each cuts
// one at most; a warp for each row of 1024 elements' groups took as long as the
// attention) the CTAs: the group in which the next CTA's run starts, unless an
// earlier run starts in it, too.  The lengths are inputs of
// the whole call, complete before the attention kernel lets this one start, so
// the division of work is computed while that one runs; then the rows of
// up to kParts parts and their (m, l) are asked for at once, and what is left
// is one trip to L2 (part after part it was 5.6 us of a 17 us call).
constexpr int kParts = 20;

// Groups of a launch, of every length; below 2^31 (the host refuses more).
__host__ __device__ inline uint32_t combine_groups(const TreeParams& p, int rows) {
  return static_cast<uint32_t>(p.B) * p.Hkv * ((p.G * p.T + rows - 1) / rows);
}

template <int D, int ROWS, int TR>
__global__ void __launch_bounds__(128) tree_combine_kernel(const __grid_constant__ TreeParams p) {
  const int lane = threadIdx.x & 31;
  TreeSched<TR, ROWS> sched(p);
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5);  // of the block of rows
  int b = 0, g = 0, mb = 0;
  uint32_t x0 = 0, nt = 0;  // the group's tiles
  TreeElem e{0, 0};
  if (combine_groups(p, ROWS) <= static_cast<uint32_t>(p.grid)) {
    const int mbs = (p.G * p.T + ROWS - 1) / ROWS, bg = static_cast<int>(blockIdx.x) / mbs;
    mb = static_cast<int>(blockIdx.x) - bg * mbs;
    b = bg / p.Hkv;
    g = bg - b * p.Hkv;
    while (b >= sched.b0 + 32) sched.window(sched.b0 + 32, __shfl_sync(0xffffffffu, sched.upto, 31));
    e = sched.elem(b);
    nt = static_cast<uint32_t>((e.n + TR - 1) / TR);
    x0 = __shfl_sync(0xffffffffu, sched.upto - sched.tiles, b - sched.b0) + static_cast<uint32_t>(g * sched.blocks(e) + mb) * nt;
  } else {
    const uint32_t cut = sched.begin(blockIdx.x + 1);
    if (cut < sched.total) {
      const TreePiece pc = piece_at<TR, ROWS>(sched, cut, cut + 1);
      x0 = cut - pc.t0;
      if (pc.t0 > 0 && sched.begin(blockIdx.x) <= x0) {
        b = pc.b;
        g = pc.g;
        mb = pc.mb;
        e = pc.e;
        nt = static_cast<uint32_t>(pc.nt);
      }
    }
  }
  const int i = mb * ROWS + row, t = i / p.G, h = g * p.G + i % p.G;
  int c0 = 0, c1 = 0;
  if (row < ROWS && t < e.cnt) {
    c0 = static_cast<int>(sched.owner(x0));
    c1 = static_cast<int>(sched.owner(x0 + nt - 1));
  }
  // the tcgen05 kernel's blocks of few rows: each CTA's part is in several copies
  const int copies = ROWS == 128 ? tree_copies(e.cnt * p.G - mb * ROWS) : 1;
  pdl_wait();
  pdl_launch_dependents();
  if (c0 == c1) return;  // nothing to do, or its CTA wrote the output
  constexpr int V = D / 32;
  typedef typename std::conditional<V == 4, float4, float2>::type Part;
  const int parts = (c1 - c0 + 1) * copies;
  // part k: copy k % copies of CTA c0 + k / copies; a group's first CTA has it in its second slot
  auto row_of = [&](int k) {
    const int c = c0 + k / copies;
    return (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * ROWS + (k % copies) * (ROWS / copies) + row;
  };
  const float NEG = -INFINITY;
  float M = NEG, L = 0.f, acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  for (int k0 = 0; k0 < parts; k0 += kParts) {
    Part u[kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (k0 + k < parts) u[k] = *reinterpret_cast<const Part*>(p.part_o + row_of(k0 + k) * D + lane * V);
    float2 ml = make_float2(NEG, 0.f);
    if (lane < kParts && k0 + lane < parts) ml = p.part_ml[row_of(k0 + lane)];
    float m = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float top = fmaxf(M, m);
    const float keep = M == NEG ? 1.f : ex2(M - top);  // 1: the state is zero, or NaN
    const float f = ml.x == NEG ? 1.f : ex2(ml.x - top);
    M = top;
    L = fmaf(L, keep, ml.y * f);  // lane j sums parts j, j + kParts, ...
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] *= keep;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      if (k0 + k < parts) {
        const float* v = reinterpret_cast<const float*>(&u[k]);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(v[c], fk, acc[c]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = L == 0.f ? 0.f : p.sum_unit / L;
  unsigned char* dst = p.out + 2 * (b * p.o_batch + t * p.o_token + h * p.o_head + lane * V);
#pragma unroll
  for (int k = 0; k < V; k += 2)
    reinterpret_cast<uint32_t*>(dst)[k / 2] = pack16<false>(acc[k] * inv, acc[k + 1] * inv);
}

template <class C>
cudaError_t launch_mma(const TreeParams* p, int device, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // per device; setting the attribute twice does no harm
  if (device >= 64 || !configured[device].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(tree_mma_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (device < 64) configured[device].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p->grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_mma_kernel<C>, *p);
}

template <int D, int ROWS, int TR>
cudaError_t launch_combine(const TreeParams* p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  const int rows = p->G * p->T < ROWS ? p->G * p->T : ROWS;
  const uint32_t groups = combine_groups(*p, ROWS), grid = static_cast<uint32_t>(p->grid);
  cfg.gridDim = dim3(groups < grid ? groups : grid, static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, ROWS, TR>, *p);
}

}  // namespace

int tree_mma_tile_rows(int head_dim, int cache_type) {
  return 8 * 4096 / (head_dim * (cache_type == LYC_CACHE_E4M3 ? 1 : 2));
}

int tree_mma_block_rows(int rows) { return rows <= 16 ? 16 : 32; }

cudaError_t tree_mma_launch(const TreeParams* p, int head_dim, int cache_type, int block_rows, int device,
                            cudaStream_t stream) {
  const bool f8 = cache_type == LYC_CACHE_E4M3;
#define LYC_TREE(DD, FF)                                                           \
  (block_rows == 16 ? launch_mma<TmCfg<DD, FF, 1>>(p, device, stream)              \
                    : launch_mma<TmCfg<DD, FF, 2>>(p, device, stream))
  if (head_dim == 128) return f8 ? LYC_TREE(128, true) : LYC_TREE(128, false);
  return f8 ? LYC_TREE(64, true) : LYC_TREE(64, false);
#undef LYC_TREE
}

cudaError_t tree_combine_launch(const TreeParams* p, int head_dim, int block_rows, int tile_rows,
                                cudaStream_t stream) {
  if (block_rows == 128) return launch_combine<128, 128, 128>(p, stream);  // tcgen05 kernel
#define LYC_COMBINE(DD, TT) \
  (block_rows == 16 ? launch_combine<DD, 16, TT>(p, stream) : launch_combine<DD, 32, TT>(p, stream))
  if (head_dim == 128) return tile_rows == 128 ? LYC_COMBINE(128, 128) : LYC_COMBINE(128, 256);
  return tile_rows == 256 ? LYC_COMBINE(64, 256) : LYC_COMBINE(64, 512);
#undef LYC_COMBINE
}

}  // namespace lyc
