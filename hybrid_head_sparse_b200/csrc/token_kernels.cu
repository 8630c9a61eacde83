// token_kernels.cu -- what a decode step does with each new token before and
// after attention: the per-head norm and rotation of its queries and keys
// (lyc_qk_norm_rope), the same with the keys and values written into the
// cache in 8 bits or bf16 (lyc_cache_append), and rows of the cache read back
// (lyc_cache_read).
//
// All three move bytes: a few operations on each, so HBM bounds the large
// calls and launch latency the small ones.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lyc_device.cuh"
#include "serve_plan.h"

namespace lyc {

namespace {

// 16 bytes of bf16 or fp32 as floats.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(w[i]);
      f[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Two floats as e4m3 codes, the first in the low byte (to nearest, ties to even).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The scale byte of a row whose largest magnitude has these bits: the
// smallest e >= -100 with max <= 448 * 2^e = 1.75 * 2^(e+8); 255 for a NaN
// or an infinity in the row.
__device__ __forceinline__ int scale_byte(uint32_t max_bits) {
  if (max_bits >= 0x7f800000u) return 255;
  const int b = static_cast<int>(max_bits >> 23) - 8 + ((max_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(b, 27);
}

// ---------------------------------------------------------------- tokens
// One block per token; LPH lanes hold a head's row, 16 bytes each, so a row's
// sums are shuffles within the LPH lanes and a rotation's partner elements
// are either in the lane (adjacent pairs) or in the lane half/N away.  The
// token's half angles are taken once, in 64 bits: the turn pos * inv_freq /
// 2 pi less its nearest whole number, then sincospi of that in 32 bits
// (positions reach 2^20, where a 32-bit product is off by up to 2^-4 rad).
// Heads 0..Hq-1 of the block's list are the queries, then the keys, then the
// values.
constexpr int kTokenThreads = 256;

template <typename T, int D, bool APPEND, bool F8>
__global__ void __launch_bounds__(kTokenThreads) token_kernel(const __grid_constant__ TokenParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int LPH = D / N;
  constexpr int ES = sizeof(T);
  __shared__ float2 turn[D / 2];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const int b = static_cast<int>(r / p.T), t = static_cast<int>(r % p.T);
  int64_t pos = 0;
  RowAt at{0, 0};
  bool stored = true;
  if (APPEND) {
    const int n = p.n[b];
    const int cnt = p.t_len ? p.t_len[b] : p.T;
    if (cnt < 0 || cnt > p.T || n < cnt || n > p.cache.cap) {
      if (t == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, LYC_OP_BAD_LENGTH);
      return;
    }
    if (t >= cnt) return;
    const int row = n - cnt + t;
    pos = p.pos ? p.pos[r] : row;
    stored = cache_row(p.cache, b, row, &at);
    if (!stored && threadIdx.x == 0 && p.status) atomicOr(p.status, LYC_OP_BAD_PAGE);
  } else if (p.half > 0) {
    pos = p.pos[r];
    if (pos < 0) return;
  }
  for (int i = threadIdx.x; i < p.half; i += kTokenThreads) {
    double x = static_cast<double>(pos) * static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;  // 1 / (2 pi)
    x -= rint(x);
    float s, c;
    sincospif(2.f * static_cast<float>(x), &s, &c);
    turn[i] = make_float2(c, s);
  }
  __syncthreads();

  const int lane = threadIdx.x % LPH;  // within the head's row
  const int total = p.Hq + p.Hk + p.Hv;
  // every lane of a warp takes part in the shuffles: whole warps go around
  const int rounds = (total * LPH + kTokenThreads - 1) / kTokenThreads;
  for (int it = 0; it < rounds; ++it) {
    const int h = (it * kTokenThreads + static_cast<int>(threadIdx.x)) / LPH;
    const bool isq = h < p.Hq, isk = !isq && h < p.Hq + p.Hk;
    const bool live = h < total && (isq || !APPEND || stored);
    const int hh = isq ? h : isk ? h - p.Hq : h - p.Hq - p.Hk;
    float x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = 0.f;
    if (live) {
      const unsigned char* src = isq   ? p.q + (b * p.q_batch + t * p.q_token + hh * p.q_head) * ES
                                 : isk ? p.k + (b * p.k_batch + t * p.k_token + hh * p.k_head) * ES
                                       : p.v + (b * p.v_batch + t * p.v_token + hh * p.v_head) * ES;
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + lane * 16), x);
    }
    const unsigned char* w = isq ? p.q_weight : isk ? p.k_weight : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w) {
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      float g[N];
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(w + lane * 16), g);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = x[j] * inv * g[j];
    }
    if (p.half > 0) {
      if (p.interleaved) {
        if ((isq || isk) && lane * N < 2 * p.half) {
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            const float2 cs = turn[lane * (N / 2) + j / 2];
            const float a = x[j], c = x[j + 1];
            x[j] = a * cs.x - c * cs.y;
            x[j + 1] = c * cs.x + a * cs.y;
          }
        }
      } else {
        const int hl = p.half / N;  // lanes of the first elements of the pairs
        const bool lo = lane < hl, rot = (isq || isk) && lane < 2 * hl;
        const int base = static_cast<int>(threadIdx.x & 31) - lane;
        const int from = rot ? base + (lo ? lane + hl : lane - hl) : base + lane;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float other = __shfl_sync(0xffffffffu, x[j], from);
          if (rot) {
            const float2 cs = turn[(lo ? lane : lane - hl) * N + j];
            x[j] = lo ? x[j] * cs.x - other * cs.y : x[j] * cs.x + other * cs.y;
          }
        }
      }
    }
    uint32_t mx = 0;
    if (APPEND && F8) {  // magnitudes as integers: a NaN is above every number
#pragma unroll
      for (int j = 0; j < N; ++j) mx = max(mx, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (!live) continue;
    if (isq) {
      *reinterpret_cast<uint4*>(p.q_out + (b * p.qo_batch + t * p.qo_token + hh * p.qo_head) * ES + lane * 16) =
          Vec<T>::pack(x);
    } else if (!APPEND) {
      *reinterpret_cast<uint4*>(p.k_out + (b * p.ko_batch + t * p.ko_token + hh * p.ko_head) * ES + lane * 16) =
          Vec<T>::pack(x);
    } else if (!F8) {
      unsigned char* dst = (isk ? p.cache.k : p.cache.v) + (at.kv + hh * p.cache.s_head) * ES;
      *reinterpret_cast<uint4*>(dst + lane * 16) = Vec<T>::pack(x);
    } else {
      const int e = scale_byte(mx);
      // 2^-(e - 127); a row that is not finite gets zero codes
      const float inv = e == 255 ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      uint32_t c[N / 4];
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        c[j] = e4m3x2(x[4 * j] * inv, x[4 * j + 1] * inv) | (e4m3x2(x[4 * j + 2] * inv, x[4 * j + 3] * inv) << 16);
      if (e == 255)
#pragma unroll
        for (int j = 0; j < N / 4; ++j) c[j] = 0u;
      unsigned char* dst = (isk ? p.cache.k : p.cache.v) + at.kv + hh * p.cache.s_head + lane * N;
      if (N == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[N / 4 - 1]);
      else
        *reinterpret_cast<uint32_t*>(dst) = c[0];
      if (lane == 0) (isk ? p.cache.ks : p.cache.vs)[at.sc + hh * p.cache.ss_head] = static_cast<unsigned char>(e);
    }
  }
}

// ---------------------------------------------------------------- read back
// Each thread takes 16 bytes of K and of V of one row; a block takes
// kReadThreads / LPR entries of one (element, head).
constexpr int kReadThreads = 256;

__device__ __forceinline__ float e8m0(int byte) {
  if (byte == 255) return __uint_as_float(0x7fffffffu);
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(byte) << 23);
}

// four e4m3 codes as floats, exactly (finite codes)
__device__ __forceinline__ void e4m3_to_f32(uint32_t w, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    const uint16_t c = static_cast<uint16_t>(w >> (16 * i));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
        : "r"(h));
  }
}

template <typename T, bool F8>
__device__ __forceinline__ void read_store(const uint4& u, int scale, unsigned char* dst) {
  if (F8) {
    const float s = e8m0(scale);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3_to_f32(w[i], f + 4 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= s;
#pragma unroll
    for (int i = 0; i < 16 / Vec<T>::N; ++i)
      *reinterpret_cast<uint4*>(dst + 16 * i) = Vec<T>::pack(f + Vec<T>::N * i);
  } else {
    float f[8];
    Vec<__nv_bfloat16>::unpack(u, f);
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::N; ++i)
      *reinterpret_cast<uint4*>(dst + 16 * i) = Vec<T>::pack(f + Vec<T>::N * i);
  }
}

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int CES = F8 ? 1 : 2;          // bytes of a cached element
  constexpr int LPR = D * CES / 16;        // lanes of a row
  constexpr int RPB = kReadThreads / LPR;  // entries of a block
  pdl_wait();
  pdl_launch_dependents();
  const int chunks = (p.m + RPB - 1) / RPB;
  const int64_t x = blockIdx.x;
  const int bh = static_cast<int>(x / chunks);
  const int i = static_cast<int>(x % chunks) * RPB + static_cast<int>(threadIdx.x) / LPR;
  const int lane = threadIdx.x % LPR;
  const int b = bh / p.H, h = bh % p.H;
  if (i >= p.m) return;
  const int n = p.n[b];
  if (n < 0 || n > p.cache.cap) {
    if (p.status) atomicOr(p.status, LYC_OP_BAD_LENGTH);
    return;
  }
  int64_t row = p.first + i;
  if (p.sets) {
    row = p.sets[(static_cast<int64_t>(b) * p.H + h) * p.m + i];
    if (row < -1 || row >= n) {
      if (p.status) atomicOr(p.status, LYC_OP_BAD_INDEX);
      return;
    }
    if (row < 0) return;
  }
  if (row >= n) return;
  RowAt at;
  if (!cache_row(p.cache, b, static_cast<int>(row), &at)) {
    if (p.status) atomicOr(p.status, LYC_OP_BAD_PAGE);
    return;
  }
  const int g = h / p.hdiv;
  const int64_t off = (at.kv + g * p.cache.s_head) * CES + lane * 16;
  const uint4 ku = *reinterpret_cast<const uint4*>(p.cache.k + off);
  const uint4 vu = *reinterpret_cast<const uint4*>(p.cache.v + off);
  int ks = 0, vs = 0;
  if (F8) {
    ks = p.cache.ks[at.sc + g * p.cache.ss_head];
    vs = p.cache.vs[at.sc + g * p.cache.ss_head];
  }
  const int64_t o = (b * p.o_batch + h * p.o_head + i * p.o_row + lane * (16 / CES)) * static_cast<int>(sizeof(T));
  read_store<T, F8>(ku, ks, p.k_out + o);
  read_store<T, F8>(vu, vs, p.v_out + o);
}

template <typename K, typename P>
cudaError_t launch_pdl(K kernel, const P& p, unsigned grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t token_launch(const TokenParams* p, int head_dim, int dtype, bool append, int cache_type,
                         cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p->rows);
  const bool f8 = cache_type == LYC_CACHE_E4M3;
  if (append) {
    if (head_dim == 128)
      return f8 ? launch_pdl(token_kernel<__nv_bfloat16, 128, true, true>, *p, grid, kTokenThreads, stream)
                : launch_pdl(token_kernel<__nv_bfloat16, 128, true, false>, *p, grid, kTokenThreads, stream);
    return f8 ? launch_pdl(token_kernel<__nv_bfloat16, 64, true, true>, *p, grid, kTokenThreads, stream)
              : launch_pdl(token_kernel<__nv_bfloat16, 64, true, false>, *p, grid, kTokenThreads, stream);
  }
  if (dtype == LYC_BF16)
    return head_dim == 128
               ? launch_pdl(token_kernel<__nv_bfloat16, 128, false, false>, *p, grid, kTokenThreads, stream)
               : launch_pdl(token_kernel<__nv_bfloat16, 64, false, false>, *p, grid, kTokenThreads, stream);
  return head_dim == 128 ? launch_pdl(token_kernel<float, 128, false, false>, *p, grid, kTokenThreads, stream)
                         : launch_pdl(token_kernel<float, 64, false, false>, *p, grid, kTokenThreads, stream);
}

cudaError_t read_launch(const ReadParams* p, int head_dim, int dtype, int cache_type, cudaStream_t stream) {
  const bool f8 = cache_type == LYC_CACHE_E4M3;
  const int rpb = kReadThreads / (head_dim * (f8 ? 1 : 2) / 16);
  const int64_t chunks = (p->m + rpb - 1) / rpb;
  const int64_t grid = chunks * p->B * p->H;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(grid);
#define LYC_READ(TT, DD)                                                              \
  (f8 ? launch_pdl(read_kernel<TT, DD, true>, *p, g, kReadThreads, stream)            \
      : launch_pdl(read_kernel<TT, DD, false>, *p, g, kReadThreads, stream))
  if (dtype == LYC_BF16) return head_dim == 128 ? LYC_READ(__nv_bfloat16, 128) : LYC_READ(__nv_bfloat16, 64);
  return head_dim == 128 ? LYC_READ(float, 128) : LYC_READ(float, 64);
#undef LYC_READ
}

}  // namespace lyc
