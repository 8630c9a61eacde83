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

// Two fp32 operations an instruction (sm_100's packed forms).
__device__ __forceinline__ unsigned long long as_u64(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 as_f2(unsigned long long r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(r);
}

// 16 or 8 bytes of bf16 or fp32 as floats.
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
  static __device__ __forceinline__ void unpack(const uint2& u, float2* f) {
    f[0] = make_float2(bf16lo(u.x), bf16hi(u.x));
    f[1] = make_float2(bf16lo(u.y), bf16hi(u.y));
  }
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
  static __device__ __forceinline__ uint2 pack(const float2* f) {
    return make_uint2(pair(f[0].x, f[0].y), pair(f[1].x, f[1].y));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint2& u, float2* f) {
    f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ uint2 pack(const float2* f) {
    return make_uint2(__float_as_uint(f[0].x), __float_as_uint(f[0].y));
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
// One block per token.  LPH lanes hold a head's row, two 8-byte chunks each:
// the chunks of rotation partners (elements i and i + rot_dim/2, or adjacent
// ones) lie in one lane, so a row's only shuffles are those of its sum.  A
// lane has the same elements of every head, so its turns and weights stay in
// registers, and fp32 runs two operations an instruction: the first form (a
// lane with 16 adjacent bytes, partners by shuffle, turns from shared memory)
// was bound by instructions, 250 a row against about 60.  8192 tokens of 32/8
// heads of 128 bf16: 36.8 us, 4.6 TB/s, 0.70 of the copy rate, and still six
// issue slots of ten; written into an e4m3 cache, with the values, 43.7 us (0.64),
// into a bf16 cache 43 (0.71).  (Two
// rounds of heads in flight instead of one: 35.8 and 44.3.)
//
// The token's angles are taken once, in 64 bits: the turn pos * inv_freq /
// 2 pi less its nearest whole number, then sincospi of that in 32 bits
// (positions reach 2^20, where a 32-bit product is off by up to 2^-4 rad).
template <typename T, int D, bool APPEND, bool F8>
__global__ void __launch_bounds__(512) token_kernel(const __grid_constant__ TokenParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int CE = N / 2;   // elements of a chunk
  constexpr int C2 = CE / 2;  // pairs of a chunk
  constexpr int LPH = D / N;
  constexpr int ES = sizeof(T);
  __shared__ float2 turn[D / 2];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const int b = static_cast<int>(r / p.T), t = static_cast<int>(r - static_cast<int64_t>(b) * p.T);
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

  const int lane = threadIdx.x % LPH;  // within the head's row
  const int slot = threadIdx.x / LPH, slots = blockDim.x / LPH;
  // the lane's chunks: partners, and past the rotated elements neighbours
  const int hl = p.interleaved ? 0 : p.half / CE;
  const int ca = lane < hl ? lane : 2 * lane, cb = lane < hl ? lane + hl : 2 * lane + 1;
  const bool rot = p.interleaved ? lane * N < 2 * p.half : lane < hl;

  auto load = [&](const unsigned char* row, bool live, float2* x) {
    uint2 ua = make_uint2(0u, 0u), ub = ua;
    if (live) {
      ua = *reinterpret_cast<const uint2*>(row + ca * 8);
      ub = *reinterpret_cast<const uint2*>(row + cb * 8);
    }
    Vec<T>::unpack(ua, x);
    Vec<T>::unpack(ub, x + C2);
  };
  auto fetch = [&](const unsigned char* row, bool live, uint2* u) {
    u[0] = u[1] = make_uint2(0u, 0u);
    if (live) {
      u[0] = *reinterpret_cast<const uint2*>(row + ca * 8);
      u[1] = *reinterpret_cast<const uint2*>(row + cb * 8);
    }
  };
  const unsigned char* qrow = p.q + (b * p.q_batch + t * p.q_token) * ES;
  const unsigned char* krow = p.k + (b * p.k_batch + t * p.k_token) * ES;
  const unsigned char* vrow = p.v + (b * p.v_batch + t * p.v_token) * ES;
  // asked for before the angles: the block's first rows
  uint2 uq[2], uk[2], uv[2];
  fetch(qrow + slot * p.q_head * ES, slot < p.Hq, uq);
  fetch(krow + slot * p.k_head * ES, slot < p.Hk, uk);
  if (APPEND) fetch(vrow + slot * p.v_head * ES, slot < p.Hv, uv);

  for (int i = threadIdx.x; i < p.half; i += blockDim.x) {
    double x = static_cast<double>(pos) * static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;  // 1 / (2 pi)
    x -= rint(x);
    float s, c;
    sincospif(2.f * static_cast<float>(x), &s, &c);
    turn[i] = make_float2(c, s);
  }
  __syncthreads();
  // cosines and sines of the lane's pairs: [j] of elements 2j, 2j+1 of both
  // chunks (partners), or of each chunk's pairs in turn (adjacent)
  float2 cs[C2], sn[C2], ns[C2];
  if (rot && !p.interleaved) {
#pragma unroll
    for (int j = 0; j < C2; ++j) {
      const float2 u = turn[lane * CE + 2 * j], v = turn[lane * CE + 2 * j + 1];
      cs[j] = make_float2(u.x, v.x);
      sn[j] = make_float2(u.y, v.y);
      ns[j] = make_float2(-u.y, -v.y);
    }
  }

  // norm (w != NULL) and rotation of one row; whole warps
  auto turned = [&](float2* x, bool norm, const float2* w) {
    if (norm) {
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 2 * C2; ++j) a = fma2(x[j], x[j], a);
      float ss = a.x + a.y;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int j = 0; j < 2 * C2; ++j) x[j] = mul2(mul2(x[j], inv2), w[j]);
    }
    if (rot) {
      if (!p.interleaved) {
#pragma unroll
        for (int j = 0; j < C2; ++j) {
          const float2 u = x[j], v = x[j + C2];
          x[j] = fma2(v, ns[j], mul2(u, cs[j]));
          x[j + C2] = fma2(u, sn[j], mul2(v, cs[j]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2 * C2; ++j) {
          const float2 cv = turn[lane * (N / 2) + j];
          x[j] = make_float2(x[j].x * cv.x - x[j].y * cv.y, x[j].y * cv.x + x[j].x * cv.y);
        }
      }
    }
  };
  auto store = [&](unsigned char* row, const float2* x) {
    *reinterpret_cast<uint2*>(row + ca * 8) = Vec<T>::pack(x);
    *reinterpret_cast<uint2*>(row + cb * 8) = Vec<T>::pack(x + C2);
  };
  // one row into the cache
  auto keep = [&](unsigned char* rows, unsigned char* scales, int h, bool live, const float2* x) {
    if (!F8) {
      if (live) store(rows + (at.kv + h * p.cache.s_head) * ES, x);
      return;
    }
    uint32_t mx = 0;  // magnitudes as integers: a NaN is above every number
#pragma unroll
    for (int j = 0; j < 2 * C2; ++j)
      mx = max(mx, max(__float_as_uint(x[j].x) & 0x7fffffffu, __float_as_uint(x[j].y) & 0x7fffffffu));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (!live) return;
    const int e = scale_byte(mx);
    const float inv = __uint_as_float(static_cast<uint32_t>(max(254 - e, 0)) << 23);  // 2^-(e - 127)
    unsigned char* dst = rows + at.kv + h * p.cache.s_head;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float2* y = x + c * C2;
      uint32_t code = 0u;  // a row that is not finite gets zero codes
      if (e != 255) code = e4m3x2(y[0].x * inv, y[0].y * inv);
      if (C2 == 2 && e != 255) code |= e4m3x2(y[C2 - 1].x * inv, y[C2 - 1].y * inv) << 16;
      *reinterpret_cast<uint32_t*>(dst + (c ? cb : ca) * 4) = code;
    }
    if (lane == 0) scales[at.sc + h * p.cache.ss_head] = static_cast<unsigned char>(e);
  };

  const int qrounds = (p.Hq + slots - 1) / slots;
  if (qrounds > 0) {
    float2 w[2 * C2];
    const bool norm = p.q_weight != nullptr;
    load(p.q_weight, norm, w);
    unsigned char* out = p.q_out + (b * p.qo_batch + t * p.qo_token) * ES;
    for (int it = 0; it < qrounds; ++it) {
      const int h = it * slots + slot, next = h + slots;
      float2 x[2 * C2];
      Vec<T>::unpack(uq[0], x);
      Vec<T>::unpack(uq[1], x + C2);
      fetch(qrow + next * p.q_head * ES, next < p.Hq, uq);
      turned(x, norm, w);
      if (h < p.Hq) store(out + h * p.qo_head * ES, x);
    }
  }
  const int krounds = (p.Hk + slots - 1) / slots;
  if (krounds > 0) {
    float2 w[2 * C2];
    const bool norm = p.k_weight != nullptr;
    load(p.k_weight, norm, w);
    unsigned char* out = p.k_out + (b * p.ko_batch + t * p.ko_token) * ES;
    for (int it = 0; it < krounds; ++it) {
      const int h = it * slots + slot, next = h + slots;
      float2 x[2 * C2];
      Vec<T>::unpack(uk[0], x);
      Vec<T>::unpack(uk[1], x + C2);
      fetch(krow + next * p.k_head * ES, next < p.Hk, uk);
      turned(x, norm, w);
      if (APPEND)
        keep(p.cache.k, p.cache.ks, h, h < p.Hk && stored, x);
      else if (h < p.Hk)
        store(out + h * p.ko_head * ES, x);
    }
  }
  if (APPEND) {
    const int vrounds = (p.Hv + slots - 1) / slots;
    for (int it = 0; it < vrounds; ++it) {
      const int h = it * slots + slot, next = h + slots;
      float2 x[2 * C2];
      Vec<T>::unpack(uv[0], x);
      Vec<T>::unpack(uv[1], x + C2);
      fetch(vrow + next * p.v_head * ES, next < p.Hv, uv);
      keep(p.cache.v, p.cache.vs, h, h < p.Hv && stored, x);
    }
  }
}

// ---------------------------------------------------------------- read back
// Each thread takes 16 bytes of K and of V of one row; a block takes
// kReadThreads / LPR entries of one (element, head).  32768 rows of 8 heads of
// 128, e4m3 to bf16: 37.7 us, 5.4 TB/s, 0.82 of the copy rate; e4m3 to fp32 74 us
// (0.69); a bf16 cache to bf16 40.8 us (1.00).  (Two or four rows a thread, asked for
// together: 43.)
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

// Threads of a token's block.  Few tokens: enough for all its heads at once, the
// call is a chain of latencies (32/8 heads of 128 bf16, 128 tokens: 3.3 us, of 64
// threads 4.3).  Many: 64, so that the block's start (the position, the angles, the
// lanes' turns) is spent by two warps and the SM holds more tokens (1024 tokens:
// 5.6 us, of 512 threads 12.4; 8192: 36.5, of 128 38.2, of 256 51).
static int token_threads(const TokenParams* p, int head_dim, int dtype) {
  if (p->rows > 256) return 64;
  const int lanes = head_dim / (dtype == LYC_BF16 ? 8 : 4);
  const int want = (p->Hq > p->Hk ? p->Hq : p->Hk) * lanes;
  return want <= 128 ? 128 : want <= 256 ? 256 : 512;
}

cudaError_t token_launch(const TokenParams* p, int head_dim, int dtype, bool append, int cache_type,
                         cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p->rows);
  const int kTokenThreads = token_threads(p, head_dim, dtype);
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
