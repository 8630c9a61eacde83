// serve_plan.h -- launch parameters of the serving operators (include/lyc.h,
// "Serving operators"): token_kernels.cu, tree_mma_kernel.cu; filled in by
// serve_api.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/lyc.h"

namespace lyc {

// One layer's cache as the kernels address it (lyc_layer_cache).  Strides in
// elements of K/V and in scale bytes.
struct CacheView {
  unsigned char* k;
  unsigned char* v;
  unsigned char* ks;
  unsigned char* vs;
  int64_t s_batch, s_head, s_token, s_page;
  int64_t ss_batch, ss_head, ss_token, ss_page;
  const int32_t* bt;
  int64_t num_pages;
  int32_t page_rows, max_blocks;
  int32_t cap;  // rows an element can hold
  // row / page_rows = row * page_mul >> page_shift, for rows below 2^30
  uint32_t page_mul, page_shift;
};

__device__ __forceinline__ int page_of(const CacheView& c, int row) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(row)) * c.page_mul) >> c.page_shift);
}

// Offsets of row i of element b's head 0 in K/V (elements) and in the scales;
// false where the block table names no page of the pool.
struct RowAt {
  int64_t kv, sc;
};
__device__ __forceinline__ bool cache_row(const CacheView& c, int b, int i, RowAt* at) {
  if (c.bt == nullptr) {
    at->kv = b * c.s_batch + i * c.s_token;
    at->sc = b * c.ss_batch + i * c.ss_token;
    return true;
  }
  const int blk = page_of(c, i), r = i - blk * c.page_rows;
  const int32_t page = c.bt[static_cast<int64_t>(b) * c.max_blocks + blk];
  if (page < 0 || page >= c.num_pages) return false;
  at->kv = page * c.s_page + r * c.s_token;
  at->sc = page * c.ss_page + r * c.ss_token;
  return true;
}

// Per-token heads (rope, append): blockIdx.x is a token.
struct TokenParams {
  const unsigned char* q;
  const unsigned char* k;
  const unsigned char* v;
  unsigned char* q_out;
  unsigned char* k_out;
  // element strides; a token's offset is (r / T) * batch + (r % T) * token
  int64_t q_batch, q_token, q_head, qo_batch, qo_token, qo_head;
  int64_t k_batch, k_token, k_head, ko_batch, ko_token, ko_head;
  int64_t v_batch, v_token, v_head;
  const int32_t* pos;
  const float* inv_freq;
  const unsigned char* q_weight;
  const unsigned char* k_weight;
  const int32_t* n;      // append only
  const int32_t* t_len;  // append only, or NULL
  uint32_t* status;
  int64_t rows;
  int32_t T, Hq, Hk, Hv;  // Hv: heads of v (append), 0 for rope
  int32_t half;           // rotated pairs (rot_dim / 2)
  int32_t interleaved;
  float eps;
  CacheView cache;        // append only
};

struct ReadParams {
  unsigned char* k_out;
  unsigned char* v_out;
  int64_t o_batch, o_head, o_row;
  const int32_t* n;
  const int32_t* sets;
  uint32_t* status;
  int64_t first;
  int32_t m, H, hdiv;  // output head h reads KV head h / hdiv
  int32_t B;
  CacheView cache;
};

// Over e4m3 rows a row's part of the softmax's sum is p' 2^-e, where p' = 2^(z + e - m')
// lies below 2^16 and e is its scale of V, -100 at least (kMinScaleV, the writer's
// smallest; a smaller one counts as that).  Held as 2^-16 of itself the sum of 2^27 such
// rows is finite; at e = 120 one row's is 2^-130, a number yet.
constexpr float kSumUnitE4m3 = 0x1p-16f;
constexpr uint32_t kMinScaleV = 27;  // 2^-100

struct TreeParams {
  const unsigned char* q;
  unsigned char* out;
  int64_t q_batch, q_token, q_head, o_batch, o_token, o_head;
  const int32_t* n;
  const int32_t* t_len;
  const unsigned long long* mask;
  uint32_t* status;
  float* part_o;    // [2 * grid][rows per block][d]
  float2* part_ml;  // [2 * grid][rows per block]: running maximum (log2 units) and sum
  int32_t B, T, W, Hq, Hkv, G;
  int32_t grid;
  int32_t box_rows;  // tcgen05 kernel, bf16: rows of one TMA box
  float scale_log2;
  float sum_unit;    // the sums are held in this: 1, or kSumUnitE4m3
  CacheView cache;
};

struct TreeTcParams {
  CUtensorMap tmk, tmv;
  TreeParams t;
};

// token_kernels.cu
cudaError_t token_launch(const TokenParams* p, int head_dim, int dtype, bool append, int cache_type,
                         cudaStream_t stream);
cudaError_t read_launch(const ReadParams* p, int head_dim, int dtype, int cache_type, cudaStream_t stream);
// tree_mma_kernel.cu
int tree_mma_tile_rows(int head_dim, int cache_type);
int tree_mma_block_rows(int rows);
cudaError_t tree_mma_launch(const TreeParams* p, int head_dim, int cache_type, int block_rows, int device,
                            cudaStream_t stream);
// tree_tc_kernel.cu: head_dim 128; 128 rows a tile, 128 query rows a block
int tree_tc_box_rows(const CacheView& c);
bool tree_tc_maps(TreeTcParams* P);
cudaError_t tree_tc_launch(const TreeTcParams* P, int cache_type, int device, cudaStream_t stream);
cudaError_t tree_combine_launch(const TreeParams* p, int head_dim, int block_rows, int tile_rows,
                                cudaStream_t stream);

}  // namespace lyc
