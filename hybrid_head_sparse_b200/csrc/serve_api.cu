// serve_api.cu -- host side of the serving operators (include/lyc.h, "Serving
// operators"): argument checks and launches.  No state but the per-thread
// message and code of the last failure; nothing here allocates or throws.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <atomic>

#include "serve_plan.h"

using namespace lyc;

namespace {

thread_local char g_error[256];
thread_local lyc_status g_status = LYC_OK;

lyc_status refuse(lyc_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof g_error, fmt, ap);
  va_end(ap);
  return g_status = s;
}

lyc_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return LYC_OK;
  cudaGetLastError();
  return refuse(LYC_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The call's device, current for as long as the guard lives.
struct OnDevice {
  int before = -1;
  bool ok = false;
  explicit OnDevice(int device) {
    if (cudaGetDevice(&before) != cudaSuccess) return;
    ok = before == device || cudaSetDevice(device) == cudaSuccess;
    if (before == device) before = -1;
  }
  ~OnDevice() {
    if (ok && before >= 0) cudaSetDevice(before);
  }
};

// Words that the kernels read one at a time (lengths, positions, masks, the status).
bool off_word(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) != 0; }
bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

constexpr int64_t kMaxRows = 1ll << 30;
constexpr int kMaxHeads = 1 << 14;
constexpr int64_t kMaxBatch = 1 << 20;

// A tensor's strides: used ones (entries > 1) are whole 16 bytes, >= 0.
bool stride_bad(int64_t s, int64_t entries, int per16) {
  return entries > 1 && (s < 0 || s % per16 != 0 || s > (1ll << 48));
}

lyc_status check_cache(const lyc_layer_cache* c, bool writes) {
  if (!c) return refuse(LYC_ERR_INVALID_ARG, "NULL cache");
  if (c->type != LYC_CACHE_BF16 && c->type != LYC_CACHE_E4M3)
    return refuse(LYC_ERR_INVALID_ARG, "unknown cache type %d", c->type);
  if (c->head_dim != 64 && c->head_dim != 128)
    return refuse(LYC_ERR_UNSUPPORTED, "head_dim %d is not 64 or 128", c->head_dim);
  if (c->batch < 1 || c->batch > kMaxBatch || c->num_kv_heads < 1 || c->num_kv_heads > kMaxHeads)
    return refuse(LYC_ERR_INVALID_ARG, "batch %d or num_kv_heads %d out of range", c->batch, c->num_kv_heads);
  if (!c->k || !c->v || misaligned(c->k) || misaligned(c->v))
    return refuse(LYC_ERR_INVALID_ARG, "k and v must be 16-byte aligned device pointers");
  const bool f8 = c->type == LYC_CACHE_E4M3;
  if (f8 && (!c->k_scale || !c->v_scale)) return refuse(LYC_ERR_INVALID_ARG, "an e4m3 cache needs k_scale and v_scale");
  if (!f8 && (c->k_scale || c->v_scale)) return refuse(LYC_ERR_INVALID_ARG, "a bf16 cache has no scales");
  const int per16 = f8 ? 16 : 8;
  int64_t cap = c->rows;
  if (off_word(c->block_table, 4)) return refuse(LYC_ERR_INVALID_ARG, "block_table must be 4-byte aligned");
  if (c->block_table) {
    if (c->page_rows < 1 || c->max_blocks < 1 || c->num_pages < 1 || c->num_pages > 0x7fffffffll)
      return refuse(LYC_ERR_INVALID_ARG, "paged cache needs page_rows, max_blocks and num_pages >= 1");
    cap = static_cast<int64_t>(c->page_rows) * c->max_blocks;
    if (stride_bad(c->s_page, c->num_pages, per16) || stride_bad(c->s_token, c->page_rows, per16))
      return refuse(LYC_ERR_INVALID_ARG, "page and token strides must be whole 16 bytes");
  } else {
    if (c->rows < 1) return refuse(LYC_ERR_INVALID_ARG, "rows must be >= 1");
    if (stride_bad(c->s_batch, c->batch, per16) || stride_bad(c->s_token, c->rows, per16))
      return refuse(LYC_ERR_INVALID_ARG, "batch and token strides must be whole 16 bytes");
  }
  if (cap > kMaxRows) return refuse(LYC_ERR_INVALID_ARG, "capacity above 2^30 rows");
  if (stride_bad(c->s_head, c->num_kv_heads, per16))
    return refuse(LYC_ERR_INVALID_ARG, "the head stride must be whole 16 bytes");
  const int64_t per = c->block_table ? c->page_rows : c->rows;
  if ((per > 1 && c->s_token < c->head_dim) || (c->num_kv_heads > 1 && c->s_head < c->head_dim))
    return refuse(LYC_ERR_INVALID_ARG, "token and head strides must be at least head_dim");
  if (writes && c->block_table == nullptr && c->batch > 1 && c->s_batch < c->head_dim)
    return refuse(LYC_ERR_INVALID_ARG, "a cache that is written needs a batch stride of its own");
  if (writes && c->block_table && c->num_pages > 1 && c->s_page < c->head_dim)
    return refuse(LYC_ERR_INVALID_ARG, "a cache that is written needs a page stride of its own");
  if (f8 && (c->ss_batch < 0 || c->ss_head < 0 || c->ss_token < 0 || c->ss_page < 0))
    return refuse(LYC_ERR_INVALID_ARG, "negative scale stride");
  if (f8 && writes && ((per > 1 && c->ss_token < 1) || (c->num_kv_heads > 1 && c->ss_head < 1) ||
                       (c->block_table ? c->num_pages > 1 && c->ss_page < 1 : c->batch > 1 && c->ss_batch < 1)))
    return refuse(LYC_ERR_INVALID_ARG, "scales that are written need strides of their own");
  return LYC_OK;
}

CacheView view(const lyc_layer_cache* c) {
  CacheView w;
  w.k = static_cast<unsigned char*>(c->k);
  w.v = static_cast<unsigned char*>(c->v);
  w.ks = c->k_scale;
  w.vs = c->v_scale;
  w.s_batch = c->s_batch;
  w.s_head = c->s_head;
  w.s_token = c->s_token;
  w.s_page = c->s_page;
  w.ss_batch = c->ss_batch;
  w.ss_head = c->ss_head;
  w.ss_token = c->ss_token;
  w.ss_page = c->ss_page;
  w.bt = c->block_table;
  w.num_pages = c->num_pages;
  w.page_rows = c->page_rows;
  w.max_blocks = c->max_blocks;
  // with s = ceil(log2 d) and m = ceil(2^(30+s) / d), m d = 2^(30+s) + r, r < d <= 2^s:
  // n m / 2^(30+s) exceeds n / d by n r / (d 2^(30+s)) < 1 / d, so its floor is right
  w.page_mul = w.page_shift = 0;
  if (c->block_table) {
    uint32_t s = 0;
    while ((1u << s) < static_cast<uint32_t>(c->page_rows)) ++s;
    w.page_shift = 30 + s;
    w.page_mul = static_cast<uint32_t>(((1ull << w.page_shift) + c->page_rows - 1) / c->page_rows);
  }
  w.cap = static_cast<int32_t>(c->block_table ? static_cast<int64_t>(c->page_rows) * c->max_blocks : c->rows);
  return w;
}

lyc_status check_rotation(int rot_dim, int head_dim, const float* inv_freq, float eps) {
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0)
    return refuse(LYC_ERR_INVALID_ARG, "rot_dim %d must be a multiple of 16 up to head_dim", rot_dim);
  if (rot_dim > 0 && !inv_freq) return refuse(LYC_ERR_INVALID_ARG, "a rotation needs inv_freq");
  if (!(eps >= 0.f) || isinf(eps)) return refuse(LYC_ERR_INVALID_ARG, "eps must be a finite number >= 0");
  return LYC_OK;
}

int sm_count(int device) {
  static std::atomic<int> known[64];
  if (device >= 0 && device < 64 && known[device] > 0) return known[device];
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms < 1) return 0;
  if (device >= 0 && device < 64) known[device] = sms;
  return sms;
}

// The most query rows of a KV head that the mma.sync kernel takes where the tcgen05
// kernel could.  Times in us, 32/8 heads of 128, over 131072 rows, 4 x 8192, 2048, 16 x
// 1024 and 32 x 300:
//   bf16, 16 rows   mma.sync  86   32  10   23  24
//   bf16, 32 rows   mma.sync  99   43  14   35  42   tcgen05  90  33  14  29  33
//   e4m3, 32 rows   mma.sync 122   44  15   32  36   tcgen05 106  48  20  41  49
//   e4m3, 36 rows   mma.sync 214   62  16   51  57   tcgen05 111  50  21  43  50
// (mma.sync has blocks of 16 or 32 rows, so more read the cache again; the capacity
// that the host knows says little of the lengths.)
constexpr int mma_most_rows(int cache_type) { return cache_type == LYC_CACHE_BF16 ? 16 : 32; }

struct TreeShape {
  bool tc;  // the tcgen05 kernel
  int block_rows, tile_rows, mblocks, grid;
  int64_t cap_tiles;  // tiles of a group at the cache's capacity
  uint64_t bytes;
};

// The division of the work counts tiles (and rows of query blocks) in 32 bits.
bool tree_too_large(const lyc_layer_cache* c, int T, int Hq) {
  const int64_t tiles = (static_cast<int64_t>(view(c).cap) + 127) / 128;
  const int64_t groups = static_cast<int64_t>(c->batch) * c->num_kv_heads;
  const int64_t rows = static_cast<int64_t>(Hq / c->num_kv_heads) * T;
  return static_cast<double>(tiles) * groups * ((rows + 15) / 16) >= 2147483648.0 ||
         static_cast<double>(groups) * rows >= 2147483648.0;
}

bool tree_shape(const lyc_layer_cache* c, int T, int Hq, bool may_tc, TreeShape* s) {
  const int sms = sm_count(c->device);
  if (sms < 1) return false;
  const int rows = Hq / c->num_kv_heads * T;
  s->tc = may_tc && c->head_dim == 128 && rows > mma_most_rows(c->type) &&
          (c->type == LYC_CACHE_E4M3 || tree_tc_box_rows(view(c)) > 0);
  s->block_rows = s->tc ? 128 : tree_mma_block_rows(rows);
  s->tile_rows = s->tc ? 128 : tree_mma_tile_rows(c->head_dim, c->type);
  s->mblocks = (rows + s->block_rows - 1) / s->block_rows;
  const int64_t cap = view(c).cap;
  s->cap_tiles = (cap + s->tile_rows - 1) / s->tile_rows;
  // one CTA an SM; never more than there can be tiles
  const int64_t most = s->cap_tiles * c->batch * c->num_kv_heads * s->mblocks;
  s->grid = static_cast<int>(most < sms ? most : sms);
  const uint64_t per = static_cast<uint64_t>(s->block_rows) * (c->head_dim + 2) * 4;
  s->bytes = s->cap_tiles > 1 ? 2ull * s->grid * per : 16;
  return true;
}

lyc_status check_tree(const lyc_layer_cache* c, int T, int Hq) {
  const lyc_status st = check_cache(c, false);
  if (st != LYC_OK) return st;
  if (T < 1 || T > 256) return refuse(LYC_ERR_UNSUPPORTED, "T %d is not in [1, 256]", T);
  if (Hq < c->num_kv_heads || Hq > kMaxHeads || Hq % c->num_kv_heads != 0)
    return refuse(LYC_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d", Hq, c->num_kv_heads);
  if (tree_too_large(c, T, Hq)) return refuse(LYC_ERR_UNSUPPORTED, "capacity * batch * heads * T is too large");
  return LYC_OK;
}

}  // namespace

extern "C" {

const char* lyc_operator_error(void) { return g_error; }
lyc_status lyc_operator_status(void) { return g_status; }

lyc_status lyc_qk_norm_rope(const lyc_rope_args* a, void* stream) {
  if (!a) return refuse(LYC_ERR_INVALID_ARG, "NULL arguments");
  if (a->dtype != LYC_BF16 && a->dtype != LYC_FP32) return refuse(LYC_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->head_dim != 64 && a->head_dim != 128)
    return refuse(LYC_ERR_UNSUPPORTED, "head_dim %d is not 64 or 128", a->head_dim);
  if (a->rows < 0 || a->rows > kMaxRows) return refuse(LYC_ERR_INVALID_ARG, "rows out of range");
  if (a->rows == 0) return LYC_OK;  // empty tensors have no address
  if (!a->q && !a->k) return refuse(LYC_ERR_INVALID_ARG, "neither q nor k");
  const int per16 = a->dtype == LYC_BF16 ? 8 : 4;
  const lyc_status st = check_rotation(a->rot_dim, a->head_dim, a->inv_freq, a->eps);
  if (st != LYC_OK) return st;
  if (a->rot_dim > 0 && !a->pos) return refuse(LYC_ERR_INVALID_ARG, "a rotation needs pos");
  if (a->rot_dim > 0 && (off_word(a->pos, 4) || off_word(a->inv_freq, 4)))
    return refuse(LYC_ERR_INVALID_ARG, "pos and inv_freq must be 4-byte aligned");
  if (a->q) {
    if (!a->q_out || misaligned(a->q) || misaligned(a->q_out) || misaligned(a->q_weight))
      return refuse(LYC_ERR_INVALID_ARG, "q, q_out and q_weight must be 16-byte aligned");
    if (a->num_q_heads < 1 || a->num_q_heads > kMaxHeads) return refuse(LYC_ERR_INVALID_ARG, "num_q_heads out of range");
    if (stride_bad(a->q_row, a->rows, per16) || stride_bad(a->q_head, a->num_q_heads, per16) ||
        stride_bad(a->qo_row, a->rows, per16) || stride_bad(a->qo_head, a->num_q_heads, per16))
      return refuse(LYC_ERR_INVALID_ARG, "strides of q and q_out must be whole 16 bytes");
    if ((a->rows > 1 && a->qo_row < a->head_dim) || (a->num_q_heads > 1 && a->qo_head < a->head_dim))
      return refuse(LYC_ERR_INVALID_ARG, "rows of q_out overlap");
  }
  if (a->k) {
    if (!a->k_out || misaligned(a->k) || misaligned(a->k_out) || misaligned(a->k_weight))
      return refuse(LYC_ERR_INVALID_ARG, "k, k_out and k_weight must be 16-byte aligned");
    if (a->num_kv_heads < 1 || a->num_kv_heads > kMaxHeads)
      return refuse(LYC_ERR_INVALID_ARG, "num_kv_heads out of range");
    if (stride_bad(a->k_row, a->rows, per16) || stride_bad(a->k_head, a->num_kv_heads, per16) ||
        stride_bad(a->ko_row, a->rows, per16) || stride_bad(a->ko_head, a->num_kv_heads, per16))
      return refuse(LYC_ERR_INVALID_ARG, "strides of k and k_out must be whole 16 bytes");
    if ((a->rows > 1 && a->ko_row < a->head_dim) || (a->num_kv_heads > 1 && a->ko_head < a->head_dim))
      return refuse(LYC_ERR_INVALID_ARG, "rows of k_out overlap");
  }
  OnDevice on(a->device);
  if (!on.ok) return refuse(LYC_ERR_CUDA, "device %d cannot be used", a->device);
  TokenParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const unsigned char*>(a->q);
  p.k = static_cast<const unsigned char*>(a->k);
  p.q_out = static_cast<unsigned char*>(a->q_out);
  p.k_out = static_cast<unsigned char*>(a->k_out);
  p.q_batch = a->q_row;
  p.q_head = a->q_head;
  p.qo_batch = a->qo_row;
  p.qo_head = a->qo_head;
  p.k_batch = a->k_row;
  p.k_head = a->k_head;
  p.ko_batch = a->ko_row;
  p.ko_head = a->ko_head;
  p.pos = a->pos;
  p.inv_freq = a->inv_freq;
  p.q_weight = static_cast<const unsigned char*>(a->q_weight);
  p.k_weight = static_cast<const unsigned char*>(a->k_weight);
  p.rows = a->rows;
  p.T = 1;
  p.Hq = a->q ? a->num_q_heads : 0;
  p.Hk = a->k ? a->num_kv_heads : 0;
  p.half = a->rot_dim / 2;
  p.interleaved = a->interleaved != 0;
  p.eps = a->eps;
  return launched(token_launch(&p, a->head_dim, a->dtype, false, LYC_CACHE_BF16, static_cast<cudaStream_t>(stream)),
                  "norm and rotation launch");
}

lyc_status lyc_cache_append(const lyc_layer_cache* c, const lyc_append_args* a, void* stream) {
  lyc_status st = check_cache(c, true);
  if (st != LYC_OK) return st;
  if (!a || !a->k || !a->v || !a->n) return refuse(LYC_ERR_INVALID_ARG, "NULL k, v or n");
  if (a->T < 1 || a->T > kMaxRows || static_cast<int64_t>(a->T) * c->batch > 0x7fffffffll)
    return refuse(LYC_ERR_INVALID_ARG, "T out of range");
  st = check_rotation(a->rot_dim, c->head_dim, a->inv_freq, a->eps);
  if (st != LYC_OK) return st;
  if (misaligned(a->k) || misaligned(a->v) || misaligned(a->k_weight))
    return refuse(LYC_ERR_INVALID_ARG, "k, v and k_weight must be 16-byte aligned");
  if (off_word(a->n, 4) || off_word(a->t_len, 4) || off_word(a->pos, 4) || off_word(a->inv_freq, 4) || off_word(a->status, 4))
    return refuse(LYC_ERR_INVALID_ARG, "n, t_len, pos, inv_freq and status must be 4-byte aligned");
  if (stride_bad(a->k_batch, c->batch, 8) || stride_bad(a->k_token, a->T, 8) ||
      stride_bad(a->k_head, c->num_kv_heads, 8) || stride_bad(a->v_batch, c->batch, 8) ||
      stride_bad(a->v_token, a->T, 8) || stride_bad(a->v_head, c->num_kv_heads, 8))
    return refuse(LYC_ERR_INVALID_ARG, "strides of k and v must be whole 16 bytes");
  if (a->q) {
    if (!a->q_out || misaligned(a->q) || misaligned(a->q_out) || misaligned(a->q_weight))
      return refuse(LYC_ERR_INVALID_ARG, "q, q_out and q_weight must be 16-byte aligned");
    if (a->num_q_heads < 1 || a->num_q_heads > kMaxHeads) return refuse(LYC_ERR_INVALID_ARG, "num_q_heads out of range");
    if (stride_bad(a->q_batch, c->batch, 8) || stride_bad(a->q_token, a->T, 8) || stride_bad(a->q_head, a->num_q_heads, 8) ||
        stride_bad(a->qo_batch, c->batch, 8) || stride_bad(a->qo_token, a->T, 8) ||
        stride_bad(a->qo_head, a->num_q_heads, 8))
      return refuse(LYC_ERR_INVALID_ARG, "strides of q and q_out must be whole 16 bytes");
    if ((c->batch > 1 && a->qo_batch < c->head_dim) || (a->T > 1 && a->qo_token < c->head_dim) ||
        (a->num_q_heads > 1 && a->qo_head < c->head_dim))
      return refuse(LYC_ERR_INVALID_ARG, "rows of q_out overlap");
  } else if (a->q_out || a->q_weight) {
    return refuse(LYC_ERR_INVALID_ARG, "q_out or q_weight without q");
  }
  OnDevice on(c->device);
  if (!on.ok) return refuse(LYC_ERR_CUDA, "device %d cannot be used", c->device);
  TokenParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const unsigned char*>(a->q);
  p.k = static_cast<const unsigned char*>(a->k);
  p.v = static_cast<const unsigned char*>(a->v);
  p.q_out = static_cast<unsigned char*>(a->q_out);
  p.q_batch = a->q_batch;
  p.q_token = a->q_token;
  p.q_head = a->q_head;
  p.qo_batch = a->qo_batch;
  p.qo_token = a->qo_token;
  p.qo_head = a->qo_head;
  p.k_batch = a->k_batch;
  p.k_token = a->k_token;
  p.k_head = a->k_head;
  p.v_batch = a->v_batch;
  p.v_token = a->v_token;
  p.v_head = a->v_head;
  p.pos = a->pos;
  p.inv_freq = a->inv_freq;
  p.q_weight = static_cast<const unsigned char*>(a->q_weight);
  p.k_weight = static_cast<const unsigned char*>(a->k_weight);
  p.n = a->n;
  p.t_len = a->t_len;
  p.status = a->status;
  p.rows = static_cast<int64_t>(c->batch) * a->T;
  p.T = a->T;
  p.Hq = a->q ? a->num_q_heads : 0;
  p.Hk = p.Hv = c->num_kv_heads;
  p.half = a->rot_dim / 2;
  p.interleaved = a->interleaved != 0;
  p.eps = a->eps;
  p.cache = view(c);
  return launched(token_launch(&p, c->head_dim, LYC_BF16, true, c->type, static_cast<cudaStream_t>(stream)),
                  "append launch");
}

lyc_status lyc_cache_read(const lyc_layer_cache* c, const lyc_read_args* a, void* stream) {
  const lyc_status st = check_cache(c, false);
  if (st != LYC_OK) return st;
  if (a && a->m == 0) return LYC_OK;  // empty tensors have no address
  if (!a || !a->k_out || !a->v_out || !a->n) return refuse(LYC_ERR_INVALID_ARG, "NULL k_out, v_out or n");
  if (a->dtype != LYC_BF16 && a->dtype != LYC_FP32) return refuse(LYC_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->m < 0 || a->m > kMaxRows || a->first < 0 || a->first > kMaxRows)
    return refuse(LYC_ERR_INVALID_ARG, "m or first out of range");
  if (a->num_heads < 1 || a->num_heads > kMaxHeads || a->num_heads % c->num_kv_heads != 0 ||
      (!a->sets && a->num_heads != c->num_kv_heads))
    return refuse(LYC_ERR_INVALID_ARG, "num_heads %d does not fit num_kv_heads %d", a->num_heads, c->num_kv_heads);
  if (off_word(a->n, 4) || off_word(a->sets, 4) || off_word(a->status, 4))
    return refuse(LYC_ERR_INVALID_ARG, "n, sets and status must be 4-byte aligned");
  if (a->sets && a->first != 0) return refuse(LYC_ERR_INVALID_ARG, "sets and first do not go together");
  const int per16 = a->dtype == LYC_BF16 ? 8 : 4;
  if (misaligned(a->k_out) || misaligned(a->v_out) || stride_bad(a->o_batch, c->batch, per16) ||
      stride_bad(a->o_head, a->num_heads, per16) || stride_bad(a->o_row, a->m, per16))
    return refuse(LYC_ERR_INVALID_ARG, "outputs must be 16-byte aligned with strides of whole 16 bytes");
  if ((c->batch > 1 && a->o_batch < c->head_dim) || (a->num_heads > 1 && a->o_head < c->head_dim) ||
      (a->m > 1 && a->o_row < c->head_dim))
    return refuse(LYC_ERR_INVALID_ARG, "rows of the outputs overlap");
  OnDevice on(c->device);
  if (!on.ok) return refuse(LYC_ERR_CUDA, "device %d cannot be used", c->device);
  ReadParams p;
  memset(&p, 0, sizeof p);
  p.k_out = static_cast<unsigned char*>(a->k_out);
  p.v_out = static_cast<unsigned char*>(a->v_out);
  p.o_batch = a->o_batch;
  p.o_head = a->o_head;
  p.o_row = a->o_row;
  p.n = a->n;
  p.sets = a->sets;
  p.status = a->status;
  p.first = a->first;
  p.m = a->m;
  p.H = a->num_heads;
  p.hdiv = a->num_heads / c->num_kv_heads;
  p.B = c->batch;
  p.cache = view(c);
  return launched(read_launch(&p, c->head_dim, a->dtype, c->type, static_cast<cudaStream_t>(stream)), "read launch");
}

uint64_t lyc_tree_workspace_bytes(const lyc_layer_cache* c, int T, int num_q_heads) {
  if (check_tree(c, T, num_q_heads) != LYC_OK) return 0;
  TreeShape s;
  if (!tree_shape(c, T, num_q_heads, true, &s)) {
    refuse(LYC_ERR_CUDA, "device %d cannot be used", c->device);
    return 0;
  }
  return s.bytes;
}

lyc_status lyc_tree_attention(const lyc_layer_cache* c, const lyc_tree_args* a, void* stream) {
  if (!a) return refuse(LYC_ERR_INVALID_ARG, "NULL arguments");
  const lyc_status st = check_tree(c, a->T, a->num_q_heads);
  if (st != LYC_OK) return st;
  if (!a->q || !a->out || !a->n || misaligned(a->q) || misaligned(a->out))
    return refuse(LYC_ERR_INVALID_ARG, "q and out must be 16-byte aligned device pointers, n not NULL");
  if (off_word(a->n, 4) || off_word(a->t_len, 4) || off_word(a->mask, 8) || off_word(a->status, 4))
    return refuse(LYC_ERR_INVALID_ARG, "n, t_len and status must be 4-byte aligned, mask 8");
  if (!(a->scale > 0.f) || isinf(a->scale)) return refuse(LYC_ERR_INVALID_ARG, "scale must be a finite number > 0");
  if (stride_bad(a->q_batch, c->batch, 8) || stride_bad(a->q_token, a->T, 8) || stride_bad(a->q_head, a->num_q_heads, 8) ||
      stride_bad(a->o_batch, c->batch, 8) || stride_bad(a->o_token, a->T, 8) || stride_bad(a->o_head, a->num_q_heads, 8))
    return refuse(LYC_ERR_INVALID_ARG, "strides of q and out must be whole 16 bytes");
  if ((c->batch > 1 && a->o_batch < c->head_dim) || (a->T > 1 && a->o_token < c->head_dim) ||
      (a->num_q_heads > 1 && a->o_head < c->head_dim))
    return refuse(LYC_ERR_INVALID_ARG, "rows of out overlap");
  OnDevice on(c->device);
  TreeShape s;
  if (!on.ok || !tree_shape(c, a->T, a->num_q_heads, true, &s))
    return refuse(LYC_ERR_CUDA, "device %d cannot be used", c->device);
  if (!a->workspace || misaligned(a->workspace) || a->workspace_bytes < s.bytes)
    return refuse(LYC_ERR_INVALID_ARG, "the workspace needs %llu bytes, 16-byte aligned",
                  static_cast<unsigned long long>(s.bytes));
  TreeTcParams P;
  memset(&P, 0, sizeof P);
  TreeParams& p = P.t;
  p.q = static_cast<const unsigned char*>(a->q);
  p.out = static_cast<unsigned char*>(a->out);
  p.q_batch = a->q_batch;
  p.q_token = a->q_token;
  p.q_head = a->q_head;
  p.o_batch = a->o_batch;
  p.o_token = a->o_token;
  p.o_head = a->o_head;
  p.n = a->n;
  p.t_len = a->t_len;
  p.mask = reinterpret_cast<const unsigned long long*>(a->mask);
  p.status = a->status;
  p.B = c->batch;
  p.T = a->T;
  p.W = (a->T + 63) / 64;
  p.Hq = a->num_q_heads;
  p.Hkv = c->num_kv_heads;
  p.G = a->num_q_heads / c->num_kv_heads;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.sum_unit = c->type == LYC_CACHE_E4M3 ? kSumUnitE4m3 : 1.f;
  p.cache = view(c);
  if (s.tc && c->type == LYC_CACHE_BF16) {
    p.box_rows = tree_tc_box_rows(p.cache);
    // a layout that TMA cannot describe (a stride of 2^40 bytes, say); needs no more workspace
    if (!tree_tc_maps(&P)) tree_shape(c, a->T, a->num_q_heads, false, &s);
  }
  p.grid = s.grid;
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2ll * s.grid * s.block_rows * c->head_dim);
  const cudaStream_t str = static_cast<cudaStream_t>(stream);
  lyc_status rc = launched(s.tc ? tree_tc_launch(&P, c->type, c->device, str)
                                : tree_mma_launch(&p, c->head_dim, c->type, s.block_rows, c->device, str),
                           "tree attention launch");
  // a group of one tile is never cut: nothing to merge
  if (rc == LYC_OK && s.cap_tiles > 1)
    rc = launched(tree_combine_launch(&p, c->head_dim, s.block_rows, s.tile_rows, str), "tree merge launch");
  return rc;
}

}  // extern "C"
