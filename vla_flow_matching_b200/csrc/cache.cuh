// Internal interface of the paged prefix cache kernels (k_cache.cu, k_cache_attn.cu),
// called by cache_api.cu and pi0x_api.cu.  Not part of the ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pi0x.h"

namespace pi0x {

typedef __nv_bfloat16 bf16;

// Rows of a (batch, token, head, head_dim) tensor, strides in elements.
struct RowsPtr {
  void *data;
  int64_t sb, st, sh;
};

// One pool of a layer: row r = page * page_size + offset holds kv_heads * head_dim codes.
struct PoolPtr {
  void *codes;
  float *scale;
};

// n / d for 0 <= n < 2^31 by a product: q = (hi32(n * m) + n) >> l with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1 (Granlund and Montgomery, 1994).
struct FastDiv {
  uint32_t d, m, l;
  FastDiv() = default;
  __host__ explicit FastDiv(uint32_t div) : d(div), l(0) {
    while ((1ull << l) < div) ++l;
    m = (uint32_t)(((1ull << 32) * ((1ull << l) - div)) / div + 1);
  }
  __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)((((uint64_t)n * m >> 32) + n) >> l);
  }
};

struct PageTable {
  const int *table;   // (B, max_pages)
  int max_pages, page_size, num_pages;
  FastDiv by_page;    // by page_size
};

// Row of the pool that holds slot `pos` of sample b, or -1 (no page there).
__host__ __device__ __forceinline__ int cache_row(const PageTable &pt, int b, int64_t pos) {
  if (pos < 0 || pos >= (int64_t)pt.max_pages * pt.page_size) return -1;
  const uint32_t at = pt.by_page.div((uint32_t)pos), off = (uint32_t)pos - at * (uint32_t)pt.page_size;
  const int page = pt.table[(int64_t)b * pt.max_pages + at];
  return page >= 0 && page < pt.num_pages ? page * pt.page_size + (int)off : -1;
}

// ---- norm, rotation and page writes (k_cache.cu) ---------------------------------
struct RowArgs {
  int B, T, hq, hk;            // heads of q, of k and v
  RowsPtr q, k, v, q_out, k_out;
  const int *start, *count, *positions;
  const float *q_gain, *k_gain;
  float eps;
  int rotate, to_cache;
  PoolPtr kp, vp;              // to_cache: the layer's pools
  PageTable pt;
  int per;                     // heads of a token that one lane group rotates
  uint32_t q_blocks;           // blocks of q rows, before those of k (and v) rows
  FastDiv by_q, by_k, by_t;    // by a token's items of q and of k, by T
  // pair i turns by pos * f_i of a full turn, f_i = base^(-2i/D) / 2 pi as a 64-bit fraction:
  // 1 / 2 pi times ratio[k] = base^(-2 * 2^k / D) for every bit k of i
  uint64_t ratio[7];
};
cudaError_t launch_rows(const RowArgs &a, int dtype, int pool_dtype, int head_dim, cudaStream_t s);

struct ReadArgs {
  int layers, B, kv, P;
  int64_t layer_rows;          // num_pages * page_size
  PoolPtr kp, vp;              // of the first layer
  PageTable pt;
  const int *lens;
  const uint8_t *mask;
  void *k_out, *v_out;
  uint8_t *mask_out;
  FastDiv by_p, by_kv, by_b;
};
cudaError_t launch_cache_read(const ReadArgs &a, int dtype, int pool_dtype, int head_dim, cudaStream_t s);

// ---- attention of one new token (k_cache_attn.cu) --------------------------------
struct AttendArgs {
  int B, heads, kv;
  const bf16 *q;
  int64_t q_sb, q_sh;
  PoolPtr kp, vp;              // of the layer
  PageTable pt;
  const int *lens;
  const uint8_t *mask;
  int mask_len;
  float scale_log2;            // scale * log2(e)
  bf16 *out;
  float *lse;
  float *part;                 // workspace
};
size_t attend_workspace(int B, int heads, int kv, int head_dim, int pool_dtype, int page_size, int max_pages);
cudaError_t launch_attend(const AttendArgs &a, int pool_dtype, int head_dim, cudaStream_t s);

// Host checks of a cache descriptor and its page table (PI0X_OK or the status to return).
int check_cache(const pi0x_cache *c, int layer0, int layers, int B, const int32_t *table, int max_pages);
PoolPtr layer_pool(const pi0x_cache *c, int layer, bool v);
PageTable page_table(const pi0x_cache *c, const int32_t *table, int max_pages);
inline size_t pool_elem(int dtype) { return dtype == PI0X_DTYPE_BF16 ? 2 : 1; }

}  // namespace pi0x
