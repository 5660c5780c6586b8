// C ABI of the paged prefix cache (include/pi0x.h): checks of arguments and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "../../include/pi0x.h"
#include "cache.cuh"
#include "common.cuh"
#include "kernels.cuh"

namespace pi0x {
namespace {

int refuse(int status, const char *why) {
  set_last_error(why);
  return status;
}
int launched(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return PI0X_OK;
  cudaGetLastError();
  set_last_error((std::string(what) + ": " + cudaGetErrorString(e)).c_str());
  return e == cudaErrorMemoryAllocation ? PI0X_ENOMEM : PI0X_ECUDA;
}
bool aligned(const void *p, size_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
constexpr float kLog2e = 1.4426950408889634f;
bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Rows of `elem`-byte elements: data and strides in whole 16 bytes.
bool rows_ok(const pi0x_rows *r, int elem) {
  const int64_t n = 16 / elem;
  return r && r->data && aligned(r->data) && r->batch_stride % n == 0 && r->token_stride % n == 0 &&
         r->head_stride % n == 0;
}
// No two of an output's rows share memory: each stride, from the least on, is beyond all that the
// lesser ones span.
bool apart(const pi0x_rows *r, int B, int T, int heads, int head_dim) {
  typedef __int128 Wide;
  struct {
    int n;
    Wide stride;
  } dim[3] = {{B, r->batch_stride}, {T, r->token_stride}, {heads, r->head_stride}};
  for (auto &d : dim) d.stride = d.stride < 0 ? -d.stride : d.stride;
  std::sort(dim, dim + 3, [](const auto &x, const auto &y) { return x.stride < y.stride; });
  Wide span = head_dim;
  for (const auto &d : dim) {
    if (d.n < 2) continue;
    if (d.stride < span) return false;
    span += (d.n - 1) * d.stride;
  }
  return true;
}
RowsPtr rows_of(const pi0x_rows *r) { return RowsPtr{r->data, r->batch_stride, r->token_stride, r->head_stride}; }

bool rotation_ok(const pi0x_rotation *r) {
  const bool gains = r->q_gain || r->k_gain;
  return aligned(r->q_gain, 4) && aligned(r->k_gain, 4) && aligned(r->positions, 4) && (!gains || (r->eps > 0.0f && isfinite(r->eps))) &&
         (r->rope_base == 0.0f || (r->rope_base >= 1.0f && isfinite(r->rope_base)));
}

// The ratios of a rotation's angles (RowArgs) as 64-bit fractions; one of 1 is a step below it.
// They depend on (base, D) alone; the last ones formed are kept per thread.
void set_ratios(RowArgs &a, float base, int head_dim) {
  static thread_local float last_base = 0.0f;
  static thread_local int last_dim = 0;
  static thread_local uint64_t ratio[7];
  if (base != last_base || head_dim != last_dim) {
    for (int k = 0; k < 7; ++k) {
      const long double r = powl((long double)base, -2.0L * (1 << k) / head_dim) * 18446744073709551616.0L;
      ratio[k] = r >= 18446744073709551615.0L ? UINT64_MAX : (uint64_t)r;
    }
    last_base = base;
    last_dim = head_dim;
  }
  for (int k = 0; k < 7; ++k) a.ratio[k] = ratio[k];
}

// The norms and the rotation of a RowArgs whose heads are set.
void set_rotation(RowArgs &a, const pi0x_rotation *rot, int head_dim) {
  a.q_gain = a.hq ? rot->q_gain : nullptr;
  a.k_gain = a.hk ? rot->k_gain : nullptr;
  a.eps = rot->eps;
  a.positions = rot->positions;
  a.rotate = rot->rope_base > 0.0f;
  if (a.rotate) set_ratios(a, rot->rope_base, head_dim);
}

// The sizes of an attention call on a cache that check_cache() has seen.
int check_attend(const pi0x_cache *c, int B, int q_heads, int max_pages) {
  if (q_heads < 1 || q_heads % c->kv_heads)
    return refuse(PI0X_EINVAL, "pi0x_cache_attention: no heads, or heads that kv_heads does not divide");
  if (B > 65535 || q_heads > 65535 || (int64_t)B * q_heads > INT32_MAX)
    return refuse(PI0X_EINVAL, "pi0x_cache_attention: over 65535 samples or heads, or 2^31 rows or more");
  if ((int64_t)B > INT32_MAX / (((int64_t)max_pages * c->page_size + 63) / 64))
    return refuse(PI0X_EINVAL, "pi0x_cache_attention: 2^31 blocks of 64 slots or more");
  return PI0X_OK;
}

}  // namespace

int check_cache(const pi0x_cache *c, int layer0, int layers, int B, const int32_t *table, int max_pages) {
  if (!c || !c->k || !c->v || !table || !aligned(table, 4) || B < 1 || max_pages < 1 || c->layers < 1 || c->num_pages < 1 ||
      c->page_size < 1 || c->kv_heads < 1 || layer0 < 0 || layers < 1 || layers > c->layers - layer0)
    return refuse(PI0X_EINVAL, "paged cache: null or misaligned pointer, size below 1 or layer out of range");
  if (c->dtype != PI0X_DTYPE_BF16 && c->dtype != PI0X_DTYPE_E4M3 && c->dtype != PI0X_DTYPE_INT8)
    return refuse(PI0X_EUNSUPPORTED, "paged cache: pages are bf16, e4m3 or int8");
  if (!head_dim_ok(c->head_dim)) return refuse(PI0X_EUNSUPPORTED, "paged cache: head_dim is 64, 128 or 256");
  if (c->dtype != PI0X_DTYPE_BF16 && (!c->k_scale || !c->v_scale))
    return refuse(PI0X_EINVAL, "paged cache: 8-bit pages need k_scale and v_scale");
  if (!aligned(c->k) || !aligned(c->v) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return refuse(PI0X_EINVAL, "paged cache: pools must be 16-byte aligned");
  const int64_t most = INT32_MAX;
  if ((int64_t)c->num_pages * c->page_size > most / c->layers || c->kv_heads > 65535)
    return refuse(PI0X_EINVAL, "paged cache: 2^31 rows or more, or over 65535 kv heads");
  if ((int64_t)max_pages * c->page_size > most - 4096)  // kernels look a few blocks of keys ahead in 32 bits
    return refuse(PI0X_EINVAL, "paged cache: a page table of 2^31 - 4096 slots or more");
  return PI0X_OK;
}

PoolPtr layer_pool(const pi0x_cache *c, int layer, bool v) {
  const int64_t cells = (int64_t)layer * c->num_pages * c->page_size * c->kv_heads;
  uint8_t *codes = (uint8_t *)(v ? c->v : c->k) + cells * c->head_dim * (int64_t)pool_elem(c->dtype);
  return PoolPtr{codes, c->dtype == PI0X_DTYPE_BF16 ? nullptr : (v ? c->v_scale : c->k_scale) + cells};
}
PageTable page_table(const pi0x_cache *c, const int32_t *table, int max_pages) {
  return PageTable{table, max_pages, c->page_size, c->num_pages, FastDiv(c->page_size)};
}

}  // namespace pi0x

using namespace pi0x;

extern "C" {

int pi0x_qk_norm_rope(int dtype, int B, int T, int q_heads, int k_heads, int head_dim, const pi0x_rows *q,
                      const pi0x_rows *k, const int32_t *start, const pi0x_rotation *rot, const pi0x_rows *q_out,
                      const pi0x_rows *k_out, void *stream) {
  if (!rot || !aligned(start, 4) || B < 1 || T < 1 || q_heads < 0 || k_heads < 0 || (q_heads == 0 && k_heads == 0))
    return refuse(PI0X_EINVAL, "pi0x_qk_norm_rope: null rotation, misaligned start, size below 1 or no heads");
  if (dtype != PI0X_DTYPE_BF16 && dtype != PI0X_DTYPE_F32)
    return refuse(PI0X_EUNSUPPORTED, "pi0x_qk_norm_rope: rows are bf16 or f32");
  if (!head_dim_ok(head_dim)) return refuse(PI0X_EUNSUPPORTED, "pi0x_qk_norm_rope: head_dim is 64, 128 or 256");
  const int elem = dtype == PI0X_DTYPE_F32 ? 4 : 2;
  if ((q_heads && (!rows_ok(q, elem) || !rows_ok(q_out, elem))) ||
      (k_heads && (!rows_ok(k, elem) || !rows_ok(k_out, elem))))
    return refuse(PI0X_EINVAL, "pi0x_qk_norm_rope: rows must be given, with data and strides in whole 16 bytes");
  if ((q_heads && !apart(q_out, B, T, q_heads, head_dim)) || (k_heads && !apart(k_out, B, T, k_heads, head_dim)))
    return refuse(PI0X_EINVAL, "pi0x_qk_norm_rope: rows of an output overlap");
  if (!rotation_ok(rot)) return refuse(PI0X_EINVAL, "pi0x_qk_norm_rope: gain alignment, eps or rope_base");
  if ((int64_t)B * T > INT32_MAX / ((int64_t)q_heads + k_heads))
    return refuse(PI0X_EINVAL, "pi0x_qk_norm_rope: 2^31 rows or more");
  RowArgs a = {};
  a.B = B;
  a.T = T;
  a.hq = q_heads;
  a.hk = k_heads;
  if (q_heads) a.q = rows_of(q), a.q_out = rows_of(q_out);
  if (k_heads) a.k = rows_of(k), a.k_out = rows_of(k_out);
  a.start = start;
  set_rotation(a, rot, head_dim);
  return launched(launch_rows(a, dtype, PI0X_DTYPE_BF16, head_dim, (cudaStream_t)stream), "pi0x_qk_norm_rope");
}

int pi0x_cache_write(const pi0x_cache *cache, int layer, int dtype, int B, int T, const pi0x_rows *k,
                     const pi0x_rows *v, const int32_t *table, int max_pages, const int32_t *start,
                     const int32_t *count, const pi0x_rotation *rot, int q_heads, const pi0x_rows *q,
                     const pi0x_rows *q_out, void *stream) {
  const int st = check_cache(cache, layer, 1, B, table, max_pages);
  if (st) return st;
  if (T < 1 || !start || !aligned(start, 4) || !aligned(count, 4) || q_heads < 0 || (q_heads && !rot))
    return refuse(PI0X_EINVAL, "pi0x_cache_write: T below 1, start missing, start or count misaligned, or q without a rotation");
  if (dtype != PI0X_DTYPE_BF16 && dtype != PI0X_DTYPE_F32)
    return refuse(PI0X_EUNSUPPORTED, "pi0x_cache_write: rows are bf16 or f32");
  const int elem = dtype == PI0X_DTYPE_F32 ? 4 : 2;
  if (!rows_ok(k, elem) || !rows_ok(v, elem) || (q_heads && (!rows_ok(q, elem) || !rows_ok(q_out, elem))))
    return refuse(PI0X_EINVAL, "pi0x_cache_write: rows must be given, with data and strides in whole 16 bytes");
  if (q_heads && !apart(q_out, B, T, q_heads, cache->head_dim))
    return refuse(PI0X_EINVAL, "pi0x_cache_write: rows of q_out overlap");
  if (rot && !rotation_ok(rot)) return refuse(PI0X_EINVAL, "pi0x_cache_write: gain alignment, eps or rope_base");
  if ((int64_t)B * T > INT32_MAX / ((int64_t)q_heads + 2 * cache->kv_heads))
    return refuse(PI0X_EINVAL, "pi0x_cache_write: 2^31 rows or more");
  RowArgs a = {};
  a.B = B;
  a.T = T;
  a.hq = q_heads;
  a.hk = cache->kv_heads;
  if (q_heads) a.q = rows_of(q), a.q_out = rows_of(q_out);
  a.k = rows_of(k);
  a.v = rows_of(v);
  a.start = start;
  a.count = count;
  if (rot) set_rotation(a, rot, cache->head_dim);
  a.to_cache = 1;
  a.kp = layer_pool(cache, layer, false);
  a.vp = layer_pool(cache, layer, true);
  a.pt = page_table(cache, table, max_pages);
  return launched(launch_rows(a, dtype, cache->dtype, cache->head_dim, (cudaStream_t)stream), "pi0x_cache_write");
}

int pi0x_cache_read(const pi0x_cache *cache, int layer0, int layers, int B, int P, const int32_t *table,
                    int max_pages, const int32_t *lens, const uint8_t *mask, int dtype, void *k_out, void *v_out,
                    uint8_t *mask_out, void *stream) {
  const int st = check_cache(cache, layer0, layers, B, table, max_pages);
  if (st) return st;
  if (P < 1 || !lens || !aligned(lens, 4) || !k_out || !v_out || !aligned(k_out) || !aligned(v_out))
    return refuse(PI0X_EINVAL, "pi0x_cache_read: P below 1, a null or misaligned pointer");
  if (dtype != PI0X_DTYPE_BF16 && dtype != PI0X_DTYPE_F32)
    return refuse(PI0X_EUNSUPPORTED, "pi0x_cache_read: outputs are bf16 or f32");
  if ((int64_t)B * P > INT32_MAX / layers / cache->kv_heads)
    return refuse(PI0X_EINVAL, "pi0x_cache_read: 2^31 rows or more");
  ReadArgs a = {};
  a.layers = layers;
  a.B = B;
  a.kv = cache->kv_heads;
  a.P = P;
  a.layer_rows = (int64_t)cache->num_pages * cache->page_size;
  a.kp = layer_pool(cache, layer0, false);
  a.vp = layer_pool(cache, layer0, true);
  a.pt = page_table(cache, table, max_pages);
  a.lens = lens;
  a.mask = mask;
  a.k_out = k_out;
  a.v_out = v_out;
  a.mask_out = mask_out;
  return launched(launch_cache_read(a, dtype, cache->dtype, cache->head_dim, (cudaStream_t)stream), "pi0x_cache_read");
}

size_t pi0x_cache_attention_workspace(const pi0x_cache *c, int B, int q_heads, int max_pages) {
  int dummy = 0;
  if (check_cache(c, 0, 1, B, &dummy, max_pages) || check_attend(c, B, q_heads, max_pages)) return 0;
  return attend_workspace(B, q_heads, c->kv_heads, c->head_dim, c->dtype, c->page_size, max_pages);
}

int pi0x_cache_attention(const pi0x_cache *cache, int layer, int B, int q_heads, const pi0x_rows *q,
                         const int32_t *table, int max_pages, const int32_t *lens, const uint8_t *mask, int mask_len,
                         float scale, void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  const int st = check_cache(cache, layer, 1, B, table, max_pages);
  if (st) return st;
  const int sizes = check_attend(cache, B, q_heads, max_pages);
  if (sizes) return sizes;
  const pi0x_rows one = q ? pi0x_rows{q->data, q->batch_stride, 0, q->head_stride} : pi0x_rows{};  // a token a sample
  if (!lens || !aligned(lens, 4) || !out || !aligned(out) || !aligned(lse, 4) || !rows_ok(&one, 2) ||
      (mask && mask_len < 1) || !isfinite(scale * kLog2e))
    return refuse(PI0X_EINVAL, "pi0x_cache_attention: a null or misaligned pointer, an empty mask or a scale that is "
                               "not finite or beyond 2e38");
  const size_t need =
      attend_workspace(B, q_heads, cache->kv_heads, cache->head_dim, cache->dtype, cache->page_size, max_pages);
  if (need && (!workspace || !aligned(workspace) || workspace_bytes < need))
    return refuse(PI0X_EINVAL, "pi0x_cache_attention: workspace missing, misaligned or too small");
  AttendArgs a = {};
  a.B = B;
  a.heads = q_heads;
  a.kv = cache->kv_heads;
  a.q = (const bf16 *)q->data;
  a.q_sb = q->batch_stride;
  a.q_sh = q->head_stride;
  a.kp = layer_pool(cache, layer, false);
  a.vp = layer_pool(cache, layer, true);
  a.pt = page_table(cache, table, max_pages);
  a.lens = lens;
  a.mask = mask;
  a.mask_len = mask_len;
  a.scale_log2 = scale * kLog2e;
  a.out = (bf16 *)out;
  a.lse = lse;
  a.part = (float *)workspace;
  return launched(launch_attend(a, cache->dtype, cache->head_dim, (cudaStream_t)stream), "pi0x_cache_attention");
}

}  // extern "C"
