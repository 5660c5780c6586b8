// Attention of one new token a sample over the paged prefix cache.
//
// s_j = scale * q . k_j, out = sum_j e^(s_j - m) v_j / l, l = sum_j e^(s_j - m), with the
// running maximum m and sum l of one pass over the keys.
#include "cache.cuh"
#include "common.cuh"
#include "kernels.cuh"

#include <cuda_fp8.h>
#include <math.h>

namespace pi0x {

namespace {
constexpr int kWarps = 4;

__device__ __forceinline__ float code_value(const bf16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float code_value(const __nv_fp8_e4m3 *p) { return (float)*p; }
__device__ __forceinline__ float code_value(const int8_t *p) { return (float)*p; }
}  // namespace

// One block a (sample, query head): warps take every fourth key, a lane D/32 dims.
template <typename C, int D>
__global__ void __launch_bounds__(kWarps * 32) k_attend(const __grid_constant__ AttendArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = D / 32;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = h / (a.heads / a.kv);
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(a.q[b * a.q_sb + h * a.q_sh + lane + 32 * i]) * a.scale_log2;
    o[i] = 0.0f;
  }
  const int64_t cap = (int64_t)a.pt.max_pages * a.pt.page_size;
  int n = (int)min((int64_t)a.lens[b], cap);
  if (a.mask) n = min(n, a.mask_len);
  for (int p = warp; p < n; p += kWarps) {
    if (a.mask && !a.mask[(int64_t)b * a.mask_len + p]) continue;
    const int cell = cache_row(a.pt, b, p);
    if (cell < 0) continue;
    const int64_t at = (int64_t)cell * a.kv + g;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += q[i] * code_value((const C *)a.kp.codes + at * D + lane + 32 * i);
    s = warp_sum(s);
    if (a.kp.scale) s *= a.kp.scale[at];
    const float m2 = fmaxf(m, s), keep = m == -INFINITY ? 0.0f : exp2f(m - m2);
    const float e = exp2f(s - m2), w = a.vp.scale ? e * a.vp.scale[at] : e;
    l = l * keep + e;
    m = m2;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * code_value((const C *)a.vp.codes + at * D + lane + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) sm_o[warp][lane + 32 * i] = o[i];
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
  __syncthreads();
  float mm = -INFINITY, ll = 0.0f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sm_m[w] == -INFINITY ? 0.0f : exp2f(sm_m[w] - mm);
    ll += f[w] * sm_l[w];
  }
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x += f[w] * sm_o[w][d];
    a.out[((int64_t)b * a.heads + h) * D + d] = __float2bfloat16_rn(ll == 0.0f ? 0.0f : x / ll);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)b * a.heads + h] = ll == 0.0f ? -INFINITY : mm * 0.69314718f + logf(ll);
}

size_t attend_workspace(int, int, int, int, int, int, int) { return 0; }

namespace {
template <typename C, int D>
cudaError_t attend_go(const AttendArgs &a, cudaStream_t s) {
  return launch_pdl(k_attend<C, D>, dim3(a.heads, a.B), kWarps * 32, 0, s, a);
}
template <typename C>
cudaError_t attend_dim(const AttendArgs &a, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? attend_go<C, 64>(a, s) : head_dim == 128 ? attend_go<C, 128>(a, s) : attend_go<C, 256>(a, s);
}
}  // namespace

cudaError_t launch_attend(const AttendArgs &a, int pool_dtype, int head_dim, cudaStream_t s) {
  return pool_dtype == PI0X_DTYPE_E4M3   ? attend_dim<__nv_fp8_e4m3>(a, head_dim, s)
         : pool_dtype == PI0X_DTYPE_INT8 ? attend_dim<int8_t>(a, head_dim, s)
                                         : attend_dim<bf16>(a, head_dim, s);
}

}  // namespace pi0x
