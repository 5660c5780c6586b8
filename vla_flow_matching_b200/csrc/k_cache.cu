// Rows of queries, keys and values on their way into and out of the paged prefix
// cache: per-head RMSNorm and rotate-half rotation, 8-bit codes with a scale a row,
// page writes (k_rows) and the read of many layers back into contiguous tensors
// (k_cache_read).
//
// Both kernels move every byte once and compute little (about 10 operations an
// element), so they are bound by HBM at size and by one launch when small.
#include "cache.cuh"
#include "common.cuh"
#include "kernels.cuh"

#include <cuda_fp8.h>

namespace pi0x {

namespace {
constexpr unsigned kFull = 0xffffffffu;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4 *>(p);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void load4(const bf16 *p, float (&v)[4]) {
  const uint2 x = *reinterpret_cast<const uint2 *>(p);
  v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16 *p, const float (&v)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// Pool element types: bf16 rows as they are, or codes of a scaled row.
struct PoolBf16 {
  static constexpr bool kScaled = false;
};
struct PoolE4m3 {
  static constexpr bool kScaled = true;
  // Least power of two that brings `top` within 448 = 1.75 * 2^8: a power of two makes
  // the division exact, so a code depends on its value alone, and what a code stands
  // for is exact in bf16.  top = f * 2^e, 1 <= f < 2: 2^(e-8), or 2^(e-7) above 1.75.
  static __device__ __forceinline__ float scale(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
  }
  static __device__ __forceinline__ uint32_t codes(const float (&v)[4], float scale) {
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));  // exact: 2^-n of 2^n
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  static __device__ __forceinline__ void values(uint32_t w, float (&v)[4]) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(a), y = __half22float2(b);
    v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
  }
};
struct PoolInt8 {
  static constexpr bool kScaled = true;
  static __device__ __forceinline__ float scale(uint32_t top) {
    return fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), kMinScale);
  }
  // A division per element, not a product with 1/scale: the code is then the nearest
  // one, with nothing rounded before the last step.
  static __device__ __forceinline__ uint32_t codes(const float (&v)[4], float scale) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = max(-127, min(127, __float2int_rn(__fdiv_rn(v[i], scale))));
      w |= ((uint32_t)c & 0xffu) << (8 * i);
    }
    return w;
  }
  static __device__ __forceinline__ void values(uint32_t w, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)((int)(w << (24 - 8 * i)) >> 24);
  }
};

// cos and sin of 2 pi t, t = `turn` * 2^-32 of a full turn.  The integer is split into
// the nearest quarter turn and a rest of at most an eighth (|y| <= pi/4), where the
// Taylor polynomials of degree 9 and 10 are within 2e-9 and 2e-10.
__device__ __forceinline__ void turn_cos_sin(uint32_t turn, float &c, float &s) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float y = (float)(int)(turn - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float z = y * y;
  const float sp = y + y * z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880))));
  const float cp =
      1.0f + z * (-0.5f + z * (1.0f / 24 + z * (-1.0f / 720 + z * (1.0f / 40320 + z * (-1.0f / 3628800)))));
  const float a = (quarter & 1) ? sp : cp, b = (quarter & 1) ? cp : sp;
  c = ((quarter + 1) & 2) ? -a : a;
  s = (quarter & 2) ? -b : b;
}

}  // namespace

// A group of D/8 lanes holds a row: lane l the pairs (i, i + D/2), i = 4l..4l+3, so
// that the rotation needs no exchange and loads are 8 (bf16) or 16 (fp32) bytes a lane,
// consecutive over the group.  A group takes `per` rows of one token and forms the
// token's cosines and sines once for them.
template <typename T, typename Pool, int D>
__global__ void __launch_bounds__(256) k_rows(const __grid_constant__ RowArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kLanes = D / 8;
  const int rows = a.hq + a.hk + a.hv;
  const int chunks = (rows + a.per - 1) / a.per;
  const int64_t items = (int64_t)a.B * a.T * chunks;
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  const int l4 = (threadIdx.x % kLanes) * 4;
  const bool live = item < items;
  const int64_t tok = live ? item / chunks : 0;
  const int row0 = live ? (int)(item - tok * chunks) * a.per : 0;
  const int row1 = live ? min(rows, row0 + a.per) : 0;
  const int b = (int)(tok / a.T), t = (int)(tok - (int64_t)b * a.T);
  const int64_t slot = (int64_t)(a.start ? a.start[b] : 0) + t;

  int cell = -1;  // row of the pools
  if (a.to_cache && live && row1 > a.hq && (!a.count || t < a.count[b])) cell = cache_row(a.pt, b, slot);

  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 1.0f, s[i] = 0.0f;
  if (a.rotate && row0 < a.hq + a.hk) {
    const uint64_t pos = (uint64_t)(a.positions ? (int64_t)a.positions[tok] : slot);
#pragma unroll
    for (int i = 0; i < 4; ++i) turn_cos_sin((uint32_t)((pos * a.turn[l4 + i] + 0x80000000u) >> 32), c[i], s[i]);
  }

  for (int r = 0; r < a.per; ++r) {
    const int row = row0 + r;
    const bool is_q = row < a.hq, is_k = !is_q && row < a.hq + a.hk;
    const bool put = row < row1 && (is_q || !a.to_cache || cell >= 0);
    const int h = is_q ? row : is_k ? row - a.hq : row - a.hq - a.hk;
    float x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
    if (put) {
      const RowsPtr &src = is_q ? a.q : is_k ? a.k : a.v;
      const T *p = (const T *)src.data + b * src.sb + t * src.st + h * src.sh + l4;
      load4(p, x);
      load4(p + D / 2, y);
    }
    const float *gain = is_q ? a.q_gain : is_k ? a.k_gain : nullptr;
    if (a.q_gain || a.k_gain) {  // the same for every lane: the sums below are warp-wide
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      if (gain) {
        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
        float g[4], g2[4];
        load4(gain + l4, g);
        load4(gain + D / 2 + l4, g2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = x[i] * inv * (1.0f + g[i]);
          y[i] = y[i] * inv * (1.0f + g2[i]);
        }
      }
    }
    if (a.rotate && (is_q || is_k)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = x[i] * c[i] - y[i] * s[i];
        y[i] = y[i] * c[i] + x[i] * s[i];
        x[i] = lo;
      }
    }
    if constexpr (Pool::kScaled) {  // launched with to_cache only
      // Largest magnitude as bits: NaN and infinity order above every finite value.
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = max(top, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(y[i]) & 0x7fffffffu));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
      if (put && !is_q) {
        const PoolPtr &pool = is_k ? a.kp : a.vp;
        const int64_t at = (int64_t)cell * a.hk + h;
        const bool finite = top < 0x7f800000u;
        const float scale = finite ? Pool::scale(top) : __uint_as_float(0x7fc00000u);
        uint32_t lo = 0, hi = 0;
        if (finite) {
          lo = Pool::codes(x, scale);
          hi = Pool::codes(y, scale);
        }
        uint8_t *dst = (uint8_t *)pool.codes + at * D + l4;
        *reinterpret_cast<uint32_t *>(dst) = lo;
        *reinterpret_cast<uint32_t *>(dst + D / 2) = hi;
        if (l4 == 0) pool.scale[at] = scale;
      }
    }
    if (put && (is_q || !a.to_cache)) {
      const RowsPtr &dst = is_q ? a.q_out : a.k_out;
      T *p = (T *)dst.data + b * dst.sb + t * dst.st + h * dst.sh + l4;
      store4(p, x);
      store4(p + D / 2, y);
    }
    if (put && !is_q && a.to_cache && !Pool::kScaled) {
      bf16 *p = (bf16 *)(is_k ? a.kp : a.vp).codes + ((int64_t)cell * a.hk + h) * D + l4;
      store4(p, x);
      store4(p + D / 2, y);
    }
  }
}

// A lane group of D/8 lanes moves a row of keys and the row of values beside it.
template <typename T, typename Pool, int D>
__global__ void __launch_bounds__(256) k_cache_read(const __grid_constant__ ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kLanes = D / 8;
  const int64_t items = (int64_t)a.layers * a.B * a.kv * a.P;
  const int64_t step = (int64_t)gridDim.x * blockDim.x / kLanes;
  const int l8 = (threadIdx.x % kLanes) * 8;
  for (int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kLanes; item < items; item += step) {
    const int p = (int)(item % a.P);
    const int64_t rest = item / a.P;
    const int h = (int)(rest % a.kv), b = (int)(rest / a.kv % a.B), layer = (int)(rest / a.kv / a.B);
    int cell = -1;
    if (p < a.lens[b] && (!a.mask || a.mask[(int64_t)b * a.P + p])) cell = cache_row(a.pt, b, p);
    if (a.mask_out && layer == 0 && h == 0 && l8 == 0) a.mask_out[(int64_t)b * a.P + p] = cell >= 0;
    const int64_t at = (layer * a.layer_rows + cell) * a.kv + h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const PoolPtr &pool = i ? a.vp : a.kp;
      float x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
      if (cell >= 0) {
        if constexpr (Pool::kScaled) {
          const uint2 w = *reinterpret_cast<const uint2 *>((const uint8_t *)pool.codes + at * D + l8);
          const float scale = pool.scale[at];
          Pool::values(w.x, x);
          Pool::values(w.y, y);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] *= scale, y[j] *= scale;
        } else {
          load4((const bf16 *)pool.codes + at * D + l8, x);
          load4((const bf16 *)pool.codes + at * D + l8 + 4, y);
        }
      }
      T *dst = (T *)(i ? a.v_out : a.k_out) + item * D + l8;
      store4(dst, x);
      store4(dst + 4, y);
    }
  }
}

namespace {

template <typename T, typename Pool, int D>
cudaError_t rows_go(RowArgs a, cudaStream_t s) {
  constexpr int kLanes = D / 8;
  const int rows = a.hq + a.hk + a.hv;
  a.per = 1;
  const int64_t threads = (int64_t)a.B * a.T * ((rows + a.per - 1) / a.per) * kLanes;
  return launch_pdl(k_rows<T, Pool, D>, dim3((unsigned)((threads + 255) / 256)), 256, 0, s, a);
}
template <typename T, typename Pool, int D>
cudaError_t read_go(const ReadArgs &a, cudaStream_t s) {
  const int64_t threads = (int64_t)a.layers * a.B * a.kv * a.P * (D / 8);
  const int64_t blocks = (threads + 255) / 256;
  return launch_pdl(k_cache_read<T, Pool, D>, dim3((unsigned)(blocks < 148 * 32 ? blocks : 148 * 32)), 256, 0, s, a);
}

#define PI0X_PICK(fn, ...)                                                                    \
  auto by_dim = [&](auto t, auto p) -> cudaError_t {                                          \
    using T = decltype(t);                                                                    \
    using P = decltype(p);                                                                    \
    return head_dim == 64 ? fn<T, P, 64>(__VA_ARGS__)                                         \
                          : head_dim == 128 ? fn<T, P, 128>(__VA_ARGS__) : fn<T, P, 256>(__VA_ARGS__); \
  };                                                                                          \
  auto by_pool = [&](auto t) -> cudaError_t {                                                 \
    return pool_dtype == PI0X_DTYPE_E4M3 ? by_dim(t, PoolE4m3())                              \
                                         : pool_dtype == PI0X_DTYPE_INT8 ? by_dim(t, PoolInt8()) : by_dim(t, PoolBf16()); \
  };                                                                                          \
  return dtype == PI0X_DTYPE_F32 ? by_pool(float()) : by_pool(bf16())

}  // namespace

cudaError_t launch_rows(const RowArgs &a, int dtype, int pool_dtype, int head_dim, cudaStream_t s) {
  PI0X_PICK(rows_go, a, s);
}
cudaError_t launch_cache_read(const ReadArgs &a, int dtype, int pool_dtype, int head_dim, cudaStream_t s) {
  PI0X_PICK(read_go, a, s);
}

}  // namespace pi0x
