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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&x);
}
// Two fp32 values in a 64-bit register pair: sm_100 multiplies and adds both in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split(f32x2 a, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 16 bytes of a row: 8 bf16 or 4 fp32 values, in pairs.
template <typename T>
struct Vec;
template <>
struct Vec<bf16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4 &w, f32x2 (&v)[4]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 put(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4 &w, f32x2 (&v)[2]) {
    v[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
    v[1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  static __device__ __forceinline__ uint4 put(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
// N = 4 or 8 values as bf16.
template <int N>
__device__ __forceinline__ void store_bf16(bf16 *p, const float (&v)[N]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4 *>(p) = Vec<bf16>::put(v);
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// Pool element types: bf16 rows as they are, or codes of a scaled row.  kDouble: keys are normed
// and rotated in 64 bits on their way in.  What e4m3 codes stand for is exact, so all the error
// of a page is in codes next to the border of two, a whole step each; in fp32 one value in 2.5
// million falls on the wrong side, in 64 bits next to none.
struct PoolBf16 {
  static constexpr bool kScaled = false, kDouble = false;
};
struct PoolE4m3 {
  static constexpr bool kScaled = true, kDouble = true;
  // Least power of two that brings `top` within 448 = 1.75 * 2^8: a power of two makes
  // the division exact, so a code depends on its value alone, and what a code stands
  // for is exact in bf16.  top = f * 2^e, 1 <= f < 2: 2^(e-8), or 2^(e-7) above 1.75.
  static __device__ __forceinline__ float scale(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
  }
  template <int N>
  static __device__ __forceinline__ void codes(const float (&v)[N], float scale, uint32_t (&w)[N / 4]) {
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));  // exact: 2^-n of 2^n
    uint32_t c[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      c[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = c[2 * i] | c[2 * i + 1] << 16;
  }
  static __device__ __forceinline__ void values(uint32_t w, f32x2 *v) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(a), y = __half22float2(b);
    v[0] = pair(x.x, x.y), v[1] = pair(y.x, y.y);
  }
};
struct PoolInt8 {
  static constexpr bool kScaled = true, kDouble = false;
  static __device__ __forceinline__ float scale(uint32_t top) {
    return fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), kMinScale);
  }
  // x / scale, correctly rounded before the last step, so that a code is the nearest one: with
  // the rounded reciprocal r, q = x r and then q + (x - q scale) r is the rounded quotient
  // (Markstein, 1990) as long as the residual is exact, which scales of 2^-100 and more
  // guarantee.  |x / scale| is at most 127 and a rounding, so the code needs no clamp, and the sum
  // with 1.5 * 2^23, where a step is 1, has the rounded integer in its low bits.  (In packed pairs
  // and without conversions 64 x 816 tokens of one head of 256 dims, written and read back, take
  // 43.5 us instead of 47.5.)
  template <int N>
  static __device__ __forceinline__ void codes(const float (&v)[N], float scale, uint32_t (&w)[N / 4]) {
    constexpr float kInt = 12582912.0f;
    float c[N];
    if (scale >= 7.8886091e-31f) {
      const float r = __frcp_rn(scale);
      const f32x2 r2 = pair(r, r), minus = pair(-scale, -scale);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const f32x2 x = pair(v[2 * i], v[2 * i + 1]), q = mul2(x, r2);
        split(add2(fma2(fma2(q, minus, x), r2, q), pair(kInt, kInt)), c[2 * i], c[2 * i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) c[i] = __fdiv_rn(v[i], scale) + kInt;
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t lo = __byte_perm(__float_as_uint(c[4 * i]), __float_as_uint(c[4 * i + 1]), 0x0040);
      const uint32_t hi = __byte_perm(__float_as_uint(c[4 * i + 2]), __float_as_uint(c[4 * i + 3]), 0x0040);
      w[i] = __byte_perm(lo, hi, 0x5410);
    }
  }
  // x + 128 as the low bits of a float in [2^23, 2^24), whose steps are 1; minus 2^23 + 128.
  static __device__ __forceinline__ void values(uint32_t w, f32x2 *v) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7650 + i));
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = add2(pair(x[2 * i], x[2 * i + 1]), pair(-8388736.0f, -8388736.0f));
  }
};

// f_i of RowArgs.  Every product loses up to a unit of 2^-64 and takes over the part of the last ones'
// losses that its ratio leaves: f_i is less than 2 units off at bases of 100 and more, 7.5 at base 1, and
// the angle of a 32-bit position, rounded to 32 bits, less than 1.5 * 2^-32 of a turn, 4.3 * 2^-32 at base 1
// (all i, in exact arithmetic).  (A table of them in the parameters, which lanes index apart, is read
// one lane after another.)
__device__ __forceinline__ uint64_t turn_of(const RowArgs &a, int i) {
  uint64_t f = 2935890503282001226ull;  // 2^64 / 2 pi
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (i >> k & 1) f = __umul64hi(f, a.ratio[k]);
  return f;
}
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

// The same to 2^-20 or so with sin.approx and cos.approx, for rows that are rounded to bf16
// (2^-9) on their way in or out: a third of the instructions.
__device__ __forceinline__ void turn_cos_sin_approx(uint32_t turn, float &c, float &s) {
  const float y = (float)(int)turn * 1.4629180792671596e-9f;  // 2 pi 2^-32: [-pi, pi]
  c = __cosf(y);
  s = __sinf(y);
}

}  // namespace

// A lane holds 16 bytes of each half of a row, the pairs (i, i + D/2), so the rotation needs
// no exchange; D/16 (bf16) or D/8 (fp32) lanes hold a row.  RowMath has what is done to a row.
// kExact: sines and cosines to fp32 (fp32 rows, and those on their way into 8-bit codes).
template <typename T, int D, bool kExact>
struct RowMath {
  static constexpr int kN = Vec<T>::kN, kP = kN / 2, kLanes = D / 2 / kN;
  f32x2 c[kP], s[kP];           // cosines and sines of the lane's pairs
  f32x2 ns[kExact ? kP : 1];    // kExact: negative sines, which save a rounding

  // The tables in shared memory are laid out so that the lanes of a group read consecutive
  // words: entry i of lane l is turn i * kLanes + l; gains go four at a time.
  static __device__ __forceinline__ int turn_at(int p) { return p % kN * kLanes + p / kN; }
  static __device__ __forceinline__ int gain_at(int d) {
    const int p = d % (D / 2);
    return d / (D / 2) * (D / 2) + (p % kN / 4 * kLanes + p / kN) * 4 + p % 4;
  }

  // table: the lane's first entry
  __device__ __forceinline__ void turn(int64_t pos, const uint64_t *table) {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      float cs[2], sn[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t t = (uint32_t)(((uint64_t)pos * table[(2 * i + k) * kLanes] + 0x80000000u) >> 32);
        if constexpr (kExact)
          turn_cos_sin(t, cs[k], sn[k]);
        else
          turn_cos_sin_approx(t, cs[k], sn[k]);
      }
      c[i] = pair(cs[0], cs[1]);
      s[i] = pair(sn[0], sn[1]);
      if constexpr (kExact) ns[i] = pair(-sn[0], -sn[1]);
    }
  }
  __device__ __forceinline__ void rotate(f32x2 (&x)[kP], f32x2 (&y)[kP]) const {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      f32x2 v;
      if constexpr (kExact)
        v = fma2(y[i], ns[i], mul2(x[i], c[i]));
      else
        v = fma2(mul2(y[i], s[i]), pair(-1.0f, -1.0f), mul2(x[i], c[i]));
      y[i] = fma2(y[i], c[i], mul2(x[i], s[i]));
      x[i] = v;
    }
  }
  // gain: the lane's first 1 + g of the first half; the second half's are D/2 further
  static __device__ __forceinline__ void norm(f32x2 (&x)[kP], f32x2 (&y)[kP], const float *gain, float eps) {
    f32x2 sum = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < kP; ++i) sum = fma2(x[i], x[i], sum);
#pragma unroll
    for (int i = 0; i < kP; ++i) sum = fma2(y[i], y[i], sum);
    float ss, s1;
    split(sum, ss, s1);
    ss += s1;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float inv = rsqrtf(ss * (1.0f / D) + eps);
    const f32x2 inv2 = pair(inv, inv);
#pragma unroll
    for (int i = 0; i < kP / 2; ++i) {
      const ulonglong2 g = *reinterpret_cast<const ulonglong2 *>(gain + 4 * kLanes * i);
      const ulonglong2 g2 = *reinterpret_cast<const ulonglong2 *>(gain + D / 2 + 4 * kLanes * i);
      x[2 * i] = mul2(x[2 * i], mul2(inv2, g.x));
      x[2 * i + 1] = mul2(x[2 * i + 1], mul2(inv2, g.y));
      y[2 * i] = mul2(y[2 * i], mul2(inv2, g2.x));
      y[2 * i + 1] = mul2(y[2 * i + 1], mul2(inv2, g2.y));
    }
  }
  static __device__ __forceinline__ void floats(const f32x2 (&x)[kP], float (&u)[kN]) {
#pragma unroll
    for (int i = 0; i < kP; ++i) split(x[i], u[2 * i], u[2 * i + 1]);
  }
};

// cos and sin of 2 pi t 2^-64 as turn_cos_sin, to 2^-32: the Taylor terms from y^5 and y^6 on are
// small enough for fp32 (below 2^-8, so their roundings below 2^-32), the others are in 64 bits.
__device__ __forceinline__ void turn_cos_sin(uint64_t t, double &c, double &s) {
  const uint64_t quarter = (t + (1ull << 61)) >> 62;
  const double y = (double)(int64_t)(t - (quarter << 62)) * 3.4061215800865545e-19;  // 2 pi 2^-64
  const double z = y * y;
  const float w = (float)z;
  const float st = 1.0f / 120 + w * (-1.0f / 5040 + w * (1.0f / 362880 + w * (-1.0f / 39916800)));
  const float ct = -1.0f / 720 + w * (1.0f / 40320 + w * (-1.0f / 3628800 + w * (1.0f / 479001600)));
  const double sp = fma(y * z, fma((double)st, z, -1.0 / 6), y);
  const double cp = fma(fma(fma((double)ct, z, 1.0 / 24), z, -0.5), z, 1.0);
  const double a = (quarter & 1) ? sp : cp, b = (quarter & 1) ? cp : sp;
  c = ((quarter + 1) & 2) ? -a : a;
  s = (quarter & 2) ? -b : b;
}
// x to fp32, rounded to odd: towards zero, with the last bit set where that lost something, so that
// a later rounding to fewer bits (twice as few or more) is that of x itself.  (Below 2^-126 fp32 keeps
// fewer bits, and more than the 29 looked at may be lost; that those are all zero takes a sine and
// cosine of few bits, and there is none but 0 and 1, whose products lose nothing.)
__device__ __forceinline__ float to_odd(double x) {
  const uint32_t lost = __double2loint(x) & 0x1fffffffu;
  return __uint_as_float(__float_as_uint(__double2float_rz(x)) | (lost != 0));
}
// A lane's share of a row normed (gain, or nullptr) and rotated (table, or nullptr) in 64 bits.
template <typename M, int D, int kN>
__device__ __forceinline__ void turn_double(float (&u)[kN], float (&v)[kN], const float *gain, float eps, int64_t pos,
                                            const uint64_t *table) {
  double x[kN], y[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = u[i], y[i] = v[i];
  if (gain) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < kN; ++i) ss = fma(x[i], x[i], fma(y[i], y[i], ss));
#pragma unroll
    for (int o = M::kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const double inv = rsqrt(ss * (1.0 / D) + (double)eps);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = i / 4 * 4 * M::kLanes + i % 4;
      x[i] *= inv * (1.0 + (double)gain[at]);
      y[i] *= inv * (1.0 + (double)gain[D / 2 + at]);
    }
  }
  if (table) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      double c, s;
      turn_cos_sin((uint64_t)pos * table[i * M::kLanes], c, s);
      const double w = x[i] * c - y[i] * s;
      y[i] = y[i] * c + x[i] * s;
      x[i] = w;
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) u[i] = to_odd(x[i]), v[i] = to_odd(y[i]);
}

// Kinds of blocks, in this order: of q rows, of k rows (rotated into k_out), or, with kPages,
// of k and v rows on their way into pages (kTurned: there are blocks of the first two kinds).
// An item of the first two is `per` heads of one token: a group of lanes forms the token's
// cosines and sines once for them and keeps the next kAhead rows on their way; an item of the
// third is one head's key and value.  One item a group, so that the rows are on their way
// before anything else is read, and blocks of padding (tokens beyond a sample's count) end at
// once.  Bound by HBM at size and not far from it by instructions (packed fp32 where it can
// be): 32 prefixes of 816 tokens, 9 rows of 512 bytes each, move 241 MB in 42 us; 64 padded ones
// of 2 rows go into e4m3 pages in 21 us (17 with the keys turned in fp32).
template <typename T, typename Pool, int D, bool kTurned, bool kPages>
__global__ void __launch_bounds__(256, kTurned ? 3 : 4) k_rows(const __grid_constant__ RowArgs a) {
  using M = RowMath<T, D, sizeof(T) == 4 || Pool::kScaled>;
  constexpr int kN = M::kN, kP = M::kP, kLanes = M::kLanes, kGroups = 256 / kLanes, kAhead = kTurned ? 3 : 2;
  __shared__ uint64_t sm_turn[D / 2];
  __shared__ __align__(16) float sm_gain[D];  // 1 + gain (in 64 bits: the gain)
  pdl_wait();
  pdl_trigger();
  const bool is_q = kTurned && blockIdx.x < a.q_blocks;
  const bool to_pages = kPages && !is_q;
  const uint32_t block = is_q ? blockIdx.x : blockIdx.x - a.q_blocks;
  const uint32_t item = block * kGroups + threadIdx.x / kLanes;
  const int l0 = threadIdx.x % kLanes * kN;
  const FastDiv &by_items = is_q ? a.by_q : a.by_k;  // items of a token
  const float *gain = is_q ? a.q_gain : a.k_gain;
  const int heads = is_q ? a.hq : a.hk, per = to_pages ? 1 : min(a.per, heads);
  const uint32_t tok = by_items.div(item), b = a.by_t.div(tok);
  const int t = (int)(tok - b * a.T), h0 = (int)(item - tok * by_items.d) * per;
  const bool inside = item < (uint32_t)a.B * a.T * by_items.d;
  const bool kept = inside && (!to_pages || !a.count || t < a.count[b]);

  const RowsPtr &in = is_q ? a.q : a.k;
  const T *src = (const T *)in.data + (kept ? b * in.sb + t * in.st + h0 * in.sh + l0 : 0);
  const int n = kept ? min(per, heads - h0) : 0;
  uint4 lo[kAhead], hi[kAhead];
  auto load = [&](int j, const T *p, bool on) {
    lo[j] = hi[j] = make_uint4(0, 0, 0, 0);
    if (on) {
      lo[j] = *reinterpret_cast<const uint4 *>(p);
      hi[j] = *reinterpret_cast<const uint4 *>(p + D / 2);
    }
  };
  if (to_pages) {
    load(0, src, kept);
    load(1, (const T *)a.v.data + (kept ? b * a.v.sb + t * a.v.st + h0 * a.v.sh + l0 : 0), kept);
    if (a.count && !__syncthreads_or(kept)) return;
  } else {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      load(j, src, j < n);
      src += in.sh;
    }
  }
  const int64_t slot = (int64_t)(a.start && kept ? a.start[b] : 0) + t;
  const int64_t pos = a.positions && kept ? (int64_t)a.positions[tok] : slot;
  const int cell = to_pages && kept ? cache_row(a.pt, b, slot) : -1;  // row of the pools
  if (a.rotate)
    for (int i = threadIdx.x; i < D / 2; i += 256) sm_turn[M::turn_at(i)] = turn_of(a, i);
  if (gain)
    for (int i = threadIdx.x; i < D; i += 256)
      sm_gain[M::gain_at(i)] = Pool::kDouble && to_pages ? gain[i] : 1.0f + gain[i];
  __syncthreads();
  M math;
  if (a.rotate && !(Pool::kDouble && to_pages)) math.turn(pos, sm_turn + l0 / kN);

  if constexpr (kTurned) {
    if (!to_pages) {
      const RowsPtr &to = is_q ? a.q_out : a.k_out;
      T *dst = (T *)to.data + (kept ? b * to.sb + t * to.st + h0 * to.sh + l0 : 0);
      for (int r0 = 0; r0 < per; r0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (r0 + j >= per) break;  // the same for all: the exchanges below are warp-wide
          f32x2 x[kP], y[kP];
          Vec<T>::get(lo[j], x);
          Vec<T>::get(hi[j], y);
          load(j, src, r0 + j + kAhead < n);
          src += in.sh;
          if (gain) M::norm(x, y, sm_gain + l0 / kN * 4, a.eps);
          if (a.rotate) math.rotate(x, y);
          float u[kN], v[kN];
          M::floats(x, u);
          M::floats(y, v);
          if (r0 + j < n) {
            *reinterpret_cast<uint4 *>(dst) = Vec<T>::put(u);
            *reinterpret_cast<uint4 *>(dst + D / 2) = Vec<T>::put(v);
          }
          dst += to.sh;
        }
      }
      return;
    }
  }
  if constexpr (kPages) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // the key, the value
      f32x2 x[kP], y[kP];
      Vec<T>::get(lo[j], x);
      Vec<T>::get(hi[j], y);
      if constexpr (!Pool::kDouble) {
        if (j == 0 && gain) M::norm(x, y, sm_gain + l0 / kN * 4, a.eps);
        if (j == 0 && a.rotate) math.rotate(x, y);
      }
      float u[kN], v[kN];
      M::floats(x, u);
      M::floats(y, v);
      if constexpr (Pool::kDouble)
        if (j == 0 && (gain || a.rotate))
          turn_double<M, D>(u, v, gain ? sm_gain + l0 / kN * 4 : nullptr, a.eps, pos,
                            a.rotate ? sm_turn + l0 / kN : nullptr);
      const PoolPtr &pool = j ? a.vp : a.kp;
      const int64_t at = (int64_t)cell * a.hk + h0;
      if constexpr (Pool::kScaled) {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i) most = max_nan(max_nan(most, fabsf(u[i])), fabsf(v[i]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(kFull, most, o));
        if (cell >= 0) {
          const uint32_t top = __float_as_uint(most);
          const bool finite = top < 0x7f800000u;
          const float scale = finite ? Pool::scale(top) : __uint_as_float(0x7fc00000u);
          uint32_t w[kN / 4] = {}, w2[kN / 4] = {};
          if (finite) {
            Pool::codes(u, scale, w);
            Pool::codes(v, scale, w2);
          }
          uint8_t *dst = (uint8_t *)pool.codes + at * D + l0;
          if constexpr (kN == 8) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(dst + D / 2) = make_uint2(w2[0], w2[1]);
          } else {
            *reinterpret_cast<uint32_t *>(dst) = w[0];
            *reinterpret_cast<uint32_t *>(dst + D / 2) = w2[0];
          }
          if (l0 == 0) pool.scale[at] = scale;
        }
      } else if (cell >= 0) {
        bf16 *dst = (bf16 *)pool.codes + at * D + l0;
        store_bf16(dst, u);
        store_bf16(dst + D / 2, v);
      }
    }
  }
}

// A group of lanes moves a row of keys and the row of values beside it: a lane has kChunks pieces
// of each, 16 bytes of output (8 bf16 or 4 fp32 values) and kLanes pieces apart, so that loads
// and stores are consecutive over the lanes, and kAtOnce such pairs of rows on their way
// together.  Bound by HBM: 18 layers of 16 prefixes of 560 tokens move 321 MB.
template <typename T, typename Pool, int D>
__global__ void __launch_bounds__(256) k_cache_read(const __grid_constant__ ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kN = Vec<T>::kN, kChunks = 2, kLanes = D / kN / kChunks, kAtOnce = 2;
  constexpr int kWords = kN * (Pool::kScaled ? 1 : 2) / 4, kBytes = Pool::kScaled ? 1 : 2;
  const uint32_t items = (uint32_t)a.layers * a.B * a.kv * a.P;  // below 2^31
  const uint32_t step = gridDim.x * (256 / kLanes);
  const int l0 = threadIdx.x % kLanes * kN;
  for (uint32_t first = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes; first < items; first += kAtOnce * step) {
    int64_t at[kAtOnce];  // row of the pools, -1: zeros
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t item = first + u * step;
      at[u] = -1;
      if (item < items) {
        const uint32_t rest = a.by_p.div(item), up = a.by_kv.div(rest), layer = a.by_b.div(up);
        const int h = (int)(rest - up * a.kv), p = (int)(item - rest * a.P), b = (int)(up - layer * a.B);
        int cell = -1;
        if (p < a.lens[b] && (!a.mask || a.mask[(int64_t)b * a.P + p])) cell = cache_row(a.pt, b, p);
        if (a.mask_out && layer == 0 && h == 0 && l0 == 0) a.mask_out[(int64_t)b * a.P + p] = cell >= 0;
        if (cell >= 0) at[u] = (layer * a.layer_rows + cell) * a.kv + h;
      }
    }
    uint32_t w[kAtOnce][2][kChunks][kWords];  // codes of the lane's values
    float scale[kAtOnce][2];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const PoolPtr &pool = i ? a.vp : a.kp;
        const uint8_t *p = (const uint8_t *)pool.codes + (at[u] * D + l0) * kBytes;
        scale[u][i] = 0.0f;
        if constexpr (Pool::kScaled)
          if (at[u] >= 0) scale[u][i] = pool.scale[at[u]];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int j = 0; j < kWords; ++j) w[u][i][c][j] = 0;
          if (at[u] >= 0) {
            const uint8_t *q = p + c * kLanes * kN * kBytes;
            if constexpr (kWords == 4)
              *reinterpret_cast<uint4 *>(w[u][i][c]) = *reinterpret_cast<const uint4 *>(q);
            else if constexpr (kWords == 2)
              *reinterpret_cast<uint2 *>(w[u][i][c]) = *reinterpret_cast<const uint2 *>(q);
            else
              w[u][i][c][0] = *reinterpret_cast<const uint32_t *>(q);
          }
        }
      }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t item = first + u * step;
      if (item >= items) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        T *dst = (T *)(i ? a.v_out : a.k_out) + (int64_t)item * D + l0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint4 out;
          if constexpr (!Pool::kScaled && sizeof(T) == 2) {
            out = *reinterpret_cast<const uint4 *>(w[u][i][c]);  // bits as they are
          } else {
            float x[kN];
            if constexpr (Pool::kScaled) {
              f32x2 y[kN / 2];
#pragma unroll
              for (int j = 0; j < kWords; ++j) Pool::values(w[u][i][c][j], y + 2 * j);
#pragma unroll
              for (int j = 0; j < kN / 2; ++j)
                split(mul2(y[j], pair(scale[u][i], scale[u][i])), x[2 * j], x[2 * j + 1]);
            } else {
#pragma unroll
              for (int j = 0; j < kWords; ++j) {
                x[2 * j] = __uint_as_float(w[u][i][c][j] << 16);
                x[2 * j + 1] = __uint_as_float(w[u][i][c][j] & 0xffff0000u);
              }
            }
            out = Vec<T>::put(x);
          }
          *reinterpret_cast<uint4 *>(dst + c * kLanes * kN) = out;
        }
      }
    }
  }
}

namespace {

template <typename T, typename Pool, int D>
cudaError_t rows_go(RowArgs a, cudaStream_t s) {
  constexpr uint32_t kGroups = 256 / RowMath<T, D, true>::kLanes;
  const uint32_t tokens = (uint32_t)a.B * a.T;
  // Heads of an item: all of a token's (up to 16) where there are enough tokens for two
  // blocks an SM, one where there are few.
  const uint32_t most = (uint32_t)((uint64_t)tokens * (a.hq + a.hk) / (148 * 2 * kGroups));
  a.per = most < 1 ? 1 : most > 16 ? 16 : (int)most;
  auto items = [&](int heads, int per) { return (uint32_t)((heads + per - 1) / per); };
  auto blocks = [&](uint32_t n) { return (tokens * n + kGroups - 1) / kGroups; };
  const uint32_t nq = items(a.hq, a.per), nk = items(a.hk, a.to_cache ? 1 : a.per);
  a.by_q = FastDiv(nq ? nq : 1);
  a.by_k = FastDiv(nk ? nk : 1);
  a.by_t = FastDiv(a.T);
  a.q_blocks = blocks(nq);
  const dim3 grid(a.q_blocks + blocks(nk));
  if (!a.to_cache) return launch_pdl(k_rows<T, PoolBf16, D, true, false>, grid, 256, 0, s, a);
  if (a.hq) return launch_pdl(k_rows<T, Pool, D, true, true>, grid, 256, 0, s, a);
  return launch_pdl(k_rows<T, Pool, D, false, true>, grid, 256, 0, s, a);
}
template <typename T, typename Pool, int D>
cudaError_t read_go(ReadArgs a, cudaStream_t s) {
  a.by_p = FastDiv(a.P);
  a.by_kv = FastDiv(a.kv);
  a.by_b = FastDiv(a.B);
  const int64_t threads = (int64_t)a.layers * a.B * a.kv * a.P * (D / Vec<T>::kN / 2);
  const int64_t blocks = (threads + 255) / 256;
  return launch_pdl(k_cache_read<T, Pool, D>, dim3((unsigned)(blocks < 148 * 16 ? blocks : 148 * 16)), 256, 0, s, a);
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
