// Attention of one new token a sample over the paged prefix cache.
//
// s_j = scale * q . k_j, out = sum_j e^(s_j - m) v_j / l, l = sum_j e^(s_j - m), with the
// running maximum m and sum l of one pass over the keys.
//
// What bounds it: every key and value is read once and used by the query heads of its
// kv head, at most 4 * heads / bytes-per-code operations a byte (16 for 8 heads in bf16),
// far below the tensor cores' share, above what the FP32 pipes could do beside the loads.
// So the products go to the tensor cores with the small side, the heads, as the 8
// columns of m16n8k16: S^T = K Q^T takes 16 keys as rows, O^T = V^T P^T 16 dims, and the
// scores' layout transposed 8 x 8 is the weights' layout.  Beside bf16 pages a weight is two
// bf16 values, and its product two.
//
// A warp works through steps of 16 to 64 keys on its own: it copies their rows, whole rows at
// a time, into a ring of three buffers (K, V, K, ...) in shared memory and reads operands
// from there, so that two or three buffers of 8 KB are on their way at any time - 130 to 200
// KB an SM, above what HBM's latency needs - and no barrier stands between warps until their
// keys end.  (Loads straight into the products' registers, without shared memory, measured
// the same for long bf16 keys and slower for 8-bit ones, 57 against 52 us for 24 samples of up to
// 16k: a lane's share of V^T is 16 bytes of four different rows, so a request of 8 lanes covers
// 32-byte pieces of 4 rows.)
#include "cache.cuh"
#include "common.cuh"
#include "kernels.cuh"

#include <math.h>

#include <atomic>
#include <type_traits>

namespace pi0x {

namespace {
constexpr int kWarps = 4;
constexpr int kJoinThreads = 512;
constexpr float kWeightBits = 15.0f;
constexpr int kMaxCluster = 8, kClusterBlocks = 16;
constexpr unsigned kFull = 0xffffffffu;

// Four 8x8 matrices of 16-bit elements, lane i's address the row i % 8 of matrix i / 8.
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// cp.async of 16 bytes, or of 16 zero bytes, whose line is the first to leave the L2: keys and values
// are read once, page numbers, parts and the kernels' own code are wanted again.
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
// The 8x8 matrix of 16-bit elements spread over the warp, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Distributed shared memory: all threads of the cluster, and the address of a peer's copy of a variable.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_peer(const void *p, uint32_t rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// What the lane that keeps key i of 16-key tile u holds.
template <typename V, int N>
__device__ __forceinline__ V of_key(const V (&v)[N], int u, int i) {
  return __shfl_sync(kFull, v[(u * 16) / 32], (u * 16) % 32 + i);
}
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Code types.  halves(): two consecutive codes of a 32-bit word of codes as the 16-bit pair
// of the product; 8-bit codes become fp16, which holds both types' values exactly.
struct CodeBf16 {
  static constexpr int kBytes = 2;
  static constexpr bool kScaled = false;
  // A weight w as the sum of two bf16 values: its upper half, and the rest, rounded (w is then exact
  // to 2^-15).  The rest of a weight above 0 is above 0, so that infinite values stay infinite.
  static __device__ __forceinline__ uint32_t upper(float lo, float hi) {
    return prmt(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
  }
  static __device__ __forceinline__ uint32_t rest(float lo, float hi) {
    constexpr float kLeast = 9.18354962e-41f;  // 2^-133, the least bf16
    auto of = [](float w) {
      return fmaxf(w - __uint_as_float(__float_as_uint(w) & 0xffff0000u), fminf(w, kLeast));
    };
    return pack(of(lo), of(hi));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
struct Code8 {
  static constexpr int kBytes = 1;
  static constexpr bool kScaled = true;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 x = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
struct CodeE4m3 : Code8 {
  static __device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
};
struct CodeInt8 : Code8 {
  // x + 128 as the low bits of an fp16 in [1024, 2048), whose steps are 1; minus 1152.
  static __device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2 bias = __half2(__half_raw{0x6480}, __half_raw{0x6480});  // 1152
    const uint32_t u = w ^ 0x80808080u;
    uint32_t a = prmt(u, 0x64646464u, 0x4140), b = prmt(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), bias), y = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
  }
};

// Shapes of a variant: code type, head_dim, and how many products of 8 columns a unit has (1, or 2
// where a kv head has more than 8 query heads: keys and values are then read and converted
// once for 16; 8 x 10k-20k int8 keys of 128 dims, 20 heads on 2: 31 -> 26 us).
template <typename C, int D, int NT>
struct Shape {
  static constexpr int kHeads = 8 * NT;  // query heads of one kv head that share a pass
  static constexpr int kRowBytes = D * C::kBytes;
  static constexpr int kPitch = kRowBytes + 16;  // 8 rows of a matrix fall into different banks
  // keys a warp takes at once: 16 per product, 32 where rows are short and registers allow it
  // (64 at 128-byte rows with two blocks an SM instead of three: 54 against 48 us for 24 ragged
  // int8 samples)
  static constexpr int kTiles = kRowBytes >= 512 || NT * D >= 512 ? 1 : 2;
  static constexpr int kKeys = 16 * kTiles;
  static constexpr int kBlock = kWarps * kKeys;  // keys of a scheduling block
  static constexpr int kMTiles = D / 16;
  static constexpr int kBuf = kKeys * kPitch;    // bytes of a buffer
  static constexpr int kHeadPitch = D + 4;       // floats: the warps' sums on their way to each other
  static constexpr int kSums = kHeads * kHeadPitch * 4;
  static constexpr int kRing = 3 * kBuf > kSums ? 3 * kBuf : kSums;  // a warp's sums take its ring
  static constexpr int kSmem = kWarps * kRing;
  static constexpr int kBlocksPerSm = kRowBytes >= 256 || NT * D >= 256 ? 2 : 3;  // registers allow no more
  static constexpr int kGrid = 148 * kBlocksPerSm;
};

// Work: units u = (sample, kv head, group of up to 8 or 16 query heads), each of ceil(len/kBlock)
// blocks of keys (at least one).  Two ways to share them out:
//  * kCluster: a cluster of 1 to 8 CTAs takes a unit, its CTAs in turn a block each, and adds
//    up the CTAs' sums through distributed shared memory.  One launch, no workspace, and a CTA
//    knows its first keys before it knows the sample's length, so that page numbers, mask, q
//    and length are on their way together.
//  * else the units are laid end to end and a CTA takes an equal share of all blocks,
//    whichever units they belong to.  A unit inside one CTA is finished there; of a longer one
//    every CTA leaves its part (m, l and the unnormalised sum) in the workspace, and
//    k_attend_join adds them up in order.
// attend_go() has the choice between them.  Split units are listed in the workspace: by unit
// if there are no more units than CTAs, else by the CTA that a unit starts in (each CTA starts
// at most one that goes on).
struct __align__(16) Split {
  int unit;         // -1: none here
  int first, last;  // its CTAs
  int slot;         // the first CTA's part; that of CTA c > first is 2c
};
// n / d, in 32 bits where n fits (a 64-bit division takes several times as long).
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  return (uint64_t)n < (1ull << 32) && (uint64_t)d < (1ull << 32) ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}
template <int N>
struct Look {
  int page[N];
  uint8_t on[N];
};
template <int N>
struct Step {
  int rows[N];           // pool rows, -1: unseen
  unsigned seen[N];      // a bit for each visible key
  float ks[N], vs[N];    // 8-bit codes: scales
};
__device__ __forceinline__ int keys_of(const AttendArgs &a, int b) {
  int64_t n = a.lens[b];
  n = min(n, (int64_t)a.pt.max_pages * a.pt.page_size);
  if (a.mask) n = min(n, (int64_t)a.mask_len);
  return n > 0 ? (int)n : 0;
}
__host__ __device__ inline int head_groups(int heads, int kv, int per) { return (heads / kv + per - 1) / per; }
// Floats of a part: the heads' sums, then their m and l.
template <int D, int NT>
constexpr int kPartFloats = 8 * NT * (D + 2);

}  // namespace

template <typename C, int D, int NT, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, Shape<C, D, NT>::kBlocksPerSm)
    k_attend(const __grid_constant__ AttendArgs a, int cluster) {
  using S = Shape<C, D, NT>;
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t sm_ring[];
  __shared__ __align__(16) uint8_t sm_q[S::kHeads][D * 2 + 16];
  __shared__ float sm_m[kWarps][S::kHeads], sm_l[kWarps][S::kHeads], sm_qf[S::kHeads];
  __shared__ float2 sm_ml[S::kHeads];  // kCluster: this CTA's m and l
  __shared__ int64_t sm_at;
  __shared__ int sm_scan[kWarps], sm_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = a.heads / a.kv, groups = head_groups(a.heads, a.kv, S::kHeads), upb = a.kv * groups;
  auto blocks_of = [](int len) { return max(1, (int)(((uint32_t)len + S::kBlock - 1) / S::kBlock)); };

  // ---- this CTA's blocks [c0, c1), its first sample, and where in the sample's units it starts
  int b, held = 0;  // up to 32 samples: lane i holds the keys of sample i
  int64_t c0, c1, at, share = 1, longer = 0;  // a CTA's blocks; the first `longer` CTAs have one more
  Split *splits = reinterpret_cast<Split *>(a.part);
  float *parts = a.part + gridDim.x * (sizeof(Split) / 4);
  const bool by_unit = (int64_t)a.B * upb <= gridDim.x;
  const int rank = kCluster ? (int)(blockIdx.x % cluster) : 0;
  if constexpr (kCluster) {
    b = blockIdx.x / cluster / upb;
    c0 = c1 = at = 0;
  } else {
    // Up to 256 samples are counted by every warp on its own, more by the block.
    const bool alone = a.B <= 256;
    const int counters = alone ? 32 : kWarps * 32, id = alone ? lane : tid;
    const int per = (a.B + counters - 1) / counters, b_lo = min(a.B, id * per), b_hi = min(a.B, b_lo + per);
    int mine = 0;  // blocks of all samples are below 2^31
    if (a.B <= 32) {
      held = lane < a.B ? keys_of(a, lane) : 0;
      mine = lane < a.B ? blocks_of(held) : 0;
    } else {
#pragma unroll 4
      for (int i = b_lo; i < b_hi; ++i) mine += blocks_of(keys_of(a, i));
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    int before = 0, all = __shfl_sync(kFull, incl, 31);
    if (!alone) {
      if (lane == 31) sm_scan[warp] = incl;
      __syncthreads();
      all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm_scan[w];
        all += sm_scan[w];
      }
    }
    const int64_t total = (int64_t)all * upb, ctas = min((int64_t)gridDim.x, total);  // with at least a block each
    share = quotient(total, ctas);
    longer = total - share * ctas;
    c0 = min(total, blockIdx.x * share + min((int64_t)blockIdx.x, longer));
    c1 = min(total, c0 + share + (blockIdx.x < longer));
    if (!by_unit && tid == 0) splits[blockIdx.x].unit = -1;
    if (c0 >= c1) return;
    int64_t off = (int64_t)(before + incl - mine) * upb;
    const bool here = c0 >= off && c0 < off + (int64_t)mine * upb;
    b = b_lo;
    if (here && a.B > 32)
      for (;; ++b) {
        const int64_t n = (int64_t)blocks_of(keys_of(a, b)) * upb;
        if (c0 < off + n) break;
        off += n;
      }
    at = c0 - off;  // blocks into the sample's units
    if (alone) {
      const int who = __ffs(__ballot_sync(kFull, here)) - 1;
      b = __shfl_sync(kFull, b, who);
      at = __shfl_sync(kFull, at, who);
    } else {
      if (here) sm_b = b, sm_at = at;
      __syncthreads();
      b = sm_b;
      at = sm_at;
    }
  }

  // ---- one segment after another: the blocks of one unit that are this CTA's
  for (int64_t c = c0;;) {
    constexpr int kRegs = (S::kKeys + 31) / 32;  // a lane keeps key i of a step, and key 32 + i of longer ones
    int len = 0, nblk = 1, ub, blk0 = 0, nseg = 0, key_0, key_end, look_end;
    const int hop = kCluster ? cluster * S::kBlock : S::kBlock;  // from a step's keys to the next's
    if constexpr (kCluster) {
      ub = (int)(blockIdx.x / cluster) - b * upb;
      key_0 = rank * S::kBlock + warp * S::kKeys;
      look_end = a.mask ? min(a.mask_len, a.pt.max_pages * a.pt.page_size) : a.pt.max_pages * a.pt.page_size;
    } else {
      len = a.B <= 32 ? __shfl_sync(kFull, held, b) : keys_of(a, b), nblk = blocks_of(len);
      ub = (int)quotient(at, nblk), blk0 = (int)(at - (int64_t)ub * nblk);
      nseg = (int)min((int64_t)(nblk - blk0), c1 - c);
      key_0 = blk0 * S::kBlock + warp * S::kKeys;
      look_end = key_end = (int)min((int64_t)len, ((int64_t)blk0 + nseg) * S::kBlock);
    }
    const int h = ub / groups, h0 = h * group + (ub % groups) * S::kHeads;
    const int nh = min(S::kHeads, group - (ub % groups) * S::kHeads);

    // look() issues the loads of a step's page numbers and mask, settle(), a step later, takes
    // what came.  Unseen keys are not read: their rows are filled with zeros.
    auto look = [&](int key) {
      Look<kRegs> k;
#pragma unroll
      for (int r = 0; r < kRegs; ++r) {
        const int i = r * 32 + lane, p = key + i;
        k.page[r] = -1;
        k.on[r] = 1;
        if (i < S::kKeys && p < look_end) {
          k.page[r] = a.pt.table[(int64_t)b * a.pt.max_pages + a.pt.by_page.div((uint32_t)p)];
          if (a.mask) k.on[r] = a.mask[(int64_t)b * a.mask_len + p];
        }
      }
      return k;
    };
    Look<kRegs> k0 = look(key_0), ahead = look(key_0 + hop);
    if constexpr (kCluster) key_end = len = keys_of(a, b);

    // q: 16 threads a head.  fp16 products take q times a power of two (so that the largest
    // element is in [1, 2)): exact for all that matters of a bf16 q.
#pragma unroll
    for (int n = tid >> 4; n < S::kHeads; n += kWarps * 2) {
      constexpr int E = D / 16;
      const int e0 = (tid & 15) * E;
      uint32_t w[E / 2];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[i] = 0;
      if (n < nh) {
        const bf16 *src = a.q + b * a.q_sb + (h0 + n) * a.q_sh + e0;
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const uint2 v = *reinterpret_cast<const uint2 *>(src + 4 * i);
          w[2 * i] = v.x, w[2 * i + 1] = v.y;
        }
      }
      float factor = a.scale_log2;
      if constexpr (C::kScaled) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        const int e = min(max((int)(top >> 7), 1), 253);  // biased exponent of the largest element
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        factor *= __uint_as_float((uint32_t)e << 23);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
          w[i] = C::pack(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
      }
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        *reinterpret_cast<uint2 *>(&sm_q[n][e0 * 2 + 8 * i]) = make_uint2(w[2 * i], w[2 * i + 1]);
      if ((tid & 15) == 0) sm_qf[n] = factor;
    }
    __syncthreads();

    // Q^T: column (head) 8 nt + g, in the order in which a lane's keys come; in registers where
    // they have room for it.
    constexpr bool kHoldQ = NT * D <= 256;
    auto read_q = [&](int nt, int i, uint32_t (&r)[2]) {
      const uint8_t *p = &sm_q[8 * nt + g][32 * i + (C::kScaled ? 8 : 4) * t];
      r[0] = *reinterpret_cast<const uint32_t *>(p);
      r[1] = *reinterpret_cast<const uint32_t *>(p + (C::kScaled ? 4 : 16));
    };
    uint32_t qb[kHoldQ ? NT : 1][kHoldQ ? S::kMTiles : 1][2];
    float qf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      qf[nt][0] = sm_qf[8 * nt + 2 * t], qf[nt][1] = sm_qf[8 * nt + 2 * t + 1];
      if constexpr (kHoldQ) {
#pragma unroll
        for (int i = 0; i < S::kMTiles; ++i) read_q(nt, i, qb[nt][i]);
      }
    }
    // Product i of the scores: 16 keys and 16 dims against every 8 heads.
    auto score = [&](float (&x)[NT][4], int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (kHoldQ) {
          C::mma(x[nt], a0, a1, a2, a3, qb[nt][i][0], qb[nt][i][1]);
        } else {
          uint32_t q[2];
          read_q(nt, i, q);
          C::mma(x[nt], a0, a1, a2, a3, q[0], q[1]);
        }
      }
    };

    const uint32_t row_bytes = (uint32_t)a.kv * S::kRowBytes;
    const uint8_t *kbase = (const uint8_t *)a.kp.codes + (int64_t)h * S::kRowBytes;
    const uint8_t *vbase = (const uint8_t *)a.vp.codes + (int64_t)h * S::kRowBytes;

    float o[NT][S::kMTiles][4];
    float m[NT][2], l[NT][2];  // of the lane's two columns of every product
    float w[NT][2];            // 8-bit codes: running maximum of s + log2(value scale) - 15
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < S::kMTiles; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
      m[nt][0] = m[nt][1] = w[nt][0] = w[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }

    auto settle = [&](const Look<kRegs> &k, int key) {
      Step<kRegs> st;
#pragma unroll
      for (int r = 0; r < kRegs; ++r) {
        const uint32_t p = key + r * 32 + lane;
        const bool ok = k.on[r] && k.page[r] >= 0 && k.page[r] < a.pt.num_pages && (!kCluster || (int)p < key_end);
        const uint32_t off = p - a.pt.by_page.div(p) * a.pt.page_size;
        st.rows[r] = ok ? k.page[r] * a.pt.page_size + (int)off : -1;
        st.seen[r] = __ballot_sync(kFull, ok);
        st.ks[r] = st.vs[r] = 0.0f;
        if constexpr (C::kScaled)
          if (ok) {
            st.ks[r] = a.kp.scale[(int64_t)st.rows[r] * a.kv + h];
            st.vs[r] = a.vp.scale[(int64_t)st.rows[r] * a.kv + h];
          }
      }
      return st;
    };
    const uint32_t ring = smem_u32(sm_ring) + warp * S::kRing;
    const uint64_t policy = evict_first();
    // A step's rows into a buffer: kRowBytes / 16 lanes a row, consecutive bytes.
    auto copy = [&](const Step<kRegs> &st, const uint8_t *base, int buf) {
      constexpr int kLanes = S::kRowBytes / 16, kAtOnce = 32 / kLanes;
      const uint8_t *src = base + lane % kLanes * 16;
      const uint32_t dst = ring + buf * S::kBuf + lane / kLanes * S::kPitch + lane % kLanes * 16;
#pragma unroll
      for (int i = 0; i < S::kKeys; i += kAtOnce) {
        const int row = __shfl_sync(kFull, st.rows[i / 32], i % 32 + lane / kLanes);
        copy16(dst + i * S::kPitch, src + (uint64_t)(uint32_t)max(row, 0) * row_bytes, row >= 0, policy);
      }
    };
    auto next_buf = [](int buf) { return buf == 2 ? 0 : buf + 1; };

    Step<kRegs> now = settle(k0, key_0);
    int kbuf = 0;
    if (key_0 < key_end) {
      copy(now, kbase, 0);
      cp_async_commit();
      copy(now, vbase, 1);
      cp_async_commit();
    }
    Step<kRegs> next = settle(ahead, key_0 + hop);
    if (key_0 + hop < key_end) copy(next, kbase, 2);
    cp_async_commit();
    ahead = look(key_0 + 2 * hop);
    for (int key = key_0; key < key_end; key += hop) {
      // committed by now: this step's K and V and the next one's K
      cp_async_wait<2>();
      __syncwarp();
      // S^T = K Q^T: rows (keys) g and g + 8, columns (heads) 2t and 2t + 1
      float s[NT][S::kTiles][4];
#pragma unroll
      for (int u = 0; u < S::kTiles; ++u) {
        float x[2][NT][4] = {};  // two chains
        const uint32_t at_k = ring + kbuf * S::kBuf + (u * 16 + lane % 16) * S::kPitch + lane / 16 * 16;
#pragma unroll
        for (int i = 0; i < S::kRowBytes / 32; ++i) {
          uint32_t r[4];
          ldsm(r, at_k + 32 * i);
          if constexpr (C::kScaled) {
            uint32_t a0, a1, a2, a3;
            C::halves(r[0], a0, a2);
            C::halves(r[1], a1, a3);
            score(x[0], 2 * i, a0, a1, a2, a3);
            C::halves(r[2], a0, a2);
            C::halves(r[3], a1, a3);
            score(x[1], 2 * i + 1, a0, a1, a2, a3);
          } else {
            score(x[i & 1], i, r[0], r[1], r[2], r[3]);
          }
        }
        float ka = 1.0f, kb = 1.0f;
        if constexpr (C::kScaled) ka = of_key(now.ks, u, g), kb = of_key(now.ks, u, 8 + g);
        const unsigned seen = now.seen[(u * 16) / 32] >> ((u * 16) % 32 + g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[nt][u][i] = (x[0][nt][i] + x[1][nt][i]) * qf[nt][i & 1];
            if constexpr (C::kScaled) s[nt][u][i] *= i < 2 ? ka : kb;
          }
          if (!(seen & 1)) s[nt][u][0] = s[nt][u][1] = -INFINITY;
          if (!(seen >> 8 & 1)) s[nt][u][2] = s[nt][u][3] = -INFINITY;
        }
      }
      __syncwarp();
      if (key + hop < key_end) copy(next, vbase, kbuf);  // the next step's V takes K's buffer
      cp_async_commit();
      const int vbuf = next_buf(kbuf);

      // online softmax: columns are heads, so a lane's two factors serve its scores and its sums
      float p[NT][S::kTiles][4];
      float lv[kRegs];
      // A bit for each key whose value scale is below 0 (24 ragged int8 samples 44.5 -> 45.0 us).
      unsigned minus[kRegs];
      if constexpr (C::kScaled) {  // (braces: nvcc 12.9 loses code after `if constexpr` without, before a #pragma)
#pragma unroll
        for (int r = 0; r < kRegs; ++r) {
          lv[r] = log2_approx(fabsf(now.vs[r]));
          minus[r] = __ballot_sync(kFull, now.vs[r] < 0.0f);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float n0 = m[nt][0], n1 = m[nt][1];
#pragma unroll
        for (int u = 0; u < S::kTiles; ++u) {
          n0 = fmaxf(n0, fmaxf(s[nt][u][0], s[nt][u][2]));
          n1 = fmaxf(n1, fmaxf(s[nt][u][1], s[nt][u][3]));
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, d));
          n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, d));
        }
        const float z0 = n0 == -INFINITY ? 0.0f : n0, z1 = n1 == -INFINITY ? 0.0f : n1;
        float f0 = ex2_approx(m[nt][0] - z0), f1 = ex2_approx(m[nt][1] - z1);
        l[nt][0] *= f0, l[nt][1] *= f1;
        m[nt][0] = n0, m[nt][1] = n1;
#pragma unroll
        for (int u = 0; u < S::kTiles; ++u) {
          p[nt][u][0] = ex2_approx(s[nt][u][0] - z0), p[nt][u][2] = ex2_approx(s[nt][u][2] - z0);
          p[nt][u][1] = ex2_approx(s[nt][u][1] - z1), p[nt][u][3] = ex2_approx(s[nt][u][3] - z1);
          l[nt][0] += p[nt][u][0] + p[nt][u][2];
          l[nt][1] += p[nt][u][1] + p[nt][u][3];
        }
        if constexpr (C::kScaled) {
          // A value's scale goes into its weight: 2^(s + log2 |scale| - w + 15) with a maximum w of
          // its own, which keeps the fp16 weights in range whatever the scales are: the largest is
          // 2^15, and one of 2^-29 of it still has all 11 bits.  The scale's sign follows below.
          float e0 = w[nt][0] + kWeightBits, e1 = w[nt][1] + kWeightBits;
#pragma unroll
          for (int u = 0; u < S::kTiles; ++u) {
            const float va = of_key(lv, u, g), vb = of_key(lv, u, 8 + g);
            s[nt][u][0] += va, s[nt][u][1] += va, s[nt][u][2] += vb, s[nt][u][3] += vb;
            e0 = fmaxf(e0, fmaxf(s[nt][u][0], s[nt][u][2]));
            e1 = fmaxf(e1, fmaxf(s[nt][u][1], s[nt][u][3]));
          }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            e0 = fmaxf(e0, __shfl_xor_sync(kFull, e0, d));
            e1 = fmaxf(e1, __shfl_xor_sync(kFull, e1, d));
          }
          e0 -= kWeightBits, e1 -= kWeightBits;
          const float y0 = e0 == -INFINITY ? 0.0f : e0, y1 = e1 == -INFINITY ? 0.0f : e1;
          f0 = ex2_approx(w[nt][0] - y0), f1 = ex2_approx(w[nt][1] - y1);
          w[nt][0] = e0, w[nt][1] = e1;
#pragma unroll
          for (int u = 0; u < S::kTiles; ++u) {
            p[nt][u][0] = ex2_approx(s[nt][u][0] - y0), p[nt][u][2] = ex2_approx(s[nt][u][2] - y0);
            p[nt][u][1] = ex2_approx(s[nt][u][1] - y1), p[nt][u][3] = ex2_approx(s[nt][u][3] - y1);
          }
        }
        if (__any_sync(kFull, !(f0 == 1.0f && f1 == 1.0f))) {
#pragma unroll
          for (int i = 0; i < S::kMTiles; ++i)
            o[nt][i][0] *= f0, o[nt][i][1] *= f1, o[nt][i][2] *= f0, o[nt][i][3] *= f1;
        }
      }

      // O^T += V^T P^T: rows are dims (16i + g and 16i + 8 + g in bf16, 16i + 2g and + 1 of 8-bit codes)
      cp_async_wait<2>();
      __syncwarp();
#pragma unroll
      for (int u = 0; u < S::kTiles; ++u) {
        // Weights of one bf16 value each (2^-8) would show in the outputs: they are two, and two
        // products, beside bf16 pages (one robot 7.0 -> 7.2 us, 128 robots 21.1 -> 21.4, 40 x 1000-2000
        // keys 17.7 -> 18.6).  fp16 ones beside 8-bit codes are exact to 2^-11.
        uint32_t b0[NT], b1[NT], r0[NT], r1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float(&w)[4] = p[nt][u];
          if constexpr (C::kScaled) {
            const unsigned below = minus[(u * 16) / 32] >> ((u * 16) % 32 + g);
            b0[nt] = transpose8x8(C::pack(w[0], w[1]) ^ (below & 1 ? 0x80008000u : 0u));
            b1[nt] = transpose8x8(C::pack(w[2], w[3]) ^ (below >> 8 & 1 ? 0x80008000u : 0u));
          } else {
            b0[nt] = transpose8x8(C::upper(w[0], w[1]));
            b1[nt] = transpose8x8(C::upper(w[2], w[3]));
            r0[nt] = transpose8x8(C::rest(w[0], w[1]));
            r1[nt] = transpose8x8(C::rest(w[2], w[3]));
          }
        }
        const int half = lane / 16, odd = lane / 8 % 2;  // bf16: keys, dims; 8-bit codes: dims, keys
        const uint32_t at_v = ring + vbuf * S::kBuf + (u * 16 + (C::kScaled ? odd : half) * 8 + lane % 8) * S::kPitch +
                              (C::kScaled ? half : odd) * 16;
#pragma unroll
        for (int i = 0; i < S::kRowBytes / 32; ++i) {
          uint32_t r[4];
          ldsm_t(r, at_v + 32 * i);
          if constexpr (C::kScaled) {
            // a word: (dim 2g, 2g + 1) of key 2t, then of key 2t + 1
            uint32_t a0, a1, a2, a3;
            C::halves(prmt(r[0], 0, 0x3120), a0, a1);
            C::halves(prmt(r[1], 0, 0x3120), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) C::mma(o[nt][2 * i], a0, a1, a2, a3, b0[nt], b1[nt]);
            C::halves(prmt(r[2], 0, 0x3120), a0, a1);
            C::halves(prmt(r[3], 0, 0x3120), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) C::mma(o[nt][2 * i + 1], a0, a1, a2, a3, b0[nt], b1[nt]);
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              C::mma(o[nt][i], r[0], r[1], r[2], r[3], b0[nt], b1[nt]);
              C::mma(o[nt][i], r[0], r[1], r[2], r[3], r0[nt], r1[nt]);
            }
          }
        }
      }
      __syncwarp();
      now = next;
      next = settle(ahead, key + 2 * hop);
      if (key + 2 * hop < key_end) copy(next, kbase, vbuf);  // the K after the next takes V's buffer
      cp_async_commit();
      ahead = look(key + 3 * hop);
      kbuf = next_buf(vbuf);
    }

    // ---- the warps' sums together
    cp_async_wait<0>();  // the ring is empty: its first bytes take this warp's sums
    __syncwarp();
    float *mine_o = reinterpret_cast<float *>(sm_ring + warp * S::kRing);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[nt][0] += __shfl_xor_sync(kFull, l[nt][0], d);
        l[nt][1] += __shfl_xor_sync(kFull, l[nt][1], d);
      }
      const int n = 8 * nt + 2 * t;
      if (g == 0) {
        sm_m[warp][n] = m[nt][0], sm_m[warp][n + 1] = m[nt][1];
        sm_l[warp][n] = l[nt][0], sm_l[warp][n + 1] = l[nt][1];
      }
      float f0 = 1.0f, f1 = 1.0f;
      if constexpr (C::kScaled) {  // from the weights' maximum back to the scores'
        f0 = m[nt][0] == -INFINITY || w[nt][0] == -INFINITY ? 0.0f : ex2_approx(w[nt][0] - m[nt][0]);
        f1 = m[nt][1] == -INFINITY || w[nt][1] == -INFINITY ? 0.0f : ex2_approx(w[nt][1] - m[nt][1]);
      }
#pragma unroll
      for (int i = 0; i < S::kMTiles; ++i) {
        const float(&x)[4] = o[nt][i];
        float *p0 = mine_o + n * S::kHeadPitch + 16 * i + (C::kScaled ? 2 : 1) * g, *p1 = p0 + S::kHeadPitch;
        if constexpr (C::kScaled) {
          *reinterpret_cast<float2 *>(p0) = make_float2(x[0] * f0, x[2] * f0);
          *reinterpret_cast<float2 *>(p1) = make_float2(x[1] * f1, x[3] * f1);
        } else {
          p0[0] = x[0], p0[8] = x[2];
          p1[0] = x[1], p1[8] = x[3];
        }
      }
    }
    __syncthreads();
    const bool whole = kCluster ? cluster == 1 : nseg == nblk;
    const int slot = 2 * (int)blockIdx.x + (c > c0);
    float *part = parts + (int64_t)slot * kPartFloats<D, NT>;
    auto finish = [&](int n, int d, const float4 &x, float m, float l) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t at_out = ((int64_t)b * a.heads + h0 + n);
      *reinterpret_cast<uint2 *>(a.out + at_out * D + d) =
          make_uint2(CodeBf16::pack(x.x * inv, x.y * inv), CodeBf16::pack(x.z * inv, x.w * inv));
      if (d == 0 && a.lse) a.lse[at_out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    };
#pragma unroll 2
    for (int i = tid; i < nh * (D / 4); i += kWarps * 32) {
      const int n = i / (D / 4), d = i % (D / 4) * 4;
      float mm = sm_m[0][n];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][n]);
      float4 x = make_float4(0, 0, 0, 0);
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm_m[w][n] == -INFINITY ? 0.0f : ex2_approx(sm_m[w][n] - mm);
        const float4 y = *reinterpret_cast<const float4 *>(sm_ring + w * S::kRing + (n * S::kHeadPitch + d) * 4);
        x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
        l += f * sm_l[w][n];
      }
      if (whole) {
        finish(n, d, x, mm, l);
      } else if constexpr (kCluster) {  // over warp 0's sum, which this thread alone has read
        *reinterpret_cast<float4 *>(sm_ring + (n * S::kHeadPitch + d) * 4) = x;
        if (d == 0) sm_ml[n] = make_float2(mm, l);
      } else {
        *reinterpret_cast<float4 *>(part + n * D + d) = x;
        if (d == 0) part[S::kHeads * D + 2 * n] = mm, part[S::kHeads * D + 2 * n + 1] = l;
      }
    }
    if constexpr (kCluster) {
      if (whole) return;
      // Vectors of 4 dims in turn over the CTAs.  (Reading every warp's sums of the peers here,
      // without the step above, measured slower: four times the remote bytes, 27 against 23 us
      // for 128 robots; so did CTAs putting their sums into the shared memory of the one that
      // adds them up, 12.5 against 9.5 us for 32 robots.)
      cluster_sync();
      for (int i = rank * kWarps * 32 + tid; i < nh * (D / 4); i += cluster * kWarps * 32) {
        const int n = i / (D / 4), d = i % (D / 4) * 4;
        float2 ml[kMaxCluster];
        float4 y[kMaxCluster], x = make_float4(0, 0, 0, 0);
        float mm = -INFINITY, l = 0.0f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < cluster) {
            ml[r] = peer_load2(at_peer(&sm_ml[n], r));
            y[r] = peer_load4(at_peer(sm_ring + (n * S::kHeadPitch + d) * 4, r));
          }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < cluster) mm = fmaxf(mm, ml[r].x);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < cluster) {
            const float f = ml[r].x == -INFINITY ? 0.0f : ex2_approx(ml[r].x - mm);
            x.x += f * y[r].x, x.y += f * y[r].y, x.z += f * y[r].z, x.w += f * y[r].w;
            l += f * ml[r].y;
          }
        finish(n, d, x, mm, l);
      }
      cluster_sync();  // nobody leaves while a peer may read from it
      return;
    }
    if (blk0 == 0 && tid == 0) {
      const int unit = b * upb + ub;
      if (!whole) {
        const int64_t end = c + nblk - 1, most = longer * (share + 1);  // its last block; those of the longer CTAs
        const int64_t last = end < most ? quotient(end, share + 1) : longer + quotient(end - most, share);
        splits[by_unit ? unit : blockIdx.x] = Split{unit, (int)blockIdx.x, (int)last, slot};
      } else if (by_unit && gridDim.x > 1) {  // a lone CTA has no workspace and no second kernel
        splits[unit].unit = -1;
      }
    }
    c += nseg;
    if (c >= c1) break;
    at += nseg;
    if (at == (int64_t)nblk * upb) at = 0, ++b;
    __syncthreads();
  }
}

// Adds up the parts of split unit blockIdx.x, in order of the keys.  A part is 8 NT heads x D/4
// vectors; blockIdx.y takes an equal share of them, so that a few units with hundreds of
// parts spread over many SMs.  A share's vectors take `lanes` threads, and the block's groups
// of so many threads take turns at the parts, each with a running maximum of its own, so that
// one barrier is enough.  Bound by the L2's latency: kAhead parts are loaded at once.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const __grid_constant__ AttendArgs a, int grid) {
  pdl_wait();
  pdl_trigger();
  constexpr int kAhead = 8, kStats = 8 * NT * D;
  __shared__ float4 sm_x[kJoinThreads];
  __shared__ float2 sm_ml[kJoinThreads];
  const Split sp = reinterpret_cast<const Split *>(a.part)[blockIdx.x];
  if (sp.unit < 0) return;
  const float *parts = a.part + grid * (sizeof(Split) / 4);
  const int tid = threadIdx.x;
  const int group = a.heads / a.kv, groups = head_groups(a.heads, a.kv, 8 * NT), upb = a.kv * groups;
  const int b = sp.unit / upb, ub = sp.unit % upb, h0 = ub / groups * group + ub % groups * 8 * NT;
  const int nh = min(8 * NT, group - ub % groups * 8 * NT);
  const int count = sp.last - sp.first + 1;
  const int lanes = 2 * NT * D / gridDim.y, turns = kJoinThreads / lanes, turn = tid / lanes;  // 4 <= lanes <= kJoinThreads
  const int v = blockIdx.y * lanes + tid % lanes, head = v / (D / 4);
  const bool mine = head < nh;

  float m = -INFINITY, l = 0.0f;
  float4 x = make_float4(0, 0, 0, 0);
  auto add = [&](float m2, float l2, const float4 &y) {
    const float mm = fmaxf(m, m2), f = m == -INFINITY ? 0.0f : ex2_approx(m - mm),
                f2 = m2 == -INFINITY ? 0.0f : ex2_approx(m2 - mm);
    x.x = f * x.x + f2 * y.x, x.y = f * x.y + f2 * y.y, x.z = f * x.z + f2 * y.z, x.w = f * x.w + f2 * y.w;
    l = f * l + f2 * l2;
    m = mm;
  };
  for (int j0 = turn; mine && j0 < count; j0 += kAhead * turns) {
    float4 y[kAhead];
    float2 ml[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int j = j0 + q * turns;
      if (j < count) {
        const float *part = parts + (int64_t)(j == 0 ? sp.slot : 2 * (sp.first + j)) * kPartFloats<D, NT>;
        y[q] = *reinterpret_cast<const float4 *>(part + 4 * v);
        ml[q] = *reinterpret_cast<const float2 *>(part + kStats + 2 * head);
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      if (j0 + q * turns < count) add(ml[q].x, ml[q].y, y[q]);
  }
  // turns within a warp, then the rest through shared memory
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
    if (o >= lanes) {
      const float m2 = __shfl_xor_sync(kFull, m, o), l2 = __shfl_xor_sync(kFull, l, o);
      const float4 y = make_float4(__shfl_xor_sync(kFull, x.x, o), __shfl_xor_sync(kFull, x.y, o),
                                   __shfl_xor_sync(kFull, x.z, o), __shfl_xor_sync(kFull, x.w, o));
      add(m2, l2, y);
    }
  sm_x[tid] = x;
  sm_ml[tid] = make_float2(m, l);
  __syncthreads();
  if (tid >= lanes || !mine) return;
  const int step = max(lanes, 32);
  for (int j = step; j < kJoinThreads; j += step) m = fmaxf(m, sm_ml[j + tid].x);
  x = make_float4(0, 0, 0, 0);
  l = 0.0f;
#pragma unroll 8
  for (int j = 0; j < kJoinThreads; j += step) {
    const float2 ml = sm_ml[j + tid];
    const float4 y = sm_x[j + tid];
    const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
    x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
    l += f * ml.y;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t at = (int64_t)b * a.heads + h0 + head;
  const int d = v % (D / 4) * 4;
  *reinterpret_cast<uint2 *>(a.out + at * D + d) =
      make_uint2(CodeBf16::pack(x.x * inv, x.y * inv), CodeBf16::pack(x.z * inv, x.w * inv));
  if (d == 0 && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

namespace {

// How a call is shared out (see above).  A cluster's CTAs may get more blocks than an even
// share, if its unit is long for 8 of them or the clusters do not fill whole waves of CTAs; the
// even way pays for its scan, its parts and the second kernel, about as much as 192 KB of keys
// and values in every CTA.  Clusters where that is the larger cost, and only while the even
// share is small: with more work the second kernel hardly shows, and ragged samples keep the CTAs
// of a cluster waiting (lengths are not known here: the page tables' are taken).  GPU time of a
// call in us, clusters / even shares: 1 x 816 bf16 keys of 256 dims 7.2 / 8.6, 1 x 4096
// 14.0 / 8.7, 40 x 1000-2000 18.6 / 20.2, 128 x 600-816 21.7 / 24.1, 256 x 600-816 35.9 /
// 40.8; 512 x 300-700 int8 keys of 64 dims 14.2 / 24.1.
struct Plan {
  int cluster;  // CTAs of a cluster, 0: even shares and a join
  int grid;
};
template <typename C, int D, int NT>
Plan attend_plan(int B, int heads, int kv, int page_size, int max_pages) {
  using S = Shape<C, D, NT>;
  const int64_t blocks = ((int64_t)page_size * max_pages + S::kBlock - 1) / S::kBlock;
  const int64_t units = (int64_t)B * kv * head_groups(heads, kv, S::kHeads);
  int cluster = 1;
  while (cluster < kMaxCluster && cluster < blocks && units * cluster * 2 <= S::kGrid) cluster *= 2;
  const int64_t even = (units * blocks + S::kGrid - 1) / S::kGrid;
  const int64_t waves = (units * cluster + S::kGrid - 1) / S::kGrid, mine = waves * ((blocks + cluster - 1) / cluster);
  const int slack = (192 << 10) / (2 * S::kBlock * S::kRowBytes);
  if (even <= kClusterBlocks && mine <= even + slack) return Plan{cluster, (int)(units * cluster)};
  return Plan{0, (int)(units * blocks < S::kGrid ? units * blocks : S::kGrid)};
}
template <typename C, int D, int NT>
size_t attend_bytes(int B, int heads, int kv, int page_size, int max_pages) {
  const Plan p = attend_plan<C, D, NT>(B, heads, kv, page_size, max_pages);
  return p.cluster || p.grid == 1 ? 0 : p.grid * (sizeof(Split) + 2 * kPartFloats<D, NT> * sizeof(float));
}
// Dynamic shared memory beyond 48 KB has to be asked for once a device and kernel.
template <typename C, int D, int NT, bool kCluster>
cudaError_t allow_smem() {
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && allowed.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(k_attend<C, D, NT, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<C, D, NT>::kSmem);
  if (e == cudaSuccess && dev < 64) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}
template <typename C, int D, int NT>
cudaError_t attend_go(const AttendArgs &a, cudaStream_t s) {
  using S = Shape<C, D, NT>;
  const Plan p = attend_plan<C, D, NT>(a.B, a.heads, a.kv, a.pt.page_size, a.pt.max_pages);
  if (p.cluster) {
    const cudaError_t e = allow_smem<C, D, NT, true>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_attend<C, D, NT, true>, a, p.cluster);
  }
  cudaError_t e = allow_smem<C, D, NT, false>();
  if (e == cudaSuccess) e = launch_pdl(k_attend<C, D, NT, false>, dim3(p.grid), kWarps * 32, S::kSmem, s, a, 0);
  if (e != cudaSuccess || p.grid == 1) return e;  // one CTA: nothing is split
  const int64_t units = (int64_t)a.B * a.kv * head_groups(a.heads, a.kv, S::kHeads);
  const int lists = (int)(units < p.grid ? units : p.grid);
  // Shares of a split unit: about one CTA an SM in all, of 16 vectors or more, of 4 where a unit
  // has 128 parts or more (1 x 4096 keys in 64 parts: 8.7 us with 16 vectors, 10.0 with 4;
  // 1 x 32768 in 256: 14.8 and 14.0).
  const int finest = p.grid / lists >= 128 ? D / 2 : D / 8;
  int shares = 2 * NT * D / kJoinThreads > 1 ? 2 * NT * D / kJoinThreads : 1;
  while (shares < finest && lists * shares * 2 <= 148) shares *= 2;
  return launch_pdl(k_attend_join<D, NT>, dim3(lists, shares), kJoinThreads, 0, s, a, p.grid);
}

#define PI0X_PICK(fn, dtype, dim, group, ...)                                                     \
  auto by_group = [&](auto c, auto d) {                                                           \
    using C = decltype(c);                                                                        \
    return (group) > 8 ? fn<C, d(), 2>(__VA_ARGS__) : fn<C, d(), 1>(__VA_ARGS__);                  \
  };                                                                                              \
  auto by_dim = [&](auto c) {                                                                     \
    return (dim) == 64    ? by_group(c, std::integral_constant<int, 64>())                        \
           : (dim) == 128 ? by_group(c, std::integral_constant<int, 128>())                       \
                          : by_group(c, std::integral_constant<int, 256>());                      \
  };                                                                                              \
  return (dtype) == PI0X_DTYPE_E4M3   ? by_dim(CodeE4m3())                                        \
         : (dtype) == PI0X_DTYPE_INT8 ? by_dim(CodeInt8())                                        \
                                      : by_dim(CodeBf16())

}  // namespace

size_t attend_workspace(int B, int heads, int kv, int head_dim, int pool_dtype, int page_size, int max_pages) {
  PI0X_PICK(attend_bytes, pool_dtype, head_dim, heads / kv, B, heads, kv, page_size, max_pages);
}
cudaError_t launch_attend(const AttendArgs &a, int pool_dtype, int head_dim, cudaStream_t s) {
  PI0X_PICK(attend_go, pool_dtype, head_dim, a.heads / a.kv, a, s);
}

}  // namespace pi0x
