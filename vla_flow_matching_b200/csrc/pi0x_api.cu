// C ABI of libpi0x (include/pi0x.h): handle life cycle, weight repack, workspace,
// tensor maps and the per-call kernel sequence of the pi0 Euler loop.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "../../include/pi0x.h"
#include "../../include/pi0x_debug.h"
#include "cache.cuh"
#include "common.cuh"
#include "kernels.cuh"

using namespace pi0x;

namespace {

thread_local std::string g_last_error;

int cuda_fail(cudaError_t e, const char *what) {
  g_last_error = std::string(what) + ": " + cudaGetErrorString(e);
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? PI0X_ENOMEM : PI0X_ECUDA;
}
#define CK(call)                                  \
  do {                                            \
    cudaError_t e_ = (call);                      \
    if (e_ != cudaSuccess) return cuda_fail(e_, #call); \
  } while (0)

// ---- device arena: one cudaMalloc, 1 KiB aligned sub-allocations -------------
struct Arena {
  uint8_t *base = nullptr;
  size_t size = 0, used = 0;
  void *take(size_t bytes) {
    size_t off = (used + 1023) & ~size_t(1023);
    if (off + bytes > size) return nullptr;
    used = off + bytes;
    return base + off;
  }
};
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace

namespace pi0x {

// ---- cuTensorMapEncodeTiled through the runtime's driver entry point ---------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}
// 2-D bf16 K-major map: `rows` x `cols` elements with row pitch `pitch` elements,
// box = 64 columns x box_rows rows, 128-byte swizzle, zero fill out of bounds.
bool make_map(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t pitch, uint32_t box_rows) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {pitch * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pi0x

namespace {

uint16_t f32_to_bf16_bits(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0x7fc0;  // NaN
  u += 0x7fffu + ((u >> 16) & 1u);
  return (uint16_t)(u >> 16);
}
float bf16_bits_to_f32(uint16_t b) {
  uint32_t u = (uint32_t)b << 16;
  float f;
  memcpy(&f, &u, 4);
  return f;
}

struct LayerW {
  float *in_norm, *post_norm;
  void *qkv, *o, *gu, *down;   // activation-type weights
};

struct Workspace {
  int B = 0, P = 0, N = 0, R = 0;
  Arena arena;
  int *nvalid, *vidx;
  float *tvec, *xw, *h, *raw;
  float *part;   // split-KV attention partials (bf16 mode)
  float *gpart;  // split-K GEMM partial tiles (bf16 mode)
  int *counters; // split-K per-tile arrival counters
  float *ss_a, *ss_m;  // fused RMSNorm partial sums of squares, kNormSlots x ss_ld (bf16 mode)
  int ss_ld = 0;
  // persistent small-batch loop (bf16 mode): 64-slot norm sums, stage done-counters
  float *ss64_a = nullptr, *ss64_m = nullptr;
  int *done = nullptr;
  int *mt_cnt = nullptr;  // persistent loop: per (stage, m-tile) partial-tile counters
  float *rope_tab;     // (cos, sin) per position and pair (bf16 mode)
  void *xn, *q, *ks, *vs, *att, *act, *a_emb, *u_emb;
  // host-input staging (device side), allocated lazily
  Arena stage;
  bf16 *st_k = nullptr, *st_v = nullptr;
  uint8_t *st_mask = nullptr;
  float *st_state = nullptr, *st_x = nullptr;
  // tensor maps of the activation operands (bf16 mode)
  ActMap m_xn, m_att, m_act, m_aemb, m_uemb;
};

}  // namespace

struct pi0x_handle {
  pi0x_config cfg;
  int device = 0;
  bool bf16 = true;
  size_t act_bytes = 2;  // element size of activation-type tensors
  Arena warena;
  // weights (device)
  void *state_w, *ain_w, *tin_a, *tin_t, *tout_w;
  float *state_b, *ain_b, *tin_b, *tout_b, *aout_w, *aout_b, *fnorm, *inv_freq;
  // persistent loop (bf16 mode): action_in folded into the action-time MLP input,
  // w_xa = W_in[:, :W] W_action_in (W x A) and tin_b_loop = b_in + W_in[:, :W] b_action_in
  float *w_xa = nullptr, *tin_b_loop = nullptr;
  LayerW layer[kMaxDepth];
  // weight-side tensor maps + tile widths (bf16 mode)
  TcWeight g_tin, g_tout, g_qkv[kMaxDepth], g_o[kMaxDepth], g_gu[kMaxDepth], g_down[kMaxDepth];
  // the persistent loop's copy of the GEMM weights in its unit order (k_tile_weight):
  // tout, then per layer qkv, o, gu, down
  void *wtile = nullptr;
  pi0x::bf16 *wt_tout = nullptr, *wt_qkv[kMaxDepth], *wt_o[kMaxDepth], *wt_gu[kMaxDepth], *wt_down[kMaxDepth];
  int loop_grid = 0;          // CTAs of the persistent loop (0: the loop cannot launch here)
  bool loop_direct = false;   // the cooperative launch could not be captured: launch it directly
  bool loop_off = false;      // pi0x_debug_set_loop(h, 0): small batches take the multi-kernel path
  int dbg_stall = -1;         // next call's loop waits on a counter nothing raises at this stage
  unsigned long long dbg_wait_ns = 0;
  Workspace ws;
  CallPtrs *d_ptrs = nullptr;
  unsigned *d_err = nullptr;
  cudaStream_t last_stream = nullptr;  // stream of the last call (NULL = legacy default)
  bool called = false;
  // solver / convention variant (pi0x_set_variant)
  int time_grid = PI0X_TIME_PI0, x_pred = 0, causal = 0;
  cudaStream_t cap = nullptr;   // capture stream (graphs are launched on the caller's stream)
  struct Graph {
    int B, P, N, prof;
    cudaGraphExec_t exec;
    std::vector<std::pair<int, int>> marks;  // profiling graphs: (class, start event)
  };
  std::vector<Graph> graphs;
  // per-kernel-class event timing (pi0x_profile_*)
  bool prof_on = false;
  std::vector<cudaEvent_t> prof_ev;
  std::vector<std::pair<int, int>> prof_marks;  // marks of the last profiled call
};

namespace {

int validate_config(const pi0x_config *c) {
  if (!c) return PI0X_EINVAL;
  if (c->width != kWidth || c->mlp_dim != kMlp || c->num_heads != kHeads || c->num_kv_heads != 1 ||
      c->head_dim != kHeadDim)
    return PI0X_EUNSUPPORTED;
  if (c->depth < 1 || c->depth > kMaxDepth || c->horizon < 1 || c->horizon > 64 || c->action_dim < 1 ||
      c->action_dim > 64 || c->state_dim < 1 || c->state_dim > 64)
    return PI0X_EINVAL;
  if (c->precision != PI0X_BF16 && c->precision != PI0X_FP32) return PI0X_EINVAL;
  return PI0X_OK;
}

// Read `n` elements of a weight array (host or device memory) as fp32.
int fetch(const void *p, size_t n, int dtype, std::vector<float> &out) {
  if (!p) {
    g_last_error = "null weight pointer";
    return PI0X_EINVAL;
  }
  out.resize(n);
  if (dtype == PI0X_DTYPE_F32) {
    CK(cudaMemcpy(out.data(), p, n * 4, cudaMemcpyDefault));
  } else {
    std::vector<uint16_t> tmp(n);
    CK(cudaMemcpy(tmp.data(), p, n * 2, cudaMemcpyDefault));
    for (size_t i = 0; i < n; ++i) out[i] = bf16_bits_to_f32(tmp[i]);
  }
  return PI0X_OK;
}

// Upload fp32 values as fp32 or as the activation type.
int upload(pi0x_handle *h, const std::vector<float> &v, bool as_act, void **dst) {
  const size_t es = as_act ? h->act_bytes : 4;
  void *d = h->warena.take(v.size() * es);
  if (!d) return PI0X_ENOMEM;
  if (as_act && h->bf16) {
    std::vector<uint16_t> b(v.size());
    for (size_t i = 0; i < v.size(); ++i) b[i] = f32_to_bf16_bits(v[i]);
    CK(cudaMemcpy(d, b.data(), b.size() * 2, cudaMemcpyHostToDevice));
  } else {
    CK(cudaMemcpy(d, v.data(), v.size() * 4, cudaMemcpyHostToDevice));
  }
  *dst = d;
  return PI0X_OK;
}

// Row orders of the fused-epilogue GEMM operands (bf16 mode).  Output column c of
// the GEMM lies in group c/16 of 16 columns.
//  * [q; k; v] (2560 rows): group g holds, for head hd = g/16 (8 = k, 9 = v) and
//    pairs i = 8*(g%16) .. +7, the 8 features i (first half of the head) followed
//    by the 8 features i + 128 they rotate with.
//  * [gate; up] (8192 rows): group g holds gate features 8g..8g+7 then the up
//    features with the same indices.
int qkv_row_source(int c) {
  const int g = c >> 4, w = c & 15;
  return (g >> 4) * kHeadDim + (w >> 3) * (kHeadDim / 2) + (g & 15) * 8 + (w & 7);
}
int gu_row_source(int c) {
  const int g = c >> 4, w = c & 15;
  return (w >> 3) * kMlp + g * 8 + (w & 7);
}
void permute_rows(std::vector<float> &m, size_t cols, int (*src)(int)) {
  const size_t rows = m.size() / cols;
  std::vector<float> out(m.size());
  for (size_t r = 0; r < rows; ++r) memcpy(&out[r * cols], &m[(size_t)src((int)r) * cols], cols * 4);
  m.swap(out);
}

size_t weight_bytes(const pi0x_config &c, size_t es) {
  const size_t W = kWidth;
  size_t act = W * c.state_dim + W * c.action_dim + 2 * W * W + W * W +
               (size_t)c.depth * ((size_t)kQkvDim * W + W * kQDim + 2 * (size_t)kMlp * W + W * kMlp);
  size_t f32 = 4 * W + (size_t)c.action_dim * W + c.action_dim + W + 128 + (size_t)c.depth * 2 * W +
               (size_t)c.action_dim * W + W;  // + the loop's folded action-time MLP input
  return act * es + f32 * 4 + 64 * 1024 * (size_t)(16 + 6 * c.depth);
}

int build_weight_maps(pi0x_handle *h) {
  const int L = h->cfg.depth;
  auto mk = [&](TcWeight &g, const void *w, int N, int K) {
    g.N = N;
    g.K = K;
    g.bn_wide = plan_gemm_tc(1 << 20, N, K).bn;
    return make_map(&g.tm64, w, N, K, K, 64) && make_map(&g.tm_wide, w, N, K, K, g.bn_wide);
  };
  bool ok = mk(h->g_tin, h->tin_a, kWidth, kWidth) && mk(h->g_tout, h->tout_w, kWidth, kWidth);
  for (int l = 0; l < L && ok; ++l) {
    ok = mk(h->g_qkv[l], h->layer[l].qkv, kQkvDim, kWidth) && mk(h->g_o[l], h->layer[l].o, kWidth, kQDim) &&
         mk(h->g_gu[l], h->layer[l].gu, 2 * kMlp, kWidth) && mk(h->g_down[l], h->layer[l].down, kWidth, kMlp);
  }
  if (!ok) {
    g_last_error = "cuTensorMapEncodeTiled failed for a weight operand";
    return PI0X_ECUDA;
  }
  return PI0X_OK;
}

// The persistent loop's copy of every GEMM weight, as 128-row m-tiles of swizzled K-blocks.
int build_loop_weights(pi0x_handle *h) {
  const int L = h->cfg.depth;
  const size_t W = kWidth;
  const size_t per_layer = (size_t)kQkvDim * W + W * kQDim + 2 * (size_t)kMlp * W + W * kMlp;
  CK(cudaMalloc(&h->wtile, 2 * (W * W + (size_t)L * per_layer)));
  bf16 *p = (bf16 *)h->wtile;
  auto tile = [&](const void *src, int kind, bf16 *&dst) -> cudaError_t {
    const LoopGemm g = loop_gemm_plan(kind, h->loop_grid);
    dst = p;
    p += (size_t)g.N * g.K;
    return launch_tile_weight((const bf16 *)src, g.N, g.K, dst, 0);
  };
  CK(tile(h->tout_w, LK_TOUT, h->wt_tout));
  for (int l = 0; l < L; ++l) {
    CK(tile(h->layer[l].qkv, LK_QKV, h->wt_qkv[l]));
    CK(tile(h->layer[l].o, LK_O, h->wt_o[l]));
    CK(tile(h->layer[l].gu, LK_GU, h->wt_gu[l]));
    CK(tile(h->layer[l].down, LK_DOWN, h->wt_down[l]));
  }
  CK(cudaStreamSynchronize(0));
  return PI0X_OK;
}

void drop_graphs(pi0x_handle *h) {
  for (auto &g : h->graphs) cudaGraphExecDestroy(g.exec);
  h->graphs.clear();
}

void free_workspace(Workspace &ws) {
  if (ws.arena.base) cudaFree(ws.arena.base);
  ws.arena = Arena();
  ws.B = ws.P = ws.N = ws.R = 0;
}

int ensure_workspace(pi0x_handle *h, int B, int P, int N) {
  Workspace &ws = h->ws;
  if (ws.arena.base && B <= ws.B && P <= ws.P && N <= ws.N) return PI0X_OK;
  const int nB = B > ws.B ? B : ws.B, nP = P > ws.P ? P : ws.P, nN = N > ws.N ? N : ws.N;
  if (h->called) cudaStreamSynchronize(h->last_stream);
  drop_graphs(h);
  free_workspace(ws);
  const int H = h->cfg.horizon, A = h->cfg.action_dim, L = h->cfg.depth;
  const size_t R = (size_t)nB + (size_t)nB * H;
  const size_t es = h->act_bytes;
  const size_t Rp = round_up(R, 128);  // TMA boxes may cover up to 127 rows past R
  size_t bytes = 0;
  auto add = [&](size_t b) { bytes += round_up(b, 1024) + 1024; };
  add(4 * nB);
  add(4 * (size_t)nB * (nP > 0 ? nP : 1));
  add(4 * (size_t)nN * kWidth);
  add(4 * (size_t)nB * H * A);
  add(4 * Rp * kWidth);
  // fp32 mode: raw GEMM outputs before the RoPE / GeGLU kernels; bf16 mode fuses both
  const size_t raw_floats = h->bf16 ? 0 : Rp * 2 * kMlp;
  add(4 * raw_floats);
  // bf16 split-K GEMMs: split-K is used only while tiles x splits <= 148 (plan_gemm_tc)
  // split-K partial tiles: the multi-kernel GEMMs' and the loop's (one 128 x box_rows
  // tile per unit, at most one unit per CTA and stage)
  const size_t gpart_floats =
      h->bf16 ? std::max((size_t)148 * 128 * 64, (size_t)std::max(h->loop_grid, 148) * 128 * kLoopMaxRows) : 0;
  add(4 * gpart_floats);
  add(4 * 1024);
  const size_t ss_floats = h->bf16 ? (size_t)kNormSlots * Rp : 0;
  add(4 * ss_floats);
  add(4 * ss_floats);
  // positions 0 .. P + H (n_b <= P), 128 (cos, sin) pairs each
  const size_t rope_floats = h->bf16 ? (size_t)(nP + H + 1) * (kHeadDim / 2) * 2 : 0;
  add(4 * rope_floats);
  // xn, att, act and u hold kLoopReps replicas for the persistent loop (bf16 mode)
  const size_t reps = h->bf16 ? kLoopReps : 1;
  add(reps * es * Rp * kWidth);
  // q: the persistent loop stores it per 128-row query tile (up to one partial tile per sample more)
  const size_t q_elems = Rp * kQDim + (h->bf16 ? (size_t)128 * nB * kHeadDim : 0);
  add(es * q_elems);
  add(es * (size_t)L * Rp * kHeadDim);
  add(es * (size_t)L * Rp * kHeadDim);
  add(reps * es * Rp * kQDim);
  add(reps * es * Rp * kMlp);
  add(es * Rp * kWidth);
  add(reps * es * Rp * kWidth);
  // split-KV partials: splits*mtiles*B stays below 96 + 148 CTAs (attn_tc_splits)
  const size_t part_floats = h->bf16 ? (size_t)256 * 128 * (kHeadDim + 2) : 0;
  add(4 * part_floats);
  // persistent loop: 64-slot norm sums (two sets), one done-counter per stage, maps
  const size_t ss64_floats = h->bf16 ? (size_t)kLoopNormSlots * Rp : 0;
  const size_t done_ints = h->bf16 ? (size_t)loop_total_stages(nN, L, 2) : 0;
  add(4 * ss64_floats);
  add(4 * ss64_floats);
  add(4 * done_ints);
  add(4 * done_ints * kLoopMaxMtiles);
  void *base = nullptr;
  CK(cudaMalloc(&base, bytes));
  ws.arena.base = static_cast<uint8_t *>(base);
  ws.arena.size = bytes;
  ws.nvalid = (int *)ws.arena.take(4 * nB);
  ws.vidx = (int *)ws.arena.take(4 * (size_t)nB * (nP > 0 ? nP : 1));
  ws.tvec = (float *)ws.arena.take(4 * (size_t)nN * kWidth);
  ws.xw = (float *)ws.arena.take(4 * (size_t)nB * H * A);
  ws.h = (float *)ws.arena.take(4 * Rp * kWidth);
  ws.raw = (float *)ws.arena.take(4 * raw_floats);
  ws.gpart = (float *)ws.arena.take(4 * gpart_floats);
  ws.counters = (int *)ws.arena.take(4 * 1024);
  ws.ss_a = (float *)ws.arena.take(4 * ss_floats);
  ws.ss_m = (float *)ws.arena.take(4 * ss_floats);
  ws.ss_ld = (int)Rp;
  ws.rope_tab = (float *)ws.arena.take(4 * rope_floats);
  ws.xn = ws.arena.take(reps * es * Rp * kWidth);
  ws.q = ws.arena.take(es * q_elems);
  ws.ks = ws.arena.take(es * (size_t)L * Rp * kHeadDim);
  ws.vs = ws.arena.take(es * (size_t)L * Rp * kHeadDim);
  ws.att = ws.arena.take(reps * es * Rp * kQDim);
  ws.act = ws.arena.take(reps * es * Rp * kMlp);
  ws.a_emb = ws.arena.take(es * Rp * kWidth);
  ws.u_emb = ws.arena.take(reps * es * Rp * kWidth);
  ws.part = (float *)ws.arena.take(4 * part_floats);
  ws.ss64_a = (float *)ws.arena.take(4 * ss64_floats);
  ws.ss64_m = (float *)ws.arena.take(4 * ss64_floats);
  ws.done = (int *)ws.arena.take(4 * done_ints);
  ws.mt_cnt = (int *)ws.arena.take(4 * done_ints * kLoopMaxMtiles);
  CK(cudaMemset(base, 0, bytes));
  ws.B = nB;
  ws.P = nP;
  ws.N = nN;
  ws.R = (int)R;
  if (h->bf16) {
    auto mk = [&](ActMap &m, void *p, int cols) {
      return make_map(&m.m128, p, Rp, cols, cols, 128) && make_map(&m.m64, p, Rp, cols, cols, 64);
    };
    bool ok = mk(ws.m_xn, ws.xn, kWidth) && mk(ws.m_att, ws.att, kQDim) && mk(ws.m_act, ws.act, kMlp) &&
              mk(ws.m_aemb, ws.a_emb, kWidth) && mk(ws.m_uemb, ws.u_emb, kWidth);
    if (!ok) {
      g_last_error = "cuTensorMapEncodeTiled failed for an activation operand";
      return PI0X_ECUDA;
    }

  }
  return PI0X_OK;
}

// Staging buffers for a call of B samples and P slots, cut anew from one allocation, which grows to the
// largest call's bytes and stays (its layout is not kept in a captured graph: calls pass the pointers).
int ensure_stage(pi0x_handle *h, int B, int P) {
  Workspace &ws = h->ws;
  const int L = h->cfg.depth, H = h->cfg.horizon, A = h->cfg.action_dim, S = h->cfg.state_dim;
  const size_t slots = (size_t)B * (P > 0 ? P : 1), kv = (size_t)L * slots * kHeadDim * 2;
  const size_t bytes = 2 * round_up(kv, 1024) + round_up(slots, 1024) + round_up(4 * (size_t)B * S, 1024) +
                       round_up(4 * (size_t)B * H * A, 1024);
  if (bytes > ws.stage.size) {
    if (h->called) cudaStreamSynchronize(h->last_stream);
    if (ws.stage.base) cudaFree(ws.stage.base);
    ws.stage = Arena();
    void *base = nullptr;
    CK(cudaMalloc(&base, bytes));
    ws.stage.base = (uint8_t *)base;
    ws.stage.size = bytes;
  }
  ws.stage.used = 0;
  ws.st_k = (bf16 *)ws.stage.take(kv);
  ws.st_v = (bf16 *)ws.stage.take(kv);
  ws.st_mask = (uint8_t *)ws.stage.take(slots);
  ws.st_state = (float *)ws.stage.take(4 * (size_t)B * S);
  ws.st_x = (float *)ws.stage.take(4 * (size_t)B * H * A);
  return PI0X_OK;
}

bool is_device_ptr(const void *p) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
}

// ---- per-kernel-class timing marks (recorded into the profiling graph) ---------
struct Marker {
  pi0x_handle *h;
  cudaStream_t s;
  int cls = 0;
  void begin(int c) {
    if (!h->prof_on) return;
    cls = c;
    const size_t i = h->prof_marks.size() * 2;
    while (h->prof_ev.size() < i + 2) {
      cudaEvent_t e;
      cudaEventCreate(&e);
      h->prof_ev.push_back(e);
    }
    cudaEventRecord(h->prof_ev[i], s);
  }
  void end() {
    if (!h->prof_on) return;
    const size_t i = h->prof_marks.size() * 2;
    cudaEventRecord(h->prof_ev[i + 1], s);
    h->prof_marks.push_back({cls, (int)i});
  }
};
#define RUN(cls, ...) \
  do {                \
    mk.begin(cls);    \
    __VA_ARGS__;      \
    mk.end();         \
  } while (0)

// ---- the Euler loop -------------------------------------------------------------
template <typename T>
int enqueue_loop(pi0x_handle *h, int B, int P, int N, cudaStream_t s) {
  Marker mk{h, s};
  if (h->prof_on) h->prof_marks.clear();
  Workspace &ws = h->ws;
  const pi0x_config &c = h->cfg;
  const int H = c.horizon, A = c.action_dim, L = c.depth;
  Geo g{B, H, A, c.state_dim, P, B + B * H};
  const int R = g.R, BH = B * H;
  // step sizes: the pi0 grid steps by fp32(-1/N); the linspace grid by the fp32
  // difference of consecutive fp32(k/N)
  const bool linspace = h->time_grid == PI0X_TIME_LINSPACE;
  auto step_dt = [&](int k) -> float {
    if (!linspace) return (float)(-1.0 / (double)N);
    const float t0 = (float)((double)k / (double)N), t1 = (float)((double)(k + 1) / (double)N);
    return t1 - t0;
  };
  const bool tc = h->bf16;
  T *xn = (T *)ws.xn, *q = (T *)ws.q, *att = (T *)ws.att, *act = (T *)ws.act;
  T *aemb = (T *)ws.a_emb, *uemb = (T *)ws.u_emb;
  const size_t kv_stride = (size_t)R * kHeadDim;
  // tcgen05 GEMM with its tile plan for M rows; weight row orders of QKV and gate/up
  // were permuted at create time for the fused RoPE / GeGLU epilogues
  EpiArgs ebase;
  ebase.nvalid = ws.nvalid;
  ebase.inv_freq = h->inv_freq;
  ebase.B = B;
  ebase.H = H;
  ebase.part = ws.gpart;
  ebase.counters = ws.counters;
  ebase.rope_tab = ws.rope_tab;
  auto gemm = [&](int epi, const ActMap &am, const TcWeight &w, int a_row0, int M, const EpiArgs &e) {
    const TcPlan p = plan_gemm_tc(M, w.N, w.K);
    launch_gemm_tc(epi, am.get(p.a_rows), w.map(p.bn), p, a_row0, M, w.N, w.K, e, h->d_err, s);
  };

  // Cross-CTA arrival counters start every call at zero, also after a call whose
  // bounded waits gave up part-way (a memset node of the graph).
  if (tc) CK(cudaMemsetAsync(ws.counters, 0, 4 * 1024, s));
  RUN(PI0X_K_PREP, launch_prep_mask(h->d_ptrs, B, P, ws.nvalid, ws.vidx, s));
  RUN(PI0X_K_PREP, launch_time_vec<T>((const T *)h->tin_t, h->tin_b, N, linspace ? 1 : 0, ws.tvec, s));
  RUN(PI0X_K_PREP, launch_copy_x1(h->d_ptrs, BH * A, ws.xw, s));
  if (tc) RUN(PI0X_K_PREP, launch_rope_table(h->inv_freq, P + H + 1, ws.rope_tab, s));

  for (int k = 0; k < N; ++k) {
    const int step0 = (k == 0);
    const int row0 = step0 ? 0 : B;
    const int M = R - row0;
    if (step0) {
      if (tc)
        RUN(PI0X_K_EMBED, launch_state_embed<T>(h->d_ptrs, (const T *)h->state_w, h->state_b, B, c.state_dim, ws.h,
                                                s, h->layer[0].in_norm, (bf16 *)xn, ws.ss_a, ws.ss_ld));
      else
        RUN(PI0X_K_EMBED, launch_state_embed<T>(h->d_ptrs, (const T *)h->state_w, h->state_b, B, c.state_dim, ws.h,
                                                s));
    }
    RUN(PI0X_K_EMBED, launch_action_in<T, T>(ws.xw, (const T *)h->ain_w, h->ain_b, BH, A, aemb, s));
    GemmOut o_u{uemb, kWidth, 0, ws.tvec + (size_t)k * kWidth};
    GemmOut o_h{ws.h, kWidth, B, h->tout_b};
    if (tc) {
      EpiArgs eu = ebase;
      eu.out_bf16 = (bf16 *)uemb;
      eu.ldo = kWidth;
      eu.vec = ws.tvec + (size_t)k * kWidth;
      RUN(PI0X_K_GEMM, gemm(EPI_VEC_SILU, ws.m_aemb, h->g_tin, 0, BH, eu));
      EpiArgs eh = ebase;
      eh.out_f32 = ws.h;
      eh.ldo = kWidth;
      eh.out_row0 = B;
      eh.vec = h->tout_b;
      eh.gain = h->layer[0].in_norm;   // fused input norm of layer 0
      eh.xn_out = (bf16 *)xn;
      eh.ss_out = ws.ss_a;
      eh.ss_ld = ws.ss_ld;
      RUN(PI0X_K_GEMM, gemm(EPI_BIAS_F32, ws.m_uemb, h->g_tout, 0, BH, eh));
    } else {
      RUN(PI0X_K_GEMM, launch_gemm_simt<float>((const float *)aemb, kWidth, (const float *)h->tin_a, kWidth, BH, kWidth, kWidth,
                              EPI_VEC_SILU, o_u, s));
      RUN(PI0X_K_GEMM, launch_gemm_simt<float>((const float *)uemb, kWidth, (const float *)h->tout_w, kWidth, BH, kWidth, kWidth,
                              EPI_BIAS_F32, o_h, s));
    }
    for (int l = 0; l < L; ++l) {
      const LayerW &lw = h->layer[l];
      T *ks = (T *)ws.ks + (size_t)l * kv_stride, *vs = (T *)ws.vs + (size_t)l * kv_stride;
      if (!tc) RUN(PI0X_K_NORM, launch_rmsnorm<T>(ws.h, row0, M, lw.in_norm, xn, s));
      GemmOut o_raw{ws.raw, kQkvDim, row0, nullptr};
      if (tc) {
        // xn holds h*(1+g_in) from the producer; rstd is applied in this epilogue
        EpiArgs eq = ebase;
        eq.out_row0 = row0;
        eq.q = (bf16 *)q;
        eq.ks = (bf16 *)ks;
        eq.vs = (bf16 *)vs;
        eq.ss_in = ws.ss_a;
        eq.ss_ld = ws.ss_ld;
        RUN(PI0X_K_GEMM, gemm(EPI_QKV_ROPE, ws.m_xn, h->g_qkv[l], row0, M, eq));
      } else {
        RUN(PI0X_K_GEMM, launch_gemm_simt<float>((const float *)xn + (size_t)row0 * kWidth, kWidth, (const float *)lw.qkv, kWidth,
                                M, kQkvDim, kWidth, EPI_STORE_F32, o_raw, s));
        RUN(PI0X_K_ROPE, launch_rope_qkv<T>(ws.raw, row0, M, g, ws.nvalid, h->inv_freq, q, ks, vs, s));
      }
      if (tc) {
        const int splits = attn_tc_splits(g, step0);
        RUN(PI0X_K_ATTN, launch_attention_tc((const bf16 *)q, (const bf16 *)ks, (const bf16 *)vs, h->d_ptrs, l,
                                             l * R, ws.nvalid, ws.vidx, g, step0, h->causal, splits, (bf16 *)att,
                                             ws.part, h->d_err, s));
      } else {
        RUN(PI0X_K_ATTN, launch_attention<T>(q, ks, vs, h->d_ptrs, l, ws.nvalid, ws.vidx, g, step0, h->causal, att,
                                             s));
      }
      GemmOut o_res{ws.h, kWidth, row0, nullptr};
      EpiArgs eres = ebase;
      eres.out_f32 = ws.h;
      eres.ldo = kWidth;
      eres.out_row0 = row0;
      if (tc) {
        EpiArgs eo = eres;  // residual add + fused post-attention norm inputs
        eo.gain = lw.post_norm;
        eo.xn_out = (bf16 *)xn;
        eo.ss_out = ws.ss_m;
        eo.ss_ld = ws.ss_ld;
        RUN(PI0X_K_GEMM, gemm(EPI_RESID_F32, ws.m_att, h->g_o[l], row0, M, eo));
      } else {
        RUN(PI0X_K_GEMM, launch_gemm_simt<float>((const float *)att + (size_t)row0 * kQDim, kQDim, (const float *)lw.o, kQDim, M,
                                kWidth, kQDim, EPI_RESID_F32, o_res, s));
      }
      if (!tc) RUN(PI0X_K_NORM, launch_rmsnorm<T>(ws.h, row0, M, lw.post_norm, xn, s));
      GemmOut o_gu{ws.raw, 2 * kMlp, row0, nullptr};
      if (tc) {
        EpiArgs eg = ebase;
        eg.out_bf16 = (bf16 *)act;
        eg.out_row0 = row0;
        eg.ss_in = ws.ss_m;
        eg.ss_ld = ws.ss_ld;
        RUN(PI0X_K_GEMM, gemm(EPI_GEGLU, ws.m_xn, h->g_gu[l], row0, M, eg));
      } else {
        RUN(PI0X_K_GEMM, launch_gemm_simt<float>((const float *)xn + (size_t)row0 * kWidth, kWidth, (const float *)lw.gu, kWidth, M,
                                2 * kMlp, kWidth, EPI_STORE_F32, o_gu, s));
        RUN(PI0X_K_GEGLU, launch_geglu<T>(ws.raw, row0, M, act, s));
      }
      if (tc) {
        EpiArgs ed = eres;  // residual add + fused input norm of the next layer
        if (l + 1 < L) {
          ed.gain = h->layer[l + 1].in_norm;
          ed.xn_out = (bf16 *)xn;
          ed.ss_out = ws.ss_a;
          ed.ss_ld = ws.ss_ld;
        }
        RUN(PI0X_K_GEMM, gemm(EPI_RESID_F32, ws.m_act, h->g_down[l], row0, M, ed));
      } else {
        RUN(PI0X_K_GEMM, launch_gemm_simt<float>((const float *)act + (size_t)row0 * kMlp, kMlp, (const float *)lw.down, kMlp, M,
                                kWidth, kMlp, EPI_RESID_F32, o_res, s));
      }
    }
    RUN(PI0X_K_FINAL, launch_final_euler(ws.h, g, h->fnorm, h->aout_w, h->aout_b, step_dt(k), ws.xw, h->d_ptrs,
                                         k == N - 1, h->x_pred, s));
  }
  CK(cudaGetLastError());
  return PI0X_OK;
}

// ---- the Euler loop of a small batch: one persistent kernel ------------------------
bool use_loop(const pi0x_handle *h, int B) {
  return h->bf16 && !h->loop_off && h->loop_grid >= kLoopMinGrid && (long)B * (h->cfg.horizon + 1) <= kLoopMaxRows &&
         h->cfg.action_dim <= 32 && h->cfg.action_dim % 4 == 0;
}

int enqueue_persistent(pi0x_handle *h, int B, int P, int N, cudaStream_t s, int stall_stage,
                       unsigned long long wait_ns) {
  Marker mk{h, s};
  if (h->prof_on) h->prof_marks.clear();
  Workspace &ws = h->ws;
  const pi0x_config &c = h->cfg;
  const int H = c.horizon, L = c.depth, R = B + B * H;
  int splits = 1, bps = 1;
  loop_attn_plan(B, H, P, h->loop_grid, splits, bps);
  const int qps0 = (kHeads * (H + 1) + 127) / 128;
  const size_t units0 = (size_t)B * qps0 * splits;
  if (units0 > 256) {
    g_last_error = "persistent loop: too many attention units for the partial buffer";
    return PI0X_EUNSUPPORTED;
  }
  CK(cudaMemsetAsync(ws.counters, 0, 4 * 1024, s));
  CK(cudaMemsetAsync(ws.done, 0, 4 * (size_t)loop_total_stages(N, L, splits), s));
  CK(cudaMemsetAsync(ws.mt_cnt, 0, 4 * (size_t)loop_total_stages(N, L, splits) * kLoopMaxMtiles, s));
  RUN(PI0X_K_PREP, launch_prep_mask(h->d_ptrs, B, P, ws.nvalid, ws.vidx, s));
  RUN(PI0X_K_PREP, launch_time_vec<bf16>((const bf16 *)h->tin_t, h->tin_b_loop, N,
                                         h->time_grid == PI0X_TIME_LINSPACE ? 1 : 0, ws.tvec, s));
  RUN(PI0X_K_PREP, launch_copy_x1(h->d_ptrs, B * H * c.action_dim, ws.xw, s));
  RUN(PI0X_K_PREP, launch_rope_table(h->inv_freq, P + H + 1, ws.rope_tab, s));
  const int rb = (R + 15) / 16 * 16;  // rows of an activation K-block tile: the GEMMs' MMA N
  RUN(PI0X_K_EMBED, launch_state_embed<bf16>(h->d_ptrs, (const bf16 *)h->state_w, h->state_b, B, c.state_dim,
                                             ws.h, s, h->layer[0].in_norm, (bf16 *)ws.xn, ws.ss64_a, ws.ss_ld,
                                             kLoopNormSlots, rb, (int)round_up((size_t)ws.R, 128)));
  LoopArgs a;
  memset(&a, 0, sizeof(a));
  a.B = B;
  a.H = H;
  a.A = c.action_dim;
  a.S = c.state_dim;
  a.P = P;
  a.R = R;
  a.L = L;
  a.N = N;
  a.linspace = h->time_grid == PI0X_TIME_LINSPACE;
  a.x_pred = h->x_pred;
  a.causal = h->causal;
  a.grid = h->loop_grid;
  a.attn_splits = splits;
  a.attn_bps = bps;
  a.box_rows = rb;
  a.rep_rows = (int)round_up((size_t)ws.R, 128);
  a.ss_ld = ws.ss_ld;
  a.debug_stall_stage = stall_stage;
  a.wait_ns = wait_ns;
  a.h = ws.h;
  a.ss_a = ws.ss64_a;
  a.ss_m = ws.ss64_m;
  a.gpart = ws.gpart;
  a.tvec = ws.tvec;
  a.xw = ws.xw;
  a.part_o = ws.part;
  a.part_ml = ws.part + units0 * 128 * kHeadDim;
  a.xn = (bf16 *)ws.xn;
  a.q = (bf16 *)ws.q;
  a.ks = (bf16 *)ws.ks;
  a.vs = (bf16 *)ws.vs;
  a.att = (bf16 *)ws.att;
  a.act = (bf16 *)ws.act;
  a.uemb = (bf16 *)ws.u_emb;
  a.counters = ws.counters;
  a.done = ws.done;
  a.mt_cnt = ws.mt_cnt;
  a.nvalid = ws.nvalid;
  a.vidx = ws.vidx;
  a.rope_tab = ws.rope_tab;
  a.cp = h->d_ptrs;
  a.err = h->d_err;
  a.w_xa = h->w_xa;
  a.tout_b = h->tout_b;
  a.aout_w = h->aout_w;
  a.aout_b = h->aout_b;
  a.fnorm = h->fnorm;
  for (int l = 0; l < L; ++l) {
    a.in_norm[l] = h->layer[l].in_norm;
    a.post_norm[l] = h->layer[l].post_norm;
    a.w_qkv[l] = h->wt_qkv[l];
    a.w_o[l] = h->wt_o[l];
    a.w_gu[l] = h->wt_gu[l];
    a.w_down[l] = h->wt_down[l];
  }
  a.w_tout = h->wt_tout;
  RUN(PI0X_K_LOOP, CK(launch_loop(a, s)));
  CK(cudaGetLastError());
  return PI0X_OK;
}

int enqueue_call(pi0x_handle *h, int B, int P, int N, cudaStream_t s) {
  if (use_loop(h, B)) return enqueue_persistent(h, B, P, N, s, -1, kWaitLimitNs);
  return h->bf16 ? enqueue_loop<bf16>(h, B, P, N, s) : enqueue_loop<float>(h, B, P, N, s);
}

// The whole call (all Euler steps) as one CUDA graph per (B, P, N, profiling),
// captured on the handle's own stream and launched on the caller's.  Every
// caller-owned pointer reaches the kernels through the device table d_ptrs, so a
// graph stays valid across calls; graphs are dropped when the workspace moves.
int get_graph(pi0x_handle *h, int B, int P, int N, cudaGraphExec_t *out) {
  const int prof = 0;
  for (auto &g : h->graphs)
    if (g.B == B && g.P == P && g.N == N && g.prof == prof) {
      *out = g.exec;
      return PI0X_OK;
    }
  cudaGraph_t graph = nullptr;
  CK(cudaStreamBeginCapture(h->cap, cudaStreamCaptureModeThreadLocal));
  int st = enqueue_call(h, B, P, N, h->cap);
  cudaError_t e = cudaStreamEndCapture(h->cap, &graph);
  if (st) {
    if (graph) cudaGraphDestroy(graph);
    return st;
  }
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamEndCapture");
  cudaGraphExec_t exec = nullptr;
  e = cudaGraphInstantiate(&exec, graph, 0);
  cudaGraphDestroy(graph);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGraphInstantiate");
  h->graphs.push_back({B, P, N, prof, exec, {}});
  *out = exec;
  return PI0X_OK;
}

}  // namespace

namespace pi0x {
void set_last_error(const char *msg) { g_last_error = msg; }
}  // namespace pi0x

// ================================ C ABI =====================================
extern "C" {

int pi0x_version(void) { return 100; }

int pi0x_debug_gemm_bf16(const void *A, const void *Bw, int M, int N, int K, float *D, int bn, int splits,
                         void *stream) {
  if (!A || !Bw || !D || M < 1 || N < 1 || K < 64 || K % 64 ||
      (bn != 32 && bn != 64 && bn != 128 && bn != 256) || N % bn || splits < 1 || splits > K / 64 ||
      (splits > 1 && (size_t)((M + 127) / 128) * (N / bn) * splits > 148) || (splits > 1 && bn != 64))
    return PI0X_EINVAL;
  static unsigned *d_err = nullptr;
  static float *d_part = nullptr;
  static int *d_cnt = nullptr;
  if (!d_err) {
    CK(cudaMalloc(&d_err, sizeof(unsigned)));
    CK(cudaMemset(d_err, 0, sizeof(unsigned)));
    CK(cudaMalloc(&d_part, sizeof(float) * 148 * 128 * 64));
    CK(cudaMalloc(&d_cnt, sizeof(int) * 1024));
    CK(cudaMemset(d_cnt, 0, sizeof(int) * 1024));
  }
  TcPlan p;
  p.bn = bn;
  p.splits = splits;
  p.a_rows = (bn == 64 && M <= 64) ? 64 : 128;  // as the sampler plans small GEMMs
  CUtensorMap tmA, tmB;
  if (!make_map(&tmA, A, M, K, K, p.a_rows) || !make_map(&tmB, Bw, N, K, K, bn)) {
    g_last_error = "cuTensorMapEncodeTiled failed";
    return PI0X_ECUDA;
  }
  cudaStream_t s = (cudaStream_t)stream;
  EpiArgs e;
  e.out_f32 = D;
  e.ldo = N;
  e.part = d_part;
  e.counters = d_cnt;
  launch_gemm_tc(EPI_STORE_F32, tmA, tmB, p, 0, M, N, K, e, d_err, s);
  CK(cudaGetLastError());
  CK(cudaStreamSynchronize(s));
  unsigned err = 0;
  CK(cudaMemcpy(&err, d_err, sizeof(err), cudaMemcpyDeviceToHost));
  if (err) {
    cudaMemset(d_err, 0, sizeof(unsigned));
    g_last_error = "device error word 0x" + std::to_string(err);
    return PI0X_ETIMEOUT;
  }
  return PI0X_OK;
}

int pi0x_debug_attention(const void *q, const void *ks, const void *vs, const void *prefix_k,
                         const void *prefix_v, const void *mask, int B, int H, int P, int step0, int impl,
                         void *out, void *stream) {
  if (!q || !ks || !vs || !out || (P > 0 && (!prefix_k || !prefix_v || !mask)) || B < 1 || H < 1 || P < 0 ||
      impl < 0 || impl > 2)
    return PI0X_EINVAL;
  cudaStream_t s = (cudaStream_t)stream;
  Geo g{B, H, 32, 32, P, B + B * H};
  CallPtrs cp;
  memset(&cp, 0, sizeof(cp));
  cp.prefix_k[0] = (const bf16 *)prefix_k;
  cp.prefix_v[0] = (const bf16 *)prefix_v;
  cp.mask = (const uint8_t *)mask;
  if (impl != 0 && !attn_tc_maps(cp, 1, B, P, ks, vs, (uint64_t)g.R)) {
    g_last_error = "pi0x_debug_attention: cuTensorMapEncodeTiled failed (pointers must be 16-byte aligned)";
    return PI0X_EINVAL;
  }
  CallPtrs *d_cp = nullptr;
  int *nvalid = nullptr, *vidx = nullptr;
  float *part = nullptr;
  unsigned *err = nullptr;
  const size_t part_floats = (size_t)256 * 128 * (kHeadDim + 2);
  int st = PI0X_OK;
  cudaError_t e = cudaMalloc(&d_cp, sizeof(cp));
  if (e == cudaSuccess) e = cudaMalloc(&nvalid, 4 * (size_t)B);
  if (e == cudaSuccess) e = cudaMalloc(&vidx, 4 * (size_t)B * (P > 0 ? P : 1));
  if (e == cudaSuccess) e = cudaMalloc(&part, 4 * part_floats);
  if (e == cudaSuccess) e = cudaMalloc(&err, 4);
  if (e == cudaSuccess) e = cudaMemset(err, 0, 4);
  if (e == cudaSuccess) e = cudaMemcpyAsync(d_cp, &cp, sizeof(cp), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) {
    launch_prep_mask(d_cp, B, P, nvalid, vidx, s);
    if (impl == 0) {
      launch_attention<bf16>((const bf16 *)q, (const bf16 *)ks, (const bf16 *)vs, d_cp, 0, nvalid, vidx, g, step0, 0,
                             (bf16 *)out, s);
    } else {
      const int splits = impl == 2 ? 1 : attn_tc_splits(g, step0);
      launch_attention_tc((const bf16 *)q, (const bf16 *)ks, (const bf16 *)vs, d_cp, 0, 0, nvalid, vidx, g, step0, 0,
                          splits, (bf16 *)out, part, err, s);
    }
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) {
    st = cuda_fail(e, "pi0x_debug_attention");
  } else {
    unsigned w = 0;
    cudaMemcpy(&w, err, 4, cudaMemcpyDeviceToHost);
    if (w) {
      g_last_error = "device error word 0x" + std::to_string(w);
      st = PI0X_ETIMEOUT;
    }
  }
  cudaFree(d_cp);
  cudaFree(nvalid);
  cudaFree(vidx);
  cudaFree(part);
  cudaFree(err);
  return st;
}

const char *pi0x_status_string(int st) {
  switch (st) {
    case PI0X_OK: return "ok";
    case PI0X_EINVAL: return "invalid argument";
    case PI0X_EUNSUPPORTED: return "unsupported configuration";
    case PI0X_ENOMEM: return "out of memory";
    case PI0X_ECUDA: return "CUDA error";
    case PI0X_ETIMEOUT: return "device wait timed out";
    case PI0X_EDEVICE: return "device reported an invalid launch";
    default: return "unknown status";
  }
}

const char *pi0x_last_error(void) { return g_last_error.c_str(); }

int pi0x_create(const pi0x_config *cfg, const pi0x_weights *w, pi0x_handle **out) {
  if (!out || !cfg || !w || !w->layers) return PI0X_EINVAL;
  *out = nullptr;
  int st = validate_config(cfg);
  if (st) return st;
  if (w->dtype != PI0X_DTYPE_BF16 && w->dtype != PI0X_DTYPE_F32) return PI0X_EINVAL;
  int dev = 0;
  CK(cudaGetDevice(&dev));
  cudaDeviceProp prop;
  CK(cudaGetDeviceProperties(&prop, dev));
  if (prop.major != 10) {
    g_last_error = "this library is built for sm_100 (B200)";
    return PI0X_EUNSUPPORTED;
  }
  pi0x_handle *h = new (std::nothrow) pi0x_handle();
  if (!h) return PI0X_ENOMEM;
  h->cfg = *cfg;
  h->device = dev;
  h->bf16 = cfg->precision == PI0X_BF16;
  h->act_bytes = h->bf16 ? 2 : 4;
  if (h->bf16 && !get_encode()) {
    g_last_error = "cuTensorMapEncodeTiled unavailable";
    delete h;
    return PI0X_ECUDA;
  }
  const pi0x_config &c = *cfg;
  const size_t W = kWidth;
  auto fail = [&](int code) {
    pi0x_destroy(h);
    return code;
  };
  void *base = nullptr;
  size_t bytes = weight_bytes(c, h->act_bytes);
  cudaError_t e = cudaMalloc(&base, bytes);
  if (e != cudaSuccess) {
    cuda_fail(e, "cudaMalloc(weights)");
    delete h;
    return PI0X_ENOMEM;
  }
  h->warena.base = (uint8_t *)base;
  h->warena.size = bytes;
  std::vector<float> v, v2, v3;
  void *p = nullptr;
#define FETCH(ptr, n, vec)                 \
  do {                                     \
    st = fetch((ptr), (n), w->dtype, vec); \
    if (st) return fail(st);               \
  } while (0)
#define UP(vec, as_act, dst)                  \
  do {                                        \
    st = upload(h, vec, as_act, (void **)&(dst)); \
    if (st) return fail(st);                  \
  } while (0)
  FETCH(w->state_proj_w, W * c.state_dim, v);  UP(v, true, h->state_w);
  FETCH(w->state_proj_b, W, v);                UP(v, false, h->state_b);
  FETCH(w->action_in_w, W * c.action_dim, v);  UP(v, true, h->ain_w);
  std::vector<float> ain_w_host = v;
  FETCH(w->action_in_b, W, v);                 UP(v, false, h->ain_b);
  std::vector<float> ain_b_host = v;
  FETCH(w->time_in_w, W * 2 * W, v);
  v2.resize(W * W);
  v3.resize(W * W);
  for (size_t n = 0; n < W; ++n)
    for (size_t i = 0; i < W; ++i) {
      v2[n * W + i] = v[n * 2 * W + i];       // action half: columns 0..W-1
      v3[n * W + i] = v[n * 2 * W + W + i];   // time half:   columns W..2W-1
    }
  UP(v2, true, h->tin_a);
  UP(v3, true, h->tin_t);
  FETCH(w->time_in_b, W, v);                   UP(v, false, h->tin_b);
  if (h->bf16) {
    // persistent loop: w_xa = W_in[:, :W] W_action_in and b_in + W_in[:, :W] b_action_in,
    // formed in float64 from the bf16 operands the other kernels use, rounded once
    const int A = c.action_dim;
    auto rb = [](float f) { return bf16_bits_to_f32(f32_to_bf16_bits(f)); };
    std::vector<float> wxa((size_t)W * A), tb(W);
    std::vector<double> ain_r(ain_w_host.size()), acc(A);
    for (size_t i = 0; i < ain_w_host.size(); ++i) ain_r[i] = (double)rb(ain_w_host[i]);
    for (size_t n = 0; n < W; ++n) {
      double bacc = (double)v[n];
      for (int j = 0; j < A; ++j) acc[j] = 0.0;
      for (size_t i = 0; i < W; ++i) {
        const double wi = (double)rb(v2[n * W + i]);
        bacc += wi * (double)ain_b_host[i];
        const double *ar = &ain_r[i * A];
        for (int j = 0; j < A; ++j) acc[j] += wi * ar[j];
      }
      for (int j = 0; j < A; ++j) wxa[n * A + j] = (float)acc[j];
      tb[n] = (float)bacc;
    }
    UP(wxa, false, h->w_xa);
    UP(tb, false, h->tin_b_loop);
  }
  FETCH(w->time_out_w, W * W, v);              UP(v, true, h->tout_w);
  FETCH(w->time_out_b, W, v);                  UP(v, false, h->tout_b);
  FETCH(w->action_out_w, W * c.action_dim, v); UP(v, false, h->aout_w);
  FETCH(w->action_out_b, (size_t)c.action_dim, v); UP(v, false, h->aout_b);
  FETCH(w->final_norm_w, W, v);                UP(v, false, h->fnorm);
  for (int l = 0; l < c.depth; ++l) {
    const pi0x_layer_weights &lw = w->layers[l];
    LayerW &d = h->layer[l];
    FETCH(lw.in_norm_w, W, v);   UP(v, false, d.in_norm);
    FETCH(lw.post_norm_w, W, v); UP(v, false, d.post_norm);
    // [q; k; v] rows -> one (2560, 1024) operand
    std::vector<float> qkv;
    FETCH(lw.q_w, (size_t)kQDim * W, v);
    qkv.insert(qkv.end(), v.begin(), v.end());
    FETCH(lw.k_w, (size_t)kHeadDim * W, v);
    qkv.insert(qkv.end(), v.begin(), v.end());
    FETCH(lw.v_w, (size_t)kHeadDim * W, v);
    qkv.insert(qkv.end(), v.begin(), v.end());
    if (h->bf16) permute_rows(qkv, W, qkv_row_source);
    UP(qkv, true, d.qkv);
    FETCH(lw.o_w, W * kQDim, v); UP(v, true, d.o);
    // [gate; up] rows -> one (8192, 1024) operand
    std::vector<float> gu;
    FETCH(lw.gate_w, (size_t)kMlp * W, v);
    gu.insert(gu.end(), v.begin(), v.end());
    FETCH(lw.up_w, (size_t)kMlp * W, v);
    gu.insert(gu.end(), v.begin(), v.end());
    if (h->bf16) permute_rows(gu, W, gu_row_source);
    UP(gu, true, d.gu);
    FETCH(lw.down_w, W * kMlp, v); UP(v, true, d.down);
  }
  // RoPE inverse frequencies: 10000^(-2i/256), evaluated in double, rounded to fp32.
  v.resize(kHeadDim / 2);
  for (int i = 0; i < kHeadDim / 2; ++i) v[i] = (float)std::pow(10000.0, -2.0 * i / (double)kHeadDim);
  UP(v, false, h->inv_freq);
#undef FETCH
#undef UP
  if (h->bf16) {
    st = build_weight_maps(h);
    if (st) return fail(st);
  }
  if (h->bf16) {
    const char *why = nullptr;
    h->loop_grid = loop_max_grid(dev, &why);
    if (why) g_last_error = std::string("persistent small-batch loop unavailable (multi-kernel path used): ") + why;
    if (h->loop_grid >= kLoopMinGrid) {
      st = build_loop_weights(h);
      if (st) return fail(st);
    }
  }
  e = cudaMalloc(&h->d_ptrs, sizeof(CallPtrs));
  if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&h->cap, cudaStreamNonBlocking);
  if (e == cudaSuccess) e = cudaMalloc(&h->d_err, sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(h->d_err, 0, sizeof(unsigned));
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMalloc(handle)"));
  *out = h;
  return PI0X_OK;
}

int pi0x_sample(pi0x_handle *h, const void *const *prefix_k, const void *const *prefix_v,
                const uint8_t *prefix_valid_mask, int B, int P, const float *state, const float *x1, int num_steps,
                float *x0, void *stream) {
  if (!h || !prefix_k || !prefix_v || !state || !x1 || !x0) return PI0X_EINVAL;
  if (P > 0 && !prefix_valid_mask) return PI0X_EINVAL;
  if (B < 1 || B > 4096 || P < 0 || P > 8192 || num_steps < 1 || num_steps > 1024) return PI0X_EINVAL;
  const pi0x_config &c = h->cfg;
  for (int l = 0; l < c.depth; ++l)
    if (P > 0 && (!prefix_k[l] || !prefix_v[l])) return PI0X_EINVAL;
  cudaStream_t s = (cudaStream_t)stream;
  int st = ensure_workspace(h, B, P, num_steps);
  if (st) return st;
  const int H = c.horizon, A = c.action_dim, L = c.depth;
  const size_t kv_elems = (size_t)B * P * kHeadDim;
  CallPtrs cp;
  memset(&cp, 0, sizeof(cp));
  bool host_any = (P > 0 && !is_device_ptr(prefix_valid_mask)) || !is_device_ptr(state) ||
                  !is_device_ptr(x1) || !is_device_ptr(x0);
  for (int l = 0; l < L && !host_any && P > 0; ++l)
    host_any = !is_device_ptr(prefix_k[l]) || !is_device_ptr(prefix_v[l]);
  if (host_any) {
    st = ensure_stage(h, B, P);
    if (st) return st;
  }
  Workspace &ws = h->ws;
  for (int l = 0; l < L; ++l) {
    for (int kvi = 0; kvi < 2; ++kvi) {
      const void *src = kvi ? prefix_v[l] : prefix_k[l];
      const bf16 **dst = kvi ? &cp.prefix_v[l] : &cp.prefix_k[l];
      if (P == 0) {
        *dst = nullptr;
      } else if (is_device_ptr(src)) {
        *dst = (const bf16 *)src;
      } else {
        bf16 *stg = (kvi ? ws.st_v : ws.st_k) + (size_t)l * kv_elems;
        CK(cudaMemcpyAsync(stg, src, kv_elems * 2, cudaMemcpyHostToDevice, s));
        *dst = stg;
      }
    }
  }
  auto stage_in = [&](const void *src, void *stg, size_t bytes, const void **dst) -> int {
    if (is_device_ptr(src)) {
      *dst = src;
    } else {
      CK(cudaMemcpyAsync(stg, src, bytes, cudaMemcpyHostToDevice, s));
      *dst = stg;
    }
    return PI0X_OK;
  };
  const void *tmp;
  if (P > 0) {
    if ((st = stage_in(prefix_valid_mask, ws.st_mask, (size_t)B * P, &tmp))) return st;
    cp.mask = (const uint8_t *)tmp;
  }
  if ((st = stage_in(state, ws.st_state, 4 * (size_t)B * c.state_dim, &tmp))) return st;
  cp.state = (const float *)tmp;
  if ((st = stage_in(x1, ws.st_x, 4 * (size_t)B * H * A, &tmp))) return st;
  cp.x1 = (const float *)tmp;
  const bool x0_host = !is_device_ptr(x0);
  cp.x0 = x0_host ? ws.st_x : x0;  // staged x1 is consumed before x0 is written
  if (h->bf16 && (!attn_tc_maps(cp, L, B, P, ws.ks, ws.vs, (uint64_t)L * (B + (size_t)B * H)) ||
                  (use_loop(h, B) && !loop_attn_maps(cp, L, B, P, ws.ks, ws.vs, (uint64_t)L * (B + (size_t)B * H))))) {
    g_last_error = "pi0x_sample: cuTensorMapEncodeTiled failed for the prefix K/V (pointers must be 16-byte aligned)";
    return PI0X_EINVAL;
  }

  CK(cudaMemcpyAsync(h->d_ptrs, &cp, sizeof(cp), cudaMemcpyHostToDevice, s));
  if (h->prof_on) {
    // Profiled call: direct launches with an event pair around each kernel.  A
    // time-bounded delay kernel holds the stream while the host enqueues the whole
    // call, so the kernels then run back to back as they do in the graph.
    const long n = pi0x_launch_count(h, B, P, num_steps);
    launch_delay_ns((unsigned long long)(20000 * n + 2000000), s);
    st = enqueue_call(h, B, P, num_steps, s);
    if (st) return st;
  } else if (use_loop(h, B) && (h->dbg_stall >= 0 || h->loop_direct)) {
    // direct launches: a test's stalled call, or a driver that cannot capture the
    // cooperative launch into a graph
    const int stall = h->dbg_stall;
    const unsigned long long limit = stall >= 0 ? h->dbg_wait_ns : kWaitLimitNs;
    h->dbg_stall = -1;
    st = enqueue_persistent(h, B, P, num_steps, s, stall, limit);
    if (st) return st;
  } else {
    cudaGraphExec_t exec = nullptr;
    st = get_graph(h, B, P, num_steps, &exec);
    if (st && use_loop(h, B)) {
      // the cooperative launch could not be captured: launch the loop directly from now on
      h->loop_direct = true;
      g_last_error.clear();
      st = enqueue_persistent(h, B, P, num_steps, s, -1, kWaitLimitNs);
      if (st) return st;
    } else {
      if (st) return st;
      CK(cudaGraphLaunch(exec, s));
    }
  }
  if (x0_host) CK(cudaMemcpyAsync(x0, ws.st_x, 4 * (size_t)B * H * A, cudaMemcpyDeviceToHost, s));
  h->last_stream = s;
  h->called = true;
  return PI0X_OK;
}

int pi0x_sample_cache(pi0x_handle *h, const pi0x_cache *cache, int B, int P, const int32_t *page_tab, int max_pages,
                      const int32_t *lens, const uint8_t *mask, const float *state, const float *x1, int num_steps,
                      float *x0, void *stream) {
  if (!h || !lens || !state || !x1 || !x0 || B < 1 || B > 4096 || P < 1 || P > 8192 || num_steps < 1 ||
      num_steps > 1024)
    return PI0X_EINVAL;
  int st = check_cache(cache, 0, 1, B, page_tab, max_pages);
  if (st) return st;
  int dev = -1;
  CK(cudaGetDevice(&dev));
  if (dev != h->device || ((uintptr_t)lens & 3)) {
    g_last_error = "pi0x_sample_cache: another device than the handle's is current, or lens is misaligned";
    return PI0X_EINVAL;
  }
  if (cache->layers != h->cfg.depth || cache->kv_heads != 1 || cache->head_dim != kHeadDim) {
    g_last_error = "pi0x_sample_cache: the cache must have the handle's depth, one kv head and head_dim 256";
    return PI0X_EINVAL;
  }
  const int L = h->cfg.depth;
  st = ensure_workspace(h, B, P, num_steps);  // before the buffers below: it may wait for the last call
  if (!st) st = ensure_stage(h, B, P);
  if (st) return st;
  Workspace &ws = h->ws;
  ReadArgs a = {};
  a.layers = L;
  a.B = B;
  a.kv = 1;
  a.P = P;
  a.layer_rows = (int64_t)cache->num_pages * cache->page_size;
  a.kp = layer_pool(cache, 0, false);
  a.vp = layer_pool(cache, 0, true);
  a.pt = page_table(cache, page_tab, max_pages);
  a.lens = lens;
  a.mask = mask;
  a.k_out = ws.st_k;
  a.v_out = ws.st_v;
  a.mask_out = ws.st_mask;
  CK(launch_cache_read(a, PI0X_DTYPE_BF16, cache->dtype, kHeadDim, (cudaStream_t)stream));
  const void *pk[kMaxDepth], *pv[kMaxDepth];
  for (int l = 0; l < L; ++l) {
    pk[l] = ws.st_k + (size_t)l * B * P * kHeadDim;
    pv[l] = ws.st_v + (size_t)l * B * P * kHeadDim;
  }
  return pi0x_sample(h, pk, pv, ws.st_mask, B, P, state, x1, num_steps, x0, stream);
}

int pi0x_sync_status(pi0x_handle *h) {
  if (!h) return PI0X_EINVAL;
  CK(cudaStreamSynchronize(h->last_stream));
  unsigned err = 0;
  CK(cudaMemcpy(&err, h->d_err, sizeof(err), cudaMemcpyDeviceToHost));
  if (err) {
    cudaMemset(h->d_err, 0, sizeof(unsigned));
    g_last_error = "device error word 0x" + std::to_string(err);
    return (err & (kErrTimeoutProducer | kErrTimeoutMma | kErrTimeoutEpilogue | kErrTimeoutFlag)) ? PI0X_ETIMEOUT
                                                                                                 : PI0X_EDEVICE;
  }
  return PI0X_OK;
}

int pi0x_set_variant(pi0x_handle *h, int time_grid, int x_prediction, int causal_actions) {
  if (!h || (time_grid != PI0X_TIME_PI0 && time_grid != PI0X_TIME_LINSPACE) || x_prediction < 0 ||
      x_prediction > 1 || causal_actions < 0 || causal_actions > 1)
    return PI0X_EINVAL;
  if (time_grid == h->time_grid && x_prediction == h->x_pred && causal_actions == h->causal) return PI0X_OK;
  // the captured graphs bake the variant in: let in-flight calls finish, then drop them
  if (h->called) CK(cudaStreamSynchronize(h->last_stream));
  drop_graphs(h);
  h->time_grid = time_grid;
  h->x_pred = x_prediction;
  h->causal = causal_actions;
  return PI0X_OK;
}

int pi0x_debug_loop_stall(pi0x_handle *h, int stage, unsigned long long wait_ns) {
  if (!h || stage < 0 || wait_ns == 0) return PI0X_EINVAL;
  h->dbg_stall = stage;
  h->dbg_wait_ns = wait_ns;
  return PI0X_OK;
}

int pi0x_uses_loop(const pi0x_handle *h, int B) { return h && B >= 1 && use_loop(h, B) ? 1 : 0; }

int pi0x_debug_set_loop(pi0x_handle *h, int enable) {
  if (!h || enable < 0 || enable > 1) return PI0X_EINVAL;
  if (h->loop_off == !enable) return PI0X_OK;
  if (h->called) CK(cudaStreamSynchronize(h->last_stream));
  drop_graphs(h);
  h->loop_off = !enable;
  return PI0X_OK;
}

int pi0x_profile_enable(pi0x_handle *h, int on) {
  if (!h) return PI0X_EINVAL;
  h->prof_on = on != 0;
  return PI0X_OK;
}

int pi0x_profile_read(pi0x_handle *h, int kclass, long *launches, double *total_ms) {
  if (!h || kclass < 0 || kclass >= PI0X_K_COUNT || !launches || !total_ms) return PI0X_EINVAL;
  if (h->called) CK(cudaStreamSynchronize(h->last_stream));
  long n = 0;
  double ms = 0.0;
  for (auto &m : h->prof_marks) {
    if (m.first != kclass) continue;
    float t = 0.f;
    CK(cudaEventElapsedTime(&t, h->prof_ev[m.second], h->prof_ev[m.second + 1]));
    ++n;
    ms += t;
  }
  *launches = n;
  *total_ms = ms;
  return PI0X_OK;
}

long pi0x_launch_count(const pi0x_handle *h, int B, int P, int num_steps) {
  if (!h || B < 1 || P < 0 || num_steps < 1) return -1;
  const long L = h->cfg.depth, H = h->cfg.horizon;
  // persistent loop: mask prep, time-MLP half, x_1 copy, RoPE table, state embed, loop
  if (use_loop(h, B)) return 6;
  Geo g{B, (int)H, h->cfg.action_dim, h->cfg.state_dim, P, B + B * (int)H};
  long n = 3 + 1 + (h->bf16 ? 1 : 0);  // mask prep, time-MLP half, x_1 copy; state embed; RoPE table
  for (int k = 0; k < num_steps; ++k) {
    // action_in, two time-MLP GEMMs, the layers, final norm + Euler.  fp32 mode: 2 norms,
    // 2 GEMMs + RoPE, attention, O GEMM, GeGLU, down GEMM; bf16 mode fuses norms, RoPE
    // and GeGLU into the GEMMs (4 GEMMs + attention [+ split-KV combine]).
    long per_layer = h->bf16 ? 5 : 9;
    if (h->bf16 && attn_tc_splits(g, k == 0) > 1) per_layer += 1;  // split-KV combine
    n += 3 + L * per_layer + 1;
  }
  return n;
}

void pi0x_destroy(pi0x_handle *h) {
  if (!h) return;
  // the handle's work runs on the stream of its calls (the capture stream only records)
  if (h->called) cudaStreamSynchronize(h->last_stream);
  drop_graphs(h);
  for (cudaEvent_t ev : h->prof_ev) cudaEventDestroy(ev);
  if (h->cap) cudaStreamDestroy(h->cap);
  free_workspace(h->ws);
  if (h->ws.stage.base) cudaFree(h->ws.stage.base);
  if (h->warena.base) cudaFree(h->warena.base);
  if (h->wtile) cudaFree(h->wtile);
  if (h->d_ptrs) cudaFree(h->d_ptrs);
  if (h->d_err) cudaFree(h->d_err);
  delete h;
}

}  // extern "C"
