/*
 * pi0x — the pi0 flow-matching denoising loop (action expert) on one B200.
 *
 * C ABI of the shared library libpi0x.so.  Every call returns an int status
 * (PI0X_OK = 0) and never aborts the process; no C++ exception crosses it.
 *
 * The operation is the one defined on the vllm-omni page
 * "vllm_omni/diffusion/models/pi0/modeling_pi0.py": given the per-layer prefix
 * K/V cache of the vision-language prefix, the robot state and the noise chunk
 * x_1, run `num_steps` Euler steps t = 1, 1+dt, ..., -dt (dt = -1/num_steps) of
 *   v_t = action_out_proj(final_norm(expert(embed_suffix(state, x_t, t), prefix_kv)))[last H]
 *   x_t <- x_t + dt * v_t
 * and return x_0 (functions `sample_actions`, `denoise_step`, `embed_suffix`,
 * `_compute_layer_suffix_only` on that page).  The expert is a Gemma decoder
 * ("gemma_300m": width 1024, 8 query heads, 1 KV head, head_dim 256, GeGLU MLP
 * 4096; `get_gemma_config`), RMSNorm x*rsqrt(mean(x^2)+1e-6)*(1+w), rotate-half
 * RoPE with base 10000, attention scale 1/sqrt(head_dim).
 */
#ifndef PI0X_H
#define PI0X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------------- */
enum {
  PI0X_OK = 0,
  PI0X_EINVAL = 1,        /* null pointer, non-positive size, num_steps <= 0, bad config */
  PI0X_EUNSUPPORTED = 2,  /* dims other than the compiled expert dims, no sm_100 device */
  PI0X_ENOMEM = 3,        /* device or host allocation failed */
  PI0X_ECUDA = 4,         /* a CUDA runtime call failed (see pi0x_last_error) */
  PI0X_ETIMEOUT = 5,      /* a bounded device-side wait expired; results are invalid */
  PI0X_EDEVICE = 6        /* a kernel reported an invalid launch configuration */
};

/* ---- precision modes ------------------------------------------------------- */
enum {
  PI0X_BF16 = 0,  /* bf16 weights and GEMM operands, fp32 accumulate, fp32 residual
                     stream, fp32 softmax with probabilities rounded to bf16 */
  PI0X_FP32 = 1   /* every operation in fp32 (no TF32) */
};

/* ---- element types: weight arrays handed to pi0x_create (bf16, f32), and the rows
 * and pages of the paged cache below ------------------------------------------- */
enum {
  PI0X_DTYPE_BF16 = 0,  /* uint16 bf16 bit patterns */
  PI0X_DTYPE_F32 = 1,
  PI0X_DTYPE_E4M3 = 2,  /* cache pages only: 8-bit floats with one fp32 scale a row */
  PI0X_DTYPE_INT8 = 3   /* cache pages only: 8-bit integers with one fp32 scale a row */
};

/* Dimensions.  The library is compiled for width 1024, mlp_dim 4096, 8 query
 * heads, 1 KV head and head_dim 256 (PI0X_EUNSUPPORTED otherwise); depth is
 * 1..32, horizon 1..64, action_dim and state_dim 1..64 (action_dim a
 * multiple of 4, state_dim a multiple of 4). */
typedef struct {
  int width, depth, mlp_dim, num_heads, num_kv_heads, head_dim;
  int horizon, action_dim, state_dim;
  int precision;      /* PI0X_BF16 or PI0X_FP32 */
} pi0x_config;

/* One expert layer, nn.Linear (out, in) row-major layout, no biases (Gemma). */
typedef struct {
  const void *in_norm_w;    /* (width)                      input_layernorm gain */
  const void *q_w;          /* (num_heads*head_dim, width)  */
  const void *k_w;          /* (head_dim, width)            */
  const void *v_w;          /* (head_dim, width)            */
  const void *o_w;          /* (width, num_heads*head_dim)  */
  const void *post_norm_w;  /* (width)                      post_attention_layernorm gain */
  const void *gate_w;       /* (mlp_dim, width)             */
  const void *up_w;         /* (mlp_dim, width)             */
  const void *down_w;       /* (width, mlp_dim)             */
} pi0x_layer_weights;

/* All weights (the pi0 projections of `Pi0ForActionPrediction.__init__` plus
 * the expert).  Pointers may be host or device memory (unified addressing
 * decides); every array is read during pi0x_create only and may be freed
 * afterwards.  `dtype` gives the element type of every array. */
typedef struct {
  const void *state_proj_w, *state_proj_b;    /* (width, state_dim), (width)   */
  const void *action_in_w, *action_in_b;      /* (width, action_dim), (width)  */
  const void *time_in_w, *time_in_b;          /* (width, 2*width), (width): action_time_mlp_in */
  const void *time_out_w, *time_out_b;        /* (width, width), (width): action_time_mlp_out  */
  const void *action_out_w, *action_out_b;    /* (action_dim, width), (action_dim) */
  const void *final_norm_w;                   /* (width) */
  const pi0x_layer_weights *layers;           /* host array of `depth` entries */
  int dtype;                                  /* PI0X_DTYPE_BF16 or PI0X_DTYPE_F32 */
} pi0x_weights;

typedef struct pi0x_handle pi0x_handle;

/* Create a sampler on the current CUDA device: validates `cfg`, copies and
 * repacks the weights into device memory owned by the handle.  On success
 * *out receives the handle (destroy with pi0x_destroy).  Synchronous. */
int pi0x_create(const pi0x_config *cfg, const pi0x_weights *weights, pi0x_handle **out);

/* Run the whole num_steps Euler loop (`sample_actions` minus the prefix pass).
 *
 *  prefix_k, prefix_v : HOST arrays of `depth` pointers; entry l points to the
 *                       layer-l prefix key/value cache, shape (B, 1, P, head_dim),
 *                       bf16, contiguous, already rotated (post-RoPE), as the
 *                       prefix pass of the page caches them.
 *  prefix_valid_mask  : (B, P) uint8, nonzero = valid prefix token (may be NULL
 *                       when P == 0).  Any pattern is allowed (holes,
 *                       all-zero rows).  Suffix
 *                       positions continue at the per-sample count of valid
 *                       prefix tokens.
 *  B, P               : batch (1..4096) and prefix length (0..8192).
 *  state              : (B, state_dim) float32.
 *  x1                 : (B, horizon, action_dim) float32, the t = 1 noise.
 *  num_steps          : Euler steps (1..1024).
 *  x0                 : (B, horizon, action_dim) float32 output; may alias x1.
 *  stream             : a cudaStream_t (NULL = legacy default stream).
 *
 * Every array may live in device memory or host memory (pinned or pageable);
 * host arrays are staged through handle-owned device buffers and x0 is copied
 * back, all on `stream`.  The call enqueues its work on `stream` and returns:
 * device inputs must stay valid and x0 must not be read until the stream
 * reaches the end of the call.  The library keeps no caller pointer after it
 * returns.  Calls on one handle must not overlap on the device (they share the
 * handle's workspace); use one handle per concurrent stream.
 * Errors: PI0X_EINVAL for null pointers or sizes out of range (num_steps <= 0
 * is rejected because dt = -1/num_steps), PI0X_ENOMEM, PI0X_ECUDA. */
int pi0x_sample(pi0x_handle *h, const void *const *prefix_k, const void *const *prefix_v,
                const uint8_t *prefix_valid_mask, int B, int P, const float *state,
                const float *x1, int num_steps, float *x0, void *stream);

/* Wait for all work of the handle's last call and read the device error word.
 * Returns PI0X_OK, PI0X_ETIMEOUT (a bounded device wait gave up; the outputs
 * of that call are invalid), PI0X_EDEVICE or PI0X_ECUDA.  Clears the word. */
int pi0x_sync_status(pi0x_handle *h);

/* ---- paged prefix cache --------------------------------------------------------
 * For inference, as the rest of the library: no call has a backward pass.
 * pi0x_sample takes the prefix keys and values as contiguous bf16 tensors.  The
 * calls below make and hold them: per-head norm and rotation of queries and keys
 * (pi0x_qk_norm_rope), a cache in pages shared by many samples, in bf16 or 8 bits
 * (pi0x_cache_write, pi0x_cache_read), attention of one new token a sample over it
 * (pi0x_cache_attention) and the denoising loop on it (pi0x_sample_cache).
 *
 * Every pointer below is device memory of the current device, of its elements'
 * alignment at least.  The calls enqueue
 * their work on `stream` and return; they allocate nothing, keep nothing of a call's data, and
 * may be captured into a CUDA graph (pi0x_sample_cache excepted).  What can be seen from the host is checked
 * (PI0X_EINVAL, PI0X_EUNSUPPORTED); what lies in device memory is bounded by the
 * kernels: a page table entry outside [0, num_pages) is a page without keys (nothing
 * is read or written there), a length below 0 counts as 0 and one above the table's
 * max_pages * page_size as that. */

/* Pages of `page_size` rows for each of `layers` layers.  A row is one position's
 * (kv_heads, head_dim) keys or values; in the 8-bit types every (row, head) has an
 * fp32 scale and stands for code * scale.  1 <= kv_heads <= 65535; head_dim 64, 128 or 256;
 * layers >= 1; layers * num_pages * page_size < 2^31; a page table has fewer than 2^31 -
 * 4096 slots. */
typedef struct {
  void *k, *v;               /* (layers, num_pages, page_size, kv_heads, head_dim), 16-byte aligned */
  float *k_scale, *v_scale;  /* (layers, num_pages, page_size, kv_heads); NULL for bf16 pages */
  int layers, num_pages, page_size, kv_heads, head_dim;
  int dtype;                 /* PI0X_DTYPE_BF16, PI0X_DTYPE_E4M3 or PI0X_DTYPE_INT8 */
} pi0x_cache;

/* Rows of `head_dim` contiguous elements at data + b * batch_stride + t * token_stride
 * + h * head_stride (elements); data and the strides are multiples of 16 bytes.
 * An input's rows may share memory (strides of 0), an output's may not: of dimensions
 * above 1 each stride, from the least on, is beyond all that the lesser ones span. */
typedef struct {
  void *data;
  int64_t batch_stride, token_stride, head_stride;
} pi0x_rows;

/* What is done to queries and keys: y = x * rsqrt(mean(x^2) + eps) * (1 + gain) over
 * each head's row where a gain is given, then the rotate-half rotation of the pairs
 * (i, i + head_dim/2) by pos * rope_base^(-2i/head_dim) where rope_base > 0 (1 or
 * more).  At every 32-bit position the angle is exact to 1.5 * 2^-32 of a turn for
 * bases of 100 and more (4.3 * 2^-32 for all); the rest is fp32 (sines and cosines of
 * bf16 rows that stay bf16 to 2^-20; 64 bits for keys on their way into e4m3 pages),
 * rounded once to the output's type.  Squares are summed in fp32: a row of values of
 * 2^60 and more may leave its norm as zeros. */
typedef struct {
  const float *q_gain, *k_gain;  /* (head_dim) fp32; NULL: no norm */
  const int32_t *positions;      /* (B, T); NULL: start[b] + t */
  float eps;                     /* > 0 where a gain is given */
  float rope_base;               /* 0: no rotation */
} pi0x_rotation;

/* Norm and rotate q (B, T, q_heads, head_dim) into q_out and k (B, T, k_heads,
 * head_dim) into k_out, all of `dtype` (PI0X_DTYPE_BF16 or PI0X_DTYPE_F32).  Either
 * may be left out (0 heads, NULL); an output may be its input's memory, row for row.
 * start: (B) first position of each sample (NULL: 0), not used with rot->positions. */
int pi0x_qk_norm_rope(int dtype, int B, int T, int q_heads, int k_heads, int head_dim, const pi0x_rows *q,
                      const pi0x_rows *k, const int32_t *start, const pi0x_rotation *rot, const pi0x_rows *q_out,
                      const pi0x_rows *k_out, void *stream);

/* Write the keys and values of T new tokens a sample, k and v (B, T, kv_heads,
 * head_dim) of `dtype` (bf16 or f32), into the pages of `layer`.  Token t of sample b
 * goes to slot pos = start[b] + t: row pos % page_size of page
 * page_table[b * max_pages + pos / page_size].  A token at t >= count[b] (count NULL:
 * T), at a negative slot or past the table is left out, and so is one whose page is
 * outside the pool; slots without a new token keep what they hold.  Samples that
 * share a page must not write the same slot.
 *   rot != NULL: keys are normed and rotated first, and so is q (B, T, q_heads,
 * head_dim), if given, into q_out - every (b, t) of it, whatever count says.
 *   8-bit pages: int8 codes are rn(x / scale) with scale = max|x| / 127 of the row,
 * e4m3 codes with the least power of two that brings max|x| within 448 (neither below
 * 2^-126).  A row with a NaN or an infinity gets a NaN scale: it stands for NaN. */
int pi0x_cache_write(const pi0x_cache *cache, int layer, int dtype, int B, int T, const pi0x_rows *k,
                     const pi0x_rows *v, const int32_t *page_table, int max_pages, const int32_t *start,
                     const int32_t *count, const pi0x_rotation *rot, int q_heads, const pi0x_rows *q,
                     const pi0x_rows *q_out, void *stream);

/* Read slots 0..P-1 of every sample for layers [layer0, layer0 + layers) into
 * contiguous k_out, v_out (layers, B, kv_heads, P, head_dim) of `dtype` (bf16 or
 * f32): with one kv head, the layout pi0x_sample takes layer by layer.  Slot p holds
 * a key if p < lens[b], its page is inside the pool and mask (B, P) uint8 (NULL: all)
 * is nonzero there; the others are not read and come out as zeros.  mask_out (B, P)
 * uint8 (may be NULL) gets 1 where there is a key, else 0. */
int pi0x_cache_read(const pi0x_cache *cache, int layer0, int layers, int B, int P, const int32_t *page_table,
                    int max_pages, const int32_t *lens, const uint8_t *mask, int dtype, void *k_out, void *v_out,
                    uint8_t *mask_out, void *stream);

/* Attention of one new token a sample over the pages of `layer`: q (B, q_heads,
 * head_dim) bf16 (q->token_stride is not used), query head h reads kv head
 * h / (q_heads / kv_heads); q_heads is a multiple of kv_heads, and B and q_heads are at most
 * 65535, B * q_heads and all tables' slots / 64 below 2^31.  Keys are the slots p <
 * lens[b] whose page is inside the pool and, with mask (B, mask_len) uint8, p <
 * mask_len and mask[b][p] nonzero; nothing else is read.
 *   out (B, q_heads, head_dim) bf16 = softmax(scale * q . k) v; lse (B, q_heads) fp32
 * (may be NULL) = log of the sum of exp(scale * q . k).  A sample without a key gets
 * zeros and -inf.  Sums and softmax statistics are fp32.  Probabilities go into the
 * matrix product as two bf16 values each (exact to 2^-15) beside bf16 pages, as fp16
 * (2^-11) beside 8-bit ones; there q is fp16 after a division by a power of two, so an
 * element far below the head's largest is exact to 2^-25 of that one.  The result of a
 * call does not depend on timing.
 *   workspace: pi0x_cache_attention_workspace() bytes, 16-byte aligned, used by this
 * call only while it runs: calls that may overlap need one each. */
int pi0x_cache_attention(const pi0x_cache *cache, int layer, int B, int q_heads, const pi0x_rows *q,
                         const int32_t *page_table, int max_pages, const int32_t *lens, const uint8_t *mask,
                         int mask_len, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                         void *stream);

/* Bytes of workspace a pi0x_cache_attention call of these sizes needs (0 if none, or
 * if the sizes are refused). */
size_t pi0x_cache_attention_workspace(const pi0x_cache *cache, int B, int q_heads, int max_pages);

/* pi0x_sample with the prefix K/V of a cache: reads slots 0..P-1 of all layers, as
 * pi0x_cache_read with `lens` and `mask` does, into buffers of the handle and runs the
 * loop on them.  The cache has the handle's depth, one kv head and head_dim 256.
 * state, x1, x0 as for pi0x_sample (device or host); page_table, lens and mask are
 * device memory. */
int pi0x_sample_cache(pi0x_handle *h, const pi0x_cache *cache, int B, int P, const int32_t *page_table,
                      int max_pages, const int32_t *lens, const uint8_t *mask, const float *state, const float *x1,
                      int num_steps, float *x0, void *stream);

/* ---- solver / convention variants --------------------------------------------
 * The default is pi0's own loop (`sample_actions` / `denoise_step` on the
 * vllm-omni pi0 page): t from 1 (noise) to 0 with dt = -1/N, the out-projection
 * is the velocity, action tokens see each other.  pi0x_set_variant selects the
 * conventions of the Wall-X flow-matching sampler instead, each independently:
 *  - time_grid PI0X_TIME_LINSPACE: t from 0 (noise) to 1 on torch.linspace(0, 1,
 *    N+1) integrated with a fixed-grid Euler step (its odeint call), taken as
 *    t_k = fp32(k/N) correctly rounded, step size fp32(t_{k+1} - t_k);
 *  - x_prediction = 1: the out-projection is the clean action x_hat and the
 *    velocity is x_hat - x_1 (its use_x_pred branch: prediction minus noise);
 *  - causal_actions = 1: action token i sees the prefix, the state and actions
 *    0..i only (its causal_action_attention_mask, a lower-triangular suffix block).
 * The setting applies to later pi0x_sample calls on the handle; changing it
 * waits for the handle's last call and drops the cached graphs.
 * Errors: PI0X_EINVAL for a null handle or a value out of range. */
enum {
  PI0X_TIME_PI0 = 0,      /* t: 1 -> 0, dt = -1/N */
  PI0X_TIME_LINSPACE = 1  /* t: 0 -> 1 on fp32(k/N) */
};
int pi0x_set_variant(pi0x_handle *h, int time_grid, int x_prediction, int causal_actions);

/* Number of kernels one pi0x_sample(B, P, num_steps) call launches (its own
 * kernels only, not memory copies), or -1 for invalid arguments.  In bf16 mode a
 * batch whose rows fit one 128-row tile (B * (horizon + 1) <= 128) runs every
 * Euler step in one persistent kernel after five small set-up kernels; larger
 * batches run one kernel per projection, attention and small step. */
long pi0x_launch_count(const pi0x_handle *h, int B, int P, int num_steps);

/* ---- per-kernel-class device timing ------------------------------------------
 * With profiling on, the next pi0x_sample calls record a CUDA event pair around
 * every kernel launch (inside the captured graph, so kernels still run back to
 * back); pi0x_profile_read then reports, for the most recent such call, how many
 * kernels of a class ran and their summed device time in milliseconds.  It
 * synchronizes the handle's last stream.  Profiled calls use a separate graph, so
 * turning profiling on does not change the unprofiled path. */
enum {
  PI0X_K_PREP = 0,   /* mask compaction, time-MLP half, x_1 copy (once per call) */
  PI0X_K_EMBED = 1,  /* state and action input projections */
  PI0X_K_GEMM = 2,   /* every Linear of the expert and of the action-time MLP */
  PI0X_K_NORM = 3,   /* RMSNorm */
  PI0X_K_ROPE = 4,   /* RoPE of q/k, v copy */
  PI0X_K_ATTN = 5,   /* masked MQA attention */
  PI0X_K_GEGLU = 6,  /* gated GELU(tanh) */
  PI0X_K_FINAL = 7,  /* final norm + action out-proj + Euler update */
  PI0X_K_LOOP = 8,   /* the persistent small-batch loop kernel (every step of a call) */
  PI0X_K_COUNT = 9
};
int pi0x_profile_enable(pi0x_handle *h, int on);
int pi0x_profile_read(pi0x_handle *h, int kclass, long *launches, double *total_ms);

/* Human-readable name of a status code; never NULL. */
const char *pi0x_status_string(int status);

/* Text of the last CUDA error seen by this thread's calls ("" if none). */
const char *pi0x_last_error(void);

/* Free everything the handle owns.  Waits for the handle's work first.
 * Accepts NULL. */
void pi0x_destroy(pi0x_handle *h);

/* Library version as major*10000 + minor*100 + patch. */
int pi0x_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PI0X_H */
