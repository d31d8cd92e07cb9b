/*
 * s3r_view.h -- C ABI of the dense operators that stand beside the sparse global attention of
 * s3r.h in a multi-view transformer, in the same library (libs3r.so):
 *   - the per-head norm of queries and keys with the rotation by position in the same pass, and
 *     its gradient: what turns a layer's projected q and k into the q and k that either attention
 *     takes;
 *   - dense attention of every query over the keys of its own segment (a view, a whole scene, or a
 *     cache of earlier views), and its gradient, which recomputes the probabilities. The layers
 *     that alternate with the sparse ones attend inside each view this way, and the dense teacher
 *     of a sparse layer is the one-segment case.
 *
 * The conventions are those of s3r.h: device pointers of the current device, 16-byte aligned
 * unless stated; asynchronous calls on `stream`; host-side validation before any launch; no
 * allocation and no synchronisation; device-side conditions OR-ed into params->dev_status; no C++
 * exception crosses the boundary; the functions are thread-safe and keep nothing between calls.
 * Rows of 64 channels are contiguous; where a params field holds a stride pair, stride[0] is the
 * elements between tokens and stride[1] between heads (both multiples of 8, rows not overlapping);
 * {0, 0} means the dense layout [L, H, 64].
 */
#ifndef S3R_VIEW_H
#define S3R_VIEW_H

#include "s3r.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the norm's rows. */
#define S3R_TYPE_BF16 0
#define S3R_TYPE_F32 1

#define S3R_NORM_NONE 0  /* y = x */
#define S3R_NORM_LAYER 1 /* y = (x - mean) / sqrt(var + eps) * weight + bias */
#define S3R_NORM_RMS 2   /* y = x / sqrt(mean(x^2) + eps) * weight */

#define S3R_ROPE_NONE 0
#define S3R_ROPE_1D 1 /* channel pairs (i, i + 32), i < 32, turned by pos * base^(-i/32) */
#define S3R_ROPE_2D 2 /* first half of the channels by pos[0] (the patch row), second half by
                         pos[1] (its column): pairs (i, i + 16) of each half, i < 16, turned by
                         pos * base^(-i/16) */

typedef struct {
  int64_t L;   /* tokens, >= 0 */
  int32_t H;   /* query heads, >= 0 */
  int32_t Hk;  /* key heads, >= 0 */
  int32_t d;   /* 64 */
  int32_t norm; /* S3R_NORM_* */
  int32_t rope; /* S3R_ROPE_* */
  int32_t dtype;      /* S3R_TYPE_* of q, k and their outputs (their gradients in the backward) */
  int32_t grad_dtype; /* backward: S3R_TYPE_* of the upstream gradients */
  float eps;          /* >= 0, finite */
  double base;        /* rotation base, > 0, finite */
  int64_t q_stride[2], k_stride[2];   /* inputs q, k */
  int64_t qo_stride[2], ko_stride[2]; /* forward: the outputs; backward: their upstream gradients */
  int64_t dq_stride[2], dk_stride[2]; /* backward: the gradients of q and k */
} s3r_qk_norm_params;

/* q_out = R(pos) norm(q), k_out = R(pos) norm(k), one pass over both. The statistics and the
 * rotation are computed in fp32, the angles in fp64 (reduced to one turn before they are rounded),
 * and each output is rounded once. Outputs may be the inputs themselves (same pointer, same
 * strides); other overlaps are not allowed.
 *   q [L, H, 64], k [L, Hk, 64]      read, of params->dtype, strided
 *   pos                              int32, 4-byte aligned: [L] (1-D) or [L, 2] (2-D); NULL
 *                                    without a rotation. Any int32 value.
 *   qw, qb, kw, kb                   [64] fp32, each may be NULL (weight 1, bias 0); a bias needs
 *                                    S3R_NORM_LAYER, a weight any norm but S3R_NORM_NONE
 *   q_out, k_out                     written, of params->dtype, strided */
s3r_status s3r_qk_norm_rope_fwd(const s3r_qk_norm_params* params, const void* q, const void* k,
                                const int32_t* pos, const float* qw, const float* qb,
                                const float* kw, const float* kb, void* q_out, void* k_out,
                                s3r_stream stream);

/* Bytes of workspace s3r_qk_norm_rope_bwd needs (0 if params are invalid). */
size_t s3r_qk_norm_rope_bwd_workspace_bytes(const s3r_qk_norm_params* params);

/* Gradients of s3r_qk_norm_rope_fwd for the upstream gradients gq, gk (of params->grad_dtype,
 * strides qo_stride, ko_stride). The statistics are recomputed from q and k.
 *   dq, dk            written, of params->dtype; each may be the upstream gradient's own buffer
 *                     (same type and strides) or the input's
 *   dw                [4, 64] fp32, written: the gradients of qw, qb, kw, kb (summed in a fixed
 *                     order, so that equal calls give equal bits); zero where nothing was summed
 *   workspace         256-byte aligned */
s3r_status s3r_qk_norm_rope_bwd(const s3r_qk_norm_params* params, const void* q, const void* k,
                                const int32_t* pos, const float* qw, const float* kw,
                                const void* gq, const void* gk, void* dq, void* dk, float* dw,
                                void* workspace, size_t workspace_bytes, s3r_stream stream);

/* Flags of s3r_view_params besides S3R_FLAG_TEST_TIMEOUT. The dense calls push no NVTX ranges. */
#define S3R_FLAG_ALL_ROWS 0x100u /* also write the rows of no segment (before the first, past the last):
                                    out and the gradients 0, lse -inf; and NaN in the rows of a
                                    segment that cannot be used. Without it all those are left as
                                    they were */

typedef struct {
  int64_t Lq;  /* rows of q, out and lse, >= 0, < 2^31 */
  int64_t Lk;  /* rows of k and v, >= 0, < 2^31 */
  int32_t H;   /* query heads */
  int32_t Hkv; /* key/value heads, a divisor of H: head h reads key head h / (H / Hkv) */
  int32_t d;   /* 64 */
  int32_t nseg;  /* segments, >= 1 */
  int32_t max_q; /* no segment holds more queries than this */
  int32_t max_k; /* no segment holds more keys than this */
  float scale;   /* softmax scale; <= 0 selects 1/sqrt(d) */
  uint32_t flags;
  int64_t q_stride[2], k_stride[2], v_stride[2];
  int64_t dq_stride[2], dk_stride[2], dv_stride[2]; /* backward's outputs */
  uint32_t* dev_status; /* optional device word that receives S3R_DEV_* bits */
} s3r_view_params;

/* Bytes of workspace for s3r_view_attn_fwd (0: none needed, or invalid params). */
size_t s3r_view_attn_workspace_bytes(const s3r_view_params* params);

/* Dense attention inside segments. Segment s holds queries q_offs[s] .. q_offs[s+1] - 1 and keys
 * k_offs[s] .. k_offs[s+1] - 1 (device arrays of nseg + 1 int32, ascending from >= 0, 4-byte
 * aligned; they are read on the device, so a captured call replays with new offsets). Queries of a
 * segment without keys get out = 0 and lse = -inf. A segment whose offsets descend, pass Lq or Lk,
 * or exceed max_q or max_k raises S3R_DEV_BAD_INDEX, and is not computed. (Where offsets
 * descend, rows that several segments name, or a segment and S3R_FLAG_ALL_ROWS' rows, hold any
 * one's result. Nothing outside the tensors is read or written.)
 *   lse[h, r] = log sum_t exp(scale <q[r,h], k[t]>),   out[r, h] = sum_t exp(scale <q, k> - lse) v[t]
 * No value of a row outside a segment, or past its end, reaches the segment's results, whatever it
 * holds (infinities and NaN included). A NaN or infinite logit of a row's own segment makes that row
 * NaN or leaves it without a defined value. A row's sums are held in fp32 relative to one of its
 * logits, and a tile of keys may pass that by 2^60: |v| has to stay below 2^44.
 * The outputs must not overlap the inputs.
 *   q [Lq, H, 64], k, v [Lk, Hkv, 64] bf16 (read, strided)
 *   out [Lq, H, 64] bf16 (written, dense); lse [H, Lq] fp32 (written if not NULL)
 *   workspace  256-byte aligned, s3r_view_attn_workspace_bytes(params); may be NULL if that is 0 */
s3r_status s3r_view_attn_fwd(const s3r_view_params* params, const s3r_bf16* q, const s3r_bf16* k,
                             const s3r_bf16* v, const int32_t* q_offs, const int32_t* k_offs,
                             s3r_bf16* out, float* lse, void* workspace, size_t workspace_bytes,
                             s3r_stream stream);

/* Bytes of workspace for s3r_view_attn_bwd (0 if params are invalid). */
size_t s3r_view_attn_bwd_workspace_bytes(const s3r_view_params* params);

/* Gradients of s3r_view_attn_fwd for the upstream gradient dout, from the forward's inputs, out and
 * lse; the probabilities are recomputed from q, k and lse:
 *   P = exp(scale q k^T - lse),  D = <dout, out>,  dS = P (dout v^T - D),
 *   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout,
 * dk and dv summed over the query heads that share a key head. Sums are held in fp32 and added in a
 * fixed order: equal calls give equal bits. In a segment of up to 256 keys D is formed as the sum of
 * P dout v^T, which is <dout, out> without out's rounding. (In longer ones that rounding takes dq's and
 * dk's error from 0.0024 of their norm to 0.0025, and to 0.0064 where softmax rows lie on few keys.)
 * Keys of a segment without queries get zero gradients.
 * The gradients must not overlap the inputs.
 *   out, dout [Lq, H, 64] bf16 (read, dense); lse [H, Lq] fp32 (read)
 *   dq [Lq, H, 64], dk, dv [Lk, Hkv, 64] bf16 (written, strided)
 *   workspace  256-byte aligned */
s3r_status s3r_view_attn_bwd(const s3r_view_params* params, const s3r_bf16* q, const s3r_bf16* k,
                             const s3r_bf16* v, const int32_t* q_offs, const int32_t* k_offs,
                             const s3r_bf16* out, const float* lse, const s3r_bf16* dout,
                             s3r_bf16* dq, s3r_bf16* dk, s3r_bf16* dv, void* workspace,
                             size_t workspace_bytes, s3r_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* S3R_VIEW_H */
