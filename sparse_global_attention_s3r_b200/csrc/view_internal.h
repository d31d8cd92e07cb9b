// view_internal.h -- launchers behind include/s3r_view.h (not part of the public interface).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "s3r_view.h"

namespace s3r {

struct Stride2 {
  int64_t tok, head;  // elements
};

// Per-head norm and rotation of queries and keys (qk_norm_rope.cu).
struct QKNormArgs {
  const void *q, *k;
  const int32_t* pos;
  const float *qw, *qb, *kw, *kb;
  void *q_out, *k_out;    // forward: outputs; backward: the upstream gradients (read)
  void *dq, *dk;          // backward
  float* part;            // backward: [blocks][2][64] partial sums of the weights' gradients
  Stride2 qs, ks, qos, kos, dqs, dks;
  int64_t L;
  int H, Hk, norm, rope;
  int chunks;  // pieces a token's heads are split into, each an 8-lane group's work
  float eps;
  double freq[32];  // rotation of each channel pair by one position, in half turns
};
// Blocks of the backward (the rows of `part`).
int qk_norm_bwd_blocks(int64_t L, int H, int Hk);
cudaError_t launch_qk_norm_fwd(QKNormArgs a, int dtype, cudaStream_t st);
cudaError_t launch_qk_norm_bwd(QKNormArgs a, int dtype, int grad_dtype, float* dw, cudaStream_t st);

// Dense attention inside segments (view_attn.cu, view_attn_bwd.cu).
struct ViewProblem {
  int64_t Lq, Lk;
  int H, Hkv, nseg, max_q, max_k;
  float scale, scale_log2;
  uint32_t flags;
  Stride2 qs, ks, vs, dqs, dks, dvs;
  uint32_t* status;
};
// Items a head's rows of no segment are filled by: their number is known on the device only, so as
// many as a tensor of that many rows keeps busy, at most 64.
inline int64_t rest_items(int64_t rows) {
  const int64_t n = (rows + 2047) / 2048;
  return n < 1 ? 1 : n < 64 ? n : 64;
}
// Pieces the keys are split into, and the bytes of their partial results (0 for one piece).
int view_fwd_splits(const ViewProblem& p);
size_t view_fwd_workspace(const ViewProblem& p);
cudaError_t launch_view_fwd(const ViewProblem& p, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const int32_t* qo, const int32_t* ko,
                            uint16_t* out, float* lse, void* ws, cudaStream_t st);
size_t view_bwd_workspace(const ViewProblem& p);
cudaError_t launch_view_bwd(const ViewProblem& p, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const int32_t* qo, const int32_t* ko,
                            const uint16_t* out, const float* lse, const uint16_t* dout,
                            uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, cudaStream_t st);

}  // namespace s3r
