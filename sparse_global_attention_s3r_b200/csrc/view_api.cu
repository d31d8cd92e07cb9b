// view_api.cu -- the extern "C" entry points of include/s3r_view.h: argument validation, workspace
// layouts and launches.
#include <climits>
#include <cmath>

#include "view_internal.h"

namespace s3r {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool row_ptr(const void* p, int64_t rows) { return rows == 0 || (p && aligned(p, 16)); }
bool vec_ptr(const float* p) { return aligned(p, 16); }

// Strides of a [L, H, 64] tensor: {0, 0} is dense; otherwise multiples of 8 whose rows do not
// overlap. A dimension of one element never steps: its stride is replaced, so that a tensor map
// of any caller's view of it is valid.
bool strides(const int64_t in[2], int64_t L, int64_t H, Stride2* out) {
  constexpr int64_t kMax = int64_t(1) << 38;  // elements: below the 2^40 bytes of a tensor map
  Stride2 s{in[0], in[1]};
  if (s.tok == 0 && s.head == 0) {
    s = Stride2{H * 64, 64};
  } else {
    if (H <= 1) s.head = 64;
    if (L <= 1) s.tok = s.head * (H < 1 ? 1 : H);
    if (s.tok < 64 || s.head < 64 || s.tok >= kMax || s.head >= kMax || s.tok % 8 || s.head % 8)
      return false;
    const bool head_inside = s.tok >= s.head * (H - 1) + 64;
    const bool tok_inside = L <= kMax / s.tok && s.head >= s.tok * (L - 1) + 64;
    if (L > 1 && H > 1 && !head_inside && !tok_inside) return false;
  }
  *out = s;
  return true;
}

s3r_status launched(cudaError_t e) { return e == cudaSuccess ? S3R_OK : S3R_ERR_CUDA; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

s3r_status derive(const s3r_qk_norm_params* p, bool bwd, QKNormArgs* out) {
  if (!p) return S3R_ERR_INVALID_ARG;
  if (p->L < 0 || p->L > INT32_MAX || p->H < 0 || p->Hk < 0 || p->H > 65535 || p->Hk > 65535 ||
      p->H + p->Hk < 1)
    return S3R_ERR_INVALID_ARG;
  if (p->d != 64) return S3R_ERR_UNSUPPORTED;
  auto type = [](int32_t t) { return t == S3R_TYPE_BF16 || t == S3R_TYPE_F32; };
  if (!type(p->dtype) || (bwd && !type(p->grad_dtype))) return S3R_ERR_UNSUPPORTED;
  if (p->norm < S3R_NORM_NONE || p->norm > S3R_NORM_RMS || p->rope < S3R_ROPE_NONE ||
      p->rope > S3R_ROPE_2D)
    return S3R_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || std::isinf(p->eps)) return S3R_ERR_INVALID_ARG;
  if (p->rope != S3R_ROPE_NONE && (!(p->base > 0.) || std::isinf(p->base)))
    return S3R_ERR_INVALID_ARG;
  QKNormArgs a{};
  a.L = p->L;
  a.H = p->H;
  a.Hk = p->Hk;
  a.norm = p->norm;
  a.rope = p->rope;
  a.eps = p->eps;
  if (!strides(p->q_stride, p->L, p->H, &a.qs) || !strides(p->k_stride, p->L, p->Hk, &a.ks) ||
      !strides(p->qo_stride, p->L, p->H, &a.qos) || !strides(p->ko_stride, p->L, p->Hk, &a.kos))
    return S3R_ERR_INVALID_ARG;
  if (bwd &&
      (!strides(p->dq_stride, p->L, p->H, &a.dqs) || !strides(p->dk_stride, p->L, p->Hk, &a.dks)))
    return S3R_ERR_INVALID_ARG;
  *out = a;
  return S3R_OK;
}

// base^(-i/32), or base^(-i/16) twice over, in half turns. A third of the calls to pow: they are a
// share of a small call's time.
void frequencies(const s3r_qk_norm_params* p, double freq[32]) {
  if (p->rope == S3R_ROPE_NONE) return;
  const int n = p->rope == S3R_ROPE_2D ? 16 : 32;
  double low[8], high[4];
  for (int i = 0; i < 8; ++i) low[i] = std::pow(p->base, -static_cast<double>(i) / n);
  for (int i = 0; i < n / 8; ++i)
    high[i] = std::pow(p->base, -8. * i / n) / 3.14159265358979323846;
  for (int i = 0; i < 32; ++i) freq[i] = high[i % n / 8] * low[i % 8];
}

size_t norm_workspace(const QKNormArgs& a) {
  const size_t n = static_cast<size_t>(qk_norm_bwd_blocks(a.L, a.H, a.Hk));
  return round256((n < 1 ? 1 : n) * 128 * sizeof(float));
}

bool check_pos(const QKNormArgs& a, const int32_t* pos) {
  return a.rope == S3R_ROPE_NONE || a.L == 0 || (pos && aligned(pos, 4));
}

s3r_status derive(const s3r_view_params* p, ViewProblem* out) {
  if (!p) return S3R_ERR_INVALID_ARG;
  if (p->Lq < 0 || p->Lk < 0 || p->Lq > INT32_MAX || p->Lk > INT32_MAX || p->H < 1 ||
      p->H > 65535 || p->Hkv < 1 || p->H % p->Hkv != 0 || p->nseg < 1 || p->max_q < 0 ||
      p->max_k < 0)
    return S3R_ERR_INVALID_ARG;
  if (std::isnan(p->scale) || std::isinf(p->scale)) return S3R_ERR_INVALID_ARG;
  if (p->d != 64) return S3R_ERR_UNSUPPORTED;
  ViewProblem v{};
  v.Lq = p->Lq;
  v.Lk = p->Lk;
  v.H = p->H;
  v.Hkv = p->Hkv;
  v.nseg = p->nseg;
  // a bound above the tensor itself says nothing more
  v.max_q = p->max_q < p->Lq ? p->max_q : static_cast<int>(p->Lq);
  v.max_k = p->max_k < p->Lk ? p->max_k : static_cast<int>(p->Lk);
  // (segment, tile of 128 rows, head) is a block of a grid
  const int64_t tiles = (v.max_q > v.max_k ? v.max_q : v.max_k) / 128 + 1;
  if (tiles > INT32_MAX / p->H / p->nseg) return S3R_ERR_INVALID_ARG;
  v.scale = p->scale > 0.f ? p->scale : 0.125f;
  v.scale_log2 = static_cast<float>(static_cast<double>(v.scale) * 1.4426950408889634);
  v.flags = p->flags;
  if (!strides(p->q_stride, p->Lq, p->H, &v.qs) || !strides(p->k_stride, p->Lk, p->Hkv, &v.ks) ||
      !strides(p->v_stride, p->Lk, p->Hkv, &v.vs) || !strides(p->dq_stride, p->Lq, p->H, &v.dqs) ||
      !strides(p->dk_stride, p->Lk, p->Hkv, &v.dks) || !strides(p->dv_stride, p->Lk, p->Hkv, &v.dvs))
    return S3R_ERR_INVALID_ARG;
  v.status = p->dev_status;
  if (!aligned(v.status, 4)) return S3R_ERR_INVALID_ARG;
  *out = v;
  return S3R_OK;
}

}  // namespace
}  // namespace s3r

using namespace s3r;

extern "C" {

s3r_status s3r_qk_norm_rope_fwd(const s3r_qk_norm_params* params, const void* q, const void* k,
                                const int32_t* pos, const float* qw, const float* qb,
                                const float* kw, const float* kb, void* q_out, void* k_out,
                                s3r_stream stream) {
  QKNormArgs a;
  s3r_status st = derive(params, false, &a);
  if (st != S3R_OK) return st;
  const int64_t nq = a.L * a.H, nk = a.L * a.Hk;
  if (!row_ptr(q, nq) || !row_ptr(k, nk) || !row_ptr(q_out, nq) || !row_ptr(k_out, nk) ||
      !check_pos(a, pos) || !vec_ptr(qw) || !vec_ptr(qb) || !vec_ptr(kw) || !vec_ptr(kb))
    return S3R_ERR_INVALID_ARG;
  if ((a.norm == S3R_NORM_NONE && (qw || kw)) || (a.norm != S3R_NORM_LAYER && (qb || kb)))
    return S3R_ERR_INVALID_ARG;
  a.q = q, a.k = k, a.pos = pos, a.qw = qw, a.qb = qb, a.kw = kw, a.kb = kb;
  a.q_out = q_out, a.k_out = k_out;
  frequencies(params, a.freq);
  return launched(launch_qk_norm_fwd(a, params->dtype, stream));
}

size_t s3r_qk_norm_rope_bwd_workspace_bytes(const s3r_qk_norm_params* params) {
  QKNormArgs a;
  return derive(params, true, &a) == S3R_OK ? norm_workspace(a) : 0;
}

s3r_status s3r_qk_norm_rope_bwd(const s3r_qk_norm_params* params, const void* q, const void* k,
                                const int32_t* pos, const float* qw, const float* kw,
                                const void* gq, const void* gk, void* dq, void* dk, float* dw,
                                void* workspace, size_t workspace_bytes, s3r_stream stream) {
  QKNormArgs a;
  s3r_status st = derive(params, true, &a);
  if (st != S3R_OK) return st;
  const int64_t nq = a.L * a.H, nk = a.L * a.Hk;
  if (!row_ptr(q, nq) || !row_ptr(k, nk) || !row_ptr(gq, nq) || !row_ptr(gk, nk) ||
      !row_ptr(dq, nq) || !row_ptr(dk, nk) || !check_pos(a, pos) || !vec_ptr(qw) || !vec_ptr(kw) ||
      !dw || !vec_ptr(dw))
    return S3R_ERR_INVALID_ARG;
  if (a.norm == S3R_NORM_NONE && (qw || kw)) return S3R_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < norm_workspace(a))
    return S3R_ERR_WORKSPACE;
  a.q = q, a.k = k, a.pos = pos, a.qw = qw, a.kw = kw;
  a.q_out = const_cast<void*>(gq), a.k_out = const_cast<void*>(gk);
  a.dq = dq, a.dk = dk;
  a.part = static_cast<float*>(workspace);
  frequencies(params, a.freq);
  return launched(launch_qk_norm_bwd(a, params->dtype, params->grad_dtype, dw, stream));
}

size_t s3r_view_attn_workspace_bytes(const s3r_view_params* params) {
  ViewProblem p;
  return derive(params, &p) == S3R_OK ? view_fwd_workspace(p) : 0;
}

s3r_status s3r_view_attn_fwd(const s3r_view_params* params, const s3r_bf16* q, const s3r_bf16* k,
                             const s3r_bf16* v, const int32_t* q_offs, const int32_t* k_offs,
                             s3r_bf16* out, float* lse, void* workspace, size_t workspace_bytes,
                             s3r_stream stream) {
  ViewProblem p;
  s3r_status st = derive(params, &p);
  if (st != S3R_OK) return st;
  if (!row_ptr(q, p.Lq) || !row_ptr(k, p.Lk) || !row_ptr(v, p.Lk) || !row_ptr(out, p.Lq) ||
      !aligned(lse, 16) || !q_offs || !aligned(q_offs, 4) || !k_offs || !aligned(k_offs, 4))
    return S3R_ERR_INVALID_ARG;
  const size_t need = view_fwd_workspace(p);
  if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return S3R_ERR_WORKSPACE;
  return launched(launch_view_fwd(p, q, k, v, q_offs, k_offs, out, lse, workspace, stream));
}

size_t s3r_view_attn_bwd_workspace_bytes(const s3r_view_params* params) {
  ViewProblem p;
  return derive(params, &p) == S3R_OK ? view_bwd_workspace(p) : 0;
}

s3r_status s3r_view_attn_bwd(const s3r_view_params* params, const s3r_bf16* q, const s3r_bf16* k,
                             const s3r_bf16* v, const int32_t* q_offs, const int32_t* k_offs,
                             const s3r_bf16* out, const float* lse, const s3r_bf16* dout,
                             s3r_bf16* dq, s3r_bf16* dk, s3r_bf16* dv, void* workspace,
                             size_t workspace_bytes, s3r_stream stream) {
  ViewProblem p;
  s3r_status st = derive(params, &p);
  if (st != S3R_OK) return st;
  if (!row_ptr(q, p.Lq) || !row_ptr(k, p.Lk) || !row_ptr(v, p.Lk) || !row_ptr(out, p.Lq) ||
      !row_ptr(lse, p.Lq) || !row_ptr(dout, p.Lq) || !row_ptr(dq, p.Lq) || !row_ptr(dk, p.Lk) ||
      !row_ptr(dv, p.Lk) || !q_offs || !aligned(q_offs, 4) || !k_offs || !aligned(k_offs, 4))
    return S3R_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < view_bwd_workspace(p))
    return S3R_ERR_WORKSPACE;
  return launched(launch_view_bwd(p, q, k, v, q_offs, k_offs, out, lse, dout, dq, dk, dv, workspace,
                                  stream));
}

}  // extern "C"
