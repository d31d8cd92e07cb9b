// qk_norm_rope.cu -- per-head norm of queries and keys with the rotation by position in the same
// pass, and its gradient.
//
// For a row x of 64 channels (one head of one token), xhat = (x - m) r with m the mean (layer norm;
// 0 for the root-mean-square norm) and r = 1 / sqrt(mean((x - m)^2) + eps), y = xhat w + b, and
// out = R y, where R turns each channel pair (a, b) by its angle t:
//   out_a = y_a cos t - y_b sin t,   out_b = y_b cos t + y_a sin t.
// The gradient for the upstream g: dy = R^T g (the opposite turn), dw += dy xhat, db += dy,
// h = dy w, dx = r (h - mean(h xhat) xhat - mean(h)), without the last term for the rms norm.
//
// The forward reads and writes every row once and the backward reads two and writes one: DRAM
// bounds both. Eight lanes take one token and walk its rows (query heads, then key heads), so the
// token's 32 cosines and sines are made once, four a lane, and stay in registers; a lane holds the
// four channel pairs those angles turn (channels c .. c+3 and their partners: two 8-byte loads in
// bf16, two 16-byte loads in fp32), so the rotation needs no exchange, and the row sums need three
// shuffles. When the tokens are too few to fill the GPU, a token's heads are split over several
// groups, which then make the same angles again.
//
// An angle is pos * freq in fp64 (in half turns), reduced to one turn before it is rounded to fp32:
// a position of 2^31 would lose every digit in fp32.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "view_internal.h"

namespace s3r {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 8;  // 8-lane groups a block

// A lane's eight channels of one row: a[i] and b[i] are pair i's first and second.
struct Row {
  float a[4], b[4];
};
// The same as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint2 a, b;
};
template <>
struct Raw<float> {
  float4 a, b;
};
__device__ __forceinline__ Raw<uint16_t> load_raw(const uint16_t* p, int ca, int cb) {
  return {*reinterpret_cast<const uint2*>(p + ca), *reinterpret_cast<const uint2*>(p + cb)};
}
__device__ __forceinline__ Raw<float> load_raw(const float* p, int ca, int cb) {
  return {*reinterpret_cast<const float4*>(p + ca), *reinterpret_cast<const float4*>(p + cb)};
}
__device__ __forceinline__ void unpack4(uint2 u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack4(float4 u, float (&v)[4]) {
  v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
}
template <typename T>
__device__ __forceinline__ Row unpack(const Raw<T>& r) {
  Row x;
  unpack4(r.a, x.a);
  unpack4(r.b, x.b);
  return x;
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Sum over the 8 lanes of a group.
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 4);
}
__device__ __forceinline__ float sum8(const Row& r) {
  return ((r.a[0] + r.a[1]) + (r.a[2] + r.a[3])) + ((r.b[0] + r.b[1]) + (r.b[2] + r.b[3]));
}

struct Lane {
  int ca, cb;       // first channel of the lane's four a-channels and of their partners
  bool first_axis;  // 2-D: turned by pos[0]
};
__device__ __forceinline__ Lane lane_channels(int rope) {
  const int l = threadIdx.x & 7;
  if (rope == S3R_ROPE_2D) return {(l >> 2) * 32 + (l & 3) * 4, (l >> 2) * 32 + (l & 3) * 4 + 16, l < 4};
  return {l * 4, l * 4 + 32, true};
}

// cos and sin of the lane's four angles for token t (1 and 0 without a rotation). The lane's first
// pair is number 4l: the 1-D pairs are 32, the 2-D halves hold the same 16 frequencies, stored twice.
__device__ __forceinline__ void angles(const QKNormArgs& a, const Lane& ln, int64_t t, float (&c)[4],
                                       float (&s)[4]) {
  if (a.rope == S3R_ROPE_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
    return;
  }
  const double p = a.rope == S3R_ROPE_2D ? a.pos[2 * t + (ln.first_axis ? 0 : 1)] : a.pos[t];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double x = p * a.freq[4 * (threadIdx.x & 7) + i];  // in half turns
    sincospif(static_cast<float>(x - 2. * rint(0.5 * x)), &s[i], &c[i]);
  }
}

// x -> x - m in place (layer norm); returns r.
__device__ __forceinline__ float centre(Row& x, int norm, float eps) {
  if (norm == S3R_NORM_NONE) return 1.f;
  if (norm == S3R_NORM_LAYER) {
    const float m = group_sum(sum8(x)) * (1.f / 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.a[i] -= m, x.b[i] -= m;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) q = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], q));
  return rsqrtf(fmaf(group_sum(q), 1.f / 64, eps));
}

// Heads [h0, h1) of n that piece `chunk` of `chunks` takes when q's and k's heads are one list;
// `base` is the position of this list's first head in it.
__device__ __forceinline__ void piece(int total, int chunks, int chunk, int base, int n, int& h0,
                                      int& h1) {
  const int lo = static_cast<int>(static_cast<int64_t>(total) * chunk / chunks) - base;
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (chunk + 1) / chunks) - base;
  h0 = lo < 0 ? 0 : lo;
  h1 = hi > n ? n : hi;
}

// Whole warps stay converged: a group past the last unit repeats the last unit's reads and writes
// nothing (it has no rows), so every shuffle has all 32 lanes. Groups of one warp may have
// different numbers of rows, so the row loops run to the warp's most.
//
// With the weights folded into the turn, an output is three products: for a pair's centred values
// da, db,  out_a = r (da (wa c) - db (wb s)) + (ba c - bb s), and likewise out_b; the products of
// weights and turn are the token's, made once.
// 64 registers: four blocks an SM. At two blocks (92 registers) too few loads were in flight: 293
// against 200 us for 137,400 tokens of 16 + 16 heads.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_fwd_kernel(const __grid_constant__ QKNormArgs a) {
  constexpr int kAhead = sizeof(T) == 2 ? 3 : 2;  // rows in flight a group
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + (threadIdx.x >> 3);
  const int64_t units = a.L * a.chunks;
  const bool live = unit < units;
  const int64_t u = live ? unit : units - 1;
  const int chunk = static_cast<int>(u / a.L);  // the groups of a warp have the same heads
  const int64_t t = u - chunk * a.L;
  const Lane ln = lane_channels(a.rope);
  float c[4], s[4];
  angles(a, ln, t, c, s);
  for (int which = 0; which < 2; ++which) {
    const int n = which ? a.Hk : a.H;
    if (n == 0) continue;
    int h0, h1;
    piece(a.H + a.Hk, a.chunks, chunk, which ? a.H : 0, n, h0, h1);
    const int rows = live && h1 > h0 ? h1 - h0 : 0;
    if (h0 > n - 1) h0 = n - 1;
    const int most = __reduce_max_sync(0xffffffffu, rows);
    if (most == 0) continue;
    const int64_t xh = which ? a.ks.head : a.qs.head, yh = which ? a.kos.head : a.qos.head;
    const T* x = static_cast<const T*>(which ? a.k : a.q) + t * (which ? a.ks.tok : a.qs.tok) + h0 * xh;
    T* y = static_cast<T*>(which ? a.k_out : a.q_out) + t * (which ? a.kos.tok : a.qos.tok) + h0 * yh;
    Raw<T> raw[kAhead] = {};
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      if (v < rows) raw[v] = load_raw(x, ln.ca, ln.cb);
      x += xh;
    }
    const float *w = which ? a.kw : a.qw, *b = which ? a.kb : a.qb;
    float ac[4], as[4], bc[4], bs[4], oa[4], ob[4];  // wa c, wa s, wb c, wb s; the turned bias
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float wa = w ? w[ln.ca + i] : 1.f, wb = w ? w[ln.cb + i] : 1.f;
      const float ba = b ? b[ln.ca + i] : 0.f, bb = b ? b[ln.cb + i] : 0.f;
      ac[i] = wa * c[i], as[i] = wa * s[i], bc[i] = wb * c[i], bs[i] = wb * s[i];
      oa[i] = ba * c[i] - bb * s[i], ob[i] = bb * c[i] + ba * s[i];
    }
    for (int r0 = 0; r0 < most; r0 += kAhead) {
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        if (r0 + v >= most) break;
        Row d = unpack(raw[v]);
        if (r0 + v + kAhead < rows) raw[v] = load_raw(x, ln.ca, ln.cb);
        x += xh;
        const float r = centre(d, a.norm, a.eps);
        float ya[4], yb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ya[i] = fmaf(r, d.a[i] * ac[i] - d.b[i] * bs[i], oa[i]);
          yb[i] = fmaf(r, d.b[i] * bc[i] + d.a[i] * as[i], ob[i]);
        }
        if (r0 + v < rows) {
          store4(y + ln.ca, ya);
          store4(y + ln.cb, yb);
        }
        y += yh;
      }
    }
  }
}

// Backward: the blocks below q_blocks walk the queries' tokens with a grid stride, the others the
// keys', keeping the weights' gradients of a lane's eight channels in registers (one list only:
// 32 sums fewer, and three blocks an SM instead of two); they are added up over the block at the end and
// written as one row of `part`, which qk_norm_dw_kernel adds in block order.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads, 3)
    qk_norm_bwd_kernel(const __grid_constant__ QKNormArgs a, int q_blocks) {
  __shared__ float red[kThreads / 32][2][64];
  constexpr int kAhead = 1;  // rows in flight a group, beside the one in work
  const bool which = static_cast<int>(blockIdx.x) >= q_blocks;
  const int block = which ? blockIdx.x - q_blocks : blockIdx.x;
  const int blocks = which ? gridDim.x - q_blocks : q_blocks;
  const int n = which ? a.Hk : a.H, chunks = a.chunks < n ? a.chunks : n;
  const Lane ln = lane_channels(a.rope);
  float acc[2][8] = {};  // [weight or bias][a channels, then b channels]
  const float* w = which ? a.kw : a.qw;
  float wa[4], wb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wa[i] = w ? w[ln.ca + i] : 1.f;
    wb[i] = w ? w[ln.cb + i] : 1.f;
  }
  const int64_t xh = which ? a.ks.head : a.qs.head, gh = which ? a.kos.head : a.qos.head;
  const int64_t dh = which ? a.dks.head : a.dqs.head;
  const int64_t units = a.L * chunks;
  const int64_t step = static_cast<int64_t>(blocks) * kGroups;
  const int64_t warp0 = static_cast<int64_t>(block) * kGroups + (threadIdx.x >> 5) * 4;
  for (int64_t base = warp0; base < units; base += step) {  // uniform in the warp
    const int64_t unit = base + ((threadIdx.x >> 3) & 3);
    const bool live = unit < units;
    const int64_t u = live ? unit : units - 1;
    const int chunk = static_cast<int>(u / a.L);
    const int64_t t = u - chunk * a.L;
    int h0, h1;
    piece(n, chunks, chunk, 0, n, h0, h1);
    const int rows = live ? h1 - h0 : 0;
    const int most = __reduce_max_sync(0xffffffffu, rows);
    const T* x = static_cast<const T*>(which ? a.k : a.q) + t * (which ? a.ks.tok : a.qs.tok) + h0 * xh;
    const G* g = static_cast<const G*>(which ? a.k_out : a.q_out) +
                 t * (which ? a.kos.tok : a.qos.tok) + h0 * gh;
    T* d = static_cast<T*>(which ? a.dk : a.dq) + t * (which ? a.dks.tok : a.dqs.tok) + h0 * dh;
    Raw<T> rx[kAhead] = {};
    Raw<G> rg[kAhead] = {};
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      if (v < rows) {
        rx[v] = load_raw(x, ln.ca, ln.cb);
        rg[v] = load_raw(g, ln.ca, ln.cb);
      }
      x += xh;
      g += gh;
    }
    float c[4], s[4];
    angles(a, ln, t, c, s);
    for (int r0 = 0; r0 < most; r0 += kAhead) {
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        if (r0 + v >= most) break;
        Row xr = unpack(rx[v]);  // a group without the row works on zeros, or on its last row again
        const Row gr = unpack(rg[v]);
        const bool mine = r0 + v < rows;
        if (r0 + v + kAhead < rows) {
          rx[v] = load_raw(x, ln.ca, ln.cb);
          rg[v] = load_raw(g, ln.ca, ln.cb);
        }
        x += xh;
        g += gh;
        const float r = centre(xr, a.norm, a.eps);
        Row h;
        float hx = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ya = gr.a[i] * c[i] + gr.b[i] * s[i], yb = gr.b[i] * c[i] - gr.a[i] * s[i];
          xr.a[i] *= r;
          xr.b[i] *= r;
          if (mine) {
            acc[0][i] = fmaf(ya, xr.a[i], acc[0][i]);
            acc[0][4 + i] = fmaf(yb, xr.b[i], acc[0][4 + i]);
            acc[1][i] += ya;
            acc[1][4 + i] += yb;
          }
          h.a[i] = ya * wa[i];
          h.b[i] = yb * wb[i];
          hx = fmaf(h.a[i], xr.a[i], fmaf(h.b[i], xr.b[i], hx));
        }
        float m1 = 0.f, m2 = 0.f;
        if (a.norm != S3R_NORM_NONE) m2 = group_sum(hx) * (1.f / 64);
        if (a.norm == S3R_NORM_LAYER) m1 = group_sum(sum8(h)) * (1.f / 64);
        const float n1 = -r * m1, n2 = -r * m2;
        float da[4], db[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          da[i] = fmaf(n2, xr.a[i], fmaf(r, h.a[i], n1));
          db[i] = fmaf(n2, xr.b[i], fmaf(r, h.b[i], n1));
        }
        if (mine) {
          store4(d + ln.ca, da);
          store4(d + ln.cb, db);
        }
        d += dh;
      }
    }
  }
  // the four groups of a warp, then the warps of the block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = acc[kind][i];
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      if (lane < 8) red[warp][kind][(i < 4 ? ln.ca : ln.cb) + (i & 3)] = x;
    }
  __syncthreads();
  if (threadIdx.x < 128) {
    const int kind = threadIdx.x >> 6, ch = threadIdx.x & 63;
    float x = 0.f;
#pragma unroll
    for (int w8 = 0; w8 < kThreads / 32; ++w8) x += red[w8][kind][ch];
    a.part[static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x] = x;
  }
}

// dw[v][ch] = sum over the blocks' rows (v: weight and bias of q, then of k): one block per vector, 16
// slices of the rows by 64 channels, in fp64.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* part, int q_blocks, int blocks,
                                                          float* dw) {
  __shared__ double red[16][64];
  const int ch = threadIdx.x & 63, slice = threadIdx.x >> 6, v = blockIdx.x;
  const int first = v < 2 ? 0 : q_blocks, last = v < 2 ? q_blocks : blocks;
  double x = 0.;
  for (int b = first + slice; b < last; b += 16)
    x += part[static_cast<int64_t>(b) * 128 + (v & 1) * 64 + ch];
  red[slice][ch] = x;
  __syncthreads();
  if (threadIdx.x < 64) {
    double y = 0.;
#pragma unroll
    for (int s = 0; s < 16; ++s) y += red[s][ch];
    dw[v * 64 + ch] = static_cast<float>(y);
  }
}

constexpr int kSMs = 148;

// Pieces a token's heads are split into: one, unless that leaves fewer 8-lane groups than about
// eight warps per SM, and at most one piece a head.
int head_chunks(int64_t L, int heads) {
  const int64_t want = static_cast<int64_t>(kSMs) * 8 * 4;
  if (L >= want || L == 0) return 1;
  const int64_t c = (want + L - 1) / L;
  return static_cast<int>(c < heads ? c : heads);
}

// Blocks of one list of the backward: as many as have work, at most three per SM for both lists
// together (what is resident), shared by their heads.
int list_blocks(int64_t L, int n, int total) {
  if (n == 0 || L == 0) return 0;
  const int chunks = head_chunks(L, total);
  const int64_t need = (L * (chunks < n ? chunks : n) + kGroups - 1) / kGroups;
  const int64_t most = static_cast<int64_t>(3) * kSMs * n / total;
  return static_cast<int>(need < (most < 1 ? 1 : most) ? need : (most < 1 ? 1 : most));
}

}  // namespace

int qk_norm_bwd_blocks(int64_t L, int H, int Hk) {
  return list_blocks(L, H, H + Hk) + list_blocks(L, Hk, H + Hk);
}

cudaError_t launch_qk_norm_fwd(QKNormArgs a, int dtype, cudaStream_t st) {
  if (a.L == 0 || a.H + a.Hk == 0) return cudaSuccess;
  a.chunks = head_chunks(a.L, a.H + a.Hk);
  const int64_t blocks = (a.L * a.chunks + kGroups - 1) / kGroups;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (dtype == S3R_TYPE_F32)
    qk_norm_fwd_kernel<float><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a);
  else
    qk_norm_fwd_kernel<uint16_t><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_bwd(QKNormArgs a, int dtype, int grad_dtype, float* dw,
                               cudaStream_t st) {
  const int q_blocks = list_blocks(a.L, a.H, a.H + a.Hk), blocks = qk_norm_bwd_blocks(a.L, a.H, a.Hk);
  if (blocks > 0) {
    a.chunks = head_chunks(a.L, a.H + a.Hk);
    if (dtype == S3R_TYPE_F32 && grad_dtype == S3R_TYPE_F32)
      qk_norm_bwd_kernel<float, float><<<blocks, kThreads, 0, st>>>(a, q_blocks);
    else if (dtype == S3R_TYPE_F32)
      qk_norm_bwd_kernel<float, uint16_t><<<blocks, kThreads, 0, st>>>(a, q_blocks);
    else if (grad_dtype == S3R_TYPE_F32)
      qk_norm_bwd_kernel<uint16_t, float><<<blocks, kThreads, 0, st>>>(a, q_blocks);
    else
      qk_norm_bwd_kernel<uint16_t, uint16_t><<<blocks, kThreads, 0, st>>>(a, q_blocks);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  qk_norm_dw_kernel<<<4, 1024, 0, st>>>(a.part, q_blocks, blocks, dw);
  count_launch();
  return cudaGetLastError();
}

}  // namespace s3r
