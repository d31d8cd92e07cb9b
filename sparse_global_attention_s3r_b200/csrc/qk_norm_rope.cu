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

struct Row {
  float a[4], b[4];  // first and second channels of the lane's four pairs
};

__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename T>
__device__ __forceinline__ Row load_row(const T* p, int ca, int cb) {
  Row r;
  load4(p + ca, r.a);
  load4(p + cb, r.b);
  return r;
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

// cos and sin of the lane's four angles for token t (1 and 0 without a rotation).
__device__ __forceinline__ void angles(const QKNormArgs& a, const double (&freq)[4],
                                       const Lane& ln, int64_t t, float (&c)[4], float (&s)[4]) {
  if (a.rope == S3R_ROPE_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
    return;
  }
  const double p = a.rope == S3R_ROPE_2D ? a.pos[2 * t + (ln.first_axis ? 0 : 1)] : a.pos[t];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double x = p * freq[i];  // in half turns
    sincospif(static_cast<float>(x - 2. * rint(0.5 * x)), &s[i], &c[i]);
  }
}
__device__ __forceinline__ void load_freq(const QKNormArgs& a, double (&freq)[4]) {
  const int l = threadIdx.x & 7;
  // pair index of the lane's first pair: 1-D pairs are 4l .. 4l+3 of 32; the 2-D halves hold the
  // same 16 frequencies, stored twice
#pragma unroll
  for (int i = 0; i < 4; ++i) freq[i] = a.freq[4 * l + i];
}

struct Weights {
  float wa[4], wb[4], ba[4], bb[4];
};
__device__ __forceinline__ Weights load_weights(const float* w, const float* b, const Lane& ln) {
  Weights r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.wa[i] = w ? w[ln.ca + i] : 1.f;
    r.wb[i] = w ? w[ln.cb + i] : 1.f;
    r.ba[i] = b ? b[ln.ca + i] : 0.f;
    r.bb[i] = b ? b[ln.cb + i] : 0.f;
  }
  return r;
}

// x -> xhat in place; returns r.
__device__ __forceinline__ float normalise(Row& x, int norm, float eps) {
  if (norm == S3R_NORM_NONE) return 1.f;
  if (norm == S3R_NORM_LAYER) {
    const float m = group_sum(sum8(x)) * (1.f / 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.a[i] -= m, x.b[i] -= m;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) q = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], q));
  const float r = rsqrtf(fmaf(group_sum(q), 1.f / 64, eps));
#pragma unroll
  for (int i = 0; i < 4; ++i) x.a[i] *= r, x.b[i] *= r;
  return r;
}

// Rows in flight a group: loads of the next rows issued before the first is used.
constexpr int kAhead = 4;

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
// nothing (its head range is empty), so every shuffle has all 32 lanes. Groups of one warp may
// have head ranges of different lengths, so the row loops run to the warp's longest.
template <typename T>
__global__ void __launch_bounds__(kThreads) qk_norm_fwd_kernel(const __grid_constant__ QKNormArgs a) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + (threadIdx.x >> 3);
  const int64_t units = a.L * a.chunks;
  const bool live = unit < units;
  const int64_t u = live ? unit : units - 1;
  const int64_t t = u / a.chunks;
  const int chunk = static_cast<int>(u - t * a.chunks);
  const Lane ln = lane_channels(a.rope);
  double freq[4];
  load_freq(a, freq);
  float c[4], s[4];
  angles(a, freq, ln, t, c, s);
  int h0, h1;
  for (int which = 0; which < 2; ++which) {
    const int n = which ? a.Hk : a.H;
    if (n == 0) continue;
    piece(a.H + a.Hk, a.chunks, chunk, which ? a.H : 0, n, h0, h1);
    int rows = live && h1 > h0 ? h1 - h0 : 0;
    if (h0 > n - 1) h0 = n - 1;
    const int most = __reduce_max_sync(0xffffffffu, rows);
    if (most == 0) continue;
    const Weights w = which ? load_weights(a.kw, a.kb, ln) : load_weights(a.qw, a.qb, ln);
    const Stride2 xs = which ? a.ks : a.qs, ys = which ? a.kos : a.qos;
    const T* x = static_cast<const T*>(which ? a.k : a.q) + t * xs.tok + h0 * xs.head;
    T* y = static_cast<T*>(which ? a.k_out : a.q_out) + t * ys.tok + h0 * ys.head;
    for (int r0 = 0; r0 < most; r0 += kAhead) {
      Row r[kAhead];
#pragma unroll
      for (int v = 0; v < kAhead; ++v)
        r[v] = load_row(x + (r0 + v < rows ? r0 + v : 0) * xs.head, ln.ca, ln.cb);
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        if (r0 + v >= most) break;
        normalise(r[v], a.norm, a.eps);
        float oa[4], ob[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ya = fmaf(r[v].a[i], w.wa[i], w.ba[i]);
          const float yb = fmaf(r[v].b[i], w.wb[i], w.bb[i]);
          oa[i] = ya * c[i] - yb * s[i];
          ob[i] = yb * c[i] + ya * s[i];
        }
        if (r0 + v < rows) {
          store4(y + (r0 + v) * ys.head + ln.ca, oa);
          store4(y + (r0 + v) * ys.head + ln.cb, ob);
        }
      }
    }
  }
}

// Backward: a block walks tokens with a grid stride, keeping the weights' gradients of its lanes'
// channels in registers; they are added up over the block at the end and written as one row of
// `part`, which qk_norm_dw_kernel adds in block order.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const __grid_constant__ QKNormArgs a) {
  __shared__ float red[kThreads / 32][4][64];
  const Lane ln = lane_channels(a.rope);
  double freq[4];
  load_freq(a, freq);
  float acc[2][2][8] = {};  // [q or k][weight or bias][a channels, then b channels]
  const int64_t units = a.L * a.chunks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const int64_t warp0 = static_cast<int64_t>(blockIdx.x) * kGroups + (threadIdx.x >> 5) * 4;
  for (int64_t base = warp0; base < units; base += step) {  // uniform in the warp
    const int64_t unit = base + ((threadIdx.x >> 3) & 3);
    const bool live = unit < units;
    const int64_t u = live ? unit : units - 1;
    const int64_t t = u / a.chunks;
    const int chunk = static_cast<int>(u - t * a.chunks);
    float c[4], s[4];
    angles(a, freq, ln, t, c, s);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int n = which ? a.Hk : a.H;
      if (n == 0) continue;
      int h0, h1;
      piece(a.H + a.Hk, a.chunks, chunk, which ? a.H : 0, n, h0, h1);
      const int rows = live && h1 > h0 ? h1 - h0 : 0;
      if (h0 > n - 1) h0 = n - 1;
      const int most = __reduce_max_sync(0xffffffffu, rows);
      if (most == 0) continue;
      float wa[4], wb[4];
      const float* w = which ? a.kw : a.qw;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wa[i] = w ? w[ln.ca + i] : 1.f;
        wb[i] = w ? w[ln.cb + i] : 1.f;
      }
      const Stride2 xs = which ? a.ks : a.qs, gs = which ? a.kos : a.qos, ds = which ? a.dks : a.dqs;
      const T* x = static_cast<const T*>(which ? a.k : a.q) + t * xs.tok + h0 * xs.head;
      const G* g = static_cast<const G*>(which ? a.k_out : a.q_out) + t * gs.tok + h0 * gs.head;
      T* d = static_cast<T*>(which ? a.dk : a.dq) + t * ds.tok + h0 * ds.head;
      constexpr int kB = 2;  // rows in flight
      for (int r0 = 0; r0 < most; r0 += kB) {
        Row rx[kB], rg[kB];
#pragma unroll
        for (int v = 0; v < kB; ++v) {
          const int64_t at = r0 + v < rows ? r0 + v : 0;
          rx[v] = load_row(x + at * xs.head, ln.ca, ln.cb);
          rg[v] = load_row(g + at * gs.head, ln.ca, ln.cb);
        }
#pragma unroll
        for (int v = 0; v < kB; ++v) {
          if (r0 + v >= most) break;
          const bool mine = r0 + v < rows;
          const float r = normalise(rx[v], a.norm, a.eps);
          Row h;
          float hx = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float ga = mine ? rg[v].a[i] : 0.f, gb = mine ? rg[v].b[i] : 0.f;
            const float ya = ga * c[i] + gb * s[i], yb = gb * c[i] - ga * s[i];
            if (mine) {
              acc[which][0][i] = fmaf(ya, rx[v].a[i], acc[which][0][i]);
              acc[which][0][4 + i] = fmaf(yb, rx[v].b[i], acc[which][0][4 + i]);
              acc[which][1][i] += ya;
              acc[which][1][4 + i] += yb;
            }
            h.a[i] = ya * wa[i];
            h.b[i] = yb * wb[i];
            hx = fmaf(h.a[i], rx[v].a[i], fmaf(h.b[i], rx[v].b[i], hx));
          }
          float m1 = 0.f, m2 = 0.f;
          if (a.norm != S3R_NORM_NONE) m2 = group_sum(hx) * (1.f / 64);
          if (a.norm == S3R_NORM_LAYER) m1 = group_sum(sum8(h)) * (1.f / 64);
          float da[4], db[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            da[i] = r * (h.a[i] - fmaf(m2, rx[v].a[i], m1));
            db[i] = r * (h.b[i] - fmaf(m2, rx[v].b[i], m1));
          }
          if (mine) {
            store4(d + (r0 + v) * ds.head + ln.ca, da);
            store4(d + (r0 + v) * ds.head + ln.cb, db);
          }
        }
      }
    }
  }
  // the four groups of a warp, then the warps of the block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = acc[which][kind][i];
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (lane < 8) red[warp][which * 2 + kind][(i < 4 ? ln.ca : ln.cb) + (i & 3)] = x;
      }
  __syncthreads();
  const int v = threadIdx.x >> 6, ch = threadIdx.x & 63;
  float x = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) x += red[w][v][ch];
  a.part[static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x] = x;
}

// dw[v][ch] = sum over the blocks' rows: one block per vector, 16 slices of the rows by 64 channels,
// in fp64.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* part, int blocks, float* dw) {
  __shared__ double red[16][64];
  const int ch = threadIdx.x & 63, slice = threadIdx.x >> 6, v = blockIdx.x;
  double x = 0.;
  for (int b = slice; b < blocks; b += 16) x += part[static_cast<int64_t>(b) * 256 + v * 64 + ch];
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

}  // namespace

// As many blocks as have work, at most four per SM (each keeps 32 partial sums a lane).
int qk_norm_bwd_blocks(int64_t L, int H, int Hk) {
  const int64_t units = L * head_chunks(L, H + Hk);
  const int64_t b = (units + kGroups - 1) / kGroups;
  return static_cast<int>(b < 4 * kSMs ? b : 4 * kSMs);
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
  const int blocks = qk_norm_bwd_blocks(a.L, a.H, a.Hk);
  if (blocks > 0 && a.H + a.Hk > 0) {
    a.chunks = head_chunks(a.L, a.H + a.Hk);
    if (dtype == S3R_TYPE_F32 && grad_dtype == S3R_TYPE_F32)
      qk_norm_bwd_kernel<float, float><<<blocks, kThreads, 0, st>>>(a);
    else if (dtype == S3R_TYPE_F32)
      qk_norm_bwd_kernel<float, uint16_t><<<blocks, kThreads, 0, st>>>(a);
    else if (grad_dtype == S3R_TYPE_F32)
      qk_norm_bwd_kernel<uint16_t, float><<<blocks, kThreads, 0, st>>>(a);
    else
      qk_norm_bwd_kernel<uint16_t, uint16_t><<<blocks, kThreads, 0, st>>>(a);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  qk_norm_dw_kernel<<<4, 1024, 0, st>>>(a.part, a.H + a.Hk > 0 ? blocks : 0, dw);
  count_launch();
  return cudaGetLastError();
}

}  // namespace s3r
