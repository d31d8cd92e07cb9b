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

// A lane's eight channels of one row, two a word: pair i's first is half i % 2 of a[i / 2], its second
// that of b[i / 2]. The packed fp32 instructions halve what the arithmetic has to issue (137,400 tokens
// of 16 + 16 heads forward: 222 -> 207 us).
struct Row {
  float2 a[2], b[2];
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
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
// The forward's rows in flight wait in shared memory, not in registers: a thread copies its own two
// pieces of a row there (cp.async) and reads them back itself, so no barrier is needed. Four rows ahead
// and four blocks an SM took 207 to 189 us in a burst; three and six ahead 193 and 195. (The backward, with two
// rows in registers, was slower with such a ring: 130 against 119 us.)
template <typename V>
__device__ __forceinline__ void copy_piece(V* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "n"(sizeof(V))
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>  // all but the newest N groups have landed
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
template <typename T>
using Piece = decltype(Raw<T>::a);
template <typename T, int kDepth>
struct Ring {
  Piece<T> a[kDepth][kThreads], b[kDepth][kThreads];
  __device__ __forceinline__ void fetch(int slot, const T* row, int ca, int cb) {
    copy_piece(&a[slot][threadIdx.x], row + ca);
    copy_piece(&b[slot][threadIdx.x], row + cb);
  }
  __device__ __forceinline__ Raw<T> get(int slot) const {
    return {a[slot][threadIdx.x], b[slot][threadIdx.x]};
  }
};
__device__ __forceinline__ void unpack4(uint2 u, float2 (&v)[2]) {
  v[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  v[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void unpack4(float4 u, float2 (&v)[2]) {
  v[0] = make_float2(u.x, u.y), v[1] = make_float2(u.z, u.w);
}
template <typename T>
__device__ __forceinline__ Row unpack(const Raw<T>& r) {
  Row x;
  unpack4(r.a, x.a);
  unpack4(r.b, x.b);
  return x;
}
__device__ __forceinline__ void store4(uint16_t* p, const float2 (&v)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y));
}
__device__ __forceinline__ void store4(float* p, const float2 (&v)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
// Two neighbouring values of a vector, or a constant where there is none.
__device__ __forceinline__ float2 two_of(const float* p, int i, float none) {
  return p ? make_float2(p[i], p[i + 1]) : both(none);
}

// Sum over the 8 lanes of a group.
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 4);
}
__device__ __forceinline__ float sum8(const Row& r) {
  const float2 x = __fadd2_rn(__fadd2_rn(r.a[0], r.a[1]), __fadd2_rn(r.b[0], r.b[1]));
  return x.x + x.y;
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
__device__ __forceinline__ void angles(const QKNormArgs& a, const Lane& ln, int64_t t, float2 (&c)[2],
                                       float2 (&s)[2]) {
  if (a.rope == S3R_ROPE_NONE) {
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = both(1.f), s[i] = both(0.f);
    return;
  }
  const double p = a.rope == S3R_ROPE_2D ? a.pos[2 * t + (ln.first_axis ? 0 : 1)] : a.pos[t];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double* freq = a.freq + 4 * (threadIdx.x & 7) + 2 * i;
    const double x = p * freq[0], y = p * freq[1];  // in half turns
    sincospif(static_cast<float>(x - 2. * rint(0.5 * x)), &s[i].x, &c[i].x);
    sincospif(static_cast<float>(y - 2. * rint(0.5 * y)), &s[i].y, &c[i].y);
  }
}

// x -> x - m in place (layer norm); returns r.
__device__ __forceinline__ float centre(Row& x, int norm, float eps) {
  if (norm == S3R_NORM_NONE) return 1.f;
  if (norm == S3R_NORM_LAYER) {
    const float2 m = both(group_sum(sum8(x)) * (-1.f / 64));
#pragma unroll
    for (int i = 0; i < 2; ++i) x.a[i] = __fadd2_rn(x.a[i], m), x.b[i] = __fadd2_rn(x.b[i], m);
  }
  float2 q = __fmul2_rn(x.a[0], x.a[0]);
  q = __ffma2_rn(x.b[0], x.b[0], q);
  q = __ffma2_rn(x.a[1], x.a[1], q);
  q = __ffma2_rn(x.b[1], x.b[1], q);
  return rsqrtf(fmaf(group_sum(q.x + q.y), 1.f / 64, eps));
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
//
// 137,400 tokens of 16 + 16 heads in bf16: 189 us (5.95 TB/s, 0.91 of a plain copy's rate) in a burst of a
// dozen passes; 218 us (5.2 TB/s, 0.79) in a long run of them, when the power limit lowers the clock to 1.6
// GHz. 43,968 tokens in fp32: 127 us (5.7 TB/s).
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_fwd_kernel(const __grid_constant__ QKNormArgs a) {
  constexpr int kDepth = 8 / sizeof(T);  // rows in flight a group: 64 KB an SM
  __shared__ Ring<T, kDepth> ring;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + (threadIdx.x >> 3);
  const int64_t units = a.L * a.chunks;
  const bool live = unit < units;
  const int64_t u = live ? unit : units - 1;
  const int chunk = a.chunks == 1 ? 0 : static_cast<int>(u / a.L);
  const int64_t t = u - chunk * a.L;
  const Lane ln = lane_channels(a.rope);
  int h0[2], rows[2], most[2];  // of the query and the key list
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    int h1;
    piece(a.H + a.Hk, a.chunks, chunk, which ? a.H : 0, which ? a.Hk : a.H, h0[which], h1);
    rows[which] = live && h1 > h0[which] ? h1 - h0[which] : 0;
    if (rows[which] == 0) h0[which] = 0;
    most[which] = __reduce_max_sync(0xffffffffu, rows[which]);
  }
  // the next row to fetch: step f of the warp's walk over both lists
  int f = 0;
  const T* x = static_cast<const T*>(a.q) + t * a.qs.tok + h0[0] * a.qs.head;
  auto fetch = [&](int slot) {
    if (f == most[0]) x = static_cast<const T*>(a.k) + t * a.ks.tok + h0[1] * a.ks.head;
    const bool k = f >= most[0];
    if (k ? f - most[0] < rows[1] : f < rows[0]) ring.fetch(slot, x, ln.ca, ln.cb);
    copies_done();
    x += k ? a.ks.head : a.qs.head;
    ++f;
  };
#pragma unroll
  for (int v = 0; v < kDepth; ++v) fetch(v);
  float2 c[2], s[2];
  angles(a, ln, t, c, s);
  int slot = 0;
  for (int which = 0; which < 2; ++which) {
    if (most[which] == 0) continue;
    const int64_t yh = which ? a.kos.head : a.qos.head;
    T* y = static_cast<T*>(which ? a.k_out : a.q_out) + t * (which ? a.kos.tok : a.qos.tok) + h0[which] * yh;
    const float *w = which ? a.kw : a.qw, *b = which ? a.kb : a.qb;
    float2 ac[2], as[2], bc[2], bs[2], oa[2], ob[2];  // wa c, wa s, wb c, -wb s; the turned bias
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 wa = two_of(w, ln.ca + 2 * i, 1.f), wb = two_of(w, ln.cb + 2 * i, 1.f);
      const float2 ba = two_of(b, ln.ca + 2 * i, 0.f), bb = two_of(b, ln.cb + 2 * i, 0.f);
      const float2 ns = make_float2(-s[i].x, -s[i].y);
      ac[i] = __fmul2_rn(wa, c[i]), as[i] = __fmul2_rn(wa, s[i]);
      bc[i] = __fmul2_rn(wb, c[i]), bs[i] = __fmul2_rn(wb, ns);
      oa[i] = __ffma2_rn(ba, c[i], __fmul2_rn(bb, ns));
      ob[i] = __ffma2_rn(bb, c[i], __fmul2_rn(ba, s[i]));
    }
    for (int r0 = 0; r0 < most[which]; ++r0) {
      copies_wait<kDepth - 1>();
      Row d = unpack(ring.get(slot));  // a group without the row works on what the slot holds
      fetch(slot);
      slot = slot + 1 < kDepth ? slot + 1 : 0;
      const float r = centre(d, a.norm, a.eps);
      float2 ya[2], yb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ya[i] = __ffma2_rn(both(r), __ffma2_rn(d.b[i], bs[i], __fmul2_rn(d.a[i], ac[i])), oa[i]);
        yb[i] = __ffma2_rn(both(r), __ffma2_rn(d.a[i], as[i], __fmul2_rn(d.b[i], bc[i])), ob[i]);
      }
      if (r0 < rows[which]) {
        store4(y + ln.ca, ya);
        store4(y + ln.cb, yb);
      }
      y += yh;
    }
  }
}

// Backward: the blocks below q_blocks walk the queries' tokens with a grid stride, the others the
// keys', keeping the weights' gradients of a lane's eight channels in registers; they are added up
// over the block at the end and written as one row of `part`, which qk_norm_dw_kernel adds in block
// order. A group takes two rows at once, so that one's row sums (three dependent shuffles each, three
// times) run in the other's shadow: 43,968 tokens of 16 + 16 heads in bf16 132 -> 119 us (4.5 TB/s),
// though it leaves two blocks an SM instead of three. What is left is issue and the latency of those
// sums: DRAM alone would need 82 us.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads, 2)
    qk_norm_bwd_kernel(const __grid_constant__ QKNormArgs a, int q_blocks) {
  __shared__ float red[kThreads / 32][2][64];
  constexpr int kRows = 2;  // at once, and as many in flight
  const bool which = static_cast<int>(blockIdx.x) >= q_blocks;
  const int block = which ? blockIdx.x - q_blocks : blockIdx.x;
  const int blocks = which ? gridDim.x - q_blocks : q_blocks;
  const int n = which ? a.Hk : a.H, chunks = a.chunks < n ? a.chunks : n;
  const Lane ln = lane_channels(a.rope);
  float2 dw[2][2] = {}, db[2][2] = {};  // [first or second of a pair][two pairs]
  const float* w = which ? a.kw : a.qw;
  float2 wa[2], wb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    wa[i] = two_of(w, ln.ca + 2 * i, 1.f);
    wb[i] = two_of(w, ln.cb + 2 * i, 1.f);
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
    Raw<T> rx[kRows] = {};
    Raw<G> rg[kRows] = {};
#pragma unroll
    for (int v = 0; v < kRows; ++v) {
      if (v < rows) {
        rx[v] = load_raw(x, ln.ca, ln.cb);
        rg[v] = load_raw(g, ln.ca, ln.cb);
      }
      x += xh;
      g += gh;
    }
    float2 c[2], s[2];
    angles(a, ln, t, c, s);
    for (int r0 = 0; r0 < most; r0 += kRows) {
      Row xr[kRows], h[kRows];
      float r[kRows], hx[kRows];
      float2 ya[kRows][2], yb[kRows][2];
#pragma unroll
      for (int v = 0; v < kRows; ++v) {
        xr[v] = unpack(rx[v]);
        const Row gr = unpack(rg[v]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 ns = make_float2(-s[i].x, -s[i].y);
          ya[v][i] = __ffma2_rn(gr.b[i], s[i], __fmul2_rn(gr.a[i], c[i]));
          yb[v][i] = __ffma2_rn(gr.a[i], ns, __fmul2_rn(gr.b[i], c[i]));
        }
        if (r0 + v + kRows < rows) {
          rx[v] = load_raw(x, ln.ca, ln.cb);
          rg[v] = load_raw(g, ln.ca, ln.cb);
        }
        x += xh;
        g += gh;
      }
      if (a.norm == S3R_NORM_LAYER) {
        float m[kRows];
#pragma unroll
        for (int v = 0; v < kRows; ++v) m[v] = sum8(xr[v]);
#pragma unroll
        for (int z = 1; z < 8; z *= 2)
#pragma unroll
          for (int v = 0; v < kRows; ++v) m[v] += __shfl_xor_sync(0xffffffffu, m[v], z);
#pragma unroll
        for (int v = 0; v < kRows; ++v)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            xr[v].a[i] = __fadd2_rn(xr[v].a[i], both(m[v] * (-1.f / 64)));
            xr[v].b[i] = __fadd2_rn(xr[v].b[i], both(m[v] * (-1.f / 64)));
          }
      }
#pragma unroll
      for (int v = 0; v < kRows; ++v) r[v] = 1.f;
      if (a.norm != S3R_NORM_NONE) {
        float q[kRows];
#pragma unroll
        for (int v = 0; v < kRows; ++v) {
          float2 y = __fmul2_rn(xr[v].a[0], xr[v].a[0]);
          y = __ffma2_rn(xr[v].b[0], xr[v].b[0], y);
          y = __ffma2_rn(xr[v].a[1], xr[v].a[1], y);
          y = __ffma2_rn(xr[v].b[1], xr[v].b[1], y);
          q[v] = y.x + y.y;
        }
#pragma unroll
        for (int z = 1; z < 8; z *= 2)
#pragma unroll
          for (int v = 0; v < kRows; ++v) q[v] += __shfl_xor_sync(0xffffffffu, q[v], z);
#pragma unroll
        for (int v = 0; v < kRows; ++v) r[v] = rsqrtf(fmaf(q[v], 1.f / 64, a.eps));
      }
#pragma unroll
      for (int v = 0; v < kRows; ++v) {
        const bool mine = r0 + v < rows;
        float2 y = both(0.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          xr[v].a[i] = __fmul2_rn(xr[v].a[i], both(r[v]));
          xr[v].b[i] = __fmul2_rn(xr[v].b[i], both(r[v]));
          if (mine) {
            dw[0][i] = __ffma2_rn(ya[v][i], xr[v].a[i], dw[0][i]);
            dw[1][i] = __ffma2_rn(yb[v][i], xr[v].b[i], dw[1][i]);
            db[0][i] = __fadd2_rn(db[0][i], ya[v][i]);
            db[1][i] = __fadd2_rn(db[1][i], yb[v][i]);
          }
          h[v].a[i] = __fmul2_rn(ya[v][i], wa[i]);
          h[v].b[i] = __fmul2_rn(yb[v][i], wb[i]);
          y = __ffma2_rn(h[v].a[i], xr[v].a[i], __ffma2_rn(h[v].b[i], xr[v].b[i], y));
        }
        hx[v] = y.x + y.y;
      }
      float m1[kRows];
#pragma unroll
      for (int v = 0; v < kRows; ++v) m1[v] = sum8(h[v]);
      if (a.norm != S3R_NORM_NONE) {
#pragma unroll
        for (int z = 1; z < 8; z *= 2)
#pragma unroll
          for (int v = 0; v < kRows; ++v) {
            hx[v] += __shfl_xor_sync(0xffffffffu, hx[v], z);
            m1[v] += __shfl_xor_sync(0xffffffffu, m1[v], z);
          }
      }
#pragma unroll
      for (int v = 0; v < kRows; ++v) {
        const float2 n1 = both(a.norm == S3R_NORM_LAYER ? -r[v] * m1[v] * (1.f / 64) : 0.f);
        const float2 n2 = both(a.norm != S3R_NORM_NONE ? -r[v] * hx[v] * (1.f / 64) : 0.f);
        float2 ga[2], gb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ga[i] = __ffma2_rn(n2, xr[v].a[i], __ffma2_rn(both(r[v]), h[v].a[i], n1));
          gb[i] = __ffma2_rn(n2, xr[v].b[i], __ffma2_rn(both(r[v]), h[v].b[i], n1));
        }
        if (r0 + v < rows) {
          store4(d + ln.ca, ga);
          store4(d + ln.cb, gb);
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
      const float2 v = kind ? db[i >> 2][i >> 1 & 1] : dw[i >> 2][i >> 1 & 1];
      float x = i & 1 ? v.y : v.x;
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

// Blocks of one list of the backward: as many as have work, at most two per SM for both lists
// together (what is resident), shared by their heads.
int list_blocks(int64_t L, int n, int total) {
  if (n == 0 || L == 0) return 0;
  const int chunks = head_chunks(L, total);
  const int64_t need = (L * (chunks < n ? chunks : n) + kGroups - 1) / kGroups;
  const int64_t most = static_cast<int64_t>(2) * kSMs * n / total;
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
