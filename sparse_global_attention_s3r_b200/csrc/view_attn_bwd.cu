// view_attn_bwd.cu -- gradients of the dense attention inside segments (view_attn.cu), on the
// sm_100a tensor cores (tcgen05 + TMEM + TMA).
//
// The probabilities are recomputed from q, k and the forward's lse. Per head and segment, with
// t = scale log2(e) <q, k>:
//   P = 2^(t - lse log2 e),  D = <dout, out> per row,  dS = P (dout v^T - D),
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout.
// dq sums over keys, dk and dv over queries. Adding both from one kernel would need either atomics
// (results that change with their order) or a fp32 dq per key tile; two kernels that recompute S
// and dout v^T each (7 products instead of 5, 2 exponentials instead of 1) write every element
// once, in a fixed order:
//   view_dq_kernel    one block per (segment, 128 query rows, head): walks the keys. A TMEM lane is a
//                     query row; dS goes to TMEM as bf16, the A operand of dq += dS k. Also
//                     writes D for the next kernel.
//   view_dkv_kernel   one block per (segment, 128 keys, key head): walks the queries of every head
//                     that shares the key head. A TMEM lane is a key: S^T = k q^T and
//                     (dout v^T)^T = v dout^T, then P^T and dS^T go to TMEM as bf16, the A
//                     operands of dv += P^T dout and dk += dS^T q.
// Both hold S and dP of one 128 x 128 tile in TMEM beside the bf16 operands, so the products of the
// next tile run while the softmax warps work on this one: eight warps, a thread per row and half
// of the columns. What bounds them: the exponential unit (1,024 clocks a tile against 868 and
// 1,224 of products), then issue slots.
// When the blocks are too few to fill the GPU, the walk is split into pieces, whose fp32 sums
// view_sum_kernel adds in order.
//
// P and dS are rounded to bf16 for the products, relative 2^-9 a term; all sums are fp32.
//
// Roles (320 threads): warps 0-7 softmax (lane quadrant warp % 4, column half warp / 4), warp 8 TMA
// producer, warp 9 TMEM owner and MMA issuer. Every wait is bounded in time and watches a block
// abort flag (S3R_DEV_TIMEOUT on expiry).
#include <climits>
#include <cmath>

#include "internal.h"
#include "view_common.cuh"

namespace s3r {
namespace {

using namespace view;

constexpr int kThreads = 320;
constexpr int kTile = 128;
constexpr uint32_t kTileBytes = kTile * 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kIdescQK = idesc_bf16_f32(kTile, kTile, 0, 0);  // both operands K-major
constexpr uint32_t kIdescMN = idesc_bf16_f32(kTile, 64, 0, 1);     // A in TMEM, B MN-major

struct BwdArgs {
  const int32_t *qo, *ko;
  const uint16_t *out, *dout;  // [Lq, H, 64]
  const float* lse;            // [H, Lq]
  float* dsum;                 // [H, Lq]: D
  uint16_t *dq, *dk, *dv;
  Stride2 dqs, dks, dvs;
  float *part0, *part1;  // splits > 1: [splits][rows, heads, 64] f32 (dq; dk and dv)
  int64_t Lq, Lk;
  int H, Hkv, group, nseg, max_q, max_k, tiles, splits;
  float scale, scale_log2;
  uint32_t flags;
  uint32_t* status;
  uint64_t limit_ns;
};

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ float2 pair_of(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// 32 fp32 sums times f -> 64 bytes of bf16 at dst.
__device__ __forceinline__ void store_bf16(uint16_t* dst, const uint32_t (&r)[32], float f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16(__uint_as_float(r[8 * j + 2 * e]) * f, __uint_as_float(r[8 * j + 2 * e + 1]) * f);
    reinterpret_cast<uint4*>(dst)[j] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void store_f32(float* dst, const uint32_t (&r)[32], float f) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    reinterpret_cast<float4*>(dst)[j] =
        make_float4(__uint_as_float(r[4 * j]) * f, __uint_as_float(r[4 * j + 1]) * f,
                    __uint_as_float(r[4 * j + 2]) * f, __uint_as_float(r[4 * j + 3]) * f);
}
// rows [r0, r1) of one head to zero, 8 threads a row
__device__ __forceinline__ void zero_grad(uint16_t* p, const Stride2& s, int head, int64_t r0,
                                          int64_t r1, int64_t first, int64_t step) {
  for (int64_t i = r0 * 8 + first; i < r1 * 8; i += step)
    reinterpret_cast<uint4*>(p + (i >> 3) * s.tok + head * s.head)[i & 7] =
        make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void zero_part(float* p, int heads, int head, int64_t r0, int rows) {
  for (int i = threadIdx.x; i < rows * 16; i += kThreads)
    reinterpret_cast<float4*>(p + ((r0 + (i >> 4)) * heads + head) * 64)[i & 15] =
        make_float4(0.f, 0.f, 0.f, 0.f);
}

// ------------------------------------------------------------------------------------------
// dq
// ------------------------------------------------------------------------------------------
namespace dq {
constexpr int kStages = 5;
constexpr uint32_t kColS = 0, kColDP = 128, kColDQ = 256, kColDS = 320, kTmemCols = 512;
constexpr uint32_t kOffQ = 0, kOffDO = kTileBytes, kOffRing = 2 * kTileBytes;  // stage: K | V
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kOffD = kOffRing + kStages * kStageBytes;  // [2][128] f32: halves of D
constexpr uint32_t kOffBars = kOffD + 1024;
struct __align__(8) Bars {
  uint64_t q_full, k_tail;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full, s_empty, dp_full, dp_empty, ds_full, ds_empty;
  uint64_t o_full, drain, never;
};
constexpr uint32_t kOffMisc = kOffBars + sizeof(Bars);
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a block");
}  // namespace dq

__global__ void __launch_bounds__(kThreads, 1)
    view_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const BwdArgs a) {
  using namespace dq;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.limit_ns;

  uint32_t b = blockIdx.x;
  const int h = b % a.H;
  b /= a.H;
  const int split = b % a.splits;
  b /= a.splits;
  const int tile = b % a.tiles, seg = b / a.tiles;
  if (seg == a.nseg) {  // rows past the last segment (S3R_FLAG_ZERO_TAIL)
    if (split) return;
    const int64_t r0 = a.qo[a.nseg] < 0 ? 0 : a.qo[a.nseg];
    zero_grad(a.dq, a.dqs, h, r0, a.Lq, static_cast<int64_t>(tile) * kThreads + threadIdx.x,
              static_cast<int64_t>(a.tiles) * kThreads);
    return;
  }
  const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
  if (!g.ok) {
    if (threadIdx.x == 0) set_status(a.status, S3R_DEV_BAD_INDEX);
    return;
  }
  const int row0 = tile * kTile;
  if (row0 >= g.nq) return;
  const int rows = g.nq - row0 < kTile ? g.nq - row0 : kTile;
  const int all = (g.nk + kTile - 1) / kTile, per = (all + a.splits - 1) / a.splits;
  const int t0 = split * per, n = all - t0 < per ? all - t0 : per;
  float* part = a.splits > 1 ? a.part0 + static_cast<int64_t>(split) * a.Lq * a.H * 64 : nullptr;
  if (n <= 0) {
    if (part)
      zero_part(part, a.H, h, g.q0 + row0, rows);
    else
      zero_grad(a.dq, a.dqs, h, g.q0 + row0, g.q0 + row0 + rows, threadIdx.x, kThreads);
    return;
  }
  const int tail = g.nk - (t0 + n - 1) * kTile;  // keys of the last tile

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->k_tail, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_empty, 8);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->dp_empty, 8);
    mbar_init(&bars->ds_full, 8);
    mbar_init(&bars->ds_empty, 1);
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->never, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmO);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 9) tmem_alloc(tmem_holder, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;

  // D of the block's rows: each of the two column-half warps of a row takes 32 channels
  const int qd = warp & 3, half = warp >> 2, r = qd * 32 + lane;
  float lse2 = 0.f, dsum = 0.f;
  if (warp < 8) {
    if (r < rows) {
      const int64_t row = g.q0 + row0 + r;
      const uint4* o = reinterpret_cast<const uint4*>(a.out + (row * a.H + h) * 64 + 32 * half);
      const uint4* d = reinterpret_cast<const uint4*>(a.dout + (row * a.H + h) * 64 + 32 * half);
      lse2 = a.lse[h * a.Lq + row] * kLog2e;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = o[j], y = d[j];
        dsum += bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x);
        dsum += bf16_lo(x.y) * bf16_lo(y.y) + bf16_hi(x.y) * bf16_hi(y.y);
        dsum += bf16_lo(x.z) * bf16_lo(y.z) + bf16_hi(x.z) * bf16_hi(y.z);
        dsum += bf16_lo(x.w) * bf16_lo(y.w) + bf16_hi(x.w) * bf16_hi(y.w);
      }
    }
    float* sd = reinterpret_cast<float*>(smem + kOffD);
    sd[half * kTile + r] = dsum;
    asm volatile("bar.sync 1, 256;\n" ::: "memory");  // the eight softmax warps
    dsum = sd[r] + sd[kTile + r];
    if (r < rows && half == 0 && split == 0) a.dsum[h * a.Lq + g.q0 + row0 + r] = dsum;
  }

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    const int hk = h / a.group;
    bool ok = true, cut = false;
    int issued = 0;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars->q_full, 2 * kTileBytes);
      tma_load_rows(sbase + kOffQ, &tmQ, h, g.q0 + row0, &bars->q_full);
      tma_load_rows(sbase + kOffDO, &tmO, h, g.q0 + row0, &bars->q_full);
    }
    for (int t = 0; t < n; ++t) {
      const int st = t % kStages;
      const uint32_t par = ((t / kStages) & 1) ^ 1, sk = sbase + kOffRing + st * kStageBytes;
      const int32_t y = g.k0 + (t0 + t) * kTile;
      cut = t == n - 1 && tail < kTile;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_empty[st], par, abort, lim)))) break;
      if (lane == 0) {
        uint64_t* full = cut ? &bars->k_tail : &bars->k_full[st];
        mbar_arrive_expect_tx(full, kTileBytes);
        tma_load_rows(sk, &tmK, hk, y, full);
      }
      issued = 2 * t + 1;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_empty[st], par, abort, lim)))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->v_full[st], kTileBytes);
        tma_load_rows(sk + kTileBytes, &tmV, hk, y, &bars->v_full[st]);
      }
      issued = 2 * t + 2;
    }
    if (ok && cut) {  // the last key tile reaches past the segment
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_tail, 0, abort, lim));
      if (ok) {
        const int st = (n - 1) % kStages;
        zero_rows(smem + kOffRing + st * kStageBytes, tail, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->k_full[st]);
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, a.status);
      int dummy = 0;
      mbar_wait(&bars->q_full, 0, &dummy, lim);
      for (int i = issued - 1; i >= 0 && i >= issued - 2 * kStages; --i) {
        const int t = i >> 1, st = t % kStages;
        if (i & 1)
          mbar_wait(&bars->v_full[st], (t / kStages) & 1, &dummy, lim);
        else if (t == n - 1 && tail < kTile)
          mbar_wait(&bars->k_tail, 0, &dummy, lim);
        else
          mbar_wait(&bars->k_full[st], (t / kStages) & 1, &dummy, lim);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      bool ok = mbar_wait(&bars->q_full, 0, abort, lim);
      const uint64_t dqd = desc_sw128(sbase + kOffQ), dod = desc_sw128(sbase + kOffDO);
      auto scores = [&](int t) -> bool {  // S = q k^T, dP = dout v^T
        const int st = t % kStages;
        const uint32_t sk = sbase + kOffRing + st * kStageBytes;
        const uint64_t dk = desc_sw128(sk), dv = desc_sw128(sk + kTileBytes);
        if (!mbar_wait(&bars->k_full[st], (t / kStages) & 1, abort, lim)) return false;
        if (!mbar_wait(&bars->s_empty, (t & 1) ^ 1, abort, lim)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(tbase + kColS, dqd + 2 * ks, dk + 2 * ks, kIdescQK, ks > 0);
        tc_commit(&bars->s_full);
        if (!mbar_wait(&bars->v_full[st], (t / kStages) & 1, abort, lim)) return false;
        if (!mbar_wait(&bars->dp_empty, (t & 1) ^ 1, abort, lim)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(tbase + kColDP, dod + 2 * ks, dv + 2 * ks, kIdescQK, ks > 0);
        tc_commit(&bars->dp_full);
        tc_commit(&bars->v_empty[st]);
        return true;
      };
      auto grad = [&](int t) -> bool {  // dq += dS k
        const int st = t % kStages;
        if (!mbar_wait(&bars->ds_full, t & 1, abort, lim)) return false;
        tc_fence_after();
        const uint64_t dk = desc_sw128(sbase + kOffRing + st * kStageBytes);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 keys a step: 16 rows x 128 B = 2048 B
          mma_ts(tbase + kColDQ, tbase + kColDS + ks * 8, dk + 128 * ks, kIdescMN,
                 (t > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&bars->ds_empty);
        tc_commit(&bars->k_empty[st]);
        return true;
      };
      if (ok) ok = scores(0);
      for (int t = 0; ok && t < n; ++t) {
        if (t + 1 < n && !(ok = scores(t + 1))) break;
        ok = grad(t);
      }
      if (ok) {
        tc_commit(&bars->o_full);
      } else {
        raise_abort(abort, a.status);
        int dummy = 0;
        tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, &dummy, lim);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warps
    const bool idle = qd * 32 >= rows;  // no rows: only keeps the barriers going
    const uint32_t tl = tbase + (static_cast<uint32_t>(qd * 32) << 16);
    const float2 mul = make_float2(a.scale_log2, a.scale_log2), off = make_float2(-lse2, -lse2);
    const float2 nd = make_float2(-dsum, -dsum);
    bool ok = true;
    if (a.flags & S3R_FLAG_TEST_TIMEOUT) ok = mbar_wait(&bars->never, 0, abort, lim);
    for (int t = 0; ok && t < n; ++t) {
      if (!(ok = mbar_wait(&bars->s_full, t & 1, abort, lim))) break;
      tc_fence_after();
      uint32_t s0[32], s1[32], d0[32], d1[32];
      if (!idle) {
        tmem_ld32(tl + kColS + 64 * half, s0);
        tmem_ld32(tl + kColS + 64 * half + 32, s1);
        tmem_wait_ld_regs(s0);
        tmem_wait_ld_regs(s1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_empty);
      if (!(ok = mbar_wait(&bars->dp_full, t & 1, abort, lim))) break;
      tc_fence_after();
      if (!idle) {
        tmem_ld32(tl + kColDP + 64 * half, d0);
        tmem_ld32(tl + kColDP + 64 * half + 32, d1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = __ffma2_rn(pair_of(s0[2 * i], s0[2 * i + 1]), mul, off);
          const float2 y = __ffma2_rn(pair_of(s1[2 * i], s1[2 * i + 1]), mul, off);
          s0[2 * i] = __float_as_uint(exp2_approx(x.x));
          s0[2 * i + 1] = __float_as_uint(exp2_approx(x.y));
          s1[2 * i] = __float_as_uint(exp2_approx(y.x));
          s1[2 * i + 1] = __float_as_uint(exp2_approx(y.y));
        }
        tmem_wait_ld_regs(d0);
        tmem_wait_ld_regs(d1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->dp_empty);
      uint32_t p[32];
      if (!idle) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = __fmul2_rn(pair_of(s0[2 * i], s0[2 * i + 1]),
                                      __fadd2_rn(pair_of(d0[2 * i], d0[2 * i + 1]), nd));
          const float2 y = __fmul2_rn(pair_of(s1[2 * i], s1[2 * i + 1]),
                                      __fadd2_rn(pair_of(d1[2 * i], d1[2 * i + 1]), nd));
          p[i] = pack_bf16(x.x, x.y);
          p[16 + i] = pack_bf16(y.x, y.y);
        }
        if (t == n - 1 && tail < kTile) {  // keys past the segment's end
          const int left = tail - 64 * half;  // columns of this half that count
#pragma unroll
          for (int i = 0; i < 32; ++i)
            p[i] = 2 * i + 1 < left ? p[i] : 2 * i < left ? (p[i] & 0xffffu) : 0u;
        }
      }
      if (!(ok = mbar_wait(&bars->ds_empty, (t & 1) ^ 1, abort, lim))) break;
      if (!idle) {
        tc_fence_after();
        tmem_st32(tl + kColDS + 32 * half, p);
        tmem_wait_st_regs(p);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ds_full);
    }
    if (ok && (ok = mbar_wait(&bars->o_full, 0, abort, lim)) && !idle) {
      tc_fence_after();
      uint32_t o[32];
      tmem_ld32(tl + kColDQ + 32 * half, o);
      tmem_wait_ld_regs(o);
      if (r < rows) {
        const int64_t row = g.q0 + row0 + r;
        if (part)
          store_f32(part + (row * a.H + h) * 64 + 32 * half, o, a.scale);
        else
          store_bf16(a.dq + row * a.dqs.tok + h * a.dqs.head + 32 * half, o, a.scale);
      }
    }
    if (!ok) raise_abort(abort, a.status);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tbase, kTmemCols);
}

// ------------------------------------------------------------------------------------------
// dk, dv
// ------------------------------------------------------------------------------------------
namespace dkv {
constexpr int kStages = 5;
constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 320, kColP = 384, kColDS = 448,
                   kTmemCols = 512;
constexpr uint32_t kOffK = 0, kOffV = kTileBytes, kOffRing = 2 * kTileBytes;  // stage: q | dout
constexpr uint32_t kStageBytes = 2 * kTileBytes;
// per stage: [2][128] f32, -lse log2 e and -D of the stage's queries
constexpr uint32_t kOffStat = kOffRing + kStages * kStageBytes;
constexpr uint32_t kOffBars = kOffStat + kStages * 1024;
struct __align__(8) Bars {
  uint64_t kv_full, q_tail;
  uint64_t full[kStages], empty[kStages], stat[kStages];
  uint64_t s_full, s_empty, dp_full, dp_empty, p_full, p_empty, ds_full, ds_empty;
  uint64_t o_full, drain, never;
};
constexpr uint32_t kOffMisc = kOffBars + sizeof(Bars);
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a block");
}  // namespace dkv

__global__ void __launch_bounds__(kThreads, 1)
    view_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const BwdArgs a) {
  using namespace dkv;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.limit_ns;

  uint32_t b = blockIdx.x;
  const int hk = b % a.Hkv;
  b /= a.Hkv;
  const int split = b % a.splits;
  b /= a.splits;
  const int tile = b % a.tiles, seg = b / a.tiles;
  if (seg == a.nseg) {  // rows past the last segment (S3R_FLAG_ZERO_TAIL)
    if (split) return;
    const int64_t r0 = a.ko[a.nseg] < 0 ? 0 : a.ko[a.nseg];
    const int64_t first = static_cast<int64_t>(tile) * kThreads + threadIdx.x;
    zero_grad(a.dk, a.dks, hk, r0, a.Lk, first, static_cast<int64_t>(a.tiles) * kThreads);
    zero_grad(a.dv, a.dvs, hk, r0, a.Lk, first, static_cast<int64_t>(a.tiles) * kThreads);
    return;
  }
  const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
  if (!g.ok) {
    if (threadIdx.x == 0) set_status(a.status, S3R_DEV_BAD_INDEX);
    return;
  }
  const int row0 = tile * kTile;
  if (row0 >= g.nk) return;
  const int rows = g.nk - row0 < kTile ? g.nk - row0 : kTile;
  // steps: (head of the group, query tile), the tile fastest
  const int qt = (g.nq + kTile - 1) / kTile;
  const int all = qt * a.group, per = (all + a.splits - 1) / a.splits;
  const int t0 = split * per, n = all - t0 < per ? all - t0 : per;
  const int64_t part_at = static_cast<int64_t>(split) * a.Lk * a.Hkv * 64;
  if (n <= 0) {
    if (a.splits > 1) {
      zero_part(a.part0 + part_at, a.Hkv, hk, g.k0 + row0, rows);
      zero_part(a.part1 + part_at, a.Hkv, hk, g.k0 + row0, rows);
    } else {
      zero_grad(a.dk, a.dks, hk, g.k0 + row0, g.k0 + row0 + rows, threadIdx.x, kThreads);
      zero_grad(a.dv, a.dvs, hk, g.k0 + row0, g.k0 + row0 + rows, threadIdx.x, kThreads);
    }
    return;
  }
  const int tail = g.nq - (qt - 1) * kTile;  // queries of a head's last tile

  if (threadIdx.x == 0) {
    mbar_init(&bars->kv_full, 1);
    mbar_init(&bars->q_tail, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
      mbar_init(&bars->stat[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_empty, 8);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->dp_empty, 8);
    mbar_init(&bars->p_full, 8);
    mbar_init(&bars->p_empty, 1);
    mbar_init(&bars->ds_full, 8);
    mbar_init(&bars->ds_empty, 1);
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->never, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmO);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 9) tmem_alloc(tmem_holder, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    bool ok = true;
    int issued = 0, tails = 0;
    bool last_cut = false;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars->kv_full, 2 * kTileBytes);
      tma_load_rows(sbase + kOffK, &tmK, hk, g.k0 + row0, &bars->kv_full);
      tma_load_rows(sbase + kOffV, &tmV, hk, g.k0 + row0, &bars->kv_full);
    }
    // the lane's four queries of a step: -lse log2 e and -D, or (past the segment's end) -inf and
    // 0, which make P and dS zero
    float nl[4], nd[4];
    auto fetch = [&](int t) {
      const int s = t0 + t, hh = hk * a.group + s / qt, y = (s % qt) * kTile;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = y + c * 32 + lane;
        const int64_t at = hh * a.Lq + g.q0 + i;
        nl[c] = i < g.nq ? -a.lse[at] * kLog2e : -INFINITY;
        nd[c] = i < g.nq ? -a.dsum[at] : 0.f;
      }
    };
    fetch(0);
    for (int t = 0; t < n; ++t) {
      const int st = t % kStages;
      const int s = t0 + t, hh = hk * a.group + s / qt, y = (s % qt) * kTile;
      const uint32_t sq = sbase + kOffRing + st * kStageBytes;
      const bool cut = s % qt == qt - 1 && tail < kTile;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->empty[st], ((t / kStages) & 1) ^ 1, abort,
                                                   lim))))
        break;
      if (lane == 0) {
        uint64_t* full = cut ? &bars->q_tail : &bars->full[st];
        mbar_arrive_expect_tx(full, 2 * kTileBytes);
        tma_load_rows(sq, &tmQ, hh, g.q0 + y, full);
        tma_load_rows(sq + kTileBytes, &tmO, hh, g.q0 + y, full);
      }
      issued = t + 1;
      last_cut = cut;
      float* stat = reinterpret_cast<float*>(smem + kOffStat + st * 1024);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        stat[c * 32 + lane] = nl[c];
        stat[kTile + c * 32 + lane] = nd[c];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->stat[st]);
      if (t + 1 < n) fetch(t + 1);
      if (cut) {  // the tile reaches past the segment's queries
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_tail, tails & 1, abort, lim)))) break;
        last_cut = false;
        ++tails;
        uint8_t* qp = smem + kOffRing + st * kStageBytes;
        zero_rows(qp, tail, lane);
        zero_rows(qp + kTileBytes, tail, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->full[st]);
      }
    }
    if (!ok && lane == 0) {
      raise_abort(abort, a.status);
      int dummy = 0;
      mbar_wait(&bars->kv_full, 0, &dummy, lim);
      if (last_cut) mbar_wait(&bars->q_tail, tails & 1, &dummy, lim);
      for (int t = issued - 1 - (last_cut ? 1 : 0); t >= 0 && t >= issued - kStages; --t)
        mbar_wait(&bars->full[t % kStages], (t / kStages) & 1, &dummy, lim);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      bool ok = mbar_wait(&bars->kv_full, 0, abort, lim);
      const uint64_t dkd = desc_sw128(sbase + kOffK), dvd = desc_sw128(sbase + kOffV);
      auto scores = [&](int t) -> bool {  // S^T = k q^T, dP^T = v dout^T
        const int st = t % kStages;
        const uint32_t sq = sbase + kOffRing + st * kStageBytes;
        const uint64_t dqd = desc_sw128(sq), dod = desc_sw128(sq + kTileBytes);
        if (!mbar_wait(&bars->full[st], (t / kStages) & 1, abort, lim)) return false;
        if (!mbar_wait(&bars->s_empty, (t & 1) ^ 1, abort, lim)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(tbase + kColS, dkd + 2 * ks, dqd + 2 * ks, kIdescQK, ks > 0);
        tc_commit(&bars->s_full);
        if (!mbar_wait(&bars->dp_empty, (t & 1) ^ 1, abort, lim)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(tbase + kColDP, dvd + 2 * ks, dod + 2 * ks, kIdescQK, ks > 0);
        tc_commit(&bars->dp_full);
        return true;
      };
      auto grads = [&](int t) -> bool {  // dv += P^T dout, dk += dS^T q
        const int st = t % kStages;
        const uint32_t sq = sbase + kOffRing + st * kStageBytes;
        const uint64_t dqd = desc_sw128(sq), dod = desc_sw128(sq + kTileBytes);
        if (!mbar_wait(&bars->p_full, t & 1, abort, lim)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 queries a step: 16 rows x 128 B = 2048 B
          mma_ts(tbase + kColDV, tbase + kColP + ks * 8, dod + 128 * ks, kIdescMN,
                 (t > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&bars->p_empty);
        if (!mbar_wait(&bars->ds_full, t & 1, abort, lim)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts(tbase + kColDK, tbase + kColDS + ks * 8, dqd + 128 * ks, kIdescMN,
                 (t > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&bars->ds_empty);
        tc_commit(&bars->empty[st]);
        return true;
      };
      if (ok) ok = scores(0);
      for (int t = 0; ok && t < n; ++t) {
        if (t + 1 < n && !(ok = scores(t + 1))) break;
        ok = grads(t);
      }
      if (ok) {
        tc_commit(&bars->o_full);
      } else {
        raise_abort(abort, a.status);
        int dummy = 0;
        tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, &dummy, lim);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warps
    const int qd = warp & 3, half = warp >> 2, r = qd * 32 + lane;
    const bool idle = qd * 32 >= rows;
    const uint32_t tl = tbase + (static_cast<uint32_t>(qd * 32) << 16);
    const float2 mul = make_float2(a.scale_log2, a.scale_log2);
    bool ok = true;
    if (a.flags & S3R_FLAG_TEST_TIMEOUT) ok = mbar_wait(&bars->never, 0, abort, lim);
    for (int t = 0; ok && t < n; ++t) {
      const int st = t % kStages;
      const float4* nl = reinterpret_cast<const float4*>(smem + kOffStat + st * 1024 + half * 256);
      const float4* nd = nl + 32;  // 128 floats on
      if (!(ok = mbar_wait(&bars->stat[st], (t / kStages) & 1, abort, lim))) break;
      if (!(ok = mbar_wait(&bars->s_full, t & 1, abort, lim))) break;
      tc_fence_after();
      uint32_t s0[32], s1[32], d0[32], d1[32], p[32];
      if (!idle) {
        tmem_ld32(tl + kColS + 64 * half, s0);
        tmem_ld32(tl + kColS + 64 * half + 32, s1);
        tmem_wait_ld_regs(s0);
        tmem_wait_ld_regs(s1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_empty);
      if (!idle) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 l0 = nl[i], l1 = nl[8 + i];
          const float2 x0 = __ffma2_rn(pair_of(s0[4 * i], s0[4 * i + 1]), mul, make_float2(l0.x, l0.y));
          const float2 x1 = __ffma2_rn(pair_of(s0[4 * i + 2], s0[4 * i + 3]), mul, make_float2(l0.z, l0.w));
          const float2 y0 = __ffma2_rn(pair_of(s1[4 * i], s1[4 * i + 1]), mul, make_float2(l1.x, l1.y));
          const float2 y1 = __ffma2_rn(pair_of(s1[4 * i + 2], s1[4 * i + 3]), mul, make_float2(l1.z, l1.w));
          const float e0 = exp2_approx(x0.x), e1 = exp2_approx(x0.y), e2 = exp2_approx(x1.x),
                      e3 = exp2_approx(x1.y);
          const float f0 = exp2_approx(y0.x), f1 = exp2_approx(y0.y), f2 = exp2_approx(y1.x),
                      f3 = exp2_approx(y1.y);
          p[2 * i] = pack_bf16(e0, e1);
          p[2 * i + 1] = pack_bf16(e2, e3);
          p[16 + 2 * i] = pack_bf16(f0, f1);
          p[16 + 2 * i + 1] = pack_bf16(f2, f3);
          s0[4 * i] = __float_as_uint(e0), s0[4 * i + 1] = __float_as_uint(e1);
          s0[4 * i + 2] = __float_as_uint(e2), s0[4 * i + 3] = __float_as_uint(e3);
          s1[4 * i] = __float_as_uint(f0), s1[4 * i + 1] = __float_as_uint(f1);
          s1[4 * i + 2] = __float_as_uint(f2), s1[4 * i + 3] = __float_as_uint(f3);
        }
      }
      if (!(ok = mbar_wait(&bars->p_empty, (t & 1) ^ 1, abort, lim))) break;
      if (!idle) {
        tc_fence_after();
        tmem_st32(tl + kColP + 32 * half, p);
        tmem_wait_st_regs(p);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full);
      if (!(ok = mbar_wait(&bars->dp_full, t & 1, abort, lim))) break;
      tc_fence_after();
      if (!idle) {
        tmem_ld32(tl + kColDP + 64 * half, d0);
        tmem_ld32(tl + kColDP + 64 * half + 32, d1);
        tmem_wait_ld_regs(d0);
        tmem_wait_ld_regs(d1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->dp_empty);
      if (!idle) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 c0 = nd[i], c1 = nd[8 + i];
          const float2 x0 = __fmul2_rn(pair_of(s0[4 * i], s0[4 * i + 1]),
                                       __fadd2_rn(pair_of(d0[4 * i], d0[4 * i + 1]), make_float2(c0.x, c0.y)));
          const float2 x1 = __fmul2_rn(pair_of(s0[4 * i + 2], s0[4 * i + 3]),
                                       __fadd2_rn(pair_of(d0[4 * i + 2], d0[4 * i + 3]), make_float2(c0.z, c0.w)));
          const float2 y0 = __fmul2_rn(pair_of(s1[4 * i], s1[4 * i + 1]),
                                       __fadd2_rn(pair_of(d1[4 * i], d1[4 * i + 1]), make_float2(c1.x, c1.y)));
          const float2 y1 = __fmul2_rn(pair_of(s1[4 * i + 2], s1[4 * i + 3]),
                                       __fadd2_rn(pair_of(d1[4 * i + 2], d1[4 * i + 3]), make_float2(c1.z, c1.w)));
          p[2 * i] = pack_bf16(x0.x, x0.y);
          p[2 * i + 1] = pack_bf16(x1.x, x1.y);
          p[16 + 2 * i] = pack_bf16(y0.x, y0.y);
          p[16 + 2 * i + 1] = pack_bf16(y1.x, y1.y);
        }
      }
      if (!(ok = mbar_wait(&bars->ds_empty, (t & 1) ^ 1, abort, lim))) break;
      if (!idle) {
        tc_fence_after();
        tmem_st32(tl + kColDS + 32 * half, p);
        tmem_wait_st_regs(p);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ds_full);
    }
    if (ok && (ok = mbar_wait(&bars->o_full, 0, abort, lim)) && !idle) {
      tc_fence_after();
      uint32_t v[32], k[32];
      tmem_ld32(tl + kColDV + 32 * half, v);
      tmem_ld32(tl + kColDK + 32 * half, k);
      tmem_wait_ld_regs(v);
      tmem_wait_ld_regs(k);
      if (r < rows) {
        const int64_t row = g.k0 + row0 + r;
        if (a.splits > 1) {
          const int64_t at = part_at + (row * a.Hkv + hk) * 64 + 32 * half;
          store_f32(a.part0 + at, k, a.scale);
          store_f32(a.part1 + at, v, 1.f);
        } else {
          store_bf16(a.dk + row * a.dks.tok + hk * a.dks.head + 32 * half, k, a.scale);
          store_bf16(a.dv + row * a.dvs.tok + hk * a.dvs.head + 32 * half, v, 1.f);
        }
      }
    }
    if (!ok) raise_abort(abort, a.status);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tbase, kTmemCols);
}

// grad[row, head] = the pieces' sums, added in piece order; 16 lanes a (row, head). Rows outside
// the segments are not touched.
__global__ void __launch_bounds__(256) view_sum_kernel(const float* part, int splits, int64_t rows,
                                                       int heads, const int32_t* offs, int nseg,
                                                       uint16_t* grad, Stride2 s) {
  const int64_t pair = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
  if (pair >= rows * heads) return;
  const int64_t row = pair / heads;
  const int h = static_cast<int>(pair - row * heads), c = threadIdx.x & 15;
  if (row < offs[0] || row >= offs[nseg]) return;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < splits; ++i) {
    const float4 y = *reinterpret_cast<const float4*>(
        part + (static_cast<int64_t>(i) * rows * heads + pair) * 64 + 4 * c);
    x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
  }
  *reinterpret_cast<uint2*>(grad + row * s.tok + h * s.head + 4 * c) =
      make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

constexpr int kSMs = 148;
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Pieces a walk of `steps` tiles is split into for `base` blocks: the count with the shortest
// estimated time in tile times (about 0.8 us): waves of blocks, each its steps plus a start of
// about 3, and for more than one piece the summing kernel (about 5 and its traffic).
int pieces(int64_t base, int64_t steps, int64_t out_rows) {
  if (base == 0 || base >= 4 * kSMs || steps < 4) return 1;
  int best = 1;
  double best_t = 1e300;
  for (int64_t s = 1; s <= 128 && s <= steps / 2; ++s) {
    const double t = static_cast<double>(ceil_div(base * s, kSMs)) * (ceil_div(steps, s) + 3) +
                     (s > 1 ? 5. + static_cast<double>(s) * out_rows * 512 / 5e6 : 0.);
    if (t < best_t) {
      best_t = t;
      best = static_cast<int>(s);
    }
  }
  return best;
}

struct ViewBwdLayout {
  int sq, skv;  // pieces of the dq and of the dk/dv walks
  size_t dsum, dq, dk, dv, total;
};
ViewBwdLayout bwd_layout(const ViewProblem& p) {
  const int64_t tq = ceil_div(p.max_q, kTile), tk = ceil_div(p.max_k, kTile);
  const size_t qrows = static_cast<size_t>(p.Lq) * p.H, krows = static_cast<size_t>(p.Lk) * p.Hkv;
  ViewBwdLayout l{};
  l.sq = pieces(tq * p.nseg * p.H, tk, qrows);
  l.skv = pieces(tk * p.nseg * p.Hkv, tq * (p.H / p.Hkv), 2 * krows);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += round256(bytes);
    return x;
  };
  l.dsum = take(qrows * 4);
  l.dq = take(l.sq > 1 ? l.sq * qrows * 256 : 0);
  l.dk = take(l.skv > 1 ? l.skv * krows * 256 : 0);
  l.dv = take(l.skv > 1 ? l.skv * krows * 256 : 0);
  l.total = at < 256 ? 256 : at;
  return l;
}

template <typename K>
cudaError_t allow_smem(K kernel, uint32_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

size_t view_bwd_workspace(const ViewProblem& p) { return bwd_layout(p).total; }

cudaError_t launch_view_bwd(const ViewProblem& p, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const int32_t* qo, const int32_t* ko,
                            const uint16_t* out, const float* lse, const uint16_t* dout,
                            uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, cudaStream_t st) {
  const ViewBwdLayout l = bwd_layout(p);
  uint8_t* w = static_cast<uint8_t*>(ws);
  CUtensorMap tq, to, tk, tv;
  // a tensor without rows is never loaded: any valid map stands in for its own
  const bool has_q = p.Lq > 0, has_k = p.Lk > 0;
  if (!has_q && !has_k) return cudaSuccess;
  const Stride2 dense{static_cast<int64_t>(p.H) * 64, 64};
  if (has_q && (!make_tmap_rows3(&tq, q, p.Lq, p.H, p.qs) || !make_tmap_rows3(&to, dout, p.Lq, p.H, dense)))
    return cudaErrorInvalidValue;
  if (has_k && (!make_tmap_rows3(&tk, k, p.Lk, p.Hkv, p.ks) || !make_tmap_rows3(&tv, v, p.Lk, p.Hkv, p.vs)))
    return cudaErrorInvalidValue;
  if (!has_q) tq = to = tk;
  if (!has_k) tk = tv = tq;
  cudaError_t e = allow_smem(view_dq_kernel, dq::kSmemBytes);
  if (e == cudaSuccess) e = allow_smem(view_dkv_kernel, dkv::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t segs = p.nseg + ((p.flags & S3R_FLAG_ZERO_TAIL) ? 1 : 0);
  BwdArgs a{qo, ko, out, dout, lse, reinterpret_cast<float*>(w + l.dsum), dq, dk, dv, p.dqs, p.dks,
            p.dvs, nullptr, nullptr, p.Lq, p.Lk, p.H, p.Hkv, p.H / p.Hkv, p.nseg, p.max_q, p.max_k,
            0, 0, p.scale, p.scale_log2, p.flags, p.status,
            (p.flags & S3R_FLAG_TEST_TIMEOUT) ? 1000000ull : 2000000000ull};
  if (has_q) {
    a.tiles = static_cast<int>(p.max_q > 0 ? ceil_div(p.max_q, kTile) : 1);
    a.splits = l.sq;
    a.part0 = reinterpret_cast<float*>(w + l.dq);
    const int64_t blocks = segs * a.tiles * a.splits * p.H;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    view_dq_kernel<<<static_cast<unsigned>(blocks), kThreads, dq::kSmemBytes, st>>>(tq, to, tk, tv, a);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (l.sq > 1) {
      view_sum_kernel<<<static_cast<unsigned>(ceil_div(p.Lq * p.H * 16, 256)), 256, 0, st>>>(
          a.part0, l.sq, p.Lq, p.H, qo, p.nseg, dq, p.dqs);
      count_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  }
  if (has_k) {
    a.tiles = static_cast<int>(p.max_k > 0 ? ceil_div(p.max_k, kTile) : 1);
    a.splits = l.skv;
    a.part0 = reinterpret_cast<float*>(w + l.dk);
    a.part1 = reinterpret_cast<float*>(w + l.dv);
    const int64_t blocks = segs * a.tiles * a.splits * p.Hkv;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    view_dkv_kernel<<<static_cast<unsigned>(blocks), kThreads, dkv::kSmemBytes, st>>>(tq, to, tk, tv, a);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (l.skv > 1) {
      const unsigned grid = static_cast<unsigned>(ceil_div(p.Lk * p.Hkv * 16, 256));
      view_sum_kernel<<<grid, 256, 0, st>>>(a.part0, l.skv, p.Lk, p.Hkv, ko, p.nseg, dk, p.dks);
      count_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      view_sum_kernel<<<grid, 256, 0, st>>>(a.part1, l.skv, p.Lk, p.Hkv, ko, p.nseg, dv, p.dvs);
      count_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace s3r
