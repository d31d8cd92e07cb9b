// view_attn.cu -- dense attention of every query over the keys of its own segment, on the sm_100a
// tensor cores (tcgen05 + TMEM + TMA).
//
// Per head and segment, with t = scale log2(e) <q, k>:  out = sum_j 2^(t_j - m) v_j / l with
// l = sum_j 2^(t_j - m), one pass over the keys. m is a row's reference, not its running maximum:
// it is set by the first key tile and moves, with O and l rescaled, only when a logit passes it by
// more than 2^8, so the rescaling is rare and P stays below 2^8 (bf16 keeps its relative precision
// at any size). lse = (m + log2 l) ln 2.
//
// One block per (segment, 256 query rows, head, piece of the keys) and one block per SM. A block
// holds two units, each 128 query rows (a TMEM lane a row) with its own S (fp32, 128 columns),
// P (bf16, 64 columns) and O (fp32, 64 columns) in TMEM, 512 columns in all, and its own four
// softmax warps, one thread a row: row maxima and sums need no exchange. While one unit's
// exponentials run, the other unit's and the next tile's products do: S of the next tile is issued
// as soon as the softmax warps have S of this one in registers.
//   two tiles   (more than 128 rows) unit u has rows 128 u .. 128 u + 127, and each key tile feeds
//               both units
//   one tile    (128 rows or fewer, down to one) both units have the same rows and take the key
//               tiles in turn, unit u those of parity u; unit 0 joins the two results at the end.
//               For a few rows this is bound by reading the keys, and the softmax of one warp
//               alone would not keep up with that; warps without rows do nothing.
// What bounds it at many rows: the exponential unit, 16 per clock per SM against 256 FLOP of products
// each. A share of the exponentials therefore runs as a polynomial on the FMA pipe (kPolyOf8 of every
// 8 pairs).
// When there are too few blocks to fill the GPU, the keys are split into pieces (view_fwd_splits)
// whose fp32 results view_join_kernel adds, in order.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax of unit 0 and 1 (lane quadrant warp % 4), warp 8
// TMA producer, warp 9 TMEM owner and MMA issuer, warps 10-11 idle (they complete the warpgroup that
// hands its registers to the softmax warps). Every wait is bounded in time and watches a block
// abort flag (S3R_DEV_TIMEOUT on expiry).
#include <climits>
#include <cmath>

#include "internal.h"
#include "view_common.cuh"

namespace s3r {
namespace {

using namespace view;

constexpr int kThreads = 384;
// registers a thread: 168 at launch (3 warps per sub-partition), then split between the softmax
// warpgroups and the third one; 2 * 216 + 72 = 3 * 168
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr int kStages = 6;  // key and value tiles in flight
constexpr int kRows = 256;  // query rows of a block
constexpr int kTile = 128;  // rows of a unit, keys of a tile
constexpr uint32_t kTileBytes = kTile * 128;
constexpr float kMoveRef = 8.f;  // base-2 margin before a row's reference moves
#ifndef S3R_VIEW_POLY
#define S3R_VIEW_POLY 2
#endif
constexpr int kPolyOf8 = S3R_VIEW_POLY;

constexpr uint32_t kColS = 0, kColP = 256, kColO = 384, kTmemCols = 512;  // unit u: +128u, +64u, +64u
constexpr uint32_t kIdescQK = idesc_bf16_f32(kTile, kTile, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16_f32(kTile, 64, 0, 1);

struct __align__(8) Bars {
  uint64_t q_full;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t v_tail;                 // TMA of a value tile that is cut by the segment's end
  uint64_t s_full[2], s_empty[2];  // S of a unit written / read into registers
  uint64_t p_full[2], p_empty[2];  // P written / its product with V completed
  uint64_t o_full[2];              // every product of the unit completed
  uint64_t joined;                 // one tile: unit 1's result is in shared memory
  uint64_t drain;
  uint64_t never;  // never signalled: waited on only under S3R_FLAG_TEST_TIMEOUT
};
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = 2 * kTileBytes;
constexpr uint32_t kOffV = kOffK + kStages * kTileBytes;
constexpr uint32_t kOffJoin = kOffK;  // [64][128] f32 over the first two key stages, once drained
constexpr uint32_t kOffML = kOffV + kStages * kTileBytes;  // [2][128] f32: m and l of unit 1
constexpr uint32_t kOffBars = kOffML + 1024;
constexpr uint32_t kOffMisc = kOffBars + sizeof(Bars);
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a block");

struct FwdArgs {
  const int32_t *qo, *ko;
  uint16_t* out;  // [Lq, H, 64] bf16
  float* lse;     // [H, Lq] or null
  float* o_part;  // splits > 1: [splits][Lq, H, 64] f32
  float* l_part;  // splits > 1: [splits][H, Lq], in base-2 units
  int64_t Lq, Lk;
  int H, group, nseg, max_q, max_k, tiles, splits;
  float scale_log2;
  uint32_t flags;
  uint32_t* status;
  uint64_t limit_ns;
};

// Columns [from, 128) of a row's tile to -inf.
template <int N>
__device__ __forceinline__ void mask_from(uint32_t (&r)[N], int from) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i >= from) r[i] = 0xff800000u;
}

// 32 logits -> 16 packed pairs of P; adds them to sum (two running sums).
__device__ __forceinline__ void exp_chunk(const uint32_t (&s)[32], float sl2, float m,
                                          uint32_t (&p)[16], float2& sum) {
  const float2 mul = make_float2(sl2, sl2), off = make_float2(-m, -m);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = __ffma2_rn(
        make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), mul, off);
    const float2 e = (i & 7) < kPolyOf8 ? exp2_poly5x2(x)
                                        : make_float2(exp2_approx(x.x), exp2_approx(x.y));
    sum = __fadd2_rn(sum, e);
    p[i] = pack_bf16(e.x, e.y);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    view_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const FwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.limit_ns;

  // block -> (segment, row tile, key piece, head), heads fastest: the blocks that run together
  // read whole token rows
  uint32_t b = blockIdx.x;
  const int h = b % a.H;
  b /= a.H;
  const int split = b % a.splits;
  b /= a.splits;
  const int tile = b % a.tiles;
  const int seg = b / a.tiles;

  if (seg == a.nseg) {  // rows past the last segment (S3R_FLAG_ZERO_TAIL)
    if (split) return;
    int64_t r = a.qo[a.nseg];
    if (r < 0) r = 0;
    for (r += static_cast<int64_t>(tile) * kThreads + threadIdx.x; r < a.Lq;
         r += static_cast<int64_t>(a.tiles) * kThreads) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (r * a.H + h) * 64);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse) a.lse[h * a.Lq + r] = -INFINITY;
    }
    return;
  }
  const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
  if (!g.ok) {
    if (threadIdx.x == 0) set_status(a.status, S3R_DEV_BAD_INDEX);
    return;
  }
  const int row0 = tile * kRows;
  if (row0 >= g.nq) return;
  const int rows = g.nq - row0 < kRows ? g.nq - row0 : kRows;
  // key tiles [t0, t0 + n) of the segment
  const int all = (g.nk + kTile - 1) / kTile;
  const int per = (all + a.splits - 1) / a.splits;
  const int t0 = split * per;
  const int n = all - t0 < per ? all - t0 : per;
  if (n <= 0) {  // no keys: zeros, or an empty piece
    if (a.splits > 1) {
      for (int r = threadIdx.x; r < rows; r += kThreads)
        a.l_part[(static_cast<int64_t>(split) * a.H + h) * a.Lq + g.q0 + row0 + r] = -INFINITY;
      return;
    }
    for (int i = threadIdx.x; i < rows * 8; i += kThreads) {
      const int64_t r = g.q0 + row0 + (i >> 3);
      reinterpret_cast<uint4*>(a.out + (r * a.H + h) * 64)[i & 7] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse && (i & 7) == 0) a.lse[h * a.Lq + r] = -INFINITY;
    }
    return;
  }
  const bool one = rows <= kTile;            // one tile: the units take the key tiles in turn
  const int steps = one ? n : 2 * n;         // (unit, key tile) pairs; unit = step & 1
  const int tail = g.nk - (t0 + n - 1) * kTile;  // keys of the last tile, 1 .. 128

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    mbar_init(&bars->v_tail, 1);
    for (int u = 0; u < 2; ++u) {
      mbar_init(&bars->s_full[u], 1);
      mbar_init(&bars->s_empty[u], 4);
      mbar_init(&bars->p_full[u], 4);
      mbar_init(&bars->p_empty[u], 1);
      mbar_init(&bars->o_full[u], 1);
    }
    mbar_init(&bars->joined, 4);
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->never, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 9) tmem_alloc(tmem_holder, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  if (warp >= 8) {
  regs_dec<kRegsOther>();
  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    const int hk = h / a.group;
    bool ok = true;
    int issued = 0;
    bool cut = false;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars->q_full, one ? kTileBytes : 2 * kTileBytes);
      tma_load_rows(sbase + kOffQ, &tmQ, h, g.q0 + row0, &bars->q_full);
      if (!one)
        tma_load_rows(sbase + kOffQ + kTileBytes, &tmQ, h, g.q0 + row0 + kTile, &bars->q_full);
    }
    for (int t = 0; t < n; ++t) {
      const int st = t % kStages;
      const uint32_t par = ((t / kStages) & 1) ^ 1;
      const int32_t y = g.k0 + (t0 + t) * kTile;
      cut = t == n - 1 && tail < kTile;
      // every lane waits, so that the warp stays together and all lanes see the tile
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_empty[st], par, abort, lim)))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->k_full[st], kTileBytes);
        tma_load_rows(sbase + kOffK + st * kTileBytes, &tmK, hk, y, &bars->k_full[st]);
      }
      issued = 2 * t + 1;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_empty[st], par, abort, lim)))) break;
      if (lane == 0) {
        uint64_t* full = cut ? &bars->v_tail : &bars->v_full[st];
        mbar_arrive_expect_tx(full, kTileBytes);
        tma_load_rows(sbase + kOffV + st * kTileBytes, &tmV, hk, y, full);
      }
      issued = 2 * t + 2;
    }
    if (ok && cut) {  // the last value tile reaches past the segment
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_tail, 0, abort, lim));
      if (ok) {
        const int st = (n - 1) % kStages;
        zero_rows(smem + kOffV + st * kTileBytes, tail, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_full[st]);
      }
    }
    if (!ok && lane == 0) {  // let the copies in flight land before the block ends
      raise_abort(abort, a.status);
      int dummy = 0;
      mbar_wait(&bars->q_full, 0, &dummy, lim);
      for (int i = issued - 1; i >= 0 && i >= issued - 2 * kStages; --i) {
        const int t = i >> 1, st = t % kStages;
        if (!(i & 1))
          mbar_wait(&bars->k_full[st], (t / kStages) & 1, &dummy, lim);
        else if (t == n - 1 && tail < kTile)
          mbar_wait(&bars->v_tail, 0, &dummy, lim);
        else
          mbar_wait(&bars->v_full[st], (t / kStages) & 1, &dummy, lim);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      bool ok = mbar_wait(&bars->q_full, 0, abort, lim);
      // step s: unit s & 1 and key tile s >> 1 (two tiles) or s (one tile); the unit's own count of
      // steps is s >> 1 either way
      auto qk = [&](int s) -> bool {
        const int u = s & 1, t = one ? s : s >> 1, i = s >> 1, st = t % kStages;
        if (!mbar_wait(&bars->k_full[st], (t / kStages) & 1, abort, lim)) return false;
        if (!mbar_wait(&bars->s_empty[u], (i & 1) ^ 1, abort, lim)) return false;
        tc_fence_after();
        const uint64_t dq = desc_sw128(sbase + kOffQ + (one ? 0 : u * kTileBytes));
        const uint64_t dk = desc_sw128(sbase + kOffK + st * kTileBytes);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(tbase + kColS + u * 128, dq + 2 * ks, dk + 2 * ks, kIdescQK, ks > 0);
        tc_commit(&bars->s_full[u]);
        if (one || u) tc_commit(&bars->k_empty[st]);
        return true;
      };
      auto pv = [&](int s) -> bool {
        const int u = s & 1, t = one ? s : s >> 1, i = s >> 1, st = t % kStages;
        if (!mbar_wait(&bars->v_full[st], (t / kStages) & 1, abort, lim)) return false;
        if (!mbar_wait(&bars->p_full[u], i & 1, abort, lim)) return false;
        tc_fence_after();
        const uint64_t dv = desc_sw128(sbase + kOffV + st * kTileBytes);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 keys a step: 16 rows x 128 B = 2048 B
          mma_ts(tbase + kColO + u * 64, tbase + kColP + u * 64 + ks * 8, dv + 128 * ks, kIdescPV,
                 (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&bars->p_empty[u]);
        if (one || u) tc_commit(&bars->v_empty[st]);
        return true;
      };
      if (ok) ok = qk(0);
      if (ok && steps > 1) ok = qk(1);
      for (int s = 0; ok && s < steps; ++s) {
        if (s + 2 < steps && !(ok = qk(s + 2))) break;
        ok = pv(s);
        if (ok && s + 2 >= steps) tc_commit(&bars->o_full[s & 1]);
      }
      if (!ok) {
        raise_abort(abort, a.status);
        int dummy = 0;
        tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, &dummy, lim);
      }
    }
  }
  } else {
  regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax warps
    const int u = warp >> 2, qd = warp & 3;
    const int r = (one ? 0 : u * kTile) + qd * 32 + lane;  // row of the block
    const int mine = one ? (n - u + 1) >> 1 : n;           // key tiles of this unit
    // a warp whose 32 rows are all past the end only keeps the barriers going: what its lanes of
    // P hold reaches no other lane of O
    const bool idle = (one ? 0 : u * kTile) + qd * 32 >= rows;
    const uint32_t tl = tbase + (static_cast<uint32_t>(qd * 32) << 16);
    const uint32_t tS = tl + kColS + u * 128, tP = tl + kColP + u * 64, tO = tl + kColO + u * 64;
    const float sl2 = a.scale_log2;
    float m = 0.f;
    float2 sum = make_float2(0.f, 0.f);
    bool ok = true;
    if (a.flags & S3R_FLAG_TEST_TIMEOUT) ok = mbar_wait(&bars->never, 0, abort, lim);
    for (int i = 0; ok && i < mine; ++i) {
      if (!(ok = mbar_wait(&bars->s_full[u], i & 1, abort, lim))) break;
      tc_fence_after();
      uint32_t s0[32], s1[32], s2[32], s3[32];
      if (!idle) {
        tmem_ld32(tS, s0);
        tmem_ld32(tS + 32, s1);
        tmem_ld32(tS + 64, s2);
        tmem_ld32(tS + 96, s3);
        tmem_wait_ld_regs(s0);
        tmem_wait_ld_regs(s1);
        tmem_wait_ld_regs(s2);
        tmem_wait_ld_regs(s3);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_empty[u]);
      const int t = one ? 2 * i + u : i;
      if (idle) {
        if (!(ok = mbar_wait(&bars->p_empty[u], (i & 1) ^ 1, abort, lim))) break;
        if (lane == 0) mbar_arrive(&bars->p_full[u]);
        continue;
      }
      if (t == n - 1 && tail < kTile) {  // keys past the segment's end
        mask_from(s0, tail);
        mask_from(s1, tail - 32);
        mask_from(s2, tail - 64);
        mask_from(s3, tail - 96);
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t(&s)[32] = c == 0 ? s0 : c == 1 ? s1 : c == 2 ? s2 : s3;
        float x = fmax3_nan(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
        float y = fmax3_nan(__uint_as_float(s[3]), __uint_as_float(s[4]), __uint_as_float(s[5]));
#pragma unroll
        for (int j = 6; j + 3 < 32; j += 4) {
          x = fmax3_nan(x, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          y = fmax3_nan(y, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
        }
        x = fmax3_nan(x, __uint_as_float(s[30]), __uint_as_float(s[31]));
        mx[c] = fmax3_nan(x, y, y);
      }
      const float top = fmax3_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * sl2;
      if (i == 0) {
        m = top == -INFINITY ? 0.f : top;
      } else if (__any_sync(0xffffffffu, !(top <= m + kMoveRef))) {
        // move the reference: O so far has to be complete, and is rescaled in place
        if (!(ok = mbar_wait(&bars->p_empty[u], (i & 1) ^ 1, abort, lim))) break;
        tc_fence_after();
        const float to = !(top <= m + kMoveRef) ? top : m;
        const float f = exp2_approx(m - to);
        m = to;
        sum = __fmul2_rn(sum, make_float2(f, f));
        uint32_t o[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_st32(tO + 32 * c, o);
          tmem_wait_st_regs(o);
        }
      }
      uint32_t p[16];
      exp_chunk(s0, sl2, m, p, sum);
      if (!(ok = mbar_wait(&bars->p_empty[u], (i & 1) ^ 1, abort, lim))) break;
      tc_fence_after();
      tmem_st32x16(tP, p);
      exp_chunk(s1, sl2, m, p, sum);
      tmem_st32x16(tP + 16, p);
      exp_chunk(s2, sl2, m, p, sum);
      tmem_st32x16(tP + 32, p);
      exp_chunk(s3, sl2, m, p, sum);
      tmem_st32x16(tP + 48, p);
      tmem_wait_st_keep16(p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full[u]);
    }
    // the unit's result, joined with the other unit's where they share rows
    if (ok && mine > 0) ok = mbar_wait(&bars->o_full[u], 0, abort, lim);
    const bool join = one && n > 1;
    if (ok && join && u == 1) {
      // the ring is free once both units' products are done
      ok = mbar_wait(&bars->o_full[0], 0, abort, lim);
    }
    if (ok && mine > 0 && !(join && u == 0 && idle)) {
      tc_fence_after();
      float l = sum.x + sum.y;
      uint32_t o0[32], o1[32];
      if (!idle) {
        tmem_ld32(tO, o0);
        tmem_ld32(tO + 32, o1);
        tmem_wait_ld_regs(o0);
        tmem_wait_ld_regs(o1);
      }
      float* jo = reinterpret_cast<float*>(smem + kOffJoin);
      float* ml = reinterpret_cast<float*>(smem + kOffML);
      if (join && u == 1) {
        if (!idle) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            jo[j * kTile + r] = __uint_as_float(o0[j]);
            jo[(j + 32) * kTile + r] = __uint_as_float(o1[j]);
          }
          ml[r] = m;
          ml[kTile + r] = l;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->joined);
      } else {
        if (join && (ok = mbar_wait(&bars->joined, 0, abort, lim))) {
          const float m1 = ml[r], l1 = ml[kTile + r];
          const float to = fmax3_nan(m, m1, m1);
          const float f0 = exp2_approx(m - to), f1 = exp2_approx(m1 - to);
          m = to;
          l = l * f0 + l1 * f1;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            o0[j] = __float_as_uint(fmaf(__uint_as_float(o0[j]), f0, jo[j * kTile + r] * f1));
            o1[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), f0, jo[(j + 32) * kTile + r] * f1));
          }
        }
        if (ok && r < rows) {
          const float inv = 1.f / l;
          const int64_t row = g.q0 + row0 + r;
          if (a.splits > 1) {
            float4* dst = reinterpret_cast<float4*>(
                a.o_part + ((static_cast<int64_t>(split) * a.Lq + row) * a.H + h) * 64);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t* o = j < 8 ? &o0[4 * j] : &o1[4 * (j - 8)];
              dst[j] = make_float4(__uint_as_float(o[0]) * inv, __uint_as_float(o[1]) * inv,
                                   __uint_as_float(o[2]) * inv, __uint_as_float(o[3]) * inv);
            }
            a.l_part[(static_cast<int64_t>(split) * a.H + h) * a.Lq + row] = m + log2f(l);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(a.out + (row * a.H + h) * 64);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t* o = j < 4 ? &o0[8 * j] : &o1[8 * (j - 4)];
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
              dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (a.lse) a.lse[h * a.Lq + row] = (m + log2f(l)) * kLn2;
          }
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

// out = sum_s 2^(l_s - l) o_s with l = log2 sum_s 2^(l_s): the pieces' results, each already divided
// by its own sum. 16 lanes a (row, head), 4 channels each. A piece without keys has l_s = -inf and
// its o_s was not written.
__global__ void __launch_bounds__(256) view_join_kernel(const FwdArgs a) {
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t pair = gid >> 4;
  if (pair >= a.Lq * a.H) return;
  const int64_t row = pair / a.H;
  const int h = static_cast<int>(pair - row * a.H);
  const bool tail = row >= a.qo[a.nseg];
  if (row < a.qo[0] || tail) return;  // outside the segments (the tail is the other kernel's)
  const int c = threadIdx.x & 15;
  const float* lp = a.l_part + h * a.Lq + row;
  const int64_t ls = a.H * a.Lq;
  float top = -INFINITY;
  bool nan = false;
  for (int s = 0; s < a.splits; ++s) {
    const float l = lp[s * ls];
    top = fmaxf(top, l);
    nan |= l != l;
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  if (top > -INFINITY || nan) {
    for (int s = 0; s < a.splits; ++s) {
      const float l = lp[s * ls];
      if (l == -INFINITY) continue;
      const float w = exp2_approx(l - top);
      const float4 x = *reinterpret_cast<const float4*>(
          a.o_part + ((static_cast<int64_t>(s) * a.Lq + row) * a.H + h) * 64 + 4 * c);
      total += w;
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
    const float inv = 1.f / total;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  }
  *reinterpret_cast<uint2*>(a.out + pair * 64 + 4 * c) =
      make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
  if (a.lse && c == 0) a.lse[h * a.Lq + row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
}

constexpr int kSMs = 148;
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

// Pieces of the keys: the count with the shortest estimated time, in key-tile times of a block
// (about 0.7 us): waves of blocks, each its tiles plus a start of about 3, and for more than one
// piece the joining kernel (about 6 and its traffic).
int view_fwd_splits(const ViewProblem& p) {
  const int64_t base = ceil_div(p.max_q, kRows) * p.nseg * p.H, tk = ceil_div(p.max_k, kTile);
  if (base == 0 || base >= 4 * kSMs || tk < 4) return 1;
  int best = 1;
  double best_t = 1e300;
  for (int64_t s = 1; s <= 128 && s <= tk / 2; ++s) {
    const double t = static_cast<double>(ceil_div(base * s, kSMs)) * (ceil_div(tk, s) + 3) +
                     (s > 1 ? 6. + static_cast<double>(s) * p.Lq * p.H * 512 / 4.5e6 : 0.);
    if (t < best_t) {
      best_t = t;
      best = static_cast<int>(s);
    }
  }
  return best;
}

size_t view_fwd_workspace(const ViewProblem& p) {
  const size_t s = view_fwd_splits(p), rows = static_cast<size_t>(p.Lq) * p.H;
  return s > 1 ? round256(s * rows * 64 * 4) + round256(s * rows * 4) : 0;
}

cudaError_t launch_view_fwd(const ViewProblem& p, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const int32_t* qo, const int32_t* ko,
                            uint16_t* out, float* lse, void* ws, cudaStream_t st) {
  if (p.Lq == 0) return cudaSuccess;
  CUtensorMap tq, tk, tv;
  if (!make_tmap_rows3(&tq, q, p.Lq, p.H, p.qs)) return cudaErrorInvalidValue;
  tk = tv = tq;  // without keys nothing is loaded through these
  if (p.Lk > 0 &&
      (!make_tmap_rows3(&tk, k, p.Lk, p.Hkv, p.ks) || !make_tmap_rows3(&tv, v, p.Lk, p.Hkv, p.vs)))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(view_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  const int splits = view_fwd_splits(p);
  const size_t rows = static_cast<size_t>(p.Lq) * p.H;
  float* o_part = splits > 1 ? static_cast<float*>(ws) : nullptr;
  float* l_part = splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                                        round256(splits * rows * 64 * 4))
                             : nullptr;
  const int64_t tiles = p.max_q > 0 ? ceil_div(p.max_q, kRows) : 1;
  const int64_t segs = p.nseg + ((p.flags & S3R_FLAG_ZERO_TAIL) ? 1 : 0);
  const int64_t blocks = segs * tiles * splits * p.H;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  FwdArgs a{qo, ko, out, lse, o_part, l_part, p.Lq, p.Lk, p.H, p.H / p.Hkv, p.nseg, p.max_q,
            p.max_k, static_cast<int>(tiles), splits, p.scale_log2, p.flags, p.status,
            (p.flags & S3R_FLAG_TEST_TIMEOUT) ? 1000000ull : 2000000000ull};
  view_fwd_kernel<<<static_cast<unsigned>(blocks), kThreads, kSmemBytes, st>>>(tq, tk, tv, a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess || splits == 1) return e;
  view_join_kernel<<<static_cast<unsigned>(ceil_div(static_cast<int64_t>(rows) * 16, 256)), 256, 0,
                     st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace s3r
