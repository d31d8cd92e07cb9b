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
//   view_d_kernel     D of every (row, head), from out as the forward rounded it
//   view_dq_kernel    item: (segment, 128 query rows, head); walks the keys. A TMEM lane is a query
//                     row; dS goes to TMEM as bf16, the A operand of dq += dS k.
//   view_dkv_kernel   item: (segment, 128 keys, key head); walks the queries of every head that
//                     shares the key head. A TMEM lane is a key: S^T = k q^T and
//                     (dout v^T)^T = v dout^T, then P^T and dS^T go to TMEM as bf16, the A
//                     operands of dv += P^T dout and dk += dS^T q.
// Both are persistent, one block per SM: the next item's tiles are on their way while this one's
// result is written. Both hold S and dP of one 128 x 128 tile in TMEM beside the bf16 operands, so
// the products of the next tile run while the softmax warps work on this one: eight warps, a thread
// per row and half of the columns. (Sixteen warps of a quarter each spilled registers: 2.3 against 1.2
// ms at 32 views of 1,374 tokens and 16 heads.) A warp packs eight pairs of columns while the next
// eight's exponentials run, and the tests of the barriers it will wait on are made ahead, since even a
// wait that is over takes about 100 clocks.
// What bounds them: the exponential unit, 1,024 clocks a tile, or the products, 868 (dq) and 1,224 (dk,
// dv); a tile takes about 1,850 and 2,050, the rest being what a warp does before its first and after
// its last exponential (all eight warps work on the same tile, so the exponential unit is idle then), and
// 4,000 and 5,500 more an item. 32 views take 1.04 ms in a burst of a dozen passes, and 1.18 ms in a long
// run of them, when the power limit lowers the clock to 1.7 GHz.
// When the items are too few to fill the GPU, the walks are split into pieces, whose fp32 sums
// view_sum_kernel adds in order.
//
// P and dS are rounded to bf16 for the products, relative 2^-8 a term at most; all sums are fp32.
//
// Roles (384 threads): warps 0-7 softmax (lane quadrant warp % 4, column half warp / 4), warp 8 TMA
// producer, warp 9 issuer of S and dP (owns the TMEM), warp 10 issuer of the gradients' products,
// warp 11 statistics of the walked queries (dk, dv). Every wait is bounded in time and watches a
// block abort flag (S3R_DEV_TIMEOUT on expiry).
#include <climits>
#include <cmath>

#include "internal.h"
#include "view_common.cuh"

namespace s3r {
namespace {

using namespace view;

constexpr int kThreads = 384;  // 3 warps at most per sub-partition: 168 registers a thread
constexpr int kSoftmax = 256;  // threads of the softmax warps
constexpr int kTile = 128;
constexpr uint32_t kTileBytes = kTile * 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kIdescQK = idesc_bf16_f32(kTile, kTile, 0, 0);  // both operands K-major
constexpr uint32_t kIdescMN = idesc_bf16_f32(kTile, 64, 0, 1);     // A in TMEM, B MN-major

struct BwdArgs {
  const int32_t *qo, *ko;
  const float* lse;   // [H, Lq]
  float* dsum;        // [H, Lq]: D
  uint16_t *dq, *dk, *dv;
  Stride2 dqs, dks, dvs;
  // splits > 1: [splits][part_rows, heads, 64] f32 (dq; dk and dv), for the rows of nseg segments of
  // the greatest length (row r of segment s: s * max + r)
  float *part0, *part1;
  int64_t Lq, Lk, part_rows;
  int H, Hkv, group, nseg, max_q, max_k, tiles, splits;
  // items: (segment, row tile, piece, head), heads fastest; then rest_items * heads for the rows of no segment
  uint32_t work_items;
  int rest_items;
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
// The exponentials are issued in a row and used afterwards (volatile: in this order).
__device__ __forceinline__ uint32_t exp2_now(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return __float_as_uint(y);
}

// s <- 2^(s mul + off), off the row's own or (dk, dv) each column's
__device__ __forceinline__ void exp_pair(uint32_t (&s)[32], int j, float2 mul, float2 off) {
  const float2 x = __ffma2_rn(pair_of(s[2 * j], s[2 * j + 1]), mul, off);
  s[2 * j] = exp2_now(x.x);
  s[2 * j + 1] = exp2_now(x.y);
}
template <int kFrom>  // eight pairs
__device__ __forceinline__ void exp_pairs(uint32_t (&s)[32], float2 mul, float2 off) {
#pragma unroll
  for (int j = 0; j < 8; ++j) exp_pair(s, kFrom + j, mul, off);
}
// values 2j, 2j + 1 of a vector in shared memory
__device__ __forceinline__ float2 pair_at(const float4* x, int j) {
  const float4 v = x[j / 2];
  return j & 1 ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
}
__device__ __forceinline__ uint32_t pack_pair(const uint32_t (&s)[32], int j) {
  return pack_bf16(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
}
// dS = P (dP - D) of columns 2j, 2j + 1, as bf16
__device__ __forceinline__ uint32_t grad_pair(const uint32_t (&p)[32], const uint32_t (&dp)[32], int j,
                                              float2 nd) {
  const float2 x = __fmul2_rn(pair_of(p[2 * j], p[2 * j + 1]),
                              __fadd2_rn(pair_of(dp[2 * j], dp[2 * j + 1]), nd));
  return pack_bf16(x.x, x.y);
}

// sum of P dP over the columns below `left`
__device__ __forceinline__ float row_dot(const uint32_t (&p)[32], const uint32_t (&dp)[32], int left) {
  float x[4] = {};
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < left) x[j & 3] = fmaf(__uint_as_float(p[j]), __uint_as_float(dp[j]), x[j & 3]);
  return (x[0] + x[1]) + (x[2] + x[3]);
}
// columns from `left` on to zero
__device__ __forceinline__ void keep_columns(uint32_t (&p)[16], int left) {
#pragma unroll
  for (int j = 0; j < 16; ++j) p[j] = 2 * j + 1 < left ? p[j] : 2 * j < left ? (p[j] & 0xffffu) : 0u;
}

// 32 fp32 sums a lane, times f, to 64 bytes of bf16 or 128 bytes of fp32 a row: rows 0 .. rows - 1 of
// the warp's 32 to dst + row * stride elements, through 4 KB of shared memory. Whole warp.
__device__ __forceinline__ void store_bf16(uint8_t* stage, int lane, uint16_t* dst, int64_t stride,
                                           int rows, const uint32_t (&r)[32], float f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16(__uint_as_float(r[8 * j + 2 * e]) * f, __uint_as_float(r[8 * j + 2 * e + 1]) * f);
    put_piece<4>(stage, lane, j, make_uint4(w[0], w[1], w[2], w[3]));
  }
  warp_rows<4>(stage, lane, dst, stride * 2, rows);
}
__device__ __forceinline__ void store_f32(uint8_t* stage, int lane, float* dst, int64_t stride, int rows,
                                          const uint32_t (&r)[32], float f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(r[4 * j + e]) * f);
    put_piece<8>(stage, lane, j, make_uint4(w[0], w[1], w[2], w[3]));
  }
  warp_rows<8>(stage, lane, dst, stride * 4, rows);
}
// What the producer tells the other warps of an item.
struct Item {
  int kind;       // kEnd, kZero (nothing to walk: write zeros), kRest (rows of no segment: zeros),
                  // kBad (a segment that cannot be used: NaN), kWork
  int row, rows;  // first row (of q, or of k) and how many (kRest: part_row from 0, others from `row`)
  int n, tail;    // steps of the walk (kRest: the item's number of the head's); dq: keys of the last one
  int h, split;   // head (of q, or of k), piece
  int part_row;   // splits > 1: the first row's place in the partial sums
  int q0, nq, t0; // dk, dv: the segment's queries, the piece's first step
  int whole;      // dq: the item walks all keys of the segment, at most kExactTiles tiles
  int sums;       // dq: steps before the n others that go over the same tiles to form D
};
enum { kEnd, kZero, kRest, kBad, kWork };

// An item without work: zeros, or NaN (kBad), in its rows of one head, 8 threads a row. kRest: part_row
// rows from 0 and the others from `row`, 32 of every 32 * rest_items.
__device__ __forceinline__ void fill_grad(const BwdArgs& a, const volatile Item* m, uint16_t* p,
                                          const Stride2& s) {
  const bool rest = m->kind == kRest;
  const uint32_t w = m->kind == kBad ? 0x7fc07fc0u : 0u;
  const int64_t row = m->row, rows = m->rows, before = rest ? m->part_row : 0;
  const int64_t first = (rest ? static_cast<int64_t>(m->n) * kSoftmax : 0) + threadIdx.x;
  for (int64_t i = first; i < rows * 8; i += (rest ? static_cast<int64_t>(a.rest_items) : 1) * kSoftmax) {
    const int64_t r = (i >> 3) < before ? i >> 3 : row + (i >> 3) - before;
    reinterpret_cast<uint4*>(p + r * s.tok + m->h * s.head)[i & 7] = make_uint4(w, w, w, w);
  }
}
__device__ __forceinline__ void zero_part(float* p, int heads, int head, int64_t r0, int rows) {
  for (int i = threadIdx.x; i < rows * 16; i += kSoftmax)
    reinterpret_cast<float4*>(p + ((r0 + (i >> 4)) * heads + head) * 64)[i & 15] =
        make_float4(0.f, 0.f, 0.f, 0.f);
}

// D = <dout, out> of every (row, head): 8 lanes a row, and [H, Lq] written in runs of 32 rows (a
// block has 32 rows of one head). Bound by reading both.
__global__ void __launch_bounds__(256) view_d_kernel(const uint16_t* out, const uint16_t* dout,
                                                     float* dsum, int64_t Lq, int H) {
  const int h = blockIdx.x % H;
  const int64_t row = static_cast<int64_t>(blockIdx.x / H) * 32 + (threadIdx.x >> 3);
  float d = 0.f;
  if (row < Lq) {
    const int64_t at = (row * H + h) * 64 + (threadIdx.x & 7) * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(out + at);
    const uint4 y = *reinterpret_cast<const uint4*>(dout + at);
    d = bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x);
    d += bf16_lo(x.y) * bf16_lo(y.y) + bf16_hi(x.y) * bf16_hi(y.y);
    d += bf16_lo(x.z) * bf16_lo(y.z) + bf16_hi(x.z) * bf16_hi(y.z);
    d += bf16_lo(x.w) * bf16_lo(y.w) + bf16_hi(x.w) * bf16_hi(y.w);
  }
  d += __shfl_xor_sync(0xffffffffu, d, 1);
  d += __shfl_xor_sync(0xffffffffu, d, 2);
  d += __shfl_xor_sync(0xffffffffu, d, 4);
  if (row < Lq && (threadIdx.x & 7) == 0) dsum[h * Lq + row] = d;
}

// Both kernels' shared memory: two items' own tiles, a ring of walked tiles with their queries'
// statistics, and the barriers.
constexpr int kStages = 4;
// Up to so many tiles of keys, D is formed from P and dP: one tile from the registers, two in a walk ahead
// (1.35 us a tile of an item). Both sides, for 8 segments of 640 queries of 16 heads: all gradients' time,
// and dq's error relative to its norm (rounding the exact dq alone: 0.0017) where the logits' deviation is
// 1.5, and where it is 8 and a row's softmax lies on few keys:
//   128 keys          formed 44 us, 0.0024, 0.0024
//   129 to 256 keys   formed 68 us, 0.0024, 0.0024;         from out 55 us, 0.0026 to 0.0025, 0.0064
//   257 to 512 keys   formed 86 to 103 us, 0.0024, 0.0024;  from out 68 to 80 us, 0.0025, 0.0064
// Two tiles are where a fifth of the time still takes off a twentieth of an ordinary row's error and more;
// at four it is three tenths for less. Rows on few keys would gain at any length.
constexpr int kExactTiles = 2;
constexpr uint32_t kStageBytes = 2 * kTileBytes;          // dq: K | V; dk, dv: q | dout
constexpr uint32_t kOffOwn = 0;                           // [2 items]: q | dout; or K | V
constexpr uint32_t kOffRing = 2 * kStageBytes;
// [2][128] f32 each, -lse log2 e and -D of 128 queries: dq has one per item, dk and dv one per stage
constexpr uint32_t kOffStat = kOffRing + kStages * kStageBytes;
// dq: [2 items][2 column halves][128] f32, sums of P dP (the half of the space it has no stages for)
constexpr uint32_t kOffPair = kOffStat + 2048;
constexpr uint32_t kOffNext = kOffStat + kStages * 1024;  // 16 bytes: the answer to a request
constexpr uint32_t kOffItem = kOffNext + 16;
constexpr uint32_t kOffBars = kOffItem + 2 * sizeof(Item);
struct __align__(8) Bars {
  uint64_t own_full[2], own_empty[2];      // an item's own tiles and its description
  uint64_t full[kStages], empty[kStages];  // a stage's tiles
  uint64_t tail;                           // TMA of tiles that are cut by the segment's end
  uint64_t s_full, s_empty;                // S and dP written / read into registers
  uint64_t p_full, p_empty;                // dS (and P) written / their products completed
  uint64_t o_full;                         // every product of the item completed
  uint64_t pair[4];  // dq: both column halves' sums of a lane quadrant written
  uint64_t next;  // the answer to a request for an item
  uint64_t drain[2];
  uint64_t never;  // never signalled: waited on only under S3R_FLAG_TEST_TIMEOUT
};
constexpr uint32_t kOffMisc = kOffBars + sizeof(Bars);
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 227 * 1024 && kOffBars % 8 == 0, "shared memory of a block");
constexpr uint32_t kTmemCols = 512;

struct Block {
  uint8_t* smem;
  uint32_t sbase;
  Bars* bars;
  Item* items;
  volatile int* abort;
};

template <bool kDKV>
__device__ __forceinline__ Block block_start(uint8_t* smem_raw) {
  const uint32_t raw_s = smem_addr(smem_raw);
  Block k;
  k.smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
  k.sbase = smem_addr(k.smem);
  k.bars = reinterpret_cast<Bars*>(k.smem + kOffBars);
  k.items = reinterpret_cast<Item*>(k.smem + kOffItem);
  k.abort = reinterpret_cast<volatile int*>(k.smem + kOffMisc + 4);
  Bars* bars = k.bars;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->own_full[i], 1);
      mbar_init(&bars->own_empty[i], kDKV ? 11 : 10);  // issuers, softmax warps, statistics warp
      mbar_init(&bars->drain[i], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], kDKV ? 2 : 1);  // the tiles, and the statistics
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->tail, 1);
    mbar_init(&bars->next, 1);
    mbar_init(&bars->s_full, kDKV ? 2 : 1);
    mbar_init(&bars->s_empty, 8);
    mbar_init(&bars->p_full, 8);
    mbar_init(&bars->p_empty, 1);
    mbar_init(&bars->o_full, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bars->pair[i], 2);
    mbar_init(&bars->never, 1);
    *k.abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x >> 5 == 9)
    tmem_alloc(reinterpret_cast<uint32_t*>(k.smem + kOffMisc), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return k;
}

// The TMEM of a block starts at column 0: all 512 are its own.
__device__ __forceinline__ void block_end() {
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x >> 5 == 9) tmem_dealloc(0, kTmemCols);
}

// Lets the producer's copies in flight land before the block ends: `items` and `stages` issued so
// far; `cut`: the last stage's went to the tail barrier and is not handed on.
__device__ __forceinline__ void drain_copies(const Block& k, int items, int stages, bool cut, int cuts,
                                             uint64_t lim) {
  int dummy = 0;
  for (int i = items - 1; i >= 0 && i >= items - 2; --i)
    wait_bar(&k.bars->own_full[i & 1], (i >> 1) & 1, &dummy, lim);
  if (cut) wait_bar(&k.bars->tail, cuts & 1, &dummy, lim);
  for (int t = stages - 1 - (cut ? 1 : 0); t >= 0 && t >= stages - kStages; --t)
    wait_bar(&k.bars->full[t % kStages], (t / kStages) & 1, &dummy, lim);
}

// The issuer of S and dP (warp 9) of both kernels: per step, two products of the item's own tiles
// with the stage's. S is written as soon as the last one is in registers, while this tile's
// exponentials run; dP once the last one is, and both are then handed on together. dk, dv: the
// issuer's own arrival hands on the stage's statistics too, which it has waited for.
template <bool kDKV>
__device__ __forceinline__ void issue_scores(const Block& k, const BwdArgs& a) {
  const uint32_t el = elect_one();
  Bars* bars = k.bars;
  const uint64_t lim = a.limit_ns;
  bool ok = true;
  int c = 0;  // steps so far
  for (int i = 0; ok; ++i) {
    const int slot = i & 1;
    if (!(ok = wait_bar_warp(&bars->own_full[slot], (i >> 1) & 1, k.abort, lim))) break;
    const volatile Item* item = k.items + slot;
    const int kind = item->kind, n = item->n + item->sums;
    if (kind == kEnd) break;
    if (kind == kWork) {
      const uint32_t own = k.sbase + kOffOwn + slot * kStageBytes;
      const uint64_t d0 = desc_sw128(own), d1 = desc_sw128(own + kTileBytes);
      for (int t = 0; t < n; ++t, ++c) {
        const int st = c % kStages;
        const uint32_t sk = k.sbase + kOffRing + st * kStageBytes;
        const uint64_t e0 = desc_sw128(sk), e1 = desc_sw128(sk + kTileBytes);
        if (!(ok = wait_bar_warp(&bars->full[st], (c / kStages) & 1, k.abort, lim))) break;
        if (!(ok = wait_bar_warp(&bars->s_empty, (c & 1) ^ 1, k.abort, lim))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_ss_if(el, 0, d0 + 2 * ks, e0 + 2 * ks, kIdescQK, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_ss_if(el, 128, d1 + 2 * ks, e1 + 2 * ks, kIdescQK, ks > 0);
        tc_commit_if(el, &bars->s_full);
        if (kDKV) mbar_arrive_if(el, &bars->s_full);
      }
      if (!ok) break;
      tc_commit_if(el, &bars->own_empty[slot]);
    } else {
      mbar_arrive_if(el, &bars->own_empty[slot]);
    }
  }
  if (!ok) {
    if (el) raise_abort(k.abort, a.status);
    int dummy = 0;
    tc_commit_if(el, &bars->drain[0]);
    wait_bar(&bars->drain[0], 0, &dummy, lim);
  }
}

// The issuer of the gradients' products (warp 10). dq: A = dS at column 320, B = K, into 256. dk, dv:
// A = P at 384, B = dout, into 256 and A = dS at 448, B = q, into 320.
template <bool kDKV>
__device__ __forceinline__ void issue_grads(const Block& k, const BwdArgs& a) {
  const uint32_t el = elect_one();
  Bars* bars = k.bars;
  const uint64_t lim = a.limit_ns;
  bool ok = true;
  int c = 0;
  for (int i = 0; ok; ++i) {
    const int slot = i & 1;
    if (!(ok = wait_bar_warp(&bars->own_full[slot], (i >> 1) & 1, k.abort, lim))) break;
    const volatile Item* item = k.items + slot;
    const int kind = item->kind, n = item->n, sums = kDKV ? 0 : item->sums;
    if (kind == kEnd) break;
    if (kind == kWork) {
      for (int t = -sums; t < n; ++t, ++c) {
        const int st = c % kStages;
        const uint32_t sk = k.sbase + kOffRing + st * kStageBytes;
        const uint64_t e0 = desc_sw128(sk), e1 = desc_sw128(sk + kTileBytes);
        if (!(ok = wait_bar_warp(&bars->p_full, c & 1, k.abort, lim))) break;
        if (!kDKV && t < 0) {  // nothing to multiply: the stage is handed back
          mbar_arrive_if(el, &bars->p_empty);
          mbar_arrive_if(el, &bars->empty[st]);
          continue;
        }
        tc_fence_after();
        // 16 rows of the stage a step: 16 x 128 B = 2048 B
        if (kDKV) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts_if(el, 256, 384 + ks * 8, e1 + 128 * ks, kIdescMN, (t > 0 || ks > 0) ? 1u : 0u);
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts_if(el, kDKV ? 320 : 256, (kDKV ? 448 : 320) + ks * 8, e0 + 128 * ks, kIdescMN,
                    (t > 0 || ks > 0) ? 1u : 0u);
        tc_commit_if(el, &bars->p_empty);
        tc_commit_if(el, &bars->empty[st]);
      }
      if (!ok) break;
      tc_commit_if(el, &bars->o_full);
    }
    mbar_arrive_if(el, &bars->own_empty[slot]);
  }
  if (!ok) {
    if (el) raise_abort(k.abort, a.status);
    int dummy = 0;
    tc_commit_if(el, &bars->drain[1]);
    wait_bar(&bars->drain[1], 0, &dummy, lim);
  }
}

// ------------------------------------------------------------------------------------------
// dq
// ------------------------------------------------------------------------------------------
// The walk ahead of the dq kernel's softmax warps: the sum of P dP over a thread's half of the columns.
// Not inlined: the registers it took cost the walk that follows 4 % (8 views: 134 against 129 us).
__device__ __noinline__ bool sum_walk(const Block& k, const BwdArgs& a, int n, int tail, bool idle, int half,
                                      uint32_t tl, float nl, uint32_t el, int* step, float* sum) {
  Bars* bars = k.bars;
  const float2 mul = make_float2(a.scale_log2, a.scale_log2), off = make_float2(nl, nl);
  int c = *step;
  float x = 0.f;
  for (int t = 0; t < n; ++t, ++c) {
    if (!wait_bar(&bars->s_full, c & 1, k.abort, a.limit_ns)) return false;
    tc_fence_after();
    if (!idle) {
      const int left = t == n - 1 ? tail - 64 * half : 64;
#pragma unroll 1
      for (int z = 0; z < 2; ++z) {
        uint32_t s[32], dp[32];
        tmem_ld32(tl + 64 * half + 32 * z, s);
        tmem_ld32(tl + 128 + 64 * half + 32 * z, dp);
        tmem_wait_ld_regs(s);
        tmem_wait_ld_regs(dp);
        exp_pairs<0>(s, mul, off);
        exp_pairs<8>(s, mul, off);
        x += row_dot(s, dp, left - 32 * z);
      }
    }
    tc_fence_before();
    __syncwarp();
    mbar_arrive_if(el, &bars->s_empty);
    // (as in the walk that follows, so that no warp is a phase ahead of another or of the issuer)
    if (!wait_bar(&bars->p_empty, (c & 1) ^ 1, k.abort, a.limit_ns)) return false;
    __syncwarp();
    mbar_arrive_if(el, &bars->p_full);
  }
  *step = c;
  *sum = x;
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    view_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const BwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const Block k = block_start<false>(smem_raw);
  Bars* bars = k.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.limit_ns;

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    bool ok = true, cut = false;
    int ni = 0, c = 0, cuts = 0;  // items, stages and cut stages so far
    uint32_t it = blockIdx.x;
    bool more = true;  // `it` is an item
    int asked = 0;     // requests so far
    uint32_t skipped = 0;  // items without rows so far
    for (bool first = true; ok; first = false) {
      if (!first) {  // the item asked for while the last one was issued
        if (!(ok = wait_bar_warp(&bars->next, (asked - 1) & 1, k.abort, lim))) break;
        more = taken_item(k.smem + kOffNext, &it);
      }
      if (more) request_item(lane == 0, k.smem + kOffNext, &bars->next), ++asked;
      Item m{};
      int key0 = 0;
      if (more) {
        uint32_t b = it;
        m.h = b % a.H;
        b /= a.H;
        if (it >= a.work_items) {
          const Rows x = rows_outside(a.qo, a.nseg, a.Lq);
          m.kind = kRest;
          m.row = x.after;
          m.part_row = x.before;
          m.rows = x.before + static_cast<int>(a.Lq) - x.after;
          m.n = (it - a.work_items) / a.H;
        } else {
          m.split = b % a.splits;
          b /= a.splits;
          const int tile = b % a.tiles, seg = b / a.tiles;
          const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
          if (!g.ok) {
            if (lane == 0) set_status(a.status, S3R_DEV_BAD_INDEX);
            const Rows x = rows_clipped(a.qo, seg, a.Lq);
            if ((a.flags & S3R_FLAG_ALL_ROWS) && tile + m.split == 0 && x.before < x.after) {
              m.kind = kBad;
              m.row = x.before;
              m.rows = x.after - x.before;
            }
          } else if (tile * kTile < g.nq) {
            const int row0 = tile * kTile;
            m.row = g.q0 + row0;
            m.part_row = a.splits > 1 ? seg * a.max_q + row0 : 0;
            m.rows = g.nq - row0 < kTile ? g.nq - row0 : kTile;
            // (one piece takes all the tiles of a segment whose D is formed here)
            const int all = (g.nk + kTile - 1) / kTile, share = (all + a.splits - 1) / a.splits;
            const int per = share > kExactTiles ? share : kExactTiles;
            const int t0 = m.split * per;
            m.n = all - t0 < per ? all - t0 : per;
            m.kind = m.n > 0 ? kWork : kZero;
            // (a piece that ends before the segment does has a whole last tile)
            const int left = g.nk - (t0 + m.n - 1) * kTile;
            m.tail = left < kTile ? left : kTile;
            m.whole = all == m.n && all <= kExactTiles;
            m.sums = m.whole && all > 1 ? all : 0;
            key0 = g.k0 + t0 * kTile;
          }
          if (m.kind == kEnd) {  // no rows
            if (++skipped % kSkips) continue;
            m.kind = kZero;
          }
        }
      }
      const int slot = ni & 1;
      // the item's statistics, lane by lane; rows past the end get zeros
      float nl[4], nd[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = x * 32 + lane;
        const bool in = m.kind == kWork && r < m.rows;
        const int64_t at = m.h * a.Lq + m.row + r;
        nl[x] = in ? -a.lse[at] * kLog2e : 0.f;
        nd[x] = in ? -a.dsum[at] : 0.f;
      }
      if (!(ok = wait_bar_warp(&bars->own_empty[slot], ((ni >> 1) & 1) ^ 1, k.abort, lim))) break;
      float* stat = reinterpret_cast<float*>(k.smem + kOffStat + slot * 1024);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        stat[x * 32 + lane] = nl[x];
        stat[kTile + x * 32 + lane] = nd[x];
      }
      if (lane == 0) k.items[slot] = m;
      __syncwarp();
      if (lane == 0) {
        if (m.kind == kWork) {
          const uint32_t own = k.sbase + kOffOwn + slot * kStageBytes;
          mbar_arrive_expect_tx(&bars->own_full[slot], kStageBytes);
          tma_load_rows(own, &tmQ, m.h, m.row, &bars->own_full[slot]);
          tma_load_rows(own + kTileBytes, &tmO, m.h, m.row, &bars->own_full[slot]);
        } else {
          mbar_arrive(&bars->own_full[slot]);
        }
      }
      ++ni;
      if (m.kind == kEnd) break;
      if (m.kind != kWork) continue;
      const int hk = m.h / a.group;
      for (int x = 0; x < m.sums + m.n; ++x) {
        const int t = x < m.sums ? x : x - m.sums;
        const int st = c % kStages;
        const uint32_t sk = k.sbase + kOffRing + st * kStageBytes;
        if (!(ok = wait_bar_warp(&bars->empty[st], ((c / kStages) & 1) ^ 1, k.abort, lim))) break;
        cut = t == m.n - 1 && m.tail < kTile;
        if (lane == 0) {
          uint64_t* full = cut ? &bars->tail : &bars->full[st];
          mbar_arrive_expect_tx(full, kStageBytes);
          tma_load_rows(sk, &tmK, hk, key0 + t * kTile, full);
          tma_load_rows(sk + kTileBytes, &tmV, hk, key0 + t * kTile, full);
        }
        ++c;
        if (cut) {  // the key tile reaches past the segment
          if (!(ok = wait_bar_warp(&bars->tail, cuts & 1, k.abort, lim))) break;
          ++cuts;
          cut = false;
          zero_rows(k.smem + kOffRing + st * kStageBytes, m.tail, lane);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->full[st]);
        }
      }
    }
    if (!ok && lane == 0) {
      raise_abort(k.abort, a.status);
      int dummy = 0;
      if (asked > 0) wait_bar(&bars->next, (asked - 1) & 1, &dummy, lim);
      drain_copies(k, ni, c, cut, cuts, lim);
    }
  } else if (warp == 9) {
    issue_scores<false>(k, a);
  } else if (warp == 10) {
    issue_grads<false>(k, a);
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax warps
    const uint32_t el = elect_one();
    const int qd = warp & 3, half = warp >> 2, r = qd * 32 + lane;
    const uint32_t tl = static_cast<uint32_t>(qd * 32) << 16;
    const float2 mul = make_float2(a.scale_log2, a.scale_log2);
    bool ok = true;
    int c = 0, done = 0, wholes = 0;
    if (a.flags & S3R_FLAG_TEST_TIMEOUT) ok = wait_bar(&bars->never, 0, k.abort, lim);
    for (int i = 0; ok; ++i) {
      const int slot = i & 1;
      if (!(ok = wait_bar(&bars->own_full[slot], (i >> 1) & 1, k.abort, lim))) break;
      const volatile Item* item = k.items + slot;
      const int kind = item->kind, n = item->n, tail = item->tail, rows = item->rows;
      if (kind == kEnd) break;
      float* sums = a.splits > 1 ? a.part0 + item->split * a.part_rows * a.H * 64 : nullptr;
      if (kind == kWork) {
        const bool idle = qd * 32 >= rows;  // no rows: only keeps the barriers going
        const volatile float* stat = reinterpret_cast<const volatile float*>(k.smem + kOffStat + slot * 1024);
        const float nl = stat[r], d = stat[kTile + r];
        const float2 off = make_float2(nl, nl);
        float2 nd = make_float2(d, d);
        // Few keys make out large beside dS, and its rounding to bf16 shows in D. So up to kExactTiles
        // tiles D is the sum of P dP, formed in a walk ahead (one tile: below, from the registers), and
        // left for dk and dv.
        const int sums_steps = item->sums;
        float x = 0.f;
        if (sums_steps > 0 && !(ok = sum_walk(k, a, sums_steps, tail, idle, half, tl, nl, el, &c, &x))) break;
        // the row's two halves
        const auto exact = [&](float mine) -> bool {
          float* pair = reinterpret_cast<float*>(k.smem + kOffPair) + (wholes & 1) * 256 + r;
          pair[half * 128] = mine;
          __syncwarp();
          mbar_arrive_if(el, &bars->pair[qd]);
          if (!wait_bar(&bars->pair[qd], wholes & 1, k.abort, lim)) return false;
          ++wholes;
          const float sum = pair[0] + pair[128];
          if (half == 0 && r < rows) a.dsum[item->h * a.Lq + item->row + r] = sum;
          nd = make_float2(-sum, -sum);
          return true;
        };
        if (sums_steps > 0 && !idle && !(ok = exact(x))) break;
        bool ready = false;  // a test of the next wait's barrier, made ahead: one takes about 100 clocks
        for (int t = 0; t < n; ++t, ++c) {
          if (!ready && !(ok = wait_bar(&bars->s_full, c & 1, k.abort, lim))) break;
          tc_fence_after();
          if (idle) {
            ready = false;
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(el, &bars->s_empty);
            if (!(ok = wait_bar(&bars->p_empty, (c & 1) ^ 1, k.abort, lim))) break;
            __syncwarp();
            mbar_arrive_if(el, &bars->p_full);
            continue;
          }
          uint32_t s0[32], s1[32], d0[32], d1[32], p[16];
          tmem_ld32(tl + 64 * half, s0);
          tmem_wait_ld_regs(s0);
          tmem_ld32(tl + 64 * half + 32, s1);
          tmem_ld32(tl + 128 + 64 * half, d0);
          tmem_ld32(tl + 128 + 64 * half + 32, d1);
          exp_pairs<0>(s0, mul, off);
          ready = mbar_peek(&bars->p_empty, (c & 1) ^ 1);
          tmem_wait_ld_regs(s1);
          tmem_wait_ld_regs(d0);
          tmem_wait_ld_regs(d1);
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(el, &bars->s_empty);
          const int left = t == n - 1 ? tail - 64 * half : 64;  // columns of this half that count
          const bool whole = item->whole && sums_steps == 0;  // one tile
          if (whole) {
            exp_pairs<8>(s0, mul, off);
            exp_pairs<0>(s1, mul, off);
            exp_pairs<8>(s1, mul, off);
            if (!(ok = exact(row_dot(s0, d0, left) + row_dot(s1, d1, left - 32)))) break;
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = grad_pair(s0, d0, j, nd);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              exp_pair(s0, 8 + j, mul, off);
              p[j] = grad_pair(s0, d0, j, nd);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              exp_pair(s1, j, mul, off);
              p[8 + j] = grad_pair(s0, d0, 8 + j, nd);
            }
          }
          if (!ready && !(ok = wait_bar(&bars->p_empty, (c & 1) ^ 1, k.abort, lim))) break;
          tc_fence_after();
          if (left < 32) keep_columns(p, left);
          tmem_st32x16(tl + 320 + 32 * half, p);
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              exp_pair(s1, 8 + j, mul, off);
              p[j] = grad_pair(s1, d1, j, nd);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = grad_pair(s1, d1, j, nd);
          }
#pragma unroll
          for (int j = 8; j < 16; ++j) p[j] = grad_pair(s1, d1, j, nd);
          if (left < 64) keep_columns(p, left - 32);
          tmem_st32x16(tl + 320 + 32 * half + 16, p);
          ready = mbar_peek(&bars->s_full, (c & 1) ^ 1);
          tmem_wait_st_keep16(p);
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(el, &bars->p_full);
        }
        if (!ok || !(ok = wait_bar(&bars->o_full, done & 1, k.abort, lim))) break;
        ++done;
        if (!idle) {
          tc_fence_after();
          uint32_t o[32];
          tmem_ld32(tl + 256 + 32 * half, o);
          tmem_wait_ld_regs(o);
          // through the item's own tiles, which no product reads any more
          uint8_t* stage = k.smem + kOffOwn + slot * kStageBytes + warp * 4096;
          const int r0 = qd * 32, h = item->h;
          if (sums)
            store_f32(stage, lane, sums + (static_cast<int64_t>(item->part_row + r0) * a.H + h) * 64 + 32 * half,
                      static_cast<int64_t>(a.H) * 64, rows - r0, o, a.scale);
          else
            store_bf16(stage, lane, a.dq + (item->row + r0) * a.dqs.tok + h * a.dqs.head + 32 * half,
                       a.dqs.tok, rows - r0, o, a.scale);
          fence_proxy_async();  // these reads and writes before the next item's tiles land there
        }
      } else if (kind == kZero && sums) {
        zero_part(sums, a.H, item->h, item->part_row, rows);
      } else {
        fill_grad(a, item, a.dq, a.dqs);
      }
      __syncwarp();
      mbar_arrive_if(el, &bars->own_empty[slot]);
    }
    if (!ok) raise_abort(k.abort, a.status);
  }
  block_end();
}

// ------------------------------------------------------------------------------------------
// dk, dv
// ------------------------------------------------------------------------------------------
// The statistics warp (11): -lse log2 e and -D of every step's 128 queries, four a lane, or (past
// the segment's end) -inf and 0, which make P and dS zero. They are read from L2 two steps ahead of
// their place in the ring, by a warp of their own: in the producer they held up its copies.
__device__ __forceinline__ void load_stats(const Block& k, const BwdArgs& a, int lane) {
  Bars* bars = k.bars;
  bool ok = true;
  int c = 0;
  for (int i = 0; ok; ++i) {
    const int slot = i & 1;
    if (!(ok = wait_bar_warp(&bars->own_full[slot], (i >> 1) & 1, k.abort, a.limit_ns))) break;
    const volatile Item* item = k.items + slot;
    const int kind = item->kind, n = item->n;
    if (kind == kEnd) break;
    if (kind == kWork) {
      const int nq = item->nq, t0 = item->t0, qt = (nq + kTile - 1) / kTile;
      const int64_t q0 = item->q0;
      int hh = item->h * a.group + t0 / qt, y = t0 % qt * kTile;
      float l0[4], d0[4], l1[4], d1[4], l2[4], d2[4];  // of steps t, t + 1, t + 2
      auto fetch = [&](float (&l)[4], float (&d)[4]) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = y + x * 32 + lane;
          const bool in = r < nq && hh < a.H;
          const int64_t at = hh * a.Lq + q0 + r;
          l[x] = in ? a.lse[at] : INFINITY;
          d[x] = in ? a.dsum[at] : 0.f;
        }
        y += kTile;
        if (y >= nq) y = 0, ++hh;
      };
      fetch(l0, d0);
      fetch(l1, d1);
      for (int t = 0; t < n; ++t, ++c) {
        const int st = c % kStages;
        fetch(l2, d2);
        if (!(ok = wait_bar_warp(&bars->empty[st], ((c / kStages) & 1) ^ 1, k.abort, a.limit_ns))) break;
        float* stat = reinterpret_cast<float*>(k.smem + kOffStat + st * 1024);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          stat[x * 32 + lane] = -l0[x] * kLog2e;
          stat[kTile + x * 32 + lane] = -d0[x];
          l0[x] = l1[x], d0[x] = d1[x];
          l1[x] = l2[x], d1[x] = d2[x];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->full[st]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->own_empty[slot]);
  }
  if (!ok && lane == 0) raise_abort(k.abort, a.status);
}

__global__ void __launch_bounds__(kThreads, 1)
    view_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const BwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const Block k = block_start<true>(smem_raw);
  Bars* bars = k.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.limit_ns;

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    bool ok = true, cut = false;
    int ni = 0, c = 0, cuts = 0;
    uint32_t it = blockIdx.x;
    bool more = true;  // `it` is an item
    int asked = 0;     // requests so far
    uint32_t skipped = 0;  // items without rows so far
    for (bool first = true; ok; first = false) {
      if (!first) {  // the item asked for while the last one was issued
        if (!(ok = wait_bar_warp(&bars->next, (asked - 1) & 1, k.abort, lim))) break;
        more = taken_item(k.smem + kOffNext, &it);
      }
      if (more) request_item(lane == 0, k.smem + kOffNext, &bars->next), ++asked;
      Item m{};
      int qt = 1;
      if (more) {
        uint32_t b = it;
        m.h = b % a.Hkv;
        b /= a.Hkv;
        if (it >= a.work_items) {
          const Rows x = rows_outside(a.ko, a.nseg, a.Lk);
          m.kind = kRest;
          m.row = x.after;
          m.part_row = x.before;
          m.rows = x.before + static_cast<int>(a.Lk) - x.after;
          m.n = (it - a.work_items) / a.Hkv;
        } else {
          m.split = b % a.splits;
          b /= a.splits;
          const int tile = b % a.tiles, seg = b / a.tiles;
          const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
          if (!g.ok) {
            if (lane == 0) set_status(a.status, S3R_DEV_BAD_INDEX);
            const Rows x = rows_clipped(a.ko, seg, a.Lk);
            if ((a.flags & S3R_FLAG_ALL_ROWS) && tile + m.split == 0 && x.before < x.after) {
              m.kind = kBad;
              m.row = x.before;
              m.rows = x.after - x.before;
            }
          } else if (tile * kTile < g.nk) {
            const int row0 = tile * kTile;
            m.row = g.k0 + row0;
            m.part_row = a.splits > 1 ? seg * a.max_k + row0 : 0;
            m.rows = g.nk - row0 < kTile ? g.nk - row0 : kTile;
            // steps: (head of the group, query tile), the tile fastest
            m.q0 = g.q0;
            m.nq = g.nq;
            qt = (g.nq + kTile - 1) / kTile;
            const int all = qt * a.group, per = (all + a.splits - 1) / a.splits;
            m.t0 = m.split * per;
            m.n = all - m.t0 < per ? all - m.t0 : per;
            m.kind = m.n > 0 ? kWork : kZero;
          }
          if (m.kind == kEnd) {  // no rows
            if (++skipped % kSkips) continue;
            m.kind = kZero;
          }
        }
      }
      const int slot = ni & 1;
      if (!(ok = wait_bar_warp(&bars->own_empty[slot], ((ni >> 1) & 1) ^ 1, k.abort, lim))) break;
      if (lane == 0) {
        k.items[slot] = m;
        if (m.kind == kWork) {
          const uint32_t own = k.sbase + kOffOwn + slot * kStageBytes;
          mbar_arrive_expect_tx(&bars->own_full[slot], kStageBytes);
          tma_load_rows(own, &tmK, m.h, m.row, &bars->own_full[slot]);
          tma_load_rows(own + kTileBytes, &tmV, m.h, m.row, &bars->own_full[slot]);
        } else {
          mbar_arrive(&bars->own_full[slot]);
        }
      }
      ++ni;
      if (m.kind == kEnd) break;
      if (m.kind != kWork) continue;
      int hh = m.h * a.group + m.t0 / qt, y = m.t0 % qt * kTile;  // head and query tile of the step
      for (int t = 0; t < m.n; ++t) {
        const int st = c % kStages, left = m.nq - y;
        const uint32_t sq = k.sbase + kOffRing + st * kStageBytes;
        if (!(ok = wait_bar_warp(&bars->empty[st], ((c / kStages) & 1) ^ 1, k.abort, lim))) break;
        cut = left < kTile;
        if (lane == 0) {
          uint64_t* full = cut ? &bars->tail : &bars->full[st];
          mbar_arrive_expect_tx(full, kStageBytes);
          tma_load_rows(sq, &tmQ, hh, m.q0 + y, full);
          tma_load_rows(sq + kTileBytes, &tmO, hh, m.q0 + y, full);
        }
        ++c;
        y += kTile;
        if (y >= m.nq) y = 0, ++hh;
        if (cut) {  // the tiles reach past the segment's queries
          if (!(ok = wait_bar_warp(&bars->tail, cuts & 1, k.abort, lim))) break;
          ++cuts;
          cut = false;
          uint8_t* qp = k.smem + kOffRing + st * kStageBytes;
          zero_rows(qp, left, lane);
          zero_rows(qp + kTileBytes, left, lane);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->full[st]);
        }
      }
    }
    if (!ok && lane == 0) {
      raise_abort(k.abort, a.status);
      int dummy = 0;
      if (asked > 0) wait_bar(&bars->next, (asked - 1) & 1, &dummy, lim);
      drain_copies(k, ni, c, cut, cuts, lim);
    }
  } else if (warp == 9) {
    issue_scores<true>(k, a);
  } else if (warp == 10) {
    issue_grads<true>(k, a);
  } else if (warp == 11) {
    load_stats(k, a, lane);
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax warps
    const uint32_t el = elect_one();
    const int qd = warp & 3, half = warp >> 2;
    const uint32_t tl = static_cast<uint32_t>(qd * 32) << 16;
    const float2 mul = make_float2(a.scale_log2, a.scale_log2);
    bool ok = true;
    int c = 0, done = 0;
    if (a.flags & S3R_FLAG_TEST_TIMEOUT) ok = wait_bar(&bars->never, 0, k.abort, lim);
    for (int i = 0; ok; ++i) {
      const int slot = i & 1;
      if (!(ok = wait_bar(&bars->own_full[slot], (i >> 1) & 1, k.abort, lim))) break;
      const volatile Item* item = k.items + slot;
      const int kind = item->kind, n = item->n, rows = item->rows;
      if (kind == kEnd) break;
      if (kind == kWork) {
        const bool idle = qd * 32 >= rows;
        bool ready = false;  // a test of the next wait's barrier, made ahead: one takes about 100 clocks
        for (int t = 0; t < n; ++t, ++c) {
          const int st = c % kStages;
          const float4* nl = reinterpret_cast<const float4*>(k.smem + kOffStat + st * 1024 + half * 256);
          const float4* nd = nl + 32;  // 128 floats on
          if (!ready && !(ok = wait_bar(&bars->s_full, c & 1, k.abort, lim))) break;
          tc_fence_after();
          if (idle) {
            ready = false;
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(el, &bars->s_empty);
            if (!(ok = wait_bar(&bars->p_empty, (c & 1) ^ 1, k.abort, lim))) break;
            __syncwarp();
            mbar_arrive_if(el, &bars->p_full);
            continue;
          }
          uint32_t s0[32], s1[32], d0[32], d1[32], p[16], g[16];
          tmem_ld32(tl + 64 * half, s0);
          tmem_wait_ld_regs(s0);
          tmem_ld32(tl + 64 * half + 32, s1);
          tmem_ld32(tl + 128 + 64 * half, d0);
          tmem_ld32(tl + 128 + 64 * half + 32, d1);
#pragma unroll
          for (int j = 0; j < 8; ++j) exp_pair(s0, j, mul, pair_at(nl, j));
          ready = mbar_peek(&bars->p_empty, (c & 1) ^ 1);
          tmem_wait_ld_regs(s1);
          tmem_wait_ld_regs(d0);
          tmem_wait_ld_regs(d1);
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(el, &bars->s_empty);
          // packing eight pairs while the next eight's exponentials run
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            exp_pair(s0, 8 + j, mul, pair_at(nl, 8 + j));
            p[j] = pack_pair(s0, j);
            g[j] = grad_pair(s0, d0, j, pair_at(nd, j));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            exp_pair(s1, j, mul, pair_at(nl, 16 + j));
            p[8 + j] = pack_pair(s0, 8 + j);
            g[8 + j] = grad_pair(s0, d0, 8 + j, pair_at(nd, 8 + j));
          }
          if (!ready && !(ok = wait_bar(&bars->p_empty, (c & 1) ^ 1, k.abort, lim))) break;
          tc_fence_after();
          tmem_st32x16(tl + 384 + 32 * half, p);
          tmem_st32x16(tl + 448 + 32 * half, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            exp_pair(s1, 8 + j, mul, pair_at(nl, 24 + j));
            p[j] = pack_pair(s1, j);
            g[j] = grad_pair(s1, d1, j, pair_at(nd, 16 + j));
          }
#pragma unroll
          for (int j = 8; j < 16; ++j) {
            p[j] = pack_pair(s1, j);
            g[j] = grad_pair(s1, d1, j, pair_at(nd, 16 + j));
          }
          tmem_st32x16(tl + 384 + 32 * half + 16, p);
          tmem_st32x16(tl + 448 + 32 * half + 16, g);
          ready = mbar_peek(&bars->s_full, (c & 1) ^ 1);
          tmem_wait_st_keep16(p);
          tmem_wait_st_keep16(g);
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(el, &bars->p_full);
        }
        if (!ok || !(ok = wait_bar(&bars->o_full, done & 1, k.abort, lim))) break;
        ++done;
        if (!idle) {
          tc_fence_after();
          uint32_t v[32], g[32];
          tmem_ld32(tl + 256 + 32 * half, v);
          tmem_ld32(tl + 320 + 32 * half, g);
          tmem_wait_ld_regs(v);
          tmem_wait_ld_regs(g);
          uint8_t* stage = k.smem + kOffOwn + slot * kStageBytes + warp * 4096;  // as for dq
          const int r0 = qd * 32, h = item->h;
          if (a.splits > 1) {
            const int64_t at =
                ((item->split * a.part_rows + item->part_row + r0) * a.Hkv + h) * 64 + 32 * half;
            store_f32(stage, lane, a.part0 + at, static_cast<int64_t>(a.Hkv) * 64, rows - r0, g, a.scale);
            store_f32(stage, lane, a.part1 + at, static_cast<int64_t>(a.Hkv) * 64, rows - r0, v, 1.f);
          } else {
            const int64_t row = item->row + r0;
            store_bf16(stage, lane, a.dk + row * a.dks.tok + h * a.dks.head + 32 * half, a.dks.tok,
                       rows - r0, g, a.scale);
            store_bf16(stage, lane, a.dv + row * a.dvs.tok + h * a.dvs.head + 32 * half, a.dvs.tok,
                       rows - r0, v, 1.f);
          }
          fence_proxy_async();
        }
      } else if (kind == kZero && a.splits > 1) {
        const int64_t at = item->split * a.part_rows * a.Hkv * 64;
        zero_part(a.part0 + at, a.Hkv, item->h, item->part_row, rows);
        zero_part(a.part1 + at, a.Hkv, item->h, item->part_row, rows);
      } else {
        fill_grad(a, item, a.dk, a.dks);
        fill_grad(a, item, a.dv, a.dvs);
      }
      __syncwarp();
      mbar_arrive_if(el, &bars->own_empty[slot]);
    }
    if (!ok) raise_abort(k.abort, a.status);
  }
  block_end();
}

// grad[row, head] = the pieces' sums, added in piece order; 16 lanes a (row, head).
__global__ void __launch_bounds__(256) view_sum_kernel(const float* part, const BwdArgs a, int heads,
                                                       bool keys, uint16_t* grad, Stride2 s) {
  const int64_t pair = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
  if (pair >= a.part_rows * heads) return;
  const int64_t slot = pair / heads;
  const int h = static_cast<int>(pair - slot * heads), c = threadIdx.x & 15;
  const int most = keys ? a.max_k : a.max_q, seg = static_cast<int>(slot / most);
  const int r = static_cast<int>(slot - int64_t(seg) * most);
  const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
  if (!g.ok || r >= (keys ? g.nk : g.nq)) return;
  const int64_t row = static_cast<int64_t>(keys ? g.k0 : g.q0) + r;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < a.splits; ++i) {
    const float4 y = *reinterpret_cast<const float4*>(
        part + (i * a.part_rows * heads + pair) * 64 + 4 * c);
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
  const size_t qrows = static_cast<size_t>(p.nseg) * p.max_q * p.H;  // of partial sums
  const size_t krows = static_cast<size_t>(p.nseg) * p.max_k * p.Hkv;
  ViewBwdLayout l{};
  l.sq = pieces(tq * p.nseg * p.H, tk, qrows);
  l.skv = pieces(tk * p.nseg * p.Hkv, tq * (p.H / p.Hkv), 2 * krows);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += round256(bytes);
    return x;
  };
  l.dsum = take(static_cast<size_t>(p.Lq) * p.H * 4);
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
  cudaError_t e = allow_smem(view_dq_kernel, kSmemBytes);
  if (e == cudaSuccess) e = allow_smem(view_dkv_kernel, kSmemBytes);
  if (e != cudaSuccess) return e;
  const bool all_rows = p.flags & S3R_FLAG_ALL_ROWS;
  float* dsum = reinterpret_cast<float*>(w + l.dsum);
  BwdArgs a{qo, ko, lse, dsum, dq, dk, dv, p.dqs, p.dks, p.dvs, nullptr, nullptr, p.Lq, p.Lk, 0, p.H,
            p.Hkv, p.H / p.Hkv, p.nseg, p.max_q, p.max_k, 0, 0, 0, 0, p.scale, p.scale_log2, p.flags,
            p.status, (p.flags & S3R_FLAG_TEST_TIMEOUT) ? 1000000ull : 2000000000ull};
  if (has_q) {
    const int64_t d_blocks = ceil_div(p.Lq, 32) * p.H;
    a.tiles = static_cast<int>(p.max_q > 0 ? ceil_div(p.max_q, kTile) : 1);
    a.splits = l.sq;
    a.part0 = reinterpret_cast<float*>(w + l.dq);
    a.part_rows = static_cast<int64_t>(p.nseg) * p.max_q;
    a.rest_items = all_rows ? static_cast<int>(rest_items(p.Lq)) : 0;
    const int64_t work = static_cast<int64_t>(p.nseg) * a.tiles * a.splits * p.H;
    const int64_t items = work + static_cast<int64_t>(a.rest_items) * p.H;
    a.work_items = static_cast<uint32_t>(work);
    if (items > INT_MAX || d_blocks > INT_MAX) return cudaErrorInvalidValue;
    view_d_kernel<<<static_cast<unsigned>(d_blocks), 256, 0, st>>>(out, dout, dsum, p.Lq, p.H);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    view_dq_kernel<<<static_cast<unsigned>(items), kThreads, kSmemBytes, st>>>(tq, to, tk, tv, a);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (l.sq > 1) {
      view_sum_kernel<<<static_cast<unsigned>(ceil_div(a.part_rows * p.H * 16, 256)), 256, 0, st>>>(
          a.part0, a, p.H, false, dq, p.dqs);
      count_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  }
  if (has_k) {
    a.tiles = static_cast<int>(p.max_k > 0 ? ceil_div(p.max_k, kTile) : 1);
    a.splits = l.skv;
    a.part0 = reinterpret_cast<float*>(w + l.dk);
    a.part1 = reinterpret_cast<float*>(w + l.dv);
    a.part_rows = static_cast<int64_t>(p.nseg) * p.max_k;
    a.rest_items = all_rows ? static_cast<int>(rest_items(p.Lk)) : 0;
    const int64_t work = static_cast<int64_t>(p.nseg) * a.tiles * a.splits * p.Hkv;
    const int64_t items = work + static_cast<int64_t>(a.rest_items) * p.Hkv;
    a.work_items = static_cast<uint32_t>(work);
    if (items > INT_MAX) return cudaErrorInvalidValue;
    view_dkv_kernel<<<static_cast<unsigned>(items), kThreads, kSmemBytes, st>>>(tq, to, tk, tv, a);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (l.skv > 1) {
      const unsigned grid = static_cast<unsigned>(ceil_div(a.part_rows * p.Hkv * 16, 256));
      view_sum_kernel<<<grid, 256, 0, st>>>(a.part0, a, p.Hkv, true, dk, p.dks);
      count_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      view_sum_kernel<<<grid, 256, 0, st>>>(a.part1, a, p.Hkv, true, dv, p.dvs);
      count_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace s3r
