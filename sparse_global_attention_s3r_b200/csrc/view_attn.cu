// view_attn.cu -- dense attention of every query over the keys of its own segment, on the sm_100a
// tensor cores (tcgen05 + TMEM + TMA).
//
// Per head and segment, with t = scale log2(e) <q, k>:  out = sum_j 2^(t_j - m) v_j / l with
// l = sum_j 2^(t_j - m), one pass over the keys. m is a row's reference, not its running maximum:
// the largest of its first 32 logits. Since P is bf16 and every sum fp32, of one exponent range, any
// m serves as long as nothing overflows, so no maximum is formed of later tiles: a tile whose sum of
// P passes 2^60 moves the reference and is done again (far_tile). lse = (m + log2 l) ln 2.
//
// Persistent, one block per SM, which walks items: (segment, 256 query rows, piece of the keys, head).
// A block holds two units, each 128 query rows (a TMEM lane a row) with its own S (fp32, 128
// columns), P (bf16, 64 columns) and O (fp32, 64 columns) in TMEM, 512 columns in all, its own issuer
// of products and its own four softmax warps, one thread a row, so a row's sum needs no exchange.
// While a unit's exponentials run, its next S, its last product with V and the other unit's products
// do; the next item's tiles are on their way while this one's result is written.
//   two tiles   (more than 128 rows) unit u has rows 128 u .. 128 u + 127, and each key tile feeds
//               both units
//   one tile    (128 rows or fewer, down to one) both units have the same rows and take the key
//               tiles in turn, unit u those of parity u; unit 0 joins the two results at the end.
//               For a few rows this is bound by reading the keys, and the softmax of one warp
//               alone would not keep up with that; warps without rows do nothing.
// What bounds it at many rows: the exponential unit, 16 per clock per SM, 2,048 clocks per 256 x 128
// logits, against 1,224 of products. A tile takes about 2,900, since the two warps of a sub-partition
// tend to run in step; an item 6,000 more (fitted over 1 to 10 key tiles). In a burst of a dozen passes 32
// views of 1,374 tokens, 16 heads, take 373 us (663 TFLOP/s), one query over 137,400 keys 105 us (5.4 TB/s,
// 5 us of it the joining kernel); in a long run of passes, when the power limit lowers the clock to 1.8 GHz,
// 396 us (625 TFLOP/s) and 118 us (4.8 TB/s).
// When there are too few blocks to fill the GPU, the keys are split into pieces (view_fwd_splits)
// whose fp32 results view_join_kernel adds, in order.
//
// Roles (352 threads): warps 0-3 and 4-7 softmax of unit 0 and 1 (lane quadrant warp % 4), warp 8
// TMA producer, warps 9 and 10 MMA issuers of unit 0 and 1 (9 owns the TMEM). Every wait is bounded
// in time and watches a block abort flag (S3R_DEV_TIMEOUT on expiry).
#include <climits>
#include <cmath>

#include "internal.h"
#include "view_common.cuh"

namespace s3r {
namespace {

using namespace view;

constexpr int kThreads = 352;  // 3 warps at most per sub-partition: 168 registers a thread
constexpr int kStages = 5;  // key and value tiles in flight
constexpr int kRows = 256;  // query rows of a block
constexpr int kTile = 128;  // rows of a unit, keys of a tile
constexpr uint32_t kTileBytes = kTile * 128;
// of every 8 pairs of exponentials, on the FMA pipe as a polynomial: 1 took 2 to 3 % off (32 views of
// 1,374 tokens: 406 -> 396 us), 2 and more lost it again to the issue slots and to spilled registers
constexpr int kPolyOf8 = 1;
constexpr float kFarSum = 1152921504606846976.f;  // 2^60: a row's reference moves beyond this

constexpr uint32_t kColS = 0, kColP = 256, kColO = 384, kTmemCols = 512;  // unit u: +128u, +64u, +64u
constexpr uint32_t kIdescQK = idesc_bf16_f32(kTile, kTile, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16_f32(kTile, 64, 0, 1);

struct __align__(8) Bars {
  uint64_t q_full[2], q_empty[2];          // an item's queries and its description
  uint64_t full[kStages], empty[kStages];  // key and value tile of a stage
  uint64_t tail;                   // TMA of the tiles that are cut by the segment's end
  uint64_t s_full[2], s_empty[2];  // S of a unit written / read into registers
  uint64_t p_full[2], p_empty[2];  // P written / its product with V completed
  uint64_t o_full[2];              // every product of the unit for this item completed
  uint64_t joined, join_done;      // one tile: unit 1's m, l and O can be read / have been read
  uint64_t next;  // the answer to a request for an item
  uint64_t drain[2];
  uint64_t never;  // never signalled: waited on only under S3R_FLAG_TEST_TIMEOUT
};
// What the producer tells the other warps of an item.
struct Item {
  int kind;  // kEnd, kZero (no keys: write zeros), kRest (rows of no segment: zeros), kBad (a segment
             // that cannot be used: NaN), kWork
  int row, rows;  // first row of q and how many (kRest: part_row from 0, the others from `row`)
  int n, tail;    // key tiles, keys of the last one (kRest: n is the item's number of the head's)
  int h, split;
  int part_row;  // splits > 1: the first row's place in the partial results
};
enum { kEnd, kZero, kRest, kBad, kWork };
constexpr uint32_t kOffQ = 0;  // [2 items][2 tiles]
constexpr uint32_t kOffRing = 4 * kTileBytes;  // stage: K | V
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kOffML = kOffRing + kStages * kStageBytes;  // [2][128] f32: m and l of unit 1
constexpr uint32_t kOffNext = kOffML + 1024;  // 16 bytes: the answer to a request for an item
constexpr uint32_t kOffItem = kOffNext + 16;  // [2] Item
constexpr uint32_t kOffBars = kOffItem + 2 * sizeof(Item);
constexpr uint32_t kOffMisc = kOffBars + sizeof(Bars);
constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 227 * 1024 && sizeof(Item) % 4 == 0 && kOffBars % 8 == 0,
              "shared memory of a block");

struct FwdArgs {
  const int32_t *qo, *ko;
  uint16_t* out;  // [Lq, H, 64] bf16
  float* lse;     // [H, Lq] or null
  // splits > 1, for part_rows = nseg * max_q rows (row r of segment s: s * max_q + r):
  float* o_part;  // [splits][part_rows, H, 64] f32
  float* l_part;  // [splits][H, part_rows], in base-2 units
  int64_t Lq, Lk, part_rows;
  int H, group, nseg, max_q, max_k, tiles, splits;
  // items: (segment, row tile, key piece, head), heads fastest; then rest_items * H for the rows of no segment
  uint32_t work_items;
  int rest_items;
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

__device__ __forceinline__ float row_max(const uint32_t (&s)[32]) {
  float x[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t* v = s + 8 * c;
    x[c] = fmax3_nan(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
    x[c] = fmax3_nan(x[c], __uint_as_float(v[3]), __uint_as_float(v[4]));
    x[c] = fmax3_nan(x[c], __uint_as_float(v[5]), __uint_as_float(v[6]));
    x[c] = fmax3_nan(x[c], __uint_as_float(v[7]), x[c]);
  }
  return fmax3_nan(fmax3_nan(x[0], x[1], x[2]), x[3], x[3]);
}

// The exponentials of 32 logits in two steps, so that the results of one chunk are packed while the
// exponential unit works on the next: the volatile statements keep that order. (Left to the
// compiler, each result was used soon after its exponential was issued, and a chunk of 32 took 370
// clocks instead of 290.)
__device__ __forceinline__ float exp2_now(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float clamp_nan(float x) {
  asm("{\n max.NaN.f32 %0, %0, %1;\n min.NaN.f32 %0, %0, %2;\n}\n" : "+f"(x) : "f"(-127.f), "f"(127.f));
  return x;
}
// s <- 2^(s sl2 - m)
__device__ __forceinline__ void exp_issue(uint32_t (&s)[32], float sl2, float m) {
  const float2 mul = make_float2(sl2, sl2), off = make_float2(-m, -m);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = __ffma2_rn(
        make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), mul, off);
    // (clamped where 2^x ends: a far logit has to make the sum large, a NaN has to stay one)
    const float2 e = (i & 7) < kPolyOf8
                         ? exp2_poly5x2_in(make_float2(clamp_nan(x.x), clamp_nan(x.y)))
                         : make_float2(exp2_now(x.x), exp2_now(x.y));
    s[2 * i] = __float_as_uint(e.x);
    s[2 * i + 1] = __float_as_uint(e.y);
  }
}
// p <- 16 packed pairs of bf16; sum += s
__device__ __forceinline__ void exp_finish(const uint32_t (&s)[32], uint32_t (&p)[16], float2& sum) {
  float2 acc[2];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 e = make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
    asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(p[i]) : "f"(e.y), "f"(e.x));
    acc[i & 1] = i < 2 ? e : __fadd2_rn(acc[i & 1], e);
  }
  sum = __fadd2_rn(sum, __fadd2_rn(acc[0], acc[1]));
}

// A tile in which some row's logits are so far above its reference that the sum of its P passed
// kFarSum: every row of the warp moves its reference up to the tile's maximum where that is larger,
// O so far (complete: p_empty has been waited for) is rescaled, and P is formed again. S has been
// handed back by then, so the logits are formed from the tiles in shared memory, on the FMA pipe:
// 68 us against 1.5 of an ordinary tile, for logits that rise by more than 40 (base e) above a row's reference.
// Returns the new reference, the sum of P and the factor of what was summed before. Whole warp.
__device__ __noinline__ float3 far_tile(const uint8_t* q_tile, int row, const uint8_t* k_tile, int keys,
                                        float sl2, float m, uint32_t tP, uint32_t tO, bool rescale) {
  auto chunk = [](const uint8_t* tile, int r, int i) {  // 16 bytes of a 128-byte swizzled row
    return *reinterpret_cast<const uint4*>(tile + r * 128 + ((i ^ (r & 7)) << 4));
  };
  auto dot = [&](int j) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 a = chunk(q_tile, row, i), b = chunk(k_tile, j, i);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), x);
        x = fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(v[e] & 0xffff0000u), x);
      }
    }
    return x * sl2;
  };
  float top = -INFINITY;
  for (int j = 0; j < keys; ++j) top = fmax3_nan(top, dot(j), top);
  const float to = !(top <= m) ? top : m;
  const float f = exp2_approx(m - to);
  if (rescale) {
    for (int z = 0; z < 4; ++z) {
      uint32_t o[16];
      tmem_ld32x16(tO + 16 * z, o);
      tmem_wait_ld_n<16>(o);
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st32x16(tO + 16 * z, o);
      tmem_wait_st_keep16(o);
    }
  }
  float sum = 0.f;
  for (int j = 0; j < kTile; j += 2) {
    const float a = j < keys ? exp2_approx(dot(j) - to) : 0.f;
    const float b = j + 1 < keys ? exp2_approx(dot(j + 1) - to) : 0.f;
    sum += a + b;
    tmem_st1(tP + j / 2, pack_bf16(a, b));
  }
  tmem_wait_st_all();
  return make_float3(to, sum, f);
}

// Items without work, by the 256 softmax threads: zeros and lse = -inf (kZero; with several key
// pieces only the piece's lse, which the joining kernel goes by), the same for rows of no segment
// (kRest: 256 rows of every 256 * rest_items), or NaN (kBad).
__device__ __forceinline__ void fill_item(const FwdArgs& a, const volatile Item* m, int kind, int warp,
                                          int lane) {
  const int h = m->h, rows = m->rows, before = kind == kRest ? m->part_row : 0;
  const int64_t row = m->row;
  const uint32_t w = kind == kBad ? 0x7fc07fc0u : 0u;
  const float l = kind == kBad ? __int_as_float(0x7fc00000) : -INFINITY;
  const int64_t first = (kind == kRest ? static_cast<int64_t>(m->n) * kRows : 0) + warp * 32 + lane;
  for (int64_t i = first; i < rows; i += (kind == kRest ? static_cast<int64_t>(a.rest_items) : 1) * kRows) {
    if (kind == kZero && a.splits > 1) {
      a.l_part[(static_cast<int64_t>(m->split) * a.H + h) * a.part_rows + m->part_row + i] = l;
      continue;
    }
    const int64_t r = i < before ? i : row + i - before;
    uint4* o = reinterpret_cast<uint4*>(a.out + (r * a.H + h) * 64);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = make_uint4(w, w, w, w);
    if (a.lse) a.lse[h * a.Lq + r] = l;
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
  Item* items = reinterpret_cast<Item*>(smem + kOffItem);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 2);  // both MMA warps
    }
    mbar_init(&bars->tail, 1);
    mbar_init(&bars->next, 1);
    for (int u = 0; u < 2; ++u) {
      mbar_init(&bars->q_full[u], 1);
      mbar_init(&bars->q_empty[u], 10);  // both MMA warps, the eight softmax warps
      mbar_init(&bars->s_full[u], 1);
      mbar_init(&bars->s_empty[u], 4);
      mbar_init(&bars->p_full[u], 4);
      mbar_init(&bars->p_empty[u], 1);
      mbar_init(&bars->o_full[u], 1);
      mbar_init(&bars->drain[u], 1);
    }
    mbar_init(&bars->joined, 4);
    mbar_init(&bars->join_done, 4);
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
  constexpr uint32_t tbase = 0;  // all 512 columns are this block's, so they start at 0

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    bool ok = true;
    bool cut = false;        // the last issued tiles land on `tail`, not yet handed on
    int k = 0, tile_no = 0, cuts = 0;  // items, key tiles and cut tiles so far
    uint32_t it = blockIdx.x;
    bool more = true;  // `it` is an item
    int asked = 0;     // requests so far
    uint32_t skipped = 0;  // items without rows so far
    for (bool first = true; ok; first = false) {
      if (!first) {  // the item asked for while the last one was issued
        if (!(ok = wait_bar_warp(&bars->next, (asked - 1) & 1, abort, lim))) break;
        more = taken_item(smem + kOffNext, &it);
      }
      if (more) request_item(lane == 0, smem + kOffNext, &bars->next), ++asked;
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
          } else if (tile * kRows < g.nq) {
            const int row0 = tile * kRows;
            m.row = g.q0 + row0;
            m.part_row = a.splits > 1 ? seg * a.max_q + row0 : 0;
            m.rows = g.nq - row0 < kRows ? g.nq - row0 : kRows;
            // key tiles [t0, t0 + n) of the segment
            const int all = (g.nk + kTile - 1) / kTile;
            const int per = (all + a.splits - 1) / a.splits;
            const int t0 = m.split * per;
            m.n = all - t0 < per ? all - t0 : per;
            m.kind = m.n > 0 ? kWork : kZero;
            // (a piece that ends before the segment does has a whole last tile)
            const int left = g.nk - (t0 + m.n - 1) * kTile;
            m.tail = left < kTile ? left : kTile;
            key0 = g.k0 + t0 * kTile;
          }
          if (m.kind == kEnd) {  // no rows
            if (++skipped % kSkips) continue;
            m.kind = kZero;
          }
        }
      }
      const int slot = k & 1;
      if (!(ok = wait_bar_warp(&bars->q_empty[slot], ((k >> 1) & 1) ^ 1, abort, lim))) break;
      const bool one = m.rows <= kTile;
      if (lane == 0) {
        items[slot] = m;
        if (m.kind == kWork) {
          const uint32_t q = sbase + kOffQ + slot * 2 * kTileBytes;
          mbar_arrive_expect_tx(&bars->q_full[slot], one ? kTileBytes : 2 * kTileBytes);
          tma_load_rows(q, &tmQ, m.h, m.row, &bars->q_full[slot]);
          if (!one) tma_load_rows(q + kTileBytes, &tmQ, m.h, m.row + kTile, &bars->q_full[slot]);
        } else {
          mbar_arrive(&bars->q_full[slot]);
        }
      }
      ++k;
      if (m.kind == kEnd) break;
      if (m.kind != kWork) continue;
      const int hk = m.h / a.group;
      for (int t = 0; t < m.n; ++t) {
        const int st = tile_no % kStages;
        const uint32_t sk = sbase + kOffRing + st * kStageBytes;
        // every lane waits, so that the warp stays together and all lanes see the tile
        if (!(ok = wait_bar_warp(&bars->empty[st], ((tile_no / kStages) & 1) ^ 1, abort, lim))) break;
        cut = t == m.n - 1 && m.tail < kTile;
        if (lane == 0) {
          uint64_t* full = cut ? &bars->tail : &bars->full[st];
          mbar_arrive_expect_tx(full, kStageBytes);
          tma_load_rows(sk, &tmK, hk, key0 + t * kTile, full);
          tma_load_rows(sk + kTileBytes, &tmV, hk, key0 + t * kTile, full);
        }
        ++tile_no;
        if (cut) {  // the value tile reaches past the segment
          if (!(ok = wait_bar_warp(&bars->tail, cuts & 1, abort, lim))) break;
          ++cuts;
          cut = false;
          zero_rows(smem + kOffRing + st * kStageBytes + kTileBytes, m.tail, lane);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->full[st]);
        }
      }
    }
    if (!ok && lane == 0) {  // let the copies in flight land before the block ends
      raise_abort(abort, a.status);
      int dummy = 0;
      if (asked > 0) wait_bar(&bars->next, (asked - 1) & 1, &dummy, lim);
      for (int i = k - 1; i >= 0 && i >= k - 2; --i)
        wait_bar(&bars->q_full[i & 1], (i >> 1) & 1, &dummy, lim);
      if (cut) wait_bar(&bars->tail, cuts & 1, &dummy, lim);
      for (int t = tile_no - 1 - (cut ? 1 : 0); t >= 0 && t >= tile_no - kStages; --t)
        wait_bar(&bars->full[t % kStages], (t / kStages) & 1, &dummy, lim);
    }
  } else if (warp >= 9) {
    // ------------------------------------------------------------------ MMA issuers, one a unit
    const uint32_t el = elect_one();
    const int u = warp - 9;
    bool ok = true;
    int tile_no = 0, c = 0;  // key tiles so far, steps of this unit so far
    for (int k = 0; ok; ++k) {
      const int slot = k & 1;
      if (!(ok = wait_bar_warp(&bars->q_full[slot], (k >> 1) & 1, abort, lim))) break;
      const volatile Item* item = items + slot;
      const int kind = item->kind, n = item->n;
      if (kind == kEnd) break;
      const bool one = item->rows <= kTile;
      if (kind == kWork) {
        const uint64_t dq =
            desc_sw128(sbase + kOffQ + slot * 2 * kTileBytes + (one ? 0 : u * kTileBytes));
        const int step = one ? 2 : 1, first = one ? u : 0;
        // S of the unit's step x, key tile t of the item
        auto qk = [&](int x, int t) -> bool {
          const int st = (tile_no + t) % kStages;
          if (!wait_bar_warp(&bars->full[st], ((tile_no + t) / kStages) & 1, abort, lim)) return false;
          if (!wait_bar_warp(&bars->s_empty[u], (x & 1) ^ 1, abort, lim)) return false;
          tc_fence_after();
          const uint64_t dk = desc_sw128(sbase + kOffRing + st * kStageBytes);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss_if(el, tbase + kColS + u * 128, dq + 2 * ks, dk + 2 * ks, kIdescQK, ks > 0);
          tc_commit_if(el, &bars->s_full[u]);
          return true;
        };
        auto pv = [&](int x, int t) -> bool {
          const int st = (tile_no + t) % kStages;
          if (!wait_bar_warp(&bars->p_full[u], x & 1, abort, lim)) return false;
          tc_fence_after();
          const uint64_t dv = desc_sw128(sbase + kOffRing + st * kStageBytes + kTileBytes);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)  // 16 keys a step: 16 rows x 128 B = 2048 B
            mma_ts_if(el, tbase + kColO + u * 64, tbase + kColP + u * 64 + ks * 8, dv + 128 * ks,
                      kIdescPV, (t > first || ks > 0) ? 1u : 0u);
          tc_commit_if(el, &bars->p_empty[u]);
          tc_commit_if(el, &bars->empty[st]);
          return true;
        };
        // a key tile that is the other unit's: handed back once it has landed
        auto skip = [&](int t) -> bool {
          const int st = (tile_no + t) % kStages;
          if (!wait_bar_warp(&bars->full[st], ((tile_no + t) / kStages) & 1, abort, lim)) return false;
          mbar_arrive_if(el, &bars->empty[st]);
          return true;
        };
        if (one && u == 1) ok = skip(0);
        if (ok && first < n) ok = qk(c, first);
        for (int t = first; ok && t < n; t += step) {
          if (one && t + 1 < n && !(ok = skip(t + 1))) break;
          if (t + step < n && !(ok = qk(c + 1, t + step))) break;
          ok = pv(c, t);
          ++c;
        }
        if (!ok) break;
        if (first < n) tc_commit_if(el, &bars->o_full[u]);
        tile_no += n;
        tc_commit_if(el, &bars->q_empty[slot]);
      } else {
        mbar_arrive_if(el, &bars->q_empty[slot]);
      }
    }
    if (!ok) {
      if (el) raise_abort(abort, a.status);
      int dummy = 0;
      tc_commit_if(el, &bars->drain[u]);
      wait_bar(&bars->drain[u], 0, &dummy, lim);
    }
  } else {
    // ------------------------------------------------------------------ softmax warps
    const uint32_t el = elect_one();
    const int u = warp >> 2, qd = warp & 3;
    const uint32_t tl = tbase + (static_cast<uint32_t>(qd * 32) << 16);
    const uint32_t tS = tl + kColS + u * 128, tP = tl + kColP + u * 64, tO = tl + kColO + u * 64;
    const float sl2 = a.scale_log2;
    bool ok = true;
    int c = 0, done = 0, joins = 0, tile_no = 0;  // steps, items with steps, joined items, tiles
    if (a.flags & S3R_FLAG_TEST_TIMEOUT) ok = wait_bar(&bars->never, 0, abort, lim);
    for (int k = 0; ok; ++k) {
      const int slot = k & 1;
      if (!(ok = wait_bar(&bars->q_full[slot], (k >> 1) & 1, abort, lim))) break;
      const volatile Item* item = items + slot;
      const int kind = item->kind, n = item->n, tail = item->tail, rows = item->rows;
      if (kind == kEnd) break;
      if (kind != kWork) {
        fill_item(a, item, kind, warp, lane);
        __syncwarp();
        mbar_arrive_if(el, &bars->q_empty[slot]);
        continue;
      }
      const bool one = rows <= kTile;            // one tile: the units take the key tiles in turn
      const int r = (one ? 0 : u * kTile) + qd * 32 + lane;  // row of the item
      const int mine = one ? (n - u + 1) >> 1 : n;           // key tiles of this unit
      // a warp whose 32 rows are all past the end only keeps the barriers going: what its lanes of
      // P hold reaches no other lane of O
      const bool idle = (one ? 0 : u * kTile) + qd * 32 >= rows;
      float m = 0.f;
      float sum = 0.f;
      bool ready = false;  // a test of the next wait's barrier, made ahead: one takes about 100 clocks
      for (int i = 0; i < mine; ++i, ++c) {
        if (!ready && !(ok = wait_bar(&bars->s_full[u], c & 1, abort, lim))) break;
        tc_fence_after();
        const int t = one ? 2 * i + u : i;
        if (idle) {
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(el, &bars->s_empty[u]);
          ready = false;
          if (!(ok = wait_bar(&bars->p_empty[u], (c & 1) ^ 1, abort, lim))) break;
          __syncwarp();
          mbar_arrive_if(el, &bars->p_full[u]);
          continue;
        }
        const bool cut = t == n - 1 && tail < kTile;  // keys past the segment's end
        uint32_t s0[32], s1[32], s2[32], s3[32], p[16];
        tmem_ld32(tS, s0);
        tmem_ld32(tS + 32, s1);
        tmem_wait_ld_regs(s0);
        tmem_wait_ld_regs(s1);
        tmem_ld32(tS + 64, s2);
        tmem_ld32(tS + 96, s3);
        if (cut) {
          mask_from(s0, tail);
          mask_from(s1, tail - 32);
        }
        if (i == 0) {  // the reference (a branch: the other tiles have no maximum to wait for)
          m = row_max(s0) * sl2;
          m = m == -INFINITY ? 0.f : m;
          asm volatile("" : "+f"(m));
        }
        float2 part = make_float2(0.f, 0.f);
        exp_issue(s0, sl2, m);
        tmem_wait_ld_regs(s2);
        tmem_wait_ld_regs(s3);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(el, &bars->s_empty[u]);
        if (cut) {
          mask_from(s2, tail - 64);
          mask_from(s3, tail - 96);
        }
        exp_issue(s1, sl2, m);
        ready = mbar_peek(&bars->p_empty[u], (c & 1) ^ 1);
        exp_finish(s0, p, part);
        if (!ready && !(ok = wait_bar(&bars->p_empty[u], (c & 1) ^ 1, abort, lim))) break;
        tc_fence_after();
        tmem_st32x16(tP, p);
        exp_issue(s2, sl2, m);
        exp_finish(s1, p, part);
        tmem_st32x16(tP + 16, p);
        exp_issue(s3, sl2, m);
        ready = mbar_peek(&bars->s_full[u], (c & 1) ^ 1);
        exp_finish(s2, p, part);
        tmem_st32x16(tP + 32, p);
        exp_finish(s3, p, part);
        tmem_st32x16(tP + 48, p);
        tmem_wait_st_keep16(p);
        float tile_sum = part.x + part.y;
        if (__any_sync(0xffffffffu, tile_sum > kFarSum)) {
          const int tt = tile_no + t;
          if (!(ok = wait_bar(&bars->full[tt % kStages], (tt / kStages) & 1, abort, lim))) break;
          const float3 x = far_tile(
              smem + kOffQ + (slot * 2 + (one ? 0 : u)) * kTileBytes, qd * 32 + lane,
              smem + kOffRing + (tt % kStages) * kStageBytes, t == n - 1 ? tail : kTile, sl2, m, tP,
              tO, i > 0);
          m = x.x;
          tile_sum = x.y;
          sum *= x.z;
        }
        sum += tile_sum;
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(el, &bars->p_full[u]);
      }
      if (!ok) break;
      tile_no += n;
      // the unit's result, joined with the other unit's where they share rows
      const bool join = one && n > 1;
      if (mine > 0) {
        if (!(ok = wait_bar(&bars->o_full[u], done & 1, abort, lim))) break;
        ++done;
        tc_fence_after();
      }
      float* ml = reinterpret_cast<float*>(smem + kOffML) + qd * 32 + lane;
      float l = sum;
      if (join && u == 1) {  // unit 0 reads O from this unit's columns of the same lanes
        ml[0] = m;
        ml[kTile] = l;
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(el, &bars->joined);
        if (!(ok = wait_bar(&bars->join_done, joins & 1, abort, lim))) break;
        ++joins;
      } else if (mine > 0) {
        float f0 = 1.f, f1 = 0.f;
        if (join) {
          if (!(ok = wait_bar(&bars->joined, joins & 1, abort, lim))) break;
          ++joins;
          tc_fence_after();
          const float m1 = ml[0], l1 = ml[kTile];
          const float to = fmax3_nan(m, m1, m1);
          f0 = exp2_approx(m - to);
          f1 = exp2_approx(m1 - to);
          m = to;
          l = l * f0 + l1 * f1;
        }
        if (!idle) {
          const float inv = 1.f / l;
          const int64_t row = item->row + r;
          const int h = item->h;
          // through the unit's rows of q, which no product reads any more
          uint8_t* stage = smem + kOffQ + (slot * 2 + (one ? 0 : u)) * kTileBytes + qd * 4096;
          const int left = rows - (r - lane);  // rows of this warp that count, or more
          const int64_t base = row - lane;
          const int64_t part = item->split * a.part_rows + item->part_row + r - lane;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * z, o);
            tmem_wait_ld_regs(o);
            if (join) {
              uint32_t o1[32];
              tmem_ld32(tO + 64 + 32 * z, o1);
              tmem_wait_ld_regs(o1);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * f0 + __uint_as_float(o1[j]) * f1);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
            if (a.splits > 1) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                put_piece<8>(stage, lane, j, make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
              warp_rows<8>(stage, lane, a.o_part + (part * a.H + h) * 64 + 32 * z,
                           static_cast<int64_t>(a.H) * 256, left);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack_bf16(__uint_as_float(o[8 * j + 2 * e]), __uint_as_float(o[8 * j + 2 * e + 1]));
                put_piece<8>(stage, lane, 4 * z + j, make_uint4(w[0], w[1], w[2], w[3]));
              }
            }
          }
          if (a.splits == 1)
            warp_rows<8>(stage, lane, a.out + (base * a.H + h) * 64, static_cast<int64_t>(a.H) * 128, left);
          fence_proxy_async();  // these reads and writes before the next item's queries land there
          if (r < rows) {
            const float lse2 = m + log2f(l);
            if (a.splits > 1)
              a.l_part[(static_cast<int64_t>(item->split) * a.H + h) * a.part_rows + item->part_row + r] =
                  lse2;
            else if (a.lse)
              a.lse[h * a.Lq + row] = lse2 * kLn2;
          }
        }
        if (join) {
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(el, &bars->join_done);
        }
      }
      __syncwarp();
      mbar_arrive_if(el, &bars->q_empty[slot]);
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
  const int64_t pair = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
  if (pair >= a.part_rows * a.H) return;
  const int64_t slot = pair / a.H;
  const int h = static_cast<int>(pair - slot * a.H);
  const int seg = static_cast<int>(slot / a.max_q), r = static_cast<int>(slot - int64_t(seg) * a.max_q);
  const Segment g = load_segment(a.qo, a.ko, seg, a.Lq, a.Lk, a.max_q, a.max_k);
  if (!g.ok || r >= g.nq) return;
  const int64_t row = static_cast<int64_t>(g.q0) + r;
  const int c = threadIdx.x & 15;
  const float* lp = a.l_part + h * a.part_rows + slot;
  const int64_t ls = a.H * a.part_rows;
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
          a.o_part + (s * a.part_rows * a.H + pair) * 64 + 4 * c);
      total += w;
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
    const float inv = 1.f / total;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  }
  *reinterpret_cast<uint2*>(a.out + (row * a.H + h) * 64 + 4 * c) =
      make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
  if (a.lse && c == 0) a.lse[h * a.Lq + row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
}

constexpr int kSMs = 148;
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

// Pieces of the keys: the count with the shortest estimated time, in key-tile times of a block
// (0.8 us for few rows): waves of blocks, each its tiles plus a start of about 3, and for more than one
// piece the joining kernel (about 6 and its traffic).
int view_fwd_splits(const ViewProblem& p) {
  const int64_t base = ceil_div(p.max_q, kRows) * p.nseg * p.H, tk = ceil_div(p.max_k, kTile);
  if (base == 0 || base >= 4 * kSMs || tk < 4) return 1;
  int best = 1;
  double best_t = 1e300;
  for (int64_t s = 1; s <= 128 && s <= tk / 2; ++s) {
    const double t = static_cast<double>(ceil_div(base * s, kSMs)) * (ceil_div(tk, s) + 3) +
                     (s > 1 ? 6. + static_cast<double>(s) * p.nseg * p.max_q * p.H * 512 / 4.5e6 : 0.);
    if (t < best_t) {
      best_t = t;
      best = static_cast<int>(s);
    }
  }
  return best;
}

size_t view_fwd_workspace(const ViewProblem& p) {
  const size_t s = view_fwd_splits(p), rows = static_cast<size_t>(p.nseg) * p.max_q * p.H;
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
  const int64_t part_rows = static_cast<int64_t>(p.nseg) * p.max_q;
  const size_t rows = static_cast<size_t>(part_rows) * p.H;
  float* o_part = splits > 1 ? static_cast<float*>(ws) : nullptr;
  float* l_part = splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                                        round256(splits * rows * 64 * 4))
                             : nullptr;
  const int64_t tiles = p.max_q > 0 ? ceil_div(p.max_q, kRows) : 1;
  const int64_t work = static_cast<int64_t>(p.nseg) * tiles * splits * p.H;
  const int64_t rest = (p.flags & S3R_FLAG_ALL_ROWS) ? rest_items(p.Lq) : 0;
  const int64_t blocks = work + rest * p.H;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  FwdArgs a{qo, ko, out, lse, o_part, l_part, p.Lq, p.Lk, part_rows, p.H, p.H / p.Hkv, p.nseg, p.max_q,
            p.max_k, static_cast<int>(tiles), splits, static_cast<uint32_t>(work),
            static_cast<int>(rest), p.scale_log2, p.flags, p.status,
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
