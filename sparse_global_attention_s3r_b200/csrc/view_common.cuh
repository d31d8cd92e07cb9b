// view_common.cuh -- what the dense attention kernels (view_attn.cu, view_attn_bwd.cu) share.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"
#include "s3r_view.h"
#include "sm100.cuh"
#include "view_internal.h"

namespace s3r {
namespace view {

using namespace sm100;

// One head's [128, 64] tile of a [L, H, 64] tensor in any token and head stride: 128-byte rows,
// 128-byte swizzle.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int head,
                                              int32_t row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(row), "r"(smem_addr(bar))
      : "memory");
}

// Generic-proxy writes to shared memory before tcgen05 / TMA reads of it.
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

// One TMEM column of a warp's 32 lanes, and the wait for every store so far.
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(r) : "memory");
}
__device__ __forceinline__ void tmem_wait_st_all() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// Three-input maximum that keeps a NaN: a NaN logit has to reach its row's result.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void raise_abort(volatile int* abort, uint32_t* status) {
  *abort = 1;
  set_status(status, S3R_DEV_TIMEOUT);
}

// One lane of a converged warp. The MMA warps stay whole: all lanes run the loop and its waits, and
// the tensor instructions are predicated on this one's flag. Their descriptors and addresses are
// then uniform to the compiler and live in uniform registers. Issued from a branch of one lane,
// every operand of every instruction was first moved there: 110 clocks a MMA instead of about 20,
// and the issuing thread bounded the kernel (attention of one head over 10,992 keys, per 256 x 128
// tile: 3,800 clocks of issue).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(e));
  return e;
}
// D[tmem] (+)= A B by the elected lane: A in shared memory (ss) or TMEM (ts).
__device__ __forceinline__ void mma_ss_if(uint32_t e, uint32_t d_tmem, uint64_t a_desc,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t e, uint32_t d_tmem, uint32_t a_tmem,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}
// Arrive once on `bar` when every tcgen05 operation the elected lane issued so far has completed.
__device__ __forceinline__ void tc_commit_if(uint32_t e, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar)),
      "r"(e)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_if(uint32_t e, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_addr(bar)),
      "r"(e)
      : "memory");
}
// mbar_wait with a shorter way through: the waits of the softmax loops mostly end within the first
// suspension, so the clock and the abort flag are looked at from the fourth one on.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t n = 0; !mbar_test_suspend(bar, parity, kSuspendNs); ++n) {
    if (n < 4) continue;
    if (*abort) return false;
    const uint64_t now = globaltimer_ns();
    if (n == 4)
      t0 = now;
    else if (now - t0 > limit_ns)
      return false;
  }
  return true;
}
// Whether a phase has completed, without waiting; warp-uniform.
__device__ __forceinline__ bool mbar_peek(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// wait_bar of a whole warp: true only if it was for every lane.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, volatile int* abort,
                                              uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, limit_ns));
}

// Dynamic scheduling of the persistent kernels. The grid has a block per item; a block that has
// started takes the items of blocks that have not (cluster launch control), so that the SMs finish
// together however unequal the items are. One request is in flight at a time: its answer, 16 bytes
// in shared memory, completes `bar`.
__device__ __forceinline__ void request_item(uint32_t e, void* answer, uint64_t* bar) {
  if (e) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::
            "r"(smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
  }
}
// The answer, once `bar` has completed: whether an item was taken, and its number. Whole warp.
__device__ __forceinline__ bool taken_item(const void* answer, uint32_t* item) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n"
      " mov.u32 %1, 0;\n @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
      : "=r"(got), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  fence_proxy_async();  // this read before the next answer's write
  __syncwarp();
  *item = x;
  return got != 0;
}

// Items in a row that hold no rows (tiles past their segment's end, unusable segments) are passed over by
// the producer alone, in about 0.5 us each; after so many it hands on an item of no rows, so that the warps
// that wait for the next one do not take it for lost.
constexpr uint32_t kSkips = 1u << 16;

// Rows of one segment. ok is false where the offsets cannot be used: the caller's block then
// writes nothing.
struct Segment {
  int q0, nq, k0, nk;
  bool ok;
};
__device__ __forceinline__ Segment load_segment(const int32_t* qo, const int32_t* ko, int s,
                                                int64_t Lq, int64_t Lk, int max_q, int max_k) {
  const int64_t a = qo[s], b = qo[s + 1], c = ko[s], d = ko[s + 1];
  Segment g;
  g.ok = a >= 0 && a <= b && b <= Lq && b - a <= max_q && c >= 0 && c <= d && d <= Lk &&
         d - c <= max_k;
  g.q0 = static_cast<int>(a);
  g.nq = static_cast<int>(b - a);
  g.k0 = static_cast<int>(c);
  g.nk = static_cast<int>(d - c);
  return g;
}

// S3R_FLAG_ALL_ROWS: the rows of no segment, [0, before) and [after, L) of a tensor of L rows, and the
// rows of a segment that cannot be used, clipped to the tensor.
struct Rows {
  int before, after;
};
__device__ __forceinline__ Rows rows_outside(const int32_t* offs, int nseg, int64_t L) {
  const int top = static_cast<int>(L), first = offs[0], last = offs[nseg];
  Rows r;
  r.before = first < 0 ? 0 : first > top ? top : first;
  r.after = last < r.before ? r.before : last > top ? top : last;
  return r;
}
__device__ __forceinline__ Rows rows_clipped(const int32_t* offs, int s, int64_t L) {
  const int top = static_cast<int>(L), a = offs[s], b = offs[s + 1];
  Rows r;
  r.before = a < 0 ? 0 : a;
  r.after = b > top ? top : b;
  return r;
}

// Zero the 128-byte rows [from, 128) of a 128-row tile (32 lanes): rows that TMA brought in but
// that belong to another segment. Their products would be 0 * x, which is not 0 for an infinity or
// a NaN.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
  for (int i = from * 8 + lane; i < 128 * 8; i += 32)
    reinterpret_cast<uint4*>(tile)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// A warp's way from a row a lane to whole rows in memory: 16-byte piece i of the lane's row of
// kPieces (8 or 4) goes to at most 4 KB of shared memory, swizzled so that neither side has bank
// conflicts, and warp_rows writes 32 rows from there, kPieces lanes a row. Stored from the lanes as
// they hold them, every instruction touched 32 lines: 4,200 clocks for a block's 256 rows of a result.
template <int kPieces>
__device__ __forceinline__ uint8_t* piece_at(uint8_t* stage, int row, int i) {
  return stage + row * (16 * kPieces) + ((i ^ (kPieces == 8 ? row & 7 : (row >> 1) & 3)) << 4);
}
template <int kPieces>
__device__ __forceinline__ void put_piece(uint8_t* stage, int lane, int i, uint4 x) {
  *reinterpret_cast<uint4*>(piece_at<kPieces>(stage, lane, i)) = x;
}
// Rows 0 .. rows - 1 (at most 32) to dst + row * stride bytes. Whole warp.
template <int kPieces>
__device__ __forceinline__ void warp_rows(uint8_t* stage, int lane, void* dst, int64_t stride, int rows) {
  constexpr int kStep = 32 / kPieces;  // rows an instruction
  const int i = lane % kPieces, r0 = lane / kPieces;
  uint8_t* d = static_cast<uint8_t*>(dst) + r0 * stride + i * 16;
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 32; r += kStep, d += kStep * stride)
    if (r + r0 < rows)
      *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(piece_at<kPieces>(stage, r + r0, i));
  __syncwarp();
}

}  // namespace view

// Tensor map of a [rows, H, 64] bf16 tensor with the given strides, for boxes of one head's
// [128, 64] rows (tma_host.cu). With no rows the map covers nothing and must not be used.
bool make_tmap_rows3(CUtensorMap* map, const void* base, int64_t rows, int H, Stride2 s);

}  // namespace s3r
