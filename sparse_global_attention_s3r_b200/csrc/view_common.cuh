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

// Moves registers between the warpgroups of a block (whole warpgroups call it).
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
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

// Zero the 128-byte rows [from, 128) of a 128-row tile (32 lanes): rows that TMA brought in but
// that belong to another segment. Their products would be 0 * x, which is not 0 for an infinity or
// a NaN.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
  for (int i = from * 8 + lane; i < 128 * 8; i += 32)
    reinterpret_cast<uint4*>(tile)[i] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace view

// Tensor map of a [rows, H, 64] bf16 tensor with the given strides, for boxes of one head's
// [128, 64] rows (tma_host.cu). With no rows the map covers nothing and must not be used.
bool make_tmap_rows3(CUtensorMap* map, const void* base, int64_t rows, int H, Stride2 s);

}  // namespace s3r
