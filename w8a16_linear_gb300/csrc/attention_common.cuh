// What the attention kernels share: tile sizes, TMA copies of four and five
// dimensions, TMEM and register helpers, and the encoding of their tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace w8 {
namespace {

constexpr int kRows = 128;                        // query rows per slot
constexpr int kKeys = 128;                        // keys per tile
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per wait
constexpr int kAtom = 128 * 128;                  // 128 rows of one 128-byte swizzle span

// Rescaling the accumulator is put off until the row maximum has grown by
// more than this many powers of two: P stays below 2^8, exact scaling is kept
// (m is whatever the sums used), and most tiles touch O_i not at all.
constexpr float kLazyMax = 8.0f;

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

__device__ __forceinline__ void tma_store_5d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Waits for this thread's TMEM loads; naming the registers keeps their uses
// behind the wait while other loads are still under way.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// mbar_wait_warp with every lane asking first: no broadcast on the way of a
// phase that is complete or about to be.
__device__ __forceinline__ bool mbar_wait_lanes(uint32_t bar, uint32_t parity, volatile int* abort) {
  bool done = false;
#pragma unroll 1
  for (int k = 0; k < 64 && !done; ++k) done = mbar_try_wait(bar, parity);
  done = __all_sync(0xFFFFFFFFu, done);
  if (!done) done = mbar_wait_warp(bar, parity, abort, kWaitLimitNs);
  __syncwarp();   // the TMEM instructions that follow want the warp together
  return done;
}

// The roles' registers a thread: softmax warps hold a row of 128 scores.  The
// block starts with 128 x 512; 176 x 256 + 88 x 128 + 72 x 128 is the same sum.
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory descriptor of V as the MN-major B operand: 64 head dimensions
// (one 128-byte swizzle span) by 8 keys make a core group of 1024 bytes; key
// groups are 1024 bytes apart, spans of 64 dimensions one atom.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
  d |= (uint64_t)(kAtom >> 4) << 16;   // leading dimension: the next 64 of MN
  d |= (uint64_t)(1024 >> 4) << 32;    // stride dimension: the next 8 of K
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;              // 128-byte swizzle
  return d;
}

// n / d for n < 2^32 (d from the host), with by = 2^64 / d rounded up.
__device__ __forceinline__ int quotient(int n, uint64_t by) {
  return by ? (int)__umul64hi((uint64_t)(uint32_t)n, by) : n;
}

// Where CTA k of `ctas` begins in a row of `total` tiles: total k / ctas, in 32 bits.
__device__ __forceinline__ uint32_t share_begin(uint32_t total, uint32_t k, uint32_t ctas) {
  const uint32_t q = total / ctas;
  return k * q + k * (total - q * ctas) / ctas;
}

// A dimension of one entry, or one that the samples share, gets the stride
// of the dimension before it: its own is never used, and may be anything.
bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
            const int64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B,
            CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const cuuint64_t bytes = type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : 2;
  cuuint64_t st[4];
  for (int i = 0; i + 1 < rank; ++i) st[i] = dims[i + 1] > 1 ? (cuuint64_t)strides[i] * bytes : i ? st[i - 1] : dims[0] * bytes;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return fn(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace w8
