// Attention over a paged cache for units of at most N = 16 query rows (the
// new token, or a few, of a sequence, times the query heads of a key head): the
// formula, units and pages of paged_attention.cu with the operands the other way round.
//
// Padding the rows to the 128 of an MMA would make 128 scores of each key, nearly all for
// nothing, and the way from a tile's copy to its stages' release so long that the
// copies wait for it.  Here the 128 keys of a tile are the MMA's M and the rows its N:
//   S^T = K_j Q^T        K from shared memory (K-major), 128 keys x N, to TMEM
//   P^T = exp2(S^T c - m)  a thread a key; 16-bit, row by row to shared memory
//   O^T += V_j^T P^T     V as MN-major A, so that dimensions are the lanes
// A row's maximum is over the lanes then.  The eight softmax warps keep the maxima of all
// rows in registers, alike, and one barrier a tile tells whether any score exceeds its
// maximum by more than 2^8; only then the maxima are made and O^T is scaled.
// The CTA's two groups of four softmax warps take the even and the odd tiles,
// with accumulators of their own, which the epilogue joins.
//
// E4M3 cells go to the tensor core as they are.  What stands beside them is split
// into three E4M3 terms, x = (t0 + t1 / 16 + t2 / 256) 2^e, which leaves at most 2^-12 of
// each value or 2^-18 in units of the terms: the queries, with the row's largest value in [2^7, 2^8)
// of those (so that at most 2^-25 of it is left, and nothing of a bf16 value from 2^-17 of it on, of an f16
// value from 2^-14 on), and P, whose largest is kept between 2^6 and 2^8 (so that 2^-24 of it is left).  Terms are rows of their own,
// 3 N, and the softmax and epilogue threads add the three results.  A group's scores of a tile
// are started before the products of the one before: two sets of S^T and P.
//
// Bound by the bytes of K and V.  Measured (GB300, a replayed graph), 32 query and 8 key
// heads of 128: 8 single tokens over 10335 to 20670 positions 87-92 us = 5.5-5.9 TB/s (0.83-0.88 of the
// measured copy; by the 128-row kernel, as that was then, 115 us), 16 of them 160 us = 6.3 TB/s, 16 over
// E4M3 cells 90 to 100 us = 5.1-5.7 TB/s (by the 128-row kernel 347; with V converted here 140, with its
// codes as they are 115, with rows without a query left out of Q's terms 99).  One token over 512
// positions: 8.4 us, a chain of latencies.  What runs once is mostly the
// fetching of instructions: loops are not unrolled and rows without a query left out, four at
// a time, where that makes the code shorter.
//
// Up to 16 rows.  A form of 32 against the 128-row kernel, both as they were then: 25 rows over 4133
// positions 32.2 against 25.1 us, 32 rows over 4133 51.9 against 41.7, 32 over 512 20.4 against
// 16.0; 20 rows over 20670 106 against 116, over E4M3 cells 283 against 331.  It won where few
// rows meet a long cache and lost elsewhere, and spilled registers: left out.
//
// Roundings below 32 bits: P (its sum l is taken before), since the tensor core takes 32-bit weights
// beside 32-bit values alone, which would be twice the bytes of V; beside E4M3 cells the terms
// above; and the output.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attention_common.cuh"
#include "few_ring.h"
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {
namespace {

constexpr int N = kFewRows;

template <int DP, bool kCodes>
struct Few {
  static constexpr int kAtoms = kCodes ? 1 : DP / 64;    // 128-byte spans of a row of K and V
  static constexpr int kTile = kAtoms * kAtom;           // bytes of 128 rows of them
  // Stages of a group's ring: of K and V in turn, or of E4M3 cells of each (of 16 bits
  // there is no room for two whole rings).
  static constexpr int kR = kCodes ? 0 : DP == 128 ? 3 : 5;
  static constexpr int kRK = kCodes ? 3 : 0, kRV = kCodes ? 2 : 0;
  static constexpr int kStages = kCodes ? kRK + kRV : kR;
  static constexpr int kCols = kCodes ? 3 * N : N;       // rows of Q and P, columns of S^T and O^T
  static constexpr int kAhead = kCodes ? 2 : 1;   // sets of S^T and P of a group
  static constexpr int kRing = 0;                        // codes: K's stages, then V's, of each group
  static constexpr int kQAtom = kCols * 128;
  static constexpr int kQ = kRing + 2 * kStages * kTile;
  static constexpr int kPAtom = kCols * 128;             // 128 bytes a row: 64 keys in 16 bits, 128 codes
  static constexpr int kPSet = (kCodes ? 1 : 2) * kPAtom;
  static constexpr int kP = kQ + kAtoms * kQAtom;
  static constexpr int kStat = kP + 2 * kAhead * kPSet;  // m[2][N], l[2][4][N], tops[2][4][N], factor[2][N], running m[2][N], f[2][N]
  static constexpr int kSeq = kStat + (2 + 8 + 8 + 2 + 2 + 2) * N * 4;
  static constexpr int kTiles = kSeq + kMaxSeqs * 16;
  static constexpr int kFirst = kTiles + kMaxSeqs * 4;
  static constexpr int kState = kFirst + (kMaxSeqs + 4) * 4;
  static constexpr int kBar = kState + 16 * 4;
  // full[2 S], empty[2 S], clean[2 S], q_full, q_empty, s_full[2][A], p_full[2][A], done[2][A],
  // o_full[2], l_full[2], o_free[2], drain[2]
  static constexpr int kNumBars = 6 * kStages + 2 + 6 * kAhead + 8;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kDirty = kAbort + 4;
  static constexpr int kAlloc = kDirty + 4 + 1024;       // slack for 1024-byte alignment
  static constexpr int kTmemCols = kCodes ? 512 : 128;   // of each group: S^T of the sets, O^T
  static_assert(kAlloc <= 232448, "shared memory budget");
  static_assert(2 * (kAhead + 1) * kCols <= kTmemCols, "TMEM");
  // Heads of 64 dimensions: the MMA's other 64 rows of V^T are what stands behind
  // the tile; their lanes are never read, but the ring must not end the memory.
  static_assert(kRing + 2 * kStages * kTile + kAtom <= kAlloc - 1024, "128 rows of the last stage");
};

// Warps: 0-7 softmax, 8-11 epilogue, 12 and 15 MMA issue, 13 and 16 copies of K and V,
// 14 clearing, 17 the queries' terms.
constexpr int kFewThreads = 18 * 32;

// Whether any of the 128 threads of a group says so (named barrier `id`).
__device__ __forceinline__ bool group_any(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)mine), "r"(id)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// The largest of a warp's values, NaN aside: by integers of the same order.
__device__ __forceinline__ float warp_max(float v) {
  if (!(v == v)) v = -INFINITY;
  int k = __float_as_int(v);
  k ^= (k >> 31) & 0x7FFFFFFF;
  k = __reduce_max_sync(0xFFFFFFFFu, k);
  return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
}

template <int DP, bool kF16, bool kCodes>
__global__ void __launch_bounds__(kFewThreads, 1)
    paged_few_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedArgs a) {
  using C = Few<DP, kCodes>;
  constexpr int R = C::kR, RK = C::kRK, RV = C::kRV, S = C::kStages, A = C::kAhead;
  constexpr uint32_t kFmt = kCodes || kF16 ? 0 : 1;  // E4M3 of its kind, binary16 of the other
  constexpr uint32_t kIdescS = make_idesc(kFmt, kFmt, kKeys, C::kCols);
  constexpr uint32_t kIdescO = make_idesc(kFmt, kFmt, 128, C::kCols) | (1u << 15);   // A is MN-major

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBar;
  auto bar = [&](int k) { return bar0 + 8u * (uint32_t)k; };
  auto full_bar = [&](int s) { return bar(s); };
  auto empty_bar = [&](int s) { return bar(2 * S + s); };
  auto clean_bar = [&](int s) { return bar(4 * S + s); };
  constexpr int kRest = 6 * S + 2;
  const uint32_t q_full = bar(6 * S), q_empty = bar(6 * S + 1);
  // of the group's tile t, by its set
  auto s_full = [&](int i, uint32_t t) { return bar(kRest + i * A + (int)(t % A)); };
  auto p_full = [&](int i, uint32_t t) { return bar(kRest + 2 * A + i * A + (int)(t % A)); };
  auto done_bar = [&](int i, uint32_t t) { return bar(kRest + 4 * A + i * A + (int)(t % A)); };
  const auto set_phase = [](uint32_t t) { return (t / A) & 1; };
  auto o_full = [&](int i) { return bar(kRest + 6 * A + i); };
  auto l_full = [&](int i) { return bar(kRest + 6 * A + 2 + i); };
  auto o_free = [&](int i) { return bar(kRest + 6 * A + 4 + i); };
  auto drain_bar = [&](int i) { return bar(kRest + 6 * A + 6 + i); };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kAbort);
  volatile int* dirty = reinterpret_cast<volatile int*>(smem + C::kDirty);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  float* stat_m = reinterpret_cast<float*>(smem + C::kStat);   // [2][N]
  float* stat_l = stat_m + 2 * N;                              // [2][4][N]: each softmax warp's sum
  float* tops = stat_l + 8 * N;                                // [2][4][N]
  float* factor = tops + 8 * N;                                // [2][N]: of codes, of even and odd items
  float* run_m = factor + 2 * N;                               // [2][N]: the groups' running maxima
  float* run_f = run_m + 2 * N;                                // [2][N]: what O^T and the sums are scaled by
  Seq* seqs = a.B <= kMaxSeqs ? reinterpret_cast<Seq*>(smem + C::kSeq) : nullptr;
  uint32_t* tiles = reinterpret_cast<uint32_t*>(smem + C::kTiles);
  int* state = reinterpret_cast<int*>(smem + C::kState);
  int* copied = state + 8;                                     // [2][2]: the next filling by K's and V's copies of each group; passes' Q

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 6 * S; ++s) mbar_init(bar(s), 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      for (uint32_t t = 0; t < A; ++t) {
        mbar_init(s_full(i, t), 1);
        mbar_init(p_full(i, t), 4);
        mbar_init(done_bar(i, t), 1);
      }
      mbar_init(o_full(i), 1);
      mbar_init(l_full(i), 4);
      mbar_init(o_free(i), 4);
      mbar_init(drain_bar(i), 1);
    }
    *abort = 0;
    *dirty = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == 12) {
    tmem_alloc(sbase + C::kTmemSlot, C::kTmemCols);
    tmem_relinquish();
  }
  // Rows without a query hold zeros (of codes their writer clears them): no copy writes them.
  const uint32_t q_bytes = (uint32_t)(a.G * a.rows_l * 128);
  if (!kCodes && q_bytes < (uint32_t)C::kQAtom) {
    for (uint32_t at = q_bytes + 16 * threadIdx.x; at < (uint32_t)C::kQAtom; at += 16 * kFewThreads)
#pragma unroll
      for (int k = 0; k < C::kAtoms; ++k)
        *reinterpret_cast<uint4*>(smem + C::kQ + k * C::kQAtom + at) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  griddep_wait();   // from here on what earlier kernels wrote may be read
  if (warp == 0 && seqs) share_out_whole(a, seqs, tiles, reinterpret_cast<uint32_t*>(smem + C::kFirst), state,
                                             kCodes ? kCutFewCodes : kCutFew);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();   // the next kernel may start its prologue
  const uint32_t tmem = *tmem_slot;
  const auto s_col = [&](int i, uint32_t t) { return tmem + (uint32_t)(i * (A + 1) * C::kCols) + (t % A) * C::kCols; };
  const auto o_col = [&](int i) { return tmem + (uint32_t)((i * (A + 1) + A) * C::kCols); };
  // The stage of a group's entry: of its one ring (K and V in turn), or of its ring of K or of V.
  const auto stage_of = [](bool is_v, int i, uint32_t e) {
    return kCodes ? (is_v ? 2 * RK + i * RV + (int)(e % (RV ? RV : 1)) : i * RK + (int)(e % (RK ? RK : 1))) : i * R + (int)(e % (R ? R : 1));
  };
  const auto stage_phase = [](bool is_v, uint32_t e) {
    constexpr uint32_t k = kCodes ? RK : R, v = kCodes ? RV : R;
    return (is_v ? e / v : e / k) & 1;
  };
  const auto group_tiles = [](int n, int i) { return (n + 1 - i) / 2; };

  // Each group has rings of its own: a waiter has to see every filling of its stages.
  //
  // The page of box `lane` of a tile as the table has it (checked when it is used:
  // the load is in flight until then), or one behind the last: a copy then writes zeros.
  const auto ask_page = [&](const Item& x, int tile) {
    const int key = tile * kKeys + lane * a.box;
    int page = a.pages;
    if (lane < a.boxes && key < x.limit) page = ld_i32(a.table + x.b * a.table_stride + quotient(key, a.by_page));
    return page;
  };

  if (warp == 13 || warp == 16) {
    // ---------------------------------------------------------------- copies of K (and Q), and of V
    const bool is_v = warp == 16;
    const CUtensorMap* map = is_v ? &maps.v : &maps.k;
    // entries of a group's ring; where K and V share it this warp's are every other one
    constexpr uint32_t step = kCodes ? 1 : 2;
    uint32_t entry[2] = {!kCodes && is_v ? 1u : 0u, !kCodes && is_v ? 1u : 0u}, qcount = 0;
    const uint32_t ring = sbase + C::kRing + lane * a.box * 128;
    bool ok = true;
    WholeUnits units(a, seqs, tiles, state);
    Item x;
    while (ok && units.next(x)) {
      if (x.n() == 0) continue;
      int page = ask_page(x, x.t0);
      if (!kCodes && !is_v) {
        ok = mbar_wait_lanes(q_empty, (qcount & 1) ^ 1, abort);
        if (!ok) break;
        ++qcount;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, C::kAtoms * q_bytes);
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_4d(sbase + C::kQ + at * C::kQAtom, &maps.q, q_full, 64 * at, 0, x.row0, x.hk);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int t = x.t0; t < x.t1; ++t) {
        const int next = ask_page(x, t + 1);     // a tile ahead
        const int i = (t - x.t0) & 1;
        const uint32_t e = i ? entry[1] : entry[0];
        const int st = stage_of(is_v, i, e);
        ok = mbar_wait_lanes(empty_bar(st), stage_phase(is_v, e) ^ 1, abort);
        if (!ok) break;
        if (i) entry[1] += step;
        else entry[0] += step;
        if (lane == 0) mbar_arrive_expect_tx(full_bar(st), C::kTile);
        __syncwarp();
        if (lane < a.boxes) {
          const int key = t * kKeys + lane * a.box, slot = key - quotient(key, a.by_page) * a.page_size;
          if (page < 0 || page > a.pages) page = a.pages;
          const uint32_t dst = ring + st * C::kTile;
          tma_load_4d(dst, map, full_bar(st), 0, x.hk, slot, page);
          if (C::kAtoms == 2) tma_load_4d(dst + kAtom, map, full_bar(st), 64, x.hk, slot, page);
        }
        __syncwarp();
        page = next;
      }
    }
    if (lane == 0) {
      copied[2 * is_v] = (int)entry[0];
      copied[2 * is_v + 1] = (int)entry[1];
      if (!is_v) copied[4] = (int)qcount;
      if (!ok) record_timeout(abort);
    }
  } else if (warp == 12 || warp == 15) {
    // ---------------------------------------------------------------- MMA issue, a thread for each group
    if (elect_one()) {
      const int i = warp == 12 ? 0 : 1;
      uint32_t tile = 0;                         // of the group's
      uint32_t qcount = 0, icount = 0;
      bool ok = true;
      const uint64_t qd = sw128_kmajor_desc(sbase + C::kQ);
      // Scores of the group's tile t.
      auto scores = [&](uint32_t t) {
        const uint32_t e = kCodes ? t : 2 * t;
        const int st = stage_of(false, i, e);
        // a ring of both goes by way of the clearing warp, which has to see every filling of it
        if (!mbar_wait_awake(kCodes ? full_bar(st) : clean_bar(st), stage_phase(false, e), abort)) return false;
        tc_fence_after();
        const uint64_t kd = sw128_kmajor_desc(sbase + C::kRing + st * C::kTile);
        if constexpr (kCodes) {
#pragma unroll
          for (int k = 0; k < DP / 32; ++k) mma_f8f6f4(s_col(i, t), kd + 2 * k, qd + 2 * k, kIdescS, k != 0);
        } else {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)      // descriptors count in 16 bytes
            mma_f16(s_col(i, t), kd + (((k >> 2) * kAtom + 32 * (k & 3)) >> 4), qd + (((k >> 2) * C::kQAtom + 32 * (k & 3)) >> 4),
                    kIdescS, k != 0);
        }
        mma_commit(s_full(i, t));
        mma_commit(empty_bar(st));
        return true;
      };
      WholeUnits units(a, seqs, tiles, state);
      Item x;
      while (ok && units.next(x)) {
        if (x.n() == 0) continue;
        const int n = group_tiles(x.n(), i);
        // also by a group without a tile: its word on Q below belongs to this Q
        ok = mbar_wait_awake(q_full, qcount++ & 1, abort);
        if (!ok) break;
        tc_fence_after();
        int started = 0;                         // tiles whose scores are under way
        for (int j = 0; ok && j < n; ++j, ++tile) {
          // The set of S^T that tile j + A's scores go to has been read: P of tile j was waited for.
          for (; ok && started < n && started < j + A; ++started) ok = scores(tile + (uint32_t)(started - j));
          if (!ok) break;
          if (started == n && j + A >= n && j == max(n - A, 0)) mma_commit(q_empty);
          const uint32_t e = kCodes ? tile : 2 * tile + 1;
          const int st = stage_of(true, i, e);
          ok = mbar_wait_awake(clean_bar(st), stage_phase(true, e), abort);
          if (j == 0) ok = ok && mbar_wait_awake(o_free(i), (icount++ & 1) ^ 1, abort);   // the epilogue has read O_i
          ok = ok && mbar_wait_awake(p_full(i, tile), set_phase(tile), abort);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sw128_mnmajor_desc(sbase + C::kRing + st * C::kTile);
          const uint64_t pd = sw128_kmajor_desc(sbase + C::kP + (i * A + (int)(tile % A)) * C::kPSet);
          if constexpr (kCodes) {
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k) mma_f8f6f4(o_col(i), vd + (4096 * k >> 4), pd + 2 * k, kIdescO, j != 0 || k != 0);
          } else {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_f16(o_col(i), vd + (2048 * k >> 4), pd + (((k >> 2) * C::kPAtom + 32 * (k & 3)) >> 4), kIdescO, j != 0 || k != 0);
          }
          mma_commit(empty_bar(st));
          if (A > 1) mma_commit(done_bar(i, tile));
          if (j + 1 == n) mma_commit(o_full(i));
        }
        if (n == 0) mma_commit(q_empty);         // no tile of its own
      }
      if (!ok) record_timeout(abort);
      // All MMAs complete before TMEM is freed.
      mma_commit(drain_bar(i));
      volatile int never = 0;
      if (!mbar_wait(drain_bar(i), 0, &never, kWaitLimitNs)) atomicOr(&g_paged_err, kErrTimeout);
    }
  } else if (warp == 14) {
    // ---------------------------------------------------------------- V rows that not all rows see
    uint32_t entry[2] = {0, 0};
    bool ok = true;
    WholeUnits units(a, seqs, tiles, state);
    Item x;
    while (ok && units.next(x)) {
      constexpr int kKinds = kCodes ? 1 : 2;     // entries of a ring for each tile: V, or K and V
#pragma unroll 1
      for (int k = 0; ok && k < kKinds * x.n(); ++k) {
        const int j = k / kKinds, i = j & 1;
        const uint32_t e = i ? entry[1]++ : entry[0]++;
        const int st = stage_of(true, i, e), key0 = (x.t0 + j) * kKeys;
        ok = mbar_wait_lanes(full_bar(st), stage_phase(true, e), abort);
        if (!ok) break;
        if ((kCodes || (k & 1)) && key0 + kKeys > x.lim0) {
          if (clear_rows<kF16, kCodes, C::kAtoms>(smem + C::kRing + st * C::kTile, lane, x.lim0 - key0, x.limit - key0, a.box)) *dirty = 1;
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(clean_bar(st));
      }
    }
    if (!ok && lane == 0) record_timeout(abort);
  } else if (warp == 17) {
    if constexpr (kCodes) {
      // ---------------------------------------------------------------- queries as E4M3 terms
      // Row r's terms are rows r, N + r and 2 N + r of the operand.  Four rows at a
      // time, eight lanes a row, sixteen dimensions a lane; rows without a query are
      // left as they are, four at a time.
      bool ok = true;
      uint32_t qcount = 0;
      const float scale = a.scale_log2 * ld_f32(a.k_scale);
      const int part = lane & 7;
      WholeUnits units(a, seqs, tiles, state);
      Item x;
      while (ok && units.next(x)) {
        if (x.n() == 0) continue;
        const int valid = x.left * a.G;
        uint4 w[2];
        auto load = [&](int r) {
          w[0] = w[1] = make_uint4(0, 0, 0, 0);
          if (r >= valid || 16 * part >= a.D) return;
          const int l = r / a.G, h = r - l * a.G;
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (int64_t)(x.row0 + l) * a.q_l +
                                                          (int64_t)(x.hk * a.G + h) * a.q_h + 16 * part);
          w[0] = q[0];
          w[1] = q[1];
        };
        load(lane >> 3);
        ok = mbar_wait_lanes(q_empty, (qcount & 1) ^ 1, abort);
        if (!ok) break;
#pragma unroll 1
        for (int r0 = 0; r0 < valid; r0 += 4) {
          const int r = r0 + (lane >> 3);
          const uint32_t words[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
          F2 v[8];
          float top = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[k] = unpack16<kF16>(words[k]);
            top = max_nan(top, max_nan(fabsf(v[k].x), fabsf(v[k].y)));
          }
          load(r + 4);
#pragma unroll
          for (int o = 4; o >= 1; o /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          // 2^-e takes the largest value to [128, 256) (less where it is below 2^-120); not finite: the row becomes NaN
          const uint32_t bits = __float_as_uint(top);
          const bool bad = bits >= 0x7F800000u;
          const int e = (int)(bits >> 23) - 127 - 7;
          const float down = bad ? 1.0f : pow2i(-e > 127 ? 127 : -e);
          uint32_t t[3][4] = {};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float x0 = v[k].x * down, x1 = v[k].y * down;
            if (bad) x0 = x1 = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int s = 0; s < 3; ++s) {
              const uint32_t c = cvt_e4m3x2(x0, x1);
              t[s][k >> 1] |= c << (16 * (k & 1));
              float y0, y1;
              f16x2_to_f32(cvt_e4m3x2_to_f16x2((uint16_t)c), y0, y1);
              x0 = (x0 - y0) * 16.0f;
              x1 = (x1 - y1) * 16.0f;
            }
          }
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            const int row = s * N + r;
            *reinterpret_cast<uint4*>(smem + C::kQ + row * 128 + ((part ^ (row & 7)) << 4)) = make_uint4(t[s][0], t[s][1], t[s][2], t[s][3]);
          }
          if (part == 0) factor[(qcount & 1) * N + r] = scale / down;
        }
        ++qcount;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      if (!ok && lane == 0) record_timeout(abort);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax: a thread a key
    const int i = warp >> 2;                     // group
    const int key_in = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const int id = 1 + i;                        // the group's barrier
    // What a new maximum leaves room for: with codes its weight is 2^7.  It grows to 2^8 either way.
    constexpr float kTop = kCodes ? 7.0f : 0.0f, kGrow = kLazyMax;
    // where this key's column of P stands, row 0 of set 0, before the swizzle
    uint8_t* p_at = smem + C::kP + i * A * C::kPSet + (kCodes ? key_in & 15 : (key_in >> 6) * C::kPAtom + (key_in & 7) * 2);
    const int p_chunk = kCodes ? key_in >> 4 : (key_in & 63) >> 3;
    uint32_t tile = 0, icount = 0, items = 0;
    // A warp whose wait gave up goes on to the group's next vote, so that no barrier
    // waits for it, and the group leaves together.
    bool ok = true, out = false;
    WholeUnits units(a, seqs, tiles, state);
    Item x;
    while (!out && units.next(x)) {
      if (x.n() == 0) continue;
      const float* row_factor = factor + (items++ & 1) * N;
      const int n = group_tiles(x.n(), i);
      if (n == 0) continue;
      // Rows that have a query, four at a time: the others' scores, weights and sums are
      // left out, and what stands in their columns reaches no row's result.
      const int valid = x.left * a.G;
      float l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.0f;
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++tile) {
        const int key0 = (x.t0 + 2 * j + i) * kKeys;
        ok = ok && mbar_wait_lanes(s_full(i, tile), set_phase(tile), abort);
        float s[N];                              // scaled scores, in powers of two
        bool grow = !ok || j == 0;
        if (ok) {
          tc_fence_after();
          // A position that a row does not see has the weight exp2(-inf) = 0.
          const int key = key0 + key_in;
          const bool edge = key0 + kKeys > x.lim0, there = !edge || key < x.len;
          const int ahead = edge && a.causal ? key - x.pos0 : 0;   // rows of tokens before that do not see it
          int token = 0, head = 0;
#pragma unroll
          for (int r0 = 0; r0 < N; r0 += 4) {
            if (r0 >= valid) break;
            uint32_t t[4];
            tmem_ld_32x32b_x4(s_col(i, tile) + quad + (kCodes ? 2 * N : 0) + r0, t);
            if constexpr (kCodes) {              // t0 + (t1 + t2 / 16) / 16
              uint32_t t1[4], t0[4];
              tmem_ld_32x32b_x4(s_col(i, tile) + quad + N + r0, t1);
              tmem_ld_32x32b_x4(s_col(i, tile) + quad + r0, t0);
              tmem_ld_wait();
              const float4 f = *reinterpret_cast<const float4*>(row_factor + r0);
              const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s[r0 + e] = fmaf(fmaf(__uint_as_float(t[e]), 0.0625f, __uint_as_float(t1[e])), 0.0625f, __uint_as_float(t0[e])) * ff[e];
            } else {
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 4; ++e) s[r0 + e] = __uint_as_float(t[e]) * a.scale_log2;
            }
            const float4 m4 = *reinterpret_cast<const float4*>(run_m + i * N + r0);
            const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (edge) {
                if (!there || token < ahead) s[r0 + e] = -INFINITY;
                if (++head == a.G) head = 0, ++token;
              }
              // a row without a query has no say: what it holds must not decide on roundings
              grow |= r0 + e < valid && (s[r0 + e] > mm[e] + kGrow || (mm[e] == -INFINITY && s[r0 + e] > -INFINITY));
            }
          }
        }
        // P's set has been read by the product of A tiles before (with one set that is complete
        // as the scores are, which were started behind it).
        if (A > 1 && tile >= A) ok = ok && mbar_wait_lanes(done_bar(i, tile), set_phase(tile - A), abort);
        grow |= !ok;
        __syncwarp();
        if (group_any(id, grow)) {
          if (group_any(id, !ok)) {
            out = true;
            break;
          }
          float top = -INFINITY;                 // lane r: row r's in this warp
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r >= valid) break;
            const float t = warp_max(s[r]);
            if (lane == r) top = t;
          }
          if (lane < N) tops[(i * 4 + (warp & 3)) * N + lane] = top;
          group_sync(id);
          if ((warp & 3) == 0 && lane < N) {
            const float* t = tops + i * 4 * N + lane;
            const float m = j > 0 ? run_m[i * N + lane] : -INFINITY;
            const float m_new = fmaxf(m, fmaxf(fmaxf(t[0], t[N]), fmaxf(t[2 * N], t[3 * N])) - kTop);
            run_m[i * N + lane] = m_new;
            run_f[i * N + lane] = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
          }
          group_sync(id);
          // O_i may be rescaled when the group's product with the previous tile is complete
          // (with one set it is as the scores are, which were started behind it).
          if (j > 0) {
            if (A > 1) ok = mbar_wait_lanes(done_bar(i, tile - 1), set_phase(tile - 1), abort);
            tc_fence_after();
#pragma unroll
            for (int r0 = 0; r0 < N; r0 += 4) {
              if (r0 >= valid) break;
              const float4 f4 = *reinterpret_cast<const float4*>(run_f + i * N + r0);
              const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) l[r0 + e] *= f[e];
#pragma unroll
              for (int c = 0; c < C::kCols; c += N) {
                uint32_t o[4];
                tmem_ld_32x32b_x4(o_col(i) + quad + c + r0, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
                tmem_st_32x32b_x4(o_col(i) + quad + c + r0, o);
              }
            }
            tmem_st_wait();
          }
        }
        uint8_t* p_set = p_at + (int)(tile % A) * C::kPSet;
#pragma unroll
        for (int r0 = 0; r0 < N; r0 += 4) {
          if (r0 >= valid) break;
          const float4 m4 = *reinterpret_cast<const float4*>(run_m + i * N + r0);
          const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(s[r0 + e] - (mm[e] == -INFINITY ? 0.0f : mm[e]));
            l[r0 + e] += p[e];
          }
          if constexpr (kCodes) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {   // two rows' terms and what they leave
                const int row = k * N + r0 + e;
                const uint32_t c = cvt_e4m3x2(p[e], p[e + 1]);
                p_set[row * 128 + ((p_chunk ^ (row & 7)) << 4)] = (uint8_t)c;
                p_set[(row + 1) * 128 + ((p_chunk ^ ((row + 1) & 7)) << 4)] = (uint8_t)(c >> 8);
                float y0, y1;
                f16x2_to_f32(cvt_e4m3x2_to_f16x2((uint16_t)c), y0, y1);
                p[e] = (p[e] - y0) * 16.0f;
                p[e + 1] = (p[e + 1] - y1) * 16.0f;
              }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = r0 + e;
              *reinterpret_cast<uint16_t*>(p_set + row * 128 + ((p_chunk ^ (row & 7)) << 4)) = (uint16_t)cvt16x2(kF16, p[e], 0.0f);
            }
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i, tile));
      }
      if (out) break;
      float mine = 0.0f;                         // lane r: row r's
#pragma unroll
      for (int r = 0; r < N; ++r) {
        if (r >= valid) break;
        float t = l[r];
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        if (lane == r) mine = t;
      }
      // the epilogue has read the previous item's sums
      ok = ok && mbar_wait_lanes(o_free(i), (icount & 1) ^ 1, abort);
      ++icount;
      if (!ok) continue;
      if (lane < N) {
        stat_l[(i * 4 + (warp & 3)) * N + lane] = mine;
        if ((warp & 3) == 0) stat_m[i * N + lane] = run_m[i * N + lane];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(l_full(i));
    }
    if (!ok && lane == 0) record_timeout(abort);
  } else {
    // ---------------------------------------------------------------- epilogue
    const int d = (warp & 3) * 32 + lane;        // this thread's dimension
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    float inv_s = 1.0f, v_scale = 1.0f;
    if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
    if constexpr (kCodes) v_scale = ld_f32(a.v_scale);
    uint32_t icount[2] = {0, 0};
    bool ok = true;

    auto put = [&](int64_t at, float y) {
      if (a.s_out) static_cast<uint8_t*>(a.out)[at] = (uint8_t)cvt_e4m3x2(y * inv_s, 0.0f);
      else static_cast<uint16_t*>(a.out)[at] = (uint16_t)cvt16x2(kF16, y, 0.0f);
    };
    auto put_zeros = [&](const Item& x) {
      if (d >= a.D) return;
      for (int t = 0; t < x.left; ++t)
        for (int h = 0; h < a.G; ++h) put((int64_t)(x.row0 + t) * a.o_l + (int64_t)(x.hk * a.G + h) * a.o_h + d, 0.0f);
    };
    // Rows that see a position, which not every row of the unit sees, where dimension d is +inf,
    // and where it is -inf; NaN counts as both (it was cleared).  Seldom called, and slow.
    auto spoilt_rows = [&](const Item& x, uint32_t (&rows)[2]) {
      if (d >= a.D) return;
      const int end = min(x.limit, x.t1 * kKeys);
      for (int j = max(x.lim0, x.t0 * kKeys); j < end; ++j) {
        const int at = quotient(j, a.by_page), page = ld_i32(a.table + x.b * a.table_stride + at);
        if (page < 0 || page >= a.pages) continue;
        const uint8_t* v = a.v + page * a.vs[0] + (j - at * a.page_size) * a.vs[1] + x.hk * a.vs[2];
        bool plus, minus;
        if (kCodes) {
          plus = minus = (v[d] & 0x7F) == 0x7F;
        } else {
          const uint32_t w = reinterpret_cast<const uint16_t*>(v)[d], inf = kF16 ? 0x7C00u : 0x7F80u;
          if ((w & inf) != inf) continue;
          plus = w != (inf | 0x8000u);
          minus = w != inf;
        }
        for (int r = 0; r < x.left * a.G; ++r)
          if (j < seen(a, x.pos0, x.len, r / a.G + 1)) rows[0] |= (uint32_t)plus << r, rows[1] |= (uint32_t)minus << r;
      }
    };
    if (a.may_cut && state[kShares] > 0 && state[kZeros]) {   // units without a tile: their rows are zeros
      for (int it = blockIdx.x; it < a.B * a.Hkv; it += gridDim.x) {
        Item x;
        x.b = it / a.Hkv;
        x.hk = it - x.b * a.Hkv;
        const Seq s = seqs[x.b];
        if (seen(a, s.base, s.len, s.tokens) > 0) continue;
        x.row0 = s.row0;
        x.left = s.tokens;
        put_zeros(x);
      }
    }
    WholeUnits units(a, seqs, tiles, state);
    Item x;
    while (ok && units.next(x)) {
      if (x.n() == 0) {
        put_zeros(x);
        continue;
      }
      const bool two = x.n() > 1;
      for (int i = 0; i < (two ? 2 : 1) && ok; ++i) {
        if (!mbar_wait_lanes(l_full(i), icount[i] & 1, abort) ||
            !mbar_wait_lanes(o_full(i), icount[i] & 1, abort))
          ok = false;
        ++icount[i];
      }
      if (!ok) break;
      tc_fence_after();
      // Lane r: o = (a0 O0 + a1 O1) / (a0 l0 + a1 l1) of row r, a_i = 2^(m_i - max m).
      // A group whose scores are all -inf has the sum 0, or NaN where one is NaN, which stays.
      float a0 = 0.0f, a1 = 0.0f;
      {
        const int r = lane < N ? lane : 0;
        const float m0 = stat_m[r], m1 = two ? stat_m[N + r] : -INFINITY;
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l0 += stat_l[k * N + r];
          if (two) l1 += stat_l[(4 + k) * N + r];
        }
        const float top = fmaxf(m0, m1);
        a0 = m0 == -INFINITY ? (l0 == 0.0f ? 0.0f : 1.0f) : ex2(m0 - top);
        a1 = m1 == -INFINITY ? (l1 == 0.0f ? 0.0f : 1.0f) : ex2(m1 - top);
        const float sum = a0 * l0 + a1 * l1;
        if (x.part >= 0 && warp == 8 && lane < N)
          a.part_lse[(int64_t)x.part * N + r] = sum == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top) + log2f(sum);
        const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum) * v_scale;
        a0 *= f;
        a1 *= f;
      }
      uint32_t inf_rows[2] = {0, 0};
      if (*dirty) spoilt_rows(x, inf_rows);
      __syncwarp();   // together again for the TMEM loads
      const int valid = x.left * a.G;
      int64_t at = (int64_t)x.row0 * a.o_l + (int64_t)x.hk * a.G * a.o_h + d;
      int head = 0;
#pragma unroll 1
      for (int r0 = 0; r0 < valid; r0 += 4) {
        float o[2][4];                           // of codes the three terms' sum
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !two) break;
          uint32_t t[3][4];
#pragma unroll
          for (int c = 0; c < C::kCols / N; ++c) tmem_ld_32x32b_x4(o_col(i) + quad + c * N + r0, t[c]);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[i][e] = __uint_as_float(t[0][e]);
            if (kCodes) o[i][e] = fmaf(fmaf(__uint_as_float(t[2][e]), 0.0625f, __uint_as_float(t[1][e])), 0.0625f, o[i][e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + e;
          const float f0 = __shfl_sync(0xFFFFFFFFu, a0, r & 31), f1 = __shfl_sync(0xFFFFFFFFu, a1, r & 31);
          float y = o[0][e] * f0;
          if (two) y = fmaf(o[1][e], f1, y);
          if (inf_rows[0] >> r & 1) y += INFINITY;
          if (inf_rows[1] >> r & 1) y -= INFINITY;
          if (r < valid && d < a.D) {
            if (x.part >= 0) a.part[((int64_t)x.part * N + r) * DP + d] = y;
            else put(at, y);
          }
          at += a.o_h;
          if (++head == a.G) head = 0, at += a.o_l - a.G * a.o_h;
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free(0));
        if (two) mbar_arrive(o_free(1));
      }
    }
    if (!ok && lane == 0) record_timeout(abort);
  }

  tc_fence_before();
  __syncthreads();
  // Every copy has landed before the block ends: each was waited for by those that read
  // it, unless they gave up, and then here.
  if (*abort && threadIdx.x == 0) {
    volatile int never = 0;
    auto landed = [&](uint32_t b, uint32_t parity) {
      if (!mbar_wait(b, parity, &never, kWaitLimitNs)) atomicOr(&g_paged_err, kErrTimeout);
    };
    for (int v = 0; v < 2; ++v)
      for (int i = 0; i < 2; ++i) {
        const int ring = !kCodes ? R : v ? RV : RK;
        for (int j = 1; j <= ring; ++j) {
          const int e = unread_filling(copied[2 * v + i], copied[2 * (1 - v) + i], kCodes ? 1 : 2, ring, j);
          if (e >= 0) landed(full_bar(stage_of(v, i, (uint32_t)e)), stage_phase(v, (uint32_t)e));
        }
      }
    if (!kCodes && copied[4] > 0) landed(q_full, (uint32_t)(copied[4] - 1) & 1);
  }
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joining cut units: as paged_join_kernel, with rows of DP floats; a thread
// takes four columns of a row.
template <int DP, bool kF16>
__global__ void __launch_bounds__(256) few_join_kernel(const PagedArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kBlocks = N * DP / 4 / 256;     // of a cut
  const int c = 1 + (int)blockIdx.x / kBlocks;
  const int4 lo = *reinterpret_cast<const int4*>(a.info + c * kInfo), hi = *reinterpret_cast<const int4*>(a.info + c * kInfo + 4);
  const int shares = lo.x, hk = lo.w, row0 = hi.x, left = hi.y;
  if (c >= shares) return;
  const uint32_t tile = (uint32_t)lo.y, tiles = (uint32_t)lo.z, total = (uint32_t)hi.z;
  auto start = [&](int k) { return share_begin(total, (uint32_t)k, (uint32_t)shares); };
  const uint32_t s0 = start(c) - tile, s1 = s0 + tiles;
  if (tile == 0 || start(c - 1) > s0) return;   // not inside a unit, or not its first cut
  const int at = ((int)blockIdx.x % kBlocks) * 256 + (int)threadIdx.x;
  const int r = at / (DP / 4), d = 4 * (at % (DP / 4));
  if (r >= left * a.G || d >= a.D) return;
  float inv_s = 1.0f;
  if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
  const int k0 = c - 1, k1 = (int)min((uint64_t)shares, ((uint64_t)s1 * shares + total - 1) / total);
  const int first = 2 * k0 + (start(k0) < s0 ? 1 : 0);
  auto row = [&](int k) { return (int64_t)(k == k0 ? first : 2 * k) * N + r; };
  float top = -INFINITY;
#pragma unroll 8
  for (int k = k0; k < k1; ++k) top = fmaxf(top, a.part_lse[row(k)]);
  if (top == -INFINITY) top = 0.0f;
  float sum = 0.0f, acc[4] = {};
#pragma unroll 8
  for (int k = k0; k < k1; ++k) {
    const float lse = a.part_lse[row(k)], weight = exp2f(lse - top);
    float4 v = *reinterpret_cast<const float4*>(a.part + row(k) * DP + d);
    if (lse == -INFINITY) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // nothing seen
    sum += weight;
    acc[0] = fmaf(weight, v.x, acc[0]);
    acc[1] = fmaf(weight, v.y, acc[1]);
    acc[2] = fmaf(weight, v.z, acc[2]);
    acc[3] = fmaf(weight, v.w, acc[3]);
  }
  const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
  const int l = r / a.G;
  const int64_t off = (int64_t)(row0 + l) * a.o_l + (int64_t)(hk * a.G + r - l * a.G) * a.o_h + d;
  if (a.s_out) {
    const float g = f * inv_s;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + off) =
        cvt_e4m3x2(acc[0] * g, acc[1] * g) | (cvt_e4m3x2(acc[2] * g, acc[3] * g) << 16);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + off) =
        make_uint2(cvt16x2(kF16, acc[0] * f, acc[1] * f), cvt16x2(kF16, acc[2] * f, acc[3] * f));
  }
}

template <int DP, bool kF16, bool kCodes>
cudaError_t launch_kernel(const PagedMaps& maps, const PagedArgs& a, int grid, cudaStream_t st) {
  using C = Few<DP, kCodes>;
  auto* k = paged_few_kernel<DP, kF16, kCodes>;
  static std::atomic<uint64_t> allowed{0};   // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kFewThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k, maps, a)) != cudaSuccess) return e;
  if (a.may_cut && grid > 1) {
    cfg.gridDim = dim3((unsigned)((grid - 1) * (N * DP / 4 / 256)), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, few_join_kernel<DP, kF16>, a)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DP>
cudaError_t launch_dims(const PagedMaps& maps, const PagedArgs& a, bool f16, bool codes, int grid, cudaStream_t st) {
  if (codes) return f16 ? launch_kernel<DP, true, true>(maps, a, grid, st) : launch_kernel<DP, false, true>(maps, a, grid, st);
  return f16 ? launch_kernel<DP, true, false>(maps, a, grid, st) : launch_kernel<DP, false, false>(maps, a, grid, st);
}

}  // namespace

cudaError_t launch_paged_few(const PagedMaps& maps, const PagedArgs& a, int DP, bool f16, bool codes, int grid, cudaStream_t st) {
  return DP == 64 ? launch_dims<64>(maps, a, f16, codes, grid, st) : launch_dims<128>(maps, a, f16, codes, grid, st);
}

cudaError_t paged_few_read_error(cudaStream_t st, uint32_t* err) { return read_paged_error(st, err); }

}  // namespace w8
