// Attention over a paged cache for units of at most N = 16 or 32 query rows (the
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
// E4M3 cells.  K goes to the tensor core as it is: the queries are split into
// three E4M3 terms, q = (t0 + t1 / 16 + t2 / 256) 2^e with 2^e from the row's
// largest value, which leaves less than 2^-12 of each value (nothing of a bf16
// one) or 2^-27 of the largest; the terms are 3 N rows, and the softmax threads add
// their scores.  V has to be beside 16-bit weights: four warps write its codes
// to the operands' ring as binary16 (exact), and P is binary16 too.
//
// Bound by the bytes of K and V.  Roundings below 32 bits: P (its sum l is taken
// before) and the output.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attention_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {
namespace {

template <int DP, bool kCodes, int N>
struct Few {
  static constexpr int kAtoms = DP / 64;
  static constexpr int kTile = kAtoms * kAtom;           // bytes of 128 rows of K or V in 16 bits
  static constexpr int kRawTile = kKeys * DP;            // of V's codes
  // Stages of a group's ring: of K and V in turn (16 bits), or of V and of K's codes.
  static constexpr int kR = kCodes ? (DP == 128 ? 1 : 2) : (DP == 128 ? 3 : 5);
  static constexpr int kRK = kCodes ? 2 : 0;
  static constexpr int kRaws = !kCodes ? 0 : DP == 64 ? 3 : N == 16 ? 2 : 1;   // and of V's codes, of a group
  static constexpr int kRing = 0;
  static constexpr int kKRing = kRing + 2 * kR * kTile;  // rows of 128 bytes
  static constexpr int kRaw = kKRing + 2 * kRK * kAtom;
  static constexpr int kQRows = kCodes ? 3 * N : N;
  static constexpr int kQAtom = kQRows * 128;
  static constexpr int kQ = kRaw + 2 * kRaws * kRawTile;
  static constexpr int kP = kQ + (kCodes ? 1 : kAtoms) * kQAtom;     // of each group 2 x N x 128 bytes
  static constexpr int kStat = kP + 2 * 2 * N * 128;     // m[2][N], l[2][4][N], tops[2][4][N], factor[2][N], running m[2][N], f[2][N]
  static constexpr int kSeq = kStat + (2 + 8 + 8 + 2 + 2 + 2) * N * 4;
  static constexpr int kTiles = kSeq + kMaxSeqs * 16;
  static constexpr int kFirst = kTiles + kMaxSeqs * 4;
  static constexpr int kState = kFirst + (kMaxSeqs + 4) * 4;
  static constexpr int kBar = kState + 16 * 4;
  // full[2R], empty[2R], clean[2R], k_full[2RK], k_empty[2RK], raw_full[2RW], raw_empty[2RW], q_full, q_empty,
  // s_full[2], p_full[2], o_full[2], l_full[2], o_free[2], drain[2]
  static constexpr int kNumBars = 6 * kR + 4 * kRK + 4 * kRaws + 14;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kDirty = kAbort + 4;
  static constexpr int kAlloc = kDirty + 4 + 1024;       // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448, "shared memory budget");
  // Heads of 64 dimensions: the MMA's other 64 rows of V^T are what stands behind
  // the tile; their lanes are never read, but the ring must not end the memory.
  static_assert(kRing + 2 * kR * kTile + kAtom <= kAlloc - 1024, "128 rows of the last stage");
};

// Warps: 0-7 softmax, 8-11 epilogue and conversion of the first group's V, 12 and 15 MMA
// issue, 13 and 16 copies of K and V, 14 clearing, or the queries' terms and with 17-19 the
// conversion of the second group's V.
template <bool kCodes>
constexpr int kFewThreads = (kCodes ? 20 : 17) * 32;

constexpr uint32_t kFewTmem = 256;   // columns: S^T of the groups from 0 and 96, O^T from 192 and 224

// mbar_wait that asks some times before it lets the thread sleep: a sleeping
// thread is woken late, and every hand-over between roles is on a tile's way.
__device__ __forceinline__ bool mbar_wait_awake(uint32_t bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int k = 0; k < 256; ++k)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, kWaitLimitNs);
}

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

// The sequences to shared memory and, where units may be cut, how the work is
// shared out (see share_out): by one warp, since a sequence is one unit of a key head.
__device__ __forceinline__ void share_out_few(const PagedArgs& a, Seq* seqs, uint32_t* tiles, uint32_t* first, int* state) {
  const int lane = threadIdx.x & 31;
  uint32_t total = 0, units = 0, longest = 0, zeros = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    uint32_t mine = 0;
    if (b < a.B) {
      const Seq s = load_seq(a, b);
      seqs[b] = s;
      if (s.tokens > 0) {
        mine = (uint32_t)(seen(a, s.base, s.len, s.tokens) + kKeys - 1) / kKeys;
        ++units;
        zeros |= mine == 0;
      }
      tiles[b] = mine;
    }
    if (!a.may_cut) continue;
    longest = max(longest, mine);
    mine *= (uint32_t)a.Hkv;
    uint32_t to = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
      if (lane >= o) to += v;
    }
    if (b < a.B) first[b] = total + to - mine;
    total += __shfl_sync(0xFFFFFFFFu, to, 31);
  }
  if (!a.may_cut) return;
  __syncwarp();
  units = __reduce_add_sync(0xFFFFFFFFu, units) * (uint32_t)a.Hkv;
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  zeros = __reduce_or_sync(0xFFFFFFFFu, zeros);
  const uint32_t ctas = gridDim.x;
  const uint32_t share = max((total + ctas - 1) / ctas, (uint32_t)kCutFew.least);
  const float even = (float)total / (float)ctas;
  const float whole = units <= ctas ? (float)longest : fmaxf((float)longest, even + 0.5f * (float)longest);
  const bool cut = kCutFew.slope * (float)share + kCutFew.plus < whole;
  const uint32_t shares = cut ? (total + share - 1) / share : 0;
  if (lane == 0) {
    a.info[blockIdx.x * kInfo] = (int)shares;
    state[kShares] = (int)shares;
    state[kZeros] = (int)zeros;
  }
  if (blockIdx.x >= shares) {
    if (lane == 0) state[kBegin] = state[kEnd] = (int)total;
    return;
  }
  const uint32_t p = share_begin(total, blockIdx.x, shares);
  int n = 0;                                 // sequences that begin at tile p or before it, the first aside
  for (int k = lane + 1; k < a.B; k += 32) n += first[k] <= p;
  const int b = __reduce_add_sync(0xFFFFFFFFu, n);
  if (lane != 0) return;
  const Seq s = seqs[b];
  const uint32_t at = p - first[b], hk = at / tiles[b], t = at - hk * tiles[b];
  state[kBegin] = (int)p;
  state[kEnd] = (int)share_begin(total, blockIdx.x + 1, shares);
  state[kAtB] = b;
  state[kAtHk] = (int)hk;
  state[kAtBlk] = 0;
  state[kAtTile] = (int)t;
  int* info = a.info + blockIdx.x * kInfo;
  info[1] = (int)t;
  info[2] = (int)tiles[b];
  info[3] = (int)hk;
  info[4] = s.row0;
  info[5] = s.tokens;
  info[6] = (int)total;
}

template <int DP, bool kF16, bool kCodes, int N>
__global__ void __launch_bounds__(kFewThreads<kCodes>, 1)
    paged_few_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedArgs a) {
  using C = Few<DP, kCodes, N>;
  constexpr int R = C::kR, RK = C::kRK, RW = C::kRaws;
  constexpr bool kP16 = kF16 || kCodes;            // P and V are binary16
  constexpr uint32_t kIdescS = kCodes ? make_idesc(0, 0, kKeys, 3 * N) : make_idesc(kF16 ? 0 : 1, kF16 ? 0 : 1, kKeys, N);
  constexpr uint32_t kIdescO = make_idesc(kP16 ? 0 : 1, kP16 ? 0 : 1, 128, N) | (1u << 15);   // A is MN-major

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBar;
  auto bar = [&](int k) { return bar0 + 8u * (uint32_t)k; };
  auto full_bar = [&](int s) { return bar(s); };
  auto empty_bar = [&](int s) { return bar(2 * R + s); };
  auto clean_bar = [&](int s) { return bar(4 * R + s); };
  auto k_full = [&](int s) { return bar(6 * R + s); };
  auto k_empty = [&](int s) { return bar(6 * R + 2 * RK + s); };
  auto raw_full = [&](int r) { return bar(6 * R + 4 * RK + r); };
  auto raw_empty = [&](int r) { return bar(6 * R + 4 * RK + 2 * RW + r); };
  constexpr int kRest = 6 * R + 4 * RK + 4 * RW;
  const uint32_t q_full = bar(kRest), q_empty = bar(kRest + 1);
  auto s_full = [&](int i) { return bar(kRest + 2 + i); };
  auto p_full = [&](int i) { return bar(kRest + 4 + i); };
  auto o_full = [&](int i) { return bar(kRest + 6 + i); };
  auto l_full = [&](int i) { return bar(kRest + 8 + i); };
  auto o_free = [&](int i) { return bar(kRest + 10 + i); };
  auto drain_bar = [&](int i) { return bar(kRest + 12 + i); };
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

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * R; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(clean_bar(s), kCodes ? 4 : 1);
    }
    for (int s = 0; s < 2 * RK; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int r = 0; r < 2 * RW; ++r) {
      mbar_init(raw_full(r), 1);
      mbar_init(raw_empty(r), 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 4);
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
    tmem_alloc(sbase + C::kTmemSlot, kFewTmem);
    tmem_relinquish();
  }
  // Rows without a query hold zeros (of codes their writer clears them): no copy writes them.
  const uint32_t q_bytes = (uint32_t)(a.G * a.rows_l * 128);
  if (!kCodes && q_bytes < (uint32_t)C::kQAtom) {
    for (uint32_t at = q_bytes + 16 * threadIdx.x; at < (uint32_t)C::kQAtom; at += 16 * kFewThreads<kCodes>)
#pragma unroll
      for (int k = 0; k < C::kAtoms; ++k)
        *reinterpret_cast<uint4*>(smem + C::kQ + k * C::kQAtom + at) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  griddep_wait();   // from here on what earlier kernels wrote may be read
  if (warp == 0 && seqs) share_out_few(a, seqs, tiles, reinterpret_cast<uint32_t*>(smem + C::kFirst), state);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const auto s_col = [&](int i) { return tmem + (uint32_t)(96 * i); };
  const auto o_col = [&](int i) { return tmem + 192u + (uint32_t)(32 * i); };
  const auto group_tiles = [](int n, int i) { return (n + 1 - i) / 2; };

  // Each group has rings of its own, of its K and V tiles in turn: a waiter has
  // to see every filling of its stages.
  //
  // The page of box `lane` of a tile as the table has it (checked when it is used:
  // the load is in flight until then), or one behind the last: a copy then writes zeros.
  const auto ask_page = [&](const Item& x, int tile) {
    const int key = tile * kKeys + lane * a.box;
    int page = a.pages;
    if (lane < a.boxes && key < x.limit) page = ld_i32(a.table + x.b * a.table_stride + quotient(key, a.by_page));
    return page;
  };

  // A quarter of a tile of V's codes of group i from its raw ring to the operands' ring, as
  // binary16 in the 128-byte swizzle; `count` is of the group's tiles.
  auto convert = [&](const Item& x, int i, int tile, int quarter, uint32_t count) {
    constexpr int kW = RW ? RW : 1;
    const int rs = i * kW + (int)(count % kW), st = i * R + (int)(count % R);
    if (!mbar_wait_lanes(raw_full(rs), (count / kW) & 1, abort) ||
        !mbar_wait_lanes(empty_bar(st), ((count / R) & 1) ^ 1, abort))
      return false;
    const int key0 = tile * kKeys;
    if (convert_rows<DP, true>(smem + C::kRaw + rs * C::kRawTile, smem + C::kRing + st * C::kTile, quarter, lane,
                               key0 + kKeys > x.lim0 ? x.lim0 - key0 : kKeys, x.limit - key0))
      *dirty = 1;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(clean_bar(st));
      mbar_arrive(raw_empty(rs));
    }
    return true;
  };

  if (warp == 13 || warp == 16) {
    // ---------------------------------------------------------------- copies of K (and Q), and of V
    const bool is_v = warp == 16;
    const CUtensorMap* map = is_v ? &maps.v : &maps.k;
    // The ring that a group's copies go to: of S stages of `stage` bytes, this warp's
    // entries `step` apart (16 bits: K and V in turn).
    constexpr int kStages = kCodes ? 0 : R;
    const int S = kCodes ? (is_v ? RW : RK) : kStages, step = kCodes ? 1 : 2;
    uint32_t entry[2] = {!kCodes && is_v ? 1u : 0u, !kCodes && is_v ? 1u : 0u}, qcount = 0;
    const auto stage_of = [&](int i, uint32_t e) { return i * S + (int)(e % (uint32_t)S); };
    const auto full_of = [&](int st) { return kCodes ? (is_v ? raw_full(st) : k_full(st)) : full_bar(st); };
    const auto empty_of = [&](int st) { return kCodes ? (is_v ? raw_empty(st) : k_empty(st)) : empty_bar(st); };
    const uint32_t stage_bytes = kCodes ? (is_v ? C::kRawTile : kAtom) : C::kTile, row_bytes = kCodes && is_v ? DP : 128;
    const uint32_t ring = sbase + (kCodes ? (is_v ? C::kRaw : C::kKRing) : C::kRing) + lane * a.box * row_bytes;
    bool ok = true;
    Units units(a, seqs, tiles, state);
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
        const int st = stage_of(i, e);
        ok = mbar_wait_lanes(empty_of(st), ((e / (uint32_t)S) & 1) ^ 1, abort);
        if (!ok) break;
        if (i) entry[1] += step;
        else entry[0] += step;
        if (lane == 0) mbar_arrive_expect_tx(full_of(st), stage_bytes);
        __syncwarp();
        if (lane < a.boxes) {
          const int key = t * kKeys + lane * a.box, slot = key - quotient(key, a.by_page) * a.page_size;
          if (page < 0 || page > a.pages) page = a.pages;
          const uint32_t dst = ring + st * stage_bytes;
          tma_load_4d(dst, map, full_of(st), 0, x.hk, slot, page);
          if (!kCodes && C::kAtoms == 2) tma_load_4d(dst + kAtom, map, full_of(st), 64, x.hk, slot, page);
        }
        __syncwarp();
        page = next;
      }
    }
    if (!ok && lane == 0) record_timeout(abort);
  } else if (warp == 12 || warp == 15) {
    // ---------------------------------------------------------------- MMA issue, a thread for each group
    if (elect_one()) {
      const int i = warp == 12 ? 0 : 1;
      uint32_t entry = 0, k_entry = 0;           // of this group's rings
      uint32_t qcount = 0, pcount = 0, icount = 0;
      bool ok = true;
      Units units(a, seqs, tiles, state);
      Item x;
      while (ok && units.next(x)) {
        const int n = x.n();
        if (n == 0) continue;
        // also by a group without a tile: its word on Q below belongs to this Q
        ok = mbar_wait_awake(q_full, qcount & 1, abort);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = sw128_kmajor_desc(sbase + C::kQ);
        for (int j = i; ok && j < n; j += 2) {
          const bool first = j == i, last = j + 2 >= n;
          if constexpr (kCodes) {
            const int st = i * RK + (int)(k_entry % RK);
            ok = mbar_wait_awake(k_full(st), (k_entry / RK) & 1, abort);
            if (!ok) break;
            ++k_entry;
            tc_fence_after();
            const uint64_t kd = sw128_kmajor_desc(sbase + C::kKRing + st * kAtom);
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) mma_f8f6f4(s_col(i), kd + 2 * k, qd + 2 * k, kIdescS, k != 0);
            mma_commit(s_full(i));
            mma_commit(k_empty(st));
          } else {
            const int st = i * R + (int)(entry % R);
            ok = mbar_wait_awake(clean_bar(st), (entry / R) & 1, abort);
            if (!ok) break;
            ++entry;
            tc_fence_after();
            const uint64_t kd = sw128_kmajor_desc(sbase + C::kRing + st * C::kTile);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)     // descriptors count in 16 bytes
              mma_f16(s_col(i), kd + (((k >> 2) * kAtom + 32 * (k & 3)) >> 4), qd + (((k >> 2) * C::kQAtom + 32 * (k & 3)) >> 4),
                      kIdescS, k != 0);
            mma_commit(s_full(i));
            mma_commit(empty_bar(st));
          }
          if (last) mma_commit(q_empty);

          const int st = i * R + (int)(entry % R);
          ok = mbar_wait_awake(clean_bar(st), (entry / R) & 1, abort);
          if (!ok) break;
          ++entry;
          if (first) ok = mbar_wait_awake(o_free(i), (icount++ & 1) ^ 1, abort);   // the epilogue has read O_i
          ok = ok && mbar_wait_awake(p_full(i), pcount & 1, abort);
          if (!ok) break;
          ++pcount;
          tc_fence_after();
          const uint64_t vd = sw128_mnmajor_desc(sbase + C::kRing + st * C::kTile);
          const uint64_t pd = sw128_kmajor_desc(sbase + C::kP + i * 2 * N * 128);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_f16(o_col(i), vd + (2048 * k >> 4), pd + (((k >> 2) * (N * 128) + 32 * (k & 3)) >> 4), kIdescO, !first || k != 0);
          mma_commit(empty_bar(st));
          if (last) mma_commit(o_full(i));
        }
        if (i == 1 && n == 1) mma_commit(q_empty);   // no tile of its own
        ++qcount;
      }
      if (!ok) record_timeout(abort);
      // All MMAs complete before TMEM is freed.
      mma_commit(drain_bar(i));
      volatile int never = 0;
      if (!mbar_wait(drain_bar(i), 0, &never, kWaitLimitNs)) atomicOr(&g_paged_err, kErrTimeout);
    }
  } else if (warp == 14 || warp > 16) {
    bool ok = true;
    Units units(a, seqs, tiles, state);
    Item x;
    if constexpr (kCodes) {
      // ---------------------------------------------------------------- queries as E4M3 terms
      // Row r's terms are rows r, N + r and 2 N + r of the operand, four dimensions a lane.
      uint32_t qcount = 0, tiles_done = 0;
      const float scale = a.scale_log2 * ld_f32(a.k_scale);
      while (ok && units.next(x)) {
        if (x.n() == 0) continue;
        if (warp == 14) {
        ok = mbar_wait_lanes(q_empty, (qcount & 1) ^ 1, abort);
        if (!ok) break;
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)x.row0 * a.q_l + (int64_t)x.hk * a.G * a.q_h + 4 * lane;
        const int valid = x.left * a.G;
#pragma unroll 4
        for (int r = 0; r < N; ++r) {
          const int l = r / a.G, h = r - l * a.G;
          float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (r < valid && 4 * lane < a.D) {
            const uint2 w = *reinterpret_cast<const uint2*>(q + l * a.q_l + h * a.q_h);
            const F2 lo = unpack16<kF16>(w.x), hi = unpack16<kF16>(w.y);
            v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
          }
          float top = max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])));
          // bits of values of one sign are in the values' order, NaN last
          const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
          // 2^-e takes the largest value to [128, 256) (less where it is below 2^-120); not finite: the row becomes NaN
          const int e = (int)(bits >> 23) - 127 - 7;
          const bool bad = bits >= 0x7F800000u;
          const float down = bad ? 1.0f : pow2i(-e > 127 ? 127 : -e);
          uint32_t t[3] = {0, 0, 0};
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            float x0 = v[k] * down, x1 = v[k + 1] * down;
            if (bad) x0 = x1 = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int s = 0; s < 3; ++s) {
              const uint32_t c = cvt_e4m3x2(x0, x1);
              t[s] |= c << (8 * k);
              float y0, y1;
              f16x2_to_f32(cvt_e4m3x2_to_f16x2((uint16_t)c), y0, y1);
              x0 = (x0 - y0) * 16.0f;
              x1 = (x1 - y1) * 16.0f;
            }
          }
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            const int row = s * N + r;
            *reinterpret_cast<uint32_t*>(smem + C::kQ + row * 128 + (((lane >> 2) ^ (row & 7)) << 4) + 4 * (lane & 3)) = t[s];
          }
          if (lane == 0) factor[(qcount & 1) * N + r] = scale / down;
        }
        ++qcount;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        }
#pragma unroll 1
        for (int t = x.t0 + 1; ok && t < x.t1; t += 2) ok = convert(x, 1, t, warp == 14 ? 0 : warp - 16, tiles_done++);
      }
    } else {
      // ---------------------------------------------------------------- V rows that not all rows see
      uint32_t entry[2] = {0, 0};
      while (ok && units.next(x)) {
#pragma unroll 1
        for (int k = 0; ok && k < 2 * x.n(); ++k) {   // K and V of a tile in turn
          const int i = (k >> 1) & 1;
          const uint32_t e = i ? entry[1]++ : entry[0]++;
          const int st = i * R + (int)(e % R), key0 = (x.t0 + (k >> 1)) * kKeys;
          ok = mbar_wait_lanes(full_bar(st), (e / R) & 1, abort);
          if (!ok) break;
          if ((k & 1) && key0 + kKeys > x.lim0) {
            if (clear_rows<kF16, C::kAtoms>(smem + C::kRing + st * C::kTile, lane, x.lim0 - key0, x.limit - key0)) *dirty = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(clean_bar(st));
        }
      }
    }
    if (!ok && lane == 0) record_timeout(abort);
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax: a thread a key
    const int i = warp >> 2;                     // group
    const int key_in = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const int id = 1 + i;                        // the group's barrier
    // where this key's column of P stands, row 0, before the swizzle
    uint8_t* p_at = smem + C::kP + i * 2 * N * 128 + (key_in >> 6) * (N * 128) + (key_in & 7) * 2;
    const int p_chunk = (key_in & 63) >> 3;
    uint32_t scount = 0, icount = 0, items = 0;
    // A warp whose wait gave up goes on to the group's next vote, so that no barrier
    // waits for it, and the group leaves together.
    bool ok = true, out = false;
    Units units(a, seqs, tiles, state);
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
      for (int j = 0; j < n; ++j) {
        const int key0 = (x.t0 + 2 * j + i) * kKeys;
        ok = ok && mbar_wait_lanes(s_full(i), scount & 1, abort);
        ++scount;
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
            tmem_ld_32x32b_x4(s_col(i) + quad + (kCodes ? 2 * N : 0) + r0, t);
            if constexpr (kCodes) {              // t0 + (t1 + t2 / 16) / 16
              uint32_t t1[4], t0[4];
              tmem_ld_32x32b_x4(s_col(i) + quad + N + r0, t1);
              tmem_ld_32x32b_x4(s_col(i) + quad + r0, t0);
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
              grow |= r0 + e < valid && (s[r0 + e] > mm[e] + kLazyMax || (mm[e] == -INFINITY && s[r0 + e] > -INFINITY));
            }
          }
        }
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
            const float m_new = fmaxf(fmaxf(fmaxf(m, t[0]), t[N]), fmaxf(t[2 * N], t[3 * N]));
            run_m[i * N + lane] = m_new;
            run_f[i * N + lane] = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
          }
          group_sync(id);
          // Scores of this tile are complete, so the group's product with the previous
          // one is too (issued before them): O_i may be rescaled here.
          if (j > 0) {
#pragma unroll
            for (int r0 = 0; r0 < N; r0 += 4) {
              if (r0 >= valid) break;
              uint32_t o[4];
              tmem_ld_32x32b_x4(o_col(i) + quad + r0, o);
              tmem_ld_wait();
              const float4 f4 = *reinterpret_cast<const float4*>(run_f + i * N + r0);
              const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                l[r0 + e] *= f[e];
                o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
              }
              tmem_st_32x32b_x4(o_col(i) + quad + r0, o);
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int r0 = 0; r0 < N; r0 += 4) {
          if (r0 >= valid) break;
          const float4 m4 = *reinterpret_cast<const float4*>(run_m + i * N + r0);
          const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + e;
            const float p = ex2(s[r] - (mm[e] == -INFINITY ? 0.0f : mm[e]));
            l[r] += p;
            *reinterpret_cast<uint16_t*>(p_at + r * 128 + ((p_chunk ^ (r & 7)) << 4)) = (uint16_t)cvt16x2(kP16, p, 0.0f);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i));
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
    // ---------------------------------------------------------------- epilogue (and conversion of V's codes)
    const int d = (warp & 3) * 32 + lane;        // this thread's dimension
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    float inv_s = 1.0f, v_scale = 1.0f;
    if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
    if constexpr (kCodes) v_scale = ld_f32(a.v_scale);
    uint32_t icount[2] = {0, 0}, tiles_done = 0;
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
    // Rows that see a position, which not every row of the unit sees, where dimension d
    // is not finite (and was cleared).  Seldom called, and slow.
    auto spoilt_rows = [&](const Item& x) {
      uint32_t rows = 0;
      if (d >= a.D) return rows;
      const int end = min(x.limit, x.t1 * kKeys);
      for (int j = max(x.lim0, x.t0 * kKeys); j < end; ++j) {
        const int at = quotient(j, a.by_page), page = ld_i32(a.table + x.b * a.table_stride + at);
        if (page < 0 || page >= a.pages) continue;
        const uint8_t* v = a.v + page * a.vs[0] + (j - at * a.page_size) * a.vs[1] + x.hk * a.vs[2];
        const bool bad = kCodes ? (v[d] & 0x7F) == 0x7F : (not_finite<kF16>(reinterpret_cast<const uint16_t*>(v)[d]) & 0x8000u) != 0;
        if (!bad) continue;
        for (int r = 0; r < x.left * a.G; ++r)
          if (j < seen(a, x.pos0, x.len, r / a.G + 1)) rows |= 1u << r;
      }
      return rows;
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
    Units units(a, seqs, tiles, state);
    Item x;
    while (ok && units.next(x)) {
      if (x.n() == 0) {
        put_zeros(x);
        continue;
      }
      if constexpr (kCodes) {
#pragma unroll 1
        for (int t = x.t0; ok && t < x.t1; t += 2) ok = convert(x, 0, t, warp & 3, tiles_done++);
        if (!ok) break;
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
      const uint32_t nan_rows = *dirty ? spoilt_rows(x) : 0;
      __syncwarp();   // together again for the TMEM loads
      const int valid = x.left * a.G;
      int64_t at = (int64_t)x.row0 * a.o_l + (int64_t)x.hk * a.G * a.o_h + d;
      int head = 0;
#pragma unroll 1
      for (int r0 = 0; r0 < valid; r0 += 4) {
        uint32_t o0[4], o1[4];
        tmem_ld_32x32b_x4(o_col(0) + quad + r0, o0);
        if (two) tmem_ld_32x32b_x4(o_col(1) + quad + r0, o1);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + e;
          const float f0 = __shfl_sync(0xFFFFFFFFu, a0, r & 31), f1 = __shfl_sync(0xFFFFFFFFu, a1, r & 31);
          float y = __uint_as_float(o0[e]) * f0;
          if (two) y = fmaf(__uint_as_float(o1[e]), f1, y);
          if (nan_rows >> r & 1) y = __uint_as_float(0x7FC00000u);
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
  // Every copy has landed: each was waited for by those that read it, unless they gave
  // up.  Then the block stays for 5 ms, in which any copy under way lands.
  if (*abort && threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 5000000ull) {
    }
  }
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kFewTmem);
  }
}

// Joining cut units: as paged_join_kernel, with rows of DP floats; a thread
// takes four columns of a row.
template <int DP, bool kF16, int N>
__global__ void __launch_bounds__(256) few_join_kernel(const PagedArgs a) {
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

template <int DP, bool kF16, bool kCodes, int N>
cudaError_t launch_kernel(const PagedMaps& maps, const PagedArgs& a, int grid, cudaStream_t st) {
  using C = Few<DP, kCodes, N>;
  auto* k = paged_few_kernel<DP, kF16, kCodes, N>;
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
  cfg.blockDim = dim3(kFewThreads<kCodes>, 1, 1);
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
    if ((e = cudaLaunchKernelEx(&cfg, few_join_kernel<DP, kF16, N>, a)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DP, bool kF16, bool kCodes>
cudaError_t launch_rows(const PagedMaps& maps, const PagedArgs& a, int rows, int grid, cudaStream_t st) {
  return rows == 16 ? launch_kernel<DP, kF16, kCodes, 16>(maps, a, grid, st) : launch_kernel<DP, kF16, kCodes, 32>(maps, a, grid, st);
}

template <int DP>
cudaError_t launch_dims(const PagedMaps& maps, const PagedArgs& a, int rows, bool f16, bool codes, int grid, cudaStream_t st) {
  if (codes) return f16 ? launch_rows<DP, true, true>(maps, a, rows, grid, st) : launch_rows<DP, false, true>(maps, a, rows, grid, st);
  return f16 ? launch_rows<DP, true, false>(maps, a, rows, grid, st) : launch_rows<DP, false, false>(maps, a, rows, grid, st);
}

}  // namespace

cudaError_t launch_paged_few(const PagedMaps& maps, const PagedArgs& a, int rows, int DP, bool f16, bool codes, int grid,
                             cudaStream_t st) {
  return DP == 64 ? launch_dims<64>(maps, a, rows, f16, codes, grid, st) : launch_dims<128>(maps, a, rows, f16, codes, grid, st);
}

cudaError_t paged_few_read_error(cudaStream_t st, uint32_t* err) { return read_paged_error(st, err); }

}  // namespace w8
