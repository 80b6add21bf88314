// Attention of new tokens over a paged cache, on tcgen05: for each token at
// position t of its sequence (of len positions) and query head h, with the key
// head h / (Hq / Hkv),
//
//   s_j = scale * sum_d q_d k_jd,   j < len, and j <= t where causal
//   o   = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max)       (0 where no j counts)
//
// in one pass over the positions, with the running maximum m and sum l as in cross
// attention, whose roles, TMEM layout and hand-overs this kernel has: two slots
// of 128 rows (row = token * group + head in group), both on the same key tiles, or
// where 128 rows hold all tokens of a sequence on its even and odd tiles.  What is its own:
//
// Sequences.  Starts, lengths and pages are the device's.  A unit of work is a
// block of tokens of one sequence and key head; it has the key tiles up to its last
// token's position.  A block takes whole units, the longest first, dealt out to and fro, or, where the
// lengths make that uneven or leave SMs idle, all tiles of all units stand in
// one row of which each CTA takes an even share; every CTA decides that for itself from the
// lengths, alike, and a second kernel joins the partial results.
//
// Pages.  A tile of 128 positions comes in boxes of gcd(page_size, 128) rows, one
// TMA copy a box and 64 dimensions, issued by a lane each; the page numbers of a tile are
// asked for a tile ahead.  A box of no page (beyond the unit's positions, the table
// or the cache) starts behind the last page, where a copy writes zeros.
//
// E4M3 cells.  The tensor core takes no E4M3 beside 16 bits.  Codes are copied
// as they are to a ring of their own, and the epilogue's warps, idle between
// units, write them to the operands' ring as 16-bit values (exact): K in the
// queries' type, V as binary16, whose P is binary16 too.  The scales go into the
// scores' factor and the output's.
//
// Positions that a row does not see have P = 0, but 0 * NaN would spoil the
// product: V rows behind the unit's last position are cleared in shared memory.
// Those that only some of a unit's rows see cannot be; if they hold a value that
// is not finite, it is cleared too, and added at the end to the rows that see it (restore: prompts with NaN in
// every hundredth value of a dimension 59 -> 181 us, the chunk over 8192 positions 329 -> 413).
//
// Measured (GB300, a replayed graph / one call among others): a chunk of 4096 tokens
// over 20670 positions, 32 query and 8 key heads of 128, bf16: 911-942 / 953-961 us = 1.30-1.37
// PFLOP/s; with 1024 tokens the tensor pipe is active in 53% of the cycles.  Over E4M3 cells
// the chunk takes 1233-1268 us: the conversion in shared memory is what differs.  Six prompts of
// 629 to 1077 tokens, E4M3 out: 58.8-59.2 / 58.9-59.6 us; a tile of both slots takes 3450 cycles there (stamped in a
// copy of the kernel), the two products at the nominal rate 2048 of them, and the first tile of a
// unit 1900 to 4100 more.  At most 25 rows (up to five tokens of seven sequences) over up to 4133
// positions, 20/4 heads of 64, f16: 22.5-23.1 / 22.6-23.3 us, latency.
//
// Waits: a thread that sleeps on a barrier is woken about 1 us late, so the products' warp asks 256
// times before it sleeps; page numbers are loaded raw and checked when they are used, since checked at
// once each tile's copies waited for that load.  These two, and warps without rows left idle: prompts
// 91.6 -> 75.4 us.
//
// Roundings below 32 bits: P (its sum l is taken before), since the tensor core takes 32-bit weights
// beside 32-bit values alone, which would be twice the bytes of V and half the rate; and the output.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "attention_common.cuh"
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {

namespace {

// With 256 rows a unit cutting costs the time of about 10 tiles, with 128 rows about 8
// (cross attention's figures, whose tiles these are).  Measured with 5 and 4, 10 and 8, 16 and 14 tiles, 32/8 heads of
// 128, us: a chunk of 2000 tokens over 2500 positions 77.0, 61.2 and 56.4, over E4M3 cells 117.5, 82.1 and
// 76.5; drafts over up to 1500 positions 18.1, 16.4 and 16.4, over E4M3 cells 22.2, 20.7 and 20.7; 16 sequences' drafts
// over up to 3000 27.3, 27.4 and 32.1; chunks of 256 to 1024 over 4096 to 20670 positions, and ragged prompts, alike.
constexpr Cutting kCutShared{8, 1.0f, 10.0f}, kCutSplit{4, 1.4f, 8.0f};

template <int DP, bool kCodes, bool kShared>
struct Cfg {
  static constexpr int kAtoms = DP / 64;
  static constexpr int kTile = kAtoms * kAtom;           // bytes of 128 rows of Q, K or V in 16 bits
  static constexpr int kRawTile = kKeys * DP;            // of codes
  static constexpr int kQs = kShared ? 2 : 1;            // tiles of queries
  static constexpr int kStages = DP == 128 ? (kCodes && kShared ? 3 : 4) : (kCodes || kShared ? 6 : 8);
  static constexpr int kRaws = !kCodes ? 0 : DP == 128 ? (kShared ? 2 : 3) : (kShared ? 4 : 8);
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + kQs * kTile;
  static constexpr int kRaw = kRing + kStages * kTile;
  static constexpr int kOut = kRaw + kRaws * kRawTile;   // 32 rows of 128 bytes for each epilogue warp
  static constexpr int kSum = kOut + (kShared ? 4 * 32 * 128 : 0);   // l[2][128], m[2][128]
  static constexpr int kSeq = kSum + 4 * kRows * 4;      // row0, tokens, base, len of each sequence
  static constexpr int kTiles = kSeq + kMaxSeqs * 16;    // tiles of one key head's units
  static constexpr int kFirst = kTiles + kMaxSeqs * 4;   // where they begin in the row of all tiles
  static constexpr int kOrder = kFirst + (kMaxSeqs + 4) * 4;   // sequences by their units
  static constexpr int kState = kOrder + kMaxSeqs * 2;
  static constexpr int kBar = kState + 16 * 4;
  // full[S], empty[S], clean[S], raw_full[R], raw_empty[R], q_full[2], q_empty[2], s_full[2], p_full[2],
  // o_full[2], l_full[2], o_free[2], p_half[2], drain[2]
  static constexpr int kNumBars = 3 * kStages + 2 * kRaws + 18;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kDirty = kAbort + 4;
  static constexpr int kAlloc = kDirty + 4 + 1024;       // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448, "shared memory budget");
};

// With 128 rows a sequence is one unit of a key head.
template <bool kShared>
struct UnitsKind {
  using type = Units;
};
template <>
struct UnitsKind<false> {
  using type = WholeUnits;
};
template <bool kShared>
using UnitsOf = typename UnitsKind<kShared>::type;

// kShared: both slots work on the same key tiles (256 query rows); otherwise
// they take the even and odd tiles of the same 128 rows.
template <int DP, bool kF16, bool kCodes, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedArgs a) {
  using C = Cfg<DP, kCodes, kShared>;
  constexpr int S = C::kStages, RW = C::kRaws;
  constexpr bool kP16 = kF16 || kCodes;            // P and V are binary16
  constexpr uint32_t kIdescS = make_idesc(kF16 ? 0 : 1, kF16 ? 0 : 1, kRows, kKeys);
  constexpr uint32_t kIdescO = make_idesc(kP16 ? 0 : 1, kP16 ? 0 : 1, kRows, DP) | (1u << 16);  // B is MN-major

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBar;
  auto bar = [&](int k) { return bar0 + 8u * (uint32_t)k; };
  auto full_bar = [&](int s) { return bar(s); };
  auto empty_bar = [&](int s) { return bar(S + s); };
  auto clean_bar = [&](int s) { return bar(2 * S + s); };
  auto raw_full = [&](int r) { return bar(3 * S + r); };
  auto raw_empty = [&](int r) { return bar(3 * S + RW + r); };
  constexpr int kRest = 3 * S + 2 * RW;
  auto q_full = [&](int i) { return bar(kRest + i); };
  auto q_empty = [&](int i) { return bar(kRest + 2 + i); };
  auto s_full = [&](int i) { return bar(kRest + 4 + i); };
  auto p_full = [&](int i) { return bar(kRest + 6 + i); };
  auto o_full = [&](int i) { return bar(kRest + 8 + i); };
  auto l_full = [&](int i) { return bar(kRest + 10 + i); };
  auto o_free = [&](int i) { return bar(kRest + 12 + i); };
  auto p_half = [&](int i) { return bar(kRest + 14 + i); };
  auto drain_bar = [&](int i) { return bar(kRest + 16 + i); };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kAbort);
  volatile int* dirty = reinterpret_cast<volatile int*>(smem + C::kDirty);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  float* sum_l = reinterpret_cast<float*>(smem + C::kSum);
  float* sum_m = sum_l + 2 * kRows;
  Seq* seqs = a.B <= kMaxSeqs ? reinterpret_cast<Seq*>(smem + C::kSeq) : nullptr;
  uint32_t* tiles = reinterpret_cast<uint32_t*>(smem + C::kTiles);
  int* state = reinterpret_cast<int*>(smem + C::kState);
  uint16_t* order = reinterpret_cast<uint16_t*>(smem + C::kOrder);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), kShared ? 2 : 1);   // the slots that read the tile
      mbar_init(clean_bar(s), kCodes ? 4 : 1);
    }
    for (int r = 0; r < RW; ++r) {
      mbar_init(raw_full(r), 1);
      mbar_init(raw_empty(r), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), kShared ? 1 : 2);     // the slots that read Q
      mbar_init(s_full(i), 1);
      mbar_init(p_half(i), 4);
      mbar_init(p_full(i), 4);
      mbar_init(o_full(i), 1);
      mbar_init(l_full(i), 4);
      mbar_init(o_free(i), 4);
    }
    mbar_init(drain_bar(0), 1);
    mbar_init(drain_bar(1), 1);
    *abort = 0;
    *dirty = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == 12) {
    tmem_alloc(sbase + C::kTmemSlot, kTmemCols);
    tmem_relinquish();
  }
  // Rows of a slot without a query (groups that do not divide 128) hold zeros:
  // no copy writes them, and the rows' maxima have to be the same in every call.
  const uint32_t q_bytes = (uint32_t)(a.G * a.rows_l * 128);
  if (q_bytes < kAtom) {
    for (uint32_t at = q_bytes + 16 * threadIdx.x; at < kAtom; at += 16 * kThreads)
#pragma unroll
      for (int k = 0; k < C::kQs * C::kAtoms; ++k)
        *reinterpret_cast<uint4*>(smem + C::kQ + k * kAtom + at) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  griddep_wait();   // from here on what earlier kernels wrote may be read
  uint32_t* tiles_first = reinterpret_cast<uint32_t*>(smem + C::kFirst);
  if constexpr (kShared) {
    if (seqs) {
      for (int b = threadIdx.x; b < a.B; b += kThreads) seqs[b] = load_seq(a, b);
      __syncthreads();
      order_units(a, seqs, order);
      if (a.may_cut) share_out(a, seqs, tiles, tiles_first, state, kCutShared);
    }
  } else if (warp == 0 && seqs) {
    share_out_whole(a, seqs, tiles, tiles_first, state, kCutSplit);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The next kernel (the joining one) may start its prologue.  Not with 256 rows: what is launched
  // early there costs 3 to 5% (chunks 911 -> 936 us, prompts 75 -> 79).
  if (!kShared) griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const auto s_col = [&](int i) { return tmem + (uint32_t)(i * kKeys); };
  const auto o_col = [&](int i) { return tmem + 256u + (uint32_t)(i * DP); };

  // Tiles that slot i works on in an item of n tiles.
  const auto slot_tiles = [](int n, int i) { return kShared ? n : (n + 1 - i) / 2; };

  // The stages are one ring in the shared form, which both slots go through
  // tile by tile (K and V in turn), and a ring for each slot in the separate form: a
  // waiter has to see every filling of its stages.
  constexpr int R = kShared ? S : S / 2;                              // stages of a ring
  const auto stage_of = [](int i, uint32_t e) { return (kShared ? 0 : i * R) + (int)(e % R); };
  const auto phase_of = [](uint32_t e) { return (e / R) & 1; };

  // The order in which K and V tiles are loaded, cleared and converted:
  //   shared:   K0 V0 K1 V1 ...
  //   separate: K0 K1 V0 V1 K2 K3 V2 V3 ...   (slots 0 and 1 in turn)
  const auto walk = [&](const Item& x, auto&& f) {   // f(V?, ring, tile)
    const int n = x.n();
    if constexpr (kShared) {
      for (int j = 0; j < n; ++j)
        if (!f(false, 0, x.t0 + j) || !f(true, 0, x.t0 + j)) return false;
    } else {
      for (int j = 0; j < n; j += 2) {
        const bool two = j + 1 < n;
        if (!f(false, 0, x.t0 + j) || (two && !f(false, 1, x.t0 + j + 1)) || !f(true, 0, x.t0 + j) ||
            (two && !f(true, 1, x.t0 + j + 1)))
          return false;
      }
    }
    return true;
  };
  // The page of box `lane` of a tile as the table has it (checked when it is used:
  // the load is in flight until then), or one behind the last: a copy then writes zeros.
  const auto ask_page = [&](const Item& x, int tile) {
    const int key = tile * kKeys + lane * a.box;
    int page = a.pages;
    if (lane < a.boxes && key < x.limit) page = ld_i32(a.table + x.b * a.table_stride + quotient(key, a.by_page));
    return page;
  };

  if (warp >= 12) {
  regs_down<72>();
  if (warp == 13) {
    // ---------------------------------------------------------------- loads
    uint32_t filled[2] = {0, 0}, raws = 0, qcount[2] = {0, 0};
    bool ok = true;
    auto load_q = [&](const Item& x, int i) {
      if (!mbar_wait_lanes(q_empty(i), (qcount[i] & 1) ^ 1, abort)) return false;
      ++qcount[i];
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full(i), C::kAtoms * q_bytes);
        for (int at = 0; at < C::kAtoms; ++at)
          tma_load_4d(sbase + C::kQ + i * C::kTile + at * kAtom, &maps.q, q_full(i), 64 * at, 0, x.row0 + i * a.rows_l, x.hk);
      }
      __syncwarp();
      return true;
    };
    UnitsOf<kShared> units(a, seqs, tiles, state, order);
    Item x;
    while (ok && units.next(x)) {
      if (x.n() == 0) continue;
      bool first = true;
      // pages of the tiles that come next, asked for a tile ahead: [ring]
      int page[2], ahead[2];
      page[0] = ask_page(x, x.t0);
      page[1] = kShared ? 0 : ask_page(x, x.t0 + 1);
      ahead[0] = ahead[1] = 0;
      ok = load_q(x, 0);
      ok = ok && walk(x, [&](bool is_v, int ring, int tile) {
        if (!is_v) ahead[ring] = ask_page(x, tile + (kShared ? 1 : 2));
        const int key = tile * kKeys + lane * a.box;
        const int slot = key - quotient(key, a.by_page) * a.page_size;
        uint32_t dst, full;
        if constexpr (kCodes) {
          const int r = (int)(raws % RW);
          if (!mbar_wait_lanes(raw_empty(r), ((raws / RW) & 1) ^ 1, abort)) return false;
          ++raws;
          full = raw_full(r);
          dst = sbase + C::kRaw + r * C::kRawTile + lane * a.box * DP;
          if (lane == 0) mbar_arrive_expect_tx(full, C::kRawTile);
        } else {
          const uint32_t e = filled[ring];
          const int st = stage_of(ring, e);
          if (!mbar_wait_lanes(empty_bar(st), phase_of(e) ^ 1, abort)) return false;
          ++filled[ring];
          full = full_bar(st);
          dst = sbase + C::kRing + st * C::kTile + lane * a.box * 128;
          if (lane == 0) mbar_arrive_expect_tx(full, C::kTile);
        }
        __syncwarp();
        if (lane < a.boxes) {
          if (page[ring] < 0 || page[ring] > a.pages) page[ring] = a.pages;
          if constexpr (kCodes) {
            tma_load_4d(dst, is_v ? &maps.v : &maps.k, full, 0, x.hk, slot, page[ring]);
          } else {
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              tma_load_4d(dst + at * kAtom, is_v ? &maps.v : &maps.k, full, 64 * at, x.hk, slot, page[ring]);
          }
        }
        __syncwarp();
        if (is_v) page[ring] = ahead[ring];
        if (kShared && first) {
          first = false;
          return load_q(x, 1);
        }
        return true;
      });
    }
    if (!ok && lane == 0) record_timeout(abort);
    // Every copy must have landed before the block ends.
    volatile int never = 0;
    if (lane == 0) {
      if constexpr (kCodes) {
        for (uint32_t j = 1; j <= (uint32_t)RW && j <= raws; ++j) {
          const uint32_t e = raws - j;
          if (!mbar_wait(raw_full((int)(e % RW)), (e / RW) & 1, &never, kWaitLimitNs)) atomicOr(&g_paged_err, kErrTimeout);
        }
      } else {
        for (int i = 0; i < (kShared ? 1 : 2); ++i)
          for (uint32_t j = 1; j <= R && j <= filled[i]; ++j) {
            const uint32_t e = filled[i] - j;
            if (!mbar_wait(full_bar(stage_of(i, e)), phase_of(e), &never, kWaitLimitNs)) atomicOr(&g_paged_err, kErrTimeout);
          }
      }
      for (int i = 0; i < 2; ++i)
        if (qcount[i] > 0 && !mbar_wait(q_full(i), (qcount[i] - 1) & 1, &never, kWaitLimitNs))
          atomicOr(&g_paged_err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 12 || warp == 15) {
    // ---------------------------------------------------------------- MMA issue
    // One thread for each slot.  A slot's MMAs run in the order of their issue:
    // the scores of tile j + 1 may be written over P of tile j, and when they are
    // complete so is the product of tile j.
    if (elect_one()) {
      const int i = warp == 12 ? 0 : 1;
      uint32_t entry = 0;                        // of this slot's ring
      uint32_t qcount = 0, pcount = 0, icount = 0;
      bool ok = true;
      // Waits for the ring's next entry; returns its stage.  V goes by way of the
      // clearing warp, and so does K in the separate form, where a stage holds K
      // and V in no fixed order (that warp then sees every filling of a stage);
      // codes all go by way of the converting warps.
      auto take = [&](bool is_v) {
        const uint32_t e = entry++;
        const int st = stage_of(i, e);
        ok = ok && mbar_wait_awake(kCodes || is_v || !kShared ? clean_bar(st) : full_bar(st), phase_of(e), abort);
        tc_fence_after();
        return st;
      };
      UnitsOf<kShared> units(a, seqs, tiles, state, order);
      Item x;
      while (ok && units.next(x)) {
        const int n = x.n();
        if (n == 0) continue;
        // also by a slot without a tile: its word on Q below belongs to this Q
        ok = mbar_wait_awake(q_full(kShared ? i : 0), qcount & 1, abort);
        if (!ok) break;
        tc_fence_after();
        for (int j = kShared ? 0 : i; ok && j < n; j += kShared ? 1 : 2) {
          const bool first = j == (kShared ? 0 : i), last = j + (kShared ? 1 : 2) >= n;
          // The slots take turns: a slot's scores are started when the other's
          // are complete.
          if (kShared && (i == 1 || pcount > 0))
            ok = ok && mbar_wait_awake(s_full(1 - i), (pcount - (1 - i)) & 1, abort);
          int st = take(false);
          if (!ok) break;
          const uint64_t qd = sw128_kmajor_desc(sbase + C::kQ + (kShared ? i : 0) * C::kTile);
          const uint64_t kd = sw128_kmajor_desc(sbase + C::kRing + st * C::kTile);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {   // descriptors count in 16 bytes
            const uint64_t at = ((k >> 2) * kAtom + 32 * (k & 3)) >> 4;
            mma_f16(s_col(i), qd + at, kd + at, kIdescS, k != 0);
          }
          mma_commit(s_full(i));
          mma_commit(empty_bar(st));
          if (last) mma_commit(q_empty(kShared ? i : 0));

          st = take(true);
          if (first) ok = ok && mbar_wait_awake(o_free(i), (icount++ & 1) ^ 1, abort);   // the epilogue has read O_i
          const uint64_t vd = sw128_mnmajor_desc(sbase + C::kRing + st * C::kTile);
#pragma unroll
          for (int h = 0; h < 2; ++h) {          // 64 keys at a time, as the softmax hands them over
            ok = ok && mbar_wait_awake(h ? p_full(i) : p_half(i), pcount & 1, abort);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = h * kKeys / 32; k < (h + 1) * kKeys / 32; ++k)
              mma_f16_tmem_a(o_col(i), s_col(i) + 8 * k, vd + (2048 * k >> 4), kIdescO, !first || k != 0);
          }
          ++pcount;
          if (!ok) break;
          mma_commit(empty_bar(st));
          if (last) mma_commit(o_full(i));
        }
        if (!kShared && i == 1 && n == 1) mma_commit(q_empty(0));   // no tile of its own
        ++qcount;
      }
      if (!ok) record_timeout(abort);
      // All MMAs complete before TMEM is freed.
      mma_commit(drain_bar(i));
      volatile int never = 0;
      if (!mbar_wait(drain_bar(i), 0, &never, kWaitLimitNs)) atomicOr(&g_paged_err, kErrTimeout);
    }
  } else if (warp == 14) {
    // ---------------------------------------------------------------- V rows that not all rows see
    if constexpr (!kCodes) {
      uint32_t seen_tiles[2] = {0, 0};
      bool ok = true;
      UnitsOf<kShared> units(a, seqs, tiles, state, order);
      Item x;
      while (ok && units.next(x)) {
        ok = walk(x, [&](bool is_v, int ring, int tile) {
          const uint32_t e = ring ? seen_tiles[1]++ : seen_tiles[0]++;
          const int st = stage_of(ring, e);
          const bool pass = kShared && !is_v;
          if (!pass && !mbar_wait_lanes(full_bar(st), phase_of(e), abort)) return false;
          const int key0 = tile * kKeys;
          if (is_v && key0 + kKeys > x.lim0) {
            if (clear_rows<kF16, false, C::kAtoms>(smem + C::kRing + st * C::kTile, lane, x.lim0 - key0, x.limit - key0, a.box)) *dirty = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (!pass && lane == 0) mbar_arrive(clean_bar(st));
          return true;
        });
      }
      if (!ok && lane == 0) record_timeout(abort);
    }
  }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_up<176>();
    const int i = warp >> 2;                     // slot
    const int row = (warp & 3) * 32 + lane;
    const int token = (kShared ? i * a.rows_l : 0) + row / a.G;   // of the unit
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    float scale_log2 = a.scale_log2;
    if constexpr (kCodes) scale_log2 *= ld_f32(a.k_scale);
    uint32_t scount = 0, icount = 0;
    bool ok = true;
    UnitsOf<kShared> units(a, seqs, tiles, state, order);
    Item x;
    while (ok && units.next(x)) {
      const int n = slot_tiles(x.n(), i);
      if (n == 0) continue;
      float m = -INFINITY, l = 0.0f;             // m in powers of two: scaled scores
      // Positions that the row sees.  A row without a query sees none and has no say in when the maxima are
      // raised (its scores may be another sequence's): what it holds must not decide on the other rows' roundings.
      const bool mine = row / a.G < a.rows_l && token < x.left;
      const int limit = mine ? seen(a, x.pos0, x.len, token + 1) : 0;
      // A warp without a query leaves its weights as they are: they reach its own rows alone.
      const bool busy = __any_sync(0xFFFFFFFFu, mine);
      for (int j = 0; j < n; ++j) {
        if (!busy) {
          if (!mbar_wait_lanes(s_full(i), scount & 1, abort)) {
            ok = false;
            break;
          }
          ++scount;
          if (lane == 0) {
            mbar_arrive(p_half(i));
            mbar_arrive(p_full(i));
          }
          continue;
        }
        const int key0 = (x.t0 + (kShared ? j : 2 * j + i)) * kKeys;
        const bool masked = key0 + kKeys > x.lim0;
        if (!mbar_wait_lanes(s_full(i), scount & 1, abort)) {
          ok = false;
          break;
        }
        ++scount;
        tc_fence_after();
        uint32_t r[4][32];
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        tmem_ld_32x32b_x32(s_col(i) + quad, r[0]);
        tmem_ld_32x32b_x32(s_col(i) + quad + 32, r[1]);
        tmem_ld_wait_for(r[0]);
        tmem_ld_wait_for(r[1]);
        tmem_ld_32x32b_x32(s_col(i) + quad + 64, r[2]);
        tmem_ld_32x32b_x32(s_col(i) + quad + 96, r[3]);
        if (__builtin_expect(masked, 0)) {   // a position that the row does not see has the weight exp2(-inf) = 0
          tmem_ld_wait_for(r[2]);
          tmem_ld_wait_for(r[3]);
          const int rel = limit - key0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= rel) r[c][e] = 0xFF800000u;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c == 2) {
            tmem_ld_wait_for(r[2]);
            tmem_ld_wait_for(r[3]);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            tops[(e >> 1) & 3] = fmaxf(fmaxf(tops[(e >> 1) & 3], __uint_as_float(r[c][e])), __uint_as_float(r[c][e + 1]));
        }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale_log2;
        // Scores of slot i are complete, so its product with the previous tile
        // is too (issued before them): O_i may be rescaled here.
        const bool grow = mine && (top > m + kLazyMax || (m == -INFINITY && top > m));
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, grow), 0)) {
          const float m_new = fmaxf(m, top);
          if (j > 0) {
            const float f = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
            l *= f;
#pragma unroll 1
            for (int c = 0; c < DP / 16; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(o_col(i) + quad + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(o_col(i) + quad + c * 16, o);
            }
          }
          m = m_new;
        }
        const F2 scale = splat(scale_log2), minus_m = splat(m == -INFINITY ? 0.0f : -m);
        F2 sums[2] = {splat(0.0f), splat(0.0f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const F2 t = fma2(F2{__uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1])}, scale, minus_m);
            const F2 w = F2{ex2(t.x), ex2(t.y)};
            sums[(e >> 1) & 1] = add2(sums[(e >> 1) & 1], w);
            p[e >> 1] = cvt16x2(kP16, w.x, w.y);
          }
          // P takes the first half of S_i's columns, all of which are in registers
          tmem_st_32x32b_x16(s_col(i) + quad + c * 16, p);
          if (c & 1) {   // 64 keys of P: the product with V may start on them
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c == 1 ? p_half(i) : p_full(i));
          }
        }
        sums[0] = add2(sums[0], sums[1]);
        l += sums[0].x + sums[0].y;
      }
      if (!ok) break;
      // the epilogue has read the previous item's sums
      if (!mbar_wait_lanes(o_free(i), (icount & 1) ^ 1, abort)) {
        ok = false;
        break;
      }
      ++icount;
      sum_l[i * kRows + row] = l;
      sum_m[i * kRows + row] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(l_full(i));
    }
    if (!ok && lane == 0) record_timeout(abort);
  } else {
    // ---------------------------------------------------------------- epilogue (and conversion of codes)
    regs_down<88>();
    const int row = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const int pos = row / a.G, g = row - pos * a.G, warp_l = 32 / a.G;
    float inv_s = 1.0f, v_scale = 1.0f;
    if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
    if constexpr (kCodes) v_scale = ld_f32(a.v_scale);
    uint32_t icount[2] = {0, 0}, raws = 0, filled[2] = {0, 0};
    bool ok = true;

    const int out_kind = a.s_out ? 0 : 1;      // log2 of a value's bytes
    int kind = out_kind;                       // 2 in a unit that writes a partial result
    constexpr int kUnitRows = kShared ? 2 * kRows : kRows;
    // Where 4 columns of a row of a partial result stand: those of a warp's 32
    // rows together, so that a store is 512 bytes in one piece.
    auto part_at = [&](const Item& x, int row_group, int quad_col) {
      return reinterpret_cast<float4*>(a.part) + (((int64_t)x.part * (kUnitRows / 32) + row_group) * (DP / 4) + quad_col) * 32 + lane;
    };
    // 32 columns (chunk c) of a partial result.
    auto put_part = [&](const Item& x, int row_group, int c, const uint32_t (&r)[32], float f) {
      float4* dst = part_at(x, row_group, 8 * c);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dst[k * 32] = make_float4(__uint_as_float(r[4 * k]) * f, __uint_as_float(r[4 * k + 1]) * f,
                                  __uint_as_float(r[4 * k + 2]) * f, __uint_as_float(r[4 * k + 3]) * f);
    };
    // Where this thread's row (token l of the unit) starts, or null.
    auto out_row = [&](const Item& x, int l) -> uint8_t* {
      if (pos >= a.rows_l || l >= x.left) return nullptr;
      return static_cast<uint8_t*>(a.out) + (((int64_t)(x.row0 + l) * a.o_l + (int64_t)(x.hk * a.G + g) * a.o_h) << kind);
    };
    // Packs 32 scaled columns: 8 words of codes or 16 of 16-bit values.
    auto pack = [&](const uint32_t (&r)[32], float f, uint32_t* w) {
      const F2 ff = splat(kind == 0 ? f * inv_s : f);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const F2 v = mul2(F2{__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])}, ff);
        if (kind == 0) {
          const uint32_t c = cvt_e4m3x2(v.x, v.y);
          w[k >> 1] = k & 1 ? w[k >> 1] | (c << 16) : c;
        } else {
          w[k] = cvt16x2(kF16, v.x, v.y);
        }
      }
    };
    // A thread's packed row (or 32 columns of it): whole 32-byte sectors where
    // the rows allow it.
    auto put_words = [&](uint8_t* at, int words, int bytes, const uint32_t* w) {
#pragma unroll
      for (int k = 0; k < words; k += 8) {
        if (a.wide) {
          if (4 * k < bytes) st_global_32(at + 4 * k, w[k], w[k + 1], w[k + 2], w[k + 3], w[k + 4], w[k + 5], w[k + 6], w[k + 7]);
        } else {
#pragma unroll
          for (int h = 0; h < 8; h += 2)   // rows of codes are 8-byte aligned
            if (4 * (k + h) < bytes) *reinterpret_cast<uint2*>(at + 4 * (k + h)) = make_uint2(w[k + h], w[k + h + 1]);
        }
      }
    };
    // A warp's packed rows by way of its 4 KB of shared memory and a bulk copy
    // for each 128 bytes of a row (64 for codes of small heads).
    auto put_bulk = [&](int token0, int hk, const uint32_t* w) {
      constexpr int kHalves = DP / 64;                               // 16-bit rows: 64 columns at a time
      uint8_t* stage = smem + C::kOut + (warp & 3) * 32 * 128;
      const uint32_t stage_at = sbase + C::kOut + (uint32_t)((warp & 3) * 32 * 128);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (kind == 0 && h > 0) break;
        if (lane == 0) tma_store_wait_read<0>();                     // the copy before has read the stage
        __syncwarp();
        if (kind == 0 && DP == 64) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int at = (kind == 0 ? 0 : 32 * h) + 4 * k;
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(w[at], w[at + 1], w[at + 2], w[at + 3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_4d(&maps.o, stage_at, kind == 0 ? 0 : 64 * h, 0, token0, hk);
          tma_store_commit();
        }
      }
    };
    auto put_zeros = [&](uint8_t* row_at) {
      if (!row_at) return;
      const int bytes = a.D << kind;
      for (int k = 0; k < bytes; k += 8) *reinterpret_cast<uint2*>(row_at + k) = make_uint2(0, 0);
    };
    auto put_lse = [&](const Item& x, int r, float m, float sum) {
      if (kind == 2) a.part_lse[(int64_t)x.part * kUnitRows + r] = sum == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) + log2f(sum);
    };
    // V's values that are not finite, at positions that this row (token l of the unit) sees
    // but not every row of the unit, were cleared: they are added to its accumulator, as if
    // their weights were 1, by the whole warp.  Seldom called, and slow: the warp's lanes first look through
    // the positions for the dimensions, four at a time, in which there is any.
    auto restore = [&](const Item& x, int i, int l) {
      const bool mine = pos < a.rows_l && l < x.left;
      const int from = max(x.lim0, x.t0 * kKeys), last = min(x.limit, x.t1 * kKeys);
      const int end = mine ? min(seen(a, x.pos0, x.len, l + 1), last) : 0;
      uint32_t found = 0;
#pragma unroll 1
      for (int j = from + lane; j < last; j += 32) {
        if (!kShared && ((j / kKeys - x.t0) & 1) != i) continue;     // the other slot's tile
        const int at = quotient(j, a.by_page), page = ld_i32(a.table + x.b * a.table_stride + at);
        if (page < 0 || page >= a.pages) continue;
        const uint8_t* v = a.v + page * a.vs[0] + (j - at * a.page_size) * a.vs[1] + x.hk * a.vs[2];
#pragma unroll 4
        for (int d = 0; d < a.D; d += 8) {
          uint32_t low, high;
          if (kCodes) {
            const uint2 w = *reinterpret_cast<const uint2*>(v + d);
            low = nan_codes(w.x), high = nan_codes(w.y);
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(v + 2 * d);
            low = not_finite<kP16>(w.x) | not_finite<kP16>(w.y), high = not_finite<kP16>(w.z) | not_finite<kP16>(w.w);
          }
          found |= (low ? 1u : 0u) << (d >> 2) | (high ? 2u : 0u) << (d >> 2);
        }
      }
      __syncwarp();
#pragma unroll 1
      for (found = __reduce_or_sync(0xFFFFFFFFu, found); found; found &= found - 1) {
        const int d = 4 * (__ffs(found) - 1);
        float add[4] = {};
        bool some = false;
#pragma unroll 1
        for (int j = from; j < end; ++j) {
          if (!kShared && ((j / kKeys - x.t0) & 1) != i) continue;   // the other slot's tile
          const int at = quotient(j, a.by_page), page = ld_i32(a.table + x.b * a.table_stride + at);
          if (page < 0 || page >= a.pages) continue;
          const uint8_t* v = a.v + page * a.vs[0] + (j - at * a.page_size) * a.vs[1] + x.hk * a.vs[2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint16_t w;                                              // as it was in the tile, in P's type
            if (kCodes) w = (v[d + e] & 0x7F) == 0x7F ? 0x7E00 : 0;
            else w = reinterpret_cast<const uint16_t*>(v)[d + e];
            if (!(not_finite<kP16>(w) & 0x8000u)) continue;
            some = true;
            add[e] += unpack16<kP16>(w).x;
          }
        }
        __syncwarp();
        if (!__any_sync(0xFFFFFFFFu, some)) continue;
        uint32_t o[4];
        tmem_ld_32x32b_x4(o_col(i) + quad + d, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + add[e]);
        tmem_st_32x32b_x4(o_col(i) + quad + d, o);
        tmem_st_wait();
      }
    };

    // A quarter of a tile of codes from the raw ring to the operands' ring, as
    // 16-bit values in the 128-byte swizzle: this warp's 32 rows, 16 codes of a lane at a time.
    auto convert = [&](const Item& x, bool is_v, int ring, int tile) {
      const int rs = (int)(raws % (RW ? RW : 1));
      const uint32_t e = filled[ring];
      const int st = stage_of(ring, e);
      if (!mbar_wait_lanes(raw_full(rs), (raws / (RW ? RW : 1)) & 1, abort) ||
          !mbar_wait_lanes(empty_bar(st), phase_of(e) ^ 1, abort))
        return false;
      ++raws;
      ++filled[ring];
      const uint8_t* raw = smem + C::kRaw + rs * C::kRawTile;
      uint8_t* to = smem + C::kRing + st * C::kTile;
      const int key0 = tile * kKeys;
      if (!is_v) convert_rows<DP, kF16>(raw, to, warp & 3, lane, kKeys, kKeys);
      else if (convert_rows<DP, true>(raw, to, warp & 3, lane, key0 + kKeys > x.lim0 ? x.lim0 - key0 : kKeys, x.limit - key0)) *dirty = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(clean_bar(st));
        mbar_arrive(raw_empty(rs));
      }
      return true;
    };

    if (a.may_cut && state[kShares] > 0 && state[kZeros]) {   // units without a tile: their rows are zeros
      Item x;
      const int units = a.Hkv * a.blocks;
      for (int b = 0; b < a.B; ++b)
        for (int it = blockIdx.x; it < units; it += gridDim.x) {
          x.b = b;
          x.hk = it / a.blocks;
          const int first = (it - x.hk * a.blocks) * a.per;
          const Seq s = seqs[b];
          if (first >= s.tokens) continue;
          x.left = min(a.per, s.tokens - first);
          if (seen(a, s.base, s.len, first + x.left) > 0) continue;
          x.row0 = s.row0 + first;
          for (int i = 0; i < (kShared ? 2 : 1); ++i) put_zeros(out_row(x, i * a.rows_l + pos));
        }
    }
    UnitsOf<kShared> units(a, seqs, tiles, state, order);
    Item x;
    while (ok && units.next(x)) {
      kind = x.part < 0 ? out_kind : 2;
      if constexpr (kCodes) {
        ok = walk(x, [&](bool is_v, int ring, int tile) { return convert(x, is_v, ring, tile); });
        if (!ok) break;
      }
      if constexpr (kShared) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int l = i * a.rows_l + pos;
          uint8_t* row_at = out_row(x, l);
          const int l_warp = l - pos + (warp & 3) * warp_l;   // token of the warp's first row
          if (x.n() == 0) {
            put_zeros(row_at);
            continue;
          }
          if (!mbar_wait_lanes(l_full(i), icount[i] & 1, abort) ||
              !mbar_wait_lanes(o_full(i), icount[i] & 1, abort)) {
            ok = false;
            break;
          }
          ++icount[i];
          tc_fence_after();
          const float sum = sum_l[i * kRows + row];
          const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum) * v_scale;
          put_lse(x, i * kRows + row, sum_m[i * kRows + row], sum);
          const bool spoilt = __any_sync(0xFFFFFFFFu, *dirty != 0);   // a later tile may say so just now: the warp as one
          // A bulk copy writes whole rows of a warp: only where all of them are the sequence's.
          const bool bulk = a.tma_out && l_warp + warp_l <= x.left;
          __syncwarp();   // together again for the TMEM loads
          if (__builtin_expect(spoilt, 0)) restore(x, i, l);
          // The accumulator goes to registers, packed, before anything is
          // stored: the next item's first product waits for it.
          auto free_o = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free(i));
          };
          if (kind == 2) {
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(o_col(i) + quad + c * 32, r);
              tmem_ld_wait_for(r);
              if (c == DP / 32 - 1) free_o();
              put_part(x, 4 * i + (warp & 3), c, r, f);
              __syncwarp();
            }
          } else if (kind == 0) {
            uint32_t w[DP / 4];
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(o_col(i) + quad + c * 32, r);
              tmem_ld_wait_for(r);
              if (c == DP / 32 - 1) free_o();
              pack(r, f, w + 8 * c);
            }
            if (bulk) put_bulk(x.row0 + l_warp, x.hk, w);
            else if (row_at) put_words(row_at, DP / 4, a.D, w);
          } else {
            uint32_t w[DP / 2];
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(o_col(i) + quad + c * 32, r);
              tmem_ld_wait_for(r);
              if (c == DP / 32 - 1) free_o();
              pack(r, f, w + 16 * c);
            }
            if (bulk) put_bulk(x.row0 + l_warp, x.hk, w);
            else if (row_at) put_words(row_at, DP / 2, 2 * a.D, w);
          }
          __syncwarp();
        }
      } else {
        uint8_t* row_at = out_row(x, pos);
        const bool any = __any_sync(0xFFFFFFFFu, row_at != nullptr);
        const int n0 = slot_tiles(x.n(), 0), n1 = slot_tiles(x.n(), 1);
        if (n0 == 0) {
          put_zeros(row_at);
          continue;
        }
        for (int i = 0; i < (n1 > 0 ? 2 : 1) && ok; ++i) {
          if (!mbar_wait_lanes(l_full(i), icount[i] & 1, abort) ||
              !mbar_wait_lanes(o_full(i), icount[i] & 1, abort))
            ok = false;
          ++icount[i];
        }
        if (!ok) break;
        tc_fence_after();
        // o = (a0 O0 + a1 O1) / (a0 l0 + a1 l1), a_i = 2^(m_i - max m)
        const float m0 = sum_m[row], m1 = n1 > 0 ? sum_m[kRows + row] : -INFINITY;
        const float top = fmaxf(m0, m1);
        // A slot whose scores are all -inf has the sum 0, or NaN where one is NaN, which stays.
        const float l0 = sum_l[row], l1 = n1 > 0 ? sum_l[kRows + row] : 0.0f;
        float a0 = m0 == -INFINITY ? (l0 == 0.0f ? 0.0f : 1.0f) : ex2(m0 - top);
        float a1 = m1 == -INFINITY ? (l1 == 0.0f ? 0.0f : 1.0f) : ex2(m1 - top);
        const float sum = a0 * l0 + a1 * l1;
        put_lse(x, row, top, sum);
        const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum) * v_scale;
        a0 *= f;
        a1 *= f;
        const bool spoilt = __any_sync(0xFFFFFFFFu, *dirty != 0);
        __syncwarp();   // together again for the TMEM loads
        if (__builtin_expect(spoilt, 0)) {
          restore(x, 0, pos);
          if (n1 > 0) restore(x, 1, pos);
        }
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t r[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r0[16], r1[16];
            tmem_ld_32x32b_x16(o_col(0) + quad + c * 32 + h * 16, r0);
            if (n1 > 0) tmem_ld_32x32b_x16(o_col(1) + quad + c * 32 + h * 16, r1);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float y = __uint_as_float(r0[e]) * a0;
              if (n1 > 0) y = fmaf(__uint_as_float(r1[e]), a1, y);
              r[16 * h + e] = __float_as_uint(y);
            }
          }
          if (c == DP / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(o_free(0));
              if (n1 > 0) mbar_arrive(o_free(1));
            }
          }
          if (kind == 2) {
            if (any) put_part(x, warp & 3, c, r, 1.0f);
          } else if (row_at && kind == 0) {
            uint32_t w[8];
            pack(r, 1.0f, w);
            put_words(row_at + 32 * c, 8, a.D - 32 * c, w);
          } else if (row_at) {
            uint32_t w[16];
            pack(r, 1.0f, w);
            put_words(row_at + 64 * c, 16, 2 * a.D - 64 * c, w);
          }
          __syncwarp();
        }
        __syncwarp();
      }
    }
    if (lane == 0) tma_store_wait_all();
    if (!ok && lane == 0) record_timeout(abort);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ joining cut units
//
// o = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s - max) over the parts of a
// unit that CTAs shared; a part whose positions the row does not see has lse = -inf.  Blocks go
// by the places where the row of all tiles was cut: the first cut inside a unit
// stands for it.  A warp takes 16 columns of 32 rows, a lane a row, in the
// order in which the parts were written (and have been left in L2).
template <int DP, bool kF16>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedArgs a, int unit_rows) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  constexpr int kChunks = DP / 16;
  const int groups = unit_rows / 32;
  const int w = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int c = 1 + w / (groups * kChunks);
  const int chunk = w % kChunks, group = w / kChunks % groups;
  const int4 lo = *reinterpret_cast<const int4*>(a.info + c * kInfo), hi = *reinterpret_cast<const int4*>(a.info + c * kInfo + 4);
  const int shares = lo.x, hk = lo.w, row0 = hi.x, left = hi.y;
  if (c >= shares) return;
  const uint32_t tile = (uint32_t)lo.y, tiles = (uint32_t)lo.z, total = (uint32_t)hi.z;
  auto start = [&](int k) { return share_begin(total, (uint32_t)k, (uint32_t)shares); };
  const uint32_t s0 = start(c) - tile, s1 = s0 + tiles;
  if (tile == 0 || start(c - 1) > s0) return;   // not inside a unit, or not its first cut
  const int r = 32 * group + lane;              // row of the unit
  const int row = r % kRows, pos = row / a.G, g = row - pos * a.G;
  const int l = (r / kRows) * a.rows_l + pos;
  const bool on = pos < a.rows_l && l < left && 16 * chunk < a.D;
  if (!__any_sync(0xFFFFFFFFu, on)) return;
  float inv_s = 1.0f;
  if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
  // Parts: of share c - 1, which begins in the unit (its first part) or before it
  // (its second), and of those that begin after it: k < shares s1 / total.
  const int k0 = c - 1, k1 = (int)min((uint64_t)shares, ((uint64_t)s1 * shares + total - 1) / total);
  const int first = 2 * k0 + (start(k0) < s0 ? 1 : 0);
  auto lse = [&](int k) { return a.part_lse[(int64_t)(k == k0 ? first : 2 * k) * unit_rows + r]; };
  float top = -INFINITY;
#pragma unroll 8
  for (int k = k0; k < k1; ++k) top = fmaxf(top, lse(k));
  if (top == -INFINITY) top = 0.0f;
  float sum = 0.0f, acc[16] = {};
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
    const float at = lse(k), weight = exp2f(at - top);
    const float4* src = reinterpret_cast<const float4*>(a.part) +
                        (((int64_t)(k == k0 ? first : 2 * k) * groups + group) * (DP / 4) + 4 * chunk) * 32 + lane;
    sum += weight;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 v = src[e * 32];
      if (at == -INFINITY) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // nothing seen
      acc[4 * e] = fmaf(weight, v.x, acc[4 * e]);
      acc[4 * e + 1] = fmaf(weight, v.y, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(weight, v.z, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(weight, v.w, acc[4 * e + 3]);
    }
  }
  if (!on) return;
  const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
  const int64_t off = (int64_t)(row0 + l) * a.o_l + (int64_t)(hk * a.G + g) * a.o_h + 16 * chunk;
#pragma unroll
  for (int e = 0; e < 16; e += 8) {             // eight columns: 16 bytes, or 8 of codes
    if (16 * chunk + e >= a.D) break;
    if (a.s_out) {
      uint32_t c8[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c8[k] = cvt_e4m3x2(acc[e + 2 * k] * f * inv_s, acc[e + 2 * k + 1] * f * inv_s);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + off + e) = make_uint2(c8[0] | (c8[1] << 16), c8[2] | (c8[3] << 16));
    } else {
      uint32_t v8[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v8[k] = cvt16x2(kF16, acc[e + 2 * k] * f, acc[e + 2 * k + 1] * f);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + off + e) = make_uint4(v8[0], v8[1], v8[2], v8[3]);
    }
  }
}

// ------------------------------------------------------------------ host side

struct Plan {
  bool few;         // at most kFewRows rows a unit (paged_few.cu)
  bool shared;      // 256 rows a unit, else 128 rows over even and odd tiles
  bool may_cut;
  int DP, G, rows_l, blocks, ctas;
  int64_t items;
  int unit_rows() const { return few ? kFewRows : shared ? 2 * kRows : kRows; }
  int64_t part_rows() const { return may_cut ? 2ll * ctas * unit_rows() : 0; }
};

// The host knows the sizes but not the lengths.  Units may be cut (by the CTAs, see
// share_out) where the table has room for more tiles than cutting costs.
Plan make_plan(const PagedAttnProblem& p, const PagedCache& c, int sms) {
  Plan x;
  x.DP = p.D <= 64 ? 64 : 128;
  x.G = p.Hq / p.Hkv;
  const int64_t rows = (int64_t)p.max_q * x.G;
  x.few = rows <= kFewRows;
  x.rows_l = (x.few ? kFewRows : kRows) / x.G;
  const int slots = (p.max_q + x.rows_l - 1) / x.rows_l;
  x.shared = slots > 1;
  x.blocks = x.shared ? (slots + 1) / 2 : 1;
  x.items = (int64_t)c.B * p.Hkv * x.blocks;
  const Cutting cost = x.few ? (c.codes ? kCutFewCodes : kCutFew) : x.shared ? kCutShared : kCutSplit;
  const int64_t tiles = ((int64_t)c.cols * c.page_size + kKeys - 1) / kKeys;
  const double total = (double)x.items * (double)tiles;
  x.may_cut = c.B <= kMaxSeqs && (double)tiles > cost.slope * cost.least + cost.plus && total < (double)(1ll << 31);
  int64_t ctas = x.may_cut ? ((int64_t)total + cost.least - 1) / cost.least : x.items;
  if (x.may_cut && ctas < x.items) ctas = x.items;
  x.ctas = (int)(ctas < sms ? ctas : sms);
  return x;
}

template <int DP, bool kF16, bool kCodes, bool kShared>
cudaError_t launch_kernel(const PagedMaps& maps, const PagedArgs& a, int grid, cudaStream_t st) {
  using C = Cfg<DP, kCodes, kShared>;
  auto* k = paged_attention_kernel<DP, kF16, kCodes, kShared>;
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
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k, maps, a)) != cudaSuccess) return e;
  if (a.may_cut && grid > 1) {
    const int unit_rows = kShared ? 2 * kRows : kRows;
    cfg.gridDim = dim3((unsigned)((grid - 1) * (unit_rows / 32 * (DP / 16) / 8)), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, paged_join_kernel<DP, kF16>, a, unit_rows)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DP, bool kF16>
cudaError_t launch_type(const PagedMaps& maps, const PagedArgs& a, bool codes, bool shared, int grid, cudaStream_t st) {
  if (codes)
    return shared ? launch_kernel<DP, kF16, true, true>(maps, a, grid, st) : launch_kernel<DP, kF16, true, false>(maps, a, grid, st);
  return shared ? launch_kernel<DP, kF16, false, true>(maps, a, grid, st) : launch_kernel<DP, kF16, false, false>(maps, a, grid, st);
}

}  // namespace

int64_t paged_attention_ws_floats(const PagedAttnProblem& p, const PagedCache& c, int sms) {
  const Plan x = make_plan(p, c, sms);
  return x.may_cut ? x.part_rows() * (x.DP + 1) + (int64_t)x.ctas * kInfo : 0;
}

cudaError_t launch_paged_attention(const PagedAttnProblem& p, const PagedCache& c, int sms, cudaStream_t st, int* tmap_err) {
  *tmap_err = 0;
  const Plan x = make_plan(p, c, sms);
  PagedMaps maps;
  PagedArgs a;
  std::memset(&maps, 0, sizeof(maps));
  std::memset(&a, 0, sizeof(a));
  a.B = c.B;
  a.T = (int)p.T;
  a.Hkv = p.Hkv;
  a.G = x.G;
  a.D = p.D;
  a.rows_l = x.rows_l;
  a.per = x.shared ? 2 * x.rows_l : x.rows_l;
  a.max_q = p.max_q;
  a.blocks = x.blocks;
  a.items = (int)x.items;
  auto by = [](int64_t d) { return d == 1 ? 0ull : ~0ull / (uint64_t)d + 1; };
  a.by_hkv = by(p.Hkv);
  a.by_page = by(c.page_size);
  a.causal = p.causal;
  a.may_cut = x.may_cut;
  a.pages = c.pages;
  a.page_size = c.page_size;
  a.cols = c.cols;
  a.box = c.page_size & -c.page_size;             // the largest power of two in it
  if (a.box > kKeys) a.box = kKeys;
  a.boxes = kKeys / a.box;
  a.table_stride = c.table_stride;
  a.table = c.table;
  a.q_start = c.q_start;
  a.kv_len = c.kv_len;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  const int64_t cell = c.codes ? 1 : 2;
  a.q = p.q;
  a.q_l = p.qs[0];
  a.q_h = p.qs[1];
  a.v = static_cast<const uint8_t*>(c.v);
  for (int i = 0; i < 3; ++i) a.vs[i] = c.vs[i] * cell;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.s_out = p.s_out;
  a.out = p.out;
  a.o_l = p.os[0];
  a.o_h = p.os[1];
  const int64_t bytes = p.s_out ? 1 : 2;
  auto odd = [&](int64_t stride, int64_t n, int unit) { return n > 1 && stride * bytes % unit != 0; };
  a.wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.D * bytes % 32 == 0 && !odd(a.o_l, p.T, 32) && !odd(a.o_h, p.Hq, 32);
  if (x.may_cut) {
    a.part = p.ws;
    a.part_lse = a.part + x.part_rows() * x.DP;
    a.info = reinterpret_cast<int*>(a.part_lse + x.part_rows());
  }
  const cuuint64_t D = p.D;
  const CUtensorMapDataType type16 = p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  bool ok = true;
  {
    // (dimension, head of the group, token, key head)
    const cuuint64_t dims[4] = {D, (cuuint64_t)x.G, (cuuint64_t)p.T, (cuuint64_t)p.Hkv};
    const int64_t s[3] = {p.qs[1], p.qs[0], p.qs[1] * x.G};
    const cuuint32_t box[4] = {64, (cuuint32_t)x.G, (cuuint32_t)x.rows_l, 1};
    ok = ok && encode(&maps.q, type16, p.q, 4, dims, s, box);
  }
  for (int kv = 0; kv < 2; ++kv) {
    // (dimension, key head, position, page)
    const int64_t* t = kv ? c.vs : c.ks;
    const cuuint64_t dims[4] = {D, (cuuint64_t)p.Hkv, (cuuint64_t)c.page_size, (cuuint64_t)c.pages};
    const int64_t s[3] = {t[2], t[1], t[0]};
    const bool operand = !c.codes || x.few;   // the tensor core reads the copy as it is
    const cuuint32_t box[4] = {!c.codes ? 64 : operand ? 128 : (cuuint32_t)x.DP, 1, (cuuint32_t)a.box, 1};
    ok = ok && encode(kv ? &maps.v : &maps.k, c.codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16, kv ? c.v : c.k, 4, dims, s, box,
                      operand ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                      c.codes ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  }
  a.tma_out = x.shared && 32 % x.G == 0 && p.D * bytes % 16 == 0 && !odd(a.o_l, p.T, 16) && !odd(a.o_h, p.Hq, 16);
  if (a.tma_out) {
    const cuuint64_t dims[4] = {D, (cuuint64_t)x.G, (cuuint64_t)p.T, (cuuint64_t)p.Hkv};
    const int64_t s[3] = {p.os[1], p.os[0], p.os[1] * x.G};
    const cuuint32_t box[4] = {p.s_out ? (cuuint32_t)x.DP : 64, (cuuint32_t)x.G, (cuuint32_t)(32 / x.G), 1};
    ok = ok && encode(&maps.o, p.s_out ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16, p.out, 4, dims, s, box,
                      p.s_out && x.DP == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) {
    *tmap_err = 1;
    return cudaSuccess;
  }
  if (x.few) return launch_paged_few(maps, a, x.DP, p.f16, c.codes, x.ctas, st);
  if (x.DP == 64) return p.f16 ? launch_type<64, true>(maps, a, c.codes, x.shared, x.ctas, st) : launch_type<64, false>(maps, a, c.codes, x.shared, x.ctas, st);
  return p.f16 ? launch_type<128, true>(maps, a, c.codes, x.shared, x.ctas, st) : launch_type<128, false>(maps, a, c.codes, x.shared, x.ctas, st);
}

cudaError_t paged_attention_read_error(cudaStream_t st, uint32_t* err) {
  uint32_t few = 0;
  cudaError_t e = read_paged_error(st, err);
  if (e == cudaSuccess) e = paged_few_read_error(st, &few);
  *err |= few;
  return e;
}

}  // namespace w8
