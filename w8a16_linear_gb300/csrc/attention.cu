// Cross attention on tcgen05: softmax attention of [B, Lq, Hq, D] queries over
// the [B, Lk, Hkv, D] keys and values of an encoder, Hq a multiple of Hkv,
// with key lengths and / or a key mask for each sample.  For each query row
//
//   s_j = scale * sum_d q_d k_jd,   m = max_j s_j,   p_j = exp(s_j - m)
//   o   = sum_j p_j v_j / sum_j p_j                  (0 where no key counts)
//
// in one pass over the keys: with the running maximum m and sum l, a tile of
// keys adds P V to an accumulator that is scaled by exp(m_old - m_new) first.
//
// Work: 4 B Hq Lq Lk D operations on the tensor cores against 2 B Hq Lq D +
// 4 B Hkv Lk D bytes in and 2 (or 1, as codes) B Hq Lq D out.  Long query
// sides are bound by the tensor cores, single tokens by the bytes of K and V.
//
// A CTA (one per SM, persistent over work items) has two slots of 128 query
// rows each.  The query heads that share a key head are packed into the rows
// (row = position * group + head in group), so K and V are read once for all
// of them.  While one slot's scores are in the softmax warps, the tensor core
// works on the other slot's products:
//   S_i = Q_i K_j^T     both operands in 128-byte-swizzled shared memory, by TMA
//   P_i = exp2(S_i c - m)  16-bit, written over S_i in TMEM
//   O_i += P_i V_j      P_i from TMEM, V_j from shared memory (MN-major)
// TMEM: S_0, S_1 (128 columns each), O_0, O_1.  With at most 128 rows
// the two slots take the even and the odd key tiles of the same rows, and the
// epilogue joins them.  Where whole items would leave CTAs without work or with
// uneven work, items are cut along the keys into partial results that a second
// kernel joins.
//
// Roles: warps 0-3 and 4-7 softmax of slot 0 / 1 (a thread per row, so row
// maxima and sums need no shuffles), 8-11 epilogue, 12 and 15 MMA issue of slot 0 / 1,
// 13 TMA loads, 14 clearing of masked V rows (0 * NaN would spoil the products).
//
// Measured (GB300; in a replayed graph / one call among others, where the clocks are
// lower): 4096 queries over 20670 keys, 32 query and 8 key heads of 128:
// 937 / 985 us = 1.48 / 1.41 PFLOP/s, 0.76 / 0.73 of the measured bf16 peak; 41340 queries
// over prompts of 256 to 512 keys, 32 heads, E4M3 out: 277 / 262-277 us = 0.94 / 0.94-0.99 PFLOP/s;
// 8 single tokens over 10335 to 20670 keys: 97 / 90-95 us = 5.2-5.6 TB/s, 0.78 to 0.84 of
// the measured copy, joining included.
// Registers: every form with 256 rows a unit spills (64 dimensions 72 to 148 bytes of
// stores, 128 dimensions 112 to 176, the masked forms most), since the epilogue
// holds a packed row beside 32 columns of the accumulator in its 88 registers.
// What bounds the first is the way from a tile's scores to the next tile's: 512
// cycles of scores, some 1450 of softmax, 256 of P V and four hand-overs
// of about 200, in which both slots together use the tensor core 2048 cycles;
// the second adds the finished rows and the start of each item to that every
// four tiles.
//
// Roundings below 32 bits: P to the inputs' 16-bit type (the tensor core takes
// no wider operand beside 16-bit V; its sum l is taken before the rounding,
// in 32 bits) and the output.  S, O, m and l are binary32.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "attention_common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {

__device__ uint32_t g_attn_err;   // kErrTimeout when a pipeline wait gives up

namespace {

// Samples with lengths of their own whose items may be cut (their tile counts
// are kept in shared memory).
constexpr int kMaxCutSamples = 128;

template <int DP>
struct Cfg {
  static constexpr int kAtoms = DP / 64;
  static constexpr int kTile = kAtoms * kAtom;           // bytes of 128 rows of Q, K or V
  static constexpr int kStages = DP == 128 ? 4 : 6;      // even: see the cleaning warp
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTile;
  static constexpr int kOut = kRing + kStages * kTile;   // 32 rows of 128 bytes for each epilogue warp
  static constexpr int kBound = kOut + 4 * 32 * 128;     // 128 bounds of scores for each softmax warp
  static constexpr int kSum = kBound + 8 * kKeys * 4;    // l[2][128], m[2][128]
  static constexpr int kTab = kSum + 4 * kRows * 4;      // first tile and tiles per item of each sample
  static constexpr int kBar = kTab + (2 * kMaxCutSamples + 2) * 4;
  // full[S], empty[S], clean[S], q_full[2], q_empty[2], s_full[2], p_full[2],
  // o_full[2], l_full[2], o_free[2], p_half[2], drain[2]
  static constexpr int kNumBars = 3 * kStages + 18;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;       // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448, "shared memory budget");
};

constexpr int kThreads = 512;

struct AttnArgs {
  int B, Lq, Lk, Hkv, G, D;
  int rows_l;                 // query positions per slot: 128 / G
  int blocks;                 // query blocks per (sample, key head)
  int items;
  uint64_t by_blocks, by_hkv; // 2^64 / d rounded up, 0 for d = 1
  int cut;                    // CTAs share out tiles, not items
  int groups;                 // entries of the tile table: samples with lengths of their own, else 1
  int q_bmul, k_bmul, v_bmul; // 0 where the samples share one array
  uint32_t q_bytes;           // bytes of one Q atom's box
  float scale_log2;
  const int32_t* kv_len;
  const uint8_t* kv_mask;
  int64_t mask_stride;
  const float* s_out;         // not null: E4M3 output
  void* out;
  int64_t o_b, o_l, o_h;      // element strides of the output
  int wide;                   // output rows are 32-byte aligned and whole multiples of 32 bytes
  int tma_out;                // a warp's 32 rows are whole positions, which one bulk copy can write
  float* part;                // cut: two partial results of each CTA, normalised
  float* part_lse;            // and the log2 of their sums
  uint32_t* tab;              // and the tile table, for the joining kernel
};

struct AttnMaps {
  CUtensorMap q, k, v, o;
};

// One unit of work: a block of query rows of one (sample, key head), and its
// key tiles [t0, t1).
struct Item {
  int b, hk, blk;
  int len;        // keys that may count
  int t0, t1;
  int part;       // the partial result it writes, or -1: its output rows
  __device__ __forceinline__ int n() const { return t1 - t0; }
};

// kLens / kMask: which of the two limits a kernel has.  Each form is compiled
// by itself, without tests of optional pointers, and what limits the keys is read
// by plain volatile loads: an earlier kernel may have written it just before.
__device__ __forceinline__ int load_len(const int32_t* p) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_mask(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// A CTA's units, in the order in which each of its roles goes through them.
//
// Whole items: CTA c takes items c, c + CTAs, ...  Cut items: all key tiles of
// all items stand in one row, of which CTA c takes its even share, so that no
// CTA waits for another one's longer or additional item: it begins and
// ends inside an item, as a rule, and writes partial results for those two.
template <bool kLens>
struct Units {
  const AttnArgs& a;
  const uint32_t* tab;   // cut: first tile of each table entry (groups + 1), then its items' tiles
  uint32_t cur;          // the next item, or cut: the next tile
  int entry = 0;         // cut: its table entry
  int raw = 0;           // whole items with lengths: the next item's

  __device__ __forceinline__ Units(const AttnArgs& args, const uint32_t* table) : a(args), tab(table) {
    cur = a.cut ? begin(blockIdx.x) : blockIdx.x;
    if (!a.cut) ask();
  }
  __device__ __forceinline__ uint32_t begin(uint32_t cta) const {
    return share_begin(tab[a.groups], cta, gridDim.x);
  }
  // The number of keys of the next item's sample, asked for an item ahead: its
  // latency (some 700 cycles) would stand between two items in every role.
  __device__ __forceinline__ void ask() {
    if constexpr (kLens) {
      if (cur < (uint32_t)a.items) raw = load_len(a.kv_len + quotient(quotient((int)cur, a.by_blocks), a.by_hkv));
    }
  }
  __device__ __forceinline__ void place(Item& x, int item) const {
    const int q = quotient(item, a.by_blocks);
    x.blk = item - q * a.blocks;
    x.b = quotient(q, a.by_hkv);
    x.hk = q - x.b * a.Hkv;
  }
  __device__ __forceinline__ bool next(Item& x) {
    x.part = -1;
    if (!a.cut) {
      if (cur >= (uint32_t)a.items) return false;
      place(x, (int)cur);
      x.len = kLens ? min(max(raw, 0), a.Lk) : a.Lk;
      x.t0 = 0;
      x.t1 = (x.len + kKeys - 1) / kKeys;
      cur += gridDim.x;
      ask();
      return true;
    }
    const uint32_t end = begin(blockIdx.x + 1);
    if (cur >= end) return false;
    while (cur >= tab[entry + 1]) ++entry;
    const uint32_t tiles = tab[a.groups + 1 + entry];
    const uint32_t at = cur - tab[entry], item = at / tiles;
    place(x, (int)item);
    x.len = a.Lk;
    if (kLens) {   // a table entry is a sample, and its items are counted from 0
      x.b = entry;
      x.len = min(max(load_len(a.kv_len + entry), 0), a.Lk);
    }
    x.t0 = (int)(at - item * tiles);
    x.t1 = (int)min(tiles, (uint32_t)x.t0 + (end - cur));
    if (x.n() < (int)tiles) x.part = 2 * blockIdx.x + (cur == begin(blockIdx.x) ? 0 : 1);
    cur += (uint32_t)x.n();
    return true;
  }
};

__device__ __forceinline__ void record_timeout(volatile int* abort) {
  *abort = 1;
  atomicOr(&g_attn_err, kErrTimeout);
}

// kShared: both slots work on the same key tiles (256 query rows); otherwise
// they take the even and odd tiles of the same 128 rows.
template <int DP, bool kF16, bool kLens, bool kMask, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    cross_attention_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs a) {
  using C = Cfg<DP>;
  constexpr int S = C::kStages;
  constexpr bool kClean = kLens || kMask;
  constexpr uint32_t kIdescS = make_idesc(kF16 ? 0 : 1, kF16 ? 0 : 1, kRows, kKeys);
  constexpr uint32_t kIdescO = make_idesc(kF16 ? 0 : 1, kF16 ? 0 : 1, kRows, DP) | (1u << 16);  // B is MN-major

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBar;
  auto bar = [&](int k) { return bar0 + 8u * (uint32_t)k; };
  auto full_bar = [&](int s) { return bar(s); };
  auto empty_bar = [&](int s) { return bar(S + s); };
  auto clean_bar = [&](int s) { return bar(2 * S + s); };
  auto q_full = [&](int i) { return bar(3 * S + i); };
  auto q_empty = [&](int i) { return bar(3 * S + 2 + i); };
  auto s_full = [&](int i) { return bar(3 * S + 4 + i); };
  auto p_full = [&](int i) { return bar(3 * S + 6 + i); };
  auto o_full = [&](int i) { return bar(3 * S + 8 + i); };
  auto l_full = [&](int i) { return bar(3 * S + 10 + i); };
  auto o_free = [&](int i) { return bar(3 * S + 12 + i); };
  auto p_half = [&](int i) { return bar(3 * S + 14 + i); };
  auto drain_bar = [&](int i) { return bar(3 * S + 16 + i); };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  float* sum_l = reinterpret_cast<float*>(smem + C::kSum);
  float* sum_m = sum_l + 2 * kRows;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), kShared ? 2 : 1);   // the slots that read the tile
      mbar_init(clean_bar(s), 1);
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
  // no copy writes them, and a warp raises the maxima of all of its rows together, so
  // what an earlier kernel left there would decide on the other rows' roundings.
  if (a.q_bytes < kAtom) {
    for (uint32_t at = a.q_bytes + 16 * threadIdx.x; at < kAtom; at += 16 * kThreads)
#pragma unroll
      for (int k = 0; k < 2 * C::kAtoms; ++k)
        *reinterpret_cast<uint4*>(smem + C::kQ + k * kAtom + at) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const auto s_col = [&](int i) { return tmem + (uint32_t)(i * kKeys); };
  const auto o_col = [&](int i) { return tmem + 256u + (uint32_t)(i * DP); };
  griddep_wait();   // from here on what earlier kernels wrote may be read
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem + C::kTab);
  if (a.cut) {
    // Tiles of each sample's items, and where they begin in the row of all tiles.
    const int per = a.Hkv * a.blocks;
    if constexpr (kLens) {
      for (int b = threadIdx.x; b < a.groups; b += kThreads)
        tab[a.groups + 1 + b] = (uint32_t)(min(max(load_len(a.kv_len + b), 0), a.Lk) + kKeys - 1) / kKeys;
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t sum = 0;
        for (int b = 0; b < a.groups; ++b) {
          tab[b] = sum;
          sum += tab[a.groups + 1 + b] * (uint32_t)per;
        }
        tab[a.groups] = sum;
      }
    } else if (threadIdx.x == 0) {
      tab[2] = (uint32_t)(a.Lk + kKeys - 1) / kKeys;
      tab[0] = 0;
      tab[1] = tab[2] * (uint32_t)a.items;
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int k = threadIdx.x; k < 2 * a.groups + 1; k += kThreads) a.tab[k] = tab[k];
  }

  // Tiles that slot i works on in an item of n tiles.
  const auto slot_tiles = [](int n, int i) { return kShared ? n : (n + 1 - i) / 2; };

  // The stages are one ring in the shared form, which both slots go through
  // tile by tile (K and V in turn), and a ring for each slot in the separate form.  A
  // waiter then sees every filling of its stages: waiting by parity for a
  // filling whose predecessor, another slot's, is still to come would not wait.
  constexpr int R = kShared ? S : S / 2;                              // stages of a ring
  const auto stage_of = [](int i, uint32_t e) { return (kShared ? 0 : i * R) + (int)(e % R); };
  const auto phase_of = [](uint32_t e) { return (e / R) & 1; };

  // The order in which K and V tiles are loaded and cleared:
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

  if (warp >= 12) {
  regs_down<72>();
  if (warp == 13) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      uint32_t filled[2] = {0, 0}, qcount[2] = {0, 0};
      bool ok = true;
      auto load_q = [&](const Item& x, int i) {
        if (!mbar_wait(q_empty(i), (qcount[i] & 1) ^ 1, abort, kWaitLimitNs)) return false;
        ++qcount[i];
        mbar_arrive_expect_tx(q_full(i), C::kAtoms * a.q_bytes);
        const int l0 = (kShared ? 2 * x.blk + i : x.blk) * a.rows_l;
        for (int at = 0; at < C::kAtoms; ++at)
          tma_load_5d(sbase + C::kQ + i * C::kTile + at * kAtom, &maps.q, q_full(i), 64 * at, 0, l0, x.hk, x.b * a.q_bmul);
        return true;
      };
      Units<kLens> units(a, tab);
      Item x;
      while (ok && units.next(x)) {
        if (x.n() == 0) continue;
        bool first = true;
        ok = load_q(x, 0);
        ok = ok && walk(x, [&](bool is_v, int ring, int tile) {
          const uint32_t e = ring ? filled[1]++ : filled[0]++;
          const int st = stage_of(ring, e);
          if (!mbar_wait(empty_bar(st), phase_of(e) ^ 1, abort, kWaitLimitNs)) {
            --filled[ring];
            return false;
          }
          mbar_arrive_expect_tx(full_bar(st), C::kTile);
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_4d(sbase + C::kRing + st * C::kTile + at * kAtom, is_v ? &maps.v : &maps.k, full_bar(st), 64 * at,
                        x.hk, tile * kKeys, x.b * (is_v ? a.v_bmul : a.k_bmul));
          if (kShared && first) {
            first = false;
            return load_q(x, 1);
          }
          return true;
        });
      }
      if (!ok) record_timeout(abort);
      // Every copy must have landed before the block ends.
      volatile int never = 0;
      for (int i = 0; i < (kShared ? 1 : 2); ++i)
        for (uint32_t j = 1; j <= R && j <= filled[i]; ++j) {
          const uint32_t e = filled[i] - j;
          if (!mbar_wait(full_bar(stage_of(i, e)), phase_of(e), &never, kWaitLimitNs)) atomicOr(&g_attn_err, kErrTimeout);
        }
      for (int i = 0; i < 2; ++i)
        if (qcount[i] > 0 && !mbar_wait(q_full(i), (qcount[i] - 1) & 1, &never, kWaitLimitNs))
          atomicOr(&g_attn_err, kErrTimeout);
    }
  } else if (warp == 12 || warp == 15) {
    // ---------------------------------------------------------------- MMA issue
    // One thread for each slot: issuing an MMA takes about as long as the
    // tensor core takes to run it, so one thread for both left it idle half of
    // the time.  A slot's MMAs run in the order of their issue: the scores
    // of tile j + 1 may be written over P of tile j, and when they are complete
    // so is the product of tile j.
    if (elect_one()) {
      const int i = warp == 12 ? 0 : 1;
      uint32_t entry = 0;                        // of this slot's ring
      uint32_t qcount = 0, pcount = 0, icount = 0;
      bool ok = true;
      // Waits for the ring's next entry; returns its stage.  With limits V goes by
      // way of the cleaning warp.  So does K in the separate form, where a stage
      // holds K and V in no fixed order: that warp then sees every filling of
      // a stage before it can be replaced.  In the shared form V has the odd
      // stages (S is even) and the cleaning warp waits for those alone.
      auto take = [&](bool is_v) {
        const uint32_t e = entry++;
        const int st = stage_of(i, e);
        ok = ok && mbar_wait(kClean && (is_v || !kShared) ? clean_bar(st) : full_bar(st), phase_of(e), abort, kWaitLimitNs);
        tc_fence_after();
        return st;
      };
      Units<kLens> units(a, tab);
      Item x;
      while (ok && units.next(x)) {
        const int n = x.n();
        if (n == 0) continue;
        // also by a slot without a tile: its word on Q below belongs to this Q
        ok = mbar_wait(q_full(kShared ? i : 0), qcount & 1, abort, kWaitLimitNs);
        if (!ok) break;
        tc_fence_after();
        for (int j = kShared ? 0 : i; ok && j < n; j += kShared ? 1 : 2) {
          const bool first = j == (kShared ? 0 : i), last = j + (kShared ? 1 : 2) >= n;
          // The slots take turns: a slot's scores are started when the other's
          // are complete.  Left alone the two fall into step, and the tensor core
          // idles while both are in their softmax warps.
          if (kShared && (i == 1 || pcount > 0))
            ok = ok && mbar_wait(s_full(1 - i), (pcount - (1 - i)) & 1, abort, kWaitLimitNs);
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
          if (first) ok = ok && mbar_wait(o_free(i), (icount++ & 1) ^ 1, abort, kWaitLimitNs);   // the epilogue has read O_i
          const uint64_t vd = sw128_mnmajor_desc(sbase + C::kRing + st * C::kTile);
#pragma unroll
          for (int h = 0; h < 2; ++h) {          // 64 keys at a time, as the softmax hands them over
            ok = ok && mbar_wait(h ? p_full(i) : p_half(i), pcount & 1, abort, kWaitLimitNs);
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
      if (!mbar_wait(drain_bar(i), 0, &never, kWaitLimitNs)) atomicOr(&g_attn_err, kErrTimeout);
    }
  } else if (warp == 14) {
    // ---------------------------------------------------------------- masked V rows
    // Keys that do not count have P = 0, but their V may be anything, NaN and
    // infinities included: those rows are cleared before the product.
    if constexpr (kClean) {
      uint32_t seen[2] = {0, 0};
      bool ok = true;
      Units<kLens> units(a, tab);
      Item x;
      while (ok && units.next(x)) {
        // The mask of a tile's keys lane + 32 e, asked for a V tile ahead: its
        // latency would stand before the clearing of every tile.
        uint32_t ahead[4];
        const auto ask = [&](int tile) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = tile * kKeys + 32 * e + lane;
            ahead[e] = 0;
            if (j < x.len) ahead[e] = load_mask(a.kv_mask + x.b * a.mask_stride + j);
          }
        };
        if constexpr (kMask) ask(x.t0);
        ok = walk(x, [&](bool is_v, int ring, int tile) {
          const uint32_t e = ring ? seen[1]++ : seen[0]++;
          const int st = stage_of(ring, e);
          const bool pass = kShared && !is_v;
          // Bit lane of word e: row 32 e + lane of the tile is to be cleared
          // (beyond the array the copy has written zeros).  The mask does not
          // wait for the copy.
          uint32_t word[4] = {0, 0, 0, 0};
          if (is_v) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = tile * kKeys + 32 * e + lane;
              bool off = j < a.Lk && j >= x.len;
              if constexpr (kMask)
                if (j < x.len) off = ahead[e] == 0;
              word[e] = __ballot_sync(0xFFFFFFFFu, off);
            }
            if constexpr (kMask)
              if (tile + 1 < x.t1) ask(tile + 1);
            __syncwarp();   // lanes past the last key took another path
          }
          if (!pass && !mbar_wait_warp(full_bar(st), phase_of(e), abort, kWaitLimitNs)) return false;
          if (word[0] | word[1] | word[2] | word[3]) {
            // eight lanes to a row's 128 bytes, four rows at a time
            uint8_t* v = smem + C::kRing + st * C::kTile + (lane & 7) * 16;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const int r = k + (lane >> 3);
                if (word[e] >> r & 1)
#pragma unroll
                  for (int at = 0; at < C::kAtoms; ++at)
                    *reinterpret_cast<uint4*>(v + at * kAtom + (32 * e + r) * 128) = make_uint4(0, 0, 0, 0);
              }
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
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    float4* bounds = reinterpret_cast<float4*>(smem + C::kBound) + warp * (kKeys / 4);
    uint32_t scount = 0, icount = 0;
    bool ok = true;
    Units<kLens> units(a, tab);
    Item x;
    while (ok && units.next(x)) {
      const int n = slot_tiles(x.n(), i);
      if (n == 0) continue;
      float m = -INFINITY, l = 0.0f;             // m in powers of two: scaled scores
      const auto first_key = [&](int j) { return (x.t0 + (kShared ? j : 2 * j + i)) * kKeys; };
      // The mask of the lane's four keys, asked for a tile ahead.
      uint32_t ahead[4];
      const auto ask = [&](int key0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 4 * lane + e;
          ahead[e] = 0;
          if (key < x.len) ahead[e] = load_mask(a.kv_mask + x.b * a.mask_stride + key);
        }
      };
      if constexpr (kMask) ask(first_key(0));
      for (int j = 0; j < n; ++j) {
        const int key0 = first_key(j);
        // A key's bound is +inf if it counts and -inf if not: the minimum of score
        // and bound is one instruction a score, where bits of a word take three
        // (and NaN scores of keys that do not count are gone too; one of a key that
        // counts becomes +inf, which makes its row NaN all the same).
        // The masking and the rescaling below are kept out of the line of the
        // loop, which is long enough to weigh on the instruction cache.
        const bool masked = kMask || __builtin_expect(key0 + kKeys > x.len, 0);
        if (masked) {
          float bound[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            bound[e] = (kMask ? ahead[e] != 0 : key0 + 4 * lane + e < x.len) ? INFINITY : -INFINITY;
          bounds[lane] = make_float4(bound[0], bound[1], bound[2], bound[3]);
          if constexpr (kMask)
            if (j + 1 < n) ask(first_key(j + 1));
          __syncwarp();   // lanes past the last key took another path
        }
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
        if (masked) {   // a key that does not count has the weight exp2(-inf) = 0
          tmem_ld_wait_for(r[2]);
          tmem_ld_wait_for(r[3]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 b = bounds[8 * c + e / 4];
              r[c][e] = __float_as_uint(fminf(__uint_as_float(r[c][e]), b.x));
              r[c][e + 1] = __float_as_uint(fminf(__uint_as_float(r[c][e + 1]), b.y));
              r[c][e + 2] = __float_as_uint(fminf(__uint_as_float(r[c][e + 2]), b.z));
              r[c][e + 3] = __float_as_uint(fminf(__uint_as_float(r[c][e + 3]), b.w));
            }
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
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a.scale_log2;
        // Scores of slot i are complete, so its product with the previous tile
        // is too (issued before them): O_i may be rescaled here.
        const bool grow = top > m + kLazyMax || (m == -INFINITY && top > m);
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
        const F2 scale = splat(a.scale_log2), minus_m = splat(m == -INFINITY ? 0.0f : -m);
        F2 sums[2] = {splat(0.0f), splat(0.0f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const F2 t = fma2(F2{__uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1])}, scale, minus_m);
            const F2 w = F2{ex2(t.x), ex2(t.y)};
            sums[(e >> 1) & 1] = add2(sums[(e >> 1) & 1], w);
            p[e >> 1] = cvt16x2(kF16, w.x, w.y);
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
      if (!mbar_wait_warp(o_free(i), (icount & 1) ^ 1, abort, kWaitLimitNs)) {
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
    // ---------------------------------------------------------------- epilogue
    regs_down<88>();
    const int row = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const int pos = row / a.G, g = row - pos * a.G, warp_l = 32 / a.G;
    float inv_s = 1.0f;
    if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
    uint32_t icount[2] = {0, 0};
    bool ok = true;

    const int out_kind = a.s_out ? 0 : 1;      // log2 of a value's bytes
    int kind = out_kind;                       // 2 in a unit that writes a partial result
    constexpr int kUnitRows = kShared ? 2 * kRows : kRows;
    // 32 columns (chunk c) of a partial result.  Four columns of a warp's 32 rows
    // stand together, so that a store is 512 bytes in one piece: row by row they
    // were 4096 sectors a slot, and 16 us.
    auto put_part = [&](const Item& x, int row_group, int c, const uint32_t (&r)[32], float f) {
      float4* dst = reinterpret_cast<float4*>(a.part) + (((int64_t)x.part * (kUnitRows / 32) + row_group) * (DP / 4) + 8 * c) * 32 + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dst[k * 32] = make_float4(__uint_as_float(r[4 * k]) * f, __uint_as_float(r[4 * k + 1]) * f,
                                  __uint_as_float(r[4 * k + 2]) * f, __uint_as_float(r[4 * k + 3]) * f);
    };
    // Where this thread's row (position l) starts, or null.
    auto out_row = [&](const Item& x, int l) -> uint8_t* {
      if (pos >= a.rows_l || l >= a.Lq) return nullptr;
      return static_cast<uint8_t*>(a.out) + ((x.b * a.o_b + l * a.o_l + (int64_t)(x.hk * a.G + g) * a.o_h) << kind);
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
    // for each 128 bytes of a row (64 for codes of small heads).  Stores from the
    // rows' own threads, a sector each, kept the load/store path busy for some
    // 4000 cycles a slot, and the other roles' barriers and the next slot's rows behind them.
    auto put_bulk = [&](const Item& x, int l_warp, const uint32_t* w) {
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
        if (lane == 0 && l_warp < a.Lq) {
          tma_store_5d(&maps.o, stage_at, kind == 0 ? 0 : 64 * h, 0, l_warp, x.hk, x.b);
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

    if (kLens && a.cut) {   // samples without keys have no tiles: their rows are zeros
      for (int b = 0; b < a.groups; ++b) {
        if (tab[a.groups + 1 + b] != 0) continue;
        Item x;
        for (int it = blockIdx.x; it < a.Hkv * a.blocks; it += gridDim.x) {
          x.blk = it % a.blocks;
          x.hk = it / a.blocks;
          x.b = b;
          for (int i = 0; i < (kShared ? 2 : 1); ++i) put_zeros(out_row(x, (kShared ? 2 * x.blk + i : x.blk) * a.rows_l + pos));
        }
      }
    }
    Units<kLens> units(a, tab);
    Item x;
    while (ok && units.next(x)) {
      kind = x.part < 0 ? out_kind : 2;
      if constexpr (kShared) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int l = (2 * x.blk + i) * a.rows_l + pos;
          uint8_t* row_at = out_row(x, l);
          const int l_warp = l - pos + (warp & 3) * warp_l;   // position of the warp's first row
          if (x.n() == 0) {
            put_zeros(row_at);
            continue;
          }
          if (!mbar_wait_warp(l_full(i), icount[i] & 1, abort, kWaitLimitNs) ||
              !mbar_wait_warp(o_full(i), icount[i] & 1, abort, kWaitLimitNs)) {
            ok = false;
            break;
          }
          ++icount[i];
          tc_fence_after();
          const float sum = sum_l[i * kRows + row];
          const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
          put_lse(x, i * kRows + row, sum_m[i * kRows + row], sum);
          __syncwarp();   // together again for the TMEM loads
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
            if (a.tma_out) put_bulk(x, l_warp, w);
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
            if (a.tma_out) put_bulk(x, l_warp, w);
            else if (row_at) put_words(row_at, DP / 2, 2 * a.D, w);
          }
          __syncwarp();
        }
      } else {
        const int l = x.blk * a.rows_l + pos;
        uint8_t* row_at = out_row(x, l);
        const bool any = __any_sync(0xFFFFFFFFu, row_at != nullptr);
        const int n0 = slot_tiles(x.n(), 0), n1 = slot_tiles(x.n(), 1);
        if (n0 == 0) {
          put_zeros(row_at);
          continue;
        }
        for (int i = 0; i < (n1 > 0 ? 2 : 1) && ok; ++i) {
          if (!mbar_wait_warp(l_full(i), icount[i] & 1, abort, kWaitLimitNs) ||
              !mbar_wait_warp(o_full(i), icount[i] & 1, abort, kWaitLimitNs))
            ok = false;
          ++icount[i];
        }
        if (!ok) break;
        tc_fence_after();
        // o = (a0 O0 + a1 O1) / (a0 l0 + a1 l1), a_i = 2^(m_i - max m)
        const float m0 = sum_m[row], m1 = n1 > 0 ? sum_m[kRows + row] : -INFINITY;
        const float top = fmaxf(m0, m1);
        float a0 = m0 == -INFINITY ? 0.0f : ex2(m0 - top), a1 = m1 == -INFINITY ? 0.0f : ex2(m1 - top);
        const float l0 = sum_l[row], l1 = n1 > 0 ? sum_l[kRows + row] : 0.0f;
        const float sum = a0 * l0 + a1 * l1;
        put_lse(x, row, top, sum);
        const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        a0 *= f;
        a1 *= f;
        __syncwarp();   // together again for the TMEM loads
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

// ------------------------------------------------------------------ joining cut items
//
// o = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s - max) over the parts of an
// item that CTAs shared; a part without counting keys has lse = -inf.  Blocks go
// by the places where the row of all tiles was cut: the first cut inside an item
// stands for it.  A warp takes 16 columns of 32 rows, a lane a row, in the
// order in which the parts were written (and have been left in L2).
template <int DP, bool kF16>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnArgs a, int ctas, int unit_rows) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  constexpr int kChunks = DP / 16;
  const int groups = unit_rows / 32;
  const int w = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int c = 1 + w / (groups * kChunks);
  const int chunk = w % kChunks, group = w / kChunks % groups;
  const uint32_t total = a.tab[a.groups];
  auto start = [&](int k) { return share_begin(total, (uint32_t)k, (uint32_t)ctas); };
  const uint32_t p = start(c);
  if (p >= total) return;
  int entry = 0;   // the table entry that holds tile p
  for (int k = lane + 1; k <= a.groups; k += 32) entry += a.tab[k] <= p;
  for (int o = 16; o >= 1; o /= 2) entry += __shfl_xor_sync(0xFFFFFFFFu, entry, o);
  const uint32_t tiles = a.tab[a.groups + 1 + entry], base = a.tab[entry];
  const uint32_t item = (p - base) / tiles, s0 = base + item * tiles, s1 = s0 + tiles;
  if (p == s0 || start(c - 1) > s0) return;   // not inside an item, or not its first cut
  const int q = quotient((int)item, a.by_blocks);
  const int blk = (int)item - q * a.blocks;
  int b = quotient(q, a.by_hkv);
  const int hk = q - b * a.Hkv;
  if (a.groups > 1) b = entry;
  const int r = 32 * group + lane;            // row of the unit
  const int row = r % kRows, pos = row / a.G, g = row - pos * a.G;
  const int l = (unit_rows > kRows ? 2 * blk + r / kRows : blk) * a.rows_l + pos;
  const bool on = pos < a.rows_l && l < a.Lq && 16 * chunk < a.D;
  if (!__any_sync(0xFFFFFFFFu, on)) return;
  float inv_s = 1.0f;
  if (a.s_out) inv_s = __frcp_rn(ld_f32(a.s_out));
  // Parts: of CTA c - 1, which begins in the item (its first unit) or before it
  // (its second), and of those that begin after it: k < ctas s1 / total.  A CTA
  // without a share (fewer tiles than CTAs) has none.
  const int k0 = c - 1, k1 = (int)min((uint64_t)ctas, ((uint64_t)s1 * ctas + total - 1) / total);
  const int first = 2 * k0 + (start(k0) < s0 ? 1 : 0);
  auto lse = [&](int k) {
    return total >= (uint32_t)ctas || start(k) < start(k + 1) ? a.part_lse[(int64_t)(k == k0 ? first : 2 * k) * unit_rows + r] : -INFINITY;
  };
  float top = -INFINITY;
#pragma unroll 8
  for (int k = k0; k < k1; ++k) top = fmaxf(top, lse(k));
  if (top == -INFINITY) top = 0.0f;
  float sum = 0.0f, acc[16] = {};
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
    const float weight = exp2f(lse(k) - top);
    const float4* src = reinterpret_cast<const float4*>(a.part) +
                        (((int64_t)(k == k0 ? first : 2 * k) * groups + group) * (DP / 4) + 4 * chunk) * 32 + lane;
    sum += weight;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 v = src[e * 32];
      if (weight == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // a part that nobody wrote
      acc[4 * e] = fmaf(weight, v.x, acc[4 * e]);
      acc[4 * e + 1] = fmaf(weight, v.y, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(weight, v.z, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(weight, v.w, acc[4 * e + 3]);
    }
  }
  if (!on) return;
  const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
  const int64_t off = b * a.o_b + l * a.o_l + (int64_t)(hk * a.G + g) * a.o_h + 16 * chunk;
#pragma unroll
  for (int e = 0; e < 16; e += 8) {           // eight columns: 16 bytes, or 8 of codes
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
  bool shared;      // 256 rows a unit, else 128 rows over even and odd tiles
  bool cut;
  int DP, G, rows_l, blocks, ctas, groups;
  int64_t items;
  int unit_rows() const { return shared ? 2 * kRows : kRows; }
  int64_t part_rows() const { return cut ? 2ll * ctas * unit_rows() : 0; }
};

// Whole items or cut ones: by an estimate of either's time, in tiles of one CTA.
// Cutting costs the writing and joining of the partial results and a second
// launch: with 256 rows a unit the time of about 10 tiles (2 x 2000 queries,
// 2000 keys, 16 heads: 65 us whole in 32 tiles, 74 cut in 27), with 128 rows about 8,
// and the tiles get slower as more CTAs load at once (one token, 8 key heads: 2048 keys
// 19.9 whole, 14.5 cut, 1024 keys 12.8 and 13.1; 8 tokens: 2048 keys 21.6 and 23.8 us).
Plan make_plan(const AttnProblem& p, bool lens, int sms) {
  Plan x;
  x.DP = p.D <= 64 ? 64 : 128;
  x.G = p.Hq / p.Hkv;
  x.rows_l = kRows / x.G;
  const int slots = (p.Lq + x.rows_l - 1) / x.rows_l;
  x.shared = slots > 1;
  x.blocks = x.shared ? (slots + 1) / 2 : 1;
  x.items = (int64_t)p.B * p.Hkv * x.blocks;
  const int64_t tiles = (p.Lk + kKeys - 1) / kKeys, total = x.items * tiles;
  x.groups = lens ? p.B : 1;
  const int64_t share = (total + sms - 1) / sms, least = x.shared ? 8 : 4;   // tiles a CTA
  const int64_t per = share > least ? share : least;
  const int64_t rounds = (x.items + sms - 1) / sms;
  double whole = (double)(rounds * tiles), mine = (double)per;
  // Lengths of their own (by half of the range on average) make whole items
  // uneven, the more so the fewer a CTA has.
  if (lens && p.B > 1) {
    whole *= rounds < 8 ? 1.0 : 0.8;
    mine *= 0.8;
  }
  const double cut = x.shared ? mine + 10.0 : 1.4 * mine + 8.0;
  x.cut = cut < whole && total < (1ll << 31) && x.groups <= kMaxCutSamples;
  x.ctas = (int)(x.cut ? (total + per - 1) / per : x.items < sms ? x.items : sms);
  return x;
}

template <int DP, bool kF16, bool kLens, bool kMask, bool kShared>
cudaError_t launch_kernel(const AttnMaps& maps, const AttnArgs& a, int grid, cudaStream_t st) {
  auto* k = cross_attention_kernel<DP, kF16, kLens, kMask, kShared>;
  static std::atomic<uint64_t> allowed{0};   // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP>::kAlloc);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<DP>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k, maps, a)) != cudaSuccess) return e;
  if (a.cut && grid > 1) {
    const int unit_rows = kShared ? 2 * kRows : kRows;
    cfg.gridDim = dim3((unsigned)((grid - 1) * (unit_rows / 32 * (DP / 16) / 8)), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, attention_join_kernel<DP, kF16>, a, grid, unit_rows)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DP, bool kF16, bool kLens, bool kMask>
cudaError_t launch_rows(const AttnMaps& maps, const AttnArgs& a, bool shared, int grid, cudaStream_t st) {
  return shared ? launch_kernel<DP, kF16, kLens, kMask, true>(maps, a, grid, st)
                : launch_kernel<DP, kF16, kLens, kMask, false>(maps, a, grid, st);
}

template <int DP, bool kF16>
cudaError_t launch_type(const AttnMaps& maps, const AttnArgs& a, bool shared, int grid, cudaStream_t st) {
  if (a.kv_mask)
    return a.kv_len ? launch_rows<DP, kF16, true, true>(maps, a, shared, grid, st)
                    : launch_rows<DP, kF16, false, true>(maps, a, shared, grid, st);
  return a.kv_len ? launch_rows<DP, kF16, true, false>(maps, a, shared, grid, st)
                  : launch_rows<DP, kF16, false, false>(maps, a, shared, grid, st);
}

}  // namespace

int64_t cross_attention_ws_floats(const AttnProblem& p, int sms) {
  // With lengths and without them items are cut by different rules, and the tile
  // table has other sizes: enough for both, since the lengths come with the call.
  int64_t most = 0;
  for (int lens = 0; lens < 2; ++lens) {
    const Plan x = make_plan(p, lens != 0, sms);
    const int64_t n = x.cut ? x.part_rows() * (x.DP + 1) + 2 * x.groups + 1 : 0;
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_cross_attention(const AttnProblem& p, int sms, cudaStream_t st, int* tmap_err) {
  *tmap_err = 0;
  const Plan x = make_plan(p, p.kv_len != nullptr, sms);
  AttnMaps maps;
  AttnArgs a;
  std::memset(&maps, 0, sizeof(maps));
  std::memset(&a, 0, sizeof(a));
  a.B = p.B;
  a.Lq = p.Lq;
  a.Lk = p.Lk;
  a.Hkv = p.Hkv;
  a.G = x.G;
  a.D = p.D;
  a.rows_l = x.rows_l;
  a.blocks = x.blocks;
  a.cut = x.cut;
  a.groups = x.groups;
  a.items = (int)x.items;
  auto by = [](int d) { return d == 1 ? 0ull : ~0ull / (uint64_t)d + 1; };
  a.by_blocks = by(x.blocks);
  a.by_hkv = by(p.Hkv);
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.kv_len = p.kv_len;
  a.kv_mask = p.kv_mask;
  a.mask_stride = p.mask_stride;
  a.s_out = p.s_out;
  a.out = p.out;
  a.o_b = p.os[0];
  a.o_l = p.os[1];
  a.o_h = p.os[2];
  {
    const int64_t bytes = p.s_out ? 1 : 2;
    auto odd = [&](int64_t stride, int n) { return n > 1 && stride * bytes % 32 != 0; };
    a.wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.D * bytes % 32 == 0 && !odd(a.o_b, p.B) &&
             !odd(a.o_l, p.Lq) && !odd(a.o_h, p.Hq);
  }
  if (x.cut) {
    a.part = p.ws;
    a.part_lse = a.part + x.part_rows() * x.DP;
    a.tab = reinterpret_cast<uint32_t*>(a.part_lse + x.part_rows());
  }
  a.q_bytes = (uint32_t)(x.G * x.rows_l * 128);
  const cuuint64_t D = p.D, B = p.B;
  a.q_bmul = p.qs[0] != 0;
  a.k_bmul = p.ks[0] != 0;
  a.v_bmul = p.vs[0] != 0;
  const CUtensorMapDataType type16 = p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  bool ok = true;
  {
    // (dimension, head of the group, position, key head, sample)
    const cuuint64_t dims[5] = {D, (cuuint64_t)x.G, (cuuint64_t)p.Lq, (cuuint64_t)p.Hkv, a.q_bmul ? B : 1};
    const int64_t s[4] = {p.qs[2], p.qs[1], p.qs[2] * x.G, p.qs[0]};
    const cuuint32_t box[5] = {64, (cuuint32_t)x.G, (cuuint32_t)x.rows_l, 1, 1};
    ok = ok && encode(&maps.q, type16, p.q, 5, dims, s, box);
  }
  for (int kv = 0; kv < 2; ++kv) {
    const int64_t* t = kv ? p.vs : p.ks;
    // without keys nothing is loaded: the map needs an array all the same
    const cuuint64_t dims[4] = {D, (cuuint64_t)p.Hkv, (cuuint64_t)(p.Lk ? p.Lk : 1), (kv ? a.v_bmul : a.k_bmul) ? B : 1};
    const int64_t s[3] = {t[2], t[1], t[0]};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)kKeys, 1};
    ok = ok && encode(kv ? &maps.v : &maps.k, type16, !p.Lk ? p.q : kv ? p.v : p.k, 4, dims, s, box);
  }
  {
    const int64_t bytes = p.s_out ? 1 : 2;
    auto odd = [&](int64_t stride, int n) { return n > 1 && stride * bytes % 16 != 0; };
    a.tma_out = x.shared && 32 % x.G == 0 && p.D * bytes % 16 == 0 && !odd(a.o_b, p.B) && !odd(a.o_l, p.Lq) && !odd(a.o_h, p.Hq);
    if (a.tma_out) {
      const cuuint64_t dims[5] = {D, (cuuint64_t)x.G, (cuuint64_t)p.Lq, (cuuint64_t)p.Hkv, B};
      const int64_t s[4] = {p.os[2], p.os[1], p.os[2] * x.G, p.os[0]};
      const cuuint32_t box[5] = {p.s_out ? (cuuint32_t)x.DP : 64, (cuuint32_t)x.G, (cuuint32_t)(32 / x.G), 1, 1};
      ok = ok && encode(&maps.o, p.s_out ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16, p.out, 5, dims, s, box,
                        p.s_out && x.DP == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    }
  }
  if (!ok) {
    *tmap_err = 1;
    return cudaSuccess;
  }
  const int grid = x.ctas;
  if (x.DP == 64) return p.f16 ? launch_type<64, true>(maps, a, x.shared, grid, st) : launch_type<64, false>(maps, a, x.shared, grid, st);
  return p.f16 ? launch_type<128, true>(maps, a, x.shared, grid, st) : launch_type<128, false>(maps, a, x.shared, grid, st);
}

cudaError_t attention_read_error(cudaStream_t st, uint32_t* err) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(err, g_attn_err, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *err) {
    e = cudaMemcpyToSymbolAsync(g_attn_err, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace w8
