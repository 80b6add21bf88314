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
// epilogue joins them; few items are further split along the keys into partial
// results that a second kernel joins.
//
// Roles: warps 0-3 and 4-7 softmax of slot 0 / 1 (a thread per row, so row
// maxima and sums need no shuffles), 8-11 epilogue, 12 MMA issue, 13 TMA
// loads, 14 clearing of masked V rows (0 * NaN would spoil the products).
//
// Roundings below 32 bits: P to the inputs' 16-bit type (the tensor core takes
// no wider operand beside 16-bit V; its sum l is taken before the rounding,
// in 32 bits) and the output.  S, O, m and l are binary32.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {

__device__ uint32_t g_attn_err;   // kErrTimeout when a pipeline wait gives up

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

template <int DP>
struct Cfg {
  static constexpr int kAtoms = DP / 64;
  static constexpr int kTile = kAtoms * kAtom;           // bytes of 128 rows of Q, K or V
  static constexpr int kStages = DP == 128 ? 4 : 6;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTile;
  static constexpr int kSum = kRing + kStages * kTile;   // l[2][128], m[2][128]
  static constexpr int kBar = kSum + 4 * kRows * 4;
  // full[S], empty[S], clean[S], q_full[2], q_empty[2], s_full[2], p_full[2],
  // o_full[2], l_full[2], o_free[2], drain
  static constexpr int kNumBars = 3 * kStages + 15;
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
  int splits;                 // parts of the key axis
  int items;
  int q_bmul, k_bmul, v_bmul; // 0 where the samples share one array
  uint32_t q_bytes;           // bytes of one Q atom's box
  float scale_log2;
  const int32_t* kv_len;
  const uint8_t* kv_mask;
  int64_t mask_stride;
  const float* s_out;         // not null: E4M3 output
  void* out;
  int64_t o_b, o_l, o_h;      // element strides of the output
  float* part;                // splits > 1: normalised partial outputs, then their log2 sums
  float* part_lse;
};

struct AttnMaps {
  CUtensorMap q, k, v;
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
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

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
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

// One work item: a block of query rows of one (sample, key head), and the key
// tiles [t0, t1) of one split.
struct Item {
  int b, hk, blk, split;
  int len;        // keys that may count
  int t0, t1;
  __device__ __forceinline__ int n() const { return t1 - t0; }
};

__device__ __forceinline__ Item decode(const AttnArgs& a, int it) {
  Item x;
  x.blk = it % a.blocks;
  it /= a.blocks;
  x.split = it % a.splits;
  it /= a.splits;
  x.hk = it % a.Hkv;
  x.b = it / a.Hkv;
  x.len = a.Lk;
  if (a.kv_len) x.len = min(max(__ldg(a.kv_len + x.b), 0), a.Lk);
  const int tiles = (x.len + kKeys - 1) / kKeys;
  x.t0 = (int)((int64_t)tiles * x.split / a.splits);
  x.t1 = (int)((int64_t)tiles * (x.split + 1) / a.splits);
  return x;
}

__device__ __forceinline__ void record_timeout(volatile int* abort) {
  *abort = 1;
  atomicOr(&g_attn_err, kErrTimeout);
}

// kShared: both slots work on the same key tiles (256 query rows); otherwise
// they take the even and odd tiles of the same 128 rows.
template <int DP, bool kF16, bool kMask, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    cross_attention_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs a) {
  using C = Cfg<DP>;
  constexpr int S = C::kStages;
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
  const uint32_t drain_bar = bar(3 * S + 14);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  float* sum_l = reinterpret_cast<float*>(smem + C::kSum);
  float* sum_m = sum_l + 2 * kRows;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(clean_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 4);
      mbar_init(o_full(i), 1);
      mbar_init(l_full(i), 4);
      mbar_init(o_free(i), 4);
    }
    mbar_init(drain_bar, 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const auto s_col = [&](int i) { return tmem + (uint32_t)(i * kKeys); };
  const auto o_col = [&](int i) { return tmem + 256u + (uint32_t)(i * DP); };
  griddep_wait();   // from here on what earlier kernels wrote may be read

  // Tiles that slot i works on in an item of n tiles.
  const auto slot_tiles = [](int n, int i) { return kShared ? n : (n + 1 - i) / 2; };

  // The order in which K and V tiles pass through the ring, which the loader,
  // the cleaner and the MMA issue all follow:
  //   shared:   K0 V0 K1 V1 ...
  //   separate: K(0) K(1) | V(0) K(2) V(1) K(3) | ...   (tiles of the item)
  const auto walk = [&](const Item& x, auto&& f) {
    const int n = x.n();
    if constexpr (kShared) {
      for (int j = 0; j < n; ++j)
        if (!f(false, x.t0 + j) || !f(true, x.t0 + j)) return false;
    } else {
      for (int j = 0; j < 2 && j < n; ++j)
        if (!f(false, x.t0 + j)) return false;
      for (int j = 0; j < n; ++j)
        if (!f(true, x.t0 + j) || (j + 2 < n && !f(false, x.t0 + j + 2))) return false;
    }
    return true;
  };

  if (warp == 13) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0, issued = 0, qcount[2] = {0, 0};
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
      for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
        const Item x = decode(a, it);
        if (x.n() == 0) continue;
        bool first = true;
        ok = load_q(x, 0);
        ok = ok && walk(x, [&](bool is_v, int tile) {
          if (!mbar_wait(empty_bar(st), ph ^ 1, abort, kWaitLimitNs)) return false;
          mbar_arrive_expect_tx(full_bar(st), C::kTile);
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_4d(sbase + C::kRing + st * C::kTile + at * kAtom, is_v ? &maps.v : &maps.k, full_bar(st), 64 * at,
                        x.hk, tile * kKeys, x.b * (is_v ? a.v_bmul : a.k_bmul));
          ++issued;
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
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
      for (int j = 0; j < S && (uint32_t)j < issued; ++j) {
        const uint32_t l = issued - 1 - j;
        if (!mbar_wait(full_bar((int)(l % S)), (l / S) & 1, &never, kWaitLimitNs)) atomicOr(&g_attn_err, kErrTimeout);
      }
      for (int i = 0; i < 2; ++i)
        if (qcount[i] > 0 && !mbar_wait(q_full(i), (qcount[i] - 1) & 1, &never, kWaitLimitNs))
          atomicOr(&g_attn_err, kErrTimeout);
    }
  } else if (warp == 12) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      uint32_t qcount = 0;                       // items whose Q has been waited for
      uint32_t pcount[2] = {0, 0};               // tiles of each slot whose P has been waited for
      uint32_t ocount[2] = {0, 0};               // items of each slot whose O has been started
      bool ok = true;
      // Waits for the stage at the ring's head, and takes it.  With masks the
      // cleaning warp passes every stage first, K's too: a stage can then not
      // be refilled before that warp has seen it.
      auto take = [&](int& s) {
        s = st;
        ok = ok && mbar_wait(kMask ? clean_bar(st) : full_bar(st), ph, abort, kWaitLimitNs);
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
        tc_fence_after();
      };
      auto qk = [&](int i, int s) {
        const uint32_t qa = sbase + C::kQ + (kShared ? i : 0) * C::kTile, ka = sbase + C::kRing + s * C::kTile;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          mma_f16(s_col(i), sw128_kmajor_desc(qa + (k >> 2) * kAtom + 32 * (k & 3)),
                  sw128_kmajor_desc(ka + (k >> 2) * kAtom + 32 * (k & 3)), kIdescS, k != 0);
        mma_commit(s_full(i));
      };
      auto pv = [&](int i, int s, bool first) {
        const uint32_t va = sbase + C::kRing + s * C::kTile;
        ok = ok && mbar_wait(p_full(i), pcount[i] & 1, abort, kWaitLimitNs);
        ++pcount[i];
        if (first) {   // the epilogue has read the accumulator's previous item
          ok = ok && mbar_wait(o_free(i), (ocount[i] & 1) ^ 1, abort, kWaitLimitNs);
          ++ocount[i];
        }
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_f16_tmem_a(o_col(i), s_col(i) + 8 * k, sw128_mnmajor_desc(va + 2048 * k), kIdescO, !first || k != 0);
      };
      auto wait_q = [&](int i, uint32_t count) {
        ok = ok && mbar_wait(q_full(i), count & 1, abort, kWaitLimitNs);
        tc_fence_after();
      };
      auto next_item = [&](int it) {             // the next item with any keys, or items
        for (it += gridDim.x; it < a.items; it += gridDim.x)
          if (decode(a, it).n() > 0) break;
        return min(it, a.items);
      };
      int it = next_item((int)blockIdx.x - (int)gridDim.x);
      if constexpr (kShared) {
        // The scores of the next tile -- of the next item after an item's last
        // tile -- are issued behind each slot's product with V, so that the
        // tensor core has the other slot's work while a softmax runs.
        bool have = false;
        int s = 0;
        while (ok && it < a.items) {
          const int n = decode(a, it).n();
          const int nx = next_item(it);
          const int n_next = nx < a.items ? decode(a, nx).n() : 0;
          if (!have) {
            take(s);
            for (int i = 0; i < 2 && ok; ++i) {
              wait_q(i, qcount);
              if (!ok) break;
              qk(i, s);
              if (n == 1) mma_commit(q_empty(i));
            }
            mma_commit(empty_bar(s));
          }
          for (int j = 0; j < n && ok; ++j) {
            const bool more = j + 1 < n;
            int vs, ks = 0;
            take(vs);
            for (int i = 0; i < 2 && ok; ++i) {
              pv(i, vs, j == 0);
              if (!ok) break;
              if (i == 1) mma_commit(empty_bar(vs));
              if (!more) mma_commit(o_full(i));
              if (more || n_next > 0) {
                if (i == 0) take(ks);
                if (!more) wait_q(i, qcount + 1);
                if (!ok) break;
                qk(i, ks);
                if (more ? j + 2 == n : n_next == 1) mma_commit(q_empty(i));
                if (i == 1) mma_commit(empty_bar(ks));
              }
            }
          }
          ++qcount;
          have = n_next > 0;
          it = nx;
        }
      } else {
        while (ok && it < a.items) {
          const int n = decode(a, it).n();
          int s = 0;
          wait_q(0, qcount);
          ++qcount;
          for (int j = 0; j < 2 && j < n && ok; ++j) {
            take(s);
            if (!ok) break;
            qk(j, s);
            mma_commit(empty_bar(s));
          }
          for (int j = 0; j < n && ok; ++j) {
            take(s);
            if (!ok) break;
            pv(j & 1, s, j < 2);
            if (!ok) break;
            mma_commit(empty_bar(s));
            if (j + 2 >= n) mma_commit(o_full(j & 1));
            if (j + 2 < n) {
              take(s);
              if (!ok) break;
              qk(j & 1, s);
              mma_commit(empty_bar(s));
            }
          }
          mma_commit(q_empty(0));
          it = next_item(it);
        }
      }
      if (!ok) record_timeout(abort);
      // All MMAs complete before TMEM is freed.
      mma_commit(drain_bar);
      volatile int never = 0;
      if (!mbar_wait(drain_bar, 0, &never, kWaitLimitNs)) atomicOr(&g_attn_err, kErrTimeout);
    }
  } else if (warp == 14) {
    // ---------------------------------------------------------------- masked V rows
    // Keys that do not count have P = 0, but their V may be anything, NaN and
    // infinities included: those rows are cleared before the product.
    if constexpr (kMask) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
        const Item x = decode(a, it);
        ok = walk(x, [&](bool is_v, int tile) {
          if (!mbar_wait_warp(full_bar(st), ph, abort, kWaitLimitNs)) return false;
          if (is_v) {
            uint8_t* v = smem + C::kRing + st * C::kTile;
            bool wrote = false;
            for (int r = lane; r < kKeys; r += 32) {
              const int j = tile * kKeys + r;
              // beyond the array the copy has written zeros
              if (j >= a.Lk || (j < x.len && (!a.kv_mask || a.kv_mask[x.b * a.mask_stride + j]))) continue;
              wrote = true;
              for (int at = 0; at < C::kAtoms; ++at)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  *reinterpret_cast<uint4*>(v + at * kAtom + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            }
            if (wrote) fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(clean_bar(st));
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
          return true;
        });
      }
      if (!ok && lane == 0) record_timeout(abort);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int i = warp >> 2;                     // slot
    const int row = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t scount = 0, icount = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
      const Item x = decode(a, it);
      const int n = slot_tiles(x.n(), i);
      if (n == 0) continue;
      float m = -INFINITY, l = 0.0f;             // m in powers of two: scaled scores
      for (int j = 0; j < n; ++j) {
        const int key0 = (x.t0 + (kShared ? j : 2 * j + i)) * kKeys;
        // Bit lane of word e: key 4 lane + e of the tile counts.
        bool masked = false;
        uint32_t word[4] = {~0u, ~0u, ~0u, ~0u};
        if (kMask || key0 + kKeys > x.len) {
          masked = true;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 4 * lane + e;
            bool on = key < x.len;
            if (kMask && a.kv_mask && on) on = a.kv_mask[x.b * a.mask_stride + key] != 0;
            word[e] = __ballot_sync(0xFFFFFFFFu, on);
          }
        }
        if (!mbar_wait_warp(s_full(i), scount & 1, abort, kWaitLimitNs)) {
          ok = false;
          break;
        }
        ++scount;
        tc_fence_after();
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(s_col(i) + quad + c * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float v = __uint_as_float(r[e]);
            if (masked && !((word[e & 3] >> (8 * c + (e >> 2))) & 1)) v = -INFINITY;
            top = fmaxf(top, v);
          }
        }
        top *= a.scale_log2;
        // Scores of slot i are complete, so its product with the previous tile
        // is too (issued before them): O_i may be rescaled here.
        const bool grow = top > m + kLazyMax || (m == -INFINITY && top > m);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float m_new = fmaxf(m, top);
          if (j > 0) {
            const float f = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
            l *= f;
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(o_col(i) + quad + c * 32, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st_32x32b_x32(o_col(i) + quad + c * 32, r);
            }
          }
          m = m_new;
        }
        const float ms = m == -INFINITY ? 0.0f : m;
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32], p[16];
          tmem_ld_32x32b_x32(s_col(i) + quad + c * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0 = ex2(fmaf(__uint_as_float(r[e]), a.scale_log2, -ms));
            float p1 = ex2(fmaf(__uint_as_float(r[e + 1]), a.scale_log2, -ms));
            if (masked) {
              if (!((word[e & 3] >> (8 * c + (e >> 2))) & 1)) p0 = 0.0f;
              if (!((word[(e + 1) & 3] >> (8 * c + (e >> 2))) & 1)) p1 = 0.0f;
            }
            l0 += p0;
            l1 += p1;
            p[e >> 1] = cvt16x2(kF16, p0, p1);
          }
          // 32 scores leave 16 columns of P over the first half of S_i; chunk
          // c's are read before: columns 16 c .. 16 c + 15 lie at or below 32 c
          tmem_st_32x32b_x16(s_col(i) + quad + c * 16, p);
        }
        l += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i));
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
  } else if (warp < 12) {
    // ---------------------------------------------------------------- epilogue
    const int row = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const int pos = row / a.G, g = row - pos * a.G;
    float inv_s = 1.0f;
    if (a.s_out) inv_s = __frcp_rn(__ldg(a.s_out));
    uint32_t icount[2] = {0, 0};
    bool ok = true;

    // 32 columns of this thread's row, scaled, to the output or the partials.
    auto put = [&](const Item& x, int l, int c, const float (&v)[32]) {
      if (pos >= a.rows_l || l >= a.Lq) return;
      const int d0 = 32 * c;
      if (a.splits > 1) {
        const int64_t at = (((int64_t)x.split * a.B + x.b) * a.Hkv + x.hk) * ((int64_t)a.Lq * a.G) + (int64_t)l * a.G + g;
        float4* dst = reinterpret_cast<float4*>(a.part + at * DP + d0);
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        return;
      }
      const int64_t off = x.b * a.o_b + l * a.o_l + (int64_t)(x.hk * a.G + g) * a.o_h + d0;
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        if (d0 + e >= a.D) break;
        if (a.s_out) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = cvt_e4m3x2(v[e + 2 * k] * inv_s, v[e + 2 * k + 1] * inv_s);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + off + e) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = cvt16x2(kF16, v[e + 2 * k], v[e + 2 * k + 1]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + off + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    auto put_lse = [&](const Item& x, int l, float m, float sum) {
      if (a.splits == 1 || pos >= a.rows_l || l >= a.Lq) return;
      const int64_t at = (((int64_t)x.split * a.B + x.b) * a.Hkv + x.hk) * ((int64_t)a.Lq * a.G) + (int64_t)l * a.G + g;
      a.part_lse[at] = sum == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) + log2f(sum);
    };

    for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
      const Item x = decode(a, it);
      if constexpr (kShared) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int l = (2 * x.blk + i) * a.rows_l + pos;
          if (x.n() == 0) {
            float z[32] = {};
            for (int c = 0; c < DP / 32; ++c) put(x, l, c, z);
            put_lse(x, l, 0.0f, 0.0f);
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
          put_lse(x, l, sum_m[i * kRows + row], sum);
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(o_col(i) + quad + c * 32, r);
            tmem_ld_wait();
            if (c == DP / 32 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(o_free(i));
            }
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = f == 0.0f ? 0.0f : __uint_as_float(r[e]) * f;
            put(x, l, c, v);
          }
        }
      } else {
        const int l = x.blk * a.rows_l + pos;
        const int n0 = slot_tiles(x.n(), 0), n1 = slot_tiles(x.n(), 1);
        if (n0 == 0) {
          float z[32] = {};
          for (int c = 0; c < DP / 32; ++c) put(x, l, c, z);
          put_lse(x, l, 0.0f, 0.0f);
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
        put_lse(x, l, top, sum);
        const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        a0 *= f;
        a1 *= f;
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t r0[32], r1[32];
          tmem_ld_32x32b_x32(o_col(0) + quad + c * 32, r0);
          if (n1 > 0) tmem_ld_32x32b_x32(o_col(1) + quad + c * 32, r1);
          tmem_ld_wait();
          if (c == DP / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(o_free(0));
              if (n1 > 0) mbar_arrive(o_free(1));
            }
          }
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v[e] = f == 0.0f ? 0.0f : __uint_as_float(r0[e]) * a0;
            if (n1 > 0 && f != 0.0f) v[e] = fmaf(__uint_as_float(r1[e]), a1, v[e]);
          }
          put(x, l, c, v);
        }
      }
    }
    if (!ok && lane == 0) record_timeout(abort);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ joining the splits
//
// o = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s - max), a warp per output row;
// a split without keys has lse = -inf.  Its bytes are splits x 4 D a row, which
// the kernel before has just left in L2.
template <bool kF16>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnArgs a, int DP) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.B * a.Hkv * a.Lq * a.G;   // (b, hk, l, g)
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const float inv_s = a.s_out ? __frcp_rn(__ldg(a.s_out)) : 1.0f;
  float top = -INFINITY;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.part_lse[s * rows + r]);
  if (top == -INFINITY) top = 0.0f;
  float sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const bool on = 4 * lane < a.D;
  for (int s = 0; s < a.splits; ++s) {
    const float w = exp2f(a.part_lse[s * rows + r] - top);
    if (w == 0.0f) continue;
    sum += w;
    if (on) {
      const float4 v = *reinterpret_cast<const float4*>(a.part + (s * rows + r) * DP + 4 * lane);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  if (!on) return;
  const float f = sum == 0.0f ? 0.0f : __frcp_rn(sum);
  const int g = (int)(r % a.G);
  int64_t q = r / a.G;
  const int64_t l = q % a.Lq;
  q /= a.Lq;
  const int hk = (int)(q % a.Hkv);
  const int64_t off = (q / a.Hkv) * a.o_b + l * a.o_l + (int64_t)(hk * a.G + g) * a.o_h + 4 * lane;
  acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
  if (a.s_out)
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + off) =
        cvt_e4m3x2(acc.x * inv_s, acc.y * inv_s) | (cvt_e4m3x2(acc.z * inv_s, acc.w * inv_s) << 16);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + off) =
        make_uint2(cvt16x2(kF16, acc.x, acc.y), cvt16x2(kF16, acc.z, acc.w));
}

// ------------------------------------------------------------------ host side

// A dimension of one entry, or one that the samples share, gets the stride
// of the dimension before it: its own is never used, and may be anything.
bool encode(CUtensorMap* map, bool f16, const void* base, int rank, const cuuint64_t* dims, const int64_t* strides,
            const cuuint32_t* box) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  cuuint64_t st[4];
  for (int i = 0; i + 1 < rank; ++i) st[i] = dims[i + 1] > 1 ? (cuuint64_t)strides[i] * 2 : i ? st[i - 1] : dims[0] * 2;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
            const_cast<void*>(base), dims, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
  bool shared;      // 256 rows a work item, else 128 rows over even and odd tiles
  int DP, G, rows_l, blocks, splits;
  int64_t items;
};

Plan make_plan(const AttnProblem& p, int sms) {
  Plan x;
  x.DP = p.D <= 64 ? 64 : 128;
  x.G = p.Hq / p.Hkv;
  x.rows_l = kRows / x.G;
  const int slots = (p.Lq + x.rows_l - 1) / x.rows_l;
  x.shared = slots > 1;
  x.blocks = x.shared ? (slots + 1) / 2 : 1;
  const int64_t base = (int64_t)p.B * p.Hkv * x.blocks;
  const int tiles = (p.Lk + kKeys - 1) / kKeys;
  const int per = x.shared ? 2 : 4;    // fewest tiles of a split that are worth its partials
  int64_t s = base >= sms ? 1 : sms / base;
  if (s > tiles / per) s = tiles / per;
  x.splits = s < 1 ? 1 : (int)s;
  x.items = base * x.splits;
  return x;
}

template <int DP, bool kF16, bool kMask, bool kShared>
cudaError_t launch_kernel(const AttnMaps& maps, const AttnArgs& a, int grid, cudaStream_t st) {
  auto* k = cross_attention_kernel<DP, kF16, kMask, kShared>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP>::kAlloc);
  if (e != cudaSuccess) return e;
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
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.B * a.Hkv * a.Lq * a.G;
    cfg.gridDim = dim3((unsigned)((rows + 3) / 4), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, attention_join_kernel<kF16>, a, DP)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DP, bool kF16>
cudaError_t launch_type(const AttnMaps& maps, const AttnArgs& a, bool mask, bool shared, int grid, cudaStream_t st) {
  if (mask)
    return shared ? launch_kernel<DP, kF16, true, true>(maps, a, grid, st) : launch_kernel<DP, kF16, true, false>(maps, a, grid, st);
  return shared ? launch_kernel<DP, kF16, false, true>(maps, a, grid, st) : launch_kernel<DP, kF16, false, false>(maps, a, grid, st);
}

}  // namespace

int64_t cross_attention_ws_floats(const AttnProblem& p, int sms) {
  const Plan x = make_plan(p, sms);
  if (x.splits == 1) return 0;
  return (int64_t)x.splits * p.B * p.Hq * p.Lq * (x.DP + 1);
}

cudaError_t launch_cross_attention(const AttnProblem& p, int sms, cudaStream_t st, int* tmap_err) {
  *tmap_err = 0;
  const Plan x = make_plan(p, sms);
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
  a.splits = x.splits;
  a.items = (int)x.items;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.kv_len = p.kv_len;
  a.kv_mask = p.kv_mask;
  a.mask_stride = p.mask_stride;
  a.s_out = p.s_out;
  a.out = p.out;
  a.o_b = p.os[0];
  a.o_l = p.os[1];
  a.o_h = p.os[2];
  a.part = p.ws;
  a.part_lse = p.ws + (int64_t)x.splits * p.B * p.Hq * p.Lq * x.DP;   // not used with one split
  a.q_bytes = (uint32_t)(x.G * x.rows_l * 128);
  const cuuint64_t D = p.D, B = p.B;
  a.q_bmul = p.qs[0] != 0;
  a.k_bmul = p.ks[0] != 0;
  a.v_bmul = p.vs[0] != 0;
  bool ok = true;
  {
    // (dimension, head of the group, position, key head, sample)
    const cuuint64_t dims[5] = {D, (cuuint64_t)x.G, (cuuint64_t)p.Lq, (cuuint64_t)p.Hkv, a.q_bmul ? B : 1};
    const int64_t s[4] = {p.qs[2], p.qs[1], p.qs[2] * x.G, p.qs[0]};
    const cuuint32_t box[5] = {64, (cuuint32_t)x.G, (cuuint32_t)x.rows_l, 1, 1};
    ok = ok && encode(&maps.q, p.f16, p.q, 5, dims, s, box);
  }
  for (int kv = 0; kv < 2; ++kv) {
    const int64_t* t = kv ? p.vs : p.ks;
    // without keys nothing is loaded: the map needs an array all the same
    const cuuint64_t dims[4] = {D, (cuuint64_t)p.Hkv, (cuuint64_t)(p.Lk ? p.Lk : 1), (kv ? a.v_bmul : a.k_bmul) ? B : 1};
    const int64_t s[3] = {t[2], t[1], t[0]};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)kKeys, 1};
    ok = ok && encode(kv ? &maps.v : &maps.k, p.f16, !p.Lk ? p.q : kv ? p.v : p.k, 4, dims, s, box);
  }
  if (!ok) {
    *tmap_err = 1;
    return cudaSuccess;
  }
  const bool mask = p.kv_len || p.kv_mask;
  const int grid = (int)(x.items < sms ? x.items : sms);
  if (x.DP == 64) return p.f16 ? launch_type<64, true>(maps, a, mask, x.shared, grid, st) : launch_type<64, false>(maps, a, mask, x.shared, grid, st);
  return p.f16 ? launch_type<128, true>(maps, a, mask, x.shared, grid, st) : launch_type<128, false>(maps, a, mask, x.shared, grid, st);
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
