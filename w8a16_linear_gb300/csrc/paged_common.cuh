// What the kernels of attention over a paged cache share: their arguments, the
// sequences and units of work, how those are shared out, and their error word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace w8 {
namespace {
__device__ uint32_t g_paged_err;   // kErrTimeout when a pipeline wait gives up (one of each translation unit)
}

// Sequences that are kept in shared memory; of more, units are never cut.
constexpr int kMaxSeqs = 256;
constexpr int kThreads = 512;
constexpr int kInfo = 8;           // words about a share for the joining kernel

// Words of kState: how the work is shared out, and where this CTA begins.
enum { kShares, kBegin, kEnd, kZeros, kAtB, kAtHk, kAtBlk, kAtTile };

struct PagedArgs {
  int B, T, Hkv, G, D;
  int rows_l;                 // tokens per slot: 128 / G
  int per;                    // tokens of a unit
  int max_q;
  int blocks;                 // units of a sequence and key head at most
  int items;                  // B * Hkv * blocks
  uint64_t by_hkv, by_page;          // 2^64 / d rounded up, 0 for d = 1
  int causal;
  int may_cut;
  int pages, page_size, cols, box, boxes;   // rows of a copy, copies of a tile and 64 dimensions
  int64_t table_stride;
  const int32_t *table, *q_start, *kv_len;
  const float *k_scale, *v_scale;           // of codes
  const void* q;              // queries and their element strides, where a kernel reads them itself
  int64_t q_l, q_h;
  const uint8_t* v;           // the cache and its strides in bytes, for values that are cleared in shared memory
  int64_t vs[3];
  float scale_log2;
  const float* s_out;         // not null: E4M3 output
  void* out;
  int64_t o_l, o_h;           // element strides of the output
  int wide;                   // output rows are 32-byte aligned and whole multiples of 32 bytes
  int tma_out;                // a warp's 32 rows are whole tokens, which one bulk copy can write
  float* part;                // may_cut: two partial results of each CTA, normalised
  float* part_lse;            // and the log2 of their sums
  int* info;                  // and kInfo words about each share
};

struct PagedMaps {
  CUtensorMap q, k, v, o;
};

struct Cutting {
  int least;
  float slope, plus;
};

// What is known of a sequence: the row of its first token, its tokens (of those
// that are worked on), the position of the first and the positions that there are.
struct Seq {
  int row0, tokens, base, len;
};

__device__ __forceinline__ Seq load_seq(const PagedArgs& a, int b) {
  int q0, q1;
  if (a.q_start) {
    q0 = min(max(ld_i32(a.q_start + b), 0), a.T);
    q1 = min(max(ld_i32(a.q_start + b + 1), q0), a.T);
  } else {
    q0 = a.T / a.B * b;
    q1 = q0 + a.T / a.B;
  }
  const int kv = min(max(ld_i32(a.kv_len + b), 0), 1 << 30);
  return Seq{q0, min(q1 - q0, a.max_q), kv - (q1 - q0), min(kv, a.cols * a.page_size)};
}

// One unit of work (or the part of one that is a CTA's).
struct Item {
  int b, hk;
  int row0, left; // row of its first token; its tokens
  int pos0;       // position of the first
  int limit;      // positions that some token sees, and that the first sees
  int lim0;
  int len;
  int t0, t1;     // key tiles
  int part;       // the partial result it writes, or -1: its output rows
  __device__ __forceinline__ int n() const { return t1 - t0; }
};

// Positions that the tokens before token `end` of a sequence see, `base` being the first one's.
__device__ __forceinline__ int seen(const PagedArgs& a, int base, int len, int end) {
  return a.causal ? min(max(base + end, 0), len) : len;
}

// The sequences in the order of their numbers of units, the most first (all threads).
__device__ __forceinline__ void order_units(const PagedArgs& a, const Seq* seqs, uint16_t* order) {
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const int mine = (seqs[b].tokens + a.per - 1) / a.per;
    int before = 0;
    for (int k = 0; k < a.B; ++k) {
      const int n = (seqs[k].tokens + a.per - 1) / a.per;
      before += n > mine || (n == mine && k < b);
    }
    order[before] = (uint16_t)b;
  }
}

// A CTA's units, in the order in which each of its roles goes through them.
//
// Whole units: block by block from the last (the longest, where causal), of the
// sequences that have it, and dealt out to the CTAs to and fro.  (Counted over all blocks
// of all sequences instead, prompts of 539 to 1077 tokens gave one CTA 30 tiles
// where 18 are the average.)
struct Units {
  const PagedArgs& a;
  const Seq* seqs;            // in shared memory, or null
  const uint32_t* tiles;
  const uint16_t* order;
  uint32_t cur, end;          // cut: the next tile and the share's end
  int b, hk, blk, t;          // cut: where that tile is; whole: the block
  uint32_t begin;
  int count;                  // whole: sequences that have the block
  int at, turn;               // the next unit among theirs; whether the last round went back
  bool cut;

  __device__ __forceinline__ Units(const PagedArgs& args, const Seq* s, const uint32_t* tl, const volatile int* st,
                                   const uint16_t* ord)
      : a(args), seqs(s), tiles(tl), order(ord) {
    cut = a.may_cut && st[kShares] > 0;
    if (cut) {
      begin = cur = (uint32_t)st[kBegin];
      end = (uint32_t)st[kEnd];
      b = st[kAtB], hk = st[kAtHk], blk = st[kAtBlk], t = st[kAtTile];
    } else {
      blk = a.blocks - 1;
      count = seqs ? 0 : a.B;
      at = (int)blockIdx.x;
      turn = 0;
    }
  }
  // The unit of block `at`; false where the sequence has no such tokens.
  __device__ __forceinline__ bool fill(Item& x, int at) const {
    const Seq s = seqs ? seqs[x.b] : load_seq(a, x.b);
    const int first = at * a.per;
    if (first >= s.tokens) return false;
    x.left = min(a.per, s.tokens - first);
    x.row0 = s.row0 + first;
    x.pos0 = s.base + first;
    x.len = s.len;
    x.limit = seen(a, s.base, s.len, first + x.left);
    x.lim0 = seen(a, s.base, s.len, first + 1);
    x.t0 = 0;
    x.t1 = (x.limit + kKeys - 1) / kKeys;
    return true;
  }
  __device__ __forceinline__ bool next(Item& x) {
    x.part = -1;
    if (!cut) {
      while (blk >= 0) {
        while (seqs && count < a.B && seqs[order[count]].tokens > blk * a.per) ++count;
        const int n = count * a.Hkv;
        if (at >= n) {
          at -= n;
          --blk;
          continue;
        }
        const int k = quotient(at, a.by_hkv);
        x.b = seqs ? order[k] : k;
        x.hk = at - k * a.Hkv;
        at += turn ? 1 + 2 * (int)blockIdx.x : 2 * ((int)gridDim.x - (int)blockIdx.x) - 1;
        turn ^= 1;
        if (fill(x, blk)) return true;   // without a table of sequences one may lack the block
      }
      return false;
    }
    if (cur >= end) return false;
    for (;;) {                                        // the unit that holds tile `cur`
      x.b = b;
      if (!fill(x, blk)) {
        blk = 0;
        if (++hk == a.Hkv) {
          hk = 0;
          while (++b < a.B - 1 && tiles[b] == 0) {
          }
        }
      } else if (x.t1 == 0) {
        ++blk;
      } else {
        break;
      }
    }
    x.hk = hk;
    const int all = x.t1;
    x.t0 = t;
    x.t1 = (int)min((uint32_t)all, (uint32_t)t + (end - cur));
    if (x.n() < all) x.part = 2 * blockIdx.x + (cur == begin ? 0 : 1);
    cur += (uint32_t)x.n();
    t = x.t1;
    if (t == all) {
      t = 0;
      ++blk;
    }
    return true;
  }
};

namespace {
__device__ __forceinline__ void record_timeout(volatile int* abort) {
  *abort = 1;
  atomicOr(&g_paged_err, kErrTimeout);
}
}

// mbar_wait that asks some times before it lets the thread sleep: a sleeping
// thread is woken late, and every hand-over between roles is on a tile's way.
__device__ __forceinline__ bool mbar_wait_awake(uint32_t bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int k = 0; k < 256; ++k)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, kWaitLimitNs);
}

// Whether a half of one of the words (two 16-bit values each) is not finite.
template <bool kF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t kExp = kF16 ? 0x7C007C00u : 0x7F807F80u, kOne = kF16 ? 0x04000400u : 0x00800080u;
  return ((w & kExp) + kOne) & 0x80008000u;
}

// The word with its values that are not finite replaced by zeros.
template <bool kF16>
__device__ __forceinline__ uint32_t finite(uint32_t w) {
  const uint32_t bad = not_finite<kF16>(w);
  return w & ~((bad >> 15 & 1u ? 0xFFFFu : 0u) | (bad >> 31 ? 0xFFFF0000u : 0u));
}

// The same for four E4M3 codes: those of NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// V rows of a tile in shared memory that not every row of a unit sees (one warp;
// eight lanes to a row's 128 bytes): rows `to` and on, which none sees, are cleared up to
// the end of their copy of `box` rows (the copies behind it wrote zeros); of rows from .. to - 1 the
// values that are not finite.  Whether this lane met one of
// those.  It stands between the tile's copy and its product: 16 rows' loads are under way at a time.
template <bool kF16, bool kCells8, int kAtoms>
__device__ __forceinline__ bool clear_rows(uint8_t* tile, int lane, int from, int to, int box) {
  const auto bad_of = [](const uint4& w) {
    return kCells8 ? nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w)
                   : not_finite<kF16>(w.x) | not_finite<kF16>(w.y) | not_finite<kF16>(w.z) | not_finite<kF16>(w.w);
  };
  const auto kept = [](uint32_t w) { return kCells8 ? w & ~((nan_codes(w) >> 7) * 0xFFu) : finite<kF16>(w); };
  uint8_t* v = tile + (lane & 7) * 16;
  const int sub = lane >> 3;
  bool bad = false;
  from = max(from, 0);
#pragma unroll 1
  for (int r0 = from & ~3; r0 < min(to, kKeys); r0 += 16) {
    uint4 w[4][kAtoms];
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int at = 0; at < kAtoms; ++at)   // rows of 128 at most: the tile's last ones stand for those behind it
        w[k][at] = *reinterpret_cast<const uint4*>(v + at * kAtom + min(r0 + 4 * k + sub, kKeys - 1) * 128);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + 4 * k + sub;
#pragma unroll
      for (int at = 0; at < kAtoms; ++at)
        if (r >= from && r < to) any |= bad_of(w[k][at]);
    }
    if (__builtin_expect(any != 0, 0)) {
      bad = true;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + 4 * k + sub;
#pragma unroll
        for (int at = 0; at < kAtoms; ++at)
          if (r >= from && r < min(to, kKeys))
            *reinterpret_cast<uint4*>(v + at * kAtom + r * 128) =
                make_uint4(kept(w[k][at].x), kept(w[k][at].y), kept(w[k][at].z), kept(w[k][at].w));
      }
    }
  }
#pragma unroll 2
  for (int r = max(to, 0) + sub; r < min((max(to, 0) + box - 1) & -box, kKeys); r += 4)
#pragma unroll
    for (int at = 0; at < kAtoms; ++at) *reinterpret_cast<uint4*>(v + at * kAtom + r * 128) = make_uint4(0, 0, 0, 0);
  return bad;
}

// A quarter (32 rows) of a tile of E4M3 codes, rows of DP bytes, to 16-bit values in
// the 128-byte swizzle, exactly: binary16 where kHalf, else bfloat16; one warp, 16
// codes of a lane at a time.  Rows from `from` and `to` on as in clear_rows.
template <int DP, bool kHalf>
__device__ __forceinline__ bool convert_rows(const uint8_t* raw, uint8_t* tile, int quarter, int lane, int from, int to) {
  constexpr int kLanes = DP / 16;            // lanes of a row
  const uint8_t* src = raw + quarter * 32 * DP + lane * 16;
  const int c16 = lane % kLanes;
  const bool edge = from < quarter * 32 + 32;
  bool bad = false;
#pragma unroll 4
  for (int k = 0; k < kLanes; ++k) {         // 32 / kLanes rows at a time
    const int r = quarter * 32 + k * (32 / kLanes) + lane / kLanes;
    const uint4 c = *reinterpret_cast<const uint4*>(src + k * 512);
    const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      w[q] = cvt_e4m3x2_to_f16x2((uint16_t)(cw[q >> 1] >> (16 * (q & 1))));
      if (!kHalf) {
        float lo, hi;
        f16x2_to_f32(w[q], lo, hi);
        w[q] = cvt_bf16x2(lo, hi);
      }
    }
    if (edge && r >= from) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (r < to && not_finite<kHalf>(w[q])) bad = true;
        w[q] = r < to ? finite<kHalf>(w[q]) : 0;
      }
    }
    // Eight lanes' first stores have eight different places modulo 128 bytes (a
    // row's two halves begin with the other one of their two).
    uint8_t* at = tile + (c16 >> 2) * kAtom + r * 128;
    const int turn = c16 >> 2 & 1, ch = 2 * (c16 & 3);
    *reinterpret_cast<uint4*>(at + (((ch + turn) ^ (r & 7)) << 4)) =
        turn ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(at + (((ch + 1 - turn) ^ (r & 7)) << 4)) =
        turn ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(w[4], w[5], w[6], w[7]);
  }
  return bad;
}

// How the work is shared out, from the sequences in shared memory (all threads).
// Whole units or even shares of their tiles: by an estimate of either's time, in
// tiles of one CTA, where cutting (the writing and joining of partial results) costs
// `plus` tiles, tiles are `slope` times slower since more CTAs load at once, and a
// share has `least` tiles.
__device__ __forceinline__ void share_out(const PagedArgs& a, const Seq* seqs, uint32_t* tiles, uint32_t* first, int* state,
                                          const Cutting cost) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = warp; b < a.B; b += kThreads / 32) {
    const Seq s = seqs[b];
    uint32_t sum = 0;
    for (int f = lane * a.per; f < s.tokens; f += 32 * a.per)
      sum += (uint32_t)(seen(a, s.base, s.len, min(f + a.per, s.tokens)) + kKeys - 1) / kKeys;
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (lane == 0) tiles[b] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t total = 0, items = 0, longest = 0, zeros = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      uint32_t mine = 0;
      if (b < a.B) {
        const Seq s = seqs[b];
        mine = tiles[b] * (uint32_t)a.Hkv;
        const uint32_t units = (uint32_t)(s.tokens + a.per - 1) / (uint32_t)a.per;
        items += units * (uint32_t)a.Hkv;
        if (units) {
          longest = max(longest, (uint32_t)(seen(a, s.base, s.len, s.tokens) + kKeys - 1) / kKeys);
          zeros |= seen(a, s.base, s.len, min(a.per, s.tokens)) == 0;
        }
      }
      uint32_t to = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
        if (lane >= o) to += v;
      }
      if (b < a.B) first[b] = total + to - mine;
      total += __shfl_sync(0xFFFFFFFFu, to, 31);
    }
    __syncwarp();   // first[] is read by other lanes than wrote it, and shuffles do not order memory
    items = __reduce_add_sync(0xFFFFFFFFu, items);
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    zeros = __reduce_or_sync(0xFFFFFFFFu, zeros);
    const uint32_t ctas = gridDim.x;
    const uint32_t share = max((total + ctas - 1) / ctas, (uint32_t)cost.least);
    const float whole = items <= ctas ? (float)longest : fmaxf((float)longest, (float)total / (float)ctas + 0.5f * (float)longest);
    const float mine = cost.slope * (float)share + cost.plus;
    const uint32_t shares = mine < whole ? (total + share - 1) / share : 0;
    int at_b = 0, at_hk = 0, at_blk = 0, at_t = 0, at_tiles = 0;
    if (blockIdx.x < shares) {
      const uint32_t p = share_begin(total, blockIdx.x, shares);
      int n = 0;                               // sequences that begin at tile p or before it, the first aside
      for (int k = lane + 1; k < a.B; k += 32) n += first[k] <= p;
      at_b = __reduce_add_sync(0xFFFFFFFFu, n);
      const Seq s = seqs[at_b];
      const uint32_t at = p - first[at_b];
      at_hk = (int)(at / tiles[at_b]);
      uint32_t rest = at - (uint32_t)at_hk * tiles[at_b];
      for (int blk0 = 0;; blk0 += 32) {        // its unit, 32 at a time
        const int f = (blk0 + lane) * a.per;
        const uint32_t mine_t = f < s.tokens ? (uint32_t)(seen(a, s.base, s.len, min(f + a.per, s.tokens)) + kKeys - 1) / kKeys : 0;
        uint32_t to = mine_t;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
          if (lane >= o) to += v;
        }
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, to > rest);
        if (over) {
          const int l = __ffs(over) - 1;
          at_blk = blk0 + l;
          at_t = (int)(rest - __shfl_sync(0xFFFFFFFFu, to - mine_t, l));
          at_tiles = (int)__shfl_sync(0xFFFFFFFFu, mine_t, l);
          break;
        }
        rest -= __shfl_sync(0xFFFFFFFFu, to, 31);
        if ((blk0 + 32) * a.per >= s.tokens) break;   // never: the sequence has the tile
      }
      if (lane == 0) {
        int* info = a.info + blockIdx.x * kInfo;
        const int f = at_blk * a.per;
        info[1] = at_t;
        info[2] = at_tiles;
        info[3] = at_hk;
        info[4] = s.row0 + f;
        info[5] = min(a.per, s.tokens - f);
        info[6] = (int)total;
      }
    }
    if (lane == 0) {
      a.info[blockIdx.x * kInfo] = (int)shares;
      state[kShares] = (int)shares;
      state[kBegin] = (int)(blockIdx.x < shares ? share_begin(total, blockIdx.x, shares) : total);
      state[kEnd] = (int)(blockIdx.x < shares ? share_begin(total, blockIdx.x + 1, shares) : total);
      state[kZeros] = (int)zeros;
      state[kAtB] = at_b;
      state[kAtHk] = at_hk;
      state[kAtBlk] = at_blk;
      state[kAtTile] = at_t;
    }
  }
}

// A CTA's units, in the order in which each of its roles goes through them: as
// Units has them, where a sequence is one unit of each key head.
struct WholeUnits {
  const PagedArgs& a;
  const Seq* seqs;            // in shared memory, or null
  const uint32_t* tiles;
  uint32_t cur, end, step;    // the next item, or cut: the next tile and the share's end
  int b, hk, t;               // cut: where that tile is
  int part;
  bool cut;

  __device__ __forceinline__ WholeUnits(const PagedArgs& args, const Seq* s, const uint32_t* tl, const volatile int* st,
                                        const uint16_t* = nullptr)
      : a(args), seqs(s), tiles(tl) {
    cut = a.may_cut && st[kShares] > 0;
    part = 2 * blockIdx.x;
    cur = cut ? (uint32_t)st[kBegin] : blockIdx.x;
    end = cut ? (uint32_t)st[kEnd] : (uint32_t)a.items;
    if (cut) b = st[kAtB], hk = st[kAtHk], t = st[kAtTile];
  }
  __device__ __forceinline__ bool next(Item& x) {
    Seq s;
    do {
      if (cur >= end) return false;
      if (!cut) {
        b = quotient((int)cur, a.by_hkv);
        hk = (int)cur - b * a.Hkv;
        cur += gridDim.x;
      }
      s = seqs ? seqs[b] : load_seq(a, b);
    } while (s.tokens == 0);   // where units are cut it is one with tiles
    x.b = b;
    x.hk = hk;
    x.left = s.tokens;
    x.row0 = s.row0;
    x.pos0 = s.base;
    x.len = s.len;
    x.limit = seen(a, s.base, s.len, s.tokens);
    x.lim0 = seen(a, s.base, s.len, 1);
    x.t0 = 0;
    x.t1 = (x.limit + kKeys - 1) / kKeys;
    x.part = -1;
    if (cut) {
      const int all = x.t1;
      x.t0 = t;
      x.t1 = (int)min((uint32_t)all, (uint32_t)t + (end - cur));
      if (x.n() < all) x.part = part;
      part = 2 * blockIdx.x + 1;
      cur += (uint32_t)x.n();
      t = x.t1;
      if (t == all) {
        t = 0;
        if (++hk == a.Hkv) {
          hk = 0;
          while (++b < a.B - 1 && tiles[b] == 0) {
          }
        }
      }
    }
    return true;
  }
};

// The sequences to shared memory and, where units may be cut, how the work is
// shared out (see share_out): by one warp, since a sequence is one unit of a key head.
__device__ __forceinline__ void share_out_whole(const PagedArgs& a, Seq* seqs, uint32_t* tiles, uint32_t* first, int* state,
                                                const Cutting cost) {
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
  const uint32_t share = max((total + ctas - 1) / ctas, (uint32_t)cost.least);
  const float even = (float)total / (float)ctas;
  const float whole = units <= ctas ? (float)longest : fmaxf((float)longest, even + 0.5f * (float)longest);
  const bool cut = cost.slope * (float)share + cost.plus < whole;
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

// Reads and clears this translation unit's error word.
namespace {
inline cudaError_t read_paged_error(cudaStream_t st, uint32_t* err) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(err, g_paged_err, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *err) {
    e = cudaMemcpyToSymbolAsync(g_paged_err, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}
}  // namespace

// Units of few rows: cutting costs the time of 8 tiles, or of 12 of E4M3 cells, which are half
// the bytes and take less.  Measured, 32/8 heads of 128, us with 5 / 8 / 12: one token over
// 1024 and 1536 positions 12.0 / 11.8 / 11.8 and 12.9 / 12.9 / 15.0, 8 over up to 1500 and
// 2500 18.7 / 17.9 / 15.9 and 23.4 / 23.4 / 23.8; over E4M3 cells, 16 up to 2500 and 4133
// 28.1 / 22.5 / 22.5 and 32.7 / 32.7 / 28.8, one over 1536 13.4 / 12.5 / 11.1.
constexpr Cutting kCutFew{2, 1.0f, 8.0f}, kCutFewCodes{2, 1.0f, 12.0f};

// Units of at most kFewRows rows (paged_few.cu).
constexpr int kFewRows = 16;
cudaError_t launch_paged_few(const PagedMaps& maps, const PagedArgs& a, int DP, bool f16, bool codes, int grid, cudaStream_t st);
cudaError_t paged_few_read_error(cudaStream_t st, uint32_t* err);

}  // namespace w8
