// Root-mean-square norm of single heads and their rotation by position, in one
// pass, with the keys (and values) going to a tensor or into a paged cache.
// For each head x of D values of a token at position t:
//
//   h = fl32(fl32(x * w) * rsqrt(fl32(sum x^2 * fl32(1/D)) + eps))     (or h = x)
//   (a, b) -> (a c - b s, b c + a s),  c, s = amplitude * cos, sin(t * freq_i)
//
// for the pairs (i, i + rot/2), or (2i, 2i + 1) where interleaved, of the first
// rot dimensions; the others keep h.  All in 32 bits, rounded once, to 16 bits or
// to the E4M3 code of fl32(y * fl32(1/scale)).
//
// The angle: a frequency comes as the part of a turn that a position adds, in
// units of 2^-64 turns.  Position times that, modulo 2^64, is the phase exactly
// as far as the 2^-65 of the frequency's rounding go, at positions of either sign
// and any size: no reduction of a large argument, and none of its rounding (t * freq in
// binary32 is off by 2^-5 radians at t = 10^6).  Its upper 32 bits go to sincospi.
//
// Bound by HBM: 2 bytes a value in, 2 (or 1, as a code) out.  A warp works on one
// token (or, of few tokens, on some of its heads): its lanes compute the cosines and sines
// of their four pairs once, and then go through the heads, two chunks of 512 bytes at a time, with four
// more on their way by asynchronous copies.  A lane has both values of each of its pairs:
// with half-split pairs four dimensions of either half, so that a rotation needs no exchange
// (16 contiguous bytes a lane, with the partner from another lane: 98.8 us for the first case
// below, where the change to this layout alone gave 81.4).
//
// Measured (GB300, a replayed graph): 20670 tokens of 32 and 8 heads of 128, normed, three
// axes, bf16: 68 us = 6.2 TB/s, 0.93 of the measured copy, with the issue slots 74% busy; two
// chunks of 4096 tokens into E4M3 cells, 32 / 8 / 8 heads: 37 us = 5.0 TB/s, the issue slots 69% busy, in
// 2.25 rounds of blocks; one token of each of 8 sequences: 2.8 us, one round trip for the sequence,
// one for the page.  Tried before two chunks went at a time, when the first case took 74.2 us: 8
// chunks in flight 76.0, 40 warps an SM 90.5.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {
namespace {

constexpr int kWarps = 4;          // of a block
constexpr int kAhead = 4;          // chunks of heads that are copied ahead of the two that are worked on
constexpr int kRing = 8;           // places for them

struct RopeArgs {
  RopeProblem p;
  PagedCache c;
  int split, per;   // warps of a token, chunks of heads of each
  float inv_d;
};

// Copies of 16 and 8 bytes to shared memory that the thread waits for by groups.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// kLanes: lanes of a head (a power of two), of eight dimensions each: 8 u .. 8 u + 7
// in lane u, or where pairs are half-split four of either half, 4 u .. and rot / 2 + 4 u ..,
// so that a pair is in one lane.  kPaged: k and v go into the cache; else k to k_out.
template <bool kF16, int kLanes, bool kInterleaved, bool kPaged>
__global__ void __launch_bounds__(32 * kWarps, 6) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  griddep_launch_dependents();
  constexpr int kHeads = 32 / kLanes;                       // heads that a warp has at a time
  const RopeProblem& p = a.p;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, head0 = lane / kLanes;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = a.split == 1 ? w : w / a.split;
  const int part = (int)(w - t * a.split);
  const bool on = 8 * sub < p.D;                            // lanes beyond D hold nothing
  griddep_wait();   // from here on what earlier kernels wrote may be read
  if (t >= p.M) return;

  // The lane's dimensions: four from d0 and four from d1.
  const bool turned = 8 * sub < p.rot;
  const bool split_pairs = !kInterleaved && turned;
  const int d0 = split_pairs ? 4 * sub : 8 * sub, d1 = split_pairs ? (p.rot >> 1) + 4 * sub : 8 * sub + 4;
  // The token's heads, kHeads of a kind at a time: queries, keys and, into a cache, values.
  const int q_chunks = (p.Hq + kHeads - 1) / kHeads, k_chunks = (p.Hkv + kHeads - 1) / kHeads;
  const int chunks = q_chunks + k_chunks * (kPaged ? 2 : 1);
  const uint16_t* q_at = static_cast<const uint16_t*>(p.q) + t * p.qs[0] + head0 * p.qs[1];
  const uint16_t* k_at = static_cast<const uint16_t*>(p.k) + t * p.ks[0] + head0 * p.ks[1];
  const uint16_t* v_at = static_cast<const uint16_t*>(p.v) + t * p.vs[0] + head0 * p.vs[1];
  const int end = min(chunks, (part + 1) * a.per);
  // A lane's own 16 bytes of each chunk that is under way.
  __shared__ uint4 ring[kWarps][kRing][32];
  uint4* mine = &ring[threadIdx.x >> 5][0][lane];
  auto fetch = [&](int c) {
    const int ck = c - q_chunks, cv = ck - k_chunks;
    const bool is_q = c < q_chunks, is_v = kPaged && cv >= 0;
    const int h = (is_q ? c : is_v ? cv : ck) * kHeads;
    if (c < end && on && h + head0 < (is_q ? p.Hq : p.Hkv)) {
      const uint16_t* from = is_q ? q_at + h * p.qs[1] : is_v ? v_at + h * p.vs[1] : k_at + h * p.ks[1];
      const uint32_t to = smem_u32(mine + (c % kRing) * 32);
      if (kInterleaved) {
        copy16(to, from + d0);
      } else {
        copy8(to, from + d0);
        copy8(to + 8, from + d1);
      }
    }
    copy_commit();
  };
  // before the places and angles, which they do not need
#pragma unroll 1
  for (int k = 0; k < kAhead; ++k) fetch(part * a.per + k);

  auto leave = [] { copy_wait<0>(); };   // no copy may outlive its thread's block

  // Where the token stands: its sequence, its position there, and that one's page.
  int64_t pos = 0;
  int page = -1, slot = 0;
  if (kPaged) {
    const PagedCache& c = a.c;
    int b, kv;
    int64_t begin, end;
    if (c.q_start && c.B < 32) {   // a lane for each sequence: one round trip
      const int start = ld_i32(c.q_start + min(lane, c.B)), len = ld_i32(c.kv_len + min(lane, c.B - 1));
      b = __popc(__ballot_sync(0xFFFFFFFFu, lane >= 1 && lane <= c.B && start <= t));
      begin = __shfl_sync(0xFFFFFFFFu, start, b);
      end = __shfl_sync(0xFFFFFFFFu, start, min(b + 1, c.B));
      kv = __shfl_sync(0xFFFFFFFFu, len, min(b, c.B - 1));
      if (b >= c.B || t < begin || t >= end) return leave();   // of no sequence
    } else if (c.q_start) {
      int n = 0;   // sequences that begin at t or before it, the first aside
      for (int k = lane + 1; k <= c.B; k += 32) n += ld_i32(c.q_start + k) <= t;
      b = __reduce_add_sync(0xFFFFFFFFu, n);
      if (b >= c.B) return leave();
      begin = ld_i32(c.q_start + b);
      end = ld_i32(c.q_start + b + 1);
      kv = ld_i32(c.kv_len + b);
      if (t < begin || t >= end) return leave();
    } else {
      const int per = (int)(p.M / c.B);
      b = (int)t / per;
      end = (int64_t)(b + 1) * per;
      kv = ld_i32(c.kv_len + b);
    }
    pos = kv - (end - t);
    if (pos >= 0 && pos < (int64_t)c.cols * c.page_size) {
      const int page_at = (int)pos / c.page_size;
      slot = (int)pos - page_at * c.page_size;
      page = ld_i32(c.table + b * c.table_stride + page_at);   // used with the first key: in flight until then
    }
  }

  // Cosines and sines of the lane's pairs.
  float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (turned) {
    int64_t at[3] = {pos, pos, pos};
    if (p.positions)
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (x < p.axes) at[x] = ld_i32(p.positions + x * p.pos_stride + t);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 4 * sub + j;
      const int64_t q = i < p.axis_pairs[0] ? at[0] : i < p.axis_pairs[0] + p.axis_pairs[1] ? at[1] : at[2];
      const uint64_t phase = (uint64_t)q * __ldg(p.turns + i);
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn[j], &cs[j]);   // 2^-31 of a half turn
      cs[j] *= p.amplitude;
      sn[j] *= p.amplitude;
    }
  }
  auto put = [&](uint16_t* to, const uint32_t (&w)[4]) {
    if (kInterleaved) {
      *reinterpret_cast<uint4*>(to + d0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(to + d0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(to + d1) = make_uint2(w[2], w[3]);
    }
  };
  const bool codes = kPaged && a.c.codes, placed = page >= 0 && page < a.c.pages;   // else a position without a page

  // The chunks lo .. hi - 1, of one kind (0 queries, 1 keys, 2 values), which begin with chunk
  // c0: two at a time, so that one's reduction is under way with the other's.
  auto section = [&](auto kind, int c0, int lo, int hi) {
    constexpr int kKind = decltype(kind)::value;
    constexpr bool kCache = kPaged && kKind > 0;
    const int H = kKind == 0 ? p.Hq : p.Hkv;
    const bool norm = kKind == 0 ? p.norm_q : kKind == 1 && p.norm_k;
    F2 w[4] = {};
    if (norm && on) {
      const uint16_t* from = static_cast<const uint16_t*>(kKind == 0 ? p.q_weight : p.k_weight);
      const uint2 w0 = __ldg(reinterpret_cast<const uint2*>(from + d0)), w1 = __ldg(reinterpret_cast<const uint2*>(from + d1));
      w[0] = unpack16<kF16>(w0.x), w[1] = unpack16<kF16>(w0.y), w[2] = unpack16<kF16>(w1.x), w[3] = unpack16<kF16>(w1.y);
    }
    const int64_t* cell = kKind == 2 ? a.c.vs : a.c.ks;
    const int64_t* row = kKind == 0 ? p.qos : p.kos;
    const int64_t head = kCache ? cell[2] : row[1];
    const int64_t first = kCache ? page * cell[0] + slot * cell[1] : t * row[0];
    void* to = kKind == 0 ? p.q_out : !kPaged ? p.k_out : kKind == 1 ? a.c.k : a.c.v;
    float inv_s = 1.0f;
    if (kCache && codes) inv_s = __frcp_rn(ld_f32(kKind == 1 ? a.c.k_scale : a.c.v_scale));
#pragma unroll 1
    for (int c = lo; c < hi; c += 2) {
      fetch(c + kAhead);
      if (c + 1 < hi) fetch(c + kAhead + 1);
      copy_wait<kAhead>();
      F2 v[2][4];
      uint32_t out[2][4];
      bool there[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        there[u] = on && c + u < hi && (c + u - c0) * kHeads + head0 < H;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (there[u]) x = mine[((c + u) % kRing) * 32];
        out[u][0] = x.x, out[u][1] = x.y, out[u][2] = x.z, out[u][3] = x.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = unpack16<kF16>(out[u][e]);
      }
      if (kKind < 2) {
        if (norm) {
          float ss[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            F2 s2 = mul2(v[u][0], v[u][0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) s2 = fma2(v[u][e], v[u][e], s2);
            ss[u] = __fadd_rn(s2.x, s2.y);
          }
#pragma unroll
          for (int o = kLanes / 2; o >= 1; o /= 2)
#pragma unroll
            for (int u = 0; u < 2; ++u) ss[u] = __fadd_rn(ss[u], __shfl_xor_sync(0xFFFFFFFFu, ss[u], o));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const F2 inv = splat(rsqrtf(fmaf(ss[u], a.inv_d, p.eps)));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[u][e] = mul2(mul2(v[u][e], w[e]), inv);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (turned) {
            if (kInterleaved) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[u][e] = fma2(v[u][e], splat(cs[e]), mul2(F2{v[u][e].y, v[u][e].x}, F2{-sn[e], sn[e]}));
            } else {   // pairs of v[0], v[1] and v[2], v[3]
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const F2 c2 = F2{cs[2 * e], cs[2 * e + 1]}, s2 = F2{sn[2 * e], sn[2 * e + 1]};
                const F2 x0 = v[u][e], x1 = v[u][e + 2];
                v[u][e] = fma2(x0, c2, mul2(neg(x1), s2));
                v[u][e + 2] = fma2(x1, c2, mul2(x0, s2));
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) out[u][e] = cvt16x2(kF16, v[u][e].x, v[u][e].y);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!there[u] || (kCache && !placed)) continue;
        const int64_t at = first + ((c + u - c0) * kHeads + head0) * head;
        if (kCache && codes) {
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const F2 y = mul2(v[u][e], splat(inv_s));
            q[e] = cvt_e4m3x2(y.x, y.y);
          }
          uint8_t* cells = static_cast<uint8_t*>(to) + at;
          *reinterpret_cast<uint32_t*>(cells + d0) = q[0] | (q[1] << 16);
          *reinterpret_cast<uint32_t*>(cells + d1) = q[2] | (q[3] << 16);
        } else {
          put(static_cast<uint16_t*>(to) + at, out[u]);
        }
      }
    }
  };
  const int begin = part * a.per, k0 = q_chunks, v0 = q_chunks + k_chunks;
  section(std::integral_constant<int, 0>{}, 0, begin, min(end, k0));
  section(std::integral_constant<int, 1>{}, k0, max(begin, k0), min(end, v0));
  if (kPaged) section(std::integral_constant<int, 2>{}, v0, max(begin, v0), end);
  copy_wait<0>();
}

template <bool kF16, int kLanes, bool kInterleaved>
cudaError_t launch_layout(const RopeArgs& a, bool paged, int64_t blocks, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = paged ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<kF16, kLanes, kInterleaved, true>, a)
                        : cudaLaunchKernelEx(&cfg, norm_rope_kernel<kF16, kLanes, kInterleaved, false>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kF16, int kLanes>
cudaError_t launch_lanes(const RopeArgs& a, bool paged, int64_t blocks, cudaStream_t st) {
  return a.p.interleaved ? launch_layout<kF16, kLanes, true>(a, paged, blocks, st)
                         : launch_layout<kF16, kLanes, false>(a, paged, blocks, st);
}

template <bool kF16>
cudaError_t launch_type(const RopeArgs& a, bool paged, int64_t blocks, cudaStream_t st) {
  if (a.p.D <= 64) return launch_lanes<kF16, 8>(a, paged, blocks, st);
  if (a.p.D <= 128) return launch_lanes<kF16, 16>(a, paged, blocks, st);
  return launch_lanes<kF16, 32>(a, paged, blocks, st);
}

}  // namespace

// Warps of a token: with few tokens as many as its heads give work to (each
// computes the cosines and sines again), with tokens enough to fill the GPU one.  Measured
// with 64, 128 and 256 warps an SM as the aim: two chunks of 4096 tokens into E4M3 cells 36.8, 39.8 and 49.7 us,
// 5000 tokens of 32/8 heads 21.3, 23.8 and 34.0, 1000 of them 8.2, 8.7 and 14.6; up to 300 alike.
cudaError_t launch_norm_rope(const RopeProblem& p, const PagedCache* cache, int sms, cudaStream_t st) {
  RopeArgs a{};
  a.p = p;
  if (cache) a.c = *cache;
  a.inv_d = 1.0f / (float)p.D;
  const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
  const int per = 32 / lanes;                                  // heads of a chunk
  const int chunks = (p.Hq + per - 1) / per + (p.Hkv + per - 1) / per * (cache ? 2 : 1);
  int64_t split = 64ll * sms / p.M;                            // 64 warps an SM
  split = split < 1 ? 1 : split > chunks ? chunks : split;
  a.per = (int)((chunks + split - 1) / split);
  a.split = (chunks + a.per - 1) / a.per;
  const int64_t blocks = (p.M * a.split + kWarps - 1) / kWarps;
  return p.f16 ? launch_type<true>(a, cache != nullptr, blocks, st) : launch_type<false>(a, cache != nullptr, blocks, st);
}

}  // namespace w8
