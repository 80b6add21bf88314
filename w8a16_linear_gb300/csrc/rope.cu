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
// Bound by HBM: 2 bytes a value in, 2 (or 1, as a code) out.  A warp works on
// one token: its lanes compute the cosines and sines of their eight dimensions once, and
// then go through the token's heads, 16 bytes a lane, four loads at a time
// in flight; the partner of a half-split pair is another lane's.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {
namespace {

constexpr int kWarps = 4;          // of a block
constexpr int kAhead = 4;          // chunks of heads that are copied ahead

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
__global__ void __launch_bounds__(32 * kWarps, 8) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
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
  __shared__ uint4 ring[kWarps][kAhead][32];
  uint4* mine = &ring[threadIdx.x >> 5][0][lane];
  auto fetch = [&](int c) {
    const int ck = c - q_chunks, cv = ck - k_chunks;
    const bool is_q = c < q_chunks, is_v = kPaged && cv >= 0;
    const int h = (is_q ? c : is_v ? cv : ck) * kHeads;
    if (c < end && on && h + head0 < (is_q ? p.Hq : p.Hkv)) {
      const uint16_t* from = is_q ? q_at + h * p.qs[1] : is_v ? v_at + h * p.vs[1] : k_at + h * p.ks[1];
      const uint32_t to = smem_u32(mine + (c % kAhead) * 32);
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
  for (int k = 0; k < kAhead - 1; ++k) fetch(part * a.per + k);

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
  auto put = [&](uint16_t* to, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
    if (kInterleaved) {
      *reinterpret_cast<uint4*>(to + 8 * sub) = make_uint4(w0, w1, w2, w3);
    } else {
      *reinterpret_cast<uint2*>(to + d0) = make_uint2(w0, w1);
      *reinterpret_cast<uint2*>(to + d1) = make_uint2(w2, w3);
    }
  };
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  auto weight = [&](const void* w) {
    const uint2 lo = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + d0));
    const uint2 hi = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + d1));
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  };
  if (on && p.norm_q) wq = weight(p.q_weight);
  if (on && p.norm_k) wk = weight(p.k_weight);

  float inv_ks = 1.0f, inv_vs = 1.0f;
  if (kPaged && a.c.codes) {
    inv_ks = __frcp_rn(ld_f32(a.c.k_scale));
    inv_vs = __frcp_rn(ld_f32(a.c.v_scale));
  }

#pragma unroll 1
  for (int c = part * a.per; c < end; ++c) {
    fetch(c + kAhead - 1);   // to the place of the chunk before
    copy_wait<kAhead - 1>();
    // kinds and counts of a chunk are the same for the whole warp
    const int ck = c - q_chunks, cv = ck - k_chunks;
    const bool is_q = c < q_chunks, is_v = kPaged && cv >= 0;
    const int h = (is_q ? c : is_v ? cv : ck) * kHeads + head0;
    const bool there = on && h < (is_q ? p.Hq : p.Hkv);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (there) x = mine[(c % kAhead) * 32];
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[4] = {xw[0], xw[1], xw[2], xw[3]};
    F2 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = unpack16<kF16>(xw[e]);
    if (!is_v) {
      if (is_q ? p.norm_q : p.norm_k) {
        F2 s2 = mul2(v[0], v[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(v[e], v[e], s2);
        float ss = __fadd_rn(s2.x, s2.y);
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o /= 2) ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, o));
        const F2 inv = splat(rsqrtf(fmaf(ss, a.inv_d, p.eps)));
        const uint32_t ww[4] = {is_q ? wq.x : wk.x, is_q ? wq.y : wk.y, is_q ? wq.z : wk.z, is_q ? wq.w : wk.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(v[e], unpack16<kF16>(ww[e])), inv);
      }
      if (turned) {
        if (kInterleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = fma2(v[e], splat(cs[e]), mul2(F2{v[e].y, v[e].x}, F2{-sn[e], sn[e]}));
        } else {   // pairs of v[0], v[1] and v[2], v[3]
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const F2 c2 = F2{cs[2 * e], cs[2 * e + 1]}, s2 = F2{sn[2 * e], sn[2 * e + 1]};
            const F2 lo = v[e], hi = v[e + 2];
            v[e] = fma2(lo, c2, mul2(neg(hi), s2));
            v[e + 2] = fma2(hi, c2, mul2(lo, s2));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = cvt16x2(kF16, v[e].x, v[e].y);
    }
    if (!there) continue;
    if (is_q) {
      put(static_cast<uint16_t*>(p.q_out) + t * p.qos[0] + h * p.qos[1], out[0], out[1], out[2], out[3]);
    } else if (!kPaged) {
      put(static_cast<uint16_t*>(p.k_out) + t * p.kos[0] + h * p.kos[1], out[0], out[1], out[2], out[3]);
    } else {
      if (page < 0 || page >= a.c.pages) continue;        // a position without a page
      const int64_t* cs3 = is_v ? a.c.vs : a.c.ks;
      const int64_t at = page * cs3[0] + slot * cs3[1] + h * cs3[2];
      void* cache = is_v ? a.c.v : a.c.k;
      if (a.c.codes) {
        const F2 f = splat(is_v ? inv_vs : inv_ks);
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 y = mul2(v[e], f);
          q[e] = cvt_e4m3x2(y.x, y.y);
        }
        uint8_t* to = static_cast<uint8_t*>(cache) + at;
        *reinterpret_cast<uint32_t*>(to + d0) = q[0] | (q[1] << 16);
        *reinterpret_cast<uint32_t*>(to + d1) = q[2] | (q[3] << 16);
      } else {
        put(static_cast<uint16_t*>(cache) + at, out[0], out[1], out[2], out[3]);
      }
    }
  }
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
// computes the cosines and sines again), with tokens enough to fill the GPU one.
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
