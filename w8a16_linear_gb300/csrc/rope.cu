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
constexpr int kAhead = 4;          // loads of a lane in flight

struct RopeArgs {
  RopeProblem p;
  PagedCache c;
  int split;        // warps of a token
  float inv_d;
};

// kLanes: lanes of a head (a power of two; 8 dimensions each).  kPaged: k and v
// go into the cache; else k to k_out.
template <bool kF16, int kLanes, bool kInterleaved, bool kPaged>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  griddep_launch_dependents();
  constexpr int kHeads = 32 / kLanes;                       // heads that a warp has at a time
  const RopeProblem& p = a.p;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, head0 = lane / kLanes;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = w / a.split;
  const int part = (int)(w - t * a.split);
  const bool on = 8 * sub < p.D;                            // lanes beyond D hold nothing
  griddep_wait();   // from here on what earlier kernels wrote may be read
  if (t >= p.M) return;

  // Where the token stands: its sequence, and there its position and cell.
  int64_t pos = 0, cell_k = -1, cell_v = -1;
  if (kPaged) {
    const PagedCache& c = a.c;
    int b;
    int64_t begin, end;
    if (c.q_start) {
      int n = 0;   // sequences that begin at t or before it, the first aside
      for (int k = lane + 1; k <= c.B; k += 32) n += ld_i32(c.q_start + k) <= t;
      b = __reduce_add_sync(0xFFFFFFFFu, n);
      if (b >= c.B) return;                                 // behind the last sequence
      begin = ld_i32(c.q_start + b);
      end = ld_i32(c.q_start + b + 1);
      if (t < begin || t >= end) return;
    } else {
      const int64_t per = p.M / c.B;
      b = (int)(t / per);
      end = (b + 1) * per;
    }
    pos = ld_i32(c.kv_len + b) - (end - t);
    const int64_t page_at = pos / c.page_size;
    if (pos >= 0 && page_at < c.cols) {
      const int page = ld_i32(c.table + b * c.table_stride + page_at);
      const int64_t slot = pos - page_at * c.page_size;
      if (page >= 0 && page < c.pages) {
        cell_k = page * c.ks[0] + slot * c.ks[1];
        cell_v = page * c.vs[0] + slot * c.vs[1];
      }
    }
  }

  // Cosines and sines of the lane's dimensions.
  constexpr int kTurns = kInterleaved ? 4 : 8;
  float cs[kTurns], sn[kTurns];
  const bool turned = 8 * sub < p.rot;
  const int half = p.rot >> 1;
  const bool second = !kInterleaved && 8 * sub >= half;     // of a half-split pair
  const int partner = kInterleaved || !turned ? lane : second ? lane - (half >> 3) : lane + (half >> 3);
  if (turned) {
    const int pair0 = kInterleaved ? 4 * sub : 8 * sub - (second ? half : 0);
    int64_t at[3] = {pos, pos, pos};
    if (p.positions)
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (x < p.axes) at[x] = ld_i32(p.positions + x * p.pos_stride + t);
#pragma unroll
    for (int j = 0; j < kTurns; ++j) {
      const int i = pair0 + j;
      const int64_t q = i < p.axis_pairs[0] ? at[0] : i < p.axis_pairs[0] + p.axis_pairs[1] ? at[1] : at[2];
      const uint64_t phase = (uint64_t)q * __ldg(p.turns + i);
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn[j], &cs[j]);   // 2^-31 of a half turn
      cs[j] *= p.amplitude;
      sn[j] *= second ? -p.amplitude : p.amplitude;         // b takes + a s, a takes - b s
    }
  }
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (on && p.norm_q) wq = ldg16(static_cast<const uint16_t*>(p.q_weight) + 8 * sub);
  if (on && p.norm_k) wk = ldg16(static_cast<const uint16_t*>(p.k_weight) + 8 * sub);
  float inv_ks = 1.0f, inv_vs = 1.0f;
  if (kPaged && a.c.codes) {
    inv_ks = __frcp_rn(ld_f32(a.c.k_scale));
    inv_vs = __frcp_rn(ld_f32(a.c.v_scale));
  }

  // The token's heads: queries, keys and, into a cache, values.
  const int heads = p.Hq + p.Hkv + (kPaged ? p.Hkv : 0);
  const int chunks = (heads + kHeads - 1) / kHeads;
  for (int first = part * kAhead; first < chunks; first += a.split * kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = (first + u) * kHeads + head0;
      x[u] = make_uint4(0, 0, 0, 0);
      if (!on || h >= heads) continue;
      const uint16_t* from;
      if (h < p.Hq) from = static_cast<const uint16_t*>(p.q) + t * p.qs[0] + h * p.qs[1];
      else if (h < p.Hq + p.Hkv) from = static_cast<const uint16_t*>(p.k) + t * p.ks[0] + (h - p.Hq) * p.ks[1];
      else from = static_cast<const uint16_t*>(p.v) + t * p.vs[0] + (h - p.Hq - p.Hkv) * p.vs[1];
      x[u] = ld16_once(from + 8 * sub);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (first + u >= chunks) break;                       // the same for the whole warp
      const int h = (first + u) * kHeads + head0;
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float v[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const F2 f = unpack16<kF16>(xw[c]);
        v[2 * c] = f.x;
        v[2 * c + 1] = f.y;
      }
      if (p.norm_q || p.norm_k) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o /= 2) ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, o));
        if (is_q ? p.norm_q : p.norm_k && !is_v) {
          const float inv = rsqrtf(fmaf(ss, a.inv_d, p.eps));
          const uint32_t ww[4] = {is_q ? wq.x : wk.x, is_q ? wq.y : wk.y, is_q ? wq.z : wk.z, is_q ? wq.w : wk.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const F2 f = unpack16<kF16>(ww[c]);
            v[2 * c] = __fmul_rn(__fmul_rn(v[2 * c], f.x), inv);
            v[2 * c + 1] = __fmul_rn(__fmul_rn(v[2 * c + 1], f.y), inv);
          }
        }
      }
      float y[8];
      if (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = v[2 * j];
          y[2 * j + 1] = v[2 * j + 1];
          if (turned && !is_v) {
            y[2 * j] = fmaf(v[2 * j], cs[j % kTurns], -__fmul_rn(v[2 * j + 1], sn[j % kTurns]));
            y[2 * j + 1] = fmaf(v[2 * j + 1], cs[j % kTurns], __fmul_rn(v[2 * j], sn[j % kTurns]));
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_sync(0xFFFFFFFFu, v[e], partner);
          y[e] = v[e];
          if (turned && !is_v) y[e] = fmaf(v[e], cs[e % kTurns], -__fmul_rn(other, sn[e % kTurns]));
        }
      }
      if (!on || h >= heads) continue;
      uint16_t* to = nullptr;
      if (is_q) {
        to = static_cast<uint16_t*>(p.q_out) + t * p.qos[0] + h * p.qos[1];
      } else if (!kPaged) {
        to = static_cast<uint16_t*>(p.k_out) + t * p.kos[0] + (h - p.Hq) * p.kos[1];
      } else {
        const int64_t cell = is_v ? cell_v : cell_k;
        if (cell < 0) continue;                             // a position without a page
        const int64_t at = cell + (is_v ? (h - p.Hq - p.Hkv) * a.c.vs[2] : (h - p.Hq) * a.c.ks[2]) + 8 * sub;
        if (a.c.codes) {
          const float f = is_v ? inv_vs : inv_ks;
          uint32_t q[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) q[c] = cvt_e4m3x2(__fmul_rn(y[2 * c], f), __fmul_rn(y[2 * c + 1], f));
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + at) =
              make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
          continue;
        }
        to = static_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at - 8 * sub;
      }
      uint32_t q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) q[c] = is_v ? xw[c] : cvt16x2(kF16, y[2 * c], y[2 * c + 1]);
      *reinterpret_cast<uint4*>(to + 8 * sub) = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
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
  const int heads = p.Hq + p.Hkv * (cache ? 2 : 1);
  const int chunks = (heads * lanes + 31) / 32, rounds = (chunks + kAhead - 1) / kAhead;   // that one warp would make
  int64_t split = 16ll * sms / p.M;                            // 16 warps an SM
  split = split < 1 ? 1 : split > rounds ? rounds : split;
  a.split = (int)split;
  const int64_t blocks = (p.M * split + kWarps - 1) / kWarps;
  return p.f16 ? launch_type<true>(a, cache != nullptr, blocks, st) : launch_type<false>(a, cache != nullptr, blocks, st);
}

}  // namespace w8
