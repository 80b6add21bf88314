// Attention of new tokens over a paged cache: for each token at position t of
// its sequence (of len positions) and query head h, with the key head h / (Hq / Hkv),
//
//   s_j = scale * sum_d q_d k_jd,   j < len, and j <= t where causal
//   o   = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max)       (0 where no j counts)
//
// A warp works on one row: a lane holds four dimensions, keys go by one at a time
// with the running maximum m and sum l.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {
namespace {

struct Args {
  PagedAttnProblem p;
  PagedCache c;
};

template <bool kF16, bool kCodes>
__global__ void __launch_bounds__(128) paged_attention_kernel(const __grid_constant__ Args a) {
  griddep_wait();
  const PagedAttnProblem& p = a.p;
  const PagedCache& c = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t t = w / p.Hq;
  const int h = (int)(w - t * p.Hq);
  if (t >= p.T) return;
  int b;
  int64_t begin, end;
  if (c.q_start) {
    for (b = 0; b < c.B && c.q_start[b + 1] <= t; ++b) {
    }
    if (b >= c.B) return;
    begin = c.q_start[b];
    end = c.q_start[b + 1];
    if (t < begin || t >= end) return;
  } else {
    const int64_t per = p.T / c.B;
    b = (int)(t / per);
    begin = b * per;
    end = begin + per;
  }
  if (t - begin >= p.max_q) return;
  const int64_t len = c.kv_len[b], all = (int64_t)c.cols * c.page_size;
  int64_t n = len < all ? len : all;
  const int64_t pos = len - (end - t);
  if (p.causal && pos + 1 < n) n = pos + 1;
  const int hk = h / (p.Hq / p.Hkv);
  const bool on = 4 * lane < p.D;
  auto load = [&](const void* base, int64_t at, bool codes, float* v) {
    if (codes) {
      const uint32_t r = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + at);
      f16x2_to_f32(cvt_e4m3x2_to_f16x2((uint16_t)r), v[0], v[1]);
      f16x2_to_f32(cvt_e4m3x2_to_f16x2((uint16_t)(r >> 16)), v[2], v[3]);
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
      const F2 x = unpack16<kF16>(r.x), y = unpack16<kF16>(r.y);
      v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
    }
  };
  float q[4] = {}, k[4] = {}, v[4] = {}, o[4] = {};
  if (on) load(p.q, t * p.qs[0] + h * p.qs[1] + 4 * lane, false, q);
  float scale = p.scale, vs = 1.0f;
  if (kCodes) scale *= ld_f32(c.k_scale), vs = ld_f32(c.v_scale);
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = 0; j < n; ++j) {
    const int page = c.table[b * c.table_stride + j / c.page_size];
    const int64_t slot = j % c.page_size;
    const bool there = page >= 0 && page < c.pages;
    for (int e = 0; e < 4; ++e) k[e] = v[e] = 0.0f;
    if (on && there) {
      load(c.k, page * c.ks[0] + slot * c.ks[1] + hk * c.ks[2] + 4 * lane, kCodes, k);
      load(c.v, page * c.vs[0] + slot * c.vs[1] + hk * c.vs[2] + 4 * lane, kCodes, v);
    }
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
    for (int x = 16; x >= 1; x /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= scale;
    const float mn = fmaxf(m, s), f = mn == -INFINITY ? 1.0f : expf(m - mn), w = mn == -INFINITY && s == s ? 0.0f : expf(s - mn);
    m = mn;
    l = l * f + w;
    for (int e = 0; e < 4; ++e) o[e] = o[e] * f + w * v[e];
  }
  if (!on) return;
  const float f = l == 0.0f ? 0.0f : vs / l;
  const int64_t at = t * p.os[0] + h * p.os[1] + 4 * lane;
  if (p.s_out) {
    const float g = __frcp_rn(ld_f32(p.s_out));
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + at) =
        cvt_e4m3x2(o[0] * f * g, o[1] * f * g) | (cvt_e4m3x2(o[2] * f * g, o[3] * f * g) << 16);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint2(cvt16x2(kF16, o[0] * f, o[1] * f), cvt16x2(kF16, o[2] * f, o[3] * f));
  }
}

}  // namespace

int64_t paged_attention_ws_floats(const PagedAttnProblem&, const PagedCache&, int) { return 0; }

cudaError_t launch_paged_attention(const PagedAttnProblem& p, const PagedCache& c, int, cudaStream_t st, int* tmap_err) {
  *tmap_err = 0;
  Args a{p, c};
  const unsigned blocks = (unsigned)((p.T * p.Hq + 3) / 4);
  if (p.f16) {
    if (c.codes) paged_attention_kernel<true, true><<<blocks, 128, 0, st>>>(a);
    else paged_attention_kernel<true, false><<<blocks, 128, 0, st>>>(a);
  } else {
    if (c.codes) paged_attention_kernel<false, true><<<blocks, 128, 0, st>>>(a);
    else paged_attention_kernel<false, false><<<blocks, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t paged_attention_read_error(cudaStream_t, uint32_t* err) {
  *err = 0;
  return cudaSuccess;
}

}  // namespace w8
