// Residual addition, root-mean-square norm and E4M3 quantization in one pass:
// what stands between one linear site of a transformer block and the next.
// Per row of K values (x and the residual in bf16 or binary16):
//
//   r = fl32(x + res)                       res_out = round16(r)
//   i = rsqrt(fl32(sum r^2 * fl32(1/K)) + eps)
//   h = fl32(fl32(r * w) * i)
//   s = s_in, or for this row max(fl32(max|h| / 448), 2^-126)
//   q = E4M3_satRNE(fl32(h * fl32(1/s)))
//
// The sum of squares and max|r w| are taken together, in one reduction: since
// rounding is monotone, max|h| = fl32(max|r w| * i) exactly, so a row's scale
// needs no second pass and no second barrier.  r is not rounded before the norm and h not
// before the quantization: each output is rounded once, from 32 bits.
//
// Bound by HBM: 2 K bytes of x and of the residual in, 2 K of the residual and
// K codes out, about 5 operations a value.  A row is held in registers (kV
// 16-byte vectors of each input per thread), so every byte moves once; a block
// keeps its weights packed in registers over all its rows and has the next
// row's loads in flight while it reduces and writes the present one.  20670 x
// 4096, bf16, per-token scales: 90.7 us = 6.5 TB/s, 0.97 of the measured copy;
// one row of 4096: 2.1 us, the launch and one round trip to memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "swiglu_spec.cuh"

namespace w8 {
namespace {

constexpr int kMaxThreads = 512;              // K <= 8 * 4 * 512 = 16384
constexpr float kTinyScale = 1.17549435e-38f; // 2^-126: a zero row's scale, so that its codes are zero

struct NormArgs {
  const uint16_t *x, *res, *w;
  int64_t M;
  int K;
  float eps, inv_k;
  const float* s_in;
  float* s_tok;
  uint8_t* q;
  uint16_t *h, *res_out;
};

// blockDim = (threads of a row, rows of a block); more than one row only
// where a row is one warp's.
template <bool kF16, int kV, bool kRes, bool kTok>
__global__ void __launch_bounds__(kMaxThreads) add_rms_norm_quant_kernel(const NormArgs a) {
  __shared__ float2 slots[2][kMaxThreads / 32];
  griddep_launch_dependents();   // a GEMM launched next may start its prologue
  const int T = (int)blockDim.x, t = (int)threadIdx.x;
  const int nvec = a.K / 8;
  const int warps = T / 32;
  uint4 wv[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i)
    wv[i] = t + i * T < nvec ? ldg16(a.w + 8 * (t + i * T)) : make_uint4(0, 0, 0, 0);
  float inv_s = 1.0f;
  if (!kTok && a.q) inv_s = __frcp_rn(__ldg(a.s_in));

  const int64_t stride = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  uint4 xv[kV], rv[kV];
  auto load = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int j = t + i * T;
      xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
      if (j < nvec && m < a.M) {
        xv[i] = ld16_once(a.x + m * a.K + 8 * j);
        if (kRes) rv[i] = ld16_once(a.res + m * a.K + 8 * j);
      }
    }
  };
  load(row);
  // Every row group of a block makes the same number of rounds: the block's
  // barrier below is reached by all of its threads.
  const int64_t first = (int64_t)blockIdx.x * blockDim.y;
  for (int64_t base = first, buf = 0; base < a.M; base += stride, row += stride, buf ^= 1) {
    F2 v[kV][4];
    float ss = 0.0f, top = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
      const uint32_t rw[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
      const uint32_t ww[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
      uint32_t o[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        F2 r = unpack16<kF16>(xw[c]);
        if (kRes) r = add2(r, unpack16<kF16>(rw[c]));
        ss = fmaf(r.x, r.x, ss);
        ss = fmaf(r.y, r.y, ss);
        o[c] = cvt16x2(kF16, r.x, r.y);
        v[i][c] = mul2(r, unpack16<kF16>(ww[c]));
        // max_nan: a NaN in a row makes its scale and codes NaN
        if (kTok) top = max_nan(top, max_nan(fabsf(v[i][c].x), fabsf(v[i][c].y)));
      }
      const int j = t + i * T;
      if (kRes && a.res_out && j < nvec && row < a.M)
        *reinterpret_cast<uint4*>(a.res_out + row * a.K + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    load(row + stride);
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
      ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, o));
      if (kTok) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    if (warps > 1) {   // one row in the block: its warps' sums in a fixed order
      // Two sets of slots in turn: a set is written again only after the next
      // row's barrier, which every reader of it has passed by then.
      if ((t & 31) == 0) slots[buf][t >> 5] = make_float2(ss, top);
      __syncthreads();
      ss = slots[buf][0].x;
      top = slots[buf][0].y;
      for (int k = 1; k < warps; ++k) {
        const float2 p = slots[buf][k];
        ss = __fadd_rn(ss, p.x);
        if (kTok) top = max_nan(top, p.y);
      }
    }
    const float inv = rsqrtf(fmaf(ss, a.inv_k, a.eps));
    if (kTok) {
      const float s = max_nan(__fdiv_rn(__fmul_rn(top, inv), 448.0f), kTinyScale);
      inv_s = __frcp_rn(s);
      if (t == 0 && row < a.M) a.s_tok[row] = s;
    }
    if (row >= a.M) continue;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int j = t + i * T;
      if (j >= nvec) continue;
      uint32_t hw[4], code[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const F2 h = mul2(v[i][c], splat(inv));
        hw[c] = cvt16x2(kF16, h.x, h.y);
        const F2 y = mul2(h, splat(inv_s));
        code[c] = cvt_e4m3x2(y.x, y.y);
      }
      if (a.q)
        *reinterpret_cast<uint2*>(a.q + row * a.K + 8 * j) =
            make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
      if (a.h) *reinterpret_cast<uint4*>(a.h + row * a.K + 8 * j) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    }
  }
}

template <bool kF16, int kV>
cudaError_t launch_v(const NormArgs& a, dim3 block, int sms, cudaStream_t st) {
  void (*k)(NormArgs) = nullptr;
  if (a.res) k = a.s_tok ? add_rms_norm_quant_kernel<kF16, kV, true, true> : add_rms_norm_quant_kernel<kF16, kV, true, false>;
  else k = a.s_tok ? add_rms_norm_quant_kernel<kF16, kV, false, true> : add_rms_norm_quant_kernel<kF16, kV, false, false>;
  // blocks that fit on an SM, by block size (a multiple of 32 up to 512)
  static std::atomic<int> occ[2][2][kMaxThreads / 32 + 1];
  std::atomic<int>& o = occ[a.res != nullptr][a.s_tok != nullptr][block.x * block.y / 32];
  int b = o.load(std::memory_order_relaxed);
  if (b == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, k, (int)(block.x * block.y), 0) != cudaSuccess || b < 1) b = 1;
    o.store(b, std::memory_order_relaxed);
  }
  const int64_t want = (a.M + block.y - 1) / block.y, most = (int64_t)b * sms;
  k<<<(int)(want < most ? want : most), block, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Threads of a row and vectors of a thread: with few rows as many threads as
// the row has vectors (the fewest loads one after the other); with rows enough
// to fill the GPU up to four vectors a thread, so that reductions and barriers
// are spread over more values.
cudaError_t launch_add_rms_norm_quant(const void* x, const void* res, bool f16, int64_t M, int K, const void* w,
                                      float eps, const float* s_in, float* s_tok, uint8_t* q, void* h, void* res_out,
                                      int sms, cudaStream_t st) {
  NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(res), static_cast<const uint16_t*>(w), M, K,
             eps, 1.0f / (float)K, s_in, s_tok, q, static_cast<uint16_t*>(h), static_cast<uint16_t*>(res_out)};
  const int nvec = K / 8;
  const bool many = M >= 4 * (int64_t)sms;
  int kv = 1;
  auto threads = [&] { return ((nvec + kv - 1) / kv + 31) / 32 * 32; };
  while (kv < 4 && (threads() > kMaxThreads || (many && threads() > 128))) kv *= 2;
  const int T = threads();
  const dim3 block(T, T == 32 ? 4 : 1);
  if (f16) return kv == 1 ? launch_v<true, 1>(a, block, sms, st) : kv == 2 ? launch_v<true, 2>(a, block, sms, st) : launch_v<true, 4>(a, block, sms, st);
  return kv == 1 ? launch_v<false, 1>(a, block, sms, st) : kv == 2 ? launch_v<false, 2>(a, block, sms, st) : launch_v<false, 4>(a, block, sms, st);
}

}  // namespace w8
