// The expert layer of a few tokens over MX-quantized weights.
//
//   xq = MXFP8(x);  g, u = W13[e] xq;  hq = MXFP8(silu(g) * u);
//   out[t] = sum_j weights[t, j] * W2[e_j] hq_j
//
// Plain form: the row-wise quantizer for x, one warp per gate/up pair of 32
// channels' dot products, one warp per output value.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mxg {
namespace {

MXG_DEVINL float e4m3_f32(uint8_t c) {
  const uint32_t ex = (c >> 3) & 15, man = c & 7;
  const float m = ex ? __uint_as_float((ex + 120) << 23 | man << 20) : (float)man * 0.001953125f;
  return (c & 0x80) ? -m : m;
}
MXG_DEVINL float e2m1_f32(uint32_t c) {
  const uint32_t ex = (c >> 1) & 3, man = c & 1;
  const float m = ex ? __uint_as_float((ex + 126) << 23 | man << 22) : (float)man * 0.5f;
  return (c & 8) ? -m : m;
}
MXG_DEVINL float ue8m0_f32(uint8_t s) { return s ? __uint_as_float((uint32_t)s << 23) : __uint_as_float(1u << 22); }

// Dot product over `cols` of weight row `row` (packed scales, RT row tiles)
// and an MXFP8 vector; every lane returns the sum.
MXG_DEVINL float mx_dot(const uint8_t* w, int64_t ld, const uint8_t* ws, int64_t RT, int64_t row, int elem,
                        const uint8_t* q, const uint8_t* s, int cols, int lane) {
  float acc = 0.0f;
  for (int b = lane; b < cols / 32; b += 32) {
    const uint8_t sc = ws[((b >> 2) * RT + (row >> 7)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (b & 3)];
    const float f = ue8m0_f32(sc) * ue8m0_f32(s[b]);
    float d = 0.0f;
    for (int i = 0; i < 32; ++i) {
      const int c = b * 32 + i;
      const float wv = elem == MXG_E2M1 ? e2m1_f32((w[row * ld + (c >> 1)] >> (4 * (c & 1))) & 15)
                                        : e4m3_f32(w[row * ld + c]);
      d += wv * e4m3_f32(q[c]);
    }
    acc += d * f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  return acc;
}

struct MoeWs {
  uint8_t *xq, *xs, *hq, *hs;
  int32_t* bad;
};
size_t moe_ws(const MoeArgs& a, uint8_t* p, MoeWs* w) {
  const int64_t P = (int64_t)a.T * a.k;
  size_t o = 0;
  auto take = [&](int64_t n) { uint8_t* r = p + o; o += ((size_t)n + 255) & ~(size_t)255; return r; };
  w->bad = reinterpret_cast<int32_t*>(take(4));
  w->xq = take((int64_t)a.T * a.H);
  w->xs = take((int64_t)a.T * a.H / 32);
  w->hq = take(P * a.I);
  w->hs = take(P * a.I / 32);
  return o;
}

__global__ void moe_check_kernel(MoeArgs a, MoeWs w) {
  bool bad = false;
  for (int i = threadIdx.x; i < a.T * a.k; i += blockDim.x) bad |= a.ids[i] >= a.E;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    *w.bad = bad;
    if (bad) report(a.status, MXG_ERR_INDEX);
  }
}

// one warp per (slot, 32 channels)
__global__ void __launch_bounds__(256) moe_up_kernel(MoeArgs a, MoeWs w) {
  if (*w.bad) return;
  const int lane = threadIdx.x & 31;
  const int nb = a.I / 32;
  const int64_t n = (int64_t)a.T * a.k * nb;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
    const int64_t p = i / nb;
    const int b = (int)(i - p * nb);
    const int e = a.ids[p];
    if (e < 0) continue;
    const uint8_t* q = w.xq + p / a.k * a.H;
    const uint8_t* s = w.xs + p / a.k * (a.H / 32);
    const int64_t RT = (int64_t)a.E * 2 * a.I / 128;
    float h = 0.0f;
    for (int c = 0; c < 32; ++c) {
      const int64_t row = (int64_t)e * 2 * a.I + b * 32 + c;
      const float g = mx_dot(a.w13, a.ld13, a.s13, RT, row, a.elem, q, s, a.H, lane);
      const float u = mx_dot(a.w13, a.ld13, a.s13, RT, row + a.I, a.elem, q, s, a.H, lane);
      if (lane == c) h = g / (1.0f + expf(-g)) * u;
    }
    const uint32_t am = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu);
    int ex = (int)(am >> 23) - 127 - 8;
    if ((am >> 23) == 0) ex = -127;
    ex = max(ex, -127);
    w.hq[p * a.I + b * 32 + lane] = (uint8_t)cvt_e4m3x4(h * pow2_neg(ex), 0.0f, 0.0f, 0.0f);
    if (lane == 0) w.hs[p * nb + b] = (uint8_t)(ex + 127);
  }
}

// one warp per output value
template <typename TOut>
__global__ void __launch_bounds__(256) moe_down_kernel(MoeArgs a, MoeWs w) {
  if (*w.bad) return;
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)a.T * a.H;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
    const int64_t t = i / a.H;
    const int c = (int)(i - t * a.H);
    float y = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int64_t p = t * a.k + j;
      const int e = a.ids[p];
      if (e < 0) continue;
      y += a.weights[p] * mx_dot(a.w2, a.ld2, a.s2, (int64_t)a.E * a.H / 128, (int64_t)e * a.H + c, a.elem,
                                 w.hq + p * a.I, w.hs + p * (a.I / 32), a.I, lane);
    }
    if (lane == 0) static_cast<TOut*>(a.out)[t * a.ld_out + c] = (TOut)y;
  }
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int k, int E, int64_t H, int64_t I) {
  MoeArgs a{};
  a.T = (int)T; a.k = k; a.E = E; a.H = (int)H; a.I = (int)I;
  MoeWs w;
  return moe_ws(a, nullptr, &w);
}

mxg_status launch_moe_experts(const MoeArgs& a, cudaStream_t stream, int num_sms) {
  MoeWs w;
  moe_ws(a, static_cast<uint8_t*>(a.ws), &w);
  const int64_t cap = (int64_t)num_sms * 8;
  moe_check_kernel<<<1, 256, 0, stream>>>(a, w);
  if (launch_mx_rowwise(a.x, a.T, a.H, a.ld_x, MXG_E4M3, w.xq, a.H, w.xs, a.H / 32, stream, num_sms) != cudaSuccess)
    return MXG_ERR_CUDA;
  moe_up_kernel<<<(unsigned)std::min<int64_t>(((int64_t)a.T * a.k * (a.I / 32) + 7) / 8, cap), 256, 0, stream>>>(a, w);
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.T * a.H + 7) / 8, cap);
  if (a.out_dtype == MXG_OUT_BF16) moe_down_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, w);
  else moe_down_kernel<float><<<grid, 256, 0, stream>>>(a, w);
  return cudaGetLastError() == cudaSuccess ? MXG_OK : MXG_ERR_CUDA;
}

}  // namespace mxg
