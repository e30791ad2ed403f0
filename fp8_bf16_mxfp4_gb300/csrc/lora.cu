// Low-rank adapters of many requests beside a shared projection:
//   out[t] = y[t] + scale[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// Two kernels: the shrink u[t] = A[a] x[t] (one warp per token and rank row)
// and the expand (one thread per output value, the token's u in shared
// memory).  Sums in fp32, one rounding at the end.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mxg {
namespace {

MXG_DEVINL float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__global__ void __launch_bounds__(256) lora_shrink_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t total = a.T * a.R;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += (int64_t)gridDim.x * 8) {
    const int64_t t = w / a.R;
    const int r = (int)(w - t * a.R);
    const int id = a.ids[t];
    float s = 0.0f;
    if (id >= a.n) {
      if (lane == 0) report(a.status, MXG_ERR_INDEX);
    } else if (id >= 0) {
      const uint16_t* x = a.x + t * a.ld_x;
      const uint16_t* A = a.A + ((int64_t)id * a.R + r) * a.K;
      for (int64_t c = lane; c < a.K; c += 32) s += bf16_f32(x[c]) * bf16_f32(A[c]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) a.ws[w] = s;
  }
}

template <typename TOut>
__global__ void __launch_bounds__(256) lora_expand_kernel(LoraArgs a) {
  __shared__ float u[128];
  const int64_t nb = (a.N + 255) / 256;
  for (int64_t b = blockIdx.x; b < a.T * nb; b += gridDim.x) {
    const int64_t t = b / nb;
    const int64_t c = (b - t * nb) * 256 + threadIdx.x;
    const int id = a.ids[t];
    const bool on = id >= 0 && id < a.n;
    __syncthreads();
    if (threadIdx.x < a.R) u[threadIdx.x] = on ? a.ws[t * a.R + threadIdx.x] : 0.0f;
    __syncthreads();
    if (c < a.N) {
      float d = 0.0f;
      if (on) {
        const uint16_t* B = a.B + ((int64_t)id * a.N + c) * a.R;
        for (int r = 0; r < a.R; ++r) d += bf16_f32(B[r]) * u[r];
        if (a.scale != nullptr) d *= a.scale[id];
      }
      const float y = (float)static_cast<const TOut*>(a.y)[t * a.ld_y + c];
      static_cast<TOut*>(a.out)[t * a.ld_out + c] = (TOut)(on ? y + d : y);
    }
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int R) {
  (void)K;
  return (size_t)std::max<int64_t>(T, 1) * R * sizeof(float);
}

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t cap = (int64_t)num_sms * 16;
  lora_shrink_kernel<<<(unsigned)std::min((a.T * a.R + 7) / 8, cap), 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min(a.T * ((a.N + 255) / 256), cap);
  if (a.dtype == MXG_OUT_BF16) lora_expand_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
  else lora_expand_kernel<float><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mxg
