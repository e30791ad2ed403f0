// Top-k routing: router logits -> expert ids and combine weights.
//
// One warp per token.  Lane i holds the logits of experts i, i + 32, ...; each
// of the k rounds takes the largest value left (a warp max over the values as
// order-preserving integers) and, among its holders, the lowest expert (a warp
// min over indices), so equal logits resolve to the lower expert and the
// choice is exact.  Weights are exp(l - max) over a sum taken in fp32.
//
// Bound: the logits are read once (T * E values) and 8 bytes per slot written;
// below a few thousand tokens the launch is the cost: one token 2.1 us, 16384
// tokens of 32 experts, top 8, 7.3 us (0.46 us of memory traffic), where the k
// dependent rounds of a warp are what is left.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mxg {
namespace {

constexpr int kRouteWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;

// An unsigned key in the order of the float values; NaN and -inf are 0, below
// every other logit, and -0 equals +0.
MXG_DEVINL uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0;  // NaN compares false
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
MXG_DEVINL float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}
// exp(v - top) with the value 1 at v == top (also when both are infinite).
MXG_DEVINL float route_exp(float v, float top) { return v == top ? 1.0f : expf(v - top); }

MXG_DEVINL float load_logit(const float* p) { return __ldg(p); }
MXG_DEVINL float load_logit(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// kPer: logits per lane, the least that holds the experts (<= 32 * kPer): 16384
// tokens of 32 experts, top 8, take 7.6 us with one, 8.5 with two and 26.7 with
// sixteen; 4096 tokens of 128 experts 5.2 with four and 10.2 with sixteen.
template <typename TIn, int kPer>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const TIn* __restrict__ logits, int64_t T, int E,
                                                                     int64_t ld, int k, bool renorm,
                                                                     int32_t* __restrict__ ids,
                                                                     float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < T;
       t += (int64_t)gridDim.x * kRouteWarps) {
    const TIn* row = logits + t * ld;
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < E ? order_key(load_logit(row + e)) : 0u;
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = max(best, key[i]);
    const uint32_t top_key = __reduce_max_sync(kFull, best);
    const float top = key_value(top_key);
    float total = 0.0f;  // all experts' sum (renorm: the chosen ones', below)
    if (!renorm && top_key != 0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (key[i] != 0) total += route_exp(key_value(key[i]), top);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
    }
    int my_id = -1;  // lane j: slot j
    uint32_t my_key = 0;
    for (int j = 0; j < k; ++j) {
      const uint32_t m = __reduce_max_sync(kFull, best);
      if (m == 0) break;  // nothing left to choose (warp-uniform)
      int e;
      if constexpr (kPer == 1) {
        e = __ffs(__ballot_sync(kFull, best == m)) - 1;
      } else {
        int at = 0x7FFFFFFF;
        if (best == m) {
#pragma unroll
          for (int i = kPer - 1; i >= 0; --i)
            if (key[i] == m) at = lane + 32 * i;
        }
        e = __reduce_min_sync(kFull, at);
      }
      if ((e & 31) == lane) {  // the winner's lane drops it
        best = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (e == lane + 32 * i) key[i] = 0;
          best = max(best, key[i]);
        }
      }
      if (lane == j) {
        my_id = e;
        my_key = m;
      }
    }
    const float my_p = my_id >= 0 ? route_exp(key_value(my_key), top) : 0.0f;
    if (renorm) {
      total = my_p;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
    }
    if (lane < k) {
      ids[t * k + lane] = my_id;
      weights[t * k + lane] = my_id < 0 ? 0.0f : my_p / total;
    }
  }
}

template <typename TIn>
cudaError_t launch_route(const TIn* logits, int64_t T, int E, int64_t ld, int k, bool renorm, int32_t* ids,
                         float* weights, cudaStream_t stream, int num_sms) {
  const int64_t want = (T + kRouteWarps - 1) / kRouteWarps;
  const unsigned grid = (unsigned)std::min<int64_t>(want, (int64_t)num_sms * 8);
  const dim3 block(kRouteWarps * 32);
  const int per = (E + 31) / 32;
  if (per <= 1) moe_route_kernel<TIn, 1><<<grid, block, 0, stream>>>(logits, T, E, ld, k, renorm, ids, weights);
  else if (per <= 2) moe_route_kernel<TIn, 2><<<grid, block, 0, stream>>>(logits, T, E, ld, k, renorm, ids, weights);
  else if (per <= 4) moe_route_kernel<TIn, 4><<<grid, block, 0, stream>>>(logits, T, E, ld, k, renorm, ids, weights);
  else if (per <= 8) moe_route_kernel<TIn, 8><<<grid, block, 0, stream>>>(logits, T, E, ld, k, renorm, ids, weights);
  else moe_route_kernel<TIn, 16><<<grid, block, 0, stream>>>(logits, T, E, ld, k, renorm, ids, weights);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Gradient of the routing weights.  With s = sum_j w_j dw_j over a token's slots:
//   weights over the chosen experts   dl[id_j] = w_j (dw_j - s), zeros elsewhere
//   weights over all experts          dl_e = [e = id_j] w_j dw_j - p_e s,  p = softmax(l)
// One warp per token, a lane holding the experts lane, lane + 32, ...: the row goes
// through shared memory, where the lane of a slot adds its part, and is written once.
// An expert that is named twice (its lanes do not read back what they wrote) gets both
// in the order of the slots.  p is made as the forward makes it: a logit of -inf or NaN
// has 0, one that equals the maximum exp(0).  Bound by issue and latency: 16384 tokens
// of 256 experts, 34 MB, 8.2 us (12.2 with every slot offered to every expert in
// registers and a maximum of shuffles), with weights over the chosen experts 5.7; 77
// tokens 2.1 us, a launch.  Two or four tokens of a warp at once: 12.8 and 17; two
// experts in one load: the same, with BF16 12.1 for 9.6.
// ---------------------------------------------------------------------------
MXG_DEVINL void store_grad(float* p, float v) { *p = v; }
MXG_DEVINL void store_grad(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename TIn, int kPer>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_backward_kernel(
    const float* __restrict__ dweights, const int32_t* __restrict__ ids, const float* __restrict__ weights,
    const TIn* __restrict__ logits, int64_t T, int E, int64_t ld, int k, TIn* __restrict__ dlogits, int64_t ld_d,
    int32_t* __restrict__ status) {
  __shared__ float rows[kRouteWarps][32 * kPer];
  const int lane = threadIdx.x & 31;
  float* row = rows[threadIdx.x >> 5];
  const bool renorm = logits == nullptr;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < T;
       t += (int64_t)gridDim.x * kRouteWarps) {
    float v[kPer], top = -INFINITY;
    if (!renorm) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < E ? load_logit(logits + t * ld + e) : -INFINITY;
      }
    }
    int id = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < k) {  // loaded together, before it is known whether the slot is empty
      id = __ldg(ids + t * k + lane);
      w = __ldg(weights + t * k + lane);
      dw = __ldg(dweights + t * k + lane);
    }
    if (id >= E) {
      report(status, MXG_ERR_INDEX);
      id = -1;
    }
    if (id < 0) w = dw = 0.0f;
    if (id >= 0) row[id] = __int_as_float(lane);
    __syncwarp();
    const bool twice = __any_sync(kFull, id >= 0 && __float_as_int(row[id]) != lane);
    float s = w * dw;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    const float add = renorm ? w * (dw - s) : w * dw;
    if (renorm) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, v[i]);  // passes over NaN
      asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(top));
      float total = 0.0f;
      if (top < INFINITY) {
        const float from = top > -INFINITY ? top : 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = fmaxf(expf(v[i] - from), 0.0f);  // 0 of -inf and NaN
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = v[i] == top ? 1.0f : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) total += v[i];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
      const float per = total > 0.0f ? s / total : 0.0f;  // a row without logits has no slots
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] *= -per;
    }
    if (!twice) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) row[lane + 32 * i] = v[i];
      __syncwarp();
      if (id >= 0) row[id] += add;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = row[lane + 32 * i];
    } else {
      for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(kFull, id, j);
        const float a = __shfl_sync(kFull, add, j);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (e == lane + 32 * i) v[i] += a;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e < E) store_grad(dlogits + t * ld_d + e, v[i]);
    }
    __syncwarp();
  }
}

template <typename TIn>
cudaError_t launch_route_backward(const float* dweights, const int32_t* ids, const float* weights, const TIn* logits,
                                  int64_t T, int E, int64_t ld, int k, TIn* dlogits, int64_t ld_d, int32_t* status,
                                  cudaStream_t stream, int num_sms) {
  const int per = (E + 31) / 32;
  const auto fn = per <= 1   ? moe_route_backward_kernel<TIn, 1>
                  : per <= 2 ? moe_route_backward_kernel<TIn, 2>
                  : per <= 4 ? moe_route_backward_kernel<TIn, 4>
                  : per <= 8 ? moe_route_backward_kernel<TIn, 8>
                             : moe_route_backward_kernel<TIn, 16>;
  const int64_t want = (T + kRouteWarps - 1) / kRouteWarps;
  fn<<<(unsigned)std::min<int64_t>(want, (int64_t)num_sms * 8), kRouteWarps * 32, 0, stream>>>(
      dweights, ids, weights, logits, T, E, ld, k, dlogits, ld_d, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_route_backward(const float* dweights, const int32_t* ids, const float* weights, const void* logits,
                                      int64_t T, int E, int64_t ld, bool bf16, int k, void* dlogits, int64_t ld_d,
                                      int32_t* status, cudaStream_t stream, int num_sms) {
  if (bf16)
    return launch_route_backward(dweights, ids, weights, static_cast<const __nv_bfloat16*>(logits), T, E, ld, k,
                                 static_cast<__nv_bfloat16*>(dlogits), ld_d, status, stream, num_sms);
  return launch_route_backward(dweights, ids, weights, static_cast<const float*>(logits), T, E, ld, k,
                               static_cast<float*>(dlogits), ld_d, status, stream, num_sms);
}

cudaError_t launch_moe_route(const void* logits, int64_t T, int E, int64_t ld, bool bf16, int k, bool renorm,
                             int32_t* ids, float* weights, cudaStream_t stream, int num_sms) {
  if (bf16)
    return launch_route(static_cast<const __nv_bfloat16*>(logits), T, E, ld, k, renorm, ids, weights, stream, num_sms);
  return launch_route(static_cast<const float*>(logits), T, E, ld, k, renorm, ids, weights, stream, num_sms);
}

}  // namespace mxg
