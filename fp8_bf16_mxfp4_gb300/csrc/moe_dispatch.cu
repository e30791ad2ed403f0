// Tokens to the experts and back.  With T tokens of k slots each (P = T k):
//
//   sort              ids [T, k] -> m_splits [E] and every slot's row in expert order
//   gather            xs[row] = x[t]
//   combine           out[t] = sum_j w[t, j] y[row]         (w = 1: gather's gradient)
//   combine_backward  dy[row] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[row]>
//
// An empty slot (id < 0) owns one of the rows behind all others: its entry is
// -1 - row, gather and combine_backward write zeros there, combine skips it.  So
// every one of the P rows is written and the splits add up to P, which is what
// the grouped GEMMs ask for.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace mxg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Sort: a stable counting sort.  Chunks of the slots go to CTAs, equal runs of a
// chunk to its warps, and a warp takes its run 32 slots at a time, where
// __match_any finds the slots of one expert.  A slot's row is the rows of lower
// experts, of earlier chunks, of earlier warps and of earlier slots of its run.
// Up to 4096 slots are one CTA's; above, a first kernel leaves every chunk's counts
// and the second, which counts its own chunk again while that one ends, adds up those
// of the chunks before.  Bound by latency: 64 slots 2.5 us, 65536 slots of 32 experts
// 11 us (4 and 7, overlapping); no atomics, so equal ids keep their order.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 2048;  // least slots of a chunk, where there are several
constexpr int kSortMaxChunks = 256;

int64_t sort_chunk(int64_t P) {
  if (P <= 2 * kSortChunk) return 2 * kSortChunk;  // one CTA, one launch
  const int64_t per = (P + kSortMaxChunks - 1) / kSortMaxChunks;
  return (std::max<int64_t>(per, kSortChunk) + kSortThreads - 1) / kSortThreads * kSortThreads;
}
int64_t sort_chunks(int64_t P) { const int64_t c = sort_chunk(P); return (P + c - 1) / c; }

// Calls f(i, e) for every 32 slots of [i0, i1), a slot per lane: e is the slot's
// expert, E for an empty one (and for an id that is not below E), -1 past the end.
// Four loads are in flight.
constexpr int kSortFlight = 4;
template <typename F>
MXG_DEVINL bool for_slots(const int32_t* ids, int64_t i0, int64_t i1, int E, F f) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int64_t i = i0; i < i1; i += 32 * kSortFlight) {
    int id[kSortFlight];
#pragma unroll
    for (int q = 0; q < kSortFlight; ++q) id[q] = i + 32 * q + lane < i1 ? __ldg(ids + i + 32 * q + lane) : -1;
#pragma unroll
    for (int q = 0; q < kSortFlight; ++q) {
      const int64_t at = i + 32 * q + lane;
      if (at - lane >= i1) break;
      bad |= id[q] >= E;
      f(at, at >= i1 ? -1 : id[q] < 0 || id[q] >= E ? E : id[q]);
    }
  }
  return bad;
}

// cnt[0..E]: the slots of each expert in the warp's run.
MXG_DEVINL bool count_run(const int32_t* ids, int64_t i0, int64_t i1, int E, uint32_t* cnt) {
  const int lane = threadIdx.x & 31;
  return for_slots(ids, i0, i1, E, [&](int64_t, int e) {
    const uint32_t same = __match_any_sync(kFull, e);
    if (e >= 0 && lane == __ffs(same) - 1) cnt[e] += __popc(same);
    __syncwarp();
  });
}

// counts[e][chunk], e = 0 .. E
__global__ void __launch_bounds__(kSortThreads) moe_sort_count_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                                      int64_t chunk, int32_t* counts) {
  extern __shared__ uint32_t cnt[];  // [warps][E + 1]
  const int keys = E + 1, warp = threadIdx.x >> 5;
  ptx::pdl_launch_dependents();
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * chunk, run = chunk / kSortWarps;
  const int64_t i0 = min(P, c0 + warp * run), i1 = min(P, i0 + run);
  count_run(ids, i0, i1, E, cnt + warp * keys);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += kSortThreads) {
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) v += cnt[w * keys + e];
    counts[(int64_t)e * gridDim.x + blockIdx.x] = (int32_t)v;
  }
}

__global__ void __launch_bounds__(kSortThreads) moe_sort_place_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                                      int64_t chunk, const int32_t* counts,
                                                                      int32_t* __restrict__ m_splits,
                                                                      int32_t* __restrict__ rows, int32_t* status) {
  extern __shared__ uint32_t cnt[];  // [warps][E + 1]
  __shared__ uint32_t total[2 * kSortThreads], before[2 * kSortThreads];  // of a key: all slots, those of earlier chunks
  __shared__ uint32_t warp_sum[kSortWarps];
  const int keys = E + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * chunk, run = chunk / kSortWarps;
  const int64_t i0 = min(P, c0 + warp * run), i1 = min(P, i0 + run);
  const bool bad = count_run(ids, i0, i1, E, cnt + warp * keys);
  if (__syncthreads_or(bad) && threadIdx.x == 0) report(status, MXG_ERR_INDEX);

  if (gridDim.x == 1) {
    for (int e = threadIdx.x; e < keys; e += kSortThreads) {
      uint32_t v = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) v += cnt[w * keys + e];
      total[e] = v;
      before[e] = 0;
    }
  } else {
    ptx::pdl_wait();  // the counts are complete
    const int chunks = (int)gridDim.x;
#pragma unroll 4
    for (int e = warp; e < keys; e += kSortWarps) {  // a warp takes a key, its lanes the chunks
      uint32_t all = 0, early = 0;
      for (int c = lane; c < chunks; c += 32) {
        const uint32_t v = (uint32_t)__ldcg(counts + (int64_t)e * chunks + c);
        all += v;
        if (c < (int)blockIdx.x) early += v;
      }
      all = __reduce_add_sync(kFull, all);
      early = __reduce_add_sync(kFull, early);
      if (lane == 0) {
        total[e] = all;
        before[e] = early;
      }
    }
  }
  __syncthreads();
  // Thread t has the two keys 2 t and 2 t + 1 (at most 513).
  const int key0 = 2 * (int)threadIdx.x;
  const uint32_t t0 = key0 < keys ? total[key0] : 0u, t1 = key0 + 1 < keys ? total[key0 + 1] : 0u;
  uint32_t incl = t0 + t1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t at = incl - t0 - t1;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = key0 + q;
    if (e < keys) {
      if (blockIdx.x == 0) {
        // the tail of empty slots counts as the last expert's
        if (e < E - 1) m_splits[e] = (int32_t)(q ? t1 : t0);
        else if (e == E - 1) m_splits[e] = (int32_t)((uint32_t)P - at);
      }
      uint32_t pos = at + before[e];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t m = cnt[w * keys + e];
        cnt[w * keys + e] = pos;
        pos += m;
      }
    }
    at += q ? t1 : t0;
  }
  __syncthreads();

  uint32_t* mine = cnt + warp * keys;
  for_slots(ids, i0, i1, E, [&](int64_t i, int e) {
    const uint32_t same = __match_any_sync(kFull, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const uint32_t first = e >= 0 ? mine[e] : 0u;
    __syncwarp();
    if (e >= 0) {
      const int r = (int)(first + rank);
      rows[i] = e == E ? -1 - r : r;
      if (rank == 0) mine[e] = first + __popc(same);
    }
    __syncwarp();
  });
}

// ---------------------------------------------------------------------------
// Rows of 16-byte pieces.  The entry of a slot -> its row, or -1 where that is
// not below `count` (reported).
// ---------------------------------------------------------------------------
MXG_DEVINL int64_t row_of(int32_t entry, int64_t count, int32_t* status) {
  const int64_t r = entry < 0 ? -1 - (int64_t)entry : entry;
  if (r < count) return r;
  report(status, MXG_ERR_INDEX);
  return -1;
}

template <typename T>
struct Piece {
  static constexpr int n = 16 / sizeof(T);
};
template <typename T>
MXG_DEVINL void widen(const uint4& w, float* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  } else {
    v[0] = bf16lo_to_f32(w.x); v[1] = bf16hi_to_f32(w.x); v[2] = bf16lo_to_f32(w.y); v[3] = bf16hi_to_f32(w.y);
    v[4] = bf16lo_to_f32(w.z); v[5] = bf16hi_to_f32(w.z); v[6] = bf16lo_to_f32(w.w); v[7] = bf16hi_to_f32(w.w);
  }
}
MXG_DEVINL uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
MXG_DEVINL uint4 narrow(const float* v) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  }
}

// A CTA takes one token and `threads` pieces of its row at a time.
constexpr int kRowThreads = 256;
// As many threads as share a row's pieces equally (896 pieces: 4 times 224; with
// 256 threads combine takes 186 us instead of 173 for 65536 rows of 7168).
int row_threads(int64_t pieces) {
  const int64_t turns = (pieces + kRowThreads - 1) / kRowThreads;
  return (int)(((pieces + turns - 1) / turns + 31) / 32 * 32);
}

// A token's row is read once and written to its k rows.  Bound by HBM: 8192 tokens of
// 7168, top 8, 162 us, 6.5 TB/s, nearly all of it writes.
__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(const uint4* __restrict__ x, int64_t ld_x,
                                                                 const int32_t* __restrict__ rows, int k, int64_t P,
                                                                 int64_t pieces, uint4* __restrict__ out, int64_t ld_out,
                                                                 int32_t* status) {
  const int64_t t = blockIdx.x;
  const int32_t* mine = rows + t * k;
  for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < pieces; c += (int64_t)gridDim.y * blockDim.x) {
    const uint4 v = __ldg(x + t * ld_x + c);
    for (int j = 0; j < k; ++j) {
      const int32_t e = __ldg(mine + j);
      const int64_t r = row_of(e, P, status);
      if (r >= 0) out[r * ld_out + c] = e >= 0 ? v : make_uint4(0, 0, 0, 0);
    }
  }
}

// A thread sums one piece over the slots, eight rows in flight.  Every row is read once
// and not again, so the loads and stores are marked as streaming: 65536 rows of 7168 to
// 8192, 162 us, 6.5 TB/s; 173 with plain ones.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const uint4* __restrict__ y, int64_t ld_y, int64_t y_rows,
                                                                  const int32_t* __restrict__ rows,
                                                                  const float* __restrict__ weights, int k,
                                                                  int64_t pieces, uint4* __restrict__ out,
                                                                  int64_t ld_out, int32_t* status) {
  constexpr int n = Piece<T>::n;
  constexpr int kFlight = 8;  // rows in flight
  const int64_t t = blockIdx.x;
  for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < pieces; c += (int64_t)gridDim.y * blockDim.x) {
    float s[n];
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kFlight) {
      uint4 v[kFlight];
      float w[kFlight];
      bool on[kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        on[j] = false;
        if (j0 + j < k) {
          const int32_t e = __ldg(rows + t * k + j0 + j);
          const int64_t r = e >= 0 ? row_of(e, y_rows, status) : -1;
          on[j] = r >= 0;
          if (on[j]) {
            v[j] = __ldcs(y + r * ld_y + c);
            w[j] = weights != nullptr ? __ldg(weights + t * k + j0 + j) : 1.0f;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        if (!on[j]) continue;
        float f[n];
        widen<T>(v[j], f);
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = fmaf(w[j], f[i], s[i]);
      }
    }
    __stcs(out + t * ld_out + c, narrow<T>(s));
  }
}

// A CTA takes a token: its pieces of dout once for every kFlight slots, whose
// products with y it sums per thread, then over the CTA in a fixed order.  y and
// dy may be one buffer: a piece is read by the thread that writes it.  Bound by HBM:
// 65536 rows of 4096, 172 us, 6.6 TB/s (177 with streaming loads and stores).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) moe_combine_backward_kernel(
    const uint4* __restrict__ dout, int64_t ld_dout, const uint4* y, int64_t ld_y, const int32_t* __restrict__ rows,
    const float* __restrict__ weights, int k, int64_t P, int64_t pieces, uint4* dy, int64_t ld_dy,
    float* __restrict__ dweights, int32_t* status) {
  constexpr int n = Piece<T>::n;
  constexpr int kFlight = 4;  // slots at a time; with 8 there are too few warps (65536 rows of 4096: 199 us, 173)
  __shared__ float part[kRowThreads / 32][kFlight];
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int j0 = 0; j0 < k; j0 += kFlight) {
    int64_t at[kFlight];
    float w[kFlight], dot[kFlight];
    bool on[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      at[j] = -1;
      on[j] = false;
      w[j] = dot[j] = 0.0f;
      if (j0 + j < k) {
        const int32_t e = __ldg(rows + t * k + j0 + j);
        at[j] = row_of(e, P, status);
        on[j] = e >= 0 && at[j] >= 0;
        if (on[j]) w[j] = __ldg(weights + t * k + j0 + j);
      }
    }
    for (int64_t c = threadIdx.x; c < pieces; c += blockDim.x) {
      float d[n];
      widen<T>(__ldg(dout + t * ld_dout + c), d);
      uint4 v[kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j)
        if (on[j]) v[j] = y[at[j] * ld_y + c];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        float f[n];
        if (on[j]) {
          widen<T>(v[j], f);
#pragma unroll
          for (int i = 0; i < n; ++i) {
            dot[j] = fmaf(d[i], f[i], dot[j]);
            f[i] = w[j] * d[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < n; ++i) f[i] = 0.0f;
        }
        if (at[j] >= 0) dy[at[j] * ld_dy + c] = narrow<T>(f);
      }
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(kFull, dot[j], s);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kFlight && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
      for (int q = 0; q < warps; ++q) s += part[q][threadIdx.x];
      dweights[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// Launch with programmatic stream serialization: the kernel starts while the one
// before it ends, and waits for its results itself.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

}  // namespace

size_t moe_sort_workspace_bytes(int64_t P, int E) {
  const int64_t n = sort_chunks(P);
  return std::max<size_t>(256, n > 1 ? (size_t)n * (E + 1) * sizeof(int32_t) : 0);
}

cudaError_t launch_moe_sort(const int32_t* ids, int64_t P, int E, int32_t* m_splits, int32_t* rows, void* ws,
                            int32_t* status, cudaStream_t stream) {
  const int64_t chunk = sort_chunk(P);
  const unsigned chunks = (unsigned)std::max<int64_t>(1, sort_chunks(P));
  const size_t smem = (size_t)kSortWarps * (E + 1) * sizeof(uint32_t);
  int32_t* counts = static_cast<int32_t*>(ws);
  if (chunks == 1) {
    moe_sort_place_kernel<<<1, kSortThreads, smem, stream>>>(ids, P, E, chunk, counts, m_splits, rows, status);
    return cudaGetLastError();
  }
  moe_sort_count_kernel<<<chunks, kSortThreads, smem, stream>>>(ids, P, E, chunk, counts);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_overlapped(moe_sort_place_kernel, dim3(chunks), kSortThreads, smem, stream, ids, P, E, chunk,
                           static_cast<const int32_t*>(counts), m_splits, rows, status);
}

cudaError_t launch_moe_gather(const void* x, int64_t ld_x, const int32_t* rows, int64_t T, int k, int64_t pieces,
                              void* out, int64_t ld_out, int32_t* status, cudaStream_t stream) {
  const int threads = row_threads(pieces);
  const dim3 grid((unsigned)T, (unsigned)std::min<int64_t>(65535, (pieces + threads - 1) / threads));
  moe_gather_kernel<<<grid, threads, 0, stream>>>(static_cast<const uint4*>(x), ld_x, rows, k, T * k, pieces,
                                                  static_cast<uint4*>(out), ld_out, status);
  return cudaGetLastError();
}

cudaError_t launch_moe_combine(const void* y, int64_t ld_y, int64_t y_rows, const int32_t* rows, const float* weights,
                               int64_t T, int k, int64_t pieces, bool bf16, void* out, int64_t ld_out, int32_t* status,
                               cudaStream_t stream) {
  const int threads = row_threads(pieces);
  const dim3 grid((unsigned)T, (unsigned)std::min<int64_t>(65535, (pieces + threads - 1) / threads));
  const auto fn = bf16 ? moe_combine_kernel<__nv_bfloat16> : moe_combine_kernel<float>;
  fn<<<grid, threads, 0, stream>>>(static_cast<const uint4*>(y), ld_y, y_rows, rows, weights, k, pieces,
                                   static_cast<uint4*>(out), ld_out, status);
  return cudaGetLastError();
}

cudaError_t launch_moe_combine_backward(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y,
                                        const int32_t* rows, const float* weights, int64_t T, int k, int64_t pieces,
                                        bool bf16, void* dy, int64_t ld_dy, float* dweights, int32_t* status,
                                        cudaStream_t stream) {
  const auto fn = bf16 ? moe_combine_backward_kernel<__nv_bfloat16> : moe_combine_backward_kernel<float>;
  fn<<<(unsigned)T, row_threads(pieces), 0, stream>>>(static_cast<const uint4*>(dout), ld_dout,
                                                      static_cast<const uint4*>(y), ld_y, rows, weights, k, T * k, pieces,
                                                      static_cast<uint4*>(dy), ld_dy, dweights, status);
  return cudaGetLastError();
}

}  // namespace mxg
