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
// votes find the slots of one expert.  A slot's row is the rows of lower
// experts, of earlier chunks, of earlier warps and of earlier slots of its run.
// Up to 1024 slots are one CTA's; above, a first kernel leaves every chunk's counts
// and the last, which counts its own chunk again while the one before ends, needs the
// sums over those of the chunks before.  Where a warp has all chunks of eight keys in
// one load each CTA adds them up itself; a kernel between the two does it for more.
// Bound by latency: 512 slots of 32 experts 2.8 us, 16384 4.1, 65536 5.1, of 512
// experts 6.8; 262144 of 512 9.8.  (Chunks of 2048 slots, one CTA up to 4096: 4096 of
// 32 experts 8.4 us instead of 4.7; without the kernel between 65536 of 32 7.5 instead
// of 6.1; votes again for the placement and counters without atomics: 5.5 and 7.2 for
// the 5.1 and 6.8.)  Atomics only add within a warp's own counters, so equal ids keep
// their order.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 512;  // least slots of a chunk, where there are several
constexpr int kSortMaxChunks = 256;
constexpr int kSortKeys = 128;  // the most keys whose counts every CTA adds up itself, of at most 32 chunks

int64_t sort_chunk(int64_t P) {
  if (P <= 2 * kSortChunk) return 2 * kSortChunk;  // one CTA, one launch
  const int64_t per = (P + kSortMaxChunks - 1) / kSortMaxChunks;
  return (std::max<int64_t>(per, kSortChunk) + kSortThreads - 1) / kSortThreads * kSortThreads;
}
int64_t sort_chunks(int64_t P) { const int64_t c = sort_chunk(P); return (P + c - 1) / c; }

// Calls f(q, i, e) for every 32 slots of [i0, i1), a slot per lane: e is the slot's
// expert, E for an empty one (and for an id that is not below E), -1 past the end.
// Four loads are in flight, q counts them.
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
      f(q, at, at >= i1 ? -1 : id[q] < 0 || id[q] >= E ? E : id[q]);
    }
  }
  return bad;
}

// The lanes whose slot has this one's expert: a vote for each bit of e, of which
// those past the end (-1) have all, the others not.  (__match_any takes 200 clocks
// for 32 different experts: 262144 slots of 512 experts 9.8 us, 10.5 with it; 1048576
// of 8 13.7, 11.2.)
MXG_DEVINL uint32_t same_expert(int e, int bits) {
  uint32_t same = kFull;
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    if (b >= bits) break;
    const bool on = (e >> b) & 1;
    const uint32_t with = __ballot_sync(kFull, on);
    same &= on ? with : ~with;
  }
  return same;
}
MXG_DEVINL int expert_bits(int E) { return 32 - __clz(E + 1); }

// cnt[0..E]: the slots of each expert in the warp's run.  Of its last 32 kSortFlight
// slots e and same are the experts and the lanes that share them.
MXG_DEVINL bool count_run(const int32_t* ids, int64_t i0, int64_t i1, int E, uint32_t* cnt, int* e, uint32_t* same) {
  const int lane = threadIdx.x & 31, bits = expert_bits(E);
  return for_slots(ids, i0, i1, E, [&](int q, int64_t, int at) {
    e[q] = at;
    same[q] = same_expert(at, bits);
    if (at >= 0 && lane == __ffs(same[q]) - 1) atomicAdd(cnt + at, __popc(same[q]));
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
  int e_of[kSortFlight];
  uint32_t same_of[kSortFlight];
  count_run(ids, i0, i1, E, cnt + warp * keys, e_of, same_of);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += kSortThreads) {
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) v += cnt[w * keys + e];
    counts[(int64_t)e * gridDim.x + blockIdx.x] = (int32_t)v;
  }
}

// counts[e][.] -> their exclusive prefix sums, totals[e].  A warp takes a key.
__global__ void __launch_bounds__(kSortThreads) moe_sort_scan_kernel(int32_t* counts, int32_t* totals, int keys, int chunks) {
  const int lane = threadIdx.x & 31, e = blockIdx.x * kSortWarps + (threadIdx.x >> 5);
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  if (e >= keys) return;
  uint32_t v[kSortMaxChunks / 32], at = 0;
#pragma unroll
  for (int i = 0; i < kSortMaxChunks / 32; ++i) {
    const int c = 32 * i + lane;
    v[i] = c < chunks ? (uint32_t)ptx::ld_global_s32(counts + (int64_t)e * chunks + c) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kSortMaxChunks / 32; ++i) {
    if (32 * i >= chunks) break;
    uint32_t incl = v[i];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += o;
    }
    const int c = 32 * i + lane;
    if (c < chunks) counts[(int64_t)e * chunks + c] = (int32_t)(at + incl - v[i]);
    at += __shfl_sync(kFull, incl, 31);
  }
  if (lane == 0) totals[e] = (int32_t)at;
}

__global__ void __launch_bounds__(kSortThreads) moe_sort_place_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                                      int64_t chunk, const int32_t* counts,
                                                                      const int32_t* totals,  // with prefix sums in counts
                                                                      int32_t* __restrict__ m_splits,
                                                                      int32_t* __restrict__ rows, int32_t* status) {
  extern __shared__ uint32_t cnt[];  // [warps][E + 1]
  __shared__ uint32_t total[2 * kSortThreads], before[2 * kSortThreads];  // of a key: all slots, those of earlier chunks
  __shared__ uint32_t warp_sum[kSortWarps];
  const int keys = E + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::pdl_launch_dependents();
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * chunk, run = chunk / kSortWarps;
  const int64_t i0 = min(P, c0 + warp * run), i1 = min(P, i0 + run);
  int e_of[kSortFlight];
  uint32_t same_of[kSortFlight];
  const bool bad = count_run(ids, i0, i1, E, cnt + warp * keys, e_of, same_of);
  if (__syncthreads_or(bad) && threadIdx.x == 0) report(status, MXG_ERR_INDEX);

  if (gridDim.x == 1) {
    for (int e = threadIdx.x; e < keys; e += kSortThreads) {
      uint32_t v = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) v += cnt[w * keys + e];
      total[e] = v;
      before[e] = 0;
    }
  } else if (totals != nullptr) {
    ptx::pdl_wait();  // the counts are complete
    for (int e = threadIdx.x; e < keys; e += kSortThreads) {
      total[e] = (uint32_t)ptx::ld_global_s32(totals + e);
      before[e] = (uint32_t)ptx::ld_global_s32(counts + (int64_t)e * gridDim.x + blockIdx.x);
    }
  } else {
    ptx::pdl_wait();  // the counts are complete
    // at most kSortKeys keys and 32 chunks: eight keys of a warp in flight, its lanes the chunks
    const int chunks = (int)gridDim.x;
    uint32_t v[kSortKeys / kSortWarps];
#pragma unroll
    for (int q = 0; q < kSortKeys / kSortWarps; ++q) {
      const int e = warp + q * kSortWarps;
      v[q] = e < keys && lane < chunks ? (uint32_t)ptx::ld_global_s32(counts + (int64_t)e * chunks + lane) : 0u;
    }
#pragma unroll
    for (int q = 0; q < kSortKeys / kSortWarps; ++q) {
      const int e = warp + q * kSortWarps;
      const uint32_t all = __reduce_add_sync(kFull, v[q]);
      const uint32_t early = __reduce_add_sync(kFull, lane < (int)blockIdx.x ? v[q] : 0u);
      if (lane == 0 && e < keys) {
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
      uint32_t pos = at + before[e], m[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) m[w] = cnt[w * keys + e];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        cnt[w * keys + e] = pos;
        pos += m[w];
      }
    }
    at += q ? t1 : t0;
  }
  __syncthreads();

  uint32_t* mine = cnt + warp * keys;
  auto place = [&](int64_t i, int e, uint32_t same) {
    const int rank = __popc(same & ((1u << lane) - 1u));
    uint32_t first = 0;
    if (e >= 0 && rank == 0) first = atomicAdd(mine + e, __popc(same));
    first = __shfl_sync(kFull, first, __ffs(same) - 1);
    if (e >= 0) {
      const int r = (int)(first + rank);
      rows[i] = e == E ? -1 - r : r;
    }
    __syncwarp();  // one 32 slots after another
  };
  if (run <= 32 * kSortFlight) {  // as counted
#pragma unroll
    for (int q = 0; q < kSortFlight; ++q)
      if (i0 + 32 * q < i1) place(i0 + 32 * q + lane, e_of[q], same_of[q]);
  } else {
    const int bits = expert_bits(E);
    for_slots(ids, i0, i1, E, [&](int, int64_t i, int e) { place(i, e, same_expert(e, bits)); });
  }
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

// Gather and combine: blockDim.x threads share a row's pieces, blockDim.y tokens a CTA.
constexpr int kRowThreads = 256;
// As many threads as share a row's pieces equally (896 pieces: 4 times 224; with
// 256 threads combine takes 186 us instead of 173 for 65536 rows of 7168); of short rows
// as many tokens as make up a CTA of 128 (8 rows of 32 BF16 values for each of 32768
// tokens: 5.6 us, 19.7 with a CTA for every token; top 8 of 256 6.1 TB/s, 5.7 with 256
// threads).
dim3 row_block(int64_t pieces) {
  const int64_t turns = (pieces + kRowThreads - 1) / kRowThreads;
  const unsigned x = (unsigned)((pieces + turns - 1) / turns);
  return x > kRowThreads / 4 ? dim3((x + 31) / 32 * 32) : dim3(x, kRowThreads / 2 / x);
}
dim3 row_grid(int64_t tokens, int64_t pieces, dim3 block) {
  return dim3((unsigned)((tokens + block.y - 1) / block.y),
              (unsigned)std::min<int64_t>(65535, (pieces + block.x - 1) / block.x));
}

// A token's row is read once and written to its k rows.  Bound by HBM: 8192 tokens of
// 7168, top 8, 162 us, 6.5 TB/s, nearly all of it writes.
__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(const uint4* __restrict__ x, int64_t ld_x,
                                                                 const int32_t* __restrict__ rows, int64_t T, int k,
                                                                 int64_t pieces, uint4* __restrict__ out, int64_t ld_out,
                                                                 int32_t* status) {
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, P = T * k;
  if (t >= T) return;
  const int32_t* mine = rows + t * k;
  ptx::pdl_wait();  // rows, and x too, may come from the kernel before
  for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < pieces; c += (int64_t)gridDim.y * blockDim.x) {
    const uint4 v = ptx::ld_global_v4(x + t * ld_x + c);
    for (int j = 0; j < k; ++j) {
      const int32_t e = ptx::ld_global_s32(mine + j);
      const int64_t r = row_of(e, P, status);
      if (r >= 0) out[r * ld_out + c] = e >= 0 ? v : make_uint4(0, 0, 0, 0);
    }
  }
}

// A thread sums one piece over a token's slots, four rows in flight (8192 tokens, top 8
// of 4096: 6.2 TB/s, 5.8 with eight, which take more registers).  Every row is read
// once and not again, so the loads and stores are marked as streaming: 65536 rows of
// 7168 to 8192, 163 us, 6.5 TB/s; 173 with plain ones.  kShort: rows so short that a CTA
// has several tokens.
template <typename T, bool kShort>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const uint4* __restrict__ y, int64_t ld_y, int64_t y_rows,
                                                                  const int32_t* __restrict__ rows,
                                                                  const float* __restrict__ weights, int64_t tokens, int k,
                                                                  int64_t pieces, uint4* __restrict__ out,
                                                                  int64_t ld_out, int32_t* status) {
  constexpr int n = Piece<T>::n;
  constexpr int kFlight = 4;  // rows in flight
  const int64_t t = kShort ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
  if (kShort && t >= tokens) return;
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

// The same for up to kSlots slots, all in flight, of kTokens tokens at a time: four where
// there is one slot (32768 rows of 2048: 44 us, 94 with the above), else one, which
// leaves room for more CTAs (top 4 of 4096: 6.0 TB/s, 4.6 with two; top 2: 6.2, 5.0 with
// four; top 6: 5.9, 5.8 with the above).
template <typename T, int kTokens, int kSlots>
__global__ void __launch_bounds__(kRowThreads) moe_combine_few_kernel(const uint4* __restrict__ y, int64_t ld_y,
                                                                      int64_t y_rows, const int32_t* __restrict__ rows,
                                                                      const float* __restrict__ weights, int64_t tokens,
                                                                      int k, int pieces, uint4* __restrict__ out,
                                                                      int64_t ld_out, int32_t* status) {
  constexpr int n = Piece<T>::n;
  const int64_t t0 = (int64_t)blockIdx.x * (blockDim.y * kTokens) + threadIdx.y;  // then every blockDim.y-th
  int64_t row[kTokens][kSlots];
  float w[kTokens][kSlots];
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    const int64_t t = t0 + (int64_t)u * blockDim.y;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      row[u][j] = -1;
      w[u][j] = 1.0f;
      if (t < tokens && j < k) {
        const int32_t e = __ldg(rows + t * k + j);
        if (weights != nullptr) w[u][j] = __ldg(weights + t * k + j);
        if (e >= 0) row[u][j] = row_of(e, y_rows, status);
      }
    }
  }
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < pieces; c += gridDim.y * blockDim.x) {
    uint4 v[kTokens][kSlots];
#pragma unroll
    for (int u = 0; u < kTokens; ++u)
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (row[u][j] >= 0) v[u][j] = __ldcs(y + row[u][j] * ld_y + c);
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      float s[n];
#pragma unroll
      for (int i = 0; i < n; ++i) s[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (row[u][j] < 0) continue;
        float f[n];
        widen<T>(v[u][j], f);
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = fmaf(w[u][j], f[i], s[i]);
      }
      const int64_t t = t0 + (int64_t)u * blockDim.y;
      if (t < tokens) __stcs(out + t * ld_out + c, narrow<T>(s));
    }
  }
}

// `share` threads take a token: kPieces pieces of dout at a time, once for every kFlight
// slots, whose products with y they sum, then over the threads in a fixed order.  share
// is a power of two up to 32 (lanes of a warp, 256 / share tokens a CTA) or the whole
// CTA.  y and dy may be one buffer: a piece is read by the thread that writes it.
// Bound by HBM: 65536 rows of 4096, 172 us, 6.6 TB/s (177 with streaming loads and
// stores, 199 with eight slots in flight and fewer warps for it).
template <typename T, int kPieces, int kFlight, int kThreads, bool kLanes>
__global__ void __launch_bounds__(kThreads) moe_combine_backward_kernel(
    const uint4* __restrict__ dout, int64_t ld_dout, const uint4* y, int64_t ld_y, const int32_t* __restrict__ rows,
    const float* __restrict__ weights, int64_t tokens, int k, int pieces, int share, uint4* dy, int64_t ld_dy,
    float* __restrict__ dweights, int32_t* status) {
  constexpr int n = Piece<T>::n;
  __shared__ float part[kThreads / 32][kFlight];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = kLanes ? threadIdx.x & (share - 1) : threadIdx.x;
  const int64_t t = kLanes ? (int64_t)blockIdx.x * (blockDim.x / share) + threadIdx.x / share : blockIdx.x;
  const int last = !kLanes || t < tokens ? pieces : 0;  // all threads of a warp take part in its sums
  const int slots = !kLanes || t < tokens ? k : 0;
  rows += t * k;
  weights += t * k;
  dweights += t * k;
  dout += t * ld_dout;
  for (int j0 = 0; j0 < k; j0 += kFlight) {
    int64_t at[kFlight];
    float w[kFlight], dot[kFlight];
    bool on[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      at[j] = -1;
      on[j] = false;
      w[j] = dot[j] = 0.0f;
      if (j0 + j < slots) {
        const int32_t e = __ldg(rows + j0 + j);
        at[j] = row_of(e, tokens * k, status);
        on[j] = e >= 0 && at[j] >= 0;
        if (on[j]) w[j] = __ldg(weights + j0 + j);
      }
    }
    for (int c0 = me; c0 < last; c0 += kPieces * share) {
      uint4 d4[kPieces], v[kPieces][kFlight];
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int c = c0 + q * share;
        if (kPieces == 1 || c < pieces) {
          d4[q] = __ldg(dout + c);
#pragma unroll
          for (int j = 0; j < kFlight; ++j)
            if (on[j]) v[q][j] = y[at[j] * ld_y + c];
        }
      }
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int c = c0 + q * share;
        if (kPieces == 1 || c < pieces) {
          float d[n];
          widen<T>(d4[q], d);
#pragma unroll
          for (int j = 0; j < kFlight; ++j) {
            float f[n];
            if (on[j]) {
              widen<T>(v[q][j], f);
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
      }
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      for (int s = kLanes ? share >> 1 : 16; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(kFull, dot[j], s);
    if constexpr (kLanes) {
#pragma unroll
      for (int j = 0; j < kFlight; ++j)
        if (me == 0 && j0 + j < slots) dweights[j0 + j] = dot[j];
    } else {
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kFlight; ++j) part[warp][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < kFlight && j0 + (int)threadIdx.x < k) {
        float s = 0.0f;
        for (int q = 0; q < (int)(blockDim.x >> 5); ++q) s += part[q][threadIdx.x];
        dweights[j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

}  // namespace

size_t moe_sort_workspace_bytes(int64_t P, int E) {
  const int64_t n = sort_chunks(P);
  return std::max<size_t>(256, n > 1 ? ((size_t)n + 1) * (E + 1) * sizeof(int32_t) : 0);  // counts, totals
}

cudaError_t launch_moe_sort(const int32_t* ids, int64_t P, int E, int32_t* m_splits, int32_t* rows, void* ws,
                            int32_t* status, cudaStream_t stream) {
  const int64_t chunk = sort_chunk(P);
  const unsigned chunks = (unsigned)std::max<int64_t>(1, sort_chunks(P));
  const size_t smem = (size_t)kSortWarps * (E + 1) * sizeof(uint32_t);
  int32_t* counts = static_cast<int32_t*>(ws);
  if (chunks == 1) {
    moe_sort_place_kernel<<<1, kSortThreads, smem, stream>>>(ids, P, E, chunk, counts, nullptr, m_splits, rows, status);
    return cudaGetLastError();
  }
  moe_sort_count_kernel<<<chunks, kSortThreads, smem, stream>>>(ids, P, E, chunk, counts);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int32_t* totals = nullptr;
  if (chunks > 32 || E + 1 > kSortKeys) {
    int32_t* sums = counts + (int64_t)chunks * (E + 1);
    const cudaError_t s = launch_overlapped(moe_sort_scan_kernel, dim3((unsigned)((E + kSortWarps) / kSortWarps)), dim3(kSortThreads),
                                            0, stream, counts, sums, E + 1, (int)chunks);
    if (s != cudaSuccess) return s;
    totals = sums;
  }
  return launch_overlapped(moe_sort_place_kernel, dim3(chunks), dim3(kSortThreads), smem, stream, ids, P, E, chunk,
                           static_cast<const int32_t*>(counts), totals, m_splits, rows, status);
}

cudaError_t launch_moe_gather(const void* x, int64_t ld_x, const int32_t* rows, int64_t T, int k, int64_t pieces,
                              void* out, int64_t ld_out, int32_t* status, cudaStream_t stream) {
  const dim3 block = row_block(pieces);
  return launch_overlapped(moe_gather_kernel, row_grid(T, pieces, block), block, 0, stream, static_cast<const uint4*>(x), ld_x, rows, T, k,
                           pieces, static_cast<uint4*>(out), ld_out, status);
}

namespace {
template <typename T>
cudaError_t combine(const void* y, int64_t ld_y, int64_t y_rows, const int32_t* rows, const float* weights, int64_t tokens,
                    int k, int64_t pieces, void* out, int64_t ld_out, int32_t* status, cudaStream_t stream) {
  const dim3 block = row_block(pieces);
  const uint4* from = static_cast<const uint4*>(y);
  uint4* to = static_cast<uint4*>(out);
  if (k > 6) {
    const auto fn = block.y > 1 ? moe_combine_kernel<T, true> : moe_combine_kernel<T, false>;
    fn<<<row_grid(tokens, pieces, block), block, 0, stream>>>(from, ld_y, y_rows, rows, weights, tokens, k, pieces, to,
                                                             ld_out, status);
    return cudaGetLastError();
  }
  const int each = k > 1 ? 1 : 4;  // tokens of a thread
  const auto fn = k > 5   ? moe_combine_few_kernel<T, 1, 6>
                  : k > 4 ? moe_combine_few_kernel<T, 1, 5>
                  : k > 3 ? moe_combine_few_kernel<T, 1, 4>
                  : k > 2 ? moe_combine_few_kernel<T, 1, 3>
                  : k > 1 ? moe_combine_few_kernel<T, 1, 2>
                          : moe_combine_few_kernel<T, 4, 1>;
  fn<<<row_grid((tokens + each - 1) / each, pieces, block), block, 0, stream>>>(from, ld_y, y_rows, rows, weights, tokens, k,
                                                                               (int)pieces, to, ld_out, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t combine_backward(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y, const int32_t* rows,
                             const float* weights, int64_t tokens, int k, int64_t pieces, void* dy, int64_t ld_dy,
                             float* dweights, int32_t* status, cudaStream_t stream, int num_sms) {
  // Four rows of a thread in flight: of four slots, of three where that leaves fewer
  // unused (top 6 of 2880: 6.4 TB/s, 6.0 with four), or of fewer slots' pieces.  A
  // token has lanes of a warp, or a CTA of as many threads as share its pieces equally:
  // from 32 (top 8 of 256: 6.1 TB/s, 4.9 with eight tokens' warps in a CTA) up to 256,
  // or 1024 where there are few tokens (64 of 7168, top 8: 8.2 us, 11.9).
  const int each = k > 2 ? 1 : k > 1 ? 2 : 4;
  const int64_t want = (pieces + each - 1) / each;
  const bool lanes = want <= 16, few = !lanes && tokens < 4 * num_sms;
  int share = 1, threads = kRowThreads;
  if (lanes) {
    while (share < want) share *= 2;
  } else {
    const int64_t most = few ? 1024 : kRowThreads, turns = (want + most - 1) / most;
    share = threads = (int)(((want + turns - 1) / turns + 31) / 32 * 32);
  }
  const bool three = (k + 2) / 3 * 3 < (k + 3) / 4 * 4;
  const auto pick = [&](auto one, auto one3, auto two, auto four) {
    return each == 1 ? (three ? one3 : one) : each == 2 ? two : four;
  };
  const auto fn = lanes ? pick(moe_combine_backward_kernel<T, 1, 4, kRowThreads, true>,
                               moe_combine_backward_kernel<T, 1, 3, kRowThreads, true>,
                               moe_combine_backward_kernel<T, 2, 2, kRowThreads, true>,
                               moe_combine_backward_kernel<T, 4, 1, kRowThreads, true>)
                  : few ? pick(moe_combine_backward_kernel<T, 1, 4, 1024, false>,
                               moe_combine_backward_kernel<T, 1, 3, 1024, false>,
                               moe_combine_backward_kernel<T, 2, 2, 1024, false>,
                               moe_combine_backward_kernel<T, 4, 1, 1024, false>)
                        : pick(moe_combine_backward_kernel<T, 1, 4, kRowThreads, false>,
                               moe_combine_backward_kernel<T, 1, 3, kRowThreads, false>,
                               moe_combine_backward_kernel<T, 2, 2, kRowThreads, false>,
                               moe_combine_backward_kernel<T, 4, 1, kRowThreads, false>);
  const int64_t ctas = lanes ? (tokens + threads / share - 1) / (threads / share) : tokens;
  fn<<<(unsigned)ctas, threads, 0, stream>>>(static_cast<const uint4*>(dout), ld_dout, static_cast<const uint4*>(y), ld_y,
                                             rows, weights, tokens, k, (int)pieces, share, static_cast<uint4*>(dy), ld_dy,
                                             dweights, status);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_moe_combine(const void* y, int64_t ld_y, int64_t y_rows, const int32_t* rows, const float* weights,
                               int64_t T, int k, int64_t pieces, bool bf16, void* out, int64_t ld_out, int32_t* status,
                               cudaStream_t stream) {
  const auto fn = bf16 ? combine<__nv_bfloat16> : combine<float>;
  return fn(y, ld_y, y_rows, rows, weights, T, k, pieces, out, ld_out, status, stream);
}

cudaError_t launch_moe_combine_backward(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y,
                                        const int32_t* rows, const float* weights, int64_t T, int k, int64_t pieces,
                                        bool bf16, void* dy, int64_t ld_dy, float* dweights, int32_t* status,
                                        cudaStream_t stream, int num_sms) {
  const auto fn = bf16 ? combine_backward<__nv_bfloat16> : combine_backward<float>;
  return fn(dout, ld_dout, y, ld_y, rows, weights, T, k, pieces, dy, ld_dy, dweights, status, stream, num_sms);
}

}  // namespace mxg
