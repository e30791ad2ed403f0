// Low-rank adapters of many requests beside a shared projection:
//   out[t] = y[t] + scale[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// shrink: u[t] = A[a] x[t], split over K, fp32 partials to the workspace;
// expand: sums the partials in order and adds scale * B u to y.
// Both are bound by memory: x, y, and R (K + N) values of each adapter used.
//
// Few tokens: a CTA works for one token, reads the token's adapter rows 16 bytes
// a lane and multiplies in fp32.  Tokens that share an adapter read it again,
// from L2; every load of a CTA is in flight at once.  64 tokens of 64 adapters
// (K = N = 7168, rank 16): 7.8 us from DRAM, 6.2 from L2, about half of it the two
// launches; one token 3.8 us.
//
// Many tokens: the tokens are ordered by adapter (a third kernel), and a CTA
// runs a tile of 128 of them against the adapters that occur in it on the
// tensor core (tcgen05, BF16 x BF16 + FP32); products of rows that are not
// wanted cost little.  A row of the result is selected, never masked by a
// product: an adapter's infinities or NaN reach its own tokens only.  u keeps its
// fp32 accuracy as a sum of two BF16 terms (2^-17; BF16 output) or three (2^-25;
// FP32 output); a product that comes out infinite or NaN is done again in fp32.
//   8192 tokens, 8192 x 28672, rank 32, prompts of 1024 tokens: 206 us, 5.4 TB/s
//   of the 1.11 GB it has to move (164 us at the copy rate).  Expand is about
//   three quarters of that; reads and writes of y share DRAM at 67 to 80 %.
//   Left in the batch's order the same takes about 5 us less, but 1024 tokens of 64 mixed
//   adapters (4096 x 4096, rank 16) take 200 us instead of 37.
//   Tokens without an adapter are copied by the last tiles of a segment, a load
//   behind each store: the first such tile lengthens a call by 30 to 120 us (206 ->
//   318 here); in place there is nothing to copy.
//   mma.sync runs at 1/16 of the tcgen05 rate here: a form on it took 264 us.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "gemm_common.cuh"
#include "sm100_ptx.cuh"

namespace mxg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kLoraWarps = 4;
constexpr int kLoraThreads = kLoraWarps * 32;

struct LoraParams {
  LoraArgs a;
  float* u;         // [ksplit][T][R] partial sums (tiles: rows in the order of `order`)
  int32_t* order;   // tiles: [T] tokens, by adapter within each segment
  int ksplit;
  int blocks;       // tiles: 64-element steps of K per CTA of the shrink
  int cols;         // tiles: columns per CTA of the expand
  uint64_t timeout_ns, drain_ns;
};

// ---------------------------------------------------------------------------
// Few tokens: shrink, grid (K split, tokens, rank groups of 16).  A warp takes
// 256 elements of K, 8 a lane.
// ---------------------------------------------------------------------------
constexpr int kTokK = 8 * 32 * kLoraWarps;  // elements of K per CTA
constexpr int kTokR = 16;

// acc += sum of the products of two 8-element BF16 vectors
MXG_DEVINL float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t* u = &a.x;
  const uint32_t* v = &b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf16lo_to_f32(u[i]), bf16lo_to_f32(v[i]), acc);
    acc = fmaf(bf16hi_to_f32(u[i]), bf16hi_to_f32(v[i]), acc);
  }
  return acc;
}

__global__ void __launch_bounds__(kLoraThreads) lora_shrink_token_kernel(const LoraParams p) {
  __shared__ float red[kLoraWarps][kTokR];
  ptx::pdl_launch_dependents();
  const LoraArgs& a = p.a;
  const int64_t t = blockIdx.y;
  const int id = __ldg(a.ids + t);
  if (id < 0) return;
  if (id >= a.n) {
    if (threadIdx.x == 0) report(a.status, MXG_ERR_INDEX);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t k = (int64_t)blockIdx.x * kTokK + threadIdx.x * 8;
  const int r0 = blockIdx.z * kTokR;
  float v[kTokR];
  if (k < a.K) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.x + t * a.ld_x + k));
    const uint16_t* A = a.A + ((int64_t)id * a.R + r0) * a.K + k;
    uint4 w[kTokR];
#pragma unroll
    for (int r = 0; r < kTokR; ++r) {
      w[r] = make_uint4(0, 0, 0, 0);
      if (r0 + r < a.R) w[r] = __ldg(reinterpret_cast<const uint4*>(A + r * a.K));
    }
#pragma unroll
    for (int r = 0; r < kTokR; ++r) v[r] = r0 + r < a.R ? dot8(x, w[r], 0.0f) : 0.0f;
  } else {
#pragma unroll
    for (int r = 0; r < kTokR; ++r) v[r] = 0.0f;
  }
  // sum over the lanes, halving the ranks a lane holds: lane l ends with rank l / 2
#pragma unroll
  for (int d = 16; d >= 2; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < d / 2; ++i) {
      const float send = up ? v[i] : v[i + d / 2];
      const float keep = up ? v[i + d / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(kFull, send, d);
    }
  }
  v[0] += __shfl_xor_sync(kFull, v[0], 1);
  if ((lane & 1) == 0) red[warp][lane >> 1] = v[0];
  __syncthreads();
  const int r = threadIdx.x;
  if (r < kTokR && r0 + r < a.R)
    p.u[((int64_t)blockIdx.x * a.T + t) * a.R + r0 + r] = (red[0][r] + red[1][r]) + (red[2][r] + red[3][r]);
}

// Sum of a token's partial u, in order of the split.
MXG_DEVINL float sum_u(const LoraParams& p, int64_t t, int r) {
  const float* src = p.u + t * p.a.R + r;
  const int64_t step = p.a.T * p.a.R;
  float s = 0.0f;
  for (int k0 = 0; k0 < p.ksplit; k0 += 8) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k0 + k < p.ksplit ? __ldcg(src + (k0 + k) * step) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[k];
  }
  return s;
}

// Few tokens: expand, grid (column chunks, tokens).  A thread takes four columns
// a CTA's width apart; the first ranks of B and y are loaded before u is awaited.
constexpr int kTokCols = 4;

template <typename TOut>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_token_kernel(const LoraParams p) {
  __shared__ float us[128];
  const LoraArgs& a = p.a;
  const int64_t t = blockIdx.y;
  const int id = __ldg(a.ids + t);
  const bool on = id >= 0 && id < a.n;
  const int64_t c0 = (int64_t)blockIdx.x * (kLoraThreads * kTokCols) + threadIdx.x;
  const TOut* y = static_cast<const TOut*>(a.y) + t * a.ld_y;
  TOut* out = static_cast<TOut*>(a.out) + t * a.ld_out;
  const uint16_t* B = a.B + (int64_t)(on ? id : 0) * a.N * a.R;
  float acc[kTokCols], yv[kTokCols];
  uint4 w[kTokCols][2];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < kTokCols; ++i) {
      const int64_t c = c0 + i * kLoraThreads;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[i][h] = make_uint4(0, 0, 0, 0);
        if (on && c < a.N && r + 8 * h < a.R) w[i][h] = __ldg(reinterpret_cast<const uint4*>(B + c * a.R + r) + h);
      }
    }
  };
  load(0);
#pragma unroll
  for (int i = 0; i < kTokCols; ++i) {
    const int64_t c = c0 + i * kLoraThreads;
    acc[i] = 0.0f;
    yv[i] = c < a.N ? (float)y[c] : 0.0f;
  }
  ptx::pdl_wait();
  if (on) {
    for (int r = threadIdx.x; r < a.R; r += kLoraThreads) {
      const float s = sum_u(p, t, r);
      us[r] = a.scale != nullptr ? s * __ldg(a.scale + id) : s;
    }
    __syncthreads();
    for (int r = 0; r < a.R; r += 16) {
      if (r > 0) load(r);
#pragma unroll
      for (int i = 0; i < kTokCols; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r + 8 * h < a.R) {
            const uint32_t* b = &w[i][h].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[i] = fmaf(bf16lo_to_f32(b[j]), us[r + 8 * h + 2 * j], acc[i]);
              acc[i] = fmaf(bf16hi_to_f32(b[j]), us[r + 8 * h + 2 * j + 1], acc[i]);
            }
          }
    }
  }
#pragma unroll
  for (int i = 0; i < kTokCols; ++i) {
    const int64_t c = c0 + i * kLoraThreads;
    if (c < a.N) out[c] = (TOut)(on ? yv[i] + acc[i] : yv[i]);
  }
}

// ---------------------------------------------------------------------------
// Many tokens
// ---------------------------------------------------------------------------
constexpr int kTile = 128;          // tokens of a tile (TMEM lanes)
constexpr int kRowBytes = 128;      // one swizzled shared-memory row: 64 BF16 of the contraction
constexpr int kTileBytes = kTile * kRowBytes;

// Order of the tokens: within each segment of 8192, by adapter, tokens without
// one last; a CTA per segment counts, sums and places.  So a tile meets about
// 1 + adapters / (tiles of its segment, 64 at most) instead of up to 128.  The order among a
// segment's tokens of one adapter goes by the atomics; a token's result does not
// depend on its place.  Where the counters do not fit, the order is the batch's.
constexpr int kSegment = 8192;
constexpr int kOrderThreads = 1024;
constexpr int kOrderPer = kSegment / kOrderThreads;
constexpr int kCounters = 8192;  // adapters + 1 at most
constexpr int kCountPer = kCounters / kOrderThreads;

__global__ void __launch_bounds__(kOrderThreads) lora_order_kernel(const LoraParams p) {
  __shared__ int count[kCounters];
  __shared__ int warp_sum[32];
  ptx::pdl_launch_dependents();
  const LoraArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = (int64_t)blockIdx.x * kSegment;
  const bool sort = a.n < kCounters;
  int bucket[kOrderPer], rank[kOrderPer];
#pragma unroll
  for (int i = 0; i < kOrderPer; ++i) {
    const int64_t t = t0 + i * kOrderThreads + tid;
    const int id = t < a.T ? __ldg(a.ids + t) : -1;
    if (id >= a.n) report(a.status, MXG_ERR_INDEX);
    bucket[i] = t >= a.T ? -1 : id < 0 || id >= a.n ? a.n : id;  // -1: no token
  }
  if (!sort) {
#pragma unroll
    for (int i = 0; i < kOrderPer; ++i) {
      const int64_t t = t0 + i * kOrderThreads + tid;
      if (t < a.T) p.order[t] = (int32_t)t;
    }
    return;
  }
  for (int i = tid; i <= a.n; i += kOrderThreads) count[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOrderPer; ++i) {
    if (t0 + i * kOrderThreads >= a.T) continue;
    const uint32_t same = __match_any_sync(kFull, bucket[i]);
    const int leader = __ffs(same) - 1;
    int base = 0;
    if (lane == leader && bucket[i] >= 0) base = atomicAdd(&count[bucket[i]], __popc(same));
    rank[i] = __shfl_sync(kFull, base, leader) + __popc(same & ((1u << lane) - 1u));
  }
  __syncthreads();
  // exclusive sums: a thread has kCountPer counters in a row
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kCountPer; ++i) {
    const int b = tid * kCountPer + i;
    if (b <= a.n) sum += count[b];
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  const int before = __reduce_add_sync(kFull, lane < warp ? warp_sum[lane] : 0);
  int at = before + incl - sum;
#pragma unroll
  for (int i = 0; i < kCountPer; ++i) {
    const int b = tid * kCountPer + i;
    if (b <= a.n) {
      const int c = count[b];
      count[b] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOrderPer; ++i) {
    const int64_t t = t0 + i * kOrderThreads + tid;
    if (bucket[i] >= 0) p.order[t0 + count[bucket[i]] + rank[i]] = (int32_t)t;
  }
}

// The tokens of a tile and the adapters of their runs.
struct Tile {
  int tok[kTile];      // token (-1: past the last)
  int id[kTile];       // its adapter (-1: none)
  int16_t ord[kTile];  // the number of its run in the list (-1: none)
  int list[kTile];     // adapter of each run
  int warp_runs[4];
  int count;
};

// All threads of the CTA (at least kTile), once the order is written.
MXG_DEVINL void read_tile(Tile& s, const LoraParams& p, int64_t t0) {
  const int tid = threadIdx.x, lane = tid & 31;
  int id = -1;
  if (tid < kTile) {
    const int tok = t0 + tid < p.a.T ? __ldcg(p.order + t0 + tid) : -1;
    if (tok >= 0) id = __ldg(p.a.ids + tok);
    if (id >= p.a.n) id = -1;  // reported with the order
    s.tok[tid] = tok;
    s.id[tid] = id;
  }
  __syncthreads();
  uint32_t starts = 0;
  bool first = false;
  if (tid < kTile) {
    first = id >= 0 && (tid == 0 || s.id[tid - 1] != id);
    starts = __ballot_sync(kFull, first);
    if (lane == 0) s.warp_runs[tid >> 5] = __popc(starts);
  }
  __syncthreads();
  if (tid < kTile) {
    int o = __popc(starts & (0xFFFFFFFFu >> (31 - lane))) - 1;
    for (int w = 0; w < (tid >> 5); ++w) o += s.warp_runs[w];
    s.ord[tid] = (int16_t)(id >= 0 ? o : -1);
    if (first) s.list[o] = id;
    if (tid == kTile - 1) s.count = o + 1;
  }
  __syncthreads();
}

// Instruction descriptor of kind::f16: BF16 x BF16 -> FP32, both K-major, M = 128.
MXG_DEVINL uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// shrink: grid (K split, tiles, passes), 320 threads: warp 0 loads A (TMA), warp 1 issues
// the MMAs, warps 2-5 store, warps 6-9 gather the tokens' rows of x.  x is the M
// operand; the rows of up to 256 / R adapters of the tile form one N operand, a
// pass; passes go to several CTAs where there are few tiles.
constexpr int kShrinkThreads = 320;
constexpr int kShrinkRows = 256;  // adapter rows of one pass
constexpr int kShrinkStage = kTileBytes + kShrinkRows * kRowBytes;
constexpr int kShrinkStages = 4;
constexpr int kShrinkSmem = kShrinkStages * kShrinkStage + 1024;
constexpr int kShrinkTmem = 256;

__global__ void __launch_bounds__(kShrinkThreads, 1)
    lora_shrink_tile_kernel(const __grid_constant__ CUtensorMap tmA, const LoraParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  __shared__ Tile tile;
  __shared__ __align__(8) uint64_t bars[2 * kShrinkStages + 3];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const LoraArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kShrinkStages + s); };
  const uint32_t acc_full = bar0 + 16u * kShrinkStages, acc_empty = acc_full + 8, drain = acc_full + 16;
  ptx::pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kShrinkStages; ++s) {
      ptx::mbar_init(full_bar(s), 1 + kTile);  // warp 0; the threads of warps 6-9
      ptx::mbar_init(empty_bar(s), 1);
    }
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(acc_empty, 4);
    ptx::mbar_init(drain, 1);
    abort_word = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), kShrinkTmem);
    ptx::tmem_relinquish();
  }
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  ptx::tc_fence_before();
  ptx::pdl_wait();
  read_tile(tile, p, t0);
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int s0 = blockIdx.x * p.blocks;
  const int s1 = (int)min((a.K + 63) / 64, (int64_t)s0 + p.blocks);  // 64-element steps of this CTA
  const int per_pass = kShrinkRows / a.R;
  const int o_first = blockIdx.z * per_pass, o_step = gridDim.z * per_pass;
  const int count = tile.count;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      for (int o0 = o_first; ok && o0 < count; o0 += o_step) {
        const int na = min(per_pass, count - o0);
        for (int k = s0; k < s1; ++k) {
          if (!ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, a.status, p.timeout_ns)) { ok = false; break; }
          const uint32_t fb = full_bar(stage), sx = sbase + stage * kShrinkStage;
          ptx::mbar_arrive_expect_tx(fb, (uint32_t)(na * a.R * kRowBytes));
          armed |= 1u << stage;
          armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          for (int i = 0; i < na; ++i)
            ptx::tma_load_2d(sx + kTileBytes + i * a.R * kRowBytes, &tmA, k * 64, tile.list[o0 + i] * a.R, fb);
          if (++stage == kShrinkStages) { stage = 0; phase ^= 1u; }
        }
      }
      for (int s = 0; s < kShrinkStages; ++s)  // no copies are left in flight
        if ((armed >> s) & 1u) {
          volatile int no_abort = 0;
          ptx::mbar_wait(full_bar(s), (armed_phase >> s) & 1u, &no_abort, a.status, p.drain_ns);
        }
    }
  } else if (warp == 1) {
    const uint32_t el = ptx::elect_one();
    int stage = 0, pass = 0;
    uint32_t phase = 0;
    bool ok = true, issued = false;
    for (int o0 = o_first; ok && o0 < count; o0 += o_step, ++pass) {
      const uint32_t idesc = idesc_bf16((min(per_pass, count - o0) * a.R + 15) & ~15);
      ok = ptx::mbar_wait_warp(acc_empty, (pass & 1u) ^ 1u, abort_flag, a.status, p.timeout_ns);
      if (!ok) break;
      ptx::tc_fence_after();
      for (int k = s0; k < s1; ++k) {
        ok = ptx::mbar_wait_warp(full_bar(stage), phase, abort_flag, a.status, p.timeout_ns);
        if (!ok) break;
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_after();
        const uint64_t xd = ptx::smem_desc(sbase + stage * kShrinkStage, 16, 1024, 2);
        const uint64_t ad = ptx::smem_desc(sbase + stage * kShrinkStage + kTileBytes, 16, 1024, 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) ptx::mma_f16_if(el, tmem, xd + 2 * j, ad + 2 * j, idesc, k != s0 || j != 0);
        issued = true;
        ptx::tc_commit_if(el, empty_bar(stage));
        if (++stage == kShrinkStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      ptx::tc_commit_if(el, acc_full);
    }
    if (issued) {  // every MMA has retired before TMEM is released
      ptx::tc_commit_if(el, drain);
      volatile int no_abort = 0;
      ptx::mbar_wait(drain, 0, &no_abort, a.status, p.drain_ns);
    }
  } else if (warp >= 6) {
    // 16 bytes c of rows tid / 8, tid / 8 + 16, ...; chunk c of a row sits at c ^ (row % 8)
    const int tid = threadIdx.x - 6 * 32, c = tid & 7, r0 = tid >> 3;
    const uint32_t at = sbase + r0 * kRowBytes + ((c ^ (r0 & 7)) << 4);
    const uint16_t* src[8];
    uint32_t on = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = r0 + 16 * i;
      const bool used = tile.ord[row] >= 0;
      on |= (uint32_t)used << i;
      src[i] = a.x + (int64_t)(used ? tile.tok[row] : 0) * a.ld_x + c * 8;
    }
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int o0 = o_first; ok && o0 < count; o0 += o_step)
      for (int k = s0; k < s1; ++k) {
        ok = ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, a.status, p.timeout_ns);
        if (!ok) break;
        const bool in = k * 64 + c * 8 < a.K;  // past K: zeros
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((on >> i) & 1u)
            ptx::cp_async_16_fill(at + stage * kShrinkStage + i * 16 * kRowBytes, in ? src[i] + k * 64 : a.x, in ? 16 : 0);
        ptx::cp_async_arrive(full_bar(stage));
        if (++stage == kShrinkStages) { stage = 0; phase ^= 1u; }
      }
    ptx::cp_async_wait_all();
  } else {
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int ord = tile.ord[row];
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    float* dst = p.u + ((int64_t)blockIdx.x * a.T + t0 + row) * a.R;
    int pass = 0;
    for (int o0 = o_first; o0 < count; o0 += o_step, ++pass) {
      const bool ready = ptx::mbar_wait(acc_full, pass & 1u, abort_flag, a.status, p.timeout_ns);
      if (!__all_sync(kFull, ready)) break;
      ptx::tc_fence_after();
      const int na = min(per_pass, count - o0);
      for (int i = 0; i < na; ++i) {
        const bool mine = ord == o0 + i;
        if (!__any_sync(kFull, mine)) continue;
        for (int r = 0; r < a.R; r += 8) {
          uint32_t v[8];
          ptx::tmem_ld_32x32b_x8(tq + i * a.R + r, v);
          ptx::tmem_ld_wait();
          if (mine) ptx::st_global_v8(dst + r, v);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(acc_empty);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kShrinkTmem);
  }
}

// expand: grid (column chunks, tiles, adapter groups), 320 threads: warp 0 loads
// blocks of 128 columns of B (TMA), warp 1 issues u * B^T into one of two TMEM
// accumulators, warps 2-9 add y.  u is the M operand, as kTerms BF16 terms; a
// token's row of u is its own adapter's, and of the product with another
// adapter's B the row is not used.
// An epilogue warp has 32 rows and half of the block's columns.  Its y moves in
// pieces of 32 rows x 128 bytes through a ring of shared-memory buffers, so that
// global memory sees whole lines and two pieces are always on their way.
constexpr int kExpThreads = 320;
constexpr int kExpCols = 128;
constexpr int kPiecePitch = kRowBytes + 16;
constexpr int kPieceBytes = 32 * kPiecePitch;
constexpr int kExpTmem = 256;

template <typename TOut>
struct Exp {
  static constexpr int kTerms = sizeof(TOut) == 2 ? 2 : 3;
  static constexpr int kStages = sizeof(TOut) == 2 ? 3 : 2;  // 128 columns x 64 ranks of B each
  static constexpr int kPieces = sizeof(TOut) == 2 ? 3 : 2;
  static int smem(int R) { return (kTerms * ((R + 63) / 64) + kStages) * kTileBytes + 8 * kPieces * kPieceBytes + 1024; }
};

// y + d for the 16 bytes of a row's piece, rounded once.
template <typename TOut>
MXG_DEVINL uint4 add16(const uint4& y, const float* d);
template <>
MXG_DEVINL uint4 add16<__nv_bfloat16>(const uint4& y, const float* d) {
  uint4 o;
  const uint32_t* w = &y.x;
  uint32_t* r = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(bf16lo_to_f32(w[i]) + d[2 * i], bf16hi_to_f32(w[i]) + d[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return o;
}
template <>
MXG_DEVINL uint4 add16<float>(const uint4& y, const float* d) {
  return make_uint4(__float_as_uint(__uint_as_float(y.x) + d[0]), __float_as_uint(__uint_as_float(y.y) + d[1]),
                    __float_as_uint(__uint_as_float(y.z) + d[2]), __float_as_uint(__uint_as_float(y.w) + d[3]));
}

// u as a sum of BF16 terms: the next term of a pair of values, and what it leaves.
// A finite value past the largest BF16 starts with that one, so that the rest is
// finite too; an infinite one or NaN is the same in every term, so that each
// product has its sign.
MXG_DEVINL uint32_t bf16_term(float a, float b) {
  constexpr float kMax = 3.3895313892515355e38f;  // largest BF16
  const float ca = fabsf(a) > kMax && fabsf(a) < INFINITY ? copysignf(kMax, a) : a;
  const float cb = fabsf(b) > kMax && fabsf(b) < INFINITY ? copysignf(kMax, b) : b;
  const __nv_bfloat162 h = __floats2bfloat162_rn(ca, cb);
  return *reinterpret_cast<const uint32_t*>(&h);
}
MXG_DEVINL float left_of(float v, float term) { return fabsf(v) < INFINITY ? v - term : v; }

// Row `row` of u in shared memory ([term][64 ranks][128 rows], chunks of 16 bytes
// swizzled) for one adapter's token.
template <int kTerms>
struct URow {
  const uint8_t* at;
  int row, atoms;
  MXG_DEVINL uint4 chunk(int q, int r) const {  // ranks r .. r + 7 of term q
    return *reinterpret_cast<const uint4*>(at + (q * atoms + (r >> 6)) * kTileBytes + row * kRowBytes +
                                           ((((r & 63) >> 3) ^ (row & 7)) << 4));
  }
  MXG_DEVINL bool has_nan(int R) const {
    bool n = false;
    for (int r = 0; r < R; r += 8) {
      const uint4 w = chunk(0, r);
      const uint32_t* h = &w.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) n |= bf16x2_absmax_bits(h[j]) > 0x7F80u;
    }
    return n;
  }
  // The product with one column of B, term by term of the sum of u itself.
  MXG_DEVINL float dot(const uint16_t* b, int R) const {
    float acc = 0.0f;
    for (int r = 0; r < R; r += 8) {
      const uint4 bw = __ldg(reinterpret_cast<const uint4*>(b + r));
      float u[8] = {};
#pragma unroll
      for (int q = kTerms - 1; q >= 0; --q) {
        const uint4 w = chunk(q, r);
        const uint32_t* h = &w.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) { u[2 * j] += bf16lo_to_f32(h[j]); u[2 * j + 1] += bf16hi_to_f32(h[j]); }
      }
      const uint32_t* h = &bw.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc = fmaf(bf16lo_to_f32(h[j]), u[2 * j], acc);
        acc = fmaf(bf16hi_to_f32(h[j]), u[2 * j + 1], acc);
      }
    }
    return acc;
  }
};

// Whether all 64 values are finite: d * 0 summed in packed pairs.  The check costs
// 1024 tokens of 64 mixed adapters (4096 x 4096, rank 16) 34.5 -> 36 us, 8192 of
// them 81 -> 84, and long prompts nothing (206).
MXG_DEVINL bool all_finite(const float* d) {
  uint64_t s[4] = {};
#pragma unroll
  for (int i = 0; i < 32; ++i) ptx::fma_f32x2(s[i & 3], ptx::f32x2_pack(d[2 * i], d[2 * i + 1]), 0ull);
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) z += __uint_as_float((uint32_t)s[i]) + __uint_as_float((uint32_t)(s[i] >> 32));
  return z == 0.0f;
}
// Bit i: d[i] is infinite or NaN.
MXG_DEVINL uint64_t not_finite(const float* d) {
  uint64_t m = 0;
#pragma unroll
  for (int i = 0; i < 64; ++i) m |= (uint64_t)!(fabsf(d[i]) < INFINITY) << i;
  return m;
}

template <typename TOut>
__global__ void __launch_bounds__(kExpThreads, 1)
    lora_expand_tile_kernel(const __grid_constant__ CUtensorMap tmB, const LoraParams p) {
  constexpr int kTerms = Exp<TOut>::kTerms, kStages = Exp<TOut>::kStages, kPieces = Exp<TOut>::kPieces;
  constexpr int kPieceCols = kRowBytes / (int)sizeof(TOut);  // 64 or 32
  constexpr int kPer = 64 / kPieceCols;                      // pieces of a warp's 64 columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - ptx::smem_u32(smem_raw));
  __shared__ Tile tile;
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const LoraArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };
  const uint32_t drain = bar0 + 8u * (2 * kStages + 4);
  const int atoms = (a.R + 63) >> 6;                       // 64-rank rows of u and B
  const int ubytes = kTerms * atoms * kTileBytes;          // [term][atom][128 rows]
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(acc_full(b), 1);
      ptx::mbar_init(acc_empty(b), 8);
    }
    ptx::mbar_init(drain, 1);
    abort_word = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), kExpTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  ptx::pdl_wait();
  read_tile(tile, p, t0);
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int count = tile.count;
  const bool idle = (int)blockIdx.z >= max(count, 1);  // no adapter for this CTA
  // u: ranks past R up to the product's depth are zero
  const int depth = (a.R + 15) & ~15;
  for (int i = threadIdx.x; !idle && i < kTile * (depth >> 3); i += kExpThreads) {
    const int row = i / (depth >> 3), r0 = (i - row * (depth >> 3)) * 8;
    float v[8] = {};
    if (tile.ord[row] >= 0 && r0 < a.R) {
      const float* src = p.u + (t0 + row) * a.R + r0;
      for (int k0 = 0; k0 < p.ksplit; k0 += 4) {
        float4 w[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k][0] = w[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (k0 + k < p.ksplit) {
            const float4* part = reinterpret_cast<const float4*>(src + (int64_t)(k0 + k) * a.T * a.R);
            w[k][0] = __ldcg(part);
            w[k][1] = __ldcg(part + 1);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[0] += w[k][0].x; v[1] += w[k][0].y; v[2] += w[k][0].z; v[3] += w[k][0].w;
          v[4] += w[k][1].x; v[5] += w[k][1].y; v[6] += w[k][1].z; v[7] += w[k][1].w;
        }
      }
      const float sc = a.scale != nullptr ? __ldg(a.scale + tile.id[row]) : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= sc;
    }
    // 16-byte chunk c of a row sits at c ^ (row % 8)
    const int at = (r0 >> 6) * kTileBytes + row * kRowBytes + ((((r0 & 63) >> 3) ^ (row & 7)) << 4);
#pragma unroll
    for (int q = 0; q < kTerms; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = bf16_term(v[2 * j], v[2 * j + 1]);
        v[2 * j] = left_of(v[2 * j], bf16lo_to_f32(w[j]));
        v[2 * j + 1] = left_of(v[2 * j + 1], bf16hi_to_f32(w[j]));
      }
      *reinterpret_cast<uint4*>(smem + q * atoms * kTileBytes + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  ptx::fence_proxy_async_smem();
  __syncthreads();

  const int64_t c0 = (int64_t)blockIdx.x * p.cols;
  const int ncols = (int)(min(a.N, c0 + p.cols) - c0);
  const int blocks = (ncols + kExpCols - 1) / kExpCols;
  const int o_first = blockIdx.z, o_step = gridDim.z;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      for (int o = o_first; ok && o < count; o += o_step) {
        // rows past the adapter's last column belong to the next one (or lie past the tensor and read as zero)
        const int64_t row0 = (int64_t)tile.list[o] * a.N + c0;
        for (int b = 0; ok && b < blocks; ++b)
          for (int q = 0; q < atoms; ++q) {
            ok = ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, a.status, p.timeout_ns);
            if (!ok) break;
            const uint32_t fb = full_bar(stage);
            ptx::mbar_arrive_expect_tx(fb, kTileBytes);
            armed |= 1u << stage;
            armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
            ptx::tma_load_2d(sbase + ubytes + stage * kTileBytes, &tmB, q * 64, (int)(row0 + b * kExpCols), fb);
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
          }
      }
      for (int s = 0; s < kStages; ++s)
        if ((armed >> s) & 1u) {
          volatile int no_abort = 0;
          ptx::mbar_wait(full_bar(s), (armed_phase >> s) & 1u, &no_abort, a.status, p.drain_ns);
        }
    }
  } else if (warp == 1) {
    const uint32_t el = ptx::elect_one();
    const uint32_t idesc = idesc_bf16(kExpCols);
    int stage = 0, n = 0;
    uint32_t phase = 0;
    bool ok = true, issued = false;
    for (int o = o_first; ok && o < count; o += o_step)
      for (int b = 0; ok && b < blocks; ++b, ++n) {
        ok = ptx::mbar_wait_warp(acc_empty(n & 1), ((n >> 1) & 1u) ^ 1u, abort_flag, a.status, p.timeout_ns);
        if (!ok) break;
        const uint32_t d = tmem + (n & 1) * kExpCols;
        for (int at = 0; at < atoms; ++at) {
          ok = ptx::mbar_wait_warp(full_bar(stage), phase, abort_flag, a.status, p.timeout_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t bd = ptx::smem_desc(sbase + ubytes + stage * kTileBytes, 16, 1024, 2);
          const int steps = min(4, (depth - at * 64) >> 4);
          for (int q = kTerms - 1; q >= 0; --q) {  // the smallest term first
            const uint64_t ud = ptx::smem_desc(sbase + (q * atoms + at) * kTileBytes, 16, 1024, 2);
            for (int j = 0; j < steps; ++j)
              ptx::mma_f16_if(el, d, ud + 2 * j, bd + 2 * j, idesc, at != 0 || q != kTerms - 1 || j != 0);
          }
          issued = true;
          ptx::tc_commit_if(el, empty_bar(stage));
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (ok) ptx::tc_commit_if(el, acc_full(n & 1));
      }
    if (issued) {
      ptx::tc_commit_if(el, drain);
      volatile int no_abort = 0;
      ptx::mbar_wait(drain, 0, &no_abort, a.status, p.drain_ns);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16) + half * 64;
    uint8_t* ring = smem + ubytes + kStages * kTileBytes + (warp - 2) * kPieces * kPieceBytes;
    const uint32_t ring_a = sbase + ubytes + kStages * kTileBytes + (warp - 2) * kPieces * kPieceBytes;
    // moving: lane l has 16 bytes (l % 8) of rows l / 8, l / 8 + 4, ...; adding: row l
    const int mrow = lane >> 3, mcol = (lane & 7) * (16 / (int)sizeof(TOut));
    const TOut* ybase = static_cast<const TOut*>(a.y) + c0 + half * 64 + mcol;
    TOut* obase = static_cast<TOut*>(a.out) + c0 + half * 64 + mcol;
    int64_t tok[8];  // of rows mrow + 4 i
#pragma unroll
    for (int i = 0; i < 8; ++i) tok[i] = tile.tok[quarter * 32 + mrow + 4 * i];
    const bool in_place = a.out == a.y && a.ld_out == a.ld_y;
    const URow<kTerms> u_row{smem, quarter * 32 + lane, atoms};
    uint32_t rows = 0;  // bit i: row mrow + 4 i is moved in this pass
    auto pick = [&](int o) {
      rows = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (tok[i] >= 0 && tile.ord[quarter * 32 + mrow + 4 * i] == o) rows |= 1u << i;
      }
    };
    if (blockIdx.z == 0 && !in_place) {  // rows without an adapter are copied
      pick(-1);
      if (__any_sync(kFull, rows != 0))
        for (int c = 0; c < ncols; c += kExpCols)
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const int col = c + q * kPieceCols;
            if (half * 64 + col + mcol < ncols) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if ((rows >> i) & 1)
                  *reinterpret_cast<uint4*>(obase + tok[i] * a.ld_out + col) =
                      *reinterpret_cast<const uint4*>(ybase + tok[i] * a.ld_y + col);
            }
          }
    }
    int n = 0;  // accumulators taken
    for (int o = o_first; o < count; o += o_step) {
      pick(o);
      const bool wanted = __any_sync(kFull, rows != 0);
      const int pieces = wanted ? blocks * kPer : 0;
      auto fetch = [&](int k) {  // piece k of the pass into its buffer
        if (k < pieces) {
          const int col = (k / kPer) * kExpCols + (k % kPer) * kPieceCols;
          const uint32_t dst = ring_a + (k % kPieces) * kPieceBytes + mrow * kPiecePitch + (lane & 7) * 16;
          if (half * 64 + col + mcol < ncols) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              ptx::cp_async_16_if((rows >> i) & 1, dst + 4 * i * kPiecePitch, ybase + tok[i] * a.ld_y + col);
          }
        }
        ptx::cp_async_commit();
      };
#pragma unroll
      for (int k = 0; k < kPieces - 1; ++k) fetch(k);
      bool ok = true;
      const bool mine_o = tile.ord[quarter * 32 + lane] == o;  // this lane's row is the adapter's
      for (int b = 0; b < blocks; ++b, ++n) {
        ok = ptx::mbar_wait(acc_full(n & 1), (n >> 1) & 1u, abort_flag, a.status, p.timeout_ns);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        float d[64];
        if (wanted) {
          ptx::tmem_ld_32x32b_x32(tq + (n & 1) * kExpCols, reinterpret_cast<uint32_t*>(d));
          ptx::tmem_ld_32x32b_x32(tq + (n & 1) * kExpCols + 32, reinterpret_cast<uint32_t*>(d) + 32);
          ptx::tmem_ld_wait();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(acc_empty(n & 1));
        if (!wanted) continue;
        // `redo`: the lane's columns that are added by themselves, d being 0 there.
        auto add_pieces = [&](uint64_t redo) {
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const int k = b * kPer + q;
            fetch(k + kPieces - 1);
            ptx::cp_async_wait<kPieces - 1>();
            __syncwarp();
            uint8_t* piece = ring + (k % kPieces) * kPieceBytes;
            uint4* mine = reinterpret_cast<uint4*>(piece + lane * kPiecePitch);
            constexpr int kVals = 16 / (int)sizeof(TOut);
#pragma unroll
            for (int j = 0; j < 8; ++j) mine[j] = add16<TOut>(mine[j], d + q * kPieceCols + j * kVals);
            const int col = b * kExpCols + q * kPieceCols;
            for (uint64_t m = kPer == 1 ? redo : (redo >> (q * 32)) & 0xFFFFFFFFu; m != 0; m &= m - 1) {
              const int i = __ffsll((long long)m) - 1;
              if (half * 64 + col + i >= ncols) break;       // past the adapter's columns: not stored
              TOut* e = reinterpret_cast<TOut*>(mine) + i;  // y as it was
              *e = (TOut)((float)*e + u_row.dot(a.B + ((int64_t)tile.list[o] * a.N + c0 + half * 64 + col + i) * a.R, a.R));
            }
            __syncwarp();
            if (half * 64 + col + mcol < ncols) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                ptx::st_v4_if((rows >> i) & 1, obase + tok[i] * a.ld_out + col,
                              *reinterpret_cast<const uint4*>(piece + (mrow + 4 * i) * kPiecePitch + (lane & 7) * 16));
            }
            __syncwarp();
          }
        };
        if (!__any_sync(kFull, mine_o && !all_finite(d))) {
          add_pieces(0);
        } else {
          // A product that is not finite is done again without the split, whose
          // lower terms may be zero or of the other sign against an infinity of B
          // (with NaN in u it is what it has to be).
          const uint64_t redo = mine_o && !u_row.has_nan(a.R) ? not_finite(d) : 0;
#pragma unroll
          for (int i = 0; i < 64; ++i) d[i] = (redo >> i) & 1 ? 0.0f : d[i];
          add_pieces(redo);
        }
      }
      ptx::cp_async_wait<0>();
      if (!ok) break;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kExpTmem);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// The per-token kernels read T R (K + N) BF16 values of adapters, from L2 where
// tokens share them, at 6 to 8 TB/s; the tiles take 16 to 50 us before the size
// shows.  Per token against tiles, in us:
//   4096 x 4096, rank 16, 64 adapters: 256 tokens (67 MB) 11 / 31, 512 (134 MB)
//   19 / 32, 1024 (268 MB) 36 / 32; with 8 adapters 11 / 16, 18 / 16, 33 / 17
//   4096 x 4096, rank 64, 16 adapters: 64 tokens (67 MB) 21 / 20, 128 (134 MB)
//   26 / 21, 256 (268 MB) 49 / 22
//   2048 x 8192, rank 32, 32 adapters: 256 tokens (168 MB) 26 / 29, 512 47 / 31
// The rule knows bytes alone: where few adapters or high ranks bring the tiles
// ahead below it, it leaves 1 to 5 us.
constexpr double kTokenBytes = 150e6;
constexpr int kLoraSms = 152;

// Tiles: 64-element steps of K per shrink CTA.  Among the splits that leave
// eight steps a CTA (and at most sixteen splits), the one that ends soonest in
// whole waves of CTAs, with a CTA's start counted as eight steps.
int shrink_steps(int64_t T, int64_t K) {
  const int64_t tiles = (T + kTile - 1) / kTile, steps = (K + 63) / 64;
  int64_t best = steps, best_cost = INT64_MAX;
  for (int64_t split = 1; split <= 16 && (split == 1 || steps / split >= 8); ++split) {
    const int64_t per = (steps + split - 1) / split;
    const int64_t ctas = tiles * ((steps + per - 1) / per);
    const int64_t cost = (ctas + kLoraSms - 1) / kLoraSms * (per + 8);
    if (cost < best_cost) {
      best_cost = cost;
      best = per;
    }
  }
  return (int)best;
}

int64_t tile_splits(int64_t T, int64_t K) {
  const int64_t per = shrink_steps(T, K);
  return ((K + 63) / 64 + per - 1) / per;
}

constexpr int kLoraMaxDevices = 64;
std::mutex g_lora_mu;

// The dynamic shared-memory opt-in of the tile kernels, once per device.
cudaError_t ensure_lora_attr() {
  static bool done[kLoraMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_lora_mu);
  if (dev < kLoraMaxDevices && done[dev]) return cudaSuccess;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute((const void*)lora_shrink_tile_kernel, attr, kShrinkSmem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute((const void*)lora_expand_tile_kernel<float>, attr, Exp<float>::smem(128))) != cudaSuccess ||
      (e = cudaFuncSetAttribute((const void*)lora_expand_tile_kernel<__nv_bfloat16>, attr,
                                Exp<__nv_bfloat16>::smem(128))) != cudaSuccess)
    return e;
  if (dev < kLoraMaxDevices) done[dev] = true;
  return cudaSuccess;
}

cudaError_t launch(const void* fn, dim3 grid, int threads, size_t smem, void** args, bool overlap, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

bool lora_per_token(int64_t T, int64_t N, int64_t K, int R) {
  return (double)T * R * (double)(K + N) * 2.0 <= kTokenBytes && T <= 65535;
}

// About what a tile of sorted tokens meets, with room for one more where it
// meets several (a CTA that gets a second adapter takes twice as long: 512
// tokens of 64 adapters, 4096 x 4096, rank 16: 40 us without the room, 36 with).
// Tokens are sorted within a segment, whose tiles share its adapters out.
int64_t lora_tile_adapters(int64_t T, int64_t n) {
  const int64_t tiles = std::min<int64_t>((T + kTile - 1) / kTile, kSegment / kTile);
  return n < tiles ? 1 : std::min<int64_t>({kTile, n, 2 + n / tiles});
}

// For every N: the per-token form's partial sums only where some N takes it.
size_t lora_workspace_bytes(int64_t T, int64_t K, int R) {
  T = std::max<int64_t>(T, 1);
  const int64_t split = std::max<int64_t>(tile_splits(T, K), lora_per_token(T, 8, K, R) ? (K + kTokK - 1) / kTokK : 0);
  return (size_t)(split * T * R) * sizeof(float) + (size_t)T * sizeof(int32_t);  // u, order
}

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t stream, int num_sms) {
  LoraParams p{};
  p.a = a;
  p.u = a.ws;
  const bool f32 = a.dtype == MXG_OUT_F32;
  cudaError_t e;
  if (lora_per_token(a.T, a.N, a.K, a.R)) {
    p.ksplit = (int)((a.K + kTokK - 1) / kTokK);
    void* args[] = {(void*)&p};
    e = launch((const void*)lora_shrink_token_kernel,
               dim3((unsigned)p.ksplit, (unsigned)a.T, (unsigned)((a.R + kTokR - 1) / kTokR)), kLoraThreads, 0, args,
               false, stream);
    if (e != cudaSuccess) return e;
    return launch(f32 ? (const void*)lora_expand_token_kernel<float> : (const void*)lora_expand_token_kernel<__nv_bfloat16>,
                  dim3((unsigned)((a.N + kLoraThreads * kTokCols - 1) / (kLoraThreads * kTokCols)), (unsigned)a.T),
                  kLoraThreads, 0, args, true, stream);
  }
  const int64_t tiles = (a.T + kTile - 1) / kTile;
  if ((e = ensure_lora_attr()) != cudaSuccess) return e;
  p.blocks = shrink_steps(a.T, a.K);
  p.ksplit = (int)tile_splits(a.T, a.K);
  const int64_t met = lora_tile_adapters(a.T, a.n);
  const int64_t passes = (met * a.R + kShrinkRows - 1) / kShrinkRows;
  const int64_t pass_groups = std::max<int64_t>(1, std::min(passes, num_sms / (tiles * p.ksplit)));
  p.order = reinterpret_cast<int32_t*>(a.ws + (int64_t)p.ksplit * a.T * a.R);
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = std::max<uint64_t>(p.timeout_ns, 200000000ull);
  // The split of columns, and of a tile's adapters, that ends soonest in whole
  // waves of CTAs, with a CTA's start (its u) counted as four blocks.
  const int64_t blocks = (a.N + kExpCols - 1) / kExpCols;
  int64_t best = blocks, groups = 1, best_cost = INT64_MAX;
  for (int64_t g = 1; g <= met; g = g < met ? std::min(2 * g, met) : g + 1)
    for (int64_t per = blocks; per >= 1;
         per = std::min(per - 1, (blocks + (blocks + per - 1) / per) / ((blocks + per - 1) / per + 1))) {
      const int64_t ctas = tiles * ((blocks + per - 1) / per) * g;
      const int64_t cost = (ctas + num_sms - 1) / num_sms * (per * ((met + g - 1) / g) + 4);
      if (cost < best_cost) {
        best_cost = cost;
        best = per;
        groups = g;
      }
    }
  p.cols = (int)best * kExpCols;
  CUtensorMap tmA, tmB;
  const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!make_tmap(&tmA, a.A, dt, a.K, (int64_t)a.n * a.R, a.K * 2, 64, a.R) ||
      !make_tmap(&tmB, a.B, dt, a.R, (int64_t)a.n * a.N, (int64_t)a.R * 2, 64, kExpCols))
    return cudaErrorInvalidValue;
  void* oargs[] = {(void*)&p};
  e = launch((const void*)lora_order_kernel, dim3((unsigned)((a.T + kSegment - 1) / kSegment)), kOrderThreads, 0, oargs,
             false, stream);
  if (e != cudaSuccess) return e;
  void* sargs[] = {(void*)&tmA, (void*)&p};
  e = launch((const void*)lora_shrink_tile_kernel, dim3((unsigned)p.ksplit, (unsigned)tiles, (unsigned)pass_groups),
             kShrinkThreads, kShrinkSmem, sargs, true, stream);
  if (e != cudaSuccess) return e;
  void* eargs[] = {(void*)&tmB, (void*)&p};
  return launch(f32 ? (const void*)lora_expand_tile_kernel<float> : (const void*)lora_expand_tile_kernel<__nv_bfloat16>,
                dim3((unsigned)((a.N + p.cols - 1) / p.cols), (unsigned)tiles, (unsigned)groups), kExpThreads,
                (size_t)(f32 ? Exp<float>::smem(a.R) : Exp<__nv_bfloat16>::smem(a.R)), eargs, true, stream);
}

}  // namespace mxg
