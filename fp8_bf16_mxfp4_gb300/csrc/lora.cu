// Low-rank adapters of many requests beside a shared projection:
//   out[t] = y[t] + scale[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// Two kernels: shrink, u[t] = A[a] x[t], split over K, fp32 partials to the
// workspace; expand, which sums the partials in order and adds scale * B u to y.
// Both are bound by memory: x, y, and R (K + N) values of each adapter used.
//
// Few tokens: a CTA works for one token, reads the token's adapter rows 16 bytes
// a lane and multiplies in fp32.  Tokens that share an adapter read it again,
// from L2; that is as fast as it gets while all adapters read for all tokens
// are a few tens of MB, because every load of a CTA is in flight at once.
//
// Many tokens: a CTA takes a tile of 32 tokens as they come in the batch, and
// for every adapter that occurs in the tile runs the tile's tokens against the
// adapter's rows on the tensor core (mma.sync, BF16 x BF16 + FP32), which has
// work for a few clocks per line loaded: products of rows that are not wanted
// cost nothing, and there is no sorting.  A token's row belongs to one adapter,
// so the adapters of a tile are shared out over CTAs without any sum across
// them, and a row is selected, never masked by a product: an adapter's
// infinities or NaN reach its own tokens only.  Fragments are loaded straight
// from global memory, 16 bytes a lane: the contraction may be taken in any
// order, so lane t of a row's four takes elements 8t .. 8t+7 of a 32-element
// block for both operands.  In the expand the output columns are permuted the
// same way, so that a lane has 8 neighbouring columns of a row.  u keeps its
// fp32 accuracy as a sum of two BF16 terms (2^-17; BF16 output) or three
// (2^-25; FP32 output).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace mxg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kLoraWarps = 4;
constexpr int kLoraThreads = kLoraWarps * 32;
constexpr int kGroups = 2;                // 16-token groups of a tile
constexpr int kTile = 16 * kGroups;

struct LoraParams {
  LoraArgs a;
  float* u;         // [ksplit][T][R] partial sums
  int ksplit;
  int blocks;       // tiles: 32-element blocks of K per CTA of the shrink
  int cols;         // tiles: columns per CTA of the expand
};

MXG_DEVINL void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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
// The adapters of a tile of tokens, in order of first use.
struct Tile {
  int id[kTile];           // adapter of each token (-1: none)
  int ord[kTile];          // its number in the list (-1: none)
  int list[kTile];         // adapter by number
  uint32_t groups[kTile];  // 16-token groups in which it occurs (bit mask)
  int count;
};

MXG_DEVINL void read_tile(Tile& s, const LoraArgs& a, int64_t t0) {
  static_assert(kTile == 32, "a lane per token");
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int id = t0 + lane < a.T ? __ldg(a.ids + t0 + lane) : -1;
    if (id >= a.n) {
      report(a.status, MXG_ERR_INDEX);
      id = -1;
    }
    const uint32_t same = __match_any_sync(kFull, id);
    const int leader = __ffs(same) - 1;
    const uint32_t firsts = __ballot_sync(kFull, id >= 0 && leader == lane);
    const int o = id >= 0 ? __popc(firsts & ((1u << leader) - 1u)) : -1;
    s.id[lane] = id;
    s.ord[lane] = o;
    if (id >= 0 && leader == lane) {
      s.list[o] = id;
      s.groups[o] = ((same & 0xFFFFu) ? 1u : 0u) | ((same >> 16) ? 2u : 0u);
    }
    if (lane == 0) s.count = __popc(firsts);
  }
  __syncthreads();
}

// shrink: grid (K split, tiles, adapter groups).  The warps of a CTA take every
// fourth 32-element block of its K range, up to 32 ranks at a time.
__global__ void __launch_bounds__(kLoraThreads, 4) lora_shrink_tile_kernel(const LoraParams p) {
  constexpr int kUnroll = 2;  // blocks in flight
  __shared__ Tile tile;
  __shared__ float red[kLoraWarps][kTile][33];
  ptx::pdl_launch_dependents();
  const LoraArgs& a = p.a;
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  read_tile(tile, a, t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int64_t kblocks = (a.K + 31) >> 5;
  const int64_t b0 = (int64_t)blockIdx.x * p.blocks;
  const int nb = (int)min((int64_t)p.blocks, kblocks - b0);
  const uint16_t* xk = a.x + t0 * a.ld_x + b0 * 32 + 8 * tq;
  const int kleft = (int)min(a.K - b0 * 32, (int64_t)nb * 32) - 8 * tq;  // of this lane's first block on
  for (int o = blockIdx.z; o < tile.count; o += gridDim.z) {
    const uint32_t groups = tile.groups[o];
    for (int r0 = 0; r0 < a.R; r0 += 32) {
      const int nt = min(4, (a.R - r0) >> 3);
      const uint16_t* ak = a.A + ((int64_t)tile.list[o] * a.R + r0 + g) * a.K + b0 * 32 + 8 * tq;
      float acc[kGroups][4][4];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      for (int b = warp; b < nb; b += kLoraWarps * kUnroll) {
        uint4 xv[kUnroll][kGroups][2], av[kUnroll][4];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
          const int k = (b + q * kLoraWarps) * 32;
          const bool in = k < kleft;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            av[q][n] = make_uint4(0, 0, 0, 0);
            if (in && n < nt) av[q][n] = __ldg(reinterpret_cast<const uint4*>(ak + (int64_t)n * 8 * a.K + k));
          }
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = m * 16 + g + 8 * h;
              xv[q][m][h] = make_uint4(0, 0, 0, 0);
              if (in && ((groups >> m) & 1) && t0 + row < a.T)
                xv[q][m][h] = __ldg(reinterpret_cast<const uint4*>(xk + row * a.ld_x + k));
            }
        }
#pragma unroll
        for (int q = 0; q < kUnroll; ++q)
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
            if ((groups >> m) & 1) {
              const uint4 lo = xv[q][m][0], hi = xv[q][m][1];
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (n < nt) {
                  mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, av[q][n].x, av[q][n].y);
                  mma_bf16(acc[m][n], lo.z, hi.z, lo.w, hi.w, av[q][n].z, av[q][n].w);
                }
            }
      }
      // the four warps' sums, in order
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float* d = &red[warp][m * 16 + g][n * 8 + 2 * tq];
          d[0] = acc[m][n][0];
          d[1] = acc[m][n][1];
          d[8 * 33] = acc[m][n][2];
          d[8 * 33 + 1] = acc[m][n][3];
        }
      __syncthreads();
      for (int i = threadIdx.x; i < kTile * 32; i += kLoraThreads) {
        const int row = i >> 5, r = i & 31;
        if (tile.ord[row] == o && r < nt * 8) {
          const float s = (red[0][row][r] + red[1][row][r]) + (red[2][row][r] + red[3][row][r]);
          __stcg(p.u + ((int64_t)blockIdx.x * a.T + t0 + row) * a.R + r0 + r, s);
        }
      }
      __syncthreads();
    }
  }
}

// expand: grid (column chunks, tiles, adapter groups).  A warp takes 32 columns
// at a time; the next columns' y is on its way meanwhile.
template <typename TOut>
struct Row8;  // 8 neighbouring columns of a row
template <>
struct Row8<__nv_bfloat16> {
  uint4 v;
  MXG_DEVINL void load(const void* p, int64_t i) {
    v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
  }
  MXG_DEVINL void store(void* p, int64_t i) const {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i), v);
  }
  MXG_DEVINL void add(const float* d) {
    uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 r =
          __floats2bfloat162_rn(bf16lo_to_f32(w[i]) + d[2 * i], bf16hi_to_f32(w[i]) + d[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};
template <>
struct Row8<float> {
  float4 v[2];
  MXG_DEVINL void load(const void* p, int64_t i) {
    v[0] = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    v[1] = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i) + 1);
  }
  MXG_DEVINL void store(void* p, int64_t i) const {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + i), v[0]);
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + i) + 1, v[1]);
  }
  MXG_DEVINL void add(const float* d) {
    float* w = &v[0].x;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] += d[i];
  }
};

template <typename TOut>
__global__ void __launch_bounds__(kLoraThreads, 4) lora_expand_tile_kernel(const LoraParams p) {
  constexpr int kTerms = sizeof(TOut) == 2 ? 2 : 3;
  __shared__ Tile tile;
  extern __shared__ __align__(16) uint16_t us[];  // [kTerms][kTile][R + 8]: scale * u as a sum of BF16 terms
  const LoraArgs& a = p.a;
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  read_tile(tile, a, t0);
  if (blockIdx.z > 0 && (int)blockIdx.z >= tile.count) return;
  const int pitch = a.R + 8;
  ptx::pdl_wait();
  for (int i = threadIdx.x; i < kTile * a.R; i += kLoraThreads) {
    const int row = i / a.R, r = i - row * a.R;
    const int o = tile.ord[row];
    if (o < 0 || o % (int)gridDim.z != (int)blockIdx.z) continue;
    float s = sum_u(p, t0 + row, r);
    if (a.scale != nullptr) s *= __ldg(a.scale + tile.id[row]);
#pragma unroll
    for (int q = 0; q < kTerms; ++q) {
      const __nv_bfloat16 h = __float2bfloat16_rn(s);
      us[(q * kTile + row) * pitch + r] = *reinterpret_cast<const uint16_t*>(&h);
      s -= __bfloat162float(h);
    }
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int64_t first = (int64_t)blockIdx.x * p.cols + warp * 32;
  const int64_t c1 = min(a.N, (int64_t)(blockIdx.x + 1) * p.cols);
  for (int o = blockIdx.z; o < max(tile.count, 1); o += gridDim.z) {
    const bool any = o < tile.count;
    const uint32_t groups = any ? tile.groups[o] : 0u;
    // this lane's rows: those of adapter o, and the ones without adapter in the first pass
    bool mine[kGroups][2], sum[kGroups][2];
#pragma unroll
    for (int m = 0; m < kGroups; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = m * 16 + g + 8 * h;
        const int ro = tile.ord[row];
        sum[m][h] = any && ro == o;
        mine[m][h] = t0 + row < a.T && (sum[m][h] || (ro < 0 && o == 0));
      }
    Row8<TOut> y[kGroups][2];
    auto load = [&](int64_t c) {
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (mine[m][h] && c + 8 * tq < c1) y[m][h].load(a.y, (t0 + m * 16 + g + 8 * h) * a.ld_y + c + 8 * tq);
    };
    load(first);
    for (int64_t c0 = first; c0 < c1; c0 += kLoraWarps * 32) {
      float acc[kGroups][4][4];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      if (any) {
        // column g of product n is output column 8 (g / 2) + 2 n + g % 2
        const int64_t col = c0 + 8 * (g >> 1) + (g & 1);
        const uint16_t* bk = a.B + ((int64_t)tile.list[o] * a.N + col) * a.R;
        const bool bin = c0 + 8 * (g >> 1) < c1;
        int r0 = 0;
        for (; r0 + 32 <= a.R; r0 += 32) {
          uint4 bv[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            bv[n] = make_uint4(0, 0, 0, 0);
            if (bin) bv[n] = __ldg(reinterpret_cast<const uint4*>(bk + (int64_t)2 * n * a.R + r0 + 8 * tq));
          }
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
            if ((groups >> m) & 1) {
#pragma unroll
              for (int q = kTerms - 1; q >= 0; --q) {
                const uint16_t* u = us + (q * kTile + m * 16 + g) * pitch + r0 + 8 * tq;
                const uint4 lo = *reinterpret_cast<const uint4*>(u), hi = *reinterpret_cast<const uint4*>(u + 8 * pitch);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, bv[n].x, bv[n].y);
                  mma_bf16(acc[m][n], lo.z, hi.z, lo.w, hi.w, bv[n].z, bv[n].w);
                }
              }
            }
        }
        if (a.R & 16) {  // 16 ranks: 8 bytes a lane
          uint2 bv[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            bv[n] = make_uint2(0, 0);
            if (bin) bv[n] = __ldg(reinterpret_cast<const uint2*>(bk + (int64_t)2 * n * a.R + r0 + 4 * tq));
          }
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
            if ((groups >> m) & 1) {
#pragma unroll
              for (int q = kTerms - 1; q >= 0; --q) {
                const uint16_t* u = us + (q * kTile + m * 16 + g) * pitch + r0 + 4 * tq;
                const uint2 lo = *reinterpret_cast<const uint2*>(u), hi = *reinterpret_cast<const uint2*>(u + 8 * pitch);
#pragma unroll
                for (int n = 0; n < 4; ++n) mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, bv[n].x, bv[n].y);
              }
            }
          r0 += 16;
        }
        if (a.R & 8) {  // 8 ranks: 4 bytes a lane, half of the product's depth
          uint32_t bv[4];
#pragma unroll
          for (int n = 0; n < 4; ++n)
            bv[n] = bin ? __ldg(reinterpret_cast<const uint32_t*>(bk + (int64_t)2 * n * a.R + r0 + 2 * tq)) : 0u;
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
            if ((groups >> m) & 1) {
#pragma unroll
              for (int q = kTerms - 1; q >= 0; --q) {
                const uint16_t* u = us + (q * kTile + m * 16 + g) * pitch + r0 + 2 * tq;
                const uint32_t lo = *reinterpret_cast<const uint32_t*>(u);
                const uint32_t hi = *reinterpret_cast<const uint32_t*>(u + 8 * pitch);
#pragma unroll
                for (int n = 0; n < 4; ++n) mma_bf16(acc[m][n], lo, hi, 0u, 0u, bv[n], 0u);
              }
            }
        }
      }
      Row8<TOut> now[kGroups][2];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) now[m][h] = y[m][h];
      load(c0 + kLoraWarps * 32);
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (mine[m][h] && c0 + 8 * tq < c1) {  // N is a multiple of 8
            if (sum[m][h]) {
              float d[8];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                d[2 * n] = acc[m][n][2 * h];
                d[2 * n + 1] = acc[m][n][2 * h + 1];
              }
              now[m][h].add(d);
            }
            now[m][h].store(a.out, (t0 + m * 16 + g + 8 * h) * a.ld_out + c0 + 8 * tq);
          }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Adapter bytes that the per-token kernels would read, from L2 where tokens
// share them, against this limit.
constexpr double kTokenBytes = 64e6;

bool per_token(int64_t T, int64_t N, int64_t K, int R) {
  return (double)T * R * (double)(K + N) * 2.0 <= kTokenBytes && T <= 65535;
}

// Tiles: 32-element blocks of K per shrink CTA, a multiple of the warps, so
// that there are about eight CTAs per SM if K allows.
int shrink_blocks(int64_t T, int64_t K) {
  const int64_t tiles = (T + kTile - 1) / kTile;
  const int64_t kblocks = (K + 31) / 32;
  const int64_t split = std::max<int64_t>(1, (8 * 152 + tiles - 1) / tiles);
  const int64_t per = std::max<int64_t>((kblocks + split - 1) / split, 2 * kLoraWarps);
  return (int)std::min<int64_t>((per + kLoraWarps - 1) / kLoraWarps * kLoraWarps, 1 << 20);
}

int64_t tile_splits(int64_t T, int64_t K) {
  const int64_t per = shrink_blocks(T, K);
  return ((K + 31) / 32 + per - 1) / per;
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int R) {
  T = std::max<int64_t>(T, 1);
  const int64_t split = std::max<int64_t>(tile_splits(T, K), T <= 65535 ? (K + kTokK - 1) / kTokK : 0);
  return (size_t)(split * T * R) * sizeof(float);
}

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t stream, int num_sms) {
  LoraParams p{};
  p.a = a;
  p.u = a.ws;
  const bool f32 = a.dtype == MXG_OUT_F32;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kLoraThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  const void *shrink, *expand;
  dim3 sgrid, egrid;
  size_t smem = 0;
  if (per_token(a.T, a.N, a.K, a.R)) {
    p.ksplit = (int)((a.K + kTokK - 1) / kTokK);
    shrink = (const void*)lora_shrink_token_kernel;
    expand = f32 ? (const void*)lora_expand_token_kernel<float> : (const void*)lora_expand_token_kernel<__nv_bfloat16>;
    sgrid = dim3((unsigned)p.ksplit, (unsigned)a.T, (unsigned)((a.R + kTokR - 1) / kTokR));
    egrid = dim3((unsigned)((a.N + kLoraThreads * kTokCols - 1) / (kLoraThreads * kTokCols)), (unsigned)a.T);
  } else {
    const int64_t tiles = (a.T + kTile - 1) / kTile;
    if (tiles > 65535) return cudaErrorInvalidConfiguration;
    // adapters of a tile over CTAs: more where there are few tiles
    const int groups = std::min<int>(a.n, tiles < 64 ? 8 : 2);
    p.blocks = shrink_blocks(a.T, a.K);
    p.ksplit = (int)tile_splits(a.T, a.K);
    // columns per CTA: as many as leave about sixteen CTAs per SM, in steps of 128
    const int64_t chunks = std::max<int64_t>(1, 16 * (int64_t)num_sms / tiles);
    p.cols = (int)std::min<int64_t>(8192, std::max<int64_t>(128, (a.N / chunks + 127) / 128 * 128));
    shrink = (const void*)lora_shrink_tile_kernel;
    expand = f32 ? (const void*)lora_expand_tile_kernel<float> : (const void*)lora_expand_tile_kernel<__nv_bfloat16>;
    sgrid = dim3((unsigned)p.ksplit, (unsigned)tiles, (unsigned)groups);
    egrid = dim3((unsigned)((a.N + p.cols - 1) / p.cols), (unsigned)tiles, (unsigned)groups);
    smem = (size_t)(f32 ? 3 : 2) * kTile * (a.R + 8) * 2;
  }
  void* args[] = {(void*)&p};
  cfg.gridDim = sgrid;
  cudaError_t e = cudaLaunchKernelExC(&cfg, shrink, args);
  if (e != cudaSuccess) return e;
  cfg.gridDim = egrid;
  cfg.dynamicSmemBytes = smem;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, expand, args);
}

}  // namespace mxg
