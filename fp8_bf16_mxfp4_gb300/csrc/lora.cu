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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
  // rows past the batch are read from its last token (their products are not used)
  const uint16_t* xr[kGroups][2];
#pragma unroll
  for (int m = 0; m < kGroups; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xr[m][h] = a.x + min(t0 + m * 16 + g + 8 * h, a.T - 1) * a.ld_x + b0 * 32 + 8 * tq;
  const int whole = (int)min((int64_t)nb, (a.K >> 5) - b0);  // blocks that do not end past K
  for (int o = blockIdx.z; o < tile.count; o += gridDim.z) {
    const uint32_t groups = tile.groups[o];
    for (int r0 = 0; r0 < a.R; r0 += 32) {
      const int nt = min(4, (a.R - r0) >> 3);
      // products past the ranks are skipped; their loads repeat the first eight rows
      const uint16_t* ar[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        ar[n] = a.A + ((int64_t)tile.list[o] * a.R + r0 + (n < nt ? 8 * n : 0) + g) * a.K + b0 * 32 + 8 * tq;
      float acc[kGroups][4][4];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      // two blocks' loads are in flight while a third is multiplied
      uint4 xv[2][kGroups][2], av[2][4];
      auto load = [&](int b, int q) {
#pragma unroll
        for (int n = 0; n < 4; ++n) av[q][n] = __ldg(reinterpret_cast<const uint4*>(ar[n] + b * 32));
#pragma unroll
        for (int m = 0; m < kGroups; ++m)
          if ((groups >> m) & 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) xv[q][m][h] = __ldg(reinterpret_cast<const uint4*>(xr[m][h] + b * 32));
          }
      };
      auto multiply = [&](int q) {  // eight independent products between dependent ones
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
            if ((groups >> m) & 1) {
              const uint4 lo = xv[q][m][0], hi = xv[q][m][1];
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (n < nt) {
                  if (h == 0) mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, av[q][n].x, av[q][n].y);
                  else mma_bf16(acc[m][n], lo.z, hi.z, lo.w, hi.w, av[q][n].z, av[q][n].w);
                }
            }
      };
      if (warp < whole) load(warp, 0);
      if (warp + kLoraWarps < whole) load(warp + kLoraWarps, 1);
      for (int b = warp; b < whole; b += 2 * kLoraWarps) {
        multiply(0);
        if (b + 2 * kLoraWarps < whole) load(b + 2 * kLoraWarps, 0);
        if (b + kLoraWarps < whole) multiply(1);
        if (b + 3 * kLoraWarps < whole) load(b + 3 * kLoraWarps, 1);
      }
      if (whole < nb && warp == 0) {  // the block that ends past K: lanes without elements give zeros
        const bool in = (b0 + whole) * 32 + 8 * tq < a.K;
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < 4; ++n) av[0][n] = in ? __ldg(reinterpret_cast<const uint4*>(ar[n] + whole * 32)) : zero;
#pragma unroll
        for (int m = 0; m < kGroups; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            xv[0][m][h] = in ? __ldg(reinterpret_cast<const uint4*>(xr[m][h] + whole * 32)) : zero;
        multiply(0);
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
// at a time; the next columns' y and B are on their way meanwhile.
template <typename TOut>
struct Row8;  // 8 neighbouring columns of a row
template <>
struct Row8<__nv_bfloat16> {
  uint4 v;
  MXG_DEVINL void load(const void* p) { v = *static_cast<const uint4*>(p); }
  MXG_DEVINL void store(void* p) const { *static_cast<uint4*>(p) = v; }
  // values j, j + 1 of the row
  MXG_DEVINL void get(int j, float& lo, float& hi) const {
    lo = bf16lo_to_f32((&v.x)[j >> 1]);
    hi = bf16hi_to_f32((&v.x)[j >> 1]);
  }
  MXG_DEVINL void set(int j, float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    (&v.x)[j >> 1] = *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Row8<float> {
  float4 v[2];
  MXG_DEVINL void load(const void* p) {
    v[0] = *static_cast<const float4*>(p);
    v[1] = *(static_cast<const float4*>(p) + 1);
  }
  MXG_DEVINL void store(void* p) const {
    *static_cast<float4*>(p) = v[0];
    *(static_cast<float4*>(p) + 1) = v[1];
  }
  MXG_DEVINL void get(int j, float& lo, float& hi) const {
    lo = (&v[0].x)[j];
    hi = (&v[0].x)[j + 1];
  }
  MXG_DEVINL void set(int j, float lo, float hi) {
    (&v[0].x)[j] = lo;
    (&v[0].x)[j + 1] = hi;
  }
};

// One product's fragments of B for a chunk of kChunk ranks: 32 ranks are 16
// bytes of a row a lane, 16 ranks 8 bytes, 8 ranks 4 bytes (half of the depth).
template <int kChunk>
struct Frag {
  uint32_t v[kChunk / 8];
  MXG_DEVINL void load(const uint16_t* row, int tq) {
    const uint16_t* src = row + kChunk / 4 * tq;
    if constexpr (kChunk == 32) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(src));
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else if constexpr (kChunk == 16) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
      v[0] = w.x; v[1] = w.y;
    } else {
      v[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
    }
  }
};

// acc += u * B over a chunk; u: this lane's row g (and g + 8, `pitch` 8 rows on)
// of the 16-token group, in shared memory.
template <int kChunk>
MXG_DEVINL void chunk_products(float (*acc)[4], const uint16_t* u, int pitch, const Frag<kChunk>* b, int tq) {
  const uint16_t* lo = u + kChunk / 4 * tq;
  const uint16_t* hi = lo + 8 * pitch;
  if constexpr (kChunk == 32) {
    const uint4 l = *reinterpret_cast<const uint4*>(lo), h = *reinterpret_cast<const uint4*>(hi);
#pragma unroll
    for (int n = 0; n < 4; ++n) mma_bf16(acc[n], l.x, h.x, l.y, h.y, b[n].v[0], b[n].v[1]);
#pragma unroll
    for (int n = 0; n < 4; ++n) mma_bf16(acc[n], l.z, h.z, l.w, h.w, b[n].v[2], b[n].v[3]);
  } else if constexpr (kChunk == 16) {
    const uint2 l = *reinterpret_cast<const uint2*>(lo), h = *reinterpret_cast<const uint2*>(hi);
#pragma unroll
    for (int n = 0; n < 4; ++n) mma_bf16(acc[n], l.x, h.x, l.y, h.y, b[n].v[0], b[n].v[1]);
  } else {
    const uint32_t l = *reinterpret_cast<const uint32_t*>(lo), h = *reinterpret_cast<const uint32_t*>(hi);
#pragma unroll
    for (int n = 0; n < 4; ++n) mma_bf16(acc[n], l, h, 0u, 0u, b[n].v[0], 0u);
  }
}

// kChunk: the ranks are taken 32, 16 or 8 at a time (the largest that divides
// R).  The loop over columns has no branches: fragments past the last column
// repeat others, and 16-token groups without the adapter are multiplied too.
template <typename TOut, int kChunk>
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
  const int64_t c_first = (int64_t)blockIdx.x * p.cols + warp * 32;
  // columns of this warp from its first on (N < 2^31)
  const int left = (int)(min(a.N, (int64_t)(blockIdx.x + 1) * p.cols) - c_first);
  const TOut* y0 = static_cast<const TOut*>(a.y) + (t0 + g) * a.ld_y + c_first + 8 * tq;
  TOut* out0 = static_cast<TOut*>(a.out) + (t0 + g) * a.ld_out + c_first + 8 * tq;
  const int64_t ystep = 8 * a.ld_y, ostep = 8 * a.ld_out;
  // column g of product n is output column 8 (g / 2) + 2 n + g % 2
  const int bcol = 8 * (g >> 1) + (g & 1);

  if (blockIdx.z == 0 && (a.out != a.y || a.ld_out != a.ld_y)) {  // rows without an adapter
    bool none[kGroups][2], any = false;
#pragma unroll
    for (int i = 0; i < 2 * kGroups; ++i) {
      none[i >> 1][i & 1] = t0 + 8 * i + g < a.T && tile.ord[8 * i + g] < 0;
      any |= none[i >> 1][i & 1];
    }
    if (__any_sync(kFull, any))
      for (int c = 0; c + 8 * tq < left; c += kLoraWarps * 32)
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i)
          if (none[i >> 1][i & 1]) {
            Row8<TOut> v;
            v.load(y0 + i * ystep + c);
            v.store(out0 + i * ostep + c);
          }
  }

  for (int o = blockIdx.z; o < tile.count; o += gridDim.z) {
    const uint16_t* B = a.B + ((int64_t)tile.list[o] * a.N + c_first) * a.R;
    bool mine[2 * kGroups];  // row 8 i + g belongs to the adapter
#pragma unroll
    for (int i = 0; i < 2 * kGroups; ++i) mine[i] = t0 + 8 * i + g < a.T && tile.ord[8 * i + g] == o;
    Row8<TOut> y[2 * kGroups];
    Frag<kChunk> b[4];
    auto load_y = [&](int c) {
#pragma unroll
      for (int i = 0; i < 2 * kGroups; ++i)
        if (mine[i] && c + 8 * tq < left) y[i].load(y0 + i * ystep + c);
    };
    auto load_b = [&](int c, int r) {
      const uint16_t* row = B + (int64_t)(c + bcol < left ? c + bcol : 0) * a.R + r;
      const int step = c + bcol < left ? 2 * a.R : 0;
#pragma unroll
      for (int n = 0; n < 4; ++n) b[n].load(row + n * step, tq);
    };
    if (left <= 0) continue;
    load_y(0);
    load_b(0, 0);
    for (int c = 0; c < left; c += kLoraWarps * 32) {
      // the products add to y (a lane's columns 2 n, 2 n + 1 of product n)
      float acc[kGroups][4][4];
#pragma unroll
      for (int i = 0; i < 2 * kGroups; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) y[i].get(2 * n, acc[i >> 1][n][2 * (i & 1)], acc[i >> 1][n][2 * (i & 1) + 1]);
      load_y(c + kLoraWarps * 32);
      for (int r = 0; r < a.R; r += kChunk) {
        if (r > 0) load_b(c, r);
#pragma unroll
        for (int q = kTerms - 1; q >= 0; --q)
#pragma unroll
          for (int m = 0; m < kGroups; ++m)
            chunk_products<kChunk>(acc[m], us + (q * kTile + m * 16 + g) * pitch + r, pitch, b, tq);
      }
      load_b(c + kLoraWarps * 32, 0);
#pragma unroll
      for (int i = 0; i < 2 * kGroups; ++i)
        if (mine[i] && c + 8 * tq < left) {
          Row8<TOut> v;
#pragma unroll
          for (int n = 0; n < 4; ++n) v.set(2 * n, acc[i >> 1][n][2 * (i & 1)], acc[i >> 1][n][2 * (i & 1) + 1]);
          v.store(out0 + i * ostep + c);
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

template <typename TOut>
const void* expand_tile(int R) {
  if (R % 32 == 0) return (const void*)lora_expand_tile_kernel<TOut, 32>;
  if (R % 16 == 0) return (const void*)lora_expand_tile_kernel<TOut, 16>;
  return (const void*)lora_expand_tile_kernel<TOut, 8>;
}

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
    expand = f32 ? expand_tile<float>(a.R) : expand_tile<__nv_bfloat16>(a.R);
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
