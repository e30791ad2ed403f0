// Low-rank adapters of many requests beside a shared projection:
//   out[t] = y[t] + scale[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// Two kernels over tiles of tokens as they come in the batch (16 tokens, or 64
// in long batches):
//   shrink  u[t] = A[a] x[t]: for every adapter that occurs in the tile, the
//           tile's tokens against the adapter's rows, split over K; fp32
//           partials of the split go to the workspace;
//   expand  sums the partials in order, and for every adapter of the tile adds
//           scale * B u to the rows that use it.
// A token's row belongs to one adapter, so the adapters of a tile are shared
// out over CTAs without any sum across them, and a row is selected, never
// masked by a product: an adapter's infinities or NaN reach its own tokens only.
//
// Both are bound by memory (x, y, and R (K + N) values of each adapter used):
// the tensor core (mma.sync, BF16 x BF16 + FP32) has work for a few clocks per
// line loaded, so a product of 16 rows of which one is wanted costs nothing, and
// there is no sorting.  Fragments are loaded straight from global memory, 16
// bytes a lane: the contraction may be taken in any order, so lane t of a row's
// four takes elements 8t .. 8t+7 of a 32-element block for both operands.
// In the expand the output columns are permuted the same way, so that a lane
// has 8 neighbouring columns of a row.  u keeps its fp32 accuracy as a sum of
// two BF16 terms (2^-17; BF16 output) or three (2^-25; FP32 output).
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
constexpr int kMaxTile = 64;

struct LoraParams {
  LoraArgs a;
  float* u;         // [ksplit][T][R] partial sums
  int ksplit;
  int blocks;       // 32-element blocks of K per CTA of the shrink
  int cols;         // columns per CTA of the expand
};

MXG_DEVINL void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The adapters of a tile of tokens, in order of first use.
struct Tile {
  int id[kMaxTile];     // adapter of each token (-1: none)
  int ord[kMaxTile];    // its number in the list (-1: none)
  int list[kMaxTile];   // adapter by number
  uint32_t rows16[kMaxTile];  // 16-token groups in which it occurs (bit mask)
  int count;
};

template <int kTok>
MXG_DEVINL void read_tile(Tile& s, const LoraArgs& a, int64_t t0) {
  const int tid = threadIdx.x;
  if (tid < kTok) {
    int id = t0 + tid < a.T ? __ldg(a.ids + t0 + tid) : -1;
    if (id >= a.n) {
      report(a.status, MXG_ERR_INDEX);
      id = -1;
    }
    s.id[tid] = id;
  }
  if (tid == 0) s.count = 0;
  __syncthreads();
  if (tid < 32) {  // one warp numbers the first uses, 32 tokens at a time
    int count = 0;
    for (int base = 0; base < kTok; base += 32) {
      const int i = base + tid;
      bool first = i < kTok && s.id[i < kTok ? i : 0] >= 0;
      if (first)
        for (int j = 0; j < i; ++j)
          if (s.id[j] == s.id[i]) { first = false; break; }
      const uint32_t m = __ballot_sync(kFull, first);
      if (first) {
        const int o = count + __popc(m & ((1u << tid) - 1u));
        s.list[o] = s.id[i];
        s.rows16[o] = 0;
      }
      count += __popc(m);
    }
    if (tid == 0) s.count = count;
  }
  __syncthreads();
  if (tid < kTok) {
    int o = -1;
    if (s.id[tid] >= 0) {
      o = 0;
      while (s.list[o] != s.id[tid]) ++o;
      atomicOr(&s.rows16[o], 1u << (tid >> 4));
    }
    s.ord[tid] = o;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// shrink: grid (K split, tiles, adapter groups).  The warps of a CTA take every
// fourth 32-element block of its K range; kM groups of 16 tokens, up to 32
// ranks at a time.
// ---------------------------------------------------------------------------
template <int kM>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(const LoraParams p) {
  constexpr int kTok = 16 * kM;
  constexpr int kUnroll = kM == 1 ? 4 : 2;  // blocks in flight
  __shared__ Tile tile;
  __shared__ float red[kLoraWarps][kTok][33];
  ptx::pdl_launch_dependents();
  const LoraArgs& a = p.a;
  const int64_t t0 = (int64_t)blockIdx.y * kTok;
  read_tile<kTok>(tile, a, t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int64_t kblocks = (a.K + 31) >> 5;
  const int64_t b0 = (int64_t)blockIdx.x * p.blocks;
  const int nb = (int)min((int64_t)p.blocks, kblocks - b0);
  const uint16_t* xk = a.x + t0 * a.ld_x + b0 * 32 + 8 * tq;
  const int kleft = (int)min(a.K - b0 * 32, (int64_t)nb * 32) - 8 * tq;  // of this lane's first block on
  for (int o = blockIdx.z; o < tile.count; o += gridDim.z) {
    const uint32_t groups = tile.rows16[o];
    for (int r0 = 0; r0 < a.R; r0 += 32) {
      const int nt = min(4, (a.R - r0) >> 3);
      const uint16_t* ak = a.A + ((int64_t)tile.list[o] * a.R + r0 + g) * a.K + b0 * 32 + 8 * tq;
      float acc[kM][4][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      for (int b = warp; b < nb; b += kLoraWarps * kUnroll) {
        uint4 xv[kUnroll][kM][2], av[kUnroll][4];
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
          for (int m = 0; m < kM; ++m)
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
          for (int m = 0; m < kM; ++m)
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
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float* d = &red[warp][m * 16 + g][n * 8 + 2 * tq];
          d[0] = acc[m][n][0];
          d[1] = acc[m][n][1];
          d[8 * 33] = acc[m][n][2];
          d[8 * 33 + 1] = acc[m][n][3];
        }
      __syncthreads();
      for (int i = threadIdx.x; i < kTok * 32; i += kLoraThreads) {
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

// ---------------------------------------------------------------------------
// expand: grid (column chunks, tiles, adapter groups).  A warp takes 32 columns
// at a time.
// ---------------------------------------------------------------------------
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

template <int kM, typename TOut>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(const LoraParams p) {
  constexpr int kTok = 16 * kM;
  constexpr int kTerms = sizeof(TOut) == 2 ? 2 : 3;
  __shared__ Tile tile;
  extern __shared__ __align__(16) uint16_t us[];  // [kTerms][kTok][R + 8]: scale * u as a sum of BF16 terms
  const LoraArgs& a = p.a;
  const int64_t t0 = (int64_t)blockIdx.y * kTok;
  read_tile<kTok>(tile, a, t0);
  if (blockIdx.z > 0 && (int)blockIdx.z >= tile.count) return;
  const int pitch = a.R + 8;
  ptx::pdl_wait();
  for (int i = threadIdx.x; i < kTok * a.R; i += kLoraThreads) {
    const int row = i / a.R, r = i - row * a.R;
    const int o = tile.ord[row];
    if (o < 0 || o % (int)gridDim.z != (int)blockIdx.z) continue;
    const float* src = p.u + (t0 + row) * a.R + r;
    const int64_t step = a.T * a.R;
    float s = 0.0f;
    for (int k0 = 0; k0 < p.ksplit; k0 += 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k0 + k < p.ksplit ? __ldcg(src + (k0 + k) * step) : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    if (a.scale != nullptr) s *= __ldg(a.scale + tile.id[row]);
#pragma unroll
    for (int q = 0; q < kTerms; ++q) {
      const __nv_bfloat16 h = __float2bfloat16_rn(s);
      us[((int64_t)q * kTok + row) * pitch + r] = *reinterpret_cast<const uint16_t*>(&h);
      s -= __bfloat162float(h);
    }
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int64_t c1 = min(a.N, (int64_t)(blockIdx.x + 1) * p.cols);
  for (int64_t c0 = (int64_t)blockIdx.x * p.cols + warp * 32; c0 < c1; c0 += kLoraWarps * 32) {
    const bool cin = c0 + 8 * tq < c1;  // N is a multiple of 8
    for (int o = blockIdx.z; o < max(tile.count, 1); o += gridDim.z) {
      const bool any = o < tile.count;
      const uint32_t groups = any ? tile.rows16[o] : 0u;
      // this lane's rows: those of adapter o, and the ones without adapter in the first pass
      Row8<TOut> y[kM][2];
      bool mine[kM][2];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = m * 16 + g + 8 * h;
          const int ro = tile.ord[row];
          mine[m][h] = cin && t0 + row < a.T && (ro == o && any || ro < 0 && o == 0);
          if (mine[m][h]) y[m][h].load(a.y, (t0 + row) * a.ld_y + c0 + 8 * tq);
        }
      float acc[kM][4][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
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
          for (int m = 0; m < kM; ++m)
            if ((groups >> m) & 1) {
#pragma unroll
              for (int q = kTerms - 1; q >= 0; --q) {
                const uint16_t* u = us + ((int64_t)q * kTok + m * 16 + g) * pitch + r0 + 8 * tq;
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
          for (int m = 0; m < kM; ++m)
            if ((groups >> m) & 1) {
#pragma unroll
              for (int q = kTerms - 1; q >= 0; --q) {
                const uint16_t* u = us + ((int64_t)q * kTok + m * 16 + g) * pitch + r0 + 4 * tq;
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
          for (int m = 0; m < kM; ++m)
            if ((groups >> m) & 1) {
#pragma unroll
              for (int q = kTerms - 1; q >= 0; --q) {
                const uint16_t* u = us + ((int64_t)q * kTok + m * 16 + g) * pitch + r0 + 2 * tq;
                const uint32_t lo = *reinterpret_cast<const uint32_t*>(u);
                const uint32_t hi = *reinterpret_cast<const uint32_t*>(u + 8 * pitch);
#pragma unroll
                for (int n = 0; n < 4; ++n) mma_bf16(acc[m][n], lo, hi, 0u, 0u, bv[n], 0u);
              }
            }
        }
      }
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (mine[m][h]) {
            const int row = m * 16 + g + 8 * h;
            if (tile.ord[row] >= 0) {
              float d[8];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                d[2 * n] = acc[m][n][2 * h];
                d[2 * n + 1] = acc[m][n][2 * h + 1];
              }
              y[m][h].add(d);
            }
            y[m][h].store(a.out, (t0 + row) * a.ld_out + c0 + 8 * tq);
          }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kLongBatch = 1024;  // tokens from which tiles have 64 tokens

int tile_tokens(int64_t T) { return T >= kLongBatch ? 64 : 16; }

// 32-element blocks of K per shrink CTA: about four CTAs per SM if K allows,
// at least one block and at most 64 for each warp.
int shrink_blocks(int64_t T, int64_t K) {
  const int64_t tiles = (T + tile_tokens(T) - 1) / tile_tokens(T);
  const int64_t kblocks = (K + 31) / 32;
  const int64_t split = std::max<int64_t>(1, (640 + tiles - 1) / tiles);
  const int64_t per = (kblocks + split - 1) / split;
  const int64_t warp4 = (per + kLoraWarps - 1) / kLoraWarps * kLoraWarps;
  return (int)std::min<int64_t>(warp4, 64 * kLoraWarps);
}

template <int kM>
cudaError_t launch_lora(const LoraParams& p, cudaStream_t stream, int num_sms) {
  const LoraArgs& a = p.a;
  const int64_t tiles = (a.T + 16 * kM - 1) / (16 * kM);
  const int groups = std::min<int>(a.n, kM == 1 ? 16 : 4);
  if (tiles > 65535) return cudaErrorInvalidConfiguration;
  lora_shrink_kernel<kM><<<dim3((unsigned)p.ksplit, (unsigned)tiles, (unsigned)groups), kLoraThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool f32 = a.dtype == MXG_OUT_F32;
  const void* fn = f32 ? (const void*)lora_expand_kernel<kM, float> : (const void*)lora_expand_kernel<kM, __nv_bfloat16>;
  const size_t smem = (size_t)(f32 ? 3 : 2) * 16 * kM * (a.R + 8) * 2;
  if (smem > 40 * 1024) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * 16 * kM * (128 + 8) * 2);
    if (e != cudaSuccess) return e;
  }
  LoraParams q = p;
  // columns per CTA: as many as leave about eight CTAs per SM, in steps of 128
  const int64_t chunks = std::max<int64_t>(1, 8 * (int64_t)num_sms / tiles);
  q.cols = (int)std::min<int64_t>(4096, std::max<int64_t>(128, (a.N / chunks + 127) / 128 * 128));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((a.N + q.cols - 1) / q.cols), (unsigned)tiles, (unsigned)groups);
  cfg.blockDim = dim3(kLoraThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {(void*)&q};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int R) {
  const int64_t per = shrink_blocks(std::max<int64_t>(T, 1), K);
  return (size_t)(((K + 31) / 32 + per - 1) / per) * std::max<int64_t>(T, 1) * R * sizeof(float);
}

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t stream, int num_sms) {
  LoraParams p{};
  p.a = a;
  p.u = a.ws;
  p.blocks = shrink_blocks(a.T, a.K);
  p.ksplit = (int)(((a.K + 31) / 32 + p.blocks - 1) / p.blocks);
  return tile_tokens(a.T) == 16 ? launch_lora<1>(p, stream, num_sms) : launch_lora<4>(p, stream, num_sms);
}

}  // namespace mxg
