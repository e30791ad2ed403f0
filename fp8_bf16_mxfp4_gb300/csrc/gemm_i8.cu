// Products of 8-bit integers with a scale per token and per channel, grouped over
// experts, and the quantizer in front of them:
//
//   quantize   a = max(max |x[t]|, 2^-100), s = a / 127, q = rint(x (127 / a))
//   product    y[i, n] = sa[i] sw[g N + n] sum_k qa[i, k] qw[g N + n, k],  g row i's expert
//
// sm_103a has no integer kind of tcgen05.mma, and its integer mma.sync runs at the
// rate of dp4a.  Every integer up to 2048 is an FP16 value, so products are taken as
// FP16's: exact, with fp32 sums (exact up to 2^24; the tensor core cuts off what is below
// the last of a sum's 24 bits, 16 elements at a time).  Weights stay 8-bit integers as
// far as the SM.  Three forms:
//
//   few      tiles of 8 or 16 rows, mma.sync, weights from global memory to registers;
//   cut      tiles of 32, 64 or 128 rows on the tensor cores, the contraction of all
//            tiles cut into equal runs;
//   whole    tiles of 256 rows on the tensor cores.
//
// 8192 rows of 8 experts, 4096 x 14336: 505 us, 1.9 PFLOP/s (0.95 and more of what
// torch's BF16 product of two such matrices reaches), where the tensor pipe is busy 81 %
// of the time.  128 rows of 32 experts, 4096 x 7168: 155 us, 6.1 TB/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "gemm_common.cuh"
#include "sm100_ptx.cuh"

namespace mxg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Quantizer
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;  // at most
constexpr int kQKeep = 4;  // 16-byte pieces of a row that a thread keeps between its two passes

// A CTA takes a token (and, where there are few, every gridDim.y-th of its slots):
// its largest value, then its codes, once for every output row.

// q = rint(x r) in the low 16 bits: the sum with 1.5 2^23 rounds the exact product
// to an integer, to nearest even, in one step.
MXG_DEVINL uint32_t round_code(float x, float r) { return __float_as_uint(fmaf(x, r, 12582912.0f)); }

template <bool kF16>
__global__ void __launch_bounds__(kQThreads) int8_quantize_kernel(const uint4* __restrict__ x, int64_t ld_x,
                                                                  const int32_t* __restrict__ rows, int k, int64_t out_rows,
                                                                  int64_t pieces, uint8_t* __restrict__ q, int64_t ld_q,
                                                                  float* __restrict__ scale, int32_t* status) {
  __shared__ uint32_t part[kQThreads / 32];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();  // rows, and x too, may come from the kernel before
  const int64_t t = blockIdx.x;
  const uint4* src = x + t * ld_x;
  uint4 keep[kQKeep];
  uint32_t m = 0;
  auto amax = [&](const uint4& v) {
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  };
#pragma unroll
  for (int i = 0; i < kQKeep; ++i) {
    const int64_t c = threadIdx.x + (int64_t)i * blockDim.x;
    keep[i] = c < pieces ? ptx::ld_global_v4(src + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kQKeep; ++i) amax(keep[i]);
  for (int64_t c = threadIdx.x + (int64_t)kQKeep * blockDim.x; c < pieces; c += blockDim.x) amax(ptx::ld_global_v4(src + c));
  m = __reduce_max_sync(kFull, max(m & 0xFFFFu, m >> 16));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) m = max(m, part[w]);
  // A row with an infinity or NaN has the scale NaN and codes 0.
  const bool finite = m < 0x7F80u;
  const float a = fmaxf(__uint_as_float(m << 16), 0x1p-100f);
  const float r = finite ? 127.0f / a : 0.0f;
  const float s = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);
  constexpr float kLeast = 0x1p-100f / 127.0f;  // the scale of a row of zeros

  const int64_t first = rows != nullptr ? t * k : t;
  auto row_at = [&](int j, bool& on) -> int64_t {
    if (rows == nullptr) { on = true; return t; }
    const int32_t e = ptx::ld_global_s32(rows + first + j);
    const int64_t at = e < 0 ? -1 - (int64_t)e : e;
    on = e >= 0;
    return at < out_rows ? at : -1;
  };
  for (int j = blockIdx.y + threadIdx.x * gridDim.y; j < k; j += blockDim.x * gridDim.y) {
    bool on;
    const int64_t at = row_at(j, on);
    if (at >= 0) scale[at] = on ? s : kLeast;
    else report(status, MXG_ERR_INDEX);
  }
  auto emit = [&](int64_t c, const uint4& v) {
    uint4 o = make_uint4(0, 0, 0, 0);
    if (finite) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[2 * i] = round_code(bf16lo_to_f32(w[i]), r);
        b[2 * i + 1] = round_code(bf16hi_to_f32(w[i]), r);
      }
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kF16) {
          const __half2 f = __floats2half2_rn(__uint_as_float(b[2 * i]) - 12582912.0f,
                                              __uint_as_float(b[2 * i + 1]) - 12582912.0f);
          h[i] = *reinterpret_cast<const uint32_t*>(&f);
        } else {
          h[i] = __byte_perm(b[2 * i], b[2 * i + 1], 0x0040);  // two bytes
        }
      }
      if constexpr (kF16) o = make_uint4(h[0], h[1], h[2], h[3]);
      else o = make_uint4(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410), 0, 0);
    }
    for (int j = blockIdx.y; j < k; j += gridDim.y) {
      bool on;
      const int64_t at = row_at(j, on);
      if (at < 0) continue;
      uint8_t* dst = q + at * ld_q + c * (kF16 ? 16 : 8);
      const uint4 z = on ? o : make_uint4(0, 0, 0, 0);
      if constexpr (kF16) *reinterpret_cast<uint4*>(dst) = z;
      else *reinterpret_cast<uint2*>(dst) = make_uint2(z.x, z.y);
    }
  };
#pragma unroll
  for (int i = 0; i < kQKeep; ++i) {
    const int64_t c = threadIdx.x + (int64_t)i * blockDim.x;
    if (c < pieces) emit(c, keep[i]);
  }
  for (int64_t c = threadIdx.x + (int64_t)kQKeep * blockDim.x; c < pieces; c += blockDim.x) emit(c, ptx::ld_global_v4(src + c));
}

// Four 8-bit integers -> four FP16 values: with the sign bit flipped a byte is
// q + 128, which under the exponent of 1024 is 1152 + q.
MXG_DEVINL void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}

// In front of the product: the join counters zeroed, 8-bit activations widened.
constexpr int kPrepThreads = 256;
__global__ void __launch_bounds__(kPrepThreads) int8_prep_kernel(uint32_t* sync, int words, const uint8_t* __restrict__ a,
                                                                 int64_t ld_a, int64_t S, int64_t per_row,
                                                                 uint4* __restrict__ wide) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();  // the activations may come from the kernel before, which may also be at work with the counters
  const int64_t i0 = (int64_t)blockIdx.x * kPrepThreads + threadIdx.x;
  if (i0 < words) sync[i0] = 0;
  for (int64_t i = i0; i < S * per_row; i += (int64_t)gridDim.x * kPrepThreads) {
    const int64_t r = i / per_row, c = i - r * per_row;
    const uint4 v = ptx::ld_global_v4(a + r * ld_a + c * 16);
    uint32_t o[8];
    widen4(v.x, o[0], o[1]);
    widen4(v.y, o[2], o[3]);
    widen4(v.z, o[4], o[5]);
    widen4(v.w, o[6], o[7]);
    wide[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    wide[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// One warp: the first row off[g] and first unit tile[g] of every expert, `per_tile`
// units for every `tok` of its rows; *bad where a split is negative or they do not
// add up to S.  Lane l has experts [l * per, l * per + per).
MXG_DEVINL void plan_units(const int32_t* splits, int G, int S, int tok, int per_tile, int32_t* off, int32_t* tile, int* bad) {
  const int lane = threadIdx.x & 31, per = (G + 31) >> 5;
  int64_t rows = 0, units = 0;
  bool neg = false;
  auto split = [&](int g) -> int64_t { return splits != nullptr ? (int64_t)ptx::ld_global_s32(splits + g) : (int64_t)S; };
  auto units_of = [&](int64_t m) { return (m + tok - 1) / tok * per_tile; };
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i;
    const int64_t m = g < G ? split(g) : 0;
    neg |= m < 0;
    rows += m;
    units += units_of(m > 0 ? m : 0);
  }
  int64_t rs = rows, us = units;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t orow = __shfl_up_sync(kFull, rs, d), ou = __shfl_up_sync(kFull, us, d);
    if (lane >= d) { rs += orow; us += ou; }
  }
  const bool wrong = __any_sync(kFull, neg) || __shfl_sync(kFull, rs, 31) != S;
  rows = rs - rows;
  units = us - units;
  for (int i = 0; i < per && !wrong; ++i) {
    const int g = lane * per + i;
    if (g < G) {
      off[g] = (int32_t)rows;
      tile[g] = (int32_t)units;
      const int64_t m = split(g);
      rows += m;
      units += units_of(m);
    }
  }
  if (lane == 31) {
    off[G] = (int32_t)rs;
    tile[G] = (int32_t)us;
    *bad = wrong;
  }
}

MXG_DEVINL uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ---------------------------------------------------------------------------
// A few rows per expert.  A unit is 16 channels of one expert against a tile of up
// to 16 of its rows.  Weights go from global memory to registers, 16 bytes a lane,
// and are widened there to the A fragments of mma.sync (m16n8k16, FP16): a lane has
// the same four bytes of a channel that it has of a row, in whatever order mma.sync
// numbers them, so nothing is moved between lanes.  The rows' bytes are in shared
// memory (FP16 codes narrowed again: half the room) and are widened as they are used.
// A CTA has 16 warps: `split` of them share a unit's contraction, 128 elements in
// turn, and 16 / split units are on their way at a time; partial sums are added
// through shared memory in the warps' order.  A CTA takes an equal run of units, in
// the order expert, tile of rows, channels, and its loads run ahead over units.
// mma.sync makes 974 products of FP16 codes a clock and SM (of 8-bit integers 255, as
// does dp4a), of which 8 rows at the rate of memory need 190: bound by HBM.
// 128 rows of 32 experts, 4096 x 7168: 155 us, 6.1 TB/s (167 with dp4a, 184 in the
// form for more rows; 180 where one expert has 9 rows); 1 row, 28672 x 8192: 43 us, of
// which 6 are start and end; 1 row, 4096 x 7168: 11 us.  Loads of 32 bytes a lane, 8 warps with twice the loads in
// flight, and joins that no warp waits for measured the same or worse.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewChan = 16;
constexpr int kFewDepth = 4;   // chunks of 128 elements that a warp has in flight
constexpr int kFewCol = 20;    // words between columns of a partial tile (16 channels each): 4 columns, 32 banks

struct FewParams {
  const int32_t* splits;
  int G, S, N, K;
  int tok;           // rows of a tile: 8 or 16
  int per_tile;      // units of a tile of rows
  int split;         // warps of a unit, a power of two up to 16
  const uint8_t* a;
  int64_t ld_a;
  int f16;           // the rows' codes are FP16
  const float* sa;
  const uint8_t* w;
  int64_t ld_w;
  const float* sw;
  void* out;
  int64_t ld_out;
  int out_f32;
  int32_t* status;
};

// Bytes between rows in shared memory: 64 past a multiple of 128, so that two rows'
// 64 bytes are in different banks.
__host__ __device__ inline int few_stride(int64_t K) { return (int)((K + 127) / 128 * 128) + 64; }
inline int64_t few_part_bytes(int tok) { return (int64_t)2 * kFewWarps * tok * kFewCol * 4; }

// 16 FP16 codes -> 16 bytes: q + 1536 has q in its low byte.
MXG_DEVINL uint4 narrow16(const uint4& a, const uint4& b) {
  const __half2 bias = __half2half2(__ushort_as_half(0x6600));
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 s = __hadd2(*reinterpret_cast<const __half2*>(&w[i]), bias);
    h[i] = *reinterpret_cast<const uint32_t*>(&s);
  }
  return make_uint4(__byte_perm(h[0], h[1], 0x6420), __byte_perm(h[2], h[3], 0x6420), __byte_perm(h[4], h[5], 0x6420),
                    __byte_perm(h[6], h[7], 0x6420));
}

// The tile's rows to shared memory, as bytes.
MXG_DEVINL void few_stage(const FewParams& p, uint8_t* x, int tok0, int n) {
  const int pieces = p.K / 16, stride = few_stride(p.K);
  __syncthreads();  // the rows before are no longer read
  for (int i = threadIdx.x; i < n * pieces; i += kFewThreads) {
    const int t = i / pieces, c = i - t * pieces;
    const uint8_t* src = p.a + (int64_t)(tok0 + t) * p.ld_a;
    uint4 r;
    if (p.f16) {
      const uint4* s = reinterpret_cast<const uint4*>(src) + 2 * c;
      r = narrow16(s[0], s[1]);
    } else {
      r = reinterpret_cast<const uint4*>(src)[c];
    }
    *reinterpret_cast<uint4*>(x + t * stride + c * 16) = r;
  }
  __syncthreads();
}

// Channels [c0, c1) of one expert for a tile of n <= 8 kNT rows.
template <int kNT>
MXG_DEVINL void few_tile(const FewParams& p, uint8_t* x, float* part, int e, int tok0, int n, int c0, int c1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q16 = (lane & 3) * 16;
  const int split = p.split, kp = warp & (split - 1), ug = warp / split, at_once = kFewWarps / split;
  const int chunks = (p.K + 127) >> 7, turns = (chunks + split - 1) / split;  // a warp's chunks: kp, kp + split, ...
  const int slots = (turns + kFewDepth - 1) / kFewDepth * kFewDepth;  // of the ring, for one unit
  const int step = at_once * kFewChan, iters = (c1 - c0 + step - 1) / step;
  const int stride = few_stride(p.K);

  // what is loaded next: chunk kp + split l_i of this warp's unit of turn l_it
  int l_it = 0, l_i = 0;
  const uint8_t *w0 = nullptr, *w8 = nullptr;  // this lane's rows: channels g and g + 8 of the unit
  auto point = [&]() {  // past the last channel: not stored
    const uint32_t chan = c0 + ((uint32_t)l_it * at_once + ug) * kFewChan + g, most = c1 - 1;  // up to 512 above N
    w0 = p.w + ((int64_t)e * p.N + min(chan, most)) * p.ld_w + q16;
    w8 = p.w + ((int64_t)e * p.N + min(chan + 8, most)) * p.ld_w + q16;
  };
  point();
  uint4 v[kFewDepth][4];
  auto load = [&](uint4* d) {  // channel g, g + 8 of bytes 0-63, then 64-127 of the chunk
    const int k = (kp + split * l_i) << 7;
    const uint4 z = make_uint4(0, 0, 0, 0);
    const bool on = l_i < turns && l_it < iters;
    const bool lo = on && k + q16 < p.K, hi = on && k + q16 + 64 < p.K;
    d[0] = lo ? ptx::ld_global_v4(w0 + k) : z;
    d[1] = lo ? ptx::ld_global_v4(w8 + k) : z;
    d[2] = hi ? ptx::ld_global_v4(w0 + k + 64) : z;
    d[3] = hi ? ptx::ld_global_v4(w8 + k + 64) : z;
    if (++l_i == slots) {
      l_i = 0;
      ++l_it;
      point();
    }
  };
#pragma unroll
  for (int s = 0; s < kFewDepth; ++s) load(v[s]);

  few_stage(p, x, tok0, n);  // while the first weights are on their way

  float acc[kNT][4];
#pragma unroll
  for (int t = 0; t < kNT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
  const uint32_t xs = ptx::smem_u32(x) + g * stride + q16;
  auto multiply = [&](const uint4* d, int k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t b[kNT][4];
#pragma unroll
      for (int t = 0; t < kNT; ++t) ptx::ld_shared_v4(xs + t * 8 * stride + k + h * 64, b[t]);
      const uint32_t r0[4] = {d[2 * h].x, d[2 * h].y, d[2 * h].z, d[2 * h].w};
      const uint32_t r8[4] = {d[2 * h + 1].x, d[2 * h + 1].y, d[2 * h + 1].z, d[2 * h + 1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a0, a1, a2, a3;
        widen4(r0[j], a0, a2);
        widen4(r8[j], a1, a3);
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          uint32_t b0, b1;
          widen4(b[t][j], b0, b1);
          asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                       : "+f"(acc[t][0]), "+f"(acc[t][1]), "+f"(acc[t][2]), "+f"(acc[t][3])
                       : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        }
      }
    }
  };
  for (int it = 0; it < iters; ++it) {
    for (int i = 0; i < turns; i += kFewDepth) {
#pragma unroll
      for (int s = 0; s < kFewDepth; ++s) {
        const int c = kp + split * (i + s);
        if (c < chunks) multiply(v[s], c << 7);
        load(v[s]);
      }
    }
    // partial tiles: lane (g, q) has channels g and g + 8 of columns 2 q and 2 q + 1
    float* to_part = part + ((it & 1) * kFewWarps + warp) * (kNT * 8 * kFewCol);
    const int col = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      float* at = to_part + (t * 8 + col) * kFewCol + g;
      at[0] = acc[t][0];
      at[kFewCol] = acc[t][1];
      at[8] = acc[t][2];
      at[kFewCol + 8] = acc[t][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
    }
    __syncthreads();  // (the buffer is written again after the next one)
    for (int o = threadIdx.x; o < at_once * kNT * 128; o += kFewThreads) {
      const int which = o / (kNT * 128), t = (o >> 4) & (kNT * 8 - 1), r = o & 15;
      const int chan = c0 + (it * at_once + which) * kFewChan + r;
      if (t >= n || chan >= c1) continue;
      const float* src = part + ((it & 1) * kFewWarps + which * split) * (kNT * 8 * kFewCol) + t * kFewCol + r;
      float sum = 0.0f;
      for (int q = 0; q < split; ++q) sum += src[q * (kNT * 8 * kFewCol)];
      const float y = sum * p.sw[(int64_t)e * p.N + chan] * p.sa[tok0 + t];
      const int64_t to = (int64_t)(tok0 + t) * p.ld_out + chan;
      if (p.out_f32) static_cast<float*>(p.out)[to] = y;
      else static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(y);
    }
  }
}

__global__ void __launch_bounds__(kFewThreads, 1) int8_few_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t few_smem[];  // rows [tok][stride], then partial tiles
  __shared__ int32_t off[kMaxExperts + 1], tile[kMaxExperts + 1];
  __shared__ int bad;
  ptx::pdl_wait();  // all operands may come from the kernel before
  if (threadIdx.x < 32) plan_units(p.splits, p.G, p.S, p.tok, p.per_tile, off, tile, &bad);
  __syncthreads();
  if (bad) {  // every CTA sees it: nothing is written
    if (threadIdx.x == 0) report(p.status, MXG_ERR_SPLITS);
    return;
  }
  uint8_t* x = few_smem;
  float* part = reinterpret_cast<float*>(few_smem + p.tok * few_stride(p.K));
  const int64_t units = tile[p.G];
  int u = (int)(units * blockIdx.x / gridDim.x);
  const int end = (int)(units * (blockIdx.x + 1) / gridDim.x);
  while (u < end) {  // a tile of rows at a time
    const int e = find_prefix(tile, p.G, u), tt = (u - tile[e]) / p.per_tile;
    const int first = tile[e] + tt * p.per_tile, last = min(end, first + p.per_tile);
    const int tok0 = off[e] + tt * p.tok, n = min(p.tok, off[e + 1] - tok0);
    const int c0 = (u - first) * kFewChan, c1 = min(p.N, (last - first) * kFewChan);
    if (n <= 8) few_tile<1>(p, x, part, e, tok0, n, c0, c1);
    else few_tile<2>(p, x, part, e, tok0, n, c0, c1);
    u = last;
  }
}

// ---------------------------------------------------------------------------
// Product on the tensor cores (tcgen05, kind::f16)
//
// Weights are the M operand, which the tensor core reads from TMEM: a warp that turns
// a row's bytes into FP16 writes them where they are needed, and shared memory never
// holds them twice as wide.  Activations are the N operand, from shared memory, as
// FP16 (the quantizer writes them so, or a kernel in front widens them once).  A pair
// of CTAs on neighbouring SMs (a cluster) shares a tile of 256 channels through the
// 2-SM MMA: each has 128 channels and half of the rows, so that shared memory takes
// 96 bytes a clock; a single CTA's 160 would not fit its 128.  Per CTA:
//   warp 0       producer: 128 channels x 128 bytes of weights and the rows' 128
//                elements a stage, by TMA;
//   warp 1       TMEM owner; in the even CTA MMA issuer for both, 8 MMAs a stage;
//   warps 2-5    epilogue, one per TMEM lane quarter (a lane is a channel);
//   warps 6-9    weights to FP16, shared memory to TMEM;
//   warp 10      waits for the issuer (cut form);
//   warps 10-13  epilogue (whole tiles): with one accumulator the next tile waits
//                for it (1024 rows of 32 experts each, 2048 x 1024: 97 us, 119 with four
//                warps; x 2048, 4096 channels: 302, 306; 14 warps leave 128 registers a
//                thread, of which 60 bytes spill).
// Cut form: the stages of all units (expert, channel tile, row tile) are cut into one
// equal run per pair, so that every SM streams the same number of weight bytes; cut
// units are joined through fp32 partials, added in run order by the last to arrive.
// Bound there: an MMA of 16 contraction elements takes about 110 clocks whatever its
// rows while the widening warps write TMEM (152 us for 1024 rows of 32 experts, 4096 x
// 7168, without those writes; 184 with them; 138 of HBM).  One row tile of few rows is
// latency: 20 rows, 4096 x 4096, 14 us, of which 4 are the loads', 1 the start, 3 the
// join and 3 two launches.
// ---------------------------------------------------------------------------
constexpr int kChan = kUnitChan / 2;       // channels of a CTA's tile (TMEM lanes)
constexpr int kWBytes = kChan * kStageK;
constexpr int kI8TmemCols = 512;
constexpr int kACols = kStageK / 2;        // TMEM columns of a stage's weights (two FP16 a column)
constexpr uint32_t kWatchBar = 1;          // named barrier of the issuer and the warp that waits for it

// kTok: the tokens of a tile.  Accumulators first (two of them, but for 256
// columns), then the ring of widened weights.
template <int kTok>
struct I8Cfg {
  static constexpr int kBufs = kTok == 256 ? 1 : 2;
  static constexpr bool kCut = kTok < 256;             // units may be cut over pairs
  static constexpr int kWatch = 10;                    // the warp that waits for the issuer
  static constexpr int kEpi = kCut ? 4 : 8;            // epilogue warps
  static constexpr int kThreads = 32 * (kWatch + (kCut ? 1 : 4));
  static constexpr int kRows = kTok / 2;               // tokens whose elements a CTA loads
  static constexpr int kXBox = kRows * 128;            // 64 elements of each
  static constexpr int kStageBytes = kWBytes + 2 * kXBox;
  static constexpr int kACol = kTok >= 128 ? 256 : (kTok >= 64 ? 128 : 64);
  // Slots of widened weights in TMEM, and stages in shared memory: more of them
  // where a stage is small, since the loads' latency under load (about 2.3 us) is
  // most of a stage's time.
  static constexpr int kSlots = (kI8TmemCols - kACol) / kACols;
  static constexpr int kStages = kTok == 32 ? 10 : kTok == 64 ? 8 : kTok == 128 ? 6 : 4;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kBars = 3 * kStages + 5;
  static constexpr int kMiscOff = kBarOff + ((kBars * 8 + 15) & ~15);
  static constexpr int kOffOff = kMiscOff + 16;                      // int32 [G + 1]: first row of each expert
  static constexpr int kTileOff = kOffOff + (kMaxExperts + 4) * 4;   // int32 [G + 1]: first unit of each expert
  static constexpr int kSaOff = kTileOff + (kMaxExperts + 4) * 4;    // float [8][128]: the tile's token scales (256 tokens)
  static constexpr int kTotal = kSaOff + (kCut ? 0 : 4 * kTok * 4) + 1024;  // + alignment slack
  static_assert(kSaOff % 16 == 0, "token scales are read 16 bytes at a time");
  static_assert(kBufs * kTok <= kACol && kACol + kSlots * kACols <= kI8TmemCols, "TMEM holds accumulators and ring");
  static_assert(kStageBytes % 1024 == 0 && kXBox % 1024 == 0, "tiles keep the swizzle-atom alignment");
  static_assert(kTotal <= 232448, "fits the 227 KB of one CTA");
  static_assert(kSlots <= kStages, "a slot's MMAs are those of an earlier stage of the ring");
};

struct I8Params : I8Order {
  const int32_t* splits;  // null: one expert of all S rows
  int S, N;
  const float* sa;
  const float* sw;
  void* out;
  int64_t ld_out;
  int out_f32;
  float* part;            // [2 * pairs][2][kTok][128] partial sums of cut units
  uint32_t* sync;         // [pairs][8] arrivals at a cut unit
  int32_t* status;
  uint64_t timeout_ns, drain_ns;
  uint32_t idesc;
};

// Tokens that the MMAs of a tile take: its own, to a multiple of 16 (half of them
// in each CTA).  An expert's last tile is often short.
MXG_DEVINL int mma_tokens(int n) { return (n + 15) & ~15; }

// The even CTA issues the MMAs of both (M = 256: its TMEM has channels 0-127 of the
// tile, the odd CTA's 128-255; each has half of the tokens' elements in shared
// memory).  The widening warps and the epilogues of both arrive on the even CTA's
// barriers, and every commit reaches the barriers of both.
template <int kTok>
__global__ void __launch_bounds__(I8Cfg<kTok>::kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8Params p) {
  using L = I8Cfg<kTok>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank();

  const uint32_t bar0 = sbase + L::kBarOff;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };                     // the stage's bytes are here
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };        // its MMAs have read them
  auto ready_bar = [&](int s) { return bar0 + 8u * (2 * kStages + s); };    // its weights are in TMEM
  auto acc_full = [&](int b) { return bar0 + 8u * (3 * kStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8u * (3 * kStages + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (3 * kStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int* bad_flag = reinterpret_cast<int*>(smem + L::kMiscOff + 8);
  int32_t* off = reinterpret_cast<int32_t*>(smem + L::kOffOff);
  int32_t* tile = reinterpret_cast<int32_t*>(smem + L::kTileOff);
  // arrive on the issuing CTA's barrier (the even CTA of a pair)
  auto arrive_issuer = [&](uint32_t bar) { ptx::mbar_arrive_cluster(ptx::mapa_shared(bar, 0)); };

  if (warp == 0) {
    ptx::pdl_wait();  // all operands may come from the kernel before
    plan_units(p.splits, p.G, p.S, kTok, p.n_chan, off, tile, bad_flag);
    if (lane == 0) *abort_flag = 0;
  } else if (warp == 1) {
    ptx::tmem_alloc_g<2>(ptx::smem_u32(tmem_slot), kI8TmemCols);
    ptx::tmem_relinquish_g<2>();
  } else if (threadIdx.x == 64) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
      ptx::mbar_init(ready_bar(s), 8);  // four warps of either CTA
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(acc_full(b), 1);
      ptx::mbar_init(acc_empty(b), 2 * L::kEpi);  // the epilogue warps of either CTA
    }
    ptx::mbar_init(drain_bar, 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the peer's barriers are initialised before any remote arrival or commit reaches them
  ptx::cluster_sync();
  ptx::tc_fence_after();
  ptx::pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const bool bad = *bad_flag != 0;  // every CTA sees it: nothing is written
  if (bad && threadIdx.x == 0) report(p.status, MXG_ERR_SPLITS);

  const int units = bad ? 0 : tile[p.G];
  const int pair = (int)ptx::cluster_id_x(), pairs = (int)ptx::nclusters_x();
  const I8Runs runs(units, p.nk, units > 0 ? off[p.G] / (units / p.n_chan) : 0, pairs);  // (the mean rows of a tile)
  I8Walker<kTok, L::kCut> w;
  if constexpr (L::kCut) {
    w.s = w.end = 0;
    if (pair < runs.pairs) runs.run(pair, w.s, w.end);
    w.per_unit = p.nk;
  } else {
    w.s = pair;
    w.end = units;
    w.per_unit = pairs;
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      while (ok && w.next(p, off, tile)) {
        const int row_w = w.e * p.N + w.chan0 + rank * kChan;
        const int row_x = w.tok0 + rank * mma_tokens(w.n) / 2;
        for (int kc = w.k0; kc < w.k1; ++kc) {
          if (!ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.timeout_ns)) { ok = false; break; }
          const uint32_t fb = full_bar(stage);
          ptx::mbar_arrive_expect_tx(fb, L::kStageBytes);  // whole boxes: what lies past the matrix is zero
          armed |= 1u << stage;
          armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          const uint32_t sw = sbase + stage * L::kStageBytes;
          ptx::tma_load_2d(sw, &tmW, kc * kStageK, row_w, fb);
          ptx::tma_load_2d(sw + kWBytes, &tmX, kc * kStageK, row_x, fb);
          ptx::tma_load_2d(sw + kWBytes + L::kXBox, &tmX, kc * kStageK + 64, row_x, fb);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // do not leave copies in flight: wait (bounded) for every armed stage
      for (int s = 0; s < kStages; ++s)
        if ((armed >> s) & 1u) {
          volatile int no_abort = 0;
          ptx::mbar_wait(full_bar(s), (armed_phase >> s) & 1u, &no_abort, p.status, p.drain_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop in step (each wait ends in a vote) and one
    // lane issues and hands the stages back.  A wait on an mbarrier by the thread
    // that issues holds it until its MMAs are done.  256 tokens' MMAs take longer
    // than that; for fewer a second warp waits and meets the issuer at a named
    // barrier (128 rows of 32 experts, 4096 x 7168: 184 us, 201 with the waits here).
    if (rank == 0) {
      const uint32_t el = lane == 0;
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      int stage = 0, slot = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      while (ok && w.next(p, off, tile)) {
        const int buf = L::kBufs == 2 ? count & 1 : 0;
        if constexpr (!L::kCut) {
          ok = ptx::mbar_wait_warp(acc_empty(buf), (count & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns);
          if (!ok) break;
        }
        const uint32_t d = tm + buf * kTok;
        const uint32_t idesc = p.idesc | ((uint32_t)(mma_tokens(w.n) >> 3) << 17);
        for (int kc = w.k0; kc < w.k1; ++kc) {
          if constexpr (L::kCut) ok = !ptx::named_bar_or(kWatchBar, 64, false);
          else ok = ptx::mbar_wait_warp(ready_bar(stage), phase, abort_flag, p.status, p.timeout_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t a = tm + L::kACol + slot * kACols;
          const uint64_t b = ptx::smem_desc(sbase + stage * L::kStageBytes + kWBytes, 16, 1024, 2);
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 16 contraction elements: 8 columns, 32 bytes of each token's row
            ptx::mma_f16_ts_pair_if(el, d, a + 8 * j, b + (uint64_t)((j >> 2) * (L::kXBox >> 4) + 2 * (j & 3)), idesc,
                                    (kc != w.k0) || j != 0);
          issued = true;
          ptx::tc_commit_pair_if(el, empty_bar(stage));
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
          if (++slot == L::kSlots) slot = 0;
        }
        if (!ok) break;
        ptx::tc_commit_pair_if(el, acc_full(buf));
        ++count;
      }
      if (issued) {  // every MMA has retired before TMEM is released
        if (lane == 0) ptx::tc_commit_g<2>(drain_bar);
        volatile int no_abort = 0;
        ptx::mbar_wait(drain_bar, 0, &no_abort, p.status, p.drain_ns);
      }
    }
  } else if (L::kCut && warp == L::kWatch) {
    // ------------------------------------------------------------ the issuer's waits
    if (rank == 0) {
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && w.next(p, off, tile)) {
        ok = ptx::mbar_wait_warp(acc_empty(count & 1), ((count >> 1) & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns);
        for (int kc = w.k0; kc < w.k1; ++kc) {
          if (ok) ok = ptx::mbar_wait_warp(ready_bar(stage), phase, abort_flag, p.status, p.timeout_ns);
          if (ptx::named_bar_or(kWatchBar, 64, !ok)) break;  // the issuer leaves as well
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        ++count;
      }
    }
  } else if (warp >= 6 && warp < 10) {
    // ------------------------------------------------------------ weights to FP16
    // A thread takes a channel: 128 bytes of its row (16-byte piece c at
    // c ^ (row % 8)) become 64 TMEM columns of its lane.  The slot there is free
    // once the MMAs of kSlots stages ago have completed: they were committed to
    // that stage's empty barrier (with as many slots as stages, before this
    // stage's bytes were even loaded).
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16) + L::kACol;
    const uint32_t src0 = sbase + row * 128;
    int stage = 0, slot = 0, old = 0;  // old: the stage of kSlots ago
    uint32_t phase = 0, old_phase = 0;
    bool ok = true, wrapped = false;   // wrapped: the slots have been used before
    while (ok && w.next(p, off, tile)) {
      for (int kc = w.k0; kc < w.k1; ++kc) {
        ok = ptx::mbar_wait_warp(full_bar(stage), phase, abort_flag, p.status, p.timeout_ns);
        if (!ok) break;
        if (L::kSlots < kStages && wrapped) {
          ok = ptx::mbar_wait_warp(empty_bar(old), old_phase, abort_flag, p.status, p.timeout_ns);
          if (!ok) break;
        }
        ptx::tc_fence_after();
        const uint32_t src = src0 + stage * L::kStageBytes, dst = tq + slot * kACols;
        uint32_t o[64];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t v[4];
          ptx::ld_shared_v4(src + ((c ^ (row & 7)) << 4), v);
#pragma unroll
          for (int i = 0; i < 4; ++i) widen4(v[i], o[8 * c + 2 * i], o[8 * c + 2 * i + 1]);
        }
        ptx::tmem_st_32x32b_x64(dst, o);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_issuer(ready_bar(stage));
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
        if (wrapped && ++old == kStages) { old = 0; old_phase ^= 1u; }
        if (++slot == L::kSlots) { slot = 0; wrapped = true; }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2-5; 256 tokens: 10-13 too)
    // Warp q has TMEM lanes 32 q .. 32 q + 31: a lane is a channel, a column a token.
    const int quarter = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int kCols = 32;  // columns of a read
    int count = 0;
    while (w.next(p, off, tile)) {
      const int buf = L::kBufs == 2 ? count & 1 : 0;
      const uint32_t round = L::kBufs == 2 ? (uint32_t)(count >> 1) : (uint32_t)count;
      const int chan = w.chan0 + rank * kChan + quarter * 32 + lane;
      const bool in = chan < p.N;
      const float sw = in ? p.sw[(int64_t)w.e * p.N + chan] : 0.0f;
      // 256 tokens: of a quarter's two warps each takes every second 32 columns
      const int half = warp >= 10;
      float* sa_tile = reinterpret_cast<float*>(smem + L::kSaOff) + (2 * quarter + half) * (kTok / 2);
      if constexpr (!L::kCut) {  // the warp's copy of the token scales
        __syncwarp();
        for (int i = 32 * half + lane; i < kTok; i += 64) sa_tile[(i >> 6) * 32 + lane] = i < w.n ? p.sa[w.tok0 + i] : 0.0f;
        __syncwarp();
      }
      if (!ptx::mbar_wait_warp(acc_full(buf), round & 1u, abort_flag, p.status, p.timeout_ns)) break;
      ptx::tc_fence_after();
      ++count;
      const uint32_t d = tq + buf * kTok;
      if constexpr (!L::kCut) {
        // BF16: the warp's values as 64 pairs of tokens in registers, the
        // accumulator handed back, then the stores, while the next tile's MMAs run.
        auto release = [&]() {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_issuer(acc_empty(buf));
        };
        auto scaled = [&](int c, float* v) {  // the warp's c-th 32 columns
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(d + 64 * c + 32 * half, reinterpret_cast<uint32_t*>(v));
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 s = *reinterpret_cast<const float4*>(sa_tile + 32 * c + i);
            v[i] = v[i] * sw * s.x;
            v[i + 1] = v[i + 1] * sw * s.y;
            v[i + 2] = v[i + 2] * sw * s.z;
            v[i + 3] = v[i + 3] * sw * s.w;
          }
        };
        if (p.out_f32) {
          float* dst = static_cast<float*>(p.out) + (int64_t)w.tok0 * p.ld_out + chan;
          if (32 * half >= w.n) release();  // nothing for this warp
          for (int c = 0; 64 * c + 32 * half < w.n; ++c) {
            const int at = 64 * c + 32 * half;
            float v[32];
            scaled(c, v);
            if (at + 64 >= w.n) release();
#pragma unroll
            for (int i = 0; i < 32; ++i) ptx::st_f32_if(in && at + i < w.n, dst + (at + i) * p.ld_out, v[i]);
          }
        } else {
          uint32_t pk[kTok / 4];
#pragma unroll
          for (int c = 0; c < kTok / 64; ++c) {
            if (64 * c + 32 * half < w.n) {
              float v[32];
              scaled(c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[16 * c + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            }
          }
          release();
          // lanes 2 l and 2 l + 1 exchange: the even one takes the first token's two
          // channels, the odd one the second's
          const int odd = lane & 1;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (int64_t)(w.tok0 + odd) * p.ld_out + (chan - odd);
#pragma unroll
          for (int c = 0; c < kTok / 64; ++c) {
            if (64 * c + 32 * half < w.n) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t mine = pk[16 * c + i], other = __shfl_xor_sync(kFull, mine, 1);
                const int at = 64 * c + 32 * half + 2 * i;
                ptx::st_u32_if(in && at + odd < w.n, dst + at * p.ld_out, __byte_perm(mine, other, odd ? 0x3276 : 0x5410));
              }
            }
          }
        }
        continue;
      }
      const bool whole = w.k0 == 0 && w.k1 == runs.per_unit;
      auto read = [&](int c0, float* v) {
        __syncwarp();
        ptx::tmem_ld_32x32b_x32(d + c0, reinterpret_cast<uint32_t*>(v));
        ptx::tmem_ld_wait();
        if (c0 + kCols >= w.n) {  // last read: hand the accumulator back
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_issuer(acc_empty(buf));
        }
      };
      int first = 0, last = -1;  // the pairs of a cut unit
      if (!whole) {
        float* mine = p.part + (int64_t)(2 * I8Runs::buffer(pair, w.k0 == 0) + rank) * kTok * kChan + quarter * 32 + lane;
        for (int c0 = 0; c0 < w.n; c0 += kCols) {
          float v[kCols];
          read(c0, v);
#pragma unroll
          for (int i = 0; i < kCols; ++i) ptx::st_cg_f32_if(c0 + i < w.n, mine + (c0 + i) * kChan, v[i]);
        }
        first = runs.first(w.unit);
        last = runs.last(w.unit);
        __threadfence();
        __syncwarp();
        uint32_t got = 0;
        if (lane == 0) got = atomicInc(p.sync + I8Runs::counter(first) + rank * 4 + quarter, (uint32_t)(last - first));
        got = __shfl_sync(kFull, got, 0);
        if (got != (uint32_t)(last - first)) continue;
        __threadfence();
      }
      for (int c0 = 0; c0 < w.n; c0 += kCols) {
        float v[kCols];
        if (whole) {
          read(c0, v);
        } else {
#pragma unroll
          for (int i = 0; i < kCols; ++i) v[i] = 0.0f;
          // in run order, the first pair's from the unit's start; two of them in flight
          for (int b = first; b <= last; b += 2) {
            const float* s0 = p.part + ((int64_t)(2 * I8Runs::buffer(b, b == first) + rank) * kTok + c0) * kChan + quarter * 32 + lane;
            const float* s1 = p.part + ((int64_t)(2 * I8Runs::buffer(b + 1, false) + rank) * kTok + c0) * kChan + quarter * 32 + lane;
            float a0[kCols], a1[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) a0[i] = c0 + i < w.n ? __ldcg(s0 + i * kChan) : 0.0f;
#pragma unroll
            for (int i = 0; i < kCols; ++i) a1[i] = b < last && c0 + i < w.n ? __ldcg(s1 + i * kChan) : 0.0f;
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = v[i] + a0[i] + a1[i];
          }
        }
        const float sa = c0 + lane < w.n ? p.sa[w.tok0 + c0 + lane] : 0.0f;
        if (p.out_f32) {
          float* dst = static_cast<float*>(p.out) + (int64_t)(w.tok0 + c0) * p.ld_out + chan;
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            const float r = v[i] * sw * __shfl_sync(kFull, sa, i);
            ptx::st_f32_if(in && c0 + i < w.n, dst + i * p.ld_out, r);
          }
        } else {
          // two tokens at a time: the even lane of a pair takes the first one's two
          // channels, the odd lane the second one's
          const bool odd = lane & 1;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (int64_t)(w.tok0 + c0 + odd) * p.ld_out + (chan - odd);
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            const float r0 = v[i] * sw * __shfl_sync(kFull, sa, i), r1 = v[i + 1] * sw * __shfl_sync(kFull, sa, i + 1);
            const float other = __shfl_xor_sync(kFull, odd ? r0 : r1, 1);
            const uint32_t o = odd ? pack_bf16(other, r1) : pack_bf16(r0, other);
            ptx::st_u32_if(in && c0 + i + odd < w.n, dst + i * p.ld_out, o);
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  // neither CTA of a pair leaves while the other's MMAs or arrivals may reach it
  ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_g<2>(tmem, kI8TmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct I8Form {
  const void* fn;
  int tok, smem, threads;
  bool cut;
};
template <int kTok>
I8Form form_of() {
  return {(const void*)int8_gemm_kernel<kTok>, kTok, I8Cfg<kTok>::kTotal, I8Cfg<kTok>::kThreads, I8Cfg<kTok>::kCut};
}
constexpr int kI8Forms = 4;
I8Form i8_form(int i) {
  switch (i) {
    case 0: return form_of<32>();
    case 1: return form_of<64>();
    case 2: return form_of<128>();
    default: return form_of<256>();
  }
}

// Rows of a tile of the few-rows form: 16 where they fit its share of shared memory,
// else 8; 0 where not even these do.  What shared memory takes is missing from L1,
// through which the weights' loads pass (one row, 8192 channels, tiles of 8: K = 16384,
// 149 KB, 31 us, 36 in the next form; 18432, 165 KB, 41 and 40; 22016, 193 KB, 73 and 45).
constexpr int64_t kFewSmem = 156 * 1024;
int few_tok(int64_t S, int64_t K) {
  for (int tok = S > 8 ? 16 : 8; tok >= 8; tok -= 8)
    if (tok * (int64_t)few_stride(K) + few_part_bytes(tok) <= kFewSmem) return tok;
  return 0;
}

// Microseconds that S rows over G experts take in a tensor-core form, as far as sizes
// tell: the stages of the longest run (I8Runs) and the epilogues of its units, with
// constants fitted to 150 shapes of 1 to 64 experts, where the form so chosen is 1.6 %
// slower than the best one in the geometric mean (8.8 % by the mean expert's rows
// alone: 150 rows, 1024 x 7168, 33.5 us in whole tiles of 256, 18.4 in cut ones of
// 64).  An expert of routed rows has half a short tile.
double i8_cost(int form, int64_t S, int G, int64_t N, int64_t K) {
  constexpr double kPairs = 76, kStage[3] = {0.434, 0.443, 0.482}, kUnit[3] = {0.92, 1.35, 2.03};
  const int tok = i8_form(form).tok;
  const double used = (double)std::max<int64_t>(1, std::min<int64_t>(S, G)), nk = (double)cdiv(K, kStageK);
  const double tiles = G == 1 ? (double)std::max<int64_t>(1, cdiv(S, tok)) : used * std::max(1.0, S / used / tok + 0.53);
  const double units = tiles * cdiv(N, 2 * kChan), rounds = std::max(1.0, std::ceil(units / kPairs - 0.02));
  if (form == 3) return 3.8 + rounds * (0.514 * nk + 2.56);
  const double c32 = std::max(1.0, std::ceil(S / tiles / 32)), run = std::max(units * nk / kPairs, (double)kI8MinStages);
  double stages = std::min(rounds * nk, run + (run >= 2 * nk ? 3 : 8 + 0.625 * c32 * (nk / run + 3)));
  if (2 * units <= kPairs && nk > 1) {
    const double parts = std::min({std::floor(kPairs / units), nk, std::max(2.0, std::round(std::sqrt(1.6 * nk / c32)))});
    stages = std::min(stages, nk / parts + 4 + 0.625 * c32 * parts);
  }
  return 7.2 + kStage[form] * stages + kUnit[form] * units / kPairs;
}

// Warps of a unit in the few-rows form: all, or fewer where that leaves a warp less than
// its loads in flight and there are units for every CTA all the same.
int few_split(int64_t S, int G, int64_t N, int64_t K, int num_sms) {
  const int64_t units = std::max<int64_t>(1, std::min<int64_t>(S, G)) * cdiv(N, kFewChan);
  int split = kFewWarps;
  while (split > 1 && cdiv(K, 128) < split * kFewDepth && units >= 2 * (int64_t)num_sms * (2 * kFewWarps / split)) split /= 2;
  return split;
}

// Microseconds in the few-rows form, in tiles of `tok` rows, as they compare with
// i8_cost: the iterations of the longest run of units, without the weights' stream,
// which is the same in all forms.  Rows fall to experts at random (Poisson); more than 8
// of a tile of 16 are widened and multiplied twice, and a run inside one expert's channels
// is as slow as that expert's.  A run that ends in another expert than it began (never
// where the SMs are a multiple of the tiles) starts its loads again.
double few_cost(int64_t S, int G, int64_t N, int64_t K, int tok) {
  constexpr int kSms = 152;
  double tiles = (double)cdiv(S, tok), over = S > 8, over_used = over;  // over: the share of experts with more than 8 rows
  if (G > 1) {
    const double mean = (double)S / G, none = std::exp(-mean);
    double p = none;
    tiles = over = 0;
    for (int i = 1; i < mean || p > 1e-7; ++i) {
      p *= mean / i;
      tiles += G * p * ((i + tok - 1) / tok);
      if (i > 8) over += p;
    }
    over_used = over / (1 - none);
  }
  const int split = few_split(S, G, N, K, kSms), at_once = kFewWarps / split;
  const int64_t turns = cdiv(cdiv(K, 128), split), slots = cdiv(turns, kFewDepth) * kFewDepth;
  const double chans = (double)cdiv(N, kFewChan), run = std::max(1.0, std::ceil(std::max(1.0, tiles) * chans / kSms - 0.02));
  double iters, two = over_used;
  if (tiles <= 1 && G == 1) {
    iters = std::ceil(run / at_once);
  } else if (run <= chans) {
    const bool ends_elsewhere = kSms % std::max<int64_t>(1, std::llround(tiles)) != 0;
    iters = std::max(1.0, run / at_once + 0.48 + (ends_elsewhere ? 0.75 : 0.0));
    if (G > 1) two = 1 - std::pow(1 - over, 0.42 * G);
  } else {
    iters = run / chans * std::ceil(chans / at_once);
  }
  if (tok == 8) two = 0;
  return 3.0 + iters * (at_once * (0.14 + 0.097 * two) + 0.11 * slots + (0.58 + 0.31 * two) * turns);
}

// The form for S rows over G experts: what takes the least time by these estimates, the
// few-rows form (-1) up to a mean of 16 rows for an expert that has some.  Of 2855
// products of 1 to 16 rows for each of 1 to 256 experts the form so chosen is 0.7 % slower
// than the faster of the two in the geometric mean, 65 of them by more than 10 % (with a
// limit of 8 to 16 rows for any size 3.6 %).  Both sides, this form and the next: 12
// rows, 4096 x 14336 (tiles of 8): 27.5 us, 22.9; 8 rows 20.1, 23.0; three experts of 12,
// 11008 x 2048: 28.9, 23.4, 2048 x 2048: 10.3, 12.6; 8 of 6, 4096 x 7168: 46, 55; 64 of 5,
// 1024 x 1024: 28.4, 23.0; 22 of 4, 96 x 2336: 6.4, 13.0.
constexpr int kFew = -1;
int i8_choose(int64_t S, int G, int64_t N, int64_t K) {
  thread_local int64_t of[4] = {};  // a call asks for its form several times
  thread_local int best = 0;
  if (of[0] != S || of[1] != G || of[2] != N || of[3] != K) {
    best = 0;
    double least = i8_cost(0, S, G, N, K);
    for (int i = 1; i < kI8Forms; ++i) {
      const double c = i8_cost(i, S, G, N, K);
      if (c < least) {
        least = c;
        best = i;
      }
    }
    const int64_t used = std::max<int64_t>(1, std::min<int64_t>(S, G));
    const int tok = K <= 0x7FFFFF && S <= 16 * used ? few_tok(S, K) : 0;
    if (tok > 0 && (S == 0 || few_cost(S, G, N, K, tok) < least)) best = kFew;
    of[0] = S;
    of[1] = G;
    of[2] = N;
    of[3] = K;
  }
  return best;
}

struct I8Ws {
  uint32_t* sync;
  float* part;
  uint8_t* wide;
  size_t total;
};
I8Ws i8_ws(int64_t S, int G, int64_t N, int64_t K, int codes, uint8_t* p) {
  const int form = i8_choose(S, G, N, K);
  I8Ws w{};
  w.total = 256;
  if (form == kFew) return w;  // needs none
  const I8Form f = i8_form(form);
  size_t o = 0;
  auto take = [&](int64_t n) {
    uint8_t* r = p + o;
    o += ((size_t)n + 255) & ~(size_t)255;
    return r;
  };
  if (f.cut) {
    w.sync = reinterpret_cast<uint32_t*>(take(kI8SyncWords * 4));
    w.part = reinterpret_cast<float*>(take((int64_t)2 * I8Runs::buffer(kI8MaxPairs, false) * f.tok * kChan * 4));
  }
  if (codes == MXG_CODES_INT8) w.wide = take(S * K * 2);
  w.total = std::max<size_t>(o, 256);
  return w;
}

constexpr int kI8MaxDevices = 64;
std::mutex g_i8_mu;

cudaLaunchAttribute pair_attr() {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = 2;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

// Per device and form, once: the dynamic shared-memory opt-in and the number of
// pairs that run together.  0 where none can.
int i8_pairs(int form, int dev) {
  static int pairs[kI8MaxDevices][kI8Forms] = {};
  std::lock_guard<std::mutex> lk(g_i8_mu);
  if (dev < 0 || dev >= kI8MaxDevices) return 0;
  int& n = pairs[dev][form];
  if (n == 0) {
    const I8Form f = i8_form(form);
    cudaLaunchAttribute attr = pair_attr();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3((unsigned)f.threads);
    cfg.dynamicSmemBytes = (size_t)f.smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, f.fn, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = std::min(n, kI8MaxPairs);
  }
  return n;
}

// K-major FP16 map with a 128-byte swizzle: 64 elements x `box_rows`.
bool make_f16_tmap(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld_bytes, int box_rows) {
  return make_tmap(m, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, cols, rows, ld_bytes, 64, box_rows);
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int64_t ld_x, const int32_t* rows, int64_t T, int k, int64_t cols,
                                 int codes, void* q, int64_t ld_q, float* scale, int32_t* status, cudaStream_t stream, int num_sms) {
  const int64_t pieces = cols / 8;
  // Pieces of a row that a thread takes: as many as it keeps (4096 x 4096 to 8192 rows:
  // 19.1 us, 22.6 with one), or one where there are few CTAs (173 x 1040: 2.5 us, 3.1).
  const int64_t each = T < 4 * num_sms ? 1 : kQKeep;
  const int threads = (int)std::min<int64_t>(kQThreads, ((pieces + each - 1) / each + 31) / 32 * 32);
  const auto fn = codes == MXG_CODES_F16 ? int8_quantize_kernel<true> : int8_quantize_kernel<false>;
  const dim3 grid((unsigned)T, (unsigned)std::max<int64_t>(1, std::min<int64_t>(k, 2 * num_sms / T)));
  return launch_overlapped(fn, grid, dim3((unsigned)threads), 0, stream, static_cast<const uint4*>(x), ld_x / 8, rows, k, T * k, pieces,
                           static_cast<uint8_t*>(q), ld_q, scale, status);
}

size_t int8_gemm_workspace_bytes(int64_t S, int G, int64_t N, int64_t K, int codes) {
  return i8_ws(S, G, N, K, codes, nullptr).total;
}
int int8_gemm_tile_tokens(int64_t S, int G, int64_t N, int64_t K) {
  const int form = i8_choose(S, G, N, K);
  return form == kFew ? few_tok(S, K) : i8_form(form).tok;
}

bool int8_gemm_sizes_fit(int64_t S, int G, int64_t N, int64_t K) {
  const int form = i8_choose(S, G, N, K);
  const int64_t tiles = S / (form == kFew ? 8 : i8_form(form).tok) + std::min<int64_t>(S, G);
  if (form == kFew) return tiles <= 0x7FFFFFFF / cdiv(N, kFewChan);
  return tiles * cdiv(N, 2 * kChan) <= (0x7FFFFFFF - 256) / cdiv(K, kStageK);  // (sums of them and the pairs are taken too)
}

namespace {
mxg_status launch_int8_few(const Int8GemmArgs& a, cudaStream_t stream, int num_sms, int dev) {
  {
    static bool ready[kI8MaxDevices] = {};
    std::lock_guard<std::mutex> lk(g_i8_mu);
    if (dev < 0 || dev >= kI8MaxDevices) return MXG_ERR_CUDA;
    if (!ready[dev] && cudaFuncSetAttribute(int8_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmem) != cudaSuccess) {
      cudaGetLastError();
      return MXG_ERR_CUDA;
    }
    ready[dev] = true;
  }
  FewParams p{};
  p.splits = a.splits;
  p.G = a.G; p.S = (int)a.S; p.N = (int)a.N; p.K = (int)a.K;
  p.tok = few_tok(a.S, a.K);
  p.per_tile = (int)cdiv(a.N, kFewChan);
  p.split = few_split(a.S, a.G, a.N, a.K, num_sms);
  p.a = a.a; p.ld_a = a.ld_a; p.f16 = a.codes == MXG_CODES_F16; p.sa = a.sa;
  p.w = a.w; p.ld_w = a.ld_w; p.sw = a.sw;
  p.out = a.out; p.ld_out = a.ld_out; p.out_f32 = a.out_dtype == MXG_OUT_F32;
  p.status = a.status;
  const size_t smem = (size_t)(p.tok * (int64_t)few_stride(a.K) + few_part_bytes(p.tok));
  // started while the kernel before ends (1 token's quantizer and product: 12.7 us, 13.3 without)
  if (launch_overlapped(int8_few_kernel, dim3((unsigned)num_sms), dim3(kFewThreads), smem, stream, p) != cudaSuccess) {
    cudaGetLastError();
    return MXG_ERR_CUDA;
  }
  return MXG_OK;
}
}  // namespace

mxg_status launch_int8_gemm(const Int8GemmArgs& a, cudaStream_t stream, int num_sms) {
  const int form = i8_choose(a.S, a.G, a.N, a.K);
  int dev = 0;
  cudaGetDevice(&dev);
  if (form == kFew) return launch_int8_few(a, stream, num_sms, dev);
  const I8Form f = i8_form(form);
  const int pairs = i8_pairs(form, dev);
  if (pairs == 0) return MXG_ERR_CUDA;
  const I8Ws ws = i8_ws(a.S, a.G, a.N, a.K, a.codes, static_cast<uint8_t*>(a.ws));
  const bool widen = a.codes == MXG_CODES_INT8 && a.S > 0;

  I8Params p{};
  p.splits = a.splits;
  static_cast<I8Order&>(p) = i8_order(a.G, a.N, a.K, f.tok);
  p.S = (int)a.S; p.N = (int)a.N;
  p.sa = a.sa; p.sw = a.sw;
  p.out = a.out; p.ld_out = a.ld_out; p.out_f32 = a.out_dtype == MXG_OUT_F32;
  p.part = ws.part; p.sync = ws.sync;
  p.status = a.status;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = std::max<uint64_t>(p.timeout_ns, 200000000ull);
  // instruction descriptor: FP16 operands, K-major, fp32 sums, M = 256 (N goes by the tile)
  p.idesc = (1u << 4) | ((2 * kChan >> 4) << 24);

  const bool prep = f.cut || widen;
  if (prep) {
    const int64_t per_row = a.K / 16, items = std::max<int64_t>(widen ? a.S * per_row : 0, kI8SyncWords);
    const unsigned grid = (unsigned)std::min<int64_t>((items + kPrepThreads - 1) / kPrepThreads, (int64_t)num_sms * 16);
    if (launch_overlapped(int8_prep_kernel, dim3(grid), dim3(kPrepThreads), 0, stream, ws.sync, f.cut ? kI8SyncWords : 0, a.a, a.ld_a,
                          widen ? a.S : 0, per_row, reinterpret_cast<uint4*>(ws.wide)) != cudaSuccess) {
      cudaGetLastError();
      return MXG_ERR_CUDA;
    }
  }
  CUtensorMap tmW, tmX;
  if (!make_tmap(&tmW, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.K, (int64_t)a.G * a.N, a.ld_w, kStageK, kChan)) return MXG_ERR_CUDA;
  // without rows there is nothing to load and the map only has to be well formed
  const bool ok = a.S == 0 ? make_f16_tmap(&tmX, a.w, 8, 1, 16, f.tok / 2)
                  : widen  ? make_f16_tmap(&tmX, ws.wide, a.K, a.S, a.K * 2, f.tok / 2)
                           : make_f16_tmap(&tmX, a.a, a.K, a.S, a.ld_a, f.tok / 2);
  if (!ok) return MXG_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {pair_attr()};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3((unsigned)f.threads);
  cfg.dynamicSmemBytes = (size_t)f.smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {(void*)&tmW, (void*)&tmX, (void*)&p};
  if (cudaLaunchKernelExC(&cfg, f.fn, args) != cudaSuccess) {
    cudaGetLastError();
    return MXG_ERR_CUDA;
  }
  return MXG_OK;
}

}  // namespace mxg
