// The expert layer of a few tokens (a decode step) over MX-quantized weights:
//
//   xq = MXFP8(x[t]);  g, u = W13[e] xq;  hq = MXFP8(g / (1 + exp(-g)) * u)
//   out[t] = sum_j weights[t, j] * (W2[e_j] hq_j),   e_j = ids[t, j]
//
// With a handful of tokens per expert the layer is a stream of the used
// experts' weights: 3 H I (1/2 or 1, + 1/32) bytes each, against which
// activations, partial sums and arithmetic are small.  Two kernels:
//
//   up    units of 128 channels: the 128 gate rows and the 128 up rows of one
//         expert, against its tokens; writes hq (MXFP8 codes and scales);
//   down  units of 256 output rows of one expert; writes weighted fp32 rows
//         per slot, and the warp that completes a token's last slot sums the
//         slots in order and writes the output.
//
// Weights are the M operand of the tensor core (128 rows = TMEM lanes), the
// expert's tokens the N operand (16 to 64 columns), so a few tokens fill the
// tile: block-scaled tcgen05.mma (kind::mxf8f6f4, E4M3 activations against
// E2M1 or E4M3 weights) needs no dequantization and no instruction issue per
// weight.  One CTA per SM, 320 threads:
//   warp 0     weight producer: TMA tiles (E2M1 unpacked to bytes on the way)
//              and their packed scale chunks into a 5-stage ring, 128
//              contraction elements a stage;
//   warp 1     TMEM owner and MMA issuer: scale copies to TMEM and 8 MMAs a stage;
//   warps 2-5  epilogue, one per TMEM lane quarter;
//   warps 6-9  activations: each thread takes 32-element blocks of a token,
//              rounds them to MXFP8 (up) or copies hq (down), and writes the
//              swizzled tile and the scale bytes.
// The stages of all units (row tile, expert, 64-token tile; in that order) are
// cut into one equal run per CTA, so every SM streams the same number of bytes
// whatever the routing.  A unit cut by a run boundary is joined through
// fp32 partials in global memory: the last of its CTAs to arrive (a counter
// that wraps to zero) adds them in run order, so results do not depend on
// timing.  Nothing waits for another CTA.  The down kernel is launched with
// programmatic stream serialization: each of its CTAs starts on its SM as soon
// as the up kernel's has left and streams W2 while the others finish; only its
// activation and epilogue warps wait for the up kernel's results.
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
constexpr int kMoeThreads = 320;
constexpr int kMoeStages = 5;
constexpr int kTok = 64;                  // tokens of one unit (TMEM columns of one accumulator)
constexpr int kWTile = 128 * 128;         // one weight tile in shared memory (a byte per element)
constexpr int kActTile = kTok * 128;
constexpr int kChunk = 512;               // 128 rows x 4 scale bytes
constexpr int kStageBytes = 2 * kWTile + kActTile;
constexpr int kStageSf = 3 * kChunk;      // two weight chunks, one activation chunk
constexpr int kMoeMaxSlots = 4096;
constexpr int kMaxCtas = 160;             // partial buffers are sized for this many CTAs
constexpr int kMoeTmemCols = 512;
constexpr int kSfCol = 256;               // two accumulator buffers of 2 x 64 columns, then the scale slots
constexpr int kSfSlot = 12;               // columns of one stage's scales
constexpr int kMinStages = 2;             // shortest run of a CTA

constexpr int kSfOff = kMoeStages * kStageBytes;
constexpr int kBarOff = kSfOff + kMoeStages * kStageSf;
constexpr int kNumBars = 3 * kMoeStages + 5;
constexpr int kMiscOff = kBarOff + kNumBars * 8;
constexpr int kOffOff = kMiscOff + 32;                       // int32 [E + 1]: first sorted slot of each expert
constexpr int kTileOff = kOffOff + (kMaxExperts + 4) * 4;    // int32 [E + 1]: first token tile of each expert
constexpr int kPosOff = kTileOff + (kMaxExperts + 4) * 4;    // uint16 [E]: running position of the sort
constexpr int kSortOff = kPosOff + kMaxExperts * 2;          // uint16 [slots]: slots by expert
constexpr int kMaskOff = kSortOff + kMoeMaxSlots * 2;        // bytes: each token's used slots, (k + 7) / 8 bytes
constexpr int kMoeSmem = kMaskOff + kMoeMaxSlots + 1024;     // + alignment slack
static_assert(kBarOff % 8 == 0 && kMiscOff % 16 == 0, "barriers and TMEM address are aligned");
static_assert(kMoeSmem <= 232448, "fits the 227 KB of dynamic shared memory of one CTA");
static_assert(kSfCol + kMoeStages * kSfSlot <= kMoeTmemCols, "the scale slots fit the TMEM allocation");

struct MoeParams {
  const uint16_t* x;
  int64_t ld_x;
  const int32_t* ids;
  const float* weights;
  int T, k, E, H, I;
  const uint8_t* ws;     // packed weight scales of this kernel's matrix
  uint8_t* hq;           // [slots, I] codes
  uint8_t* hs;           // [slots, I/32] scale bytes
  float* rows;           // [slots, H] weighted down rows
  uint32_t* tok_cnt;     // [row tiles][4][T] arrivals at a token's rows
  float* part;           // [2 * CTAs][part_tok][256] partial sums of cut units
  int part_tok;
  uint32_t* sync;        // [CTAs][4] arrivals at a cut unit
  void* out;
  int64_t ld_out;
  int out_f32;
  int32_t* status;
  uint64_t timeout_ns, drain_ns;
  uint32_t idesc;
};

// The contraction stages of all units cut into equal runs, one per CTA.
struct Runs {
  int64_t total;  // stages of all units
  int per_unit;   // stages of one unit
  int ctas;       // runs (every one has at least one stage)
  MXG_DEVINL int64_t start(int b) const { return (int64_t)b * total / ctas; }
  MXG_DEVINL int owner(int64_t s) const { return (int)(((s + 1) * ctas - 1) / total); }
};

// Walks the segments (the part of one unit inside a run) of this CTA's run.
struct Walker {
  int64_t s, end;
  // the current segment: unit, its stages [k0, k1), row tile, expert, tokens sorted[tok0 .. tok0 + n)
  int unit, k0, k1, rt, e, tok0, n;
  MXG_DEVINL bool next(const Runs& r, const int32_t* off, const int32_t* tile, int E) {
    if (s >= end) return false;
    unit = (int)(s / r.per_unit);
    k0 = (int)(s - (int64_t)unit * r.per_unit);
    k1 = (int)min((int64_t)r.per_unit, k0 + (end - s));
    s += k1 - k0;
    rt = unit / tile[E];
    const int ti = unit - rt * tile[E];
    e = find_prefix(tile, E, ti);  // the last expert that starts at or before ti: it has tiles
    tok0 = (ti - tile[e]) * kTok;
    n = min(kTok, off[e + 1] - off[e] - tok0);
    tok0 += off[e];
    return true;
  }
};

// FP32 magnitude bits -> MX exponent of E4M3 (floor(log2) - 8, at least -127).
MXG_DEVINL int mx_exponent_f32(uint32_t amax_bits) { return max((int)(amax_bits >> 23) - 127 - 8, -127); }

// Eight BF16 values scaled by `sinv` -> eight E4M3 codes.
MXG_DEVINL uint2 quantize8_e4m3(const uint4& w, float sinv) {
  uint2 o;
  o.x = cvt_e4m3x4(bf16lo_to_f32(w.x) * sinv, bf16hi_to_f32(w.x) * sinv, bf16lo_to_f32(w.y) * sinv,
                   bf16hi_to_f32(w.y) * sinv);
  o.y = cvt_e4m3x4(bf16lo_to_f32(w.z) * sinv, bf16hi_to_f32(w.z) * sinv, bf16lo_to_f32(w.w) * sinv,
                   bf16hi_to_f32(w.w) * sinv);
  return o;
}

// kDown: the down kernel (else up).  kFp4: E2M1 weights (else E4M3).
template <bool kDown, bool kFp4>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_kernel(const __grid_constant__ CUtensorMap tmW, const MoeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = p.T * p.k;

  const uint32_t bar0 = sbase + kBarOff;
  auto full_w = [&](int s) { return bar0 + 8u * s; };
  auto full_a = [&](int s) { return bar0 + 8u * (kMoeStages + s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * (2 * kMoeStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8u * (3 * kMoeStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8u * (3 * kMoeStages + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (3 * kMoeStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);
  int32_t* off = reinterpret_cast<int32_t*>(smem + kOffOff);
  int32_t* tile = reinterpret_cast<int32_t*>(smem + kTileOff);
  uint16_t* pos = reinterpret_cast<uint16_t*>(smem + kPosOff);
  uint16_t* sorted = reinterpret_cast<uint16_t*>(smem + kSortOff);
  uint8_t* mask = smem + kMaskOff;

  // ---------------------------------------------------------------- plan
  // Every CTA counts the slots of each expert (the ids are a few KB).
  for (int e = threadIdx.x; e < p.E; e += kMoeThreads) off[e] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMoeStages; ++s) {
      ptx::mbar_init(full_w(s), 1);
      ptx::mbar_init(full_a(s), 4);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(acc_full(b), 1);
      ptx::mbar_init(acc_empty(b), 4);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kMoeTmemCols);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  bool bad = false;
  const int mask_bytes = (p.k + 7) >> 3;
  for (int t = threadIdx.x; t < p.T; t += kMoeThreads) {
    for (int b = 0; b < mask_bytes; ++b) {
      uint32_t m = 0;
      for (int j = b * 8; j < min(p.k, b * 8 + 8); ++j) {
        const int e = __ldg(p.ids + t * p.k + j);
        bad |= e >= p.E;
        if (e >= 0 && e < p.E) {
          m |= 1u << (j & 7);
          atomicAdd(&off[e], 1);
        }
      }
      mask[t * mask_bytes + b] = (uint8_t)m;
    }
  }
  ptx::tc_fence_before();
  bad = __syncthreads_or(bad);
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (bad) {  // every CTA sees it: nothing is written
    if (threadIdx.x == 0) report(p.status, MXG_ERR_INDEX);
    if (warp == 1) ptx::tmem_dealloc(tmem, kMoeTmemCols);
    return;
  }
  if (warp == 0) {  // prefix sums: lane l has experts [l * per, l * per + per)
    const int per = (p.E + 31) >> 5;
    int c = 0, nt = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      const int v = e < p.E ? off[e] : 0;
      c += v;
      nt += (v + kTok - 1) / kTok;
    }
    int cs = c, ns = nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int oc = __shfl_up_sync(kFull, cs, d), on = __shfl_up_sync(kFull, ns, d);
      if (lane >= d) { cs += oc; ns += on; }
    }
    c = cs - c;
    nt = ns - nt;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < p.E) {
        const int v = off[e];
        off[e] = c;
        tile[e] = nt;
        pos[e] = (uint16_t)c;
        c += v;
        nt += (v + kTok - 1) / kTok;
      }
    }
    if (lane == 31) { off[p.E] = cs; tile[p.E] = ns; }
  }
  __syncthreads();
  if constexpr (!kDown) ptx::pdl_launch_dependents();

  const int row_tiles = kDown ? (p.H + 255) >> 8 : p.I >> 7;
  Runs runs;
  runs.per_unit = (kDown ? p.I : p.H) >> 7;
  runs.total = (int64_t)tile[p.E] * row_tiles * runs.per_unit;
  runs.ctas = (int)min((int64_t)gridDim.x, (runs.total + kMinStages - 1) / kMinStages);
  const int cta = blockIdx.x;
  const bool active = cta < runs.ctas;
  Walker w;
  w.s = active ? runs.start(cta) : 0;
  w.end = active ? runs.start(cta + 1) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      constexpr uint32_t kTileTx = kFp4 ? kWTile / 2 : kWTile;  // the unpacking load counts its source bytes
      const int64_t rt_all = kDown ? (int64_t)p.E * (p.H >> 7) : (int64_t)p.E * 2 * (p.I >> 7);
      while (ok && w.next(runs, off, tile, p.E)) {
        const int row0 = kDown ? w.e * p.H + w.rt * 256 : w.e * 2 * p.I + w.rt * 128;
        const int row1 = kDown ? row0 + 128 : row0 + p.I;
        const bool two = !kDown || w.rt * 256 + 128 < p.H;
        for (int kc = w.k0; kc < w.k1; ++kc) {
          if (!ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.timeout_ns)) { ok = false; break; }
          const uint32_t fb = full_w(stage);
          ptx::mbar_arrive_expect_tx(fb, (kTileTx + kChunk) * (two ? 2u : 1u));
          armed |= 1u << stage;
          armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          const uint32_t sw = sbase + stage * kStageBytes;
          const uint32_t sf = sbase + kSfOff + stage * kStageSf;
          const uint8_t* src = p.ws + (int64_t)kc * rt_all * kChunk;
          ptx::tma_load_2d(sw, &tmW, kc * 128, row0, fb);
          if (two) ptx::tma_load_2d(sw + kWTile, &tmW, kc * 128, row1, fb);
          ptx::bulk_load(sf, src + (int64_t)(row0 >> 7) * kChunk, kChunk, fb);
          if (two) ptx::bulk_load(sf + kChunk, src + (int64_t)(row1 >> 7) * kChunk, kChunk, fb);
          if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
        }
      }
      // do not leave copies in flight: wait (bounded) for every armed stage
      for (int s = 0; s < kMoeStages; ++s)
        if ((armed >> s) & 1u) {
          volatile int no_abort = 0;
          ptx::mbar_wait(full_w(s), (armed_phase >> s) & 1u, &no_abort, p.status, p.drain_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      while (ok && w.next(runs, off, tile, p.E)) {
        const int buf = count & 1;
        if (!ptx::mbar_wait(acc_empty(buf), ((count >> 1) & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns)) break;
        ptx::tc_fence_after();
        const uint32_t d0 = tmem + buf * 2 * kTok, d1 = d0 + kTok;
        const bool two = !kDown || w.rt * 256 + 128 < p.H;
        const uint32_t idesc_n = p.idesc | ((uint32_t)((w.n + 15) >> 4) << 18);  // N / 8, N a multiple of 16
        for (int kc = w.k0; kc < w.k1; ++kc) {
          if (!ptx::mbar_wait(full_w(stage), phase, abort_flag, p.status, p.timeout_ns) ||
              !ptx::mbar_wait(full_a(stage), phase, abort_flag, p.status, p.timeout_ns)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sw = sbase + stage * kStageBytes;
          const uint32_t sf = sbase + kSfOff + stage * kStageSf;
          const uint32_t tsf = tmem + kSfCol + stage * kSfSlot;
          ptx::tc_cp_32x128b_warpx4(tsf, ptx::smem_desc(sf, 0, 128, 0));
          if (two) ptx::tc_cp_32x128b_warpx4(tsf + 4, ptx::smem_desc(sf + kChunk, 0, 128, 0));
          ptx::tc_cp_32x128b_warpx4(tsf + 8, ptx::smem_desc(sf + 2 * kChunk, 0, 128, 0));
          const uint64_t a0 = ptx::smem_desc(sw, 16, 1024, 2), a1 = ptx::smem_desc(sw + kWTile, 16, 1024, 2);
          const uint64_t b = ptx::smem_desc(sw + 2 * kWTile, 16, 1024, 2);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // 32 contraction elements (32 bytes of each row) per MMA
            const uint32_t idesc = idesc_n | (j << 4) | (j << 29);
            const uint32_t acc = (kc != w.k0) || j != 0;
            ptx::mma_mxf8f6f4(d0, a0 + 2 * j, b + 2 * j, idesc, tsf, tsf + 8, acc);
            if (two) ptx::mma_mxf8f6f4(d1, a1 + 2 * j, b + 2 * j, idesc, tsf + 4, tsf + 8, acc);
          }
          issued = true;
          ptx::tc_commit(empty_bar(stage));
          if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        ptx::tc_commit(acc_full(buf));
        ++count;
      }
      if (issued) {  // every MMA has retired before TMEM is released
        ptx::tc_commit(drain_bar);
        volatile int no_abort = 0;
        ptx::mbar_wait(drain_bar, 0, &no_abort, p.status, p.drain_ns);
      }
    }
  } else {
    // the sorted slots are only needed by the activation and epilogue warps:
    // warp 6 sorts (stable, so slots of an expert stay in order) while the
    // first weights are on their way
    if (warp == 6) {
      for (int i0 = 0; i0 < P; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < P ? __ldg(p.ids + i) : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int at = e >= 0 ? pos[e] + rank : 0;
        __syncwarp();
        if (e >= 0) {
          sorted[at] = (uint16_t)i;
          if (rank == 0) pos[e] = (uint16_t)(at + __popc(same));
        }
        __syncwarp();
      }
    }
    ptx::named_bar_sync(1, kMoeThreads - 64);

    if (warp >= 6) {
      // ---------------------------------------------------------- activations
      // Item i of a stage: token i / 4 of the unit, 32-block i % 4; a thread
      // takes items tid and tid + 128.  Two stages of loads are in flight.
      if constexpr (kDown) ptx::pdl_wait();  // hq is complete
      const int tid = threadIdx.x - 6 * 32;
      const int blk = tid & 3;
      constexpr int kVec = kDown ? 2 : 4;  // 16-byte loads of a block
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && w.next(runs, off, tile, p.E)) {
        const uint4* src[2];
        const uint8_t* ssrc[2];
        bool on[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = (tid >> 2) + 32 * q;
          on[q] = i < w.n;
          const int slot = on[q] ? sorted[w.tok0 + i] : 0;
          if constexpr (kDown) {
            src[q] = reinterpret_cast<const uint4*>(p.hq + (int64_t)slot * p.I + blk * 32);
            ssrc[q] = p.hs + (int64_t)slot * (p.I >> 5) + blk;
          } else {
            src[q] = reinterpret_cast<const uint4*>(p.x + (int64_t)(slot / p.k) * p.ld_x + blk * 32);
            ssrc[q] = nullptr;
          }
        }
        uint4 buf[2][2][kVec];
        uint8_t sbuf[2][2];
        auto load = [&](int kc, uint4 (*v)[kVec], uint8_t* sv) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (on[q]) {
#pragma unroll
              for (int i = 0; i < kVec; ++i)
                v[q][i] = kDown ? __ldcg(src[q] + kc * 8 + i) : __ldg(src[q] + kc * 16 + i);
              if constexpr (kDown) sv[q] = __ldcg(ssrc[q] + kc * 4);
            }
        };
        auto store = [&](const uint4 (*v)[kVec], const uint8_t* sv) {
          const uint32_t st = stage * kStageBytes + 2 * kWTile;
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (on[q]) {
              const int i = (tid >> 2) + 32 * q;
              uint4 c0, c1;
              uint8_t sc;
              if constexpr (kDown) {
                c0 = v[q][0];
                c1 = v[q][1];
                sc = sv[q];
              } else {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  m = __vmaxu2(m, v[q][j].x & 0x7FFF7FFFu);
                  m = __vmaxu2(m, v[q][j].y & 0x7FFF7FFFu);
                  m = __vmaxu2(m, v[q][j].z & 0x7FFF7FFFu);
                  m = __vmaxu2(m, v[q][j].w & 0x7FFF7FFFu);
                }
                const int ex = mx_exponent_from_amax_bits(max(m & 0xFFFFu, m >> 16), 8);
                const float sinv = pow2_neg(ex);
                const uint2 r0 = quantize8_e4m3(v[q][0], sinv), r1 = quantize8_e4m3(v[q][1], sinv);
                const uint2 r2 = quantize8_e4m3(v[q][2], sinv), r3 = quantize8_e4m3(v[q][3], sinv);
                c0 = make_uint4(r0.x, r0.y, r1.x, r1.y);
                c1 = make_uint4(r2.x, r2.y, r3.x, r3.y);
                sc = (uint8_t)(ex + 127);
              }
              uint8_t* row = smem + st + i * 128;  // 16-byte chunk c of row i sits at c ^ (i % 8)
              *reinterpret_cast<uint4*>(row + ((2 * blk) ^ (i & 7)) * 16) = c0;
              *reinterpret_cast<uint4*>(row + ((2 * blk + 1) ^ (i & 7)) * 16) = c1;
              smem[kSfOff + stage * kStageSf + 2 * kChunk + (i & 31) * 16 + (i >> 5) * 4 + blk] = sc;
            }
        };
        load(w.k0, buf[0], sbuf[0]);
        if (w.k0 + 1 < w.k1) load(w.k0 + 1, buf[1], sbuf[1]);
        for (int kc = w.k0; ok && kc < w.k1; kc += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (kc + h < w.k1) {
              const bool free = ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.timeout_ns);
              if (!__all_sync(kFull, free)) { ok = false; break; }
              store(buf[h], sbuf[h]);
              if (kc + h + 2 < w.k1) load(kc + h + 2, buf[h], sbuf[h]);
              ptx::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(full_a(stage));
              if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
            }
          }
        }
      }
    } else {
      // ---------------------------------------------------------- epilogue (warps 2-5)
      // Warp q has TMEM lanes 32 q .. 32 q + 31: lane l is row 32 q + l of
      // either weight tile, a column is a token.  Each warp works alone.
      const int quarter = warp & 3;
      const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
      if constexpr (kDown) {
        ptx::pdl_wait();  // the counters and partial buffers are free, hq's writer is done
        // tokens without slots: zeros
        for (int t = cta; t < p.T; t += gridDim.x) {
          uint32_t any = 0;
          for (int b = 0; b < mask_bytes; ++b) any |= mask[t * mask_bytes + b];
          if (any == 0)
            for (int c = quarter * 32 + lane; c < p.H; c += 128) {
              if (p.out_f32) static_cast<float*>(p.out)[t * p.ld_out + c] = 0.0f;
              else static_cast<uint16_t*>(p.out)[t * p.ld_out + c] = 0;
            }
        }
      } else {
        // the down kernel's counters start at zero
        const int words = ((p.H + 255) >> 8) * 4 * p.T;
        for (int i = cta * 128 + quarter * 32 + lane; i < words; i += gridDim.x * 128) p.tok_cnt[i] = 0;
      }
      int count = 0;
      while (w.next(runs, off, tile, p.E)) {
        const int buf = count & 1;
        float wt_lo = 0.0f, wt_hi = 0.0f;  // down: lane l has the weights of tokens l and l + 32
        if constexpr (kDown) {
          if (lane < w.n) wt_lo = __ldg(p.weights + sorted[w.tok0 + lane]);
          if (lane + 32 < w.n) wt_hi = __ldg(p.weights + sorted[w.tok0 + lane + 32]);
        }
        const bool ready = ptx::mbar_wait(acc_full(buf), (count >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
        if (!__all_sync(kFull, ready)) break;
        ptx::tc_fence_after();
        ++count;
        const uint32_t d0 = tq + buf * 2 * kTok, d1 = d0 + kTok;
        const bool two = !kDown || w.rt * 256 + 128 < p.H;
        const int64_t u0 = (int64_t)w.unit * runs.per_unit;
        const bool whole = w.k0 == 0 && w.k1 == runs.per_unit;

        // 16 tokens' pairs of values (gate and up, or two output rows) of this
        // lane's row; computed for all 16 so that they interleave, stored for
        // the unit's tokens only
        auto finish = [&](int c0, const float* v0, const float* v1) {
          if constexpr (kDown) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c0 + i < w.n) {
                const float wt = __shfl_sync(kFull, c0 < 32 ? wt_lo : wt_hi, (c0 + i) & 31);
                const int slot = sorted[w.tok0 + c0 + i];
                float* dst = p.rows + (int64_t)slot * p.H + w.rt * 256 + quarter * 32 + lane;
                __stcg(dst, v0[i] * wt);
                if (two) __stcg(dst + 128, v1[i] * wt);
              }
            }
          } else {
            uint32_t code[16];
            int ex[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float h = v0[i] / (1.0f + expf(-v0[i])) * v1[i];
              // the block of 32 channels is this warp's 32 lanes
              ex[i] = mx_exponent_f32(__reduce_max_sync(kFull, __float_as_uint(h) & 0x7FFFFFFFu));
              code[i] = cvt_e4m3x4(h * pow2_neg(ex[i]), 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c0 + i < w.n) {
                const int slot = sorted[w.tok0 + c0 + i];
                p.hq[(int64_t)slot * p.I + w.rt * 128 + quarter * 32 + lane] = (uint8_t)code[i];
                if (lane == 0) p.hs[(int64_t)slot * (p.I >> 5) + w.rt * 4 + quarter] = (uint8_t)(ex[i] + 127);
              }
            }
          }
        };
        float* mine = p.part + (int64_t)(2 * cta + (w.k0 == 0)) * p.part_tok * 256 + quarter * 32 + lane;
        for (int c0 = 0; c0 < w.n; c0 += 16) {
          uint32_t r0[16], r1[16];
          __syncwarp();
          ptx::tmem_ld_32x32b_x16(d0 + c0, r0);
          ptx::tmem_ld_32x32b_x16(d1 + c0, r1);
          ptx::tmem_ld_wait();
          if (c0 + 16 >= w.n) {  // last read: hand the accumulator back
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(acc_empty(buf));
          }
          float v0[16], v1[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) { v0[i] = __uint_as_float(r0[i]); v1[i] = __uint_as_float(r1[i]); }
          if (whole) {
            finish(c0, v0, v1);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c0 + i < w.n) {
                __stcg(mine + (c0 + i) * 256, v0[i]);
                if (two) __stcg(mine + (c0 + i) * 256 + 128, v1[i]);
              }
          }
        }
        if (!whole) {
          // join: the last of the unit's CTAs adds the partials in run order
          const int first = runs.owner(u0), last = runs.owner(u0 + runs.per_unit - 1);
          __threadfence();
          __syncwarp();
          uint32_t got = 0;
          if (lane == 0) got = atomicInc(p.sync + (first + 1) * 4 + quarter, (uint32_t)(last - first));
          got = __shfl_sync(kFull, got, 0);
          if (got != (uint32_t)(last - first)) continue;
          __threadfence();
          const int64_t step = (int64_t)p.part_tok * 256;
          for (int c0 = 0; c0 < w.n; c0 += 16) {
            float v0[16], v1[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v0[i] = v1[i] = 0.0f;
            // buffers 2 first + 1, 2 (first + 1), 2 (first + 2), ...
            for (int b = first; b <= last; ++b) {
              const float* src = p.part + (2 * b + (b == first)) * step + c0 * 256 + quarter * 32 + lane;
              float a0[16], a1[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                a0[i] = c0 + i < w.n ? __ldcg(src + i * 256) : 0.0f;
                a1[i] = two && c0 + i < w.n ? __ldcg(src + i * 256 + 128) : 0.0f;
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) { v0[i] += a0[i]; v1[i] += a1[i]; }
            }
            finish(c0, v0, v1);
          }
        }
        if constexpr (kDown) {
          // this warp's rows of the unit's slots are in place; whoever brings
          // a token's last slot sums the token's slots
          __threadfence();
          __syncwarp();
          uint32_t* cnt = p.tok_cnt + (int64_t)(w.rt * 4 + quarter) * p.T;
#pragma unroll 1
          for (int c0 = 0; c0 < w.n; c0 += 32) {
            bool done = false;
            int t = 0;
            if (c0 + lane < w.n) {
              t = sorted[w.tok0 + c0 + lane] / p.k;
              int v = 0;
              for (int b = 0; b < mask_bytes; ++b) v += __popc((uint32_t)mask[t * mask_bytes + b]);
              done = atomicInc(cnt + t, (uint32_t)(v - 1)) == (uint32_t)(v - 1);
            }
            uint32_t todo = __ballot_sync(kFull, done);
            if (todo) __threadfence();
            // Four tokens at a time.  Lane 8 a + b reads rows 4 b .. 4 b + 3
            // (16 bytes) of slots a, a + 4, ...; the four partial sums are
            // then added across the lanes.
            const int a = lane >> 3;
            const int64_t r = w.rt * 256 + quarter * 32 + 4 * (lane & 7);
            while (todo) {
              int tt[4];
              float4 s0[4], s1[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                tt[q] = todo ? __shfl_sync(kFull, t, __ffs(todo) - 1) : -1;
                todo &= todo - 1;
                s0[q] = s1[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              }
              for (int j = a; j < ((p.k + 3) & ~3); j += 4) {
                float4 x0[4], x1[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  x0[q] = x1[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  if (tt[q] >= 0 && j < p.k && (mask[tt[q] * mask_bytes + (j >> 3)] >> (j & 7)) & 1) {
                    const float4* src = reinterpret_cast<const float4*>(p.rows + (int64_t)(tt[q] * p.k + j) * p.H + r);
                    x0[q] = __ldcg(src);
                    if (two) x1[q] = __ldcg(src + 32);
                  }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  s0[q].x += x0[q].x; s0[q].y += x0[q].y; s0[q].z += x0[q].z; s0[q].w += x0[q].w;
                  s1[q].x += x1[q].x; s1[q].y += x1[q].y; s1[q].z += x1[q].z; s1[q].w += x1[q].w;
                }
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float* f0 = &s0[q].x;
                float* f1 = &s1[q].x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  f0[i] += __shfl_xor_sync(kFull, f0[i], 8);
                  f0[i] += __shfl_xor_sync(kFull, f0[i], 16);
                  f1[i] += __shfl_xor_sync(kFull, f1[i], 8);
                  f1[i] += __shfl_xor_sync(kFull, f1[i], 16);
                }
                if (tt[q] >= 0 && a < (two ? 2 : 1)) {  // lanes 0-7 write the first tile's rows, 8-15 the second's
                  const float4 o = a == 0 ? s0[q] : s1[q];
                  const int64_t at = tt[q] * p.ld_out + r + 128 * a;
                  if (p.out_f32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
                  } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                  }
                }
              }
            }
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kMoeTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct MoeWs {
  uint8_t *hq, *hs;
  float* rows;
  uint32_t* tok_cnt;
  float* part;
  int part_tok;
  size_t total;
};

MoeWs moe_ws(int64_t T, int k, int64_t H, int64_t I, uint8_t* p) {
  const int64_t P = T * k;
  MoeWs w{};
  size_t o = 0;
  auto take = [&](int64_t n) {
    uint8_t* r = p + o;
    o += ((size_t)n + 255) & ~(size_t)255;
    return r;
  };
  w.hq = take(P * I);
  w.hs = take(P * (I / 32));
  w.rows = reinterpret_cast<float*>(take(P * H * 4));
  w.tok_cnt = reinterpret_cast<uint32_t*>(take((H + 255) / 256 * 4 * T * 4));
  w.part_tok = (int)std::min<int64_t>(kTok, P);
  w.part = reinterpret_cast<float*>(take((int64_t)2 * kMaxCtas * w.part_tok * 256 * 4));
  w.total = o;
  return w;
}

constexpr int kMoeMaxDevices = 64;
std::mutex g_moe_mu;

const void* moe_fn(bool down, bool fp4) {
  if (down) return fp4 ? (const void*)moe_kernel<true, true> : (const void*)moe_kernel<true, false>;
  return fp4 ? (const void*)moe_kernel<false, true> : (const void*)moe_kernel<false, false>;
}

// The dynamic shared-memory opt-in, once per device.
bool ensure_moe_attr(int dev) {
  static bool done[kMoeMaxDevices] = {};
  std::lock_guard<std::mutex> lk(g_moe_mu);
  if (dev >= 0 && dev < kMoeMaxDevices && done[dev]) return true;
  for (int i = 0; i < 4; ++i)
    if (cudaFuncSetAttribute(moe_fn(i & 1, i & 2), cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeSmem) !=
        cudaSuccess) {
      cudaGetLastError();
      return false;
    }
  if (dev >= 0 && dev < kMoeMaxDevices) done[dev] = true;
  return true;
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int k, int E, int64_t H, int64_t I) {
  (void)E;
  return moe_ws(T, k, H, I, nullptr).total;
}

mxg_status launch_moe_experts(const MoeArgs& a, cudaStream_t stream, int num_sms) {
  const bool fp4 = a.elem == MXG_E2M1;
  if ((int64_t)a.E * 2 * a.I > 0x7FFFFFFF || (int64_t)a.E * a.H > 0x7FFFFFFF) return MXG_ERR_SHAPE;
  const MoeWs ws = moe_ws(a.T, a.k, a.H, a.I, static_cast<uint8_t*>(a.ws));
  int dev = 0;
  cudaGetDevice(&dev);
  if (!ensure_moe_attr(dev)) return MXG_ERR_CUDA;

  MoeParams p{};
  p.x = a.x; p.ld_x = a.ld_x;
  p.ids = a.ids; p.weights = a.weights;
  p.T = a.T; p.k = a.k; p.E = a.E; p.H = a.H; p.I = a.I;
  p.hq = ws.hq; p.hs = ws.hs; p.rows = ws.rows; p.tok_cnt = ws.tok_cnt;
  p.part = ws.part; p.part_tok = ws.part_tok;
  p.sync = reinterpret_cast<uint32_t*>(a.sync);
  p.out = a.out; p.ld_out = a.ld_out; p.out_f32 = a.out_dtype == MXG_OUT_F32;
  p.status = a.status;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = std::max<uint64_t>(p.timeout_ns, 200000000ull);
  // instruction descriptor: weights (A) E2M1 or E4M3, activations (B) E4M3,
  // both K-major, UE8M0 scales, M = 128; N is added per unit
  p.idesc = ((fp4 ? 5u : 0u) << 7) | (1u << 23) | ((128u >> 4) << 24);

  const CUtensorMapDataType dt = fp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tm13, tm2;
  if (!make_tmap(&tm13, a.w13, dt, a.H, (int64_t)a.E * 2 * a.I, a.ld13, 128, 128) ||
      !make_tmap(&tm2, a.w2, dt, a.I, (int64_t)a.E * a.H, a.ld2, 128, 128))
    return MXG_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(num_sms, kMaxCtas));
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.stream = stream;
  p.ws = a.s13;
  {
    void* args[] = {(void*)&tm13, (void*)&p};
    if (cudaLaunchKernelExC(&cfg, moe_fn(false, fp4), args) != cudaSuccess) { cudaGetLastError(); return MXG_ERR_CUDA; }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  p.ws = a.s2;
  void* args[] = {(void*)&tm2, (void*)&p};
  if (cudaLaunchKernelExC(&cfg, moe_fn(true, fp4), args) != cudaSuccess) { cudaGetLastError(); return MXG_ERR_CUDA; }
  return MXG_OK;
}

}  // namespace mxg
