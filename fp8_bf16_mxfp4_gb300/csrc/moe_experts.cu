// The expert layer of a few tokens (a decode step) over MX-quantized weights:
//
//   xq = MXFP8(x[t]);  g, u = W13[e] xq;  hq = MXFP8(g / (1 + exp(-g)) * u)
//   out[t] = sum_j weights[t, j] * (W2[e_j] hq_j),   e_j = ids[t, j]
//
// With a handful of tokens per expert the layer is a stream of the used
// experts' weights: 3 H I (1/2 or 1, + 1/32) bytes each, against which
// activations, partial sums and arithmetic are small.  Four kernels:
//
//   quant x to MXFP8, once;
//   up    units of 128 channels: the 128 gate rows and the 128 up rows of one
//         expert, against its tokens; writes hq (MXFP8 codes and scales);
//   down  units of 256 output rows of one expert; writes a weighted fp32 row
//         per slot;
//   sum   adds each token's slots in order and rounds once.
//
// Weights are the M operand of the tensor core (128 rows = TMEM lanes), the
// expert's tokens the N operand (16 to 64 columns), so a few tokens fill the
// tile: block-scaled tcgen05.mma (kind::mxf8f6f4, E4M3 activations against
// E2M1 or E4M3 weights) needs no dequantization and no instruction per weight.
// One CTA per SM:
//   warp 0       weight producer: E4M3 tiles by TMA, E2M1 tiles prefetched into
//                L2 by TMA; packed scale chunks; 128 contraction elements a stage;
//   warp 1       TMEM owner and MMA issuer: scale copies to TMEM and 8 MMAs a stage;
//   warps 2-5    epilogue, one per TMEM lane quarter;
//   warps 6-9    activations: the unit's tokens' codes and scale bytes;
//   warps 10-13  E2M1 weights only: L2 to the tensor core's 4-bit layout.
// The stages of all units (row tile, expert, 64-token tile; in that order) are
// cut into one equal run per CTA, so every SM streams the same number of bytes
// whatever the routing.  A unit cut by a run boundary is joined through
// fp32 partials in global memory: the last of its CTAs to arrive (a counter
// that wraps to zero) adds them in run order, so results do not depend on
// timing; a run takes its cut units first, so that the joins hide behind the
// rest.  Nothing waits for another CTA.  All but the first kernel are launched
// with programmatic stream serialization: they plan and start to stream their
// weights while the kernel before still runs (a down CTA as soon as the up
// kernel's has left its SM), and only their activation and epilogue warps wait
// for its results.
//
// Bound: HBM with E4M3 weights (4 tokens, top 2 of 8 experts, 4096 x 14336: 137 us
// for 0.85 GB of weights, 4 to 5 experts used, 6.2 TB/s).  E2M1 tiles cannot use the TMA for
// the tensor core's layout at full rate (it moves a row of up to 128 bytes in
// 2.9 ns an SM, so 64-byte rows stop at 3.3 TB/s); 8-byte copies out of L2 bring
// them at about 20 bytes a clock an SM: 13 tokens, top 8 of 32 experts,
// 7168 x 2048: 133 us, 5.5 TB/s; 128 tokens 155 us, joins and epilogues growing
// with the tokens; 1 token 52 us for 0.19 GB, of which the four kernels' plans
// and tails are a third.  A small layer (33 tokens, top 3 of 12, 1152 x 640,
// 27 MB) takes 17 us, nearly all of it latency.
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
constexpr int kMoeThreads = 320;  // warps 0-9
constexpr int kUnpackThreads = 128;  // warps 10-13 (E2M1 weights)
constexpr int kTok = 64;                  // tokens of one unit (TMEM columns of one accumulator)
constexpr int kWTile = 128 * 128;         // one weight tile in shared memory (a byte per element)
constexpr int kActTile = kTok * 128;
constexpr int kChunk = 512;               // 128 rows x 4 scale bytes
constexpr int kStageBytes = 2 * kWTile + kActTile;
constexpr int kStageSf = 3 * kChunk;      // two weight chunks, one activation chunk
constexpr int kMoeMaxSlots = 4096;
constexpr int kMaxCtas = 160;             // partial buffers are sized for this many CTAs
constexpr int kSyncWords = 4 * kMaxCtas;  // join counters: [CTAs][4]
constexpr int kMoeTmemCols = 512;
constexpr int kSfCol = 256;               // two accumulator buffers of 2 x 64 columns, then the scale slots
constexpr int kSfSlot = 12;               // columns of one stage's scales
constexpr int kMinStages = 4;             // shortest run of cut units
constexpr int kPlanWarps = 8;             // warps 2-9 sort the slots

// Shared memory.  E2M1 stages hold half of their bytes' worth of weights (4-bit
// elements in 16-byte slots), and the 8-byte copies that fill them land through
// L1: with less than about 30 KB of it left they drop from 6.0 to 3.9 TB/s, so
// there are four stages instead of five.  E4M3 takes five: 4 tokens, 8 experts,
// 4096 x 14336: 136.5 us against 137.7 with four.
template <bool kFp4>
struct Lay {
  static constexpr int kStages = kFp4 ? 4 : 5;
  static constexpr int kSfOff = kStages * kStageBytes;
  static constexpr int kBarOff = kSfOff + kStages * kStageSf;
  static constexpr int kMiscOff = (kBarOff + (2 * kStages + 5) * 8 + 15) & ~15;
  static constexpr int kOffOff = kMiscOff + 32;                     // int32 [E + 1]: first sorted slot of each expert
  static constexpr int kTileOff = kOffOff + (kMaxExperts + 4) * 4;  // int32 [E + 1]: first token tile of each expert
  static constexpr int kSortOff = kTileOff + (kMaxExperts + 4) * 4; // uint16 [slots]: slots by expert
  static constexpr int kTotal = kSortOff + kMoeMaxSlots * 2 + 1024; // + alignment slack
  static_assert(kBarOff % 8 == 0, "barriers are aligned");
  static_assert(kTotal <= (kFp4 ? 195 : 227) * 1024, "fits, and leaves L1 for the E2M1 copies");
  static_assert(kSfCol + kStages * kSfSlot <= kMoeTmemCols, "the scale slots fit the TMEM allocation");
};
static_assert(kMoeMaxSlots * 2 <= kActTile && kPlanWarps * kMaxExperts * 2 <= kActTile,
              "the ids and the counts of the plan fit an activation tile each");

struct MoeParams {
  const uint16_t* x;
  int64_t ld_x;
  const int32_t* ids;
  const float* weights;
  int T, k, E, H, I;
  const uint8_t* ws;     // packed weight scales of this kernel's matrix
  uint8_t* xq;           // [T, H] codes of x
  uint8_t* xs;           // [T, H/32] scale bytes
  uint8_t* hq;           // [slots, I] codes
  uint8_t* hs;           // [slots, I/32] scale bytes
  float* rows;           // [slots, H] weighted down rows
  int32_t* bad;          // set when an id is out of range
  float* part;           // [2 * CTAs][part_tok][256] partial sums of cut units
  int part_tok;
  uint32_t* sync;        // [CTAs][4] arrivals at a cut unit
  void* out;
  int64_t ld_out;
  int32_t* status;
  uint64_t timeout_ns, drain_ns;
  uint32_t idesc;
  const uint8_t* w;      // this kernel's weight codes (E2M1: read by warps 10-13)
  int64_t ld_w;
};

// The contraction stages of all units cut into equal runs (to one grain), one per CTA.
struct Runs {
  int per_unit;   // stages of one unit
  int grain;      // runs start at multiples of this many stages
  int ctas;       // runs (every one has at least one grain)
  int q, r;       // grains of a run: q + 1 for the first r runs, q for the others
  MXG_DEVINL Runs(int units, int per_unit_, int tokens, int max_ctas) : per_unit(per_unit_) {
    // whole units to every CTA, or units cut into equal runs: what ends sooner
    const int total = units * per_unit;
    const int whole = (units + max_ctas - 1) / max_ctas * per_unit;
    // A join takes as long as about 12 + tokens / 2 stages, mostly hidden where
    // the run has whole units to follow.  32 experts, top 8, 7168 x 2048, E2M1:
    // 13 tokens 130 us cut, 141 whole; 1 token 53 cut, 50 whole; 33 tokens of
    // 12 experts, top 3, 1152 x 640, E4M3: 23 cut, 16 whole.
    const int run = max((total + max_ctas - 1) / max_ctas, kMinStages);
    const int cut = run + (run >= 2 * per_unit ? 4 : 12 + tokens / 2);
    grain = whole <= cut ? per_unit : 1;
    ctas = min(max_ctas, grain > 1 || per_unit == 1 ? units : (total + kMinStages - 1) / kMinStages);
    q = ctas > 0 ? total / grain / ctas : 0;
    r = ctas > 0 ? total / grain - q * ctas : 0;
  }
  MXG_DEVINL int start(int b) const { return (b * q + min(b, r)) * grain; }
  MXG_DEVINL int owner(int s) const {
    const int g = s / grain;
    return g < r * (q + 1) ? g / (q + 1) : r + (g - r * (q + 1)) / q;
  }
};

// Walks the segments (the part of one unit inside a run) of this CTA's run:
// the cut unit at its start, the cut unit at its end, then the whole units.
struct Walker {
  int s, end;           // what is left of the run
  // the current segment: unit, its stages [k0, k1), row tile, expert, tokens sorted[tok0 .. tok0 + n)
  int unit, k0, k1, rt, e, tok0, n;
  MXG_DEVINL bool next(const Runs& r, const int32_t* off, const int32_t* tile, int E) {
    if (s >= end) return false;
    const int first = s / r.per_unit, last = end / r.per_unit;
    const int head = s - first * r.per_unit, tail = end - last * r.per_unit;
    if (head != 0 || first == last) {  // up to the unit's end, or the run's
      unit = first;
      k0 = head;
      k1 = first == last ? tail : r.per_unit;
      s += k1 - k0;
    } else if (tail != 0) {
      unit = last;
      k0 = 0;
      k1 = tail;
      end -= tail;
    } else {
      unit = first;
      k0 = 0;
      k1 = r.per_unit;
      s += k1;
    }
    rt = unit / tile[E];
    const int ti = unit - rt * tile[E];
    e = find_prefix(tile, E, ti);  // the last expert that starts at or before ti: it has tiles
    tok0 = (ti - tile[e]) * kTok;
    n = min(kTok, off[e + 1] - off[e] - tok0);
    tok0 += off[e];
    return true;
  }
};

// g / (1 + exp(-g)), by exp(-|g|): exp(-g) would pass the FP32 range below -88.7,
// where the quotient does not.  The divisor is in [1, 2], where the fast division
// is within 2 units; the result is rounded to 4 bits next.  A rounded division
// takes 33 tokens of a small layer (1152 x 640) from 16.9 to 18.0 us.
MXG_DEVINL float silu(float g) {
  const float e = expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * e : g, 1.0f + e);
}

// FP32 magnitude bits -> MX exponent of E4M3 (floor(log2) - 8, at least -127).
MXG_DEVINL int mx_exponent_f32(uint32_t amax_bits) { return max((int)(amax_bits >> 23) - 127 - 8, -127); }

__host__ __device__ constexpr int moe_threads(bool fp4) { return kMoeThreads + (fp4 ? kUnpackThreads : 0); }

// kDown: the down kernel (else up).  kFp4: E2M1 weights (else E4M3).
template <bool kDown, bool kFp4>
__global__ void __launch_bounds__(moe_threads(kFp4), 1)
    moe_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS, const MoeParams p) {
  using L = Lay<kFp4>;
  constexpr int kMoeStages = L::kStages;
  constexpr int kSfOff = L::kSfOff;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = p.T * p.k;
  constexpr int kThreads = moe_threads(kFp4);

  const uint32_t bar0 = sbase + L::kBarOff;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMoeStages + s); };
  auto acc_full = [&](int b) { return bar0 + 8u * (2 * kMoeStages + b); };
  auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kMoeStages + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kMoeStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int32_t* off = reinterpret_cast<int32_t*>(smem + L::kOffOff);
  int32_t* tile = reinterpret_cast<int32_t*>(smem + L::kTileOff);
  uint16_t* sorted = reinterpret_cast<uint16_t*>(smem + L::kSortOff);

  // ---------------------------------------------------------------- plan
  // Every CTA sorts the slots by expert (the ids are a few KB), stably: warps
  // 2-9 take a range of slots each and count its experts, the counts become
  // running positions, and the slots are placed.  Ids and counts live in two
  // activation tiles, which are first written after the sort.
  int16_t* eid = reinterpret_cast<int16_t*>(smem + 2 * kWTile);
  uint16_t* cnt = reinterpret_cast<uint16_t*>(smem + kStageBytes + 2 * kWTile);  // [8][E]
  const int plan_warp = warp - 2;
  const bool planner = plan_warp >= 0 && plan_warp < kPlanWarps;
  const int per_warp = (((P + kPlanWarps - 1) / kPlanWarps) + 31) & ~31;
  const int slot0 = min(P, plan_warp * per_warp), slot1 = min(P, slot0 + per_warp);
  int next_id = planner && slot0 + lane < slot1 ? __ldg(p.ids + slot0 + lane) : -1;  // on its way during the set-up
  for (int i = threadIdx.x; i < (kPlanWarps * p.E + 1) / 2; i += kThreads) reinterpret_cast<uint32_t*>(cnt)[i] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMoeStages; ++s) {
      ptx::mbar_init(full_bar(s), 1 + 128 + (kFp4 ? kUnpackThreads : 0));  // warp 0; the threads of warps 6-9, 10-13
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
    ptx::prefetch_tmap(&tmS);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kMoeTmemCols);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  bool bad = false;
  uint16_t* my_cnt = cnt + plan_warp * p.E;
  if (planner) {
    for (int i0 = slot0; i0 < slot1; i0 += 32) {
      const int i = i0 + lane;
      int e = next_id;
      next_id = i + 32 < slot1 ? __ldg(p.ids + i + 32) : -1;
      bad |= e >= p.E;
      if (e < 0 || e >= p.E) e = -1;
      if (i < slot1) eid[i] = (int16_t)e;
      const uint32_t same = __match_any_sync(kFull, e);
      if (e >= 0 && lane == __ffs(same) - 1) my_cnt[e] += (uint16_t)__popc(same);
      __syncwarp();
    }
  }
  ptx::tc_fence_before();
  bad = __syncthreads_or(bad);
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (!kDown) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.bad = bad;
  }
  ptx::pdl_launch_dependents();
  if (bad) {  // every CTA sees it: nothing is written
    if (threadIdx.x == 0) report(p.status, MXG_ERR_INDEX);
    ptx::pdl_wait();  // a kernel ends after the one before it: the sum kernel finds the flag in place
    if (warp == 1) ptx::tmem_dealloc(tmem, kMoeTmemCols);
    return;
  }
  if (warp == 0) {  // prefix sums: lane l has experts [l * per, l * per + per)
    const int per = (p.E + 31) >> 5;
    int c = 0, nt = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      int v = 0;
      if (e < p.E) {
#pragma unroll
        for (int q = 0; q < kPlanWarps; ++q) v += cnt[q * p.E + e];
        off[e] = v;
      }
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
        int at = c;
#pragma unroll
        for (int q = 0; q < kPlanWarps; ++q) {
          const int m = cnt[q * p.E + e];
          cnt[q * p.E + e] = (uint16_t)at;
          at += m;
        }
        c += v;
        nt += (v + kTok - 1) / kTok;
      }
    }
    if (lane == 31) { off[p.E] = cs; tile[p.E] = ns; }
  }
  __syncthreads();

  const int row_tiles = kDown ? (p.H + 255) >> 8 : p.I >> 7;
  const Runs runs(tile[p.E] * row_tiles, (kDown ? p.I : p.H) >> 7, off[p.E] / max(tile[p.E], 1), gridDim.x);
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
      constexpr uint32_t kTileTx = kFp4 ? 0 : kWTile;  // E2M1 tiles come from warps 10-13
      const int64_t rt_all = kDown ? (int64_t)p.E * (p.H >> 7) : (int64_t)p.E * 2 * (p.I >> 7);
      // E2M1: the stages to come are fetched into L2 four at a time, 256 bytes
      // of every row, kAhead stages before they are asked for: a stage's ring
      // slots cover too little of the memory's latency.
      // The distance grows from the start, so that the first stages' own loads
      // do not queue behind the prefetches.  13 tokens of the sizes above: 136,
      // 133, 130 and 148 us at 2, 4, 6 and 12 stages.
      constexpr int kAhead = 6;
      Walker pw = w;
      int pk = 0, pk1 = 0, prow0 = 0, prow1 = 0, ahead = 0, issued = 0;
      bool ptwo = false, more = kFp4;
      auto fetch_ahead = [&]() {
        while (more && ahead < min(kAhead, issued)) {
          if (pk >= pk1) {
            more = pw.next(runs, off, tile, p.E);
            if (!more) return;
            pk = pw.k0;
            pk1 = pw.k1;
            prow0 = kDown ? pw.e * p.H + pw.rt * 256 : pw.e * 2 * p.I + pw.rt * 128;
            prow1 = kDown ? prow0 + 128 : prow0 + p.I;
            ptwo = !kDown || pw.rt * 256 + 128 < p.H;
          }
          ptx::tma_prefetch_2d(&tmW, pk * 64, prow0);
          ptx::tma_prefetch_3d(&tmS, 0, prow0 >> 7, pk);
          if (ptwo) {
            ptx::tma_prefetch_2d(&tmW, pk * 64, prow1);
            ptx::tma_prefetch_3d(&tmS, 0, prow1 >> 7, pk);
          }
          const int step = min(4, pk1 - pk);
          pk += step;
          ahead += step;
        }
      };
      while (ok && w.next(runs, off, tile, p.E)) {
        const int row0 = kDown ? w.e * p.H + w.rt * 256 : w.e * 2 * p.I + w.rt * 128;
        const int row1 = kDown ? row0 + 128 : row0 + p.I;
        const bool two = !kDown || w.rt * 256 + 128 < p.H;
        for (int kc = w.k0; kc < w.k1; ++kc) {
          if constexpr (kFp4) fetch_ahead();
          if (!ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.timeout_ns)) { ok = false; break; }
          --ahead;
          ++issued;
          const uint32_t fb = full_bar(stage);
          ptx::mbar_arrive_expect_tx(fb, (kTileTx + kChunk) * (two ? 2u : 1u));
          armed |= 1u << stage;
          armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          const uint32_t sw = sbase + stage * kStageBytes;
          const uint32_t sf = sbase + kSfOff + stage * kStageSf;
          const uint8_t* src = p.ws + (int64_t)kc * rt_all * kChunk;
          if constexpr (!kFp4) {
            ptx::tma_load_2d(sw, &tmW, kc * 128, row0, fb);
            if (two) ptx::tma_load_2d(sw + kWTile, &tmW, kc * 128, row1, fb);
          }
          ptx::bulk_load(sf, src + (int64_t)(row0 >> 7) * kChunk, kChunk, fb);
          if (two) ptx::bulk_load(sf + kChunk, src + (int64_t)(row1 >> 7) * kChunk, kChunk, fb);
          if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
        }
      }
      // do not leave copies in flight: wait (bounded) for every armed stage
      for (int s = 0; s < kMoeStages; ++s)
        if ((armed >> s) & 1u) {
          volatile int no_abort = 0;
          ptx::mbar_wait(full_bar(s), (armed_phase >> s) & 1u, &no_abort, p.status, p.drain_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop in step (each wait ends in a vote) and one
    // lane issues and hands the stages back.
    const uint32_t el = ptx::elect_one();
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    int stage = 0, count = 0;
    uint32_t phase = 0;
    bool ok = true, issued = false;
    while (ok && w.next(runs, off, tile, p.E)) {
      const int buf = count & 1;
      ok = ptx::mbar_wait_warp(acc_empty(buf), ((count >> 1) & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t d0 = tm + buf * 2 * kTok, d1 = d0 + kTok;
      for (int kc = w.k0; kc < w.k1; ++kc) {
        ok = ptx::mbar_wait_warp(full_bar(stage), phase, abort_flag, p.status, p.timeout_ns);
        if (!ok) break;
        // The stage's plain stores (released by the barrier's arrivals) come
        // before the MMAs' reads.  The fence is here and not at the writers,
        // where it would wait for their loads in flight (1000 clocks a stage).
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_after();
        const uint32_t sw = sbase + stage * kStageBytes;
        const uint32_t sf = sbase + kSfOff + stage * kStageSf;
        const uint32_t tsf = tm + kSfCol + stage * kSfSlot;
        ptx::tc_cp_32x128b_warpx4_if(el, tsf, ptx::smem_desc(sf, 0, 128, 0));
        ptx::tc_cp_32x128b_warpx4_if(el, tsf + 4, ptx::smem_desc(sf + kChunk, 0, 128, 0));
        ptx::tc_cp_32x128b_warpx4_if(el, tsf + 8, ptx::smem_desc(sf + 2 * kChunk, 0, 128, 0));
        // Always both tiles (the second of the last row tile may be stale, and
        // its rows are not stored) and the same N: a branch or an operand that
        // depends on the unit costs a third more per stage.
        const uint64_t a0 = ptx::smem_desc(sw, 16, 1024, 2), a1 = ptx::smem_desc(sw + kWTile, 16, 1024, 2);
        const uint64_t b = ptx::smem_desc(sw + 2 * kWTile, 16, 1024, 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 32 contraction elements (32 bytes of each row) per MMA
          const uint32_t idesc = p.idesc | (j << 4) | (j << 29);
          const uint32_t acc = (kc != w.k0) || j != 0;
          ptx::mma_mxf8f6f4_if(el, d0, a0 + 2 * j, b + 2 * j, idesc, tsf, tsf + 8, acc);
          ptx::mma_mxf8f6f4_if(el, d1, a1 + 2 * j, b + 2 * j, idesc, tsf + 4, tsf + 8, acc);
        }
        issued = true;
        ptx::tc_commit_if(el, empty_bar(stage));
        if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      ptx::tc_commit_if(el, acc_full(buf));
      ++count;
    }
    if (issued) {  // every MMA has retired before TMEM is released
      ptx::tc_commit_if(el, drain_bar);
      volatile int no_abort = 0;
      ptx::mbar_wait(drain_bar, 0, &no_abort, p.status, p.drain_ns);
    }
  } else if (kFp4 && warp >= 10) {
    // ------------------------------------------------------------ E2M1 weights
    // The tensor core takes 4-bit elements as 8 bytes of 16 elements in a
    // 16-byte slot.  A TMA load that unpacks to this moves a row in 2.9 ns
    // whatever its length, 3.3 TB/s over the device for rows of 64 bytes;
    // 8-byte asynchronous copies into the slots reach 6.1 TB/s.
    // A thread copies piece c of rows r, r + 16, ... of either tile.
    const int tid = threadIdx.x - kMoeThreads;
    const int c = tid & 7, r = tid >> 3;
    const uint32_t slot = r * 128 + ((c ^ (r & 7)) << 4);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && w.next(runs, off, tile, p.E)) {
      const int64_t row0 = kDown ? (int64_t)w.e * p.H + w.rt * 256 : (int64_t)w.e * 2 * p.I + w.rt * 128;
      const int64_t row1 = kDown ? row0 + 128 : row0 + p.I;
      const bool two = !kDown || w.rt * 256 + 128 < p.H;
      const uint8_t* src0 = p.w + (row0 + r) * p.ld_w + c * 8;
      const uint8_t* src1 = p.w + (row1 + r) * p.ld_w + c * 8;
      const int64_t step = 16 * p.ld_w;
      for (int kc = w.k0; kc < w.k1; ++kc) {
        ok = ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.timeout_ns);
        if (!ok) break;
        const uint32_t dst = sbase + stage * kStageBytes + slot;
#pragma unroll
        for (int i = 0; i < 8; ++i) ptx::cp_async_8(dst + i * 2048, src0 + kc * 64 + i * step);
        if (two) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ptx::cp_async_8(dst + kWTile + i * 2048, src1 + kc * 64 + i * step);
        }
        ptx::cp_async_arrive(full_bar(stage));
        if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
      }
    }
    ptx::cp_async_wait_all();
  } else {
    // the sorted slots are only needed by the activation and epilogue warps:
    // placed while the first weights are on their way
    for (int i0 = slot0; i0 < slot1; i0 += 32) {
      const int i = i0 + lane;
      const int e = i < slot1 ? eid[i] : -1;
      const uint32_t same = __match_any_sync(kFull, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int at = e >= 0 ? my_cnt[e] + rank : 0;
      __syncwarp();
      if (e >= 0) {
        sorted[at] = (uint16_t)i;
        if (rank == 0) my_cnt[e] = (uint16_t)(at + __popc(same));
      }
      __syncwarp();
    }
    ptx::named_bar_sync(1, kMoeThreads - 64);

    if (warp >= 6) {
      // ---------------------------------------------------------- activations
      // Codes and scale bytes go from global to shared memory asynchronously.
      // Item i of a stage is 32-block i % 4 of token i / 4; a thread takes items
      // tid and tid + 128, and the scale word of token tid.
      const int tid = threadIdx.x - 6 * 32;
      const int blk = tid & 3;
      const int width = kDown ? p.I : p.H;
      const uint8_t* codes = kDown ? p.hq : p.xq;
      const uint8_t* scales = kDown ? p.hs : p.xs;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      ptx::pdl_wait();  // the codes are complete
      while (ok && w.next(runs, off, tile, p.E)) {
        const uint8_t* src[2];
        const uint8_t* ssrc = nullptr;
        bool on[2];
        auto row_of = [&](int i) { return kDown ? (int)sorted[w.tok0 + i] : sorted[w.tok0 + i] / p.k; };
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = (tid >> 2) + 32 * q;
          on[q] = i < w.n;
          src[q] = codes + (int64_t)(on[q] ? row_of(i) : 0) * width + blk * 32;
        }
        if (tid < w.n) ssrc = scales + (int64_t)row_of(tid) * (width >> 5);
        for (int kc = w.k0; kc < w.k1; ++kc) {
          ok = ptx::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status, p.timeout_ns);
          if (!ok) break;
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (on[q]) {
              const int i = (tid >> 2) + 32 * q;
              // 16-byte chunk c of row i sits at c ^ (i % 8)
              const uint32_t row = sbase + stage * kStageBytes + 2 * kWTile + i * 128;
              ptx::cp_async_16(row + ((2 * blk) ^ (i & 7)) * 16, src[q] + kc * 128);
              ptx::cp_async_16(row + ((2 * blk + 1) ^ (i & 7)) * 16, src[q] + kc * 128 + 16);
            }
          if (ssrc != nullptr)
            ptx::cp_async_4(sbase + kSfOff + stage * kStageSf + 2 * kChunk + (tid & 31) * 16 + (tid >> 5) * 4,
                            ssrc + kc * 4);
          ptx::cp_async_arrive(full_bar(stage));
          if (++stage == kMoeStages) { stage = 0; phase ^= 1u; }
        }
      }
      ptx::cp_async_wait_all();
    } else {
      // ---------------------------------------------------------- epilogue (warps 2-5)
      // Warp q has TMEM lanes 32 q .. 32 q + 31: lane l is row 32 q + l of
      // either weight tile, a column is a token.  Each warp works alone.
      const int quarter = warp & 3;
      const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
      ptx::pdl_wait();  // the kernel before is done with the counters and partial buffers
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
        const bool whole = w.k0 == 0 && w.k1 == runs.per_unit;
        auto read = [&](int c0, float* v0, float* v1) {  // 8 tokens' pairs of values of this lane's row
          __syncwarp();
          ptx::tmem_ld_32x32b_x8(d0 + c0, reinterpret_cast<uint32_t*>(v0));
          ptx::tmem_ld_32x32b_x8(d1 + c0, reinterpret_cast<uint32_t*>(v1));
          ptx::tmem_ld_wait();
          if (c0 + 8 >= w.n) {  // last read: hand the accumulator back
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(acc_empty(buf));
          }
        };
        int first = 0, last = -1;  // the CTAs of a cut unit
        if (!whole) {
          float* mine = p.part + (int64_t)(2 * cta + (w.k0 == 0)) * p.part_tok * 256 + quarter * 32 + lane;
          for (int c0 = 0; c0 < w.n; c0 += 8) {
            float v0[8], v1[8];
            read(c0, v0, v1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const bool in = c0 + i < w.n;
              ptx::st_cg_f32_if(in, mine + (c0 + i) * 256, v0[i]);
              ptx::st_cg_f32_if(in && two, mine + (c0 + i) * 256 + 128, v1[i]);
            }
          }
          first = runs.owner(w.unit * runs.per_unit);
          last = runs.owner(w.unit * runs.per_unit + runs.per_unit - 1);
          __threadfence();
          __syncwarp();
          uint32_t got = 0;
          if (lane == 0) got = atomicInc(p.sync + (first + 1) * 4 + quarter, (uint32_t)(last - first));
          got = __shfl_sync(kFull, got, 0);
          if (got != (uint32_t)(last - first)) continue;
          __threadfence();
        }
        // Eight tokens at a time (all eight are computed, so that they
        // interleave, and the unit's stored, under predicates: a branch for each
        // store took 1100 clocks for eight tokens).  The last CTA of a cut unit adds
        // the partials in run order: buffers 2 first + 1, 2 (first + 1), ...
        for (int c0 = 0; c0 < w.n; c0 += 8) {
          float v0[8], v1[8];
          int64_t slot[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) slot[i] = sorted[w.tok0 + min(c0 + i, w.n - 1)];
          if (whole) {
            read(c0, v0, v1);
          } else {
            constexpr int kSegs = 3;  // partials in flight
#pragma unroll
            for (int i = 0; i < 8; ++i) v0[i] = v1[i] = 0.0f;
            for (int b = first; b <= last; b += kSegs) {
              float a0[kSegs][8], a1[kSegs][8];
#pragma unroll
              for (int g = 0; g < kSegs; ++g) {
                const float* src = p.part + (int64_t)(2 * (b + g) + (b + g == first)) * p.part_tok * 256 + c0 * 256 +
                                   quarter * 32 + lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const bool in = b + g <= last && c0 + i < w.n;
                  a0[g][i] = in ? __ldcg(src + i * 256) : 0.0f;
                  a1[g][i] = in && two ? __ldcg(src + i * 256 + 128) : 0.0f;
                }
              }
#pragma unroll
              for (int g = 0; g < kSegs; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) { v0[i] += a0[g][i]; v1[i] += a1[g][i]; }
            }
          }
          if constexpr (kDown) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float wt = __shfl_sync(kFull, c0 < 32 ? wt_lo : wt_hi, (c0 + i) & 31);
              const bool in = c0 + i < w.n;
              float* dst = p.rows + slot[i] * p.H + w.rt * 256 + quarter * 32 + lane;
              ptx::st_cg_f32_if(in, dst, v0[i] * wt);
              ptx::st_cg_f32_if(in && two, dst + 128, v1[i] * wt);
            }
          } else {
            uint32_t code[8];
            int ex[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float h = silu(v0[i]) * v1[i];
              // the block of 32 channels is this warp's 32 lanes
              ex[i] = mx_exponent_f32(__reduce_max_sync(kFull, __float_as_uint(h) & 0x7FFFFFFFu));
              code[i] = cvt_e4m3x4(h * pow2_neg(ex[i]), 0.0f, 0.0f, 0.0f);
            }
            int my_ex = 0;  // lane i has the scale of token i
            int64_t my_slot = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              ptx::st_u8_if(c0 + i < w.n, p.hq + slot[i] * p.I + w.rt * 128 + quarter * 32 + lane, code[i]);
              my_ex = lane == i ? ex[i] : my_ex;
              my_slot = lane == i ? slot[i] : my_slot;
            }
            ptx::st_u8_if(lane < 8 && c0 + lane < w.n, p.hs + my_slot * (p.I >> 5) + w.rt * 4 + quarter, my_ex + 127);
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
// x rounded to MXFP8, a 32-element block per thread (the rule and bytes of the
// row-wise quantizer), and the counters of the joins zeroed.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 128;

// Eight BF16 values scaled by `sinv` -> eight E4M3 codes.
MXG_DEVINL uint2 quantize8_e4m3(const uint4& w, float sinv) {
  uint2 o;
  o.x = cvt_e4m3x4(bf16lo_to_f32(w.x) * sinv, bf16hi_to_f32(w.x) * sinv, bf16lo_to_f32(w.y) * sinv,
                   bf16hi_to_f32(w.y) * sinv);
  o.y = cvt_e4m3x4(bf16lo_to_f32(w.z) * sinv, bf16hi_to_f32(w.z) * sinv, bf16lo_to_f32(w.w) * sinv,
                   bf16hi_to_f32(w.w) * sinv);
  return o;
}

__global__ void __launch_bounds__(kQuantThreads) moe_quant_kernel(const MoeParams p) {
  ptx::pdl_launch_dependents();
  const int i = blockIdx.x * kQuantThreads + threadIdx.x;
  if (i < kSyncWords) p.sync[i] = 0;
  const int nb = p.H >> 5;
  if (i >= p.T * nb) return;
  const int t = i / nb, b = i - t * nb;
  const uint4* src = reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.ld_x + b * 32);
  uint4 v[4];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = __ldg(src + j);
    m = __vmaxu2(m, v[j].x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v[j].y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v[j].z & 0x7FFF7FFFu);
    m = __vmaxu2(m, v[j].w & 0x7FFF7FFFu);
  }
  const int ex = mx_exponent_from_amax_bits(max(m & 0xFFFFu, m >> 16), 8);
  const float sinv = pow2_neg(ex);
  const uint2 r0 = quantize8_e4m3(v[0], sinv), r1 = quantize8_e4m3(v[1], sinv);
  const uint2 r2 = quantize8_e4m3(v[2], sinv), r3 = quantize8_e4m3(v[3], sinv);
  uint4* dst = reinterpret_cast<uint4*>(p.xq + (int64_t)i * 32);
  dst[0] = make_uint4(r0.x, r0.y, r1.x, r1.y);
  dst[1] = make_uint4(r2.x, r2.y, r3.x, r3.y);
  p.xs[i] = (uint8_t)(ex + 127);
}

// ---------------------------------------------------------------------------
// Sum of each token's slots, in order; a token without slots gives zeros.
// A thread takes four columns of a token; eight slots' rows are in flight.
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 128;

template <typename TOut>
__global__ void __launch_bounds__(kSumThreads) moe_sum_kernel(const MoeParams p) {
  const int t = blockIdx.x;
  const int c = (blockIdx.y * kSumThreads + threadIdx.x) * 4;
  ptx::pdl_wait();
  if (c >= p.H || *p.bad) return;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t slot = (int64_t)t * p.k + j0 + j;
      v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (j0 + j < p.k && __ldg(p.ids + slot) >= 0) v[j] = __ldcg(reinterpret_cast<const float4*>(p.rows + slot * p.H + c));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) { s.x += v[j].x; s.y += v[j].y; s.z += v[j].z; s.w += v[j].w; }
  }
  TOut* o = static_cast<TOut*>(p.out) + t * p.ld_out + c;
  if constexpr (sizeof(TOut) == 4) {
    *reinterpret_cast<float4*>(o) = s;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2*>(o) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// 2-D byte map without swizzle.
bool make_plain_tmap(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t ld, int box_inner, int box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MoeWs {
  uint8_t *xq, *xs, *hq, *hs;
  uint32_t* sync;
  float* rows;
  int32_t* bad;
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
  w.sync = reinterpret_cast<uint32_t*>(take(kSyncWords * 4));
  w.xq = take(T * H);
  w.xs = take(T * (H / 32));
  w.hq = take(P * I);
  w.hs = take(P * (I / 32));
  w.rows = reinterpret_cast<float*>(take(P * H * 4));
  w.bad = reinterpret_cast<int32_t*>(take(4));
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
    if (cudaFuncSetAttribute(moe_fn(i & 1, i & 2), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             i & 2 ? Lay<true>::kTotal : Lay<false>::kTotal) !=
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
  p.xq = ws.xq; p.xs = ws.xs; p.hq = ws.hq; p.hs = ws.hs; p.sync = ws.sync; p.rows = ws.rows; p.bad = ws.bad;
  p.part = ws.part; p.part_tok = ws.part_tok;
  p.out = a.out; p.ld_out = a.ld_out;
  p.status = a.status;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = std::max<uint64_t>(p.timeout_ns, 200000000ull);
  // instruction descriptor: weights (A) E2M1 or E4M3, activations (B) E4M3,
  // both K-major, UE8M0 scales, M = 128, N for the most tokens of a unit
  p.idesc = ((fp4 ? 5u : 0u) << 7) | ((uint32_t)((ws.part_tok + 15) / 16) << 18) | (1u << 23) | ((128u >> 4) << 24);

  CUtensorMap tmW[2], tmS[2];  // E4M3: the stages' tiles; E2M1: 256 bytes of 128 rows for the L2 prefetch
  for (int i = 0; i < 2; ++i) {
    const uint8_t* w = i ? a.w2 : a.w13;
    const int64_t rows = i ? (int64_t)a.E * a.H : (int64_t)a.E * 2 * a.I, cols = i ? a.I : a.H, ld = i ? a.ld2 : a.ld13;
    const bool ok = fp4 ? make_plain_tmap(&tmW[i], w, cols / 2, rows, ld, 256, 128)
                        : make_tmap(&tmW[i], w, CU_TENSOR_MAP_DATA_TYPE_UINT8, cols, rows, ld, 128, 128);
    if (!ok || !make_scale_tmap(&tmS[i], i ? a.s2 : a.s13, rows / 128, cols / 128, 1, 4)) return MXG_ERR_CUDA;
  }

  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = stream;
  cfg.attrs = attr;
  auto launch = [&](const void* fn, dim3 grid, int threads, int smem, void** args, bool overlap) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.numAttrs = overlap ? 1 : 0;
    if (cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
  };
  void* pargs[] = {(void*)&p};
  const int64_t blocks = std::max<int64_t>((int64_t)a.T * (a.H / 32), kSyncWords);
  if (!launch((const void*)moe_quant_kernel, dim3((unsigned)((blocks + kQuantThreads - 1) / kQuantThreads)),
              kQuantThreads, 0, pargs, false))
    return MXG_ERR_CUDA;
  for (int i = 0; i < 2; ++i) {
    p.ws = i ? a.s2 : a.s13;
    p.w = i ? a.w2 : a.w13;
    p.ld_w = i ? a.ld2 : a.ld13;
    void* args[] = {(void*)&tmW[i], (void*)&tmS[i], (void*)&p};
    if (!launch(moe_fn(i == 1, fp4), dim3((unsigned)std::min(num_sms, kMaxCtas)), moe_threads(fp4),
                fp4 ? Lay<true>::kTotal : Lay<false>::kTotal, args, true))
      return MXG_ERR_CUDA;
  }
  const void* sum = a.out_dtype == MXG_OUT_F32 ? (const void*)moe_sum_kernel<float>
                                               : (const void*)moe_sum_kernel<__nv_bfloat16>;
  if (!launch(sum, dim3((unsigned)a.T, (unsigned)((a.H / 4 + kSumThreads - 1) / kSumThreads)), kSumThreads, 0, pargs,
              true))
    return MXG_ERR_CUDA;
  return MXG_OK;
}

}  // namespace mxg
