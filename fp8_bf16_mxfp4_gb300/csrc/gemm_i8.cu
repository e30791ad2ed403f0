// Products of 8-bit integers with a scale per token and per channel, grouped over
// experts, and the quantizer in front of them:
//
//   quantize   a = max(max |x[t]|, 2^-100), s = a / 127, q = rint(x (127 / a))
//   product    y[i, n] = sa[i] sw[g N + n] sum_k qa[i, k] qw[g N + n, k],  g row i's expert
//
// sm_103a has no integer kind of tcgen05.mma, and its mma.sync runs at a small
// fraction of the tensor cores' rate.  Every integer up to 2048 is an FP16 value,
// so the products are taken by kind::f16: exact, with fp32 sums (exact up to 2^24).
// Weights stay 8-bit integers as far as the SM: they are the M operand, which the
// tensor core reads from TMEM, so a warp that turns a row's bytes into FP16 writes
// them where they are needed and shared memory never holds them twice as wide.
// Activations are the N operand, from shared memory, as FP16 (the quantizer writes
// them so, or a kernel in front widens them once).  One CTA per SM:
//   warp 0       producer: 128 channels x 128 bytes of weights and the tokens' 128
//                elements a stage, by TMA;
//   warp 1       TMEM owner and MMA issuer, 8 MMAs a stage;
//   warps 2-5    epilogue, one per TMEM lane quarter (a lane is a channel);
//   warps 6-13   weights to FP16, shared memory to TMEM: two groups of four warps
//                take turns at the stages.
// Two forms.  Few rows per expert: tiles of 16 to 128 tokens on single CTAs; the
// stages of all units (expert, channel tile, token tile) are cut into one equal run
// per CTA, so that every SM streams the same number of weight bytes, and cut units
// are joined through fp32 partials, added in run order by the last to arrive.
// Many rows: 256 channels x 256 tokens on CTA pairs (the 2-SM MMA), whole units.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
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
constexpr int kQThreads = 256;
constexpr int kQKeep = 4;  // 16-byte pieces of a row that a thread keeps between its two passes

// q = rint(x r) in the low 16 bits: the sum with 1.5 2^23 rounds the exact product
// to an integer, to nearest even, in one step.
MXG_DEVINL uint32_t round_code(float x, float r) { return __float_as_uint(fmaf(x, r, 12582912.0f)); }

template <bool kF16>
__global__ void __launch_bounds__(kQThreads) int8_quantize_kernel(const uint4* __restrict__ x, int64_t ld_x,
                                                                  const int32_t* __restrict__ rows, int k, int64_t out_rows,
                                                                  int64_t pieces, uint8_t* __restrict__ q, int64_t ld_q,
                                                                  float* __restrict__ scale, int32_t* status) {
  __shared__ uint32_t part[kQThreads / 32];
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
    keep[i] = c < pieces ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kQKeep; ++i) amax(keep[i]);
  for (int64_t c = threadIdx.x + (int64_t)kQKeep * blockDim.x; c < pieces; c += blockDim.x) amax(__ldg(src + c));
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
    const int32_t e = __ldg(rows + first + j);
    const int64_t at = e < 0 ? -1 - (int64_t)e : e;
    on = e >= 0;
    return at < out_rows ? at : -1;
  };
  for (int j = threadIdx.x; j < k; j += blockDim.x) {
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
    for (int j = 0; j < k; ++j) {
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
  for (int64_t c = threadIdx.x + (int64_t)kQKeep * blockDim.x; c < pieces; c += blockDim.x) emit(c, __ldg(src + c));
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
  const int64_t i0 = (int64_t)blockIdx.x * kPrepThreads + threadIdx.x;
  if (i0 < words) sync[i0] = 0;
  for (int64_t i = i0; i < S * per_row; i += (int64_t)gridDim.x * kPrepThreads) {
    const int64_t r = i / per_row, c = i - r * per_row;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(a + r * ld_a) + c);
    uint32_t o[8];
    widen4(v.x, o[0], o[1]);
    widen4(v.y, o[2], o[3]);
    widen4(v.z, o[4], o[5]);
    widen4(v.w, o[6], o[7]);
    wide[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    wide[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------
constexpr int kChan = 128;                 // channels of a CTA's tile (TMEM lanes)
constexpr int kStageK = 128;               // contraction elements of a stage
constexpr int kWBytes = kChan * kStageK;
constexpr int kI8TmemCols = 512;
constexpr int kACols = kStageK / 2;        // TMEM columns of a stage's weights (two FP16 a column)
constexpr int kI8MaxCtas = 160;            // partial buffers are sized for this many CTAs
constexpr int kI8SyncWords = 4 * kI8MaxCtas;
constexpr int kI8MinStages = 4;            // shortest run of cut units

// kCta: CTAs of a tile, kTok: its tokens.  Accumulators first (two of them, but
// for the pairs' 256 columns), then the ring of widened weights.
template <int kCta, int kTok>
struct I8Cfg {
  static constexpr int kBufs = kTok == 256 ? 1 : 2;
  // Groups of four widening warps.  A pair's stage lasts 1024 clocks, which one
  // group keeps up with, and its epilogue needs the registers.
  static constexpr int kGroups = kCta == 2 ? 1 : 2;
  static constexpr int kThreads = 32 * (6 + 4 * kGroups);
  static constexpr int kRows = kTok / kCta;            // tokens whose elements this CTA loads
  static constexpr int kXBox = kRows * 128;            // 64 elements of each
  static constexpr int kStageBytes = kWBytes + 2 * kXBox;
  static constexpr int kACol = kTok >= 128 ? 256 : (kTok >= 64 ? 128 : 64);
  // An even number: each group of widening warps then has its own stages and waits
  // for every round of them (a group that came to a stage every other round could
  // take the round before for its own).
  static constexpr int kStages = (kI8TmemCols - kACol) / kACols & ~1;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kBars = 3 * kStages + 5;
  static constexpr int kMiscOff = kBarOff + ((kBars * 8 + 15) & ~15);
  static constexpr int kOffOff = kMiscOff + 16;                      // int32 [G + 1]: first row of each expert
  static constexpr int kTileOff = kOffOff + (kMaxExperts + 4) * 4;   // int32 [G + 1]: first unit of each expert
  static constexpr int kSaOff = kTileOff + (kMaxExperts + 4) * 4;    // float [4][256]: the tile's token scales (pairs)
  static constexpr int kTotal = kSaOff + (kCta == 2 ? 4 * kTok * 4 : 0) + 1024;  // + alignment slack
  static_assert(kSaOff % 16 == 0, "token scales are read 16 bytes at a time");
  static_assert(kBufs * kTok <= kACol && kACol + kStages * kACols <= kI8TmemCols, "TMEM holds accumulators and ring");
  static_assert(kStageBytes % 1024 == 0 && kXBox % 1024 == 0, "tiles keep the swizzle-atom alignment");
  static_assert(kTotal <= 232448, "fits the 227 KB of one CTA");
};

struct I8Params {
  const int32_t* splits;  // null: one expert of all S rows
  int G, S, N, nk, n_chan;  // nk: stages of a unit; n_chan: channel tiles
  int group_t;            // token tiles per group of the unit order
  const float* sa;
  const float* sw;
  void* out;
  int64_t ld_out;
  int out_f32;
  float* part;            // [2 * CTAs][kTok][128] partial sums of cut units
  uint32_t* sync;         // [CTAs][4] arrivals at a cut unit
  int wide_from_prep;     // the activations come from the kernel before
  int32_t* status;
  uint64_t timeout_ns, drain_ns;
  uint32_t idesc;
};

// The stages of all units cut into equal runs (to one grain), one per CTA.
struct I8Runs {
  int per_unit, grain, ctas, q, r;
  MXG_DEVINL I8Runs(int units, int per_unit_, int tokens, int max_ctas) : per_unit(per_unit_) {
    // whole units to every CTA, or units cut into equal runs: what ends sooner,
    // a join taking as long as some 8 + tokens / 4 stages
    const int total = units * per_unit;
    const int whole = (units + max_ctas - 1) / max_ctas * per_unit;
    const int run = max((total + max_ctas - 1) / max_ctas, kI8MinStages);
    const int cut = run + (run >= 2 * per_unit ? 3 : 8 + tokens / 4);
    grain = whole <= cut ? per_unit : 1;
    ctas = min(max_ctas, grain > 1 || per_unit == 1 ? units : (total + kI8MinStages - 1) / kI8MinStages);
    q = ctas > 0 ? total / grain / ctas : 0;
    r = ctas > 0 ? total / grain - q * ctas : 0;
  }
  MXG_DEVINL int start(int b) const { return (b * q + min(b, r)) * grain; }
  MXG_DEVINL int owner(int s) const {
    const int g = s / grain;
    return g < r * (q + 1) ? g / (q + 1) : r + (g - r * (q + 1)) / q;
  }
};

// Walks a CTA's units: of a run, the cut unit at its start, the cut unit at its
// end, then the whole units; of a pair, every npairs-th unit.
template <int kCta, int kTok>
struct I8Walker {
  int s, end, per_unit;      // what is left of the run (pairs: the next unit, all units, the stride)
  int unit, k0, k1;          // the current unit and its stages [k0, k1)
  int e, tok0, n, chan0;     // expert, first row, rows, first channel of the tile
  MXG_DEVINL bool next(const I8Params& p, const int32_t* off, const int32_t* tile) {
    if (s >= end) return false;
    if constexpr (kCta == 2) {
      unit = s;
      s += per_unit;
      k0 = 0;
      k1 = p.nk;
    } else {
      const int first = s / per_unit, last = end / per_unit;
      const int head = s - first * per_unit, tail = end - last * per_unit;
      if (head != 0 || first == last) {  // up to the unit's end, or the run's
        unit = first;
        k0 = head;
        k1 = first == last ? tail : per_unit;
        s += k1 - k0;
      } else if (tail != 0) {
        unit = last;
        k0 = 0;
        k1 = tail;
        end -= tail;
      } else {
        unit = first;
        k0 = 0;
        k1 = per_unit;
        s += k1;
      }
    }
    e = find_prefix(tile, p.G, unit);
    int tt, ct;
    tile_mn(unit - tile[e], tile[e + 1] - tile[e], p.n_chan, p.group_t, tt, ct);
    const int rows = off[e + 1] - off[e];
    n = min(kTok, rows - tt * kTok);
    tok0 = off[e] + tt * kTok;
    chan0 = ct * kChan * kCta;
    return true;
  }
};

// Tokens that a pair's MMAs take: the tile's, to a multiple of 32 (half of them in
// each CTA).  The last tile of an expert is often short: 8192 rows of 8 experts,
// 4096 x 14336, take ZZ us with it and ZZ with 256 throughout.
MXG_DEVINL int pair_tokens(int n) { return (n + 31) & ~31; }

MXG_DEVINL uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A pair (kCta = 2, a cluster of two CTAs): the even CTA issues the MMAs of both
// (M = 256: its TMEM has channels 0-127 of the tile, the odd CTA's 128-255; each
// has half of the tokens' elements in shared memory).  The widening warps and the
// epilogues of both arrive on the even CTA's barriers, and every commit reaches
// the barriers of both.
template <int kCta, int kTok>
__global__ void __launch_bounds__(I8Cfg<kCta, kTok>::kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8Params p) {
  using L = I8Cfg<kCta, kTok>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCta == 2 ? (int)ptx::cluster_ctarank() : 0;

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
  auto arrive_issuer = [&](uint32_t bar) {
    if constexpr (kCta == 2) ptx::mbar_arrive_cluster(ptx::mapa_shared(bar, 0));
    else ptx::mbar_arrive(bar);
  };

  // ---------------------------------------------------------------- plan
  if (warp == 0) {  // rows and units of every expert: lane l has experts [l * per, l * per + per)
    const int per = (p.G + 31) >> 5;
    int64_t rows = 0, units = 0;
    bool neg = false;
    auto split = [&](int g) -> int64_t { return p.splits != nullptr ? (int64_t)__ldg(p.splits + g) : (int64_t)p.S; };
    auto units_of = [&](int64_t m) { return (m + kTok - 1) / kTok * p.n_chan; };
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      const int64_t m = g < p.G ? split(g) : 0;
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
    const bool bad = __any_sync(kFull, neg) || __shfl_sync(kFull, rs, 31) != p.S;
    rows = rs - rows;
    units = us - units;
    for (int i = 0; i < per && !bad; ++i) {
      const int g = lane * per + i;
      if (g < p.G) {
        off[g] = (int32_t)rows;
        tile[g] = (int32_t)units;
        const int64_t m = split(g);
        rows += m;
        units += units_of(m);
      }
    }
    if (lane == 31) {
      off[p.G] = (int32_t)rs;
      tile[p.G] = (int32_t)us;
    }
    if (lane == 0) {
      *bad_flag = bad;
      *abort_flag = 0;
    }
  } else if (warp == 1) {
    ptx::tmem_alloc_g<kCta>(ptx::smem_u32(tmem_slot), kI8TmemCols);
    ptx::tmem_relinquish_g<kCta>();
  } else if (threadIdx.x == 64) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
      ptx::mbar_init(ready_bar(s), 4 * kCta);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(acc_full(b), 1);
      ptx::mbar_init(acc_empty(b), 4 * kCta);
    }
    ptx::mbar_init(drain_bar, 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the peer's barriers are initialised before any remote arrival or commit reaches them
  if constexpr (kCta == 2) ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool bad = *bad_flag != 0;  // every CTA sees it: nothing is written
  if (bad && threadIdx.x == 0) report(p.status, MXG_ERR_SPLITS);

  const int units = bad ? 0 : tile[p.G];
  const int cta = blockIdx.x;
  const I8Runs runs(units, p.nk, units > 0 ? off[p.G] / (units / p.n_chan) : 0, gridDim.x);
  I8Walker<kCta, kTok> w;
  if constexpr (kCta == 2) {
    w.s = (int)ptx::cluster_id_x();
    w.end = units;
    w.per_unit = (int)ptx::nclusters_x();
  } else {
    const bool active = cta < runs.ctas;
    w.s = active ? runs.start(cta) : 0;
    w.end = active ? runs.start(cta + 1) : 0;
    w.per_unit = p.nk;
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      if (p.wide_from_prep) ptx::pdl_wait();  // the widened activations are complete
      while (ok && w.next(p, off, tile)) {
        const int row_w = w.e * p.N + w.chan0 + rank * kChan;
        const int row_x = w.tok0 + (kCta == 2 ? rank * pair_tokens(w.n) / 2 : 0);
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
    // lane issues and hands the stages back.
    if (rank == 0) {
      const uint32_t el = lane == 0;
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      while (ok && w.next(p, off, tile)) {
        const int buf = L::kBufs == 2 ? count & 1 : 0;
        const uint32_t round = L::kBufs == 2 ? (uint32_t)(count >> 1) : (uint32_t)count;
        ok = ptx::mbar_wait_warp(acc_empty(buf), (round & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = tm + buf * kTok;
        const uint32_t idesc = kCta == 2 ? p.idesc | ((uint32_t)(pair_tokens(w.n) >> 3) << 17) : p.idesc;
        for (int kc = w.k0; kc < w.k1; ++kc) {
          ok = ptx::mbar_wait_warp(ready_bar(stage), phase, abort_flag, p.status, p.timeout_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t a = tm + L::kACol + stage * kACols;
          const uint64_t b = ptx::smem_desc(sbase + stage * L::kStageBytes + kWBytes, 16, 1024, 2);
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 16 contraction elements: 8 columns, 32 bytes of each token's row
            ptx::mma_f16_ts_if<kCta>(el, d, a + 8 * j, b + (uint64_t)((j >> 2) * (L::kXBox >> 4) + 2 * (j & 3)), idesc,
                                     (kc != w.k0) || j != 0);
          issued = true;
          ptx::tc_commit_pair_if<kCta>(el, empty_bar(stage));
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        ptx::tc_commit_pair_if<kCta>(el, acc_full(buf));
        ++count;
      }
      if (issued) {  // every MMA has retired before TMEM is released
        if (lane == 0) ptx::tc_commit_g<kCta>(drain_bar);
        volatile int no_abort = 0;
        ptx::mbar_wait(drain_bar, 0, &no_abort, p.status, p.drain_ns);
      }
    }
  } else if (warp >= 6) {
    // ------------------------------------------------------------ weights to FP16
    // A thread takes a channel: 128 bytes of its row (16-byte piece c at
    // c ^ (row % 8)) become 64 TMEM columns of its lane.  The stage's slot in TMEM
    // is free: its bytes were loaded after the MMAs that read it had completed.
    const int group = (warp - 6) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16) + L::kACol;
    const uint32_t src0 = sbase + row * 128;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && w.next(p, off, tile)) {
      for (int kc = w.k0; kc < w.k1; ++kc) {
        if (L::kGroups == 1 || (stage & 1) == group) {
          ok = ptx::mbar_wait_warp(full_bar(stage), phase, abort_flag, p.status, p.timeout_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t src = src0 + stage * L::kStageBytes, dst = tq + stage * kACols;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t v[4];
              ptx::ld_shared_v4(src + (((4 * h + c) ^ (row & 7)) << 4), v);
#pragma unroll
              for (int i = 0; i < 4; ++i) widen4(v[i], o[8 * c + 2 * i], o[8 * c + 2 * i + 1]);
            }
            ptx::tmem_st_32x32b_x32(dst + 32 * h, o);
          }
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_issuer(ready_bar(stage));
        }
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2-5)
    // Warp q has TMEM lanes 32 q .. 32 q + 31: a lane is a channel, a column a token.
    const int quarter = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int kCols = kTok >= 32 ? 32 : 16;  // columns of a read
    int count = 0;
    if constexpr (kCta == 1) ptx::pdl_wait();  // the kernel before has zeroed the counters
    while (w.next(p, off, tile)) {
      const int buf = L::kBufs == 2 ? count & 1 : 0;
      const uint32_t round = L::kBufs == 2 ? (uint32_t)(count >> 1) : (uint32_t)count;
      const int chan = w.chan0 + rank * kChan + quarter * 32 + lane;
      const bool in = chan < p.N;
      const float sw = in ? __ldg(p.sw + (int64_t)w.e * p.N + chan) : 0.0f;
      float* sa_tile = reinterpret_cast<float*>(smem + L::kSaOff) + quarter * kTok;
      if constexpr (kCta == 2) {  // the warp's copy of the token scales
        __syncwarp();
        for (int i = lane; i < kTok; i += 32) sa_tile[i] = i < w.n ? __ldg(p.sa + w.tok0 + i) : 0.0f;
        __syncwarp();
      }
      if (!ptx::mbar_wait_warp(acc_full(buf), round & 1u, abort_flag, p.status, p.timeout_ns)) break;
      ptx::tc_fence_after();
      ++count;
      const uint32_t d = tq + buf * kTok;
      if constexpr (kCta == 2) {
        // BF16: the tile's values as 128 pairs of tokens in registers, the
        // accumulator handed back, then the stores, while the next tile's MMAs run.
        auto release = [&]() {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_issuer(acc_empty(buf));
        };
        auto scaled = [&](int c, float* v) {  // columns 32 c .. 32 c + 31
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(d + 32 * c, reinterpret_cast<uint32_t*>(v));
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
          for (int c = 0; 32 * c < w.n; ++c) {
            float v[32];
            scaled(c, v);
            if (32 * c + 32 >= w.n) release();
#pragma unroll
            for (int i = 0; i < 32; ++i) ptx::st_f32_if(in && 32 * c + i < w.n, dst + (32 * c + i) * p.ld_out, v[i]);
          }
        } else {
          uint32_t pk[kTok / 2];
#pragma unroll
          for (int c = 0; c < kTok / 32; ++c) {
            if (32 * c < w.n) {
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
          for (int c = 0; c < kTok / 32; ++c) {
            if (32 * c < w.n) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t mine = pk[16 * c + i], other = __shfl_xor_sync(kFull, mine, 1);
                const int at = 32 * c + 2 * i;
                ptx::st_u32_if(in && at + odd < w.n, dst + at * p.ld_out, __byte_perm(mine, other, odd ? 0x3276 : 0x5410));
              }
            }
          }
        }
        continue;
      }
      const bool whole = kCta == 2 || (w.k0 == 0 && w.k1 == runs.per_unit);
      auto read = [&](int c0, float* v) {
        __syncwarp();
        if constexpr (kCols == 32) {
          ptx::tmem_ld_32x32b_x32(d + c0, reinterpret_cast<uint32_t*>(v));
        } else {
          ptx::tmem_ld_32x32b_x8(d + c0, reinterpret_cast<uint32_t*>(v));
          ptx::tmem_ld_32x32b_x8(d + c0 + 8, reinterpret_cast<uint32_t*>(v) + 8);
        }
        ptx::tmem_ld_wait();
        if (c0 + kCols >= w.n) {  // last read: hand the accumulator back
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_issuer(acc_empty(buf));
        }
      };
      int first = 0, last = -1;  // the CTAs of a cut unit
      if (!whole) {
        float* mine = p.part + ((int64_t)(2 * cta + (w.k0 == 0)) * kTok) * kChan + quarter * 32 + lane;
        for (int c0 = 0; c0 < w.n; c0 += kCols) {
          float v[kCols];
          read(c0, v);
#pragma unroll
          for (int i = 0; i < kCols; ++i) ptx::st_cg_f32_if(c0 + i < w.n, mine + (c0 + i) * kChan, v[i]);
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
      for (int c0 = 0; c0 < w.n; c0 += kCols) {
        float v[kCols];
        if (whole) {
          read(c0, v);
        } else {
#pragma unroll
          for (int i = 0; i < kCols; ++i) v[i] = 0.0f;
          for (int b = first; b <= last; ++b) {  // in run order: buffers 2 first + 1, 2 (first + 1), ...
            const float* src = p.part + ((int64_t)(2 * b + (b == first)) * kTok + c0) * kChan + quarter * 32 + lane;
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] += c0 + i < w.n ? __ldcg(src + i * kChan) : 0.0f;
          }
        }
        const float sa = c0 + lane < w.n && lane < kCols ? __ldg(p.sa + w.tok0 + c0 + lane) : 0.0f;
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
  if constexpr (kCta == 2) ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_g<kCta>(tmem, kI8TmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct I8Form {
  const void* fn;
  int cta, tok, smem, threads;
};
template <int kCta, int kTok>
I8Form form_of() {
  return {(const void*)int8_gemm_kernel<kCta, kTok>, kCta, kTok, I8Cfg<kCta, kTok>::kTotal,
          I8Cfg<kCta, kTok>::kThreads};
}
constexpr int kI8Forms = 5;
I8Form i8_form(int i) {
  switch (i) {
    case 0: return form_of<1, 16>();
    case 1: return form_of<1, 32>();
    case 2: return form_of<1, 64>();
    case 3: return form_of<1, 128>();
    default: return form_of<2, 256>();
  }
}

// The form for S rows over G experts: tiles that hold half as many tokens again as
// the mean expert's, pairs from there on.
int i8_choose(int64_t S, int G, int64_t N, int64_t K) {
  (void)N;
  (void)K;
  const int64_t mean = S / std::max<int64_t>(1, std::min<int64_t>(S, G));
  for (int i = 0; i < 4; ++i)
    if (mean + mean / 2 <= i8_form(i).tok || (G == 1 && mean <= i8_form(i).tok)) return i;
  return 4;
}

struct I8Ws {
  uint32_t* sync;
  float* part;
  uint8_t* wide;
  size_t total;
};
I8Ws i8_ws(int64_t S, int G, int64_t N, int64_t K, int codes, uint8_t* p) {
  const I8Form f = i8_form(i8_choose(S, G, N, K));
  I8Ws w{};
  size_t o = 0;
  auto take = [&](int64_t n) {
    uint8_t* r = p + o;
    o += ((size_t)n + 255) & ~(size_t)255;
    return r;
  };
  if (f.cta == 1) {
    w.sync = reinterpret_cast<uint32_t*>(take(kI8SyncWords * 4));
    w.part = reinterpret_cast<float*>(take((int64_t)2 * kI8MaxCtas * f.tok * kChan * 4));
  }
  if (codes == MXG_CODES_INT8) w.wide = take(S * K * 2);
  w.total = std::max<size_t>(o, 256);
  return w;
}

constexpr int kI8MaxDevices = 64;
std::mutex g_i8_mu;

// Per device and form, once: the dynamic shared-memory opt-in and the number of
// pairs that can run together (0 where none can).
bool i8_ready(int form, int dev, int* pairs) {
  static bool done[kI8MaxDevices][kI8Forms] = {};
  static int clusters[kI8MaxDevices] = {};
  std::lock_guard<std::mutex> lk(g_i8_mu);
  if (dev < 0 || dev >= kI8MaxDevices) return false;
  const I8Form f = i8_form(form);
  if (!done[dev][form]) {
    if (cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    if (f.cta == 2) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2);
      cfg.blockDim = dim3((unsigned)f.threads);
      cfg.dynamicSmemBytes = (size_t)f.smem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&clusters[dev], f.fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return false;
      }
    }
    done[dev][form] = true;
  }
  *pairs = clusters[dev];
  return true;
}

// K-major FP16 map with a 128-byte swizzle: 64 elements x `box_rows`.
bool make_f16_tmap(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld_bytes, int box_rows) {
  return make_tmap(m, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, cols, rows, ld_bytes, 64, box_rows);
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int64_t ld_x, const int32_t* rows, int64_t T, int k, int64_t cols,
                                 int codes, void* q, int64_t ld_q, float* scale, int32_t* status, cudaStream_t stream) {
  const int64_t pieces = cols / 8;
  const int threads = (int)std::min<int64_t>(kQThreads, (pieces + 31) / 32 * 32);
  const auto fn = codes == MXG_CODES_F16 ? int8_quantize_kernel<true> : int8_quantize_kernel<false>;
  fn<<<(unsigned)T, threads, 0, stream>>>(static_cast<const uint4*>(x), ld_x / 8, rows, k, T * k, pieces,
                                          static_cast<uint8_t*>(q), ld_q, scale, status);
  return cudaGetLastError();
}

size_t int8_gemm_workspace_bytes(int64_t S, int G, int64_t N, int64_t K, int codes) {
  return i8_ws(S, G, N, K, codes, nullptr).total;
}
int int8_gemm_tile_tokens(int64_t S, int G, int64_t N, int64_t K) { return i8_form(i8_choose(S, G, N, K)).tok; }

bool int8_gemm_sizes_fit(int64_t S, int G, int64_t N, int64_t K) {
  const I8Form f = i8_form(i8_choose(S, G, N, K));
  const int64_t units = (S / f.tok + std::min<int64_t>(S, G)) * cdiv(N, (int64_t)kChan * f.cta);
  return units <= 0x7FFFFFFF / cdiv(K, kStageK);
}

mxg_status launch_int8_gemm(const Int8GemmArgs& a, cudaStream_t stream, int num_sms) {
  int form = i8_choose(a.S, a.G, a.N, a.K);
  const I8Form f = i8_form(form);
  int dev = 0, pairs = 0;
  cudaGetDevice(&dev);
  if (!i8_ready(form, dev, &pairs) || (f.cta == 2 && pairs == 0)) return MXG_ERR_CUDA;
  const I8Ws ws = i8_ws(a.S, a.G, a.N, a.K, a.codes, static_cast<uint8_t*>(a.ws));
  const bool widen = a.codes == MXG_CODES_INT8 && a.S > 0;

  I8Params p{};
  p.splits = a.splits;
  p.G = a.G; p.S = (int)a.S; p.N = (int)a.N;
  p.nk = (int)cdiv(a.K, kStageK);
  p.n_chan = (int)cdiv(a.N, (int64_t)kChan * f.cta);
  // token tiles whose activations (about 32 MiB) stay in L2 over all channel tiles
  p.group_t = (int)std::max<int64_t>(1, (int64_t(32) << 20) / (f.tok * a.K * 2));
  p.sa = a.sa; p.sw = a.sw;
  p.out = a.out; p.ld_out = a.ld_out; p.out_f32 = a.out_dtype == MXG_OUT_F32;
  p.part = ws.part; p.sync = ws.sync;
  p.wide_from_prep = widen;
  p.status = a.status;
  p.timeout_ns = wait_timeout_ns();
  p.drain_ns = std::max<uint64_t>(p.timeout_ns, 200000000ull);
  // instruction descriptor: FP16 operands, K-major, fp32 sums
  p.idesc = (1u << 4) | ((uint32_t)((kChan * f.cta) >> 4) << 24);
  if (f.cta == 1) p.idesc |= (uint32_t)(f.tok >> 3) << 17;  // a pair's tokens go by the tile

  const bool prep = f.cta == 1 || widen;
  if (prep) {
    const int64_t per_row = a.K / 16, items = std::max<int64_t>(widen ? a.S * per_row : 0, kI8SyncWords);
    const unsigned grid = (unsigned)std::min<int64_t>((items + kPrepThreads - 1) / kPrepThreads, (int64_t)num_sms * 16);
    int8_prep_kernel<<<grid, kPrepThreads, 0, stream>>>(ws.sync, f.cta == 1 ? kI8SyncWords : 0, a.a, a.ld_a,
                                                        widen ? a.S : 0, per_row, reinterpret_cast<uint4*>(ws.wide));
    if (cudaGetLastError() != cudaSuccess) return MXG_ERR_CUDA;
  }
  CUtensorMap tmW, tmX;
  if (!make_tmap(&tmW, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.K, (int64_t)a.G * a.N, a.ld_w, kStageK, kChan)) return MXG_ERR_CUDA;
  // without rows there is nothing to load and the map only has to be well formed
  const bool ok = a.S == 0 ? make_f16_tmap(&tmX, a.w, 8, 1, 16, f.tok / f.cta)
                  : widen  ? make_f16_tmap(&tmX, ws.wide, a.K, a.S, a.K * 2, f.tok / f.cta)
                           : make_f16_tmap(&tmX, a.a, a.K, a.S, a.ld_a, f.tok / f.cta);
  if (!ok) return MXG_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (f.cta == 2) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  } else {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.gridDim = dim3((unsigned)(f.cta == 2 ? 2 * pairs : std::min(num_sms, kI8MaxCtas)));
  cfg.blockDim = dim3((unsigned)f.threads);
  cfg.dynamicSmemBytes = (size_t)f.smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  void* args[] = {(void*)&tmW, (void*)&tmX, (void*)&p};
  if (cudaLaunchKernelExC(&cfg, f.fn, args) != cudaSuccess) {
    cudaGetLastError();
    return MXG_ERR_CUDA;
  }
  return MXG_OK;
}

}  // namespace mxg
