// Which tile a number in the order of a product's work stands for, and which pair of
// CTAs takes which work.  Plain arithmetic, which a host compiler takes too, with the
// same results (the tests do).
#pragma once
#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define MXG_HD __host__ __device__ __forceinline__
#else
#define MXG_HD inline
#endif

namespace mxg {

MXG_HD int least(int a, int b) { return a < b ? a : b; }
MXG_HD int most(int a, int b) { return a > b ? a : b; }

MXG_HD int find_prefix(const int32_t* pre, int G, int x) {  // last g with pre[g] <= x
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tile order inside an expert: groups of `group_m` m-tiles; inside a group m
// runs fastest and n outer, so CTAs running at the same time share a B tile
// and the group's A rows stay in L2 across all of its n-tiles (B is then read
// once per group instead of once per m-tile).  A group has at most the expert's
// m-tiles, so that no product here is above expert_tiles.
MXG_HD void tile_mn(int local, int expert_tiles, int ntn, int group_m, int& mt, int& nt) {
  const int mtn = expert_tiles / ntn;
  group_m = least(group_m, mtn);
  const int span = group_m * ntn;
  const int grp = local / span;
  const int first = grp * group_m;
  const int rows = least(group_m, mtn - first);
  const int idx = local - grp * span;
  mt = first + idx % rows;
  nt = idx / rows;
}

// The integer products on the tensor cores: a unit is a tile of 256 channels (of a
// pair of CTAs) and kTok rows, its contraction nk stages.
constexpr int kUnitChan = 256;
constexpr int kStageK = 128;  // contraction elements of a stage
struct I8Order {
  int G, nk, n_chan;  // n_chan: channel tiles
  int group_t;        // token tiles per group of the unit order
};

constexpr int kI8MaxPairs = 80;  // what partial sums and join counters are sized for
constexpr int kI8SyncWords = 8 * kI8MaxPairs;
constexpr int kI8MinStages = 4;  // shortest run of cut units

// How the stages of all units are shared out, a run per pair: whole units; or cut into
// equal runs wherever these end; or, where there are pairs for it, every unit into
// `parts` equal runs of its own.  What ends soonest, in stages (0.46 us): a unit that
// is joined costs 4, and 0.6 for each run and 32 tokens of it, which the last to
// arrive adds up (100 rows, K = 16384, 256 channels: 46 us in runs of 4 stages, 25 in
// runs of 16 to 24; 100 rows, 1024 x 7168: 29 and 21).
struct I8Runs {
  int per_unit, grain, pairs, q, r, parts;  // parts > 0: of every unit
  MXG_HD I8Runs(int units, int per_unit_, int tokens, int max_pairs) : per_unit(per_unit_), parts(0) {
    const int total = units * per_unit, c32 = most((tokens + 31) >> 5, 1);
    const int whole = (int)((unsigned)(units + max_pairs - 1) / (unsigned)max_pairs) * per_unit;
    const int run = most((int)((unsigned)(total + max_pairs - 1) / (unsigned)max_pairs), kI8MinStages);
    const int cut = run + (run >= 2 * per_unit ? 3 : 8 + c32 * ((int)((unsigned)per_unit / (unsigned)run) + 3) * 5 / 8);
    grain = whole <= cut ? per_unit : 1;
    pairs = least(max_pairs, grain > 1 || per_unit == 1 ? units : (total + kI8MinStages - 1) / kI8MinStages);
    if (units > 0 && units <= max_pairs / 2 && per_unit > 1) {
      const float share = c32 == 1 ? 1.6f : c32 == 2 ? 0.8f : c32 == 3 ? 1.6f / 3 : 0.4f;  // 1.6 / c32, of at most 128 tokens
      int n = least((int)((unsigned)max_pairs / (unsigned)units), most(2, (int)(sqrtf(share * per_unit) + 0.5f)));
      n = least(n, per_unit);
      if ((int)((unsigned)per_unit / (unsigned)n) + 5 + c32 * n * 5 / 8 < least(whole, cut)) {
        parts = n;
        grain = 1;
        pairs = units * n;
      }
    }
    const int items = parts > 0 ? per_unit : grain > 1 ? units : total, to = parts > 0 ? parts : pairs;
    q = to > 0 ? (int)((unsigned)items / (unsigned)to) : 0;
    r = items - q * to;
  }
  // pair b's run
  MXG_HD void run(int b, int& s, int& end) const {
    const int u = parts > 0 ? (int)((unsigned)b / (unsigned)parts) : 0, i = b - u * parts;
    s = u * per_unit + (i * q + least(i, r)) * grain;
    end = s + (q + (i < r)) * grain;
  }
  // the first and the last pair of a cut unit
  MXG_HD int owner(int s) const { return s < r * (q + 1) ? s / (q + 1) : r + (s - r * (q + 1)) / q; }
  MXG_HD int first(int unit) const { return parts > 0 ? unit * parts : owner(unit * per_unit); }
  MXG_HD int last(int unit) const { return parts > 0 ? unit * parts + parts - 1 : owner(unit * per_unit + per_unit - 1); }
  // where a pair's partial sums go, of the cut unit that it begins or of the one that an
  // earlier pair began; the words that count the arrivals at a cut unit
  static MXG_HD int buffer(int pair, bool from_start) { return 2 * pair + from_start; }
  static MXG_HD int counter(int first_pair) { return (first_pair + 1) * 8; }
};

// Walks a pair's units: of a run (kCut), the cut unit at its start, the cut unit at
// its end, then the whole units; else every `per_unit`-th unit.
template <int kTok, bool kCut>
struct I8Walker {
  int s, end, per_unit;      // what is left of the run (else: the next unit, all units, the stride)
  int unit, k0, k1;          // the current unit and its stages [k0, k1)
  int e, tok0, n, chan0;     // expert, first row, rows, first channel of the tile
  MXG_HD bool next(const I8Order& p, const int32_t* off, const int32_t* tile) {
    if (s >= end) return false;
    if constexpr (!kCut) {
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
    // The expert's full tiles, then its short ones: in the order of the tiles every
    // second unit would be short where there are two, and always the same pairs'
    // (12000 rows of 32 experts, 4096 x 7168: 447 us, 481).
    const int rows = off[e + 1] - off[e], local = unit - tile[e], whole = rows / kTok * p.n_chan;
    int tt = rows / kTok, ct = local - whole;
    if (local < whole) tile_mn(local, whole, p.n_chan, p.group_t, tt, ct);
    n = least(kTok, rows - tt * kTok);
    tok0 = off[e] + tt * kTok;
    chan0 = ct * kUnitChan;
    return true;
  }
};

// The order for K and N, whose G experts' rows are taken `tok` at a time: groups of
// token tiles whose activations (about 32 MiB of FP16) stay in L2 over all channel tiles.
inline I8Order i8_order(int G, int64_t N, int64_t K, int tok) {
  const int64_t group = (int64_t(32) << 20) / (tok * K * 2);
  return {G, (int)((K + kStageK - 1) / kStageK), (int)((N + kUnitChan - 1) / kUnitChan), (int)(group < 1 ? 1 : group)};
}

}  // namespace mxg
