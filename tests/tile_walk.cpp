// The tile order of the sources, run on the host: what test_tile_walk.py asks for on
// standard input, as 32-bit integers on standard output.
//   mn LOCAL TILES NTN GROUP            -> m-tile, n-tile
//   walk TOK N K G SPLITS...            -> (unit, k0, k1, expert, first row, rows, first channel) of every unit,
//                                          walked by one pair
//   runs PAIRS TOK N K G SPLITS...      -> runs.pairs, whether units have parts, whether runs are of whole units, then
//                                          (pair, unit, k0, k1, first pair, last pair, buffer, first's buffer, counter)
//                                          of every piece of every pair's run
#include <cstdio>
#include <cstring>
#include <vector>

#include "tile_walk.h"

using namespace mxg;

static void put(std::vector<int32_t>& out, std::initializer_list<int> v) { out.insert(out.end(), v.begin(), v.end()); }

template <int kTok, bool kCut>
static void walk(const I8Order& o, const std::vector<int32_t>& off, const std::vector<int32_t>& tile, int s, int end,
                 std::vector<int32_t>& out) {
  I8Walker<kTok, kCut> w;
  w.s = s;
  w.end = end;
  w.per_unit = kCut ? o.nk : 1;
  while (w.next(o, off.data(), tile.data())) put(out, {w.unit, w.k0, w.k1, w.e, w.tok0, w.n, w.chan0});
}

template <int kTok>
static void runs(const I8Order& o, const std::vector<int32_t>& off, const std::vector<int32_t>& tile, int max_pairs,
                 std::vector<int32_t>& out) {
  const int units = tile[o.G];
  const I8Runs r(units, o.nk, units > 0 ? off[o.G] / (units / o.n_chan) : 0, max_pairs);
  put(out, {r.pairs, r.parts > 0, r.grain > 1});
  for (int b = 0; b < r.pairs; ++b) {
    I8Walker<kTok, true> w;
    r.run(b, w.s, w.end);
    w.per_unit = o.nk;
    while (w.next(o, off.data(), tile.data())) {
      const bool cut = w.k0 != 0 || w.k1 != o.nk;
      const int first = cut ? r.first(w.unit) : b, last = cut ? r.last(w.unit) : b;
      put(out, {b, w.unit, w.k0, w.k1, first, last, I8Runs::buffer(b, w.k0 == 0), I8Runs::buffer(b, b == first),
                I8Runs::counter(first)});
    }
  }
}

int main() {
  char what[16];
  std::vector<int32_t> out;
  while (std::scanf("%15s", what) == 1) {
    if (std::strcmp(what, "mn") == 0) {
      int local, tiles, ntn, group, mt = -1, nt = -1;
      if (std::scanf("%d %d %d %d", &local, &tiles, &ntn, &group) != 4) return 1;
      tile_mn(local, tiles, ntn, group, mt, nt);
      put(out, {mt, nt});
    } else {
      int tok, G, pairs = 0;
      long long N, K;
      if (std::strcmp(what, "runs") == 0 && std::scanf("%d", &pairs) != 1) return 1;
      if (std::scanf("%d %lld %lld %d", &tok, &N, &K, &G) != 4) return 1;
      const I8Order o = i8_order(G, N, K, tok);
      std::vector<int32_t> off(G + 1, 0), tile(G + 1, 0);
      for (int g = 0; g < G; ++g) {
        int m;
        if (std::scanf("%d", &m) != 1) return 1;
        off[g + 1] = off[g] + m;
        tile[g + 1] = tile[g] + (m + tok - 1) / tok * o.n_chan;
      }
      if (pairs > 0) {
        if (tok == 32) runs<32>(o, off, tile, pairs, out);
        else if (tok == 64) runs<64>(o, off, tile, pairs, out);
        else runs<128>(o, off, tile, pairs, out);
      } else if (tok == 32) walk<32, true>(o, off, tile, 0, tile[G] * o.nk, out);
      else if (tok == 64) walk<64, true>(o, off, tile, 0, tile[G] * o.nk, out);
      else if (tok == 128) walk<128, true>(o, off, tile, 0, tile[G] * o.nk, out);
      else walk<256, false>(o, off, tile, 0, tile[G], out);
    }
  }
  return std::fwrite(out.data(), 4, out.size(), stdout) == out.size() ? 0 : 1;
}
