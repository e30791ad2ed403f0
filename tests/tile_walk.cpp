// The tile order of the sources, run on the host: what test_tile_walk.py asks for on
// standard input, as 32-bit integers on standard output.
//   mn LOCAL TILES NTN GROUP            -> m-tile, n-tile
//   walk TOK N K G SPLITS...            -> (unit, k0, k1, expert, first row, rows, first channel) of every unit,
//                                          walked by one pair
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
      int tok, G;
      long long N, K;
      if (std::scanf("%d %lld %lld %d", &tok, &N, &K, &G) != 4) return 1;
      const I8Order o = i8_order(G, N, K, tok);
      std::vector<int32_t> off(G + 1, 0), tile(G + 1, 0);
      for (int g = 0; g < G; ++g) {
        int m;
        if (std::scanf("%d", &m) != 1) return 1;
        off[g + 1] = off[g] + m;
        tile[g + 1] = tile[g] + (m + tok - 1) / tok * o.n_chan;
      }
      if (tok == 32) walk<32, true>(o, off, tile, 0, tile[G] * o.nk, out);
      else if (tok == 64) walk<64, true>(o, off, tile, 0, tile[G] * o.nk, out);
      else if (tok == 128) walk<128, true>(o, off, tile, 0, tile[G] * o.nk, out);
      else walk<256, false>(o, off, tile, 0, tile[G], out);
    }
  }
  return std::fwrite(out.data(), 4, out.size(), stdout) == out.size() ? 0 : 1;
}
