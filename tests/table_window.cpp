// Walks the tile streams of random few-token calls as the warps of the split kernel do, and prints what the table
// window would load and use: argv = seed, block size, new tokens per sequence, tokens per row group, longest context.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "pa_table_window.h"

struct Group {
  int s, L, nt;
};

int main(int argc, char **argv) {
  if (argc != 6) return 2;
  std::mt19937 rng((unsigned)std::atoi(argv[1]));
  const int bs = std::atoi(argv[2]), fresh = std::atoi(argv[3]), per = std::atoi(argv[4]), longest = std::atoi(argv[5]);
  const int S = 40, HC = 3, stride = 8192 / bs;
  std::vector<Group> groups;
  for (int s = 0; s < S; ++s) {
    const int ctx = fresh + (int)(rng() % (unsigned)(longest - fresh + 1));
    for (int i = 0; i < fresh; i += per) {
      const int L = ctx - fresh + (i + per < fresh ? i + per : fresh);
      groups.push_back({s, L, (L + pa::TILE8 - 1) / pa::TILE8});
    }
  }
  struct Tile {
    int g, j;
  };
  std::vector<Tile> stream;
  for (int g = 0; g < (int)groups.size(); ++g)
    for (int h = 0; h < HC; ++h)
      for (int j = 0; j < groups[g].nt; ++j) stream.push_back({g, j});
  long missing = 0, past = 0, loads = 0;
  for (int chunk : {2, 7, 31, 200}) {  // stretches of the stream, one window each
    for (size_t at = 0; at < stream.size(); at += (size_t)chunk) {
      pa::TableWindow w;
      std::vector<int> held(32, -1);  // the row * stride + entry that each lane holds
      for (size_t t = at; t < stream.size() && t < at + (size_t)chunk; ++t) {
        const Group &g = groups[stream[t].g];
        if (w.ask(g.s, stream[t].j, g.L, bs)) {
          ++loads;
          for (int i = 0; i < 32; ++i) held[i] = w.base + i < w.end ? g.s * stride + w.base + i : -1;
          if (w.end > (g.L + bs - 1) / bs) ++past;  // an entry behind the last one that the group needs
        }
        const int j = stream[t].j, first = bs == 16 ? 2 * j : j, last = (std::min((j + 1) * 32, g.L) - 1) / bs;
        for (int e = first; e <= last; ++e)
          if (e < w.base || e >= w.base + 32 || held[e - w.base] != g.s * stride + e) ++missing;
      }
    }
  }
  std::printf("%ld %ld %ld\n", missing, past, loads);
  return 0;
}
