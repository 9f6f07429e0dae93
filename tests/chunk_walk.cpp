// Runs the chunk hand-out of the 8-bit split kernel with one warp after the other taking a step: each warp's copies run
// up to a ring ahead of its arithmetic.  argv: tiles of the stream, warps, the caller's cut in tiles, chunks that the
// workspace holds.  Prints tiles used under another's name, tiles left in a ring at the end, tiles used, chunk length.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <vector>

#include "pa_chunk8.h"

int main(int argc, char **argv) {
  if (argc != 5) return 2;
  const long long total = std::atoll(argv[1]), warps = std::atoll(argv[2]), max_chunks = std::atoll(argv[4]);
  const long long c = pa::chunk8_tiles(total, warps, std::atoi(argv[3]), max_chunks);
  const long long count = (total + c - 1) / c;
  auto length = [&](long long k) { return std::min(c, total - k * c); };
  long long ticket = std::min(warps, count), wrong = 0, left = 0, used = 0;
  struct Warp {
    long long prod_c, prod_left, prod_at, cons_c, cons_left, k;
    bool prod_done, done;
    std::deque<long long> ring;  // tiles on their way, by their place in the stream
  };
  std::vector<Warp> w;
  auto issue = [&](Warp &x) {
    if (x.prod_left == 0) {
      if (x.prod_done) return;
      if (ticket >= count) {
        x.prod_done = true;
        return;
      }
      x.prod_c = ticket++;
      x.prod_left = length(x.prod_c);
      x.prod_at = x.prod_c * c;
    }
    x.ring.push_back(x.prod_at++);
    --x.prod_left;
  };
  for (long long i = 0; i < std::min(warps, count); ++i) {
    Warp x{i, length(i), i * c, i, length(i), 0, false, false, {}};
    w.push_back(x);
  }
  for (Warp &x : w)
    for (int s = 0; s < pa::STAGES8; ++s) issue(x);
  for (bool busy = true; busy;) {
    busy = false;
    for (Warp &x : w) {
      if (x.done) continue;
      busy = true;
      if (x.cons_left == 0) {
        if (x.prod_c == x.cons_c) {
          x.done = true;
          left += (long long)x.ring.size();
          continue;
        }
        x.cons_c = x.prod_c;
        x.cons_left = length(x.cons_c);
        x.k = 0;
      }
      if (x.ring.empty() || x.ring.front() != x.cons_c * c + x.k) ++wrong;
      if (!x.ring.empty()) x.ring.pop_front();
      ++used;
      issue(x);
      --x.cons_left;
      ++x.k;
    }
  }
  std::printf("%lld %lld %lld %lld\n", wrong, left, used, c);
  return 0;
}
