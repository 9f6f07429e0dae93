// Which entries of a block table row a warp of the 8-bit decode kernels holds: one per lane, of the row it read last.
// Host code too, so that the choice can be tested without a GPU.
#pragma once

#ifndef PA_HOST_DEVICE
#ifdef __CUDACC__
#define PA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PA_HOST_DEVICE inline
#endif
#endif

namespace pa {

constexpr int TILE8 = 32;  // tokens per tile of the 8-bit kernels

struct TableWindow {
  int row = -1, base = 0, end = 0;  // lane i holds entry base + i of table row `row` while that is below `end`
  int first = 0, last = 0;          // entries of the tile asked for last

  // Asks for the entries (of blocks of 16 or 32 tokens) of tile j of a row group that sees L > 0 tokens of table row r.
  // Returns whether the lanes have to be loaded, with entries base .. end - 1: none behind the group's last block, since
  // the row may be the last of a table that ends there.  Row groups of one sequence share its row, and a later one may
  // need an entry that an earlier one did not load: holding the row and the window is not enough.
  PA_HOST_DEVICE bool ask(int r, int j, int L, int block_size) {
    const bool two = block_size == 16;
    first = two ? 2 * j : j;
    last = two && L - j * TILE8 > 16 ? first + 1 : first;  // first is even: the same window
    if (r == row && first >= base && last < end) return false;
    const int blocks = ((L - 1) >> (two ? 4 : 5)) + 1;  // at most the row's entries: contexts are checked against them
    row = r;
    base = first & ~31;
    end = base + 32 < blocks ? base + 32 : blocks;
    return true;
  }
};

}  // namespace pa
