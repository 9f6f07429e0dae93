// How the 8-bit split kernel's tile stream is cut into chunks.  Host code too, so that the choice can be tested without a
// GPU.
#pragma once

#ifndef PA_HOST_DEVICE
#ifdef __CUDACC__
#define PA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PA_HOST_DEVICE inline
#endif
#endif

namespace pa {

constexpr int STAGES8 = 2;  // ring slots of a warp of the split kernel

// Uniform chunks, `tail` of them per warp on average.  Long streams take several, so that warps that run ahead take over
// from those that lag (8 contexts of 16k-32k tokens: 278 us with one, 268 with three); short ones one, since each cut
// leaves pieces to merge (256 sequences of 32 q / 8 kv heads, 31 tiles per warp: 1, 3 and 5 us more with two, three and
// five).
constexpr int TAIL8_TILES = 16, TAIL8_MOST = 3;
// No chunk but the stream's last is shorter than the ring: a warp's copies run up to a ring ahead of its arithmetic, which
// follows them from one chunk into the next and would miss one that lies between.  This holds for a caller's cut too.
constexpr int MIN_CHUNK8_TILES = 2;
static_assert(MIN_CHUNK8_TILES >= STAGES8, "the arithmetic may be at most one chunk behind the copies");

PA_HOST_DEVICE long long ceil_div8(long long x, long long y) {
  return x < 0x7fffffffLL && y < 0x7fffffffLL ? (long long)(((unsigned)x + (unsigned)y - 1u) / (unsigned)y)
                                               : (x + y - 1) / y;
}

// Tiles of a chunk of a stream of `total` tiles over `warps` warps; chunk_tiles: the caller's cut (0: none), max_chunks:
// what the workspace holds.
PA_HOST_DEVICE long long chunk8_tiles(long long total, long long warps, int chunk_tiles, long long max_chunks) {
  long long c = chunk_tiles;
  if (c == 0) {
    long long tail = total / (warps * TAIL8_TILES);
    tail = tail < 1 ? 1 : tail > TAIL8_MOST ? TAIL8_MOST : tail;
    c = ceil_div8(total, warps * tail);
  }
  const long long least = ceil_div8(total, max_chunks);
  c = c < least ? least : c;
  return c < MIN_CHUNK8_TILES ? MIN_CHUNK8_TILES : c;
}

}  // namespace pa
