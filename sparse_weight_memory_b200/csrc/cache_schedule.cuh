// cache_schedule.cuh -- which tokens and table entries the cache's calls may
// touch, and how fwpkm_cache_attend divides its work.  Plain integer
// arithmetic, the same on the device and on the host (where the tests check
// it).
//
// A tile is TT consecutive tokens of one sequence (aligned to TT), a segment
// all visible tiles of one sequence for one cached head and one block of 16 of
// the query heads that share it.  Segments are laid end to end in the order
// (sequence, cached head, row block), and the line of all tiles is cut into
// `warps` pieces whose sizes differ by at most one tile: every warp reads the
// same number of bytes whatever the lengths are.  A segment that a cut falls
// into is summed in parts:
//   - the part that begins with the segment lies in the tail slot 2w+1 of its
//     warp w,
//   - the part of each later warp w' lies in that warp's head slot 2w'.
// So a segment's parts are slots 2w+1, 2(w+1), ..., 2*last.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define FWPKM_HD __host__ __device__ __forceinline__
#else
#define FWPKM_HD inline
#endif

namespace fwpkm {

// A sequence's length within what a row of the table can hold; `bad` where it
// is not the given one.
FWPKM_HD int cache_length(int len, int width, int page_size, bool &bad) {
  const int64_t most = (int64_t)width * page_size;
  bad = len < 0 || len > most;
  return len < 0 ? 0 : len > most ? (int)most : len;
}
// The position of a new token with `before` rows of its sequence in front of
// it and `after` rows from it to the sequence's end, or -1 where the length
// does not leave it one.  `bad` where the row may not be stored: its sequence
// has more rows than tokens, or its page would lie behind the table.
FWPKM_HD int append_position(int len, int before, int after, int width, int page_size, bool &bad) {
  if (len < 0 || after < 1 || len < after) {
    bad = true;
    return -1;
  }
  const int pos = len - after;
  bad = before < 0 || pos < before || pos / page_size >= width;
  return pos;
}
// Visible tokens [lo, len) of a sequence, as tiles first .. first + count - 1.
// A sequence without visible tokens still has one (empty) tile, so that some
// warp writes its result.
struct Span {
  int lo, len, first, count;
};
FWPKM_HD Span cache_span(int len, int window, int tile) {
  Span s;
  s.len = len;
  s.lo = window > 0 && len > window ? len - window : 0;
  s.first = s.lo / tile;
  s.count = len > s.lo ? (len - 1) / tile + 1 - s.first : 1;
  return s;
}

// Warps that share `total` tiles: all of them once each has `least` tiles.
FWPKM_HD int cache_warps(int64_t total, int most, int least) {
  const int64_t w = total / least;
  return w < 1 ? 1 : w < most ? (int)w : most;
}
// First tile of warp w's piece (w == warps: the end of the line).
FWPKM_HD int64_t cache_cut(int64_t total, int warps, int w) { return total * w / warps; }
// The warp whose piece holds the tile before `end`.
FWPKM_HD int cache_last_warp(int64_t total, int warps, int64_t end) {
  return (int)((end * warps + total - 1) / total) - 1;
}

}  // namespace fwpkm
