// cache_schedule.cuh -- which tokens and table entries the cache's calls may
// touch, and how fwpkm_cache_attend divides its work.  Plain integer
// arithmetic, the same on the device and on the host (where the tests check
// it).
//
// A tile is TT consecutive tokens of one sequence (aligned to TT), a segment
// all visible tiles of one sequence for one cached head and one block of the
// query heads that share it.  A segment costs its tiles and `extra` tiles' worth
// beside them (its queries, its result): so many units.  Segments are laid end
// to end in the order (sequence, cached head, block), and the line of all units
// is cut into `warps` pieces whose sizes differ by at most one unit.  A warp
// takes the tiles whose first unit lies in its piece: tile 0 of a segment is at
// the segment's first unit, tile j at unit extra + j.  Where there are no more
// tiles than warps, each is a piece of its own (extra = 0): the shortest time.
// A segment that a cut falls into is summed in parts:
//   - the part that begins with the segment lies in the tail slot 2w+1 of its
//     warp w,
//   - the part of each later warp w' lies in that warp's head slot 2w'.
// So a segment's parts are slots 2w+1, 2(w+1), ..., 2*last (no warp between
// them is without a tile, since pieces have more than `extra` units).
// Where every segment is short, the line is first cut into a piece for each CTA,
// each cut moved to the next segment's start, and then those pieces for the
// CTA's warps: no segment lies in two CTAs, and no second kernel is needed.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define FWPKM_HD __host__ __device__ __forceinline__
#else
#define FWPKM_HD inline
#endif

namespace fwpkm {

// Division by a fixed page size as a product and a shift: exact for 0 <= t < 2^31
// (mul is the first integer from 2^shift / d up, 2^31 <= 2^(shift - log2 d) <= 2^32).
struct PageDiv {
  uint32_t mul;
  int shift;
};
inline PageDiv page_div(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  const uint64_t top = 1ull << (31 + s);
  return {(uint32_t)((top + d - 1) / d), 31 + s};
}
FWPKM_HD int page_of(PageDiv p, int t) {
  return (int)(((uint64_t)(uint32_t)t * p.mul) >> p.shift);
}
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

// Unit of tile j, and the first tile at or after unit u of the segment (which
// may be its number of tiles: none).
FWPKM_HD int64_t tile_unit(int j, int extra) { return j == 0 ? 0 : (int64_t)j + extra; }
FWPKM_HD int tile_from(int64_t u, int extra) {
  return u == 0 ? 0 : u <= extra ? 1 : (int)(u - extra);
}
// Tiles of a segment of `count` that lie before unit u of it.
FWPKM_HD int tiles_before(int64_t u, int count, int extra) {
  return u <= 0 ? 0 : u <= extra + 1 ? 1 : u - extra < count ? (int)(u - extra) : count;
}
// A line of units cut into `warps` pieces: `more` of q + 1 units, then the
// others of q.
struct Line {
  int64_t q;
  int warps, more;
};
FWPKM_HD Line cut_line(int64_t units, int warps) {
  Line l;
  l.warps = warps;
  l.q = units / warps;
  l.more = (int)(units - l.q * warps);
  return l;
}
// First unit of piece w (w == warps: the end of the line).
FWPKM_HD int64_t line_cut(const Line &l, int w) { return l.q * w + (w < l.more ? w : l.more); }
// The piece that holds a unit.
FWPKM_HD int line_owner(const Line &l, int64_t unit) {
  const int64_t big = (l.q + 1) * l.more;
  return unit < big ? (int)(unit / (l.q + 1)) : l.more + (int)((unit - big) / l.q);
}
// The line in pieces for at most `most` warps, none of them too small to be
// worth one (nor, with units beside the tiles, without a tile).
FWPKM_HD Line piece_line(int64_t units, int most, int extra) {
  const int64_t w = units / (extra ? extra + 2 : 1);
  return cut_line(units, w < 1 ? 1 : w < most ? (int)w : most);
}
// What a segment costs beside its tiles, in tiles (512 short sequences of 16
// heads take 84 us with 0, 67 with 1, 64 with 2 and 4); nothing where every tile
// has a warp of its own.
FWPKM_HD int extra_units(int64_t tiles, int most) { return tiles <= most ? 0 : 2; }

}  // namespace fwpkm
