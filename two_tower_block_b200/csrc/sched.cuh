// Work split shared by the attention kernels, the split combine and the host.
//
// A "unit" is one (sequence, KV head[, block]) problem: its S*g packed query
// rows attend to one key list.  Its key list is cut into tiles: tile 0 is the
// block's own S keys, tiles 1.. are the visible context keys, key_tile at a
// time.  All units' tiles are laid end to end (unit-major) into one global
// sequence of T tiles, and range c of C' = min(C, T) gets tiles [floor(c*T/C'),
// floor((c+1)*T/C')); ranges c >= C' are empty.  Every range therefore carries the same work up to one
// tile, whatever the length mix, and a unit is cut only where a range
// boundary falls inside it.
//
// A range's pieces of units are "segments".  A segment that covers a whole
// unit writes the final output.  Otherwise it writes a partial (O / l and its
// lse) to slot 2*c + which, where which = 0 if the segment begins at the
// range's first tile and 1 otherwise; a cut unit is then finished by the
// combine kernel.  Only a range's first and last segment can belong to a cut
// unit, so 2*C slots always suffice.
//
// A unit may also carry a fixed cost of F tiles (the Q load and the pipeline's restart before it, the
// output after it): the global sequence then has F / 2 empty places before each unit's tiles and the
// rest after them, T counts them too, and a boundary that falls on empty places cuts no unit.  A
// range costs its tiles and one F for each unit's edge inside it, which is what the even split of
// that sequence evens out.  F is kept small enough that every range holds a tile (fixed_cost).
//
// A plan may instead give the boundaries as a table starts[0..C'] (starts[0] = 0,
// starts[C'] = T, strictly increasing), which the block-causal calls of the default
// kernel use to weigh each unit's fixed cost (built by the plan on the host); everything
// above holds for it unchanged.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define TT_HD __host__ __device__ __forceinline__
#else
#define TT_HD inline
#endif

namespace tt {

// (32-bit divisions where they hold: these sit on the path before a kernel's first load)
TT_HD long long range_start(long long T, int C, int c) {
  if (T < (1ll << 31) / C) return (uint32_t)c * (uint32_t)T / (uint32_t)C;
  return (long long)c * T / C;
}

// Ranges actually used: min(C, T), so that every used range holds at least one
// tile and the ranges touching a cut unit are consecutive and all non-empty.
TT_HD int used_ranges(long long T, int C) { return T < (long long)C ? (int)T : C; }

// Index of the range whose [start, end) contains global tile x (0 <= x < T):
// the largest c with floor(c*T/C) <= x, i.e. ceil((x+1)*C/T) - 1.
TT_HD int range_of_tile(long long T, int C, long long x) {
  if (T < (1ll << 30) / C) return (int)((((uint32_t)x + 1u) * (uint32_t)C + (uint32_t)T - 1u) / (uint32_t)T) - 1;
  return (int)(((x + 1) * (long long)C + T - 1) / T) - 1;
}

// The fixed cost per unit that leaves a tile to every range: at most `want`, for U units of T tiles in
// all over C ranges (any range is at least floor((T + U F) / C) places long, and must be longer than
// the F empty places between two units).
TT_HD int fixed_cost(long long T, long long U, int C, int want) {
  if (U >= C) return want;
  if (T < C) return 0;
  const long long most = (T - C) / (C - U);
  return most < want ? (int)most : want;
}

// The cost per unit of a decode call whose units have `least` to `most` tiles: units of one length over ranges
// that divide them evenly need no weighing.
TT_HD int decode_cost(long long T, int U, int C, int want, int least, int most) {
  return want > 0 && !(least == most && C % U == 0) ? fixed_cost(T, U, C, want) : 0;
}
// Short units: range c is unit c.
TT_HD bool whole_units(int U, int C, int most, int whole_tiles) { return U <= C && most <= whole_tiles; }

// The same two for a boundary table (null: the uniform split).
TT_HD long long range_start_tab(const long long* tab, long long T, int C, int c) {
  return tab ? tab[c] : range_start(T, C, c);
}
TT_HD int range_of_tile_tab(const long long* tab, long long T, int C, long long x) {
  if (!tab) return range_of_tile(T, C, x);
  int lo = 0, hi = C - 1;  // the largest c with tab[c] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// (a >= 0; unsigned, since the positions of a page table go up to 2^31 - 16)
TT_HD int ceil_div(int a, int b) { return (int)(((uint32_t)a + (uint32_t)b - 1u) / (uint32_t)b); }

// Number of tiles of a unit whose visible context has L keys.
TT_HD int unit_tiles(int L, int key_tile) { return 1 + ceil_div(L, key_tile); }

// The visible context of a unit with L committed positions on a layer with a sliding window:
// positions [0, sinks) and [L - window, L), as two runs of tiles.  When the two meet (or the
// layer has no window, window = 0) there is one run over [0, L).  Runs begin at a multiple of
// `align` positions (1, or the slice of a page that one load brings in); the `head` positions
// before the window's first one are then loaded but not visible.
struct CtxSpan {
  int sink_tiles;  // tiles of the first run (positions [0, sinks)); 0: a single run
  int wstart;      // first position of the second run
  int head;        // positions at its start that are not visible
  int tiles;       // tiles of both runs
};
TT_HD CtxSpan ctx_span(int L, int window, int sinks, int align, int key_tile) {
  CtxSpan s;
  if (window <= 0 || (long long)L - window <= sinks) {
    s.sink_tiles = s.wstart = s.head = 0;
  } else {
    const int wlo = L - window;
    s.sink_tiles = ceil_div(sinks, key_tile);
    s.wstart = wlo / align * align;
    s.head = wlo - s.wstart;
  }
  s.tiles = s.sink_tiles + ceil_div(L - s.wstart, key_tile);
  return s;
}

// The scale bytes of a quantised tile (D / 32 a row) are brought in by words of four bytes, aligned on both
// sides.  With head_dim 64 a word holds two rows: a contiguous cache's tile may begin at an odd row, and
// its words then begin one row earlier (the scales lie mx_odd rows into the tile's buffer).  A page, and
// so every slice of a paged tile, begins at an even row.
TT_HD int mx_odd(int D, bool paged, int row0) { return D == 64 && !paged ? row0 & 1 : 0; }
struct ScaleWord {
  int row;     // its first row within the tile (-1: the row in front of the tile)
  int slice;   // slice of 1 << psh rows it lies in: its rows follow the slice's first pool row
  int bytes;   // bytes of it that belong to the tile, 0: none
};
TT_HD ScaleWord scale_word(int word, int D, bool paged, int psh, int odd, int count) {
  const int row_bytes = D / 32;
  ScaleWord w;
  w.row = word * 4 / row_bytes - odd;
  w.slice = paged ? w.row >> psh : 0;
  const int left = (count - w.row) * row_bytes;
  w.bytes = left < 0 ? 0 : left < 4 ? left : 4;
  return w;
}
// Byte offset of the word, whose slice begins at pool row `slice_row`.
TT_HD long long scale_word_at(const ScaleWord& w, int D, int psh, int slice_row) {
  return ((long long)slice_row - (w.slice << psh) + w.row) * (D / 32);
}

// Per-range record the attention kernel leaves for the combine: the unit that
// is cut and begins in this range (or -1), the last range touching it, and
// the slot choice of this range's piece.
struct SplitRecord {
  int unit;
  int last_range;
  int first_which;
  int pad;
};

// One unit, as the kernels walk over them.
struct Unit {
  int u;          // unit index
  int tiles;      // number of key tiles
  int L;          // visible context keys
  int n, h, b;    // sequence, KV head, block index within the sequence
  int ns;         // block-sequence index n * NB + b (row block of q / k_blk / out)
  int sink_tiles, wstart, head;  // context runs of a windowed layer (CtxSpan)
  int cost;       // its fixed cost, cost / 2 places of it before the tiles
  long long Tu;   // first global place of the unit
};

// Global places of the unit's first tile, and behind its last.
TT_HD long long first_tile(const Unit& x) { return x.Tu + x.cost / 2; }
TT_HD long long end_tile(const Unit& x) { return first_tile(x) + x.tiles; }
// Whether no later unit has a tile before `end`, and no earlier one a tile at or after `start`.
TT_HD bool last_before(const Unit& x, long long end) { return end_tile(x) + x.cost >= end; }
TT_HD bool first_after(const Unit& x, long long start) {
  return first_tile(x) - x.cost <= start;
}

// Segment of the current unit inside [start, end).
struct Segment {
  int lo, hi;     // unit-local tiles [lo, hi)
  bool full;      // covers the whole unit: write the final output
  int slot;       // partial slot when !full
  bool last;      // last segment of the range
};

TT_HD Segment segment_of(const Unit& x, long long start, long long end, int c) {
  Segment s;
  const long long f = first_tile(x);
  s.lo = start > f ? (int)(start - f) : 0;
  s.hi = end - f < x.tiles ? (int)(end - f) : x.tiles;
  s.full = (s.lo == 0 && s.hi == x.tiles);
  s.slot = 2 * c + (s.lo > 0 || first_after(x, start) ? 0 : 1);
  s.last = last_before(x, end);
  return s;
}

// The record of range c: the cut unit that begins in c and runs past its end.
// C is the plan's range count; the split uses min(C, T) of them.
TT_HD SplitRecord record_of(const Unit& last, long long T, int C, long long start, long long end,
                            const long long* tab) {
  C = used_ranges(T, C);
  SplitRecord r;
  r.unit = -1;
  r.last_range = -1;
  r.first_which = 0;
  r.pad = 0;
  if (first_tile(last) >= start && end_tile(last) > end) {
    r.unit = last.u;
    r.last_range = range_of_tile_tab(tab, T, C, end_tile(last) - 1);
    r.first_which = first_after(last, start) ? 0 : 1;
  }
  return r;
}

}  // namespace tt
