// How the query rows of a paged batch are shared out over the CTAs of paged_mla_kernel.
//
// The rows stand behind each other on a line, and a CTA takes what lies in an equal share of it.  Split, a row is as long
// as the cost of its start and then its 128-key tiles: every CTA walks the same length, and rows that end in another CTA
// leave partial results.  Whole, every row is as long as any other: no row is split, and a CTA walks at most
// (longest row + start) * ceil(rows / CTAs).  Whole rows are taken where that is little more than the share of the split
// ones.  Measured on 148 CTAs, whole and split: 64 rows of 256, 512, 1024 keys 16.8 and 24.8, 23.2 and 30.5, 35.3 and
// 37.3 us; 543 selected rows of 8 tiles 123 and 138 us; rows of 1 to 1024 keys, 100 of them 35.3 and 37.1, 148 of them 36.9
// and 42.9 us; of 1 to 1536 keys, 148 of them 47.3 and 51.2, 100 of them (split by the rule) 45.9 and 41.7 us; a chunk of 148
// rows around 8100 keys 188 and 211 us.  (Dealing whole rows out by where they begin on the line of tiles can put nearly two
// shares into one CTA: that chunk took 357 us.)
//
// Plain integers, for the kernel and for a check on the host.
#pragma once

#ifdef __CUDACC__
#define DSA_HD __host__ __device__ __forceinline__
#else
#define DSA_HD inline
#endif

namespace dsa {

constexpr int kPgRowCost = 2;    // what a CTA's change to another query row costs, in tiles
constexpr int kPgMaxGrid = 160;  // CTAs at most (the workspace is sized for it)

// sum of ceil(i / 128) over i = 1 .. n
DSA_HD long long tiles_below(long long n) {
  const long long q = n >> 7, r = n & 127;
  return 64 * q * (q + 1) + r * (q + 1);
}

// Tiles of the first j query rows of a sequence with nq rows and length len (len < 0: a bad one, rows that see nothing);
// topk_tiles: of each row, where positions are selected, or 0.
DSA_HD long long tiles_of(int nq, long long len, int topk_tiles, int j) {
  if (topk_tiles) return (long long)j * topk_tiles;
  if (len < 0) return j;
  const long long base = len - nq;                            // positions before the first query row
  const long long blind = base < 0 ? (j < -base ? j : -base) : 0;  // rows that see nothing: one (empty) tile each
  return blind + tiles_below(base + j > 0 ? base + j : 0) - tiles_below(base > 0 ? base : 0);
}

struct PagedShares {
  bool whole;
  int cost;         // of a row's start, in tiles
  long long share;  // split: length of a CTA's part of the line
  int ctas;
  long long rows_each;  // whole: rows of each CTA ...
  int rows_rest;        // ... and the remainder (64 bits: a cu_q out of order may count rows many times)

  // Length of rows with that many tiles on the line.
  DSA_HD long long line(long long tiles, long long rows) const { return whole ? rows : tiles + cost * rows; }
  // Where a CTA's part begins, and (of the next one) ends.
  DSA_HD long long begin(int cta) const {
    return whole ? cta * rows_each + unsigned(cta * rows_rest) / unsigned(ctas) : share * cta;
  }
  // The row of a sequence, and its tile, that point `off` of the sequence's part of the line lies in; and the tiles of
  // the rows before it.
  DSA_HD int cut(int nq, long long len, int topk_tiles, long long off, long long& tiles_before, int& tile) const {
    int lo = whole ? int(off) : 0;
    for (int hi = whole ? lo + 1 : nq; hi - lo > 1;) {  // the last row that begins at or before it
      const int mid = (lo + hi) >> 1;
      if (line(tiles_of(nq, len, topk_tiles, mid), mid) <= off) lo = mid;
      else hi = mid;
    }
    tiles_before = tiles_of(nq, len, topk_tiles, lo);
    const long long in = off - line(tiles_before, lo) - cost;
    tile = whole || in < 0 ? 0 : int(in);
    return lo;
  }
};

// Of a batch with that many tiles and rows, the longest row of `longest` tiles.
DSA_HD PagedShares paged_shares(long long tiles, long long rows, int longest, int ctas) {
  PagedShares s;
  s.cost = tiles > ctas ? kPgRowCost : 0;  // (at most one tile each: nothing to balance)
  s.share = (tiles + s.cost * rows + ctas - 1) / ctas;
  s.ctas = ctas;
  s.rows_each = rows / ctas;
  s.rows_rest = int(rows % ctas);
  const long long walk = (longest + s.cost) * (s.rows_each + (s.rows_rest ? 1 : 0));
  // One tile more, and up to four as more CTAs would leave partial results.
  s.whole = walk <= s.share + 1 + 5 * (tiles < ctas ? tiles : ctas) / kPgMaxGrid;
  return s;
}

}  // namespace dsa
