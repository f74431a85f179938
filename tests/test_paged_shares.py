"""How the paged attention shares its rows out over the CTAs (csrc/paged_share.cuh), on the CPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include "paged_share.cuh"
// Where each CTA's part begins (and the last one's ends): tiles and rows before it, and the tile within its row.
extern "C" int cuts(const int* nq, const int* len, int batch, int topk_tiles, int ctas, long long* tiles_at, long long* rows_at,
                    int* tile_at, long long* share) {
  long long tiles = 0, rows = 0;
  int longest = 0;
  for (int b = 0; b < batch; ++b) {
    tiles += dsa::tiles_of(nq[b], len[b], topk_tiles, nq[b]);
    rows += nq[b];
    const int most = topk_tiles ? topk_tiles : (len[b] > 1 ? len[b] : 1) / 128 + ((len[b] > 1 ? len[b] : 1) % 128 != 0);
    if (nq[b] > 0 && most > longest) longest = most;
  }
  const dsa::PagedShares sh = dsa::paged_shares(tiles, rows, longest, ctas);
  *share = sh.share;
  for (int c = 0; c <= ctas; ++c) {
    const long long g = sh.begin(c);
    long long x = 0, y = 0, at = 0;
    tiles_at[c] = tiles, rows_at[c] = rows, tile_at[c] = 0;  // (at or behind the line's end)
    for (int b = 0; b < batch; ++b) {
      const long long n = dsa::tiles_of(nq[b], len[b], topk_tiles, nq[b]), end = at + sh.line(n, nq[b]);
      if (g >= at && g < end) {
        long long first;
        int tile;
        const int row = sh.cut(nq[b], len[b], topk_tiles, g - at, first, tile);
        tiles_at[c] = x + first + tile, rows_at[c] = y + row, tile_at[c] = tile;
        break;
      }
      x += n, y += nq[b], at = end;
    }
  }
  return sh.whole;
}
extern "C" long long row_tiles(int nq, long long len, int topk_tiles, int j) { return dsa::tiles_of(nq, len, topk_tiles, j); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("shares")
    (d / "driver.cpp").write_text(DRIVER)
    so = str(d / "driver.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-I",
                           os.path.join(ROOT, "indexer_selected_sparse_dsa_b200", "csrc"), str(d / "driver.cpp"), "-o", so])
    L = ctypes.CDLL(so)
    L.row_tiles.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    L.row_tiles.restype = ctypes.c_longlong
    return L


def row_list(new, lens, topk_tiles):
    """Tiles of every query row, in order, by definition."""
    return [topk_tiles or max(1, -(-(m - n + j + 1) // 128)) for n, m in zip(new, lens) for j in range(n)]


def cuts(L, new, lens, topk_tiles, ctas):
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    nq, ln = np.array(new, np.int32), np.array(lens, np.int32)
    tiles, rows, tile = np.zeros(ctas + 1, np.int64), np.zeros(ctas + 1, np.int64), np.zeros(ctas + 1, np.int32)
    share = np.zeros(1, np.int64)
    whole = L.cuts(p(nq), p(ln), len(new), topk_tiles, ctas, p(tiles), p(rows), p(tile), p(share))
    return bool(whole), tiles, rows, tile, int(share[0])


def walks(rows, begin_row, begin_tile, cost):
    """What each CTA walks, in tiles with the starts of its rows."""
    out = []
    for c in range(len(begin_row) - 1):
        r0, t0, r1, t1 = int(begin_row[c]), int(begin_tile[c]), int(begin_row[c + 1]), int(begin_tile[c + 1])
        if (r0, t0) == (r1, t1):
            out.append(0)
            continue
        n = sum(rows[r0:r1]) - t0 + t1
        starts = (r1 - r0) + (1 if t1 > 0 else 0) - (1 if t0 > 0 else 0)
        out.append(n + cost * starts)
    return out


def check(L, new, lens, topk_tiles=0, ctas=148):
    rows = row_list(new, lens, topk_tiles)
    whole, tiles_at, rows_at, tile_at, share = cuts(L, new, lens, topk_tiles, ctas)
    total = sum(rows)
    before = np.concatenate([[0], np.cumsum(rows)])
    assert tiles_at[0] == 0 and tiles_at[-1] == total and (np.diff(tiles_at) >= 0).all()
    for t, r, i in zip(tiles_at, rows_at, tile_at):  # the row and tile are the place that the count of tiles says
        assert t == before[r] + i and 0 <= i < (rows[r] if r < len(rows) else 1)
    cost = 2 if total > ctas else 0
    assert share == -(-(total + cost * len(rows)) // ctas)
    most = max(walks(rows, rows_at, tile_at, cost))
    if whole:
        assert not tile_at.any()
        assert most <= share + 1 + 5 * min(total, ctas) / 160, (most, share)
    else:
        assert most <= share + cost, (most, share)  # (a share that begins inside a row's start walks that start whole)
    return whole, most, share


@pytest.mark.parametrize("batch", [1, 2, 40, 64, 100, 128, 144, 148, 149, 200, 296, 297, 1000])
@pytest.mark.parametrize("longest", [100, 300, 1024, 1536, 8000])
def test_no_walk_is_longer_than_said_decode(lib, batch, longest):
    r = np.random.default_rng(batch * 10007 + longest)
    for lo in (1, max(1, longest * 15 // 16), longest):
        for _ in range(4):
            lens = [int(x) for x in r.integers(lo, longest + 1, batch)]
            check(lib, [1] * batch, lens)


@pytest.mark.parametrize("new,lens", [
    ([148], [8150]), ([144], [2000]), ([512], [512]), ([512, 266], [8192, 2369]), ([40, 0, 1, 90], [4000, 3, 2500, 700]),
    ([6, 1, 3, 2, 5] * 4, [8192, 300, 77, 5000, 6] * 4), ([0, 0, 1], [9, 0, 1]), ([3], [1]), ([5, 2], [0, 100]),
    ([1], [300]), ([1], [128]), ([0, 0], [5, 0]), ([1] * 400, [1 + i % 300 for i in range(400)])])
@pytest.mark.parametrize("topk_tiles", [0, 1, 3, 8, 16])
@pytest.mark.parametrize("ctas", [1, 3, 132, 148, 160])
def test_no_walk_is_longer_than_said_chunks(lib, new, lens, topk_tiles, ctas):
    check(lib, new, lens, topk_tiles, ctas)


def test_rows_near_the_number_of_ctas_are_dealt_out_one_by_one(lib):
    """Unequal rows, as many as CTAs or a few less: whole, and no CTA has two."""
    r = np.random.default_rng(5)
    for batch in (140, 148):
        lens = [int(x) for x in r.integers(60 * 128, 64 * 128, batch)]
        whole, most, share = check(lib, [1] * batch, lens)
        assert whole and most <= 66


def test_rows_counted_many_times_over(lib):
    """A cu_q that goes back and forth: more rows than 32 bits hold, and every place on the line still found."""
    batch, rows = 12000, 1 << 25
    for topk_tiles, m in ((1, 1 << 26), (16, 1 << 26), (0, rows)):
        whole, tiles_at, rows_at, tile_at, _ = cuts(lib, [rows] * batch, [m] * batch, topk_tiles, 148)
        each = lib.row_tiles(rows, m, topk_tiles, rows)
        assert tiles_at[0] == rows_at[0] == 0 and tiles_at[-1] == batch * each and rows_at[-1] == batch * rows
        assert (np.diff(tiles_at) > 0).all()
        for t, r, i in zip(tiles_at, rows_at, tile_at):
            b, j = divmod(int(r), rows)
            assert int(t) == b * each + lib.row_tiles(rows, m, topk_tiles, j) + int(i)


def test_tiles_of_by_definition(lib):
    for nq, m in ((1, 1), (5, 5), (7, 3), (4, 0), (300, 1000), (130, 129), (2, 1 << 20)):
        for j in range(0, nq + 1, max(1, nq // 9)):
            assert lib.row_tiles(nq, m, 0, j) == sum(max(1, -(-(m - nq + i + 1) // 128)) for i in range(j))
            assert lib.row_tiles(nq, m, 16, j) == 16 * j
    assert lib.row_tiles(9, -1, 0, 9) == 9
    assert lib.row_tiles(1, 2 ** 31 - 1, 0, 1) == 1 << 24
