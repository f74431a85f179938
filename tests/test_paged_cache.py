"""The paged 8-bit latent cache: writing, reading back, and latent attention over it."""
import ctypes

import numpy as np
import pytest

from indexer_selected_sparse_dsa_b200 import binding as B
from indexer_selected_sparse_dsa_b200 import build
from paged_util import (HEADS, LATENT, ROW, ROW8, SCALE, Batch, check_attention, e4m3_values, quantise64, selection)


# ------------------------------------------------------------------ the definition itself (CPU)

def test_definition_of_the_row_against_first_principles():
    """quantise64 on rows whose codes are known: grid values come back, midpoints go to the even code."""
    import torch
    v = e4m3_values()
    grid = v[:127]
    row = np.zeros((4, ROW))
    row[0, :127] = grid                                    # 448 is the largest: k = 0
    row[1, :126] = (grid[1:] + grid[:-1]) / 2              # midpoints of neighbouring codes
    row[1, 200] = 448.0
    row[2, 0], row[2, 512:] = 449.0, 3.0                   # just above 448: k = 1
    codes, rope, scale = (x.numpy() for x in quantise64(torch.from_numpy(row)))
    assert list(codes[0, :127]) == list(range(127)) and scale[0] == 1.0
    assert all(c % 2 == 0 for c in codes[1, :126]) and scale[1] == 1.0
    assert scale[2] == 2.0 and v[codes[2, 0]] == 224.0 and (rope[2] == 1.5).all()
    assert scale[3] == 2.0 ** -60 and not codes[3].any()
    assert np.abs(v[codes[0]] * scale[0] - row[0, :512]).max() == 0


# ------------------------------------------------------------------ refusals (no kernel is launched)

@pytest.fixture(scope="module")
def L():
    build.build()
    return B.lib()


P = ctypes.c_void_p
FAKE, ODD, NIL = P(1 << 20), P((1 << 20) + 2), P(0)


def _calls(L, **kw):
    """The four entry points with good host arguments, some of them replaced."""
    a = dict(rows=FAKE, ld=576, T=4, cu=FAKE, sl=FAKE, pt=FAKE, B=2, mp=8, kv8=FAKE, ks=FAKE, np=16, ps=64, start=FAKE,
             kv=FAKE, cr=1000, q=FAKE, idx=FAKE, topk=64, scale=0.0625, o=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    plan = (a["cu"], a["sl"], a["pt"], a["B"], a["mp"])
    cache = (a["kv8"], a["ks"], a["np"], a["ps"])
    out = (ctypes.c_float(a["scale"]), a["o"], a["lse"], a["ws"], a["wsb"], NIL)
    return dict(
        write=lambda: L.dsa_cache_write(a["rows"], a["ld"], a["T"], *plan, *cache, NIL),
        read=lambda: L.dsa_cache_read(*cache, a["sl"], a["pt"], a["B"], a["mp"], a["start"], a["kv"], a["cr"], NIL),
        attn=lambda: L.dsa_paged_mla_attn(a["q"], a["T"], *plan, *cache, *out),
        sparse=lambda: L.dsa_paged_sparse_mla_attn(a["q"], a["T"], *plan, a["idx"], a["topk"], *cache, *out))


ALL = ("write", "read", "attn", "sparse")


@pytest.mark.parametrize("which,bad", [
    (ALL, dict(B=-1)), (ALL, dict(mp=0)), (ALL, dict(np=0)), (ALL, dict(ps=0)), (ALL, dict(np=1 << 20, ps=1 << 12)),
    (ALL, dict(kv8=NIL)), (ALL, dict(kv8=P((1 << 20) + 8))), (ALL, dict(ks=NIL)), (ALL, dict(pt=NIL)),
    (ALL, dict(pt=ODD)), (ALL, dict(sl=NIL)),
    (("write", "attn", "sparse"), dict(T=-1)), (("write", "attn", "sparse"), dict(cu=NIL)),
    (("write",), dict(rows=NIL)), (("write",), dict(rows=ODD)), (("write",), dict(ld=575)), (("write",), dict(ld=580)),
    (("read",), dict(start=NIL)), (("read",), dict(kv=NIL)), (("read",), dict(kv=ODD)), (("read",), dict(cr=0)),
    (("attn", "sparse"), dict(q=NIL)), (("attn", "sparse"), dict(q=ODD)), (("attn", "sparse"), dict(o=NIL)),
    (("attn", "sparse"), dict(lse=ODD)), (("attn", "sparse"), dict(scale=0.0)),
    (("attn", "sparse"), dict(scale=float("nan"))), (("attn", "sparse"), dict(T=1 << 26)),
    (("sparse",), dict(topk=0)), (("sparse",), dict(topk=2049)), (("sparse",), dict(idx=NIL)),
    (("sparse",), dict(idx=ODD)), (("attn", "sparse"), dict(ws=NIL)), (("attn", "sparse"), dict(ws=P((1 << 20) + 128))),
], ids=str)
def test_host_arguments_are_refused(L, which, bad):
    calls = _calls(L, **bad)
    for name in which:
        assert calls[name]() == B.DSA_ERR_INVALID_ARG, name
        assert B.last_error() != ""


def test_workspace_is_checked_and_bounded(L):
    for name, topk in (("attn", 0), ("sparse", 64)):
        need = B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 4, 8 * 64, topk)
        assert need > 0 and need % 256 == 0
        assert _calls(L, wsb=need - 1)[name]() == B.DSA_ERR_WORKSPACE and B.last_error() != ""
    # partial results are a matter of the machine, not of the batch: the size stops growing with either
    big = B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 1 << 16, 1 << 20, 0)
    assert big == B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 1 << 20, 1 << 30, 0) < 48 << 20
    assert B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 1, 128, 0) < B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 1, 129, 0)
    assert B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 0, 128, 0) == 0


def test_empty_batches_are_no_ops(L):
    for kw in (dict(T=0), dict(B=0, cu=NIL, sl=NIL, pt=NIL, kv8=NIL, ks=NIL)):
        calls = _calls(L, **kw)
        for name in ALL if "B" in kw else ("write", "attn", "sparse"):
            assert calls[name]() == B.DSA_OK, name


def test_binding_refuses_wrong_tensors(L):
    """On CPU tensors: whatever is wrong is found before a pointer is taken."""
    import torch
    i32 = torch.zeros(3, dtype=torch.int32)
    kv8, sc = torch.zeros(4, 8, ROW8, dtype=torch.uint8), torch.zeros(4, 8)
    with pytest.raises(TypeError):
        B.dsa_cache_write(torch.zeros(2, ROW, dtype=torch.bfloat16), i32, i32[:2], i32.view(1, 3), kv8, sc)
    with pytest.raises(TypeError):
        B.dsa_cache_read(kv8, sc, i32, i32.view(3, 1), i32.long(), torch.zeros(9, ROW, dtype=torch.bfloat16))


# ------------------------------------------------------------------ write and read (GPU)

def special_rows(r, n):
    """Ordinary rows, with the values at which a quantiser goes wrong in the first ones."""
    x = r.standard_normal((n, ROW)) * np.exp(2 * r.standard_normal((n, 1)))
    grid = e4m3_values()[:127]
    rows = [np.zeros(ROW), np.concatenate([grid, -grid, np.zeros(ROW - 254)]),
            np.concatenate([(grid[1:] + grid[:-1]) / 2, [448.0], np.ones(ROW - 127)]),
            np.full(ROW, 449.0), np.full(ROW, 448.0), np.full(ROW, 1e-38), np.full(ROW, -3e38),
            x[0] * 2.0 ** -70, x[0] * 2.0 ** 66]
    rows[6][512:] = 1.0                       # its rope half is divided by 2^60
    rows[5][512:] = 2.0 ** -40
    rows[7][512:], rows[8][512:] = 0.0, 1.0
    for i, v in enumerate(rows[:n]):
        x[i] = v
    return x


def nonfinite_rows(r, n):
    x = r.standard_normal((n, ROW))
    x[0, 5], x[0, 100], x[0, 101] = np.nan, np.inf, -np.inf
    x[1 % n, :512] = np.inf
    x[2 % n, 520] = np.nan
    return x


WRITES = [  # new tokens, lengths, page size, spare query rows
    ([1], [1], 1, 0), ([1], [1000], 7, 3), ([5], [5], 64, 0), ([1, 0, 3, 2], [130, 0, 3, 77], 16, 2),
    ([0, 0], [5, 0], 8, 1), ([200, 1, 33], [200, 5000, 40], 50, 0), ([1] * 70, list(range(1, 71)), 3, 0),
    ([2] * 1100, [2 + i % 5 for i in range(1100)], 4, 5),
]


@pytest.mark.gpu
@pytest.mark.parametrize("values", [None, special_rows, nonfinite_rows], ids=["normal", "special", "nonfinite"])
@pytest.mark.parametrize("ld", [ROW, 600])
@pytest.mark.parametrize("new,lens,page,pad", WRITES, ids=range(len(WRITES)))
def test_write(new, lens, page, pad, ld, values):
    import torch
    c = Batch(new, lens, page, seed=1, pad=pad)
    r = np.random.default_rng(2)
    make = values or (lambda r, n: r.standard_normal((n, ROW)))
    x = torch.from_numpy(make(r, max(c.T, 1)).astype(np.float32)).to(torch.bfloat16).cuda()[:c.T]
    wide = torch.full((c.T, ld), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :ROW] = x
    want8, want_scale = c.kv8.clone().view(-1, ROW8), c.kv_scale.clone().view(-1)
    t = 0
    for b, (n, m) in enumerate(zip(new, lens)):
        if n:
            codes, rope, scale = quantise64(x[t:t + n].double())
            at = torch.from_numpy(c.slots(b, np.arange(m - n, m))).cuda()
            want8[at] = torch.cat([codes, rope.to(torch.bfloat16).view(torch.uint8)], 1)
            want_scale[at] = scale.float()
        t += n
    B.dsa_cache_write(wide[:, :ROW], *c.plan, c.kv8, c.kv_scale)
    B.dsa_sync_status()
    assert torch.equal(c.kv_scale.view(-1), want_scale)
    got, want = c.kv8.view(-1, ROW8), want8
    # a NaN has several codes and patterns; everything else has to agree bit for bit
    nan_g, nan_w = got[:, :LATENT] & 127 == 127, want[:, :LATENT] & 127 == 127
    assert torch.equal(nan_g, nan_w)
    assert torch.equal(got[:, :LATENT][~nan_g], want[:, :LATENT][~nan_w])
    rg, rw = (z[:, LATENT:].contiguous().view(torch.bfloat16) for z in (got, want))
    assert torch.equal(rg.isnan(), rw.isnan())
    assert torch.equal(rg[~rg.isnan()], rw[~rw.isnan()])


@pytest.mark.gpu
@pytest.mark.parametrize("values", [None, special_rows], ids=["normal", "special"])
@pytest.mark.parametrize("lens,page", [([1], 1), ([0], 8), ([777], 16), ([0, 130, 0, 1, 64, 0], 16), ([5000, 3], 50),
                                       (list(range(300)), 7), ([1] * 2000, 5)], ids=range(7))
def test_read(lens, page, values):
    import torch
    c = Batch([0] * len(lens), lens, page, seed=3, values=values)
    gap = 2
    start = np.cumsum([gap] + [m + gap for m in lens])[:-1]
    kv = torch.full((int(start[-1] + lens[-1] + gap), ROW), 5.0, dtype=torch.bfloat16, device="cuda")
    want = kv.double()
    for b, m in enumerate(lens):
        if m:
            want[start[b]:start[b] + m] = c.values(b, m)
    want16 = want.to(torch.bfloat16)
    lat = want[:, :LATENT]
    tiny = lat.abs() < 2.0 ** -126                          # bf16's subnormal values have fewer bits
    assert torch.equal(want16[:, :LATENT].double()[~tiny], lat[~tiny])   # a code times its power of two needs no rounding
    B.dsa_cache_read(c.kv8, c.kv_scale, c.seq_len, c.page_table, torch.from_numpy(start).cuda(), kv)
    B.dsa_sync_status()
    assert torch.equal(kv, want16)


# ------------------------------------------------------------------ attention (GPU)

ATTN = [  # new tokens, lengths, page size, spare query rows
    ([1], [1], 1, 0), ([1], [300], 16, 0), ([1], [127], 64, 2), ([1], [128], 64, 0), ([1], [129], 64, 0),
    ([1], [20000], 64, 0), ([3], [3], 7, 1), ([130], [130], 128, 0), ([17], [1000], 50, 0),
    ([1, 0, 6, 2, 0], [1000, 0, 6, 513, 40], 16, 3), ([1] * 64, [1 + 37 * i for i in range(64)], 32, 0),
    ([1] * 400, [1 + i % 300 for i in range(400)], 24, 0), ([2, 200], [9000, 700], 200, 0),
    ([1] * 1500, [1 + i % 7 for i in range(1500)], 8, 2),
]


def large_logits(r, n):
    """Scores up to some hundreds, largest late in the sequence: the running maximum moves on many times."""
    return r.standard_normal((n, ROW)) * np.linspace(1, 12, n)[:, None]


def unlike_scales(r, n):
    """Tokens whose sizes differ by many powers of two."""
    return r.standard_normal((n, ROW)) * 2.0 ** r.integers(-30, 4, (n, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("values", [None, large_logits, unlike_scales], ids=["normal", "large", "scales"])
@pytest.mark.parametrize("new,lens,page,pad", ATTN, ids=range(len(ATTN)))
def test_dense_attention(new, lens, page, pad, values):
    c = Batch(new, lens, page, seed=4, pad=pad, values=values)
    o, lse = c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * page, 0)
    B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, SCALE, o, lse, ws)
    B.dsa_sync_status()
    check_attention(c, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("holes", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("topk", [1, 64, 129, 2048])
@pytest.mark.parametrize("new,lens,page,pad", [ATTN[i] for i in (0, 1, 6, 8, 9, 10, 12)], ids=range(7))
def test_selected_attention(new, lens, page, pad, topk, holes):
    import torch
    c = Batch(new, lens, page, seed=5, pad=pad)
    idx = selection(c, topk, seed=6, holes=holes)
    o, lse = c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * page, topk)
    B.dsa_paged_sparse_mla_attn(c.q, *c.plan, torch.from_numpy(idx).cuda(), c.kv8, c.kv_scale, SCALE, o, lse, ws)
    B.dsa_sync_status()
    check_attention(c, o, lse, idx)


def run_dense(c, out=None):
    o, lse = out or c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, max(c.T, 1), c.table.shape[1] * c.page, 0)
    B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, SCALE, o, lse, ws)
    return o, lse


def run_selected(c, idx, out=None):
    import torch
    o, lse = out or c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * c.page, idx.shape[1])
    B.dsa_paged_sparse_mla_attn(c.q, *c.plan, torch.from_numpy(idx).cuda(), c.kv8, c.kv_scale, SCALE, o, lse, ws)
    return o, lse


# ------------------------------------------------------------------ what must not be read, and what must be seen

@pytest.mark.gpu
def test_unseen_rows_may_hold_anything():
    """NaN codes, scales and rope values in every cache row that no position maps to, and in the positions of a chunk
    that a query row does not see yet."""
    import torch
    c = Batch([3, 130, 1], [200, 300, 129], 50, seed=7)
    used = np.concatenate([c.slots(b, np.arange(m)) for b, m in enumerate(c.lens)])
    rest = torch.from_numpy(np.setdiff1d(np.arange(c.n_pages * c.page), used)).cuda()
    c.kv8.view(-1, ROW8)[rest] = 0x7f
    c.kv8.view(-1, ROW8)[rest, LATENT:] = torch.full((ROW8 - LATENT,), 0xff, dtype=torch.uint8, device="cuda")
    c.kv_scale.view(-1)[rest] = float("nan")
    o, lse = run_dense(c)
    B.dsa_sync_status()
    check_attention(c, o, lse)
    idx = selection(c, 129, seed=8, holes=0.3)
    o, lse = run_selected(c, idx)
    B.dsa_sync_status()
    check_attention(c, o, lse, idx)
    # the last token of the second sequence: only its own query row sees it
    last = int(c.slots(1, 299))
    c.kv8.view(-1, ROW8)[last, :LATENT] = 0x7f
    o2, lse2 = run_dense(c)
    B.dsa_sync_status()
    row = int(c.cu[2]) - 1
    assert bool(o2[row].isnan().all()) and bool(lse2[row].isnan().all())
    keep = [t for t in range(c.T) if t != row]
    assert not bool(o2[keep].isnan().any()) and not bool(lse2[keep].isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dim", [3, 300, 540])
def test_a_nonfinite_query_value_stays_in_its_head(bad, dim):
    """Two of the heads hold one; the row is split over CTAs, so the merge carries it too."""
    import torch
    c = Batch([1, 2], [3000, 90], 16, seed=9)
    good, good_lse = run_dense(c)
    c.q[0, 5, dim] = bad
    c.q[2, 63, dim] = bad
    o, lse = run_dense(c)
    B.dsa_sync_status()
    for t, h in ((0, 5), (2, 63)):
        assert bool(o[t, h].isnan().all()) and bool(lse[t, h].isnan())
        o[t, h], lse[t, h] = good[t, h], good_lse[t, h]
    assert torch.equal(o, good) and torch.equal(lse, good_lse)


@pytest.mark.gpu
def test_rows_that_see_nothing_ignore_their_query():
    """An all-empty selection gives 0 and -inf, NaN queries or not; so does one empty tile beside a full one."""
    c = Batch([2, 1], [400, 300], 16, seed=19)
    idx = selection(c, 256, seed=20)
    idx[0] = -1
    idx[2, :128] = -1
    c.q[0] = float("nan")
    o, lse = run_selected(c, idx)
    B.dsa_sync_status()
    c.q[0] = 0
    check_attention(c, o, lse, idx)


@pytest.mark.gpu
def test_large_and_small_queries():
    """Heads of one row whose queries differ by many powers of two, and an all-zero one (the mean of the values)."""
    import torch
    c = Batch([1, 1], [700, 50], 16, seed=10)
    c.q[0] *= torch.exp2(torch.arange(64, device="cuda").float() - 40)[:, None].bfloat16()
    c.q[0, 7] = 0
    c.q[0, 8, :512] = 0
    o, lse = run_dense(c)
    B.dsa_sync_status()
    check_attention(c, o, lse)


@pytest.mark.gpu
def test_a_position_selected_twice_counts_twice():
    c = Batch([1, 2], [300, 90], 16, seed=21)
    idx = selection(c, 200, seed=22)
    idx[0, 100:110] = idx[0, 3]
    idx[2, 50:] = idx[2, 49]
    o, lse = run_selected(c, idx)
    B.dsa_sync_status()
    check_attention(c, o, lse, idx)


@pytest.mark.gpu
@pytest.mark.parametrize("new, lens", [
    ([1] * 64, [100 + 9 * b for b in range(64)]),                  # whole rows: one of up to six tiles a CTA
    ([1] * 150, [130 + 2 * b for b in range(150)]),                # more rows than CTAs
    ([3] * 110, [5 + 3 * b for b in range(110)]),                  # several short rows a CTA
    ([1] * 20 + [0, 0] + [1] * 20, [300] * 20 + [0, 77] + [500] * 20),
    ([1, 1, 1] + [1] * 60, [6000, 129, 128] + [20] * 60),          # long and short ones: split
    ([40, 0, 1, 90], [4000, 3, 2500, 700]),
])
def test_rows_shared_out_over_the_ctas(new, lens):
    c = Batch(new, lens, 32, seed=25)
    o, lse = run_dense(c)
    B.dsa_sync_status()
    check_attention(c, o, lse)
    for topk in (100, 256, 900):
        idx = selection(c, topk, seed=topk, holes=0.1)
        o, lse = run_selected(c, idx)
        B.dsa_sync_status()
        check_attention(c, o, lse, idx)


@pytest.mark.gpu
def test_sequences_may_share_pages():
    """A common prefix of four pages, read by both sequences."""
    import torch
    c = Batch([2, 1], [400, 300], 64, seed=23)
    c.table[1, :4] = c.table[0, :4]
    c.page_table = torch.from_numpy(c.table).cuda()
    o, lse = run_dense(c)
    B.dsa_sync_status()
    check_attention(c, o, lse)


@pytest.mark.gpu
def test_query_rows_before_the_first_sequence():
    """cu_q may begin behind row 0: the rows before it belong to no sequence."""
    import torch
    c = Batch([1, 2], [40, 50], 16, seed=24)
    want = run_dense(c)
    front = torch.full_like(c.q[:2], 3.0)
    c.q, c.cu_q, c.T = torch.cat([front, c.q]), c.cu_q + 2, c.T + 2
    o, lse = run_dense(c)
    B.dsa_sync_status()
    assert bool((o[:2] == 7.0).all()) and bool((lse[:2] == 7.0).all())
    c.q = c.q[2:]
    check_attention(c, o[2:], lse[2:])
    check_attention(c, *want)
    before = c.kv8.clone(), c.kv_scale.clone()
    at = torch.from_numpy(np.concatenate([c.slots(0, [39]), c.slots(1, [48, 49])])).cuda()
    c.kv8.view(-1, ROW8)[at] = 0
    c.kv_scale.view(-1)[at] = 0
    rows = torch.cat([torch.full((2, ROW), 9.0, dtype=torch.bfloat16, device="cuda"), c.rows[at]])
    B.dsa_cache_write(rows, *c.plan, c.kv8, c.kv_scale)
    B.dsa_sync_status()
    assert torch.equal(c.kv8, before[0]) and torch.equal(c.kv_scale, before[1])


# ------------------------------------------------------------------ rows and pages that do not fit

def bad_status(fn):
    with pytest.raises(B.DSAError) as e:
        fn()
        B.dsa_sync_status()
    assert e.value.code == B.DSA_ERR_BAD_ROW


@pytest.mark.gpu
def test_pages_outside_the_cache_are_skipped():
    import torch
    for page in (-1, 1 << 30):
        c = Batch([1, 1], [100, 40], 16, seed=11)
        lost = np.arange(32, 48)                                     # positions of sequence 0's third page
        c.page_table[0, 2] = page
        out = c.outputs()
        bad_status(lambda: run_dense(c, out))
        idx = np.full((2, 128), -1, np.int32)
        idx[0, :84] = np.setdiff1d(np.arange(100), lost)
        idx[1, :40] = np.arange(40)
        check_attention(c, *out, idx)                                # as if they were not there
        start = torch.tensor([0, 100], device="cuda")
        kv = torch.full((140, ROW), 5.0, dtype=torch.bfloat16, device="cuda")
        bad_status(lambda: B.dsa_cache_read(c.kv8, c.kv_scale, c.seq_len, c.page_table, start, kv))
        assert bool((kv[32:48] == 5.0).all()) and not bool((kv[:32] == 5.0).all(1).any())
        before = c.kv8.clone()
        c.page_table[0, 6] = page                                    # where sequence 0's new token goes
        bad_status(lambda: B.dsa_cache_write(c.rows[:2], *c.plan, c.kv8, c.kv_scale))
        changed = (c.kv8 != before).any(2).view(-1).nonzero().flatten().cpu().tolist()
        assert changed == [int(c.slots(1, 39))]


@pytest.mark.gpu
def test_lengths_that_do_not_fit():
    """Longer than the page table, shorter than the new tokens, negative: those rows see nothing and are not written; the
    others are as they should be."""
    import torch
    for wrong, blind in ((-5, 3), (0, 3), (2, 1), (1 << 30, 3)):
        c = Batch([2, 3, 1], [50, 60, 70], 16, seed=12)
        c.seq_len[1] = wrong
        out = c.outputs()
        bad_status(lambda: run_dense(c, out))
        o, lse = out
        assert bool((o[2:2 + blind] == 0).all()) and bool(torch.isinf(lse[2:2 + blind]).all())
        c.lens[1] = wrong if blind == 1 else 0
        ro, rl, to, tl = c.reference()
        # (with two positions for three new tokens, the last two stand at positions 0 and 1)
        for t in [0, 1, 5] + ([3, 4] if blind == 1 else []):
            assert bool(((o[t].double() - ro[t]).abs() <= to[t]).all())
            assert bool(((lse[t].double() - rl[t]).abs() <= tl[t]).all())
        before = c.kv8.clone()
        bad_status(lambda: B.dsa_cache_write(c.rows[:6], *c.plan, c.kv8, c.kv_scale))
        changed = set((c.kv8 != before).any(2).view(-1).nonzero().flatten().cpu().tolist())
        want = {int(c.slots(0, 48)), int(c.slots(0, 49)), int(c.slots(2, 69))}
        assert changed == want | ({int(c.slots(1, 0)), int(c.slots(1, 1))} if blind == 1 else set())
        if wrong != 2 and wrong != 0:
            kv = torch.full((300, ROW), 5.0, dtype=torch.bfloat16, device="cuda")
            start = torch.tensor([0, 60, 130], device="cuda")
            bad_status(lambda: B.dsa_cache_read(c.kv8, c.kv_scale, c.seq_len, c.page_table, start, kv))
            assert bool((kv[60:130] == 5.0).all()) and not bool((kv[:50] == 5.0).all(1).any())


@pytest.mark.gpu
@pytest.mark.parametrize("start", [-1, 999, 1 << 40])
def test_flat_rows_outside_the_destination(start):
    import torch
    c = Batch([0, 0], [20, 30], 16, seed=13)
    kv = torch.full((1000, ROW), 5.0, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([start, 100], device="cuda")
    bad_status(lambda: B.dsa_cache_read(c.kv8, c.kv_scale, c.seq_len, c.page_table, at, kv))
    assert bool((kv[:100] == 5.0).all()) and bool((kv[130:] == 5.0).all())
    assert torch.equal(kv[100:130], c.values(1, 30).bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 3, 1, 4], [0, 2, 1 << 30, 4], [-2, 1, 2, 4]])
def test_query_rows_out_of_order(cu):
    """Only that nothing is read or written where it should not be: the sequences that are in order come out."""
    import torch
    c = Batch([2, 1, 1], [50, 60, 70], 16, seed=14)
    c.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    bad_status(lambda: run_dense(c))
    before = c.kv8.clone()
    bad_status(lambda: B.dsa_cache_write(c.rows[:4], *c.plan, c.kv8, c.kv_scale))
    changed = set((c.kv8 != before).any(2).view(-1).nonzero().flatten().cpu().tolist())
    allowed = {int(s) for b, m in enumerate(c.lens) for s in c.slots(b, np.arange(m))}
    assert changed <= allowed


@pytest.mark.gpu
def test_selected_positions_out_of_sight():
    c = Batch([2], [100], 16, seed=15)
    idx = selection(c, 64, seed=16)
    idx[0, 3], idx[0, 9], idx[1, 63] = 99, 1 << 30, 100               # row 0 sees 0 .. 98, row 1 0 .. 99
    out = c.outputs()
    bad_status(lambda: run_selected(c, idx, out))
    idx[idx >= 99] = -1
    full = idx.copy()
    check_attention(c, *out, full)


# ------------------------------------------------------------------ together, captured, elsewhere

@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 50])
def test_a_step_through_all_four(page):
    """New tokens are written, attended to densely and by selection; the cache is read back, and the flat kernels give the
    same on the rows that come out."""
    import torch
    c = Batch([2, 1, 5], [400, 1, 3000], page, seed=17)
    new = torch.randn(c.T, ROW, device="cuda").bfloat16()
    B.dsa_cache_write(new, *c.plan, c.kv8, c.kv_scale)
    o, lse = run_dense(c)
    idx = selection(c, 256, seed=18)
    o_s, lse_s = run_selected(c, idx)
    start = torch.tensor([0, 400, 401], device="cuda")
    kv = torch.empty(sum(c.lens), ROW, dtype=torch.bfloat16, device="cuda")
    B.dsa_cache_read(c.kv8, c.kv_scale, c.seq_len, c.page_table, start, kv)
    rows = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(c.new, device="cuda"))
    o_f = torch.empty(c.T, HEADS, LATENT, device="cuda")
    lse_f = torch.empty(c.T, HEADS, device="cuda")
    B.dsa_sparse_mla_attn(c.q, kv, start[rows].contiguous(), torch.from_numpy(idx).cuda(), SCALE, o_f, lse_f)
    B.dsa_sync_status()
    check_attention(c, o, lse)
    check_attention(c, o_s, lse_s, idx)
    # the flat kernel rounds its probabilities to bf16, 2^-8, and its sums take the rounded ones
    assert float((lse_f - lse_s).abs().max()) < 2.0 ** -8 + 1e-4
    assert float((o_f - o_s.float()).norm() / o_f.norm()) < 2 * 2.0 ** -8


@pytest.mark.gpu
def test_captured_graphs_share_a_workspace():
    """Two graphs over one workspace, replayed in turn on new inputs, lengths and pages."""
    import torch
    a, b = Batch([1] * 8, [900 + 7 * i for i in range(8)], 16, seed=20), Batch([3, 4], [2000, 77], 50, seed=21)
    ws = torch.empty(48 << 20, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for c in (a, b):
        o, lse = c.outputs()
        run = lambda: B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, SCALE, o, lse, ws)  # noqa: E731,B023
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        outs.append((o, lse))
        graphs.append(g)
    for seed in (22, 23):
        a2, b2 = Batch(a.new, [700 + 11 * i for i in range(8)], 16, seed=seed, width=a.table.shape[1], spare=a.n_pages), \
            Batch(b.new, [1500, 60], 50, seed=seed + 50, width=b.table.shape[1], spare=b.n_pages)
        for c, n, (o, lse) in ((a, a2, outs[0]), (b, b2, outs[1])):
            P_ = c.n_pages
            keep = torch.from_numpy((n.table >= P_) & (n.table < 1 << 30)).cuda()
            n.page_table[keep] %= P_
            n.table = n.page_table.cpu().numpy()
            used = n.table[n.table < 1 << 30]
            if len(set(used.tolist())) < len(used):                   # two of them fell together: place them apart
                fresh = iter(np.random.default_rng(seed).permutation(P_))
                n.table = np.where(n.table < 1 << 30, -1, n.table)
                n.table[n.table == -1] = [next(fresh) for _ in range(len(used))]
                n.page_table = torch.from_numpy(n.table).cuda()
            c.q.copy_(n.q)
            c.seq_len.copy_(n.seq_len)
            c.page_table.copy_(n.page_table)
            c.lens, c.table = n.lens, n.table
            o.fill_(7.0)
            lse.fill_(7.0)
        for g in graphs:
            g.replay()
        graphs[0].replay()
        B.dsa_sync_status()
        check_attention(a, *outs[0])
        check_attention(b, *outs[1])


@pytest.mark.gpu
def test_on_another_stream_the_calls_follow_each_other():
    """Write and both attentions on a side stream, right behind each other; the same twice, bit for bit."""
    import torch
    c = Batch([1, 4], [2500, 600], 16, seed=24)
    new = torch.randn(c.T, ROW, device="cuda").bfloat16()
    idx = selection(c, 300, seed=25)
    idx_d = torch.from_numpy(idx).cuda()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * c.page, 0)
    outs = [c.outputs() for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(2):
        B.dsa_cache_write(new, *c.plan, c.kv8, c.kv_scale, stream=side)
        B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, SCALE, *outs[2 * k], ws, stream=side)
        B.dsa_paged_sparse_mla_attn(c.q, *c.plan, idx_d, c.kv8, c.kv_scale, SCALE, *outs[2 * k + 1], ws, stream=side)
    B.dsa_sync_status(side)
    check_attention(c, *outs[0])
    check_attention(c, *outs[1], idx)
    for x, y in zip(outs[0] + outs[1], outs[2] + outs[3]):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams, a workspace each, with nothing between them: what each gives alone, bit for bit."""
    import torch
    cs = [Batch([1] * 40, [1500 + 20 * b for b in range(40)], 16, seed=27), Batch([60, 3], [900, 4000], 64, seed=28)]
    picks = [torch.from_numpy(selection(c, 700, seed=29)).cuda() for c in cs]
    ws = [B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * c.page, 0) for c in cs]

    def calls(k, outs, stream):
        c = cs[k]
        B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, SCALE, *outs[0], ws[k], stream=stream)
        B.dsa_paged_sparse_mla_attn(c.q, *c.plan, picks[k], c.kv8, c.kv_scale, SCALE, *outs[1], ws[k], stream=stream)

    alone = [[c.outputs(), c.outputs()] for c in cs]
    for k in range(2):
        calls(k, alone[k], None)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    both = [[[c.outputs(), c.outputs()] for c in cs] for _ in range(4)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for outs in both:
        for k in (0, 1):
            calls(k, outs[k], streams[k])
    for st in streams:
        B.dsa_sync_status(st)
    for outs in both:
        for k in range(2):
            for got, want in zip(outs[k], alone[k]):
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_cache_larger_than_32_bit_offsets():
    """A sequence in the last pages of a cache of more than 2^32 bytes."""
    import torch
    c = Batch([2], [500], 64, seed=26)
    pages = (1 << 32) // (64 * ROW8) + 200
    kv8 = torch.empty(pages, 64, ROW8, dtype=torch.uint8, device="cuda")
    scale = torch.empty(pages, 64, device="cuda")
    shift = pages - c.n_pages
    kv8[shift:] = c.kv8
    scale[shift:] = c.kv_scale
    table = torch.from_numpy(np.where(c.table < 1 << 30, c.table + shift, -1).astype(np.int32)).cuda()
    o, lse = c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * 64, 0)
    B.dsa_paged_mla_attn(c.q, c.cu_q, c.seq_len, table, kv8, scale, SCALE, o, lse, ws)
    kv = torch.empty(500, ROW, dtype=torch.bfloat16, device="cuda")
    B.dsa_cache_read(kv8, scale, c.seq_len, table, torch.zeros(1, dtype=torch.int64, device="cuda"), kv)
    B.dsa_sync_status()
    check_attention(c, o, lse)
    assert torch.equal(kv, c.values(0, 500).bfloat16())
    new = torch.randn(2, ROW, device="cuda").bfloat16()
    B.dsa_cache_write(new, c.cu_q, c.seq_len, table, kv8, scale)
    B.dsa_cache_write(new, c.cu_q, c.seq_len, c.page_table, c.kv8, c.kv_scale)
    B.dsa_sync_status()
    assert torch.equal(kv8[shift:], c.kv8) and torch.equal(scale[shift:], c.kv_scale)


CHILD = r"""
import sys
sys.path[:0] = [ROOT, ROOT + "/tests"]
import torch
from indexer_selected_sparse_dsa_b200 import binding as B
from paged_util import Batch, check_attention, selection
from test_paged_cache import run_dense, run_selected
c = Batch([1, 6, 2], [3000, 700, 90], 16, seed=30)
idx = selection(c, 300, seed=31)
def status(fn):
    try:
        fn()
        B.dsa_sync_status()
        return "OK"
    except B.DSAError as e:
        return {B.DSA_ERR_TIMEOUT: "TIMEOUT"}.get(e.code, str(e))
B.dsa_set_wait_limit_ns(1)
got = [status(lambda: run_dense(c)), status(lambda: run_selected(c, idx))]
B.dsa_set_wait_limit_ns(0)
check_attention(c, *run_dense(c))
check_attention(c, *run_selected(c, idx), idx)
got.append(status(lambda: None))
print("RESULT", *got, flush=True)
"""


@pytest.mark.gpu
def test_waits_give_up_and_leave_the_context_usable():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\n" + CHILD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "RESULT TIMEOUT TIMEOUT OK" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
