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
    (("sparse",), dict(idx=ODD)),
], ids=str)
def test_host_arguments_are_refused(L, which, bad):
    calls = _calls(L, **bad)
    for name in which:
        assert calls[name]() == B.DSA_ERR_INVALID_ARG, name
        assert B.last_error() != ""


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
