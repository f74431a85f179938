"""Paged latent cache and attention: values, plans and calls at the edges of what their description allows."""
import math

import numpy as np
import pytest

from indexer_selected_sparse_dsa_b200 import binding as B
from paged_util import HEADS, LATENT, ROW, ROW8, SCALE, Batch, check_attention, quantise64, selection
from test_paged_cache import bad_status, run_dense, run_selected


def put(c, b, pos, rows):
    """Store latent rows (64-bit, bf16 values) at positions `pos` of sequence b, as dsa_cache_write does."""
    import torch
    codes, rope, scale = quantise64(rows)
    at = torch.from_numpy(c.slots(b, pos)).cuda()
    c.kv8.view(-1, ROW8)[at] = torch.cat([codes, rope.to(torch.bfloat16).view(torch.uint8)], 1)
    c.kv_scale.view(-1)[at] = scale.float()


# ------------------------------------------------------------------ scales far apart

@pytest.mark.gpu
@pytest.mark.parametrize("gap", [2.0, 8.0, 16.0])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n", [100, 1000, 6000])
def test_rows_of_the_largest_and_the_smallest_scale(n, first, gap):
    """One position of scale 2^60 and many zero rows (2^-60), whose scores are `gap` below its own: together they weigh as
    much as the softmax says.  What is looked at: o = p v and lse.  The scores come from the rope half alone (the latent
    half of the query is 0, its products are exact), so besides the sums, 2^-17 of them, what is rounded is the
    probability, 2^-11, and the result, 2^-8."""
    import torch
    c = Batch([1], [n], 16, seed=41)
    one = 0 if first else n - 1
    rows = torch.zeros(n, ROW, dtype=torch.float64, device="cuda")
    rows[one, :LATENT] = 448.0 * 2.0 ** 60
    rows[one, 100:LATENT] = 32.0 * 2.0 ** 60
    rows[one, LATENT] = 1.0
    put(c, 0, np.arange(n), rows)
    assert set(c.kv_scale.view(-1)[torch.from_numpy(c.slots(0, np.arange(n))).cuda()].tolist()) == {2.0 ** 60, 2.0 ** -60}
    c.q[:, :, :] = 0
    c.q[:, :, LATENT] = gap / SCALE
    o, lse = run_dense(c)
    B.dsa_sync_status()
    x = torch.zeros(n, dtype=torch.float64)
    x[one] = gap
    want = torch.softmax(x, 0)[one].item() * rows[one, :LATENT]
    e = 2.0 ** -16 * gap + 2.0 ** -20
    assert bool(((o[0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 + 2 * e) * want.abs()).all())
    assert float((lse[0].double() - torch.logsumexp(x, 0).item()).abs().max()) <= e + 2.0 ** -16


# ------------------------------------------------------------------ infinite rope values

@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[300], [3000], [129, 700], [90]])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_an_infinite_rope_value_weighs_nothing_where_its_score_is_minus_infinity(lens, bad):
    """Heads whose product with it is -inf give its position the weight 0, as the softmax does; the others, +inf, have no
    finite result.  The row is the highest of the cache in its tile, the one that places without a key read too."""
    import torch
    c = Batch([1] * len(lens), lens, 16, seed=40)
    c.q[:, :, LATENT:] = torch.where(c.q[:, :, LATENT:] == 0, 1, c.q[:, :, LATENT:])
    idx = np.full((c.T, max(lens)), -1, np.int32)
    for b, m in enumerate(lens):
        tile = np.arange((m - 1) // 128 * 128, m)
        hit = int(tile[np.argmax(c.slots(b, tile))])
        c.kv8.view(-1, ROW8)[int(c.slots(b, hit)), LATENT:].view(torch.bfloat16)[9 + b] = bad
        idx[b, :m - 1] = np.delete(np.arange(m), hit)
    ro, rl, to, tl = c.reference(idx)                                 # without that position
    wide = np.full((c.T, max(lens) + 40), -1, np.int32)               # with it, and with empty slots
    for b, m in enumerate(lens):
        wide[b, 20:20 + m] = np.arange(m)
    for o, lse in (run_dense(c), run_selected(c, wide) if wide.shape[1] <= 2048 else run_dense(c)):
        B.dsa_sync_status()
        for t in range(c.T):
            gone = (torch.sign(c.q[t, :, LATENT + 9 + t].float()) * bad) < 0
            assert 0 < int(gone.sum()) < HEADS
            assert bool(((o[t].double() - ro[t]).abs() <= to[t])[gone].all())
            assert bool(((lse[t].double() - rl[t]).abs() <= tl[t])[gone].all())
            assert not bool(o[t, ~gone].isfinite().any()) and not bool(lse[t, ~gone].isfinite().any())


# ------------------------------------------------------------------ plans that do not fit

@pytest.mark.gpu
def test_a_sequence_whose_rows_pass_the_end():
    """Only cu_q[batch] is above T: that sequence is skipped by the writer as by the attention, with the status bit."""
    import torch
    c = Batch([2, 3], [50, 60], 16, seed=42)
    out = run_dense(c)
    new = torch.randn(5, ROW, device="cuda").bfloat16()
    c.cu_q = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    got = c.outputs()
    bad_status(lambda: run_dense(c, got))
    assert torch.equal(got[0][:2], out[0][:2]) and torch.equal(got[1][:2], out[1][:2])
    before = c.kv8.clone()
    bad_status(lambda: B.dsa_cache_write(new, *c.plan, c.kv8, c.kv_scale))
    changed = (c.kv8 != before).any(2).view(-1).nonzero().flatten().cpu().tolist()
    assert set(changed) == {int(s) for s in c.slots(0, [48, 49])}


@pytest.mark.gpu
@pytest.mark.parametrize("cu,rows", [([0, 3, 1, 4], {0: (0, 47, 3), 3: (2, 69, 3)}),
                                     ([0, 2, 1 << 30, 4], {0: (0, 48, 2), 1: (0, 49, 2)}),
                                     ([-2, 1, 2, 4], {1: (1, 59, 1), 2: (2, 68, 2), 3: (2, 69, 2)})])
def test_sequences_in_order_beside_others_that_are_not(cu, rows):
    """Rows that one sequence in order has to itself come out and are written; nothing lies around the tensors' ends."""
    import torch
    c = Batch([2, 1, 1], [50, 60, 70], 16, seed=43)
    c.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full((c.T + 4, HEADS, LATENT), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T + 4, HEADS), 7.0, device="cuda")
    bad_status(lambda: run_dense(c, (o[2:-2], lse[2:-2])))
    for x in (o, lse):
        assert bool((x[:2] == 7.0).all()) and bool((x[-2:] == 7.0).all())
    alone = Batch([1], [1], 16, seed=43)
    for t, (b, pos, _) in rows.items():
        alone.q, alone.T, alone.new, alone.lens = c.q[t:t + 1], 1, [1], [pos + 1]
        alone.kv8, alone.kv_scale, alone.table = c.kv8, c.kv_scale, c.table[b:b + 1]
        check_attention(alone, o[2 + t:3 + t], lse[2 + t:3 + t])
    new = torch.randn(c.T, ROW, device="cuda").bfloat16()
    codes, rope, scale = quantise64(new.double())
    want = torch.cat([codes, rope.to(torch.bfloat16).view(torch.uint8)], 1)
    bad_status(lambda: B.dsa_cache_write(new, *c.plan, c.kv8, c.kv_scale))
    for t, (b, pos, _) in rows.items():
        at = int(c.slots(b, [pos])[0])
        assert torch.equal(c.kv8.view(-1, ROW8)[at], want[t]) and float(c.kv_scale.view(-1)[at]) == float(scale[t])


# ------------------------------------------------------------------ short wait limits

SHORT = r"""
import sys
sys.path[:0] = [ROOT, ROOT + "/tests"]
from indexer_selected_sparse_dsa_b200 import binding as B
from paged_util import Batch, check_attention, selection
from test_paged_cache import run_dense, run_selected
def limited(ns, call, c, *pick):
    B.dsa_set_wait_limit_ns(ns)
    out = c.outputs()
    try:
        call(c, *pick, out=out)
        B.dsa_sync_status()
        check_attention(c, *out, *pick)
        return "OK"
    except B.DSAError as e:
        assert e.code == B.DSA_ERR_TIMEOUT, e
        return "TIMEOUT"
    finally:
        B.dsa_set_wait_limit_ns(0)
        check_attention(c, *call(c, *pick), *pick)
        B.dsa_sync_status()
seen = {}
for new, lens in (([1, 6, 2], [3000, 700, 90]), ([60, 3], [2000, 9000])):
    c = Batch(new, lens, 16, seed=30)
    idx = selection(c, 300, seed=31)
    for ns in LIMITS:
        for call, pick in ((run_dense, ()), (run_selected, (idx,))):
            seen.setdefault(ns, []).append(limited(ns, call, c, *pick))
c = Batch([1], [1], 16, seed=32)
in_time = [limited(3900, run_dense, c) for _ in range(20)]
print("RESULT", all(s == "TIMEOUT" for s in seen[1]), all(s == "OK" for s in seen[200000]), "OK" in in_time, flush=True)
"""


@pytest.mark.gpu
def test_a_short_limit_times_out_or_gives_the_result():
    """Limits from a nanosecond to 0.2 ms over a few tiles a CTA: waits give up at the start, in the middle of the pipeline or
    not at all.  A call that reports no timeout is right, and so is the next call after one that does.  No wait is complete
    within 1 ns everywhere, none of so small a batch is 0.2 ms late, and one key's waits (2.5 us) are not 3.9 us late."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    limits = [1, 300, 1000, 2000, 3000, 4000, 5000, 6000, 7000, 8000, 9000, 10000, 12000, 14000, 16000, 20000, 200000]
    r = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\nLIMITS = {limits!r}\n" + SHORT], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "RESULT True True True" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


# ------------------------------------------------------------------ other arguments

@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0416, 0.1352, 1.7])
def test_scales_that_are_no_power_of_two(scale):
    import torch
    c = Batch([1, 4, 40], [2500, 300, 700], 16, seed=44)
    o, lse = c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * c.page, 0)
    B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, scale, o, lse, ws)
    B.dsa_sync_status()
    check_attention(c, o, lse, scale=scale)
    idx = selection(c, 300, seed=45, holes=0.2)
    B.dsa_paged_sparse_mla_attn(c.q, *c.plan, torch.from_numpy(idx).cuda(), c.kv8, c.kv_scale, scale, o, lse, ws)
    B.dsa_sync_status()
    check_attention(c, o, lse, idx, scale=scale)


@pytest.mark.gpu
def test_without_lse():
    """The outputs are the same; whole rows and rows split over CTAs (the merge) alike."""
    import torch
    c = Batch([1, 1, 1] + [1] * 60, [6000, 129, 128] + [20] * 60, 16, seed=46)
    idx = selection(c, 900, seed=47)
    idx_d = torch.from_numpy(idx).cuda()
    want, want_s = run_dense(c)[0], run_selected(c, idx)[0]
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * c.page, 0)
    o, o_s = c.outputs()[0], c.outputs()[0]
    B.dsa_paged_mla_attn(c.q, *c.plan, c.kv8, c.kv_scale, SCALE, o, None, ws)
    B.dsa_paged_sparse_mla_attn(c.q, *c.plan, idx_d, c.kv8, c.kv_scale, SCALE, o_s, None, ws)
    B.dsa_sync_status()
    assert torch.equal(o, want) and torch.equal(o_s, want_s)


@pytest.mark.gpu
@pytest.mark.parametrize("topk", [64, 2048])
def test_what_the_indexer_selects_is_what_is_attended_to(topk):
    """The selected step of a server: new rows written, positions ranked by the indexer, attention over what it wrote, one
    behind the other on a stream; then all of it captured and replayed with other queries and lengths."""
    import torch
    c = Batch([1, 3, 1, 20], [5000, 900, 1, 2600], 16, seed=48)
    g = torch.Generator(device="cuda").manual_seed(49)
    q_I = torch.randn(c.T, B.INDEX_HEADS, B.INDEX_DIM, generator=g, device="cuda").bfloat16()
    w = torch.rand(c.T, B.INDEX_HEADS, generator=g, device="cuda").bfloat16()
    k_I = torch.randn(sum(c.lens), B.INDEX_DIM, generator=g, device="cuda").bfloat16()
    first = np.concatenate([[0], np.cumsum(c.lens)[:-1]])
    kv_start = torch.from_numpy(np.repeat(first, c.new)).cuda()
    n_vis = torch.tensor([m - n + j + 1 for n, m in zip(c.new, c.lens) for j in range(n)], dtype=torch.int32, device="cuda")
    new = torch.randn(c.T, ROW, generator=g, device="cuda").bfloat16()
    idx = torch.full((c.T, topk), 7, dtype=torch.int32, device="cuda")
    o, lse = c.outputs()
    ws_i = B.workspace(B.DSA_OP_INDEXER_TOPK, c.T, max(c.lens), topk)
    ws = B.workspace(B.DSA_OP_PAGED_MLA, c.T, c.table.shape[1] * c.page, topk)

    def step():
        B.dsa_cache_write(new, *c.plan, c.kv8, c.kv_scale)
        B.dsa_indexer_topk(q_I, w, k_I, kv_start, n_vis, max(c.lens), topk, idx, ws_i)
        B.dsa_paged_sparse_mla_attn(c.q, *c.plan, idx, c.kv8, c.kv_scale, SCALE, o, lse, ws)

    def look():
        B.dsa_sync_status()
        kept = torch.minimum(n_vis, torch.tensor(topk, device="cuda"))
        assert torch.equal((idx >= 0).sum(1, dtype=torch.int32), kept) and bool((idx < n_vis[:, None]).all())
        check_attention(c, o, lse, idx.cpu().numpy())

    step()
    look()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([4000, 700, 1, 2000], [130, 3, 1, 20]):
        q_I.normal_(generator=g)
        c.q.normal_(generator=g)
        new.normal_(generator=g)
        c.lens = lens
        c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        n_vis.copy_(torch.tensor([m - n + j + 1 for n, m in zip(c.new, lens) for j in range(n)], dtype=torch.int32))
        graph.replay()
        look()


# ------------------------------------------------------------------ the longest sequence

def test_workspace_of_any_length():
    """Lengths end at 2^31 - 1, whatever max_pages * page_size says: the size does not shrink again."""
    most = B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 1 << 20, 1 << 30, 0)
    for T, keys in ((1 << 24, 1 << 60), (1 << 11, (1 << 62) - 1), (1 << 20, 1 << 50)):
        assert B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, T, keys, 0) == most
    assert B.dsa_workspace_size(B.DSA_OP_PAGED_MLA, 1, (1 << 63) - 1, 0) == most


@pytest.mark.gpu
def test_a_sequence_as_long_as_the_type_allows():
    """2^31 - 64 positions, all of them the same page: o is the page's own, lse is log(number of pages) more.  A thread adds
    2^31 / 128 / 148 * 16 weights of a head and 32 keys one by one in fp32, so its sum may be off by 2^-24 of it each,
    0.108 in all (0.115 in lse); the value product's, in half as many steps of up to 2^-23, by as much."""
    import torch
    c = Batch([1], [64], 64, seed=50)
    ro, rl, _, _ = c.reference()
    pages = (1 << 25) - 1
    table = torch.full((1, pages), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    length = torch.tensor([64 * pages], dtype=torch.int32, device="cuda")
    o, lse = c.outputs()
    ws = B.workspace(B.DSA_OP_PAGED_MLA, 1, 64 * pages, 0)
    B.dsa_paged_mla_attn(c.q, c.cu_q, length, table, c.kv8, c.kv_scale, SCALE, o, lse, ws)
    B.dsa_sync_status()
    assert float((lse.double() - (rl + math.log(pages))).abs().max()) <= 0.115 + 2.0 ** -8
    assert float((o.double() - ro).norm() / ro.norm()) <= 0.25 + 2.0 ** -8


# ------------------------------------------------------------------ arguments that are no tensors (CPU)

@pytest.mark.parametrize("bad", [None, 3, [1.0]], ids=str)
def test_arguments_that_are_no_tensors(bad):
    """As everywhere: a TypeError that names the argument, whichever it is."""
    import torch
    i32 = torch.zeros(3, dtype=torch.int32)
    good = dict(q=torch.zeros(2, HEADS, ROW, dtype=torch.bfloat16), cu_q=i32, seq_len=i32[:2], page_table=i32[:2].view(2, 1),
                idx=torch.zeros(2, 5, dtype=torch.int32), kv8=torch.zeros(4, 8, ROW8, dtype=torch.uint8),
                kv_scale=torch.zeros(4, 8), o=torch.zeros(2, HEADS, LATENT, dtype=torch.bfloat16),
                ws=torch.zeros(1 << 10, dtype=torch.uint8), rows=torch.zeros(2, ROW, dtype=torch.bfloat16),
                start=torch.zeros(2, dtype=torch.int64), kv=torch.zeros(9, ROW, dtype=torch.bfloat16))
    calls = dict(
        q=lambda a: B.dsa_paged_mla_attn(a["q"], a["cu_q"], a["seq_len"], a["page_table"], a["kv8"], a["kv_scale"], SCALE,
                                         a["o"], None, a["ws"]),
        idx=lambda a: B.dsa_paged_sparse_mla_attn(a["q"], a["cu_q"], a["seq_len"], a["page_table"], a["idx"], a["kv8"],
                                                  a["kv_scale"], SCALE, a["o"], None, a["ws"]),
        rows=lambda a: B.dsa_cache_write(a["rows"], a["cu_q"], a["seq_len"], a["page_table"], a["kv8"], a["kv_scale"]),
        kv=lambda a: B.dsa_cache_read(a["kv8"], a["kv_scale"], a["seq_len"], a["page_table"], a["start"], a["kv"]))
    for which, names in (("q", ("q", "ws", "kv8")), ("idx", ("q", "ws", "idx", "page_table")), ("rows", ("seq_len", "page_table")),
                         ("kv", ("kv", "kv8"))):
        for name in names:
            with pytest.raises(TypeError, match=f"^{name} must be"):
                calls[which]({**good, name: bad})
