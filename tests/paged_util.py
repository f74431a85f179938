"""Seeded paged batches, the paged operators' definitions in 64 bits, and their tolerances."""
import math

import numpy as np

LATENT, ROPE, ROW, ROW8, HEADS = 512, 64, 576, 640, 64
SCALE = 1.0 / 16.0


def e4m3_values():
    """The values of the 256 e4m3 codes."""
    v = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        v[c] = math.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


def quantise64(rows):
    """rows [n, 576] float64 (exact bf16 values) -> (codes uint8 [n, 512], rope float64, scale float64), by definition."""
    import torch
    lat = rows[:, :LATENT]
    amax = torch.where(lat.isfinite(), lat.abs(), 0.0).amax(1)
    scale = torch.full_like(amax, 2.0 ** -60)
    for k in range(-60, 60):
        scale[amax > 448.0 * 2.0 ** k] = 2.0 ** (k + 1)
    grid = torch.from_numpy(e4m3_values()[:127]).to(rows.device)
    a = torch.where(lat.isfinite(), lat / scale[:, None], 0.0).abs().clamp(max=448.0)
    hi = torch.bucketize(a, grid).clamp(max=126)           # grid[hi - 1] < a <= grid[hi]
    lo = (hi - 1).clamp(min=0)
    dh, dl = grid[hi] - a, a - grid[lo]
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi) + torch.where(lat.signbit(), 128, 0)
    return torch.where(lat.isfinite(), pick, 127).to(torch.uint8), rows[:, LATENT:] / scale[:, None], scale


class Batch:
    """A paged batch on the device: pages in random order, the unused entries of the page table poisoned."""

    def __init__(self, new, lens, page, seed, spare=2, pad=0, width=None, values=None):
        import torch
        r = np.random.default_rng(seed)
        self.new, self.lens, self.page = list(new), list(lens), page
        used = [-(-m // page) for m in lens]
        self.n_pages = sum(used) + spare
        order = r.permutation(self.n_pages)
        width = max(max(used, default=0), 1) if width is None else width
        table = np.full((len(lens), width), 1 << 30, np.int32)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.T = sum(new) + pad
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = r.standard_normal((self.n_pages * page, ROW)) if values is None else values(r, self.n_pages * page)
        self.rows = torch.from_numpy(rows.astype(np.float32)).to(torch.bfloat16).cuda()
        self.q = torch.from_numpy(r.standard_normal((self.T, HEADS, ROW)).astype(np.float32)).to(torch.bfloat16).cuda()
        codes, rope, scale = quantise64(self.rows.double())
        self.kv8 = torch.cat([codes, rope.to(torch.bfloat16).view(torch.uint8)], 1).view(self.n_pages, page, ROW8)
        self.kv_scale = scale.float().view(self.n_pages, page)
        self.cu_q = torch.from_numpy(self.cu).cuda()
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.page_table = torch.from_numpy(table).cuda()

    @property
    def plan(self):
        return self.cu_q, self.seq_len, self.page_table

    def slots(self, b, pos):
        pos = np.asarray(pos, np.int64)
        return self.table[b, pos // self.page].astype(np.int64) * self.page + pos % self.page

    def values(self, b, n):
        """Positions 0 .. n-1 of sequence b in 64 bits, as the cache holds them."""
        import torch
        at = torch.from_numpy(self.slots(b, np.arange(n))).cuda()
        raw = self.kv8.view(-1, ROW8)[at]
        tab = torch.from_numpy(e4m3_values()).cuda()
        x = torch.cat([tab[raw[:, :LATENT].long()], raw[:, LATENT:].contiguous().view(torch.bfloat16).double()], 1)
        return x * self.kv_scale.view(-1)[at].double()[:, None]

    def scales(self, b, n):
        import torch
        return self.kv_scale.view(-1)[torch.from_numpy(self.slots(b, np.arange(n))).cuda()].double()

    def outputs(self):
        import torch
        o = torch.full((self.T, HEADS, LATENT), 7.0, dtype=torch.bfloat16, device="cuda")
        return o, torch.full((self.T, HEADS), 7.0, device="cuda")

    def reference(self, idx=None, scale=SCALE):
        """(o, lse, tolerance of o, tolerance of lse) in 64 bits.

        What the kernels may round (each at most half a step): q to 2^-22 of its head's largest value; the products'
        sums in 32 bits over the 36 steps of 16 or 32 dims, 36 * 2^-23 < 2^-17 of the sum of magnitudes; so a score is
        off by at most e = scale * (2^-17 sum |q||k| + 2^-22 max|q| sum |k|) plus 2^-20 for the exponential's argument
        and itself.  Probabilities are rounded to fp16, 2^-11, and sums in 32 bits again, 2^-17; the output to bf16,
        2^-8 of itself.  A relative error e of every weight moves a mean by at most 2 e times the mean magnitude.
        fp16 has a floor besides its relative step: what is rounded is u = p 2^k, held so that the largest u of a head
        is at least 2^4 (the running maximum stands at 2^4 and is never above a score already seen); values below 2^-14
        are rounded to multiples of 2^-24, so each u is off by up to 2^-25 more, 2^-29 of the largest, times its code.
        """
        import torch
        o = torch.zeros(self.T, HEADS, LATENT, dtype=torch.float64, device="cuda")
        lse = torch.full((self.T, HEADS), -math.inf, dtype=torch.float64, device="cuda")
        to, tl = torch.zeros_like(o), torch.zeros_like(lse)
        for b, (n, m) in enumerate(zip(self.new, self.lens)):
            if n == 0 or m == 0:
                continue
            seq, sc = self.values(b, m), self.scales(b, m)
            for j in range(n):
                t = int(self.cu[b]) + j
                seen = max(m - n + j + 1, 0)
                k, ks = seq[:seen], sc[:seen]
                if idx is not None:
                    s = torch.as_tensor(idx[t]).long().cuda()
                    s = s[(s >= 0) & (s < seen)]
                    k, ks = seq[s], sc[s]
                if k.shape[0] == 0:
                    continue
                q = self.q[t].double()
                x = q @ k.T * scale
                lse[t] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1)
                v = k[:, :LATENT]
                o[t] = p @ v
                e = scale * (2.0 ** -17 * (q.abs() @ k.abs().T)
                             + 2.0 ** -22 * q.abs().amax(1, keepdim=True) * k.abs().sum(1)[None]).amax(1) + 2.0 ** -20
                tl[t] = e + 2.0 ** -22 * lse[t].abs()
                to[t] = 2.0 ** -8 * o[t].abs() + (2 * e[:, None] + 2.0 ** -11 + 2.0 ** -16) * (p @ v.abs())
                to[t] += 2.0 ** -29 * (p * ks).amax(1)[:, None] * (v.abs() / ks[:, None]).sum(0)[None]
        return o, lse, to, tl


def check_attention(batch, o, lse, idx=None, scale=SCALE):
    import torch
    ro, rl, to, tl = batch.reference(idx, scale)
    used = int(batch.cu[-1])
    assert bool((o[used:] == 7.0).all()) and bool((lse[used:] == 7.0).all()), "rows behind the last sequence changed"
    o, lse, ro, rl, to, tl = (x[:used] for x in (o.double(), lse.double(), ro, rl, to, tl))
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert bool((o[empty] == 0).all())
    over = ((o - ro).abs() - to).amax() if used else 0
    assert over <= 0, f"o off by {float((o - ro).abs().max()):.3e}, {float(over):.3e} over the tolerance"
    d = torch.where(empty, 0.0, (lse - rl).abs() - tl)
    assert bool((d <= 0).all()), f"lse off: {float(d.max()):.3e} over the tolerance"


def selection(batch, topk, seed, holes=0.0):
    """A random selection as the top-k writes it (ascending, -1 behind); `holes`: that share of it emptied in place."""
    r = np.random.default_rng(seed)
    idx = np.full((batch.T, topk), -1, np.int32)
    for b, (n, m) in enumerate(zip(batch.new, batch.lens)):
        for j in range(n):
            seen = m - n + j + 1
            k = min(topk, seen)
            idx[batch.cu[b] + j, :k] = np.sort(r.permutation(seen)[:k])
    idx[r.random(idx.shape) < holes] = -1
    return idx
