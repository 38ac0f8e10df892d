"""Plain 64-bit forms of attention with sinks and of drafted trees, with the tolerances of chunk_reference.

A row's trees are lists of parents; everything is written from the definitions in include/pkv.h and
include/pkv_tree.h, token by token."""
from __future__ import annotations

import math

import torch

import chunk_reference as R


def forest(n, gen, roots=0.1, near=False):
    """Parents of n drafted tokens: each hangs from the context with probability `roots` (the first always), else
    from an earlier token (`near`: one of the last four)."""
    out = []
    for j in range(n):
        top = j == 0 or float(torch.rand(1, generator=gen)) < roots
        low = max(0, j - 4) if near else 0
        out.append(-1 if top else low + int(torch.randint(j - low, (1,), generator=gen)))
    return out


def branch(tree, leaf):
    """Token leaf of a tree and its ancestors, the oldest first."""
    out = []
    while leaf >= 0:
        out.append(leaf)
        leaf = tree[leaf]
    return out[::-1]


def seen(n, L, window=0, sinks=0, prefix=0, tree=None):
    """[n][L]: which tokens of a row of L tokens, its last n new, each new one attends to."""
    C = L - n
    out = torch.zeros(n, L, dtype=torch.bool)
    where = torch.arange(L)  # positions
    lines = None
    if tree is not None:
        lines = [branch(tree, j) for j in range(n)]
        where[C:] = torch.tensor([C + len(x) - 1 for x in lines])
    for j in range(n):
        P = int(where[C + j])
        near = where > P - window if window else torch.ones(L, dtype=torch.bool)
        near = near | (where < sinks)
        if tree is None:
            out[j] = near & (where < max(P + 1, prefix))
        else:
            out[j, :C] = near[:C]
            for a in lines[j]:
                out[j, C + a] = bool(near[C + a])
    return out


def attention(c, q, scale, trees=None, window=0, sinks=0, softcap=0.0, slopes=None, prefix_lens=None, fp32=False):
    """(out, its tolerance, lse, its tolerance) in float64, as chunk_reference.attention.  `fp32`: queries and
    outputs of the single-token step, whose products carry both halves of a weight (2^-21) and round nothing to
    16 bits."""
    io = torch.float32 if fp32 else R.IO[c.kv]
    out = torch.zeros(c.tokens, c.n_q, R.D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((c.tokens, c.n_q), -math.inf, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for i, (n, L) in enumerate(c.rows):
        if n == 0 or L < n:
            continue
        a = int(c.cu[i])
        show = seen(n, L, window, sinks, 0 if prefix_lens is None else int(prefix_lens[i]),
                    None if trees is None else trees[i]).to(q.device)
        kq = c.stored("k", i).repeat_interleave(c.n_q // c.n_kv, 0)
        v = c.stored("v", i).repeat_interleave(c.n_q // c.n_kv, 0)
        used = show.any(0)  # what no query attends to may be anything
        kq, v = kq.masked_fill(~used[:, None], 0), v.masked_fill(~used[:, None], 0)
        qd = q[a:a + n].double().transpose(0, 1)
        s = qd @ kq.transpose(1, 2) * scale
        size = qd.abs() @ kq.abs().transpose(1, 2) * abs(scale)
        if softcap > 0:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            far = (torch.arange(L - n, L)[:, None] - torch.arange(L)[None]).abs().double().to(q.device)
            s = s - slopes.double()[:, None, None] * far
            size = size + slopes.double().abs()[:, None, None] * far * 2 ** -2
        s, size = s.masked_fill(~show, -math.inf), size.masked_fill(~show, 0.0)
        ds = size.amax(-1) * R.SCORE_STEPS + s.masked_fill(~show, 0).abs().amax(-1) * 2.0 ** -22 + 2.0 ** -20
        p = torch.softmax(s, -1)
        o, mag = p @ v, p @ v.abs()
        z = torch.logsumexp(s, -1)
        weights = 2.0 ** -20 if fp32 else R.half_step(io)
        t = R.half_step(io) * o.abs() + (weights + 2 * ds[..., None] + 2.0 ** -20) * mag + R.tiny(io)
        out[a:a + n], tol[a:a + n] = o.transpose(0, 1), t.transpose(0, 1)
        lse[a:a + n] = z.transpose(0, 1)
        ltol[a:a + n] = (ds + z.abs() * 2.0 ** -22 + 2.0 ** -20).transpose(0, 1)
    return out, tol, lse, ltol


def check(c, q, out, lse, scale, status=0, **kw):
    want, tol, wl, lt = attention(c, q, scale, fp32=lse is None, **kw)
    n = int(c.cu[-1])
    assert torch.isfinite(out[:n]).all()
    err = (out[:n].double() - want[:n]).abs()
    assert (err <= tol[:n]).all(), f"{float((err - tol[:n]).max())} over the tolerance, error {float(err.max())}"
    if lse is not None:
        none = wl[:n] == -math.inf
        assert (lse[:n][none] == -math.inf).all()
        lerr = (lse[:n].double() - wl[:n]).abs()[~none]
        assert (lerr <= lt[:n][~none]).all(), float(lerr.max())
    assert c.pool.read_status() == status


def spoil(c, tokens, value=math.nan):
    """K and V of the given tokens [(row, token)] become `value` (q8_0: their scales), in the call's layer."""
    for i, t in tokens:
        page, slot = int(c.bt[i, t // R.PAGE]), t % R.PAGE
        for name in ("k", "v"):
            x = getattr(c.pool, name + "_scales") if c.pool.k_scales is not None else getattr(c.pool, name + "_data")
            x[c.layer, page, :, slot] = value
