"""Weights far below a row's largest: chunk attention holds a block's weights in 16 bits, beside a maximum that later
groups of the block's columns may raise."""
import math

import pytest
import torch

import chunk_reference as R
import tree_reference as T
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu


def write(c, which, i, t, x):
    """K or V of token t of row i in every KV head, as c's pool holds it."""
    page, slot = int(c.bt[i, t // 16]), t % 16
    data, scales = (getattr(c.pool, which + s) for s in ("_data", "_scales"))
    if c.kv == api.Q8_0:
        b = x.reshape(4, 32)
        d = (b.abs().amax(-1, keepdim=True) / 127.0).half()
        code = torch.where(d > 0, b / d.float().clamp_min(1e-30), torch.zeros_like(b)).round().clamp(-127, 127)
        data[c.layer, page, :, slot] = (code + 128).to(torch.uint8).reshape(128)
        scales[c.layer, page, :, slot] = d[:, 0]
    else:
        data[c.layer, page, :, slot] = x.to(data.dtype)


@pytest.mark.parametrize("call", ["chunk", "bias", "sinks", "tree"])
@pytest.mark.parametrize("up", [10.0, 15.5, 17.5, 19.0])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_a_maximum_raised_within_a_block(kv, up, call):
    """One token's score lies `up` above those of the tokens before it, in a later group of the same block, and its
    value is 0: the output is what the others leave."""
    rows, heavy = [(1, 60), (1, 50), (3, 64)], [45, 33, 60]
    c = R.Chunk(kv, 1, 4, rows, seed=1)
    kw, window, sinks = {}, 0, 0
    if call == "sinks":
        window, sinks = 40, 16
        c.pool.set_window(0, window)
        c.pool.set_sinks(0, sinks)
    if call == "bias":
        kw["slopes"] = torch.full((4,), 2.0 ** -12, device=c.device)
    one = torch.zeros(128, device=c.device)
    one[0] = 1.0
    for i, (n, L) in enumerate(rows):
        for t in range(L):
            write(c, "k", i, t, one * (up if t == heavy[i] else 0.0))
            write(c, "v", i, t, torch.full((128,), 0.0 if t == heavy[i] else 900.0 + t, device=c.device))
    q = torch.zeros(c.tokens, c.n_q, 128, dtype=R.IO[kv], device=c.device)
    q[:, :, 0] = 16.0
    out = torch.zeros_like(q)
    if call == "tree":
        parents = torch.tensor([-1, -1, -1, 0, 1], dtype=torch.int32, device=c.device)
        trees = [[-1], [-1], [-1, 0, 1]]
        api.paged_tree_attention(c.pool, 0, q, parents, c.cu, c.bt, c.lens, 1 / 16, out=out)
    else:
        trees = None
        api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, 1 / 16, out=out, **kw)
    want, tol, _, _ = T.attention(c, q, 1 / 16, trees=trees, window=window, sinks=sinks, **kw)
    # A weight in f16, scaled by 2^7, is off by half a step of the subnormals too: 2^-25 of it.  (A weight made under
    # the lower maximum is normal then, and rounded to a subnormal as it is rescaled.)  bf16 has none here.
    least = 0.0 if kv == api.BF16 else 2.0 ** -32 * sum(900.0 + t for t in range(64))
    assert c.pool.read_status() == 0
    err = (out.double() - want).abs()
    assert (want > 8 * (tol + least)).all()  # what is lost would show
    assert (err <= tol + least).all(), float((err - tol - least).max())
