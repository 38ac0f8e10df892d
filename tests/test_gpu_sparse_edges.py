"""The widest and deepest trees under windows and sinks, and values that are not finite, query by query and head by
head: what chunk attention's kernels do where not every token from a query's first on is visible."""
import math

import pytest
import torch

import chunk_reference as R
import tree_reference as T
from test_gpu_tree import drafted, parents_of, run
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
TYPES = [api.F16, api.BF16, api.Q8_0]


def close_gap(c, window, sinks):
    """Context tokens that no drafted token attends to are NaN, the table entries of pages without any other -1.
    Returns the table as it was."""
    full = c.bt.clone()
    for i, (n, L) in enumerate(c.rows):
        first = max(0, L - n + 1 - window)
        T.spoil(c, [(i, t) for t in range(sinks, first)])
        c.bt[i, -(-sinks // 16):max(-(-sinks // 16), first // 16)] = -1
    return full


@pytest.mark.parametrize("window,sinks", [(3, 0), (300, 17), (700, 400)])
@pytest.mark.parametrize("kv,group", [(api.F16, 4), (api.BF16, 1), (api.Q8_0, 4)])
def test_the_widest_and_deepest_trees(kv, group, window, sinks):
    """1024 drafted tokens, whose depths are found by walking to their roots: a chain, a star, a binary tree, a deep
    forest.  Windows that end among the context and among the drafted tokens, in every tile."""
    n = 1024
    c = R.Chunk(kv, 1, group, [(n, n + 5), (n, n + 500), (n, n), (n - 1, n + 77)], seed=window)
    c.pool.set_window(0, window)
    c.pool.set_sinks(0, sinks)
    trees = [list(range(-1, n - 1)), [-1] + [0] * (n - 1), [(j - 1) // 2 if j else -1 for j in range(n)],
             T.forest(n - 1, c.gen, roots=0.002, near=True)]
    full = close_gap(c, window, sinks)
    q, out, lse = run(c, parents_of(c, trees))
    c.bt = full
    T.check(c, q, out, lse, SCALE, trees=trees, window=window, sinks=sinks)


@pytest.mark.parametrize("kv", TYPES)
def test_a_chain_behind_a_long_context_under_a_window(kv):
    """A chain whose every block of context is masked for some of its queries: a causal chunk of that window."""
    c = R.Chunk(kv, 1, 4, [(600, 2000), (1, 900)], seed=2)
    c.pool.set_window(0, 777)
    q, out, lse = run(c, parents_of(c, [list(range(-1, m - 1)) for m, _ in c.rows]))
    want, tol, wl, lt = R.attention(c, q, SCALE, window=777)
    assert ((out.double() - want).abs() <= tol).all() and ((lse.double() - wl).abs() <= lt).all()


def reached(out, hit):
    """Every head of every query in `hit` holds a value that is not finite."""
    assert (~torch.isfinite(out[hit])).any(-1).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("kv", TYPES)
def test_seen_values_reach_every_query_that_sees_them(kv, bad):
    c = R.Chunk(kv, 2, 4, [(300, 300), (60, 420), (1, 90)], seed=5)
    c.pool.set_window(0, 50)
    c.pool.set_sinks(0, 4)
    tokens = [(0, 2), (0, 100), (1, 375), (2, 60)]
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    T.spoil(c, tokens, bad)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE)
    for i, (n, L) in enumerate(c.rows):
        show = T.seen(n, L, 50, 4)
        hit = torch.stack([show[:, t] for r, t in tokens if r == i]).any(0).to(c.device)
        mine = out[int(c.cu[i]):int(c.cu[i]) + n]
        reached(mine, hit)
        assert torch.isfinite(mine[~hit]).all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("kv", TYPES)
def test_seen_values_reach_every_descendant(kv, bad, window, sinks):
    c = R.Chunk(kv, 2, 4, [(64, 200), (1, 90), (100, 331)], seed=5)
    c.pool.set_window(0, window)
    c.pool.set_sinks(0, sinks)
    trees, parents = drafted(c, near=True)
    tokens = [(0, 125), (0, 200 - 64 + 9), (1, 88), (2, 331 - 100 + 30), (2, 331 - 100 + 80)]
    T.spoil(c, tokens, bad)
    _, out, _ = run(c, parents)
    for i, (n, L) in enumerate(c.rows):
        show = T.seen(n, L, window, sinks, tree=trees[i])
        hit = torch.stack([show[:, t] for r, t in tokens if r == i]).any(0).to(c.device)
        mine = out[int(c.cu[i]):int(c.cu[i]) + n]
        reached(mine, hit)
        assert torch.isfinite(mine[~hit]).all()
