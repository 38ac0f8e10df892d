"""paged_tree_attention and kv_tree_commit on the GPU against their definitions, and a run of the calls of
speculative decoding together."""
import math

import pytest
import torch

import chunk_reference as R
import tree_reference as T
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
TYPES = [api.F16, api.BF16, api.Q8_0]
RAGGED = [(1, 1), (1, 17), (3, 3), (16, 40), (0, 12), (33, 33), (5, 300), (70, 131), (0, 0), (64, 700), (129, 500), (40, 168)]


def drafted(c, **kw):
    """A forest for each row, and the parents array of the call."""
    trees = [T.forest(n, c.gen, **kw) for n, _ in c.rows]
    return trees, parents_of(c, trees)


def parents_of(c, trees):
    flat = [x for t in trees for x in t]
    return torch.tensor(flat + [7] * (c.tokens - len(flat)), dtype=torch.int32, device=c.device)


def run(c, parents, q=None, workspace=None, **kw):
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[c.kv]) if q is None else q
    out = torch.full((c.tokens, c.n_q, 128), 7.0, dtype=q.dtype, device=c.device)
    lse = torch.full((c.tokens, c.n_q), 7.0, device=c.device)
    scale = kw.pop("scale", SCALE)
    api.paged_tree_attention(c.pool, c.layer, q, parents, c.cu, c.bt, c.lens, scale, out=out, lse=lse,
                             workspace=workspace, **kw)
    return q, out, lse


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("kv", TYPES)
def test_ragged_trees(kv, group, near):
    c = R.Chunk(kv, 2, group, RAGGED, seed=group, behind=3)
    trees, parents = drafted(c, near=near)
    q, out, lse = run(c, parents)
    T.check(c, q, out, lse, SCALE, trees=trees)
    assert (out[int(c.cu[-1]):] == 7).all() and (lse[int(c.cu[-1]):] == 7).all()  # tokens of no row


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (5, 2), (16, 4), (100, 17), (60, 200), (128, 128), (300, 1)])
@pytest.mark.parametrize("kv", TYPES)
def test_windows_and_sinks(kv, window, sinks):
    """Windows shorter than the trees and longer; sinks that reach into the drafted tokens."""
    c = R.Chunk(kv, 2, 4, RAGGED, seed=window)
    c.pool.set_window(0, window)
    c.pool.set_sinks(0, sinks)
    trees, parents = drafted(c, near=True)
    full = c.bt.clone()
    for i, (n, L) in enumerate(c.rows):  # no query attends to these
        first = max(0, L - n + 1 - window)
        T.spoil(c, [(i, t) for t in range(sinks, first)])
        c.bt[i, -(-sinks // 16):max(-(-sinks // 16), first // 16)] = -1
    q, out, lse = run(c, parents)
    c.bt = full
    T.check(c, q, out, lse, SCALE, trees=trees, window=window, sinks=sinks)


@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(softcap=2.0), dict(softcap=1e12), dict(scale=-0.2), dict(scale=0.0)])
@pytest.mark.parametrize("kv", TYPES)
def test_scores(kv, kw):
    c = R.Chunk(kv, 2, 4, [(64, 200), (40, 500), (1, 700), (129, 260)], seed=3)
    c.pool.set_window(0, 90)
    trees, parents = drafted(c)
    q, out, lse = run(c, parents, **kw)
    kw = dict(kw)
    T.check(c, q, out, lse, kw.pop("scale", SCALE), trees=trees, window=90, **kw)


@pytest.mark.parametrize("chunks", [1, 2, 7, 152, 400])
@pytest.mark.parametrize("kv", TYPES)
def test_splits(kv, chunks):
    c = R.Chunk(kv, 2, 4, [(60, 1000), (1, 2100), (200, 310), (64, 640)], seed=4)
    trees, parents = drafted(c)
    q, out, lse = run(c, parents, workspace=api.WorkspaceChunk(c.pool, c.n_q, chunks))
    T.check(c, q, out, lse, SCALE, trees=trees)


@pytest.mark.parametrize("kv", TYPES)
def test_the_widest_and_deepest_trees(kv):
    """1024 drafted tokens: a chain, a star, a binary tree, and 1023 of a forest; more than one warp plans."""
    n = 1024
    c = R.Chunk(kv, 1, 4, [(n, n + 5), (n, n + 300), (n, n), (n - 1, n + 77)], seed=1)
    trees = [list(range(-1, n - 1)), [-1] + [0] * (n - 1), [(j - 1) // 2 if j else -1 for j in range(n)],
             T.forest(n - 1, c.gen)]
    q, out, lse = run(c, parents_of(c, trees))
    T.check(c, q, out, lse, SCALE, trees=trees)


@pytest.mark.parametrize("kv", TYPES)
def test_a_chain_is_a_chunk(kv):
    c = R.Chunk(kv, 2, 4, [(40, 300), (1, 50), (100, 100)], seed=2)
    q, out, lse = run(c, parents_of(c, [list(range(-1, n - 1)) for n, _ in c.rows]))
    want, tol, wl, lt = R.attention(c, q, SCALE)
    assert ((out.double() - want).abs() <= tol).all() and ((lse.double() - wl).abs() <= lt).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("kv", TYPES)
def test_other_branches_never_reach_an_output(kv, bad):
    """K and V of a drafted token that are not finite reach its descendants alone."""
    c = R.Chunk(kv, 2, 4, [(64, 200), (1, 90), (100, 331)], seed=5)
    trees, parents = drafted(c)
    tokens = [(0, 200 - 64 + 9), (2, 331 - 100 + 30), (2, 331 - 100 + 80)]
    T.spoil(c, tokens, bad)
    q, out, lse = run(c, parents)
    T.spoil(c, tokens, 1.0)
    want, tol, wl, lt = T.attention(c, q, SCALE, trees=trees)
    for i, (n, L) in enumerate(c.rows):
        hit = [any(r == i and t - (L - n) in T.branch(trees[i], j) for r, t in tokens) for j in range(n)]
        a = int(c.cu[i])
        whole = torch.tensor([a + j for j in range(n) if not hit[j]], device=c.device)
        assert ((out[whole].double() - want[whole]).abs() <= tol[whole]).all()
        assert ((lse[whole].double() - wl[whole]).abs() <= lt[whole]).all()
        for j in range(n):
            assert not hit[j] or not torch.isfinite(out[a + j]).all()


def test_parents_outside_their_tree():
    """A parent that is not an earlier token, or below -1, is reported and stands for -1."""
    c = R.Chunk(api.F16, 2, 4, [(8, 100), (6, 30)], seed=5)
    trees = [[-1, 0, 1, 1, 3, 4, 0, 6], [-1, 0, 0, 1, 2, 2]]
    parents = parents_of(c, trees)
    for j, p in ((3, 3), (3, 7), (3, 2 ** 31 - 1), (3, -2), (3, -2 ** 31), (0, 0), (8 + 5, 900)):
        wrong = parents.clone()
        wrong[j] = p
        q, out, lse = run(c, wrong)
        mended = [list(t) for t in trees]
        mended[0 if j < 8 else 1][j % 8] = -1
        T.check(c, q, out, lse, SCALE, trees=mended, status=api.DEV_BAD_TREE)


def test_rows_that_are_skipped():
    """More drafted tokens than a tree may have, and lengths that do not fit."""
    c = R.Chunk(api.F16, 2, 2, [(3, 40), (1025, 1100), (9, 60), (4, 20)], seed=1)
    trees = [T.forest(n, c.gen) for n, _ in c.rows]
    c.lens[2] = 8
    q, out, lse = run(c, parents_of(c, trees))
    assert c.pool.read_status() == api.DEV_BAD_LENGTH
    c.rows = [(3, 40), (1025, 0), (9, 0), (4, 20)]
    assert (out[3:3 + 1025 + 9] == 0).all() and (lse[3:3 + 1025 + 9] == -math.inf).all()
    T.check(c, q, out, lse, SCALE, trees=trees)


def test_strided_queries_streams_and_graph():
    """Queries inside a projection's output; the call on another stream; captured, with other trees at its replay."""
    c = R.Chunk(api.BF16, 2, 4, [(20, 300), (33, 90), (1, 400)], seed=6, layers=2, layer=1)
    trees, parents = drafted(c)
    qkv = c.normal(c.tokens, c.n_q + 4, 128, dtype=torch.bfloat16)
    q = qkv[:, :c.n_q]
    ws = api.WorkspaceChunk(c.pool, c.n_q)
    _, out, lse = run(c, parents, q, ws)
    T.check(c, q, out, lse, SCALE, trees=trees)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    side.wait_stream(torch.cuda.current_stream())
    api.paged_tree_attention(c.pool, 1, q, parents, c.cu, c.bt, c.lens, SCALE, out=out2, lse=lse2, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_tree_attention(c.pool, 1, q, parents, c.cu, c.bt, c.lens, SCALE, out=out2, lse=lse2, workspace=ws)
    for rows in ([(20, 300), (33, 90), (1, 400)], [(0, 10), (50, 60), (4, 390)]):
        c.rows = rows
        c.cu.copy_(torch.tensor([0] + [n for n, _ in rows]).cumsum(0))
        c.lens.copy_(torch.tensor([L for _, L in rows]))
        trees = [T.forest(n, c.gen) for n, _ in rows]
        parents.copy_(parents_of(c, trees))
        qkv.copy_(c.normal(*qkv.shape, dtype=qkv.dtype))
        graph.replay()
        torch.cuda.synchronize()
        T.check(c, q, out2, lse2, SCALE, trees=trees)


def test_two_calls_at_once():
    c = R.Chunk(api.F16, 2, 4, [(60, 3000), (64, 700)] + [(5, 200)] * 10, seed=16)
    trees, parents = drafted(c)
    q, out, lse = run(c, parents)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [api.WorkspaceChunk(c.pool, c.n_q) for _ in streams]
    outs = [(torch.zeros_like(out), torch.zeros_like(lse)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, ws, (o, z) in zip(streams, spaces, outs):
            api.paged_tree_attention(c.pool, 0, q, parents, c.cu, c.bt, c.lens, SCALE, out=o, lse=z, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for o, z in outs:
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("kv", TYPES)
def test_many_calls_back_to_back(kv):
    """Thousands of calls that nothing waits between, on three sets of inputs in turn: the bits of the first, and no wait
    that gave up."""
    sets = []
    for seed in range(3):
        c = R.Chunk(kv, 8, 4, [(128, 9000 + 500 * seed), (7, 4000), (30, 2500 + seed)], seed=seed)
        c.pool.set_window(0, 1500)
        c.pool.set_sinks(0, 40)
        trees, parents = drafted(c)
        q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
        sets.append((c, parents, q, api.WorkspaceChunk(c.pool, c.n_q), torch.zeros_like(q), torch.zeros_like(q)))

    def calls(tree, chunk):
        for (c, parents, q, ws, _, _), a, b in zip(sets, tree, chunk):
            api.paged_tree_attention(c.pool, 0, q, parents, c.cu, c.bt, c.lens, SCALE, out=a, workspace=ws)
            api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=b, workspace=ws)

    first = [torch.empty_like(x[2]) for x in sets], [torch.empty_like(x[2]) for x in sets]
    calls(*first)
    torch.cuda.synchronize()
    for _ in range(10):
        for _ in range(100):
            calls([x[4] for x in sets], [x[5] for x in sets])
        torch.cuda.synchronize()
        for x, a, b in zip(sets, *first):
            assert torch.equal(x[4], a) and torch.equal(x[5], b)
            assert x[0].pool.read_status() == 0


def test_nothing_to_do_and_bad_pages():
    c = R.Chunk(api.F16, 2, 2, [(0, 5), (0, 0)], seed=1)
    assert api.paged_tree_attention(c.pool, 0, torch.empty(0, 4, 128, dtype=torch.float16, device=c.device),
                                    torch.empty(0, dtype=torch.int32, device=c.device), c.cu, c.bt, c.lens,
                                    SCALE).shape == (0, 4, 128)
    c = R.Chunk(api.F16, 2, 2, [(4, 50)], seed=1)
    trees, parents = drafted(c)
    c.bt[0, 1] = c.num_pages
    run(c, parents)
    assert c.pool.read_status() == api.DEV_BAD_PAGE


def test_bounded_waits():
    c = R.Chunk(api.F16, 2, 4, [(30, 500), (1, 900)], seed=6)
    trees, parents = drafted(c)
    c.pool.set_test_stall(2_000_000)
    q, _, _ = run(c, parents)
    assert c.pool.read_status() & api.DEV_TIMEOUT
    c.pool.set_test_stall(0)
    q, out, lse = run(c, parents, q)
    T.check(c, q, out, lse, SCALE, trees=trees)


# ------------------------------------------------------------------------ commit ----
POOLS = [api.F16, api.BF16, api.F32, api.Q8_0]


def arrays(pool):
    return [x for x in (pool.k_data, pool.v_data, pool.k_scales, pool.v_scales) if x is not None]


def filled(kv, rows, layers=1, n_kv=2, seed=0):
    """A pool whose every byte is random (whole numbers: values do not matter here)."""
    c = R.Chunk(kv, n_kv, 1, rows, seed=seed, layers=layers)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for x in arrays(c.pool):
        b = x.view(torch.uint8)
        b.copy_(torch.randint(0, 256, b.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def committed(c, trees, leaves, layers, before):
    """The pool's arrays after the commit, and the paths, token by token."""
    out, paths = [x.clone() for x in before], []
    for i, (n, L) in enumerate(c.rows):
        path = T.branch(trees[i], leaves[i])
        paths.append(path)
        for d, x in enumerate(path):
            a, b = L - n + x, L - n + d
            for was, now in zip(before, out):
                now[layers, int(c.bt[i, b // 16]), :, b % 16] = was[layers, int(c.bt[i, a // 16]), :, a % 16]
    return out, paths


def same(xs, ys):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(xs, ys))


@pytest.mark.parametrize("kv", POOLS)
def test_commit(kv):
    """Paths that stay, shift by one and jump, over page borders; leaves of every kind; one layer of three and all."""
    rows = [(1, 1), (9, 9), (40, 100), (17, 33), (0, 20), (64, 78), (200, 207), (33, 1000), (12, 12), (0, 0), (100, 131)]
    for first, layers, seed in ((0, 3, 1), (1, 1, 2), (2, 0, 3)):
        c = filled(kv, rows, layers=3, seed=seed)
        trees = [T.forest(n, c.gen, near=bool(seed & 1)) for n, _ in rows]
        trees[2] = list(range(-1, 39))               # a chain: nothing moves
        trees[6] = [-1, -1] + list(range(1, 199))    # all but one token, each one slot down
        leaves = [n - 1 for n, _ in rows]
        leaves[3], leaves[7] = -1, 0
        before = [x.clone() for x in arrays(c.pool)]
        path = torch.full((len(rows), 250), -5, dtype=torch.int32, device=c.device)
        leaf = torch.tensor(leaves, dtype=torch.int32, device=c.device)
        new = api.kv_tree_commit(c.pool, parents_of(c, trees), leaf, c.cu, c.bt, c.lens, first_layer=first,
                                 num_layers=layers, path=path)
        want, paths = committed(c, trees, leaves, slice(first, first + layers), before)
        assert same(arrays(c.pool), want)
        assert new.tolist() == [L - n + len(p) for (n, L), p in zip(rows, paths)]
        for i, p in enumerate(paths):
            assert path[i].tolist() == p + [-5] * (250 - len(p))
        assert c.pool.read_status() == 0


@pytest.mark.parametrize("kv", POOLS)
@pytest.mark.parametrize("n_kv", [1, 3, 8])
def test_commit_of_long_paths(kv, n_kv):
    """Up to 1023 tokens that move by one slot or more: far more than a warp holds at once."""
    n = 1024
    rows = [(n, n + 7), (n, n), (n, n + 30)]
    c = filled(kv, rows, layers=2, n_kv=n_kv, seed=n_kv)
    every_other = [-1, 0] + [max(0, j - 2) for j in range(2, n)]
    trees = [[-1, -1] + list(range(1, n - 1)), every_other, T.forest(n, c.gen, roots=0.0, near=True)]
    leaves = [n - 1, n - 1, n - 1]
    before = [x.clone() for x in arrays(c.pool)]
    new = api.kv_tree_commit(c.pool, parents_of(c, trees), torch.tensor(leaves, dtype=torch.int32, device=c.device),
                             c.cu, c.bt, c.lens)
    want, paths = committed(c, trees, leaves, slice(0, 2), before)
    assert same(arrays(c.pool), want)
    assert new.tolist() == [L - m + len(p) for (m, L), p in zip(rows, paths)]


def test_commit_of_wrong_input():
    """Leaves outside their tree accept nothing, wrong parents end the path, rows of wrong lengths stay."""
    rows = [(5, 40), (5, 40), (6, 30), (1025, 1030), (4, 20), (3, 3)]
    c = filled(api.F16, rows, seed=4)
    trees = [T.forest(n, c.gen) for n, _ in rows]
    trees[2] = [-1, -1, 1, 5, 2, 4]
    leaves = [5, -2, 5, 3, 1, 2]
    c.lens[4] = 3
    before = [x.clone() for x in arrays(c.pool)]
    parents = parents_of(c, trees)
    parents[10 + 2] = 2  # token 2 of row 2: its own parent
    path = torch.full((len(rows), 2), -5, dtype=torch.int32, device=c.device)
    new = api.kv_tree_commit(c.pool, parents, torch.tensor(leaves, dtype=torch.int32, device=c.device), c.cu, c.bt,
                             c.lens, path=path)
    assert c.pool.read_status() == api.DEV_BAD_TREE | api.DEV_BAD_LENGTH
    last = T.branch(trees[5], 2)
    assert new.tolist() == [35, 35, 24 + 3, 1030, 3, len(last)]
    assert path.tolist()[:5] == [[-5, -5], [-5, -5], [2, 4], [-5, -5], [-5, -5]]  # cut at the stride
    c.rows = [(0, 0), (0, 0), (6, 30), (0, 0), (0, 0), (3, 3)]
    trees[2] = [-1, -1, -1, 5, 2, 4]
    want, _ = committed(c, trees, [-1, -1, 5, -1, -1, 2], slice(0, 1), before)
    assert same(arrays(c.pool), want)


def test_commit_of_pages_outside_the_pool():
    c = filled(api.F16, [(40, 60)], seed=4)
    trees = [[-1, -1] + list(range(1, 39))]
    before = [x.clone() for x in arrays(c.pool)]
    good = c.bt.clone()
    c.bt[0, 2] = c.num_pages
    new = api.kv_tree_commit(c.pool, parents_of(c, trees), torch.tensor([39], dtype=torch.int32, device=c.device), c.cu,
                             c.bt, c.lens)
    assert c.pool.read_status() == api.DEV_BAD_PAGE and new.tolist() == [59]
    c.bt = good
    want, _ = committed(c, trees, [39], slice(0, 1), before)
    for d in range(39):  # the tokens that would come from or go to the page stay
        if 32 <= 20 + d < 48 or 32 <= 21 + d < 48:
            at = int(good[0, (20 + d) // 16]), (20 + d) % 16
            for w, b in zip(want, before):
                w[0, at[0], :, at[1]] = b[0, at[0], :, at[1]]
    assert same(arrays(c.pool), want)


def test_commit_without_tokens_and_in_a_graph():
    c = filled(api.F16, [(0, 0), (0, 33)], seed=4)
    before = [x.clone() for x in arrays(c.pool)]
    none = torch.full((2,), -1, dtype=torch.int32, device=c.device)
    new = api.kv_tree_commit(c.pool, torch.empty(0, dtype=torch.int32, device=c.device), none, c.cu, c.bt, c.lens)
    assert new.tolist() == [0, 33] and same(arrays(c.pool), before)
    c = filled(api.F16, [(20, 90), (30, 30)], seed=5, layers=2)
    parents = parents_of(c, [T.forest(20, c.gen), T.forest(30, c.gen)])
    leaf = torch.tensor([19, 29], dtype=torch.int32, device=c.device)
    new = torch.zeros(2, dtype=torch.int32, device=c.device)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        api.kv_tree_commit(c.pool, parents, leaf, c.cu, c.bt, c.lens, new_lens=new, stream=side)
    for _ in range(3):
        trees = [T.forest(20, c.gen), T.forest(30, c.gen)]
        leaves = [int(torch.randint(-1, 20, (1,), generator=c.gen)), int(torch.randint(-1, 30, (1,), generator=c.gen))]
        parents.copy_(parents_of(c, trees))
        leaf.copy_(torch.tensor(leaves))
        before = [x.clone() for x in arrays(c.pool)]
        graph.replay()
        torch.cuda.synchronize()
        want, paths = committed(c, trees, leaves, slice(0, 2), before)
        assert same(arrays(c.pool), want)
        assert new.tolist() == [70 + len(paths[0]), len(paths[1])]


# ---------------------------------------------------------------------- together ----
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 6)])
@pytest.mark.parametrize("kv", TYPES)
def test_a_step_of_speculative_decoding(kv, window, sinks):
    """Draft, store, attend, accept, commit, go on: each drafted token gets what it gets as the last token of a row
    that holds its branch alone, and the committed cache is that row's, bit for bit."""
    gen = torch.Generator().manual_seed(7)
    rows, n_kv, group = [(12, 100), (20, 33), (7, 7)], 2, 4
    c = R.Chunk(kv, n_kv, group, rows, seed=7, layers=2, layer=1)
    io = R.IO[kv]
    for layer in (0, 1):
        c.pool.set_window(layer, window)
        c.pool.set_sinks(layer, sinks)
    trees, parents = drafted(c)
    depth = torch.tensor([len(T.branch(t, j)) - 1 for t in trees for j in range(len(t))], dtype=torch.int32)
    past = torch.tensor([L - n for n, L in rows for _ in range(n)], dtype=torch.int32)
    positions = (past + depth)[None].to(c.device)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(c.device)
    q, k, v = (torch.randn(c.tokens, h, 128, generator=gen).to(c.device).to(io) for h in (c.n_q, n_kv, n_kv))
    context = [x.clone() for x in arrays(c.pool)]
    qr = torch.empty_like(q)
    for layer in (0, 1):
        api.kv_rope_append(c.pool, layer, q, k, v, positions, inv, (64,), c.cu, c.bt, c.lens, q_out=qr)
    _, out, lse = run(c, parents, qr)
    T.check(c, qr, out, lse, SCALE, trees=trees, window=window, sinks=sinks)
    stored = [x.clone() for x in arrays(c.pool)]

    leaves = [int(torch.randint(0, n, (1,), generator=gen)) for n, _ in rows]
    new = api.kv_tree_commit(c.pool, parents, torch.tensor(leaves, dtype=torch.int32, device=c.device), c.cu, c.bt, c.lens)
    after = [x.clone() for x in arrays(c.pool)]
    for i, ((n, L), leaf) in enumerate(zip(rows, leaves)):
        line = T.branch(trees[i], leaf)
        at = int(c.cu[i]) + torch.tensor(line, device=c.device)
        assert int(new[i]) == L - n + len(line)
        # the branch alone: its tokens appended in turn to the context
        for x, y in zip(arrays(c.pool), context):
            x.copy_(y)
        cu = torch.tensor([0, len(line)], dtype=torch.int32, device=c.device)
        pos = torch.arange(L - n, L - n + len(line), dtype=torch.int32, device=c.device)[None].contiguous()
        for layer in (0, 1):
            turned = api.kv_rope_append(c.pool, layer, q[at], k[at], v[at], pos, inv, (64,), cu, c.bt[i:i + 1],
                                        new[i:i + 1])
        assert torch.equal(turned, qr[at])
        for x, y in zip(arrays(c.pool), after):
            for t in range(L - n + len(line)):
                page = int(c.bt[i, t // 16])
                assert torch.equal(x[:, page, :, t % 16].contiguous().view(torch.uint8),
                                   y[:, page, :, t % 16].contiguous().view(torch.uint8))
        alone = api.paged_chunk_attention(c.pool, 1, turned, cu, c.bt[i:i + 1], new[i:i + 1], SCALE)
        want, tol, _, _ = T.attention(one_row(c, i, len(line), L - n + len(line)), turned, SCALE, window=window, sinks=sinks)
        assert ((alone.double() - want).abs() <= tol).all()
        assert ((out[at].double() - want).abs() <= tol).all()
    for x, y in zip(arrays(c.pool), after):
        x.copy_(y)
    # the next token of each row, on the committed cache
    lens = new + 1
    x, kn, vn = (torch.randn(3, h, 128, generator=gen).to(c.device) for h in (c.n_q, n_kv, n_kv))
    c.bt = c.bt.clone()
    spare = c.spare.to(c.device)
    for i, L in enumerate(lens.tolist()):  # a row whose whole tree was accepted needs a page more
        if int(c.bt[i, (L - 1) // 16]) < 0:
            c.bt[i, (L - 1) // 16] = spare[i]
    step = api.decode_step(c.pool, 1, x, kn, vn, c.bt, lens, SCALE)
    c.rows = [(1, L) for L in lens.tolist()]
    c.cu = torch.arange(4, dtype=torch.int32, device=c.device)
    c.tokens = 3
    T.check(c, x, step, None, SCALE, window=window, sinks=sinks)


def one_row(c, i, n, L):
    class Row:
        pass

    r = Row()
    r.kv, r.n_kv, r.n_q, r.rows, r.tokens = c.kv, c.n_kv, c.n_q, [(n, L)], n
    r.cu = torch.tensor([0, n])
    r.stored = lambda which, _: c.stored(which, i, L)
    return r


@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_pages_beyond_32_bits(kv):
    """Rows in the last pages of a pool whose K alone is more than 4 GiB: the bits of the same rows in a small pool."""
    rows, n_kv = [(33, 200), (1, 700), (64, 90)], 8
    c = R.Chunk(kv, n_kv, 4, rows, seed=3)
    per_page = n_kv * 16 * 128 * (1 if kv == api.Q8_0 else 2)
    pages = (5 << 30) // per_page
    big = api.KVPool(1, pages, n_kv, kv, device="cuda")
    for x, y in zip(arrays(big), arrays(c.pool)):
        x[0, pages - c.num_pages:] = y[0]
    bt = torch.where(c.bt >= 0, c.bt + (pages - c.num_pages), c.bt)
    trees, parents = drafted(c)
    leaves = torch.tensor([32, 0, 63], dtype=torch.int32, device=c.device)
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    x = c.normal(3, c.n_q, 128)
    got = []
    for pool, table in ((c.pool, c.bt), (big, bt)):
        pool.set_window(0, 100)
        pool.set_sinks(0, 5)
        out = [api.paged_tree_attention(pool, 0, q, parents, c.cu, table, c.lens, SCALE),
               api.paged_decode_attention(pool, 0, x, table, c.lens, SCALE, num_chunks=1),
               api.kv_tree_commit(pool, parents, leaves, c.cu, table, c.lens)]
        assert pool.read_status() == 0
        got.append(out + [y[0, -c.num_pages:].contiguous().view(torch.uint8) for y in arrays(pool)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
