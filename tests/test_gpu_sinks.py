"""Layers whose first tokens stay visible under their window (kv_pool_set_sinks), on the GPU against the 64-bit
definition: the single-token step, the fused append, and chunk attention."""
import ctypes
import math

import pytest
import torch

import chunk_reference as R
import tree_reference as T
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
ALL = [api.F16, api.BF16, api.F32, api.Q8_0]
LENGTHS = [1, 2, 5, 16, 17, 33, 100, 118, 300, 0, 1000, 5000]


def set_layer(c, window, sinks):
    c.pool.set_window(c.layer, window)
    c.pool.set_sinks(c.layer, sinks)
    assert c.pool.sinks(c.layer) == sinks


def close_gap(c, window, sinks):
    """Tokens that no query of the row attends to are NaN, the table entries of pages without any other -1.
    Returns the table as it was."""
    full = c.bt.clone()
    for i, (n, L) in enumerate(c.rows):
        first = max(0, L - n + 1 - window)  # of the first query's window
        T.spoil(c, [(i, t) for t in range(sinks, first)])
        for p in range(-(-sinks // 16), first // 16):
            c.bt[i, p] = -1
    return full


@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (17, 16), (100, 17), (100, 200), (7, 3), (5, 33), (1000, 64),
                                          (90, 0), (4096, 4)])
@pytest.mark.parametrize("kv", ALL)
def test_step(kv, window, sinks):
    c = R.Chunk(kv, 2, 4, [(min(1, L), L) for L in LENGTHS], seed=window)
    set_layer(c, window, sinks)
    q = c.normal(len(LENGTHS), c.n_q, 128)
    full = close_gap(c, window, sinks)
    out = api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE)
    c.bt = full
    assert (out[LENGTHS.index(0)] == 0).all()
    has = torch.tensor([L > 0 for L in LENGTHS], device=c.device)
    check_rows(c, q[has], out[has], window=window, sinks=sinks)


def check_rows(c, q, out, **kw):
    """The rows with a token, as the tokens of a chunk."""
    T.check(c, q, out, None, SCALE, **kw)


@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("kv", ALL)
def test_step_groups_chunks_and_layers(kv, group):
    """Work splits from one CTA to many more than there are pages, in the second layer of a pool."""
    c = R.Chunk(kv, 2, group, [(1, L) for L in (700, 40, 3000, 1)], seed=group, layers=2, layer=1)
    set_layer(c, 333, 21)
    q = c.normal(4, c.n_q, 128)
    full = close_gap(c, 333, 21)
    for chunks in (1, 3, 60, 456, 1000):
        out = api.paged_decode_attention(c.pool, 1, q, c.bt, c.lens, SCALE, num_chunks=chunks)
        bt, c.bt = c.bt, full
        check_rows(c, q, out, window=333, sinks=21)
        c.bt = bt


@pytest.mark.parametrize("window,sinks", [(1, 4), (2, 4), (20, 5), (64, 16), (300, 1)])
@pytest.mark.parametrize("kv", ALL)
def test_fused_step_stores_and_attends(kv, window, sinks):
    """The new token lands in its slot, in pages that hold sinks too, and counts."""
    rows = [(1, L) for L in (1, 4, 5, 6, 7, 16, 17, 18, 30, 400, 401)]
    c = R.Chunk(kv, 2, 2, rows, seed=sinks)
    set_layer(c, window, sinks)
    q, k, v = (c.normal(len(rows), h, 128) for h in (c.n_q, 2, 2))
    full = close_gap(c, window, sinks)
    before = [x.clone() for x in (c.pool.k_data, c.pool.v_data)]
    out = api.decode_step(c.pool, 0, q, k, v, c.bt, c.lens, SCALE)
    stored = [x.clone() for x in (c.pool.k_data, c.pool.v_data)]
    c.bt = full
    check_rows(c, q, out, window=window, sinks=sinks)
    for x, y in zip((c.pool.k_data, c.pool.v_data), before):
        x.copy_(y)
    api.kv_append(c.pool, 0, k, v, c.bt, c.lens)
    for x, y in zip((c.pool.k_data, c.pool.v_data), stored):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def run(c, q=None, workspace=None, **kw):
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[c.kv]) if q is None else q
    out = torch.full((c.tokens, c.n_q, 128), 7.0, dtype=q.dtype, device=c.device)
    lse = torch.full((c.tokens, c.n_q), 7.0, device=c.device)
    api.paged_chunk_attention(c.pool, c.layer, q, c.cu, c.bt, c.lens, SCALE, out=out, lse=lse, workspace=workspace, **kw)
    return q, out, lse


@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (100, 17), (50, 150), (128, 128), (200, 3), (333, 64), (30, 400)])
@pytest.mark.parametrize("kv,group", [(api.F16, 4), (api.F16, 1), (api.BF16, 4), (api.BF16, 2), (api.Q8_0, 4), (api.Q8_0, 2)])
def test_chunk(kv, group, window, sinks):
    """Chunks and single tokens: gaps inside a block, between blocks, and none."""
    c = R.Chunk(kv, 2, group, [(1, 1), (1, 700), (40, 40), (0, 12), (70, 900), (300, 300), (5, 1500), (260, 1100)],
                seed=window, behind=2)
    set_layer(c, window, sinks)
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    full = close_gap(c, window, sinks)
    _, out, lse = run(c, q)
    c.bt = full
    T.check(c, q, out, lse, SCALE, window=window, sinks=sinks)
    assert (out[int(c.cu[-1]):] == 7).all() and (lse[int(c.cu[-1]):] == 7).all()


@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(softcap=2.0), dict(bias=True), dict(prefix=True),
                                dict(softcap=20.0, bias=True, prefix=True)])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_chunk_scores(kv, kw):
    rows = [(200, 200), (40, 500), (1, 700), (129, 460)]
    c = R.Chunk(kv, 2, 4, rows, seed=3)
    set_layer(c, 77, 9)
    a = {k: v for k, v in kw.items() if k == "softcap"}
    if kw.get("bias"):
        a["slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(c.n_q)], device=c.device)
    if kw.get("prefix"):
        a["prefix_lens"] = torch.tensor([150, 470, 0, 9999], dtype=torch.int32, device=c.device)
    q, out, lse = run(c, **a)
    T.check(c, q, out, lse, SCALE, window=77, sinks=9, **a)


@pytest.mark.parametrize("chunks", [1, 2, 7, 152, 400])
@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_chunk_splits(kv, chunks):
    c = R.Chunk(kv, 2, 4, [(90, 1000), (1, 2100), (300, 310), (64, 640)], seed=4)
    set_layer(c, 400, 130)
    q, out, lse = run(c, workspace=api.WorkspaceChunk(c.pool, c.n_q, chunks))
    T.check(c, q, out, lse, SCALE, window=400, sinks=130)


def test_chunk_planned_by_the_cta():
    """More rows and tiles than one warp plans."""
    c = R.Chunk(api.F16, 1, 4, [(1, 30 + 9 * i) for i in range(70)] + [(2100, 2200)], seed=8)
    set_layer(c, 150, 20)
    q, out, lse = run(c)
    T.check(c, q, out, lse, SCALE, window=150, sinks=20)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_unseen_values_never_reach_an_output(kv, bad):
    """A token that the first queries of a tile see and the later ones do not, in the sinks' block and behind it:
    the later ones are whole."""
    c = R.Chunk(kv, 2, 4, [(300, 300), (60, 420)], seed=5)
    set_layer(c, 50, 4)
    tokens = [(0, 20), (0, 100), (1, 375)]
    q, clean, clean_lse = run(c)
    T.check(c, q, clean, clean_lse, SCALE, window=50, sinks=4)
    T.spoil(c, tokens, bad)
    _, out, lse = run(c, q)
    for i, (n, L) in enumerate(c.rows):
        show = T.seen(n, L, 50, 4)
        hit = torch.zeros(n, dtype=torch.bool)
        for r, t in tokens:
            if r == i:
                hit |= show[:, t]
        a = int(c.cu[i])
        whole = torch.arange(a, a + n)[~hit].to(c.device)
        want, tol, wl, lt = T.attention(clean_copy(c, tokens), q, SCALE, window=50, sinks=4)
        assert ((out[whole].double() - want[whole]).abs() <= tol[whole]).all()
        assert ((lse[whole].double() - wl[whole]).abs() <= lt[whole]).all()
        assert not torch.isfinite(out[torch.arange(a, a + n)[hit].to(c.device)]).all()


def clean_copy(c, tokens):
    T.spoil(c, tokens, 1.0)
    return c


def test_no_window_no_effect():
    """Sinks without a window, and a window that reaches them: the results without sinks, bit for bit where one CTA
    does all the work (the pieces of a split row are merged in the order in which they finish)."""
    for kv in ALL:
        c = R.Chunk(kv, 2, 2, [(1, 300), (1, 40)], seed=2)
        q = c.normal(2, c.n_q, 128)
        plain = api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE, num_chunks=1)
        for window, sinks in ((0, 5), (290, 10), (1000, 3)):
            set_layer(c, window, sinks)
            assert torch.equal(plain, api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE, num_chunks=1))
            T.check(c, q, api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE), None, SCALE)


def test_step_without_a_workspace():
    """The entry point with scratch of the library's own serves sinks as well."""
    c = R.Chunk(api.Q8_0, 2, 4, [(1, L) for L in (700, 40, 3, 1500)], seed=3)
    set_layer(c, 200, 33)
    q = c.normal(4, c.n_q, 128)
    out = torch.zeros_like(q)
    fn = api.lib().paged_decode_attention_static
    fn.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                   ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    assert fn(c.pool.handle, 0, q.data_ptr(), c.bt.data_ptr(), c.bt.shape[1], c.lens.data_ptr(), 4, c.n_q, SCALE,
              out.data_ptr(), 0, torch.cuda.current_stream().cuda_stream) == 0
    check_rows(c, q, out, window=200, sinks=33)


def test_calls_that_refuse_sinks():
    c = R.Chunk(api.F16, 2, 2, [(2, 300)], seed=2)
    set_layer(c, 100, 4)
    q = c.normal(1, 2, c.n_q, 128)
    lse = torch.zeros(2, c.n_q, device=c.device)
    ws = api.Workspace(c.pool, c.n_q, 1)
    calls = [
        lambda: api.paged_decode_attention_mq(c.pool, 0, q, c.bt, c.lens, SCALE),
        lambda: api.decode_step_mq(c.pool, 0, q, q[:, :, :2].contiguous(), q[:, :, :2].contiguous(), c.bt, c.lens, SCALE),
        lambda: api.paged_decode_split(c.pool, 0, q[:, 0].contiguous(), c.bt, c.lens, SCALE, torch.empty_like(q[:, 0]), ws),
        lambda: api.paged_attention_mass(c.pool, 0, q[0].half(), lse, c.cu, c.bt, c.lens, SCALE,
                                         mass_out=torch.zeros(1, 2, 300, device=c.device)),
    ]
    for call in calls:
        with pytest.raises(api.PkvError, match="sinks"):
            call()
    c.pool.set_window(0, 0)  # without a window they are no sinks
    for call in calls:
        call()
    assert c.pool.read_status() == 0


def test_graph_with_other_lengths():
    """A captured step and a captured chunk follow the lengths on the device."""
    c = R.Chunk(api.F16, 2, 4, [(1, 900), (1, 300), (1, 2000)], seed=9)
    set_layer(c, 200, 18)
    q = c.normal(3, c.n_q, 128)
    qh = q.half()
    out, outh, lse = torch.zeros_like(q), torch.zeros_like(qh), torch.zeros(3, c.n_q, device=c.device)
    ws, wc = api.Workspace(c.pool, c.n_q, 3), api.WorkspaceChunk(c.pool, c.n_q)

    def call():
        api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE, out=out, workspace=ws)
        api.paged_chunk_attention(c.pool, 0, qh, c.cu, c.bt, c.lens, SCALE, out=outh, lse=lse, workspace=wc)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ((900, 300, 2000), (5, 219, 218), (217, 1, 1999)):
        c.rows = [(1, L) for L in lengths]
        c.lens.copy_(torch.tensor(lengths))
        graph.replay()
        torch.cuda.synchronize()
        T.check(c, q, out, None, SCALE, window=200, sinks=18)
        T.check(c, qh, outh, lse, SCALE, window=200, sinks=18)


@pytest.mark.parametrize("kv", ALL)
def test_bounded_waits(kv):
    c = R.Chunk(kv, 2, 4, [(1, 500), (1, 900)], seed=6)
    set_layer(c, 100, 20)
    q = c.normal(2, c.n_q, 128)
    c.pool.set_test_stall(2_000_000)
    api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE)
    assert c.pool.read_status() & api.DEV_TIMEOUT
    if kv != api.F32:
        run(c)
        assert c.pool.read_status() & api.DEV_TIMEOUT
    c.pool.set_test_stall(0)
    T.check(c, q, api.paged_decode_attention(c.pool, 0, q, c.bt, c.lens, SCALE), None, SCALE, window=100, sinks=20)
    if kv != api.F32:
        qh, out, lse = run(c)
        T.check(c, qh, out, lse, SCALE, window=100, sinks=20)
