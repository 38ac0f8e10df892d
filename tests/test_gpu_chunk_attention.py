"""paged_chunk_attention and paged_attention_mass on the GPU against their 64-bit definitions: formats, groups,
ragged rows, masks, caps and biases, strides, splits, streams and graphs."""
import math

import pytest
import torch

import chunk_reference as R
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
RAGGED = [(1, 1), (1, 17), (3, 3), (16, 40), (0, 12), (33, 33), (5, 300), (130, 131), (0, 0), (257, 700)]


def check(c, q, out, lse, **kw):
    want, tol, wl, lt = R.attention(c, q, SCALE, **kw)
    n = int(c.cu[-1])
    err = (out[:n].double() - want[:n]).abs()
    assert torch.isfinite(out[:n]).all()
    worst = (err - tol[:n]).max()
    assert worst <= 0, f"{float(worst)} over the tolerance, error {float(err.max())}"
    skipped = wl[:n] == -math.inf
    assert (lse[:n][skipped] == -math.inf).all()
    lerr = (lse[:n].double() - wl[:n]).abs()[~skipped]
    assert (lerr <= lt[:n][~skipped]).all(), float(lerr.max())
    assert c.pool.read_status() == 0


def run(c, q=None, workspace=None, **kw):
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[c.kv]) if q is None else q
    out = torch.full((c.tokens, c.n_q, 128), 7.0, dtype=q.dtype, device=c.device)
    lse = torch.full((c.tokens, c.n_q), 7.0, device=c.device)
    api.paged_chunk_attention(c.pool, c.layer, q, c.cu, c.bt, c.lens, SCALE, out=out, lse=lse, workspace=workspace,
                              **kw)
    return q, out, lse


@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_ragged_rows(kv, group):
    c = R.Chunk(kv, 2, group, RAGGED, seed=group, behind=3)
    q, out, lse = run(c)
    check(c, q, out, lse)
    assert (out[int(c.cu[-1]):] == 7).all() and (lse[int(c.cu[-1]):] == 7).all()  # tokens of no row


@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
@pytest.mark.parametrize("rows", [[(1, 5000)], [(1, 128)], [(1, 129)], [(64, 64)], [(600, 5003)], [(1, 1)] * 40,
                                  [(2, 2000), (1, 4097), (1, 3), (300, 2300)]])
def test_lengths(kv, rows):
    c = R.Chunk(kv, 2, 4, rows, seed=5)
    check(c, *run(c))


@pytest.mark.parametrize("window", [1, 16, 100, 128, 1000])
@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_window_reads_only_its_pages(kv, window):
    rows = [(70, 900), (1, 333), (300, 300)]
    c = R.Chunk(kv, 2, 2, rows, seed=window)
    c.pool.set_window(0, window)
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    full = c.bt.clone()
    for i, (n, L) in enumerate(rows):  # entries before the first page any query sees
        c.bt[i, :max(0, L - n + 1 - window) // 16] = -1
    _, out, lse = run(c, q)
    c.bt = full
    check(c, q, out, lse, window=window)


@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(softcap=2.0), dict(bias=True), dict(prefix=True),
                                dict(softcap=20.0, bias=True, prefix=True, window=77)])
@pytest.mark.parametrize("kv", [api.F16, api.BF16])
def test_scores(kv, kw):
    rows = [(200, 200), (40, 500), (1, 700), (129, 260)]
    c = R.Chunk(kv, 2, 4, rows, seed=3)
    a, b = {}, {}
    if "softcap" in kw:
        a["softcap"] = b["softcap"] = kw["softcap"]
    if kw.get("bias"):
        a["slopes"] = b["slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(c.n_q)], device=c.device)
    if kw.get("prefix"):
        a["prefix_lens"] = b["prefix_lens"] = torch.tensor([150, 470, 0, 9999], dtype=torch.int32, device=c.device)
    if "window" in kw:
        c.pool.set_window(0, kw["window"])
        b["window"] = kw["window"]
    q, out, lse = run(c, **a)
    check(c, q, out, lse, **b)


@pytest.mark.parametrize("kw", [dict(softcap=8.0), dict(softcap=1.5), dict(softcap=1e-3), dict(softcap=1e5),
                                dict(softcap=1e12), dict(scale=-0.2), dict(scale=0.0), dict(scale=-0.2, softcap=6.0),
                                dict(slope=-0.05), dict(slope=8.0), dict(slope=0.5, softcap=30.0, window=90),
                                dict(softcap=3.0, window=40, prefix=True), dict(slope=1.0, prefix=True)])
@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_scores_at_their_ends(kv, kw):
    """Caps near and far from the scores, scales that are not positive, biases that rise and fall steeply: chunks
    of both halves of a tile and single tokens."""
    rows = [(150, 700), (1, 650), (20, 20), (64, 300), (1, 1)]
    c = R.Chunk(kv, 2, 4, rows, seed=13)
    b = {k: v for k, v in kw.items() if k == "softcap"}
    if "slope" in kw:
        b["slopes"] = torch.tensor([kw["slope"] * 0.9 ** h for h in range(c.n_q)], device=c.device)
    if kw.get("prefix"):
        b["prefix_lens"] = torch.tensor([690, 0, 20, 128, 5], dtype=torch.int32, device=c.device)
    a, scale = dict(b), kw.get("scale", SCALE)
    if "window" in kw:
        c.pool.set_window(0, kw["window"])
        b["window"] = kw["window"]
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    lse = torch.empty(c.tokens, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, scale, lse=lse, **a)
    want, tol, wl, lt = R.attention(c, q, scale, **b)
    assert ((out.double() - want).abs() <= tol).all(), float(((out.double() - want).abs() - tol).max())
    assert ((lse.double() - wl).abs() <= lt).all(), float(((lse.double() - wl).abs() - lt).max())
    got = torch.zeros(len(rows), 2, 700, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, scale, mass_out=got, **a)
    want, tol = R.mass(c, q, lse, scale, torch.zeros_like(got), **b)
    for i, (n, L) in enumerate(rows):
        # a steep bias takes weights below fp32's normal numbers, where each of a token's n (n_q / n_kv) terms is
        # lost: less than 2^-126 each
        lost = n * (c.n_q // c.n_kv) * 2.0 ** -126
        assert ((got[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L] + lost).all(), i


def test_large_scores():
    """Scores of several hundred: the running maximum is raised by far more than exp's range."""
    c = R.Chunk(api.F16, 1, 4, [(140, 900)], seed=2, spread=30.0)
    check(c, *run(c))


@pytest.mark.parametrize("bad", [math.nan, math.inf, 6e4])
@pytest.mark.parametrize("kv", [api.F16, api.BF16])
def test_unseen_values_never_reach_an_output(kv, bad):
    """K and V of a token of the chunk are not finite: queries before it, and queries whose window has passed it,
    are unaffected; a query that sees it shows it."""
    n, L, at = 150, 340, 250
    c = R.Chunk(kv, 2, 2, [(n, L), (3, 50)], seed=8)
    q, out, lse = run(c)
    page, slot = c.bt[0, at // 16].long(), at % 16
    c.pool.v_data[0, page, :, slot, 5] = bad
    c.pool.k_data[0, page, :, slot] = 0 if bad == 6e4 else bad
    _, out2, lse2 = run(c, q)
    first = at - (L - n)  # the first query that sees the token
    want, tol, wl, lt = R.attention(R.Chunk(kv, 2, 2, [(n, L), (3, 50)], seed=8), q, SCALE)
    assert ((out2.double() - want).abs() <= tol)[:first].all() and ((lse2.double() - wl).abs() <= lt)[:first].all()
    assert torch.equal(out2[n:], out[n:])
    if bad != 6e4:
        assert not torch.isfinite(out2[first:n, :, 5]).any()
    c.pool.set_window(0, 20)
    _, out3, _ = run(c, q)
    assert torch.isfinite(out3[first + 20:n]).all() and torch.isfinite(out3[:first]).all()


@pytest.mark.parametrize("chunks", [1, 2, 7, 50, 152, 400])
@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_splits(kv, chunks):
    c = R.Chunk(kv, 2, 4, [(90, 1500), (1, 2600), (200, 200), (1, 5)], seed=9)
    ws = api.WorkspaceChunk(c.pool, c.n_q, chunks)
    ws.tensor.fill_(255)  # NaN: no initialisation is needed
    check(c, *run(c, workspace=ws))


def test_strided_queries_and_other_layer():
    c = R.Chunk(api.BF16, 2, 4, [(70, 150), (1, 40)], seed=4, layers=3, layer=1)
    qkv = c.normal(c.tokens, c.n_q + 2 * c.n_kv, 128, dtype=torch.bfloat16)
    q = qkv[:, :c.n_q]
    assert not q.is_contiguous()
    _, out, lse = run(c, q)
    check(c, q, out, lse)


def test_rows_that_are_skipped():
    """Lengths that do not fit record BAD_LENGTH: zeros for a valid chunk, nothing for an invalid one."""
    c = R.Chunk(api.F16, 2, 2, [(4, 20), (5, 33), (6, 100)], seed=1)
    c.lens[1] = 3  # fewer tokens than new ones
    q, out, lse = run(c)
    assert c.pool.read_status() == api.DEV_BAD_LENGTH
    assert (out[4:9] == 0).all() and (lse[4:9] == -math.inf).all()
    c.lens[1] = 33
    want, tol, _, _ = R.attention(c, q, SCALE)
    ok = (out.double() - want).abs() <= tol
    assert ok[:4].all() and ok[9:].all()
    c.lens[1] = 16 * c.stride + 1
    run(c, q)
    assert c.pool.read_status() == api.DEV_BAD_LENGTH
    c.lens[1] = 33
    c.cu[2] = 2  # entries decrease: row 1 holds no valid chunk
    run(c, q)
    assert c.pool.read_status() == api.DEV_BAD_LENGTH


def test_pages_outside_the_pool_are_reported():
    c = R.Chunk(api.F16, 2, 2, [(4, 20), (5, 33)], seed=1)
    c.bt[1, 1] = c.num_pages
    run(c)
    assert c.pool.read_status() == api.DEV_BAD_PAGE


def test_no_rows_and_no_tokens():
    c = R.Chunk(api.F16, 2, 2, [(0, 5), (0, 0)], seed=1)
    _, out, _ = run(c)
    assert out.shape[0] == 0 and c.pool.read_status() == 0


def test_streams_and_graph():
    """The same calls on another stream, and captured and replayed with new inputs."""
    c = R.Chunk(api.F16, 2, 4, [(65, 500), (1, 900)], seed=6)
    ws = api.WorkspaceChunk(c.pool, c.n_q)
    q, out, lse = run(c, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    mass = torch.zeros(2, 2, 1000, device=c.device)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=out2, lse=lse2, workspace=ws)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=out2, lse=lse2, workspace=ws)
        api.paged_attention_mass(c.pool, 0, q, lse2, c.cu, c.bt, c.lens, SCALE, mass_out=mass)
    q.copy_(c.normal(*q.shape, dtype=q.dtype))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check(c, q, out2, lse2)
    want, tol = R.mass(c, q, lse2, SCALE, torch.zeros_like(mass))
    for i, (_, L) in enumerate(c.rows):
        assert ((mass[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all()


@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_replayed_with_other_lengths(kv):
    """A captured call follows the lengths that the device holds when it is replayed: other rows, fewer tokens, a
    row without any."""
    c = R.Chunk(kv, 2, 4, [(65, 500), (1, 900), (200, 260)], seed=6)
    ws, wm = api.WorkspaceChunk(c.pool, c.n_q), api.WorkspaceMass(c.pool, c.n_q)
    q, out, lse = run(c, workspace=ws)
    mass = torch.zeros(3, 2, 1000, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=mass, workspace=wm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=out, lse=lse, workspace=ws)
        api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=mass, workspace=wm)
    for rows in ([(1, 120), (150, 900), (0, 10)], [(266, 400), (0, 0), (0, 260)], [(1, 1), (1, 900), (1, 2)]):
        c.rows = rows
        c.cu.copy_(torch.tensor([0] + [n for n, _ in rows]).cumsum(0))
        c.lens.copy_(torch.tensor([L for _, L in rows]))
        mass.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        check(c, q, out, lse)
        want, tol = R.mass(c, q, lse, SCALE, torch.zeros_like(mass))
        for i, (_, L) in enumerate(rows):
            assert ((mass[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all()
            assert (mass[i, :, L:] == -1).all()


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace, give the bits that they give alone."""
    c = R.Chunk(api.BF16, 2, 4, [(65, 500), (1, 4000), (300, 1500)] + [(1, 700)] * 20, seed=16)
    q, out, lse = run(c)
    mass = api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE,
                                    mass_out=torch.zeros(23, 2, 4000, device=c.device))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [(api.WorkspaceChunk(c.pool, c.n_q), api.WorkspaceMass(c.pool, c.n_q)) for _ in streams]
    outs = [(torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(mass)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (ws, wm), (o, l, m) in zip(streams, spaces, outs):
            api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=o, lse=l, workspace=ws, stream=st)
            api.paged_attention_mass(c.pool, 0, q, l, c.cu, c.bt, c.lens, SCALE, mass_out=m, workspace=wm, stream=st)
    torch.cuda.synchronize()
    for o, l, m in outs:
        assert torch.equal(o, out) and torch.equal(l, lse) and torch.equal(m, mass)


def test_scratch_belongs_to_the_calls_stream(monkeypatch):
    """Scratch that a call makes for a stream of its own is not handed to the current stream while that one may
    still use it."""
    c = R.Chunk(api.F16, 2, 4, [(65, 500), (1, 900)], seed=6)
    made = []
    for name in ("WorkspaceChunk", "WorkspaceMass"):
        def note(*a, make=getattr(api, name)):
            made.append(make(*a))
            return made[-1]
        monkeypatch.setattr(api, name, note)
    side = torch.cuda.Stream()
    q, out, lse = run(c)
    del made[:]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    _, out2, lse2 = run(c, q, stream=side)  # its outputs are filled before, on the current stream
    mass = api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, stream=side,
                                    mass_out=torch.zeros(2, 2, 900, device=c.device))
    at, sizes = [w.tensor.data_ptr() for w in made], [w.nbytes for w in made]
    assert len(at) == 2
    del made[:]
    for size in sizes:
        assert torch.empty(size, dtype=torch.uint8, device=c.device).data_ptr() not in at
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and bool((mass[0, :, :500] > 0).all())


# ------------------------------------------------------------------------ mass ----
@pytest.mark.parametrize("last", [0, 1, 20])
@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_mass(kv, group, last):
    c = R.Chunk(kv, 2, group, RAGGED + [(300, 1400)], seed=group)
    q, _, lse = run(c)
    before = torch.rand(len(c.rows), c.n_kv, 1403, device=c.device)
    got = torch.full_like(before, 5.0)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, last_queries=last, mass_in=before,
                             mass_out=got)
    want, tol = R.mass(c, q, lse, SCALE, before, last=last)
    for i, (_, L) in enumerate(c.rows):
        err = (got[i, :, :L].double() - want[i, :, :L]).abs()
        assert (err <= tol[i, :, :L]).all(), (i, float(err.max()))
        assert (got[i, :, L:] == 5).all()
    again = before.clone()  # in place, and the same bits
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, last_queries=last, mass_in=again)
    for i, (_, L) in enumerate(c.rows):
        assert torch.equal(again[i, :, :L], got[i, :, :L])
    assert c.pool.read_status() == 0


@pytest.mark.parametrize("chunks", [1, 2, 7, 152, 400])
@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_mass_splits(kv, chunks):
    c = R.Chunk(kv, 2, 4, [(90, 1500), (1, 2600), (700, 900), (1, 5)], seed=9)
    q, _, lse = run(c)
    ws = api.WorkspaceMass(c.pool, c.n_q, chunks)
    ws.tensor.fill_(255)  # NaN: no initialisation is needed
    before = torch.rand(4, 2, 2600, device=c.device)
    got = api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_in=before,
                                   mass_out=torch.empty_like(before), workspace=ws)
    want, tol = R.mass(c, q, lse, SCALE, before)
    for i, (_, L) in enumerate(c.rows):
        assert ((got[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all(), i
    assert c.pool.read_status() == 0


def test_mass_ignores_what_is_not_a_query():
    """Tokens behind the last row, another row's queries and a query without an lse may hold anything."""
    c = R.Chunk(api.F16, 2, 4, [(5, 90), (40, 300)], seed=2, behind=20)
    q, _, lse = run(c)
    want, tol = R.mass(c, q, lse, SCALE, torch.zeros(2, 2, 300, device=c.device))
    q[45:], lse[45:] = math.nan, math.nan
    got = torch.zeros(2, 2, 300, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=got)
    for i, (_, L) in enumerate(c.rows):
        assert ((got[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all(), i
    q[5:45], lse[7, 3] = math.nan, math.nan  # row 1's queries: NaN
    lse[5:45] = math.nan
    got = torch.zeros(2, 2, 300, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=got)
    assert ((got[0, :, :90].double() - want[0, :, :90]).abs() <= tol[0, :, :90]).all()
    assert (got[1] == 0).all()


@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(bias=True), dict(prefix=True), dict(window=50),
                                dict(softcap=20.0, bias=True, prefix=True, window=77)])
def test_mass_scores(kw):
    c = R.Chunk(api.F16, 2, 4, [(200, 200), (40, 500), (1, 700), (129, 260)], seed=3)
    a, b = {}, {}
    if "softcap" in kw:
        a["softcap"] = b["softcap"] = kw["softcap"]
    if kw.get("bias"):
        a["slopes"] = b["slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(c.n_q)], device=c.device)
    if kw.get("prefix"):
        a["prefix_lens"] = b["prefix_lens"] = torch.tensor([150, 470, 0, 9999], dtype=torch.int32, device=c.device)
    if "window" in kw:
        c.pool.set_window(0, kw["window"])
        b["window"] = kw["window"]
    q, _, lse = run(c, **a)
    got = torch.zeros(4, 2, 700, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=got, **a)
    want, tol = R.mass(c, q, lse, SCALE, torch.zeros_like(got), **b)
    for i, (n, L) in enumerate(c.rows):
        assert ((got[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all(), i
        total = got[i, :, :L].sum()  # every query and head hands out a weight of 1
        assert abs(float(total) - n * c.n_q) <= 1e-3 * n * c.n_q


def test_mass_of_rows_that_do_not_fit():
    c = R.Chunk(api.F16, 2, 2, [(4, 20), (5, 33), (6, 100)], seed=1)
    q, _, lse = run(c)
    got = torch.full((3, 2, 40), 5.0, device=c.device)  # too narrow for row 2
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=got)
    assert c.pool.read_status() == api.DEV_BAD_LENGTH
    assert (got[2] == 5).all() and (got[0, :, 20:] == 5).all()
    want, tol = R.mass(c, q, lse, SCALE, torch.zeros(3, 2, 100, device=c.device))
    for i, (_, L) in enumerate(c.rows[:2]):
        assert ((got[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all()


def test_mass_skips_queries_without_a_finite_lse():
    c = R.Chunk(api.F16, 2, 2, [(40, 90)], seed=1)
    q, _, lse = run(c)
    lse[5], lse[7, 1], lse[9] = -math.inf, math.nan, math.inf
    got = torch.zeros(1, 2, 90, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=got)
    finite = lse.masked_fill(~torch.isfinite(lse), math.inf)  # exp(s - inf) = 0
    want, tol = R.mass(c, q, finite, SCALE, torch.zeros_like(got))
    assert ((got.double() - want).abs() <= tol).all()


def test_bounded_waits():
    """The test hook stalls every wait: the call gives up, says so, and the next one is whole again."""
    c = R.Chunk(api.F16, 2, 4, [(65, 500), (1, 900)], seed=6)
    c.pool.set_test_stall(2_000_000)
    q, _, lse = run(c)
    assert c.pool.read_status() & api.DEV_TIMEOUT
    mass = torch.zeros(2, 2, 900, device=c.device)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=mass)
    assert c.pool.read_status() & api.DEV_TIMEOUT
    c.pool.set_test_stall(0)
    q, out, lse = run(c, q)
    check(c, q, out, lse)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=mass)
    want, tol = R.mass(c, q, lse, SCALE, torch.zeros_like(mass))
    for i, (_, L) in enumerate(c.rows):
        assert ((mass[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all()
