"""Values at the ends of the stored formats, and values that must not reach a result, in paged_chunk_attention and
paged_attention_mass."""
import math

import pytest
import torch

import chunk_reference as R
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
ROWS = [(150, 340), (1, 70), (3, 50)]
AT = (250, 33, 49)  # a token of each row: inside the chunk, before the only query, the last one
KW = [{}, {"softcap": 30.0}, {"slope": 0.01}, {"slope": 0.01, "softcap": 30.0}]


def test_rows_computed_again_do_not_stop_the_rest():
    """A value that is not finite in the last token of a long row: the 252 (query, head) rows of the tile that do
    not attend to it are computed again, two KV heads by one CTA.  Row by row in the middle of the pipeline that
    took 1.5 seconds a head, beyond the limit of the waits behind it (a second)."""
    n, L = 64, 200_000
    c = R.Chunk(api.F16, 2, 4, [(n, L)], seed=31)
    c.pool.v_data[0, c.bt[0, (L - 1) // 16].long(), :, (L - 1) % 16, 5] = math.inf
    q = c.normal(n, c.n_q, 128, dtype=torch.float16)
    lse = torch.empty(n, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse,
                                    workspace=api.WorkspaceChunk(c.pool, c.n_q, 1))
    torch.cuda.synchronize()
    assert c.pool.read_status() == 0
    assert torch.isinf(out[-1, :, 5]).all()
    assert torch.isfinite(out[:-1]).all() and torch.isfinite(out[-1, :, 6:]).all()
    c.pool.v_data[0, c.bt[0, (L - 1) // 16].long(), :, (L - 1) % 16, 5] = 0
    want, tol, wl, lt = R.attention(c, q, SCALE)
    assert ((out.double() - want).abs() <= tol)[:-1].all() and ((lse.double() - wl).abs() <= lt).all()


@pytest.mark.parametrize("kv", [api.F16, api.BF16])
def test_pieces_beyond_those_told_apart(kv):
    """1400 pieces in one CTA's range, values that are not finite in the first and the last ones: the queries before
    such a value are whole in every row."""
    rows = [(2, 19 + i % 5) for i in range(700)]
    c = R.Chunk(kv, 2, 2, rows, seed=32)
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    want, tol, wl, lt = R.attention(c, q, SCALE)
    bad = (0, 5, 350, 650, 698, 699)
    for i in bad:
        L = rows[i][1]
        c.pool.v_data[0, c.bt[i, (L - 1) // 16].long(), :, (L - 1) % 16, 9] = math.nan
    lse = torch.empty(c.tokens, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse,
                                    workspace=api.WorkspaceChunk(c.pool, c.n_q, 1))
    sees = torch.tensor([2 * i + 1 for i in bad], device=c.device)
    assert torch.isnan(out[sees][..., 9]).all()
    out[sees] = want[sees].to(out.dtype)
    assert ((out.double() - want).abs() <= tol).all() and ((lse.double() - wl).abs() <= lt).all()
    assert c.pool.read_status() == 0


# ------------------------------------------------------- q8_0: a block's scale may be any f16 ----
def put(c, which, scale, code, block=1, dim=37):
    """Token AT of each row: one 32-wide block of K or V is `code` in one dim and 0 in the others, under `scale`."""
    for i, t in enumerate(AT):
        page = c.bt[i, t // 16].long()
        data, scales = getattr(c.pool, which + "_data")[0], getattr(c.pool, which + "_scales")[0]
        data[page, :, t % 16, 32 * block:32 * block + 32] = 128
        data[page, :, t % 16, dim] = 128 + code
        scales[page, :, t % 16, block] = scale


def queries(c, which):
    q = c.normal(c.tokens, c.n_q, 128, dtype=torch.float16)
    if which == "k":
        q[..., 37] *= 2.0 ** -12  # scores of the size of the others
    return q


def zero_key(c):
    """K of the tokens AT is 0: their weights stay far from 1, and V times weight within f16's range."""
    for i, t in enumerate(AT):
        c.pool.k_data[0][c.bt[i, t // 16].long(), :, t % 16] = 128


def scores_of(c, kw):
    a = {k: v for k, v in kw.items() if k == "softcap"}
    if "slope" in kw:
        a["slopes"] = torch.full((c.n_q,), kw["slope"], device=c.device)
    return a


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("chunks", [1, 152])
@pytest.mark.parametrize("kw", KW)
@pytest.mark.parametrize("scale,code", [(511.5, -128), (512.0, 127), (600.0, -127), (-600.0, 127), (60000.0, 2)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_large_q8_0_values(which, scale, code, kw, chunks, window):
    """Stored values around and beyond f16's 65504, for queries that see them and queries that do not."""
    c = R.Chunk(api.Q8_0, 2, 4, ROWS, seed=21)
    c.pool.set_window(0, window)
    q = queries(c, which)
    if which == "v":
        zero_key(c)
    put(c, which, scale, code)
    a = scores_of(c, kw)
    out, lse = torch.empty(c.tokens, c.n_q, 128, dtype=torch.float16, device=c.device), \
        torch.empty(c.tokens, c.n_q, device=c.device)
    api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=out, lse=lse,
                              workspace=api.WorkspaceChunk(c.pool, c.n_q, chunks), **a)
    want, tol, wl, lt = R.attention(c, q, SCALE, window=window, **a)
    assert want.abs().max() < 65000
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert ((out.double() - want).abs() <= tol).all(), float(((out.double() - want).abs() - tol).max())
    assert ((lse.double() - wl).abs() <= lt).all()
    assert c.pool.read_status() == 0


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("kw", KW)
@pytest.mark.parametrize("scale,code", [(511.5, -128), (512.0, 127), (600.0, -127), (-600.0, 127), (60000.0, 2)])
def test_mass_of_large_q8_0_keys(scale, code, kw, window):
    c = R.Chunk(api.Q8_0, 2, 4, ROWS, seed=22)
    c.pool.set_window(0, window)
    q = queries(c, "k")
    put(c, "k", scale, code)
    a = scores_of(c, kw)
    lse = R.attention(c, q, SCALE, window=window, **a)[2].float()
    before = torch.rand(3, 2, 340, device=c.device)
    got = api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_in=before,
                                   mass_out=torch.empty_like(before), **a)
    want, tol = R.mass(c, q, lse, SCALE, before, window=window, **a)
    for i, (_, L) in enumerate(c.rows):
        assert ((got[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all(), i
    assert c.pool.read_status() == 0


@pytest.mark.parametrize("group", [1, 2])
def test_large_q8_0_values_of_other_groups(group):
    """One and two query heads a KV head; every tenth token has values beyond f16's range, in K and in V."""
    c = R.Chunk(api.Q8_0, 2, group, [(300, 900), (1, 77)], seed=25)
    q = queries(c, "k")
    for i, (_, L) in enumerate(c.rows):
        t = torch.arange(3, L, 10, device=c.device)
        page = c.bt[i][t // 16].long()
        for name, scale in (("k", 700.0), ("v", -900.0)):
            data, scales = getattr(c.pool, name + "_data")[0], getattr(c.pool, name + "_scales")[0]
            data[page, :, t % 16, 32:64] = 128
            data[page, :, t % 16, 37] = 128 + 100
            scales[page, :, t % 16, 1] = scale
    lse = torch.empty(c.tokens, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse)
    want, tol, wl, lt = R.attention(c, q, SCALE)
    over = want.abs() - tol >= 65520  # infinite in f16
    assert (out[over].double() == want[over].sign() * math.inf).all()
    held = want.abs() + tol < 65504
    assert ((out.double() - want).abs() <= tol)[held].all() and ((lse.double() - wl).abs() <= lt).all()
    assert held.float().mean() > 0.99
    mass = torch.rand(2, 2, 900, device=c.device)
    want, tol = R.mass(c, q, lse, SCALE, mass)
    api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_in=mass)  # in place
    for i, (_, L) in enumerate(c.rows):
        assert ((mass[i, :, :L].double() - want[i, :, :L]).abs() <= tol[i, :, :L]).all(), i
    assert c.pool.read_status() == 0


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("kw", KW)
@pytest.mark.parametrize("scale,code", [(math.nan, 1), (math.inf, -3), (600.0, 127)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_unseen_q8_0_values_never_reach_an_output(which, scale, code, kw, window):
    """Queries before the token, and queries whose window has passed it, are as without it."""
    c = R.Chunk(api.Q8_0, 2, 4, ROWS, seed=23)
    c.pool.set_window(0, window)
    q, a = queries(c, which), scores_of(c, kw)
    if which == "v":
        zero_key(c)
    want, tol, wl, lt = R.attention(c, q, SCALE, window=window, **a)
    put(c, which, scale, code)
    lse = torch.empty(c.tokens, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse, **a)
    for i, (n, L) in enumerate(ROWS):
        s = int(c.cu[i])
        pos = torch.arange(L - n, L, device=c.device)
        sees = (pos >= AT[i]) & ((pos < AT[i] + window) | (window == 0))
        off = s + torch.nonzero(~sees).flatten()
        assert ((out.double() - want).abs() <= tol)[off].all() and ((lse.double() - wl).abs() <= lt)[off].all(), i
        if not math.isfinite(scale):
            assert not torch.isfinite(out[s + torch.nonzero(sees).flatten()][..., 37]).any()


# ------------------------------------------------------------------------ caps ----
@pytest.mark.parametrize("kw", [{"softcap": 30.0}, {"slope": 0.02, "softcap": 30.0}])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_capped_scores_do_not_depend_on_what_is_not_seen(kv, kw):
    """Keys behind a row's end, keys that come after a query, and queries behind the last row may hold anything:
    the same bits come out (a cap's arithmetic is chosen for groups of scores together)."""
    rows = [(70, 250), (1, 301), (3, 77), (1, 1)]
    c = R.Chunk(kv, 2, 4, rows, seed=24, behind=30)
    a = scores_of(c, kw)
    a["prefix_lens"] = torch.tensor([400, 0, 100, 9], dtype=torch.int32, device=c.device)
    n = int(c.cu[-1])
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    one = 128 + 127 if kv == api.Q8_0 else 1.0

    def fill(big, last):
        """Slots behind the rows' ends and queries behind the last row: 0, or far beyond the cap."""
        for i, (_, L) in enumerate(rows):
            page = c.bt[i, (L - 1) // 16].long()
            c.pool.k_data[0, page, :, (L - 1) % 16 + 1:] = one
            if kv == api.Q8_0:
                c.pool.k_scales[0, page, :, (L - 1) % 16 + 1:] = 100.0 * big
            else:
                c.pool.k_data[0, page, :, (L - 1) % 16 + 1:] *= 1000.0 * big
        q[n:] = 1000.0 * big
        page = c.bt[0, 249 // 16].long()  # the last token of row 0's chunk
        if last is not None:
            c.pool.k_data[0, page, :, 249 % 16] = 128 if kv == api.Q8_0 else last

    def both():
        lse = torch.zeros(c.tokens, c.n_q, device=c.device)
        out = torch.zeros_like(q)
        api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, out=out, lse=lse, **a)
        mass = torch.zeros(4, 2, 310, device=c.device)
        api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_out=mass, last_queries=40, **a)
        return out, lse, mass

    fill(0.0, None)
    want = both()
    fill(1.0, None)
    got = both()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    # no prefix: a key that only the last query of row 0 sees
    a["prefix_lens"] = torch.zeros(4, dtype=torch.int32, device=c.device)
    if kv != api.Q8_0:
        fill(0.0, 0.0)
        want = both()
        fill(0.0, 500.0)
        got = both()
        for x, y in zip(got[:2], want[:2]):
            assert torch.equal(x[:69], y[:69]) and torch.equal(x[70:], y[70:])
