"""kv_rope_append and kv_evict on the GPU against their definitions, and the four long-prompt calls in a row."""
import math

import numpy as np
import pytest
import torch

import chunk_reference as R
import oracle as O
from helpers import int8_codes
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

FORMATS = [api.F16, api.BF16, api.F32, api.Q8_0]
TYPES = [torch.float16, torch.bfloat16, torch.float32]


def sections_of(half, axes):
    a = half // (axes + 1)
    return tuple([a] * (axes - 1) + [half - a * (axes - 1)])


def positions_of(c, axes, far=0):
    p = torch.randint(0, 4000, (axes, c.tokens), generator=c.gen).to(torch.int32)
    return (p + far).to(torch.int32).to(c.device)


def freqs(rot, device):
    h = rot // 2
    return (500000.0 ** (-torch.arange(h, dtype=torch.float64) / h)).float().to(device)


def rotated_tolerance(x, pair, t):
    # cos and sin: the fp32 argument is off by 2^-25 of a half turn (9.4e-8), sincospif by 2 ulp (1.2e-7); two
    # products and a sum in fp32 add 3 * 2^-24: 4e-7 of |x| + |y| in all.  Then the rounding to t.
    return 4e-7 * pair + R.half_step(t) * x.abs() + R.tiny(t)


@pytest.mark.parametrize("t_out", TYPES)
@pytest.mark.parametrize("t_in", TYPES)
@pytest.mark.parametrize("rot,axes,interleaved", [(128, 1, False), (96, 3, False), (64, 2, True), (16, 1, True),
                                                  (128, 4, True), (32, 2, False)])
def test_queries_and_keys(t_in, t_out, rot, axes, interleaved):
    c = R.Chunk(api.F32, 2, 4, [(3, 3), (1, 40), (0, 9), (20, 61)], seed=rot, behind=2)
    qkv = c.normal(c.tokens, c.n_q + 2 * c.n_kv, 128, dtype=t_in)
    q, k, v = qkv[:, :c.n_q], qkv[:, c.n_q:c.n_q + c.n_kv], qkv[:, c.n_q + c.n_kv:]
    pos, inv, sec = positions_of(c, axes), freqs(rot, c.device), sections_of(rot // 2, axes)
    q_out = torch.full((c.tokens, c.n_q, 128), 9.0, dtype=t_out, device=c.device)
    kd, vd = c.pool.k_data.clone(), c.pool.v_data.clone()
    api.kv_rope_append(c.pool, 0, q, k, v, pos, inv, sec, c.cu, c.bt, c.lens, q_out=q_out, interleaved=interleaved)
    n = int(c.cu[-1])
    want, pair = R.rotate(q, pos, inv, sec, interleaved)
    assert ((q_out.double() - want).abs() <= rotated_tolerance(want, pair, t_out))[:n].all()
    assert (q_out[n:] == 9).all()
    wk, pk = R.rotate(k, pos, inv, sec, interleaved)
    for i, (m, L) in enumerate(c.rows):
        a = int(c.cu[i])
        for j in range(m):
            p = L - m + j
            at = (0, c.bt[i, p // 16].long(), slice(None), p % 16)
            err = (c.pool.k_data[at].double() - wk[a + j]).abs()
            assert (err <= rotated_tolerance(wk[a + j], pk[a + j], torch.float32)).all()
            assert torch.equal(c.pool.v_data[at], v[a + j].float())
            c.pool.k_data[at], c.pool.v_data[at] = kd[at], vd[at]
    same = lambda x, y: torch.equal(x.view(torch.int32), y.view(torch.int32))  # noqa: E731
    assert same(c.pool.k_data, kd) and same(c.pool.v_data, vd)  # nothing else was written
    assert c.pool.read_status() == 0


@pytest.mark.parametrize("rot", [128, 96, 64, 16])
@pytest.mark.parametrize("kv", FORMATS)
def test_stored_formats_are_the_appends(kv, rot):
    """At position 0 nothing turns: K and V are stored bit for bit as the oracle encodes them."""
    c = R.Chunk(kv, 3, 2, [(5, 21), (1, 16), (40, 70)], seed=rot, layers=2, layer=1)
    k, v = c.normal(c.tokens, 3, 128), c.normal(c.tokens, 3, 128)
    k[3, 1, 32:64] = 0  # a q8_0 block of zeros
    pos = torch.zeros(1, c.tokens, dtype=torch.int32, device=c.device)
    assert api.kv_rope_append(c.pool, 1, None, k, v, pos, freqs(rot, c.device), (rot // 2,), c.cu, c.bt, c.lens) is None
    torch.cuda.synchronize()
    assert c.pool.read_status() == 0
    for name, x in (("k", k), ("v", v)):
        data, scales = O.encode_pool(kv, x.cpu().numpy()[None])
        got = getattr(c.pool, name + "_data")[1]
        for i, (n, L) in enumerate(c.rows):
            a = int(c.cu[i])
            for j in range(n):
                p = L - n + j
                row = got[c.bt[i, p // 16].long(), :, p % 16].cpu()
                if kv == api.Q8_0:
                    np.testing.assert_array_equal(int8_codes(row.numpy()), data[0, a + j])
                    sc = getattr(c.pool, name + "_scales")[1][c.bt[i, p // 16].long(), :, p % 16].cpu()
                    np.testing.assert_array_equal(sc.view(torch.int16).numpy().view(np.uint16), scales[0, a + j])
                elif kv == api.F32:
                    np.testing.assert_array_equal(row.numpy(), data[0, a + j])
                else:
                    np.testing.assert_array_equal(row.view(torch.int16).numpy().view(np.uint16), data[0, a + j])


@pytest.mark.parametrize("rot,interleaved", [(128, False), (96, False), (64, True)])
def test_q8_0_keys(rot, interleaved):
    """A stored key is off by half a code, the scale's f16 rounding (127 codes of it) and the rotation."""
    c = R.Chunk(api.Q8_0, 2, 1, [(70, 100)], seed=rot)
    k, v = c.normal(c.tokens, 2, 128, dtype=torch.bfloat16), c.normal(c.tokens, 2, 128, dtype=torch.bfloat16)
    pos, inv = positions_of(c, 1), freqs(rot, c.device)
    api.kv_rope_append(c.pool, 0, None, k, v, pos, inv, (rot // 2,), c.cu, c.bt, c.lens, interleaved=interleaved)
    want, pair = R.rotate(k, pos, inv, (rot // 2,), interleaved)
    got = c.stored("k", 0)[:, 30:].transpose(0, 1)
    d = want.reshape(70, 2, 4, 32).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 32).reshape(70, 2, 128) / 127
    tol = d * (0.5 + 127 * R.half_step(torch.float16)) * (1 + 1e-5) + 4e-7 * pair + 127 * R.tiny(torch.float16)
    assert ((got - want).abs() <= tol).all()


def test_far_positions():
    """Positions near 2^31 keep fp32 accuracy: the angle is reduced in 64 bits."""
    c = R.Chunk(api.F32, 1, 1, [(64, 64)], seed=3)
    q, k, v = (c.normal(c.tokens, 1, 128) for _ in range(3))
    inv = freqs(128, c.device)
    for far in (1_000_000, 2**31 - 5000, -(2**31)):
        pos = (torch.randint(0, 4000, (1, c.tokens), generator=c.gen) + far).to(torch.int32).to(c.device)
        got = api.kv_rope_append(c.pool, 0, q, k, v, pos, inv, (64,), c.cu, c.bt, c.lens)
        want, pair = R.rotate(q, pos, inv, (64,), False)
        # the reference's own product, 55 bits in 53, is off by 2^-53 * 2^31 = 2.4e-7 of a radian
        assert ((got.double() - want).abs() <= rotated_tolerance(want, pair, torch.float32) + 2.4e-7 * pair).all()


def test_in_place_and_many_tokens():
    c = R.Chunk(api.F16, 2, 4, [(4500, 4600), (1, 9)], seed=2)
    q = c.normal(c.tokens, c.n_q, 128, dtype=torch.float16)
    k, v = c.normal(c.tokens, 2, 128, dtype=torch.float16), c.normal(c.tokens, 2, 128, dtype=torch.float16)
    pos, inv = positions_of(c, 1), freqs(128, c.device)
    apart = api.kv_rope_append(c.pool, 0, q, k, v, pos, inv, (64,), c.cu, c.bt, c.lens)
    want, pair = R.rotate(q, pos, inv, (64,), False)
    assert ((apart.double() - want).abs() <= rotated_tolerance(want, pair, torch.float16)).all()
    api.kv_rope_append(c.pool, 0, q, k, v, pos, inv, (64,), c.cu, c.bt, c.lens, q_out=q)
    assert torch.equal(q, apart)


def test_rope_skips_what_does_not_fit():
    c = R.Chunk(api.F16, 2, 1, [(4, 20), (5, 33), (6, 100)], seed=1)
    q, k, v = (c.normal(c.tokens, 2, 128) for _ in range(3))
    pos, inv = positions_of(c, 1), freqs(128, c.device)
    args = (pos, inv, (64,), c.cu, c.bt)
    kd = c.pool.k_data.clone()
    lens = c.lens.clone()
    lens[1] = 4
    got = api.kv_rope_append(c.pool, 0, q, k, v, *args, lens)
    assert c.pool.read_status() == api.DEV_BAD_LENGTH
    want, pair = R.rotate(q, pos, inv, (64,), False)
    assert ((got.double() - want).abs() <= rotated_tolerance(want, pair, torch.float32)).all()
    row = c.bt[1, :3].long()
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731
    assert same(c.pool.k_data[0, row], kd[0, row])
    c.bt[2, 6] = -7
    api.kv_rope_append(c.pool, 0, q, k, v, *args, c.lens)
    assert c.pool.read_status() == api.DEV_BAD_PAGE


# ----------------------------------------------------------------------- evict ----
def evict_case(kv, rows, budgets, seed=0, n_kv=2, layers=1, layer=0):
    """A Chunk of rows whose last pages are fresh ones for the kept tokens."""
    c = R.Chunk(kv, n_kv, 1, [(0, L) for L in rows] + [(0, max(1, B)) for B in budgets], seed=seed, layers=layers,
                layer=layer)
    n = len(rows)
    return c, c.bt[:n].contiguous(), c.lens[:n].contiguous(), c.bt[n:].contiguous()


def check_evict(c, bt, lens, dst, mass, budgets, first, recent):
    n = len(budgets)
    rows = [int(x) for x in lens]
    arrays = [x for x in (c.pool.k_data, c.pool.v_data, c.pool.k_scales, c.pool.v_scales) if x is not None]
    before = [x.clone() for x in arrays]
    keep_lens = torch.tensor(budgets, dtype=torch.int32, device=c.device)
    width = max(max(min(L, B) for L, B in zip(rows, budgets)), 1) + 1
    idx = torch.full((n, c.n_kv, width), -5, dtype=torch.int32, device=c.device)
    kept_mass = torch.full((n, c.n_kv, width), -5.0, device=c.device)
    _, new = api.kv_evict(c.pool, c.layer, mass, bt, lens, keep_lens, dst, first=first, recent=recent, keep_idx=idx,
                          dst_mass=kept_mass)
    assert new.tolist() == [min(L, B) for L, B in zip(rows, budgets)]
    assert c.pool.read_status() == 0
    for i, (L, B) in enumerate(zip(rows, budgets)):
        for h in range(c.n_kv):
            want = R.keep(mass[i, h].tolist(), L, B, first, recent)
            m = len(want)
            assert idx[i, h, :m].tolist() == want
            assert (idx[i, h, m:] == -5).all() and (kept_mass[i, h, m:] == -5).all()
            if not m:
                continue
            w = torch.tensor(want, device=c.device)
            assert torch.equal(kept_mass[i, h, :m].view(torch.int32), mass[i, h][w].view(torch.int32))
            b = torch.arange(m, device=c.device)
            for x, old in zip(arrays, before):
                got = x[c.layer][dst[i][b // 16].long(), h, b % 16]
                src = old[c.layer][bt[i][w // 16].long(), h, w % 16]
                assert torch.equal(got.view(torch.uint8), src.view(torch.uint8))
                x[c.layer][dst[i][b // 16].long(), h, b % 16] = old[c.layer][dst[i][b // 16].long(), h, b % 16]
    for x, old in zip(arrays, before):
        assert torch.equal(x.view(torch.uint8), old.view(torch.uint8))  # nothing else was written


@pytest.mark.parametrize("first,recent", [(0, 0), (4, 32), (1, 0), (0, 500), (500, 3)])
@pytest.mark.parametrize("kv", FORMATS)
def test_evict(kv, first, recent):
    rows, budgets = [1, 17, 700, 1033, 300, 0, 64], [1, 16, 250, 100, 300, 5, 0]
    c, bt, lens, dst = evict_case(kv, rows, budgets, seed=first + recent)
    mass = torch.exp(2 * c.normal(len(rows), c.n_kv, 1040))
    check_evict(c, bt, lens, dst, mass, budgets, first, recent)


def test_evict_ties_and_special_weights():
    rows, budgets = [900, 900, 900, 900], [400, 400, 899, 33]
    c, bt, lens, dst = evict_case(api.F16, rows, budgets, seed=4)
    mass = torch.randint(0, 3, (4, 2, 900), generator=c.gen).float().to(c.device)
    mass[1] = 0.0
    mass[1, :, ::2] = -0.0  # equal to 0
    mass[2, 0, 100:200], mass[2, 1, 300:] = math.nan, math.inf
    mass[3, 0], mass[3, 1] = -math.inf, math.nan
    check_evict(c, bt, lens, dst, mass, budgets, 4, 16)


@pytest.mark.parametrize("L", [5000, 20000, 70001])
def test_evict_long_rows(L):
    c, bt, lens, dst = evict_case(api.Q8_0, [L, 33], [1500, 20], seed=L)
    mass = torch.exp(2 * c.normal(2, c.n_kv, L + 3))
    mass = torch.where(torch.rand(mass.shape, generator=c.gen).to(c.device) < 0.3, torch.zeros_like(mass), mass)
    check_evict(c, bt, lens, dst, mass, [1500, 20], 4, 64)


def test_evict_clamps_and_reports():
    c, bt, lens, dst = evict_case(api.F16, [100, 200], [40, 50])
    mass = torch.rand(2, 2, 150, device=c.device)  # too narrow for row 1: its first 150 tokens count
    keep = torch.tensor([-3, 50], dtype=torch.int32, device=c.device)
    idx, new = api.kv_evict(c.pool, 0, mass, bt, lens, keep, dst)
    assert c.pool.read_status() == api.DEV_BAD_LENGTH and new.tolist() == [0, 50]
    assert idx[1, 1, :50].tolist() == R.keep(mass[1, 1].tolist(), 150, 50, 0, 0)
    dst[1, 2] = -1
    api.kv_evict(c.pool, 0, mass, bt, torch.tensor([100, 150], dtype=torch.int32, device=c.device),
                 torch.tensor([40, 50], dtype=torch.int32, device=c.device), dst)
    assert c.pool.read_status() == api.DEV_BAD_PAGE


def test_evict_on_a_stream_of_its_own():
    """The kept indices that the call makes are filled on its stream, not behind the current one's work."""
    rows, budgets = [700, 300], [250, 300]
    c, bt, lens, dst = evict_case(api.F16, rows, budgets, seed=3)
    mass = torch.rand(2, c.n_kv, 700, generator=c.gen).to(c.device)
    keep = torch.tensor(budgets, dtype=torch.int32, device=c.device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy
    idx, new = api.kv_evict(c.pool, 0, mass, bt, lens, keep, dst, first=4, recent=16, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert new.tolist() == budgets
    for h in range(c.n_kv):
        assert idx[0, h, :250].tolist() == R.keep(mass[0, h].tolist(), 700, 250, 4, 16)
        assert idx[1, h, :300].tolist() == list(range(300))


# ---------------------------------------------------------------- all together ----
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.Q8_0])
def test_long_prompt_in_chunks_then_eviction_then_a_step(kv):
    """Two prompts taken in by chunks, evicted to a budget, and continued by one token: pages from the allocator,
    every value checked against the definitions at each step."""
    n_kv, group, layer = 2, 4, 0
    total, budget, recent = [150, 333], 96, 16
    c = R.Chunk(kv, n_kv, group, [(0, 1)], seed=11)  # only its generator and helpers
    alloc = api.PageAllocator(80, 8, 40)
    pool = c.pool = api.KVPool(1, 80, n_kv, kv, device=c.device)
    for t in (pool.k_scales, pool.v_scales) if kv == api.Q8_0 else (pool.k_data, pool.v_data):
        t.fill_(math.nan)
    seqs = [alloc.open(), alloc.open()]
    mass = torch.full((2, n_kv, 400), math.nan, device=c.device)
    done = [0, 0]
    inv = freqs(128, c.device)

    def step(new):
        c.rows = [(n, d + n) for n, d in zip(new, done)]
        for s, n in zip(seqs, new):
            alloc.reserve(s, n)
        for s, n in zip(seqs, new):
            alloc.commit(s, n)
        bt, sl = alloc.batch(seqs, 0, 40)
        assert sl.tolist() == [L for _, L in c.rows]
        c.bt, c.lens = torch.from_numpy(bt).to(c.device), torch.from_numpy(sl).to(c.device)
        c.cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device=c.device)
        c.tokens = sum(new)
        q, k, v = (c.normal(c.tokens, h, 128, dtype=R.IO[kv]) for h in (c.n_q, n_kv, n_kv))
        pos = torch.cat([torch.arange(p, p + n) for p, n in zip(text, new)])[None].to(torch.int32).to(c.device)
        for i, n in enumerate(new):
            text[i] += n
        qr = api.kv_rope_append(pool, layer, q, k, v, pos, inv, (64,), c.cu, c.bt, c.lens)
        want, pair = R.rotate(q, pos, inv, (64,), False)
        assert ((qr.double() - want).abs() <= rotated_tolerance(want, pair, qr.dtype)).all()
        lse = torch.empty(c.tokens, c.n_q, device=c.device)
        out = api.paged_chunk_attention(pool, layer, qr, c.cu, c.bt, c.lens, 1 / math.sqrt(128), lse=lse)
        o, tol, z, zt = R.attention(c, qr, 1 / math.sqrt(128))
        assert ((out.double() - o).abs() <= tol).all() and ((lse.double() - z).abs() <= zt).all()
        api.paged_attention_mass(pool, layer, qr, lse, c.cu, c.bt, c.lens, 1 / math.sqrt(128), mass_in=mass)
        for i in range(2):
            done[i] += new[i]

    text = [0, 0]
    step([100, 200])
    step([50, 133])
    assert done == total
    for i in range(2):
        got = float(mass[i, :, :total[i]].double().sum())
        assert abs(got - total[i] * c.n_q) <= 1e-3 * got  # every query and head handed out a weight of 1
    fresh = [alloc.open(), alloc.open()]
    alloc.reserve_many(fresh, budget)
    alloc.commit_many(fresh, budget)
    dst = torch.from_numpy(alloc.batch(fresh, 0, 40)[0]).to(c.device)
    keep = torch.full((2,), budget, dtype=torch.int32, device=c.device)
    kept_mass = torch.zeros(2, n_kv, 400, device=c.device)
    idx = torch.full((2, n_kv, 400), -1, dtype=torch.int32, device=c.device)
    old = [c.stored("k", i) for i in range(2)]
    _, new_lens = api.kv_evict(pool, layer, mass, c.bt, c.lens, keep, dst, first=2, recent=recent, keep_idx=idx,
                               dst_mass=kept_mass)
    for s in seqs:
        alloc.release(s)
    seqs[:], done[:] = fresh, [budget, budget]
    assert new_lens.tolist() == done
    c.bt, c.rows = dst, [(0, budget), (0, budget)]
    for i in range(2):
        now = c.stored("k", i)
        for h in range(n_kv):
            kept = R.keep(mass[i, h].tolist(), total[i], budget, 2, recent)
            assert idx[i, h, :budget].tolist() == kept
            assert torch.equal(now[h], old[i][h][kept])
    mass = kept_mass
    step([1, 1])
    assert pool.read_status() == 0
