"""Long-prompt calls at sizes that take the other forms of their work split: plans made by the whole CTA, more tiles
than it has threads, 64-bit unit counts, and four tokens a CTA of the rotated append."""
import math

import pytest
import torch

import chunk_reference as R
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


class Part:
    """The queries j .. j + 63 of row i of a chunk, as a chunk of their own."""

    def __init__(self, c, i, j):
        n, L = c.rows[i]
        m = min(64, n - j)
        self.at = int(c.cu[i]) + j
        self.kv, self.n_kv, self.n_q, self.layer, self.pool, self.device = c.kv, c.n_kv, c.n_q, c.layer, c.pool, c.device
        self.rows, self.bt, self.tokens = [(m, L - n + j + m)], c.bt[i:i + 1], m
        self.cu = torch.tensor([0, m], dtype=torch.int32)
    stored = R.Chunk.stored


@pytest.mark.parametrize("window", [0, 900])
@pytest.mark.parametrize("kv", [api.F16, api.Q8_0])
def test_attention_of_more_tiles_than_threads(kv, window):
    """407 tiles for 384 threads; 690,000 units of work over the KV heads (beyond the 32-bit form) in f16 without a
    window."""
    c = R.Chunk(kv, 4, 4, [(26000, 26500), (1, 300)], seed=41)
    c.pool.set_window(0, window)
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    lse = torch.empty(c.tokens, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse)
    assert c.pool.read_status() == 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for i, j in ((0, 0), (0, 64), (0, 9984), (0, 12345), (0, 20000), (0, 25936), (1, 0)):
        p = Part(c, i, j)
        at = slice(p.at, p.at + p.tokens)
        want, tol, wl, lt = R.attention(p, q[at], SCALE, window=window)
        assert ((out[at].double() - want).abs() <= tol).all(), (i, j)
        assert ((lse[at].double() - wl).abs() <= lt).all(), (i, j)


def sampled_mass(c, q, lse, i, tokens):
    """Weights of some tokens of row i in float64 [n_kv][tokens], without mass_in, and their tolerance."""
    n, L = c.rows[i]
    a = int(c.cu[i])
    k = c.stored("k", i)[:, tokens].repeat_interleave(c.n_q // c.n_kv, 0)
    qd = q[a:a + n].double().transpose(0, 1)
    s = qd @ k.transpose(1, 2) * SCALE
    size = qd.abs() @ k.abs().transpose(1, 2) * SCALE
    pos = torch.arange(L - n, L, device=c.device)[:, None]
    seen = tokens[None] <= pos
    w = torch.exp(s - lse[a:a + n].double().transpose(0, 1)[..., None]).masked_fill(~seen, 0.0)
    ds = size * R.SCORE_STEPS + s.abs() * 2.0 ** -22 + 2.0 ** -20
    both = torch.stack([w, w * ds]).sum(2).reshape(2, c.n_kv, -1, len(tokens)).sum(2)
    return both[0], both[1] + both[0] * 2.0 ** -18


@pytest.mark.parametrize("kv,rows", [
    (api.F16, [(5000, 120000)]),  # 469 tiles, 590,000 units
    (api.Q8_0, [(300, 9000), (0, 5000), (7, 4097)]),  # a stride beyond 4096 tokens
    (api.BF16, [(2 + i % 3, 90 + 20 * i) for i in range(40)]),  # more than 32 rows
])
def test_mass_planned_by_the_cta(kv, rows):
    n_kv = 8 if rows[0][1] == 120000 else 2
    c = R.Chunk(kv, n_kv, 4, rows, seed=42)
    q = c.normal(c.tokens, c.n_q, 128, dtype=R.IO[kv])
    lse = torch.empty(c.tokens, c.n_q, device=c.device)
    api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse)
    stride = max(L for _, L in rows) + 3
    before = torch.rand(len(rows), n_kv, stride, device=c.device)
    got = api.paged_attention_mass(c.pool, 0, q, lse, c.cu, c.bt, c.lens, SCALE, mass_in=before,
                                   mass_out=torch.full_like(before, -1.0))
    assert c.pool.read_status() == 0
    for i, (n, L) in enumerate(rows):
        assert (got[i, :, L:] == -1).all()
        if n == 0:
            assert torch.equal(got[i, :, :L], before[i, :, :L])
            continue
        old = before[i, :, :L].clone()
        old[:, L - n:] = 0
        total = (got[i, :, :L].double() - old.double()).sum()  # every query and head hands out a weight of 1
        assert abs(float(total) - n * c.n_q) <= 1e-3 * n * c.n_q
        tokens = torch.unique(torch.randint(0, L, (60,), generator=c.gen).clamp(0, L - 1)).to(c.device)
        tokens = torch.unique(torch.cat([tokens, torch.tensor([0, max(0, L - n), L - 1], device=c.device)]))
        want, tol = sampled_mass(c, q, lse, i, tokens)
        want = want + old[:, tokens].double()
        err = (got[i][:, tokens].double() - want).abs()
        assert (err <= tol + want.abs() * 2.0 ** -23).all(), (i, float(err.max()))


@pytest.mark.parametrize("t_in", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.F32, api.Q8_0])
def test_append_of_many_tokens_is_the_append_of_few(kv, t_in):
    """One call of 4201 tokens (four to a CTA) stores and turns what a call for each row does (one to a CTA)."""
    rows = [(2100, 2105), (2099, 2099), (2, 40)]
    c = R.Chunk(kv, 2, 2, rows, seed=43)
    qkv = c.normal(c.tokens, c.n_q + 2 * c.n_kv, 128, dtype=t_in)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    pos = torch.randint(0, 100000, (2, c.tokens), generator=c.gen).to(torch.int32).to(c.device)
    inv = (500000.0 ** (-torch.arange(48, dtype=torch.float64) / 48)).float().to(c.device)
    arrays = [x for x in (c.pool.k_data, c.pool.v_data, c.pool.k_scales, c.pool.v_scales) if x is not None]
    start = [x.clone() for x in arrays]
    whole = api.kv_rope_append(c.pool, 0, q, k, v, pos, inv, (20, 28), c.cu, c.bt, c.lens)
    after = [x.clone() for x in arrays]
    for x, old in zip(arrays, start):
        assert not torch.equal(x.view(torch.uint8), old.view(torch.uint8))
        x.copy_(old)
    for i, (n, _) in enumerate(rows):
        at = slice(int(c.cu[i]), int(c.cu[i]) + n)
        part = api.kv_rope_append(c.pool, 0, q[at], k[at], v[at], pos[:, at].contiguous(), inv, (20, 28),
                                  torch.tensor([0, n], dtype=torch.int32, device=c.device), c.bt[i:i + 1],
                                  c.lens[i:i + 1])
        assert torch.equal(part, whole[at])
    for x, y in zip(arrays, after):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert c.pool.read_status() == 0
