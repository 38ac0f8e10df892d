"""Plain 64-bit forms of the long-prompt operators, and the inputs of their tests.

Everything here is written from the definitions in include/pkv_chunk.h with torch in float64, token by token or
row by row; the kernels' outputs are compared with it under tolerances derived from their roundings:
  half step of a type t: torch.finfo(t).eps / 2, relative to the value (plus half its smallest subnormal);
  a score: q and K are exact in the products, which accumulate in fp32 over 128 dims in at most 16 rounded steps of
  the tensor core or 128 fused steps of a CUDA core, each off by at most 2^-23 (truncation) of the running sum,
  itself at most S = scale * sum |q k|.  Typical sums are far smaller than S, whose terms cancel; 16 * 2^-23 * S is
  taken for both (the CUDA-core chain rounds to nearest, 128 steps of random sign: sqrt(128) * 2^-24 * S)."""
from __future__ import annotations

import math

import torch

from paged_kv_decode_09_gb300 import api

D, PAGE, QB = 128, 16, 32
IO = {api.F16: torch.float16, api.BF16: torch.bfloat16, api.Q8_0: torch.float16, api.F32: torch.float32}
STORE = {api.F16: torch.float16, api.BF16: torch.bfloat16, api.F32: torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of the type's subnormals."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def pages(n):
    return (n + PAGE - 1) // PAGE


class Chunk:
    """A pool with random contents and the rows [(new tokens, tokens in the cache)] of a chunk call.

    Unused table entries are -1; slots behind a row's last token and pages of no row hold NaN.  The token arrays
    carry `behind` tokens behind the last row."""

    def __init__(self, kv, n_kv, group, rows, seed=0, behind=0, layers=1, layer=0, device="cuda", spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.n_kv, self.n_q, self.rows, self.layer = kv, n_kv, n_kv * group, rows, layer
        self.device = torch.device(device, torch.cuda.current_device()) if device == "cuda" else torch.device(device)
        need = [pages(L) for _, L in rows]
        self.num_pages = sum(need) + 3
        ids = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.stride = max(need + [1]) + 1
        bt = torch.full((len(rows), self.stride), -1, dtype=torch.int32)
        at = 0
        used = torch.zeros(self.num_pages, PAGE, dtype=torch.bool)
        for i, x in enumerate(need):
            bt[i, :x] = ids[at:at + x]
            for p in range(x):
                used[bt[i, p].long(), :min(PAGE, rows[i][1] - PAGE * p)] = True
            at += x
        self.spare = ids[at:]
        self.bt = bt.to(self.device)
        self.cu = torch.tensor([0] + [n for n, _ in rows], dtype=torch.int32).cumsum(0).to(torch.int32).to(self.device)
        self.lens = torch.tensor([L for _, L in rows], dtype=torch.int32, device=self.device)
        self.tokens = sum(n for n, _ in rows) + behind
        self.pool = api.KVPool(layers, self.num_pages, n_kv, kv, device=self.device)
        shape = (self.num_pages, n_kv, PAGE, D)
        mask = used.to(self.device)[:, None, :, None].expand(self.num_pages, n_kv, PAGE, 1)
        for data, scales in ((self.pool.k_data, self.pool.k_scales), (self.pool.v_data, self.pool.v_scales)):
            x = (torch.randn(shape, generator=g) * spread).to(self.device)
            if kv == api.Q8_0:
                b = x.reshape(*shape[:-1], D // QB, QB)
                d = (b.abs().amax(-1, keepdim=True) / 127.0).half()
                c = (b / d.float()).round().clamp(-127, 127)
                data[layer].copy_((c + 128).to(torch.uint8).reshape(shape))
                scales[layer].copy_(d.squeeze(-1).masked_fill(~mask, float("nan")))
            else:
                data[layer].copy_(x.to(STORE[kv]).masked_fill(~mask, float("nan")))
        self.gen = g

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.gen).to(self.device).to(dtype)

    def stored(self, which, i, L=None):
        """K ("k") or V ("v") of row i in float64: [n_kv][L][128]."""
        L = self.rows[i][1] if L is None else L
        pg = self.bt[i, :pages(L)].long()
        data = getattr(self.pool, which + "_data")[self.layer][pg].double()
        if self.kv == api.Q8_0:
            sc = getattr(self.pool, which + "_scales")[self.layer][pg].double()
            data = (data - 128) * sc.repeat_interleave(QB, -1)
        return data.transpose(0, 1).reshape(self.n_kv, -1, D)[:, :L]


def scores(c, q, i, scale, window=0, softcap=0.0, slopes=None, prefix=0):
    """(scores [n_q][n][L] of row i in float64, -inf where not attended; their rounding bound S)."""
    n, L = c.rows[i]
    a = int(c.cu[i])
    k = c.stored("k", i).repeat_interleave(c.n_q // c.n_kv, 0)
    qd = q[a:a + n].double().transpose(0, 1)
    dot = qd @ k.transpose(1, 2)
    size = qd.abs() @ k.abs().transpose(1, 2) * abs(scale)
    s = dot * scale
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    p = torch.arange(L - n, L, device=q.device)[:, None]
    t = torch.arange(L, device=q.device)[None]
    if slopes is not None:
        s = s - slopes.double()[:, None, None] * (p - t).abs().double()
        size = size + slopes.double().abs()[:, None, None] * (p - t).abs().double() * 2 ** -2
    seen = t < torch.clamp(p + 1, min=prefix)
    if window:
        seen = seen & (t >= p + 1 - window)
    return s.masked_fill(~seen, -math.inf), size.masked_fill(~seen, 0.0)


SCORE_STEPS = 16 * 2.0 ** -23


def attention(c, q, scale, prefix_lens=None, **kw):
    """(out, its tolerance, lse, its tolerance) in float64; rows without tokens stay zero / -inf."""
    io = IO[c.kv]
    out = torch.zeros(c.tokens, c.n_q, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((c.tokens, c.n_q), -math.inf, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for i, (n, L) in enumerate(c.rows):
        if n == 0 or L < n:
            continue
        a = int(c.cu[i])
        s, size = scores(c, q, i, scale, prefix=0 if prefix_lens is None else int(prefix_lens[i]), **kw)
        v = c.stored("v", i).repeat_interleave(c.n_q // c.n_kv, 0)
        # the largest score error of each query; exp2 and the division add a few 2^-22
        ds = size.amax(-1) * SCORE_STEPS + s.masked_fill(s == -math.inf, 0).abs().amax(-1) * 2.0 ** -22 + 2.0 ** -20
        p = torch.softmax(s, -1)
        o, mag = p @ v, p @ v.abs()
        z = torch.logsumexp(s, -1)
        # weights rounded to the io type (q8_0: V as two f16 parts, 2^-21), the output rounded once
        t = half_step(io) * o.abs() + (half_step(io) + 2 * ds[..., None] + 2.0 ** -20) * mag + tiny(io)
        out[a:a + n], tol[a:a + n] = o.transpose(0, 1), t.transpose(0, 1)
        lse[a:a + n] = z.transpose(0, 1)
        ltol[a:a + n] = (ds + z.abs() * 2.0 ** -22 + 2.0 ** -20).transpose(0, 1)
    return out, tol, lse, ltol


def mass(c, q, lse, scale, mass_in, last=0, prefix_lens=None, **kw):
    """(mass_out [rows][n_kv][stride], its tolerance) in float64; entries from L on are NaN."""
    rows, n_kv, stride = mass_in.shape
    out = torch.full((rows, n_kv, stride), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for i, (n, L) in enumerate(c.rows):
        if L < n:
            continue
        out[i, :, :L] = mass_in[i, :, :L].double()
        out[i, :, L - n:L] = 0
        if n == 0:
            continue
        a = int(c.cu[i])
        s, size = scores(c, q, i, scale, prefix=0 if prefix_lens is None else int(prefix_lens[i]), **kw)
        w = torch.exp(s - lse[a:a + n].double().transpose(0, 1)[..., None])
        ds = size * SCORE_STEPS + s.masked_fill(s == -math.inf, 0).abs() * 2.0 ** -22 + 2.0 ** -20
        j0 = max(0, n - last) if last else 0
        out[i, :, :L] += w[:, j0:].sum(1).reshape(n_kv, -1, L).sum(1)
        tol[i, :, :L] = (w * ds)[:, j0:].sum(1).reshape(n_kv, -1, L).sum(1)
    # the fp32 sum of the weights: at most one rounding per addition of a few hundred terms in pairs
    return out, tol + out.abs() * 2.0 ** -18


def keep(w, L, B, first, recent):
    """Kept tokens of one (row, KV head) from its weights w [>= L] (a list), ascending."""
    B = min(L, B)
    r = min(recent, B)
    f = min(first, B - r)

    def rank(t):  # NaN below every number
        return (1, 0.0) if math.isnan(w[t]) else (0, -w[t])

    middle = sorted(range(f, L - r), key=lambda t: (rank(t), t))[:B - f - r]
    return sorted([*range(f), *middle, *range(L - r, L)])


def rotate(x, positions, inv_freq, sections, interleaved):
    """x [tokens][heads][128] turned by the angles, in float64; |x| + |y| of each dim's pair."""
    half = inv_freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    angle = positions[axis].double() * inv_freq.double()[:, None]  # [half][tokens]
    c, s = torch.cos(angle).t()[:, None], torch.sin(angle).t()[:, None]
    y = x.double().clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    y[..., one] = x[..., one].double() * c - x[..., two].double() * s
    y[..., two] = x[..., one].double() * s + x[..., two].double() * c
    pair = torch.zeros_like(y)
    pair[..., one] = pair[..., two] = x[..., one].double().abs() + x[..., two].double().abs()
    return y, pair
