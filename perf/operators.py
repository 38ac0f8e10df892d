"""Workloads of the long-prompt operators: a ragged chunk of new tokens rotated and stored in the paged
cache, attention of the chunk over the cache, the attention weight each cached token has received, and
eviction from the cache by that weight.

Every case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` is one pass (in
elementary torch operations, or through the library's entry points when `own` is true), `exact` is the same
operator in 64 bits written from its definition, and `work` counts what a pass cannot do without."""
import math
import random

import torch

own = False

PAGE, D, QB = 16, 128, 32
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}
_KV_BYTES = {"f16": 256, "bf16": 256, "f32": 512, "q8_0": 136}  # one token of one KV head, K or V
_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases ----
def _case(op, kv, n_q, n_kv, rows, chunk_rows, new, past, mix, **more):
    """`chunk_rows` of the rows bring new[0] .. new[1] tokens, the others one; every row has past[0] ..
    past[1] tokens in the cache before them (`mix` picks the lengths, over their logarithm)."""
    return {"op": op, "kv": kv, "n_q": n_q, "n_kv": n_kv, "rows": rows, "chunk_rows": chunk_rows,
            "new_min": new[0], "new_max": new[1], "past_min": past[0], "past_max": past[1], "mix": mix, **more}


def _rope(io, n_q, n_kv, rows, chunk_rows, new, past, mix, axes, rot, interleaved):
    return _case("rope_append", io, n_q, n_kv, rows, chunk_rows, new, past, mix, axes=axes, rot=rot,
                 interleaved=interleaved)


def _attn(kv, n_q, n_kv, rows, chunk_rows, new, past, mix, window=0, softcap=0.0, bias=False, prefix=0):
    return _case("attention", kv, n_q, n_kv, rows, chunk_rows, new, past, mix, window=window, softcap=softcap,
                 bias=bias, prefix=prefix)


def _mass(kv, n_q, n_kv, rows, chunk_rows, new, past, mix, last, softcap=0.0):
    return _case("mass", kv, n_q, n_kv, rows, chunk_rows, new, past, mix, last=last, softcap=softcap)


def _evict(kv, n_kv, rows, past, mix, keep, first, recent):
    return _case("evict", kv, n_kv, n_kv, rows, 0, (1, 1), past, mix, keep=keep, first=first, recent=recent)


def listed():
    return [
        # one decode step of eight rows, rotated and stored: latency
        {"name": "rope_step_8x1", **_rope("f16", 16, 8, 8, 0, (1, 1), (256, 2048), 1, 1, 128, False)},
        # a prefill of four prompts with image positions (three axes), bf16 projections in one buffer
        {"name": "rope_prefill_bf16", **_rope("bf16", 32, 8, 4, 4, (1000, 4000), (0, 0), 2, 3, 128, False)},
        # eight rows with one query each: the shortest attention call, cache-bound
        {"name": "attn_step_f16", **_attn("f16", 32, 8, 8, 0, (1, 1), (1024, 8192), 3)},
        # one prompt of 8191 tokens from an empty cache: compute-bound
        {"name": "attn_prompt_bf16", **_attn("bf16", 32, 8, 1, 1, (8191, 8191), (0, 0), 4)},
        # the next 2048 tokens of a long prompt over a q8_0 cache
        {"name": "attn_chunk_q8_0", **_attn("q8_0", 32, 8, 1, 1, (2048, 2048), (30001, 30001), 5)},
        # a mixed batch: two chunks beside 30 decoding rows, scores capped
        {"name": "attn_mixed_cap_f16", **_attn("f16", 32, 8, 32, 2, (300, 700), (500, 6000), 6, softcap=50.0)},
        # short prompts with a distance bias and a prefix seen from everywhere
        {"name": "attn_bias_prefix_f16", **_attn("f16", 16, 8, 5, 5, (120, 900), (0, 64), 7, bias=True, prefix=200)},
        # a windowed layer over a long row
        {"name": "attn_window_bf16", **_attn("bf16", 32, 8, 2, 2, (1500, 4096), (9000, 14000), 8, window=4096)},
        # weights of the last 32 queries of each row over its whole cache, before an eviction
        {"name": "mass_last32_f16", **_mass("f16", 32, 8, 4, 4, (64, 512), (4096, 30000), 9, 32)},
        # weights of a whole chunk
        {"name": "mass_chunk_bf16", **_mass("bf16", 32, 8, 2, 2, (1500, 2048), (2000, 9000), 10, 0)},
        # a few short rows to 256 tokens each: latency
        {"name": "evict_small_f16", **_evict("f16", 8, 4, (500, 2048), 11, 256, 4, 32)},
        # eight long rows to 4096 tokens each
        {"name": "evict_long_bf16", **_evict("bf16", 8, 8, (4096, 32768), 12, 4096, 4, 128)},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "attention", "attention", "mass", "evict"])
    n_q, n_kv = rng.choice([(32, 8), (16, 8), (8, 8)])
    mix = rng.randrange(1 << 20)
    if op == "rope_append":
        rows = _log(rng, 1, 32)
        chunk_rows = rng.randrange(rows + 1)
        new_hi = _log(rng, 1, max(1, 8192 // max(chunk_rows, 1)))
        past_hi = _log(rng, 1, 4096)
        return _rope(rng.choice(["f16", "bf16"]), n_q, n_kv, rows, chunk_rows, (rng.randint(1, new_hi), new_hi),
                     (rng.randint(0, past_hi), past_hi), mix, rng.choice([1, 2, 3]), rng.choice([128, 64, 96]),
                     rng.random() < 0.3)
    if op == "attention":
        rows = _log(rng, 1, 32)
        chunk_rows = rng.randrange(min(rows, 6) + 1)
        new_hi = _log(rng, 1, max(1, 3000 // max(chunk_rows, 1)))
        past_hi = _log(rng, 1, max(1, min(16000, 60000 // rows)))
        return _attn(rng.choice(["f16", "bf16", "q8_0"]), n_q, n_kv, rows, chunk_rows,
                     (rng.randint(1, new_hi), new_hi), (rng.randint(0, past_hi), past_hi), mix,
                     window=rng.choice([0, 0, 1, 100, 1024, 4096]), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                     bias=rng.random() < 0.3, prefix=rng.choice([0, 0, 1, 77, 500]))
    if op == "mass":
        rows = _log(rng, 1, 16)
        chunk_rows = rng.randrange(min(rows, 4) + 1)
        new_hi = _log(rng, 1, max(1, 2048 // max(chunk_rows, 1)))
        past_hi = _log(rng, 1, max(1, min(16000, 60000 // rows)))
        return _mass(rng.choice(["f16", "bf16", "q8_0"]), n_q, n_kv, rows, chunk_rows,
                     (rng.randint(1, new_hi), new_hi), (rng.randint(0, past_hi), past_hi), mix,
                     rng.choice([0, 0, 1, 16, 32, 64]), softcap=rng.choice([0.0, 0.0, 30.0]))
    rows = _log(rng, 1, 8)
    past_hi = _log(rng, 16, 32768)
    keep = _log(rng, 1, 4096)
    return _evict(rng.choice(["f16", "bf16"]), n_kv, rows, (rng.randint(1, past_hi), past_hi), mix, keep,
                  rng.choice([0, 1, 4]), rng.choice([0, 1, 16, 32, 128]))


def _lengths(case):
    """(new tokens, tokens in the cache including them) of each row."""
    rng = random.Random(case["mix"])
    new, lens = [], []
    for i in range(case["rows"]):
        n = _log(rng, case["new_min"], case["new_max"]) if i < case["chunk_rows"] else 1
        lo, hi = case["past_min"], case["past_max"]
        past = _log(rng, lo + 1, hi + 1) - 1
        new.append(n)
        lens.append(past + n)
    return new, lens


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _visible(case, n, length, j):
    """[lo, hi) of the tokens query j of a row of n new and `length` tokens attends to."""
    p = length - n + j
    window, prefix = case.get("window", 0), case.get("prefix", 0)
    lo = max(0, p + 1 - window) if window else 0
    return lo, min(length, max(p + 1, prefix))


def _queries(case, n):
    """First query that counts towards the mass."""
    last = case.get("last", 0)
    return max(0, n - last) if last else 0


def work(case):
    new, lens = _lengths(case)
    tokens, n_q, n_kv, kvb = sum(new), case["n_q"], case["n_kv"], _KV_BYTES[case["kv"]]
    op = case["op"]
    if op == "rope_append":
        io = _BYTES[case["kv"]]
        b = tokens * ((n_q + 2 * n_kv) * D * io + n_q * D * io + 2 * n_kv * kvb + 4 * case["axes"])
        return {"bytes": b, "flops": 3 * tokens * (n_q + n_kv) * case["rot"]}
    if op == "evict":
        b = f = 0
        for length in lens:
            kept = min(length, case["keep"])
            b += n_kv * (4 * length + kept * (4 * kvb + 4 + 4))
            f += n_kv * length
        return {"bytes": b, "flops": f}
    pairs = touched = queries = 0
    for n, length in zip(new, lens):
        j0 = _queries(case, n)
        low = length
        for j in range(j0, n):
            lo, hi = _visible(case, n, length, j)
            pairs += hi - lo
            low = min(low, lo)
        touched += length - low
        queries += n - j0
    if op == "attention":
        b = queries * n_q * (4 * D + 4) + touched * n_kv * 2 * kvb
        return {"bytes": b, "flops": 4 * D * n_q * pairs}
    b = queries * n_q * (2 * D + 4) + touched * n_kv * kvb + n_kv * 4 * (2 * sum(lens) - tokens)
    return {"bytes": b, "flops": 2 * D * n_q * pairs}


# ------------------------------------------------------------------ inputs ----
def _q8_encode(x):
    """(codes + 128 as uint8, f16 scales) of x [..., 128], 32 values a block."""
    b = x.reshape(*x.shape[:-1], D // QB, QB)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    c = torch.where(d > 0, b / d, torch.zeros_like(b))
    c = torch.copysign(torch.floor(c.abs() + 0.5), c).clamp(-127, 127)
    return (c + 128).to(torch.uint8).reshape(x.shape), d.squeeze(-1).to(torch.float16)


def _inputs(case, seed):
    """The case's tensors on the GPU, and its lengths."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, kv, n_q, n_kv, rows = (case[k] for k in ("op", "kv", "n_q", "n_kv", "rows"))
    new, lens = _lengths(case)
    tokens = sum(new)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    s = {"new": new, "lens": lens, "tokens": tokens}
    need = [_pages(x) for x in lens]
    kept = [min(x, case["keep"]) if op == "evict" else 0 for x in lens]
    total = sum(need) + sum(_pages(x) for x in kept)
    pages = total + total // 10 + 1
    stride = max(need) + 2
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((rows, stride), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, x in enumerate(need):
        bt[i, :x] = ids[at:at + x]
        at += x
    s["pages"], s["block_table"] = pages, bt
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["starts"] = cu

    shape = (1, pages, n_kv, PAGE, D)
    s["k_scales"] = s["v_scales"] = None
    if kv == "q8_0":
        for name in ("k", "v"):
            data = torch.empty(shape, dtype=torch.uint8, device="cuda")
            scales = torch.empty((*shape[:-1], D // QB), dtype=torch.float16, device="cuda")
            for p in range(0, pages, 1024):
                data[0, p:p + 1024], scales[0, p:p + 1024] = _q8_encode(normal(min(1024, pages - p), n_kv, PAGE, D))
            s[name + "_data"], s[name + "_scales"] = data, scales
    else:
        s["k_data"], s["v_data"] = normal(*shape, dtype=_TORCH[kv]), normal(*shape, dtype=_TORCH[kv])

    if op == "rope_append":
        qkv = normal(tokens, (n_q + 2 * n_kv), D, dtype=_TORCH[kv])  # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        half = case["rot"] // 2
        s["inv_freq"] = (500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        axes = case["axes"]
        a = half // 4 if axes == 3 else half // axes
        s["sections"] = {1: (half,), 2: (a, half - a), 3: (a, (half - a) // 2, half - a - (half - a) // 2)}[axes]
        pos = []
        for n, length in zip(new, lens):
            j, past = torch.arange(n, device="cuda"), length - n
            grid = [past + j, past + j // 32, past + j % 32]  # frame, line and column of an image's patch
            pos.append(torch.stack(grid[:axes]))
        s["positions"] = torch.cat(pos, 1).to(torch.int32).contiguous()
        s["q_out"] = torch.zeros(tokens, n_q, D, dtype=_TORCH[kv], device="cuda")
    elif op == "evict":
        cap = max(kept) if kept else 1
        w = torch.exp(2.0 * normal(rows, n_kv, max(lens) + 7))
        w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
        s["mass"] = w
        s["keep_lens"] = torch.full((rows,), case["keep"], dtype=torch.int32, device="cuda")
        dst = torch.full((rows, _pages(cap) + 1), -1, dtype=torch.int32, device="cuda")
        for i, x in enumerate(kept):
            dst[i, :_pages(x)] = ids[at:at + _pages(x)]
            at += _pages(x)
        s["dst_table"], s["kept"] = dst, kept
        s["keep_idx"] = torch.full((rows, n_kv, cap), -1, dtype=torch.int32, device="cuda")
        s["dst_mass"] = torch.zeros(rows, n_kv, cap, device="cuda")
        s["new_lens"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    else:
        io = torch.bfloat16 if kv == "bf16" else torch.float16
        s["q"] = normal(tokens, n_q, D, dtype=io)
        s["scale"] = 1.0 / math.sqrt(D)
        s["slopes"] = s["prefix_lens"] = None
        if case.get("bias"):
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / n_q) for h in range(n_q)], device="cuda")
        if case.get("prefix"):
            s["prefix_lens"] = torch.full((rows,), case["prefix"], dtype=torch.int32, device="cuda")
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(tokens, n_q, device="cuda")
        if op == "mass":
            s["lse"] = _all_lse(case, s)
            s["mass_in"] = torch.rand(rows, n_kv, max(lens) + 5, generator=g, device="cuda")
            s["mass_out"] = torch.zeros_like(s["mass_in"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from paged_kv_decode_09_gb300 import api
        kv = {"f16": api.F16, "bf16": api.BF16, "f32": api.F32, "q8_0": api.Q8_0}[case["kv"]]
        tensors = [s["k_data"], s["v_data"]] + ([s["k_scales"], s["v_scales"]] if case["kv"] == "q8_0" else [])
        s["pool"] = api.KVPool(1, s["pages"], case["n_kv"], kv, tensors=tensors)
        if case.get("window"):
            s["pool"].set_window(0, case["window"])
        if case["op"] == "attention":
            s["workspace"] = api.WorkspaceChunk(s["pool"], case["n_q"])
    return s


# -------------------------------------------------------------------- runs ----
def run(s):
    return {"rope_append": _run_rope, "attention": _run_attention, "mass": _run_mass,
            "evict": _run_evict}[s["case"]["op"]](s)


def _row_kv(s, i, length, name, dtype=torch.float32):
    """K or V of the first `length` tokens of row i: [n_kv][length][128]."""
    pg = s["block_table"][i, :_pages(length)].long()
    x = s[name + "_data"][0][pg].to(dtype)
    if s[name + "_scales"] is not None:
        sc = s[name + "_scales"][0][pg].to(dtype)
        x = ((x - 128.0).reshape(*x.shape[:-1], D // QB, QB) * sc[..., None]).reshape(x.shape)
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, D)[:, :length]


def _scores(case, s, i, j0, j1, k):
    """Scores [n_kv][j1 - j0][G][hi] of the queries j0 .. j1 of row i, -inf where masked; no query of the
    range sees a token from hi on."""
    n, length, n_kv = s["new"][i], s["lens"][i], case["n_kv"]
    a = s["starts"][i]
    hi = max(length - n + j1, min(length, case.get("prefix", 0)))
    q = s["q"][a + j0:a + j1].float().reshape(j1 - j0, n_kv, -1, D)
    x = torch.einsum("jhgd,htd->hjgt", q, k[:, :hi]) * s["scale"]
    p = torch.arange(length - n + j0, length - n + j1, device="cuda")[:, None]
    t = torch.arange(hi, device="cuda")[None]
    if case.get("softcap"):
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if case.get("bias"):
        x = x - s["slopes"].reshape(n_kv, 1, -1, 1) * (p - t).abs()[:, None].float()
    seen = t < torch.clamp(p + 1, min=case.get("prefix", 0))
    if case.get("window"):
        seen = seen & (t >= p + 1 - case["window"])
    return x.masked_fill(~seen[:, None], -math.inf)


def _each(case, s, queries_from=lambda n: 0):
    """(row, first query, last query + 1, their slice of the chunk) over the batch, in ranges of at most 2^29
    scores."""
    for i, (a, n, length) in enumerate(zip(s["starts"], s["new"], s["lens"])):
        step = max(1, (1 << 29) // (case["n_q"] * length))
        for j in range(queries_from(n), n, step):
            yield i, j, min(n, j + step), slice(a + j, a + min(n, j + step))


def _all_lse(case, s):
    """log of the sum of exp of each query's scores, as the attention call that precedes the mass returns it."""
    lse = torch.zeros(s["tokens"], case["n_q"], device="cuda")
    for i, j0, j1, rows in _each(case, s):
        x = _scores(case, s, i, j0, j1, _row_kv(s, i, s["lens"][i], "k"))
        lse[rows] = torch.logsumexp(x, -1).transpose(0, 1).reshape(j1 - j0, -1)
    return lse


def _run_rope(s):
    case = s["case"]
    if own:
        from paged_kv_decode_09_gb300 import api
        api.kv_rope_append(s["pool"], 0, s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["sections"],
                           s["cu"], s["block_table"], s["seq_lens"], q_out=s["q_out"],
                           interleaved=case["interleaved"])
        return s["q_out"], s["k_data"], s["v_data"]
    half = case["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"))
    angle = s["positions"][axis].t().double() * s["inv_freq"].double()  # [tokens][half]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        x = x.float()
        y = x.clone()
        one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else \
            (slice(0, half), slice(half, 2 * half))
        y[..., one] = x[..., one] * cos - x[..., two] * sin
        y[..., two] = x[..., one] * sin + x[..., two] * cos
        return y

    s["q_out"].copy_(rotated(s["q"]))
    row = torch.repeat_interleave(torch.arange(case["rows"], device="cuda"), s["cu"].diff().long())
    tok = torch.arange(s["tokens"], device="cuda")
    slot = tok - s["cu"][1:].long()[row] + s["seq_lens"].long()[row]
    page = s["block_table"][row, slot // PAGE].long()
    s["k_data"][0][page, :, slot % PAGE] = rotated(s["k"]).to(s["k_data"].dtype)
    s["v_data"][0][page, :, slot % PAGE] = s["v"]
    return s["q_out"], s["k_data"], s["v_data"]


def _run_attention(s):
    case = s["case"]
    if own:
        from paged_kv_decode_09_gb300 import api
        api.paged_chunk_attention(s["pool"], 0, s["q"], s["cu"], s["block_table"], s["seq_lens"], s["scale"],
                                  softcap=case["softcap"], slopes=s["slopes"], prefix_lens=s["prefix_lens"],
                                  out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return s["out"], s["lse"]
    for i, j0, j1, rows in _each(case, s):
        x = _scores(case, s, i, j0, j1, _row_kv(s, i, s["lens"][i], "k"))
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        v = _row_kv(s, i, s["lens"][i], "v")[:, :x.shape[-1]]
        o = torch.einsum("hjgt,htd->hjgd", e, v) / z
        s["out"][rows] = o.transpose(0, 1).reshape(j1 - j0, -1, D).to(s["out"].dtype)
        s["lse"][rows] = (m + torch.log(z)).transpose(0, 1).reshape(j1 - j0, -1)
    return s["out"], s["lse"]


def _run_mass(s):
    case = s["case"]
    if own:
        from paged_kv_decode_09_gb300 import api
        api.paged_attention_mass(s["pool"], 0, s["q"], s["lse"], s["cu"], s["block_table"], s["seq_lens"],
                                 s["scale"], softcap=case["softcap"], last_queries=case["last"],
                                 mass_in=s["mass_in"], mass_out=s["mass_out"])
        return s["mass_out"]
    for i, (n, length) in enumerate(zip(s["new"], s["lens"])):
        s["mass_out"][i, :, :length - n] = s["mass_in"][i, :, :length - n]
        s["mass_out"][i, :, length - n:length] = 0.0
    for i, j0, j1, rows in _each(case, s, lambda n: _queries(case, n)):
        x = _scores(case, s, i, j0, j1, _row_kv(s, i, s["lens"][i], "k"))
        lse = s["lse"][rows].reshape(j1 - j0, case["n_kv"], -1, 1).transpose(0, 1)
        s["mass_out"][i, :, :x.shape[-1]] += torch.exp(x - lse).sum((1, 2))
    return s["mass_out"]


def _keep(case, w, length):
    """Kept tokens of one row, ascending [n_kv][kept], from its weights w [n_kv][>= length]."""
    kept = min(length, case["keep"])
    recent = min(case["recent"], kept)
    first = min(case["first"], kept - recent)
    w = w[:, :length].clone()
    w[:, :first] = math.inf
    w[:, length - recent:] = math.inf
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    return torch.sort(order[:, :kept], dim=-1).values


def _run_evict(s):
    case = s["case"]
    if own:
        from paged_kv_decode_09_gb300 import api
        api.kv_evict(s["pool"], 0, s["mass"], s["block_table"], s["seq_lens"], s["keep_lens"], s["dst_table"],
                     first=case["first"], recent=case["recent"], keep_idx=s["keep_idx"], new_lens=s["new_lens"],
                     dst_mass=s["dst_mass"])
        return s["keep_idx"], s["new_lens"], s["dst_mass"], s["k_data"], s["v_data"]
    head = torch.arange(case["n_kv"], device="cuda")[:, None]
    for i, (length, kept) in enumerate(zip(s["lens"], s["kept"])):
        idx = _keep(case, s["mass"][i], length)
        s["keep_idx"][i, :, :kept] = idx.to(torch.int32)
        s["dst_mass"][i, :, :kept] = s["mass"][i].gather(1, idx)
        slot = torch.arange(kept, device="cuda")[None]
        src, dst = s["block_table"][i][idx // PAGE].long(), s["dst_table"][i][slot // PAGE].long()
        for name in ("k_data", "v_data"):
            s[name][0][dst, head, slot % PAGE] = s[name][0][src, head, idx % PAGE]
    s["new_lens"].copy_(torch.clamp(s["seq_lens"], max=case["keep"]))
    return s["keep_idx"], s["new_lens"], s["dst_mass"], s["k_data"], s["v_data"]


# ------------------------------------------------------------------- exact ----
def _stored(s, name, page, head, slot):
    """The stored value in 64 bits at (page, KV head, slot), from the pool's bytes."""
    x = s[name + "_data"][0][page, head, slot].double()
    if s[name + "_scales"] is None:
        return x
    return (x - 128.0) * s[name + "_scales"][0][page, head, slot].double().repeat_interleave(QB, -1)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope_append":
        return _exact_rope(case, s)
    if op == "evict":
        return _exact_evict(case, s)
    return _exact_attention(case, s)


def _exact_rope(case, s):
    half, n_axis = case["rot"] // 2, s["sections"]
    ends = [sum(n_axis[:a + 1]) for a in range(len(n_axis))]
    turn = torch.empty(s["tokens"], half, dtype=torch.complex128, device="cuda")
    for u in range(half):
        axis = next(a for a, e in enumerate(ends) if u < e)
        angle = s["positions"][axis].double() * s["inv_freq"][u].double()
        turn[:, u] = torch.polar(torch.ones_like(angle), angle)

    def rotated(x):  # a pair of dims as one complex number, turned
        x = x.double()
        rot, rest = x[..., :2 * half], x[..., 2 * half:]
        pair = rot.reshape(*rot.shape[:-1], half, 2) if case["interleaved"] else \
            torch.stack([rot[..., :half], rot[..., half:]], -1)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
        rot = z.reshape(rot.shape) if case["interleaved"] else torch.cat([z[..., 0], z[..., 1]], -1)
        return torch.cat([rot, rest], -1)

    k, v = s["k_data"].double(), s["v_data"].double()
    rk, rv = rotated(s["k"]), s["v"].double()
    for i, a in enumerate(s["starts"][:-1]):
        n, length = s["new"][i], s["lens"][i]
        pos = torch.arange(length - n, length, device="cuda")
        page = s["block_table"][i][pos // PAGE].long()
        k[0].index_put_((page[:, None], torch.arange(case["n_kv"], device="cuda")[None], (pos % PAGE)[:, None]),
                        rk[a:a + n])
        v[0].index_put_((page[:, None], torch.arange(case["n_kv"], device="cuda")[None], (pos % PAGE)[:, None]),
                        rv[a:a + n])
    return rotated(s["q"]), k, v


def _exact_attention(case, s):
    mass = case["op"] == "mass"
    g, n_kv = case["n_q"] // case["n_kv"], case["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], case["n_q"], dtype=torch.float64, device="cuda")
    total = torch.zeros(s["mass_in"].shape, dtype=torch.float64, device="cuda") if mass else None
    for i in range(case["rows"]):
        n, length, a = s["new"][i], s["lens"][i], s["starts"][i]
        t = torch.arange(length, device="cuda")
        page, slot = s["block_table"][i][t // PAGE].long(), t % PAGE
        if mass:
            total[i, :, :length - n] = s["mass_in"][i, :, :length - n].double()
        for h in range(n_kv):
            k = _stored(s, "k", page, h, slot)
            v = None if mass else _stored(s, "v", page, h, slot)
            for j in range(_queries(case, n) if mass else 0, n, 1024):
                e = min(n, j + 1024)
                p = length - n + torch.arange(j, e, device="cuda")
                low = p + 1 - case["window"] if case.get("window") else torch.zeros_like(p)
                high = torch.maximum(p + 1, torch.full_like(p, case.get("prefix", 0)))
                hide = (t[None] < low[:, None]) | (t[None] >= high[:, None])
                for u in range(h * g, (h + 1) * g):
                    x = (s["q"][a + j:a + e, u].double() @ k.t()) / math.sqrt(D)
                    if case.get("softcap"):
                        x = torch.tanh(x / case["softcap"]) * case["softcap"]
                    if case.get("bias"):
                        x = x - s["slopes"][u].double() * (t[None] - p[:, None]).abs().double()
                    if mass:
                        w = torch.exp(x - s["lse"][a + j:a + e, u].double()[:, None])
                        total[i, h, :length] += w.masked_fill(hide, 0.0).sum(0)
                    else:
                        x = x.masked_fill(hide, -math.inf)
                        lse[a + j:a + e, u] = torch.logsumexp(x, 1)
                        out[a + j:a + e, u] = torch.softmax(x, 1) @ v
    return total if mass else (out, lse)


def _exact_evict(case, s):
    keep_idx, dst_mass = s["keep_idx"].clone(), s["dst_mass"].double()
    k, v = s["k_data"].double(), s["v_data"].double()
    for i in range(case["rows"]):
        length, kept = s["lens"][i], s["kept"][i]
        recent = min(case["recent"], kept)
        first = min(case["first"], kept - recent)
        for h in range(case["n_kv"]):
            w = s["mass"][i, h, :length].tolist()
            middle = sorted(range(first, length - recent), key=lambda t: (-w[t], t))[:kept - first - recent]
            idx = torch.tensor(sorted([*range(first), *middle, *range(length - recent, length)]), device="cuda")
            keep_idx[i, h, :kept] = idx.to(torch.int32)
            dst_mass[i, h, :kept] = s["mass"][i, h][idx].double()
            to = torch.arange(kept, device="cuda")
            src, dst = s["block_table"][i][idx // PAGE].long(), s["dst_table"][i][to // PAGE].long()
            k[0, dst, h, to % PAGE] = s["k_data"][0, src, h, idx % PAGE].double()
            v[0, dst, h, to % PAGE] = s["v_data"][0, src, h, idx % PAGE].double()
    return keep_idx, torch.tensor([min(x, case["keep"]) for x in s["lens"]], dtype=torch.int32,
                                  device="cuda"), dst_mass, k, v
