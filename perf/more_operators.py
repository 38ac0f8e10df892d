"""Workloads of speculative trees and of layers that keep their first tokens: single-token and chunk attention
under a sliding window with sinks, attention of a tree of drafted tokens over the paged cache, and the commit
of the tree's accepted path.

Every case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` is one pass (in
elementary torch operations, or through the library's entry points when `own` is true), `exact` is the same
operator in 64 bits written from its definition, and `work` counts what a pass cannot do without."""
import math
import random

import torch

own = False

PAGE, D, QB = 16, 128, 32
_KV_BYTES = {"f16": 256, "bf16": 256, "f32": 512, "q8_0": 136}  # one token of one KV head, K or V
_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases ----
def _case(op, kv, n_q, n_kv, rows, new, past, mix, **more):
    """Each row brings new[0] .. new[1] tokens and has past[0] .. past[1] in the cache before them (`mix` picks
    the lengths and the trees)."""
    return {"op": op, "kv": kv, "n_q": n_q, "n_kv": n_kv, "rows": rows, "new_min": new[0], "new_max": new[1],
            "past_min": past[0], "past_max": past[1], "mix": mix, **more}


def _step(kv, n_q, n_kv, rows, past, mix, window, sinks):
    return _case("step", kv, n_q, n_kv, rows, (1, 1), past, mix, window=window, sinks=sinks, softcap=0.0)


def _chunk(kv, n_q, n_kv, rows, new, past, mix, window, sinks, softcap=0.0):
    return _case("chunk", kv, n_q, n_kv, rows, new, past, mix, window=window, sinks=sinks, softcap=softcap)


def _tree(kv, n_q, n_kv, rows, new, past, mix, window=0, sinks=0, softcap=0.0):
    return _case("tree", kv, n_q, n_kv, rows, new, past, mix, window=window, sinks=sinks, softcap=softcap)


def _commit(kv, n_kv, rows, new, past, mix, layers):
    return _case("commit", kv, n_kv, n_kv, rows, new, past, mix, layers=layers, window=0, sinks=0, softcap=0.0)


def listed():
    return [
        # a decode step of eight conversations on a layer that keeps four sinks and its last 1024 tokens: latency
        {"name": "sink_step_f16", **_step("f16", 32, 8, 8, (1024, 8192), 1, 1024, 4)},
        # the long batch of the 8-bit cache on such a layer
        {"name": "sink_step_q8_0", **_step("q8_0", 32, 8, 32, (4096, 32768), 2, 4096, 4)},
        # many rows around the window's length, some still shorter, an odd window
        {"name": "sink_step_bf16", **_step("bf16", 16, 8, 64, (16, 4000), 3, 1001, 17)},
        # a long prompt from an empty cache: compute-bound
        {"name": "sink_prompt_bf16", **_chunk("bf16", 32, 8, 1, (8191, 8191), (0, 0), 4, 2048, 4)},
        # the next 2048 tokens of a long prompt over an 8-bit cache
        {"name": "sink_chunk_q8_0", **_chunk("q8_0", 32, 8, 1, (2048, 2048), (30001, 30001), 5, 4096, 64)},
        # a small tree in four rows of a small model: the shortest verification
        {"name": "tree_small_f16", **_tree("f16", 16, 8, 4, (5, 12), (256, 2048), 6)},
        # trees of 64 drafted tokens in eight conversations
        {"name": "tree_64_bf16", **_tree("bf16", 32, 8, 8, (64, 64), (1024, 8192), 7)},
        # trees of up to 32 tokens over an 8-bit cache
        {"name": "tree_32_q8_0", **_tree("q8_0", 32, 8, 8, (20, 32), (4096, 16384), 8)},
        # ragged trees, single tokens among them, on a capped layer with a window and sinks
        {"name": "tree_window_f16", **_tree("f16", 32, 8, 24, (1, 60), (500, 6000), 9, 1024, 4, 50.0)},
        # one layer's accepted paths: latency
        {"name": "commit_layer_f16", **_commit("f16", 8, 8, (24, 64), (16, 500), 10, 1)},
        # all 32 layers of a batch at once
        {"name": "commit_model_bf16", **_commit("bf16", 8, 32, (24, 64), (16, 200), 11, 32)},
        # a wide batch of deep trees in full precision
        {"name": "commit_wide_f32", **_commit("f32", 8, 192, (100, 256), (1, 64), 12, 16)},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "chunk", "tree", "tree", "commit"])
    n_q, n_kv = rng.choice([(32, 8), (16, 8), (8, 8)])
    mix = rng.randrange(1 << 20)
    window, sinks = _log(rng, 1, 4096), rng.choice([1, 2, 4, 16, 17, 64, 200])
    if op == "step":
        rows = _log(rng, 1, 64)
        past_hi = _log(rng, 1, max(1, min(32768, 500000 // rows)))
        return _step(rng.choice(["f16", "bf16", "f32", "q8_0"]), n_q, n_kv, rows, (rng.randint(0, past_hi), past_hi),
                     mix, window, sinks)
    if op == "chunk":
        rows = _log(rng, 1, 16)
        new_hi = _log(rng, 1, max(1, 4000 // rows))
        past_hi = _log(rng, 1, max(1, min(16000, 60000 // rows)))
        return _chunk(rng.choice(["f16", "bf16", "q8_0"]), n_q, n_kv, rows, (rng.randint(1, new_hi), new_hi),
                      (rng.randint(0, past_hi), past_hi), mix, window, sinks, rng.choice([0.0, 0.0, 30.0]))
    if op == "tree":
        rows = _log(rng, 1, 32)
        new_hi = _log(rng, 1, min(200, max(1, 2000 // rows)))
        past_hi = _log(rng, 1, max(1, min(16000, 100000 // rows)))
        if rng.random() < 0.6:
            window = sinks = 0
        return _tree(rng.choice(["f16", "bf16", "q8_0"]), n_q, n_kv, rows, (rng.randint(1, new_hi), new_hi),
                     (rng.randint(0, past_hi), past_hi), mix, window, sinks, rng.choice([0.0, 0.0, 30.0, 50.0]))
    rows, layers = _log(rng, 1, 128), _log(rng, 1, 32)
    new_hi = _log(rng, 1, 256)
    past_hi = _log(rng, 1, 200)
    return _commit(rng.choice(["f16", "bf16", "f32"]), n_kv, rows, (rng.randint(1, new_hi), new_hi),
                   (rng.randint(0, past_hi), past_hi), mix, layers)


def _lengths(case):
    """(new tokens, tokens in the cache including them, parents of the new tokens) of each row."""
    rng = random.Random(case["mix"])
    new, lens, trees = [], [], []
    for _ in range(case["rows"]):
        n = _log(rng, case["new_min"], case["new_max"])
        past = _log(rng, case["past_min"] + 1, case["past_max"] + 1) - 1
        new.append(n)
        lens.append(past + n)
        # the root is the token that the model chose last; drafts hang from it and from one another
        trees.append([-1] + [rng.randrange(j) for j in range(1, n)] if case["op"] in ("tree", "commit") else None)
    return new, lens, trees


def _path(tree, leaf):
    path = []
    while leaf >= 0:
        path.append(leaf)
        leaf = tree[leaf]
    return path[::-1]


def _accepted(tree):
    """The accepted path: the longest one whose moved tokens all lie behind its length, so that a pass on a
    committed tree moves the same values once more."""
    best = [0]
    for leaf in range(len(tree)):
        path = _path(tree, leaf)
        if len(path) > len(best) and all(x == d or x >= len(path) for d, x in enumerate(path)):
            best = path
    return best


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _context(past, position, window, sinks):
    """Tokens before `past` that a query at `position` sees."""
    low = max(0, position + 1 - window) if window else 0
    return past - max(0, min(low, past) - sinks)


def work(case):
    new, lens, trees = _lengths(case)
    n_q, n_kv, kvb, op = case["n_q"], case["n_kv"], _KV_BYTES[case["kv"]], case["op"]
    if op == "commit":
        moved = sum(sum(x != d for d, x in enumerate(_accepted(t))) for t in trees)
        return {"bytes": 4 * case["layers"] * n_kv * moved * kvb + 4 * (sum(new) + 4 * case["rows"]), "flops": 0}
    pairs = touched = 0
    for n, length, tree in zip(new, lens, trees):
        past, window, sinks = length - n, case["window"], case["sinks"]
        touched += _context(past, past, window, sinks) + n
        for j in range(n):
            if tree is None:
                pairs += _context(past + j + 1, past + j, window, sinks)
            else:
                depth = len(_path(tree, j)) - 1
                near = depth + 1 if not window else sum(depth - a < window or past + a < sinks for a in range(depth + 1))
                pairs += _context(past, past + depth, window, sinks) + near
    io = 8 * D if op == "step" else 4 * D + 4
    return {"bytes": sum(new) * n_q * io + touched * n_kv * 2 * kvb, "flops": 4 * D * n_q * pairs}


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
    new, lens, trees = _lengths(case)
    tokens, layers = sum(new), case.get("layers", 1)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    s = {"new": new, "lens": lens, "tokens": tokens, "scale": 1.0 / math.sqrt(D)}
    need = [_pages(x) for x in lens]
    pages = sum(need) + sum(need) // 10 + 1
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((rows, max(need) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, x in enumerate(need):
        bt[i, :x] = ids[at:at + x]
        at += x
    s["pages"], s["block_table"] = pages, bt
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"], s["starts"] = torch.tensor(cu, dtype=torch.int32, device="cuda"), cu

    shape = (layers, pages, n_kv, PAGE, D)
    s["k_scales"] = s["v_scales"] = None
    for name in ("k", "v"):
        data = s[name + "_data"] = torch.empty(shape, dtype=_TORCH.get(kv, torch.uint8), device="cuda")
        if kv == "q8_0":
            s[name + "_scales"] = torch.empty((*shape[:-1], D // QB), dtype=torch.float16, device="cuda")
        for layer in range(layers):
            for p in range(0, pages, 4096):
                x = normal(min(4096, pages - p), n_kv, PAGE, D)
                if kv == "q8_0":
                    data[layer, p:p + 4096], s[name + "_scales"][layer, p:p + 4096] = _q8_encode(x)
                else:
                    data[layer, p:p + 4096] = x

    if op in ("tree", "commit"):
        s["parents"] = torch.tensor([x for t in trees for x in t], dtype=torch.int32, device="cuda")
        s["depth"] = max(len(_path(t, j)) for t in trees for j in range(len(t)))  # of the deepest draft, the root 1
    if op == "commit":
        paths = [_accepted(t) for t in trees]
        s["leaves"] = torch.tensor([p[-1] for p in paths], dtype=torch.int32, device="cuda")
        s["path"] = torch.full((rows, max(len(p) for p in paths)), -1, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    elif op == "step":
        s["q"] = normal(rows, n_q, D)
        s["out"] = torch.zeros_like(s["q"])
    else:
        s["q"] = normal(tokens, n_q, D, dtype=torch.bfloat16 if kv == "bf16" else torch.float16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(tokens, n_q, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from paged_kv_decode_09_gb300 import api
        kv = {"f16": api.F16, "bf16": api.BF16, "f32": api.F32, "q8_0": api.Q8_0}[case["kv"]]
        tensors = [s["k_data"], s["v_data"]] + ([s["k_scales"], s["v_scales"]] if case["kv"] == "q8_0" else [])
        s["pool"] = api.KVPool(case.get("layers", 1), s["pages"], case["n_kv"], kv, tensors=tensors)
        if case["window"]:
            s["pool"].set_window(0, case["window"])
            s["pool"].set_sinks(0, case["sinks"])
        if case["op"] == "step":
            s["workspace"] = api.Workspace(s["pool"], case["n_q"], case["rows"])
        elif case["op"] != "commit":
            s["workspace"] = api.WorkspaceChunk(s["pool"], case["n_q"])
    return s


# -------------------------------------------------------------------- runs ----
def run(s):
    return {"step": _run_step, "chunk": _run_chunk, "tree": _run_tree, "commit": _run_commit}[s["case"]["op"]](s)


def _run_step(s):
    if own:
        from paged_kv_decode_09_gb300 import api
        return api.paged_decode_attention(s["pool"], 0, s["q"], s["block_table"], s["seq_lens"], s["scale"],
                                          out=s["out"], workspace=s["workspace"])
    for i, length in enumerate(s["lens"]):
        t = torch.arange(length, device="cuda")
        seen = ((t >= length - s["case"]["window"]) | (t < s["case"]["sinks"]))[None]
        s["out"][i], _ = _attend(s, i, s["q"][i:i + 1], seen)
    return s["out"]


def _run_chunk(s):
    case = s["case"]
    if own:
        from paged_kv_decode_09_gb300 import api
        api.paged_chunk_attention(s["pool"], 0, s["q"], s["cu"], s["block_table"], s["seq_lens"], s["scale"],
                                  softcap=case["softcap"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return s["out"], s["lse"]
    for i, (a, n, length) in enumerate(zip(s["starts"], s["new"], s["lens"])):
        step = max(1, (1 << 29) // (case["n_q"] * length))
        for j in range(0, n, step):
            e = min(n, j + step)
            p = torch.arange(length - n + j, length - n + e, device="cuda")[:, None]
            t = torch.arange(length, device="cuda")[None]
            seen = (t <= p) & ((t > p - case["window"]) | (t < case["sinks"]))
            s["out"][a + j:a + e], s["lse"][a + j:a + e] = _attend(s, i, s["q"][a + j:a + e], seen)
    return s["out"], s["lse"]


def _run_tree(s):
    case = s["case"]
    if own:
        from paged_kv_decode_09_gb300 import api
        api.paged_tree_attention(s["pool"], 0, s["q"], s["parents"], s["cu"], s["block_table"], s["seq_lens"],
                                 s["scale"], softcap=case["softcap"], out=s["out"], lse=s["lse"],
                                 workspace=s["workspace"])
        return s["out"], s["lse"]
    # each drafted token's ancestors and depth, from the parents
    row = torch.repeat_interleave(torch.arange(case["rows"], device="cuda"), s["cu"].diff().long(),
                                  output_size=s["tokens"])
    start = s["cu"].long()[row]
    at = torch.arange(s["tokens"], device="cuda")
    line = torch.zeros(s["tokens"], max(s["new"]) + 1, dtype=torch.bool, device="cuda")  # column 0: no node
    depth = torch.full_like(at, -1)
    node = at - start
    for _ in range(s["depth"]):
        line.scatter_(1, (node + 1)[:, None], True)
        depth += (node >= 0).long()
        node = torch.where(node >= 0, s["parents"][start + node.clamp(min=0)].long(), node)
    for i, (a, n, length) in enumerate(zip(s["starts"], s["new"], s["lens"])):
        past, d = length - n, depth[a:a + n]
        t = torch.arange(past, device="cuda")[None]
        before = torch.ones(n, past, dtype=torch.bool, device="cuda")
        near = line[a:a + n, 1:n + 1]
        if case["window"]:
            before = (t > past + d[:, None] - case["window"]) | (t < case["sinks"])
            near = near & ((d[:, None] - d[None] < case["window"]) | (past + d[None] < case["sinks"]))
        s["out"][a:a + n], s["lse"][a:a + n] = _attend(s, i, s["q"][a:a + n], torch.cat([before, near], 1))
    return s["out"], s["lse"]


def _attend(s, i, q, seen):
    """(outputs, logs of the softmax's sums) of the queries q [n][n_q][128] of row i over its tokens, those of
    seen [n][length]."""
    n, n_kv = q.shape[0], s["case"]["n_kv"]
    x = torch.einsum("jhgd,htd->hjgt", q.float().reshape(n, n_kv, -1, D), _row_kv(s, i, "k")) * s["scale"]
    if s["case"]["softcap"]:
        x = s["case"]["softcap"] * torch.tanh(x / s["case"]["softcap"])
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("hjgt,htd->hjgd", e, _row_kv(s, i, "v")) / z
    return o.transpose(0, 1).reshape(n, -1, D).to(q.dtype), (m + torch.log(z)).transpose(0, 1).reshape(n, -1)


def _row_kv(s, i, name):
    """K or V of row i: [n_kv][length][128]."""
    pg = s["block_table"][i, :_pages(s["lens"][i])].long()
    x = s[name + "_data"][0][pg].float()
    if s[name + "_scales"] is not None:
        sc = s[name + "_scales"][0][pg].float()
        x = ((x - 128.0).reshape(*x.shape[:-1], D // QB, QB) * sc[..., None]).reshape(x.shape)
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, D)[:, :s["lens"][i]]


def _run_commit(s):
    if own:
        from paged_kv_decode_09_gb300 import api
        api.kv_tree_commit(s["pool"], s["parents"], s["leaves"], s["cu"], s["block_table"], s["seq_lens"],
                           path=s["path"], new_lens=s["new_lens"])
        return s["path"], s["new_lens"], s["k_data"], s["v_data"]
    start, rows = s["cu"][:-1].long(), torch.arange(len(s["lens"]), device="cuda")[:, None]
    past = s["seq_lens"].long() - s["cu"].diff()
    up, node = [], s["leaves"].long()  # the path from the leaf up
    for _ in range(s["path"].shape[1]):
        up.append(node)
        node = torch.where(node >= 0, s["parents"][start + node.clamp(min=0)].long(), node)
    up = torch.stack(up, 1)
    length = (up >= 0).sum(1)
    d = torch.arange(up.shape[1], device="cuda")[None]
    on = d < length[:, None]
    path = up.gather(1, (length[:, None] - 1 - d).clamp(min=0))
    s["path"].copy_(torch.where(on, path, s["path"].long()))
    s["new_lens"].copy_(past + length)
    # behind a path's end its first token is moved again
    src = past[:, None] + torch.where(on, path, path[:, :1])
    dst = past[:, None] + torch.where(on, d, torch.zeros_like(d))
    from_page, to_page = s["block_table"][rows, src // PAGE].long(), s["block_table"][rows, dst // PAGE].long()
    for x in (s["k_data"], s["v_data"]):
        x[:, to_page, :, dst % PAGE] = x[:, from_page, :, src % PAGE]
    return s["path"], s["new_lens"], s["k_data"], s["v_data"]


# ------------------------------------------------------------------- exact ----
def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_commit(case, s) if case["op"] == "commit" else _exact_attention(case, s)


def _exact_attention(case, s):
    _, _, trees = _lengths(case)
    group, cap = case["n_q"] // case["n_kv"], case["softcap"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    for i, (a, n, length) in enumerate(zip(s["starts"], s["new"], s["lens"])):
        past = length - n
        t = torch.arange(length, device="cuda")
        page, slot = s["block_table"][i][t // PAGE].long(), t % PAGE
        # each token's own position, and whose descendant each drafted token is
        where = list(range(length))
        kin = None
        if trees[i] is not None:
            lines = [_path(trees[i], j) for j in range(n)]
            where = list(range(past)) + [past + len(x) - 1 for x in lines]
            kin = torch.zeros(n, length, dtype=torch.bool)
            for j, x in enumerate(lines):
                kin[j, :past] = True
                kin[j, [past + y for y in x]] = True
            kin = kin.cuda()
        where = torch.tensor(where, device="cuda")
        for j in range(0, n, 1024):
            e = min(n, j + 1024)
            p = where[past + j:past + e][:, None]
            show = where[None] <= p if kin is None else kin[j:e]
            if case["window"]:
                show = show & ((p - where[None] < case["window"]) | (where[None] < case["sinks"]))
            for h in range(case["n_kv"]):
                k, v = _stored(s, "k", page, h, slot), _stored(s, "v", page, h, slot)
                for u in range(h * group, (h + 1) * group):
                    x = (s["q"][a + j:a + e, u].double() @ k.t()) / math.sqrt(D)
                    if cap:
                        x = torch.tanh(x / cap) * cap
                    x = x.masked_fill(~show, -math.inf)
                    lse[a + j:a + e, u] = torch.logsumexp(x, 1)
                    out[a + j:a + e, u] = torch.softmax(x, 1) @ v
    return out if case["op"] == "step" else (out, lse)


def _stored(s, name, page, head, slot):
    """The stored value in 64 bits at (page, KV head, slot), from the pool's bytes."""
    x = s[name + "_data"][0][page, head, slot].double()
    if s[name + "_scales"] is None:
        return x
    return (x - 128.0) * s[name + "_scales"][0][page, head, slot].double().repeat_interleave(QB, -1)


def _exact_commit(case, s):
    new, lens, trees = _lengths(case)
    table = s["block_table"].tolist()
    path, new_lens = s["path"].clone(), []
    k, v = s["k_data"].double(), s["v_data"].double()
    for i, (n, length, tree) in enumerate(zip(new, lens, trees)):
        past, line = length - n, _accepted(tree)
        new_lens.append(past + len(line))
        for d, x in enumerate(line):
            path[i, d] = x
            at, to = past + x, past + d
            for mine, stored in ((k, s["k_data"]), (v, s["v_data"])):
                mine[:, table[i][to // PAGE], :, to % PAGE] = \
                    stored[:, table[i][at // PAGE], :, at % PAGE].double()
    return path, torch.tensor(new_lens, dtype=torch.int32, device="cuda"), k, v
