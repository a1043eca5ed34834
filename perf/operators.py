"""The operators of a verify round around the quantized projections, as cases that can be timed and compared.

A verify round of block-wise speculative decoding appends the rows of every sequence's block to a paged
key/value cache with their rotary positions, attends to the cache, chooses tokens from edited logits, and
then keeps the accepted rows and gives the other pages back. Each case is one of these:

  rope     rotary positions of queries and keys, the keys and values written to the cache's pages
  attn     attention of a chunk of new rows over a paged cache (also with a window and visible first tokens)
  cache    the end of a round (compact, free, reserve), forks of sequences, copies of pages
  logits   penalties, biases and grammar masks on logits, written out or fused with the greedy verify

`run` computes an operator in its plain form, in elementary torch operations, or (with `own`) by the library's call.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One sequence's verify block of 8 rows, straight from the fp32 output of a stacked q/k/v projection: latency.
        dict(name="rope block 1x8", kind="rope", into="fp32", dtype="bf16", layout="slot", seqs=1, rows=8, kv=2048, heads=32,
             kv_heads=8, dim=128, page=16, rot=128, interleaved=False, scaling="none", factor=1.0, ragged=False),
        # A prompt chunk far into a long context: interleaved pairs in half of each head, frequencies stretched.
        dict(name="rope chunk 4x2048 far", kind="rope", into="bf16", dtype="bf16", layout="head", seqs=4, rows=2048, kv=200000,
             heads=32, kv_heads=8, dim=128, page=64, rot=64, interleaved=True, scaling="yarn", factor=8.0, ragged=True),
        # One sequence's verify block over a short cache: latency.
        dict(name="attn block 1x8 kv 4k", kind="attn", dtype="bf16", layout="slot", seqs=1, rows=8, kv=4096, heads=32, kv_heads=8,
             dim=128, page=16, window=0, sinks=0, ragged=False),
        # Plain decoding, a token for each of many sequences of very different lengths.
        dict(name="attn decode 48x1 ragged", kind="attn", dtype="bf16", layout="slot", seqs=48, rows=1, kv=16383, heads=32,
             kv_heads=8, dim=128, page=16, window=0, sinks=0, ragged=True),
        # A prompt's chunk after what is already in the cache: matrix-bound.
        dict(name="attn chunk 1x2048 kv 10k", kind="attn", dtype="bf16", layout="head", seqs=1, rows=2048, kv=10240, heads=32,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, ragged=False),
        # Batched verify blocks of 16 rows with wide heads over long caches of which a window and the first tokens are seen.
        dict(name="window block 16x16 dim 256", kind="attn", dtype="fp16", layout="slot", seqs=16, rows=16, kv=32003, heads=16,
             kv_heads=4, dim=256, page=32, window=4096, sinks=4, ragged=True),
        # Ragged prompt chunks under a window, an odd page size and an odd number of query heads to a key head.
        dict(name="window chunk 3x1500", kind="attn", dtype="fp16", layout="head", seqs=3, rows=1500, kv=9001, heads=20,
             kv_heads=4, dim=64, page=24, window=1023, sinks=7, ragged=True),
        # The end of a batched round: kept rows move together, pages go back, the next block's pages are taken.
        dict(name="cache round 32x16", kind="cache", op="round", dtype="bf16", layout="slot", layers=16, seqs=32, rows=16, kv=3001,
             kv_heads=4, dim=128, page=16, ragged=True),
        # Branches of running sequences: the old ones dropped, new ones forked, their last pages copied.
        dict(name="cache fork 12x4", kind="cache", op="fork", dtype="bf16", layout="slot", layers=16, seqs=12, rows=4, kv=5001,
             kv_heads=8, dim=128, page=64, ragged=True),
        # Moving pages, as before a swap or to close gaps.
        dict(name="cache copy 3000 pages", kind="cache", op="copy", dtype="fp16", layout="head", layers=4, seqs=3000, rows=1, kv=16,
             kv_heads=8, dim=128, page=16, ragged=False),
        # Sampling parameters of a few requests on plain decoding's logits, written out.
        dict(name="logits edit 8x1", kind="logits", op="edit", seqs=8, rows=1, vocab=151936, penalties=True, bias=40, mask=True),
        # Batched verify blocks over the vocabulary, each row under its own grammar mask, chosen without writing logits.
        dict(name="logits verify 4x16", kind="logits", op="verify", seqs=4, rows=16, vocab=151936, penalties=True, bias=300, mask=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "attn", "attn", "window", "cache", "logits"])
    if kind == "logits":
        return dict(kind=kind, op=rng.choice(["edit", "verify"]), seqs=rng.randint(1, 8), rows=rng.randint(1, 8), vocab=_log_int(rng, 1000, 150000),
                    penalties=rng.random() < 0.8, bias=rng.choice([0, 3, 300]), mask=rng.random() < 0.7)
    layout, dtype, dim = rng.choice(["slot", "head"]), rng.choice(["bf16", "fp16"]), rng.choice([64, 80, 96, 128, 192, 256])
    kv_heads, page = rng.randint(1, 8), rng.choice([1, 8, 16, 20, 32, 64, 128])
    if kind == "rope":
        rows = _log_int(rng, 1, 1000)
        return dict(kind=kind, into=rng.choice(["fp32", "bf16", "fp16"]), dtype=dtype, layout=layout, seqs=rng.randint(1, 8), rows=rows,
                    kv=rows + _log_int(rng, 1, 500000), heads=kv_heads * rng.randint(1, 4), kv_heads=kv_heads, dim=dim, page=max(8, page),
                    rot=2 * rng.randint(1, dim // 2), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "smooth"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]), ragged=rng.random() < 0.7)
    if kind == "cache":
        op = rng.choice(["round", "fork", "copy"])
        rows = rng.randint(1, 24) if op == "round" else rng.randint(1, 6)
        return dict(kind=kind, op=op, dtype=dtype, layout=layout, layers=rng.randint(1, 12), seqs=_log_int(rng, 1, 24), rows=rows,
                    kv=rows + _log_int(rng, 1, 4000), kv_heads=kv_heads, dim=dim, page=max(8, page), ragged=rng.random() < 0.7)
    rows = rng.choice([1, 1, 8, 16, rng.randint(1, 16), _log_int(rng, 1, 1000)])
    per = rng.randint(1, 8)
    seqs = rng.randint(1, 32) if rows <= 16 else rng.randint(1, 3)
    kv = rows + _log_int(rng, 1, 16000 if seqs <= 8 else 6000)
    while rows > 16 and seqs * rows * kv * kv_heads * per * dim > 6e10:
        rows //= 2
    return dict(kind="attn", dtype=dtype, layout=layout, seqs=seqs, rows=rows, kv=kv, heads=kv_heads * per, kv_heads=kv_heads, dim=dim, page=page,
                window=_log_int(rng, 1, 4000) if kind == "window" else 0, sinks=rng.choice([0, 1, 4, 100]) if kind == "window" else 0,
                ragged=rng.random() < 0.7)


# ---- what the cases have in common: lengths go by the case alone, so that its work is known ----


def _spread(b):
    """Parts of one, spread evenly, 0 for the first."""
    return b * 0.6180339887498949 % 1.0


def _rows_of(c):
    """Rows of each sequence's chunk."""
    return [max(1, c["rows"] - int(c["rows"] * _spread(b))) if c["ragged"] else c["rows"] for b in range(c["seqs"])]


def _kv_of(c):
    """Tokens of each sequence, its chunk among them."""
    rows = _rows_of(c)
    if not c["ragged"]:
        return [c["kv"]] * c["seqs"]
    return [max(rows[b], c["kv"] - int(0.9 * c["kv"] * _spread(3 * b))) for b in range(c["seqs"])]


def _cdiv(a, b):
    return -(-a // b)


def _storage(c, layers, pages, gen):
    """k, v [layers, pages, slots, heads, dim], with the heads or the slots outermost in memory."""
    t = DTYPES[c["dtype"]]
    shape = (layers, pages, c["page"], c["kv_heads"], c["dim"])
    if c["layout"] == "head":
        shape = (layers, pages, c["kv_heads"], c["page"], c["dim"])
    kv = [torch.empty(shape, dtype=t, device="cuda").normal_(generator=gen) for _ in range(2)]
    return [x.transpose(2, 3) if c["layout"] == "head" else x for x in kv]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(rows):
    s = [0]
    for r in rows:
        s.append(s[-1] + r)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"rope": _prepare_rope, "attn": _prepare_attn, "cache": _prepare_cache, "logits": _prepare_logits}[case["kind"]](case, gen)


def run(state):
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "cache": _own_cache, "logits": _own_logits}[state["case"]["kind"]](state)
    return {"rope": _plain_rope, "attn": _plain_attn, "cache": _plain_cache, "logits": _plain_logits}[state["case"]["kind"]](state)


def exact(case, seed):
    return {"rope": _exact_rope, "attn": _exact_attn, "cache": _exact_cache, "logits": _exact_logits}[case["kind"]](prepare(case, seed))


def work(case):
    return {"rope": _work_rope, "attn": _work_attn, "cache": _work_cache, "logits": _work_logits}[case["kind"]](case)


def _row_places(s):
    """Sequence and place in its chunk of every row, and whether a sequence has it."""
    r = torch.arange(s["n_rows"], device="cuda")
    b = (r[:, None] >= s["row_start"][None, 1:]).sum(1).clamp(max=s["kv_len"].numel() - 1)
    return b, r - s["row_start"][b]


# ---- rope ----


def _prepare_rope(c, gen):
    rows, kv = _rows_of(c), _kv_of(c)
    n = sum(rows)
    width = _cdiv(c["kv"], c["page"]) + 1
    # Pages that the chunk's rows fall into are in the pool; what is before them is never touched here.
    tails = [(_cdiv(kv[b], c["page"]) - (kv[b] - rows[b]) // c["page"]) for b in range(c["seqs"])]
    pages = sum(tails) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(c["seqs"]):
        first = (kv[b] - rows[b]) // c["page"]
        table[b, first:first + tails[b]] = order[at:at + tails[b]]
        at += tails[b]
    heads, hk, d = c["heads"], c["kv_heads"], c["dim"]
    qkv = torch.randn((n, (heads + 2 * hk) * d), generator=gen, device="cuda").to(DTYPES[c["into"]])
    k, v = _storage(c, 1, pages, gen)
    s = dict(case=c, n_rows=n, qkv=qkv, q=qkv[:, :heads * d].view(n, heads, d), kin=qkv[:, heads * d:(heads + hk) * d].view(n, hk, d),
             vin=qkv[:, (heads + hk) * d:].view(n, hk, d), k=k, v=v, row_start=_i32(_starts(rows)), kv_len=_i32(kv), table=table)
    if own:
        import w4_gemm_vqv_amd as vqv
        s["cache"] = vqv.PagedCache(k, v)
        s["seqs"] = vqv.Sequences(s["row_start"], s["kv_len"], table, n_rows=n, max_rows=max(rows), max_kv=max(kv))
        s["rope"] = vqv.Rope(c["rot"], BASE, interleaved=c["interleaved"], scaling=c["scaling"], factor=c["factor"], original_len=ORIGINAL)
        s["q_out"] = torch.empty((n, heads, d), dtype=DTYPES[c["dtype"]], device="cuda")
    return s


BASE, ORIGINAL = 1e6, 8192


def _plain_frequencies(c):
    """Angle per position of each pair (64 bits), and the factor on cosines and sines."""
    rot, factor = c["rot"], c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base = BASE * factor ** (rot / (rot - 2)) if c["scaling"] == "ntk" and rot > 2 else BASE
    f = base ** (-2 * i / rot)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "yarn":
        def pair(turns):
            return rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    if c["scaling"] == "smooth":
        turns = ORIGINAL * f / (2 * math.pi)
        part = ((turns - 1) / (4 - 1)).clamp(0, 1)
        return f / factor * (1 - part) + f * part, 1.0
    return f, 1.0


def _plain_rotate(x, cos, sin, c):
    """x [rows, heads, dim] in 32 bits."""
    rot = c["rot"]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    c, t = s["case"], DTYPES[s["case"]["dtype"]]
    b, i = _row_places(s)
    pos = (s["kv_len"][b] - (s["row_start"][b + 1] - s["row_start"][b])).long() + i
    f, m = _plain_frequencies(c)
    angle = pos.double()[:, None] * f[None, :]
    cos, sin = (torch.cos(angle) * m).float()[:, None, :], (torch.sin(angle) * m).float()[:, None, :]
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    s["k"][0].index_put_((page, slot), _plain_rotate(s["kin"], cos, sin, c).to(t))
    s["v"][0].index_put_((page, slot), s["vin"].float().to(t))
    return _plain_rotate(s["q"], cos, sin, c).to(t), s["k"], s["v"]


def _own_rope(s):
    import w4_gemm_vqv_amd as vqv
    vqv.vqv_rope_append(s["q"], s["kin"], s["vin"], s["cache"], s["seqs"], s["rope"], q_out=s["q_out"])
    return s["q_out"], s["k"], s["v"]


def _exact_rope(s):
    c = s["case"]
    rot, half, base, factor = c["rot"], c["rot"] // 2, BASE, c["factor"]
    if c["scaling"] == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    m, f = 1.0, [math.exp(-2.0 * i / rot * math.log(base)) for i in range(half)]
    if c["scaling"] == "linear":
        f = [x / factor for x in f]
    elif c["scaling"] == "smooth":
        for i in range(half):
            wave = 2 * math.pi / f[i]
            if wave > ORIGINAL / 1.0:
                f[i] /= factor
            elif wave > ORIGINAL / 4.0:
                w = (ORIGINAL / wave - 1.0) / 3.0
                f[i] = (1 - w) * f[i] / factor + w * f[i]
    elif c["scaling"] == "yarn":
        m = 1.0 + 0.1 * math.log(factor)
        at = [half * math.log(ORIGINAL / (2 * math.pi * turns)) / math.log(BASE) for turns in (32.0, 1.0)]
        lo, hi = max(int(math.floor(at[0])), 0), min(int(math.ceil(at[1])), rot - 1)
        for i in range(half):
            w = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f[i] *= 1 - w + w / factor
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    k, v, q = s["k"].double(), s["v"].double(), s["q"].double()
    starts, lens, rows = s["row_start"].tolist(), s["kv_len"].tolist(), _rows_of(c)
    even = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    odd = even + (1 if c["interleaved"] else half)

    def turned(x, angle):
        y = x.clone()
        y[..., even] = m * (x[..., even] * angle.cos() - x[..., odd] * angle.sin())
        y[..., odd] = m * (x[..., even] * angle.sin() + x[..., odd] * angle.cos())
        return y

    for b in range(c["seqs"]):
        pos = torch.arange(lens[b] - rows[b], lens[b], device="cuda")
        angle = (pos.double()[:, None] * f)[:, None, :]
        mine = slice(starts[b], starts[b + 1])
        q[mine] = turned(q[mine], angle)
        page, slot = s["table"][b][pos // c["page"]].long(), pos % c["page"]
        k[0, page, slot] = turned(s["kin"][mine].double(), angle)
        v[0, page, slot] = s["vin"][mine].double()
    return q, k, v


def _work_rope(c):
    n = sum(_rows_of(c))
    values = n * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    return {"bytes": values * (DTYPES[c["into"]].itemsize + 2), "flops": 3 * n * (c["heads"] + c["kv_heads"]) * c["rot"]}


# ---- attn ----


def _prepare_attn(c, gen):
    rows, kv = _rows_of(c), _kv_of(c)
    n = sum(rows)
    held = [_cdiv(x, c["page"]) for x in kv]
    pages = sum(held) + 5
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], max(held)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(c["seqs"]):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    k, v = _storage(c, 1, pages, gen)
    q = (1.5 * torch.randn((n, c["heads"], c["dim"]), generator=gen, device="cuda")).to(DTYPES[c["dtype"]])
    s = dict(case=c, n_rows=n, q=q, k=k, v=v, row_start=_i32(_starts(rows)), kv_len=_i32(kv), table=table, max_rows=max(rows), scale=c["dim"] ** -0.5)
    if own:
        import w4_gemm_vqv_amd as vqv
        s["cache"] = vqv.PagedCache(k, v)
        s["seqs"] = vqv.Sequences(s["row_start"], s["kv_len"], table, n_rows=n, max_rows=max(rows), max_kv=max(kv))
        s["out"] = torch.empty_like(q)
        need = vqv.vqv_paged_attn_workspace_bytes(s["cache"], s["seqs"], c["heads"], window=c["window"], sinks=c["sinks"])
        s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return s


def _plain_attn(s):
    c = s["case"]
    hk, g, d, t, n_seqs = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], s["max_rows"], c["seqs"]
    pages = s["table"].long().clamp(min=0)
    k, v = (x[0][pages].flatten(1, 2).transpose(1, 2).float() for x in (s["k"], s["v"]))  # [seqs, kv heads, tokens, dim]
    counts = s["row_start"][1:] - s["row_start"][:-1]
    i = torch.arange(t, device="cuda")
    at = (s["row_start"][:-1, None] + i).clamp(max=s["n_rows"] - 1)
    q = s["q"][at].float().view(n_seqs, t, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n_seqs, hk, t * g, d)
    scores = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    pos = (s["kv_len"] - counts)[:, None] + i[None, :]
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j[None, None, :] <= pos[:, :, None]) & (j[None, None, :] < s["kv_len"][:, None, None])
    if c["window"]:
        seen &= (j[None, None, :] > pos[:, :, None] - c["window"]) | (j[None, None, :] < c["sinks"])
    seen = seen[:, None, :, None, :].expand(n_seqs, 1, t, g, -1).reshape(n_seqs, 1, t * g, -1)
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    o = o.view(n_seqs, hk, t, g, d).permute(0, 2, 1, 3, 4).reshape(n_seqs, t, hk * g, d)
    b, place = _row_places(s)
    return o[b, place].to(s["q"].dtype)


def _own_attn(s):
    import w4_gemm_vqv_amd as vqv
    c = s["case"]
    vqv.vqv_paged_attn(s["q"], s["cache"], s["seqs"], scale=s["scale"], window=c["window"], sinks=c["sinks"], out=s["out"], workspace=s["workspace"])
    return s["out"]


def _exact_attn(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g, starts, lens = c["heads"] // c["kv_heads"], s["row_start"].tolist(), s["kv_len"].tolist()
    for b in range(c["seqs"]):
        used = s["table"][b, :_cdiv(lens[b], c["page"])].long()
        n = starts[b + 1] - starts[b]
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")[:, None]
        key = torch.arange(lens[b], device="cuda")[None, :]
        hidden = key > pos
        if c["window"]:
            hidden = hidden | ((key <= pos - c["window"]) & (key >= c["sinks"]))
        for h in range(c["kv_heads"]):
            k = s["k"][0, used, :, h].reshape(-1, c["dim"])[:lens[b]].double()
            v = s["v"][0, used, :, h].reshape(-1, c["dim"])[:lens[b]].double()
            for e in range(h * g, (h + 1) * g):
                x = (s["q"][starts[b]:starts[b + 1], e].double() @ k.t()) * s["scale"]
                x.masked_fill_(hidden, -math.inf)
                out[starts[b]:starts[b + 1], e] = torch.softmax(x, 1) @ v
    return out


def _work_attn(c):
    values = pairs = 0
    for n, length in zip(_rows_of(c), _kv_of(c)):
        first = length - n
        window, sinks = c["window"] or length, c["sinks"] if c["window"] else 0
        low = max(first - window + 1, 0)  # the first row's window begins here
        values += 2 * (length - low + min(sinks, low)) * c["kv_heads"] * c["dim"] + 2 * n * c["heads"] * c["dim"]
        pairs += sum(min(p + 1, window) + min(sinks, max(p + 1 - window, 0)) for p in range(first, length))
    return {"bytes": 2 * values, "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---- cache ----


def _prepare_cache(c, gen):
    if c["op"] == "copy":
        k, v = _storage(c, c["layers"], 2 * c["seqs"] + 3, gen)
        order = torch.randperm(2 * c["seqs"] + 3, generator=gen, device="cuda").to(torch.int32)
        s = dict(case=c, k=k, v=v, src=order[:c["seqs"]].contiguous(), dst=order[c["seqs"]:2 * c["seqs"]].contiguous())
        if own:
            import w4_gemm_vqv_amd as vqv
            s["cache"] = vqv.PagedCache(k, v)
        return s
    rows, kv = _rows_of(c), _kv_of(c)
    held = [_cdiv(x, c["page"]) for x in kv]
    branches = c["seqs"] * c["rows"] if c["op"] == "fork" else 0
    spare = branches + 2 * c["seqs"] + 3
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"] + branches, max(held) + 2), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(c["seqs"]):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    ref[order[:at].long()] = 1
    k, v = _storage(c, c["layers"], pages, gen)
    s = dict(case=c, k=k, v=v, table=table, ref=ref, held=_i32(held + [0] * branches), length=_i32(kv + [0] * branches),
             row_start=_i32(_starts(rows)), kv_len=_i32(kv), n_rows=sum(rows))
    if c["op"] == "fork":
        s["parent"] = _i32([b for b in range(c["seqs"]) for _ in range(c["rows"])])
        s["child"] = _i32([c["seqs"] + i for i in range(branches)])
        s["none"] = _i32([0] * branches)
    else:
        # Rows that the target confirmed, along one branch of a drafted tree: row 0 always.
        s["keep"] = (torch.rand(s["n_rows"], generator=gen, device="cuda") < 0.6).to(torch.int32)
        s["keep"][s["row_start"][:-1].long()] = 1
    if own:
        import w4_gemm_vqv_amd as vqv
        s["cache"] = vqv.PagedCache(k, v)
        s["pages"] = vqv.Pages(ref, table, s["held"], s["length"], page_size=c["page"])
        s["workspace"] = torch.empty(vqv.vqv_cache_workspace_bytes(s["pages"]), dtype=torch.uint8, device="cuda")
        if c["op"] == "fork":
            s["ok"] = torch.empty(branches, dtype=torch.int32, device="cuda")
        else:
            s["seqs"] = vqv.Sequences(s["row_start"], s["kv_len"], table, n_rows=s["n_rows"], max_rows=max(rows), max_kv=max(kv))
            s["ok"] = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
    return s


def _plain_free(ref, rank_of, wanted):
    """The page that each wanted one gets: free pages in the order of their numbers."""
    free = torch.sort((ref != 0).to(torch.int32), stable=True).indices
    return torch.where(wanted, free[torch.where(wanted, rank_of, 0)], -1)


def _plain_trim(s, rows, keep_len):
    """Frees the pages of `rows` of the table that are past `keep_len` tokens."""
    c = s["case"]
    table, j = s["table"][rows], torch.arange(s["table"].shape[1], device="cuda")
    stay = torch.minimum((keep_len + c["page"] - 1) // c["page"], s["held"][rows])
    gone = (j[None, :] >= stay[:, None]) & (j[None, :] < s["held"][rows][:, None])
    s["ref"].index_add_(0, table.long().clamp(min=0).flatten(), -gone.to(torch.int32).flatten())
    s["table"][rows] = torch.where(gone, -1, table)
    s["held"][rows] = stay
    s["length"][rows] = torch.minimum(s["length"][rows], keep_len)


def _plain_cache(s):
    c = s["case"]
    if c["op"] == "copy":
        for x in (s["k"], s["v"]):
            x[:, s["dst"].long()] = x[:, s["src"].long()]
        return s["k"], s["v"]
    if c["op"] == "fork":
        parent, child = s["parent"].long(), s["child"].long()
        _plain_trim(s, child, s["none"])
        length = s["length"][parent]
        wanted = length % c["page"] != 0
        new = _plain_free(s["ref"], wanted.long().cumsum(0) - 1, wanted)
        last = ((length - 1) // c["page"]).clamp(min=0).long()
        old = s["table"][parent, last].long()
        for x in (s["k"], s["v"]):
            # A parent that ends with a page gives it as it is: that page is copied onto itself.
            x[:, torch.where(wanted, new, old)] = x[:, old]
        j = torch.arange(s["table"].shape[1], device="cuda")
        table = torch.where(wanted[:, None] & (j[None, :] == last[:, None]), new[:, None].to(torch.int32), s["table"][parent])
        one = (j[None, :] < s["held"][parent][:, None]).to(torch.int32)
        s["ref"].index_add_(0, table.long().clamp(min=0).flatten(), one.flatten())
        s["table"][child], s["held"][child], s["length"][child] = table, s["held"][parent], length
        return s["k"], s["v"], s["table"], s["ref"], s["held"], s["length"], torch.ones_like(s["child"])
    # The end of a round. The kept rows, in their order, take the chunk's first places.
    b, i = _row_places(s)
    n = s["row_start"][1:] - s["row_start"][:-1]
    kept = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda").index_add_(0, b, s["keep"])
    place = torch.sort(b * 2 + (s["keep"] == 0), stable=True).indices  # rows of a sequence: kept ones first
    source = torch.where(i < kept[b], place - s["row_start"][b], i)
    first = (s["kv_len"] - n)[b]
    to, of = first + i, first + source
    at_to, at_of = (s["table"][b, to // c["page"]].long(), to % c["page"]), (s["table"][b, of // c["page"]].long(), of % c["page"])
    for x in (s["k"], s["v"]):
        x[:, at_to[0], at_to[1]] = x[:, at_of[0], at_of[1]]
    new_len = (s["kv_len"] - n + kept).to(torch.int32)
    rows = torch.arange(c["seqs"], device="cuda")
    s["length"].copy_(new_len)
    _plain_trim(s, rows, new_len)
    # The next block may be as long as this one was.
    goal = ((s["kv_len"] + c["page"] - 1) // c["page"]).to(torch.int32)
    short = goal - s["held"]
    j = torch.arange(s["table"].shape[1], device="cuda")
    wanted = (j[None, :] >= s["held"][:, None]) & (j[None, :] < goal[:, None])
    rank_of = (short.cumsum(0) - short)[:, None] + j[None, :] - s["held"][:, None]
    new = _plain_free(s["ref"], rank_of, wanted).to(torch.int32)
    s["table"].copy_(torch.where(wanted, new, s["table"]))
    s["ref"].index_add_(0, new.long().clamp(min=0).flatten(), wanted.to(torch.int32).flatten())
    s["held"].copy_(goal)
    return s["k"], s["v"], s["table"], s["ref"], s["held"], s["length"], torch.ones_like(s["kv_len"])


def _own_cache(s):
    import w4_gemm_vqv_amd as vqv
    c = s["case"]
    if c["op"] == "copy":
        vqv.vqv_cache_copy(s["cache"], s["src"], s["dst"])
        return s["k"], s["v"]
    if c["op"] == "fork":
        vqv.vqv_cache_trim(s["pages"], s["none"], rows=s["child"])
        vqv.vqv_cache_fork(s["cache"], s["pages"], s["parent"], s["child"], ok=s["ok"], workspace=s["workspace"])
    else:
        vqv.vqv_cache_compact(s["cache"], s["seqs"], s["keep"], new_len=s["length"])
        vqv.vqv_cache_trim(s["pages"], s["length"])
        vqv.vqv_cache_reserve(s["pages"], s["kv_len"], ok=s["ok"], workspace=s["workspace"])
    return s["k"], s["v"], s["table"], s["ref"], s["held"], s["length"], s["ok"]


def _exact_cache(s):
    c = s["case"]
    k, v = s["k"].double(), s["v"].double()
    if c["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            k[:, b], v[:, b] = k[:, a], v[:, a]
        return k, v
    table, ref, held = s["table"].tolist(), s["ref"].tolist(), s["held"].tolist()
    length = s["length"].tolist()
    if c["op"] == "fork":
        for a, b in zip(s["parent"].tolist(), s["child"].tolist()):
            table[b], held[b], length[b] = list(table[a]), held[a], length[a]
            shared = table[a][:length[a] // c["page"]]
            for p in shared:
                ref[p] += 1
            if length[a] % c["page"]:
                new, old = ref.index(0), table[a][len(shared)]
                ref[new], table[b][len(shared)] = 1, new
                k[:, new], v[:, new] = k[:, old], v[:, old]
        return k, v, _i32(table), _i32(ref), _i32(held), _i32(length), torch.ones_like(s["child"])
    keep, starts = s["keep"].tolist(), s["row_start"].tolist()
    for b, total in enumerate(s["kv_len"].tolist()):
        first = to = total - (starts[b + 1] - starts[b])
        for i in range(starts[b + 1] - starts[b]):
            if keep[starts[b] + i]:
                (p0, s0), (p1, s1) = divmod(first + i, c["page"]), divmod(to, c["page"])
                k[:, table[b][p1], s1], v[:, table[b][p1], s1] = k[:, table[b][p0], s0], v[:, table[b][p0], s0]
                to += 1
        length[b] = to
        while held[b] > _cdiv(to, c["page"]):
            held[b] -= 1
            ref[table[b][held[b]]] -= 1
            table[b][held[b]] = -1
    for b, total in enumerate(s["kv_len"].tolist()):
        while held[b] < _cdiv(total, c["page"]):
            table[b][held[b]] = ref.index(0)
            ref[table[b][held[b]]] = 1
            held[b] += 1
    return k, v, _i32(table), _i32(ref), _i32(held), _i32(length), torch.ones_like(s["kv_len"])


def _work_cache(c):
    token = 2 * c["kv_heads"] * c["dim"] * 2 * c["layers"]  # bytes of a token's keys and values on all layers
    if c["op"] == "copy":
        return {"bytes": 2 * c["seqs"] * c["page"] * token, "flops": 0}
    entries = sum(_cdiv(x, c["page"]) for x in _kv_of(c))
    if c["op"] == "fork":
        copied = sum(x % c["page"] != 0 for x in _kv_of(c)) * c["rows"]
        return {"bytes": 2 * copied * c["page"] * token + 12 * entries * c["rows"], "flops": 0}
    # Of the rows after the first, 0.6 are kept, and the i-th kept one moves unless all before it were.
    moved = sum(0.6 * (1 - 0.6 ** i) for n in _rows_of(c) for i in range(n))
    return {"bytes": 2 * moved * token + 4 * sum(_rows_of(c)) + 16 * c["seqs"], "flops": 0}


# ---- logits ----


def _prepare_logits(c, gen):
    n_seqs, t, n = c["seqs"], c["rows"], c["vocab"]
    logits = 3.0 * torch.randn((n_seqs * t, n), generator=gen, device="cuda")
    s = dict(case=c, logits=logits, counts=None, seen=None, repetition=None, frequency=None, presence=None,
             bias_start=None, bias_token=None, bias_value=None, mask=None)
    s["draft"] = torch.randint(0, n, (n_seqs, t - 1), generator=gen, device="cuda").to(torch.int32)
    if t > 1:  # a good part of the drafts is what the target would choose
        good = torch.rand(n_seqs, t - 1, generator=gen, device="cuda") < 0.8
        s["draft"] = torch.where(good, logits.view(n_seqs, t, n)[:, :-1].argmax(2).to(torch.int32), s["draft"])
    words = _cdiv(n, 32)
    if c["penalties"]:
        # What a few thousand tokens of text leave: some tokens often, most never.
        at = (torch.rand(n_seqs, 2000, generator=gen, device="cuda").pow(3) * n).long().clamp(max=n - 1)
        s["counts"] = torch.zeros(n_seqs, n, dtype=torch.int32, device="cuda")
        s["counts"].scatter_add_(1, at, torch.ones_like(at, dtype=torch.int32))
        s["seen"] = _bits(torch.rand(n_seqs, 32 * words, generator=gen, device="cuda") < 0.01)
        s["repetition"] = 1 + 0.3 * torch.rand(n_seqs, generator=gen, device="cuda")
        s["frequency"] = 0.4 * torch.rand(n_seqs, generator=gen, device="cuda")
        s["presence"] = 0.8 * torch.rand(n_seqs, generator=gen, device="cuda")
    if c["bias"]:
        s["bias_start"] = _i32([b * c["bias"] for b in range(n_seqs + 1)])
        pick = torch.rand(n_seqs, n, generator=gen, device="cuda").topk(c["bias"], dim=1).indices
        s["bias_token"] = pick.flatten().to(torch.int32)
        s["bias_value"] = 4.0 * torch.randn(n_seqs * c["bias"], generator=gen, device="cuda")
    if c["mask"]:
        # Rows in free text allow nearly all tokens, rows inside a structure few.
        share = torch.where(torch.arange(n_seqs * t, device="cuda") % 3 == 0, 0.02, 0.97)
        s["mask"] = _bits(torch.rand(n_seqs * t, 32 * words, generator=gen, device="cuda") < share[:, None])
    if own:
        import w4_gemm_vqv_amd as vqv
        s["edits"] = vqv.Edits(n_seqs, n, counts=s["counts"], seen=s["seen"], repetition=s["repetition"], frequency=s["frequency"],
                               presence=s["presence"], bias_start=s["bias_start"], bias_token=s["bias_token"], bias_value=s["bias_value"])
        if c["op"] == "edit":
            s["out"] = torch.empty_like(logits)
        else:
            s["argmax"] = torch.empty(n_seqs * t, dtype=torch.int32, device="cuda")
            s["accept"] = torch.empty(n_seqs, dtype=torch.int32, device="cuda")
            s["margin"] = torch.empty(n_seqs * t, dtype=torch.float32, device="cuda")
            s["workspace"] = torch.empty(vqv.vqv_verify_workspace_bytes(n_seqs, t, n), dtype=torch.uint8, device="cuda")
    return s


def _bits(allowed):
    """[rows, 32 * words] truth values as int32 words, the lowest bit first."""
    w = allowed.view(allowed.shape[0], -1, 32).long() << torch.arange(32, device="cuda")
    w = w.sum(2)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def _plain_bits(words, n):
    return ((words[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).flatten(1)[:, :n] != 0


def _plain_logits(s):
    c = s["case"]
    n_seqs, t, n = c["seqs"], c["rows"], c["vocab"]
    x = s["logits"].view(n_seqs, t, n)
    if c["penalties"]:
        # Row i comes after the drafts that were fed at rows 1 to i.
        count = s["counts"][:, None, :].expand(n_seqs, t, n).contiguous()
        before = (torch.arange(t - 1, device="cuda")[None, :] < torch.arange(t, device="cuda")[:, None]).to(torch.int32)
        count.scatter_add_(2, s["draft"][:, None, :].expand(n_seqs, t, t - 1).long(), before[None].expand(n_seqs, t, t - 1).contiguous())
        used = count > 0
        r = s["repetition"][:, None, None]
        x = torch.where(used | _plain_bits(s["seen"], n)[:, None, :], torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None, None] * count.float()
        x = torch.where(used, x - s["presence"][:, None, None], x)
    if c["bias"]:
        bias = torch.zeros(n_seqs, n, device="cuda")
        bias.scatter_(1, s["bias_token"].view(n_seqs, -1).long(), s["bias_value"].view(n_seqs, -1))
        x = x + bias[:, None, :]
    if c["mask"]:
        x = torch.where(_plain_bits(s["mask"], n).view(n_seqs, t, n), x, float("-inf"))
    x = x.reshape(n_seqs * t, n)
    if c["op"] == "edit":
        return x
    top = x.amax(1, keepdim=True)
    j = torch.arange(n, device="cuda", dtype=torch.int32)
    best = torch.where(x == top, j, n).amin(1).to(torch.int32)
    second = torch.where(j[None, :] == best[:, None], float("-inf"), x).amax(1)
    margin = torch.where(top[:, 0] == second, 0.0, top[:, 0] - second)
    match = (best.view(n_seqs, t)[:, :t - 1] == s["draft"]).to(torch.int32)
    return best, match.cumprod(1).sum(1).to(torch.int32), margin


def _own_logits(s):
    import w4_gemm_vqv_amd as vqv
    c = s["case"]
    if c["op"] == "edit":
        vqv.vqv_logits_edit(s["logits"], s["edits"], s["draft"], c["seqs"], c["rows"], mask=s["mask"], out=s["out"])
        return s["out"]
    vqv.vqv_logits_verify(s["logits"], s["edits"], s["draft"], c["seqs"], c["rows"], mask=s["mask"], argmax=s["argmax"],
                          accept_len=s["accept"], margin=s["margin"], workspace=s["workspace"])
    return s["argmax"], s["accept"], s["margin"]


def _exact_logits(s):
    c = s["case"]
    n_seqs, t, n = c["seqs"], c["rows"], c["vocab"]
    rows, draft = [], s["draft"].tolist()
    shift = torch.arange(32, device="cuda")
    for b in range(n_seqs):
        count = s["counts"][b].double() if c["penalties"] else None
        for i in range(t):
            x = s["logits"][b * t + i].double()
            if c["penalties"]:
                if i:
                    count[draft[b][i - 1]] += 1
                told = (count > 0) | ((s["seen"][b].long()[:, None] >> shift & 1).flatten()[:n] == 1)
                r = s["repetition"][b].double()
                x = torch.where(told, torch.where(x > 0, x / r, x * r), x)
                x = x - s["frequency"][b].double() * count - s["presence"][b].double() * (count > 0)
            if c["bias"]:
                mine = slice(b * c["bias"], (b + 1) * c["bias"])
                x[s["bias_token"][mine].long()] += s["bias_value"][mine].double()
            if c["mask"]:
                x[(s["mask"][b * t + i].long()[:, None] >> shift & 1).flatten()[:n] == 0] = -math.inf
            rows.append(x)
    x = torch.stack(rows)
    if c["op"] == "edit":
        return x
    order = torch.sort(x, dim=1, descending=True, stable=True)
    best = order.indices[:, 0].view(n_seqs, t)
    accept = [next((i for i in range(t - 1) if int(best[b, i]) != draft[b][i]), t - 1) for b in range(n_seqs)]
    top = order.values[:, :2]
    return best.flatten().to(torch.int32), _i32(accept), torch.where(top[:, 0] == top[:, 1], 0.0, top[:, 0] - top[:, 1])


def _work_logits(c):
    rows, n = c["seqs"] * c["rows"], c["vocab"]
    values = 4 * rows * n * (2 if c["op"] == "edit" else 1)
    state = c["seqs"] * n * (4 + 1 / 8) if c["penalties"] else 0
    return {"bytes": values + state + (rows * n / 8 if c["mask"] else 0) + 8 * c["seqs"] * c["bias"], "flops": 5 * rows * n}
