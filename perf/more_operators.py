"""Operators that serve many requests in one verify round, as cases that can be timed and compared.

Requests share a batch although each has its own sampling, its own adapter and a long history: the cache holds keys
and values in 4 bits, drafted tokens are verified against the target's probabilities, and low-rank adapters are added
beside the shared projection. Each case is one of these:

  rope     rotary positions of queries and keys, the keys and values written to a 4-bit cache's pages, and the new
           rows read back as the cache holds them
  attn     attention of new rows over the pages of a 4-bit cache (also with a window and visible first tokens)
  sample   verification of drafted tokens against the target's probabilities, from given random numbers
  lora     low-rank adapters, one per row's request, added to a projection's output

`run` computes an operator in its plain form, in elementary torch operations, or (with `own`) by the library's call.

The cache holds a record per token and key head: dim / 2 bytes of codes, then a scale and a bias in fp16 for every 32
values (the last group may be shorter), zeros up to a multiple of 16 bytes. A 32-bit word of codes holds 8 values, value
2 i + j of them in bits 16 j + 4 i and up. A group's values are cut to +-32768, its bias is their least and its scale a
fifteenth of their spread, both rounded to fp16, a code is (x - bias) * (1 / scale) to the nearest whole number of 0 to
15, each step in fp32; value = scale * code + bias.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"


def listed():
    return [
        # One sequence's verify block of 8 rows, straight from the fp32 output of a stacked q/k/v projection: latency.
        dict(name="q4 rope block 1x8", kind="rope", into="fp32", dtype="bf16", layout="slot", seqs=1, rows=8, kv=2048, heads=32,
             kv_heads=8, dim=128, page=16, rot=128, interleaved=False, ragged=False),
        # Prompt chunks far into long contexts: interleaved pairs in half of each head.
        dict(name="q4 rope chunk 4x2048 far", kind="rope", into="bf16", dtype="bf16", layout="head", seqs=4, rows=2048, kv=200000,
             heads=32, kv_heads=8, dim=128, page=64, rot=64, interleaved=True, ragged=True),
        # One sequence's verify block over a short cache: latency.
        dict(name="q4 attn block 1x8 kv 4k", kind="attn", dtype="bf16", layout="slot", seqs=1, rows=8, kv=4096, heads=32, kv_heads=8,
             dim=128, page=16, window=0, sinks=0, ragged=False),
        # Plain decoding, a token for each of many sequences of very different lengths.
        dict(name="q4 decode 48x1 ragged", kind="attn", dtype="bf16", layout="slot", seqs=48, rows=1, kv=16383, heads=32,
             kv_heads=8, dim=128, page=16, window=0, sinks=0, ragged=True),
        # A prompt's chunk after what is already in the cache: matrix-bound.
        dict(name="q4 chunk 1x2048 kv 10k", kind="attn", dtype="bf16", layout="head", seqs=1, rows=2048, kv=10240, heads=32,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, ragged=False),
        # Batched verify blocks of 16 rows with wide heads over long caches of which a window and the first tokens are seen.
        dict(name="q4 window block 16x16 dim 256", kind="attn", dtype="fp16", layout="slot", seqs=16, rows=16, kv=32003, heads=16,
             kv_heads=4, dim=256, page=32, window=4096, sinks=4, ragged=True),
        # One request's verify block of 8 rows over the vocabulary, with the drafter's probabilities: latency.
        dict(name="sample 1x8", kind="sample", seqs=1, rows=8, vocab=151936, drafter="probs", ragged=False, greedy=0),
        # Batched verify blocks, requests with temperature and greedy ones together, some blocks cut short.
        dict(name="sample 4x16", kind="sample", seqs=4, rows=16, vocab=151936, drafter="probs", ragged=True, greedy=1),
        # Plain decoding of many requests, a token drawn for each.
        dict(name="sample 64x1", kind="sample", seqs=64, rows=1, vocab=151936, drafter="none", ragged=False, greedy=0),
        # A verify block of one request with its adapter beside the target projection: latency.
        dict(name="lora 8 rows rank 16", kind="lora", dtype="bf16", seqs=1, rows=8, K=5120, N=17408, rank=16, adapters=4, idle=0.0),
        # Plain decoding, 64 requests of 40 adapters, some of them without one.
        dict(name="lora 64x1 rank 32", kind="lora", dtype="bf16", seqs=64, rows=1, K=2560, N=18432, rank=32, adapters=40, idle=0.1),
        # Prompt chunks of three requests with wide adapters.
        dict(name="lora chunks 3x700 rank 64", kind="lora", dtype="fp16", seqs=3, rows=700, K=5120, N=17408, rank=64, adapters=3, idle=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "attn", "attn", "window", "sample", "sample", "lora", "lora"])
    if kind == "sample":
        rows = rng.choice([1, 2, 8, 16, rng.randint(1, 24)])
        return dict(kind=kind, seqs=rng.randint(1, max(1, 48 // rows)), rows=rows, vocab=_log_int(rng, 100, 160000),
                    drafter=rng.choice(["probs", "probs", "none"]), ragged=rng.random() < 0.5, greedy=rng.choice([0, 0, 1, 2]))
    if kind == "lora":
        seqs, rows = rng.randint(1, 64), rng.choice([1, 1, 8, rng.randint(1, 16)])
        if rng.random() < 0.25:
            seqs, rows = rng.randint(1, 3), _log_int(rng, 16, 600)
        return dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), seqs=seqs, rows=rows, K=64 * _log_int(rng, 1, 128),
                    N=_log_int(rng, 1, 16000), rank=8 * _log_int(rng, 1, 16), adapters=rng.randint(1, 48), idle=rng.choice([0.0, 0.1, 0.5]))
    layout, dtype, dim = rng.choice(["slot", "head"]), rng.choice(["bf16", "fp16"]), rng.choice([64, 80, 96, 128, 128, 192, 256])
    kv_heads, page = rng.randint(1, 8), rng.choice([1, 8, 16, 20, 32, 64, 128])
    if kind == "rope":
        rows = _log_int(rng, 1, 1000)
        return dict(kind=kind, into=rng.choice(["fp32", "bf16", "fp16"]), dtype=dtype, layout=layout, seqs=rng.randint(1, 8), rows=rows,
                    kv=rows + _log_int(rng, 1, 500000), heads=kv_heads * rng.randint(1, 4), kv_heads=kv_heads, dim=dim, page=max(8, page),
                    rot=2 * rng.randint(1, dim // 2), interleaved=rng.random() < 0.5, ragged=rng.random() < 0.7)
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _starts(rows):
    s = [0]
    for r in rows:
        s.append(s[-1] + r)
    return s


def _row_places(s):
    """Sequence and place in its chunk of every row."""
    r = torch.arange(s["n_rows"], device=DEVICE)
    b = (r[:, None] >= s["row_start"][None, 1:]).sum(1).clamp(max=s["kv_len"].numel() - 1)
    return b, r - s["row_start"][b]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    return {"rope": _prepare_rope, "attn": _prepare_attn, "sample": _prepare_sample, "lora": _prepare_lora}[case["kind"]](case, gen)


def run(state):
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "sample": _own_sample, "lora": _own_lora}[state["case"]["kind"]](state)
    return {"rope": _plain_rope, "attn": _plain_attn, "sample": _plain_sample, "lora": _plain_lora}[state["case"]["kind"]](state)


def exact(case, seed):
    return {"rope": _exact_rope, "attn": _exact_attn, "sample": _exact_sample, "lora": _exact_lora}[case["kind"]](prepare(case, seed))


def work(case):
    return {"rope": _work_rope, "attn": _work_attn, "sample": _work_sample, "lora": _work_lora}[case["kind"]](case)


# ---- the 4-bit records ----


def _record(dim):
    return _cdiv(dim // 2 + 4 * _cdiv(dim, 32), 16) * 16


def _shift():
    v = torch.arange(8, device=DEVICE, dtype=torch.int32)
    return 16 * (v & 1) + 4 * (v >> 1)


def _pack(x):
    """Records (uint8) of fp32 values [..., dim]."""
    dim, groups = x.shape[-1], _cdiv(x.shape[-1], 32)
    x = x.clamp(-32768.0, 32768.0)
    lo = torch.stack([g.amin(-1) for g in x.split(32, -1)], -1)
    hi = torch.stack([g.amax(-1) for g in x.split(32, -1)], -1)
    scale, bias = ((hi - lo) * (1 / 15)).half(), lo.half()
    s, b = (t.float().repeat_interleave(32, -1)[..., :dim] for t in (scale, bias))
    code = torch.where(s == 0, 0.0, torch.round((x - b) * torch.where(s == 0, 1.0, s).reciprocal()).clamp(0, 15)).to(torch.int32)
    words = (code.unflatten(-1, (dim // 8, 8)) << _shift()).sum(-1).to(torch.int32)
    rec = torch.zeros(*x.shape[:-1], _record(dim), dtype=torch.uint8, device=DEVICE)
    rec[..., :dim // 2] = words.view(torch.uint8)
    rec[..., dim // 2:dim // 2 + 4 * groups] = torch.stack([scale, bias], -1).flatten(-2).contiguous().view(torch.uint8)
    return rec


def _unpack(rec, dim):
    """Values [..., dim] in 32 bits of records (uint8)."""
    groups = _cdiv(dim, 32)
    words = rec[..., :dim // 2].contiguous().view(torch.int32)
    code = ((words[..., None] >> _shift()) & 15).flatten(-2).float()
    pairs = rec[..., dim // 2:dim // 2 + 4 * groups].contiguous().view(torch.float16).float().unflatten(-1, (groups, 2))
    s, b = (pairs[..., i].repeat_interleave(32, -1)[..., :dim] for i in (0, 1))
    return code * s + b


def _values64(rec, dim):
    """The same in 64 bits, byte by byte."""
    out = torch.empty(*rec.shape[:-1], dim, dtype=torch.float64, device=DEVICE)
    for i in range(dim):
        byte = rec[..., i // 8 * 4 + 2 * (i % 2) + i % 8 // 4].int()
        code = byte // 16 if i % 8 // 2 % 2 else byte % 16
        at = dim // 2 + i // 32 * 4
        pair = rec[..., at:at + 4].contiguous().view(torch.float16).double()
        out[..., i] = pair[..., 0] * code + pair[..., 1]
    return out


def _swap(c, x):
    """Heads outermost in a page's memory, or slots."""
    return x.transpose(2, 3).contiguous().transpose(2, 3) if c["layout"] == "head" else x


# ---- rope ----

BASE = 1e6


def _prepare_rope(c, gen):
    rows, kv = _rows_of(c), _kv_of(c)
    n = sum(rows)
    width = _cdiv(c["kv"], c["page"]) + 1
    # Pages that the chunk's rows fall into are in the pool; what is before them is never touched here.
    tails = [(_cdiv(kv[b], c["page"]) - (kv[b] - rows[b]) // c["page"]) for b in range(c["seqs"])]
    pages = sum(tails) + 3
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b in range(c["seqs"]):
        first = (kv[b] - rows[b]) // c["page"]
        table[b, first:first + tails[b]] = order[at:at + tails[b]]
        at += tails[b]
    heads, hk, d = c["heads"], c["kv_heads"], c["dim"]
    qkv = torch.randn((n, (heads + 2 * hk) * d), generator=gen, device=DEVICE)
    qkv += 0.5 * torch.randn((1, (heads + 2 * hk) * d), generator=gen, device=DEVICE)  # columns have means of their own
    qkv = qkv.to(DTYPES[c["into"]])
    shape = (1, pages, c["page"], hk, _record(d))
    k, v = (_swap(c, torch.zeros(shape, dtype=torch.uint8, device=DEVICE)) for _ in range(2))
    s = dict(case=c, n_rows=n, qkv=qkv, q=qkv[:, :heads * d].view(n, heads, d), kin=qkv[:, heads * d:(heads + hk) * d].view(n, hk, d),
             vin=qkv[:, (heads + hk) * d:].view(n, hk, d), k=k, v=v, row_start=_i32(_starts(rows)), kv_len=_i32(kv), table=table)
    if own:
        import w4_gemm_vqv_amd as vqv
        s["cache"] = vqv.PagedCacheQ4(k, v, d)
        s["seqs"] = vqv.Sequences(s["row_start"], s["kv_len"], table, n_rows=n, max_rows=max(rows), max_kv=max(kv))
        s["rope"] = vqv.Rope(c["rot"], BASE, interleaved=c["interleaved"])
        s["q_out"] = torch.empty((n, heads, d), dtype=DTYPES[c["dtype"]], device=DEVICE)
        s["k_out"], s["v_out"] = (torch.empty((n, hk, d), dtype=torch.float32, device=DEVICE) for _ in range(2))
    return s


def _plain_rotate(x, angle, c):
    """x [rows, heads, dim], in 64 bits: keys are next to a code's border."""
    rot, x = c["rot"], x.double()
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    b, i = _row_places(s)
    pos = (s["kv_len"][b] - (s["row_start"][b + 1] - s["row_start"][b])).long() + i
    f = BASE ** (-2 * torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEVICE) / c["rot"])
    angle = pos.double()[:, None] * f[None, :]
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    s["k"][0].index_put_((page, slot), _pack(_plain_rotate(s["kin"], angle, c).float()))
    s["v"][0].index_put_((page, slot), _pack(s["vin"].float()))
    q = _plain_rotate(s["q"], angle, c).float().to(DTYPES[c["dtype"]])
    return q, _unpack(s["k"][0][page, slot], c["dim"]), _unpack(s["v"][0][page, slot], c["dim"])


def _own_rope(s):
    import w4_gemm_vqv_amd as vqv
    vqv.vqv_rope_append_q4(s["q"], s["kin"], s["vin"], s["cache"], s["seqs"], s["rope"], q_out=s["q_out"])
    vqv.vqv_cache_q4_read(s["cache"], s["seqs"], k_out=s["k_out"], v_out=s["v_out"])
    return s["q_out"], s["k_out"], s["v_out"]


def _exact_held(x):
    """What the records of x [..., dim] stand for."""
    x = x.float().double().clamp(-32768.0, 32768.0)  # a key is rounded once after its turn
    out = torch.empty_like(x)
    for at in range(0, x.shape[-1], 32):
        g = x[..., at:at + 32]
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        s, b = ((hi - lo).float() * (1 / 15)).half().double(), lo.half().double()
        code = torch.where(s > 0, ((g - b).float() * s.float().reciprocal()).double().round().clamp(0, 15), 0.0)
        out[..., at:at + 32] = s * code + b
    return out


def _exact_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    f = torch.tensor([math.exp(-2.0 * i / rot * math.log(BASE)) for i in range(half)], dtype=torch.float64, device=DEVICE)
    starts, lens, rows = s["row_start"].tolist(), s["kv_len"].tolist(), _rows_of(c)
    even = torch.arange(half, device=DEVICE) * (2 if c["interleaved"] else 1)
    odd = even + (1 if c["interleaved"] else half)
    pos = torch.cat([torch.arange(lens[b] - rows[b], lens[b], device=DEVICE) for b in range(c["seqs"])])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE), (pos.double()[:, None] * f)[:, None, :])

    def turned(x):
        x = x.double()
        z = torch.complex(x[..., even], x[..., odd]) * turn
        y = x.clone()
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    return turned(s["q"]), _exact_held(turned(s["kin"])), _exact_held(s["vin"].double())


def _work_rope(c):
    n, hk, d = sum(_rows_of(c)), c["kv_heads"], c["dim"]
    into = n * (c["heads"] + 2 * hk) * d * DTYPES[c["into"]].itemsize
    out = n * (c["heads"] * d * 2 + 2 * hk * (_record(d) + 4 * d))
    return {"bytes": into + out, "flops": n * (3 * (c["heads"] + hk) * c["rot"] + 10 * hk * d)}


# ---- attn ----


def _prepare_attn(c, gen):
    rows, kv = _rows_of(c), _kv_of(c)
    n = sum(rows)
    held = [_cdiv(x, c["page"]) for x in kv]
    pages = sum(held) + 5
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((c["seqs"], max(held)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b in range(c["seqs"]):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]

    def storage(mean):
        # Columns of keys have means of their own, so that scores go by what differs between tokens.
        x = torch.empty((1, pages, c["page"], c["kv_heads"], _record(c["dim"])), dtype=torch.uint8, device=DEVICE)
        offset = mean * torch.randn((c["kv_heads"], c["dim"]), generator=gen, device=DEVICE)
        step = max(1, (1 << 26) // (c["page"] * c["kv_heads"] * c["dim"]))
        for p in range(0, pages, step):
            m = min(step, pages - p)
            x[0, p:p + m] = _pack(torch.randn((m, c["page"], c["kv_heads"], c["dim"]), generator=gen, device=DEVICE) + offset)
        return _swap(c, x)

    k, v = storage(0.5), storage(0.0)
    q = (1.5 * torch.randn((n, c["heads"], c["dim"]), generator=gen, device=DEVICE)).to(DTYPES[c["dtype"]])
    s = dict(case=c, n_rows=n, q=q, k=k, v=v, row_start=_i32(_starts(rows)), kv_len=_i32(kv), table=table, max_rows=max(rows), scale=c["dim"] ** -0.5)
    if own:
        import w4_gemm_vqv_amd as vqv
        s["cache"] = vqv.PagedCacheQ4(k, v, c["dim"])
        s["seqs"] = vqv.Sequences(s["row_start"], s["kv_len"], table, n_rows=n, max_rows=max(rows), max_kv=max(kv))
        s["out"] = torch.empty_like(q)
        need = vqv.vqv_paged_attn_q4_workspace_bytes(s["cache"], s["seqs"], c["heads"], window=c["window"], sinks=c["sinks"])
        s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEVICE)
    return s


def _plain_attn(s):
    c = s["case"]
    hk, g, d, t, n_seqs = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], s["max_rows"], c["seqs"]
    pages = s["table"].long().clamp(min=0)
    k, v = (_unpack(x[0][pages].flatten(1, 2).transpose(1, 2), d) for x in (s["k"], s["v"]))  # [seqs, kv heads, tokens, dim]
    counts = s["row_start"][1:] - s["row_start"][:-1]
    i = torch.arange(t, device=DEVICE)
    at = (s["row_start"][:-1, None] + i).clamp(max=s["n_rows"] - 1)
    q = s["q"][at].float().view(n_seqs, t, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n_seqs, hk, t * g, d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    pos = (s["kv_len"] - counts)[:, None] + i[None, :]
    j = torch.arange(k.shape[2], device=DEVICE)
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
    vqv.vqv_paged_attn_q4(s["q"], s["cache"], s["seqs"], scale=s["scale"], window=c["window"], sinks=c["sinks"], out=s["out"], workspace=s["workspace"])
    return s["out"]


def _exact_attn(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    g, starts, lens = c["heads"] // c["kv_heads"], s["row_start"].tolist(), s["kv_len"].tolist()
    for b in range(c["seqs"]):
        used = s["table"][b, :_cdiv(lens[b], c["page"])].long()
        n = starts[b + 1] - starts[b]
        pos = torch.arange(lens[b] - n, lens[b], device=DEVICE)[:, None]
        key = torch.arange(lens[b], device=DEVICE)[None, :]
        hidden = key > pos
        if c["window"]:
            hidden = hidden | ((key <= pos - c["window"]) & (key >= c["sinks"]))
        keys, values = (_values64(x[0, used].flatten(0, 1)[:lens[b]], c["dim"]) for x in (s["k"], s["v"]))
        for h in range(c["kv_heads"]):
            for e in range(h * g, (h + 1) * g):
                x = (s["q"][starts[b]:starts[b + 1], e].double() @ keys[:, h].t()) * s["scale"]
                x.masked_fill_(hidden, -math.inf)
                out[starts[b]:starts[b + 1], e] = torch.softmax(x, 1) @ values[:, h]
    return out


def _work_attn(c):
    tokens = n_q = pairs = 0
    for n, length in zip(_rows_of(c), _kv_of(c)):
        first = length - n
        window, sinks = c["window"] or length, c["sinks"] if c["window"] else 0
        low = max(first - window + 1, 0)  # the first row's window begins here
        tokens += length - low + min(sinks, low)
        n_q += n
        pairs += sum(min(p + 1, window) + min(sinks, max(p + 1 - window, 0)) for p in range(first, length))
    d = c["dim"]
    return {"bytes": 2 * tokens * c["kv_heads"] * (d // 2 + 4 * _cdiv(d, 32)) + 4 * n_q * c["heads"] * d, "flops": 4 * pairs * c["heads"] * d}


# ---- sample ----


def _prepare_sample(c, gen):
    n_seqs, t, n = c["seqs"], c["rows"], c["vocab"]
    logits = 3.0 * torch.randn((n_seqs * t, n), generator=gen, device=DEVICE)
    temperature = 0.5 + 0.7 * torch.rand(n_seqs, generator=gen, device=DEVICE)
    if c["greedy"]:  # such requests are in the batch too
        temperature[torch.arange(n_seqs, device=DEVICE) % (c["greedy"] + 1) == 0] = 0.0
    s = dict(case=c, logits=logits, temperature=temperature, probs=None, draft_len=None,
             uniform=torch.rand((n_seqs, t), generator=gen, device=DEVICE))
    # The drafter's view of what follows row i: near the target's.
    heat = torch.where(temperature > 0, temperature, 0.1)[:, None, None]
    near = logits.view(n_seqs, t, n)[:, :-1] + 0.4 * torch.randn((n_seqs, t - 1, n), generator=gen, device=DEVICE)
    probs = torch.softmax(near / heat, 2)
    if c["drafter"] == "probs":
        # Drawn from its probabilities.
        at = probs.double().cumsum(2)
        pick = torch.rand((n_seqs, t - 1, 1), generator=gen, device=DEVICE, dtype=torch.float64) * at[:, :, -1:]
        s["draft"] = torch.searchsorted(at, pick, right=True)[:, :, 0].clamp(max=n - 1).to(torch.int32)
        s["probs"] = probs
    else:
        s["draft"] = probs.argmax(2).to(torch.int32)  # its best guess, as of a lookup
    if c["ragged"]:
        s["draft_len"] = _i32([max(0, t - 1 - int(t * _spread(b))) for b in range(n_seqs)])
    if own:
        import w4_gemm_vqv_amd as vqv
        s["token"] = torch.empty(n_seqs, dtype=torch.int32, device=DEVICE)
        s["accept"] = torch.empty(n_seqs, dtype=torch.int32, device=DEVICE)
        s["logprob"] = torch.empty((n_seqs, t), dtype=torch.float32, device=DEVICE)
        s["workspace"] = torch.empty(vqv.vqv_verify_sampled_workspace_bytes(n_seqs, t, n), dtype=torch.uint8, device=DEVICE)
    return s


def _plain_sample(s):
    """In 64 bits: a drawn token is next to the borders of its neighbours."""
    c = s["case"]
    n_seqs, t, n = c["seqs"], c["rows"], c["vocab"]
    x = s["logits"].view(n_seqs, t, n)
    j = torch.arange(n, device=DEVICE)
    top = x.amax(2, keepdim=True)
    heat = s["temperature"].double()[:, None, None]
    e = torch.exp((x.double() - top) / torch.where(heat > 0, heat, 1.0))
    p = e / e.sum(2, keepdim=True)
    first = torch.where(x == top, j, n).amin(2, keepdim=True)
    p = torch.where(heat > 0, p, (j == first).double())
    accept = torch.zeros(n_seqs, dtype=torch.int32, device=DEVICE)
    if t > 1:
        d = s["draft"].long()[:, :, None]
        pd = p[:, :-1].gather(2, d)[:, :, 0]
        qd = s["probs"].gather(2, d)[:, :, 0].double() if s["probs"] is not None else 1.0
        good = s["uniform"][:, :-1].double() * qd < pd
        length = s["draft_len"] if s["draft_len"] is not None else torch.full((n_seqs,), t - 1, device=DEVICE)
        good &= torch.arange(t - 1, device=DEVICE)[None, :] < length[:, None]
        accept = good.int().cumprod(1).sum(1)
    b = torch.arange(n_seqs, device=DEVICE)
    r = p[b, accept]
    if t > 1:
        i = accept.clamp(max=t - 2)
        q = s["probs"][b, i].double() if s["probs"] is not None else (j[None, :] == s["draft"][b, i][:, None]).double()
        rest = (r - q).clamp(min=0.0)
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, r)
        r = torch.where((accept < length)[:, None], rest, r)
    at = r.cumsum(1)
    over = (at > s["uniform"][:, -1:].double() * at[:, -1:]) & (r > 0)
    lowest = torch.where(over, j, n).amin(1)
    last = torch.where(r > 0, j, 0).amax(1)
    token = torch.where(lowest < n, lowest, last)
    # What the committed tokens' logarithms of probability are, zeros behind them.
    i = torch.arange(t, device=DEVICE)[None, :]
    committed = torch.where(i == accept[:, None], token[:, None], 0)
    if t > 1:
        committed = torch.where(i < accept[:, None], torch.nn.functional.pad(s["draft"].long(), (0, 1)), committed)
    logp = torch.log(p.gather(2, committed[:, :, None])[:, :, 0])
    return token.to(torch.int32), accept.to(torch.int32), torch.where(i <= accept[:, None], logp, 0.0).float()


def _own_sample(s):
    import w4_gemm_vqv_amd as vqv
    c = s["case"]
    vqv.vqv_verify_sampled(s["logits"], s["draft"], s["uniform"], c["seqs"], c["rows"], draft_probs=s["probs"], temperature=s["temperature"],
                           draft_len=s["draft_len"], token=s["token"], accept_len=s["accept"], logprob=s["logprob"],
                           workspace=s["workspace"])
    return s["token"], s["accept"], s["logprob"]


def _exact_sample(s):
    c = s["case"]
    t, n = c["rows"], c["vocab"]
    tokens, accepts = [], []
    logprob = torch.zeros((c["seqs"], t), dtype=torch.float64, device=DEVICE)
    uniform, heat, draft = s["uniform"].tolist(), s["temperature"].tolist(), s["draft"].tolist()

    def target(b, i):
        x = s["logits"][b * t + i].double()
        if not heat[b] > 0:
            p = torch.zeros_like(x)
            p[int(torch.sort(x, descending=True, stable=True).indices[0])] = 1.0
            return p, torch.log(p)
        return torch.softmax(x / heat[b], 0), torch.log_softmax(x / heat[b], 0)

    for b in range(c["seqs"]):
        count = t - 1 if s["draft_len"] is None else int(s["draft_len"][b])
        i = 0
        while True:
            p, logs = target(b, i)
            if i >= count:
                break
            q = torch.zeros_like(p) if s["probs"] is None else s["probs"][b, i].double()
            if s["probs"] is None:
                q[draft[b][i]] = 1.0
            if not uniform[b][i] * float(q[draft[b][i]]) < float(p[draft[b][i]]):
                rest = torch.relu(p - q)
                p = rest if float(rest.sum()) > 0 else p
                break
            logprob[b, i] = logs[draft[b][i]]
            i += 1
        held = torch.nonzero(p > 0)[:, 0]
        edges = torch.cumsum(p[held], 0)
        at = int(torch.searchsorted(edges, uniform[b][t - 1] * edges[-1], right=True))
        tokens.append(int(held[min(at, held.numel() - 1)]))
        accepts.append(i)
        logprob[b, i] = logs[tokens[-1]]
    return _i32(tokens), _i32(accepts), logprob


def _work_sample(c):
    rows, n = c["seqs"] * c["rows"], c["vocab"]
    again = 4 * c["seqs"] * n if c["drafter"] == "probs" and c["rows"] > 1 else 0
    return {"bytes": 4 * rows * n + again, "flops": 4 * rows * n}


# ---- lora ----


def _prepare_lora(c, gen):
    t = DTYPES[c["dtype"]]
    weight = t if t != torch.float32 else torch.bfloat16
    m, k, n, r = c["seqs"] * c["rows"], c["K"], c["N"], c["rank"]
    x = torch.randn((m, k), generator=gen, device=DEVICE).to(t)
    a = (k ** -0.5 * torch.randn((c["adapters"], r, k), generator=gen, device=DEVICE)).to(weight)
    b = (r ** -0.5 * torch.randn((c["adapters"], n, r), generator=gen, device=DEVICE)).to(weight)
    scale = 0.5 + torch.rand(c["adapters"], generator=gen, device=DEVICE)
    pick = torch.randint(0, c["adapters"], (c["seqs"],), generator=gen, device=DEVICE)
    pick = torch.where(torch.rand(c["seqs"], generator=gen, device=DEVICE) < c["idle"], -1, pick)
    which = pick.repeat_interleave(c["rows"]).to(torch.int32)
    y = torch.randn((m, n), generator=gen, device=DEVICE)
    s = dict(case=c, x=x, a=a, b=b, scale=scale, which=which, y=y)
    if own:
        import w4_gemm_vqv_amd as vqv
        s["set"] = vqv.Adapters(a, b, scale)
        s["out"] = torch.empty_like(y)
        need = vqv.vqv_lora_add_workspace_bytes(s["set"], m)
        s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEVICE)
    return s


def _plain_lora(s):
    x, out = s["x"].float(), s["y"]
    for e in range(s["case"]["adapters"]):
        part = s["scale"][e] * torch.matmul(torch.matmul(x, s["a"][e].float().t()), s["b"][e].float().t())
        out = torch.where((s["which"] == e)[:, None], out + part, out)
    return out


def _own_lora(s):
    import w4_gemm_vqv_amd as vqv
    vqv.vqv_lora_add(s["x"], s["set"], s["which"], s["y"], out=s["out"], workspace=s["workspace"])
    return s["out"]


def _exact_lora(s):
    out = s["y"].double()
    for e in sorted(set(s["which"].tolist()) - {-1}):
        rows = torch.nonzero(s["which"] == e)[:, 0]
        low = s["x"][rows].double() @ s["a"][e].double().t()
        out[rows] += (low * s["scale"][e].double()) @ s["b"][e].double().t()
    return out


def _work_lora(c):
    m, k, n, r = c["seqs"] * c["rows"], c["K"], c["N"], c["rank"]
    # Of the adapters, those that some request is likely to pick; requests pick one at random.
    live = c["adapters"] * (1 - (1 - (1 - c["idle"]) / c["adapters"]) ** c["seqs"])
    size = DTYPES[c["dtype"]].itemsize
    return {"bytes": m * k * size + 8 * m * n + 2 * live * r * (k + n), "flops": 2 * (1 - c["idle"]) * m * r * (k + n)}
