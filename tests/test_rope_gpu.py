"""vqv_rope_append against the oracle: queries turned, keys turned and written
to the pages with the values, everything else in the cache untouched."""

import pytest
import torch

from oracle import round_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SENTINEL = 7.0


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def storage(layers, pages, ps, hk, dim, dtype, layout):
    """k or v of a cache, filled with a sentinel; "gap" leaves room between slots."""
    if layout == "head":
        return torch.full((layers, pages, hk, ps, dim), SENTINEL, dtype=dtype,
                          device="cuda").transpose(2, 3)
    if layout == "gap":
        return torch.full((layers, pages, ps + 1, hk, dim + 8), SENTINEL, dtype=dtype,
                          device="cuda")[:, :, :ps, :, :dim]
    return torch.full((layers, pages, ps, hk, dim), SENTINEL, dtype=dtype, device="cuda")


def check(vqv, rows, kv, heads, hk, dim, ps, rot, inter, scaling="none", into="fp32", dtype="bf16",
          layout="slot", layers=1, layer=0, bad=(), seed=0, base=1e6, factor=8.0):
    """bad: (sequence, page index) entries of the table that hold no page."""
    torch.manual_seed(seed)
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    n, width = start[-1], max(-(-x // ps) for x in kv) + 1
    # Only pages under the new rows exist; -1 elsewhere.
    table, used = [[-1] * width for _ in rows], 0
    for b, (r, x) in enumerate(zip(rows, kv)):
        for t in range(max(x - r, 0), x):
            if table[b][t // ps] < 0:
                table[b][t // ps] = used
                used += 1
    for b, j in bad:
        table[b][j] = -1 if j % 2 else used + 1000
    pages = used + 2
    perm = torch.randperm(pages).tolist()
    table = [[perm[p] if 0 <= p < pages else p for p in row] for row in table]
    qkv = torch.randn(n, (heads + 2 * hk) * dim).to(DT[into]).cuda()
    q, k, v = qkv.split([heads * dim, hk * dim, hk * dim], 1)
    q, k, v = q.unflatten(1, (heads, dim)), k.unflatten(1, (hk, dim)), v.unflatten(1, (hk, dim))
    ck, cv = (storage(layers, pages, ps, hk, dim, DT[dtype], layout) for _ in range(2))
    cache = vqv.PagedCache(ck, cv)
    seqs = vqv.Sequences(i32(start), i32(kv), i32(table), n_rows=n, max_rows=max(rows), max_kv=max(kv))
    rope = vqv.Rope(rot, base, inter, scaling, factor, 8192)
    out = vqv.vqv_rope_append(q, k, v, cache, seqs, rope, layer=layer)
    torch.cuda.synchronize()

    f, m = ref.rope_frequencies(rot, base, scaling, factor, 8192)
    wk = torch.full(ck.shape, SENTINEL, dtype=torch.float64)
    wv, wq = wk.clone(), torch.empty(n, heads, dim, dtype=torch.float64)
    big_k, big_q = torch.zeros_like(wk), torch.zeros_like(wq)
    for b, r, pos in ref.sequence_rows(start, kv):
        wq[r] = ref.rope_ref(q[r].cpu(), pos, f, m, rot, inter)
        big_q[r] = q[r].abs().max().item()
        p = table[b][pos // ps] if pos >= 0 else -1
        if 0 <= p < pages:
            wk[layer, p, pos % ps] = ref.rope_ref(k[r].cpu(), pos, f, m, rot, inter)
            big_k[layer, p, pos % ps] = k[r].abs().max().item()
            wv[layer, p, pos % ps] = v[r].double().cpu().to(DT[dtype]).double()
    # Half a step of the output's type, after 32-bit work: cosine and sine off by a rounded turn
    # (2^-26 turns, 2.4e-8 * 2 pi) and 2 steps, products and sum by 3 half steps, of values as
    # large as the row's largest twice.
    half = torch.finfo(DT[dtype]).eps / 2
    for got, want, big in ((out, wq, big_q), (ck, wk, big_k)):
        d32 = 2 * m * big * (2 ** -26 * 6.3 + 2 ** -22 + 3 * 2 ** -24)
        allow = half * (want.abs() + d32) + d32 + 2.0 ** -25
        err = (got.double().cpu() - want).abs()
        assert (err <= allow).all(), (err / allow).max()
    assert torch.equal(cv.double().cpu(), wv)


CASES = [
    dict(rows=[8], kv=[40], heads=4, hk=2, dim=128, ps=16, rot=128, inter=False),
    dict(rows=[1], kv=[1], heads=1, hk=1, dim=64, ps=1, rot=64, inter=True, into="bf16"),
    dict(rows=[3, 0, 5, 1], kv=[100003, 9, 5, 500001], heads=5, hk=1, dim=80, ps=20, rot=34, inter=False,
         scaling="yarn", into="fp16", dtype="fp16", layout="head"),
    dict(rows=[70, 2], kv=[90, 262144], heads=6, hk=3, dim=96, ps=24, rot=96, inter=True,
         scaling="smooth", layout="gap"),
    dict(rows=[2, 2], kv=[7, 300], heads=8, hk=8, dim=192, ps=8, rot=2, inter=False, scaling="ntk"),
    dict(rows=[17], kv=[20000], heads=2, hk=2, dim=256, ps=64, rot=254, inter=False,
         scaling="linear", layers=3, layer=2, into="bf16", dtype="fp16"),
    dict(rows=[9, 9], kv=[33, 34], heads=3, hk=1, dim=8, ps=4, rot=6, inter=True),
    dict(rows=[530, 1], kv=[530, 3], heads=2, hk=1, dim=64, ps=16, rot=48, inter=False, scaling="ntk"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['rows']}x{c['heads']}x{c['dim']}r{c['rot']}")
def test_matches_oracle(vqv, case):
    check(vqv, **case)


def test_bad_pages_and_short_lengths(vqv):
    """Rows on pages that the table does not hold, or before the first token,
    are turned but written nowhere."""
    check(vqv, rows=[8, 4, 6], kv=[40, 20, 4], heads=2, hk=2, dim=64, ps=4, rot=64, inter=False,
          bad=[(0, 8), (0, 9), (1, 4)])


def test_past_the_table(vqv):
    k = torch.full((1, 4, 4, 1, 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    cache = vqv.PagedCache(k, k.clone())
    x = torch.randn(4, 1, 64, device="cuda")
    seqs = vqv.Sequences(i32([0, 4]), i32([10]), i32([[2, 1]]), n_rows=4, max_rows=4, max_kv=10)
    vqv.vqv_rope_append(x, x, x, cache, seqs, vqv.Rope(64))
    torch.cuda.synchronize()
    for t in (cache.k, cache.v):
        assert (t[0, [0, 2, 3]] == SENTINEL).all()
        assert (t[0, 1, :2] == SENTINEL).all() and (t[0, 1, 2:] != SENTINEL).any()
    assert torch.equal(cache.v[0, 1, 2:], x[:2].to(torch.bfloat16))


def test_values_pass_unchanged(vqv):
    """Infinities and NaN past the turned part and in the values stay what and where they are."""
    x = torch.randn(1, 1, 64, device="cuda")
    x[0, 0, 40], x[0, 0, 63], x[0, 0, 50] = float("inf"), float("nan"), -0.0
    k = torch.zeros((1, 1, 4, 1, 64), dtype=torch.float16, device="cuda")
    cache = vqv.PagedCache(k, k.clone())
    seqs = vqv.Sequences(i32([0, 1]), i32([3]), i32([[0]]), n_rows=1, max_rows=1, max_kv=3)
    q = vqv.vqv_rope_append(x, x, x, cache, seqs, vqv.Rope(32, interleaved=True))
    torch.cuda.synchronize()
    want = x[0].half()
    assert torch.equal(q[0, :, 32:].view(torch.int16), want[:, 32:].view(torch.int16))
    assert torch.equal(cache.v[0, 0, 2].view(torch.int16), want.view(torch.int16))
    assert torch.isfinite(cache.k[0, 0, 2, :, :32]).all()


def test_other_stream_and_graph(vqv):
    """On a stream of its own, and replayed from a graph."""
    torch.manual_seed(3)
    n, heads, hk, dim = 6, 4, 2, 64
    qkv = torch.randn(n, heads + 2 * hk, dim, device="cuda")
    k = torch.zeros((1, 4, 8, hk, dim), dtype=torch.bfloat16, device="cuda")
    cache = vqv.PagedCache(k, torch.zeros_like(k))
    seqs = vqv.Sequences(i32([0, 2, 6]), i32([9, 7]), i32([[3, 1], [0, 2]]), n_rows=n, max_rows=4, max_kv=9)
    rope, out = vqv.Rope(64), torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        vqv.vqv_rope_append(qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:], cache,
                            seqs, rope, q_out=out, stream=stream)

    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, cache.k, cache.v)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        for t in (out, cache.k, cache.v):
            t.zero_()
        torch.cuda.synchronize()
        call(side) if rep == 0 else graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((out, cache.k, cache.v), want):
            assert torch.equal(got, w), rep


def test_refuses_wrong_tensors(vqv):
    k = torch.zeros((1, 4, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache = vqv.PagedCache(k, k.clone())
    seqs = vqv.Sequences(i32([0, 2]), i32([2]), i32([[0]]), n_rows=2, max_rows=2, max_kv=2)
    q, x, rope = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda"), vqv.Rope(64)
    for bad in ((q[:1], x, x), (q, x[:, :1], x), (q, x, x.half()), (q, x, x[..., ::2]), (q.double(), x, x)):
        with pytest.raises(ValueError):
            vqv.vqv_rope_append(*bad, cache, seqs, rope)
    with pytest.raises(ValueError):
        vqv.vqv_rope_append(q, x, x, cache, seqs, rope, q_out=torch.empty(2, 4, 64, device="cuda"))
    with pytest.raises(vqv.VqvError):
        vqv.vqv_rope_append(q, x, x, cache, seqs, vqv.Rope(128))
