"""The 4-bit paged cache: vqv_rope_append_q4, vqv_cache_q4_read and
vqv_paged_attn_q4 against the oracle in 64 bits."""

import pytest
import torch

from oracle import round_ref as ref
from oracle import serve_ref as q4

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NONE = 0xFF  # records of it have NaN scales and biases


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def device(x, layout):
    """Records [layers, pages, slots, heads, bytes] on the GPU, in memory as `layout` says."""
    if layout == "head":
        return x.transpose(2, 3).contiguous().cuda().transpose(2, 3)
    if layout == "gap":
        wide = torch.full((*x.shape[:2], x.shape[2] + 1, x.shape[3], x.shape[4] + 16), NONE, dtype=torch.uint8)
        wide[:, :, :x.shape[2], :, :x.shape[4]] = x
        return wide.cuda()[:, :, :x.shape[2], :, :x.shape[4]]
    return x.cuda()


# ---- append and read ----


def append(vqv, rows, kv, heads, hk, dim, ps, rot, inter, scaling="none", into="fp32", dtype="bf16", layout="slot",
           layers=1, layer=0, bad=(), seed=0, base=1e6, factor=8.0, change=None):
    """bad: (sequence, page index) entries of the table that hold no page; change: of the inputs."""
    torch.manual_seed(seed)
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    n, width = start[-1], max(-(-x // ps) for x in kv) + 1
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
    qkv = torch.randn(n, (heads + 2 * hk) * dim) * (1 + torch.arange((heads + 2 * hk) * dim) % 5)
    if change:
        change(qkv)
    qkv = qkv.to(DT[into])
    q, k, v = qkv.cuda().split([heads * dim, hk * dim, hk * dim], 1)
    q, k, v = q.unflatten(1, (heads, dim)), k.unflatten(1, (hk, dim)), v.unflatten(1, (hk, dim))
    size = q4.record_bytes(dim)
    ck, cv = (device(torch.full((layers, pages, ps, hk, size), NONE, dtype=torch.uint8), layout) for _ in range(2))
    cache = vqv.PagedCacheQ4(ck, cv, dim)
    seqs = vqv.Sequences(i32(start), i32(kv), i32(table), n_rows=n, max_rows=max(rows), max_kv=max(kv))
    rope = vqv.Rope(rot, base, inter, scaling, factor, 8192)
    out = vqv.vqv_rope_append_q4(q, k, v, cache, seqs, rope, layer=layer, q_dtype=DT[dtype])
    read = {t: vqv.vqv_cache_q4_read(cache, seqs, layer=layer, dtype=DT[t]) for t in DT}
    torch.cuda.synchronize()

    f, m = ref.rope_frequencies(rot, base, scaling, factor, 8192)
    turned_k, wq = torch.zeros(n, hk, dim, dtype=torch.float64), torch.zeros(n, heads, dim, dtype=torch.float64)
    big, place = torch.zeros(n, 1, 1, dtype=torch.float64), {}
    for b, r, pos in ref.sequence_rows(start, kv):
        wq[r] = ref.rope_ref(q[r].cpu(), pos, f, m, rot, inter)
        turned_k[r] = ref.rope_ref(k[r].cpu(), pos, f, m, rot, inter)
        big[r] = q[r].float().nan_to_num(0, 0, 0).abs().max().item()
        p = table[b][pos // ps] if pos >= 0 else -1
        if 0 <= p < pages:
            place[r] = (p, pos % ps)
    # Queries: as tests of vqv_rope_append derive it, 32-bit work and half a step of the output.
    half = torch.finfo(DT[dtype]).eps / 2
    d32 = 2 * m * big * (2 ** -26 * 6.3 + 2 ** -22 + 3 * 2 ** -24)
    ok = wq.isfinite()
    allow = half * (wq.abs() + d32) + d32 + 2.0 ** -25
    err = torch.where(ok, (out.double().cpu() - wq).abs(), 0.0)
    assert (err <= allow).all(), (err / allow).max()
    # Records: of the keys rounded once to fp32, and of the values; everything else untouched.
    want_k, want_v = (torch.full((layers, pages, ps, hk, size), NONE, dtype=torch.uint8) for _ in range(2))
    rk, rv = q4.pack(turned_k.float()), q4.pack(v.cpu().float())
    for r, (p, s) in place.items():
        want_k[layer, p, s], want_v[layer, p, s] = rk[r], rv[r]
    assert torch.equal(cv.cpu(), want_v)
    # mscale reaches the kernel in fp32 and the oracle in 64 bits: under YaRN a key's last bit, and
    # so a code next to a border, may differ; elsewhere all bytes are equal.
    if m == 1.0:
        assert torch.equal(ck.cpu(), want_k)
    else:
        a, c = q4.unpack(ck.cpu(), dim), q4.unpack(want_k, dim)
        step = torch.stack([g.amax(-1) - g.amin(-1) for g in c.split(32, -1)], -1).amax(-1, keepdim=True) / 15
        assert (a.isnan() == c.isnan()).all() and ((a - c).abs().nan_to_num(0) <= 1.01 * step.nan_to_num(0) + 1e-6).all()
        assert ((a - c).abs().nan_to_num(0) > 1e-3 * step.nan_to_num(0)).double().mean() < 1e-4
    # What is read back: values in fp32, rounded once more; zeros for rows on no page.
    stored = {"k": ck.cpu(), "v": cv.cpu()}
    for t, (gk, gv) in read.items():
        for got, name in ((gk, "k"), (gv, "v")):
            want = torch.zeros(n, hk, dim, dtype=torch.float64)
            for r, (p, s) in place.items():
                want[r] = q4.unpack(stored[name][layer, p, s], dim)
            held = torch.tensor([r in place or any(start[b] <= r < start[b + 1] for b in range(len(rows))) for r in range(n)])
            g, w = got.double().cpu()[held], want[held].float().to(DT[t]).double()
            assert torch.equal(g.nan_to_num(1e9), w.nan_to_num(1e9)), t
    return cache, table, place


CASES = [
    dict(rows=[8], kv=[40], heads=4, hk=2, dim=128, ps=16, rot=128, inter=False),
    dict(rows=[1], kv=[1], heads=1, hk=1, dim=64, ps=1, rot=64, inter=True, into="bf16"),
    dict(rows=[3, 0, 5, 1], kv=[100003, 9, 5, 500001], heads=5, hk=1, dim=80, ps=20, rot=34, inter=False,
         scaling="yarn", into="fp16", dtype="fp16", layout="head"),
    dict(rows=[70, 2], kv=[90, 262144], heads=6, hk=3, dim=96, ps=24, rot=96, inter=True, scaling="smooth", layout="gap"),
    dict(rows=[2, 2], kv=[7, 300], heads=8, hk=8, dim=192, ps=8, rot=2, inter=False, scaling="ntk"),
    dict(rows=[17], kv=[20000], heads=2, hk=2, dim=256, ps=64, rot=254, inter=False, scaling="linear", layers=3,
         layer=2, into="bf16", dtype="fp16"),
    dict(rows=[9, 9], kv=[33, 34], heads=3, hk=1, dim=80, ps=4, rot=6, inter=True),
    dict(rows=[530, 1], kv=[530, 3], heads=2, hk=1, dim=64, ps=16, rot=48, inter=False, scaling="ntk"),
    dict(rows=[4, 3], kv=[2, 10], heads=2, hk=1, dim=64, ps=16, rot=64, inter=False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['rows']}x{c['heads']}x{c['dim']}r{c['rot']}")
def test_append(vqv, case):
    append(vqv, **case)


def test_append_bad_pages(vqv):
    append(vqv, rows=[40, 20], kv=[100, 20], heads=4, hk=2, dim=128, ps=8, rot=64, inter=False, bad=[(0, 9), (0, 12), (1, 0)])


@pytest.mark.parametrize("dim", [64, 80, 128])
def test_append_extremes(vqv, dim):
    """NaN, infinities, values past the cut, groups of one value, of zeros and of the smallest values."""
    def change(x):
        c = x[:, 2 * dim:]                    # k and v, one head each
        c[0, 5], c[0, dim + 7] = float("nan"), float("nan")
        c[1, 3], c[1, dim + 3] = float("inf"), -float("inf")
        c[2, 1], c[2, 2], c[2, dim + 1] = 1e20, -1e20, 70000.0
        c[3], c[4] = 2.5, 0.0
        c[5] *= 1e-7
        c[6] *= 1e-30
        c[7] = 100 + 1e-3 * c[7]
    for inter in (False, True):
        append(vqv, rows=[9], kv=[9], heads=2, hk=1, dim=dim, ps=16, rot=2, inter=inter, change=change)


def test_records_move_as_bytes(vqv):
    """Copy, fork and compact over `records`: what they do to a 16-bit cache, done to records."""
    cache, table, place = append(vqv, rows=[8, 8], kv=[30, 20], heads=2, hk=2, dim=80, ps=8, rot=64, inter=False, layers=2)
    before = cache.k.cpu().clone()
    src, dst = place[0][0], [p for p in range(cache.pages) if p not in {x[0] for x in place.values()}][0]
    vqv.vqv_cache_copy(cache.records, i32([src]), i32([dst]))
    before[:, dst] = before[:, src]
    assert torch.equal(cache.k.cpu(), before)
    keep = [1, 0, 1, 1, 0, 0, 1, 0] + [1] * 8
    seqs = vqv.Sequences(i32([0, 8, 16]), i32([30, 20]), i32(table), n_rows=16, max_rows=8, max_kv=30)
    assert vqv.vqv_cache_compact(cache.records, seqs, i32(keep)).tolist() == [26, 20]
    at = [place[r] for r in range(8)]
    for to, of in enumerate([0, 2, 3, 6]):
        before[0, at[to][0], at[to][1]] = before[0, at[of][0], at[of][1]]
    assert torch.equal(cache.k.cpu()[0], before[0])


def test_read_one_of_both_and_rows_of_nobody(vqv):
    cache, table, _ = append(vqv, rows=[4], kv=[10], heads=2, hk=1, dim=64, ps=16, rot=64, inter=False)
    seqs = vqv.Sequences(i32([0, 4]), i32([10]), i32(table), n_rows=6, max_rows=4, max_kv=10)
    k, v = vqv.vqv_cache_q4_read(cache, seqs, k_out=torch.full((6, 1, 64), 3.0, device="cuda"))
    assert (k[4:] == 3.0).all() and not (k[:4] == 3.0).any()
    other = torch.full((6, 1, 64), 3.0, device="cuda")
    vqv.vqv_cache_q4_read(cache, seqs, k_out=other, v_out=v)
    assert torch.equal(other, k)


# ---- attention ----


class Case:
    """Inputs on the GPU. Every slot that no token stands in holds NaN, in K and V."""

    def __init__(self, rows, kv, heads, hk, dim, ps, dtype="bf16", layout="slot", seed=0, layers=1, layer=0,
                 max_rows=None, max_kv=None):
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.kv, self.ps, self.hk, self.dim = rows, kv, ps, hk, dim
        self.heads, self.t, self.layer, self.layout = heads, DT[dtype], layer, layout
        self.start = [0]
        for r in rows:
            self.start.append(self.start[-1] + r)
        self.n = self.start[-1]
        held = [-(-x // ps) for x in kv]
        self.pages = sum(held) + 3
        perm = torch.randperm(self.pages, generator=gen).tolist()
        self.table = [[-1] * (max(held) + 1) for _ in rows]
        for b, x in enumerate(held):
            for j in range(x):
                self.table[b][j] = perm.pop()
        # Values as the cache holds them, by token: set() writes them.
        shape = (layers, self.pages, ps, hk, q4.record_bytes(dim))
        self.rk = torch.full(shape, NONE, dtype=torch.uint8)
        self.rv = self.rk.clone()
        offset = torch.randn(hk, dim, generator=gen)
        for b, x in enumerate(kv):
            self.set(b, 0, torch.randn(x, hk, dim, generator=gen) + offset, torch.randn(x, hk, dim, generator=gen))
        self.q = (1.5 * torch.randn(self.n, heads, dim, generator=gen)).to(self.t)
        self.max_rows = max(rows) if max_rows is None else max_rows
        self.max_kv = max(kv) if max_kv is None else max_kv
        self.scale = dim ** -0.5

    def set(self, b, t, k=None, v=None):
        """Keys and values [tokens, hk, dim] of sequence b from token t on."""
        n = (k if k is not None else v).shape[0]
        at = torch.arange(t, t + n)
        page, slot = torch.tensor(self.table[b])[at // self.ps], at % self.ps
        for rec, x in ((self.rk, k), (self.rv, v)):
            if x is not None:
                rec[self.layer, page, slot] = q4.pack(x)

    def run(self, vqv, window=0, sinks=0, stream=None, scale=None):
        self.cache = vqv.PagedCacheQ4(device(self.rk, self.layout), device(self.rv, self.layout), self.dim)
        self.seqs = vqv.Sequences(i32(self.start), i32(self.kv), i32(self.table), n_rows=self.n,
                                  max_rows=self.max_rows, max_kv=self.max_kv)
        out = torch.full(self.q.shape, 9.0, dtype=self.t, device="cuda")
        self.qd = self.q.cuda()
        vqv.vqv_paged_attn_q4(self.qd, self.cache, self.seqs, scale=scale or self.scale, window=window, sinks=sinks,
                              layer=self.layer, out=out, stream=stream)
        torch.cuda.synchronize()
        return out.cpu()

    def want(self, window=0, sinks=0, scale=None, rounded=True):
        """In 64 bits, over the values as they enter the products (one rounding to fp16, but for the
        keys of fp16 queries, which enter in two values), or exact ones."""
        k, v = (q4.unpack(x[self.layer], self.dim) for x in (self.rk, self.rv))
        if rounded:
            k, v = k.half().double() if self.t == torch.bfloat16 else k, v.half().double()
        return ref.attn_ref(self.q, k, v, self.start, self.kv, self.table, scale or self.scale, window, sinks)

    def allowance(self, want, values=0.0, low=0.0, terms=None):
        """Half a step of the output, after: a score's error, which moves its weight by as much,
        relatively (`terms` products and sums in fp32 of sizes up to `size`, one scaling, one
        subtraction, an exponential of 2^-22), for the weight and for the sum of weights; keys in two
        values (2^-22) of fp16 queries; a bf16 query 2^24 below its row's largest is off by up to 2^-35 of that; weights in two fp16
        values (2^-22) for fp16 outputs of up to 64 pairs, else in one (2^-11); below 2^-29 of the largest they are
        off by 2^-40 of it, of which `low` is the sum of |v|; sums over tokens in fp32. `values`
        is the relative rounding of keys and values where it is not in `want`."""
        out, mean, size = want
        pairs = min(self.max_rows, self.n) * (self.heads // self.hk)
        weight = 2.0 ** -22 if pairs <= 64 and self.t == torch.float16 else 2.0 ** -11
        terms = self.dim if terms is None else terms
        keys = 2.0 ** -22 if self.t == torch.float16 else 0.0
        score = size * ((terms + 8) * 2.0 ** -24 + values + keys) + 2.0 ** -22
        inner = (weight + values + 2 * score + (max(self.kv) + 8) * 2.0 ** -24) * mean + 2.0 ** -40 * low
        half = torch.finfo(self.t).eps / 2
        return half * (out.abs() + inner) + inner + 2.0 ** -25

    def close(self, got, want, **kw):
        allow, err = self.allowance(want, **kw), (got.double() - want[0]).abs()
        assert (err <= allow).all(), f"error over allowance {(err / allow).nan_to_num(1e9).max():.3g}"


ATTN = [
    dict(rows=[1], kv=[1], heads=1, hk=1, dim=64, ps=1),
    dict(rows=[8], kv=[300], heads=8, hk=2, dim=128, ps=16),
    dict(rows=[1] * 5, kv=[1, 16, 129, 700, 64], heads=8, hk=2, dim=128, ps=16),
    dict(rows=[3, 0, 1], kv=[40, 9, 33], heads=6, hk=2, dim=64, ps=20, dtype="fp16", layout="head"),
    dict(rows=[16, 5], kv=[400, 37], heads=8, hk=2, dim=256, ps=32, dtype="fp16"),
    dict(rows=[16, 16], kv=[16, 200], heads=12, hk=3, dim=96, ps=24, layout="gap"),
    dict(rows=[70, 33], kv=[70, 401], heads=10, hk=2, dim=80, ps=8, layout="head"),
    dict(rows=[130], kv=[333], heads=4, hk=4, dim=192, ps=64, dtype="fp16", layout="head"),
    dict(rows=[65], kv=[257], heads=21, hk=3, dim=128, ps=128),
    dict(rows=[100], kv=[164], heads=8, hk=1, dim=64, ps=1),
    dict(rows=[40, 90], kv=[45, 91], heads=6, hk=2, dim=256, ps=16),
    dict(rows=[9], kv=[77], heads=16, hk=2, dim=192, ps=20, layers=3, layer=1),
    dict(rows=[12], kv=[90], heads=2, hk=1, dim=80, ps=16, dtype="fp16"),
    dict(rows=[1, 1], kv=[2100, 5], heads=40, hk=1, dim=128, ps=64, layout="head"),
    dict(rows=[2], kv=[1500], heads=2, hk=1, dim=96, ps=16),
    dict(rows=[30], kv=[500], heads=4, hk=2, dim=64, ps=16),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{c['rows']}kv{c['kv']}h{c['heads']}/{c['hk']}d{c['dim']}p{c['ps']}")
def test_attention(vqv, case):
    c = Case(**case)
    got = c.run(vqv)
    c.close(got, c.want())
    c.close(got, c.want(rounded=False), values=2.0 ** -11)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (37, 0), (64, 4), (100, 150), (5000, 2)])
@pytest.mark.parametrize("index", [1, 2, 5, 6, 8, 10])
def test_windows(vqv, index, window, sinks):
    c = Case(**ATTN[index])
    c.close(c.run(vqv, window, sinks), c.want(window, sinks))


# Rows of a case (two heads to a key head) that take one tile of 32 (row, head) pairs, two, and
# several work-groups' worth.
ROWS = [3, 20, 50, 90]


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 80, 96, 128, 192, 256])
def test_many_blocks_of_one_work_group(vqv, dim, dtype, rows, window, sinks):
    """A max_kv that plans one split: every wave walks over 10 blocks and more, past what it looks
    up ahead; odd pages, some of them none, NaN in every slot without a token."""
    c = Case(rows=[rows, 2], kv=[1501, 1290], heads=4, hk=2, dim=dim, ps=20, dtype=dtype,
             layout="head" if dim % 64 else "slot", seed=dim + rows, max_kv=64)
    c.table[0][70], c.table[0][31], c.table[1][50], c.table[1][3] = -1, c.pages, 1 << 30, -7
    c.close(c.run(vqv, window, sinks), c.want(window, sinks), low=5.0 * 1501)


@pytest.mark.parametrize("rows,dim,dtype", [(1, 128, "bf16"), (8, 256, "fp16"), (200, 64, "bf16"), (130, 128, "fp16")])
def test_long_sequences(vqv, rows, dim, dtype):
    """Tens of thousands of tokens in many splits, the last one short."""
    c = Case(rows=[rows], kv=[24001], heads=2, hk=1, dim=dim, ps=64, dtype=dtype, seed=rows)
    c.close(c.run(vqv), c.want(), low=5.0 * 24001)
    c.close(c.run(vqv, 9000, 100), c.want(9000, 100), low=5.0 * 24001)


def test_large_and_small_scores(vqv):
    """Scores far apart, where one weight takes nearly all; queries of the type's extremes."""
    for rows in ([8, 1], [80, 3]):
        c = Case(rows=rows, kv=[600, 900], heads=4, hk=2, dim=64, ps=16, seed=5)
        plain = c.q.clone()
        c.q = plain * 12
        c.close(c.run(vqv, scale=1.0), c.want(scale=1.0))
        for size in (1e-30, 1e-38, 1e15):
            c.q = (plain.float() * size).to(c.t)
            c.close(c.run(vqv, scale=0.125 / size if size > 1e-35 else 1.0),
                    c.want(scale=0.125 / size if size > 1e-35 else 1.0))
        c.q = plain
        c.q[0] = 0
        c.q[1, 0, 3:] = 0
        c.q[2, :, 0] = 1e6          # beside it the others of the row are small
        c.close(c.run(vqv, scale=1e-6), c.want(scale=1e-6))


def test_scores_past_any_exponent(vqv):
    """One token takes all, and the output is its values."""
    for rows, dim in ((2, 64), (20, 128), (50, 192), (100, 64)):
        for size in (1e6, 1e10, 1e20, 1e30):
            c = Case(rows=[rows], kv=[700], heads=2, hk=1, dim=dim, ps=16, max_kv=64)
            c.q = torch.full_like(c.q, size)
            k = torch.zeros(700, 1, dim)
            k[:, 0] = torch.arange(700.0)[:, None] % 650
            c.set(0, 0, k)
            got, want = c.run(vqv, scale=1.0), c.want(scale=1.0)
            assert torch.equal(got, want[0].to(c.t))


def test_bad_pages_are_hidden(vqv):
    for rows, heads in (([4, 6], 4), ([70, 40], 4)):
        c = Case(rows=rows, kv=[160, 90], heads=heads, hk=2, dim=64, ps=16)
        c.table[0][1], c.table[0][4], c.table[1][0] = -1, c.pages, 1 << 30
        c.close(c.run(vqv), c.want())
        for j in range(len(c.table[1])):
            c.table[1][j] = -1
        got = c.run(vqv)
        c.close(got, c.want())
        assert (got[rows[0]:] == 0).all()


def test_past_the_table_and_lengths(vqv):
    """kv_len past the table's width, shorter than the rows, zero."""
    c = Case(rows=[3, 5, 2], kv=[64, 40, 20], heads=2, hk=1, dim=64, ps=16)
    c.kv, c.max_kv = [100, 3, 0], 100
    got = c.run(vqv)
    c.close(got, c.want())
    assert (got[3:5] == 0).all() and (got[8:] == 0).all()


@pytest.mark.parametrize("rows", [2, 150])
def test_lengths_past_any_table(vqv, rows):
    """A kv_len near 2^31: the tokens that the table holds are seen by all rows."""
    c = Case(rows=[rows], kv=[64], heads=2, hk=1, dim=64, ps=16)
    k, v = (q4.unpack(x[0], 64).half().double() for x in (c.rk, c.rv))
    table = c.table[0][:4]
    want = ref.attn_ref(c.q, k, v, list(range(rows + 1)), [64] * rows, [table] * rows, c.scale)
    c.kv, c.table = [2 ** 31 - 1], [table]
    got = c.run(vqv)
    c.kv = [64]
    c.close(got, want)


def test_longer_than_planned(vqv):
    """A max_kv below the real lengths costs speed, not results."""
    for rows in ([2, 1], [80, 3]):
        c = Case(rows=rows, kv=[900, 500], heads=4, hk=2, dim=128, ps=16, max_kv=150)
        c.close(c.run(vqv), c.want())


def test_rows_without_a_sequence(vqv):
    """Rows past max_rows and past the last sequence are not written."""
    for rows, most in (([6], 4), ([90], 70)):
        c = Case(rows=rows, kv=[150], heads=2, hk=1, dim=64, ps=16, max_rows=most)
        got, want = c.run(vqv), c.want()
        assert (got[most:] == 9.0).all()
        c.n = most
        c.close(got[:most], tuple(x[:most] for x in want))


def test_hidden_nan(vqv):
    """Tokens that a row does not see may hold anything."""
    nan = float("nan")
    for rows, dtype, dim in (([12], "bf16", 64), ([12], "fp16", 256), ([30], "bf16", 128), ([150], "bf16", 128)):
        c = Case(rows=rows, kv=[200], heads=4, hk=1, dim=dim, ps=16, dtype=dtype)
        n = rows[0]
        clean = c.run(vqv, 40, 2)
        for t in (199, 200 - n // 2, 20, 21):
            c.set(0, t, torch.full((1, 1, dim), nan), torch.full((1, 1, dim), nan))
        got = c.run(vqv, 40, 2)
        rows_ok = [r for r in range(n // 2) if 200 - n + r - 40 >= 21]
        assert rows_ok and torch.equal(got[rows_ok], clean[rows_ok])
        assert got[-1].isnan().all()


def test_seen_nan(vqv):
    """A NaN that is seen comes out: of a key everywhere, of values in their group."""
    for rows, dim in ((2, 64), (20, 128), (50, 192), (100, 96)):
        c = Case(rows=[rows], kv=[400], heads=2, hk=1, dim=dim, ps=16)
        clean = c.run(vqv)
        keep = c.rk.clone()
        x = torch.randn(1, 1, dim)
        x[0, 0, 5] = float("nan")
        c.set(0, 17, k=x)
        assert c.run(vqv).isnan().all()
        c.rk = keep
        v = q4.unpack(c.rv[0, c.table[0][1], 1], dim).float()[None]
        v[0, 0, 40] = float("nan")
        c.set(0, 17, v=v)
        got = c.run(vqv)
        assert got[:, :, 32:64].isnan().all()
        rest = [i for i in range(dim) if not 32 <= i < 64]
        assert got[:, :, rest].isfinite().all()
        # re-packing the other groups changes the token's values by rounding only
        assert (got[:, :, rest].float() - clean[:, :, rest].float()).abs().max() < 0.1


def test_deterministic_on_streams_and_graphs(vqv):
    c = Case(rows=[8, 2], kv=[1700, 90], heads=8, hk=2, dim=128, ps=16)
    want = c.run(vqv)
    assert torch.equal(c.run(vqv, stream=torch.cuda.Stream()), want)
    out = torch.empty(c.q.shape, dtype=c.t, device="cuda")
    need = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=c.scale, out=out, workspace=ws)
    for _ in range(4):
        out.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


def test_far_offsets(vqv):
    """Pages whose place passes 2^32 bytes."""
    ps, hk, dim, pages = 64, 8, 256, 60000        # 60000 pages of 81920 bytes: 4.9e9
    k = torch.empty((1, pages, ps, hk, 160), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ids = [pages - 1, 5, pages - 2]
    c = Case(rows=[2], kv=[150], heads=hk, hk=hk, dim=dim, ps=ps)
    small = c.table[0][:3]
    for x, s in ((k, c.rk), (v, c.rv)):
        x[0, ids] = s[0, small].cuda()
    seqs = vqv.Sequences(i32([0, 2]), i32([150]), i32([ids]), n_rows=2, max_rows=2, max_kv=150)
    cache = vqv.PagedCacheQ4(k, v, dim)
    c.close(vqv.vqv_paged_attn_q4(c.q.cuda(), cache, seqs, scale=c.scale).cpu(), c.want())
    got, _ = vqv.vqv_cache_q4_read(cache, seqs)
    at = torch.tensor([148, 149])
    page = torch.tensor(small)[at // ps]
    assert torch.equal(got.cpu().double(), q4.unpack(c.rk[0, page, at % ps], dim).float().double())


def test_no_rows(vqv):
    c = Case(rows=[2, 1], kv=[20, 7], heads=4, hk=2, dim=64, ps=16)
    c.run(vqv)
    seqs = vqv.Sequences(i32([0, 0, 0]), i32([20, 7]), i32(c.table), n_rows=0, max_rows=0, max_kv=20)
    before = [c.cache.k.clone(), c.cache.v.clone()]
    q, k = (torch.empty(0, h, 64, dtype=c.t, device="cuda") for h in (4, 2))
    assert vqv.vqv_paged_attn_q4(q, c.cache, seqs, scale=1.0).shape == (0, 4, 64)
    assert vqv.vqv_rope_append_q4(q, k, k, c.cache, seqs, vqv.Rope(64)).shape == (0, 4, 64)
    assert vqv.vqv_cache_q4_read(c.cache, seqs)[0].shape == (0, 2, 64)
    assert all(torch.equal(x, y) for x, y in zip((c.cache.k, c.cache.v), before))


def test_refuses_wrong_tensors(vqv):
    c = Case(rows=[2], kv=[10], heads=2, hk=1, dim=64, ps=16)
    c.run(vqv)
    for q in (c.qd[:1], c.qd.float(), c.qd[:, :, ::2], c.qd[:, 0], c.q):
        with pytest.raises(ValueError):
            vqv.vqv_paged_attn_q4(q, c.cache, c.seqs, scale=1.0)
    with pytest.raises(ValueError):
        vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=1.0, out=torch.empty(2, 2, 64, device="cuda"))
    with pytest.raises(vqv.VqvError):
        vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=0.0)
    k = c.cache.k
    for args in ((k, k, 72), (k, k, 128), (k[:, :, :, :, ::2], k[:, :, :, :, ::2], 64), (k.view(torch.int8), k, 64),
                 (k.cpu(), k.cpu(), 64), (k[0], k[0], 64)):
        with pytest.raises(ValueError):
            vqv.PagedCacheQ4(*args)
    rope = vqv.Rope(64)
    kv = torch.zeros(2, 1, 64, device="cuda", dtype=c.t)
    with pytest.raises(ValueError):
        vqv.vqv_rope_append_q4(c.qd, kv, kv, c.cache, c.seqs, rope, q_dtype=torch.float32)
    with pytest.raises(ValueError):
        vqv.vqv_rope_append_q4(c.qd, kv[:1], kv, c.cache, c.seqs, rope)
    with pytest.raises(ValueError):
        vqv.vqv_cache_q4_read(c.cache, c.seqs, k_out=torch.empty(2, 1, 32, device="cuda"))


# ---- many rows of bf16: read through a 16-bit copy in the workspace ----


def planned(rows, heads, **kw):
    """A case whose max_kv, far above the real lengths, makes the call large enough for the copy."""
    return Case(rows=rows, heads=heads, max_kv=2 ** 27 // (max(rows) * heads) + 1, **kw)


def copies(c, vqv):
    need = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads)
    return need >= 2 * max(c.kv) * c.hk * c.dim * 2 + c.n * c.heads * c.dim * 4


COPIED = [
    dict(rows=[200], kv=[300], heads=8, hk=2, dim=128, ps=16),
    dict(rows=[129], kv=[129], heads=4, hk=1, dim=64, ps=1, layout="head"),
    dict(rows=[260], kv=[411], heads=6, hk=3, dim=80, ps=20, layout="gap"),
    dict(rows=[171], kv=[800], heads=12, hk=4, dim=96, ps=24),
    dict(rows=[512], kv=[600], heads=2, hk=2, dim=192, ps=64, layers=3, layer=1),
    dict(rows=[150], kv=[1201], heads=8, hk=2, dim=256, ps=1000),
    # 512 pairs and more, fewer, none, just as many
    dict(rows=[130, 3, 0, 128, 1, 127], kv=[400, 90, 5, 128, 700, 130], heads=8, hk=2, dim=128, ps=16),
    dict(rows=[1, 2, 1], kv=[70, 300, 9], heads=600, hk=1, dim=64, ps=8),   # rows of 600 pairs
    dict(rows=[1, 0, 0, 1, 0], kv=[40, 5, 0, 33, 2], heads=1024, hk=1, dim=96, ps=16),
    dict(rows=[0, 1, 0, 0], kv=[7, 40, 3, 33], heads=600, hk=1, dim=128, ps=16),
]


@pytest.mark.parametrize("case", COPIED, ids=lambda c: f"{c['rows']}kv{c['kv']}h{c['heads']}/{c['hk']}d{c['dim']}p{c['ps']}")
def test_copied_attention(vqv, case):
    c = planned(**case)
    c.close(c.run(vqv), c.want())
    assert copies(c, vqv)
    c.close(c.run(vqv, 100, 7), c.want(100, 7))


def test_copied_or_longer_than_planned(vqv):
    """Of one call: sequences that fit the copy, one that is longer, one of few rows; then pages that
    are not there."""
    c = Case(rows=[700, 640, 5, 700], kv=[3000, 12100, 800, 700], heads=16, hk=2, dim=64, ps=16, max_kv=12000)
    c.close(c.run(vqv), c.want(), low=5.0 * 12100)
    assert copies(c, vqv)
    c.table[0][3], c.table[0][4], c.table[1][0], c.table[3][18] = -1, c.pages, 1 << 30, -9
    c.close(c.run(vqv), c.want(), low=5.0 * 12100)
    c.table[3] = [-1] * len(c.table[3])
    got = c.run(vqv)
    c.close(got, c.want(), low=5.0 * 12100)
    assert (got[1345:] == 0).all()


def test_copied_lengths(vqv):
    """kv_len below the rows, zero, past the table; rows past max_rows."""
    c = planned(rows=[300, 290, 280], kv=[640, 300, 290], heads=4, hk=2, dim=64, ps=16)
    c.kv = [700, 3, 0]
    got = c.run(vqv)
    c.close(got, c.want())
    assert (got[300:587] == 0).all() and (got[590:] == 0).all()
    c = Case(rows=[400], kv=[450], heads=4, hk=2, dim=64, ps=16, max_rows=270, max_kv=2 ** 17)
    got, want = c.run(vqv), c.want()
    assert (got[270:] == 9.0).all()
    c.n = 270
    c.close(got[:270], tuple(x[:270] for x in want))


def test_copied_nan(vqv):
    """Hidden tokens may hold anything, a NaN that is seen comes out."""
    nan = float("nan")
    for dim in (128, 192):
        c = planned(rows=[300], kv=[700], heads=4, hk=2, dim=dim, ps=16)
        clean = c.run(vqv)
        for t in (699, 550):
            c.set(0, t, torch.full((1, 2, dim), nan), torch.full((1, 2, dim), nan))
        got = c.run(vqv)
        assert torch.equal(got[:150], clean[:150]) and got[150:].isnan().all()
        c = planned(rows=[300], kv=[700], heads=4, hk=2, dim=dim, ps=16)
        v = q4.unpack(c.rv[0, c.table[0][0], 5], dim).float()[None]
        v[0, 0, 40] = nan           # of one group of one head
        c.set(0, 5, v=v)
        got = c.run(vqv)
        assert got[:, :2, 32:64].isnan().all()
        assert got[:, 2:].isfinite().all() and got[:, :2, :32].isfinite().all() and got[:, :2, 64:].isfinite().all()


def test_copied_scores_of_any_size(vqv):
    for dim in (128, 192):
        c = planned(rows=[300], kv=[500], heads=4, hk=2, dim=dim, ps=16, seed=5)
        plain = c.q.clone()
        for size in (12.0, 1e-30, 1e-38, 1e15):
            c.q = (plain.float() * size).to(c.t)
            scale = 1.0 if size == 12.0 or size < 1e-35 else 0.125 / size
            c.close(c.run(vqv, scale=scale), c.want(scale=scale))
        c.q = plain
        c.q[0] = 0
        c.q[1, 0, 3:] = 0
        c.q[2, :, 0] = 1e6          # beside it the others of the row are small
        c.close(c.run(vqv, scale=1e-6), c.want(scale=1e-6))
        for size in (1e6, 1e30):    # one token takes all
            c.q = torch.full_like(c.q, size)
            k = torch.zeros(500, 2, dim)
            k[:] = torch.arange(500.0)[:, None, None] % 450
            c.set(0, 0, k)
            assert torch.equal(c.run(vqv, scale=1.0), c.want(scale=1.0)[0].to(c.t))


def test_copied_on_streams_and_in_graphs(vqv):
    """Two graphs that share one workspace, replayed in turn; nothing is taken from the workspace."""
    c = planned(rows=[300, 6], kv=[500, 1700], heads=4, hk=2, dim=128, ps=16)
    want = c.run(vqv)
    assert copies(c, vqv)
    assert torch.equal(c.run(vqv, stream=torch.cuda.Stream()), want)
    need = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    window = c.run(vqv, 90, 3)
    outs, graphs = [], []
    for args in ({}, dict(window=90, sinks=3)):
        out = torch.empty(c.q.shape, dtype=c.t, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=c.scale, out=out, workspace=ws, **args)
        outs.append(out)
        graphs.append(graph)
    for i in range(4):
        for out in outs:
            out.zero_()
        ws.fill_(255 if i % 2 else 0)
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0].cpu(), want) and torch.equal(outs[1].cpu(), window)


def test_copied_workspace(vqv):
    """A call needs the whole workspace; fp16 takes no copy and less."""
    c = planned(rows=[300], kv=[500], heads=4, hk=2, dim=128, ps=16)
    c.run(vqv)
    need = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads)
    out = torch.empty(c.q.shape, dtype=c.t, device="cuda")
    with pytest.raises(Exception, match="(?i)workspace"):
        vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=c.scale, out=out,
                              workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    h = planned(rows=[300], kv=[500], heads=4, hk=2, dim=128, ps=16, dtype="fp16")
    h.close(h.run(vqv), h.want())


@pytest.mark.parametrize("rows,most", [(3, 64), (3, 4000), (50, 64), (300, 2 ** 18)])
@pytest.mark.parametrize("size,scale", [(1e-38, 1e-6), (1e-30, 1e-30), (1e30, 1e30), (1.0, 3.4e38), (1.0, 1e-45)])
def test_scales_of_any_size(vqv, rows, most, size, scale):
    """All weights of a row the same, or one token that takes all: for rows of several tiles, splits and the copy."""
    c = Case(rows=[rows], kv=[500], heads=4, hk=2, dim=64, ps=16, seed=9, max_kv=most)
    c.q = (c.q.float() * size).to(c.t)
    if size * scale > 1:
        c.q = c.q.abs() + size            # the largest sum of keys takes all
        k = torch.randn(500, 2, 1).expand(500, 2, 64) * torch.arange(500)[:, None, None] / 500
        c.set(0, 0, k.contiguous())
        c.q[:] = c.q[:, :, :1]
    got, want = c.run(vqv, scale=scale), c.want(scale=scale)
    c.close(got, want)
    assert size * scale <= 1 or torch.equal(got, want[0].to(c.t))


@pytest.mark.parametrize("case", [
    dict(rows=[300, 260, 280], kv=[300, 700, 900], heads=4),             # 512 pairs and more each: the first fit
    dict(rows=[4, 300, 1, 3, 270, 2, 290], kv=[90, 300, 33, 80, 700, 9, 500], heads=4),
    dict(rows=[140, 1, 300], kv=[200, 40, 420], heads=8)])
@pytest.mark.parametrize("width", [2 ** 20, 45000])
def test_copies_that_do_not_fit(vqv, case, width):
    """Tables of so many pages that the copy holds one or two of the sequences: the others are read
    from the records, in the same call."""
    c = planned(**case, hk=2, dim=64, ps=16)
    c.max_kv = 16 * width
    c.table = [row + [-1] * (width - len(row)) for row in c.table]
    want = c.want()
    c.close(c.run(vqv), want)
    need = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads)
    assert 2 ** 30 <= need < 2 ** 30 + 2 ** 28
    c.table[-1] = [-1] * width
    got = c.run(vqv)
    assert (got[c.start[-2]:] == 0).all()
    c.close(got, c.want())


def test_workspace_of_fp16_calls(vqv):
    """fp16 calls need less than bf16 ones where those copy, and no less than they say."""
    for rows, kv, most in ([300, 9], [500, 1400], 2 ** 17), ([8], [3000], 3000):
        c = Case(rows=rows, kv=kv, heads=4, hk=2, dim=128, ps=16, dtype="fp16", max_kv=most)
        want = c.run(vqv)
        c.close(want, c.want())
        need = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads, dtype=torch.float16)
        both = vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads)
        assert need == both if max(rows) < 256 else need < both
        assert vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads, dtype=torch.bfloat16) == both
        with pytest.raises(ValueError):
            vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads, dtype=torch.float32)
        out = torch.empty(c.q.shape, dtype=c.t, device="cuda")
        ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
        vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=c.scale, out=out, workspace=ws[:need])
        assert torch.equal(out.cpu(), want) and (ws[need:] == 255).all()
        if need:
            with pytest.raises(vqv.VqvError, match="(?i)workspace"):
                vqv.vqv_paged_attn_q4(c.qd, c.cache, c.seqs, scale=c.scale, out=out, workspace=ws[:need - 16])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_sequences(vqv, dtype):
    """64 of very different lengths, that fill the GPU and are split all the same."""
    kv = [9000, 1] + [(37 * i) % 300 + 1 for i in range(62)]
    c = Case(rows=[1] * 64, kv=kv, heads=8, hk=8, dim=64, ps=16, dtype=dtype)
    c.close(c.run(vqv), c.want(), low=5.0 * 9000)
    assert vqv.vqv_paged_attn_q4_workspace_bytes(c.cache, c.seqs, c.heads) > 0
    c.close(c.run(vqv, 300, 5), c.want(300, 5))


@pytest.mark.parametrize("n", [2, 3, 4, 8, 9, 16])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_chunk_beside_decoding_rows(vqv, n, dtype):
    """Tiles of one long chunk and single rows, in batches of even and odd size, the chunk first and last."""
    for first in (True, False):
        rows = [150] + [1] * (n - 1)
        kv = [700] + [(113 * i) % 900 + 1 for i in range(1, n)]
        if not first:
            rows, kv = rows[::-1], kv[::-1]
        c = Case(rows=rows, kv=kv, heads=4, hk=2, dim=64, ps=16, dtype=dtype, seed=n)
        c.close(c.run(vqv), c.want())
        c.max_kv = 9000     # planned for longer ones: splits
        c.close(c.run(vqv), c.want())


def test_read_only_one(vqv):
    cache, table, _ = append(vqv, rows=[4], kv=[10], heads=2, hk=1, dim=64, ps=16, rot=64, inter=False)
    seqs = vqv.Sequences(i32([0, 4]), i32([10]), i32(table), n_rows=4, max_rows=4, max_kv=10)
    k, v = vqv.vqv_cache_q4_read(cache, seqs)
    for args in (dict(want_v=False), dict(k_out=torch.empty_like(k), want_k=False, want_v=False)):
        got, none = vqv.vqv_cache_q4_read(cache, seqs, **args)
        assert none is None and torch.equal(got, k)
    none, got = vqv.vqv_cache_q4_read(cache, seqs, want_k=False)
    assert none is None and torch.equal(got, v)
    assert vqv.vqv_cache_q4_read(cache, seqs, want_k=False, want_v=False) == (None, None)
