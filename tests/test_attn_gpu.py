"""vqv_paged_attn against the oracle in 64 bits."""

import pytest
import torch

from oracle import round_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Inputs on the GPU. Every slot that no token stands in holds NaN, in K and V."""

    def __init__(self, rows, kv, heads, hk, dim, ps, dtype="bf16", layout="slot", seed=0, layers=1,
                 layer=0, max_rows=None, max_kv=None):
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.kv, self.ps, self.hk, self.dim = rows, kv, ps, hk, dim
        self.heads, self.t, self.layer = heads, DT[dtype], layer
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
        shape = (layers, self.pages, ps, hk, dim)
        k = torch.full(shape, float("nan"))
        v = k.clone()
        for b, x in enumerate(kv):
            for t in range(x):
                p = self.table[b][t // ps]
                k[layer, p, t % ps] = torch.randn(hk, dim, generator=gen)
                v[layer, p, t % ps] = torch.randn(hk, dim, generator=gen)
        self.q = (1.5 * torch.randn(self.n, heads, dim, generator=gen)).to(self.t)
        self.k, self.v = k.to(self.t), v.to(self.t)
        self.layout = layout
        self.max_rows = max(rows) if max_rows is None else max_rows
        self.max_kv = max(kv) if max_kv is None else max_kv
        self.scale = dim ** -0.5

    def device(self, x):
        if self.layout == "head":
            return x.transpose(2, 3).contiguous().cuda().transpose(2, 3)
        if self.layout == "gap":
            wide = torch.full((*x.shape[:2], x.shape[2] + 1, x.shape[3], x.shape[4] + 8),
                              float("nan"), dtype=x.dtype)
            wide[:, :, :x.shape[2], :, :x.shape[4]] = x
            return wide.cuda()[:, :, :x.shape[2], :, :x.shape[4]]
        return x.cuda()

    def run(self, vqv, window=0, sinks=0, stream=None, scale=None):
        self.cache = vqv.PagedCache(self.device(self.k), self.device(self.v))
        self.seqs = vqv.Sequences(i32(self.start), i32(self.kv), i32(self.table), n_rows=self.n,
                                  max_rows=self.max_rows, max_kv=self.max_kv)
        out = torch.full(self.q.shape, 9.0, dtype=self.t, device="cuda")
        self.qd = self.q.cuda()
        vqv.vqv_paged_attn(self.qd, self.cache, self.seqs, scale=scale or self.scale, window=window,
                           sinks=sinks, layer=self.layer, out=out, stream=stream)
        torch.cuda.synchronize()
        return out.cpu()

    def want(self, window=0, sinks=0, scale=None):
        return ref.attn_ref(self.q, self.k[self.layer], self.v[self.layer], self.start, self.kv,
                            self.table, scale or self.scale, window, sinks)

    def close(self, got, want):
        """Half a step of the output; half a step of each weight; a score's error moves its weight
        by as much, relatively: `dim` products and sums in fp32 of sizes up to `size`, then one
        scaling and one subtraction (2 roundings of values up to 2 * size) and the exponential
        (2^-22), for the weight and for the sum of weights; sums over tokens in fp32. fp16 weights
        below 2^-14 are off by up to 2^-14 (the smallest normal) each."""
        out, mean, size = want
        half, n = torch.finfo(self.t).eps / 2, max(self.kv)
        score = size * (self.dim + 8) * 2.0 ** -24 + 2.0 ** -22
        inner = (half + 2 * score + (n + 8) * 2.0 ** -24) * mean
        if self.t == torch.float16:
            inner = inner + n * 2.0 ** -14 * half * 8
        allow = half * (out.abs() + inner) + inner + 2.0 ** -25
        err = (got.double() - out).abs()
        assert (err <= allow).all(), f"error over allowance {(err / allow).nan_to_num(1e9).max():.3g}"


CASES = [
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
]
WINDOWS = [(0, 0), (1, 0), (1, 3), (37, 0), (64, 4), (100, 150), (5000, 2)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['rows']}kv{c['kv']}h{c['heads']}/{c['hk']}d{c['dim']}p{c['ps']}")
def test_matches_oracle(vqv, case):
    c = Case(**case)
    c.close(c.run(vqv), c.want())


@pytest.mark.parametrize("window,sinks", WINDOWS[1:])
@pytest.mark.parametrize("index", [1, 2, 5, 6, 8, 10])
def test_windows(vqv, index, window, sinks):
    c = Case(**CASES[index])
    c.close(c.run(vqv, window, sinks), c.want(window, sinks))


def test_large_scores(vqv):
    """Scores far apart: one weight takes nearly all, and moves from block to block."""
    c = Case(rows=[8, 1], kv=[600, 900], heads=4, hk=2, dim=64, ps=16, seed=5)
    c.q *= 12
    c.close(c.run(vqv, scale=1.0), c.want(scale=1.0))


def test_bad_pages_are_hidden(vqv):
    """Pages that the table does not hold, or that are none: their tokens are
    hidden; a row with nothing left gives zeros."""
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
    c.kv = [100, 3, 0]
    c.max_kv = 100
    got = c.run(vqv)
    c.close(got, c.want())
    assert (got[3:5] == 0).all() and (got[8:] == 0).all()


@pytest.mark.parametrize("ps", [1, 16])
@pytest.mark.parametrize("rows", [2, 150])
def test_lengths_past_any_table(vqv, rows, ps):
    """A kv_len near 2^31: the tokens that the table holds are seen by all rows."""
    gen = torch.Generator().manual_seed(3)
    n = 64 // ps
    k, v = (torch.randn(1, n, ps, 1, 64, generator=gen).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(rows, 2, 64, generator=gen).to(torch.bfloat16)
    seqs = vqv.Sequences(i32([0, rows]), i32([2 ** 31 - 1]), i32([list(range(n))]), n_rows=rows,
                         max_rows=rows, max_kv=64)
    got = vqv.vqv_paged_attn(q.cuda(), vqv.PagedCache(k.cuda(), v.cuda()), seqs, scale=0.125).cpu()
    c = Case(rows=[1], kv=[64], heads=2, hk=1, dim=64, ps=ps)
    # as single rows at the end of 64 tokens
    want = ref.attn_ref(q, k[0], v[0], list(range(rows + 1)), [64] * rows, [list(range(n))] * rows, 0.125)
    c.close(got, want)


def test_longer_than_planned(vqv):
    """A max_kv below the real lengths costs speed, not results."""
    for rows in ([2, 1], [80, 3]):
        c = Case(rows=rows, kv=[900, 500], heads=4, hk=2, dim=128, ps=16, max_kv=150)
        c.close(c.run(vqv), c.want())


def test_rows_without_a_sequence(vqv):
    """Rows past max_rows and past the last sequence are not written."""
    c = Case(rows=[6], kv=[50], heads=2, hk=1, dim=64, ps=16, max_rows=4)
    got, want = c.run(vqv), c.want()
    assert (got[4:] == 9.0).all()
    c.close(got[:4], tuple(x[:4] for x in want))


def test_hidden_infinities_and_nan(vqv):
    """Tokens that a row does not see may hold anything: future tokens of the
    chunk, tokens before the window."""
    for rows, dtype, dim in (([12], "bf16", 64), ([12], "fp16", 256), ([150], "bf16", 128)):
        c = Case(rows=rows, kv=[200], heads=4, hk=1, dim=dim, ps=16, dtype=dtype)
        n = rows[0]
        clean = c.run(vqv, 40, 2)
        for t, x in ((199, float("nan")), (200 - n // 2, float("inf")), (20, float("nan")),
                     (21, float("-inf"))):
            p = c.table[0][t // 16]
            c.k[0, p, t % 16], c.v[0, p, t % 16] = x, x
        got = c.run(vqv, 40, 2)
        before = n // 2  # rows before the first bad token of the chunk that do not see 20, 21
        rows_ok = [r for r in range(before) if 200 - n + r - 40 >= 21]
        assert rows_ok and torch.equal(got[rows_ok], clean[rows_ok])
        assert got[-1].isnan().all()


def test_seen_nan(vqv):
    """A NaN that is seen comes out."""
    c = Case(rows=[2], kv=[40], heads=2, hk=1, dim=64, ps=16)
    c.k[0, c.table[0][0], 3, 0, 5] = float("nan")
    assert c.run(vqv).isnan().all()


def test_deterministic_on_streams_and_graphs(vqv):
    c = Case(rows=[8, 2], kv=[700, 90], heads=8, hk=2, dim=128, ps=16)
    want = c.run(vqv)
    assert torch.equal(c.run(vqv, stream=torch.cuda.Stream()), want)
    out = torch.empty(c.q.shape, dtype=c.t, device="cuda")
    need = vqv.vqv_paged_attn_workspace_bytes(c.cache, c.seqs, c.heads)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vqv.vqv_paged_attn(c.qd, c.cache, c.seqs, scale=c.scale, out=out, workspace=ws)
    for _ in range(4):
        out.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


def test_far_offsets(vqv):
    """Pages whose place passes 2^32 values."""
    ps, hk, dim, pages = 64, 8, 256, 36000        # 36000 pages of 131072 values: 4.7e9
    k = torch.empty((1, pages, ps, hk, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ids = [pages - 1, 5, pages - 2]
    gen = torch.Generator().manual_seed(1)
    small = [torch.randn(3, ps, hk, dim, generator=gen).to(torch.bfloat16) for _ in range(2)]
    for x, s in zip((k, v), small):
        x[0, ids] = s.cuda()
    q = torch.randn(2, hk, dim, generator=gen).to(torch.bfloat16)
    seqs = vqv.Sequences(i32([0, 2]), i32([150]), i32([ids]), n_rows=2, max_rows=2, max_kv=150)
    got = vqv.vqv_paged_attn(q.cuda(), vqv.PagedCache(k, v), seqs, scale=0.06).cpu()
    c = Case(rows=[2], kv=[150], heads=hk, hk=hk, dim=dim, ps=ps)
    c.close(got, ref.attn_ref(q, *small, [0, 2], [150], [[0, 1, 2]], 0.06))


def test_refuses_wrong_tensors(vqv):
    c = Case(rows=[2], kv=[10], heads=2, hk=1, dim=64, ps=16)
    c.run(vqv)
    for q in (c.qd[:1], c.qd.half(), c.qd[:, :, ::2], c.qd[:, 0], c.q):
        with pytest.raises(ValueError):
            vqv.vqv_paged_attn(q, c.cache, c.seqs, scale=1.0)
    with pytest.raises(ValueError):
        vqv.vqv_paged_attn(c.qd, c.cache, c.seqs, scale=1.0, out=torch.empty(2, 2, 64, device="cuda"))
    with pytest.raises(vqv.VqvError):
        vqv.vqv_paged_attn(c.qd, c.cache, c.seqs, scale=0.0)


def near(c, got, want, low=0.0, terms=1):
    """As `close`, for scores of `terms` products each, where the largest weight of a wave's tokens is 1
    exactly (`want`'s mean is then what the others come to) and fp16 weights are 2^15 times as
    large: off by up to 2^-25 of that where they are subnormal; low is the sum of |v| over tokens."""
    out, mean, size = want
    half, n = torch.finfo(c.t).eps / 2, max(c.kv)
    score = size * (terms + 8) * 2.0 ** -24 + 2.0 ** -22
    inner = (2 * score + (n + 8) * 2.0 ** -24) * torch.maximum(mean, out.abs()) + half * mean
    if c.t == torch.float16:
        inner = inner + 2.0 ** -40 * low
    allow = half * (out.abs() + inner) + inner + 2.0 ** -25
    err = (got.double() - out).abs()
    assert (err <= allow).all(), f"error over allowance {(err / allow).nan_to_num(1e9).max():.3g}"


def ladder(rows, dim, dtype, steps, heads=2, seed=0, kv=1300):
    """A case whose scores go by the first column alone: step (token, score of a row of factor 1);
    all other tokens score -30 times that. Row i's factor is between 1 and 1.5. One split."""
    c = Case(rows=[rows], kv=[kv], heads=heads, hk=1, dim=dim, ps=16, dtype=dtype, seed=seed, max_kv=64)
    c.q.zero_()
    c.q[:, :, 0] = (1 + torch.rand(rows, heads, generator=torch.Generator().manual_seed(seed)) / 2).to(c.t)
    c.k[0, c.table[0][:-(-kv // 16)], :, :, 0] = -30.0
    for t, score in steps:
        c.k[0, c.table[0][t // 16], t % 16, :, 0] = score
    c.k[0, :, :, :, 1:] = 0
    return c


SHAPES_OF_WAVES = [(2, 64), (2, 128), (2, 256), (20, 80), (20, 192), (50, 96), (50, 192), (100, 64), (100, 128)]


@pytest.mark.parametrize("rows,dim", SHAPES_OF_WAVES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_largest_weight_is_exact(vqv, rows, dim, dtype):
    """A score that passes the one before it by less than 2^8 (in a later block of the same wave)
    has the largest weight: its error is none, and the other's is multiplied by values of 0."""
    c = ladder(rows, dim, dtype, [(0, 1.0), (512, 3.5)])
    c.v[0, c.table[0][0], 0] = 0
    out, mean, size = c.want(scale=1.0)
    # all of the sum of weighted |v| but for the largest weight's part
    near(c, c.run(vqv, scale=1.0), (out, (mean - out.abs()).clamp(min=0), size))


@pytest.mark.parametrize("rows,dim", [(1, 256), (50, 192), (100, 64), (100, 128), (100, 256)])
@pytest.mark.parametrize("below", [11.0, 17.5, 21.0])
def test_many_small_weights(vqv, rows, dim, below):
    """fp16: thousands of tokens far below one of values 0 are most of the output."""
    c = Case(rows=[rows], kv=[6000], heads=1, hk=1, dim=dim, ps=16, dtype="fp16", max_kv=64)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.k.zero_()
    c.k[0, c.table[0][0], 3, :, 0] = below
    c.v[0, c.table[0][:375]] = 500 + 100 * c.v[0, c.table[0][:375]]
    c.v[0, c.table[0][0], 3] = 0
    low = c.v[0, c.table[0][:375]].double().abs().sum((0, 1, 2))
    near(c, c.run(vqv, scale=1.0), c.want(scale=1.0), low=low)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,dim", [(2, 64), (50, 192), (100, 64), (300, 128)])
def test_seen_nan_and_infinity_in_every_shape(vqv, rows, dim, dtype):
    """A NaN among the keys, and a score of infinity: NaN; an infinity among the values of a seen
    token comes out, in its column alone."""
    c = Case(rows=[rows], kv=[400], heads=2, hk=1, dim=dim, ps=16, dtype=dtype)
    p, clean = c.table[0][1], c.run(vqv)
    for x in (float("nan"), float("inf")):
        keep = c.k[0, p, 3].clone()
        c.k[0, p, 3, 0, 5] = x
        got = c.run(vqv)
        assert got[c.q[:, :, 5] * x != -float("inf")].isnan().all()
        c.k[0, p, 3] = keep
    c.v[0, p, 3, 0, 7] = -float("inf")
    got = c.run(vqv)
    assert (got[:, :, 7] == -float("inf")).all()
    assert torch.equal(got[:, :, :7], clean[:, :, :7]) and torch.equal(got[:, :, 8:], clean[:, :, 8:])


@pytest.mark.parametrize("rows,dim", SHAPES_OF_WAVES)
def test_scores_past_any_exponent(vqv, rows, dim):
    """Scores of 1e6 to 1e37: one token takes all, and the output is its values."""
    for size in (1e6, 1e10, 1e20, 1e34):
        c = ladder(rows, dim, "bf16", [(t, 2.0 ** (t / 100) * size) for t in range(0, 1200, 37)], kv=1300)
        for sign in (1, -1):
            c.k[0, :, :, :, 0] *= sign
            got, want = c.run(vqv, scale=1.0), c.want(scale=1.0)
            if sign > 0:
                assert torch.equal(got.double(), want[0])
            else:   # the many tokens at 30 to 45, of equal weights
                near(c, got, (want[0], want[1], torch.tensor(45.0)))


@pytest.mark.parametrize("rows,kv", [(8, 5), (8, 1), (50, 20), (150, 100)])
def test_window_past_any_length(vqv, rows, kv):
    """The widest window, also where the first rows stand before the first token."""
    c = Case(rows=[rows, rows], kv=[kv, kv + 30], heads=2, hk=1, dim=64, ps=16)
    plain = c.run(vqv)
    for window in (2 ** 31 - 1, 2 ** 31 - kv, 2 ** 30 + 1):
        for sinks in (0, 3, 2 ** 31 - 1):
            c.close(c.run(vqv, window, sinks), c.want())
    c.close(plain, c.want())


def test_no_rows(vqv):
    """A call without rows is a call: of attention, of the append, of compact."""
    c = Case(rows=[2, 1], kv=[20, 7], heads=4, hk=2, dim=64, ps=16)
    c.run(vqv)
    seqs = vqv.Sequences(i32([0, 0, 0]), i32([20, 7]), i32(c.table), n_rows=0, max_rows=0, max_kv=20)
    before = [c.cache.k.clone(), c.cache.v.clone()]
    q = torch.empty(0, 4, 64, dtype=c.t, device="cuda")
    assert vqv.vqv_paged_attn(q, c.cache, seqs, scale=1.0).shape == (0, 4, 64)
    k = torch.empty(0, 2, 64, dtype=c.t, device="cuda")
    assert vqv.vqv_rope_append(q, k, k, c.cache, seqs, vqv.Rope(64)).shape == (0, 4, 64)
    assert vqv.vqv_cache_compact(c.cache, seqs, i32([])).tolist() == [20, 7]
    for x, y in zip((c.cache.k, c.cache.v), before):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


# Rows of a case (two heads to a key head) that take 32, 64, 128 and, up to dim 128 without a
# window, two tiles of 128 (row, head) pairs of a work-group.
ROWS = [3, 20, 50, 90]


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 80, 96, 128, 192, 256])
def test_many_blocks_of_one_work_group(vqv, dim, dtype, rows, window, sinks):
    """A max_kv that plans one split: every work-group walks over 10 blocks and more, past what it
    looks up ahead; odd pages, some of them none, NaN in every slot without a token."""
    c = Case(rows=[rows, 2], kv=[1501, 1290], heads=4, hk=2, dim=dim, ps=20, dtype=dtype,
             layout="head" if dim % 64 else "slot", seed=dim + rows, max_kv=64)
    c.table[0][70], c.table[0][31], c.table[1][50], c.table[1][3] = -1, c.pages, 1 << 30, -7
    near(c, c.run(vqv, window, sinks), c.want(window, sinks), 5.0 * 1501, dim)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_maximum_jumps_between_blocks(vqv, dim, dtype, rows):
    """The maximum passes the one before it by far, block after block, up and then down: what was
    summed is scaled to nothing or kept as it is."""
    for sign in (1, -1):
        steps = [(i * 71, sign * 12.0 * i) for i in range(1, 18)]
        c = ladder(rows, dim, dtype, steps, seed=rows)
        near(c, c.run(vqv, scale=1.0), c.want(scale=1.0))


@pytest.mark.parametrize("rows,dim,dtype", [(1, 128, "bf16"), (8, 256, "fp16"), (200, 64, "bf16"), (130, 128, "fp16")])
def test_long_sequences(vqv, rows, dim, dtype):
    """Tens of thousands of tokens in many splits, the last one short."""
    c = Case(rows=[rows], kv=[24001], heads=2, hk=1, dim=dim, ps=64, dtype=dtype, seed=rows)
    near(c, c.run(vqv), c.want(), 5.0 * 24001, dim)
    near(c, c.run(vqv, 9000, 100), c.want(9000, 100), 5.0 * 24001, dim)


@pytest.mark.parametrize("rows,dim", [(1, 64), (3, 80), (8, 128), (16, 96), (30, 128), (25, 192), (16, 256), (32, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_few_rows_are_as_good_as_fp32(vqv, rows, dim, dtype):
    """Up to 64 (row, head) pairs the weights are held to 2^-16 (bf16) or 2^-22, twice the type's
    bits: beside the output's own rounding an error of that and of fp32 sums."""
    c = Case(rows=[rows, 1], kv=[700, 333], heads=2, hk=1, dim=dim, ps=16, dtype=dtype, seed=rows)
    for window, sinks in ((0, 0), (200, 3)):
        got, (out, mean, size) = c.run(vqv, window, sinks), c.want(window, sinks)
        half = torch.finfo(c.t).eps / 2
        score = size * (dim + 8) * 2.0 ** -24 + 2.0 ** -22
        inner = (half ** 2 + 2 * score + (700 + 8) * 2.0 ** -24) * mean
        if dtype == "fp16":
            inner = inner + 2.0 ** -40 * 5.0 * 700
        allow = half * (out.abs() + inner) + inner + 2.0 ** -25
        err = (got.double() - out).abs()
        assert (err <= allow).all(), f"error over allowance {(err / allow).max():.3g}"


@pytest.mark.parametrize("rows,dim", SHAPES_OF_WAVES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_infinity_behind_a_small_weight(vqv, rows, dim, dtype):
    """Weights that are powers of two (nothing is left over by their rounding): an infinity among
    the values comes out as one, not as NaN."""
    c = ladder(rows, dim, dtype, [(0, 0.0), (512, 0.0)])
    c.q[:, :, 0] = 1.0
    for depth in (0, 1, 7, 20, 30, 38):
        c.k[0, c.table[0][32], 0, :, 0] = -depth
        for x in (float("inf"), -float("inf")):
            c.v[0, c.table[0][32], 0, :, 11] = x
            got = c.run(vqv, scale=0.6931471805599453)
            assert (got[:, :, 11] == x).all(), depth
            assert got.isfinite().sum() == got.numel() - got[:, :, 11].numel()
