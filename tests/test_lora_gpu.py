"""vqv_lora_add against the oracle in 64 bits."""

import pytest
import torch

from oracle import serve_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


class Case:
    def __init__(self, which, K, N, rank, n, act="bf16", weight=None, ranks=None, seed=0, size=1.0):
        gen = torch.Generator().manual_seed(seed)
        M = len(which)
        t, w = DT[act], DT[weight or (act if act != "fp32" else "bf16")]
        self.x = (size * torch.randn(M, K, generator=gen)).to(t)
        self.a = (K ** -0.5 * torch.randn(n, rank, K, generator=gen)).to(w)
        self.b = (rank ** -0.5 * torch.randn(n, N, rank, generator=gen)).to(w)
        self.scale = 0.5 + torch.rand(n, generator=gen)
        self.y = torch.randn(M, N, generator=gen)
        self.which = torch.tensor(which, dtype=torch.int32)
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32)

    def set(self, vqv):
        return vqv.Adapters(self.a.cuda(), self.b.cuda(), self.scale.cuda(),
                            None if self.ranks is None else self.ranks.cuda())

    def want(self):
        return ref.lora_add(self.x, self.a, self.b, self.scale, self.which, self.y, self.ranks)

    def close(self, got, want):
        """fp32: K products summed, then `rank` products of values that hold all of the first sums'
        bits (three of the weights' type: three products each), the scaling and the last sum, each off by
        2^-24 of at most the sum of absolute products."""
        out, size = want
        terms = self.x.shape[1] + 3 * self.a.shape[1] + 16
        err = (got.cpu().double() - out).abs()
        allow = terms * 2.0 ** -24 * size + 1e-30
        assert (err <= allow).all(), f"error over allowance {(err / allow).max():.3g}"
        # Sums of many terms of either sign: their errors add up to far less than that.
        close = (err > 16 * 2.0 ** -24 * size).double().mean()
        assert close < 0.01, f"{close:.3g} of the values are far off for fp32 sums"


CASES = [
    dict(which=[0], K=64, N=1, rank=8, n=1),
    dict(which=[0] * 8, K=512, N=300, rank=16, n=2),
    dict(which=[1, 0, 1, 1, 0, 2, -1, 5], K=520, N=257, rank=16, n=3, act="fp16"),
    dict(which=list(range(40)) + [-1] * 3 + [7] * 21, K=264, N=130, rank=32, n=40),
    dict(which=[3] * 64, K=1024, N=515, rank=64, n=4, act="fp16"),
    dict(which=[i % 3 for i in range(150)], K=328, N=100, rank=40, n=3),
    dict(which=[0] * 70 + [1] * 1 + [2] * 130, K=256, N=192, rank=128, n=3),
    dict(which=[i // 50 - 1 for i in range(230)], K=8, N=33, rank=256, n=4, act="fp16"),
    dict(which=[0, 1] * 9, K=1000, N=77, rank=24, n=2, act="fp32"),
    dict(which=[1] * 33 + [0] * 20, K=512, N=90, rank=72, n=2, act="fp32", weight="fp16"),
    dict(which=[i * 7 % 64 for i in range(64)], K=128, N=64, rank=8, n=64),
    dict(which=[0, 1, 2, 3] * 16, K=5120, N=2000, rank=16, n=4),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c['which'])}x{c['K']}x{c['N']}r{c['rank']}n{c['n']}{c.get('act', 'bf16')}")
def test_matches_oracle(vqv, case):
    c = Case(**case)
    want = c.want()
    got = vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda())
    c.close(got, want)
    none = [m for m, e in enumerate(case["which"]) if not 0 <= e < case["n"]]
    assert torch.equal(got.cpu()[none], c.y[none])


@pytest.mark.parametrize("act", ["bf16", "fp16", "fp32"])
def test_ranks(vqv, act):
    """Fewer ranks than the arrays hold, none, odd ones, wrong ones: what is past them is not used."""
    c = Case([0, 1, 2, 3, 4, 5] * 4, K=320, N=100, rank=40, n=6, act=act, ranks=[40, 0, 1, 13, -5, 99])
    for e, r in enumerate([40, 0, 1, 13, 0, 40]):
        c.a[e, r:] = float("nan")
        c.b[e, :, r:] = float("nan")
    got = vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda())
    c.close(got, c.want())


@pytest.mark.parametrize("weight,size", [("bf16", 1e-30), ("bf16", 1e30), ("fp16", 1e-30), ("fp16", 1e30), ("fp16", 1e-3), ("fp16", 1e3)])
def test_sizes(vqv, weight, size):
    """Values between the products of any fp32 size, rows of very different sizes together."""
    c = Case([0, 1] * 12, K=256, N=64, rank=16, n=2, act="fp32", weight=weight, size=size)
    c.x[::3] = 0
    c.x[1::5] *= 1e-4
    c.y *= size
    c.close(vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda()), c.want())


def test_nan_and_infinity_stay_in_their_rows(vqv):
    for act in ("bf16", "fp16", "fp32"):
        c = Case([0] * 20 + [1] * 20, K=256, N=70, rank=16, n=2, act=act)
        clean = vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda()).cpu()
        c.x[3, 7], c.x[25, 0] = float("nan"), float("inf")
        got = vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda()).cpu()
        rest = [m for m in range(40) if m not in (3, 25)]
        assert torch.equal(got[rest], clean[rest])
        assert got[3].isnan().all() and not got[25].isfinite().any()


def test_in_place_and_columns(vqv):
    """out = y, columns of wider tensors, rows that are not 16-byte aligned."""
    c = Case([0, -1, 1, 1, 0] * 8, K=192, N=99, rank=16, n=2)
    want, ad, x, which = c.want(), c.set(vqv), c.x.cuda(), c.which.cuda()
    first = vqv.vqv_lora_add(x, ad, which, c.y.cuda())
    c.close(first, want)
    y = c.y.cuda()
    assert vqv.vqv_lora_add(x, ad, which, y, out=y) is y
    assert torch.equal(y, first)
    for off, width in ((0, 99), (3, 205), (4, 208)):
        wide = torch.full((40, width), 5.0, device="cuda")
        wide[:, off:off + 99] = c.y.cuda()
        part = wide[:, off:off + 99]
        vqv.vqv_lora_add(x, ad, which, part, out=part)
        assert torch.equal(part, first)
        assert (wide[:, :off] == 5).all() and (wide[:, off + 99:] == 5).all()
        out = torch.full((40, width), 5.0, device="cuda")
        vqv.vqv_lora_add(x, ad, which, c.y.cuda(), out=out[:, off:off + 99])
        assert torch.equal(out[:, off:off + 99], first)
        assert (out[:, :off] == 5).all() and (out[:, off + 99:] == 5).all()


def test_order_of_rows_does_not_matter(vqv):
    """Rows are computed alike wherever they stand, if as many share their adapter."""
    c = Case([0] * 10 + [1] * 30, K=256, N=64, rank=16, n=2)
    ad = c.set(vqv)
    got = vqv.vqv_lora_add(c.x.cuda(), ad, c.which.cuda(), c.y.cuda()).cpu()
    p = torch.randperm(40, generator=torch.Generator().manual_seed(1))
    mixed = vqv.vqv_lora_add(c.x[p].cuda(), ad, c.which[p].cuda(), c.y[p].cuda()).cpu()
    assert torch.equal(mixed, got[p])


def test_streams_and_graphs(vqv):
    c = Case([i % 5 - 1 for i in range(90)], K=640, N=200, rank=32, n=4)
    ad, x, which, y = c.set(vqv), c.x.cuda(), c.which.cuda(), c.y.cuda()
    want = vqv.vqv_lora_add(x, ad, which, y)
    torch.cuda.synchronize()
    other = vqv.vqv_lora_add(x, ad, which, y, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    out = torch.empty_like(y)
    ws = torch.empty(vqv.vqv_lora_add_workspace_bytes(ad, 90), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vqv.vqv_lora_add(x, ad, which, y, out=out, workspace=ws)
    for _ in range(4):
        out.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_no_rows_and_refusals(vqv):
    c = Case([0, 1], K=64, N=16, rank=8, n=2)
    ad = c.set(vqv)
    empty = vqv.vqv_lora_add(c.x[:0].cuda(), ad, c.which[:0].cuda(), c.y[:0].cuda())
    assert empty.shape == (0, 16)
    x, which, y = c.x.cuda(), c.which.cuda(), c.y.cuda()
    for bad in (x[:1], x[:, ::2], x.cpu()):
        with pytest.raises(ValueError):
            vqv.vqv_lora_add(bad, ad, which, y)
    with pytest.raises(vqv.VqvError):
        vqv.vqv_lora_add(x.half(), ad, which, y)
    for bad in (y[:1], y.double(), y.t().contiguous().t(), y.cpu()):
        with pytest.raises(ValueError):
            vqv.vqv_lora_add(x, ad, which, bad)
    with pytest.raises(ValueError):
        vqv.vqv_lora_add(x, ad, which.long(), y)
    with pytest.raises(vqv.VqvError):
        vqv.vqv_lora_add(x, ad, which, y, out=y[:1].expand(2, 16))
    with pytest.raises(ValueError):
        vqv.Adapters(c.a.float().cuda(), c.b.float().cuda(), c.scale.cuda())
    with pytest.raises(ValueError):
        vqv.Adapters(c.a.cuda(), c.b[:, :, :4].contiguous().cuda(), c.scale.cuda())
    with pytest.raises(ValueError):
        vqv.Adapters(c.a.cuda(), c.b.cuda(), c.scale[:1].cuda())


@pytest.mark.parametrize("weight", ["bf16", "fp16"])
def test_infinities_between_the_products(vqv, weight):
    """One rank's sum is an infinity, which decides the output by its weight's sign; the others are finite, past
    the weights' type too. Then a finite sum that the weights' type would round to an infinity."""
    c = Case([0] * 5 + [1] * 40, K=64, N=300, rank=16, n=2, act="fp32", weight=weight, size=1e6)
    c.x[:, 5] = c.x[:, 5].abs() + 1
    c.a[:, 3, 5] = float("inf")
    want, got = c.want()[0], vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda()).cpu()
    assert want.isinf().all() and torch.equal(got, want.float())
    c = Case([0] * 3 + [1] * 30, K=8, N=70, rank=8, n=2, act="fp32", weight=weight)
    c.x[:], c.a[:] = 0, 0
    c.x[:, 2], c.a[:, :, 2] = 3.3999e38, 1.0
    c.b *= 2.0 ** -9
    c.close(vqv.vqv_lora_add(c.x.cuda(), c.set(vqv), c.which.cuda(), c.y.cuda()), c.want())


# Calls whose second kernel takes 64 columns at a time: ranks of up to 128, and enough columns and slots.
WIDE = [
    dict(which=[i * 7 % 66 - 1 for i in range(64)], K=72, N=8203, rank=8, n=64),
    dict(which=[i * 5 % 64 for i in range(64)], K=136, N=8450, rank=24, n=64, act="fp16"),
    dict(which=[0] * 70 + [-1] * 3 + [1, 2] * 50 + [2] * 127, K=264, N=13999, rank=64, n=3),
    dict(which=[i % 4 - 1 for i in range(300)], K=64, N=13121, rank=96, n=3, act="fp16"),
    dict(which=[i // 101 for i in range(300)], K=200, N=13500, rank=128, n=3),
    dict(which=[2] * 60 + [0, 1] * 20 + [1] * 199, K=64, N=13315, rank=40, n=3, act="fp32", weight="fp16"),
    dict(which=[1, 0, 3] * 100, K=96, N=13077, rank=128, n=2, act="fp32"),
    dict(which=[0] * 64, K=64, N=65601, rank=16, n=1, act="fp16"),
]


def is_wide(c):
    M, n, N = len(c["which"]), c["n"], c["N"]
    slots = min(n, 64, M)
    return c["rank"] <= 128 and -(-M // 64) * max(slots // 8, 1) * -(-N // 256) >= 256


@pytest.mark.parametrize("case", WIDE, ids=lambda c: f"{len(c['which'])}x{c['K']}x{c['N']}r{c['rank']}n{c['n']}{c.get('act', 'bf16')}")
def test_many_columns(vqv, case):
    """Against the oracle; fewer ranks than the arrays hold, with NaN past them; in place, and columns of
    wider tensors, whose rows are not 16-byte aligned and whose other columns stay."""
    assert is_wide(case)
    c = Case(**case)
    x, which, N = c.x.cuda(), c.which.cuda(), case["N"]
    want, ad = c.want(), c.set(vqv)
    got = vqv.vqv_lora_add(x, ad, which, c.y.cuda())
    c.close(got, want)
    none = [m for m, e in enumerate(case["which"]) if not 0 <= e < case["n"]]
    assert torch.equal(got.cpu()[none], c.y[none])
    y = c.y.cuda()
    vqv.vqv_lora_add(x, ad, which, y, out=y)
    assert torch.equal(y, got)
    for off, width in ((3, N + 6), (4, N + 12 - N % 4)):
        wide = torch.full((len(which), width), 5.0, device="cuda")
        wide[:, off:off + N] = c.y.cuda()
        vqv.vqv_lora_add(x, ad, which, wide[:, off:off + N], out=wide[:, off:off + N])
        assert torch.equal(wide[:, off:off + N], got)
        assert (wide[:, :off] == 5).all() and (wide[:, off + N:] == 5).all()
    c.ranks = torch.tensor([(5 * e + 3) % (case["rank"] + 1) for e in range(case["n"])], dtype=torch.int32)
    for e, r in enumerate(c.ranks.tolist()):
        c.a[e, r:] = float("nan")
        c.b[e, :, r:] = float("nan")
    c.close(vqv.vqv_lora_add(x, c.set(vqv), which, c.y.cuda()), c.want())


@pytest.mark.parametrize("N", [99, 512, 8203])
def test_other_columns_of_the_same_rows(vqv, N):
    c = Case([0, -1, 1, 1, 0] * 13, K=64, N=N, rank=16, n=2)
    ad, x, which = c.set(vqv), c.x.cuda(), c.which.cuda()
    want = vqv.vqv_lora_add(x, ad, which, c.y.cuda())
    for y0, o0 in ((0, N), (N + 3, 0)):
        wide = torch.full((65, 2 * N + 5), 5.0, device="cuda")
        y, out = wide[:, y0:y0 + N], wide[:, o0:o0 + N]
        y.copy_(c.y)
        vqv.vqv_lora_add(x, ad, which, y, out=out)
        assert torch.equal(out, want) and torch.equal(y.cpu(), c.y)
        rest = [i for i in range(2 * N + 5) if not (y0 <= i < y0 + N or o0 <= i < o0 + N)]
        assert (wide[:, rest] == 5).all()
    with pytest.raises(vqv.VqvError):
        vqv.vqv_lora_add(x, ad, which, wide[:, :N], out=wide[:, 1:N + 1])
