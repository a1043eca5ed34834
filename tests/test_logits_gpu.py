"""vqv_logits_edit against the oracle in 64 bits, and vqv_logits_verify
against the greedy verify's oracle on the edited logits."""

import numpy as np
import pytest
import torch

from oracle import round_ref as ref
from oracle import verify_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


def pack(bits):
    """Truth values [rows, n] as int32 words, the lowest bit first, the last word's rest set."""
    rows, n = bits.shape
    b = torch.ones(rows, -(-n // 32) * 32, dtype=torch.int64)
    b[:, :n] = bits
    w = (b.view(rows, -1, 32) << torch.arange(32)).sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).cuda()


def case(B, T, N, seed, penalties=True, counts=True, seen=True, bias=5, mask=True):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=gen)
    c = dict(logits=3 * torch.randn(B * T, N, generator=gen), T=T, draft=None, counts=None, seen=None,
             repetition=None, frequency=None, presence=None, biases=None, allowed=None)
    c["draft"] = torch.randint(0, N, (B, T - 1), generator=gen)
    if T > 3:
        c["draft"][:, 2] = c["draft"][:, 0]      # a draft twice
    if penalties:
        c["repetition"], c["frequency"], c["presence"] = 1 + rand(B), rand(B) - 0.2, rand(B)
        if counts:
            c["counts"] = torch.where(rand(B, N) < 0.1, torch.randint(1, 9, (B, N), generator=gen), 0)
        if seen:
            c["seen"] = rand(B, N) < 0.1
    if bias:
        c["biases"] = [[(int(torch.randint(-2, N + 2, (1,), generator=gen)), (4 * rand(1) - 2).item())
                        for _ in range(bias + b)] for b in range(B)]
        c["biases"][0] += [(0, 1.5), (N - 1, -1.0), (0, 2.25)]   # the last one of a token counts
    if mask:
        c["allowed"] = rand(B * T, N) < torch.where(torch.arange(B * T) % 3 == 0, 0.05, 0.9)[:, None]
    return c


def edits(vqv, c):
    B, N = c["logits"].shape[0] // c["T"], c["logits"].shape[1]
    f = lambda x, t: None if x is None else x.to(t).cuda()
    a = dict(counts=f(c["counts"], torch.int32), seen=None if c["seen"] is None else pack(c["seen"]),
             repetition=f(c["repetition"], torch.float32), frequency=f(c["frequency"], torch.float32),
             presence=f(c["presence"], torch.float32))
    if c["biases"] is not None:
        at = np.cumsum([0] + [len(x) for x in c["biases"]])
        flat = [e for x in c["biases"] for e in x]
        a["bias_start"] = torch.tensor(at, dtype=torch.int32).cuda()
        a["bias_token"] = torch.tensor([t for t, _ in flat], dtype=torch.int32).cuda()
        a["bias_value"] = torch.tensor([v for _, v in flat], dtype=torch.float32).cuda()
    return B, vqv.Edits(B, N, **a), f(c["draft"], torch.int32), \
        None if c["allowed"] is None else pack(c["allowed"])


def run_edit(vqv, c, inplace=False, **kw):
    B, e, draft, mask = edits(vqv, c)
    x = c["logits"].cuda()
    out = vqv.vqv_logits_edit(x, e, draft, B, c["T"], mask=mask, out=x if inplace else None, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def check_edit(got, c):
    want, size = ref.logits_ref(**c)
    hidden = want == -np.inf
    assert torch.equal(got == -np.inf, hidden | (c["logits"] == -np.inf))
    # one rounding (half a step, 2^-24) of each step's result
    allow = 2.0 ** -24 * size * (1 + 1e-6) + 2.0 ** -149
    err = (got.double() - want).abs()[~hidden]
    assert (err <= allow[~hidden]).all(), (err / allow[~hidden]).max()


CASES = [dict(B=1, T=1, N=1), dict(B=2, T=1, N=33), dict(B=1, T=8, N=4096), dict(B=3, T=5, N=4097),
         dict(B=2, T=16, N=9001), dict(B=1, T=64, N=777, bias=0), dict(B=2, T=3, N=5000, counts=False),
         dict(B=2, T=4, N=1000, seen=False, mask=False), dict(B=2, T=4, N=1002, penalties=False),
         dict(B=1, T=2, N=70000, bias=900), dict(B=4, T=2, N=100, penalties=False, bias=0)]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_edit(vqv, kw):
    c = case(**kw, seed=kw["N"])
    got = run_edit(vqv, c)
    check_edit(got, c)
    assert torch.equal(run_edit(vqv, c, inplace=True), got)


@pytest.mark.parametrize("only", ["repetition", "frequency", "presence"])
def test_single_penalties(vqv, only):
    c = case(2, 4, 900, seed=4, bias=0, mask=False)
    for name in ("repetition", "frequency", "presence"):
        if name != only:
            c[name] = None
    check_edit(run_edit(vqv, c), c)


def test_without_drafts(vqv):
    c = case(2, 4, 900, seed=6)
    c["draft"] = None
    check_edit(run_edit(vqv, c), c)


def test_drafts_that_are_no_tokens(vqv):
    c = case(1, 5, 50, seed=7)
    c["draft"] = torch.tensor([[-1, 50, 1 << 30, 60]])
    check_edit(run_edit(vqv, c), c)


def run_verify(vqv, c, draft_len=None):
    B, e, draft, mask = edits(vqv, c)
    out = vqv.vqv_logits_verify(c["logits"].cuda(), e, draft, B, c["T"], mask=mask, draft_len=draft_len)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in out]


@pytest.mark.parametrize("kw", CASES, ids=str)
@pytest.mark.parametrize("limited", [False, True])
def test_verify(vqv, kw, limited):
    """Exactly the verify of the edited logits."""
    c = case(**kw, seed=kw["N"] + 1)
    B, T = kw["B"], kw["T"]
    if T > 1:   # drafts that the target confirms, as far as they do not change its choice
        first = torch.from_numpy(run_verify(vqv, c)[0]).view(B, T)
        c["draft"][:, :T // 2] = first[:, :T // 2]
    dl = torch.arange(B, dtype=torch.int32).cuda() if limited else None
    a, n, m = run_verify(vqv, c, dl)
    x = run_edit(vqv, c).numpy()
    wa, wn, wm = verify_ref(x, c["draft"].to(torch.int32).numpy(), B, T,
                            draft_len=None if dl is None else dl.cpu().numpy(), margin=True)
    np.testing.assert_array_equal(a, wa)
    np.testing.assert_array_equal(n, wn)
    np.testing.assert_array_equal(m, wm)


def test_nothing_allowed(vqv):
    c = case(1, 3, 5000, seed=9)
    c["allowed"][1] = False
    c["logits"][2, 77] = float("nan")
    c["allowed"][2, 77] = False          # a masked NaN has no influence
    a, _, m = run_verify(vqv, c)
    assert a[1] == 0 and m[1] == 0 and np.isfinite(m[2]) and a[2] != 77
    c["allowed"][2, 77] = True
    a, _, m = run_verify(vqv, c)
    assert a[2] == 77 and np.isnan(m[2])


def test_lowest_value_and_infinities(vqv):
    """Logits at the type's lowest value and infinite ones follow IEEE rules."""
    low = torch.finfo(torch.float32).min
    c = case(1, 1, 64, seed=10, bias=0, mask=False)
    c["logits"][0, :8] = torch.tensor([low, -low, float("inf"), -float("inf"), low, 0.0, -0.0, 1e-40])
    c["counts"][0, :8] = torch.tensor([1, 1, 1, 1, 0, 2, 2, 1])
    got = run_edit(vqv, c)[0].double()
    x, r = c["logits"][0], c["repetition"][0]
    f, p, n = c["frequency"][0], c["presence"][0], c["counts"][0].float()
    told = (c["counts"][0] > 0) | c["seen"][0]
    w = torch.where(told, torch.where(x > 0, x / r, x * r), x) - f * n
    w = torch.where(n > 0, w - p, w)
    assert torch.equal(got, w.double())


def test_graph_and_stream(vqv):
    c = case(2, 4, 9000, seed=12)
    B, e, draft, mask = edits(vqv, c)
    x = c["logits"].cuda()
    out = torch.empty_like(x)
    res = [torch.empty(B * 4, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"),
           torch.empty(B * 4, device="cuda")]
    ws = torch.empty(vqv.vqv_verify_workspace_bytes(B, 4, 9000), dtype=torch.uint8, device="cuda")

    def path(stream=None):
        vqv.vqv_logits_edit(x, e, draft, B, 4, mask=mask, out=out, stream=stream)
        vqv.vqv_logits_verify(x, e, draft, B, 4, mask=mask, argmax=res[0], accept_len=res[1],
                              margin=res[2], workspace=ws, stream=stream)

    path()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, *res)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path()
    for rep in range(4):
        for t in (out, *res):
            t.zero_()
        torch.cuda.synchronize()
        path(torch.cuda.Stream()) if rep == 0 else graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((out, *res), want):
            assert torch.equal(got, w)


def test_refuses_wrong_tensors(vqv):
    c = case(2, 3, 100, seed=1)
    B, e, draft, mask = edits(vqv, c)
    x = c["logits"].cuda()
    for kw in (dict(mask=mask[:, :3]), dict(mask=mask[:4]), dict(out=x.half())):
        with pytest.raises(ValueError):
            vqv.vqv_logits_edit(x, e, draft, B, 3, **kw)
    for a in ((x[:, :64], e, draft, B, 3), (x, e, draft[:, :1], B, 3), (x, e, draft, 3, 2), (x.half(), e, draft, B, 3)):
        with pytest.raises(ValueError):
            vqv.vqv_logits_edit(*a)
    with pytest.raises(vqv.VqvError):
        vqv.vqv_logits_verify(x, e, None, B, 3)
    with pytest.raises(ValueError):
        vqv.Edits(2, 100, counts=torch.zeros(2, 99, dtype=torch.int32, device="cuda"))
