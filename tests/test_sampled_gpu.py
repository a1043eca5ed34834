"""vqv_verify_sampled against the oracle in 64 bits."""

import math

import pytest
import torch

from oracle import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


class Case:
    """Drafts drawn from the drafter's probabilities (or its best guesses), which are near the target's."""

    def __init__(self, B, T, N, probs=True, seed=0, spread=3.0, near=0.4, lens=False, temperature=True):
        gen = torch.Generator().manual_seed(seed)
        self.B, self.T, self.N = B, T, N
        self.logits = spread * torch.randn(B * T, N, generator=gen)
        self.temperature = 0.5 + torch.rand(B, generator=gen) if temperature else None
        heat = self.temperature[:, None, None] if temperature else 1.0
        q = (self.logits.view(B, T, N)[:, :-1] + near * torch.randn(B, T - 1, N, generator=gen)) / heat
        q = torch.softmax(q, 2)
        self.probs = q if probs else None
        if T > 1:
            pick = torch.multinomial(q.reshape(-1, N), 1, generator=gen) if probs else q.reshape(-1, N).argmax(1)
            self.draft = pick.view(B, T - 1).to(torch.int32)
        else:
            self.draft = torch.zeros(B, 0, dtype=torch.int32)
        self.uniform = torch.rand(B, T, generator=gen)
        self.lens = torch.randint(-2, T + 2, (B,), generator=gen).to(torch.int32) if lens else None

    def run(self, vqv, **kw):
        on = lambda x: None if x is None else x.cuda()
        out = vqv.vqv_verify_sampled(self.logits.cuda(), self.draft.cuda(), self.uniform.cuda(), self.B, self.T,
                                     draft_probs=on(self.probs), temperature=on(self.temperature),
                                     draft_len=on(self.lens), **kw)
        torch.cuda.synchronize()
        return out

    def want(self):
        return ref.verify_sampled(self.logits, self.draft, self.uniform, self.B, self.T, self.probs, self.temperature,
                                  self.lens)

    def check(self, vqv, border=1e-11):
        """Tokens and lengths are equal: 64-bit exponentials to 2^-42 and sums put no decision of
        these inputs, which stay `border` away from a change, on another side. log p: one rounding to fp32
        of a 64-bit value off by 2^-40, and of p."""
        tokens, accepts, logp, near = self.want()
        assert near > border, "the inputs are next to a border"
        token, accept, got = self.run(vqv)
        assert accept.tolist() == accepts
        assert token.tolist() == tokens
        err = (got.cpu().double() - logp).abs()
        assert (err <= 2.0 ** -24 * logp.abs() + 2.0 ** -36).all(), err.max()
        return accepts


CASES = [
    dict(B=1, T=1, N=1), dict(B=1, T=2, N=1), dict(B=1, T=1, N=5), dict(B=3, T=4, N=2),
    dict(B=2, T=8, N=1000), dict(B=5, T=3, N=4095), dict(B=2, T=5, N=4096), dict(B=2, T=4, N=4097, probs=False),
    dict(B=7, T=16, N=777, lens=True), dict(B=1, T=64, N=300, near=0.05), dict(B=4, T=6, N=9001, probs=False, lens=True),
    dict(B=1, T=8, N=151936), dict(B=3, T=2, N=151936, probs=False, temperature=False), dict(B=30, T=1, N=20000),
    dict(B=2, T=2, N=300001, spread=0.5), dict(B=70, T=2, N=130, near=3.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
@pytest.mark.parametrize("seed", [0, 1])
def test_matches_oracle(vqv, case, seed):
    Case(**case, seed=seed).check(vqv)


def test_both_ends_are_reached(vqv):
    """Of many blocks some accept nothing, some everything."""
    got = Case(B=60, T=4, N=500, seed=3).check(vqv)
    assert {0, 3} <= set(got) and len(set(got)) == 4


def test_flat_rows(vqv):
    """100000 tokens of about the same probability: borders 1e-5 apart, sums up to the last one."""
    c = Case(B=16, T=1, N=100000, spread=1e-3, seed=2)
    c.uniform[:, 0] = torch.linspace(0, 1 - 2.0 ** -24, 16)
    tokens, accepts, _, _ = c.want()
    token, accept, _ = c.run(vqv)
    # the draws of 0 and the last may be on a border; they may move by one token
    assert (token.cpu() - torch.tensor(tokens)).abs().max() <= 1
    assert torch.equal(token.cpu()[1:-1], torch.tensor(tokens[1:-1], dtype=torch.int32))


def test_greedy_requests(vqv):
    """Temperatures of 0, below, NaN: as vqv_verify chooses; others beside them."""
    c = Case(B=6, T=5, N=3000, seed=4)
    c.temperature[:4] = torch.tensor([0.0, -1.0, math.nan, -0.0])
    best = c.logits.argmax(1).view(6, 5)
    c.draft[:2, :3] = best[:2, :3].to(torch.int32)
    accepts = c.check(vqv)
    am, al = vqv.vqv_verify(c.logits.cuda(), c.draft.cuda(), 6, 5)
    token, accept, logp = c.run(vqv)
    assert accept[:4].tolist() == al[:4].tolist()
    assert token[:4].tolist() == am.view(6, 5)[:4].gather(1, al[:4, None].long())[:, 0].tolist()
    assert (logp[:4] == 0).all() and accepts[0] >= 3


@pytest.mark.parametrize("temperature", [1e-40, 1e-20, 1e20, math.inf])
def test_extreme_temperatures(vqv, temperature):
    """Next to greedy, and next to every token alike."""
    c = Case(B=2, T=3, N=1000, seed=5)
    c.temperature[:] = temperature
    c.logits[:, ::3] = -math.inf
    c.draft[:] = 1
    c.check(vqv)


def test_masked_rows(vqv):
    """Masks of -inf and of the type's lowest value; rows of one token; rows of nothing; NaN and infinity."""
    c = Case(B=8, T=3, N=5000, seed=6)
    c.logits[0:3, 100:] = -math.inf
    c.logits[3:6, 7:] = torch.finfo(torch.float32).min
    c.logits[6:9] = -math.inf
    c.logits[6:9, 4321] = -5.0
    c.logits[9:12] = -math.inf
    c.logits[12, 4500], c.logits[12, 77] = math.nan, math.nan
    c.logits[15, 4500], c.logits[15, 4400] = math.inf, math.inf
    c.logits[18:21] = torch.finfo(torch.float32).max
    c.check(vqv)
    c.probs = None
    c.check(vqv)
    # drafts where the mask leaves them
    c.draft[2:7, 0] = torch.tensor([4321, 0, 77, 4400, 5], dtype=torch.int32)
    c.check(vqv)


def test_drafts_that_are_none(vqv):
    for probs in (True, False):
        c = Case(B=4, T=3, N=600, seed=7, probs=probs)
        c.draft[0, 0], c.draft[1, 1], c.draft[2, 0] = -1, 600, 2 ** 31 - 1
        accepts = c.check(vqv)
        assert accepts[0] == 0 and accepts[1] <= 1 and accepts[2] == 0


def test_random_numbers_at_the_ends(vqv):
    """0 draws the first token with a share; 1 and NaN, which are none, the last, and accept nothing
    that is not certain."""
    c = Case(B=3, T=2, N=5000, seed=8)
    c.logits[:, :10] = c.logits[:, 4900:] = -math.inf
    c.uniform[0], c.uniform[1], c.uniform[2] = 0.0, 1.0, math.nan
    c.lens = torch.zeros(3, dtype=torch.int32)
    token, accept, _ = c.run(vqv)
    assert token.tolist() == [10, 4899, 4899] and accept.tolist() == [0, 0, 0]
    c.lens = None
    c.probs = None
    _, accept, _ = c.run(vqv)
    assert accept.tolist() == [1, 0, 0]


def test_nothing_left(vqv):
    """The drafter is sure of what the target rejects, or has all that the target has."""
    c = Case(B=2, T=2, N=300, seed=9)
    c.temperature[:] = 1.0
    c.probs = torch.softmax(c.logits.view(2, 2, 300)[:, :1], 2) * 1.001    # p < q everywhere
    c.uniform[:, 0] = 1 - 2.0 ** -24
    accepts = c.check(vqv)
    assert accepts == [0, 0]
    c.probs = torch.zeros_like(c.probs)
    c.probs[0, 0, 5], c.probs[1, 0, 6] = 1.0, math.nan
    c.draft[:, 0] = torch.tensor([5, 6], dtype=torch.int32)
    token, accept, _ = c.run(vqv)
    assert accept.tolist() == [0, 0] and 5 != token[0].item() and 6 != token[1].item()


def test_rows_behind_the_last_draft_are_not_looked_at(vqv):
    c = Case(B=3, T=4, N=5000, seed=10)
    c.lens = torch.tensor([0, 1, 2], dtype=torch.int32)
    before = c.run(vqv)
    for b in range(3):
        c.logits[b * 4 + c.lens[b] + 1:b * 4 + 4] = math.nan
        c.probs[b, c.lens[b]:] = math.nan
    after = c.run(vqv)
    assert all(torch.equal(x, y) for x, y in zip(before, after))


def test_frequencies(vqv):
    """20000 blocks of one draft: first tokens come as often as the target has them (five standard
    deviations of each count)."""
    n, N = 20000, 6
    gen = torch.Generator().manual_seed(11)
    p, q = torch.tensor([0.3, 0.05, 0.25, 0.1, 0.2, 0.1]), torch.tensor([0.1, 0.3, 0.1, 0.3, 0.1, 0.1])
    c = Case(B=n, T=2, N=N, seed=11)
    c.logits = p.log().repeat(2 * n, 1)
    c.temperature = None
    c.probs = q.repeat(n, 1, 1)
    c.draft = torch.multinomial(q, n, replacement=True, generator=gen).view(n, 1).to(torch.int32)
    token, accept, _ = c.run(vqv)
    first = torch.where(accept.cpu() > 0, c.draft[:, 0], token.cpu())
    share = torch.bincount(first, minlength=N) / n
    assert ((share - p).abs() < 5 * (p * (1 - p) / n).sqrt()).all()


def test_streams_graphs_and_without_logprob(vqv):
    c = Case(B=4, T=5, N=50000, seed=12, near=1.0)
    token, accept, logp = c.run(vqv)
    again = c.run(vqv, stream=torch.cuda.Stream(), want_logprob=False)
    assert torch.equal(again[0], token) and torch.equal(again[1], accept) and again[2] is None
    args = [x.cuda() for x in (c.logits, c.draft, c.uniform)]
    probs, heat = c.probs.cuda(), c.temperature.cuda()
    out = [torch.empty_like(x) for x in (token, accept, logp)]
    ws = torch.empty(vqv.vqv_verify_sampled_workspace_bytes(4, 5, 50000), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vqv.vqv_verify_sampled(*args, 4, 5, draft_probs=probs, temperature=heat, token=out[0], accept_len=out[1],
                               logprob=out[2], workspace=ws)
    for _ in range(4):
        for x in out:
            x.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, (token, accept, logp)))


def test_after_edits(vqv):
    """Logits edited in place, then verified: what is masked is not drawn."""
    c = Case(B=2, T=3, N=4000, seed=13)
    words = torch.zeros(6, 125, dtype=torch.int32)
    words[:, 3] = -1                                # tokens 96 .. 127
    logits = c.logits.cuda()
    vqv.vqv_logits_edit(logits, vqv.Edits(2, 4000), c.draft.cuda(), 2, 3, mask=words.cuda(), out=logits)
    c.logits = logits.cpu()
    c.check(vqv)
    token, _, _ = c.run(vqv)
    assert ((token >= 96) & (token < 128)).all()


def test_refuses_wrong_tensors(vqv):
    c = Case(B=2, T=3, N=100)
    lg, d, u, q = c.logits.cuda(), c.draft.cuda(), c.uniform.cuda(), c.probs.cuda()
    for args in ((lg[:5], d, u), (lg.half(), d, u), (lg, d.long(), u), (lg, d[:, :1], u), (lg, d, u[:, :2]),
                 (lg, None, u), (lg, d, u.double()), (lg.cpu(), d, u), (lg.t().contiguous().t(), d, u)):
        with pytest.raises(ValueError):
            vqv.vqv_verify_sampled(*args, 2, 3)
    for kw in (dict(draft_probs=q[:, :1]), dict(draft_probs=q.half()), dict(temperature=torch.ones(3, device="cuda")),
               dict(draft_len=torch.ones(2, device="cuda")), dict(token=torch.empty(2, device="cuda"))):
        with pytest.raises(ValueError):
            vqv.vqv_verify_sampled(lg, d, u, 2, 3, **kw)
    with pytest.raises(vqv.VqvError):
        vqv.vqv_verify_sampled(lg, d, u, 2, 3, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,probs,uniform", [(1, False, 0.3), (2, True, 0.0), (2, True, 0.99), (2, False, 0.99)])
def test_more_chunks_than_threads(vqv, T, probs, uniform):
    """A vocabulary of more chunks (of 4096) than a draw has threads: a thread then has several."""
    N = 1024 * 4096 + 9001
    c = Case(B=1, T=T, N=N, probs=probs, seed=5, spread=1.0, near=0.2) if T == 1 else Case.__new__(Case)
    if T > 1:   # torch.multinomial has its limit at 2^24 categories; the draft is any token
        gen = torch.Generator().manual_seed(6)
        c.B, c.T, c.N, c.temperature, c.lens = 1, T, N, torch.tensor([0.8]), None
        c.logits = torch.randn(T, N, generator=gen)
        c.probs = torch.softmax(c.logits[:1] / 0.8 + 0.2 * torch.randn(1, N, generator=gen), 1)[None] if probs else None
        c.draft = torch.tensor([[N - 5]], dtype=torch.int32)
        c.uniform = torch.tensor([[uniform, 0.6180339]])
    else:
        c.uniform[:] = uniform
    tokens, accepts, logp, near = c.want()
    token, accept, got = c.run(vqv)
    assert accept.tolist() == accepts
    # borders are 2^-22 of the sum apart, 64-bit sums of 2^22 terms off by far less than one
    assert token.tolist() == tokens
    assert ((got.cpu().double() - logp).abs() <= 2.0 ** -24 * logp.abs() + 2.0 ** -36).all()
