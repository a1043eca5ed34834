"""The example runs the operators for many requests together; what it leaves
behind is that of one chunk per request over the tokens that it committed, and
the probabilities are those of that chunk's logits."""

import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_round.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("serve_round", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rounds(ex):
    rng = np.random.default_rng(2)
    prompts = [rng.integers(0, ex.VOCAB, n).tolist() for n in (21, 9, 40)]
    model = ex.Model()
    tokens, logs, accepted, cache, book = ex.decode(model, prompts, rounds=10, block=4)
    assert sum(sum(a) for a in accepted) > 0
    for b, t in enumerate(tokens):
        n = len(t) - 1                     # the last token has not been fed
        assert n == book.length[b].item() == len(prompts[b]) - 1 + sum(a[b] + 1 for a in accepted)
        assert book.held[b].item() == -(-n // ex.PAGE)
        assert len(logs[b]) == len(t) - len(prompts[b])
        fresh = ex.new_cache(8)
        table = ex.i32([[3, 1, 0, 2, 6, 4, 7, 5]])
        seqs = ex.vqv.Sequences(ex.i32([0, n]), ex.i32([n]), table, n_rows=n, max_rows=n, max_kv=n)
        logits = model.logits(ex.i32(t[:n]), ex.i32([ex.ADAPTER[b]] * n), fresh, seqs)
        own = ex.vqv.Sequences(ex.i32([0, n]), ex.i32([n]), book.table[b:b + 1], n_rows=n, max_rows=n, max_kv=n)
        # Layer 0's keys and values go by the tokens and the adapter alone: the projections differ by how
        # their sums are cut, so that a code next to a border is another one: a step, a fifteenth of
        # what its group spans, in a value of a thousand at most.
        for got, want in zip(ex.vqv.vqv_cache_q4_read(cache, own), ex.vqv.vqv_cache_q4_read(fresh, seqs)):
            span = want.unflatten(2, (2, 32))
            step = ((span.amax(3) - span.amin(3)) / 15).repeat_interleave(32, 2)
            err = (got - want).abs()
            assert (err <= 1.02 * step + 1e-3).all()
            assert (err > 0.5 * step).float().mean() < 1e-3
        # Log p of what was committed, from the chunk's logits: behind a 4-bit cache (above) and
        # projections and attention rounded to bf16 a logit is off by a few hundredths of the logits' spread.
        x = logits[len(prompts[b]) - 1:].double()
        spread = x.std().item()
        if b == 0:
            x[:, 7] = -1e4
            best = x.max(1).values - x.gather(1, torch.tensor(t[len(prompts[b]):], device="cuda")[:, None])[:, 0]
            assert (best <= 0.1 * spread).all() and logs[0] == [0.0] * len(logs[0])
            assert 7 not in t[len(prompts[b]):]
        else:
            heat = ex.TEMPERATURE[b]
            p = torch.log_softmax(x / heat, 1).gather(1, torch.tensor(t[len(prompts[b]):], device="cuda")[:, None])[:, 0]
            assert ((p.cpu() - torch.tensor(logs[b])).abs() <= 0.1 * spread / heat + 0.02).all()


def test_rounds_in_a_graph(ex):
    """A round's calls captured once: replays with other inputs give what eager calls give."""
    vqv, model = ex.vqv, ex.Model()
    B, T, n = 3, 4, 30
    table = ex.i32([[4 * b, 4 * b + 1, 4 * b + 2, 4 * b + 3] for b in range(B)])
    start, kv_len = ex.i32([b * T for b in range(B + 1)]), ex.i32([n + 2 * b for b in range(B)])
    which = ex.i32([ex.ADAPTER[b] for b in range(B) for _ in range(T)])
    cache = ex.new_cache(4 * B)
    seqs = vqv.Sequences(start, kv_len, table, n_rows=B * T, max_rows=T, max_kv=64)
    tokens, uniform = torch.zeros(B * T, dtype=torch.int32, device="cuda"), torch.zeros(B, T, device="cuda")
    draft = torch.zeros(B, T - 1, dtype=torch.int32, device="cuda")
    heat = torch.tensor(ex.TEMPERATURE, device="cuda")
    outs = [torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"),
            torch.empty(B, T, device="cuda")]

    def round_():
        logits = model.logits(tokens, which, cache, seqs)
        return vqv.vqv_verify_sampled(logits, draft, uniform, B, T, temperature=heat)

    def inputs(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        tokens.copy_(torch.randint(0, ex.VOCAB, (B * T,), generator=g, device="cuda"))
        draft.copy_(tokens.view(B, T)[:, 1:])
        uniform.copy_(torch.rand(B, T, generator=g, device="cuda"))

    inputs(0)
    round_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o, r in zip(outs, round_()):
            o.copy_(r)
    for seed in range(1, 5):
        inputs(seed)
        graph.replay()
        got = [o.clone() for o in outs]
        want = round_()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_two_streams_at_once(ex):
    """Calls on two streams with workspaces of their own do not disturb one another."""
    vqv = ex.vqv
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    logits = [3 * torch.randn(16, 50000, generator=g, device="cuda") for _ in range(2)]
    draft = [torch.randint(0, 50000, (4, 3), generator=g, device="cuda").to(torch.int32) for _ in range(2)]
    uniform = [torch.rand(4, 4, generator=g, device="cuda") for _ in range(2)]
    want = [vqv.vqv_verify_sampled(l, d, u, 4, 4) for l, d, u in zip(logits, draft, uniform)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(vqv.vqv_verify_sampled(logits[i], draft[i], uniform[i], 4, 4, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))
