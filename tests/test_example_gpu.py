"""The example runs the operators together; what it leaves behind is that of
one chunk over the tokens that it confirmed."""

import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "verify_round.py")


def test_verify_round_example():
    spec = importlib.util.spec_from_file_location("verify_round", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    prompt = np.random.default_rng(1).integers(0, ex.VOCAB, 21).tolist()
    model = ex.Model()
    plain, ones, _, _ = ex.decode(model, prompt, rounds=18, block=4)
    assert all(c == [1, 1] for c in ones)
    known = ex.i32(plain)
    known[:, ::5] = 0
    tokens, confirmed, cache, book = ex.decode(model, prompt, rounds=6, block=4, known=known)
    assert sum(c[0] for c in confirmed) > 10 and sum(c[1] for c in confirmed) > 10
    for b in range(2):
        n = min(len(tokens[b]), len(plain[b]))
        assert tokens[b][:n] == plain[b][:n]
    length = book.length.tolist()
    for b in range(2):
        n = len(tokens[b]) - 1            # the last choice has not been fed
        assert length[b] == n == len(prompt) - 1 + sum(c[b] for c in confirmed)
        assert book.held[b].item() == -(-n // ex.PAGE)
        # All of it as one chunk on a cache of its own.
        fresh = ex.new_cache(4)
        seqs = ex.vqv.Sequences(ex.i32([0, n]), ex.i32([n]), ex.i32([[2, 0, 3, 1]]), n_rows=n,
                                max_rows=n, max_kv=n)
        logits = model.logits(ex.i32(tokens[b][:n]), fresh, seqs)
        t = torch.arange(n)
        at = book.table[b].cpu()[t // ex.PAGE].long(), t % ex.PAGE
        own = torch.tensor([2, 0, 3, 1])[t // ex.PAGE], t % ex.PAGE
        for got, want in ((cache.k, fresh.k), (cache.v, fresh.v)):
            got, want = got[:, at[0], at[1]].float(), want[:, own[0], own[1]].float()
            # The projections differ by how their sums are cut, attention by its tiles: a few
            # roundings to bf16 (2^-8 each) of values around the largest of a head.
            assert ((got - want).abs() <= 6 * 2.0 ** -8 * want.abs().amax(-1, keepdim=True)).all()
        if b == 0:                        # no edits: the tokens are the greedy choices
            top = logits[len(prompt) - 1:].topk(2, 1)
            clear = top.values[:, 0] - top.values[:, 1] > 0.05 * logits.std()
            follow = torch.tensor(tokens[0][len(prompt):], device="cuda")
            assert clear.float().mean() > 0.5
            assert torch.equal(top.indices[clear[:, None].expand(-1, 2)].view(-1, 2)[:, 0], follow[clear])
    shared = book.ref.tolist().count(2)
    assert shared == (len(prompt) - 1) // ex.PAGE
