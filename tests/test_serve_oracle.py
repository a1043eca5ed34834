"""The oracle of the operators for batches of many requests against values
worked out by hand, and planted mistakes that it tells apart."""

import math

import pytest
import torch

from oracle import serve_ref as ref


def test_record_by_hand():
    """Values 0 .. 15 twice in the first group: scale 1, bias 0, codes as they are."""
    x = torch.zeros(64)
    x[:32] = torch.arange(32) % 16
    x[32:] = 3.0
    rec = ref.pack(x)
    assert rec.numel() == 48
    # word 0: value 2i + j in bits 16j + 4i: values 0 2 4 6 | 1 3 5 7
    assert rec[:8].tolist() == [0x20, 0x64, 0x31, 0x75, 0xA8, 0xEC, 0xB9, 0xFD]
    assert rec[16:32].tolist() == [0] * 16          # a group of one value: scale 0, codes 0
    meta = rec[32:40].view(torch.float16).tolist()
    assert meta == [1.0, 0.0, 0.0, 3.0]
    assert rec[40:].tolist() == [0] * 8
    assert torch.equal(ref.unpack(rec, 64), x.double())


@pytest.mark.parametrize("dim", [64, 80, 96, 128, 192, 256])
def test_records_hold_values_to_half_a_step(dim):
    x = torch.randn(50, dim, generator=torch.Generator().manual_seed(dim))
    got = ref.unpack(ref.pack(x), dim)
    for g in range(0, dim, 32):
        v = x[:, g:g + 32].double()
        step = (v.amax(1) - v.amin(1)) / 15
        # half a step, and the fp16 roundings of scale (15 times) and bias
        allow = step * (0.5 + 15 * 2.0 ** -11) + v.abs().amax(1) * 2.0 ** -11 + 1e-6
        assert ((got[:, g:g + 32] - v).abs().amax(1) <= allow).all()


def test_records_of_extremes():
    x = torch.zeros(3, 64)
    x[0, 3], x[0, 40] = math.nan, math.inf
    x[1, 0], x[1, 1] = 1e30, -1e30
    x[2, :32] = 1e-6 * torch.arange(32)     # scale rounds to a subnormal
    got = ref.unpack(ref.pack(x), 64)
    assert got[0, :32].isnan().all() and got[0, 32:].isfinite().all()
    assert abs(got[0, 40] - 32768) <= 16 and abs(got[1, 0] - 32768) <= 30 and got[1, 1] == -32768
    assert (got[2, :32] - x[2, :32].double()).abs().max() < 2e-6


def logits_of(p):
    return torch.tensor(p, dtype=torch.float64).log().float()


def test_draws_by_hand():
    p = [[0.5, 0.25, 0.25], [0.1, 0.2, 0.7]]
    q = torch.tensor([[[0.2, 0.8, 0.0]]])
    x = logits_of(p)
    call = lambda u, d, **kw: ref.verify_sampled(x, torch.tensor([[d]]), torch.tensor([u]), 1, 2, **kw)[:2]
    # draft 1: accepted where u * 0.8 < 0.25; then the second row's sums 0.1, 0.3, 1
    assert call([0.3, 0.05], 1, probs=q) == ([0], [1])
    assert call([0.3, 0.25], 1, probs=q) == ([1], [1])
    assert call([0.3, 0.31], 1, probs=q) == ([2], [1])
    # rejected: r = 0.3, 0, 0.25
    assert call([0.4, 0.5], 1, probs=q) == ([0], [0])
    assert call([0.4, 0.56], 1, probs=q) == ([2], [0])
    # a draft that was not drawn is accepted with its probability, and is not drawn behind that
    assert call([0.24, 0.0], 1) == ([0], [1])
    assert call([0.26, 0.66], 1) == ([0], [0])
    assert call([0.26, 0.67], 1) == ([2], [0])
    # no valid draft: a draw from the first row
    assert call([0.0, 0.51], 1, draft_len=[0]) == ([1], [0])
    # greedy
    assert call([0.99, 0.3], 0, temperature=[0.0]) == ([2], [1])
    assert call([0.0, 0.3], 1, temperature=[0.0]) == ([0], [0])
    # a token that is none
    assert call([0.0, 0.6], 7) == ([1], [0])


def test_drawn_as_the_target_alone():
    """Over a grid of random numbers the first committed token has the target's frequencies."""
    p, q = torch.tensor([0.1, 0.6, 0.3]), torch.tensor([0.5, 0.3, 0.2])
    n, seen = 40, torch.zeros(3, dtype=torch.float64)
    x = logits_of([p.tolist(), [0.3, 0.3, 0.4]])
    for d in range(3):
        for a in range(n):
            for c in range(n):
                u = torch.tensor([[(a + 0.5) / n, (c + 0.5) / n]])
                t, l, _, _ = ref.verify_sampled(x, torch.tensor([[d]]), u, 1, 2, probs=q.view(1, 1, 3))
                seen[d if l[0] else t[0]] += float(q[d]) / n / n
    assert (seen - p.double()).abs().max() < 1.5 / n


def test_rows_of_nothing_and_infinities():
    inf, nan = math.inf, math.nan
    for row, at in (([-inf] * 4, 0), ([1, nan, 2, nan], 1), ([0, inf, inf, 1], 1)):
        p, hot = ref.target(torch.tensor(row, dtype=torch.float32), 1.0)
        assert hot == at and p.tolist() == [float(j == at) for j in range(4)]


def test_lora_by_hand():
    a = torch.zeros(2, 8, 8)
    b = torch.zeros(2, 3, 8)
    a[1, 0, 2], b[1, 1, 0], a[1, 5, 3], b[1, 2, 5] = 2.0, 3.0, 1.0, 10.0
    x = torch.arange(16.0).view(2, 8)
    y = torch.ones(2, 3)
    out, _ = ref.lora_add(x, a, b, torch.tensor([1.0, 0.5]), torch.tensor([1, -1]), y)
    assert out.tolist() == [[1, 1 + 0.5 * 12, 1 + 0.5 * 30], [1, 1, 1]]
    out, _ = ref.lora_add(x, a, b, torch.tensor([1.0, 0.5]), torch.tensor([1, 2]), y, ranks=torch.tensor([8, 5]))
    assert out.tolist() == [[1, 7, 1], [1, 1, 1]]
