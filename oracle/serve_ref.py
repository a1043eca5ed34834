"""Oracle of the operators for batches of many requests, on the CPU in 64 bits.

Plain definitions, value by value where it is affordable; tensors are torch CPU
tensors. Shares no code with the library.
"""

from __future__ import annotations

import math

import torch


def record_bytes(dim):
    return -(-(dim // 2 + 4 * -(-dim // 32)) // 16) * 16


def _code_place(i):
    """(byte, shift) of value i's code."""
    word, at = i // 8, i % 8
    bit = 16 * (at % 2) + 4 * (at // 2)
    return 4 * word + bit // 8, bit % 8


def pack(x):
    """Records (uint8) of values [..., dim]: fp32 steps as the format says."""
    x = x.float()
    dim = x.shape[-1]
    rec = torch.zeros(*x.shape[:-1], record_bytes(dim), dtype=torch.uint8)
    x = torch.where(x > 32768.0, 32768.0, torch.where(x < -32768.0, -32768.0, x))
    for g in range(-(-dim // 32)):
        v = x[..., 32 * g:32 * g + 32]
        bad = v.isnan().any(-1)
        lo, hi = v.amin(-1), v.amax(-1)
        scale = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32)).half()
        bias = lo.half() + 0.0  # a zero is +0
        scale[bad] = bias[bad] = float("nan")
        s, b = scale.float()[..., None], bias.float()[..., None]
        code = torch.round((v - b) * (1.0 / s)).clamp(0, 15)
        code = torch.where(s > 0, code, 0.0).nan_to_num(0.0).to(torch.uint8)
        for i in range(v.shape[-1]):
            byte, shift = _code_place(32 * g + i)
            rec[..., byte] |= code[..., i] << shift
        at = dim // 2 + 4 * g
        rec[..., at:at + 2] = scale[..., None].contiguous().view(torch.uint8)
        rec[..., at + 2:at + 4] = bias[..., None].contiguous().view(torch.uint8)
    return rec


def unpack(rec, dim):
    """Values [..., dim] in 64 bits."""
    out = torch.empty(*rec.shape[:-1], dim, dtype=torch.float64)
    for i in range(dim):
        byte, shift = _code_place(i)
        at = dim // 2 + 4 * (i // 32)
        scale, bias = (rec[..., a:a + 2].contiguous().view(torch.float16)[..., 0].double() for a in (at, at + 2))
        out[..., i] = scale * (rec[..., byte] >> shift & 15).double() + bias
    return out


def target(row, temperature):
    """(probabilities, place of all of it or None) of one row of logits, in 64 bits."""
    x = row.double()
    p = torch.zeros_like(x)
    nan = x.isnan().nonzero()
    top = int(nan[0]) if nan.numel() else int((x == x.max()).nonzero()[0])
    if not temperature > 0 or nan.numel() or math.isinf(float(x[top])):
        p[top] = 1.0
        return p, top
    e = torch.where(x == -math.inf, 0.0, torch.exp((x - x[top]) / temperature))
    return e / e.sum(), None


def draw(r, u):
    """The lowest j with r_j > 0 whose running sum passes u times the sum, or the last with r_j > 0."""
    at = r.cumsum(0)
    held = (r > 0).nonzero()[:, 0].tolist()
    for j in held:
        if at[j] > u * at[-1]:
            return j
    return held[-1]


def verify_sampled(logits, draft, uniform, B, T, probs=None, temperature=None, draft_len=None):
    """Lists of tokens and accepted lengths, the committed tokens' log p [B, T] in 64 bits, and
    how near to a border the decisions came (relative, the least of all)."""
    N = logits.shape[1]
    tokens, accepts, near = [], [], math.inf
    logp = torch.zeros(B, T, dtype=torch.float64)
    for b in range(B):
        t = 1.0 if temperature is None else float(temperature[b])
        n = T - 1 if draft_len is None else min(max(int(draft_len[b]), 0), T - 1)
        r = None
        for i in range(n + 1):
            p, _ = target(logits[b * T + i], t)
            if i == n:
                r = p
                break
            d = int(draft[b, i])
            inside = 0 <= d < N
            q = torch.zeros_like(p)
            if probs is not None:
                q = probs[b, i].double()
            elif inside:
                q[d] = 1.0
            if inside:
                a, c = float(uniform[b, i]) * float(q[d]), float(p[d])
                if 0 < c < 1:
                    near = min(near, abs(a - c) / c)
                if a < c:
                    logp[b, i] = math.log(c)
                    continue
            r = torch.where(p > q, p - q, 0.0)
            if not (r > 0).any():
                r = p
            break
        u = float(uniform[b, T - 1])
        j = draw(r, u)
        at = r.cumsum(0) / r.sum()
        near = min(near, float((at - u).abs().min()) if (r > 0).sum() > 1 else math.inf)
        tokens.append(j)
        accepts.append(i)
        logp[b, i] = math.log(float(p[j]))
    return tokens, accepts, logp, near


def lora_add(x, a, b, scale, which, y, ranks=None):
    """(out in 64 bits, sums of absolute products: of the first product's terms and of all)."""
    out, size = y.double().clone(), y.double().abs()
    for m, e in enumerate(which.tolist()):
        if not 0 <= e < a.shape[0]:
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[e]), 0), a.shape[1])
        A, B = a[e, :r].double(), b[e, :, :r].double()
        out[m] += float(scale[e]) * (B @ (A @ x[m].double()))
        size[m] += abs(float(scale[e])) * (B.abs() @ (A.abs() @ x[m].double().abs()))
    return out, size
