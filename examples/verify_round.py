"""Block-wise decoding with the library's operators, on a small random model.

    python examples/verify_round.py [rounds]

Two sequences share a prompt: it is computed once and the second sequence is a
fork of the first. Each round then feeds a block of rows per sequence (the last
confirmed token and guesses for what follows), and the target confirms as many
of the guesses as its own greedy choice agrees with:

  W4 projection -> vqv_rope_append -> vqv_paged_attn -> W4 projections (SwiGLU)
  on every layer, the vocabulary projection -> vqv_logits_verify, and at the end
  vqv_cache_compact, vqv_cache_trim and vqv_cache_reserve.

A first pass guesses nothing and confirms a token a round; a second one takes
its guesses from the first pass' tokens, every fifth of them spoilt, and ends
at the same tokens in fewer rounds. Nothing is copied to the host before the
last round has run.
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gen  # noqa: E402
import w4_gemm_vqv_amd as vqv  # noqa: E402

VOCAB, HIDDEN, FFN, LAYERS = 1000, 256, 512, 2
HEADS, KV_HEADS, DIM, PAGE = 4, 2, 64, 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Weight:
    """A random W4 weight of the library's layout."""

    def __init__(self, rng, n, k):
        codes, scales, biases = gen.make_weights(rng, n, k)
        self.parts = (torch.from_numpy(codes).cuda(),
                      *(torch.from_numpy(x.view(np.int16)).view(torch.float16).cuda()
                        for x in (scales, biases)))

    def __call__(self, x):
        return vqv.vqv_qgemm(x, *self.parts)


class Model:
    def __init__(self, seed=0):
        rng = np.random.default_rng(seed)
        self.embed = torch.from_numpy(rng.standard_normal((VOCAB, HIDDEN)).astype(np.float32)).cuda()
        self.layers = [dict(qkv=Weight(rng, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN),
                            out=Weight(rng, HIDDEN, HEADS * DIM), up=Weight(rng, 2 * FFN, HIDDEN),
                            down=Weight(rng, HIDDEN, FFN)) for _ in range(LAYERS)]
        self.head = Weight(rng, VOCAB, HIDDEN)
        self.rope = vqv.Rope(DIM, 10000.0)

    @staticmethod
    def norm(h):
        return (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def logits(self, tokens, cache, seqs):
        """fp32 logits of the rows' tokens; their keys and values join the cache."""
        h = self.embed[tokens.long()]
        for l, w in enumerate(self.layers):
            qkv = w["qkv"](self.norm(h)).unflatten(1, (HEADS + 2 * KV_HEADS, DIM))
            q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
            q = vqv.vqv_rope_append(q, k, v, cache, seqs, self.rope, layer=l)
            o = vqv.vqv_paged_attn(q, cache, seqs, scale=DIM ** -0.5, layer=l)
            h = h + w["out"](o.flatten(1))
            g = vqv.vqv_qgemm_swiglu(self.norm(h), *w["up"].parts)
            h = h + w["down"](self.norm(g))
        return self.head(self.norm(h))


def new_cache(pages):
    shape = (LAYERS, pages, PAGE, KV_HEADS, DIM)
    return vqv.PagedCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))


def edits_of(n_seqs):
    """Sequence 0 as it is, sequence 1 with a penalty for repeated tokens and a biased token."""
    counts = torch.zeros(n_seqs, VOCAB, dtype=torch.int32, device="cuda")
    one = lambda a: torch.tensor([0.0, a], device="cuda")
    return counts, vqv.Edits(n_seqs, VOCAB, counts=counts, repetition=1.0 + one(0.2),
                             presence=one(0.1), bias_start=i32([0, 0, 1]), bias_token=i32([7]),
                             bias_value=torch.tensor([0.5], device="cuda"))


def decode(model, prompt, rounds, block=8, width=32, known=None):
    """Tokens of both sequences (their prompt in front), confirmed per round, and the cache with
    its book. known [2, any] int32 holds guesses for the tokens at each position."""
    B, pages = 2, 2 * width
    cache = new_cache(pages)
    book = vqv.Pages(i32([0] * pages), i32([[-1] * width] * B), i32([0] * B), i32([0] * B), page_size=PAGE)
    counts, edits = edits_of(B)

    # The prompt, but for its last token, as one chunk of sequence 0; then the fork.
    n = len(prompt) - 1
    assert vqv.vqv_cache_reserve(book, i32([n])).tolist() == [1]
    seqs = vqv.Sequences(i32([0, n]), i32([n]), book.table, n_rows=n, max_rows=n, max_kv=n)
    model.logits(i32(prompt[:n]), cache, seqs)
    book.length[0] = n
    assert vqv.vqv_cache_fork(cache, book, i32([0]), i32([1])).tolist() == [1]
    counts += torch.bincount(torch.tensor(prompt, device="cuda"), minlength=VOCAB).to(torch.int32)

    most = n + rounds * block
    rows = torch.arange(block, device="cuda")
    kv_len, ok = torch.empty_like(book.length), torch.empty_like(book.length)
    seqs = vqv.Sequences(i32([0, block, 2 * block]), kv_len, book.table, n_rows=B * block,
                         max_rows=block, max_kv=most)
    tokens = i32([[prompt[-1]] * block] * B)
    history, confirmed, good = [], [], []
    for _ in range(rounds):
        kv_len.copy_(book.length + block)
        good.append(vqv.vqv_cache_reserve(book, kv_len, ok=ok).clone())
        logits = model.logits(tokens.flatten(), cache, seqs)
        draft = tokens[:, 1:].contiguous()
        choice, accept, _ = vqv.vqv_logits_verify(logits, edits, draft, B, block, want_margin=False)
        # Row 0 and the confirmed drafts stay.
        keep = (rows[None, :] <= accept[:, None]).to(torch.int32).flatten()
        vqv.vqv_cache_compact(cache, seqs, keep, new_len=book.length)
        vqv.vqv_cache_trim(book, book.length)
        choice = choice.view(B, block)
        fresh = torch.where(rows[None, :] <= accept[:, None], choice, VOCAB)
        counts.copy_((torch.zeros(B, VOCAB + 1, dtype=torch.int32, device="cuda").scatter_add_(
            1, fresh.long(), torch.ones_like(fresh)))[:, :VOCAB] + counts)
        history.append(fresh)
        confirmed.append(accept + 1)
        # The next block: the choice after the last confirmed row, then guesses.
        tokens = choice.gather(1, accept[:, None].long()).expand(B, block)
        if known is not None:
            at = (book.length[:, None] + rows[None, :]).clamp(max=known.shape[1] - 1)
            tokens = torch.where(rows[None, :] > 0, known.gather(1, at.long()), tokens)
    assert torch.stack(good).all(), "the cache ran out of pages"
    out = []
    for b in range(B):
        chosen = torch.cat([h[b] for h in history])
        out.append(list(prompt) + chosen[chosen < VOCAB].tolist())
    return out, torch.stack(confirmed).tolist(), cache, book


def main():
    rounds = int(sys.argv[1]) if len(sys.argv) > 1 else 12
    prompt = np.random.default_rng(1).integers(0, VOCAB, 21).tolist()
    model = Model()
    first, _, _, _ = decode(model, prompt, rounds)
    known = i32(first)
    known[:, ::5] = 0
    tokens, confirmed, _, book = decode(model, prompt, rounds // 3 + 1, known=known)
    for b, (t, plain) in enumerate(zip(tokens, first)):
        n = min(len(t), len(plain))
        print(f"sequence {b}: confirmed per round {[c[b] for c in confirmed]}, "
              f"{'the same' if t[:n] == plain[:n] else 'other'} tokens as one at a time:")
        print("  " + " ".join(str(x) for x in t[len(prompt):n]))
    print(f"pages held {book.held.tolist()}, lengths {book.length.tolist()}, "
          f"{int((book.ref > 1).sum())} pages shared")


if __name__ == "__main__":
    main()
