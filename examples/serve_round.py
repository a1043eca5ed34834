"""Rounds of decoding for requests of different kinds in one batch, on a small random model.

    python examples/serve_round.py [rounds]

Three requests with prompts of their own share every call although each has an adapter (or none), a temperature (or
is greedy) and a history of its own in a 4-bit cache. Each round feeds a block of rows per request (the last committed
token and drafts), and takes the drafts that sampling accepts:

  W4 projection + vqv_lora_add -> vqv_rope_append_q4 -> vqv_paged_attn_q4 -> W4 projections (SwiGLU) on every layer,
  the vocabulary projection -> vqv_logits_edit -> vqv_verify_sampled, and at the end vqv_cache_compact (on the
  4-bit records), vqv_cache_trim and vqv_cache_reserve.

The drafter is a fixed distribution over the vocabulary: it is seldom right, and what comes out is distributed as
the target alone would draw it all the same. Nothing is copied to the host before the last round has run.
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gen  # noqa: E402
import w4_gemm_vqv_amd as vqv  # noqa: E402

VOCAB, HIDDEN, FFN, LAYERS = 200, 256, 512, 2
HEADS, KV_HEADS, DIM, PAGE, RANK = 8, 2, 64, 16, 8
ADAPTER = [-1, 1, 0]                 # of each request; -1: none
TEMPERATURE = [0.0, 0.8, 1.5]        # 0: greedy
QKV = (HEADS + 2 * KV_HEADS) * DIM


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Weight:
    """A random W4 weight of the library's layout."""

    def __init__(self, rng, n, k):
        codes, scales, biases = gen.make_weights(rng, n, k)
        self.parts = (torch.from_numpy(codes).cuda(),
                      *(torch.from_numpy(x.view(np.int16)).view(torch.float16).cuda() for x in (scales, biases)))

    def __call__(self, x):
        # A call takes 64 rows at most.
        return torch.cat([vqv.vqv_qgemm(x[i:i + 64].contiguous(), *self.parts) for i in range(0, len(x), 64)])


class Model:
    def __init__(self, seed=0):
        rng = np.random.default_rng(seed)

        def normal(*shape, size=1.0):
            return (size * torch.from_numpy(rng.standard_normal(shape).astype(np.float32))).cuda()

        self.embed = normal(VOCAB, HIDDEN)
        self.layers = [dict(qkv=Weight(rng, QKV, HIDDEN), out=Weight(rng, HIDDEN, HEADS * DIM),
                            up=Weight(rng, 2 * FFN, HIDDEN), down=Weight(rng, HIDDEN, FFN),
                            adapters=vqv.Adapters(normal(2, RANK, HIDDEN, size=HIDDEN ** -0.5).bfloat16(),
                                                  normal(2, QKV, RANK).bfloat16(),
                                                  torch.tensor([0.5, 1.0], device="cuda"))) for _ in range(LAYERS)]
        self.head = Weight(rng, VOCAB, HIDDEN)
        self.rope = vqv.Rope(DIM, 10000.0)

    @staticmethod
    def norm(h):
        return (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def logits(self, tokens, which, cache, seqs):
        """fp32 logits of the rows' tokens, of which row r's request has adapter which[r]; their keys
        and values join the cache."""
        h = self.embed[tokens.long()]
        for l, w in enumerate(self.layers):
            x = self.norm(h)
            qkv = w["qkv"](x)
            vqv.vqv_lora_add(x, w["adapters"], which, qkv, out=qkv)
            q, k, v = qkv.unflatten(1, (HEADS + 2 * KV_HEADS, DIM)).split([HEADS, KV_HEADS, KV_HEADS], 1)
            q = vqv.vqv_rope_append_q4(q, k, v, cache, seqs, self.rope, layer=l)
            o = vqv.vqv_paged_attn_q4(q, cache, seqs, scale=DIM ** -0.5, layer=l)
            h = h + w["out"](o.flatten(1))
            g = torch.cat([vqv.vqv_qgemm_swiglu(x.contiguous(), *w["up"].parts) for x in self.norm(h).split(64)])
            h = h + w["down"](self.norm(g))
        return self.head(self.norm(h))


def new_cache(pages):
    shape = (LAYERS, pages, PAGE, KV_HEADS, vqv.vqv_q4_record_bytes(DIM))
    return vqv.PagedCacheQ4(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)), DIM)


def decode(model, prompts, rounds, block=4, width=32, seed=0):
    """Per request its tokens (the prompt in front) and the log p of those it committed; the drafts accepted per
    round; the cache and its book."""
    B, pages = len(prompts), len(prompts) * width
    gen_ = torch.Generator(device="cuda")
    gen_.manual_seed(seed)
    cache = new_cache(pages)
    book = vqv.Pages(i32([0] * pages), i32([[-1] * width] * B), i32([0] * B), i32([0] * B), page_size=PAGE)
    heat = torch.tensor(TEMPERATURE[:B], device="cuda")

    # The prompts, but for their last tokens, as chunks of one call.
    n = [len(p) - 1 for p in prompts]
    lens = i32(n)
    assert vqv.vqv_cache_reserve(book, lens).tolist() == [1] * B
    start = [sum(n[:b]) for b in range(B + 1)]
    seqs = vqv.Sequences(i32(start), lens, book.table, n_rows=start[-1], max_rows=max(n), max_kv=max(n))
    which = i32([ADAPTER[b] for b in range(B) for _ in range(n[b])])
    model.logits(i32([t for p in prompts for t in p[:-1]]), which, cache, seqs)
    book.length.copy_(lens)

    kv_len, ok = torch.empty_like(book.length), torch.empty_like(book.length)
    seqs = vqv.Sequences(i32([b * block for b in range(B + 1)]), kv_len, book.table, n_rows=B * block,
                         max_rows=block, max_kv=max(n) + rounds * block)
    which = i32([ADAPTER[b] for b in range(B) for _ in range(block)])
    rows = torch.arange(block, device="cuda")
    edits = vqv.Edits(B, VOCAB, bias_start=i32([0] + [1] * B), bias_token=i32([7]),
                      bias_value=torch.tensor([-1e4], device="cuda"))       # request 0 never says token 7
    drafter = torch.softmax(torch.randn(VOCAB, generator=gen_, device="cuda"), 0)
    probs = drafter.expand(B, block - 1, VOCAB).contiguous()
    last = i32([p[-1] for p in prompts])
    history, accepted, logs, good = [], [], [], []
    for _ in range(rounds):
        draft = torch.multinomial(drafter, B * (block - 1), replacement=True, generator=gen_)
        draft = draft.view(B, block - 1).to(torch.int32)
        tokens = torch.cat([last[:, None], draft], 1)
        kv_len.copy_(book.length + block)
        good.append(vqv.vqv_cache_reserve(book, kv_len, ok=ok).clone())
        logits = model.logits(tokens.flatten(), which, cache, seqs)
        vqv.vqv_logits_edit(logits, edits, draft, B, block, out=logits)
        uniform = torch.rand(B, block, generator=gen_, device="cuda")
        last, accept, logp = vqv.vqv_verify_sampled(logits, draft, uniform, B, block, draft_probs=probs,
                                                    temperature=heat)
        # Row 0 and the accepted drafts stay.
        keep = (rows[None, :] <= accept[:, None]).to(torch.int32).flatten()
        vqv.vqv_cache_compact(cache.records, seqs, keep, new_len=book.length)
        vqv.vqv_cache_trim(book, book.length)
        fresh = torch.where(rows[None, :] == accept[:, None], last[:, None],
                            torch.nn.functional.pad(draft, (0, 1)))
        history.append(torch.where(rows[None, :] <= accept[:, None], fresh, VOCAB))
        accepted.append(accept)
        logs.append(logp)
    assert torch.stack(good).all(), "the cache ran out of pages"
    out, out_logs = [], []
    for b in range(B):
        chosen, log = (torch.cat([x[b] for x in list_]) for list_ in (history, logs))
        out.append(list(prompts[b]) + chosen[chosen < VOCAB].tolist())
        out_logs.append(log[chosen < VOCAB].tolist())
    return out, out_logs, torch.stack(accepted).tolist(), cache, book


def main():
    rounds = int(sys.argv[1]) if len(sys.argv) > 1 else 12
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (21, 9, 40)]
    tokens, logs, accepted, _, book = decode(Model(), prompts, rounds)
    for b, t in enumerate(tokens):
        print(f"request {b} (adapter {ADAPTER[b]}, temperature {TEMPERATURE[b]}): accepted per round "
              f"{[a[b] for a in accepted]}, mean log p {np.mean(logs[b]):.2f}")
        print("  " + " ".join(str(x) for x in t[len(prompts[b]):]))
    print(f"pages held {book.held.tolist()}, lengths {book.length.tolist()}")


if __name__ == "__main__":
    main()
