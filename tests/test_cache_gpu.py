"""The page operators against the oracle's book of lists: every table, count
and stored value is exactly equal."""

import pytest
import torch

from oracle import round_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vqv():
    import w4_gemm_vqv_amd as v
    v.lib()
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def storage(layers, pages, ps, hk, dim, dtype, layout, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pages, ps, hk, dim)
    if layout == "head":
        shape = (layers, pages, hk, ps, dim)
    if layout == "gap":
        shape = (layers, pages, ps + 1, hk, dim + 8)
    if layout == "pages first":
        shape = (pages, layers, ps, hk, dim)
    x = torch.randint(-32768, 32767, shape, generator=gen, device="cuda", dtype=torch.int16).view(dtype)
    if layout == "head":
        return x.transpose(2, 3)
    if layout == "gap":
        return x[:, :, :ps, :, :dim]
    return x.transpose(0, 1) if layout == "pages first" else x


SHAPES = [(1, 16, 2, 64, torch.bfloat16, "slot"), (3, 8, 1, 8, torch.float16, "head"),
          (2, 20, 3, 80, torch.float16, "head"), (2, 5, 2, 96, torch.bfloat16, "gap"),
          (2, 1, 4, 256, torch.bfloat16, "slot"), (3, 64, 2, 128, torch.bfloat16, "pages first")]


def bits(x):
    return x.contiguous().view(torch.int16).cpu()


def pair(vqv, shape, pages):
    layers, ps, hk, dim, dtype, layout = shape
    return vqv.PagedCache(*(storage(layers, pages, ps, hk, dim, dtype, layout, s) for s in (1, 2)))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("n", [0, 1, 7])
def test_copy(vqv, shape, n):
    cache = pair(vqv, shape, 20)
    want = [bits(x) for x in (cache.k, cache.v)]
    order = torch.randperm(20, generator=torch.Generator().manual_seed(3)).tolist()
    src, dst = order[:n], order[n:2 * n]
    for x in want:
        for a, b in zip(src, dst):
            x[:, b] = x[:, a]
    # pairs that name no page are left out
    vqv.vqv_cache_copy(cache, i32(src + [-1, 20, 1 << 30, 3]), i32(dst + [order[15], order[16], 2, -5]))
    torch.cuda.synchronize()
    for got, w in zip((cache.k, cache.v), want):
        assert torch.equal(bits(got), w)


def test_copy_far(vqv):
    """Pages whose place passes 2^32 values."""
    k = torch.zeros((1, 36000, 64, 8, 256), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, 1], v[0, 35999] = 3.0, 5.0
    vqv.vqv_cache_copy(vqv.PagedCache(k, v), i32([1, 35999]), i32([35998, 0]))
    torch.cuda.synchronize()
    assert (k[0, 35998] == 3).all() and (v[0, 0] == 5).all() and not k[0, 35997].any()


def random_book(seed, rows, width, ps, pages, spare_rows=0, partial=True):
    gen = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=gen).tolist()
    table = [[-1] * width for _ in range(rows + spare_rows)]
    held, length, refs = [0] * (rows + spare_rows), [0] * (rows + spare_rows), [0] * pages
    for r in range(rows):
        held[r] = int(torch.randint(0, min(width, len(order)) + 1, (1,), generator=gen))
        held[r] = min(held[r], max(pages // rows - 1, 0))
        for j in range(held[r]):
            table[r][j] = order.pop()
            refs[table[r][j]] = 1
        top = held[r] * ps
        length[r] = max(top - int(torch.randint(0, 2 * ps, (1,), generator=gen)), 0) if partial else top
    return ref.Book(refs, table, held, length, ps)


class Device:
    def __init__(self, vqv, book):
        self.t = [i32(x) for x in (book.ref, book.table, book.held, book.length)]
        self.pages = vqv.Pages(*self.t, page_size=book.ps)

    def check(self, book):
        torch.cuda.synchronize()
        for got, want, name in zip(self.t, (book.ref, book.table, book.held, book.length),
                                   ("ref", "table", "held", "length")):
            assert got.tolist() == want, name


@pytest.mark.parametrize("ps", [1, 16, 20])
@pytest.mark.parametrize("rows,width,pages", [(1, 1, 2), (5, 12, 50), (40, 70, 2500), (1500, 3, 9000)])
def test_trim_and_reserve(vqv, rows, width, pages, ps):
    gen = torch.Generator().manual_seed(rows + ps)
    book = random_book(rows + 7 * ps, rows, width, ps, pages)
    dev = Device(vqv, book)
    for step in range(3):
        keep = torch.randint(-5, width * ps + 5, (rows,), generator=gen).tolist()
        vqv.vqv_cache_trim(dev.pages, i32(keep))
        book.trim(keep)
        dev.check(book)
        goal = torch.randint(-3, width * ps + 2 * step, (rows,), generator=gen).tolist()
        ok = vqv.vqv_cache_reserve(dev.pages, i32(goal))
        assert book.reserve(goal) == ok.tolist()
        dev.check(book)


def test_trim_named_rows(vqv):
    book = random_book(4, 6, 8, 16, 60)
    dev = Device(vqv, book)
    vqv.vqv_cache_trim(dev.pages, i32([0, 20, 5, 7]), rows=i32([3, 1, -1, 6]))
    book.trim([0, 20, 5, 7], [3, 1, -1, 6])
    dev.check(book)
    # a row that is named twice gives its pages back once
    vqv.vqv_cache_trim(dev.pages, i32([0, 0, 0]), rows=i32([2, 2, 2]))
    book.trim([0, 0, 0], [2, 2, 2])
    dev.check(book)


@pytest.mark.parametrize("order", ["as drawn", "rising", "falling"])
def test_trim_rows_named_with_other_lengths(vqv, order):
    """A row that is named several times is cut to the shortest of its lengths, whatever the order."""
    for seed in range(20):
        gen = torch.Generator().manual_seed(seed)
        book = random_book(seed, 6, 40, 4, 400)
        dev = Device(vqv, book)
        keep = torch.randint(60, 170, (600,), generator=gen)
        if order != "as drawn":
            keep = keep.sort(descending=order == "falling").values
        rows = torch.randint(-1, 7, (600,), generator=gen).tolist()
        vqv.vqv_cache_trim(dev.pages, keep.to(torch.int32).cuda(), rows=i32(rows))
        book.trim(keep.tolist(), rows)
        dev.check(book)


def test_trim_bad_pages(vqv):
    """Entries that name no page leave the table and touch nothing."""
    book = ref.Book([1, 1, 0], [[0, 99, -7, 1]], [4], [60], 16)
    dev = Device(vqv, book)
    vqv.vqv_cache_trim(dev.pages, i32([5]))
    book.trim([5])
    dev.check(book)
    assert book.ref == [1, 0, 0]


def test_reserve_runs_out(vqv):
    """Rows are served in order while the free pages reach; a goal wider than
    the table takes none."""
    book = ref.Book([1, 0, 0, 1, 0], [[0, -1, -1], [-1] * 3, [3, -1, -1], [-1] * 3], [1, 0, 1, 0],
                    [4, 0, 4, 0], 4)
    dev = Device(vqv, book)
    goal = [13, 8, 12, 4]
    ok = vqv.vqv_cache_reserve(dev.pages, i32(goal))
    assert ok.tolist() == book.reserve(goal) == [0, 1, 0, 0]
    dev.check(book)
    ok = vqv.vqv_cache_reserve(dev.pages, i32([4, 12]))
    assert ok.tolist() == book.reserve([4, 12]) == [1, 1]
    dev.check(book)


@pytest.mark.parametrize("pages", [40000, 70001])
def test_reserve_many_pages(vqv, pages):
    """More pages than one step of the scan, the free ones far apart."""
    refs = [1] * pages
    for p in (5, 16383, 16384, 39999, pages - 1):
        refs[p] = 0
    book = ref.Book(refs, [[-1] * 4, [-1] * 4], [0, 0], [0, 0], 16)
    dev = Device(vqv, book)
    ok = vqv.vqv_cache_reserve(dev.pages, i32([20, 40]))
    assert ok.tolist() == book.reserve([20, 40])
    dev.check(book)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_fork(vqv, shape):
    layers, ps, hk, dim, dtype, layout = shape
    book = random_book(11, 4, 9, ps, 40, spare_rows=7)
    cache, dev = pair(vqv, shape, 40), Device(vqv, book)
    parent, child = [0, 1, 1, 3, 2, 0], [4, 5, 10, 8, 7, 6]
    for again in range(2):
        want = [bits(x) for x in (cache.k, cache.v)]
        ok = vqv.vqv_cache_fork(cache, dev.pages, i32(parent), i32(child))
        good, copies = book.fork(parent, child)
        assert ok.tolist() == good
        for x in want:
            for a, b in copies:
                x[:, b] = x[:, a]
        dev.check(book)
        for got, w in zip((cache.k, cache.v), want):
            assert torch.equal(bits(got), w)
        # drop the branches; the shared pages stay with their parents
        vqv.vqv_cache_trim(dev.pages, i32([0] * 6), rows=i32(child))
        book.trim([0] * 6, child)
        dev.check(book)


@pytest.mark.parametrize("extra", [0, 1500])
def test_reserve_on_shared_pages(vqv, extra):
    """A branch that is cut inside the pages that it shares gets no room to write there; a branch of
    the branch does, and what is appended to it does not reach the first row. extra: rows more than
    the book's work-group has threads."""
    ps, width, pages = 16, 8, 20
    book = ref.Book([1, 1, 1] + [0] * (pages - 3), [[2, 0, 1] + [-1] * 5] + [[-1] * width for _ in range(4 + extra)],
                    [3] + [0] * (4 + extra), [40] + [0] * (4 + extra), ps)
    cache, dev = pair(vqv, (2, ps, 1, 64, torch.bfloat16, "slot"), pages), Device(vqv, book)
    tail = [0] * extra

    def both(name, *a):
        got = getattr(vqv, "vqv_cache_" + name)(*([cache] if name == "fork" else []), dev.pages, *map(i32, a))
        want = getattr(book, name)(*a)
        if name != "trim":
            assert got.tolist() == (want[0] if name == "fork" else want)
        dev.check(book)
        return want

    both("fork", [0, 0, 0], [1, 2, 3])
    both("trim", [20, 32, 40], [1, 2, 3])
    # row 1 ends in a shared page, row 2 at its border, row 3 in its own; row 1 may keep what it has
    assert both("reserve", [56, 21, 33, 41, 0] + tail)[:5] == [1, 0, 1, 1, 1]
    assert both("reserve", [56, 20, 33, 41, 0] + tail)[:5] == [1, 1, 1, 1, 1]
    before = [bits(x) for x in (cache.k, cache.v)]
    both("fork", [1], [4])
    both("trim", [0], [1])
    assert both("reserve", [40, 0, 33, 41, 21] + tail)[:5] == [1, 1, 1, 1, 1]
    x = torch.ones(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    seqs = vqv.Sequences(i32([0, 0, 0, 0, 0, 1]), i32([40, 0, 32, 40, 21]), dev.t[1], n_rows=1, max_rows=1, max_kv=48)
    vqv.vqv_rope_append(x, x, x, cache, seqs, vqv.Rope(64), layer=1)
    torch.cuda.synchronize()
    held = [p for r in (0, 2, 3) for p in book.table[r] if p >= 0]
    for got, w in zip((cache.k, cache.v), before):
        assert torch.equal(bits(got)[:, held], w[:, held])
    assert (cache.v[1, book.table[4][1], 4] == 1).all()


def test_fork_refused_pairs(vqv):
    """Rows that are none, a child that holds pages, is named twice or is a
    parent, and too few free pages."""
    ps = 4
    refs = [1, 1, 1, 0, 0, 1]
    table = [[0, 1, -1], [2, -1, -1], [-1] * 3, [-1] * 3, [-1] * 3, [5, -1, -1], [-1] * 3]
    book = ref.Book(refs, table, [2, 1, 0, 0, 0, 1, 0], [6, 3, 0, 0, 0, 4, 0], ps)
    cache, dev = pair(vqv, (1, ps, 1, 8, torch.bfloat16, "slot"), 6), Device(vqv, book)
    parent, child = [0, 0, 9, 1, 0, 1, 5], [2, 2, 6, -1, 5, 3, 4]
    ok = vqv.vqv_cache_fork(cache, dev.pages, i32(parent), i32(child))
    assert ok.tolist() == book.fork(parent, child)[0] == [1, 0, 0, 0, 0, 1, 1]
    dev.check(book)
    ok = vqv.vqv_cache_fork(cache, dev.pages, i32([0]), i32([6]))   # no page is free now
    assert ok.tolist() == book.fork([0], [6])[0] == [0]
    dev.check(book)


def test_copy_many_pairs(vqv):
    """More pairs than a launch's second dimension holds."""
    n = 70001
    cache = pair(vqv, (1, 1, 1, 8, torch.bfloat16, "slot"), 2 * n)
    order = torch.randperm(2 * n, generator=torch.Generator().manual_seed(2))
    want = [bits(x) for x in (cache.k, cache.v)]
    for x in want:
        x[:, order[n:]] = x[:, order[:n]]
    vqv.vqv_cache_copy(cache, order[:n].to(torch.int32).cuda(), order[n:].to(torch.int32).cuda())
    torch.cuda.synchronize()
    for got, w in zip((cache.k, cache.v), want):
        assert torch.equal(bits(got), w)


@pytest.mark.parametrize("n", [1025, 70000])
def test_fork_many_pairs(vqv, n):
    """More branches than the book's work-group has threads, and than a launch holds; one page too few."""
    pages, ps = n + 2, 2
    cache = pair(vqv, (1, ps, 1, 8, torch.bfloat16, "slot"), pages)
    table = torch.full((n + 1, 2), -1, dtype=torch.int32, device="cuda")
    table[0] = i32([5, 2])
    refs, held, length = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (pages, n + 1, n + 1))
    refs[[5, 2, 9]] = 1                       # page 9 is another's
    held[0], length[0] = 2, 3
    book = vqv.Pages(refs, table, held, length, page_size=ps)
    child = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
    ok = vqv.vqv_cache_fork(cache, book, torch.zeros_like(child), child)
    free = torch.tensor([p for p in range(pages) if p not in (5, 2, 9)], dtype=torch.int32, device="cuda")
    good = free.numel()
    assert good == n - 1 and ok[:good].all() and ok[good] == 0
    assert (table[1:n, 0] == 5).all() and torch.equal(table[1:n, 1], free) and (table[n] == -1).all()
    assert refs[5] == n and (refs[free.long()] == 1).all() and refs[2] == refs[9] == 1
    assert (held[1:n] == 2).all() and (length[1:n] == 3).all() and held[n] == length[n] == 0
    for x in (cache.k, cache.v):
        x = x.view(torch.int16)
        assert (x[0, free.long()] == x[0, 2]).all()


@pytest.mark.parametrize("bad", [-1, 6, 1 << 30])
def test_fork_bad_pages(vqv, bad):
    """A parent whose last page is none has no branch (its tokens there are hidden; a new page
    would show another sequence's); an entry of a full page that is none is passed on."""
    ps, none = 4, [-1] * 3
    table = [[0, bad, -1], [bad, 2, -1], none[:], none[:], none[:]]
    book = ref.Book([1, 0, 1, 0, 0, 0], table, [2, 2, 0, 0, 0], [6, 7, 0, 0, 0], ps)
    cache, dev = pair(vqv, (1, ps, 1, 8, torch.bfloat16, "slot"), 6), Device(vqv, book)
    want = [bits(x) for x in (cache.k, cache.v)]
    ok = vqv.vqv_cache_fork(cache, dev.pages, i32([0, 1]), i32([2, 3]))
    good, copies = book.fork([0, 1], [2, 3])
    assert ok.tolist() == good == [0, 1] and copies == [(2, 1)]
    dev.check(book)
    for x, got in zip(want, (cache.k, cache.v)):
        x[:, 1] = x[:, 2]
        assert torch.equal(bits(got), x)


def compact(vqv, shape, rows, kv, keep, bad=()):
    layers, ps, hk, dim, dtype, layout = shape
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    held = [-(-max(x, 1) // ps) for x in kv]
    pages = sum(held) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
    table = [[-1] * max(held) for _ in rows]
    for b, x in enumerate(held):
        for j in range(x):
            table[b][j] = order.pop()
    for b, j in bad:
        table[b][j] = -1 if b % 2 else pages
    cache = pair(vqv, shape, pages)
    want, new = [bits(x) for x in (cache.k, cache.v)], []
    for b, x in enumerate(kv):
        first = to = x - rows[b]
        for i in range(rows[b]):
            if not keep[start[b] + i]:
                continue
            s, d = (table[b][t // ps] if t >= 0 else -1 for t in (first + i, to))
            if 0 <= s < pages and 0 <= d < pages:
                for w in want:
                    w[:, d, to % ps] = w[:, s, (first + i) % ps]
            to += 1
        new.append(to)
    seqs = vqv.Sequences(i32(start), i32(kv), i32(table), n_rows=start[-1], max_rows=max(rows), max_kv=max(kv))
    got = vqv.vqv_cache_compact(cache, seqs, i32(keep))
    torch.cuda.synchronize()
    assert got.tolist() == new
    for x, w in zip((cache.k, cache.v), want):
        assert torch.equal(bits(x), w)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_compact(vqv, shape):
    gen = torch.Generator().manual_seed(2)
    rows, kv = [16, 1, 0, 9, 30, 5], [40, 1, 6, 9, 100, 64]
    keep = torch.randint(0, 3, (sum(rows),), generator=gen).tolist()
    compact(vqv, shape, rows, kv, keep)
    compact(vqv, shape, rows, kv, [0] * sum(rows))
    compact(vqv, shape, rows, kv, [1] * sum(rows))


def test_compact_many_rows(vqv):
    """More rows than one run of the list; every second one kept."""
    rows = [600, 257]
    compact(vqv, SHAPES[0], rows, [605, 400], [i % 2 for i in range(sum(rows))])


def test_compact_moves_bytes(vqv):
    """A prefix stays, bit for bit; a key kept behind a dropped row is still turned for its old place."""
    x = torch.randn(5, 1, 64, generator=torch.Generator().manual_seed(4)).cuda()
    rope = vqv.Rope(64)
    seqs = vqv.Sequences(i32([0, 5]), i32([9]), i32([[2, 0, 1]]), n_rows=5, max_rows=5, max_kv=9)
    cache = pair(vqv, (1, 4, 1, 64, torch.bfloat16, "slot"), 3)
    vqv.vqv_rope_append(x, x, x, cache, seqs, rope)
    before = [bits(cache.k), bits(cache.v)]
    assert vqv.vqv_cache_compact(cache, seqs, i32([1, 1, 1, 0, 0])).tolist() == [7]
    assert torch.equal(bits(cache.k), before[0]) and torch.equal(bits(cache.v), before[1])
    assert vqv.vqv_cache_compact(cache, seqs, i32([1, 0, 0, 1, 0])).tolist() == [6]
    f, m = ref.rope_frequencies(64, 10000.0)
    got = cache.k[0, 0, 1].double().cpu()          # token 5: row 3 of positions 4..8
    old, new = (ref.rope_ref(x[3].cpu(), p, f, m, 64, False) for p in (7, 5))
    assert ((got - old).abs() <= 2.0 ** -8 * old.abs() + 1e-5).all() and (got - new).abs().max() > 0.1
    assert torch.equal(cache.v[0, 0, 1], x[3].to(torch.bfloat16))


def test_compact_bad_pages(vqv):
    """A row on a page that is none is not moved, nor is one whose place is on
    such a page; rows before the first token neither."""
    compact(vqv, (1, 4, 1, 64, torch.bfloat16, "slot"), [12, 12, 6], [20, 21, 4],
            [0, 1] * 6 + [0, 1, 1] * 4 + [1] * 6, bad=[(0, 3), (1, 2)])


@pytest.mark.parametrize("kv", [-2 ** 31, -2 ** 31 + 2, -5, 2])
def test_lengths_far_below_zero(vqv, kv):
    """Rows before the first token are stored nowhere and move nowhere, also where their positions
    pass 32 bits and the table is as wide; what stands on the pages that those would be on stays."""
    ps, width = 1 << 20, 2048
    cache = vqv.PagedCache(*(torch.full((1, 2, ps, 1, 64), x, dtype=torch.bfloat16, device="cuda") for x in (2.0, 3.0)))
    seqs = vqv.Sequences(i32([0, 4]), i32([kv]), i32([[1] * width]), n_rows=4, max_rows=4, max_kv=4)
    x = torch.randn(4, 1, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    q = vqv.vqv_rope_append(x, x, x, cache, seqs, vqv.Rope(2, interleaved=True))
    out = vqv.vqv_paged_attn(q, cache, seqs, scale=1.0)
    new = vqv.vqv_cache_compact(cache, seqs, i32([0, 1, 1, 0]))
    assert new.tolist() == [max(kv - 2, -2 ** 31)]
    first = max(kv, 0)                      # tokens that there are
    assert (out[:4 - first] == 0).all() and (out[4 - first:] != 0).all()
    for t, value in ((cache.k, 2.0), (cache.v, 3.0)):
        assert (t[0, 0] == value).all() and (t[0, 1, first:] == value).all()
        # what is not turned of the rows that there are
        assert torch.equal(t[0, 1, :first, :, 2:], x[4 - first:, :, 2:])


def test_round_in_a_graph(vqv):
    """Compact, trim and reserve replayed from a graph are as good as called."""
    ps, layers = 4, 2
    cache = vqv.PagedCache(*(storage(layers, 12, ps, 1, 64, torch.bfloat16, "slot", s) for s in (1, 2)))
    first = [cache.k.clone(), cache.v.clone()]
    book = ref.Book([1] * 6 + [0] * 6, [[3, 0, 5, -1], [1, 2, 4, -1]], [3, 3], [11, 12], ps)
    dev = Device(vqv, book)
    kv, start = i32([11, 12]), i32([0, 6, 12])
    seqs = vqv.Sequences(start, kv, dev.t[1], n_rows=12, max_rows=6, max_kv=12)
    keep, ok = i32([1, 0, 0, 1, 0, 1] + [1, 0, 0, 0, 0, 0]), i32([0, 0])
    ws = torch.empty(vqv.vqv_cache_workspace_bytes(dev.pages), dtype=torch.uint8, device="cuda")

    def path():
        vqv.vqv_cache_compact(cache, seqs, keep, new_len=dev.t[3])
        vqv.vqv_cache_trim(dev.pages, dev.t[3])
        vqv.vqv_cache_reserve(dev.pages, kv, ok=ok, workspace=ws)

    start_state = [t.clone() for t in dev.t]
    path()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*dev.t, cache.k, cache.v, ok)]
    assert want[3].tolist() == [8, 7] and ok.tolist() == [1, 1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path()
    for _ in range(3):
        for t, s in zip((*dev.t, cache.k, cache.v), (*start_state, *first)):
            t.copy_(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((*dev.t, cache.k, cache.v, ok), want):
            assert torch.equal(got.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8))


def test_refuses_wrong_tensors(vqv):
    book = random_book(1, 2, 3, 4, 9)
    dev, cache = Device(vqv, book), pair(vqv, (1, 4, 1, 64, torch.bfloat16, "slot"), 9)
    with pytest.raises(ValueError):
        vqv.vqv_cache_trim(dev.pages, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        vqv.vqv_cache_trim(dev.pages, i32([1, 2]), rows=i32([1]))
    with pytest.raises(vqv.VqvError):
        vqv.vqv_cache_reserve(dev.pages, i32([1, 2, 3]))
    with pytest.raises(ValueError):
        vqv.vqv_cache_fork(cache, dev.pages, i32([0]), i32([1, 2]))
    with pytest.raises(ValueError):
        vqv.vqv_cache_copy(cache, i32([0]), torch.tensor([1], dtype=torch.int32))
    with pytest.raises(vqv.VqvError):
        vqv.vqv_cache_fork(pair(vqv, (1, 8, 1, 64, torch.bfloat16, "slot"), 9), dev.pages, i32([0]), i32([1]))
    with pytest.raises(ValueError):
        vqv.Pages(*dev.t[:2], dev.t[2][:1], dev.t[3], page_size=4)
