"""include/vqv_round.h on the CPU: the library exports what it declares, the
binding's structs have the header's sizes, rotary plans, and every refusal (the
pointers are made up and never followed: checks come before any launch)."""

import ctypes
import math
import os
import re
import subprocess

import pytest

from oracle import round_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "vqv_round.h")
OK, ARG, UNSUP, ALIGN, WS, HIP = range(6)
BF16, FP16, FP32 = range(3)
P = [0x10000000 * i for i in range(1, 14)]


@pytest.fixture(scope="module")
def R():
    from w4_gemm_vqv_amd import vqv
    if not os.path.exists(vqv.LIB_PATH):
        from w4_gemm_vqv_amd.build import build
        build(verbose=False)
    from w4_gemm_vqv_amd import round as r
    return r


@pytest.fixture(scope="module")
def L(R):
    return R._round_lib()


def test_exports(R, L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(vqv_\w+)\s*\(", text))
    assert names == set(R.ROUND_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", R._load()._name], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (vqv_\w+)$", out, flags=re.M))


def test_struct_sizes(R, tmp_path):
    """The binding's structs against a C compiler's view of the header."""
    src = tmp_path / "s.c"
    src.write_text('#include "vqv_round.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu '
                   '%zu %zu %zu\\n", sizeof(vqv_cache), sizeof(vqv_seqs), sizeof(vqv_rope), '
                   'sizeof(vqv_pages), sizeof(vqv_edits)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(t) for t in (R._Cache, R._Seqs, R._Rope,
                                                               R._Pages, R._Edits)]


@pytest.mark.parametrize("rot", [2, 34, 64, 128, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "smooth"])
def test_rope_plan(R, rot, scaling):
    plan = R.Rope(rot, 1e6, scaling=scaling, factor=8.0, original_len=8192)
    f, m = ref.rope_frequencies(rot, 1e6, scaling, 8.0, 8192)
    assert abs(plan.c.mscale - m) <= 2.0 ** -24 * m
    for i, x in enumerate(f):
        assert abs(plan.c.turns[i] * 2 * math.pi - x) <= 1e-14 * x
    assert not any(plan.c.turns[len(f):])


@pytest.mark.parametrize("factor", [0.25, 0.5, 1.0, 1.5])
def test_yarn_does_not_shrink(R, factor):
    """Cosines and sines grow with the factor, and are left alone where it does not stretch."""
    plan = R.Rope(64, 1e6, scaling="yarn", factor=factor, original_len=8192)
    want = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    assert abs(plan.c.mscale - want) <= 2.0 ** -24 * want
    f, m = ref.rope_frequencies(64, 1e6, "yarn", factor, 8192)
    assert m == want
    for i, x in enumerate(f):
        assert abs(plan.c.turns[i] * 2 * math.pi - x) <= 1e-14 * x


@pytest.mark.parametrize("args,status", [
    ((3, 1e4, 0, 0, 1.0, 0), ARG), ((0, 1e4, 0, 0, 1.0, 0), ARG), ((258, 1e4, 0, 0, 1.0, 0), UNSUP),
    ((64, 0.0, 0, 0, 1.0, 0), ARG), ((64, math.inf, 0, 0, 1.0, 0), ARG),
    ((64, 1e4, 0, 5, 1.0, 0), ARG), ((64, 1e4, 0, 1, 0.0, 0), ARG),
    ((64, 1e4, 0, 3, 2.0, 0), ARG), ((64, 1.0, 0, 3, 2.0, 100), ARG),
    ((64, 1e4, 0, 0, 0.0, 0), OK), ((64, 1e4, 1, 4, 2.0, 100), OK)])
def test_rope_plan_refusals(R, L, args, status):
    assert L.vqv_rope_plan(R._Rope(), *args) == status


def cache(R, **kw):
    a = dict(k=P[0], v=P[1], layers=2, pages=100, page_size=16, kv_heads=8, dim=128, dtype=BF16,
             layer_stride=100 * 16 * 8 * 128, page_stride=16 * 8 * 128, slot_stride=8 * 128,
             head_stride=128)
    a.update(kw)
    return R._Cache(**a)


def seqs(R, **kw):
    a = dict(row_start=P[2], kv_len=P[3], table=P[4], table_stride=50, n_seqs=4, table_width=50,
             n_rows=32, max_rows=8, max_kv=800)
    a.update(kw)
    return R._Seqs(**a)


def pages(R, **kw):
    a = dict(ref=P[2], table=P[3], held=P[4], length=P[5], pages=100, rows=4, width=50,
             page_size=16)
    a.update(kw)
    return R._Pages(**a)


BAD_CACHE = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(layers=0), ARG), (dict(pages=0), ARG),
             (dict(page_size=0), ARG), (dict(kv_heads=0), ARG), (dict(dim=0), ARG),
             (dict(dim=12), UNSUP), (dict(dim=264), UNSUP), (dict(dtype=FP32), UNSUP),
             (dict(dtype=7), ARG), (dict(head_stride=-8), ARG), (dict(slot_stride=1028), ALIGN),
             (dict(k=P[0] + 8), ALIGN), (dict(page_stride=1 << 32), UNSUP)]
BAD_SEQS = [(dict(row_start=None), ARG), (dict(kv_len=None), ARG), (dict(table=None), ARG),
            (dict(n_seqs=0), ARG), (dict(n_rows=-1), ARG), (dict(max_rows=-1), ARG),
            (dict(max_kv=-1), ARG), (dict(table_width=0), ARG), (dict(table_stride=49), ARG),
            (dict(kv_len=P[3] + 2), ALIGN), (dict(n_seqs=70000), UNSUP)]


def rope_call(R, L, c=None, s=None, **kw):
    plan = R._Rope()
    assert L.vqv_rope_plan(plan, kw.pop("rot", 128), 1e4, 0, 0, 1.0, 0) == OK
    a = dict(q=P[5], qr=6144, qh=128, k=P[6], kr=6144, kh=128, v=P[7], vr=6144, vh=128,
             in_dtype=FP32, heads=32, layer=0, rope=plan, out=P[8])
    a.update(kw)
    return L.vqv_rope_append(a["q"], a["qr"], a["qh"], a["k"], a["kr"], a["kh"], a["v"], a["vr"],
                             a["vh"], a["in_dtype"], a["heads"], c or cache(R), a["layer"],
                             s or seqs(R), a["rope"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(out=None), ARG),
    (dict(in_dtype=5), ARG), (dict(heads=0), ARG), (dict(layer=2), ARG), (dict(layer=-1), ARG),
    (dict(rot=256), ARG), (dict(qr=-8), ARG), (dict(qr=6146), ALIGN), (dict(kh=129), ALIGN),
    (dict(q=P[5] + 4), ALIGN), (dict(out=P[8] + 8), ALIGN), (dict(out=P[5] + 1024), ARG),
    (dict(heads=70000), UNSUP)])
def test_rope_refusals(R, L, kw, status):
    assert rope_call(R, L, **kw) == status


def attn_call(R, L, c=None, s=None, **kw):
    a = dict(q=P[5], layer=0, heads=32, scale=0.1, window=0, sinks=0, out=P[6], ws=P[7],
             wn=1 << 27)
    a.update(kw)
    return L.vqv_paged_attn(a["q"], c or cache(R), a["layer"], s or seqs(R), a["heads"],
                            a["scale"], a["window"], a["sinks"], a["out"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(layer=2), ARG), (dict(heads=0), ARG),
    (dict(heads=33), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(window=-1), ARG),
    (dict(sinks=-1), ARG), (dict(q=P[5] + 8), ALIGN), (dict(out=P[6] + 2), ALIGN),
    (dict(out=P[5] + 4096), ARG), (dict(ws=None), WS), (dict(wn=64), WS), (dict(ws=P[7] + 4), WS),
    (dict(ws=P[6]), ARG), (dict(heads=8 * 2000), UNSUP)])
def test_attn_refusals(R, L, kw, status):
    assert attn_call(R, L, **kw) == status


def test_attn_grid_limits(R, L):
    """More work-groups than a launch can count."""
    assert attn_call(R, L, s=seqs(R, n_rows=1 << 20, max_rows=1 << 20), heads=1024,
                     wn=1 << 60) == UNSUP
    assert attn_call(R, L, s=seqs(R, n_rows=1 << 20, n_seqs=1), heads=32, wn=1 << 60) == UNSUP


def test_empty_calls(R, L):
    """No rows: no memory is needed for them, as of an empty tensor. What else is wrong is refused."""
    none = seqs(R, n_rows=0)
    rows = dict(q=None, k=None, v=None, out=None)
    assert rope_call(R, L, s=none, **rows) == OK
    assert rope_call(R, L, s=none, q=None) == OK
    assert rope_call(R, L, s=none, layer=2, **rows) == ARG
    assert rope_call(R, L, s=none, rot=256, **rows) == ARG
    assert rope_call(R, L, s=seqs(R), out=None) == ARG
    assert attn_call(R, L, s=none, q=None, out=None, ws=None, wn=0) == OK
    assert attn_call(R, L, s=none, q=None, out=None, ws=None, wn=0, scale=0.0) == ARG
    assert attn_call(R, L, s=none, q=None, out=None, ws=None, wn=0, heads=33) == ARG
    assert attn_call(R, L, s=seqs(R, max_rows=0), q=None) == ARG
    # pages and lists of none
    p = pages(R)
    need = L.vqv_cache_workspace_bytes(p)
    assert L.vqv_cache_copy(cache(R), None, None, 0, None) == OK
    assert L.vqv_cache_trim(p, None, None, 0, None) == OK
    assert L.vqv_cache_reserve(p, None, 0, None, P[8], need, None) == OK
    assert L.vqv_cache_fork(cache(R), p, None, None, 0, None, P[8], need, None) == OK


def test_attn_dims(R, L):
    for d in (8, 72, 136, 248):
        assert attn_call(R, L, c=cache(R, dim=d)) == UNSUP


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_refusals(R, L, kw, status):
    c = cache(R, **kw)
    assert rope_call(R, L, c=c) == status
    assert attn_call(R, L, c=c) == status
    assert L.vqv_cache_copy(c, P[5], P[6], 3, None) == status
    assert L.vqv_cache_compact(c, seqs(R), P[5], P[6], None) == status
    assert L.vqv_paged_attn_workspace_bytes(c, seqs(R), 32, 0, 0) == 0


@pytest.mark.parametrize("kw,status", BAD_SEQS)
def test_seqs_refusals(R, L, kw, status):
    s = seqs(R, **kw)
    assert rope_call(R, L, s=s) == status
    assert attn_call(R, L, s=s) == status
    assert L.vqv_cache_compact(cache(R), s, P[5], P[6], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ref=None), ARG), (dict(table=None), ARG), (dict(held=None), ARG), (dict(length=None), ARG),
    (dict(pages=0), ARG), (dict(rows=0), ARG), (dict(width=0), ARG), (dict(page_size=0), ARG),
    (dict(ref=P[2] + 1), ALIGN), (dict(rows=1 << 20, width=1 << 12), UNSUP)])
def test_pages_refusals(R, L, kw, status):
    p = pages(R, **kw)
    assert L.vqv_cache_trim(p, P[6], None, 4, None) == status
    assert L.vqv_cache_reserve(p, P[6], 4, P[7], P[8], 1 << 30, None) == status
    assert L.vqv_cache_fork(cache(R), p, P[6], P[7], 4, P[8], P[9], 1 << 30, None) == status
    assert L.vqv_cache_workspace_bytes(p) == 0


def test_book_refusals(R, L):
    p, need = pages(R), L.vqv_cache_workspace_bytes(pages(R))
    assert L.vqv_cache_trim(p, None, None, 4, None) == ARG
    assert L.vqv_cache_trim(p, P[6], None, 5, None) == ARG
    assert L.vqv_cache_trim(p, P[6], None, -1, None) == ARG
    assert L.vqv_cache_trim(p, P[6] + 2, None, 4, None) == ALIGN
    assert L.vqv_cache_reserve(p, P[6], 5, P[7], P[8], need, None) == ARG
    assert L.vqv_cache_reserve(p, P[6], 4, None, P[8], need, None) == ARG
    assert L.vqv_cache_reserve(p, P[6], 4, P[6], P[8], need, None) == ARG
    assert L.vqv_cache_reserve(p, P[6], 4, P[7], None, need, None) == WS
    assert L.vqv_cache_reserve(p, P[6], 4, P[7], P[8], need - 1, None) == WS
    assert L.vqv_cache_reserve(p, P[6], 4, P[7], P[7], need, None) == ARG
    f = lambda *a: L.vqv_cache_fork(cache(R), *a, None)
    assert f(p, P[6], P[7], 5, P[8], P[9], need) == ARG
    assert f(p, None, P[7], 4, P[8], P[9], need) == ARG
    assert f(p, P[6], P[7], 4, P[7], P[9], need) == ARG
    assert f(p, P[6], P[7], 4, P[8], P[9] + 8, need) == WS
    assert f(pages(R, pages=99), P[6], P[7], 4, P[8], P[9], need) == ARG
    assert f(pages(R, page_size=8), P[6], P[7], 4, P[8], P[9], need) == ARG
    assert L.vqv_cache_copy(cache(R), None, P[6], 3, None) == ARG
    assert L.vqv_cache_copy(cache(R), P[5], P[6], -1, None) == ARG
    assert L.vqv_cache_compact(cache(R), seqs(R), None, P[6], None) == ARG
    assert L.vqv_cache_compact(cache(R), seqs(R), P[5], P[5], None) == ARG
    assert L.vqv_cache_compact(cache(R), seqs(R), P[5], P[3], None) == ARG


def edits(R, **kw):
    a = dict(n_seqs=2, n=1000, counts=P[2], seen=P[3], repetition=P[4], frequency=P[5],
             presence=P[6], bias_start=P[7], bias_token=P[8], bias_value=P[9], n_bias=10)
    a.update(kw)
    return R._Edits(**a)


@pytest.mark.parametrize("kw,T,status", [
    (dict(n_seqs=0), 4, ARG), (dict(n=0), 4, ARG), (dict(), 0, ARG), (dict(), 65, ARG),
    (dict(n_bias=-1), 4, ARG), (dict(bias_token=None), 4, ARG), (dict(bias_value=None), 4, ARG),
    (dict(n=1 << 30), 4, ARG), (dict(counts=P[2] + 2), 4, ALIGN), (dict(n_seqs=70000), 4, UNSUP)])
def test_edits_refusals(R, L, kw, T, status):
    e = edits(R, **kw)
    assert L.vqv_logits_edit(P[0], e, P[10], T, None, P[1], None) == status
    assert L.vqv_logits_verify(P[0], e, P[10], None, T, None, P[11], P[12], None, P[1], 1 << 27,
                               None) == status


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 4095])
def test_edits_past_the_last_tile(R, L, n):
    """Tokens of the last tile that 32 bits do not count."""
    a = [i << 40 for i in range(1, 8)]   # far enough apart
    e = R._Edits(n_seqs=1, n=n)
    assert L.vqv_logits_edit(a[0], e, None, 1, a[1], a[2], None) == UNSUP
    assert L.vqv_logits_verify(a[0], e, None, None, 1, a[1], a[2], a[3], None, a[4], 1 << 39, None) == UNSUP


def test_logits_refusals(R, L):
    e = edits(R)
    ed = lambda *a: L.vqv_logits_edit(*a, None)
    assert ed(None, e, P[10], 4, None, P[1]) == ARG
    assert ed(P[0], e, P[10], 4, None, None) == ARG
    assert ed(P[0] + 4, e, P[10], 4, None, P[1]) == ALIGN
    assert ed(P[0], e, P[10], 4, None, P[0] + 16) == ARG
    assert ed(P[0], e, P[10], 4, None, P[2]) == ARG
    ve = lambda lg, d, am, al, mg, ws, wn: L.vqv_logits_verify(lg, e, d, None, 4, None, am, al, mg,
                                                              ws, wn, None)
    assert ve(P[0], None, P[11], P[12], None, P[1], 1 << 27) == ARG
    assert ve(P[0], P[10], None, P[12], None, P[1], 1 << 27) == ARG
    assert ve(P[0], P[10], P[11], P[11], None, P[1], 1 << 27) == ARG
    assert ve(P[0], P[10], P[11], P[12], P[2], P[1], 1 << 27) == ARG
    assert ve(P[0], P[10], P[11], P[12], None, None, 1 << 27) == WS
    assert ve(P[0], P[10], P[11], P[12], None, P[1], 64) == WS
    assert ve(P[0], P[10], P[11], P[12], None, P[0], 1 << 27) == ARG


def test_binding_refuses_host_tensors(R):
    import torch
    k = torch.zeros(1, 4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        R.PagedCache(k, k.clone())
    with pytest.raises(ValueError):
        R.PagedCache(k, k[:, :2])
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        R.Sequences(i, i[:2], i.view(1, 3), 0, 0, 0)
    with pytest.raises(ValueError):
        R.Rope(64, scaling="other")
    with pytest.raises(R.VqvError):
        R.Rope(63)
    with pytest.raises(ValueError):
        R.Edits(1, 10, counts=torch.zeros(1, 10, dtype=torch.int32))
