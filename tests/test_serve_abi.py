"""include/vqv_serve.h on the CPU: the library exports what it declares, the
binding's structs have the header's sizes, and every refusal (the pointers are
made up and never followed: checks come before any launch)."""

import ctypes
import math
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "vqv_serve.h")
OK, ARG, UNSUP, ALIGN, WS, HIP = range(6)
BF16, FP16, FP32 = range(3)
P = [0x100000000 * i for i in range(1, 14)]


@pytest.fixture(scope="module")
def S():
    from w4_gemm_vqv_amd import vqv
    if not os.path.exists(vqv.LIB_PATH):
        from w4_gemm_vqv_amd.build import build
        build(verbose=False)
    from w4_gemm_vqv_amd import serve
    return serve


@pytest.fixture(scope="module")
def L(S):
    return S._serve_lib()


def test_exports(S):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(vqv_\w+)\s*\(", text))
    assert names == set(S.SERVE_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", S._load()._name], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (vqv_\w+)$", out, flags=re.M))


def test_struct_sizes(S, tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "vqv_serve.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu\\n", '
                   'sizeof(vqv_cache_q4), sizeof(vqv_adapters)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(t) for t in (S._CacheQ4, S._Adapters)]


def test_record_bytes(L):
    got = {d: L.vqv_q4_record_bytes(d) for d in (64, 80, 96, 128, 192, 256)}
    assert got == {64: 48, 80: 64, 96: 64, 128: 80, 192: 128, 256: 160}
    for d in (-64, 0, 8, 32, 72, 100, 160, 320):
        assert L.vqv_q4_record_bytes(d) == 0


def cache(S, **kw):
    a = dict(k=P[0], v=P[1], layers=2, pages=100, page_size=16, kv_heads=8, dim=128, reserved=0,
             layer_stride=100 * 16 * 8 * 80, page_stride=16 * 8 * 80, slot_stride=8 * 80,
             head_stride=80)
    a.update(kw)
    return S._CacheQ4(**a)


def seqs(S, **kw):
    a = dict(row_start=P[2], kv_len=P[3], table=P[4], table_stride=50, n_seqs=4, table_width=50,
             n_rows=32, max_rows=8, max_kv=800)
    a.update(kw)
    return S._Seqs(**a)


BAD_CACHE = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(layers=0), ARG), (dict(pages=0), ARG),
             (dict(page_size=0), ARG), (dict(kv_heads=0), ARG), (dict(dim=0), ARG),
             (dict(dim=72), UNSUP), (dict(dim=320), UNSUP), (dict(head_stride=-16), ARG),
             (dict(slot_stride=648), ALIGN), (dict(k=P[0] + 8), ALIGN), (dict(v=P[1] + 4), ALIGN),
             (dict(page_stride=1 << 34), UNSUP), (dict(kv_heads=70000), UNSUP),
             (dict(layers=40000), UNSUP)]
BAD_SEQS = [(dict(row_start=None), ARG), (dict(kv_len=None), ARG), (dict(table=None), ARG),
            (dict(n_seqs=0), ARG), (dict(n_rows=-1), ARG), (dict(max_rows=-1), ARG),
            (dict(max_kv=-1), ARG), (dict(table_width=0), ARG), (dict(table_stride=49), ARG),
            (dict(kv_len=P[3] + 2), ALIGN), (dict(n_seqs=70000), UNSUP)]


def rope_call(S, L, c=None, s=None, **kw):
    plan = S.Rope(kw.pop("rot", 128), 1e4).c
    a = dict(q=P[5], qr=6144, qh=128, k=P[6], kr=6144, kh=128, v=P[7], vr=6144, vh=128,
             in_dtype=FP32, heads=32, layer=0, rope=plan, out=P[8], q_dtype=BF16)
    a.update(kw)
    return L.vqv_rope_append_q4(a["q"], a["qr"], a["qh"], a["k"], a["kr"], a["kh"], a["v"], a["vr"],
                                a["vh"], a["in_dtype"], a["heads"], c or cache(S), a["layer"],
                                s or seqs(S), a["rope"], a["out"], a["q_dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(out=None), ARG),
    (dict(in_dtype=5), ARG), (dict(heads=0), ARG), (dict(layer=2), ARG), (dict(layer=-1), ARG),
    (dict(rot=256), ARG), (dict(qr=-8), ARG), (dict(qr=6146), ALIGN), (dict(kh=129), ALIGN),
    (dict(q=P[5] + 4), ALIGN), (dict(out=P[8] + 8), ALIGN), (dict(out=P[5] + 1024), ARG),
    (dict(out=P[7]), ARG), (dict(heads=70000), UNSUP), (dict(q_dtype=FP32), UNSUP),
    (dict(q_dtype=9), ARG), (dict(rope=None), ARG)])
def test_rope_refusals(S, L, kw, status):
    assert rope_call(S, L, **kw) == status


def read_call(S, L, c=None, s=None, **kw):
    a = dict(layer=0, k=P[8], v=P[9], dtype=FP32)
    a.update(kw)
    return L.vqv_cache_q4_read(c or cache(S), a["layer"], s or seqs(S), a["k"], a["v"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), ARG), (dict(layer=-1), ARG), (dict(dtype=4), ARG), (dict(k=P[8] + 8), ALIGN),
    (dict(v=P[9] + 4), ALIGN), (dict(v=P[8]), ARG), (dict(k=P[0] + 64), ARG), (dict(v=P[1]), ARG),
    (dict(k=None, v=None), OK)])
def test_read_refusals(S, L, kw, status):
    assert read_call(S, L, **kw) == status


def attn_call(S, L, c=None, s=None, **kw):
    a = dict(q=P[5], dtype=BF16, layer=0, heads=32, scale=0.1, window=0, sinks=0, out=P[6], ws=P[7],
             wn=1 << 27)
    a.update(kw)
    return L.vqv_paged_attn_q4(a["q"], a["dtype"], c or cache(S), a["layer"], s or seqs(S), a["heads"],
                               a["scale"], a["window"], a["sinks"], a["out"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(layer=2), ARG), (dict(heads=0), ARG),
    (dict(heads=33), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(window=-1), ARG),
    (dict(sinks=-1), ARG), (dict(q=P[5] + 8), ALIGN), (dict(out=P[6] + 2), ALIGN),
    (dict(out=P[5] + 4096), ARG), (dict(ws=None), WS), (dict(wn=64), WS), (dict(ws=P[7] + 4), WS),
    (dict(ws=P[6]), ARG), (dict(heads=8 * 2000), UNSUP), (dict(dtype=FP32), UNSUP),
    (dict(dtype=3), ARG)])
def test_attn_refusals(S, L, kw, status):
    assert attn_call(S, L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(S, L, kw, status):
    c = cache(S, **kw)
    assert rope_call(S, L, c=c) == status
    assert read_call(S, L, c=c) == status
    assert attn_call(S, L, c=c) == status
    assert L.vqv_paged_attn_q4_workspace_bytes(c, seqs(S), 32, 0, 0) == 0


@pytest.mark.parametrize("kw,status", BAD_SEQS)
def test_bad_sequences(S, L, kw, status):
    s = seqs(S, **kw)
    assert rope_call(S, L, s=s) == status
    assert read_call(S, L, s=s) == status
    assert attn_call(S, L, s=s) == status


def test_attn_grid_limits(S, L):
    """More work-groups than a launch can count."""
    assert attn_call(S, L, s=seqs(S, n_rows=1 << 20, max_rows=1 << 20), heads=1024, wn=1 << 60) == UNSUP
    assert attn_call(S, L, s=seqs(S, n_rows=1 << 20, n_seqs=1), heads=32, wn=1 << 60) == UNSUP


def test_empty_calls(S, L):
    """No rows: no memory is needed for them. What else is wrong is refused."""
    none = seqs(S, n_rows=0)
    rows = dict(q=None, k=None, v=None, out=None)
    assert rope_call(S, L, s=none, **rows) == OK
    assert rope_call(S, L, s=none, layer=2, **rows) == ARG
    assert rope_call(S, L, s=none, q_dtype=FP32, **rows) == UNSUP
    assert read_call(S, L, s=none, k=None, v=None) == OK
    assert read_call(S, L, s=none) == OK
    assert attn_call(S, L, s=none, q=None, out=None, ws=None, wn=0) == OK
    assert attn_call(S, L, s=none, q=None, out=None, ws=None, wn=0, scale=0.0) == ARG
    assert attn_call(S, L, s=none, q=None, out=None, ws=None, wn=0, dtype=FP32) == UNSUP
    assert lora_call(S, L, x=None, which=None, M=0, y=None, out=None, ws=None, wn=0) == OK


def sample_call(L, **kw):
    a = dict(logits=P[0], draft=P[1], probs=P[2], draft_len=P[3], temperature=P[4], uniform=P[5], B=2, T=8,
             N=5000, token=P[6], accept=P[7], logprob=P[8], ws=P[9], wn=1 << 27)
    a.update(kw)
    return L.vqv_verify_sampled(*(a[x] for x in ("logits", "draft", "probs", "draft_len", "temperature", "uniform", "B",
                                                 "T", "N", "token", "accept", "logprob", "ws", "wn")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), ARG), (dict(draft=None), ARG), (dict(uniform=None), ARG), (dict(token=None), ARG),
    (dict(accept=None), ARG), (dict(B=0), ARG), (dict(T=0), ARG), (dict(T=65), ARG), (dict(N=0), ARG),
    (dict(B=70000, T=1, N=10), UNSUP), (dict(B=1 << 14, T=64, N=1 << 12), ARG),
    (dict(B=1, T=1, N=2 ** 31 - 4095), UNSUP), (dict(logits=P[0] + 4), ALIGN), (dict(probs=P[2] + 4), ALIGN),
    (dict(draft=P[1] + 2), ALIGN), (dict(draft_len=P[3] + 1), ALIGN), (dict(temperature=P[4] + 2), ALIGN),
    (dict(uniform=P[5] + 2), ALIGN), (dict(token=P[6] + 2), ALIGN), (dict(accept=P[7] + 2), ALIGN),
    (dict(logprob=P[8] + 2), ALIGN), (dict(ws=None), WS), (dict(wn=16), WS), (dict(ws=P[9] + 8), WS),
    (dict(token=P[0]), ARG), (dict(accept=P[1]), ARG), (dict(logprob=P[2]), ARG), (dict(token=P[3]), ARG),
    (dict(token=P[4]), ARG), (dict(logprob=P[5]), ARG), (dict(accept=P[6]), ARG), (dict(logprob=P[6]), ARG),
    (dict(ws=P[2]), ARG), (dict(ws=P[6]), ARG)])
def test_sample_refusals(L, kw, status):
    assert sample_call(L, **kw) == status


def test_sample_workspace(L):
    assert L.vqv_verify_sampled_workspace_bytes(0, 1, 1) == 0
    assert L.vqv_verify_sampled_workspace_bytes(1, 65, 1) == 0
    # a partial of 16 bytes per row and chunk, a sum per sequence and chunk, a counter per sequence
    assert L.vqv_verify_sampled_workspace_bytes(2, 8, 5000) == 2 * 8 * 2 * 16 + 2 * 2 * 8 + 16


def adapters(S, **kw):
    a = dict(a=P[0], b=P[1], scale=P[2], ranks=P[3], n=4, rank=16, K=512, N=1000, dtype=BF16, reserved=0)
    a.update(kw)
    return S._Adapters(**a)


def lora_call(S, L, ad=None, **kw):
    a = dict(x=P[4], act=BF16, which=P[5], M=8, y=P[6], ys=1000, out=P[7], os=1000, ws=P[8], wn=1 << 27)
    a.update(kw)
    return L.vqv_lora_add(a["x"], a["act"], ad or adapters(S), a["which"], a["M"], a["y"], a["ys"], a["out"], a["os"],
                          a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), ARG), (dict(b=None), ARG), (dict(scale=None), ARG), (dict(n=0), ARG), (dict(rank=0), ARG),
    (dict(rank=12), ARG), (dict(rank=264), UNSUP), (dict(K=0), ARG), (dict(K=20), ARG), (dict(K=40000), UNSUP),
    (dict(N=0), ARG), (dict(dtype=FP32), UNSUP), (dict(dtype=8), ARG), (dict(a=P[0] + 8), ALIGN),
    (dict(b=P[1] + 2), ALIGN), (dict(scale=P[2] + 2), ALIGN), (dict(ranks=P[3] + 2), ALIGN)])
def test_bad_adapters(S, L, kw, status):
    ad = adapters(S, **kw)
    assert lora_call(S, L, ad) == status
    assert L.vqv_lora_add_workspace_bytes(ad, 8) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ARG), (dict(which=None), ARG), (dict(y=None), ARG), (dict(out=None), ARG), (dict(M=-1), ARG),
    (dict(M=1 << 23), UNSUP), (dict(act=FP16), UNSUP), (dict(act=7), ARG), (dict(ys=999), ARG), (dict(os=999), ARG),
    (dict(ys=1 << 60), UNSUP), (dict(x=P[4] + 8), ALIGN), (dict(which=P[5] + 2), ALIGN), (dict(y=P[6] + 2), ALIGN),
    (dict(out=P[7] + 1), ALIGN), (dict(ws=None), WS), (dict(wn=8), WS), (dict(ws=P[8] + 8), WS),
    (dict(out=P[4]), ARG), (dict(out=P[0]), ARG), (dict(out=P[1] + 64), ARG), (dict(out=P[2]), ARG),
    (dict(out=P[3]), ARG), (dict(out=P[5]), ARG), (dict(ws=P[7]), ARG), (dict(ws=P[6]), ARG), (dict(ws=P[4]), ARG),
    (dict(out=P[6] + 4), ARG), (dict(out=P[6], os=1004), ARG)])
def test_lora_refusals(S, L, kw, status):
    assert lora_call(S, L, **kw) == status


def test_lora_grid_limits(S, L):
    """More work-groups than a launch can count."""
    ad = adapters(S, n=1000, N=100000)
    assert lora_call(S, L, ad, M=1 << 21, ys=100000, os=100000, wn=1 << 60) == UNSUP
    assert L.vqv_lora_add_workspace_bytes(ad, 1 << 21) == 0


@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 512, 2 ** 31 - 4096])
def test_lora_columns_past_32_bits(S, L, N):
    """Columns are counted in 32 bits, past the last one to the end of the work-groups' share."""
    ad = adapters(S, n=1, rank=8, K=8, N=N)
    assert lora_call(S, L, ad, M=1, ys=N, os=N, wn=1 << 60) == UNSUP
    assert L.vqv_lora_add_workspace_bytes(ad, 1) == 0
    assert L.vqv_lora_add_workspace_bytes(adapters(S, n=1, rank=8, K=8, N=2 ** 31 - 4097), 1) > 0


def attn_bytes(S, L, dtype=None, heads=32, **kw):
    width = -(-kw["max_kv"] // 64) + 1
    c = cache(S, page_size=64, page_stride=64 * 8 * 80, layers=1)
    s = seqs(S, table_width=width, table_stride=width, **kw)
    if dtype is None:
        return L.vqv_paged_attn_q4_workspace_bytes(c, s, heads, 0, 0)
    return L.vqv_paged_attn_q4_type_workspace_bytes(c, s, dtype, heads, 0, 0)


def test_copy_of_large_calls(S, L):
    """The size of a prompt chunk's workspace does not collapse where its tokens take more than 1 GiB."""
    for rows in (256, 1024, 2048):
        for n in (1, 3):
            got = [attn_bytes(S, L, n_seqs=n, n_rows=n * rows, max_rows=rows, max_kv=1 << i) for i in range(9, 24)]
            got += [attn_bytes(S, L, n_seqs=n, n_rows=n * rows, max_rows=rows, max_kv=kv)
                    for kv in (1 << 24, 20000011, 1 << 25)]
            assert got[-1] >= 1 << 30 and all(b >= 0.9 * a for a, b in zip(got, got[1:])), got
    got = [attn_bytes(S, L, n_seqs=n, n_rows=n * 1024, max_rows=1024, max_kv=32768) for n in range(1, 40)]
    assert got[0] > 1 << 27 and got[-1] >= 1 << 30 and all(b >= 0.9 * a for a, b in zip(got, got[1:])), got


def test_workspace_of_a_type(S, L):
    """bf16 calls need what either type may; fp16 ones hold no copy."""
    kw = dict(n_seqs=1, n_rows=2048, max_rows=2048, max_kv=10240)
    assert attn_bytes(S, L, BF16, **kw) == attn_bytes(S, L, **kw) > 10240 * 8 * 128 * 4
    assert attn_bytes(S, L, FP16, **kw) <= attn_bytes(S, L, **kw) - 10240 * 8 * 128 * 4
    kw = dict(n_seqs=4, n_rows=32, max_rows=8, max_kv=8000)
    assert attn_bytes(S, L, FP16, **kw) == attn_bytes(S, L, BF16, **kw) == attn_bytes(S, L, **kw) > 0
    assert attn_bytes(S, L, FP32, **kw) == attn_bytes(S, L, 7, **kw) == 0
    assert attn_bytes(S, L, FP16, heads=33, **kw) == 0


def test_long_sequences_are_split(S, L):
    """Sequences of 16383 tokens are split over work-groups however many decode (partial sums need a
    workspace), but a call is not refused for its splits."""
    for n in (8, 48, 63, 64, 128, 200):
        assert attn_bytes(S, L, n_seqs=n, n_rows=n, max_rows=1, max_kv=16383) > 0, n
    assert attn_bytes(S, L, n_seqs=48, n_rows=256 + 47, max_rows=256, max_kv=16383) > 0
    for n, heads in ((65535, 64), (40000, 128)):
        s = seqs(S, n_seqs=n, n_rows=n, max_rows=1, max_kv=1 << 20, table_width=1 << 16, table_stride=1 << 16)
        c = cache(S, kv_heads=8, page_size=16)
        assert attn_call(S, L, c=c, s=s, heads=heads, ws=None, wn=0, q=None) == ARG   # refused for q, not for its size


@pytest.mark.parametrize("off,width,ok", [(1000, 4000, True), (3000, 4000, True), (-1000, 4000, True),
                                          (4000 * 3 + 2000, 4000, True), (999, 4000, False), (3001, 4000, False),
                                          (4000 * 3, 4000, False), (1000, 1999, False), (-999, 4000, False)])
def test_lora_columns_of_the_same_rows(S, L, off, width, ok):
    """y and out as columns of one tensor do not overlap where the columns do not (off: elements)."""
    status = lora_call(S, L, out=P[6] + 4 * off, ys=width, os=width)
    assert (status != ARG) if ok else (status == ARG)


def test_not_refused_for_splits(S, L):
    """Rows past max_rows are not computed, but they count where partial sums are joined."""
    s = seqs(S, n_seqs=64, n_rows=1 << 20, max_rows=1, max_kv=1 << 15, table_width=1 << 11, table_stride=1 << 11)
    assert attn_call(S, L, s=s, ws=None, wn=0, q=None) == ARG   # refused for q, not for its size
