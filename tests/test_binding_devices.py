"""Both bindings launch on the tensors' device and its current stream, whatever
device is current (on the CPU: tensors and library are stand-ins)."""

import contextlib

import pytest
import torch


class Tensor:
    """What the bindings ask of a device tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32, device=1):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", device)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def stride(self, d=None):
        s = [self.shape[i + 1:].numel() for i in range(len(self.shape))]
        return tuple(s) if d is None else s[d]

    def data_ptr(self):
        return 4096


class Library:
    """Notes the device that is current at each call, and the call's stream."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            self.calls.append((name, self.state["device"], args[-1]))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    from w4_gemm_vqv_amd import round as r
    from w4_gemm_vqv_amd import vqv as v
    state = {"device": 0}

    @contextlib.contextmanager
    def device(d):
        before, state["device"] = state["device"], d.index
        yield
        state["device"] = before

    class Stream:
        def __init__(self, d):
            self.cuda_stream = 1000 + d.index

    L = Library(state)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: Stream(d or torch.device("cuda", state["device"])))
    monkeypatch.setattr(r, "_round_lib", lambda: L)
    monkeypatch.setattr(r, "_new", lambda shape, dtype, dev, stream: Tensor(
        *((shape,) if isinstance(shape, int) else shape), dtype=dtype, device=dev.index))
    monkeypatch.setattr(v, "lib", lambda: L)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(
        *((shape,) if isinstance(shape, int) else shape), dtype=dtype, device=device.index))
    L.r, L.v = r, v
    return L


def round_calls(r, d):
    t = lambda *s, dtype=torch.int32: Tensor(*s, dtype=dtype, device=d)
    cache = r.PagedCache(*(t(2, 8, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)))
    seqs = r.Sequences(t(3), t(2), t(2, 4), n_rows=6, max_rows=3, max_kv=64)
    pages = r.Pages(t(8), t(2, 4), t(2), t(2), page_size=16)
    edits = r.Edits(2, 100, counts=t(2, 100))
    f = torch.float32
    q, k = t(6, 4, 64, dtype=torch.bfloat16), t(6, 2, 64, dtype=torch.bfloat16)
    r.vqv_rope_append(q, k, k, cache, seqs, r.Rope(64))
    r.vqv_paged_attn(q, cache, seqs, scale=1.0)
    r.vqv_cache_copy(cache, t(3), t(3))
    r.vqv_cache_trim(pages, t(2))
    r.vqv_cache_reserve(pages, t(2))
    r.vqv_cache_fork(cache, pages, t(1), t(1))
    r.vqv_cache_compact(cache, seqs, t(6))
    r.vqv_logits_edit(t(6, 100, dtype=f), edits, t(2, 2), 2, 3)
    r.vqv_logits_verify(t(6, 100, dtype=f), edits, t(2, 2), 2, 3)
    return 9


def projection_calls(v, d):
    t = lambda *s, dtype=torch.int32: Tensor(*s, dtype=dtype, device=d)
    w = (t(100, 64, dtype=torch.uint8), t(100, 2, dtype=torch.float16), t(100, 2, dtype=torch.float16))
    x, logits, draft = t(4, 128, dtype=torch.bfloat16), t(4, 100, dtype=torch.float32), t(1, 3)
    v.vqv_qgemm(x, *w)
    v.vqv_qgemm_swiglu(x, *w)
    v.vqv_verify(logits, draft, 1, 4)
    v.vqv_verify_ex(logits, draft, 1, 4)
    v.vqv_qgemm_verify(x, *w, draft, 1, 4)
    v.vqv_qgemm_verify_ex(x, *w, draft, 1, 4)
    v.vqv_qgemm_verify_ex_noalloc(x, *w, draft, 1, 4)
    return 7


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("calls", [round_calls, projection_calls])
def test_calls_run_on_the_tensors_device(lib, calls, device):
    n = calls(lib.r if calls is round_calls else lib.v, device)
    launches = [c for c in lib.calls if c[0] != "vqv_rope_plan"]
    assert len(launches) == n
    for name, current, stream in launches:
        assert (current, stream) == (device, 1000 + device), name
    assert lib.state["device"] == 0
