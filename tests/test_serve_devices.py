"""The binding of the operators for many requests launches on the tensors' device and its current
stream, and refuses tensors of two devices (on the CPU: tensors and library are stand-ins)."""

import pytest
import torch

from .test_binding_devices import Tensor, lib  # noqa: F401 (a fixture)


@pytest.fixture
def serve(lib, monkeypatch):  # noqa: F811
    from w4_gemm_vqv_amd import serve as s
    monkeypatch.setattr(s, "_serve_lib", lambda: lib)
    monkeypatch.setattr(s, "_new", lib.r._new)
    monkeypatch.setattr(s, "vqv_q4_record_bytes", lambda dim: 48)
    return s


def calls(s, r, d, other=None):
    """Each call with all tensors on device d, or one of them on `other`."""
    here = lambda *shape, dtype=torch.int32: Tensor(*shape, dtype=dtype, device=d)
    there = lambda *shape, dtype=torch.int32: Tensor(*shape, dtype=dtype, device=d if other is None else other)
    half, f = torch.bfloat16, torch.float32
    cache = s.PagedCacheQ4(*(here(2, 8, 16, 2, 48, dtype=torch.uint8) for _ in range(2)), 64)
    seqs = r.Sequences(here(3), here(2), here(2, 4), n_rows=6, max_rows=3, max_kv=64)
    q, k = there(6, 4, 64, dtype=half), here(6, 2, 64, dtype=half)
    ad = s.Adapters(here(2, 8, 64, dtype=half), here(2, 100, 8, dtype=half), here(2, dtype=f), here(2))
    return [
        lambda: s.vqv_rope_append_q4(q, k, k, cache, seqs, r.Rope(64)),
        lambda: s.vqv_cache_q4_read(cache, seqs, k_out=there(6, 2, 64, dtype=f)),
        lambda: s.vqv_paged_attn_q4(q, cache, seqs, scale=1.0),
        lambda: s.vqv_verify_sampled(here(6, 100, dtype=f), here(2, 2), there(2, 3, dtype=f), 2, 3),
        lambda: s.vqv_lora_add(here(6, 64, dtype=half), ad, there(6), here(6, 100, dtype=f)),
    ]


@pytest.mark.parametrize("device", [0, 1])
def test_calls_run_on_the_tensors_device(lib, serve, device):  # noqa: F811
    todo = calls(serve, lib.r, device)
    for call in todo:
        call()
    launches = [c for c in lib.calls if c[0] != "vqv_rope_plan"]
    assert len(launches) == len(todo)
    for name, current, stream in launches:
        assert (current, stream) == (device, 1000 + device), name
    assert lib.state["device"] == 0


def test_tensors_of_two_devices_are_refused(lib, serve):  # noqa: F811
    for call in calls(serve, lib.r, 0, other=1):
        with pytest.raises(ValueError):
            call()
    assert not [c for c in lib.calls if c[0] != "vqv_rope_plan"]


def test_caches_and_adapters_of_two_devices_are_refused(lib, serve):  # noqa: F811
    k = Tensor(2, 8, 16, 2, 48, dtype=torch.uint8, device=0)
    with pytest.raises(ValueError):
        serve.PagedCacheQ4(k, Tensor(2, 8, 16, 2, 48, dtype=torch.uint8, device=1), 64)
    a, b = Tensor(2, 8, 64, dtype=torch.bfloat16, device=0), Tensor(2, 100, 8, dtype=torch.bfloat16, device=1)
    with pytest.raises(ValueError):
        serve.Adapters(a, b, Tensor(2, dtype=torch.float32, device=0))
