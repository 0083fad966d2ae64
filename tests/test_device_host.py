"""Sizes that depend on a device are asked for on the tensors' device, not on the current one (no GPU: the library and the
devices are stand-ins)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture
def kv(monkeypatch):
    """The module with a library whose sizes are 1000 times the current device's number, which starts at 0."""
    from moe_nvfp4_gemv_gb300 import kvcache
    current = [0]

    @contextlib.contextmanager
    def device(index):
        current.append(index)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(kvcache, "_lib", SimpleNamespace(
        fp4gemv_kv_attention_shared_scratch_bytes=lambda *a: 1000 * current[-1],
        fp4gemv_kv_attention_workspace_bytes=lambda dim: 1000 * current[-1],
        fp4gemv_stream_capture_id=lambda stream: 0))
    monkeypatch.setattr(kvcache, "_raw_stream", lambda index: 77)
    monkeypatch.setattr(kvcache, "_workspaces", {})
    return kvcache


def test_scratch_of_another_device(kv):
    cache = kv.KvCache8.allocate(2, 1, 64, 16, device="cpu")
    cache._index = 3
    assert cache.shared_scratch_bytes(2, 1, 4) == 3000


def test_workspace_of_another_device(kv, monkeypatch):
    monkeypatch.setattr(kv.torch, "zeros", lambda n, dtype, device: (n, device))
    assert kv.attention_workspace(torch.device("cuda", 2), 64) == (2000, torch.device("cuda", 2))
