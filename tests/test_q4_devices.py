"""Workspace sizes follow the current device: they are multiples of its SM
count (a stand-in library on the CPU, no launch)."""
import types

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m


@pytest.fixture
def two_devices(monkeypatch):
    """A process with a second device that needs twice the workspace. Gives the current device's holder."""
    now = types.SimpleNamespace(device=0)
    size = lambda *a: 1024 * (now.device + 1)
    stub = types.SimpleNamespace(kv_q4_attend_workspace_bytes=size, spec_logprobs_workspace_bytes=size,
                                 kv_q4_attend=lambda *a: 0, spec_logprobs=lambda *a: 0)
    monkeypatch.setattr(m, "lib", lambda: stub)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now.device)
    yield now
    m._attend_bytes.cache_clear()
    m._logprobs_bytes.cache_clear()


def test_attend_asks_for_each_device(two_devices):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    kv = torch.zeros(4, 7, 16, 72, dtype=torch.uint8)
    cache, q = m.kv_q4_cache(kv, kv.clone()), torch.zeros(3, 91, 128)
    call = lambda ws: m.kv_q4_attend(cache, q, i32(1, 4), i32(2), i32(1), torch.zeros_like(q), ws, 29, 0.1, stream=0)
    size = m.kv_q4_attend_workspace_bytes(cache, 91, 29, q.dtype)
    ws = torch.zeros(size, dtype=torch.uint8)
    call(ws)
    two_devices.device = 1
    assert m.kv_q4_attend_workspace_bytes(cache, 91, 29, q.dtype) == 2 * size
    with pytest.raises(m.MTPError):
        call(ws)
    two_devices.device = 0
    assert m.kv_q4_attend_workspace_bytes(cache, 91, 29, q.dtype) == size
    call(ws)


def test_logprobs_asks_for_each_device(two_devices):
    call = lambda ws: m.spec_logprobs(torch.zeros(2, 977), torch.zeros(2, dtype=torch.int32), torch.zeros(2), ws, stream=0)
    size = m.spec_logprobs_workspace_bytes(2, 977, 0)
    ws = torch.zeros(size, dtype=torch.uint8)
    call(ws)
    two_devices.device = 1
    assert m.spec_logprobs_workspace_bytes(2, 977, 0) == 2 * size
    with pytest.raises(m.MTPError):
        call(ws)
