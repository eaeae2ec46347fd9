"""The current stream's handle for every way of naming a device (CPU only; the
stream queries are stubbed)."""
from types import SimpleNamespace

import pytest
import torch

import fp8_fine_grained_quant_b200 as fq


@pytest.mark.parametrize("device,raw", [(0, False), (1, False), ("cuda:1", False), (torch.device("cuda"), False),
                                        (torch.device("cuda:0"), True), (torch.device("cuda:1"), True)])
@pytest.mark.parametrize("has_raw", [True, False])
def test_current_stream_of_a_device(monkeypatch, device, raw, has_raw):
    seen = []
    monkeypatch.setattr(fq, "_raw_stream", (lambda i: 100 + i) if has_raw else None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: seen.append(d) or SimpleNamespace(cuda_stream=7))
    if raw and has_raw:
        assert fq._stream(None, device) == 100 + device.index and not seen
    else:
        assert fq._stream(None, device) == 7 and seen == [device]


def test_a_given_stream_is_taken_as_it_is(monkeypatch):
    monkeypatch.setattr(fq, "_raw_stream", lambda i: 1 / 0)
    for device in (0, "cuda:0", torch.device("cuda:0")):
        assert fq._stream(SimpleNamespace(cuda_stream=41), device) == 41
        assert fq._stream(42, device) == 42


@pytest.mark.parametrize("device", [None, 0, "cuda:0", torch.device("cuda:0")])
def test_status_calls_take_a_device_in_every_form(monkeypatch, device):
    """Without a device the current one, an int."""
    class Here:
        def __init__(self, d):
            pass

        def __enter__(self):
            return self

        def __exit__(self, *a):
            return False

    got = []
    fake = SimpleNamespace(fp8q_get_device_error=lambda s: got.append(s) or 3,
                           fp8q_selftest_wait_timeout=lambda ns, s: got.append((ns, s)) or 0)
    monkeypatch.setattr(fq, "lib", lambda: fake)
    monkeypatch.setattr(fq, "_raw_stream", lambda i: 7)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "device", Here)
    assert fq.get_device_error(device=device) == 3
    fq.selftest_wait_timeout(1000, device=device)
    assert got == [7, (1000, 7)]


@pytest.mark.gpu
def test_status_calls_without_a_device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert fq.get_device_error() == fq.OK
    assert fq.get_device_error(device="cuda:0") == fq.OK
    fq.selftest_wait_timeout(1_000_000)
    assert fq.get_device_error() == fq.ERR_TIMEOUT
    assert fq.get_device_error() == fq.OK
