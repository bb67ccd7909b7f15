"""A device may be given by its number, 0 among them, on the CPU."""
import contextlib

import pytest
import torch

from dense_fp32_gemm_02_gb300 import binding as b


def test_an_empty_checkpoint_is_made_on_device_zero(monkeypatch):
    made = []
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: made.append(device))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    b.act8_empty(3, 40, device=0)
    assert made == [0, 0]
    b.act8_empty(3, 40)
    assert made[2:] == [torch.device("cuda", 1)] * 2


@pytest.mark.parametrize("call", [lambda **k: b.device_status(**k), lambda **k: b.selftest_wait_timeout(1000, **k)])
def test_the_error_word_of_device_zero(monkeypatch, call):
    used = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: 0

    @contextlib.contextmanager
    def device(d):
        used.append(d)
        yield

    monkeypatch.setattr(b, "lib", Library())
    monkeypatch.setattr(b, "_stream_handle", lambda stream, device: None)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    call(device=0)
    call()
    assert used == [0, torch.device("cuda", 1)]
