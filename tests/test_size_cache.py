"""The binding keeps the library's answers to workspace size questions, per
device: on the CPU, with a library and devices that are made up."""
import contextlib

import pytest
import torch

from paged_kv_cache_255_gb300 import pagedattn as pa


class Devices:
    """Two devices of different sizes; counts the questions asked."""

    def __init__(self):
        self.current, self.asked, self.broken = 0, 0, False

    @contextlib.contextmanager
    def device(self, index):
        before, self.current = self.current, self.current if index is None else index
        yield
        self.current = before

    def pa_decode_shared_workspace_size(self, *args):
        self.asked += 1
        return 0 if self.broken else 1000 * (self.current + 1) + args[0]


@pytest.fixture
def dev(monkeypatch):
    d = Devices()
    monkeypatch.setattr(pa, "lib", lambda: d)
    monkeypatch.setattr(pa, "_sizes", {})
    monkeypatch.setattr(torch.cuda, "device", d.device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: d.current)
    return d


@pytest.mark.parametrize("device", [None, "cuda", torch.device("cuda")])
def test_a_device_without_an_index_is_the_current_one(dev, device):
    assert pa.decode_shared_workspace_size(5, 1, 16, 8, device=device) == 1005
    dev.current = 1
    assert pa.decode_shared_workspace_size(5, 1, 16, 8, device=device) == 2005
    assert pa.decode_shared_workspace_size(5, 1, 16, 8, device="cuda:0") == 1005
    assert dev.asked == 2


def test_no_size_is_not_kept(dev):
    dev.broken = True
    with pytest.raises(ValueError):
        pa.decode_shared_workspace_size(5, 1, 16, 8)
    dev.broken = False
    assert pa.decode_shared_workspace_size(5, 1, 16, 8) == 1005


def test_the_answers_kept_are_bounded(dev):
    for n in range(1, 3 * pa._MOST_SIZES):
        assert pa.decode_shared_workspace_size(n, 1, 16, 8) == 1000 + n
        assert len(pa._sizes) <= pa._MOST_SIZES
    asked = dev.asked
    assert pa.decode_shared_workspace_size(n, 1, 16, 8) == 1000 + n and dev.asked == asked
