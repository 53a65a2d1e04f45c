"""Where a call's tensors come from when it goes to a stream of its own (no GPU: torch's allocation
and streams are stood in for)."""
import contextlib

import pytest
import torch

from post_weight_quantization_27_b200 import gq


class _Tensor:
    def __init__(self, pool):
        self.pool, self.known, self.device = pool, [], "gpu"

    def record_stream(self, s):
        self.known.append(s)


@pytest.fixture
def allocations(monkeypatch):
    """torch.empty as tensors that know the stream that was current when they were made."""
    current = ["main"]

    @contextlib.contextmanager
    def on(s):
        before, current[0] = current[0], s if s is not None else current[0]
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[0])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: _Tensor(current[0]))


def test_tensors_of_a_call_on_another_stream_are_that_streams(allocations):
    t = gq.workspace(256, "gpu", "side")
    assert t.pool == "side" and t.known == ["main"]
    q = gq._outputs(8, 64, -1, False, "gpu", True, 4, "side")
    for k in ("qpacked", "scales", "zeros", "g_idx"):
        assert q[k].pool == "side" and q[k].known == ["main"]


def test_tensors_of_a_call_on_the_current_stream_are_plain(allocations):
    t = gq.workspace(256, "gpu")
    assert t.pool == "main" and t.known == []
