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


def test_errors_of_a_chain_are_read_on_the_calls_stream(allocations, monkeypatch):
    """gptq_sequential reads the layers' errors behind the work on its stream."""
    read = []

    class Errors(_Tensor):
        def cpu(self):
            read.append(torch.cuda.current_stream())
            return torch.zeros(1, dtype=torch.float64)

        def data_ptr(self):
            return 4096

        def numel(self):
            return 0

        def __getitem__(self, k):
            return self

        def view(self, *shape):
            return self

    class Lib:
        gq_gptq_sequential_workspace_size = staticmethod(lambda *a: 256)
        gq_gptq_sequential = staticmethod(lambda *a: 0)
    monkeypatch.setattr(gq, "lib", Lib)
    monkeypatch.setattr(gq, "_stream", lambda s: 0)
    monkeypatch.setattr(gq, "_dev", lambda t, *a: t)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Errors(torch.cuda.current_stream()))
    X, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64)
    for stream, expected in (("side", "side"), (None, "main")):
        read.clear()
        gq.gptq_sequential(X, [dict(W=W)], stream=stream)
        assert read == [expected]
