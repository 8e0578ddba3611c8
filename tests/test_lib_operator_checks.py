"""CPU-only checks of what the operator classes refuse before they call the library."""
import itertools
import random
from types import SimpleNamespace

import pytest
import torch

import grouped_gemm_device_gb300 as g

F32, ONE, TWO = torch.float32, torch.device("cuda", 0), torch.device("cuda", 1)


class Stub:
    """What the checks ask of a tensor, on a device that need not exist."""
    dtype, shape, is_cuda = F32, (4, 8), True

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True


def test_tensors_of_another_device_are_refused():
    t = Stub(ONE)
    assert g._expect(t, "x", F32, (4, 8), 0) is t
    for other in (Stub(TWO), torch.zeros(4, 8)):
        with pytest.raises(ValueError, match="cuda:0"):
            g._expect(other, "x", F32, (4, 8), 0)
    for grads, outs in (([t, Stub(TWO)], None), ([t], [Stub(TWO)])):
        with pytest.raises(ValueError, match="one device"):
            g.GradClip(grads, outs)


def test_calls_need_their_device_to_be_current(monkeypatch):
    monkeypatch.setattr(g, "_cuda", SimpleNamespace(
        _cuda_getDevice=lambda: 1, _cuda_getCurrentRawStream=lambda d: 70 + d))
    assert g._call_stream(1, None) == 71 and g._call_stream(1, 5) == 5
    for stream in (None, 5):
        with pytest.raises(ValueError, match="current"):
            g._call_stream(0, stream)


def test_buffers_are_made_on_a_gpu():
    for make in (lambda: g.RouterLoss(8, 2, 4, device="cpu"),
                 lambda: g.LayerNorm(8, 4, device="cpu"),
                 lambda: g.Fp8Linear(8, 8, 4, device="cpu")):
        with pytest.raises(ValueError, match="GPU"):
            make()
    assert g._gpu("cuda:1") == TWO


def test_written_tensors_that_share_memory_are_found():
    """Against every pair of spans: two that overlap, at least one of them written."""
    r = random.Random(0)
    seen = set()
    for _ in range(3000):
        def span():
            return r.randrange(1, 60), r.choice([0, 1, 2, 5, 12])
        grads = [span() for _ in range(r.randrange(1, 5))]
        outs = [s if r.random() < 0.5 else span() for s in grads]
        items = [(o, True) for o in outs] + [(a, False) for a, o in zip(grads, outs) if a != o]
        want = any((wa or wb) and max(a[0], b[0]) < min(a[0] + a[1], b[0] + b[1])
                   for (a, wa), (b, wb) in itertools.combinations(items, 2))
        assert g._collide(grads, outs) == want
        seen.add(want)
    assert seen == {True, False}
