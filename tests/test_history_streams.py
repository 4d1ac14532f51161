"""The history tower on a stream that is not the current one: every library
call, and what torch does between them, has to go to that stream.  The library
and the stream context are recorders here; nothing runs on a device."""
from contextlib import contextmanager

import pytest
import torch

from deep_learning_recommendation_amd import history

H, W, D, V = 2, 8, 16, 10


class Recorder:
    """Stands in for the library: notes each call's stream argument and the
    stream that is current meanwhile."""

    def __init__(self):
        self.calls, self.current = [], None

    @contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def __getattr__(self, name):
        if name.startswith("DLRM_"):
            return 0
        if name.endswith("_size"):
            return lambda *a: 256
        return lambda *a: self.calls.append((name, a[-1], self.current))


def noted(lib, what, call):
    def wrapped(*a, **k):
        lib.calls.append((what, lib.current, lib.current))
        return call(*a, **k)
    return wrapped


@pytest.fixture
def lib(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(history, "C", lib)
    monkeypatch.setattr(torch.cuda, "stream", lib.stream)
    for name, what in (("empty", "buffer"), ("where", "indices")):
        monkeypatch.setattr(torch, name, noted(lib, what, getattr(torch, name)))
    return lib


def _tower(train):
    layers = [history.make_layer(torch.ones(D), torch.zeros(H * 3 * W, D), torch.zeros(D, H * W), torch.ones(H), "cpu")]
    return history.HistoryTower(torch.zeros(V, D), layers, torch.ones(D), H, W, W, train=train)


def test_every_call_goes_to_the_given_stream(lib):
    tok, off = torch.arange(5), torch.tensor([0, 2, 2, 5])
    out, S = torch.zeros(3, D), object()
    tower, serving = _tower(True), _tower(False)
    lib.calls.clear()
    tower.forward(tok, off, 3, out, D, stream=S)
    tower.backward(out, D, stream=S)
    serving.forward(tok, off, 3, out, D, stream=S)
    serving.forward(tok[:0], torch.zeros(4, dtype=torch.int64), 0, out, D, stream=S)
    serving.step(tok[:3], [None], None, out, D, stream=S)
    names = {c[0] for c in lib.calls}
    assert {"buffer", "indices", "dlrm_linattn_fwd", "dlrm_linattn_bwd", "dlrm_linattn_step"} <= names
    assert all(c[1] is S and c[2] is S for c in lib.calls), [c for c in lib.calls if c[1] is not S or c[2] is not S][:5]
    assert lib.current is None


def test_a_step_of_nobody_makes_no_call(lib):
    out, serving = torch.zeros(0, D), _tower(False)
    lib.calls.clear()
    assert serving.step(torch.zeros(0, dtype=torch.int64), [None], None, out, D) is out
    assert not lib.calls
