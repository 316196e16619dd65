"""The loss calls make what they allocate, and read their status, in the context
of the stream that they are given (no GPU: the library, the context and the
output tensors are stand-ins that note where they were used)."""

from types import SimpleNamespace

import pytest
import torch

from rnn_joint_network_02_b200 import frnnt


class Place:
    """Stands for the stream's context; `inside` while it is entered."""
    inside = False

    def __enter__(self):
        Place.inside = True

    def __exit__(self, *_):
        Place.inside = False


@pytest.fixture
def seen(monkeypatch):
    """What a call did, in order: (what, in the stream's context)."""
    log = []

    class Status:
        def __getitem__(self, _):
            return self

        def item(self):
            log.append(("status read", Place.inside))
            return 0

    class Outputs(SimpleNamespace):
        def __init__(self, f, g, *_, **__):
            log.append(("outputs", Place.inside))
            super().__init__(loss=torch.zeros(2), df=f, dg=g, status=Status(), dropped=None,
                             workspace=torch.zeros(4), **{k: f for k in ("dW_f", "dW_g", "dW_o", "db_o", "dW_d", "db_d")})

        def grads(self):
            return dict(df=self.df, dg=self.dg)

    class Library:
        def __getattr__(self, name):
            def call(*_):
                log.append((name, Place.inside))
                return 0
            return call

    def dropout(x, p, seed, offset=0, out=None, stream=None):
        log.append(("dropout", Place.inside and stream is None))
        return x if out is None else out

    empty_like = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda t: log.append(("dropped", Place.inside)) or empty_like(t))
    monkeypatch.setattr(frnnt, "Outputs", Outputs)
    monkeypatch.setattr(frnnt, "dropout", dropout)
    monkeypatch.setattr(frnnt, "lib", Library)
    monkeypatch.setattr(frnnt, "_check_call", lambda *_, **__: None)
    monkeypatch.setattr(frnnt, "_ptr", lambda t: None)
    monkeypatch.setattr(frnnt, "_queue", lambda dev: None)
    monkeypatch.setattr(frnnt, "_elsewhere", lambda dev, stream: None if stream is None else Place())
    return log


F, G, W, B = torch.zeros(2, 3, 4), torch.zeros(2, 2, 4), torch.zeros(5, 4), torch.zeros(5)
STREAM = SimpleNamespace(device=torch.device("cpu"), cuda_stream=1234)
CALLS = {
    "fwd_bwd": lambda **k: frnnt.fwd_bwd(F, G, W, W, W, B, None, None, None, **k),
    "noalloc": lambda **k: frnnt.fwd_bwd_noalloc(F, G, W, W, W, B, None, None, None, **k),
    "pruned": lambda **k: frnnt.fwd_bwd_pruned(F, G, W, W, W, B, None, None, None, None, 2, **k),
    "tdt": lambda **k: frnnt.fwd_bwd_tdt(F, G, W, W, W, B, W, B, None, None, None, (0, 1), **k),
}


@pytest.mark.parametrize("drop", [None, frnnt.Dropout(0.5, 1)])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("entry", CALLS)
def test_everything_is_done_on_the_given_stream(seen, monkeypatch, entry, own, drop):
    monkeypatch.setattr(frnnt, "_current_device", lambda: 0)
    out = frnnt.Outputs(F, G) if own else None
    del seen[:]
    CALLS[entry](stream=STREAM, dropout=drop, out=out)
    assert not Place.inside and all(inside for _, inside in seen), seen
    names = [n for n, _ in seen]
    assert ("outputs" in names) != own and "status read" in names and sum(n.startswith("frnnt_fwd") for n in names) == 1
    assert names.count("dropout") == (4 if drop else 0) and names.count("dropped") == (2 if drop and own else 0)
    if own and drop:        # the buffers are made once
        del seen[:]
        CALLS[entry](stream=STREAM, dropout=drop, out=out)
        assert "dropped" not in [n for n, _ in seen]


@pytest.mark.parametrize("entry", CALLS)
def test_no_context_without_a_stream(seen, entry):
    CALLS[entry]()
    assert seen and not any(inside for _, inside in seen)


def test_no_context_for_the_current_stream(monkeypatch):
    """A program that names the stream that is current anyway pays for no context; another stream, a stream of another
    device and another current device are not taken for it."""
    dev = torch.device("cuda", 0)
    monkeypatch.setattr(frnnt, "_current_device", lambda: 0)
    monkeypatch.setattr(frnnt, "_raw_stream", lambda index: 77 + index)
    monkeypatch.setattr(frnnt, "_elsewhere", lambda *a: a)
    same = SimpleNamespace(device=dev, cuda_stream=77)
    assert frnnt._loss_place(dev, same) is None
    assert frnnt._loss_place(dev, None) == (dev, None)
    for s in (SimpleNamespace(device=dev, cuda_stream=78), SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)):
        assert frnnt._loss_place(dev, s) == (dev, s)
    monkeypatch.setattr(frnnt, "_current_device", lambda: 1)
    assert frnnt._loss_place(dev, same) == (dev, same)
