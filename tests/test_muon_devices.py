"""Which device and stream the Newton-Schulz, Muon and embedding calls use, on a library that records its
calls: no GPU is needed, and a second one is only named."""
from __future__ import annotations

import types

import pytest
import torch

from rank_gradient_compression_powersgd_amd import binding as B
from rank_gradient_compression_powersgd_amd.group import PowerSGDGroup


class _Library:
    """Accepts every call and keeps its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            if name == "psgd_create":
                args[0]._obj.value = 4096 + args[1]                  # a handle per device
            return 0 if name != "psgd_last_error" else b""
        return call

    def args(self, name):
        return [a for n, a in self.calls if n == name]


class _On:
    """A tensor that says it lives on another device."""

    def __init__(self, t, index):
        self._t, self.device = t, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture()
def lib(monkeypatch):
    one = _Library()
    monkeypatch.setattr(B, "load_library", lambda path=None: one)
    # device 0 is current; the stream of device k is 100 + k

    def current_stream(device=None):
        index = device if isinstance(device, int) else 0 if device is None else torch.device(device).index
        return types.SimpleNamespace(cuda_stream=100 + index)

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    return one


def _hp():
    return B.muon_hparams(0.1)


def test_newton_schulz_and_muon_take_their_contexts_stream(lib):
    ctx = B.psgd_create(1, 4)
    skip = _On(torch.zeros(1, dtype=torch.int32), 1)
    B.psgd_newton_schulz(ctx, 7)
    B.psgd_muon_update(ctx, 7, skip, None, _hp())
    assert lib.args("psgd_newton_schulz")[0][-1] == 101
    assert lib.args("psgd_muon_update")[0][-1] == 101
    B.psgd_newton_schulz(ctx, 7, stream=55)
    assert lib.args("psgd_newton_schulz")[1][-1] == 55
    B.psgd_destroy(ctx)
    B.psgd_newton_schulz(ctx, 7)                                     # a context made elsewhere: the current device
    assert lib.args("psgd_newton_schulz")[2][-1] == 100


class _Group(PowerSGDGroup):
    """Its handles are no library's: nothing is destroyed."""

    def close(self):
        pass


def _group(device):
    g = _Group.__new__(_Group)
    g.torch, g.ctx, g.plan = torch, B.psgd_create(device, 4), 7
    g.err = [torch.zeros(4, 8)]
    g.scale = torch.ones(1)
    g.flags, g.skip = _On(torch.zeros(1, dtype=torch.uint8), 1), _On(torch.zeros(1, dtype=torch.int32), 1)
    g.adam_step, g.adam_norm = torch.zeros(1, dtype=torch.int32), torch.zeros(2)
    return g


def test_one_stream_through_the_whole_muon_step(lib):
    """Every launch of a step goes to one stream, the current one of the group's device."""
    g = _group(1)
    g.attach_muon([_On(torch.zeros(4, 8), 1)], [_On(torch.zeros(4, 8), 1)])
    x = torch.zeros(6)
    g.step_muon(_hp(), [(x, x, x, x)], B.psgd_adam_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0), max_norm=1.0)
    names = ["psgd_compress", "psgd_check_finite", "psgd_adam_prepare", "psgd_decompress_update", "psgd_muon_update", "psgd_adam_update"]
    assert [n for n, _ in lib.calls if n in names] == names
    for n in names:
        assert lib.args(n)[0][-1] == 101, n


def test_tensors_on_another_device_than_the_context_are_refused(lib):
    """A launch on the context's device would read the other device's memory."""
    ctx = B.psgd_create(0, 1)
    table, ids, rows = _On(torch.zeros(5, 8), 1), _On(torch.zeros(3, dtype=torch.int64), 1), _On(torch.zeros(3, 8), 1)
    for call in (lambda c: B.psgd_embed_lookup(c, table, ids, rows),
                 lambda c: B.psgd_embed_grad(c, rows, ids, table, workspace=_On(torch.zeros(1 << 16, dtype=torch.uint8), 1))):
        with pytest.raises(B.PsgdError) as ei:
            call(ctx)
        assert ei.value.status == B.PSGD_EINVAL and "context" in str(ei.value)
    g = _group(0)
    with pytest.raises(B.PsgdError) as ei:
        g.attach_muon([_On(torch.zeros(4, 8), 1)], [_On(torch.zeros(4, 8), 1)])
    assert ei.value.status == B.PSGD_EINVAL and "context" in str(ei.value)
    assert not [n for n, _ in lib.calls if n in ("psgd_embed_lookup", "psgd_embed_grad", "psgd_muon_attach")]
    there = B.psgd_create(1, 1)
    B.psgd_embed_lookup(there, table, ids, rows)
    B.psgd_embed_grad(there, rows, ids, table, workspace=_On(torch.zeros(1 << 16, dtype=torch.uint8), 1))
    assert lib.args("psgd_embed_lookup")[0][-1] == 101 and lib.args("psgd_embed_grad")[0][-1] == 101
