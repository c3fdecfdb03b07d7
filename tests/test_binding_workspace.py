"""The binding's workspaces, without a GPU: CPU tensors stand for the device's and a recorder for the library, called
behind the check for CUDA tensors."""
import gc
import weakref

import pytest
import torch

import selective_state_space_37_b200 as ss
from selective_state_space_37_b200 import _binding as bd

CPU = torch.device("cpu")


class FakeLib:
    """Answers every size with `need` bytes and hands every other call to `on_call(name, args)`."""

    def __init__(self, need, on_call):
        self.need, self.on_call = need, on_call

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: self.need
        return lambda *a: self.on_call(name, a) or ss.SS_OK


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(bd, "_stream_handle", lambda stream, device: 0)
    monkeypatch.setattr(bd, "_ws_cache", {})

    def install(need, on_call):
        monkeypatch.setattr(bd, "lib", lambda: FakeLib(need, on_call))
    return install


def gdr_args(B=1, L=20, H=2, d=64):
    x = torch.zeros(B, L, H, d)
    g = torch.zeros(B, L, H)
    return x, x, x, g, torch.zeros(H), g


def norm_args(rows=4, cols=8):
    x = torch.zeros(rows, cols)
    return x, x, torch.zeros(rows), torch.zeros(rows)


CALLS = {"ss_gdr_fwd": lambda: bd.ss_gdr_fwd.__wrapped__(*gdr_args()),
         "ss_gdr_bwd": lambda: bd.ss_gdr_bwd.__wrapped__(*gdr_args(), torch.zeros(1, 20, 2, 64)),
         "ss_norm_bwd": lambda: bd.ss_norm_bwd.__wrapped__(*norm_args())}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_workspace_lives_until_the_library_returns(name, fake, monkeypatch):
    """A larger request for the same stream replaces the cached buffer; the call that was given the first one still
    has to launch on it."""
    held = []
    plain = bd.workspace_for

    def tracked(nbytes, device, handle):
        ws = plain(nbytes, device, handle)
        held.append(weakref.ref(ws))
        return ws

    monkeypatch.setattr(bd, "workspace_for", tracked)
    alive = []

    def on_call(called, args):
        assert called == name
        plain(1 << 20, CPU, 0)
        gc.collect()
        alive.append(held[0]() is not None)

    fake(4096, on_call)
    CALLS[name]()
    assert alive == [True]
