"""The binding's workspaces, without a GPU: CPU tensors stand for the device's and a recorder for the library, called
behind the check for CUDA tensors."""
import contextlib
import gc
import threading
import time
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


def conv_call(**kw):
    x, g, s = torch.zeros(1, 8, 64), torch.zeros(1, 8, 16), torch.zeros(64)
    return bd.ss_fwd_conv(x, torch.zeros(64, 4), x, torch.zeros(64, 16), g, g, D=s, z=x, delta_bias=s, **kw)


def ssd_call(**kw):
    x, h, b = (torch.zeros(1, 8, *s, dtype=torch.bfloat16) for s in ((2, 64), (2,), (64,)))
    return bd.ss_ssd_fwd(x, h, torch.zeros(2), b, b, **kw)


SHARED = {**CALLS, "ss_fwd_conv": conv_call, "ss_ssd_fwd": ssd_call}


@pytest.mark.parametrize("name", sorted(SHARED))
def test_host_threads_on_one_stream_launch_in_turn(name, fake):
    """Two threads' calls on one stream share a workspace: no launch of the second comes between the first one's."""
    inside, most = [], []

    def on_call(called, args):   # a call's launches take a while, without the interpreter's lock
        inside.append(called)
        most.append(len(inside))
        time.sleep(0.02)
        inside.pop()

    fake(4096, on_call)
    threads = [threading.Thread(target=SHARED[n]) for n in (name, "ss_gdr_bwd", name)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(10)
    assert len(most) == 3 and max(most) == 1


def test_streams_do_not_wait_for_one_another(fake, monkeypatch):
    """The lock is the stream's: a call on another stream goes ahead."""
    monkeypatch.setattr(bd, "_stream_handle", lambda stream, device: threading.get_ident())
    both = threading.Barrier(2, timeout=10)
    fake(4096, lambda called, args: both.wait() and None)
    threads = [threading.Thread(target=CALLS["ss_norm_bwd"]) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(10)
    assert not both.broken


class FakeStream:
    cuda_stream = 7


OUTPUTS = {
    "ss_gdr_fwd": (lambda **kw: bd.ss_gdr_fwd.__wrapped__(*gdr_args(), seqlens=torch.zeros(1, dtype=torch.int32), **kw), 2),
    "ss_gdr_bwd": (lambda **kw: bd.ss_gdr_bwd.__wrapped__(*gdr_args(), torch.zeros(1, 20, 2, 64), **kw), 6),
    "ss_gdr_step": (lambda **kw: bd.ss_gdr_step.__wrapped__(torch.zeros(1, 2, 64, 64), *(t[:, 0].contiguous() if t.dim() > 1 else t
                                                                                      for t in gdr_args()), **kw), 1),
    "ss_fwd_conv": (conv_call, 2), "ss_ssd_fwd": (ssd_call, 2),
    "ss_norm_fwd": (lambda **kw: bd.ss_norm_fwd.__wrapped__(torch.zeros(4, 8), **kw), 3),
    "ss_norm_bwd": (lambda **kw: bd.ss_norm_bwd.__wrapped__(*norm_args(), **kw), 3)}


@pytest.mark.parametrize("name", sorted(OUTPUTS))
def test_outputs_are_made_on_the_calls_stream(name, fake, monkeypatch):
    """The allocator's blocks belong to a stream: every tensor that a call makes comes from the stream it launches on."""
    call, count = OUTPUTS[name]
    on, made = [], []

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        try:
            yield
        finally:
            on.pop()

    def tracked(fn):
        def make(*a, **kw):
            made.append(on[-1] if on else None)
            return fn(*a, **kw)
        return make

    fake(4096, lambda called, args: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for n in ("empty", "empty_like", "zeros", "zeros_like"):
        monkeypatch.setattr(torch, n, tracked(getattr(torch, n)))
    st = FakeStream()
    call(stream=st)   # (the inputs' own torch.zeros come first, on no stream)
    ours = made[len([m for m in made if m is None]):]
    assert made == [None] * (len(made) - len(ours)) + ours and set(ours) == {st}
    assert len(ours) >= count   # (and the workspace)


@pytest.mark.parametrize("name", sorted(SHARED))
def test_captured_calls_have_workspaces_of_their_own(name, fake, monkeypatch):
    """Graphs may be replayed at once, and the cached buffer may be replaced: a capture leaves the cache alone."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    fake(4096, lambda called, args: None)
    SHARED[name]()
    assert not bd._ws_cache
