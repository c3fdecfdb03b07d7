"""GPU tests of calls from several host threads, and of outputs made for a call on another stream."""
import threading

import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import call_args, gdr_inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def gdr_call(L, seed, **kw):
    x = gdr_inputs(2, L, 4, 2, 128, 128, seed=seed, init=True)
    dy = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)

    def call(**kw):
        y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], **kw)
        g = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], **kw)
        return [y, S, *(g[n] for n in sorted(g))]
    return call


def norm_call(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn(rows, cols, generator=g).to(BF).to(DEV) for _ in range(2))

    def call(**kw):
        y, mean, rstd = ss.ss_norm_fwd(x, **kw)
        d = ss.ss_norm_bwd(dy, x, mean, rstd, **kw)
        return [y, mean, rstd, *(d[n] for n in sorted(d))]
    return call


def test_two_threads_on_one_stream():
    """Calls with workspaces of different sizes, from two host threads on one stream: the results of the calls in
    turn."""
    calls = [[gdr_call(40 + 90 * i, i) for i in range(4)] + [norm_call(300, 640, 1)],
             [norm_call(2000, 520, 2), gdr_call(700, 9), gdr_call(20, 10), norm_call(64, 4096, 3)]]
    want = [[c() for c in some] for some in calls]
    torch.cuda.synchronize()
    ss.clear_workspaces()
    got, failed = [[], []], []

    def work(i):
        try:
            for _ in range(20):
                got[i].append([c() for c in calls[i]])
        except Exception as e:   # (a thread's exception is lost otherwise)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        for again in got[i]:
            assert all(torch.equal(a, b) for g, w in zip(again, want[i]) for a, b in zip(g, w))


@pytest.mark.parametrize("make", [lambda: gdr_call(200, 3), lambda: norm_call(500, 640, 4)], ids=["delta rule", "norm"])
def test_outputs_on_another_stream_leave_pending_work_alone(make):
    """Blocks freed while work queued on the current stream still reads them are not what a call on another stream
    writes to."""
    call = make()
    want = call()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    call(stream=st)   # (the inputs' copies are done; the stream's own workspace exists)
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.full_like(t, 7) for t in want]
        torch.cuda._sleep(20_000_000)                       # some 10 ms: the copies below wait behind it
        copies = [t.clone() for t in old]
        del old
        got = call(stream=st)
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies)
