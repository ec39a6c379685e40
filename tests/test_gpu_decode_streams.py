"""The decoding calls on other streams: with ``stream=`` while the current stream is busy, and two
streams' calls at once on pools of their own.  The results are those of calls one after the other."""
import pytest
import torch

import test_gpu_draft_step as ds
import test_gpu_draft_verify as dv
from test_gpu_state_pool import i32, pool
from test_gpu_stream_argument import WAIT, _stream_of

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def busy(kw):
    """Before a call with ``stream=``: the state is there, and the current stream has work to do."""
    if "stream" in kw:
        torch.cuda.synchronize()
        torch.cuda._sleep(WAIT)


def _calls():
    """Name -> (a call with fresh state, its outputs and what it writes)."""
    import chunked_linear_recurrence_gb300 as sf
    x = ds.case(9, 5, 4, 4, 2, 128, BF16, True, 51)
    y = ds.case(9, 12, 11, 4, 2, 64, torch.float32, False, 52)
    v = dv.make(6, 3, 5000, torch.float32, True, 53)
    small, large = pool(40, 54), pool(4200, 55, ((8,),))
    idx, parents = i32(range(1, 21)), i32([0] * 10 + list(range(10)))

    def draft(z):
        def f(**kw):
            w = dict(z, cache=z["cache"].clone())
            busy(kw)
            return [ds.call(w, **kw), w["cache"]]
        return f

    def move(fn, caches, *args):
        def f(**kw):
            c = [t.clone() for t in caches]
            busy(kw)
            return [fn(c, *args, **kw), *c]
        return f
    return {"gdn_draft_step": draft(x), "linattn_draft_step": draft(y),
            "verify": lambda **kw: busy(kw) or list(dv.call(v, **kw)),
            "fork": move(sf.sf_state_fork, small, idx, parents),
            "fork with a workspace": move(sf.sf_state_fork, large, idx, parents),
            "compact": move(sf.sf_state_compact, small, i32([39, 1, 7, 38]))}


NAMES = ["gdn_draft_step", "linattn_draft_step", "verify", "fork", "fork with a workspace", "compact"]


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream(name):
    run = _calls()[name]
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    got = run(stream=side)
    assert _stream_of(got[0]) == side.cuda_stream
    side.synchronize()
    assert not torch.cuda.current_stream().query()        # nothing waited for the current stream
    torch.cuda.synchronize()
    assert all(map(torch.equal, got, want))


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name):
    run = _calls()[name]
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT // 10)
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert all(map(torch.equal, g, want))
