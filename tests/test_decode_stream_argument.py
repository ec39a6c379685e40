"""The decoding calls with ``stream=`` make their own buffers on that stream (as
test_stream_argument has it for the others): with a recording library in place of the real one."""
import contextlib

import pytest
import torch

from test_stream_argument import Lib, Stream

N, T, P, H, HK, D = 2, 3, 2, 4, 2, 64


def calls(sf):
    z = torch.zeros
    i32 = lambda *s: z(*s, dtype=torch.int32)   # noqa: E731
    q, v, g, cache, idx, dec = z(N, T, HK, D), z(N, T, H, D), z(N, T, H), z(4, H, D, D), i32(N), z(H)
    pend = (z(N, P, HK, D), z(N, P, H, D), z(N, P, H), z(N, P, H))
    probs, x, u = z(N, T + 1, 9), i32(N, T), z(N, T + 1)
    big = z(5000, 8)
    return {
        "sf_gdn_draft_step": lambda s: sf.sf_gdn_draft_step(q, q, v, g, g, cache, idx, pending=pend, stream=s),
        "sf_linattn_draft_step": lambda s: sf.sf_linattn_draft_step(q, q, v, dec, cache, idx, pending=pend[:2], stream=s),
        "sf_draft_verify": lambda s: sf.sf_draft_verify(probs, x, u, stream=s),
        "sf_state_fork": lambda s: sf.sf_state_fork(cache, idx, idx, stream=s),
        "sf_state_fork with a workspace": lambda s: sf.sf_state_fork(big, idx, idx, stream=s),
        "sf_state_compact": lambda s: sf.sf_state_compact([cache, cache.clone()], idx, stream=s),
        "sf_state_compact in place": lambda s: sf.sf_state_compact(cache, idx, out=idx, stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls(None)))
@pytest.mark.parametrize("given", [True, False])
def test_buffers_of_a_call_are_made_on_its_stream(monkeypatch, name, given):
    import chunked_linear_recurrence_gb300 as sf
    from chunked_linear_recurrence_gb300 import _decode, _linattn
    call = calls(sf)[name]
    current, made, done = [], [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def recorded(make):
        def f(*a, **kw):
            made.append(tuple(current))
            return make(*a, **kw)
        return f

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(_linattn, "_raw_stream", None)
    monkeypatch.setattr(_decode, "load", lambda: Lib(done))
    monkeypatch.setattr(_decode, "_workspace_bytes", lambda *a: 1024)
    for f in ("zeros", "empty", "empty_like"):
        monkeypatch.setattr(torch, f, recorded(getattr(torch, f)))
    stream = Stream() if given else None
    call(stream)
    assert done and made
    assert all(c == ((stream,) if given else ()) for c in made)
