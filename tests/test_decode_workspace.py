"""Which forks and compactions make a workspace for themselves: those that the library would use one
for, with a recording library in place of the real one."""
import pytest
import torch

from test_stream_argument import Lib, Stream


@pytest.fixture
def made(monkeypatch):
    from chunked_linear_recurrence_gb300 import _decode, _linattn
    got = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: got.append(kw["dtype"]) or empty(*a, **kw))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(_linattn, "_raw_stream", None)
    monkeypatch.setattr(_decode, "load", lambda: Lib([]))
    monkeypatch.setattr(_decode, "_workspace_bytes", lambda *a: 1024)
    return got


@pytest.mark.parametrize("rows,used", [(256, False), (257, True)])
def test_many_rows_have_a_workspace(made, rows, used):
    import chunked_linear_recurrence_gb300 as sf
    cache, idx = torch.zeros(4096, 8), torch.zeros(rows, dtype=torch.int32)
    for call in (lambda: sf.sf_state_fork(cache, idx[:3], idx), lambda: sf.sf_state_compact(cache, idx)):
        made.clear()
        call()
        assert (torch.uint8 in made) == used


@pytest.mark.parametrize("out", ["none", "apart", "beside", "indices", "parents", "overlapping"])
@pytest.mark.parametrize("slots", [40, 5000])
def test_a_workspace_is_made_where_one_is_used(made, out, slots):
    import chunked_linear_recurrence_gb300 as sf
    cache, buf = torch.zeros(slots, 8), torch.zeros(64, dtype=torch.int32)
    idx, par, reserved = buf[:12], buf[12:20], torch.zeros(slots, dtype=torch.bool)
    own = torch.zeros(8, dtype=torch.int32)
    to = {"none": None, "apart": own, "beside": buf[20:28], "indices": idx[:8], "parents": par,
          "overlapping": buf[8:16]}[out]
    used = slots > 4096 or out in ("indices", "parents", "overlapping")
    sf.sf_state_fork(cache, idx, par, reserved=reserved, out=to)
    assert (torch.uint8 in made) == used
    if out in ("none", "apart", "beside", "indices"):
        made.clear()
        sf.sf_state_compact(cache, idx[:8], reserved=reserved, out=to)
        assert (torch.uint8 in made) == (slots > 4096 or out == "indices")
