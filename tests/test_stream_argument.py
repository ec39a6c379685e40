"""A call with ``stream=`` makes its own buffers on that stream: nothing of another stream's order
clears them under the kernels or hands them to other work.  Here with a recording library in
place of the real one; test_gpu_stream_argument runs the kernels."""
import contextlib

import pytest
import torch


class Lib:
    """Answers 0 (and 1024 to the sizes of workspaces) to every entry point."""

    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return 1024 if name.endswith("_workspace") else 0
        return entry


class Stream:
    cuda_stream = 77


B, T, H, HK, D = 1, 70, 4, 2, 64


def calls(sf):
    z = torch.zeros
    q, v, g = z(B, T, HK, D), z(B, T, H, D), z(B, T, H)
    dec, cache, idx = z(H), z(3, H, D, D), z(B, dtype=torch.int32)
    step = (z(2, HK, D), z(2, HK, D), z(2, H, D))
    P, S = z(2, H, D, D), z(2, H, D, D)
    offs, bounds, gb = torch.tensor([0, T], dtype=torch.int32), z(2, 2, dtype=torch.int32), z(2, H)
    n = sf._native
    return {
        "sf_linattn_chunk_fwd": lambda s: sf.sf_linattn_chunk_fwd(q, q, v, dec, output_final_state=True, stream=s),
        "sf_linattn_paged_chunk_fwd": lambda s: sf.sf_linattn_paged_chunk_fwd(q, q, v, dec, cache, idx, stream=s),
        "sf_linattn_chunk_bwd": lambda s: sf.sf_linattn_chunk_bwd(q, q, v, dec, None, v, stream=s),
        "sf_linattn_step": lambda s: sf.sf_linattn_step(*step, dec, cache, stream=s),
        "sf_gdn_step": lambda s: sf.sf_gdn_step(*step, gb, gb, cache, stream=s),
        "sf_qk_norm_rope_fwd": lambda s: sf.sf_qk_norm_rope_fwd(v, q, stream=s),
        "sf_qk_norm_rope_bwd": lambda s: sf.sf_qk_norm_rope_bwd(v, q, None, None, None, None, v, q, stream=s),
        "sf_gdn_chunk_fwd": lambda s: sf.sf_gdn_chunk_fwd(q, q, v, g, g, output_final_state=True, stream=s),
        "sf_gdn_paged_chunk_fwd": lambda s: sf.sf_gdn_paged_chunk_fwd(q, q, v, g, g, cache, idx, stream=s),
        "sf_gdn_segment_summary": lambda s: sf.sf_gdn_segment_summary(q, v, g, g, bounds, stream=s),
        "sf_state_scan": lambda s: sf.sf_state_scan(P, S, stream=s),
        "sf_gdn_segment_reverse_summary":
            lambda s: sf.sf_gdn_segment_reverse_summary(q, q, g, g, v, offs, stream=s),
        "sf_state_scan_reverse": lambda s: sf.sf_state_scan_reverse(P, S, stream=s),
        "sf_gdn_chunk_bwd": lambda s: sf.sf_gdn_chunk_bwd(q, q, v, g, g, None, v, stream=s),
        "sf_gdn_chunk_bwd_noalloc": lambda s: n.sf_gdn_chunk_bwd_noalloc(q, q, v, g, g, None, v, stream=s),
        # the stream as the last of the positional arguments
        "sf_gdn_step ": lambda s: sf.sf_gdn_step(*step, gb, gb, cache, None, None, None, s),
    }


NAMES = sorted(calls(__import__("chunked_linear_recurrence_gb300")))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", [True, False])
def test_buffers_of_a_call_are_made_on_its_stream(monkeypatch, name, given):
    import chunked_linear_recurrence_gb300 as sf
    from chunked_linear_recurrence_gb300 import _linattn, _native
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
    for m in (_linattn, _native):
        monkeypatch.setattr(m, "load", lambda: Lib(done))
    for f in ("zeros", "empty", "empty_like"):
        monkeypatch.setattr(torch, f, recorded(getattr(torch, f)))
    stream = Stream() if given else None
    call(stream)
    assert done and made
    assert all(c == ((stream,) if given else ()) for c in made)
