"""Calls with ``stream=`` that make their own workspaces and outputs, while the current stream has
work of its own queued: the results are those of a call on the current stream, and the buffers
belong to the stream that was given."""
import pytest
import torch

from test_gpu_linattn import inputs
from test_gpu_qk_norm_rope import make

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
WAIT = 20_000_000          # cycles, about 10 ms


def _calls():
    import chunked_linear_recurrence_gb300 as sf
    x = inputs(1, 2500, 4, 2, 128, BF16, seed=31)              # cut into segments, shared heads
    y = inputs(1, 700, 4, 2, 64, F32, seed=32, lengths=[400, 0, 300])
    n = make(2, 300, 4, 2, 128, BF16, 33, 128)
    g = torch.full((1, 2500, 4), -0.1, device="cuda")
    b = torch.full((1, 2500, 4), 0.5, device="cuda")
    tokens = lambda z: (z["q"], z["k"], z["v"])   # noqa: E731
    norm = (n["q"], n["k"], n["qw"], n["kw"], n["cs"], n["pos"])
    return [
        lambda **kw: sf.sf_linattn_chunk_fwd(*tokens(x), x["decay"], x["s0"], output_final_state=True, **kw),
        lambda **kw: sf.sf_linattn_chunk_bwd(*tokens(x), x["decay"], x["s0"], x["do"], x["df"], **kw),
        lambda **kw: sf.sf_linattn_chunk_bwd(*tokens(y), y["decay"], y["s0"], y["do"], y["df"],
                                             cu_seqlens=y["cu"], **kw),
        lambda **kw: sf.sf_qk_norm_rope_bwd(*norm, n["dq"], n["dk"], **kw),
        lambda **kw: sf.sf_gdn_chunk_fwd(*tokens(x), g, b, x["s0"], output_final_state=True, **kw),
        lambda **kw: sf.sf_gdn_chunk_bwd(*tokens(x), g, b, x["s0"], x["do"], x["df"], **kw),
    ]


def _tensors(r):
    return list(r.values()) if isinstance(r, dict) else list(r)


def _same(a, b, summed):
    """Equal; the delta rule's gate and beta gradients are FP32 sums in no fixed order."""
    return (a - b).norm() <= 1e-5 * b.norm() if summed else torch.equal(a, b)


def _stream_of(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("call", range(6))
def test_a_call_on_another_stream_without_a_workspace(call):
    run = _calls()[call]
    want = [t.clone() for t in _tensors(run())]
    summed = [call == 5 and i in (3, 4) for i in range(len(want))]      # dgate, dbeta
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(WAIT)                     # whatever the current stream is given now comes late
    got = _tensors(run(stream=side))
    assert all(_stream_of(t) == side.cuda_stream for t in got)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(map(_same, got, want, summed))
    with torch.cuda.stream(side):               # now the call comes late, and the current stream first
        torch.cuda._sleep(WAIT)
    got = _tensors(run(stream=side))
    held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (256, 1 << 20, 1 << 24, 1 << 26)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(h.min() == 255 for h in held)
    assert all(map(_same, got, want, summed))
