"""How far a NaN or an infinity inside a sequence reaches: that head's results from the start of its
block of 64 tokens on (blocks counted from the sequence's start; what the backward walks from the
end, dk, dv and d_initial_state, from the end of its block counted from the sequence's end), and
nothing else -- not the rows before, not another sequence, not another head.  Also a captured
backward."""
import numpy as np
import pytest
import torch

from test_gpu_linattn import BF16, F32, inputs, run_fwd

pytestmark = pytest.mark.gpu
LENGTHS, AT = [150, 1700, 70], 700          # the token of the second sequence that is hit


def grads(x):
    import chunked_linear_recurrence_gb300 as sf
    return sf.sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"],
                                   cu_seqlens=x["cu"])


def same(a, b, rows):
    return torch.equal(a[:, rows], b[:, rows])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_reach_of_a_value_that_is_not_finite(dtype, D, name, value):
    H = 2
    x = inputs(1, sum(LENGTHS), H, H, D, dtype, seed=17 + D, lengths=LENGTHS, decay=[-0.01, -0.3])
    clean, clean_g = run_fwd(x), grads(x)
    bad = x[name].clone()
    bad[0, LENGTHS[0] + AT, 1, 3] = value
    y = dict(x, **{name: bad})
    (out, fin), g = run_fwd(y), grads(y)
    lo, hi = LENGTHS[0], LENGTHS[0] + LENGTHS[1]
    first = lo + AT // 64 * 64
    last = hi - (LENGTHS[1] - 1 - AT) // 64 * 64            # one past the block counted from the end
    rows = np.arange(sum(LENGTHS))
    before, after = rows[(rows < first) | (rows >= hi)], rows[(rows < lo) | (rows >= last)]
    # the other head and the other sequences
    for a, b in ((out, clean[0]), (g["dq"], clean_g["dq"]), (g["dk"], clean_g["dk"]), (g["dv"], clean_g["dv"])):
        assert torch.equal(a[:, :, 0], b[:, :, 0])
    for a, b in ((fin, clean[1]), (g["d_initial_state"], clean_g["d_initial_state"])):
        assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(a[[0, 2]], b[[0, 2]])
    for a, b, keep in ((out, clean[0], before), (g["dq"], clean_g["dq"], before),
                       (g["dk"], clean_g["dk"], after), (g["dv"], clean_g["dv"], after)):
        assert same(a[:, :, 1:], b[:, :, 1:], keep)
    # and it does reach the token's own results and what follows from them
    at = LENGTHS[0] + AT
    hit = dict(q=(out, g["dk"]), k=(out, g["dq"]), v=(out, g["dq"]), do=(g["dq"], g["dv"]))[name]
    assert all(not torch.isfinite(t[0, at, 1].float()).all() for t in hit[:1])
    if name in ("k", "v"):
        assert not torch.isfinite(fin[1, 1]).all() and not torch.isfinite(out[0, hi - 1, 1].float()).all()
    else:
        assert torch.isfinite(fin).all()
    if name in ("q", "do"):
        assert not torch.isfinite(g["d_initial_state"][1, 1]).all()
    else:
        assert torch.isfinite(g["d_initial_state"]).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_backward_replayed_in_a_graph(dtype, D):
    """Up to four launches that start while the ones before them end; walks that are cut, shared
    heads; replayed on other tokens and other offsets in the same buffers."""
    import chunked_linear_recurrence_gb300 as sf
    T = 1600
    x = inputs(1, T, 4, 2, D, dtype, seed=5, lengths=[1300, 0, 300])
    y = inputs(1, T, 4, 2, D, dtype, seed=6, lengths=[100, 1050, 450])
    want = grads(y)
    ws = sf.sf_linattn_bwd_workspace(x["q"], x["v"], x["cu"])
    got = {n: torch.zeros_like(t) for n, t in want.items()}

    def call():
        sf.sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"], cu_seqlens=x["cu"],
                                grads=got, ws=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n, t in x.items():
        t.copy_(y[n])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    sf.sf_workspace_status(ws)
