"""Failure detection of the verification on the device without a fault: a bounded wait that runs
out.  The first CTA of every sequence gives up at once, while the others still sum their slices,
outlives them and what they send to it, and says so.  The next call is right."""
import pytest
import torch

from test_gpu_draft_verify import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V", [(1, 32000), (5, 70001), (40, 513), (600, 300)])
@pytest.mark.parametrize("nothing_left", [False, True])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(N, V, nothing_left):
    """One CTA a sequence, eight, short and long rows; where nothing is left to draw from behind a
    rejected draft the other CTAs go on to a second pass, and give up in it after two seconds."""
    import chunked_linear_recurrence_gb300 as sf
    d = make(N, 2, V, torch.float32, True, N + V)
    d["num"] = torch.full((N,), 2, dtype=torch.int32, device="cuda")
    if nothing_left:
        d["draft"] = d["target"][:, :2] * 1.5
        d["u"][:, :2] = 0.9
    if N > 1:
        d["num"][1] = -1
    check(d, call(d))
    assert sf.load().sf_testing_inject_verify_timeout() == 0
    want = [-1] * N
    if N > 1:
        want[1] = 0
    assert call(d)[1].tolist() == want
    check(d, call(d))
