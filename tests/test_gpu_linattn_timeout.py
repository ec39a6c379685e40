"""Failure detection of the tensor-core linear attention on the device without a fault: a bounded
wait that runs out.  One warp never announces a table, the warps that need it give up after a few
milliseconds, the others see the abort flag, copies and products in flight land, every CTA leaves,
and the status word reads SF_ERR_TIMEOUT.  The next call, in the same workspace, is right."""
import pytest
import torch

from test_gpu_linattn import BF16, STATE, TOL, err, inputs, ref_fwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("T,lengths", [(40, None), (130, None), (700, None), (2500, None), (2500, [1300, 0, 1200])])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(D, T, lengths):
    """One chunk, a few, more than there are stages; cut into segments, where the pieces' launch
    gives up as well; the backward's three walks."""
    import chunked_linear_recurrence_gb300 as sf
    from chunked_linear_recurrence_gb300 import _native
    lib = sf.load()
    x = inputs(1, T, 2, 1, D, BF16, seed=T + D, lengths=lengths)
    args = (x["q"], x["k"], x["v"], x["decay"], x["s0"])
    bwd = lambda **kw: sf.sf_linattn_chunk_bwd(*args, x["do"], x["df"], cu_seqlens=x["cu"], **kw)   # noqa: E731
    good = bwd()
    for call, need in ((lambda ws: run_fwd(x, ws=ws), sf.sf_linattn_fwd_workspace),
                       (lambda ws: bwd(ws=ws), sf.sf_linattn_bwd_workspace)):
        ws = need(x["q"], x["v"], x["cu"])
        assert lib.sf_testing_inject_linattn_timeout(100) == 0
        call(ws)
        with pytest.raises(_native.SfError) as e:
            sf.sf_workspace_status(ws)
        assert e.value.status == _native.SF_ERR_TIMEOUT
        sf.sf_workspace_status(ws)                        # read once, then cleared
        result = call(ws)
        sf.sf_workspace_status(ws)
        if isinstance(result, dict):
            assert all(torch.equal(result[n], good[n]) for n in good)
        else:
            ro, rf = ref_fwd(x)
            assert err(result[0], ro) <= TOL[BF16] and err(result[1], rf) <= STATE


def test_injection_rejects_bad_arguments():
    import chunked_linear_recurrence_gb300 as sf
    lib = sf.load()
    assert lib.sf_testing_inject_linattn_timeout(0) == 1
    assert lib.sf_testing_inject_linattn_timeout(10001) == 1
