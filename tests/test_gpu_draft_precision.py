"""Drafted tokens and commits: how exact they are, with bounds that a lost summand would break
(test_draft_precision_bounds derives them and plants such losses).  BF16 outputs are rounded, by 2^-8 at
the most, and hide what lies below unless they cancel."""
import numpy as np
import pytest
import torch

import test_draft_precision_bounds as bounds
from helpers import f64
from test_draft_precision_bounds import PAIRED, TOL, paired
from test_gpu_draft_step import BF16, F32, call, case, commit, err, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("start", [0.0, 1.0])
@pytest.mark.parametrize("T,P", [(1, 1), (5, 4), (8, 8), (8, 0)])
def test_states_and_fp32_outputs_are_fp32(T, P, start, D, dtype, delta):
    """From states of zeros, which are the tokens' alone then, and others."""
    x = case(6, T, P, 4, 2, D, dtype, delta, 200 + T + P + D)
    x["cache"] *= start
    y = dict(x, cache=x["cache"].clone())
    ro, rc = want(x)
    out = call(x)
    assert err(x["cache"], rc) <= TOL
    if dtype == F32:
        assert err(out, ro) <= TOL
    if P:
        commit(y, y["pend"], y["num_pend"])
        assert err(y["cache"], rc) <= TOL


def still(x, key):
    """Nothing decays, and every key is `key`."""
    for t in (x["new"], x["pend"]):
        if t is not None:
            t["k"][:] = key
            if x["delta"]:
                t["gate"].zero_()
    if not x["delta"]:
        x["decay"].zero_()


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,P", [(1, 0), (5, 4), (8, 0), (12, 0), (12, 9), (20, 3)])
def test_outputs_that_cancel_keep_the_states_bits(T, P, D, delta):
    """Keys of zeros: every draft reads the state as it is."""
    H, N = 4, 3
    x = case(N, T, P, H, 2, D, BF16, delta, 300 + T + P)
    g = torch.Generator().manual_seed(T)
    S = paired(g, *x["cache"].shape)
    x["cache"] = S.cuda()
    sign = torch.randint(0, 2, (N, T, 2, 1), generator=g) * 2.0 - 1.0
    x["new"]["q"] = (sign * 0.125).expand(N, T, 2, D).contiguous().to(BF16).cuda()
    still(x, 0.0)
    ro, _ = want(x, num=None, num_pend=None, scale=1.0)
    out = call(x, num_tokens=None, num_pending=None, scale=1.0)
    assert torch.equal(x["cache"], S.cuda())
    assert err(out, ro) <= PAIRED + 2.0 ** -8


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [0, 3, 12])
def test_keys_that_cancel_keep_the_states_bits(T, D, dtype):
    """A token's key reads what is left of the pairs; what the state then holds for it is as exact.
    Committed, and pending in front of drafts."""
    x = case(4, T, 1, 4, 2, D, dtype, True, 350 + D)
    g = torch.Generator().manual_seed(D + 1)
    x["cache"] = paired(g, *x["cache"].shape).cuda()
    still(x, 0.125)
    x["pend"]["beta"].fill_(64 / D)
    _, rc = want(x, num=None, num_pend=None)
    if T:
        call(x, num_tokens=None, num_pending=None)
    else:
        commit(x, x["pend"], None)
    rows = x["idx"].tolist()
    q = np.full(D, 0.125)
    assert bounds.err(f64(x["cache"])[rows] @ q, rc[rows] @ q) <= PAIRED


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("how", ["one call", "commit", "drafts"])
def test_a_token_that_takes_the_place_of_a_larger_one(how, dtype, D):
    """The delta rule's purpose: what the state held for a key, 2^13 times the values, is replaced by
    a token with that key, as a pending token, committed, or as a draft; then the key is asked
    for.  The key's length is exactly 1 and beta is 1, so the value is left.  Sums of 16 parts cut at
    2^-23 of 2^13: 16^0.5 2^-10 = 3.9e-3, which is all that FP32 arithmetic gives here; BF16
    outputs are rounded beside it."""
    N, H = 5, 4
    x = case(N, 2, 2, H, H, D, dtype, True, 400 + D)
    g = torch.Generator().manual_seed(D)
    key = torch.zeros(N, H, D)
    key[..., :64] = (torch.randint(0, 2, (N, H, 64), generator=g) * 2.0 - 1.0) / 8
    key = key.to(dtype).cuda()
    x["cache"] = (torch.randn(x["cache"].shape, generator=g) * 2.0 ** 13).cuda()
    x["num"] = x["num_pend"] = None
    for t in (x["new"], x["pend"]):
        t["k"][:] = key[:, None]
        t["gate"].zero_()
        t["beta"][:] = torch.tensor([1.0, 0.0], device="cuda")[:, None]
    x["new"]["q"][:] = key[:, None]
    if how != "drafts":
        x["new"]["beta"].zero_()
    else:
        x["pend"] = None
    ro, rc = want(x, scale=1.0)
    value = f64(x["new"]["v"] if how == "drafts" else x["pend"]["v"])[:, :1]
    assert np.allclose(ro, np.broadcast_to(value, ro.shape), rtol=0, atol=1e-9)
    if how == "commit":
        commit(x, x["pend"], None)
        x["pend"] = None
    out = call(x, scale=1.0)
    assert err(out, ro) <= 3.9e-3 + (2.0 ** -8 if dtype == BF16 else 0.0)
    assert err(x["cache"], rc) <= TOL


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("T,P", [(1, 1), (5, 4), (8, 8)])
def test_one_call_and_commit_then_draft_differ_in_few_roundings(T, P, delta):
    """Both ways are FP32 before the outputs' rounding to BF16, 2 x 2.9e-7 of the 2-norm apart: where
    no border of BF16, 2^-8 of a value apart, lies between them they are equal.  2^8 x 5.8e-7 of the
    values is 1.5e-4, ten times that with the small ones' closer borders; and they differ by
    one step then, 2^-7."""
    x = case(40, T, P, 4, 2, 128, BF16, delta, 500 + T)
    y = dict(x, cache=x["cache"].clone())
    out = call(x)
    commit(y, y["pend"], y["num_pend"])
    assert torch.equal(x["cache"], y["cache"])
    a, b = f64(out), f64(call(y, pending=None, num_pending=None))
    assert (a != b).mean() <= 1.5e-3
    assert (np.abs(a - b) <= 2.0 ** -7 * np.maximum(np.abs(a), np.abs(b)) + 5.8e-7 * np.abs(a).max()).all()
