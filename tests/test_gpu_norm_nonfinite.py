"""NaN and infinities in the norm of query and key heads: a head that holds one gives what the
formula gives for it (NaN in every element for a NaN, through the norm), other heads are not touched.

Where the FP64 oracle is finite the limits are those of test_gpu_qk_norm_rope."""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import linattn as la
from test_gpu_qk_norm_rope import close, make, rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BAD = ((3, 1, 5, float("nan")), (7, 0, 2, float("inf")), (8, 2, 60, -float("inf")))   # token, head, element


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("norm,eps", [("rms", 1e-6), ("l2", 1e-6), ("l2", 1e3)])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (0, False)])
def test_a_head_with_a_nan_or_an_infinity(dtype, norm, eps, rot, interleaved):
    """eps = 1e3 is above the norm of every finite head."""
    import chunked_linear_recurrence_gb300 as sf
    x = make(1, 12, 3, 3, 64, dtype, 11, rot, fused=False)
    for t, h, e, value in BAD:
        x["q"][0, t, h, e] = value
    opt = dict(norm=norm, eps=eps, interleaved=interleaved)
    args = (x["q"], x["k"], x["qw"], x["kw"], x["cs"], x["pos"])
    q, _ = sf.sf_qk_norm_rope_fwd(*args, sections=x["sections"], **opt)
    g = sf.sf_qk_norm_rope_bwd(*args, x["dq"], x["dk"], sections=x["sections"], **opt)
    cs = None if x["cs"] is None else f64(x["cs"])
    pos = None if x["pos"] is None else x["pos"].cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref = la.norm_rope(rows(x["q"]), f64(x["qw"]), cs, pos, x["sections"], **opt)
        rdx, rdw = la.norm_rope_bwd(rows(x["q"]), f64(x["qw"]), cs, pos, x["sections"], rows(x["dq"]), **opt)
    assert np.isnan(ref[3, 1]).all() and np.isnan(rdx[3, 1]).all()
    finite = np.isfinite(ref).all(-1)
    assert finite.sum() == ref.shape[0] * ref.shape[1] - len(BAD)
    for got, want in ((f64(q).reshape(ref.shape), ref), (f64(g["dq"]).reshape(rdx.shape), rdx),
                      (f64(g["dq_weight"]), rdw)):
        assert (np.isnan(got) == np.isnan(want)).all()
        assert (np.isinf(got) == np.isinf(want)).all()
    assert close(torch.from_numpy(f64(q).reshape(ref.shape)[finite]), ref[finite], dtype)
    # heads of finite numbers: as if the others were not there
    y = {n: t.clone() for n, t in x.items() if n in ("q", "dq")}
    for t, h, _, _ in BAD:
        y["q"][0, t, h] = 1
    clean = sf.sf_qk_norm_rope_bwd(y["q"], *args[1:], x["dq"], x["dk"], sections=x["sections"], **opt)["dq"]
    keep = torch.from_numpy(finite).cuda()
    assert torch.equal(g["dq"][0][keep], clean[0][keep])
    assert torch.isfinite(g["dk"].float()).all() and torch.isfinite(g["dk_weight"]).all()
