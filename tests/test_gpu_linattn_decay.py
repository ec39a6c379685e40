"""The carried factor lam^64 is a float that lacks up to 2^-25 / lam^64 of itself.  A state of any
memory must show nothing of it: neither the drift of thousands of chunks that lack it nor a
correction of rows that were never multiplied with it.

Two heads of the same tokens whose decays are next to one another, one factor rounded up and one
down as far as it goes: what the errors of their final states have in common (the same sums in
the same order) goes, and what the lack makes of it stays.  The error is taken along the state,
<S - R, R> / <R, R>, where the roundings of 16384 elements (1e-7 each) average to 1e-9; the
64 rows' weights are off by at most 2^-23 each, independently: 1.2e-7 / 64^0.5 = 1.5e-8 a head.  Limit:
1e-7.  (16 chunks' lacks at lam^64 = 0.51 are 9e-7 a head.)"""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import linattn as la
from test_gpu_linattn import BF16, inputs

pytestmark = pytest.mark.gpu


def decays(f):
    """Two float decays whose 64th powers are near f, one rounded down and one up the most."""
    d = (np.float32(np.log(f) / 64) + np.arange(4000, dtype=np.float32) * np.float32(2.0 ** -31)).astype(np.float32)
    p = np.exp(64 * d.astype(np.float64))
    lack = p / p.astype(np.float32).astype(np.float64) - 1
    return [float(d[lack.argmax()]), float(d[lack.argmin()])], lack.max() - lack.min()


@pytest.mark.parametrize("f", [0.51, 0.6, 0.83, 0.97])
@pytest.mark.parametrize("chunks,walks", [(17, 160), (40, 160), (33, 2)])
@pytest.mark.parametrize("D", [128, 64])
def test_no_bias_of_the_carried_factor(f, chunks, walks, D):
    """160 walks are not cut, 2 are."""
    import chunked_linear_recurrence_gb300 as sf
    pair, gap = decays(f)
    assert gap >= 1.5 * 2 ** -25 / f
    B, T = walks // 2, 64 * chunks + 1
    x = inputs(1, T, 2, 1, D, BF16, seed=chunks, decay=pair, s0=False)
    x["v"][:, :, 1] = x["v"][:, :, 0]
    wide = [x[n].expand(B, -1, -1, -1).contiguous() for n in ("q", "k", "v")]
    fin = f64(sf.sf_linattn_chunk_fwd(*wide, x["decay"], output_final_state=True)[1][0])
    ref = la.fwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["decay"]))[1][0]
    along = [((fin[h] - ref[h]) * ref[h]).sum() / (ref[h] ** 2).sum() for h in range(2)]
    assert abs(along[0] - along[1]) <= 1e-7, along
    assert all(np.linalg.norm(fin[h] - ref[h]) <= 1e-6 * np.linalg.norm(ref[h]) for h in range(2))
