"""Forks and compactions of middle-sized pools with a workspace and without one, on either side of the
sizes from which a plan has a launch of its own: the same slots and the same copies."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import decode as od
from test_gpu_state_pool import i32, mask, moved

pytestmark = pytest.mark.gpu


def without(caches, fn, *args):
    """The library's call without a workspace."""
    import chunked_linear_recurrence_gb300 as sf
    from chunked_linear_recurrence_gb300 import _decode
    pool, _ = _decode._state_pool(caches)
    stream = torch.cuda.current_stream().cuda_stream
    at = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    assert getattr(sf.load(), fn)(ctypes.byref(pool), *at, None, 0, stream) == 0


@pytest.mark.parametrize("slots,rows", [(512, 256), (4096, 256), (512, 257), (700, 90), (3000, 1000), (4096, 1024)])
@pytest.mark.parametrize("caches", [1, 3])
def test_both_forms_give_the_same(slots, rows, caches):
    import chunked_linear_recurrence_gb300 as sf
    r = np.random.RandomState(slots + rows)
    idx, parents = r.randint(-1, slots + 1, rows), r.randint(-1, rows + 1, rows)
    reserved = {int(s) for s in r.randint(1, slots, 9)}
    res = mask(slots, reserved)
    a = [torch.randn(slots, 4, 4 + i, device="cuda") for i in range(caches)]
    b = [t.clone() for t in a]
    new, copies = od.fork(idx, parents, slots, reserved)
    want = moved(a, copies)
    got = sf.sf_state_fork(a, i32(idx), i32(parents), reserved=res)
    out, at, par = torch.empty_like(got), i32(idx), i32(parents)
    without(b, "sf_state_fork", at, rows, par, rows, res, out)
    assert got.tolist() == new and out.tolist() == new
    assert all(map(torch.equal, a, want)) and all(map(torch.equal, b, want))
    new, moves = od.compact(idx, slots, reserved)
    want = moved(want, moves)
    got = sf.sf_state_compact(a, i32(idx), reserved=res)
    without(b, "sf_state_compact", at, rows, res, out)
    assert got.tolist() == new and out.tolist() == new
    assert all(map(torch.equal, a, want)) and all(map(torch.equal, b, want))
