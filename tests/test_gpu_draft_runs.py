"""Drafted tokens and commits of many sequences: a warp takes several strips of states one after the
other, alone, in runs of two and of four, with the tokens of a run kept, the next strip's state and
values copied ahead and runs that change to other sequences, to padding and to ones without tokens.

A strip's arithmetic knows nothing of the others, so every sequence has to give, to the bit, what it
gives in a call of a few sequences, where no warp has a second strip; some are held against the oracle
too.  The whole pool is compared: what no sequence advances stays as it was."""
import math

import pytest
import torch

from test_gpu_draft_step import BF16, F32, TOL, call, case, commit, err, want

pytestmark = pytest.mark.gpu
NAN = float("nan")


def warps(T, P, dtype, D):
    """What the machine holds of a call's kernel, each with a strip of 16 rows."""
    many = max(T, P) > 8
    return 152 * {(BF16, 128): 8, (BF16, 64): 13 if many else 14, (F32, 128): 4 if many else 7,
                  (F32, 64): 7 if many else 12}[dtype, D]


def strips_in_a_row(turns):
    """The library's choice where a warp has this many strips."""
    return min((1, 2, 4), key=lambda r: math.ceil(turns / r) * r * {1: 1.18, 2: 1.06, 4: 1.0}[r])


def at(x, rows):
    """A call's sequences `rows` alone, on the same pool."""
    cut = lambda t: None if t is None else {m: v[rows].contiguous() for m, v in t.items()}   # noqa: E731
    return dict(x, new=cut(x["new"]), pend=cut(x["pend"]), idx=x["idx"][rows],
                num=x["num"][rows], num_pend=None if x["num_pend"] is None else x["num_pend"][rows])


def write(x):
    """What a call writes: outputs (None for commits); the pool is advanced in place."""
    if x["new"]["v"].shape[1]:
        return call(x, out=torch.full_like(x["new"]["v"], NAN))
    return commit(x, x["pend"], x["num_pend"])


def compare(N, T, P, H, HK, D, dtype, delta, seed):
    x = case(N, T, P, H, HK, D, dtype, delta, seed, slots=N + 2)
    g = torch.Generator().manual_seed(seed)
    most = lambda n: torch.where(torch.rand(N, generator=g) < 0.3, torch.where(torch.rand(N, generator=g) < 0.5, 0, n),   # noqa: E731
                                 torch.randint(0, n + 1, (N,), generator=g)).to(torch.int32).cuda()
    x["num"] = most(T)
    if P:
        x["num_pend"] = most(P)
    for n in torch.randint(0, N, (N // 8 + 1,), generator=g).tolist():       # padding in the midst of others
        x["idx"][n] = [-1, 0, N + 2][n % 3]
    before = x["cache"].clone()
    out = write(x)
    y = dict(x, cache=before.clone())
    step = 152 * 4 * 16 // (D * H)            # (the fewest warps of any kernel)
    for n in range(0, N, step):
        o = write(at(y, slice(n, n + step)))
        if o is not None:
            assert torch.equal(out[n:n + step], o)
    assert torch.equal(x["cache"], y["cache"])
    for n in (0, N // 2, N - 1):
        one = at(dict(x, cache=before), slice(n, n + 1))
        slot = int(one["idx"])
        if not 0 < slot < N + 2:
            slot = 1
        small = dict(one, cache=before[[0, slot]], idx=torch.where(one["idx"] == slot, 1, -1).to(torch.int32))
        if T:
            ro, rc = want(small)
            assert err(out[n:n + 1], ro) <= TOL[dtype]
        else:
            _, rc = want(dict(small, new=small["pend"] | {"q": small["pend"]["k"]}, num=small["num_pend"] * 0))
        if int(one["idx"]) == slot:
            assert err(x["cache"][slot], rc[1]) <= TOL[F32]


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("T,P", [(4, 3), (16, 12), (32, 20), (7, 0), (12, 0), (0, 5), (0, 12), (0, 32)])
@pytest.mark.parametrize("turns,run", [(4.5, 1), (5.5, 2), (7.8, 4)])
def test_several_strips_to_a_warp(turns, run, T, P, dtype, D, delta):
    H, HK = 4, 2
    N = math.ceil(warps(T, P, dtype, D) * turns * 16 / (D * H))
    assert strips_in_a_row(N * H * D / 16 / warps(T, P, dtype, D)) == run
    compare(N, T, P, H, HK, D, dtype, delta, T + P)
