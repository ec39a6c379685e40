"""Draws from rows of many millions of tokens: sums of that many weights keep 38 bits.

The weights are whole numbers times one factor, so that sums and borders are exact here.  A draw is
the first token whose running sum passes u times the sum; the kernel's sums are off by at most 2^-38
of the whole, so a uniform whose aim lies further than that from the borders of its token has to draw
that token.  (The seeds leave no more than a few uniforms out.)  One row is read by 160 sequences,
which is as many as take one CTA each, with the longest sums."""
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu
N = 160


def draws(weights, u):
    import chunked_linear_recurrence_gb300 as sf
    rows = weights[None, None].expand(N, 1, -1)
    return sf.sf_draft_verify(rows, torch.zeros(N, 0, dtype=torch.int32, device="cuda"), u[:, None].cuda())[0][:, 0].tolist()


def check(got, u, run, total):
    """run(y): the exact sum of the first y + 1 weights."""
    near, seen = Fraction(total, 1 << 38), 0
    for y, x in zip(got, u.tolist()):
        aim = Fraction(x) * total
        low, high = run(y - 1) if y else 0, run(y)
        assert low - near <= aim < high + near
        seen += low + near <= aim < high - near
    assert seen >= N // 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [33554467, 100000007])
def test_equal_weights(V, dtype):
    u = torch.rand(N, generator=torch.Generator().manual_seed(V))
    got = draws(torch.full((V,), 0.7, dtype=dtype, device="cuda"), u)
    check(got, u, lambda y: y + 1, V)


@pytest.mark.parametrize("V", [1000003, 40000003])
def test_weights_of_all_sizes(V):
    """24 random bits each, a few of them 2^24 times the others."""
    g = torch.Generator("cuda").manual_seed(V)
    w = torch.randint(1, 1 << 24, (V,), generator=g, device="cuda")
    w[torch.randint(0, V, (9,), generator=g, device="cuda")] <<= 24
    run = w.cumsum(0)
    u = torch.rand(N, generator=torch.Generator().manual_seed(V))
    got = draws(w.float(), u)
    check(got, u, lambda y: int(run[y]), int(run[-1]))


@pytest.mark.parametrize("V", [3000, 70001])
def test_uniforms_far_outside_their_range(V):
    """Whatever lies below 0 draws the first token with weight, from 1 on the last one."""
    import chunked_linear_recurrence_gb300 as sf
    u = [-float("inf"), -3e38, -1e30, -1e-45, 1.0, 3e38, float("inf")]
    target = torch.zeros(len(u), 1, V, device="cuda")
    target[:, :, 1234:1300] = 1.0
    tokens, num = sf.sf_draft_verify(target, torch.zeros(len(u), 0, dtype=torch.int32, device="cuda"),
                                     torch.tensor(u, device="cuda")[:, None])
    assert tokens[:, 0].tolist() == [1234] * 4 + [1299] * 3 and num.tolist() == [1] * len(u)
