"""Bounds on the error of drafted tokens and commits (test_gpu_draft_precision), and that a lost part
of a number breaks them: the rule in FP64 with the state that is read, or the rows' weights, cut to two
BF16 summands (16 bits)."""
import numpy as np
import pytest
import torch

# States and FP32 outputs.  Behind up to eight tokens a value has come through some 24 roundings (the
# exponential and up to eight products of decays, sums of eight partial products, up to eight
# multiply-adds of the solve, the update), independent and of 2^-24 at the most, of the 2-norm:
TOL = 24 ** 0.5 * 2.0 ** -24
# What is read from paired() by vectors of equal numbers, 1/8 each: the d, whose sums are about 1.  The
# tensor core cuts each of 24 sums at 2^-23 of their largest product, 2^12; the rounding of an advanced
# state, 2^13 2^-24 of an element, adds (128 / 3)^0.5 / 8 of itself.
PAIRED = 24 ** 0.5 * 2.0 ** -11 + (128 / 3) ** 0.5 / 8 * 2.0 ** -11


def paired(g, *shape):
    """States whose columns come in pairs of a + d and -a, a about 2^13 and d about 1."""
    S = torch.zeros(shape)
    a = torch.randn(*shape[:-1], shape[-1] // 2, generator=g) * 2.0 ** 13
    S[..., 0::2] = a + torch.randn(a.shape, generator=g)
    S[..., 1::2] = -a
    return S


def bits16(x):
    t = torch.from_numpy(np.ascontiguousarray(x)).float()
    a = t.bfloat16().float()
    return (a.double() + (t - a).bfloat16().double()).numpy()


def err(x, ref):
    return np.linalg.norm(x - ref) / np.linalg.norm(ref)


def advance(S, k, v, gate, beta, read=lambda x: x, weight=lambda x: x):
    for t in range(k.shape[1]):
        S = np.exp(gate[:, t])[:, None, None] * S
        r = beta[:, t][:, None] * (v[:, t] - np.einsum("nvk,nk->nv", read(S), k[:, t]))
        S = S + weight(r)[:, :, None] * k[:, t][:, None]
    return S


@pytest.mark.parametrize("T", [1, 4, 8])
def test_weights_of_two_summands_break_the_bound(T):
    """From a state of zeros, which is the tokens' alone."""
    r = np.random.RandomState(T)
    k = r.randn(24, T, 128)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    args = (np.zeros((24, 128, 128)), k, r.randn(24, T, 128), -r.rand(24, T), r.rand(24, T))
    assert err(advance(*args, weight=bits16), advance(*args)) > 4 * TOL


@pytest.mark.parametrize("D", [64, 128])
def test_states_of_two_summands_break_the_bound(D):
    g = torch.Generator().manual_seed(D)
    S = paired(g, 24, D, D).double().numpy()
    q = np.full(D, 0.125)
    assert err(bits16(S) @ q, S @ q) > 3 * (PAIRED + 2.0 ** -8)
    k = np.broadcast_to(q, (24, 1, D))
    args = (S, k, torch.randn(24, 1, D, generator=g).double().numpy(), np.zeros((24, 1)), np.full((24, 1), 64 / D))
    assert err(advance(*args, read=bits16) @ q, advance(*args) @ q) > 3 * PAIRED
