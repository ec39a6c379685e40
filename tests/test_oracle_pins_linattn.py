"""Pins of the FP64 oracle of the decayed linear attention, the steps and the norm with
rotation: closed forms, identities and central differences (CPU only)."""
import numpy as np
import pytest

import oracle
from oracle import linattn as la


def _inputs(seed=0, B=2, T=9, H=2, HK=1, K=4, V=3):
    r = np.random.RandomState(seed)
    return dict(q=r.randn(B, T, HK, K), k=r.randn(B, T, HK, K), v=r.randn(B, T, H, V),
                decay=-np.abs(r.randn(H)), s0=r.randn(B, H, V, K), do=r.randn(B, T, H, V),
                df=r.randn(B, H, V, K))


def test_forward_is_the_decayed_sum():
    x = _inputs(1)
    out, fin = la.fwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], scale=0.7)
    B, T, H, V = x["v"].shape
    for b in range(B):
        for h in range(H):
            lam = np.exp(x["decay"][h])
            for i in range(T):
                w = lam ** np.arange(i, -1, -1)
                want = 0.7 * (np.einsum("j,ja,jv,a->v", w, x["k"][b, :i + 1, 0], x["v"][b, :i + 1, h],
                                        x["q"][b, i, 0]) + lam ** (i + 1) * x["s0"][b, h] @ x["q"][b, i, 0])
                np.testing.assert_allclose(out[b, i, h], want, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(fin[0, 0], np.exp(x["decay"][0]) ** T * x["s0"][0, 0] + sum(
        np.exp(x["decay"][0]) ** (T - 1 - t) * np.outer(x["v"][0, t, 0], x["k"][0, t, 0])
        for t in range(T)), rtol=1e-11)


def test_no_memory_and_plain_sums():
    x = _inputs(2)
    x["decay"] = np.array([-np.inf, 0.0])
    out, _ = la.fwd(x["q"], x["k"], x["v"], x["decay"], None, scale=1.0)
    qk = np.einsum("bta,bta->bt", x["q"][:, :, 0], x["k"][:, :, 0])
    np.testing.assert_allclose(out[:, :, 0], qk[..., None] * x["v"][:, :, 0], rtol=1e-12)
    p = np.tril(np.einsum("bia,bja->bij", x["q"][:, :, 0], x["k"][:, :, 0]))
    np.testing.assert_allclose(out[:, :, 1], p @ x["v"][:, :, 1], rtol=1e-10, atol=1e-12)


def test_split_equals_sequential_and_packed_equals_dense():
    x = _inputs(3)
    a, fa = la.fwd(x["q"][:, :4], x["k"][:, :4], x["v"][:, :4], x["decay"], x["s0"])
    b, fb = la.fwd(x["q"][:, 4:], x["k"][:, 4:], x["v"][:, 4:], x["decay"], fa)
    out, fin = la.fwd(x["q"], x["k"], x["v"], x["decay"], x["s0"])
    assert np.array_equal(np.concatenate([a, b], 1), out) and np.array_equal(fb, fin)
    flat = {n: x[n].reshape(1, 18, *x[n].shape[2:]) for n in ("q", "k", "v")}
    o, f = la.fwd(flat["q"], flat["k"], flat["v"], x["decay"], np.stack([x["s0"][0], x["s0"][0], x["s0"][1]]),
                  cu_seqlens=[0, 9, 9, 18])
    assert np.array_equal(o.reshape(out.shape), out)
    assert np.array_equal(f[[0, 2]], fin) and np.array_equal(f[1], x["s0"][0])


def test_gradients_are_central_differences():
    x = _inputs(4, T=5)
    g = la.bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])

    def loss(y):
        o, f = la.fwd(y["q"], y["k"], y["v"], y["decay"], y["s0"])
        return (o * x["do"]).sum() + (f * x["df"]).sum()

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "d_initial_state")):
        r = np.random.RandomState(5)
        for _ in range(6):
            u = r.randn(*x[name].shape)
            h = 1e-4
            d = (loss({**x, name: x[name] + h * u}) - loss({**x, name: x[name] - h * u})) / (2 * h)
            np.testing.assert_allclose((g[grad] * u).sum(), d, rtol=1e-8, atol=1e-8)


def test_steps_equal_one_token_of_the_rules():
    r = np.random.RandomState(6)
    N, H, HK, D = 3, 4, 2, 5
    q, k, v = r.randn(N, HK, D), r.randn(N, HK, D), r.randn(N, H, D)
    cache, idx, decay = r.randn(5, H, D, D), [2, -1, 4], -np.abs(r.randn(H))
    out, new = la.step(q, k, v, cache, idx, decay=decay)
    for n in (0, 2):
        o, f = la.fwd(q[n][None, None], k[n][None, None], v[n][None, None], decay, cache[idx[n]][None])
        np.testing.assert_allclose(out[n], o[0, 0], rtol=1e-12)
        np.testing.assert_allclose(new[idx[n]], f[0], rtol=1e-12)
    assert not out[1].any() and np.array_equal(new[[0, 1, 3]], cache[[0, 1, 3]])
    gate, beta = -np.abs(r.randn(N, H)), r.rand(N, H)
    out, new = la.step(q, k, v, cache, idx, gate=gate, beta=beta)
    for n in (0, 2):
        o, f = oracle.gdn_fwd(q[n][None, None], k[n][None, None], v[n][None, None], gate[n][None, None],
                              beta[n][None, None], cache[idx[n]][None])
        np.testing.assert_allclose(out[n], o[0, 0], rtol=1e-12)
        np.testing.assert_allclose(new[idx[n]], f[0], rtol=1e-12)


@pytest.mark.parametrize("norm,interleaved", [("rms", False), ("rms", True), ("l2", False)])
def test_norm_rope_keeps_lengths_and_its_gradient_is_differences(norm, interleaved):
    r = np.random.RandomState(7)
    rows, D, half = 6, 16, 6
    x, w, d = r.randn(rows, 2, D), r.rand(D) + 0.5, r.randn(rows, 2, D)
    a = r.rand(20, half) * 6
    cs = np.stack([np.cos(a), np.sin(a)], -1)
    pos, sec = r.randint(0, 20, (2, rows)), [2, 4]
    kw = dict(norm=norm, eps=1e-3, interleaved=interleaved)
    y = la.norm_rope(x, None, cs, pos, sec, **kw)
    plain = la.norm_rope(x, None, None, None, None, **kw)
    np.testing.assert_allclose((y ** 2).sum(-1), (plain ** 2).sum(-1), rtol=1e-12)
    # the angle between two rows' pairs depends on the difference of positions alone
    same = np.zeros((2, rows), int)
    np.testing.assert_allclose(la.norm_rope(x, w, np.stack([np.ones((1, half)), np.zeros((1, half))], -1),
                                            same, sec, **kw),
                               la.norm_rope(x, w, None, None, None, **kw), rtol=1e-12)
    dx, dw = la.norm_rope_bwd(x, w, cs, pos, sec, d, **kw)
    loss = lambda x, w: (la.norm_rope(x, w, cs, pos, sec, **kw) * d).sum()   # noqa: E731
    h = 1e-5
    for _ in range(4):
        u, uw = r.randn(*x.shape), r.randn(D)
        np.testing.assert_allclose((dx * u).sum(), (loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h), rtol=1e-6, atol=1e-7)
        np.testing.assert_allclose((dw * uw).sum(), (loss(x, w + h * uw) - loss(x, w - h * uw)) / (2 * h), rtol=1e-8)
