"""The norm of query and key heads with the position rotation on the GPU against the FP64
oracle.

Element by element: FP32 arithmetic of a dozen operations, 1e-6 of the head's largest value
taken ten times over, and for BF16 one rounding of the result, 2^-9 of it (a tie's neighbour:
2^-8).  The weights' gradients are FP32 sums over every token and head: 1e-5 of their 2-norm."""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import linattn as la

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def close(x, ref, dtype):
    x = f64(x).reshape(ref.shape)
    top = np.abs(ref).max(-1, keepdims=True)
    return bool((np.abs(x - ref) <= 1e-5 * top + (2.0 ** -8 * np.abs(ref) if dtype == BF16 else 0)).all())


def make(B, T, H, HK, D, dtype, seed, rot, axes=1, P=97, fused=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    qkv = rn(B, T, (H + 2 * HK) * D).to(dtype).cuda()
    half = rot // 2
    a = torch.rand(P, max(half, 1), generator=g) * 6.28
    x = dict(q=qkv[..., :H * D].view(B, T, H, D), k=qkv[..., H * D:(H + HK) * D].view(B, T, HK, D),
             qw=(rn(D) * 0.2 + 1).cuda(), kw=(rn(D) * 0.2 + 1).cuda(),
             cs=torch.stack([a.cos(), a.sin()], -1).cuda() if rot else None,
             pos=torch.randint(0, P, (axes, B * T), generator=g, dtype=torch.int32).cuda() if rot else None,
             sections=[half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1) if rot else None,
             dq=rn(B, T, H, D).to(dtype).cuda(), dk=rn(B, T, HK, D).to(dtype).cuda())
    if not fused:
        x["q"], x["k"] = x["q"].contiguous(), x["k"].contiguous()
    return x


def rows(t):
    return f64(t).reshape(-1, t.shape[2], t.shape[3])


def check(x, dtype, norm="rms", eps=1e-6, interleaved=False, weights=True):
    import chunked_linear_recurrence_gb300 as sf
    qw, kw = (x["qw"], x["kw"]) if weights else (None, None)
    opt = dict(norm=norm, eps=eps, interleaved=interleaved)
    q, k = sf.sf_qk_norm_rope_fwd(x["q"], x["k"], qw, kw, x["cs"], x["pos"], sections=x["sections"], **opt)
    g = sf.sf_qk_norm_rope_bwd(x["q"], x["k"], qw, kw, x["cs"], x["pos"], x["dq"], x["dk"],
                               sections=x["sections"], **opt)
    cs = None if x["cs"] is None else f64(x["cs"])
    pos = None if x["pos"] is None else x["pos"].cpu().numpy()
    for got, src, w, d, dx, dw in ((q, x["q"], qw, x["dq"], g["dq"], g["dq_weight"]),
                                   (k, x["k"], kw, x["dk"], g["dk"], g["dk_weight"])):
        w = None if w is None else f64(w)
        assert close(got, la.norm_rope(rows(src), w, cs, pos, x["sections"], **opt), dtype)
        rx, rw = la.norm_rope_bwd(rows(src), w, cs, pos, x["sections"], rows(d), **opt)
        # dx cancels g against its part along x: its rounding is that of its terms
        r = np.abs(rows(d)).max(-1, keepdims=True) * 4
        lim = 1e-5 * np.maximum(np.abs(rx).max(-1, keepdims=True), r) + (
            2.0 ** -8 * np.abs(rx) if dtype == BF16 else 0)
        assert (np.abs(f64(dx).reshape(rx.shape) - rx) <= lim).all()
        assert np.linalg.norm(f64(dw) - rw) <= 1e-5 * np.linalg.norm(rw)
    return q, k, g


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("norm,interleaved,axes", [("rms", False, 1), ("rms", True, 3), ("l2", False, 2)])
def test_slices_of_a_fused_projection(dtype, D, norm, interleaved, axes):
    for B, T, H, HK in ((1, 1, 1, 1), (3, 1, 5, 1), (2, 33, 4, 2), (1, 301, 6, 3)):
        check(make(B, T, H, HK, D, dtype, T + D, D, axes), dtype, norm, interleaved=interleaved)


@pytest.mark.parametrize("rot,axes", [(0, 1), (8, 1), (24, 2), (64, 4), (120, 3)])
def test_partial_rotation_sections_and_no_weights(rot, axes):
    """Sections that end inside a lane's four pairs, heads that are rotated in part or not."""
    for interleaved in (False, True):
        check(make(2, 19, 3, 3, 128, F32, rot, rot, axes, fused=False), F32, interleaved=interleaved,
              weights=False)


def test_zero_and_tiny_rows():
    """Rows of zeros, and rows shorter than eps (where the l2 norm divides by eps)."""
    for norm, eps in (("rms", 1e-6), ("l2", 1e-3)):
        x = make(1, 9, 2, 1, 64, F32, 3, 64, fused=False)
        x["q"][:, 2] = 0
        x["k"][:, 4] *= 1e-6
        check(x, F32, norm, eps)


def test_positions_outside_the_table_are_clamped():
    x = make(1, 8, 2, 2, 64, F32, 5, 64)
    x["pos"][0, :4] = torch.tensor([-1, -(1 << 31), 97, (1 << 31) - 1], device="cuda", dtype=torch.int32)
    check(x, F32)


def test_in_place_empty_and_other_stream():
    import chunked_linear_recurrence_gb300 as sf
    x = make(2, 40, 4, 2, 128, BF16, 6, 128, fused=False)
    a = lambda y: (y["q"], y["k"], y["qw"], y["kw"], y["cs"], y["pos"])   # noqa: E731
    q, k = sf.sf_qk_norm_rope_fwd(*a(x))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q2, k2 = sf.sf_qk_norm_rope_fwd(*a(x), stream=side)
    side.synchronize()
    assert torch.equal(q, q2) and torch.equal(k, k2)
    y = {**x, "q": x["q"].clone(), "k": x["k"].clone()}
    q3, k3 = sf.sf_qk_norm_rope_fwd(*a(y), q_out=y["q"], k_out=y["k"])
    assert q3 is y["q"] and torch.equal(q, q3) and torch.equal(k, k3)
    e = make(1, 0, 4, 2, 128, BF16, 6, 128, fused=False)
    assert sf.sf_qk_norm_rope_fwd(*a(e))[0].shape == (1, 0, 4, 128)
    g = sf.sf_qk_norm_rope_bwd(*a(e), e["dq"], e["dk"])
    assert not g["dq_weight"].any() and not g["dk_weight"].any()


def test_gradient_against_differences_and_repeats_bitwise():
    """Central differences of the FP32 forward: curvature of order h^2, rounding 1e-6 / h."""
    import chunked_linear_recurrence_gb300 as sf
    x = make(1, 21, 2, 1, 64, F32, 7, 64, 3, fused=False)
    kw = dict(sections=x["sections"])
    args = lambda q, qw: (q, x["k"], qw, x["kw"], x["cs"], x["pos"])   # noqa: E731
    g = sf.sf_qk_norm_rope_bwd(*args(x["q"], x["qw"]), x["dq"], x["dk"], **kw)
    h = sf.sf_qk_norm_rope_bwd(*args(x["q"], x["qw"]), x["dq"], x["dk"], **kw)
    assert all(torch.equal(g[n], h[n]) for n in g)
    loss = lambda q, qw: (sf.sf_qk_norm_rope_fwd(*args(q, qw), **kw)[0].double() * x["dq"].double()).sum()   # noqa: E731
    gen = torch.Generator().manual_seed(9)
    for name, grad in (("q", "dq"), ("qw", "dq_weight")):
        u = torch.randn(x[name].shape, generator=gen).cuda()
        e = 1e-2
        y = {n: [x[n], x[n]] for n in ("q", "qw")}
        y[name] = [x[name] + e * u, x[name] - e * u]
        d = (loss(y["q"][0], y["qw"][0]) - loss(y["q"][1], y["qw"][1])) / (2 * e)
        exact = (g[grad].double() * u.double()).sum()
        size = (g[grad].double().norm() * u.double().norm())
        assert abs(d - exact) <= 1e-3 * size, name


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("rot,axes", [(8, 1), (24, 2), (40, 3), (56, 4)])
def test_partial_rotation_of_bf16_that_ends_inside_a_group_of_eight(D, rot, axes):
    """rotary_dim / 2 is no multiple of 8: groups of four elements, 8-byte accesses."""
    for norm, interleaved in (("rms", False), ("rms", True), ("l2", False), ("l2", True)):
        check(make(2, 19, 5, 3, D, BF16, rot + D, rot, axes), BF16, norm, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_and_backward_in_a_graph(dtype):
    """Replayed on new inputs in the same buffers: bitwise the calls' results."""
    import chunked_linear_recurrence_gb300 as sf
    x, y = (make(2, 33, 4, 2, 128, dtype, s, 128, 3, fused=False) for s in (21, 22))
    ws = sf.sf_qk_norm_rope_bwd_workspace(x["q"], x["k"])

    def run(z, ws=None):
        a = (z["q"], z["k"], z["qw"], z["kw"], z["cs"], z["pos"])
        f = sf.sf_qk_norm_rope_fwd(*a, sections=z["sections"])
        return list(f) + list(sf.sf_qk_norm_rope_bwd(*a, z["dq"], z["dk"], sections=z["sections"], ws=ws).values())
    run(x, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x, ws)
    for n in ("q", "k", "qw", "kw", "cs", "pos", "dq", "dk"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(map(torch.equal, got, run(y)))
