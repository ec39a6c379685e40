"""The decayed linear attention on the GPU against the FP64 oracle.

Tolerances (2-norm of the difference over that of the reference).  FP32 outputs and states:
sums of at most ~400 terms a chunk in FP32, 400^0.5 2^-24 = 1.2e-6, and as much again for the
powers of lam: 1e-5.  BF16 outputs: three independent roundings to BF16 (the products q.k, the
state that the query reads, the result), each at most 2^-9 relative, 2^-9 3^0.5 = 3.4e-3: 5e-3.
"""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import linattn as la

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
STATE = 1e-5
TOL = {F32: 1e-5, BF16: 5e-3}


def _sf():
    import chunked_linear_recurrence_gb300 as sf
    return sf


def err(x, ref, rows=None):
    x = f64(x) if isinstance(x, torch.Tensor) else x
    if rows is not None:
        x, ref = x[:, rows], ref[:, rows]
    n = np.linalg.norm(ref)
    return np.linalg.norm(x - ref) / (n if n > 0 else 1.0)


def inputs(B, T, H, HK, D, dtype, seed, lengths=None, decay=None, s0=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    N = B if lengths is None else len(lengths)
    x = dict(q=unit(rn(B, T, HK, D)).to(dtype), k=unit(rn(B, T, HK, D)).to(dtype), v=rn(B, T, H, D).to(dtype),
             decay=torch.tensor(decay, dtype=F32) if decay is not None else -torch.rand(H, generator=g) ** 3,
             s0=rn(N, H, D, D) * 0.1 if s0 else None, do=rn(B, T, H, D).to(dtype), df=rn(N, H, D, D) * 0.1)
    cu = None if lengths is None else torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)
    return {n: (t.cuda() if t is not None else None) for n, t in dict(x, cu=cu).items()}


def ref_fwd(x, scale=None):
    return la.fwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["decay"]), f64(x["s0"]),
                  None if x["cu"] is None else x["cu"].tolist(), scale)


def ref_bwd(x, scale=None, df=True):
    return la.bwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["decay"]), f64(x["s0"]), f64(x["do"]),
                  f64(x["df"]) if df else None, None if x["cu"] is None else x["cu"].tolist(), scale)


def run_fwd(x, **kw):
    return _sf().sf_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], cu_seqlens=x["cu"],
                                      output_final_state=True, **kw)


SIZES = [(1, 1, 1, 1), (1, 2, 3, 1), (2, 63, 2, 2), (1, 64, 2, 1), (1, 65, 1, 1), (3, 130, 4, 2), (1, 257, 2, 2),
         (2, 700, 1, 1)]


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("B,T,H,HK", SIZES)
def test_dense_forward_and_backward(B, T, H, HK, dtype, D):
    x = inputs(B, T, H, HK, D, dtype, seed=T + D)
    ro, rf = ref_fwd(x)
    out, fin = run_fwd(x)
    assert err(out, ro) <= TOL[dtype] and err(fin, rf) <= STATE
    rg = ref_bwd(x)
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])
    for n in ("dq", "dk", "dv"):
        assert err(g[n], rg[n]) <= TOL[dtype], n
    assert err(g["d_initial_state"], rg["d_initial_state"]) <= STATE


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("B,T,H,HK", [(1, 1, 1, 1), (5, 1, 1, 1), (2, 5, 2, 1), (1, 33, 4, 2), (1, 64, 1, 1)])
def test_a_single_chunk_is_rounded_once(B, T, H, HK, D):
    """Up to 64 BF16 tokens with no state: every output is a sum kept in FP32 and rounded to BF16
    once.  Each element is within half a unit in its last place (8 significant bits: 2^(e - 8)
    for a value in [2^e, 2^(e+1))), and 1e-5 of the largest for the sums and for products of 16 bits."""
    x = inputs(B, T, H, HK, D, BF16, seed=900 + T + D, s0=False)

    def once(got, ref):
        half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 8)
        return (np.abs(f64(got) - ref) <= half + 1e-5 * np.abs(ref).max()).all()
    assert once(run_fwd(x)[0], ref_fwd(x)[0])
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], None, x["do"])
    rg = ref_bwd(x, df=False)
    for n in ("dq", "dk", "dv"):
        assert once(g[n], rg[n]), n


@pytest.mark.parametrize("dtype,D,H,HK", [(BF16, 128, 4, 2), (BF16, 64, 3, 1), (F32, 64, 2, 2), (F32, 128, 2, 1)])
def test_packed_sequences(dtype, D, H, HK):
    """Ragged lengths with empty and one-token sequences; rows past the last sequence hold NaN
    inputs and keep what the outputs held."""
    lengths = [130, 0, 64, 1, 0, 261, 0]
    T = sum(lengths) + 9
    x = inputs(1, T, H, HK, D, dtype, seed=50 + D, lengths=lengths)
    end = sum(lengths)
    for n in ("q", "k", "v", "do"):
        x[n][:, end:] = float("nan")
    nan = lambda t: torch.full_like(t, float("nan"))   # noqa: E731
    ro, rf = ref_fwd(x)
    out, fin = run_fwd(x, out=nan(x["v"]))
    rows = np.arange(end)
    assert err(out, ro, rows) <= TOL[dtype] and err(fin, rf) <= STATE
    assert torch.isnan(out[:, end:].float()).all()
    for n in (1, 4, 6):
        assert torch.equal(fin[n], x["s0"][n])
    grads = dict(dq=nan(x["q"]), dk=nan(x["k"]), dv=nan(x["v"]), d_initial_state=nan(x["df"]))
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"],
                                   cu_seqlens=x["cu"], grads=grads)
    rg = ref_bwd(x)
    for n in ("dq", "dk", "dv"):
        assert err(g[n], rg[n], rows) <= TOL[dtype], n
        assert torch.isnan(g[n][:, end:].float()).all(), n
    assert err(g["d_initial_state"], rg["d_initial_state"]) <= STATE


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_a_long_walk_is_cut_into_segments(dtype, D):
    """One chain over 3001 tokens runs as segments side by side; also packed, with a sequence
    of less than one segment."""
    for lengths in (None, [2011, 77, 913]):
        x = inputs(1, 3001, 1, 1, D, dtype, seed=71, lengths=lengths, decay=[-0.004])
        ro, rf = ref_fwd(x)
        out, fin = run_fwd(x)
        assert err(out, ro) <= TOL[dtype] and err(fin, rf) <= STATE
        rg = ref_bwd(x)
        g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"],
                                       cu_seqlens=x["cu"])
        for n in ("dq", "dk", "dv"):
            assert err(g[n], rg[n]) <= TOL[dtype], n
        assert err(g["d_initial_state"], rg["d_initial_state"]) <= STATE


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_one_long_sequence_among_many_walks(dtype, D):
    """More walks than SMs and one far above the even share: it alone is cut, the others (one of
    them empty) read and write the caller's states next to it; also in place on a pool."""
    lengths = [77, 1601, 0, 64, 1, 300]
    x = inputs(1, sum(lengths) + 3, 32, 8, D, dtype, seed=77, lengths=lengths)
    rows = np.arange(sum(lengths))
    ro, rf = ref_fwd(x)
    out, fin = run_fwd(x)
    assert err(out, ro, rows) <= TOL[dtype]
    for n in range(len(lengths)):
        assert err(fin[n], rf[n]) <= STATE, n
    cache = torch.full((8, 32, D, D), float("nan"), device="cuda")
    idx = torch.tensor([3, 1, 7, 2, 6, 4], dtype=torch.int32, device="cuda")
    cache[idx.long()] = x["s0"]
    paged = _sf().sf_linattn_paged_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], cache, idx, cu_seqlens=x["cu"])
    assert torch.equal(paged[:, :len(rows)], out[:, :len(rows)]) and torch.equal(cache[idx.long()], fin)
    rg = ref_bwd(x)
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"],
                                   cu_seqlens=x["cu"])
    for n in ("dq", "dk", "dv"):
        assert err(g[n], rg[n], rows) <= TOL[dtype], n
    for n in range(len(lengths)):
        assert err(g["d_initial_state"][n], rg["d_initial_state"][n]) <= STATE, n


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_decays_at_their_ends(dtype, D):
    """No decay, hardly any, one that underflows within a chunk, and no memory at all."""
    dec = [0.0, -1e-6, -50.0, -float("inf")]
    x = inputs(1, 333, 4, 2, D, dtype, seed=80, decay=dec)
    ro, rf = ref_fwd(x)
    out, fin = run_fwd(x)
    rg = ref_bwd(x)
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])
    for h in range(4):
        assert err(out[:, :, h], ro[:, :, h]) <= TOL[dtype], h
        assert err(fin[:, h], rf[:, h]) <= STATE, h
        assert err(g["dv"][:, :, h], rg["dv"][:, :, h]) <= TOL[dtype], h
        assert err(g["d_initial_state"][:, h], rg["d_initial_state"][:, h]) <= STATE, h


def test_state_keeps_fp32_accuracy_over_a_long_memory():
    """65536 tokens with a decay of 1e-5 a token: the state sums thousands of chunks, and a bias
    of one rounding in the carried power of lam (1024 chunks of 2^-25) would show."""
    T, D = 65536, 128
    x = inputs(1, T, 1, 1, D, BF16, seed=90, decay=[-1e-5])
    _, fin = run_fwd(x)
    w = torch.exp(x["decay"].double() * torch.arange(T - 1, -1, -1, device="cuda"))[:, None]
    ref = (x["v"][0, :, 0].double() * w).T @ x["k"][0, :, 0].double() + torch.exp(
        x["decay"].double() * T) * x["s0"][0, 0].double()
    assert err(fin[0, 0], f64(ref)) <= STATE


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_scale_missing_states_and_missing_cotangent(dtype, D):
    x = inputs(2, 100, 2, 2, D, dtype, seed=95, s0=False)
    ro, _ = ref_fwd(x, 0.25)
    out, none = _sf().sf_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], scale=0.25)
    assert none is None and err(out, ro) <= TOL[dtype]
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], None, x["do"], scale=0.25,
                                   want_d_initial_state=False)
    rg = ref_bwd(x, 0.25, df=False)
    assert g["d_initial_state"] is None
    for n in ("dq", "dk", "dv"):
        assert err(g[n], rg[n]) <= TOL[dtype], n


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_final_state_in_place_of_the_initial_state(dtype, D):
    """One walk, cut into segments, and packed ones of which one is not cut."""
    for lengths in (None, [1900, 60, 0]):
        x = inputs(1, 2000, 2, 1, D, dtype, seed=96, lengths=lengths)
        end = 2000 if lengths is None else sum(lengths)
        out, fin = run_fwd(x)
        state = x["s0"].clone()
        again, same = _sf().sf_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], state, cu_seqlens=x["cu"],
                                                 output_final_state=True, final_state=state)
        assert same is state and torch.equal(state, fin) and torch.equal(again[:, :end], out[:, :end])


def test_no_tokens_hand_the_state_through():
    for D, dtype in ((128, BF16), (64, F32)):
        x = inputs(2, 0, 2, 1, D, dtype, seed=1)
        out, fin = run_fwd(x)
        assert out.shape == (2, 0, 2, D) and torch.equal(fin, x["s0"])
        g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])
        assert torch.equal(g["d_initial_state"], x["df"])


@pytest.mark.parametrize("dtype,D,T", [(BF16, 128, 300), (BF16, 128, 2500), (F32, 64, 300), (BF16, 64, 2500)])
def test_paged_prefill(dtype, D, T):
    """The pool's slots advance in place (also where the walk is cut into segments); padding and
    has_initial_state as the gated delta rule's paged prefill."""
    lengths = [T - 140, 0, 75, 65]
    x = inputs(1, T + 4, 2, 1, D, dtype, seed=97, lengths=lengths)
    cache = (torch.randn(8, 2, D, D, generator=torch.Generator().manual_seed(3)) * 0.1).cuda()
    cache[6] = float("nan")
    before = cache.clone()
    idx = torch.tensor([2, 6, -1, 5], dtype=torch.int32, device="cuda")
    has = torch.tensor([True, False, True, True], device="cuda")
    out = torch.full_like(x["v"], float("nan"))
    _sf().sf_linattn_paged_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], cache, idx, cu_seqlens=x["cu"],
                                     has_initial_state=has, out=out)
    s0 = f64(before)[[2, 6, 0, 5]]
    s0[1] = 0
    ro, rf = la.fwd(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["decay"]), s0, x["cu"].tolist())
    cu = x["cu"].tolist()
    for n in (0, 3):
        assert err(out, ro, np.arange(cu[n], cu[n + 1])) <= TOL[dtype]
        assert err(cache[int(idx[n])], rf[n]) <= STATE
    assert not cache[6].any()                                       # a fresh empty sequence
    assert not out[:, cu[2]:cu[3]].float().any() and torch.isnan(out[:, cu[4]:].float()).all()
    for s in (0, 1, 3, 4, 7):
        assert torch.equal(cache[s], before[s])


def test_gradients_against_differences():
    """The loss is linear in each of q, k, v and the initial state, so its central difference
    along a direction is exact up to rounding: two FP32 losses, each off by 1e-6 of the 2-norm of
    its terms."""
    x = inputs(2, 150, 2, 1, 64, F32, seed=99)
    g = _sf().sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])

    def terms(y):
        o, f = run_fwd(y)
        return torch.cat([(o.double() * x["do"].double()).flatten(), (f.double() * x["df"].double()).flatten()])

    gen = torch.Generator().manual_seed(5)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "d_initial_state")):
        u = torch.randn(x[name].shape, generator=gen).cuda()
        a, b = terms({**x, name: x[name] + u}), terms({**x, name: x[name] - u})
        d = (a.sum() - b.sum()) / 2
        assert abs((g[grad].double() * u.double()).sum() - d) <= 2e-6 * (a.norm() + b.norm()) * 8, name


def test_repeats_bitwise_on_another_stream_and_in_a_graph():
    for D, dtype, T in ((128, BF16, 900), (64, F32, 300)):
        x = inputs(2, T, 2, 1, D, dtype, seed=101)
        sf = _sf()
        out, fin = run_fwd(x)
        g = sf.sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o2, f2 = run_fwd(x)
            g2 = sf.sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"])
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, o2) and torch.equal(fin, f2)
        assert all(torch.equal(g[n], g2[n]) for n in g)
        ws = sf.sf_linattn_fwd_workspace(x["q"], x["v"])
        o3, f3 = torch.zeros_like(out), torch.zeros_like(fin)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run_fwd(x, out=o3, final_state=f3, ws=ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o3) and torch.equal(fin, f3)
        sf.sf_workspace_status(ws)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_nothing_but_the_status_word_is_read_before_it_is_written(dtype, D):
    """Walks that are cut and shared heads, in a workspace of NaN bit patterns."""
    sf = _sf()
    for lengths in (None, [1700, 0, 300]):
        x = inputs(1, 2000, 4, 2, D, dtype, seed=103, lengths=lengths)
        args = (x["q"], x["k"], x["v"], x["decay"], x["s0"])
        for call, need in ((lambda ws: run_fwd(x, ws=ws), sf.sf_linattn_fwd_workspace),
                           (lambda ws: tuple(sf.sf_linattn_chunk_bwd(*args, x["do"], x["df"], cu_seqlens=x["cu"],
                                                                     ws=ws).values()), sf.sf_linattn_bwd_workspace)):
            ws = need(x["q"], x["v"], x["cu"])
            assert ws.numel() > 256
            clean = call(torch.zeros_like(ws))
            ws[256:] = 255
            assert all(torch.equal(a, b) for a, b in zip(call(ws), clean))
            sf.sf_workspace_status(ws)
