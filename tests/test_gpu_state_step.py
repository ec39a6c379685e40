"""The single-token steps on the GPU against the FP64 oracle.

Both compute in FP32: a row's dot products of at most 128 terms, 128^0.5 2^-24 < 1e-6 of the
terms' 2-norm; with the cancellation of v against S k the bound taken is 1e-5 of the result's
2-norm (FP32 outputs, states).  A BF16 output is rounded once: 2^-9."""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import linattn as la

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-5, BF16: 2.0 ** -9 + 1e-5}


def err(x, ref):
    n = np.linalg.norm(ref)
    return np.linalg.norm(f64(x) - ref) / (n if n > 0 else 1.0)


def inputs(N, H, HK, D, dtype, seed, slots):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    x = dict(q=unit(rn(N, HK, D)).to(dtype), k=unit(rn(N, HK, D)).to(dtype), v=rn(N, H, D).to(dtype),
             decay=-torch.rand(H, generator=g), gate=-torch.rand(N, H, generator=g) * 2,
             beta=torch.rand(N, H, generator=g), cache=rn(slots, H, D, D))
    return {n: t.cuda() for n, t in x.items()}


def call(x, delta, idx, **kw):
    import chunked_linear_recurrence_gb300 as sf
    if delta:
        return sf.sf_gdn_step(x["q"], x["k"], x["v"], x["gate"], x["beta"], x["cache"], idx, **kw)
    return sf.sf_linattn_step(x["q"], x["k"], x["v"], x["decay"], x["cache"], idx, **kw)


def want(x, delta, idx, scale=None):
    rule = dict(gate=f64(x["gate"]), beta=f64(x["beta"])) if delta else dict(decay=f64(x["decay"]))
    return la.step(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["cache"]),
                   None if idx is None else idx.tolist(), scale=scale, **rule)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("N,H,HK", [(1, 1, 1), (5, 3, 1), (7, 4, 2)])
def test_step(N, H, HK, dtype, D, delta):
    x = inputs(N, H, HK, D, dtype, N + D, N + 3)
    idx = (torch.randperm(N + 2, generator=torch.Generator().manual_seed(1))[:N] + 1).to(torch.int32).cuda()
    ro, rc = want(x, delta, idx)
    before = x["cache"].clone()
    out = call(x, delta, idx)
    assert err(out, ro) <= TOL[dtype] and err(x["cache"], rc) <= 1e-5
    free = [s for s in range(N + 3) if s not in idx.tolist()]
    assert torch.equal(x["cache"][free], before[free])


@pytest.mark.parametrize("delta", [False, True])
def test_padding_leaves_the_pool_alone(delta):
    x = inputs(6, 2, 2, 64, BF16, 4, 5)
    idx = torch.tensor([0, 3, -1, 5, 1 << 30, 2], dtype=torch.int32, device="cuda")   # 5: past the pool
    x["q"][0], x["v"][2] = float("nan"), float("nan")
    before = x["cache"].clone()
    y = {**x, "q": torch.nan_to_num(x["q"]), "v": torch.nan_to_num(x["v"])}
    ro, rc = want(y, delta, torch.tensor([-1, 3, -1, -1, -1, 2]))
    out = call(x, delta, idx, out=torch.full_like(x["v"], float("nan")))
    assert err(out, ro) <= TOL[BF16] and err(x["cache"], rc) <= 1e-5
    assert not out[[0, 2, 3, 4]].float().any()
    assert torch.equal(x["cache"][[0, 1, 4]], before[[0, 1, 4]])


@pytest.mark.parametrize("delta", [False, True])
def test_no_indices_scale_and_no_sequences(delta):
    x = inputs(3, 2, 1, 128, F32, 6, 4)
    ro, rc = want(x, delta, None, 0.5)
    out = call(x, delta, None, scale=0.5)
    assert err(out, ro) <= TOL[F32] and err(x["cache"], rc) <= 1e-5
    e = {n: (t[:0] if n not in ("decay", "cache") else t) for n, t in x.items()}
    assert call(e, delta, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 2, 128)


def test_decays_at_their_ends():
    """No decay, a large one and none of the past at all."""
    x = inputs(2, 3, 3, 64, F32, 8, 4)
    x["decay"] = torch.tensor([0.0, -90.0, -float("inf")], device="cuda")
    idx = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    ro, rc = want(x, False, idx)
    out = call(x, False, idx)
    for h in range(3):
        assert err(out[:, h], ro[:, h]) <= 1e-5 and err(x["cache"][:, h], rc[:, h]) <= 1e-5


def test_a_pool_of_more_than_2_31_elements():
    """Slots whose element offsets pass 32 bits."""
    H, D, slots = 32, 128, 4200
    cache = torch.zeros(slots, H, D, D, device="cuda")
    assert cache.numel() > 1 << 31
    x = inputs(2, H, H, D, BF16, 9, 2)
    cache[4199], cache[4100] = x["cache"][0], x["cache"][1]
    rule = dict(decay=f64(x["decay"]))
    ro, rc = la.step(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["cache"]), None, **rule)
    idx = torch.tensor([4199, 4100], dtype=torch.int32, device="cuda")
    out = call({**x, "cache": cache}, False, idx)
    assert err(out, ro) <= TOL[BF16]
    assert err(cache[4199], rc[0]) <= 1e-5 and err(cache[4100], rc[1]) <= 1e-5
    assert not cache[:4100].any()


@pytest.mark.parametrize("delta", [False, True])
def test_prefill_then_steps_equal_one_prefill(delta):
    """100 tokens by the paged prefill and 4 by steps, through the same pool, give the states and
    outputs of 104 tokens."""
    import oracle
    import chunked_linear_recurrence_gb300 as sf
    B, T, H, HK, D = 2, 104, 4, 2, 128
    g = torch.Generator().manual_seed(11)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    q, k, v = (t.to(BF16).cuda() for t in (unit(rn(B, T, HK, D)), unit(rn(B, T, HK, D)), rn(B, T, H, D)))
    gate, beta = (-torch.rand(B, T, H, generator=g)).cuda(), torch.rand(B, T, H, generator=g).cuda()
    decay = -torch.rand(H, generator=g).cuda()
    cache = torch.full((4, H, D, D), float("nan"), device="cuda")
    idx = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    fresh = torch.zeros(B, dtype=torch.bool, device="cuda")
    cut = lambda t: t[:, :100].contiguous()   # noqa: E731
    if delta:
        outs = [sf.sf_gdn_paged_chunk_fwd(cut(q), cut(k), cut(v), cut(gate), cut(beta), cache, idx,
                                          has_initial_state=fresh)]
    else:
        outs = [sf.sf_linattn_paged_chunk_fwd(cut(q), cut(k), cut(v), decay, cache, idx, has_initial_state=fresh)]
    for t in range(100, T):
        at = lambda x: x[:, t].contiguous()   # noqa: E731
        if delta:
            o = sf.sf_gdn_step(at(q), at(k), at(v), at(gate), at(beta), cache, idx)
        else:
            o = sf.sf_linattn_step(at(q), at(k), at(v), decay, cache, idx)
        outs.append(o[:, None])
    out = torch.cat(outs, 1)
    if delta:   # the chunked delta rule's own tolerance for BF16
        ro, rf = oracle.gdn_fwd(*(f64(t) for t in (q, k, v, gate, beta)))
        tol = 2e-2
    else:
        ro, rf = la.fwd(f64(q), f64(k), f64(v), f64(decay))
        tol = 5e-3
    assert err(out, ro) <= tol and err(cache[idx.long()], rf) <= (tol if delta else 1e-5)


@pytest.mark.parametrize("delta", [False, True])
def test_steps_replayed_in_a_graph(delta):
    """Three replays advance the pool as three calls do."""
    x = inputs(5, 4, 2, 128, BF16, 41, 8)
    idx = torch.tensor([3, 1, -1, 7, 2], dtype=torch.int32, device="cuda")
    y = dict(x, cache=x["cache"].clone())
    call(dict(x, cache=x["cache"].clone()), delta, idx)                 # loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(y, delta, idx)
    for _ in range(3):
        ref = call(x, delta, idx)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(x["cache"], y["cache"])
