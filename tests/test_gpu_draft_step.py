"""Drafted tokens and commits on the GPU against the FP64 oracle.

FP32 arithmetic.  A token's u has a relative error of about 4e-6 of the terms' 2-norm: dot products
of 128 terms 128^0.5 2^-24 = 7e-7, products of up to 32 decays 32 x 2^-24 = 1.9e-6, the two factors
of a coefficient.  With keys of length <= 1 and beta in [0,1] the rule does not expand an error, and
those of up to 64 tokens (pending and drafted) are independent: 64^0.5 x 4e-6 = 3.2e-5 of the
result's 2-norm.  A BF16 output is rounded once: 2^-8 at most."""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import decode as od

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TOL = {F32: 3.2e-5, BF16: 2.0 ** -8 + 3.2e-5}
NAN = float("nan")


def err(x, ref):
    n = np.linalg.norm(ref)
    return np.linalg.norm(f64(x) - ref) / (n if n > 0 else 1.0)


def tokens(g, N, T, H, HK, D, dtype, delta, q=True):
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
    t = dict(k=unit(rn(N, T, HK, D)).to(dtype), v=rn(N, T, H, D).to(dtype))
    if q:
        t["q"] = unit(rn(N, T, HK, D)).to(dtype)
    if delta:
        t["gate"] = -torch.rand(N, T, H, generator=g)
        t["beta"] = torch.rand(N, T, H, generator=g)
    return {m: x.cuda() for m, x in t.items()}


def case(N, T, P, H, HK, D, dtype, delta, seed, slots=None):
    g = torch.Generator().manual_seed(seed)
    slots = slots or N + 3
    x = dict(new=tokens(g, N, T, H, HK, D, dtype, delta), delta=delta,
             pend=tokens(g, N, P, H, HK, D, dtype, delta, q=False) if P else None,
             cache=torch.randn(slots, H, D, D, generator=g).cuda(),
             decay=None if delta else (-torch.rand(H, generator=g)).cuda())
    x["idx"] = (torch.randperm(slots - 1, generator=g)[:N] + 1).to(torch.int32).cuda()
    x["num"] = torch.randint(0, T + 1, (N,), generator=g, dtype=torch.int32).cuda()
    x["num_pend"] = torch.randint(0, P + 1, (N,), generator=g, dtype=torch.int32).cuda() if P else None
    return x


def rule(x, t):
    return (t["gate"], t["beta"]) if x["delta"] else ()


def call(x, **kw):
    import chunked_linear_recurrence_gb300 as sf
    n, p = x["new"], x["pend"]
    kw = {**dict(num_tokens=x["num"], pending=None if p is None else (p["k"], p["v"], *rule(x, p)),
                 num_pending=x["num_pend"]), **kw}
    idx = kw.pop("idx", x["idx"])
    if x["delta"]:
        return sf.sf_gdn_draft_step(n["q"], n["k"], n["v"], n["gate"], n["beta"], x["cache"], idx, **kw)
    return sf.sf_linattn_draft_step(n["q"], n["k"], n["v"], x["decay"], x["cache"], idx, **kw)


def commit(x, t, num, **kw):
    import chunked_linear_recurrence_gb300 as sf
    if x["delta"]:
        return sf.sf_gdn_commit(t["k"], t["v"], t["gate"], t["beta"], x["cache"], x["idx"], num_tokens=num, **kw)
    return sf.sf_linattn_commit(t["k"], t["v"], x["decay"], x["cache"], x["idx"], num_tokens=num, **kw)


def ints(t):
    return None if t is None else t.tolist()


def want(x, idx="own", **kw):
    wide = lambda t: None if t is None else {m: f64(v) for m, v in t.items()}   # noqa: E731
    a = dict(num=ints(x["num"]), num_pend=ints(x["num_pend"]), scale=None)
    a.update(kw)
    return od.draft_step(wide(x["new"]), a["num"], wide(x["pend"]), a["num_pend"], f64(x["cache"]),
                         ints(x["idx"]) if isinstance(idx, str) else idx,
                         None if x["delta"] else f64(x["decay"]), a["scale"])


def check(x, out, ro, rc, dtype):
    assert err(out, ro) <= TOL[dtype], err(out, ro)
    assert err(x["cache"], rc) <= TOL[F32], err(x["cache"], rc)
    assert not f64(out)[ro == 0].any()                        # rows behind num_tokens


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("N,T,P,H,HK", [(1, 1, 0, 1, 1), (1, 1, 1, 2, 1), (5, 4, 4, 3, 1), (7, 5, 3, 4, 2),
                                        (3, 8, 0, 2, 2), (2, 17, 9, 2, 1), (2, 32, 32, 1, 1), (3, 0, 5, 2, 1),
                                        (2, 3, 16, 6, 3)])
def test_draft_step(N, T, P, H, HK, dtype, D, delta):
    x = case(N, T, P, H, HK, D, dtype, delta, 100 * T + P + D)
    ro, rc = want(x)
    before = x["cache"].clone()
    out = call(x)
    check(x, out, ro, rc, dtype)
    adv = [] if x["num_pend"] is None else [s for s, n in zip(x["idx"].tolist(), x["num_pend"].tolist()) if n]
    same = [s for s in range(N + 3) if s not in adv]
    assert torch.equal(x["cache"][same], before[same])


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 13, 16, 24, 32])
def test_every_token_counts_where_no_numbers_are_given(T, dtype, D, delta):
    x = case(2, T, T, 2, 1, D, dtype, delta, T)
    ro, rc = want(x, num=None, num_pend=None, scale=0.5)
    out = call(x, num_tokens=None, num_pending=None, scale=0.5)
    check(x, out, ro, rc, dtype)


@pytest.mark.parametrize("delta", [False, True])
def test_commit_then_draft_equals_both_in_one_call(delta):
    """Committed by itself a state is, to the bit, what the draft step writes.  The drafts of one
    call come from the state before both: each way is within the tolerance of the exact outputs, so
    they are within twice that of each other."""
    x = case(6, 5, 4, 4, 2, 128, BF16, delta, 3)
    y = dict(x, cache=x["cache"].clone())
    out = call(x)
    commit(y, y["pend"], y["num_pend"])
    assert torch.equal(x["cache"], y["cache"])
    assert err(out, f64(call(y, pending=None, num_pending=None))) <= 2 * TOL[BF16]


@pytest.mark.parametrize("delta", [False, True])
def test_padding_and_bad_counts(delta):
    """Indices outside the pool and counts outside their range, on the device."""
    x = case(6, 3, 2, 2, 2, 64, BF16, delta, 4, slots=5)
    idx = torch.tensor([0, 3, -1, 5, 1 << 30, 2], dtype=torch.int32, device="cuda")     # 5: past the pool
    x["num"] = torch.tensor([3, 99, 3, 3, 3, -7], dtype=torch.int32, device="cuda")
    x["num_pend"] = torch.tensor([2, -1, 2, 2, 2, 1 << 30], dtype=torch.int32, device="cuda")
    before = x["cache"].clone()
    ro, rc = want(x, idx=idx.tolist())
    out = call(x, idx=idx, out=torch.full_like(x["new"]["v"], NAN))
    check(x, out, ro, rc, BF16)
    assert torch.equal(x["cache"][[0, 1, 3, 4]], before[[0, 1, 3, 4]])
    assert not out[[0, 2, 3, 4, 5]].float().any() and out[1].float().any()


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_do_not_count_reach_nothing(delta, dtype):
    x = case(4, 9, 6, 2, 1, 128, dtype, delta, 5)
    x["num"] = torch.tensor([0, 3, 8, 9], dtype=torch.int32, device="cuda")
    x["num_pend"] = torch.tensor([6, 0, 5, 1], dtype=torch.int32, device="cuda")
    ro, rc = want(x)
    for t, num in ((x["new"], x["num"]), (x["pend"], x["num_pend"])):
        for m in t:
            for n in range(4):
                t[m][n, num[n]:] = NAN if n % 2 else float("inf")
    out = call(x, out=torch.full_like(x["new"]["v"], NAN))
    check(x, out, ro, rc, dtype)


def test_gates_at_their_ends():
    """No decay, a large one and none of the past at all: no infinity less an infinity."""
    for delta in (False, True):
        x = case(3, 6, 5, 3, 3, 64, F32, delta, 6)
        ends = torch.tensor([0.0, -90.0, -float("inf")], device="cuda")
        if delta:
            for t in (x["new"], x["pend"]):
                t["gate"][:] = ends
                t["gate"][0, 1::2] = -0.5
                t["beta"][1] = 1.0
                t["beta"][2] = 0.0
        else:
            x["decay"] = ends
        ro, rc = want(x, num=None, num_pend=None)
        out = call(x, num_tokens=None, num_pending=None)
        assert np.isfinite(f64(out)).all()
        for h in range(3):
            assert err(out[:, :, h], ro[:, :, h]) <= TOL[F32]
            assert err(x["cache"][x["idx"].long(), h], rc[x["idx"].tolist(), h]) <= TOL[F32]


@pytest.mark.parametrize("delta", [False, True])
def test_a_sequence_owns_its_slot_without_indices(delta):
    x = case(3, 2, 2, 2, 1, 128, BF16, delta, 7, slots=4)
    ro, rc = want(x, idx=None)
    check(x, call(x, idx=None), ro, rc, BF16)


@pytest.mark.parametrize("delta", [False, True])
def test_a_pool_of_more_than_2_31_elements(delta):
    H, D, slots = 32, 128, 4200
    cache = torch.zeros(slots, H, D, D, device="cuda")
    assert cache.numel() > 1 << 31
    x = case(2, 3, 2, H, H, D, BF16, delta, 8)
    small = x["cache"][x["idx"].long()].clone()
    cache[4199], cache[4100] = small[0], small[1]
    ro, rc = want(x, num=None, num_pend=None)
    rows = x["idx"].tolist()
    x["idx"] = torch.tensor([4199, 4100], dtype=torch.int32, device="cuda")
    y = dict(x, cache=cache)
    out = call(y, num_tokens=None, num_pending=None)
    assert err(out, ro) <= TOL[BF16]
    assert err(cache[4199], rc[rows[0]]) <= TOL[F32] and err(cache[4100], rc[rows[1]]) <= TOL[F32]
    assert not cache[:4100].any()


@pytest.mark.parametrize("delta", [False, True])
def test_one_token_at_a_time_is_the_step(delta):
    """Committed tokens are those of the one-token step, drafts its outputs."""
    import chunked_linear_recurrence_gb300 as sf
    x = case(5, 6, 0, 4, 2, 128, F32, delta, 9)
    y = dict(x, cache=x["cache"].clone())
    out = call(x, num_tokens=None)
    n = y["new"]
    for t in range(6):
        at = lambda m: n[m][:, t].contiguous()   # noqa: E731
        own = (at("gate"), at("beta")) if delta else (y["decay"],)
        o = (sf.sf_gdn_step if delta else sf.sf_linattn_step)(at("q"), at("k"), at("v"), *own, y["cache"], y["idx"])
        assert err(out[:, t], f64(o)) <= 2 * TOL[F32]
    commit(x, n, None)
    assert err(x["cache"], f64(y["cache"])) <= 2 * TOL[F32]


@pytest.mark.parametrize("delta", [False, True])
def test_more_states_than_fit_the_machine_at_once(delta):
    """Thousands of states, ragged: every head against the same heads in a call of their own."""
    x = case(150, 4, 3, 16, 8, 128, BF16, delta, 10)
    y = dict(x, cache=x["cache"].clone())
    out = call(x)
    for n in (0, 77, 149):
        one = dict(y, new={m: t[n:n + 1].contiguous() for m, t in y["new"].items()},
                   pend={m: t[n:n + 1].contiguous() for m, t in y["pend"].items()},
                   idx=y["idx"][n:n + 1], num=y["num"][n:n + 1], num_pend=y["num_pend"][n:n + 1])
        ro, rc = want(one)
        assert err(out[n:n + 1], ro) <= TOL[BF16]
        slot = int(y["idx"][n])
        assert err(x["cache"][slot], rc[slot]) <= TOL[F32]
        assert torch.equal(call(one), out[n:n + 1]) and torch.equal(one["cache"][slot], x["cache"][slot])


@pytest.mark.parametrize("delta", [False, True])
def test_rounds_replayed_in_a_graph(delta):
    """Three replays advance the pool as three calls do, with counts that change in between, on a
    stream of their own."""
    x = case(5, 4, 4, 4, 2, 128, BF16, delta, 11)
    y = dict(x, cache=x["cache"].clone(), num_pend=x["num_pend"].clone(), num=x["num"].clone())
    call(dict(x, cache=x["cache"].clone()))                 # loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(y)
    for i in range(3):
        x["num_pend"] = torch.tensor([i, 4, 0, 2, 1], dtype=torch.int32, device="cuda")
        x["num"] = torch.tensor([4, i, 3, 0, 2], dtype=torch.int32, device="cuda")
        y["num_pend"].copy_(x["num_pend"])
        y["num"].copy_(x["num"])
        ref = call(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(x["cache"], y["cache"])


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("T,P", [(5, 4), (8, 8), (16, 12)])
def test_rows_that_do_not_count_reach_nothing_in_short_calls(T, P, dtype, D, delta):
    """Up to eight tokens of each kind, and up to sixteen: none counts, some do, all do."""
    x = case(4, T, P, 2, 1, D, dtype, delta, 12)
    x["num"] = torch.tensor([0, 3, T - 1, T], dtype=torch.int32, device="cuda")
    x["num_pend"] = torch.tensor([P, 0, P - 1, 1], dtype=torch.int32, device="cuda")
    ro, rc = want(x)
    for t, num in ((x["new"], x["num"]), (x["pend"], x["num_pend"])):
        for m in t:
            for n in range(4):
                t[m][n, num[n]:] = NAN if n % 2 else float("inf")
    out = call(x, out=torch.full_like(x["new"]["v"], NAN))
    check(x, out, ro, rc, dtype)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,P", [(6, 3), (6, 0), (14, 3)])
def test_a_bad_draft_reaches_the_ones_behind_it_alone(T, P, dtype, delta):
    """A NaN or an infinity in a draft: not the drafts before it, other heads' or sequences', nor the pool."""
    for what, bad in (("k", NAN), ("v", float("inf")), ("q", NAN)):
        x = case(3, T, P, 2, 2, 128, dtype, delta, 13)
        x["num"] = None
        y = dict(x, cache=x["cache"].clone(), new={m: t.clone() for m, t in x["new"].items()})
        good = call(x)
        y["new"][what][1, 4, 0, 7] = bad
        out = call(y)
        assert torch.equal(x["cache"], y["cache"])
        same = torch.ones(3, T, 2, dtype=torch.bool)
        same[1, 4:, 0] = False
        assert torch.equal(out[same.cuda()], good[same.cuda()])
        assert not torch.isfinite(out[1, 4, 0]).all()


@pytest.mark.parametrize("delta", [False, True])
def test_gates_at_their_ends_in_one_pass(delta):
    x = case(3, 6, 5, 3, 3, 64, BF16, delta, 14)
    ends = torch.tensor([0.0, -90.0, -float("inf")], device="cuda")
    if delta:
        for t in (x["new"], x["pend"]):
            t["gate"][:] = ends
            t["gate"][0, 1::2] = -0.5
            t["beta"][1] = 1.0
            t["beta"][2] = 0.0
    else:
        x["decay"] = ends
    ro, rc = want(x, num=None, num_pend=None)
    out = call(x, num_tokens=None, num_pending=None)
    assert np.isfinite(f64(out)).all()
    for h in range(3):
        assert err(out[:, :, h], ro[:, :, h]) <= TOL[BF16]
        assert err(x["cache"][x["idx"].long(), h], rc[x["idx"].tolist(), h]) <= TOL[F32]
