"""Refusals of the decoding operators: the C ABI's host checks (nothing is launched, so they run
without a GPU) and the binding's shape, type and stride checks."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
BYTE = ctypes.c_void_p((1 << 20) + 1)
HALF = ctypes.c_void_p((1 << 20) + 16)   # (states are stored 32 bytes at a time)


@pytest.fixture(scope="module")
def lib():
    from chunked_linear_recurrence_gb300 import _native
    if not os.path.exists(_native.LIB_PATH):
        from chunked_linear_recurrence_gb300 import build
        build.build()
    return _native.load()


def _shape(**kw):
    from chunked_linear_recurrence_gb300._native import sf_gdn_shape
    return ctypes.byref(sf_gdn_shape(**{**dict(B=1, T=4, H=2, K=128, V=128, N=3, dtype=1, scale=0.0), **kw}))


def _pend(P=4, k=FAKE, v=FAKE, gate=FAKE, beta=FAKE, count=FAKE):
    from chunked_linear_recurrence_gb300._native import sf_pending
    return ctypes.byref(sf_pending(P, k, v, gate, beta, count))


def _draft(lib, delta, shape, q=FAKE, k=FAKE, v=FAKE, rule=FAKE, num=FAKE, pend=None, cache=FAKE, slots=8, idx=FAKE,
           out=FAKE):
    if delta:
        return lib.sf_gdn_draft_step(shape, q, k, v, rule, FAKE, num, pend, cache, slots, idx, out, None)
    return lib.sf_linattn_draft_step(shape, q, k, v, rule, num, pend, cache, slots, idx, out, None)


def _commit(lib, delta, shape, k=FAKE, v=FAKE, rule=FAKE, num=FAKE, cache=FAKE, slots=8, idx=FAKE):
    if delta:
        return lib.sf_gdn_commit(shape, k, v, rule, FAKE, num, cache, slots, idx, None)
    return lib.sf_linattn_commit(shape, k, v, rule, num, cache, slots, idx, None)


BAD = [(dict(K=96, V=96), 2), (dict(K=128, V=64), 2), (dict(T=-1), 1), (dict(T=33), 2), (dict(H=0), 1),
       (dict(dtype=7), 1), (dict(N=-1), 1), (dict(H=4, HK=3), 1), (dict(H=4, HK=-1), 1), (dict(N=1 << 30, H=4), 2)]


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("kw,status", BAD)
def test_draft_steps_and_commits_reject_bad_shapes(lib, delta, kw, status):
    s = _shape(**kw)
    assert _draft(lib, delta, s) == status and _commit(lib, delta, s) == status
    assert len(lib.sf_last_error()) > 0


@pytest.mark.parametrize("delta", [False, True])
def test_draft_steps_and_commits_reject_bad_pointers(lib, delta):
    s = _shape()
    assert _draft(lib, delta, None) == 1 and _commit(lib, delta, None) == 1
    for kw in (dict(q=None), dict(q=ODD), dict(k=None), dict(k=ODD), dict(v=None), dict(v=ODD), dict(rule=None),
               dict(rule=BYTE), dict(num=BYTE), dict(cache=None), dict(cache=ODD), dict(out=None), dict(out=ODD),
               dict(cache=HALF), dict(idx=BYTE), dict(slots=-1), dict(idx=None, slots=2)):
        assert _draft(lib, delta, s, **kw) == 1, kw
        if not set(kw) & {"q", "out"}:
            assert _commit(lib, delta, s, **kw) == 1, kw
    for kw, status in ((dict(P=-1), 1), (dict(P=33), 2), (dict(k=None), 1), (dict(v=ODD), 1), (dict(count=BYTE), 1)):
        assert _draft(lib, delta, s, pend=_pend(**kw)) == status, kw
    if delta:
        assert _draft(lib, delta, s, pend=_pend(gate=None)) == 1 and _draft(lib, delta, s, pend=_pend(beta=None)) == 1


@pytest.mark.parametrize("delta", [False, True])
def test_nothing_to_do_is_no_error(lib, delta):
    assert _draft(lib, delta, _shape(N=0)) == 0 and _commit(lib, delta, _shape(N=0)) == 0
    assert _draft(lib, delta, _shape(T=0)) == 0 and _commit(lib, delta, _shape(T=0)) == 0
    assert _draft(lib, delta, _shape(T=0), q=None, k=None, v=None, out=None, pend=_pend(P=0, k=None)) == 0


def _verify(lib, target=FAKE, x=FAKE, u=FAKE, draft=FAKE, num=FAKE, tokens=FAKE, count=FAKE, **kw):
    from chunked_linear_recurrence_gb300._native import sf_verify_shape
    d = {**dict(N=2, T=3, V=100, dtype=0, target_seq=400, target_row=100, draft_seq=300, draft_row=100), **kw}
    return lib.sf_draft_verify(ctypes.byref(sf_verify_shape(**d)), target, x, u, draft, num, tokens, count, None)


def test_verification_rejects_bad_arguments(lib):
    for kw in (dict(N=-1), dict(T=-1), dict(V=0), dict(dtype=2), dict(target_seq=-1), dict(draft_row=-1),
               dict(target=None), dict(x=None), dict(u=None), dict(tokens=None), dict(count=None), dict(target=BYTE),
               dict(draft=BYTE), dict(x=BYTE), dict(u=BYTE), dict(num=BYTE), dict(tokens=BYTE), dict(count=BYTE),
               dict(dtype=1, target=BYTE)):
        assert _verify(lib, **kw) == 1, kw
    for kw in (dict(N=(1 << 24) + 1), dict(T=(1 << 20) + 1), dict(V=(1 << 30) + 1)):
        assert _verify(lib, **kw) == 2, kw
    assert _verify(lib, N=0, target=None) == 0
    assert lib.sf_draft_verify(None, *([FAKE] * 7), None) == 1


def _pool(slots=8, sizes=(1 << 16,), at=None):
    from chunked_linear_recurrence_gb300._native import sf_state_pool
    n = len(sizes)
    a = (ctypes.c_void_p * n)(*(at or [1 << 20] * n))
    return ctypes.byref(sf_state_pool(slots, n, a, (ctypes.c_size_t * n)(*sizes)))


def test_pool_operators_reject_bad_arguments(lib):
    need = lib.sf_state_workspace(8, 4)      # used here, because out and the indices are one
    copy = lambda p, src=FAKE, dst=FAKE, M=4: lib.sf_state_copy(p, src, dst, M, None)   # noqa: E731
    fork = lambda p, idx=FAKE, N=4, par=FAKE, M=4, res=None, out=FAKE, ws=FAKE, n=need: lib.sf_state_fork(   # noqa: E731
        p, idx, N, par, M, res, out, ws, n, None)
    comp = lambda p, idx=FAKE, N=4, res=None, out=FAKE, ws=FAKE, n=need: lib.sf_state_compact(   # noqa: E731
        p, idx, N, res, out, ws, n, None)
    for p, status in ((None, 1), (_pool(slots=0), 1), (_pool(sizes=(24,)), 1), (_pool(at=[0]), 1),
                      (_pool(at=[(1 << 20) + 8]), 1), (_pool(slots=(1 << 18) + 1), 2), (_pool(sizes=(1 << 39,)), 2)):
        assert copy(p) == status and fork(p) == status and comp(p) == status
    p = _pool()
    assert copy(p, src=None) == 1 and copy(p, dst=BYTE) == 1 and copy(p, M=-1) == 1 and copy(p, M=0) == 0
    assert fork(p, idx=None) == 1 and fork(p, par=None) == 1 and fork(p, out=None) == 1 and fork(p, N=-1) == 1
    assert fork(p, M=-1) == 1 and fork(p, par=BYTE) == 1 and fork(p, M=0) == 0
    assert fork(p, ws=None) == 3 and fork(p, ws=ODD) == 3 and fork(p, n=need - 1) == 3
    assert comp(p, idx=None) == 1 and comp(p, out=BYTE) == 1 and comp(p, N=-1) == 1 and comp(p, N=0) == 0
    assert comp(p, ws=None) == 3 and comp(p, ws=ODD) == 3 and comp(p, n=need - 1) == 3


def test_binding_checks_shapes_types_and_strides():
    import chunked_linear_recurrence_gb300 as sf
    z = torch.zeros
    N, T, P, H, HK, D = 3, 4, 2, 2, 1, 64
    a = dict(q=z(N, T, HK, D), k=z(N, T, HK, D), v=z(N, T, H, D), gate=z(N, T, H), beta=z(N, T, H),
             state_cache=z(5, H, D, D))
    with pytest.raises(ValueError, match="CUDA device"):
        sf.sf_gdn_draft_step(**a)
    # the checks that follow come after the device's, so the tensors claim to be on one
    with pytest.MonkeyPatch().context() as mp:
        mp.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
        pend = (z(N, P, HK, D), z(N, P, H, D), z(N, P, H), z(N, P, H))
        for kw, msg in ((dict(q=z(N, HK, D)), "must be"), (dict(k=z(N, T, H, D)), "k must be"),
                        (dict(v=z(N, T + 1, H, D)), "does not match"), (dict(v=z(N, T, H, D).bfloat16()), "v must be"),
                        (dict(gate=None), "gate is needed"), (dict(beta=z(N, T)), "beta must be"),
                        (dict(state_cache=z(5, H, D)), "must be"), (dict(state_cache=z(5, H + 1, D, D)), "state_cache"),
                        (dict(state_indices=z(N)), "state_indices must be"),
                        (dict(num_tokens=z(N + 1, dtype=torch.int32)), "num_tokens must be"),
                        (dict(num_pending=z(N, dtype=torch.int32)), "needs pending"),
                        (dict(pending=pend[:2]), "must be \\(k, v, gate, beta\\)"),
                        (dict(pending=(pend[0][0],) + pend[1:]), "pending k must be"),
                        (dict(pending=(pend[0].bfloat16(),) + pend[1:]), "pending k must be"),
                        (dict(pending=(pend[0], pend[1][:, :1], *pend[2:])), "pending v must be"),
                        (dict(pending=pend[:3] + (z(N, T, H),)), "pending beta must be"),
                        (dict(pending=pend, num_pending=z(N)), "num_pending must be"),
                        (dict(out=z(N, T, H, D).bfloat16()), "out must be"),
                        (dict(q=z(N, D, HK, T).permute(0, 3, 2, 1)), "contiguous"),
                        (dict(q=z(N, T, 0, D), k=z(N, T, 0, D)), "at least one head")):
            with pytest.raises(ValueError, match=msg):
                sf.sf_gdn_draft_step(**{**a, **kw})
        lin = {m: t for m, t in a.items() if m not in ("gate", "beta")}
        for kw, msg in ((dict(decay=None), "decay is needed"), (dict(decay=z(H + 1)), "decay must be"),
                        (dict(decay=z(H), pending=pend), "must be \\(k, v\\)")):
            with pytest.raises(ValueError, match=msg):
                sf.sf_linattn_draft_step(**lin, **kw)
        with pytest.raises(ValueError, match="v must be"):
            sf.sf_gdn_commit(a["k"], a["v"].bfloat16(), a["gate"], a["beta"], a["state_cache"])
        with pytest.raises(ValueError, match="decay must be"):
            sf.sf_linattn_commit(a["k"], a["v"], z(1), a["state_cache"])

        V = 10
        b = dict(target_probs=z(N, T + 1, V), draft_tokens=z(N, T, dtype=torch.int32), uniforms=z(N, T + 1))
        for kw, msg in ((dict(target_probs=z(N, V)), "target_probs must be"),
                        (dict(target_probs=z(N, V, T + 1).transpose(1, 2)), "rows must be contiguous"),
                        (dict(target_probs=z(N, T + 1, V).half()), "dtype"),
                        (dict(draft_tokens=z(N, T).long()), "draft_tokens must be"),
                        (dict(uniforms=z(N, T)), "uniforms must be"), (dict(draft_probs=z(N, T + 1, V)), "draft_probs"),
                        (dict(draft_probs=z(N, T, V).bfloat16()), "draft_probs must be"),
                        (dict(num_drafts=z(N)), "num_drafts must be"), (dict(tokens=z(N, T + 1)), "tokens must be")):
            with pytest.raises(ValueError, match=msg):
                sf.sf_draft_verify(**{**b, **kw})

        i = z(N, dtype=torch.int32)
        for call, msg in ((lambda: sf.sf_state_copy([], i, i), "at least one cache"),
                          (lambda: sf.sf_state_copy([z(4, 8), z(5, 8)], i, i), "one num_slots"),
                          (lambda: sf.sf_state_copy(z(4, 8).T, i, i), "contiguous"),
                          (lambda: sf.sf_state_copy(z(4, 8), i.long(), i), "src must be"),
                          (lambda: sf.sf_state_copy(z(4, 8), i, i[:1]), "dst must be"),
                          (lambda: sf.sf_state_fork(z(4, 8), i, i[None]), "parents must be"),
                          (lambda: sf.sf_state_fork(z(4, 8), i, i, reserved=z(3, dtype=torch.bool)), "reserved must be"),
                          (lambda: sf.sf_state_compact(z(4, 8), i, out=z(4, dtype=torch.int32)), "out must be"),
                          (lambda: sf.sf_state_compact(z(4, 8), i, ws=i), "ws must be")):
            with pytest.raises(ValueError, match=msg):
                call()
