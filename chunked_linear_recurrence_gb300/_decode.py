"""ctypes binding of include/sf_decode.h: drafted tokens on the paged state pool, their commit and
verification, and the pool's copies, forks and compaction.

Argument marshalling only, as ``_native``: every step of the computation runs in the CUDA
library, and a call that the library cannot take raises.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._linattn import _F32, _addr, _at, _need, _shape_of, _stream, _ws
from ._native import (_check, _dtype_code, load, on_its_stream, sf_pending, sf_state_pool,
                      sf_verify_shape)

_I32 = torch.int32


def _tokens(k, v, state_cache, what="k"):
    """(N, T, H, HK, K, V) of tokens k [N,T,HK,K] and v [N,T,H,V] on a pool [num_slots,H,V,K]."""
    ks, vs, cs = k.shape, v.shape, state_cache.shape
    if len(ks) != 4 or len(vs) != 4 or len(cs) != 4:
        raise ValueError(f"{what} must be [N,T,HK,K], v [N,T,H,V] and state_cache [num_slots,H,V,K]")
    N, T, HK, K = ks
    if vs[0] != N or vs[1] != T:
        raise ValueError(f"v {tuple(vs)} does not match {what} {tuple(ks)} in [N,T]")
    if HK < 1:          # (to the library 0 means H, and it would read that many)
        raise ValueError("q and k need at least one head")
    return N, T, vs[2], HK, K, vs[3]


@functools.lru_cache(maxsize=256)
def _draft_shape(N, T, H, HK, K, V, dtype, scale):
    return _shape_of(1, T, H, K, V, N, dtype, scale, HK)


def _pool(state_cache, state_indices, N, H, V, K):
    slots = state_cache.shape[0]
    return (_addr("state_cache", state_cache, (slots, H, V, K), _F32), slots,
            _addr("state_indices", state_indices, (N,), _I32))


def _draft(q, k, v, gate, beta, delta, state_cache, state_indices, num_tokens, pending, num_pending, scale,
           out):
    """Checks and addresses of a draft step: (shape, tokens, gates, num_tokens, pending, the rest), out."""
    N, T, H, HK, K, V = _tokens(q, v, state_cache, "q")
    dt = q.dtype
    vs = (N, T, H, V)
    tokens = (_at("q", q), _addr("k", k, q.shape, dt), _addr("v", v, vs, dt))
    gates = ()
    if delta:
        gates = (_addr("gate", _need("gate", gate), (N, T, H), _F32),
                 _addr("beta", _need("beta", beta), (N, T, H), _F32))
    num = _addr("num_tokens", num_tokens, (N,), _I32)
    pend = None
    if pending is not None:
        if len(pending) != (4 if delta else 2):
            raise ValueError("pending must be (k, v, gate, beta)" if delta else "pending must be (k, v)")
        pk = pending[0]
        if pk.dim() != 4:
            raise ValueError("pending k must be [N,P,HK,K]")
        P = pk.shape[1]
        pg = pb = None
        if delta:
            pg = _addr("pending gate", _need("pending gate", pending[2]), (N, P, H), _F32)
            pb = _addr("pending beta", _need("pending beta", pending[3]), (N, P, H), _F32)
        pend = sf_pending(P, _addr("pending k", pk, (N, P, HK, K), dt),
                          _addr("pending v", pending[1], (N, P, H, V), dt), pg, pb,
                          _addr("num_pending", num_pending, (N,), _I32))
    elif num_pending is not None:
        raise ValueError("num_pending needs pending tokens")
    pool = _pool(state_cache, state_indices, N, H, V, K)
    if out is None:
        out = torch.empty_like(v)
        to = out.data_ptr()
    else:
        to = _addr("out", out, vs, dt)
    return (_draft_shape(N, T, H, HK, K, V, dt, scale)[1], tokens, gates, num, pend, (*pool, to)), out


@on_its_stream
def sf_gdn_draft_step(q, k, v, gate, beta, state_cache, state_indices=None, num_tokens=None,
                      pending=None, num_pending=None, scale=None, out=None, stream=None):
    """Outputs of up to 32 drafted tokens of every sequence by the gated delta rule: q, k
    [N,T,HK,K], v [N,T,H,V], gate, beta [N,T,H] FP32, of which the first num_tokens (int32 [N];
    None: all) count.  state_cache [num_slots,H,V,K] is first advanced, at the slots
    state_indices (as sf_gdn_step), by the first num_pending (int32 [N]; None: all) of the
    ``pending`` tokens (k [N,P,HK,K], v [N,P,H,V], gate, beta [N,P,H]); the drafts leave it as
    it then is.  Returns out [N,T,H,V], zero behind num_tokens and in padding."""
    (shape, tokens, gates, num, pend, rest), out = _draft(
        q, k, v, gate, beta, True, state_cache, state_indices, num_tokens, pending, num_pending, scale, out)
    _check(load().sf_gdn_draft_step(shape, *tokens, *gates, num, pend, *rest, _stream(stream, q.device)))
    return out


@on_its_stream
def sf_linattn_draft_step(q, k, v, decay, state_cache, state_indices=None, num_tokens=None,
                          pending=None, num_pending=None, scale=None, out=None, stream=None):
    """sf_gdn_draft_step for linear attention: decay [H]; pending (k, v)."""
    (shape, tokens, _, num, pend, rest), out = _draft(
        q, k, v, None, None, False, state_cache, state_indices, num_tokens, pending, num_pending, scale, out)
    decay = _addr("decay", _need("decay", decay), (v.shape[2],), _F32)
    _check(load().sf_linattn_draft_step(shape, *tokens, decay, num, pend, *rest, _stream(stream, q.device)))
    return out


@on_its_stream
def sf_gdn_commit(k, v, gate, beta, state_cache, state_indices=None, num_tokens=None, stream=None):
    """Advances state_cache in place by the first num_tokens (int32 [N]; None: all) of up to 32
    tokens of every sequence: k [N,T,HK,K], v [N,T,H,V], gate, beta [N,T,H] FP32."""
    N, T, H, HK, K, V = _tokens(k, v, state_cache)
    shape = _draft_shape(N, T, H, HK, K, V, k.dtype, None)[1]
    _check(load().sf_gdn_commit(shape, _at("k", k), _addr("v", v, (N, T, H, V), k.dtype),
                                _addr("gate", _need("gate", gate), (N, T, H), _F32),
                                _addr("beta", _need("beta", beta), (N, T, H), _F32),
                                _addr("num_tokens", num_tokens, (N,), _I32),
                                *_pool(state_cache, state_indices, N, H, V, K),
                                _stream(stream, k.device)))


@on_its_stream
def sf_linattn_commit(k, v, decay, state_cache, state_indices=None, num_tokens=None, stream=None):
    """sf_gdn_commit for linear attention: decay [H]."""
    N, T, H, HK, K, V = _tokens(k, v, state_cache)
    shape = _draft_shape(N, T, H, HK, K, V, k.dtype, None)[1]
    _check(load().sf_linattn_commit(shape, _at("k", k), _addr("v", v, (N, T, H, V), k.dtype),
                                    _addr("decay", _need("decay", decay), (H,), _F32),
                                    _addr("num_tokens", num_tokens, (N,), _I32),
                                    *_pool(state_cache, state_indices, N, H, V, K),
                                    _stream(stream, k.device)))


@functools.lru_cache(maxsize=256)
def _verify_shape(N, T, V, dtype, strides):
    s = sf_verify_shape(N, T, V, _dtype_code(dtype), *strides)
    return s, ctypes.byref(s)


def _rows(name, t, shape, dtype):
    """Address and strides (of sequences and rows) of probabilities whose rows are contiguous."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    seq, row, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.data_ptr(), seq, row


@on_its_stream
def sf_draft_verify(target_probs, draft_tokens, uniforms, draft_probs=None, num_drafts=None,
                    tokens=None, num_tokens=None, stream=None):
    """Accepts drafted tokens and draws the one behind them: target_probs [N,T+1,V] (FP32 or
    BF16; rows contiguous), draft_tokens int32 [N,T], uniforms [N,T+1] FP32 in [0,1),
    draft_probs [N,T,V] (None: the draft is certain), num_drafts int32 [N] (None: T; negative:
    padding).  Returns (tokens int32 [N,T+1]: the accepted drafts, the drawn token, then -1;
    num_tokens int32 [N]: how many they are)."""
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise ValueError("target_probs must be [N,T+1,V]")
    N, T, V = target_probs.shape
    T -= 1
    dt = target_probs.dtype
    target, seq, row = _rows("target_probs", target_probs, (N, T + 1, V), dt)
    draft, dseq, drow = (None, 0, 0) if draft_probs is None else _rows("draft_probs", draft_probs, (N, T, V), dt)
    x = _addr("draft_tokens", _need("draft_tokens", draft_tokens), (N, T), _I32)
    u = _addr("uniforms", _need("uniforms", uniforms), (N, T + 1), _F32)
    num = _addr("num_drafts", num_drafts, (N,), _I32)
    shape = _verify_shape(N, T, V, dt, (seq, row, dseq, drow))[1]
    if tokens is None:
        tokens = torch.empty((N, T + 1), dtype=_I32, device=target_probs.device)
    if num_tokens is None:
        num_tokens = torch.empty((N,), dtype=_I32, device=target_probs.device)
    _check(load().sf_draft_verify(shape, target, x, u, draft, num,
                                  _addr("tokens", tokens, (N, T + 1), _I32),
                                  _addr("num_tokens", num_tokens, (N,), _I32),
                                  _stream(stream, target_probs.device)))
    return tokens, num_tokens


def _state_pool(caches):
    """The pool struct of one cache or several, [num_slots, ...] each, and their device."""
    if isinstance(caches, torch.Tensor):
        caches = (caches,)
    n = len(caches)
    if n == 0:
        raise ValueError("at least one cache is needed")
    first = caches[0]
    slots = first.shape[0] if first.dim() else 0
    at, size = [], []
    for c in caches:
        if c.dim() < 2 or c.shape[0] != slots or slots < 1:
            raise ValueError(f"caches must be [num_slots, ...] of one num_slots >= 1, got {tuple(c.shape)}")
        at.append(_at("caches", c))
        size.append(c.nbytes // slots)
    return sf_state_pool(slots, n, (ctypes.c_void_p * n)(*at), (ctypes.c_size_t * n)(*size)), first.device


@functools.lru_cache(maxsize=256)
def _workspace_bytes(slots, rows):
    return load().sf_state_workspace(slots, rows)


def sf_state_workspace(caches, rows):
    """A workspace for sf_state_fork (rows: the number of parents) and sf_state_compact (of
    indices) on a pool, to be kept and passed as ``ws``."""
    cache = caches if isinstance(caches, torch.Tensor) else caches[0]
    return torch.empty(_workspace_bytes(cache.shape[0], rows), dtype=torch.uint8, device=cache.device)


def _vector(name, t):
    if t is None or t.dim() != 1 or t.dtype != _I32:
        raise ValueError(f"{name} must be a 1-D int32 tensor")
    return _at(name, t), t.shape[0]


@on_its_stream
def sf_state_copy(caches, src, dst, stream=None):
    """Copies the slots src[i] of a pool into its slots dst[i] (int32 [M]; a pair with an index
    outside [1, num_slots) is skipped).  The dst are distinct and none is also a src.
    ``caches``: one cache [num_slots, ...] or several (of the layers of a model)."""
    pool, device = _state_pool(caches)
    s, M = _vector("src", src)
    _check(load().sf_state_copy(ctypes.byref(pool), s, _addr("dst", _need("dst", dst), (M,), _I32), M,
                                _stream(stream, device)))


def _plan_args(pool, device, reserved, rows, out, ws, inputs):
    """``inputs``: (address, bytes) of the indices."""
    slots = pool.num_slots
    reserved = _addr("reserved", reserved, (slots,), torch.bool)
    if out is None:
        out = torch.empty(rows, dtype=_I32, device=device)
        to, inputs = out.data_ptr(), ()
    else:
        to = _addr("out", out, (rows,), _I32)
    if (ws is None and slots <= 4096 and rows <= 256 and pool.num_caches <= 64
            and not any(to < at + n and at < to + rows * 4 for at, n in inputs)):
        return out, None, (reserved, to, None, 0)            # (none is used)
    if ws is None:
        ws = torch.empty(_workspace_bytes(slots, rows), dtype=torch.uint8, device=device)
    else:
        _ws(ws)
    return out, ws, (reserved, to, ws.data_ptr(), ws.numel())


@on_its_stream
def sf_state_fork(caches, state_indices, parents, reserved=None, out=None, ws=None, stream=None):
    """Continues sequence parents[i] (int32 [M]) of state_indices (int32 [N]) as row i: the first
    row of a slot keeps it, the others get copies in the lowest slots that no row keeps; a slot
    that is ``reserved`` (bool [num_slots]) is neither given out nor kept, so that its rows all
    get copies.  Returns the rows' slots, int32 [M] (-1: no such sequence, or no slot left)."""
    pool, device = _state_pool(caches)
    idx, N = _vector("state_indices", state_indices)
    par, M = _vector("parents", parents)
    out, ws, tail = _plan_args(pool, device, reserved, M, out, ws, ((idx, N * 4), (par, M * 4)))
    _check(load().sf_state_fork(ctypes.byref(pool), idx, N, par, M, *tail, _stream(stream, device)))
    return out


@on_its_stream
def sf_state_compact(caches, state_indices, reserved=None, out=None, ws=None, stream=None):
    """Brings the slots that state_indices (int32 [N]) names into the lowest ones of the pool, but
    for ``reserved`` slots (bool [num_slots]), which stay.  Returns where each is then, int32 [N]."""
    pool, device = _state_pool(caches)
    idx, N = _vector("state_indices", state_indices)
    out, ws, tail = _plan_args(pool, device, reserved, N, out, ws, ((idx, N * 4),))
    _check(load().sf_state_compact(ctypes.byref(pool), idx, N, *tail, _stream(stream, device)))
    return out
