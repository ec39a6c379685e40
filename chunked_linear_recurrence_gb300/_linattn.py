"""ctypes binding of include/sf_linattn.h: linear attention with a decay for each head, the
single-token steps on the paged state pool, and the norm of query and key heads with the
position rotation.

Argument marshalling only, as ``_native``: every step of the computation runs in the CUDA
library, and a call that the library cannot take raises.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._native import _check, _dtype_code, load, on_its_stream, sf_gdn_shape, sf_qk_shape

_NORMS = {"rms": 0, "l2": 1}
_F32 = torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _at(name, t):
    """Device address of a contiguous tensor."""
    if t is None:
        raise ValueError(f"{name} is needed")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    return t.data_ptr()


def _addr(name, t, shape, dtype):
    """Device address of a contiguous tensor of this shape and type (None for None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    return t.data_ptr()


def _need(name, t):
    if t is None:
        raise ValueError(f"{name} is needed")
    return t


def _tokens(q, k, v, decay, cu_seqlens):
    """Shape checks of a token stream: (B, T, H, HK, D, N)."""
    qs, vs, dt = q.shape, v.shape, q.dtype
    if len(qs) != 4 or len(vs) != 4:
        raise ValueError("q/k and v must be 4-D: [B,T,HK,K] and [B,T,H,V]")
    B, T, HK, K = qs
    H = vs[2]
    if vs[0] != B or vs[1] != T:
        raise ValueError(f"v {tuple(vs)} does not match q {tuple(qs)} in [B,T]")
    if k is not None and k.shape != qs:
        raise ValueError(f"k {tuple(k.shape)} must match q {tuple(qs)} in shape and dtype")
    if v.dtype != dt or (k is not None and k.dtype != dt):
        raise ValueError("q, k and v must share one dtype")
    if HK < 1:          # (to the library 0 means H, and it would read that many)
        raise ValueError("q and k need at least one head")
    if decay is not None and decay.shape != (H,):
        raise ValueError(f"decay must be [H] = {(H,)}, got {tuple(decay.shape)}")
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.dtype != torch.int32:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor")
        N = cu_seqlens.numel() - 1
    return B, T, H, HK, K, N


@functools.lru_cache(maxsize=256)
def _shape_of(B, T, H, K, V, N, dtype, scale, HK):
    """The shape struct of these sizes (the library only reads it), and a reference to it."""
    s = sf_gdn_shape(B, T, H, K, V, N, _dtype_code(dtype), float(scale) if scale is not None else 0.0,
                     HK)
    return s, ctypes.byref(s)


def _shape(q, v, cu_seqlens, scale, dims=None):
    B, T, H, HK, K, N = dims or _tokens(q, None, v, None, cu_seqlens)
    return _shape_of(B, T, H, K, v.shape[3], N, q.dtype, scale, HK)[1]


def _ws(ws):
    if not ws.is_cuda or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on a CUDA device")
    return ws


def workspace(nbytes, device):
    """A buffer whose status word is clear; the kernels write what else they read.  Up to 16 MB are
    cleared whole, in one call (10.4 us against 13.7 for an empty buffer and its first bytes); of
    more, which may be gigabytes, only the status word (64 MB 20.4 us, 256 MB 69.7)."""
    nbytes = max(int(nbytes), 256)
    if nbytes <= 1 << 24:
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def sf_linattn_fwd_workspace(q, v, cu_seqlens=None):
    """A workspace for sf_linattn_chunk_fwd and sf_linattn_paged_chunk_fwd on these shapes, to
    be kept and passed as ``ws`` (a call without one allocates its own)."""
    shape = _shape(q, v, cu_seqlens, None)
    need = load().sf_linattn_fwd_workspace(shape, int(cu_seqlens is not None))
    return workspace(need, q.device)


def sf_linattn_bwd_workspace(q, v, cu_seqlens=None):
    """The same for sf_linattn_chunk_bwd."""
    shape = _shape(q, v, cu_seqlens, None)
    need = load().sf_linattn_bwd_workspace(shape, int(cu_seqlens is not None))
    return workspace(need, q.device)


@on_its_stream
def sf_linattn_chunk_fwd(q, k, v, decay, initial_state=None, cu_seqlens=None, scale=None,
                         output_final_state=False, out=None, final_state=None, ws=None,
                         stream=None):
    """Linear attention with a decay for each head: S_t = exp(decay) S_{t-1} + v_t k_t^T,
    out_t = scale S_t q_t.  q, k [B,T,HK,K]; v [B,T,H,V]; decay [H] FP32 (natural log).
    Returns (out [B,T,H,V], final_state [N,H,V,K] or None)."""
    lib = load()
    dims = _tokens(q, k, v, decay, cu_seqlens)
    B, T, H, HK, K, N = dims
    shape = _shape(q, v, cu_seqlens, scale, dims)
    dt, st = q.dtype, (N, H, v.shape[3], K)
    args = (_at("q", q), _at("k", k), _at("v", v),
            _addr("decay", decay, (H,), _F32), _addr("initial_state", initial_state, st, _F32),
            _addr("cu_seqlens", cu_seqlens, (N + 1,), torch.int32))
    if out is None:
        out = torch.empty_like(v)
    else:
        _addr("out", out, v.shape, dt)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty(st, dtype=_F32, device=q.device)
    else:
        _addr("final_state", final_state, st, _F32)
    if ws is None:
        ws = workspace(lib.sf_linattn_fwd_workspace(shape, int(cu_seqlens is not None)),
                       q.device)
    ws = _ws(ws)
    _check(lib.sf_linattn_chunk_fwd(
        shape, *args, int(bool(output_final_state)), out.data_ptr(),
        None if final_state is None else final_state.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(stream, q.device)))
    return out, final_state


@on_its_stream
def sf_linattn_paged_chunk_fwd(q, k, v, decay, state_cache, state_indices, cu_seqlens=None,
                               has_initial_state=None, scale=None, out=None, ws=None, stream=None):
    """sf_linattn_chunk_fwd advancing state_cache [num_slots,H,V,K] in place at the slots
    state_indices (int32 [N]; <= 0: padding, zero output); has_initial_state (bool [N])
    False starts from zero.  Returns out [B,T,H,V]."""
    lib = load()
    dims = _tokens(q, k, v, decay, cu_seqlens)
    B, T, H, HK, K, N = dims
    shape = _shape(q, v, cu_seqlens, scale, dims)
    dt = q.dtype
    if state_cache.dim() != 4:
        raise ValueError("state_cache must be [num_slots,H,V,K]")
    slots = state_cache.shape[0]
    args = (_at("q", q), _at("k", k), _at("v", v),
            _addr("decay", decay, (H,), _F32),
            _addr("state_cache", state_cache, (slots, H, v.shape[3], K), _F32), slots,
            _addr("state_indices", state_indices, (N,), torch.int32),
            _addr("has_initial_state", has_initial_state, (N,), torch.bool),
            _addr("cu_seqlens", cu_seqlens, (N + 1,), torch.int32))
    if out is None:
        out = torch.empty_like(v)
    if ws is None:
        ws = workspace(lib.sf_linattn_fwd_workspace(shape, int(cu_seqlens is not None)),
                       q.device)
    ws = _ws(ws)
    _check(lib.sf_linattn_paged_chunk_fwd(shape, *args, _addr("out", out, v.shape, dt),
                                          ws.data_ptr(), ws.numel(), _stream(stream, q.device)))
    return out


@on_its_stream
def sf_linattn_chunk_bwd(q, k, v, decay, initial_state, d_out, d_final_state=None, cu_seqlens=None,
                         scale=None, want_d_initial_state=True, grads=None, ws=None, stream=None):
    """Backward of sf_linattn_chunk_fwd.  Returns dict dq, dk, dv, d_initial_state (the decay
    is a fixed property of the head and has no gradient)."""
    lib = load()
    dims = _tokens(q, k, v, decay, cu_seqlens)
    B, T, H, HK, K, N = dims
    shape = _shape(q, v, cu_seqlens, scale, dims)
    dt, st = q.dtype, (N, H, v.shape[3], K)
    args = (_at("q", q), _at("k", k), _at("v", v),
            _addr("decay", decay, (H,), _F32), _addr("initial_state", initial_state, st, _F32),
            _addr("cu_seqlens", cu_seqlens, (N + 1,), torch.int32),
            _addr("d_out", _need("d_out", d_out), v.shape, dt),
            _addr("d_final_state", d_final_state, st, _F32))
    if grads is None:
        grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                     d_initial_state=(torch.empty(st, dtype=_F32, device=q.device)
                                      if want_d_initial_state else None))
    if ws is None:
        ws = workspace(lib.sf_linattn_bwd_workspace(shape, int(cu_seqlens is not None)),
                       q.device)
    ws = _ws(ws)
    _check(lib.sf_linattn_chunk_bwd(
        shape, *args, _addr("dq", grads["dq"], q.shape, dt),
        _addr("dk", grads["dk"], q.shape, dt), _addr("dv", grads["dv"], v.shape, dt),
        _addr("d_initial_state", grads.get("d_initial_state"), st, _F32), ws.data_ptr(), ws.numel(),
        _stream(stream, q.device)))
    return grads


def _step_args(q, k, v, state_cache, state_indices, scale, out):
    qs, vs, cs, dt = q.shape, v.shape, state_cache.shape, q.dtype
    if len(qs) != 3 or len(vs) != 3 or len(cs) != 4:
        raise ValueError("q/k must be [N,HK,K], v [N,H,V] and state_cache [num_slots,H,V,K]")
    N, HK, K = qs
    _, H, V = vs
    if HK < 1:
        raise ValueError("q and k need at least one head")
    slots = cs[0]
    shape = _shape_of(1, 1, H, K, V, N, dt, scale, HK)[1]
    head = (_at("q", q), _addr("k", k, qs, dt), _addr("v", v, (N, H, V), dt))
    if out is None:
        out = torch.empty_like(v)
        to = out.data_ptr()
    else:
        to = _addr("out", out, (N, H, V), dt)
    tail = (_addr("state_cache", state_cache, (slots, H, V, K), _F32), slots,
            None if state_indices is None else _addr("state_indices", state_indices, (N,), torch.int32),
            to)
    return shape, N, H, head, tail, out


@on_its_stream
def sf_linattn_step(q, k, v, decay, state_cache, state_indices=None, scale=None, out=None,
                    stream=None):
    """One token of every sequence: q, k [N,HK,K], v [N,H,V], decay [H]; advances state_cache
    [num_slots,H,V,K] in place at the slots state_indices (int32 [N]; <= 0: padding, zero
    output; None: sequence n owns slot n).  Returns out [N,H,V]."""
    shape, N, H, head, tail, out = _step_args(q, k, v, state_cache, state_indices, scale, out)
    _check(load().sf_linattn_step(shape, *head, _addr("decay", decay, (H,), _F32),
                                  *tail, _stream(stream, q.device)))
    return out


@on_its_stream
def sf_gdn_step(q, k, v, gate, beta, state_cache, state_indices=None, scale=None, out=None,
                stream=None):
    """sf_linattn_step for the gated delta rule: gate, beta [N,H] FP32."""
    shape, N, H, head, tail, out = _step_args(q, k, v, state_cache, state_indices, scale, out)
    _check(load().sf_gdn_step(shape, *head, _addr("gate", gate, (N, H), _F32),
                              _addr("beta", beta, (N, H), _F32), *tail, _stream(stream, q.device)))
    return out


def _token_stride(name, t):
    """Elements between consecutive tokens of [B,T,heads,D]: a token's heads are contiguous,
    and the batch rows follow one another at the same stride."""
    B, T, h, D = t.shape
    if t.is_contiguous():
        return h * D
    sb, st, sh, sd = t.stride()
    if t.numel() == 0:
        return h * D
    if (sd != 1 and D > 1) or (sh != D and h > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if T == 1:
        st = sb if B > 1 else h * D
    elif B > 1 and sb != T * st:
        raise ValueError(f"{name}: batch rows must follow one another at one token stride")
    return st


@functools.lru_cache(maxsize=256)
def _qk_shape_of(rows, H, HK, D, dtype, norm, eps, interleaved, q_stride, k_stride, half, P, sections):
    """The shape struct of these sizes (the library only reads it), and a reference to it."""
    if len(sections) > 4:
        raise ValueError("at most 4 position axes")
    s = sf_qk_shape(rows, H, HK, D, _dtype_code(dtype), _NORMS[norm], eps, 2 * half,
                    int(bool(interleaved)), P, len(sections), (ctypes.c_int * 4)(*sections),
                    q_stride, k_stride)
    return s, ctypes.byref(s)


def _qk_shape(q, k, q_weight, k_weight, cos_sin, positions, sections, norm, eps, interleaved):
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4 or qs[0] != ks[0] or qs[1] != ks[1] or qs[3] != ks[3]:
        raise ValueError("q must be [B,T,H,D] and k [B,T,HK,D]")
    if q.dtype != k.dtype:
        raise ValueError("q and k must share one dtype")
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}, got {norm!r}")
    if not q.is_cuda or not k.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    B, T, H, D = qs
    HK = ks[2]
    table = at = None
    P = half = 0
    if cos_sin is None:
        sections = ()
    else:
        if cos_sin.dim() != 3 or cos_sin.shape[2] != 2:
            raise ValueError("cos_sin must be [table_rows, rotary_dim / 2, 2] FP32")
        P, half, _ = cos_sin.shape
        sections = (half,) if sections is None else tuple(map(int, sections))
        shape = _need("positions", positions).shape
        if len(sections) != 1 or (shape != (B * T,) and shape != (B, T)):
            shape = (len(sections), B * T)
        table = _addr("cos_sin", cos_sin, (P, half, 2), _F32)
        at = _addr("positions", positions, shape, torch.int32)
    s = _qk_shape_of(B * T, H, HK, D, q.dtype, norm, float(eps), interleaved,
                     H * D if q.is_contiguous() else _token_stride("q", q),
                     HK * D if k.is_contiguous() else _token_stride("k", k), half, P, sections)[1]
    return s, (q.data_ptr(), k.data_ptr(), _addr("q_weight", q_weight, (D,), _F32),
               _addr("k_weight", k_weight, (D,), _F32), table, at)


@on_its_stream
def sf_qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, cos_sin=None, positions=None,
                        sections=None, norm="rms", eps=1e-6, interleaved=False, q_out=None,
                        k_out=None, stream=None):
    """Norm of each head of q [B,T,H,D] and k [B,T,HK,D] ("rms" or "l2", times the weights
    [D]), then the rotation of its pairs by the angles cos_sin [table_rows, rotary_dim/2, 2] at
    ``positions`` (int32 [axes, B*T]; [B,T] or [B*T] for one axis), ``sections`` pairs to an
    axis.  q and k may be slices of one fused projection.  Returns (q_out, k_out)."""
    s, args = _qk_shape(q, k, q_weight, k_weight, cos_sin, positions, sections, norm, eps, interleaved)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _addr("q_out", q_out, q.shape, q.dtype)
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    else:
        _addr("k_out", k_out, k.shape, k.dtype)
    _check(load().sf_qk_norm_rope_fwd(s, *args, q_out.data_ptr(), k_out.data_ptr(),
                                      _stream(stream, q.device)))
    return q_out, k_out


def sf_qk_norm_rope_bwd_workspace(q, k):
    """A workspace for sf_qk_norm_rope_bwd on these shapes, to be kept and passed as ``ws``."""
    s = sf_qk_shape(0, q.shape[2], k.shape[2], q.shape[3])
    need = load().sf_qk_norm_rope_bwd_workspace(ctypes.byref(s))
    return torch.empty(need, dtype=torch.uint8, device=q.device)


@on_its_stream
def sf_qk_norm_rope_bwd(q, k, q_weight, k_weight, cos_sin, positions, d_q_out, d_k_out,
                        sections=None, norm="rms", eps=1e-6, interleaved=False,
                        want_weight_grads=True, grads=None, ws=None, stream=None):
    """Backward of sf_qk_norm_rope_fwd from its inputs and the cotangents of its outputs.
    Returns dict dq, dk (contiguous), dq_weight, dk_weight [D] FP32 (None if not wanted)."""
    s, args = _qk_shape(q, k, q_weight, k_weight, cos_sin, positions, sections, norm, eps, interleaved)
    lib, D, dev = load(), q.shape[3], q.device
    if grads is None:
        grads = dict(dq=torch.empty_like(q, memory_format=torch.contiguous_format),
                     dk=torch.empty_like(k, memory_format=torch.contiguous_format),
                     dq_weight=torch.empty(D, dtype=_F32, device=dev) if want_weight_grads else None,
                     dk_weight=torch.empty(D, dtype=_F32, device=dev) if want_weight_grads else None)
    dqw, dkw = grads.get("dq_weight"), grads.get("dk_weight")
    if ws is None and (dqw is not None or dkw is not None):
        ws = torch.empty(lib.sf_qk_norm_rope_bwd_workspace(s), dtype=torch.uint8, device=dev)
    ws = _ws(ws) if ws is not None else None
    _check(lib.sf_qk_norm_rope_bwd(
        s, *args, _addr("d_q_out", d_q_out, q.shape, q.dtype),
        _addr("d_k_out", d_k_out, k.shape, k.dtype), _addr("dq", grads["dq"], q.shape, q.dtype),
        _addr("dk", grads["dk"], k.shape, k.dtype), _addr("dq_weight", dqw, (D,), _F32),
        _addr("dk_weight", dkw, (D,), _F32), None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel(), _stream(stream, dev)))
    return grads
