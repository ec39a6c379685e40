"""FP64 CPU oracle of the decayed linear attention, of the single-token steps and of the norm
of query and key heads with the position rotation -- TEST INFRASTRUCTURE ONLY.

Token by token from the definitions, in NumPy; small cases only.  Shares no code with the
CUDA library.

    S_t = exp(decay_h) S_{t-1} + outer(v_t, k_t);   out_t = scale S_t q_t

Layouts as the library's: q, k [B,T,HK,K]; v [B,T,H,V]; decay [H]; states [N,H,V,K]; value
head h reads query/key head h // (H // HK).  Rows outside every sequence are NaN.
"""
from __future__ import annotations

import numpy as np


def _spans(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def _wide(x, H):
    x = np.asarray(x, np.float64)
    return np.repeat(x, H // x.shape[2], axis=2)


def fwd(q, k, v, decay, initial_state=None, cu_seqlens=None, scale=None):
    """(out [B,T,H,V], final states [N,H,V,K])."""
    v = np.asarray(v, np.float64)
    B, T, H, V = v.shape
    K = q.shape[-1]
    q, k = _wide(q, H), _wide(k, H)
    scale = K ** -0.5 if scale is None else scale
    lam = np.exp(np.asarray(decay, np.float64))[:, None, None]
    spans = _spans(B, T, cu_seqlens)
    out = np.full((B, T, H, V), np.nan)
    fin = np.zeros((len(spans), H, V, K))
    for n, (b, lo, hi) in enumerate(spans):
        S = np.zeros((H, V, K)) if initial_state is None else np.array(initial_state[n], np.float64)
        for t in range(lo, hi):
            S = lam * S + v[b, t][:, :, None] * k[b, t][:, None]
            out[b, t] = scale * np.einsum("hvk,hk->hv", S, q[b, t])
        fin[n] = S
    return out, fin


def bwd(q, k, v, decay, initial_state, d_out, d_final_state=None, cu_seqlens=None, scale=None):
    """Gradients of <d_out, out> + <d_final_state, final_state>: dict dq, dk, dv (NaN outside
    every sequence), d_initial_state."""
    v, d_out = np.asarray(v, np.float64), np.asarray(d_out, np.float64)
    B, T, H, V = v.shape
    HK, K = q.shape[2], q.shape[3]
    qw, kw = _wide(q, H), _wide(k, H)
    scale = K ** -0.5 if scale is None else scale
    lam = np.exp(np.asarray(decay, np.float64))[:, None, None]
    spans = _spans(B, T, cu_seqlens)
    dq, dk = np.full((B, T, H, K), np.nan), np.full((B, T, H, K), np.nan)
    dv = np.full((B, T, H, V), np.nan)
    d0 = np.zeros((len(spans), H, V, K))
    for n, (b, lo, hi) in enumerate(spans):
        S = np.zeros((H, V, K)) if initial_state is None else np.array(initial_state[n], np.float64)
        for t in range(lo, hi):
            S = lam * S + v[b, t][:, :, None] * kw[b, t][:, None]
            dq[b, t] = scale * np.einsum("hvk,hv->hk", S, d_out[b, t])
        G = np.zeros((H, V, K)) if d_final_state is None else np.array(d_final_state[n], np.float64)
        for t in range(hi - 1, lo - 1, -1):
            G = G + scale * d_out[b, t][:, :, None] * qw[b, t][:, None]
            dk[b, t] = np.einsum("hvk,hv->hk", G, v[b, t])
            dv[b, t] = np.einsum("hvk,hk->hv", G, kw[b, t])
            G = lam * G
        d0[n] = G
    group = lambda x: x.reshape(B, T, HK, H // HK, K).sum(3)   # noqa: E731
    return dict(dq=group(dq), dk=group(dk), dv=dv, d_initial_state=d0)


def step(q, k, v, cache, idx, decay=None, gate=None, beta=None, scale=None):
    """One token of every sequence on a pool of states: (out [N,H,V], the pool afterwards).
    decay [H]: linear attention; gate, beta [N,H]: the gated delta rule."""
    v = np.asarray(v, np.float64)
    N, H, V = v.shape
    K = q.shape[-1]
    scale = K ** -0.5 if scale is None else scale
    cache = np.array(cache, np.float64)
    out = np.zeros((N, H, V))
    for n in range(N):
        s = int(idx[n]) if idx is not None else n
        if (idx is not None and s <= 0) or s >= cache.shape[0]:
            continue
        for h in range(H):
            a = h // (H // q.shape[1])
            qn, kn = np.asarray(q[n, a], np.float64), np.asarray(k[n, a], np.float64)
            S = cache[s, h]
            if gate is None:
                S = np.exp(float(decay[h])) * S
                r = v[n, h]
            else:
                S = np.exp(float(gate[n, h])) * S
                r = float(beta[n, h]) * (v[n, h] - S @ kn)
            S = S + np.outer(r, kn)
            cache[s, h] = S
            out[n, h] = scale * (S @ qn)
    return out, cache


def _angles(cos_sin, positions, sections, rows):
    """cos, sin [rows, half]: each pair at the position of its axis, clamped into the table."""
    cos_sin = np.asarray(cos_sin, np.float64)
    P, half, _ = cos_sin.shape
    pos = np.clip(np.asarray(positions).reshape(-1, rows), 0, P - 1)
    axis = np.repeat(np.arange(len(sections)), sections)
    out = np.empty((rows, half, 2))
    for p in range(half):
        out[:, p] = cos_sin[pos[axis[p]], p]
    return out[..., 0][:, None], out[..., 1][:, None]


def _pairs(half, interleaved):
    p = np.arange(half)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + half)


def norm_rope(x, w, cos_sin, positions, sections, norm="rms", eps=1e-6, interleaved=False):
    """x [rows, heads, D] -> the normed and rotated heads."""
    x = np.asarray(x, np.float64)
    rows, _, D = x.shape
    ss = (x * x).sum(-1, keepdims=True)
    r = 1 / np.sqrt(ss / D + eps) if norm == "rms" else 1 / np.maximum(np.sqrt(ss), eps)
    y = x * r * (1.0 if w is None else np.asarray(w, np.float64))
    if cos_sin is None:
        return y
    c, s = _angles(cos_sin, positions, sections, rows)
    a, b = _pairs(c.shape[-1], interleaved)
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def norm_rope_bwd(x, w, cos_sin, positions, sections, d, norm="rms", eps=1e-6, interleaved=False):
    """(dx, dw) of norm_rope for the cotangent d."""
    x, d = np.asarray(x, np.float64), np.array(d, np.float64)
    rows, _, D = x.shape
    w = np.ones(D) if w is None else np.asarray(w, np.float64)
    dy = d
    if cos_sin is not None:
        c, s = _angles(cos_sin, positions, sections, rows)
        a, b = _pairs(c.shape[-1], interleaved)
        dy = d.copy()
        dy[..., a] = d[..., a] * c + d[..., b] * s
        dy[..., b] = d[..., b] * c - d[..., a] * s
    ss = (x * x).sum(-1, keepdims=True)
    g = dy * w
    gx = (g * x).sum(-1, keepdims=True)
    if norm == "rms":
        r = 1 / np.sqrt(ss / D + eps)
        dx = r * g - x * r ** 3 * gx / D
    else:
        nrm = np.sqrt(ss)
        r = 1 / np.maximum(nrm, eps)
        dx = r * g - np.where(nrm > eps, x * r ** 3 * gx, 0.0)
    return dx, (dy * x * r).sum((0, 1))
