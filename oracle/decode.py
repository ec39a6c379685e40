"""FP64 CPU oracle of decoding several tokens at a time (drafted tokens and commits on the pool of
states, verification of drafts, forks and compaction of the pool) -- TEST INFRASTRUCTURE ONLY.

From the definitions, in NumPy and plain Python; small cases only.  Shares no code with the CUDA
library.
"""
from __future__ import annotations

import numpy as np

from .linattn import step


def _count(num, n, most):
    return most if num is None else min(max(int(num[n]), 0), most)


def _slot(idx, n, slots):
    s = n if idx is None else int(idx[n])
    return s if (idx is None or s > 0) and s < slots else None


def advance(tok, num, cache, idx, decay=None, scale=None):
    """The first num[n] of the tokens (dict k, v and, for the delta rule, gate, beta; [N,T,...]; q
    or not) of every sequence, one after the other: (outputs [N,T,H,V], the pool afterwards)."""
    tok = {m: np.asarray(t, np.float64) for m, t in tok.items()}
    N, T, H, V = tok["v"].shape
    cache = np.array(cache, np.float64)
    out = np.zeros((N, T, H, V))
    for n in range(N):
        s = _slot(idx, n, cache.shape[0])
        if s is None:
            continue
        S = cache[s][None]
        for t in range(_count(num, n, T)):
            at = {m: x[n:n + 1, t] for m, x in tok.items()}
            at.setdefault("q", np.zeros_like(at["k"]))
            o, S = step(at["q"], at["k"], at["v"], S, None, decay=decay, gate=at.get("gate"), beta=at.get("beta"),
                        scale=scale)
            out[n, t] = o[0]
        cache[s] = S[0]
    return out, cache


def draft_step(tok, num, pend, num_pend, cache, idx, decay=None, scale=None):
    """(outputs of the drafts, the pool advanced by the pending tokens alone)."""
    if pend is not None:
        _, cache = advance(pend, num_pend, cache, idx, decay)
    return advance(tok, num, cache, idx, decay, scale)[0], np.array(cache, np.float64)


def verify(target, x, u, draft=None, num=None):
    """(tokens [N,T+1], num_tokens [N]) of target [N,T+1,V], x [N,T], u [N,T+1], draft [N,T,V]."""
    target, u = np.asarray(target, np.float64), np.asarray(u, np.float64)
    N, rows, V = target.shape
    T = rows - 1
    tokens, count = np.full((N, rows), -1, np.int64), np.zeros(N, np.int64)

    def positive(w):
        return np.where(w > 0, w, 0.0)          # a NaN is not

    for n in range(N):
        nd = T if num is None else min(int(num[n]), T)
        if nd < 0:
            continue
        a = 0
        while a < nd:
            y = int(x[n][a])
            if not 0 <= y < V:
                break
            if not u[n, a] * (1.0 if draft is None else float(draft[n][a][y])) < target[n, a, y]:
                break
            tokens[n, a] = y
            a += 1
        count[n] = a + 1
        w = positive(target[n, a])
        if a < nd:
            if draft is None:
                less = w.copy()
                if 0 <= int(x[n][a]) < V:
                    less[int(x[n][a])] = 0.0
            else:
                with np.errstate(invalid="ignore"):
                    less = positive(target[n, a] - np.asarray(draft[n][a], np.float64))
            if less.any():
                w = less
        total = w.sum()
        if not (total > 0 and np.isfinite(total)):
            continue
        over = (np.cumsum(w) > u[n, T] * total) & (w > 0)      # (u < 0: the first token with weight)
        tokens[n, a] = np.argmax(over) if over.any() else np.nonzero(w)[0][-1]
    return tokens, count


def fork(idx, parents, slots, reserved=()):
    """(new slots of the rows, {slot: the slot it is a copy of})."""
    reserved = set(reserved)
    src = []
    for p in parents:
        s = int(idx[p]) if 0 <= p < len(idx) else -1
        src.append(s if 0 < s < slots else -1)
    keeper = {}
    for i, s in enumerate(src):
        if s > 0 and s not in reserved:
            keeper.setdefault(s, i)
    free = [s for s in range(1, slots) if s not in keeper and s not in reserved]
    new, copies = [], {}
    for i, s in enumerate(src):
        if s < 0 or keeper.get(s) == i:
            new.append(s)
        elif free:
            to = free.pop(0)
            new.append(to)
            copies[to] = s
        else:
            new.append(-1)
    return new, copies


def compact(idx, slots, reserved=()):
    """(new slots of the rows, {slot: the slot that moved into it})."""
    reserved = set(reserved)
    live = sorted({int(s) for s in idx if 0 < s < slots} - reserved)
    low = [s for s in range(1, slots) if s not in reserved][:len(live)]
    to = dict(zip([s for s in live if s not in low], [s for s in low if s not in live]))
    return [to.get(int(s), int(s)) for s in idx], {b: a for a, b in to.items()}
