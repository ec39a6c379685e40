"""Pins of the decoding oracle on facts that do not come from it."""
import numpy as np
import pytest

import oracle
from oracle import decode as od
from oracle import linattn as la


def tokens(N, T, H, HK, D, delta, seed, q=True):
    r = np.random.RandomState(seed)
    t = dict(k=r.randn(N, T, HK, D) / D ** 0.5, v=r.randn(N, T, H, D))
    if q:
        t["q"] = r.randn(N, T, HK, D)
    if delta:
        t["gate"], t["beta"] = -r.rand(N, T, H), r.rand(N, T, H)
    return t


def test_drafts_behind_pending_tokens_equal_one_sequence():
    """Pending and drafted tokens in a row are the sequence of both, by the other oracles."""
    N, H, HK, D, P, T = 2, 4, 2, 8, 3, 4
    r = np.random.RandomState(0)
    cache, idx, decay = r.randn(4, H, D, D), [3, 1], -r.rand(H)
    for delta in (False, True):
        new, pend = tokens(N, T, H, HK, D, delta, 1), tokens(N, P, H, HK, D, delta, 2)
        out, after = od.draft_step(new, None, pend, None, cache, idx, None if delta else decay)
        both = {m: np.concatenate([pend.get(m, np.zeros_like(new[m][:, :P][:, [0] * P])), new[m]], 1) for m in new}
        if delta:
            ref, _ = oracle.gdn_fwd(*(np.repeat(both[m], H // HK, 2) if m in "qk" else both[m]
                                      for m in ("q", "k", "v", "gate", "beta")), cache[idx])
            _, fin = oracle.gdn_fwd(*(np.repeat(x, H // HK, 2) if i < 2 else x for i, x in enumerate(
                (pend["k"], pend["k"], pend["v"], pend["gate"], pend["beta"]))), cache[idx])
        else:
            ref, _ = la.fwd(both["q"], both["k"], both["v"], decay, cache[idx])
            _, fin = la.fwd(pend["k"], pend["k"], pend["v"], decay, cache[idx])
        assert np.abs(out - ref[:, P:]).max() < 1e-10
        assert np.abs(after[idx] - fin).max() < 1e-10
        assert np.array_equal(after[[0, 2]], cache[[0, 2]])


def test_verified_tokens_have_the_targets_distribution():
    """Over a fine grid of the uniforms, the first token's frequencies are the target's
    probabilities, whatever the draft's are."""
    p, q = np.array([0.5, 0.0, 0.3, 0.2]), np.array([0.1, 0.4, 0.3, 0.2])
    m = 200
    for draft in (q, None):
        freq = np.zeros(4)
        for x in range(4):
            weight = q[x] if draft is not None else float(x == 2)
            if weight == 0:
                continue
            grid = (np.arange(m) + 0.5) / m
            u = np.stack(np.meshgrid(grid, grid, indexing="ij"), -1).reshape(-1, 2)
            n = len(u)
            tok, _ = od.verify(np.broadcast_to(np.stack([p, p]), (n, 2, 4)), np.full((n, 1), x), u,
                               None if draft is None else np.broadcast_to(q[None], (n, 1, 4)))
            freq += weight * np.bincount(tok[:, 0], minlength=4) / n
        assert np.abs(freq - p).max() < 2.0 / m


@pytest.mark.parametrize("seed", range(20))
def test_forked_and_compacted_rows_keep_their_states(seed):
    r = np.random.RandomState(seed)
    slots = r.randint(3, 40)
    reserved = {int(s) for s in r.choice(np.arange(1, slots), r.randint(0, 3), replace=True)} if seed % 2 else set()
    idx = r.randint(-1, slots + 1, r.randint(1, 30))
    state = np.arange(slots) * 10
    parents = r.randint(-1, len(idx) + 1, r.randint(1, 30))
    new, copies = od.fork(idx, parents, slots, reserved)
    after = state.copy()
    for to, s in copies.items():
        assert to not in reserved and to > 0
        after[to] = state[s]
    got = [s for s in new if s > 0]
    assert len(set(got)) == len(got) and not set(got) & reserved
    for i, p in enumerate(parents):
        s = idx[p] if 0 <= p < len(idx) else -1
        if 0 < s < slots:
            assert new[i] == -1 or after[new[i]] == state[s]
        else:
            assert new[i] == -1
    lost = [i for i, p in enumerate(parents) if new[i] < 0 and 0 <= p < len(idx) and 0 < idx[p] < slots]
    assert not lost or len(got) == slots - 1 - len(reserved)

    new, moves = od.compact(idx, slots, reserved)
    after = state.copy()
    for to, s in moves.items():
        after[to] = state[s]
    for n, s in enumerate(idx):
        assert new[n] == s if not 0 < s < slots or s in reserved else after[new[n]] == state[s]
    live = {s for s, o in zip(new, idx) if 0 < o < slots and o not in reserved}
    assert live == set([s for s in range(1, slots) if s not in reserved][:len(live)])
