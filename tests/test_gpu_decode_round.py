"""The decoding operators together, as a server uses them: prompts prefilled into a pool, forked into
several continuations, rounds of drafted tokens (outputs from the states advanced by what the
round before accepted, verification, the next round), a beam dropped, the rest committed and
compacted.

Whatever was accepted, a sequence's state has to be the rule's over its tokens, from the state that
the prefill left: FP32 arithmetic, at most 4 rounds of 4 tokens, 16^0.5 x 4e-6 = 1.6e-5 of the
2-norm (the steps' own tolerance, test_gpu_draft_step).  The drafts' outputs have BF16's half step
beside it."""
import numpy as np
import pytest
import torch

from helpers import f64
from oracle import decode as od

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
V, H, HK, D, DRAFTS = 50, 4, 2, 128, 3


class Model:
    """One layer: a token's queries, keys, values and gates are rows of tables, its probabilities a
    softmax of the layer's output."""

    def __init__(self, delta, seed):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)   # noqa: E731
        self.delta = delta
        self.q, self.k = unit(rn(V, HK, D)).to(BF16).cuda(), unit(rn(V, HK, D)).to(BF16).cuda()
        self.v = rn(V, H, D).to(BF16).cuda()
        self.gate, self.beta = -torch.rand(V, H, generator=g).cuda(), torch.rand(V, H, generator=g).cuda()
        self.decay = -torch.rand(H, generator=g).cuda()
        self.head = (rn(H * D, V) * 2).cuda()

    def inputs(self, x):
        x = x.long().clamp_min(0)
        t = dict(q=self.q[x], k=self.k[x], v=self.v[x])
        if self.delta:
            t.update(gate=self.gate[x], beta=self.beta[x])
        return t

    def draft_step(self, t, pool, idx, pending, num_pending):
        import chunked_linear_recurrence_gb300 as sf
        pend = None
        if pending is not None:
            pend = tuple(pending[m] for m in (("k", "v", "gate", "beta") if self.delta else ("k", "v")))
        kw = dict(pending=pend, num_pending=num_pending)
        if self.delta:
            return sf.sf_gdn_draft_step(t["q"], t["k"], t["v"], t["gate"], t["beta"], pool, idx, **kw)
        return sf.sf_linattn_draft_step(t["q"], t["k"], t["v"], self.decay, pool, idx, **kw)

    def commit(self, t, pool, idx, num):
        import chunked_linear_recurrence_gb300 as sf
        if self.delta:
            sf.sf_gdn_commit(t["k"], t["v"], t["gate"], t["beta"], pool, idx, num_tokens=num)
        else:
            sf.sf_linattn_commit(t["k"], t["v"], self.decay, pool, idx, num_tokens=num)

    def prefill(self, x, pool, idx):
        import chunked_linear_recurrence_gb300 as sf
        t = self.inputs(x)
        fresh = torch.zeros(len(x), dtype=torch.bool, device="cuda")
        if self.delta:
            sf.sf_gdn_paged_chunk_fwd(t["q"], t["k"], t["v"], t["gate"], t["beta"], pool, idx, has_initial_state=fresh)
        else:
            sf.sf_linattn_paged_chunk_fwd(t["q"], t["k"], t["v"], self.decay, pool, idx, has_initial_state=fresh)

    def want(self, tokens, S):
        """(outputs [T,H,D], state) of the tokens of one sequence from the state S, in FP64."""
        t = {m: f64(x)[None] for m, x in self.inputs(torch.tensor(tokens, device="cuda")).items()}
        out, cache = od.advance(t, None, S[None], None, None if self.delta else f64(self.decay))
        return out[0], cache[0]


def err(x, ref):
    return np.linalg.norm(f64(x) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("delta", [False, True])
def test_rounds_of_drafted_decoding(delta):
    import chunked_linear_recurrence_gb300 as sf
    g = torch.Generator().manual_seed(5)
    model, slots = Model(delta, 4), 12
    pool = torch.full((slots, H, D, D), float("nan"), device="cuda")
    extra = torch.arange(slots * 16, device="cuda", dtype=torch.int16).view(slots, 16)   # another layer's cache
    reserved = torch.zeros(slots, dtype=torch.bool, device="cuda")
    reserved[3] = True                                            # a prompt's state kept for later
    prompts = torch.randint(0, V, (3, 70), generator=g).cuda()
    idx = torch.tensor([9, 3, 5], dtype=torch.int32, device="cuda")
    model.prefill(prompts, pool, idx)
    extra[idx.long(), 0] = torch.tensor([100, 101, 102], dtype=torch.int16, device="cuda")
    start = {i: f64(pool[s]) for i, s in enumerate(idx.tolist())}

    parents = torch.tensor([0, 0, 1, 1, 2], dtype=torch.int32, device="cuda")
    rows = sf.sf_state_fork([pool, extra], idx, parents, reserved=reserved)
    assert rows.tolist() == [9, 1, 2, 4, 5]                       # slot 3 is kept and copied twice
    assert extra[rows.long(), 0].tolist() == [100, 100, 101, 101, 102]

    N = 5
    x0 = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    done = [[] for _ in range(N)]                                 # tokens whose states count
    pending = num_pending = None
    for r in range(4):
        drafts = torch.randint(0, V, (N, DRAFTS), generator=g, dtype=torch.int32).cuda()
        x = torch.cat([x0[:, None], drafts], 1)
        t = model.inputs(x)
        out = model.draft_step(t, pool, rows, pending, num_pending)
        for n in range(N):
            ro, _ = model.want(done[n] + x[n].tolist(), start[parents[n].item()])
            assert err(out[n], ro[len(done[n]):]) <= 2.0 ** -8 + 1.6e-5
        probs = (out.float().flatten(2) @ model.head).softmax(-1)
        u = torch.rand(N, DRAFTS + 1, generator=g).cuda()
        u[0, :DRAFTS] = 0.0                                       # everything the target could say is accepted
        u[1, 0] = 1.0                                             # nothing is
        tokens, num = sf.sf_draft_verify(probs, drafts, u)
        wt, wn = od.verify(f64(probs), drafts.tolist(), f64(u))
        assert tokens.tolist() == wt.tolist() and num.tolist() == wn.tolist()
        assert num[0] == DRAFTS + 1 and num[1] == 1
        for n in range(N):
            done[n] += x[n, :num[n]].tolist()
        x0 = tokens.gather(1, num.long()[:, None] - 1)[:, 0].contiguous()
        pending, num_pending = t, num
    model.commit(pending, pool, rows, num_pending)
    finals = [model.want(done[n], start[parents[n].item()])[1] for n in range(N)]
    for n in range(N):
        assert err(pool[rows[n].item()], finals[n]) <= 1.6e-5
    assert np.array_equal(f64(pool[3]), start[1])                 # as the prefill left it

    keep = torch.tensor([4, 2, 1], dtype=torch.int32, device="cuda")   # two continuations end here
    left = sf.sf_state_fork([pool, extra], rows, keep, reserved=reserved)
    assert left.tolist() == [5, 2, 1]
    left = sf.sf_state_compact([pool, extra], left, reserved=reserved)
    assert left.tolist() == [4, 2, 1]                             # 1, 2, 4: the lowest but for the one kept
    for i, n in enumerate(keep.tolist()):
        assert err(pool[left[i].item()], finals[n]) <= 1.6e-5
    assert extra[left.long(), 0].tolist() == [102, 101, 100]


@pytest.mark.parametrize("delta", [False, True])
def test_a_round_in_one_graph(delta):
    """A round is captured once and replayed: the counts, tokens and slots of the next round come out
    of the graph's own buffers, on the device alone."""
    import chunked_linear_recurrence_gb300 as sf
    g = torch.Generator().manual_seed(6)
    model, N, slots = Model(delta, 7), 3, 6
    start = torch.randn(slots, H, D, D, generator=g).cuda() * 0.1
    idx = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    drafts = torch.randint(0, V, (5, N, DRAFTS), generator=g, dtype=torch.int32).cuda()
    us = torch.rand(5, N, DRAFTS + 1, generator=g).cuda()
    first = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()

    def fresh():
        z = model.inputs(torch.zeros(N, DRAFTS + 1, dtype=torch.int32, device="cuda"))
        return dict(pool=start.clone(), x0=first.clone(), pend={m: t.clone() for m, t in z.items()},
                    num=torch.zeros(N, dtype=torch.int32, device="cuda"), d=drafts[0].clone(), u=us[0].clone())

    def round_(s):
        t = model.inputs(torch.cat([s["x0"][:, None], s["d"]], 1))
        out = model.draft_step(t, s["pool"], idx, s["pend"], s["num"])
        tokens, num = sf.sf_draft_verify((out.float().flatten(2) @ model.head).softmax(-1), s["d"], s["u"])
        s["x0"].copy_(tokens.gather(1, num.long()[:, None] - 1)[:, 0])
        s["num"].copy_(num)
        for m, x in s["pend"].items():
            x.copy_(t[m])
        return out, tokens

    a, b = fresh(), fresh()
    round_(fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = round_(b)
    for r in range(5):
        for s in (a, b):
            s["d"].copy_(drafts[r])
            s["u"].copy_(us[r])
        want = round_(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(map(torch.equal, got, want)) and torch.equal(a["pool"], b["pool"])
        assert torch.equal(a["num"], b["num"]) and torch.equal(a["x0"], b["x0"])
