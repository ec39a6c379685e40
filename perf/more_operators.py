"""What the operators of decoding several tokens at a time are measured on.

A sequence of a linear recurrence holds one state in a pool.  A round of decoding with drafted
tokens computes the drafts' outputs from the state without advancing it (``draft_step``, which
first advances it by the tokens that the round before accepted, or ``commit``, which does that
alone), and tests the drafts against the target's probabilities (``verify``).  Sequences fork
into several continuations and leave the pool (``fork``), and what is left is moved together
(``compact``).  ``run`` computes them in plain torch operations, or, where ``own`` is true,
through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX_STATES = 4096            # states of 128 x 128 that the largest drawn step holds
MAX_PROBS = 128 * 15 * 100003


# ------------------------------------------------------------------------------- the cases
def _step(op, rule, N, T, P, H, HK, D, dtype="bf16", pad=0):
    """T tokens whose outputs are wanted (0 for a commit) behind up to P accepted ones."""
    return dict(op=op, rule=rule, N=N, T=T, P=P, H=H, HK=HK, D=D, dtype=dtype, pad=pad)


def _verify(N, T, V, dtype="f32", drafts=True):
    return dict(op="verify", N=N, T=T, V=V, dtype=dtype, drafts=drafts)


def _fork(rows, sources, slots, caches, H, D, pinned=0):
    """`rows` sequences are continued by `rows` others, all of them from the first `sources`,
    `pinned` of which stay as they are."""
    return dict(op="fork", rows=rows, sources=sources, slots=slots, caches=caches, H=H, D=D,
                pinned=pinned)


def _compact(live, moves, slots, caches, H, D, pinned=0):
    return dict(op="compact", live=live, moves=moves, slots=slots, caches=caches, H=H, D=D,
                pinned=pinned)


def listed():
    return [
        # one request that drafts three tokens behind its last one: latency
        dict(_step("draft_step", "gdn", 1, 4, 4, 16, 16, 128), name="draft_step.one"),
        # a batch of requests in the midst of decoding, grouped heads, one row of it padding
        dict(_step("draft_step", "gdn", 128, 5, 5, 32, 16, 128, pad=1), name="draft_step.batch"),
        # the other rule with long drafts
        dict(_step("draft_step", "linattn", 256, 8, 8, 16, 16, 128), name="draft_step.linattn"),
        # the first round after the prompts: nothing to advance by; FP32 tokens, small heads
        dict(_step("draft_step", "gdn", 33, 3, 0, 6, 2, 64, "f32"), name="draft_step.first"),
        # the accepted tokens of a batch brought into the states before they are forked or kept
        dict(_step("commit", "gdn", 128, 0, 8, 32, 16, 128), name="commit.batch"),
        # the same for a few requests of the other rule
        dict(_step("commit", "linattn", 5, 0, 3, 16, 4, 128), name="commit.few"),
        # one request, a small vocabulary: latency
        dict(_verify(1, 3, 32000), name="verify.one"),
        # a batch with seven drafts each and an odd vocabulary
        dict(_verify(128, 7, 100003), name="verify.batch"),
        # the best of four continuations takes the place of all: latency
        dict(_fork(4, 1, 9, 1, 16, 128), name="fork.one"),
        # the surviving continuations of a beam search take over the places of the others, eight layers
        dict(_fork(96, 40, 160, 8, 16, 128, pinned=3), name="fork.beams"),
        # a few finished requests leave holes in a small pool
        dict(_compact(6, 2, 17, 1, 16, 128), name="compact.few"),
        # a pool of eight layers is emptied to a third before its rest is given back
        dict(_compact(60, 48, 192, 8, 16, 128, pinned=2), name="compact.pool"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["draft_step", "draft_step", "draft_step", "commit", "verify", "verify", "fork",
                     "compact"])
    D = rng.choice([128, 128, 128, 64])
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    if op in ("draft_step", "commit"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        HK = rng.choice([x for x in range(1, H + 1) if H % x == 0 and x * 4 >= H])
        N = _log(rng, 1, MAX_STATES // H // 2)
        T = 0 if op == "commit" else _log(rng, 1, 16)
        P = _log(rng, 1, 16) if op == "commit" else rng.choice([0, T, T])
        return _step(op, rng.choice(["gdn", "linattn"]), N, T, P, H, HK, D, dtype,
                     rng.choice([0, 0, 1]))
    if op == "verify":
        T, V = rng.randint(0, 8), _log(rng, 100, 200000)
        N = _log(rng, 1, max(1, min(512, MAX_PROBS // 2 // ((2 * T + 1) * V))))
        return _verify(N, T, V, rng.choice(["f32", "f32", "bf16"]), rng.choice([True, True, False]))
    caches = rng.choice([1, 1, 2, 5])
    slots = _log(rng, 8, max(9, 160 * 8 * 16 // (caches * H)) if caches * H > 16 else 300)
    pinned = rng.choice([0, 0, 1])
    if op == "fork":
        rows = rng.randint(1, slots - 2 - pinned)
        return _fork(rows, rng.randint(1, rows), slots, caches, H, D, pinned)
    live = rng.randint(1, slots - 2 - pinned)
    return _compact(live, rng.randint(0, min(live, slots - 1 - pinned - live)), slots, caches, H, D, pinned)


# ------------------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def _slopes(H):
    """Decays of the heads: a geometric series, from a memory of a token or two to one of
    hundreds."""
    return [-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)]


def _pick(g, lo, hi, n):
    """n different whole numbers of [lo, hi)."""
    return torch.randperm(hi - lo, generator=g, device="cuda")[:n] + lo


def prepare(case, seed):
    g = _gen(seed)
    c = case
    s = dict(case=c)
    op = c["op"]
    if op in ("draft_step", "commit"):
        N, H, HK, D, dt = c["N"], c["H"], c["HK"], c["D"], DTYPES[c["dtype"]]

        def tokens(n):
            t = dict(k=_unit(_randn(g, N, n, HK, D)).to(dt), v=_randn(g, N, n, H, D).to(dt))
            if c["rule"] == "gdn":
                t["gate"] = -torch.nn.functional.softplus(_randn(g, N, n, H))
                t["beta"] = torch.sigmoid(_randn(g, N, n, H))
            return t
        count = lambda n: torch.randint(1, n + 1, (N,), generator=g, device="cuda",   # noqa: E731
                                        dtype=torch.int32)
        s["pend"] = tokens(c["P"]) if c["P"] else None
        s["num_pend"] = count(c["P"]) if c["P"] else None
        if op == "draft_step":
            s["new"] = tokens(c["T"])
            s["new"]["q"] = _unit(_randn(g, N, c["T"], HK, D)).to(dt)
            s["num_new"] = count(c["T"])        # some requests draft fewer tokens
        s["cache"] = _randn(g, N + 1, H, D, D) * 0.1                     # slot 0: padding's
        idx = torch.randperm(N, generator=g, device="cuda").to(torch.int32) + 1
        if c["pad"]:
            idx[N // 2:N // 2 + c["pad"]] = -1
        s["idx"] = idx
        s["decay"] = torch.tensor(_slopes(H), device="cuda")
        return s
    if op == "verify":
        N, T, V, dt = c["N"], c["T"], c["V"], DTYPES[c["dtype"]]
        s["target"] = torch.empty(N, T + 1, V, device="cuda", dtype=dt)
        s["draft"] = torch.empty(N, T, V, device="cuda", dtype=dt) if c["drafts"] else None
        s["x"] = torch.zeros(N, T, device="cuda", dtype=torch.int32)
        heat = 0.5 + 3.0 * torch.rand(N, 1, generator=g, device="cuda")   # from flat to peaked
        for t in range(T + 1):       # the draft model's logits are the target's and an error
            z = _randn(g, N, V) * heat
            s["target"][:, t] = z.softmax(-1).to(dt)
            if t == T:
                break
            p = (z + 0.5 * _randn(g, N, V)).softmax(-1).to(dt)
            if c["drafts"]:
                s["draft"][:, t] = p
                s["x"][:, t] = torch.multinomial(p.float(), 1, generator=g)[:, 0].int()
            else:                    # a looked-up continuation, often the likeliest
                s["x"][:, t] = p.argmax(-1).int()
        s["u"] = torch.rand(N, T + 1, generator=g, device="cuda")
        s["num"] = torch.randint((T + 1) // 2, T + 1, (N,), generator=g, device="cuda",
                                 dtype=torch.int32)
        return s
    H, D, S = c["H"], c["D"], c["slots"]
    s["caches"] = [_randn(g, S, H, D, D) for _ in range(c["caches"])]
    s["reserved"] = torch.zeros(S, dtype=torch.bool, device="cuda")
    if op == "fork":
        held = _pick(g, 1, S, c["rows"])            # those past the sources end here
        more = min(c["pinned"], c["sources"])
        s["reserved"][held[:more]] = True           # states kept for later: copied, never taken over
        s["idx"] = held.int()
        # every source has at least one continuation, the others go at random
        parents = torch.randint(0, c["sources"], (c["rows"],), generator=g, device="cuda")
        parents[:c["sources"]] = torch.arange(c["sources"], device="cuda")
        s["parents"] = parents[torch.randperm(c["rows"], generator=g, device="cuda")].int()
        return s
    # pinned slots first, so that the places to fill are known: the next ones
    s["reserved"][1:1 + c["pinned"]] = True
    lo = 1 + c["pinned"]
    mid = lo + c["live"]
    idx = torch.cat([_pick(g, lo, mid, c["live"] - c["moves"]), _pick(g, mid, S, c["moves"])])
    s["idx"] = idx[torch.randperm(c["live"], generator=g, device="cuda")].int()
    return s


# ------------------------------------------------------------------------- the plain forms
def _live(idx, slots):
    return (idx > 0) & (idx < slots)


def _walk(S, tok, n, decay, group, scale, on):
    """The tokens of every sequence, one after the other, from the states S [N,H,V,K]: where a
    sequence is `on` and has more than t tokens (n), token t advances it.  Returns the states
    and, with queries, the outputs."""
    wide = lambda x: torch.repeat_interleave(x.float(), group, 2)   # noqa: E731
    k, v = wide(tok["k"]), tok["v"].float()
    q = wide(tok["q"]) if "q" in tok else None
    outs = []
    for t in range(k.shape[1]):
        kt = k[:, t, :, None]
        if "gate" in tok:
            d = S * tok["gate"][:, t].exp()[..., None, None]
            r = tok["beta"][:, t][..., None] * (v[:, t] - (d * kt).sum(-1))
        else:
            d = S * decay.exp()[None, :, None, None]
            r = v[:, t]
        use = (on & (t < n))[:, None, None, None]
        S = torch.where(use, d + r[..., None] * kt, S)
        if q is not None:
            outs.append(torch.where(use[..., 0], (S * q[:, t, :, None]).sum(-1) * scale, 0.0))
    return S, torch.stack(outs, 1) if outs else None


def _plain_step(s):
    c = s["case"]
    G = c["H"] // c["HK"]
    on = _live(s["idx"], s["cache"].shape[0])
    at = torch.where(on, s["idx"], 0).long()
    S = s["cache"][at]
    if c["P"]:
        S, _ = _walk(S, s["pend"], s["num_pend"], s["decay"], G, 1.0, on)
        s["cache"][at] = S                  # padding hands slot 0 back as it was
    if c["op"] == "commit":
        return dict(cache=s["cache"])
    _, out = _walk(S, s["new"], s["num_new"], s["decay"], G, c["D"] ** -0.5, on)
    return dict(out=out.to(s["new"]["v"].dtype), cache=s["cache"])


def _plain_verify(s):
    c = s["case"]
    N, T = c["N"], c["T"]
    n = s["num"].long()
    ok = torch.zeros(N, T, dtype=torch.bool, device="cuda")
    if T:
        at = s["x"].long()[..., None]
        p = s["target"][:, :T].gather(2, at)[..., 0].double()
        q = s["draft"].gather(2, at)[..., 0].double() if c["drafts"] else torch.ones_like(p)
        ok = (s["u"][:, :T].double() * q < p) & (torch.arange(T, device="cuda") < n[:, None])
    taken = ok.long().cumprod(1).sum(1)
    row = torch.arange(N, device="cuda")
    p = s["target"][row, taken].double()
    w = p
    if T:
        which = taken.clamp_max(T - 1)
        if c["drafts"]:
            less = (p - s["draft"][row, which].double()).clamp_min(0)
        else:
            less = p.scatter(1, s["x"][row, which].long()[:, None], 0.0)
        less = torch.where(less.sum(1, keepdim=True) > 0, less, p)
        w = torch.where((taken < n)[:, None], less, p)
    run = w.cumsum(1)
    aim = s["u"][:, T].double() * run[:, -1]
    pick = (run <= aim[:, None]).sum(1).clamp_max(c["V"] - 1)
    col = torch.arange(T + 1, device="cuda")
    x = torch.cat([s["x"].long(), torch.zeros(N, 1, dtype=torch.long, device="cuda")], 1)
    tokens = torch.where(col < taken[:, None], x, torch.where(col == taken[:, None], pick[:, None], -1))
    return dict(tokens=tokens.int(), num=(taken + 1).int())


def _free_first(used):
    """The slots, those that are not used first, each kind from the lowest on."""
    return torch.sort(used.int(), stable=True).indices


def _plain_fork(s):
    S = s["case"]["slots"]
    src = s["idx"].long()[s["parents"].long()]
    M = src.numel()
    earlier = torch.ones(M, M, dtype=torch.bool, device="cuda").tril(-1)
    first = ~((src[:, None] == src[None]) & earlier).any(1)
    keep = first & ~s["reserved"][src]
    used = s["reserved"].clone()
    used[0] = True
    used[src[keep]] = True
    rank = (~keep).long().cumsum(0) - 1
    place = _free_first(used)[rank.clamp(0, S - 1)]
    new = torch.where(keep, src, torch.where(rank < (~used).sum(), place, -1))
    rows = (~keep & (new > 0)).nonzero()[:, 0]
    for cache in s["caches"]:
        cache[new[rows]] = cache[src[rows]]
    return dict(idx=new.int(), caches=s["caches"])


def _plain_compact(s):
    idx = s["idx"].long()
    live = torch.zeros(s["case"]["slots"], dtype=torch.bool, device="cuda")
    live[idx] = True
    live &= ~s["reserved"]
    usable = ~s["reserved"]
    usable[0] = False
    low = usable & (usable.long().cumsum(0) <= live.sum())
    src, dst = (live & ~low).nonzero()[:, 0], (low & ~live).nonzero()[:, 0]
    to = torch.arange(live.numel(), device="cuda")
    to[src] = dst
    for cache in s["caches"]:
        cache[dst] = cache[src]
    return dict(idx=to[idx].int(), caches=s["caches"])


# ----------------------------------------------------------------------- the package's calls
def _own(s):
    import chunked_linear_recurrence_gb300 as sf
    c = s["case"]
    op = c["op"]
    if op == "draft_step":
        n, p = s["new"], s["pend"]
        if c["rule"] == "gdn":
            pend = None if p is None else (p["k"], p["v"], p["gate"], p["beta"])
            out = sf.sf_gdn_draft_step(n["q"], n["k"], n["v"], n["gate"], n["beta"], s["cache"],
                                       s["idx"], num_tokens=s["num_new"], pending=pend,
                                       num_pending=s["num_pend"])
        else:
            pend = None if p is None else (p["k"], p["v"])
            out = sf.sf_linattn_draft_step(n["q"], n["k"], n["v"], s["decay"], s["cache"], s["idx"],
                                           num_tokens=s["num_new"], pending=pend,
                                           num_pending=s["num_pend"])
        return dict(out=out, cache=s["cache"])
    if op == "commit":
        p = s["pend"]
        if c["rule"] == "gdn":
            sf.sf_gdn_commit(p["k"], p["v"], p["gate"], p["beta"], s["cache"], s["idx"],
                             num_tokens=s["num_pend"])
        else:
            sf.sf_linattn_commit(p["k"], p["v"], s["decay"], s["cache"], s["idx"],
                                 num_tokens=s["num_pend"])
        return dict(cache=s["cache"])
    if op == "verify":
        tokens, num = sf.sf_draft_verify(s["target"], s["x"], s["u"], draft_probs=s["draft"],
                                         num_drafts=s["num"])
        return dict(tokens=tokens, num=num)
    if op == "fork":
        idx = sf.sf_state_fork(s["caches"], s["idx"], s["parents"], reserved=s["reserved"])
    else:
        idx = sf.sf_state_compact(s["caches"], s["idx"], reserved=s["reserved"])
    return dict(idx=idx, caches=s["caches"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"draft_step": _plain_step, "commit": _plain_step, "verify": _plain_verify,
            "fork": _plain_fork, "compact": _plain_compact}[op](state)


# ------------------------------------------------------------------------------ work, exact
def work(case):
    c = case
    if c["op"] in ("draft_step", "commit"):
        e = 2 if c["dtype"] == "bf16" else 4
        H, HK, D = c["H"], c["HK"], c["D"]
        N = c["N"] - c["pad"] if c["N"] > c["pad"] else max(1, c["N"] - 1)
        T, P = (c["T"] + 1) / 2, (c["P"] + 1) / 2 if c["P"] else 0     # tokens in use, on average
        gates = 8 * H if c["rule"] == "gdn" else 0
        per = (2 * HK + 2 * H) * D * e + gates
        if c["op"] == "commit":
            T = 0
        return {"bytes": N * (4 * H * D * D * (2 if c["P"] else 1) + T * per
                              + P * ((HK + H) * D * e + gates)),
                "flops": N * H * D * D * 2 * ((2 if c["rule"] == "gdn" else 1) * (T + P))}
    if c["op"] == "verify":
        e = 2 if c["dtype"] == "bf16" else 4
        # the row that is drawn from; the draft's row too, unless all drafts are accepted
        rows = 1 + (1 - 0.78 ** (0.75 * c["T"]) if c["drafts"] and c["T"] else 0)
        return {"bytes": c["N"] * c["V"] * e * rows, "flops": c["N"] * c["V"] * (rows + 1)}
    if c["op"] == "fork":
        moved = c["rows"] - c["sources"] + min(c["pinned"], c["sources"])
    else:
        moved = c["moves"]
    small = 4 * (c["rows"] if c["op"] == "fork" else c["live"]) * 2 + c["slots"]
    return {"bytes": 8 * moved * c["caches"] * c["H"] * c["D"] * c["D"] + small, "flops": 0}


def _exact_step(s):
    """From the definition in closed form: with M_t = e^{g_t} (I - beta_t k_t k_t^T) the state after
    n tokens is S M_1 .. M_n + sum_t beta_t v_t k_t^T M_{t+1} .. M_n, so that a row is followed
    backwards from the vector that reads it (outputs), and the whole matrix forwards."""
    c = s["case"]
    G, D = c["H"] // c["HK"], c["D"]
    cache = s["cache"].double()
    idx = s["idx"].tolist()
    counts = {m: s[m].tolist() for m in ("num_pend", "num_new") if s.get(m) is not None}
    eye = torch.eye(D, dtype=torch.float64, device="cuda")
    gdn = c["rule"] == "gdn"

    def rule(tok, n, t):
        k = tok["k"][n, t].double().repeat_interleave(G, 0)
        v = tok["v"][n, t].double()
        if gdn:
            return k, v, tok["gate"][n, t].double().exp(), tok["beta"][n, t].double()
        return k, v, s["decay"].double().exp(), torch.ones(c["H"], dtype=torch.float64, device="cuda")

    out = None
    if c["op"] == "draft_step":
        out = torch.zeros(c["N"], c["T"], c["H"], D, dtype=torch.float64, device="cuda")
    for n, slot in enumerate(idx):
        if not 0 < slot < cache.shape[0]:
            continue
        if c["P"]:
            S = cache[slot]
            for t in range(counts["num_pend"][n]):
                k, v, lam, beta = rule(s["pend"], n, t)
                M = eye - (beta[:, None, None] * k[:, :, None] * k[:, None] if gdn else 0.0)
                S = lam[:, None, None] * (S @ M) + (beta[:, None] * v)[:, :, None] * k[:, None]
            cache[slot] = S
        if out is None:
            continue
        steps = [rule(s["new"], n, t) for t in range(counts["num_new"][n])]
        for i in range(len(steps)):
            x = s["new"]["q"][n, i].double().repeat_interleave(G, 0) * D ** -0.5
            o = 0.0
            for k, v, lam, beta in reversed(steps[:i + 1]):
                kx = (k * x).sum(-1, keepdim=True)
                o = o + beta[:, None] * v * kx
                x = lam[:, None] * (x - (beta[:, None] * kx * k if gdn else 0.0))
            out[n, i] = o + (cache[slot] @ x[..., None])[..., 0]
    return dict(cache=cache) if out is None else dict(out=out, cache=cache)


def _exact_verify(s):
    c = s["case"]
    N, T = c["N"], c["T"]
    x, num = s["x"].tolist(), s["num"].tolist()
    u = s["u"].double().cpu().numpy()
    tokens, count = np.full((N, T + 1), -1, np.int32), np.zeros(N, np.int32)
    for n in range(N):
        a = 0
        while a < num[n]:
            p = float(s["target"][n, a, x[n][a]])
            q = float(s["draft"][n, a, x[n][a]]) if c["drafts"] else 1.0
            if not u[n, a] * q < p:
                break
            tokens[n, a] = x[n][a]
            a += 1
        p = s["target"][n, a].double().cpu().numpy()
        w = p
        if a < num[n]:
            w = p.copy()
            if c["drafts"]:
                w = np.maximum(p - s["draft"][n, a].double().cpu().numpy(), 0.0)
            else:
                w[x[n][a]] = 0.0
            w = w if w.any() else p
        run = np.cumsum(w)
        tokens[n, a] = min(int(np.searchsorted(run, u[n, T] * run[-1], side="right")), c["V"] - 1)
        count[n] = a + 1
    return dict(tokens=torch.from_numpy(tokens).cuda(), num=torch.from_numpy(count).cuda())


def _exact_move(s):
    c = s["case"]
    idx = s["idx"].tolist()
    pinned = set(s["reserved"].nonzero()[:, 0].tolist())
    moves = {}
    if c["op"] == "fork":
        want = [idx[p] for p in s["parents"].tolist()]
        kept = set(want) - pinned
        free = [x for x in range(1, c["slots"]) if x not in kept and x not in pinned]
        new, seen = [], set()
        for x in want:
            if x in pinned or x in seen:
                to = free.pop(0) if free else -1
                if to > 0:
                    moves[to] = x
                new.append(to)
            else:
                new.append(x)
            seen.add(x)
    else:
        live = sorted(set(idx) - pinned)
        places = [x for x in range(1, c["slots"]) if x not in pinned][:len(live)]
        holes = [x for x in places if x not in live]
        to = dict(zip([x for x in live if x not in places], holes))
        moves = {b: a for a, b in to.items()}
        new = [to.get(x, x) for x in idx]
    for cache in s["caches"]:
        for to, x in moves.items():
            cache[to] = cache[x]
    return dict(idx=torch.tensor(new, dtype=torch.int32, device="cuda"),
                caches=[cache.double() for cache in s["caches"]])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("draft_step", "commit"):
        return _exact_step(s)
    return _exact_verify(s) if op == "verify" else _exact_move(s)
