"""What the linear-attention operators are measured on.

The operators are the decayed linear attention (chunked forward and backward for prompts and
training, one-token step for decoding), the gated delta rule's one-token step, and the pass
that turns a projection's raw queries and keys into what both rules take: a norm of each head
and the position rotation (with one or several position axes).  ``run`` computes them in
plain 32-bit torch operations, or, where ``own`` is true, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 128          # of the plain form
EXACT_CHUNK = 64     # of the 64-bit form
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases
def _norm(op, B, T, H, HK, D, dtype="bf16", norm="rms", rot=None, axes=1, interleaved=False):
    return dict(op=op, B=B, T=T, H=H, HK=HK, D=D, dtype=dtype, norm=norm, rot=rot or D,
                axes=axes, interleaved=interleaved)


def _chunk(op, B, T, H, HK, D, dtype="bf16", packed=0, s0=True):
    return dict(op=op, B=B, T=T, H=H, HK=HK, D=D, dtype=dtype, packed=packed, s0=s0)


def _step(op, N, H, HK, D, dtype="bf16", pad=0):
    return dict(op=op, N=N, H=H, HK=HK, D=D, dtype=dtype, pad=pad)


def listed():
    return [
        # one token of each of 16 decoding requests, grouped heads: the smallest call, latency
        dict(_norm("norm_rope", 16, 1, 16, 4, 128), name="norm_rope.decode"),
        # a packed prompt of video patches: three position axes, an odd number of tokens
        dict(_norm("norm_rope", 1, 32769, 16, 16, 128, axes=3), name="norm_rope.video"),
        # the same pass's gradients in a training step
        dict(_norm("norm_rope_bwd", 2, 8192, 16, 16, 128), name="norm_rope_bwd.train"),
        # one short prompt that is no multiple of any chunk: latency
        dict(_chunk("linattn", 1, 130, 16, 16, 128, s0=False), name="linattn.prompt"),
        # a batch of prompts with carried states
        dict(_chunk("linattn", 4, 4096, 16, 16, 128), name="linattn.batch"),
        # one very long document on few heads: nothing to split but the time axis
        dict(_chunk("linattn", 1, 131072, 4, 4, 128), name="linattn.long"),
        # eight ragged prompts packed into one stream (one of them empty), grouped heads
        dict(_chunk("linattn", 1, 65536, 32, 8, 128, packed=8), name="linattn.packed"),
        # a training step's backward pass
        dict(_chunk("linattn_bwd", 2, 8192, 16, 16, 128), name="linattn_bwd.train"),
        # a small packed backward in FP32 at the smaller head size, grouped heads
        dict(_chunk("linattn_bwd", 1, 1000, 4, 2, 64, "f32", packed=3), name="linattn_bwd.f32"),
        # decoding: one token of each of 256 requests on a paged pool of states, some rows padding
        dict(_step("linattn_step", 256, 16, 16, 128, pad=3), name="linattn_step.batch"),
        # decoding one request with the delta rule: latency
        dict(_step("gdn_step", 1, 16, 16, 128), name="gdn_step.one"),
        # decoding a batch with the delta rule, grouped heads
        dict(_step("gdn_step", 128, 32, 16, 128, pad=1), name="gdn_step.batch"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "linattn", "linattn", "linattn", "linattn_bwd",
                     "linattn_bwd", "linattn_step", "gdn_step"])
    D = rng.choice([128, 128, 128, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    HK = rng.choice([x for x in range(1, H + 1) if H % x == 0 and x * 4 >= H])
    if op.startswith("norm_rope"):
        rows = 32768 * 16 * 128 // (H * D * (2 if dtype == "f32" else 1))
        if op == "norm_rope_bwd":
            rows //= 2
        B = rng.choice([1, 1, 2, 3, 5])
        T = _log(rng, 1, max(1, rows // B))
        rot = rng.choice([D, D, D // 2])
        return _norm(op, B, T, H, HK, D, dtype, rng.choice(["rms", "l2"]), rot,
                     rng.choice([1, 1, 2, 3]), rng.choice([False, False, True]))
    if op.endswith("step"):
        return _step(op, _log(rng, 1, 4096 // H), H, HK, D, dtype, rng.choice([0, 0, 1]))
    # token-heads: as many as the longest listed case of the direction; FP32 runs on the
    # CUDA cores, and a user keeps it to smaller work
    most = 65536 * 4 if op == "linattn_bwd" else 65536 * 8
    if dtype == "f32":
        most //= 8
    packed = rng.choice([0, 0, 2, 5, 8])
    B = 1 if packed else rng.choice([1, 1, 2, 4, 7])
    T = _log(rng, max(1, packed), max(packed, most // (B * H), 1))
    return _chunk(op, B, T, H, HK, D, dtype, packed, rng.choice([True, False]))


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


def _lengths(seed, n, total):
    """n ragged lengths that sum to at most `total`, one of them empty where there are several."""
    r = np.random.RandomState(seed % (1 << 31))
    w = r.uniform(0.1, 1.9, n)
    if n > 3:
        w[3] = 0.0
    L = np.floor(w / w.sum() * total).astype(int)
    if L.sum() == 0:
        L[0] = total
    return [int(x) for x in L]


def _table(P, half, base=10000.0):
    inv = base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    a = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()      # [P, half, 2]


def _sections(axes, half):
    """Rotary pairs of each position axis, in order: the first axis (time) gets the rest."""
    if axes == 1:
        return [half]
    other = (half * 3) // (8 if axes == 3 else 4)
    return [half - other * (axes - 1)] + [other] * (axes - 1)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    H, HK, D = case["H"], case["HK"], case["D"]
    s = dict(case=case)
    op = case["op"]
    if op.startswith("norm_rope"):
        B, T = case["B"], case["T"]
        # the heads of one fused projection: queries, keys and values side by side
        qkv = _randn(g, B, T, (H + 2 * HK) * D).to(dt)
        s["q"] = qkv[..., :H * D].view(B, T, H, D)
        s["k"] = qkv[..., H * D:(H + HK) * D].view(B, T, HK, D)
        s["qw"] = 1.0 + 0.1 * _randn(g, D)
        s["kw"] = 1.0 + 0.1 * _randn(g, D)
        half = case["rot"] // 2
        P = max(64, min(B * T, 32768) + 1)
        s["table"] = _table(P, half)
        if T == 1:     # decoding: every request is somewhere else
            s["pos"] = torch.randint(0, P, (case["axes"], B * T), generator=g, device="cuda",
                                     dtype=torch.int32)
        elif case["axes"] == 1:
            s["pos"] = (torch.arange(B * T, device="cuda", dtype=torch.int32) % T % P)[None].contiguous()
        else:          # frames of 24 x 24 patches: time, height, width
            t = torch.arange(B * T, device="cuda", dtype=torch.int32) % T
            s["pos"] = torch.stack([t // 576 % P, t // 24 % 24, t % 24][:case["axes"]]).contiguous()
        s["sections"] = _sections(case["axes"], half)
        if op == "norm_rope_bwd":
            s["dq"] = _randn(g, B, T, H, D).to(dt)
            s["dk"] = _randn(g, B, T, HK, D).to(dt)
        return s
    if op.endswith("step"):
        N = case["N"]
        s["q"] = _unit(_randn(g, N, HK, D)).to(dt)
        s["k"] = _unit(_randn(g, N, HK, D)).to(dt)
        s["v"] = _randn(g, N, H, D).to(dt)
        s["cache"] = _randn(g, N + 1, H, D, D) * 0.1                     # slot 0: padding's
        idx = torch.randperm(N, generator=g, device="cuda").to(torch.int32) + 1
        if case["pad"]:
            idx[N // 2:N // 2 + case["pad"]] = -1
        s["idx"] = idx
        s["decay"] = torch.tensor(_slopes(H), device="cuda")
        if op == "gdn_step":
            s["gate"] = -torch.nn.functional.softplus(_randn(g, N, H))
            s["beta"] = torch.sigmoid(_randn(g, N, H))
        return s
    B, T = case["B"], case["T"]
    s["q"] = _unit(_randn(g, B, T, HK, D)).to(dt)
    s["k"] = _unit(_randn(g, B, T, HK, D)).to(dt)
    s["v"] = _randn(g, B, T, H, D).to(dt)
    s["decay"] = torch.tensor(_slopes(H), device="cuda")
    lens = _lengths(seed, case["packed"], T) if case["packed"] else [T] * B
    N = len(lens)
    s["lens"] = lens
    s["n"] = torch.tensor(lens, device="cuda")
    if case["packed"]:
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
        starts = torch.tensor([0] + list(np.cumsum(lens))[:-1], device="cuda")
        n = s["n"]
        # row of every (sequence, position from the right end), for the plain form's padding
        Tm = max(max(lens), 1)
        at = torch.arange(Tm, device="cuda")[None] - (Tm - n)[:, None]
        s["live"] = at >= 0
        s["rows"] = torch.where(s["live"], starts[:, None] + at, T)
    else:
        s["cu"] = None
    s["s0"] = _randn(g, N, H, D, D) * 0.1 if case["s0"] else None
    if op == "linattn_bwd":
        s["dout"] = _randn(g, B, T, H, D).to(dt)
        s["dfin"] = _randn(g, N, H, D, D) * 0.01
    return s


# ------------------------------------------------------------------------- the plain forms
def _rot_cs(s):
    half = s["case"]["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=half)
    cs = s["table"][s["pos"].long()[axis].T, torch.arange(half, device="cuda")]   # [tokens, half, 2]
    B, T = s["case"]["B"], s["case"]["T"]
    return cs.view(B, T, 1, half, 2).unbind(-1)


def _rotate(x, cos, sin, rot, interleaved):
    y, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    cos, sin = _rot_cs(s)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.float()
        if c["norm"] == "rms":
            y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        else:
            y = x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(EPS)
        out.append(_rotate(y * w, cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype))
    return dict(q=out[0], k=out[1])


def _plain_norm_bwd(s):
    c = s["case"]
    D = c["D"]
    cos, sin = _rot_cs(s)
    res = {}
    for n, x, w, d in (("q", s["q"], s["qw"], s["dq"]), ("k", s["k"], s["kw"], s["dk"])):
        x = x.float()
        dy = _rotate(d.float(), cos, -sin, c["rot"], c["interleaved"])
        ss = x.square().sum(-1, keepdim=True)
        if c["norm"] == "rms":
            r = torch.rsqrt(ss / D + EPS)
            t = r * r / D
        else:
            r = 1.0 / ss.sqrt().clamp_min(EPS)
            t = torch.where(ss.sqrt() > EPS, r * r, torch.zeros_like(r))
        gw = dy * w
        res["d" + n] = (r * (gw - x * t * (gw * x).sum(-1, keepdim=True))).to(d.dtype)
        res["d" + n + "w"] = (dy * x * r).sum((0, 1, 2))
    return res


def _plain_step(s):
    c = s["case"]
    f = lambda x: torch.repeat_interleave(x.float(), c["H"] // c["HK"], 1)   # noqa: E731
    q, k, v = f(s["q"]), f(s["k"]), s["v"].float()
    live = ((s["idx"] > 0) & (s["idx"] < s["cache"].shape[0]))
    at = torch.where(live, s["idx"], 0).long()
    S = s["cache"][at]
    if c["op"] == "gdn_step":
        d = S * s["gate"].exp()[..., None, None]
        r = s["beta"][..., None] * (v - (d * k[:, :, None]).sum(-1))
    else:
        d = S * s["decay"].exp()[None, :, None, None]
        r = v
    S1 = d + r[..., None] * k[:, :, None]
    out = (S1 * q[:, :, None]).sum(-1) * (c["D"] ** -0.5)
    s["cache"][at] = torch.where(live[:, None, None, None], S1, S)
    return dict(out=torch.where(live[:, None, None], out, 0.0).to(s["v"].dtype), cache=s["cache"])


def _heads(x, s):
    """[B,T,heads,D] -> FP32 [N,Tm,H,D]: shared heads repeated, packed sequences padded at
    their left ends with zeros."""
    x = x.float()
    if s["cu"] is not None:
        x = torch.cat([x[0], torch.zeros_like(x[0, :1])])[s["rows"]]
        x = torch.where(s["live"][..., None, None], x, 0.0)
    return torch.repeat_interleave(x, s["case"]["H"] // x.shape[2], 2)


def _unpack(x, s, like):
    """The inverse of _heads' padding, rounded to the type of `like`."""
    if s["cu"] is None:
        return x.to(like.dtype)
    r = torch.zeros(like.shape[1] + 1, *x.shape[2:], device=x.device)
    r[s["rows"].flatten()] = x.flatten(0, 1)
    return r[None, :like.shape[1]].to(like.dtype)


def _mix(x, y, z, decay, scale):
    """scale sum_{j<=i} lam^(i-j) (x_i . y_j) z_j over [N,T,H,D], and sum_j lam^(T-1-j) z_j y_j^T."""
    N, T, H, D = x.shape
    C = min(CHUNK, T)
    nc = -(-T // C)
    pad = nc * C - T                       # at the left: zero rows
    cut = lambda a: torch.nn.functional.pad(a, (0, 0, 0, 0, pad, 0)).view(N, nc, C, H, D)   # noqa: E731
    x, y, z = cut(x), cut(y), cut(z)
    i = torch.arange(C, device=x.device)
    gap = (i[:, None] - i[None]).float()
    w = torch.where(gap >= 0, torch.exp(decay[:, None, None] * gap.clamp_min(0)), 0.0)      # [H,C,C]
    p = torch.einsum("nciha,ncjha->nchij", x, y) * w
    out = torch.einsum("nchij,ncjhv->ncihv", p, z)
    to_end = torch.exp(decay * (C - 1 - i)[:, None])                                        # [C,H]
    U = torch.einsum("ncjhv,ncjha->nchva", z * to_end[..., None], y)
    c = torch.arange(nc, device=x.device)
    steps = (c[:, None] - c[None]).float()
    carry = torch.where(steps >= 0, torch.exp(decay[:, None, None] * C * steps.clamp_min(0)), 0.0)
    S = torch.einsum("hcd,ndhva->nchva", carry, U)                 # state after each chunk
    entry = torch.cat([torch.zeros_like(S[:, :1]), S[:, :-1]], 1)
    rd = torch.exp(decay * (i + 1)[:, None])                                                # [C,H]
    out = out + torch.einsum("nchva,nciha->ncihv", entry, x) * rd[..., None]
    return out.reshape(N, nc * C, H, D)[:, pad:] * scale, S[:, -1]


def _since(s, decay, Tm, shift):
    """lam^(tokens since the sequence's first token, plus shift), [N,Tm,H]."""
    n = s["n"]
    at = torch.arange(Tm, device="cuda")[None] - (Tm - n)[:, None] + shift
    return torch.exp(decay * at.clamp_min(0)[..., None])


def _plain_fwd(s):
    c = s["case"]
    scale, decay = c["D"] ** -0.5, s["decay"]
    q, k, v = _heads(s["q"], s), _heads(s["k"], s), _heads(s["v"], s)
    out, fin = _mix(q, k, v, decay, scale)
    if s["s0"] is not None:
        out = out + scale * _since(s, decay, q.shape[1], 1)[..., None] * torch.einsum(
            "nhva,niha->nihv", s["s0"], q)
        fin = fin + torch.exp(decay * s["n"][:, None])[..., None, None] * s["s0"]
    return dict(out=_unpack(out, s, s["v"]), final_state=fin)


def _plain_bwd(s):
    c = s["case"]
    scale, decay, G = c["D"] ** -0.5, s["decay"], c["H"] // c["HK"]
    n = s["n"]
    q, k, v, do = (_heads(s[x], s) for x in ("q", "k", "v", "dout"))
    Tm = q.shape[1]
    dq, _ = _mix(do, v, k, decay, scale)
    if s["s0"] is not None:
        dq = dq + scale * _since(s, decay, Tm, 1)[..., None] * torch.einsum(
            "nhva,nihv->niha", s["s0"], do)
    back = lambda x: x.flip(1)   # noqa: E731
    dv, _ = _mix(back(k), back(q), back(do), decay, scale)
    dk, _ = _mix(back(v), back(do), back(q), decay, scale)
    to_end = torch.exp(decay * torch.arange(Tm - 1, -1, -1, device="cuda")[:, None])[..., None]
    dv = back(dv) + to_end * torch.einsum("nhva,niha->nihv", s["dfin"], k)
    dk = back(dk) + to_end * torch.einsum("nhva,nihv->niha", s["dfin"], v)
    since = _since(s, decay, Tm, 1)[..., None]
    d0 = scale * torch.einsum("nihv,niha->nhva", do * since, q) + torch.exp(
        decay * n[:, None])[..., None, None] * s["dfin"]
    group = lambda x: x.unflatten(2, (c["HK"], G)).sum(3)   # noqa: E731
    return dict(dq=_unpack(group(dq), s, s["q"]), dk=_unpack(group(dk), s, s["k"]),
                dv=_unpack(dv, s, s["v"]), d_initial_state=d0)


# ----------------------------------------------------------------------- the package's calls
def _kept(s, name, make):
    """A workspace or an output buffer that a program allocates once and passes every time."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    import chunked_linear_recurrence_gb300 as sf
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        q, k = sf.sf_qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["table"], s["pos"],
                                      sections=s["sections"], norm=c["norm"], eps=EPS,
                                      interleaved=c["interleaved"])
        return dict(q=q, k=k)
    if op == "norm_rope_bwd":
        ws = _kept(s, "ws", lambda: sf.sf_qk_norm_rope_bwd_workspace(s["q"], s["k"]))
        g = sf.sf_qk_norm_rope_bwd(s["q"], s["k"], s["qw"], s["kw"], s["table"], s["pos"], s["dq"],
                                   s["dk"], sections=s["sections"], norm=c["norm"], eps=EPS,
                                   interleaved=c["interleaved"], ws=ws)
        return dict(dq=g["dq"], dk=g["dk"], dqw=g["dq_weight"], dkw=g["dk_weight"])
    if op == "linattn_step":
        out = sf.sf_linattn_step(s["q"], s["k"], s["v"], s["decay"], s["cache"], s["idx"])
        return dict(out=out, cache=s["cache"])
    if op == "gdn_step":
        out = sf.sf_gdn_step(s["q"], s["k"], s["v"], s["gate"], s["beta"], s["cache"], s["idx"])
        return dict(out=out, cache=s["cache"])
    if op == "linattn":
        ws = _kept(s, "ws", lambda: sf.sf_linattn_fwd_workspace(s["q"], s["v"], s["cu"]))
        # rows past the last sequence are never written: they stay the zeros they were
        out = _kept(s, "out", lambda: torch.zeros_like(s["v"])) if s["cu"] is not None else None
        out, fin = sf.sf_linattn_chunk_fwd(s["q"], s["k"], s["v"], s["decay"], s["s0"],
                                           cu_seqlens=s["cu"], output_final_state=True, out=out,
                                           ws=ws)
        return dict(out=out, final_state=fin)
    ws = _kept(s, "ws", lambda: sf.sf_linattn_bwd_workspace(s["q"], s["v"], s["cu"]))
    grads = None
    if s["cu"] is not None:
        grads = _kept(s, "grads", lambda: dict(
            dq=torch.zeros_like(s["q"]), dk=torch.zeros_like(s["k"]), dv=torch.zeros_like(s["v"]),
            d_initial_state=torch.zeros_like(s["dfin"])))
    g = sf.sf_linattn_chunk_bwd(s["q"], s["k"], s["v"], s["decay"], s["s0"], s["dout"], s["dfin"],
                                cu_seqlens=s["cu"], grads=grads, ws=ws)
    return dict(dq=g["dq"], dk=g["dk"], dv=g["dv"], d_initial_state=g["d_initial_state"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"norm_rope": _plain_norm, "norm_rope_bwd": _plain_norm_bwd, "linattn": _plain_fwd,
            "linattn_bwd": _plain_bwd, "linattn_step": _plain_step, "gdn_step": _plain_step}[op](state)


# ------------------------------------------------------------------------------ work, exact
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    H, HK, D = c["H"], c["HK"], c["D"]
    if c["op"].startswith("norm_rope"):
        rows = c["B"] * c["T"]
        el = rows * (H + HK) * D
        small = rows * c["axes"] * 4 + rows * c["rot"] * 4 + 2 * D * 4
        n = 2 if c["op"] == "norm_rope" else 3
        return {"bytes": n * el * e + small, "flops": (8 if n == 2 else 16) * el}
    if c["op"].endswith("step"):
        N = c["N"] - c["pad"] if c["N"] > c["pad"] else max(1, c["N"] - 1)
        return {"bytes": N * (8 * H * D * D + (2 * HK + 2 * H) * D * e),
                "flops": N * H * D * D * (5 if c["op"] == "linattn_step" else 7)}
    N = c["packed"] or c["B"]
    rows = c["B"] * c["T"]
    states = N * H * D * D * 4
    if c["op"] == "linattn":
        return {"bytes": rows * (2 * HK + 2 * H) * D * e + states * (2 if c["s0"] else 1),
                "flops": rows * H * 4 * D * D}
    return {"bytes": rows * (4 * HK + 3 * H) * D * e + states * (3 if c["s0"] else 2),
            "flops": rows * H * 10 * D * D}


def _exact_scan(x, y, z, decay, S, scale, read_shift, write_shift, scale_src):
    """64-bit walk over the tokens [T,H,D] of one sequence, EXACT_CHUNK at a time:
    out_i = scale sum_{j<=i} lam^(i-j) (x_i.y_j) z_j + lam^(i+1-read_shift) S x_i (times scale
    where the sources are not scaled), the state S [H,Z,Y] advancing with it."""
    T = x.shape[0]
    out = torch.zeros(T, *z.shape[1:], dtype=torch.float64, device="cuda")
    rs = 1.0 if scale_src else scale
    for t in range(0, T, EXACT_CHUNK):
        a, b, c = x[t:t + EXACT_CHUNK], y[t:t + EXACT_CHUNK], z[t:t + EXACT_CHUNK]
        L = a.shape[0]
        i = torch.arange(L, device="cuda", dtype=torch.float64)
        gap = i[:, None] - i
        w = torch.exp(decay[:, None, None] * gap.clamp_min(0)).tril()
        p = torch.matmul(a.transpose(0, 1), b.permute(1, 2, 0)) * w * scale          # [H,i,j]
        o = torch.matmul(p, c.transpose(0, 1))
        rd = torch.exp(decay[:, None] * (i + 1 - read_shift)) * rs                   # [H,i]
        o = o + torch.matmul(a.transpose(0, 1), S.transpose(1, 2)) * rd[..., None]
        out[t:t + L] = o.transpose(0, 1)
        wr = torch.exp(decay[:, None] * (L - 1 - i + write_shift))                   # [H,j]
        if scale_src:
            wr = wr * scale
        S = S * torch.exp(decay * L)[:, None, None] + torch.matmul(
            c.permute(1, 2, 0) * wr[:, None], b.transpose(0, 1))
    return out, S


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    H, HK, D = c["H"], c["HK"], c["D"]
    G, scale = H // HK, D ** -0.5
    op = c["op"]
    if op.startswith("norm_rope"):
        half = c["rot"] // 2
        bounds = np.cumsum([0] + s["sections"])
        res = {}
        angle = torch.empty(c["B"] * c["T"], half, 2, dtype=torch.float64, device="cuda")
        for a in range(c["axes"]):
            lo, hi = int(bounds[a]), int(bounds[a + 1])
            angle[:, lo:hi] = s["table"].double()[s["pos"][a].long(), lo:hi]
        rotor = torch.view_as_complex(angle).view(c["B"], c["T"], 1, half)

        def turn(x, r):
            head = x[..., :c["rot"]]
            pair = head.unflatten(-1, (half, 2)) if c["interleaved"] else head.unflatten(
                -1, (2, half)).transpose(-1, -2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * r)
            w = w.flatten(-2) if c["interleaved"] else w.transpose(-1, -2).flatten(-2)
            return torch.cat([w, x[..., c["rot"]:]], -1)

        for n in ("q", "k"):
            x, w = s[n].double(), s[n + "w"].double()
            ss = (x * x).sum(-1, keepdim=True)
            size = (ss / D + EPS).sqrt() if c["norm"] == "rms" else ss.sqrt().clamp_min(EPS)
            if op == "norm_rope":
                res[n] = turn(x / size * w, rotor)
                continue
            dy = turn(s["d" + n].double(), rotor.conj())
            unit = x / size
            gw = dy * w
            along = (gw * unit).sum(-1, keepdim=True)
            if c["norm"] == "rms":
                along = along / D
            else:
                along = torch.where(ss.sqrt() > EPS, along, 0.0)
            res["d" + n] = (gw - unit * along) / size
            res["d" + n + "w"] = (dy * unit).flatten(0, 2).sum(0)
        return res
    if op.endswith("step"):
        idx = s["idx"].tolist()
        cache = s["cache"].double()
        out = torch.zeros(c["N"], H, D, dtype=torch.float64, device="cuda")
        for n, slot in enumerate(idx):
            if slot <= 0:
                continue
            q, k = (s[m][n].double().repeat_interleave(G, 0) for m in ("q", "k"))
            v = s["v"][n].double()
            if op == "gdn_step":
                S = cache[slot] * s["gate"][n].double().exp()[:, None, None]
                v = s["beta"][n].double()[:, None] * (v - torch.einsum("hvk,hk->hv", S, k))
            else:
                S = cache[slot] * s["decay"].double().exp()[:, None, None]
            S = S + torch.einsum("hv,hk->hvk", v, k)
            cache[slot] = S
            out[n] = scale * torch.einsum("hvk,hk->hv", S, q)
        return dict(out=out, cache=cache)
    decay = s["decay"].double()
    N = len(s["lens"])
    zero = torch.zeros(H, D, D, dtype=torch.float64, device="cuda")
    q, k = (s[m].double().repeat_interleave(G, 2) for m in ("q", "k"))
    v = s["v"].double()
    names = ("out",) if op == "linattn" else ("dq", "dk", "dv")
    res = {m: torch.zeros(c["B"], c["T"], H, D, dtype=torch.float64, device="cuda") for m in names}
    state = torch.zeros(N, H, D, D, dtype=torch.float64, device="cuda")
    at = 0
    for n, L in enumerate(s["lens"]):
        b, lo = (0, at) if c["packed"] else (n, 0)
        at += L
        row = slice(lo, lo + L)
        S0 = zero if s["s0"] is None else s["s0"][n].double()
        qs, ks, vs = q[b, row], k[b, row], v[b, row]
        if op == "linattn":
            res["out"][b, row], state[n] = _exact_scan(qs, ks, vs, decay, S0, scale, 0, 0, False)
            continue
        do, dS = s["dout"][b, row].double(), s["dfin"][n].double()
        r = lambda x: x.flip(0)   # noqa: E731
        res["dq"][b, row] = _exact_scan(do, vs, ks, decay, S0.transpose(1, 2), scale, 0, 0, False)[0]
        dv, state[n] = _exact_scan(r(ks), r(qs), r(do), decay, dS, scale, 1, 1, True)
        dk, _ = _exact_scan(r(vs), r(do), r(qs), decay, dS.transpose(1, 2), scale, 1, 1, True)
        res["dv"][b, row], res["dk"][b, row] = r(dv), r(dk)
    if op == "linattn":
        return dict(out=res["out"], final_state=state)
    for m in ("dq", "dk"):
        res[m] = res[m].unflatten(2, (HK, G)).sum(3)
    return dict(**res, d_initial_state=state)
