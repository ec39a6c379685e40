"""A linear-attention layer trained, prefilled and decoded with this package's operators.

    python examples/linear_attention_layer.py

The layer projects its input to queries, keys and values in one matrix product, norms and
rotates the query and key heads (``sf_qk_norm_rope_*``), runs the decayed linear attention
(``sf_linattn_*``) and projects back.  The script takes gradient steps on a copying task,
prefills ragged prompts into a paged pool of states, continues them token by token, and checks
that the continuation equals one prefill over the whole sequences.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_linear_recurrence_gb300 as sf  # noqa: E402


class _NormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, qw, kw, table, pos):
        ctx.save_for_backward(q, k, qw, kw, table, pos)
        return sf.sf_qk_norm_rope_fwd(q, k, qw, kw, table, pos)

    @staticmethod
    def backward(ctx, dq, dk):
        g = sf.sf_qk_norm_rope_bwd(*ctx.saved_tensors, dq.contiguous(), dk.contiguous())
        return g["dq"], g["dk"], g["dq_weight"], g["dk_weight"], None, None


class _LinAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay):
        ctx.save_for_backward(q, k, v, decay)
        return sf.sf_linattn_chunk_fwd(q, k, v, decay)[0]

    @staticmethod
    def backward(ctx, d_out):
        q, k, v, decay = ctx.saved_tensors
        g = sf.sf_linattn_chunk_bwd(q, k, v, decay, None, d_out.contiguous(),
                                    want_d_initial_state=False)
        return g["dq"], g["dk"], g["dv"], None


class Layer(torch.nn.Module):
    """Linear attention with H value heads, HK query/key heads and a fixed decay of each head."""

    def __init__(self, width=512, H=4, HK=2, D=128, max_pos=4096):
        super().__init__()
        self.H, self.HK, self.D = H, HK, D
        kw = dict(device="cuda", dtype=torch.bfloat16)
        self.inp = torch.nn.Linear(width, (2 * HK + H) * D, bias=False, **kw)
        self.out = torch.nn.Linear(H * D, width, bias=False, **kw)
        self.qw = torch.nn.Parameter(torch.ones(D, device="cuda"))
        self.kw = torch.nn.Parameter(torch.ones(D, device="cuda"))
        self.register_buffer("decay", -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H))
        a = torch.arange(max_pos, device="cuda")[:, None] * 1e4 ** (
            -torch.arange(D // 2, device="cuda") / (D // 2))
        self.register_buffer("table", torch.stack([a.cos(), a.sin()], -1).contiguous())

    def heads(self, x, pos):
        """q, k (normed and rotated) and v of x [B,T,width] at the positions pos [B*T]."""
        B, T, _ = x.shape
        n = self.HK * self.D
        qkv = self.inp(x)
        q, k = (qkv[..., i * n:(i + 1) * n].view(B, T, self.HK, self.D) for i in (0, 1))
        v = qkv[..., 2 * n:].view(B, T, self.H, self.D).contiguous()
        q, k = _NormRope.apply(q, k, self.qw, self.kw, self.table, pos)
        return q, k, v

    def forward(self, x):
        B, T, _ = x.shape
        pos = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B)
        return self.out(_LinAttn.apply(*self.heads(x, pos), self.decay).flatten(2))

    @torch.no_grad()
    def prefill(self, x, cu_seqlens, pool, slots):
        """Packed prompts x [1,T,width] into the pool's slots, from empty states."""
        cu = cu_seqlens.tolist()
        pos = torch.cat([torch.arange(b - a, dtype=torch.int32) for a, b in zip(cu, cu[1:])]).cuda()
        fresh = torch.zeros(len(slots), dtype=torch.bool, device="cuda")
        o = sf.sf_linattn_paged_chunk_fwd(*self.heads(x, pos), self.decay, pool, slots,
                                          cu_seqlens=cu_seqlens, has_initial_state=fresh)
        return self.out(o.flatten(2))

    @torch.no_grad()
    def step(self, x, pos, pool, slots):
        """The next token x [N,width] of every sequence, at the positions pos [N]."""
        q, k, v = (t[:, 0].contiguous() for t in self.heads(x[:, None], pos))
        return self.out(sf.sf_linattn_step(q, k, v, self.decay, pool, slots).flatten(1))


def main():
    torch.manual_seed(0)
    layer = Layer()
    opt = torch.optim.SGD(layer.parameters(), lr=0.05)
    x = torch.randn(2, 200, 512, device="cuda", dtype=torch.bfloat16)
    losses = []
    for _ in range(8):                                   # learn to hand the input through
        loss = (layer(x).float() - x.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print("loss", " ".join("%.4f" % v for v in losses))
    assert losses[-1] < losses[0]

    prompt, more = [130, 1, 77], 5                       # ragged prompts, five tokens each after
    seqs = [torch.randn(n + more, 512, device="cuda", dtype=torch.bfloat16) for n in prompt]

    def offsets(lengths):
        return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32).cuda()

    pool = torch.full((6, layer.H, layer.D, layer.D), float("nan"), device="cuda")
    slots = torch.tensor([4, 1, 3], dtype=torch.int32, device="cuda")
    layer.prefill(torch.cat([s[:n] for s, n in zip(seqs, prompt)])[None], offsets(prompt), pool, slots)
    for t in range(more):
        pos = torch.tensor([n + t for n in prompt], dtype=torch.int32, device="cuda")
        last = layer.step(torch.stack([s[n + t] for s, n in zip(seqs, prompt)]), pos, pool, slots)
    whole = torch.zeros_like(pool)
    cu = offsets([n + more for n in prompt])
    out = layer.prefill(torch.cat(seqs)[None], cu, whole, slots)[0]
    want = out[(cu[1:] - 1).long()]
    err = ((last - want).float().norm() / want.float().norm()).item()
    drift = ((pool - whole)[slots.long()].norm() / whole[slots.long()].norm()).item()
    print("decoded against prefilled: outputs %.1e, states %.1e" % (err, drift))
    # the outputs' BF16 roundings, the states' FP32 ones
    assert err < 1e-2 and drift < 1e-4
    print("ok")


if __name__ == "__main__":
    main()
