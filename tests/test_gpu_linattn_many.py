"""Many packed sequences, a few of them cut into segments: the places of the sequences' segments,
pieces and entry states are found 32 sequences at a time, and the remainders of up to 64 sequences
are handed out by their lengths.  Tolerances of test_gpu_linattn."""
import numpy as np
import pytest
import torch

from test_gpu_linattn import BF16, F32, STATE, TOL, err, inputs, ref_bwd, ref_fwd, run_fwd

pytestmark = pytest.mark.gpu


def lengths_of(N, long):
    """Short sequences (empty ones and ones of a token among them) around the long ones."""
    n = [(7 * i) % 23 if i % 5 else i % 2 for i in range(N)]
    for at, length in long:
        n[at] = length
    return n


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("N,H,long", [(40, 2, [(35, 1500)]), (100, 2, [(0, 900), (34, 2000), (70, 1500)]),
                                      (70, 1, [(31, 1024), (32, 1025), (69, 900)])])
def test_long_sequences_among_many_short_ones(dtype, D, N, H, long):
    import chunked_linear_recurrence_gb300 as sf
    lengths = lengths_of(N, long)
    T = sum(lengths)
    x = inputs(1, T + 3, H, 1, D, dtype, seed=N + D, lengths=lengths, decay=[-0.003, -0.2][:H])
    rows = np.arange(T)
    ro, rf = ref_fwd(x)
    out, fin = run_fwd(x)
    assert err(out, ro, rows) <= TOL[dtype]
    for n in range(N):
        assert err(fin[n], rf[n]) <= STATE, n
    g = sf.sf_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["s0"], x["do"], x["df"], cu_seqlens=x["cu"])
    rg = ref_bwd(x)
    for n in ("dq", "dk", "dv"):
        assert err(g[n], rg[n], rows) <= TOL[dtype], n
    for n in range(N):
        assert err(g["d_initial_state"][n], rg["d_initial_state"][n]) <= STATE, n


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_many_sequences_of_which_none_is_cut(dtype, D):
    """On a pool, with padding between them."""
    import chunked_linear_recurrence_gb300 as sf
    N, H = 100, 2
    lengths = [20 + i % 3 for i in range(N)]
    x = inputs(1, sum(lengths), H, 2, D, dtype, seed=7 + D, lengths=lengths)
    ro, rf = ref_fwd(x)
    idx = torch.randperm(N, generator=torch.Generator().manual_seed(1)).to(torch.int32) + 1
    idx[10::7] = -1
    cache = torch.zeros(N + 1, H, D, D, device="cuda")
    live = idx > 0
    cache[idx[live].long().cuda()] = x["s0"][live.cuda()]
    out = sf.sf_linattn_paged_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], cache, idx.cuda(), cu_seqlens=x["cu"])
    cu = x["cu"].tolist()
    for n in range(N):
        if live[n]:
            assert err(out, ro, np.arange(cu[n], cu[n + 1])) <= TOL[dtype], n
            assert err(cache[int(idx[n])], rf[n]) <= STATE, n
        else:
            assert not out[:, cu[n]:cu[n + 1]].any()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_offsets_are_free_for_reuse_when_a_call_is_over(dtype, D):
    """No walk of the first call is cut, all of the second's offsets are written over the first's
    right behind it, and one walk of those is: neither launch of the first may still read them."""
    import chunked_linear_recurrence_gb300 as sf
    T = 1536
    even, ragged = [48] * 32, [3] * 31 + [T - 93]
    x = inputs(1, T, 1, 1, D, dtype, seed=3, lengths=even, decay=[-0.01])
    y = dict(x, cu=torch.tensor([0] + list(np.cumsum(ragged)), dtype=torch.int32, device="cuda"))
    a, b = run_fwd(x), run_fwd(y)
    ws = sf.sf_linattn_fwd_workspace(x["q"], x["v"], x["cu"])
    cu = x["cu"].clone()
    for _ in range(20):
        cu.copy_(x["cu"])
        first = run_fwd(dict(x, cu=cu), ws=ws)
        cu.copy_(y["cu"])
        second = run_fwd(dict(x, cu=cu), ws=ws)
        assert all(map(torch.equal, first, a)) and all(map(torch.equal, second, b))
