"""Verification of drafted tokens on the GPU against the FP64 oracle.  Tokens are whole numbers
and have to be equal: the tests and sums behind them are exact to 2^-40, the oracle's to 2^-49 or
so, and the inputs' uniforms are at random (a draw differs if its uniform lies within that of a
border between two tokens: 1e-12 times the number of tokens)."""
import pytest
import torch

from helpers import f64
from oracle import decode as od

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(N, T, V, dtype, drafts, seed, heat=2.0, noise=0.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, T + 1, V, generator=g) * heat
    target = z.softmax(-1).to(dtype)
    q = (z[:, :T] + noise * torch.randn(N, T, V, generator=g)).softmax(-1).to(dtype)
    x = torch.zeros(N, T, dtype=torch.int32)
    if T and drafts:
        x = torch.multinomial(q.float().flatten(0, 1), 1, generator=g).view(N, T).int()
    elif T:
        x = q.argmax(-1).int()
    d = dict(target=target, x=x, u=torch.rand(N, T + 1, generator=g), draft=q if drafts else None,
             num=torch.randint(0, T + 1, (N,), generator=g, dtype=torch.int32))
    return {m: None if t is None else t.cuda() for m, t in d.items()}


def call(d, **kw):
    import chunked_linear_recurrence_gb300 as sf
    return sf.sf_draft_verify(d["target"], d["x"], d["u"], draft_probs=d["draft"], num_drafts=d["num"], **kw)


def check(d, got):
    tok, num = od.verify(f64(d["target"]), d["x"].tolist(), f64(d["u"]), None if d["draft"] is None else f64(d["draft"]),
                         None if d["num"] is None else d["num"].tolist())
    assert got[0].tolist() == tok.tolist() and got[1].tolist() == num.tolist()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("N,T,V", [(1, 0, 1), (1, 1, 1), (3, 0, 7), (2, 1, 33), (5, 3, 1000), (4, 8, 32000), (40, 4, 4099),
                                   (3, 40, 257), (200, 2, 513), (600, 1, 100), (1, 2, 200003)])
def test_verify(N, T, V, drafts, dtype):
    d = make(N, T, V, dtype, drafts, N + T + V)
    check(d, call(d))
    d["num"] = None
    check(d, call(d))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_likely_drafts_are_accepted_to_the_end(dtype):
    """All, none and every number of drafts in between, across a warp's width."""
    N, T, V = 66, 65, 90
    d = make(N, T, V, dtype, True, 1, noise=0.0)
    d["num"] = None
    d["u"].clamp_max_(0.99)                          # p = q: accepted
    for n in range(N):
        if n < T:
            d["u"][n, n] = 1.0                       # u q < p fails: the first rejection
    got = call(d)
    assert got[1].tolist() == [min(n, T) + 1 for n in range(N)]
    check(d, got)


def test_nothing_left_is_drawn_from_the_target():
    """A draft with at least the target's probability everywhere, and a rejected token."""
    d = make(6, 2, 500, F32, True, 2)
    d["draft"] = d["target"][:, :2] * 1.5
    d["u"][:, :2] = 0.9
    d["num"] = None
    got = call(d)
    assert got[1].tolist() == [1] * 6
    check(d, got)


def test_uniforms_at_their_ends_take_tokens_with_weight():
    d = make(8, 1, 3000, F32, True, 3)
    w = torch.zeros(3000)
    w[1234:1300] = torch.rand(66)
    w[1299] = 0.5
    d["target"][:] = w.cuda()
    d["u"][:, 1] = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan"), float("inf"), 0.5])
    d["num"] = torch.zeros(8, dtype=torch.int32, device="cuda")
    tok = call(d)[0][:, 0].tolist()
    assert tok[0] == 1234 and tok[4] == 1234 and tok[1:4] == [1299] * 3 and tok[5:7] == [1299] * 2
    check(d, call(d))


def test_bad_probabilities_and_tokens():
    d = make(9, 2, 700, F32, True, 4)
    d["num"] = torch.tensor([2, 2, 2, 2, -1, 99, 0, 2, 2], dtype=torch.int32, device="cuda")
    d["x"][0, 0], d["x"][1, 0] = -1, 700                       # not in the vocabulary
    d["target"][2, 0, ::3] = float("nan")
    d["target"][3, 0, ::3] *= -1
    d["target"][6, 0] = 0.0                                    # nothing to draw from
    d["target"][7, 0, 5] = float("inf")
    d["x"][7, 0], d["u"][7, 0] = 9, 1.0
    d["draft"][8, 0, ::2] = float("nan")
    d["u"][8, 0] = 1.0
    got = call(d)
    assert got[1][4] == 0 and (got[0][4] == -1).all() and got[0][6, 0] == -1
    check(d, got)


def test_an_infinite_weight_draws_nothing():
    d = make(2, 2, 700, F32, True, 10)
    d["num"] = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    d["target"][:, 0, 5] = float("inf")
    d["x"][1, 0], d["target"][1, 0, 9] = 9, 0.0                # rejected
    got = call(d)
    assert got[0].tolist() == [[-1] * 3] * 2 and got[1].tolist() == [1, 1]
    check(d, got)


def test_drafts_without_probabilities_and_out_of_the_vocabulary():
    d = make(4, 3, 50, F32, False, 5)
    d["num"] = None
    d["x"][0, 0], d["x"][1, 0] = -5, 50
    d["u"][2, 0] = 1.0
    d["target"][3, 0] = 0.0
    d["target"][3, 0, 7] = 1.0
    d["x"][3, 0], d["u"][3, 0] = 7, 1.0                        # rejected, and nothing else has weight
    got = call(d)
    assert got[0][3, 0] == 7
    check(d, got)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_a_larger_buffer(dtype):
    """Strided rows and sequences, at every alignment."""
    N, T, V = 7, 3, 1001
    d = make(N, T, V, dtype, True, 6)
    want = call(d)
    for shift in range(8):
        a = torch.full((N, T + 2, V + 40), float("nan"), dtype=dtype, device="cuda")[:, 1:, shift:shift + V]
        b = torch.full((T, N, V + 13), float("nan"), dtype=dtype, device="cuda")[:, :, 7 - shift:7 - shift + V].transpose(0, 1)
        a.copy_(d["target"])
        b.copy_(d["draft"])
        got = call(dict(d, target=a, draft=b))
        assert all(map(torch.equal, got, want))


def test_unnormalised_weights_give_the_same_tokens():
    """Times a power of two nothing changes, neither large nor small."""
    d = make(9, 3, 2000, F32, True, 7)
    want = call(d)
    for s in (2.0 ** 60, 2.0 ** -60):
        got = call(dict(d, target=d["target"] * s, draft=d["draft"] * s))
        assert all(map(torch.equal, got, want))


def test_probabilities_of_more_than_2_31_elements():
    N, T, V = 12, 1, 100_000_000
    target = torch.zeros(N, T + 1, V, dtype=BF16, device="cuda")
    assert target.numel() > 1 << 31
    at = [V - 1 - 7 * n for n in range(N)]
    for n in range(N):
        target[n, 0, at[n]] = 1.0
        target[n, 1, at[n] - 1] = 0.5
    x = torch.tensor(at, dtype=torch.int32, device="cuda")[:, None].contiguous()
    import chunked_linear_recurrence_gb300 as sf
    tok, num = sf.sf_draft_verify(target, x, torch.full((N, 2), 0.5, device="cuda"))
    assert num.tolist() == [2] * N and tok.tolist() == [[a, a - 1] for a in at]


def test_replayed_in_a_graph_and_on_another_stream():
    d = make(5, 3, 3001, F32, True, 8)
    e = make(5, 3, 3001, F32, True, 9)
    call(d)
    y = {m: t.clone() for m, t in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(y)
    for src in (d, e, d):
        for m in y:
            y[m].copy_(src[m])
        graph.replay()
        torch.cuda.synchronize()
        check(src, got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(e, stream=side)
    side.synchronize()
    check(e, got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("N,T,V", [(1, 3, 65536), (40, 2, 65537), (90, 1, 70001), (400, 1, 65535), (320, 1, 65543)])
def test_long_rows(N, T, V, drafts, dtype):
    """On either side of the length that takes more warps, with clusters of eight down to one."""
    d = make(N, T, V, dtype, drafts, N + V)
    check(d, call(d))
