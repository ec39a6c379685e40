"""Copies, forks and compaction of the pool on the GPU: whole numbers and copied bits, so
everything is equal to the oracle's."""
import numpy as np
import pytest
import torch

from oracle import decode as od

pytestmark = pytest.mark.gpu


def pool(slots, seed, sizes=((2, 64, 64),), dtypes=(torch.float32,)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(slots, *s, generator=g, device="cuda").to(d) for s, d in zip(sizes, dtypes)]


def i32(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


def moved(caches, moves):
    want = [c.clone() for c in caches]
    for to, s in moves.items():
        for w, c in zip(want, caches):
            w[to] = c[s]
    return want


def mask(slots, reserved):
    m = torch.zeros(slots, dtype=torch.bool, device="cuda")
    for s in reserved:
        m[s] = True
    return m


SIZES = [(((2, 64, 64),), (torch.float32,)),
         (((1, 128, 128), (3, 8), (5, 24)), (torch.float32, torch.bfloat16, torch.float16)),
         (((4, 128, 128), (8,)), (torch.float32, torch.int16))]


@pytest.mark.parametrize("sizes", range(3))
@pytest.mark.parametrize("seed", range(12))
def test_fork_and_compact_of_random_pools(seed, sizes):
    import chunked_linear_recurrence_gb300 as sf
    r = np.random.RandomState(seed)
    slots = int(r.choice([2, 3, 9, 31, 32, 33, 64, 65, 100]))
    reserved = [int(s) for s in r.randint(0, slots, r.randint(0, 4))] if seed % 2 else []
    idx = r.randint(-1, slots + 2, r.randint(1, slots + 5))          # padding, past the pool, shared slots
    parents = r.randint(-1, len(idx) + 1, r.randint(1, slots + 5))
    caches = pool(slots, seed, *SIZES[sizes])
    res = mask(slots, reserved) if seed % 2 else None
    new, copies = od.fork(idx, parents, slots, reserved)
    want = moved(caches, copies)
    got = sf.sf_state_fork(caches if seed % 3 else caches[0], i32(idx), i32(parents), reserved=res)
    assert got.tolist() == new
    assert all(map(torch.equal, caches if seed % 3 else caches[:1], want))

    new, moves = od.compact(idx, slots, reserved)
    want = moved(caches, moves)
    got = sf.sf_state_compact(caches, i32(idx), reserved=res)
    assert got.tolist() == new and all(map(torch.equal, caches, want))


@pytest.mark.parametrize("slots,rows", [(5000, 3000), (40000, 2500), (1 << 18, 1025)])
def test_large_pools(slots, rows):
    """More slots and rows than the plan has threads, and more slots than its shared memory holds
    numbers of."""
    import chunked_linear_recurrence_gb300 as sf
    r = np.random.RandomState(rows)
    idx = r.randint(1, slots, rows)
    parents = r.randint(0, rows, rows + 77)
    reserved = [int(s) for s in r.randint(1, slots, slots // 3)]
    caches = [torch.arange(slots * 4, device="cuda").view(slots, 4)]
    new, copies = od.fork(idx, parents, slots, reserved)
    want = moved(caches, {})
    if copies:
        want[0][torch.tensor(list(copies))] = caches[0][torch.tensor(list(copies.values()))]
    got = sf.sf_state_fork(caches, i32(idx), i32(parents), reserved=mask(slots, reserved))
    assert got.tolist() == new and torch.equal(caches[0], want[0])
    new, moves = od.compact(idx, slots, reserved)
    if moves:
        want[0][torch.tensor(list(moves))] = want[0][torch.tensor(list(moves.values()))]
    got = sf.sf_state_compact(caches, i32(idx), reserved=mask(slots, reserved))
    assert got.tolist() == new and torch.equal(caches[0], want[0])


def test_compact_edges():
    import chunked_linear_recurrence_gb300 as sf
    for slots in (2, 32, 33, 64, 1000):
        for idx in ([slots - 1], list(range(1, slots)), list(range(slots - 1, 0, -2)), [-1, 0, slots], [1, 1, slots - 1]):
            caches = pool(slots, 1, ((8,),))
            new, moves = od.compact(idx, slots)
            want = moved(caches, moves)
            assert sf.sf_state_compact(caches, i32(idx)).tolist() == new and torch.equal(caches[0], want[0])


def test_no_slot_left():
    """Rows that no slot is left for get -1, in the rows' order, and nothing else is touched."""
    import chunked_linear_recurrence_gb300 as sf
    caches = pool(5, 2)
    before = caches[0].clone()
    got = sf.sf_state_fork(caches, i32([3]), i32([0] * 6), reserved=mask(5, [1]))
    assert got.tolist() == [3, 2, 4, -1, -1, -1]
    assert torch.equal(caches[0][[0, 1, 3]], before[[0, 1, 3]])
    assert torch.equal(caches[0][2], before[3]) and torch.equal(caches[0][4], before[3])


def test_in_place_indices_and_a_kept_workspace():
    import chunked_linear_recurrence_gb300 as sf
    caches = pool(70, 3)
    ws = sf.sf_state_workspace(caches, 40)
    ws.fill_(255)
    idx = i32(range(30, 70))
    parents = i32([i // 2 for i in range(40)])
    new, copies = od.fork(idx.tolist(), parents.tolist(), 70)
    want = moved(caches, copies)
    assert sf.sf_state_fork(caches, idx, parents, out=idx, ws=ws) is idx
    assert idx.tolist() == new and torch.equal(caches[0], want[0])
    new, moves = od.compact(new, 70)
    want = moved(caches, moves)
    sf.sf_state_compact(caches, idx, out=idx, ws=ws)
    assert idx.tolist() == new and torch.equal(caches[0], want[0])
    par = i32([5, 5, 7])
    new, _ = od.fork(idx.tolist(), [5, 5, 7], 70)
    sf.sf_state_fork(caches, idx, par, out=par)
    assert par.tolist() == new


def test_no_rows_and_no_sequences():
    import chunked_linear_recurrence_gb300 as sf
    caches = pool(4, 4)
    before = caches[0].clone()
    none = i32([])
    assert sf.sf_state_fork(caches, i32([1]), none).tolist() == []
    assert sf.sf_state_fork(caches, none, i32([0, -1])).tolist() == [-1, -1]
    assert sf.sf_state_compact(caches, none).tolist() == []
    sf.sf_state_copy(caches, none, none)
    assert torch.equal(caches[0], before)


def test_copy_skips_padding():
    import chunked_linear_recurrence_gb300 as sf
    caches = pool(9, 5, *SIZES[1])
    want = moved(caches, {5: 2, 6: 2})
    sf.sf_state_copy(caches, i32([2, 2, 0, -1, 9, 3, 3, 4, 1 << 30]), i32([5, 6, 7, 8, 8, 0, 9, 4, 7]))
    assert all(map(torch.equal, caches, want))


def test_more_caches_than_a_launch_takes():
    import chunked_linear_recurrence_gb300 as sf
    caches = pool(6, 6, ((8,),) * 70, (torch.float32,) * 70)
    want = moved(caches, {1: 5, 2: 5})
    assert sf.sf_state_fork(caches, i32([5]), i32([0, 0, 0])).tolist() == [5, 1, 2]
    assert all(map(torch.equal, caches, want))


def test_a_pool_of_more_than_4_gb():
    import chunked_linear_recurrence_gb300 as sf
    cache = torch.zeros(4200, 32, 64, 128, dtype=torch.float32, device="cuda")
    assert cache.numel() * 4 > 1 << 32
    cache[4198] = torch.randn(32, 64, 128, device="cuda")
    cache[4199] = torch.randn(32, 64, 128, device="cuda")
    a, b = cache[4198].clone(), cache[4199].clone()
    assert sf.sf_state_compact(cache, i32([4199, 4198])).tolist() == [2, 1]
    assert torch.equal(cache[1], a) and torch.equal(cache[2], b)
    sf.sf_state_copy(cache, i32([1]), i32([4197]))
    assert torch.equal(cache[4197], a) and torch.equal(cache[4198], a) and not cache[4196].any()


def test_replayed_in_a_graph_and_on_another_stream():
    import chunked_linear_recurrence_gb300 as sf
    caches = pool(40, 7)
    idx, parents = i32(range(1, 21)), i32([0] * 10 + list(range(10)))
    sf.sf_state_fork(pool(40, 8), idx, parents)
    x = [c.clone() for c in caches]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mid = sf.sf_state_fork(x, idx, parents)
        got = sf.sf_state_compact(x, mid)
    for seed in range(3):
        r = np.random.RandomState(seed)
        idx.copy_(i32(r.permutation(39)[:20] + 1))
        parents.copy_(i32(r.randint(-1, 20, 20)))
        for a, c in zip(x, caches):
            a.copy_(c)
        new, copies = od.fork(idx.tolist(), parents.tolist(), 40)
        want = moved(caches, copies)
        new, moves = od.compact(new, 40)
        want = moved(want, moves)
        graph.replay()
        torch.cuda.synchronize()
        assert got.tolist() == new and torch.equal(x[0], want[0])
    side = torch.cuda.Stream()
    x = [c.clone() for c in caches]
    side.wait_stream(torch.cuda.current_stream())
    got = sf.sf_state_fork(x, idx, parents, stream=side)
    side.synchronize()
    new, copies = od.fork(idx.tolist(), parents.tolist(), 40)
    assert got.tolist() == new and torch.equal(x[0], moved(caches, copies)[0])


def test_more_rows_than_a_plan_in_every_cta_takes():
    """Both forms of the move, side by side: in place, and with the new indices apart, on either side
    of the sizes where the plan is made once."""
    import chunked_linear_recurrence_gb300 as sf
    for slots, rows in ((4096, 1024), (4097, 1024), (4096, 1025), (4100, 1100)):
        r = np.random.RandomState(slots + rows)
        idx = i32(r.randint(-1, slots + 1, rows))
        parents = i32(r.randint(-1, rows + 1, rows))
        res = mask(slots, r.randint(1, slots, 50))
        a = torch.arange(slots * 4, device="cuda").view(slots, 4)
        b, at = a.clone(), idx.clone()
        new, copies = od.fork(idx.tolist(), parents.tolist(), slots, set(res.nonzero()[:, 0].tolist()))
        got = sf.sf_state_fork(a, idx, parents, reserved=res)
        sf.sf_state_fork(b, at, parents, reserved=res, out=at)
        assert got.tolist() == new and torch.equal(got, at) and torch.equal(a, b)
        new, _ = od.compact(got.tolist(), slots, set(res.nonzero()[:, 0].tolist()))
        got = sf.sf_state_compact(a, got, reserved=res)
        sf.sf_state_compact(b, at, reserved=res, out=at)
        assert got.tolist() == new and torch.equal(got, at) and torch.equal(a, b)
