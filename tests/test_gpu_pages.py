"""The page operators on the GPU against a plain implementation with Python lists."""
import ctypes
import random
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_linear_attention_gla_gb300 import build as glabuild
    glabuild.build()
    import gated_linear_attention_gla_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_pools(S, seed=1):
    """Page sizes of one vector, of odd numbers of vectors, and above a copy block's 32 KB."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [r(S, 4), r(S, 3, 8).to(torch.bfloat16), r(S, 2, 65, 68), r(S, 36)]


def fork_ref(used, parents):
    free = [p for p, x in enumerate(used) if not x]
    children, bad, used2 = [], False, list(used)
    for p in parents:
        ok = p == -2 or (0 <= p < len(used) and used[p])
        if ok and free:
            children.append(free.pop(0))
            used2[children[-1]] = 1
        else:
            bad |= p != -1
            children.append(-1)
    return children, used2, bad


def compact_ref(used):
    L = sum(1 for x in used if x)
    holes = [p for p in range(L) if not used[p]]
    forward = []
    for p, x in enumerate(used):
        forward.append(-1 if not x else p if p < L else holes.pop(0))
    return forward, [1] * L + [0] * (len(used) - L)


def synced(gla, bad):
    if bad:
        with pytest.raises(gla.GlaError) as e:
            gla.status_sync()
        assert e.value.status == 1
    gla.status_sync()


SIZES = [1, 2, 31, 64, 1023, 1024, 1025, 2500]


@pytest.mark.parametrize("S", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(gla, S, in_place):
    r = random.Random(S)
    for trial in range(4):
        used = [int(r.random() < (0.2, 0.6, 0.95, 0.0)[trial]) for _ in range(S)]
        live = [p for p in range(S) if used[p]]
        n = r.randint(0, S + 2)
        parents = [r.choice([-2, -1] + (live[:3] if live else []) + [r.choice(live) if live else -2])
                   for _ in range(n)]
        if trial == 1 and n > 2:
            parents[0], parents[n // 2] = S, r.randrange(S)     # out of the pool; perhaps a free page
        children, used2, bad = fork_ref(used, parents)
        pools = make_pools(S)
        want = [p.clone() for p in pools]
        for p, q in zip(parents, children):
            for w, o in zip(want, pools):
                if q >= 0:
                    w[q] = 0 if p == -2 else o[p]
        table = i32(used)
        got, out = gla.fork_pages(pools, table, i32(parents),
                                  used_out=None if in_place else torch.full_like(table, 5))
        synced(gla, bad)
        assert got.tolist() == children and out.tolist() == used2
        assert table.tolist() == (used2 if in_place else used)
        assert all(torch.equal(a, b) for a, b in zip(pools, want))


@pytest.mark.parametrize("S", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(gla, S, in_place):
    r = random.Random(S + 1)
    for share in (0.0, 0.1, 0.5, 0.9, 1.0):
        used = [7 * int(r.random() < share) for _ in range(S)]   # any value but 0 is used
        forward, used2 = compact_ref(used)
        slots = [p for p in range(S) if used[p]] + [-1]
        r.shuffle(slots)
        bad = share == 0.5 and S > 2
        if bad:
            slots += [S + 3, -7]
        pools = make_pools(S)
        want = [p.clone() for p in pools]
        for p, q in enumerate(forward):
            for w, o in zip(want, pools):
                if q >= 0:
                    w[q] = o[p]
        table, sl = i32(used), i32(slots)
        if in_place:
            s2, out, fwd = gla.compact_pages(pools, table, sl, slots_out=sl)
            assert s2 is sl and out is table
        else:
            s2, out, fwd = gla.compact_pages(pools, table, sl, used_out=torch.full_like(table, 5))
            assert table.tolist() == used and sl.tolist() == slots
        synced(gla, bad)
        assert fwd.tolist() == forward and out.tolist() == used2
        assert s2.tolist() == [forward[s] if 0 <= s < S else -1 for s in slots]
        assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copy(gla):
    S = 40
    src = [0, 0, 3, -1, 5, 7, 9, 9, 11, 12, 40, 2, 30]
    dst = [1, 2, 4, 6, -1, 8, 10, 10, 12, 13, 14, -3, 30]
    # page 10 is written twice; page 12 is written by one pair and read by another, so
    # that one is skipped (12 -> 13 is copied); page 2 is written by (0 -> 2) while
    # (2 -> -3) is no pair; 40 and -3 are outside
    copied = [1, 2, 4, -1, -1, 8, -1, -1, -1, 13, -1, -1, 30]
    pools = make_pools(S)
    want = [p.clone() for p in pools]
    for s, q in zip(src, copied):
        for w, o in zip(want, pools):
            if q >= 0:
                w[q] = o[s]
    got = gla.copy_pages(pools, i32(src), i32(dst))
    synced(gla, True)
    assert got.tolist() == copied
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    assert gla.copy_pages(pools, i32([]), i32([])).tolist() == []
    synced(gla, False)


def test_copy_many_pages_and_pools(gla):
    """More pages than the planning block has threads, more pools than one launch takes."""
    S = 3000
    g = torch.Generator(device="cuda").manual_seed(3)
    pools = [torch.randn(S, 8, generator=g, device="cuda") for _ in range(70)]
    perm = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    src, dst = perm[:1500].contiguous(), perm[1500:].contiguous()
    want = [p.clone() for p in pools]
    for w in want:
        w[dst.long()] = w[src.long()]
    assert torch.equal(gla.copy_pages(pools, src, dst), dst)
    synced(gla, False)
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_pages_far_into_a_large_pool(gla):
    """Byte offsets beyond 32 bits: 3 pages of 3 GiB."""
    n = 3 * 2 ** 30
    pool = torch.empty(3, n, dtype=torch.uint8, device="cuda")
    pool[0], pool[1], pool[2] = 1, 2, 3
    pool[2, -16:] = 9
    gla.copy_pages([pool], i32([2]), i32([1]))
    synced(gla, False)
    assert torch.equal(pool[1], pool[2]) and int(pool[0].max()) == 1


def test_free(gla):
    used = i32([1, 1, 0, 3, 1, 1])
    out = gla.free_pages(used, i32([3, -1, 0]), used_out=torch.empty_like(used))
    synced(gla, False)
    assert out.tolist() == [0, 1, 0, 0, 1, 1] and used.tolist() == [1, 1, 0, 3, 1, 1]
    for slots in ([2], [1, 1], [6], [-4]):                      # free already, twice, outside
        gla.free_pages(used.clone(), i32(slots))
        synced(gla, True)
    assert gla.free_pages(used, i32([0, 1, 3, 4, 5])) is used
    synced(gla, False)
    assert used.tolist() == [0] * 6


def test_serving_round_captured(gla):
    """Requests come, fork, finish and are compacted, captured once and replayed: the tables
    and pools follow the plain implementation, with the decode step on the pages between."""
    S, H, dk, dv = 16, 2, 64, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    pool = torch.randn(S, H, dk, dv, generator=g, device="cuda")
    tail = torch.randn(S, 3, 16, generator=g, device="cuda").to(torch.bfloat16)
    used = i32([1, 0, 1, 1, 0, 0, 1, 0, 0, 0, 0, 1, 0, 0, 0, 0])
    parents, done, slots = i32([3, -2, 3, -1]), i32([2, -1]), i32([0, 3, 6, 11, -1])
    q = torch.randn(5, H, dk, generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.full((5, H), -0.1, device="cuda")

    def round_():
        children, _ = gla.fork_pages([pool, tail], used, parents)
        gla.free_pages(used, done)
        table, _, forward = gla.compact_pages([pool, tail], used, slots)
        out = gla.decode_step(q, q, q, gate, pool, slots=table)
        return children, table, forward, out

    saved = [t.clone() for t in (pool, tail, used)]
    eager = [t.clone() for t in round_()]
    gla.status_sync()
    after = [t.clone() for t in (pool, tail, used)]
    u = saved[2].tolist()
    children, u, bad = fork_ref(u, parents.tolist())
    u[2] = 0
    forward, u = compact_ref(u)
    assert not bad and eager[0].tolist() == children and eager[2].tolist() == forward
    assert used.tolist() == u
    assert eager[1].tolist() == [forward[s] if s >= 0 else -1 for s in slots.tolist()]
    assert torch.equal(after[1][forward[11]], saved[1][11])
    for t, s in zip((pool, tail, used), saved):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = round_()
    graph.replay()
    gla.status_sync()
    assert all(torch.equal(a, b) for a, b in zip((pool, tail, used), after))
    assert all(torch.equal(a[:3], b[:3]) for a, b in zip(held, eager))


def test_copies_from_several_threads(gla):
    """Host threads copy in pools of different sizes at the same time; the plans of large pools need
    more shared memory than a kernel has without asking for it.  A captured copy replays behind them."""
    sizes, turns = [524_288, 140_000, 200_000], 20_000
    pools = [torch.arange(S, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4) for S in sizes]
    src, dst = [i32([S - 1, 7]) for S in sizes], [i32([3, S - 2]) for S in sizes]
    gla.copy_pages([pools[0]], src[0], dst[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gla.copy_pages([pools[0]], src[0], dst[0])
    streams, copied = [torch.cuda.Stream() for _ in sizes], [torch.empty_like(s) for s in src]
    torch.cuda.synchronize()
    results, gate = [set() for _ in sizes], threading.Barrier(len(sizes))

    def work(i):
        pool = gla._binding.PagePool(pools[i].data_ptr(), 16)
        call = (ctypes.byref(pool), 1, sizes[i], src[i].data_ptr(), dst[i].data_ptr(),
                copied[i].data_ptr(), 2, streams[i].cuda_stream)
        copy = gla.lib().gla_pages_copy
        gate.wait()
        for _ in range(turns):
            results[i].add(copy(*call))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert results == [{0}] * len(sizes)
    graph.replay()
    synced(gla, False)
    assert held.tolist() == dst[0].tolist()
    for S, p in zip(sizes, pools):
        assert p[3].tolist() == [S - 1] * 4 and p[S - 2].tolist() == [7] * 4 and p[4].tolist() == [4] * 4


def test_largest_tables(gla):
    """As many pages as a pool may have: fork, free, compact and copy against the plain implementation."""
    S = gla._binding.GLA_MAX_PAGES
    g = torch.Generator().manual_seed(55)
    used = (torch.rand(S, generator=g) < 0.6).int().tolist()
    pool = torch.arange(S, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4)
    live = [p for p in range(S) if used[p]]
    pick = torch.randint(0, len(live), (150_000,), generator=g).tolist()
    parents = [-2 if i % 5 == 0 else -1 if i % 7 == 0 else live[p] for i, p in enumerate(pick)]
    children, used2, bad = fork_ref(used, parents)
    assert not bad
    want = list(range(S))
    for p, q in zip(parents, children):
        if q >= 0:
            want[q] = 0 if p == -2 else p
    table = i32(used)
    got, _ = gla.fork_pages([pool], table, i32(parents))
    synced(gla, False)
    assert got.tolist() == children and table.tolist() == used2
    assert torch.equal(pool, i32(want)[:, None].expand(S, 4))
    done = live[::3]
    gla.free_pages(table, i32(done))
    for p in done:
        used2[p] = 0
    assert table.tolist() == used2
    forward, used3 = compact_ref(used2)
    slots = [p for p in range(S) if used2[p]][::-1]
    moved, _, fwd = gla.compact_pages([pool], table, i32(slots))
    synced(gla, False)
    for p, q in enumerate(forward):
        if q >= 0 and q != p:
            want[q] = want[p]
    assert fwd.tolist() == forward and table.tolist() == used3
    assert moved.tolist() == [forward[p] for p in slots]
    assert torch.equal(pool, i32(want)[:, None].expand(S, 4))
    order = torch.randperm(S, generator=g).int()
    src, dst = order[:S // 2].tolist(), order[S // 2:].tolist()
    assert gla.copy_pages([pool], i32(src), i32(dst)).tolist() == dst
    synced(gla, False)
    for p, q in zip(src, dst):
        want[q] = want[p]
    assert torch.equal(pool, i32(want)[:, None].expand(S, 4))
