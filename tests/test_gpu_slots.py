"""Slot pools on the GPU against a slot-by-slot model on the host: everything is equal bit for bit."""
import random

import pytest
import torch

import ssm_ref as R
from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV

pytestmark = pytest.mark.gpu
i32 = torch.int32


def dev(x):
    return torch.tensor(x, dtype=i32, device=DEV)


def pool_of(n, seed=0):
    """Planes of every kind: slots of a multiple of 16 bytes, of 4, odd ones, and one of more than 32 KB."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, 2, 64, 72, generator=g).to(DEV), torch.randint(-128, 127, (n, 37), generator=g).to(torch.int8).to(DEV),
            torch.randn(n, 3, 10, generator=g).to(torch.bfloat16).to(DEV), torch.randn(n, 8, generator=g).to(DEV)]


def random_refs(n, share, seed):
    r = random.Random(seed)
    return [r.choice([1, 1, 2, 5]) if r.random() < share else r.choice([0, 0, 0, -1]) for _ in range(n)]


@pytest.mark.parametrize("n,share", [(1, 0.0), (1, 1.0), (2, 0.5), (33, 0.4), (200, 0.9), (1024, 0.5), (1025, 0.1), (5000, 0.6), (300, 0.0), (300, 1.0)])
def test_compact(n, share):
    refs = random_refs(n, share, n)
    r = random.Random(1)
    table = [r.randrange(-3, n + 3) for _ in range(2 * n + 5)]
    want_refs, want_table, want_used, moves = R.compact(refs, table)
    pool = pool_of(n) if n <= 300 else [torch.arange(n * 12, device=DEV, dtype=torch.float32).reshape(n, 12)]
    want = [p.clone() for p in pool]
    for p in want:
        for a, b in moves:
            p[b] = p[a]
    d_refs, d_table = dev(refs), dev(table)
    used = K.kda_slots_compact(pool, d_refs, d_table)
    torch.cuda.synchronize()
    assert used.tolist() == [want_used] and d_table.tolist() == want_table
    # a free slot's count is left as it was unless something moved there
    got = d_refs.tolist()
    assert [max(x, 0) for x in got] == [max(x, 0) for x in want_refs]
    for p, q in zip(pool, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("n,share,N", [(1, 0.0, 1), (8, 1.0, 3), (40, 0.5, 7), (40, 0.5, 40), (300, 0.7, 150), (3000, 0.9, 400)])
def test_fork(n, share, N):
    refs = random_refs(n, share, 10 * n + N)
    r = random.Random(2)
    parents = [r.randrange(-2, n + 2) for _ in range(N)]
    want_refs, want_children, sources = R.fork(refs, parents)
    pool = pool_of(n) if n <= 300 else [torch.arange(n * 12, device=DEV, dtype=torch.float32).reshape(n, 12)]
    want = [p.clone() for p in pool]
    for p in want:
        for c, s in zip(want_children, sources):
            if c >= 0:
                p[c] = 0 if s is None else p[s]
    d_refs = dev(refs)
    children = K.kda_slots_fork(pool, d_refs, dev(parents))
    torch.cuda.synchronize()
    assert children.tolist() == want_children and d_refs.tolist() == want_refs
    for p, q in zip(pool, want):
        assert torch.equal(p, q)


def test_new_sequences_and_one_plane():
    refs = dev([1, 0, 0, 2, 0])
    states = torch.ones(5, 7, 3, device=DEV)
    children = K.kda_slots_fork(states, refs, 2)
    torch.cuda.synchronize()
    assert children.tolist() == [1, 2] and refs.tolist() == [1, 1, 1, 2, 0]
    assert (states[1:3] == 0).all() and (states[[0, 3, 4]] == 1).all()
    assert K.kda_slots_fork(states, refs, 0).numel() == 0
    assert K.kda_slots_fork(states, refs, dev([])).numel() == 0
    assert K.kda_slots_fork(states, refs, 3).tolist() == [4, -1, -1]


def test_counts():
    refs = dev([0, 1, 2, 3, 1000])
    K.kda_slots_retain(refs, dev([0, 1, 1, 3, -1, 5, 4]))
    assert refs.tolist() == [0, 3, 2, 4, 1001]
    K.kda_slots_release(refs, dev([0, 1, 2, 2, 2, 2, 9, -7] + [4] * 1000))
    assert refs.tolist() == [0, 2, 0, 4, 1]
    K.kda_slots_release(refs, dev([]))
    big = torch.ones(70000, dtype=i32, device=DEV)
    K.kda_slots_release(big, torch.arange(0, 70000, 2, dtype=i32, device=DEV))
    assert (big[::2] == 0).all() and (big[1::2] == 1).all()


def test_copy_between_pools():
    src, dst = pool_of(9, 1), pool_of(12, 2)
    want = [p.clone() for p in dst]
    a, b = [3, 8, 3, -1, 9, 0, 5], [0, 11, 7, 2, 4, 12, 7]
    for p, q in zip(want, src):
        for s, d in zip(a, b):                      # in order: the last of one destination stays
            if 0 <= d < 12:
                p[d] = q[s] if 0 <= s < 9 else 0
    out = K.kda_slots_copy(src, dst, dev(a), dev(b))
    torch.cuda.synchronize()
    assert out is dst
    for p, q in zip(dst, want):
        assert torch.equal(p, q)
    # one list only, and none
    batch = torch.zeros(3, 2, 64, 72, device=DEV)
    K.kda_slots_copy(src[0], batch, src_slots=dev([8, 20, 1]))
    assert torch.equal(batch[[0, 2]], src[0][[8, 1]]) and (batch[1] == 0).all()
    K.kda_slots_copy(batch, dst[0], dst_slots=dev([5, 6, 5]))
    assert torch.equal(dst[0][[6, 5]], batch[[1, 2]])
    K.kda_slots_copy(src[0], dst[0])
    assert torch.equal(dst[0][:9], src[0]) and torch.equal(dst[0][9:11], want[0][9:11])


def test_pool_beyond_4_gb():
    """Offsets past 32 bits: the last slots of a pool of 5 GB."""
    n, per = 80, 64 << 20
    pool = torch.zeros(n, per, dtype=torch.uint8, device=DEV)
    pool[n - 1] = 7
    pool[n - 2] = 9
    refs = torch.zeros(n, dtype=i32, device=DEV)
    refs[n - 2:] = 1
    kids = K.kda_slots_fork(pool, refs, dev([n - 1]))
    assert kids.tolist() == [0] and (pool[0] == 7).all()
    table = dev([n - 1, n - 2, 0])
    used = K.kda_slots_compact(pool, refs, table)
    assert used.item() == 3 and table.tolist() == [2, 1, 0]
    assert (pool[1] == 9).all() and (pool[2] == 7).all()


def test_captured():
    """Release, compact and fork in a captured graph, replayed with eager work between."""
    n = 64
    refs0 = dev(random_refs(n, 0.6, 3))
    table0 = dev([s for s in range(n) if refs0[s] > 0])
    gone = table0[::5].contiguous()
    pool0 = torch.randn(n, 300, device=DEV)

    def work(refs, table, pool):
        K.kda_slots_release(refs, gone)
        used = K.kda_slots_compact(pool, refs, table)
        kids = K.kda_slots_fork(pool, refs, table[:9])
        return used, kids

    refs, table, pool = refs0.clone(), table0.clone(), pool0.clone()
    want = work(refs, table, pool)
    want = [t.clone() for t in (refs, table, pool) + want]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        work(refs, table, pool)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = work(refs, table, pool)
    for _ in range(4):
        refs.copy_(refs0); table.copy_(table0); pool.copy_(pool0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((refs, table, pool) + out, want):
            assert torch.equal(a, b)
        work(refs.clone(), table.clone(), pool.clone())
