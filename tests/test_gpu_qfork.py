"""Rows taken into the 4-bit cache from anywhere, and sequences taken over by others."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _qcache_ref as qref
from test_gpu_qcache import filled, gen, ints, new_rows

pytestmark = pytest.mark.gpu
DTS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def arrays(c):
    return [t for t in (c.k, c.k_scale, c.v, c.v_scale, c.weight, c.pos) if t is not None]


# ----------------------------------------------------------------------------------------------------------- append_rows

@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("B,n,H,d,S,N", [(1, 1, 1, 64, 1, 1), (3, 4, 5, 128, 9, 100), (2, 37, 3, 192, 50, 12), (4, 3, 2, 256, 7, 300)])
@pytest.mark.parametrize("scattered", [False, True])
def test_rows_from_anywhere(B, n, H, d, S, N, dt, scattered):
    """What cs_qcache_append makes of the same rows side by side; tokens without a row leave their slots as they were."""
    g = gen(B, n, H, d, S, N, scattered)
    cache, before = filled(B, H, S, d, g)
    rows = torch.randint(0, N, (B, n), generator=g)            # the same row twice, too
    rows[torch.rand(B, n, generator=g) < 0.25] = -1
    k, v = new_rows(1, N, H, d, dt, g)[0], new_rows(1, N, H, d, dt, g)[0]
    at = torch.randint(0, 1000, (B,), generator=g)
    if scattered:
        slots = torch.rand(B, H, S, generator=g).argsort(-1)[..., :n].contiguous()
        how = dict(slots=ints(slots))
    else:
        start = torch.randint(0, S - n + 1, (B,), generator=g)
        slots, how = (start[:, None, None] + torch.arange(n)).expand(B, H, n), dict(start=ints(start))
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    cs.cs_qcache_append_rows(cache, k.cuda(), v.cuda(), ints(rows), ws, pos=ints(at), **how)
    assert cs.cs_get_device_error(ws) == 0
    want = [t.clone() for t in before]
    for b in range(B):
        for t in range(n):
            if rows[b, t] < 0:
                continue
            for h in range(H):
                s = int(slots[b, h, t])
                want[0][b, h, s], want[1][b, h, s] = qref.quantise(k[rows[b, t], h][None])[0][0], qref.quantise(k[rows[b, t], h][None])[1][0]
                want[2][b, h, s], want[3][b, h, s] = qref.quantise(v[rows[b, t], h][None])[0][0], qref.quantise(v[rows[b, t], h][None])[1][0]
                want[4][b, h, s], want[5][b, h, s] = 0.0, at[b] + t
    for got, w in zip((cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos), want):
        assert torch.equal(got.cpu(), w)


def test_rows_and_slots_out_of_range_are_passed_over():
    g = gen(1)
    cache, before = filled(2, 2, 6, 64, g)
    k, v = new_rows(1, 5, 2, 64, torch.float16, g)[0].cuda(), new_rows(1, 5, 2, 64, torch.float16, g)[0].cuda()
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    cs.cs_qcache_append_rows(cache, k, v, ints([[5, -2], [2 ** 31 - 1, -(2 ** 31)]]), ws, start=ints([0, 0]), pos=ints([0, 0]))
    assert cs.cs_get_device_error(ws, clear=True) == cs.CS_DEVERR_INDEX
    cs.cs_qcache_append_rows(cache, k, v, ints([[-1, -1], [-1, -1]]), ws, start=ints([100, -9]), pos=ints([0, 0]))
    assert cs.cs_get_device_error(ws, clear=True) == 0         # no rows, so no slots either
    cs.cs_qcache_append_rows(cache, k, v, ints([[0, 1], [2, 3]]), ws, start=ints([6, -3]), pos=ints([0, 0]))
    assert cs.cs_get_device_error(ws) == cs.CS_DEVERR_INDEX
    for got, w in zip((cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos), before):
        assert torch.equal(got.cpu(), w)


@pytest.mark.parametrize("shift", [0, 1])
def test_rows_of_a_projections_output(shift):
    g = gen(2, shift)
    cache, _ = filled(2, 3, 8, 128, g)
    other, _ = filled(2, 3, 8, 128, gen(2, shift))
    x = torch.randn(20, 9, 128, generator=g).half()
    flat = torch.zeros(x.numel() + 8, dtype=torch.float16, device="cuda")
    dev = flat[shift:shift + x.numel()].view(x.shape)
    dev.copy_(x)
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    rows = torch.tensor([[3, 19, 0], [7, 8, 9]])
    cs.cs_qcache_append_rows(cache, dev[:, 3:6], dev[:, 6:], ints(rows), ws, start=ints([1, 2]), pos=ints([4, 5]))
    cs.cs_qcache_append(other, x[rows][:, :, 3:6].cuda(), x[rows][:, :, 6:].cuda(), ws, start=ints([1, 2]), pos=ints([4, 5]))
    for a, b in zip(arrays(cache), arrays(other)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------------------------------ fork

def forked(src, dst, source, length):
    want = [t.clone() for t in dst]
    for i, s in enumerate(source):
        if 0 <= s < src[0].shape[0]:
            n = min(max(int(length[s]), 0), src[0].shape[2], dst[0].shape[2])
            for w, x in zip(want, src):
                w[i, :, :n] = x[s, :, :n]
    return want


def same(got, want):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("B,H,S,d,source", [
    (4, 3, 100, 64, [0, 0, 0, 0]),                 # samples of one
    (5, 2, 37, 128, [1, 0, 2, 2, 3]),              # two change places, a chain behind them
    (6, 1, 1, 64, [1, 2, 3, 4, 5, 0]),             # a ring
    (3, 2, 1000, 192, [2, -1, 0]),
    (4, 5, 130, 256, [3, 3, 3, -1]),
    (1, 2, 9, 64, [0]),
    (33, 2, 70, 128, list(range(32, -1, -1))),
    (200, 1, 5, 64, [(7 * i + 3) % 200 for i in range(200)])])
@pytest.mark.parametrize("in_place", [True, False])
def test_forks(B, H, S, d, source, in_place):
    g = gen(B, H, S, d, in_place)
    cache, _ = filled(B, H, S, d, g)
    length = torch.randint(0, S + 1, (B,), generator=g)
    length[0] = S
    to = cache if in_place else filled(B, H, S, d, gen(99))[0]
    want = forked([t.clone() for t in arrays(cache)], arrays(to), source, length)
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    cs.cs_qcache_fork(cache, ints(source), ints(length), ws, dst=None if in_place else to)
    assert cs.cs_get_device_error(ws) == 0
    assert same(arrays(to), want)


def test_into_another_size_without_weights_and_in_views():
    g = gen(4)
    big, _ = filled(5, 4, 60, 64, g)
    cut = lambda t: t[1:4, 1:, :31]  # noqa: E731
    src = cs.QCache(cut(big.k), cut(big.v), cut(big.k_scale), cut(big.v_scale), pos=cut(big.pos))
    room, _ = filled(3, 5, 50, 64, gen(5))
    lead = lambda t: t[:2, 2:, :40]  # noqa: E731
    dst = cs.QCache(lead(room.k), lead(room.v), lead(room.k_scale), lead(room.v_scale), pos=lead(room.pos))
    before = [t.clone() for t in arrays(room)]
    ws = cs.QCacheWorkspace(src, n_heads=0)
    length = torch.tensor([31, 7, 30])
    want = forked(arrays(src), arrays(dst), [2, 1], length)
    cs.cs_qcache_fork(src, ints([2, 1]), ints(length), ws, dst=dst)
    assert cs.cs_get_device_error(ws) == 0 and same([t.contiguous() for t in arrays(dst)], want)
    for now, was in zip(arrays(room), before):   # nothing beside the copies
        inside = torch.zeros(now.shape[:3], dtype=torch.bool, device="cuda")
        inside[0, 2:, :30] = inside[1, 2:, :7] = True
        if now.data_ptr() == room.weight.data_ptr():
            inside[:] = False
        assert torch.equal(now[~inside], was[~inside])


@pytest.mark.parametrize("in_place", [True, False])
def test_wrong_sources_and_lengths_are_flagged(in_place):
    g = gen(6)
    cache, _ = filled(3, 2, 20, 64, g)
    to = cache if in_place else filled(3, 2, 10, 64, gen(7))[0]
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    for source, length, err in (([3, 0, -2], [5, 5, 5], cs.CS_DEVERR_INDEX), ([1, 1, 1], [0, 21 if in_place else 11, 0], cs.CS_DEVERR_COUNT),
                                ([-1, 2, -1], [0, 0, -4], cs.CS_DEVERR_COUNT)):
        want = forked([t.clone() for t in arrays(cache)], arrays(to), source, length)
        cs.cs_qcache_fork(cache, ints(source), ints(length), ws, dst=None if in_place else to)
        assert cs.cs_get_device_error(ws, clear=True) == err
        assert same(arrays(to), want)


def test_replayed_forks_read_their_sources_anew():
    g = gen(8)
    cache, _ = filled(4, 2, 300, 128, g)
    source, length = ints([0, 0, 2, 2]), ints([300, 5, 77, 9])
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cs.cs_qcache_fork(cache, source, length, ws)
    for s, n in (([1, 0, 3, 2], [300, 5, 77, 9]), ([-1, 3, 1, 0], [20, 300, 0, 1])):
        source.copy_(ints(s))
        length.copy_(ints(n))
        want = forked([t.clone() for t in arrays(cache)], arrays(cache), s, n)
        graph.replay()
        torch.cuda.synchronize()
        assert same(arrays(cache), want)


@pytest.mark.parametrize("B,H,S,d,step", [(600, 1, 5, 128, 1), (300, 2, 70, 64, 7), (1792, 1, 3, 256, 5), (4096, 1, 2, 64, 1)])
@pytest.mark.parametrize("how", ["in place", "in place, from a few", "into another"])
def test_many_sequences(B, H, S, d, step, how):
    """More sequences than a CTA has threads, up to as many as can change places (batch x d_head 458,752)."""
    g = gen(B, H, S, d, step)
    cache, _ = filled(B, H, S, d, g)
    if how == "in place, from a few":      # that nobody writes
        few = torch.randperm(B, generator=g)[:B // 2]
        source = torch.full((B,), -1)
        others = torch.ones(B, dtype=torch.bool)
        others[few] = False
        source[others] = few[torch.randint(0, len(few), (int(others.sum()),), generator=g)]
        source = source.tolist()
    else:
        source = [(i + step) % B for i in range(B)]
    length = torch.randint(0, S + 1, (B,), generator=g)
    to = filled(B, H, S, d, gen(98))[0] if how == "into another" else cache
    want = forked([t.clone() for t in arrays(cache)], arrays(to), source, length)
    ws = cs.QCacheWorkspace(cache, n_heads=0)
    cs.cs_qcache_fork(cache, ints(source), ints(length), ws, dst=to)
    assert cs.cs_get_device_error(ws) == 0
    assert same(arrays(to), want)
