"""Eviction and trim of long and of many rows: every kernel and cluster size of the choice, with slots given up, equal and
strange weights, empty and protected slots."""
import numpy as np
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _qcache_ref as ref

gpu = pytest.mark.gpu


def order(w, pos, sinks, recent, next_pos):
    """ref.order for long rows: by class, then NaN, then weight, then slot."""
    w = np.asarray(w, dtype=np.float64)
    cls = np.ones(len(w), dtype=int)
    if pos is not None:
        p = np.asarray(pos, dtype=np.int64)
        cls = np.where(p < 0, 0, np.where((p < sinks) | ((recent > 0) & (p >= next_pos - recent)), 2, 1))
    nan = np.isnan(w)
    return np.lexsort((np.arange(len(w)), np.where(nan, 0.0, w) + 0.0, ~nan, cls))


def weights(kind, shape, g):
    w = torch.randn(shape, generator=g).exp()
    if kind == "ties":
        w = torch.randint(0, 3, shape, generator=g).float()
    elif kind == "same":
        w = torch.full(shape, 0.5)
    elif kind == "specials":
        w = torch.randn(shape, generator=g)
        for x in (float("nan"), float("inf"), float("-inf"), 0.0, -0.0):
            w[torch.rand(shape, generator=g) < 0.1] = x
    elif kind == "close":
        w = 1.0 + torch.randint(0, 200, shape, generator=g) * 2.0 ** -23
    return w


KINDS = ["plain", "ties", "same", "specials", "close"]


def positions(shape, g):
    pos = torch.rand(shape, generator=g).argsort(-1).int() + torch.randint(0, 50, shape[:2] + (1,), generator=g).int()
    pos[torch.rand(shape, generator=g) < 0.05] = -1
    return pos


@pytest.mark.parametrize("kind", KINDS)
def test_order_is_the_plain_forms(kind):
    g = torch.Generator().manual_seed(len(kind))
    w = weights(kind, (2, 1, 300), g)
    pos = positions((2, 1, 300), g)
    for b in range(2):
        for p, sinks, recent in ((None, 0, 0), (pos[b, 0], 0, 0), (pos[b, 0], 5, 40), (pos[b, 0], 0, 1000)):
            assert order(w[b, 0], p, sinks, recent, 310).tolist() == ref.order(w[b, 0], p, sinks, recent, 310)


# rows of: one CTA with all its registers (160 x 8,192), two CTAs (160 x 20,000), 4 and 8 CTAs, 8 of 1,024 threads, and
# rows that no cluster holds
ROWS = [(20, 8, 8192), (20, 8, 20000), (1, 2, 9000), (1, 2, 20000), (2, 1, 70001), (2, 1, 140001)]


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,H,S", ROWS)
def test_evict(B, H, S, kind):
    import __graft_entry__ as graft
    graft.build()
    g = torch.Generator().manual_seed(S + len(kind))
    w, pos = weights(kind, (B, H, S), g), positions((B, H, S), g)
    length = torch.full((B,), S)
    length[B // 2:] -= torch.arange(B - B // 2) % 7
    for p, sinks, recent, n in ((None, 0, 0, 1), (None, 0, 0, S // 3), (pos, 3, 200, 37), (pos, 0, S // 2, S // 2 + 100), (pos, S, 0, 900)):
        nxt = torch.full((B,), S + 20)
        cache = cs.QCache(None, None, None, None, weight=w.cuda(), pos=None if p is None else p.cuda())
        ws = cs.QCacheWorkspace(cache)
        slots = torch.full((B, H, n), -7, dtype=torch.int32, device="cuda")
        cs.cs_qcache_evict(cache, length.int().cuda(), S, slots, ws, next_pos=nxt.int().cuda(), sinks=sinks, recent=recent)
        got = slots.cpu().numpy()
        assert cs.cs_get_device_error(ws) == 0
        for b in range(B):
            used = int(length[b])
            give = max(0, n - (S - used))
            for h in range(H):
                o = order(w[b, h, :used], None if p is None else p[b, h, :used], sinks, recent, S + 20)
                want = np.concatenate([np.sort(o[:give]), np.arange(used, used + n - give)])
                assert np.array_equal(got[b, h], want), (b, h, n)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,H,S", [(20, 8, 8192)] + ROWS[2:] + [(3, 2, 5000)])
def test_trim(B, H, S, kind):
    import __graft_entry__ as graft
    graft.build()
    d = 64
    g = torch.Generator().manual_seed(S + len(kind) + 1)
    w, pos = weights(kind, (B, H, S), g), positions((B, H, S), g)
    src = cs.QCache.empty(B, H, S, d)
    gc = torch.Generator("cuda").manual_seed(S)
    for t in (src.k, src.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=gc, device="cuda"))
    for t in (src.k_scale, src.v_scale):
        t.copy_(torch.randn(t.shape, generator=gc, device="cuda"))
    src.weight.copy_(w)
    src.pos.copy_(pos)
    length = torch.full((B,), S)
    length[B // 2:] -= torch.arange(B - B // 2) % 7 * (S // 10)
    nxt = torch.full((B,), S + 20)
    ws = cs.QCacheWorkspace(src, n_heads=0)
    for keep, sinks, recent in ((1, 0, 0), (1234, 3, 200), (S // 3, 0, S // 2), (S - 5, 2, 5)):
        dst = cs.QCache.empty(B, H, keep + 3, d)
        dst.weight.fill_(-3.0)
        cs.cs_qcache_trim(src, length.int().cuda(), keep, dst, ws, next_pos=nxt.int().cuda(), sinks=sinks, recent=recent)
        for b in range(B):
            used = int(length[b])
            for h in range(H):
                o = order(w[b, h, :used], pos[b, h, :used], sinks, recent, S + 20)
                left = torch.from_numpy(np.sort(o[max(0, used - keep):])).cuda()
                n = len(left)
                for name in ("k", "v", "k_scale", "v_scale", "pos"):
                    assert torch.equal(getattr(dst, name)[b, h, :n], getattr(src, name)[b, h, left]), (name, b, h, keep)
                assert np.array_equal(dst.weight[b, h, :n].cpu().numpy(), src.weight[b, h, left].cpu().numpy(), equal_nan=True)
                assert (dst.weight[b, h, n:] == -3.0).all()
    assert cs.cs_get_device_error(ws) == 0
