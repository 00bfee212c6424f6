"""Calls of the 4-bit cache at the ends of what their arguments allow."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _qcache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def filled(B, H, S, d, g):
    (k, ks), (v, vs) = (ref.quantise(torch.randn(B, H, S, d, generator=g)) for _ in range(2))
    w = torch.rand(B, H, S, generator=g) * 4
    pos = torch.stack([torch.randperm(S, generator=g) for _ in range(B * H)]).view(B, H, S).int()
    return cs.QCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), weight=w.cuda(), pos=pos.cuda()), (k, ks, v, vs, w, pos)


@pytest.mark.parametrize("S", [1, 70, 9001])
@pytest.mark.parametrize("decay", [1.0, 0.75, 0.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_without_tokens_decays_the_weights(S, decay, in_place):
    B, H, d = 3, 2, 64
    g = torch.Generator().manual_seed(S)
    cache, cpu = filled(B, H, S, d, g)
    length = [S, S // 2, 0]
    w = cache.weight if in_place else torch.full_like(cache.weight, -1.0)
    none = torch.empty(B, 0, H, d, device="cuda")
    ws = cs.QCacheWorkspace(cache)
    cs.cs_qcache_attention(cache, none, ints(length), none.clone(), ws, weight=w, decay=decay)
    want = cpu[4].clone() if in_place else torch.full((B, H, S), -1.0)
    for b, n in enumerate(length):
        want[b, :, :n] = decay * cpu[4][b, :, :n]
    assert torch.equal(w.cpu(), want) and cs.cs_get_device_error(ws) == 0
    cs.cs_qcache_attention(cache, none, ints([S + 1, 0, -1]), none.clone(), ws, weight=w, decay=0.0)
    assert not w[0].any() and cs.cs_get_device_error(ws) == cs.CS_DEVERR_COUNT


@pytest.mark.parametrize("group,n_q", [(1, 3), (4, 4), (8, 5)])
@pytest.mark.parametrize("last", [2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31])
def test_positions_at_the_ends_of_32_bits(group, n_q, last):
    """q_pos[b] + t past the largest position sees every token; below the first, none."""
    B, H, S, d = 2, 2, 90, 64
    g = torch.Generator().manual_seed(group)
    cache, cpu = filled(B, H, S, d, g)
    cache.pos[:, :, 7] = cpu[5][:, :, 7] = 2 ** 31 - 1
    cache.pos[:, :, 8] = cpu[5][:, :, 8] = -1
    q = torch.randn(B, n_q, H * group, d, generator=g)
    out = torch.full_like(q, float("nan"), device="cuda")
    w = torch.zeros_like(cache.weight)
    ws = cs.QCacheWorkspace(cache, n_heads=H * group, n_q=n_q)
    cs.cs_qcache_attention(cache, q.cuda(), ints([S, 50]), out, ws, q_pos=ints([last, last]), weight=w, decay=0.0)
    # (torch compares 32-bit tensors in 32 bits, whatever the other side)
    ro, re, rw, rwe = ref.attention(*cpu[:4], cpu[5].long(), q, [S, 50], q_pos=[last, last], old=cpu[4], decay=0.0)
    assert ((out.cpu().double() - ro).abs() <= re + 2.0 ** -24 * (ro.abs() + re)).all()
    assert ((w.cpu().double() - rw).abs()[0] <= rwe[0]).all() and bool(out.any()) == (last > 0)
