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
