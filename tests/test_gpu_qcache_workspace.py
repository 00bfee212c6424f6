"""The 4-bit cache's calls stay inside the workspace that they ask for on this GPU."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _qcache_ref as ref
from test_qcache_workspace import MB, SHAPES, slots_and

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("shape", SHAPES)
def test_sizes(shape):
    b, kv, cap, d, heads, n_q = shape
    assert 0 < cs.lib().cs_qcache_workspace_size(*shape) <= slots_and(b, kv, cap, heads, n_q, 15 * MB + 11 * MB)


class Guarded:
    """A workspace of exactly n bytes with a pattern behind it."""

    def __init__(self, n):
        self.nbytes = n
        self.buf = torch.full((n + 256 + MB,), 0xa5, dtype=torch.uint8, device="cuda")
        self.ptr = (self.buf.data_ptr() + 255) & ~255
        self.end = self.ptr - self.buf.data_ptr() + n
        assert cs.lib().cs_workspace_init(self.ptr, n, torch.cuda.current_stream().cuda_stream) == 0

    def whole(self):
        return bool((self.buf[self.end:] == 0xa5).all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,kv,group,n_q,S,d", [
    (1, 1, 1, 1, 9001, 64), (1, 2, 8, 1, 20011, 128), (3, 5, 4, 2, 700, 128), (70, 8, 16, 1, 300, 64), (40, 8, 8, 1, 900, 64),
    (16, 19, 1, 1, 600, 128), (5, 3, 17, 1, 400, 192), (2, 3, 8, 4, 500, 256), (300, 3, 2, 1, 33, 64)])
@pytest.mark.parametrize("ragged", [False, True])
def test_attention_stays_inside(B, kv, group, n_q, S, d, dt, ragged):
    g = torch.Generator().manual_seed(B * 31 + kv * 7 + S)
    rows = torch.randn(2, B, kv, S, d, generator=g)
    (k, ks), (v, vs) = ref.quantise(rows[0]), ref.quantise(rows[1])
    old = torch.rand(B, kv, S, generator=g)
    cache = cs.QCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), weight=old.cuda())
    lens = torch.randint(0, S + 1, (B,), generator=g) if ragged else torch.full((B,), S)
    q = torch.randn(B, n_q, kv * group, d, generator=g).to(dt)
    got = []
    for ws, weights in ((Guarded(cs.lib().cs_qcache_workspace_size(B, kv, S, d, kv * group, n_q)), True),
                        (Guarded(max(cs.lib().cs_qcache_workspace_size(B, kv, 1, d, kv * group, n_q), 512)), False)):
        w = torch.full_like(cache.weight, -1.0) if weights else None
        out = torch.full_like(q, float("nan"), device="cuda")
        cs.cs_qcache_attention(cache, q.cuda(), lens.int().cuda(), out, ws, weight=w, decay=0.5)
        assert ws.whole() and cs.cs_get_device_error(ws) == 0
        got.append(out)
        if weights and B <= 5:
            ro, re, rw, rwe = ref.attention(k, ks, v, vs, None, q, lens.tolist(), old=old, decay=0.5)
            assert ((out.cpu().double() - ro).abs() <= re + ref.half_step(dt) * (ro.abs() + re) + 1e-30).all()
            for b in range(B):
                n = int(lens[b])
                assert ((w[b, :, :n].cpu().double() - rw[b, :, :n]).abs() <= rwe[b, :, :n]).all() and (w[b, :, n:] == -1).all()
        elif weights:
            # what a head's rows give sums to the rows, beside the decayed account
            for b in range(B):
                n = int(lens[b])
                s = (w[b, :, :n].cpu() - 0.5 * old[b, :, :n]).double().sum(-1)
                assert torch.allclose(s, torch.full_like(s, float(group * n_q if n else 0)), rtol=0, atol=1e-4 * group * n_q)
    assert torch.equal(got[0], got[1])


def test_evict_and_trim_stay_inside():
    B, H, S, d, keep = 3, 5, 5000, 64, 1234
    g = torch.Generator("cuda").manual_seed(1)
    src, dst = (cs.QCache.empty(B, H, n, d) for n in (S, keep))
    src.weight.copy_(torch.rand(B, H, S, generator=g, device="cuda"))
    length = torch.full((B,), S, dtype=torch.int32, device="cuda")
    small, exact = Guarded(256), Guarded(cs.lib().cs_qcache_workspace_size(B, H, keep, d, 0, 1))
    out = torch.empty(B, H, 7, dtype=torch.int32, device="cuda")
    cs.cs_qcache_evict(src, length, S, out, small)
    assert torch.equal(out.long(), src.weight.argsort(-1)[..., :7].sort(-1).values)
    cs.cs_qcache_trim(src, length, keep, dst, exact)
    want = src.weight.argsort(-1)[..., -keep:].sort(-1).values
    assert torch.equal(dst.weight, src.weight.gather(-1, want))
    assert small.whole() and exact.whole()
    with pytest.raises(cs.CsError):
        cs.cs_qcache_trim(src, length, keep, dst, small)
