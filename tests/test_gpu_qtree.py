"""Attention of drafted trees over the 4-bit cache against its plain 64-bit form."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _prompt_ref as ref
import _qcache_ref as qref
from test_gpu_qcache import filled, gen, ints

pytestmark = pytest.mark.gpu
DTS = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def parents(B, n, g):
    p = torch.full((B, n), -1, dtype=torch.int32)
    for b in range(B):
        for t in range(1, n):
            p[b, t] = int(torch.randint(-1, t, (1,), generator=g)) if t % 5 else -1
    return p


def drafts(B, n, H, kv, d, dt, g):
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return r(B, n, H, d).to(dt), (r(B, n, kv, d) + r(kv, d)).to(dt), (2 * r(B, n, kv, d)).to(dt)


def run(cache, q, k, v, length, parent=None, n_new=None, scale=0.0, ws=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    ws = ws or cs.QCacheTreeWorkspace(cache, q.shape[2], q.shape[1])
    cs.cs_qcache_tree_attention(cache, q.cuda(), k.cuda(), v.cuda(), ints(length), out, ws, scale=scale,
                                parent=None if parent is None else ints(parent), n_new=None if n_new is None else ints(n_new))
    return out, ws


def check(cpu, cache, q, k, v, length, parent=None, n_new=None, scale=0.0, pos=True):
    out, ws = run(cache, q, k, v, length, parent, n_new, scale)
    assert cs.cs_get_device_error(ws) == 0
    want, bound = ref.tree(*cpu[:4], cpu[5] if pos else None, q, k, v, length, parent, n_new, scale)
    off = (out.cpu().double() - want).abs()
    assert (off <= bound).all(), (off / bound.clamp(min=1e-30)).max().item()
    # roundings of both signs: their mean square, not their sum, is what a whole output is off by
    if want.norm() > 0:
        assert (off.norm() / want.norm()).item() < 4 * torch.finfo(q.dtype).eps
    return out


def without_positions(cache):
    return cs.QCache(cache.k, cache.v, cache.k_scale, cache.v_scale)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("B,H,kv,d,S,n", [(1, 1, 1, 64, 1, 1), (2, 8, 8, 64, 100, 5), (1, 6, 2, 128, 300, 17), (2, 16, 2, 128, 257, 64),
                                          (1, 8, 1, 64, 129, 128), (1, 5, 1, 128, 640, 33), (1, 16, 1, 64, 130, 64), (3, 3, 1, 128, 128, 43)])
def test_trees(B, H, kv, d, S, n, dt):
    g = gen(B, H, kv, d, S, n)
    cache, cpu = filled(B, kv, S, d, g)
    check(cpu, cache, *drafts(B, n, H, kv, d, dt, g), torch.randint(S // 2, S + 1, (B,), generator=g), parents(B, n, g))


@pytest.mark.parametrize("dt", DTS)
def test_chains_empty_slots_and_ragged_trees(dt):
    g = gen(5)
    B, H, kv, d, S, n = 5, 8, 2, 128, 400, 9
    cache, cpu = filled(B, kv, S, d, g)
    gone = torch.rand(B, kv, S, generator=g) < 0.3
    gone[1] = True                       # a sequence with nothing but empty slots
    cpu[5][gone] = -1
    cache.pos.copy_(cpu[5])
    # empty slots may hold anything
    cache.k_scale[gone.cuda()] = float("nan")
    cache.v_scale[gone.cuda()] = float("inf")
    q, k, v = drafts(B, n, H, kv, d, dt, g)
    length = torch.tensor([400, 400, 0, 129, 1])
    check(cpu, cache, q, k, v, length)
    n_new = torch.tensor([9, 1, 0, 4, 8])
    out = check(cpu, cache, q, k, v, length, parents(B, n, g), n_new)
    for b in range(B):
        assert (out[b, int(n_new[b]):] == 0).all()


@pytest.mark.parametrize("H,kv,d,S,n", [(8, 1, 128, 20000, 3), (4, 4, 64, 9001, 16), (16, 2, 128, 5000, 40)])
def test_long_caches(H, kv, d, S, n):
    g = gen(H, kv, S)
    cache, cpu = filled(1, kv, S, d, g)
    check(cpu, cache, *drafts(1, n, H, kv, d, torch.float16, g), torch.tensor([S]), parents(1, n, g))


def test_without_positions_and_unused_slots():
    """Slots past the length hold anything; without positions every slot below it counts."""
    g = gen(9)
    B, H, kv, d, S, n = 2, 4, 2, 64, 300, 7
    cache, cpu = filled(B, kv, S, d, g)
    length = torch.tensor([131, 5])
    for b in range(B):
        cache.k_scale[b, :, int(length[b]):] = float("inf")
        cache.v_scale[b, :, int(length[b]):] = float("nan")
    q, k, v = drafts(B, n, H, kv, d, torch.float16, g)
    check(cpu, without_positions(cache), q, k, v, length, parents(B, n, g), pos=False)


@pytest.mark.parametrize("dt", DTS)
def test_ranges(dt):
    """Rows of very different sizes: q's beside each other, tiny and huge keys and values, drafted ones beyond fp16."""
    g = gen(11)
    H, kv, d, S, n = 4, 2, 128, 200, 6
    k = torch.randn(1, kv, S, d, generator=g)
    v = torch.randn(1, kv, S, d, generator=g) * torch.exp(4 * torch.randn(1, kv, S, 1, generator=g))
    v[0, 0, 3, :64] = torch.tensor([65504.0, -65504.0]).repeat(32)
    (kc, ks), (vc, vs) = qref.quantise(k), qref.quantise(v)
    pos = torch.arange(S, dtype=torch.int32).expand(1, kv, S).contiguous()
    cache = cs.QCache(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), pos=pos.cuda())
    q, kn, vn = drafts(1, n, H, kv, d, dt, g)
    q[0, 0] *= 1e-4
    q[0, 1] *= 30
    q[0, 2, :, 7] = 200.0
    q[0, 3] = 0.0
    out, ws = run(cache, q, kn, vn, torch.tensor([S]))
    want, bound = ref.tree(kc, ks, vc, vs, pos, q, kn, vn, torch.tensor([S]))
    off = (out.cpu().double() - want).abs()
    top = torch.finfo(dt).max
    assert ((off <= bound) | (want.abs() + bound > top)).all()
    # drafted rows beyond the cache's range, and NaN, count as it would take them
    kn[0, 1, 0, 5] = float("nan")
    vn[0, 2, 1, :] = float("inf")
    out, ws = run(cache, q, kn, vn, torch.tensor([S]))
    want, bound = ref.tree(kc, ks, vc, vs, pos, q, kn, vn, torch.tensor([S]))
    off = (out.cpu().double() - want).abs()
    assert ((off <= bound) | (want.abs() + bound > top)).all()


def test_a_row_of_nan_stays_alone():
    g = gen(13)
    cache, cpu = filled(1, 1, 200, 64, g)
    q, k, v = drafts(1, 8, 2, 1, 64, torch.float16, g)
    clean, _ = run(cache, q, k, v, [200])
    q[0, 3, 1, 9] = float("nan")
    out, _ = run(cache, q, k, v, [200])
    bad = torch.zeros(1, 8, 2, dtype=torch.bool)
    bad[0, 3, 1] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def test_wrong_parents_and_counts_are_flagged():
    g = gen(14)
    cache, cpu = filled(2, 2, 50, 64, g)
    q, k, v = drafts(2, 4, 2, 2, 64, torch.float16, g)
    ok = torch.tensor([[-1, 0, 1, 2], [-1, -1, -1, -1]])
    for parent in ([[-1, 0, 1, 3], [-1, -1, -1, -1]], [[-1, 0, 1, -7], [-1] * 4], [[-1, 0, 1, 1000], [-1] * 4]):
        out, ws = run(cache, q, k, v, [50, 50], torch.tensor(parent))
        assert cs.cs_get_device_error(ws) == cs.CS_DEVERR_INDEX
        want, _ = run(cache, q, k, v, [50, 50], torch.tensor([[-1, 0, 1, -1], [-1] * 4]))
        assert torch.equal(out, want)
    for length, n_new in (([51, 50], [4, 4]), ([50, -1], [4, 4]), ([50, 50], [5, 4]), ([50, 50], [4, -1])):
        out, ws = run(cache, q, k, v, length, ok, n_new)
        assert cs.cs_get_device_error(ws) == cs.CS_DEVERR_COUNT
        want, _ = run(cache, q, k, v, [min(max(x, 0), 50) for x in length], ok, [min(max(x, 0), 4) for x in n_new])
        assert torch.equal(out, want)


def test_strided_drafts_and_cut_caches():
    g = gen(15)
    B, H, kv, d, S, n = 2, 4, 2, 64, 150, 5
    big, cpu = filled(B + 1, kv + 1, S, d, g)
    cut = lambda t: t[1:, 1:]  # noqa: E731
    cache = cs.QCache(cut(big.k), cut(big.v), cut(big.k_scale), cut(big.v_scale), weight=cut(big.weight), pos=cut(big.pos))
    q, k, v = drafts(B, n, H, kv, d, torch.bfloat16, g)
    want, _ = run(cache, q, k, v, [150, 77])
    ref_out = check([cut(t) for t in cpu], cache, q, k, v, torch.tensor([150, 77]))
    assert torch.equal(want, ref_out)
    for shift in (0, 1):   # rows on 16-byte boundaries, or not
        both = torch.cat([q, k, v], 2)
        flat = torch.zeros(both.numel() + 8, dtype=torch.bfloat16, device="cuda")
        dev = flat[shift:shift + both.numel()].view(both.shape)
        dev.copy_(both)
        room = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
        out = room[shift:shift + q.numel()].view(q.shape)
        ws = cs.QCacheTreeWorkspace(cache, H, n)
        cs.cs_qcache_tree_attention(cache, dev[:, :, :H], dev[:, :, H:H + kv], dev[:, :, H + kv:], ints([150, 77]), out, ws)
        assert torch.equal(out, want)


def test_same_bits_again_and_captured():
    g = gen(16)
    cache, cpu = filled(2, 2, 9000, 128, g)
    q, k, v = (t.cuda() for t in drafts(2, 12, 8, 2, 128, torch.float16, g))
    p, length = ints(parents(2, 12, g)), ints([9000, 1234])
    ws = cs.QCacheTreeWorkspace(cache, 8, 12)
    out = torch.zeros_like(q)
    cs.cs_qcache_tree_attention(cache, q, k, v, length, out, ws, parent=p)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cs.cs_qcache_tree_attention(cache, q, k, v, length, out, ws, parent=p)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    length.copy_(ints([10, 9000]))
    want, _ = run(cache, q.cpu(), k.cpu(), v.cpu(), [10, 9000], p.cpu())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_chain_sees_what_appended_tokens_see():
    """Beside cs_qcache_attention over the same tokens in the cache: they differ by what 4 bits cost the drafted rows alone."""
    g = gen(17)
    B, H, kv, d, S, n = 1, 4, 2, 64, 200, 4
    cache, cpu = filled(B, kv, S, d, g)
    q, k, v = drafts(B, n, H, kv, d, torch.float16, g)
    (kc, ks), (vc, vs) = qref.quantise(k.transpose(1, 2)), qref.quantise(v.transpose(1, 2))
    # drafted rows that 4 bits hold exactly
    k, v = (qref.values(c, s).transpose(1, 2).half() for c, s in ((kc, ks), (vc, vs)))
    tree, _ = run(cache, q, k, v, [150])
    ws = cs.QCacheWorkspace(cache, n_heads=H, n_q=n)
    cache.pos.copy_(torch.arange(S, dtype=torch.int32).expand(B, kv, S))
    cache.k[:, :, 150:154], cache.k_scale[:, :, 150:154] = kc.cuda(), ks.cuda()
    cache.v[:, :, 150:154], cache.v_scale[:, :, 150:154] = vc.cuda(), vs.cuda()
    out = torch.empty_like(tree)
    cs.cs_qcache_attention(cache, q.cuda(), ints([154]), out, ws, q_pos=ints([150]))
    _, bound = ref.tree(*cpu[:4], None, q, k, v, [150])
    assert ((tree.double() - out.double()).abs().cpu() <= 3 * bound).all()


@pytest.mark.parametrize("H,kv,n", [(8, 8, 16), (8, 8, 17), (8, 1, 2), (8, 1, 3), (16, 1, 1), (17, 1, 1), (6, 2, 5), (6, 2, 6)])
@pytest.mark.parametrize("dt", DTS)
def test_on_both_sides_of_few_rows(H, kv, n, dt):
    """Rows of a cache head up to and past what the kernels of single tokens take, over a ragged batch with an empty sequence."""
    g = gen(H, kv, n, 18)
    cache, cpu = filled(4, kv, 700, 128, g)
    cpu[5][torch.rand(4, kv, 700, generator=g) < 0.05] = -1
    cache.pos.copy_(cpu[5])
    check(cpu, cache, *drafts(4, n, H, kv, 128, dt, g), torch.tensor([700, 0, 129, 1]), parents(4, n, g), torch.tensor([n, n, max(n - 1, 0), n]))


def test_a_workspace_of_larger_sizes_serves_smaller_calls():
    g = gen(19)
    cache, cpu = filled(2, 2, 300, 64, g)
    ws = cs.QCacheTreeWorkspace(cache, 16, 64)
    for H, n in ((16, 64), (2, 1), (4, 8), (16, 2), (2, 64), (8, 4), (4, 5)):
        q, k, v = drafts(2, n, H, 2, 64, torch.float16, g)
        out, _ = run(cache, q, k, v, [300, 77], ws=ws)
        want, bound = ref.tree(*cpu[:4], cpu[5], q, k, v, [300, 77])
        assert ((out.cpu().double() - want).abs() <= bound).all()
    assert cs.cs_get_device_error(ws) == 0


def test_long_chains_and_deep_trees():
    g = gen(20)
    cache, cpu = filled(1, 1, 40, 64, g)
    q, k, v = drafts(1, 128, 2, 1, 64, torch.bfloat16, g)
    check(cpu, cache, q, k, v, torch.tensor([40]))
    check(cpu, cache, q, k, v, torch.tensor([40]), torch.arange(-1, 127, dtype=torch.int32)[None])
    check(cpu, cache, q, k, v, torch.tensor([0]), torch.full((1, 128), -1, dtype=torch.int32))


def test_scales_and_negative_scales():
    g = gen(21)
    cache, cpu = filled(1, 2, 200, 128, g)
    for H, n in ((4, 2), (4, 20)):
        q, k, v = drafts(1, n, H, 2, 128, torch.float16, g)
        for scale in (0.03, -0.05):
            check(cpu, cache, q, k, v, torch.tensor([200]), parents(1, n, g), scale=scale)


@pytest.mark.parametrize("H,kv,d,S,n", [(8, 2, 128, 54, 24), (8, 8, 64, 1, 40), (16, 1, 128, 250, 30), (8, 1, 64, 256, 5), (5, 1, 128, 129, 100)])
def test_keys_of_short_contexts_count_in_full(H, kv, d, S, n):
    """fp16: over caches of up to 256 slots keys are not rounded to 16 bits, so that a logit is off by what fp32 sums are, also where
    channels are far from zero."""
    g = gen(H, kv, d, S, n)
    cache, cpu = filled(1, kv, S, d, g)
    scales = cpu[1].clone()
    scales[..., 1] += 3.0                 # the groups' offsets
    cache.k_scale.copy_(scales)
    q, k, v = drafts(1, n, H, kv, d, torch.float16, g)
    q = q - 0.5 * q.mean(-1, keepdim=True)
    tree = parents(1, n, g)
    out, ws = run(without_positions(cache), q, k, v, torch.tensor([S]), tree)
    assert cs.cs_get_device_error(ws) == 0
    own = ref.paths(tree[0], n)
    for h in range(H):
        i = h // (H // kv)
        keys = torch.cat([qref.values(cpu[0][0, i], scales[0, i]), ref.drafted(k[0, :, i])])
        vals = torch.cat([qref.values(cpu[2][0, i], cpu[3][0, i]), ref.drafted(v[0, :, i])])
        seen = torch.cat([torch.ones(n, S, dtype=torch.bool), own], 1)
        want, bound = ref.rows(q[0, :, h].double(), keys, vals, seen, d ** -0.5, torch.float16, 2.0 ** -18,
                               ref.half_step(torch.float16), ref.half_step(torch.float16))
        assert ((out[0, :, h].cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("H,n", [(8, 1), (16, 1), (8, 2), (64, 16)])
def test_a_workspace_serves_caches_of_fewer_heads(H, n):
    """Fewer cache heads under as many query heads: more rows of each, on one path or the other."""
    g = gen(22, H, n)
    ws = cs.QCacheTreeWorkspace(filled(3, H, 100, 128, g)[0], H, n)
    for kv in (1, 2, H):
        cache, cpu = filled(3, kv, 100, 128, g)
        q, k, v = drafts(3, n, H, kv, 128, torch.bfloat16, g)
        out, _ = run(cache, q, k, v, [100, 0, 57], ws=ws)
        want, _ = run(cache, q, k, v, [100, 0, 57])
        assert torch.equal(out, want) and cs.cs_get_device_error(ws) == 0


@pytest.mark.parametrize("S", [256, 257, 5000])
@pytest.mark.parametrize("H,kv,d,L,n", [(8, 2, 128, 54, 24), (16, 1, 64, 9, 40), (8, 1, 128, 250, 5)])
def test_short_contexts_in_caches_of_any_capacity(H, kv, d, L, n, S):
    """fp16: a context of few slots, in a cache that keys are rounded over and in one that they are not; within the bound of
    rounded keys, and with the same contents the same bits but for that."""
    g = gen(23, H, kv, d, L, n)
    small, cpu = filled(2, kv, L, d, g)
    cache = cs.QCache.empty(2, kv, S, d)
    for name in ("k", "v", "k_scale", "v_scale", "weight", "pos"):
        getattr(cache, name)[:, :, :L] = getattr(small, name)
    q, k, v = drafts(2, n, H, kv, d, torch.float16, g)
    tree, length = parents(2, n, g), torch.tensor([L, L - 4])
    out = check(cpu, cache, q, k, v, length, tree)
    alike, _ = run(small, q, k, v, length, tree)
    if S <= 256 or H // kv * n <= 16:
        assert torch.equal(out, alike)
    else:
        want, bound = ref.tree(*cpu[:4], cpu[5], q, k, v, length, tree)
        assert ((alike.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H,kv,n,S", [(8, 1, 24, 200), (2, 1, 40, 300), (8, 1, 24, 5000)])
def test_a_bad_row_among_many_stays_alone(H, kv, n, S, bad, dt):
    """One query row of NaN or with an infinity, beside others of its row tile: it is not finite, they keep their bits."""
    g = gen(24, H, n, S)
    cache, cpu = filled(1, kv, S, 64, g)
    q, k, v = drafts(1, n, H, kv, 64, dt, g)
    clean, _ = run(cache, q, k, v, [S])
    q[0, n - 7, H - 1, 9] = bad
    out, ws = run(cache, q, k, v, [S])
    keep = torch.ones(1, n, H, dtype=torch.bool)
    keep[0, n - 7, H - 1] = False
    assert not torch.isfinite(out[~keep]).any() and torch.equal(out[keep], clean[keep])
    assert cs.cs_get_device_error(ws) == 0
