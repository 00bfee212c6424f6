"""The calls around the 4-bit cache as a serving process makes them: packed prompts, samples of them, drafted trees, accepted paths."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _prompt_ref as ref
import _qcache_ref as qref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_prompts_samples_trees_and_accepted_paths(dt):
    g = torch.Generator("cuda").manual_seed(0)
    heads, kv, d, budget, n, B = 8, 2, 64, 160, 7, 6
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    cache = cs.QCache.empty(B, kv, budget, d)
    ws = cs.QCacheWorkspace(cache, n_heads=heads, n_q=1)
    tws = cs.QCacheTreeWorkspace(cache, heads, n)

    # ---- two prompts, packed, attend and go into sequences 0 and 3; then each is sampled three times
    lens = [150, 33]
    qkv = rand(sum(lens), heads + 2 * kv, d)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    start = ints([0, 150, 183])
    out = torch.empty(sum(lens), heads, d, dtype=dt, device="cuda")
    pws = cs.PromptWorkspace(2, heads, kv, d, sum(lens))
    cs.cs_prompt_attention(q, k, v, out, start, pws)
    want, bound = ref.prompt(q, k, v, lens, lens)
    assert ((out.double() - want).abs() <= bound).all()

    rows = torch.full((B, 150), -1, dtype=torch.int32)
    rows[0] = torch.arange(150)
    rows[3, :33] = 150 + torch.arange(33)
    zero = ints([0] * B)
    cs.cs_qcache_append_rows(cache, k, v, rows.cuda(), ws, start=zero, pos=zero)
    length = ints([150, 0, 0, 33, 0, 0])
    source = ints([0, 0, 0, 3, 3, 3])
    cs.cs_qcache_fork(cache, source, length, ws)
    length = length[source.long()].contiguous()
    used, at = length.clone(), length.clone()      # slots in use; the next position

    # ---- three rounds of drafting, the last ones with the budget used up; positions and slots kept by the caller
    gg = torch.Generator().manual_seed(1)
    cpu = [t.cpu().clone() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos)]
    for _ in range(3):
        parent = torch.tensor([[-1] + [int(torch.randint(-1, t, (1,), generator=gg)) for t in range(1, n)] for _ in range(B)])
        q, k, v = rand(B, n, heads, d), rand(B, n, kv, d), rand(B, n, kv, d)
        out = torch.empty_like(q)
        cs.cs_qcache_tree_attention(cache, q, k, v, used, out, tws, parent=ints(parent))
        want, bound = ref.tree(cpu[0], cpu[1], cpu[2], cpu[3], cpu[5], q.cpu(), k.cpu(), v.cpu(), used.cpu(), parent)
        assert ((out.cpu().double() - want).abs() <= bound).all()

        # one path of every tree is accepted; its tokens take the slots that eviction gives for so many
        paths = []
        for b in range(B):
            t = int(torch.randint(0, n, (1,), generator=gg))
            path = []
            while t >= 0:
                path.insert(0, t)
                t = int(parent[b, t])
            paths.append(path)
        most = max(len(p) for p in paths)
        slots = torch.empty(B, kv, most, dtype=torch.int32, device="cuda")
        cs.cs_qcache_evict(cache, used, budget, slots, ws, next_pos=at, sinks=2, recent=8)
        pick = torch.full((B, most), -1, dtype=torch.int32)
        for b, p in enumerate(paths):
            # a path that is shorter takes the last slots: those beyond the used ones come last
            pick[b, most - len(p):] = b * n + torch.tensor(p, dtype=torch.int32)
        first = at - ints([most - len(p) for p in paths])
        cs.cs_qcache_append_rows(cache, k.flatten(0, 1), v.flatten(0, 1), pick.cuda(), ws, slots=slots, pos=first)
        s = slots.cpu()
        for b, p in enumerate(paths):
            for i, t in enumerate(p):
                for h in range(kv):
                    j = int(s[b, h, most - len(p) + i])
                    (c, sc), (cv, sv) = qref.quantise(k[b, t, h].cpu()[None]), qref.quantise(v[b, t, h].cpu()[None])
                    cpu[0][b, h, j], cpu[1][b, h, j], cpu[2][b, h, j], cpu[3][b, h, j] = c[0], sc[0], cv[0], sv[0]
                    cpu[4][b, h, j], cpu[5][b, h, j] = 0.0, int(at[b]) + i
        for got, w in zip((cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos), cpu):
            assert torch.equal(got.cpu(), w)
        at += ints([len(p) for p in paths])
        used = torch.clamp(used + most, max=budget)

        # the next token alone, with its weight on the slots' account
        q1 = rand(B, 1, heads, d)
        o1 = torch.empty_like(q1)
        cs.cs_qcache_attention(cache, q1, used, o1, ws, q_pos=at, weight=cache.weight)
        cpu[4] = cache.weight.cpu().clone()
        assert torch.isfinite(o1).all()
    for w in (ws, tws, pws):
        assert cs.cs_get_device_error(w) == 0


def test_two_streams_at_once():
    """Calls on workspaces of their own, side by side on two streams, each as it is alone."""
    g = torch.Generator("cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    lens = [900, 70, 2000]
    q, k, v = r(2970, 8, 128), r(2970, 2, 128), r(2970, 2, 128)
    start = ints([0, 900, 970, 2970])
    cache = cs.QCache.empty(4, 2, 3000, 128)
    for t in (cache.k, cache.v):
        t.random_(0, 256, generator=g)
    cache.k_scale.uniform_(0.01, 0.1, generator=g)
    cache.v_scale.uniform_(0.01, 0.1, generator=g)
    cache.pos.copy_(torch.arange(3000, device="cuda"))
    tq, tk, tv, length = r(4, 20, 8, 128), r(4, 20, 2, 128), r(4, 20, 2, 128), ints([3000, 1, 1500, 700])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    pws, tws = cs.PromptWorkspace(3, 8, 2, 128, 2970), cs.QCacheTreeWorkspace(cache, 8, 20)
    po, to = torch.empty_like(q), torch.empty_like(tq)
    cs.cs_prompt_attention(q, k, v, po, start, pws)
    cs.cs_qcache_tree_attention(cache, tq, tk, tv, length, to, tws)
    torch.cuda.synchronize()
    want = po.clone(), to.clone()
    for _ in range(20):
        with torch.cuda.stream(a):
            cs.cs_prompt_attention(q, k, v, po, start, pws)
        with torch.cuda.stream(b):
            cs.cs_qcache_tree_attention(cache, tq, tk, tv, length, to, tws)
    torch.cuda.synchronize()
    assert torch.equal(po, want[0]) and torch.equal(to, want[1])
    assert cs.cs_get_device_error(pws) == 0 and cs.cs_get_device_error(tws) == 0


@pytest.mark.parametrize("n", [1, 20])
def test_offsets_past_32_bits(n):
    """A cache of more than 2^31 bytes of keys: the last head's slots as they are in a small cache; forks and rows there, too."""
    g = torch.Generator("cuda").manual_seed(3)
    kv, d, cap, used = 4, 128, 5_200_000, 300
    big = cs.QCache.empty(2, kv, cap, d)
    small = cs.QCache.empty(1, kv, used, d)
    for t in (small.k, small.v):
        t.random_(0, 256, generator=g)
    small.k_scale.uniform_(0.01, 0.1, generator=g)
    small.v_scale.uniform_(0.01, 0.1, generator=g)
    small.weight.uniform_(0, 1, generator=g)
    small.pos.copy_(torch.arange(used, device="cuda"))
    parts = ("k", "v", "k_scale", "v_scale", "weight", "pos")
    for name in parts:
        getattr(big, name)[1, :, :used] = getattr(small, name)[0]
    q, k, v = (torch.randn(2, n, h, d, generator=g, device="cuda").half() for h in (2 * kv, kv, kv))
    out, one = torch.empty_like(q), torch.empty_like(q[1:])
    tws = cs.QCacheTreeWorkspace(big, 2 * kv, n)
    cs.cs_qcache_tree_attention(big, q, k, v, ints([0, used]), out, tws)
    cs.cs_qcache_tree_attention(small, q[1:], k[1:], v[1:], ints([used]), one, cs.QCacheTreeWorkspace(small, 2 * kv, n))
    # the cut along the keys goes by the lengths, which are alike but for an empty sequence
    assert torch.equal(out[1:], one) and cs.cs_get_device_error(tws) == 0
    ws = cs.QCacheWorkspace(big, n_heads=0)
    cs.cs_qcache_fork(big, ints([1, -1]), ints([0, used]), ws)
    for name in parts:
        assert torch.equal(getattr(big, name)[0, :, :used], getattr(small, name)[0])
    last = cap - 2 * n
    cs.cs_qcache_append_rows(big, k.flatten(0, 1), v.flatten(0, 1), ints([list(range(n)), list(range(n, 2 * n))]), ws,
                             start=ints([last, last]), pos=ints([7, 9]))
    (kc, ks), (vc, vs) = qref.quantise(k.cpu().transpose(1, 2)), qref.quantise(v.cpu().transpose(1, 2))
    for got, want in zip((big.k, big.k_scale, big.v, big.v_scale), (kc, ks, vc, vs)):
        assert torch.equal(got[:, :, last:last + n].cpu(), want)
    assert (big.pos[:, :, last] == ints([7, 9])[:, None]).all() and cs.cs_get_device_error(ws) == 0


def test_prompts_whose_rows_lie_far_apart():
    g = torch.Generator("cuda").manual_seed(4)
    n, kv, d, wide = 4000, 2, 64, 300_000
    buf = torch.empty(n, wide, dtype=torch.bfloat16, device="cuda")      # 2.4 GB, of which few columns are used
    cut = lambda h, at: buf[:, at:at + h * d].unflatten(1, (h, d))  # noqa: E731
    q, k, v, out = cut(4, 0), cut(kv, 1024), cut(kv, wide - 1024), cut(4, 4096)
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    pws = cs.PromptWorkspace(1, 4, kv, d, n)
    cs.cs_prompt_attention(q, k, v, out, ints([0, n]), pws)
    dense = torch.empty(n, 4, d, dtype=torch.bfloat16, device="cuda")
    cs.cs_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), dense, ints([0, n]), pws)
    assert torch.equal(out, dense) and cs.cs_get_device_error(pws) == 0


def test_wide_groups_of_drafted_trees():
    g = torch.Generator().manual_seed(5)
    for heads, n in ((127, 8), (100, 10), (65, 3), (128, 1), (33, 31)):
        x = torch.randn(1, 1, 140, 64, generator=g)
        (kc, ks), (vc, vs) = qref.quantise(x), qref.quantise(torch.randn(1, 1, 140, 64, generator=g))
        cache = cs.QCache(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda())
        q, k, v = (torch.randn(1, n, h, 64, generator=g).half() for h in (heads, 1, 1))
        out = torch.empty_like(q, device="cuda")
        ws = cs.QCacheTreeWorkspace(cache, heads, n)
        cs.cs_qcache_tree_attention(cache, q.cuda(), k.cuda(), v.cuda(), ints([140]), out, ws)
        want, bound = ref.tree(kc, ks, vc, vs, None, q, k, v, [140])
        assert ((out.cpu().double() - want).abs() <= bound).all() and cs.cs_get_device_error(ws) == 0
