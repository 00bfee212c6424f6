"""The 4-bit KV cache on the GPU against its plain 64-bit forms."""
import numpy as np
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _qcache_ref as ref

pytestmark = pytest.mark.gpu
DTS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)) + 1)


def filled(B, H, S, d, g, big=False):
    """A cache of random rows, with every slot filled: (QCache on the GPU, the arrays on the CPU)."""
    x = torch.randn(B, H, S, d, generator=g) * (1 + 3 * torch.rand(H, 1, d, generator=g)) + torch.randn(H, 1, d, generator=g)
    y = torch.randn(B, H, S, d, generator=g) + 0.5 * torch.randn(H, 1, d, generator=g)
    (k, ks), (v, vs) = ref.quantise(x), ref.quantise(y)
    w = torch.rand(B, H, S, generator=g) * 4
    pos = torch.stack([torch.randperm(S, generator=g) for _ in range(B * H)]).view(B, H, S).int()
    cpu = (k, ks, v, vs, w, pos)
    k_, ks_, v_, vs_, w_, pos_ = (t.cuda() for t in cpu)
    return cs.QCache(k_, v_, ks_, vs_, weight=w_, pos=pos_), cpu


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


# ------------------------------------------------------------------------------------------------------- append and read

def new_rows(B, n, H, d, dt, g):
    x = torch.randn(B, n, H, d, generator=g) * torch.exp(2 * torch.randn(B, n, H, 1, generator=g)) + torch.randn(H, d, generator=g)
    return x.to(dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("B,n,H,d,S", [(1, 1, 1, 64, 1), (3, 1, 5, 128, 9), (2, 37, 3, 192, 50), (1, 300, 2, 256, 311), (2, 7, 1, 64, 7)])
@pytest.mark.parametrize("scattered", [False, True])
def test_append_then_read(B, n, H, d, S, dt, scattered):
    g = gen(B, n, H, d, S, scattered)
    cache, before = filled(B, H, S, d, g)
    k, v = new_rows(B, n, H, d, dt, g), new_rows(B, n, H, d, dt, g)
    at = torch.randint(0, 1000, (B,), generator=g)
    if scattered:
        slots = torch.rand(B, H, S, generator=g).argsort(-1)[..., :n].contiguous()
    else:
        start = torch.randint(0, S - n + 1, (B,), generator=g)
        slots = (start[:, None, None] + torch.arange(n)).expand(B, H, n)
    how = dict(slots=ints(slots)) if scattered else dict(start=ints(start))
    ws = cs.QCacheWorkspace(cache)
    cs.cs_qcache_append(cache, k.cuda(), v.cuda(), ws, pos=ints(at), **how)
    ki, vi = torch.empty(B, n, H, d, dtype=dt, device="cuda"), torch.empty(B, n, H, d, dtype=dt, device="cuda")
    cs.cs_qcache_read(cache, ki, vi, ws, **how)
    assert cs.cs_get_device_error(ws) == 0
    want = [t.clone() for t in before]
    ix = (torch.arange(B)[:, None, None], torch.arange(H)[None, :, None], slots.long())
    (want[0][ix], want[1][ix]), (want[2][ix], want[3][ix]) = ref.quantise(k.transpose(1, 2)), ref.quantise(v.transpose(1, 2))
    want[4][ix] = 0.0
    want[5][ix] = (at[:, None, None] + torch.arange(n)).expand(B, H, n).int()
    for got, w in zip((cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos), want):
        assert torch.equal(got.cpu(), w)
    for got, c, s in ((ki, want[0], want[1]), (vi, want[2], want[3])):
        val = ref.values(c[ix], s[ix]).transpose(1, 2)
        # one rounding to fp32 (an fma), one to dt; below dt's normal range half the smallest step
        bound = (ref.half_step(dt) + 2.0 ** -24) * val.abs() + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
        assert ((got.cpu().double() - val).abs() <= bound).all()


@pytest.mark.parametrize("dt", DTS)
def test_append_of_strange_rows(dt):
    """Infinities, NaN, constants, ranges below fp16's and values on halves between two codes."""
    d, H, n = 128, 2, 8
    x = torch.zeros(1, n, H, d)
    x[0, 0, :, :70] = float("inf")
    x[0, 0, :, 3] = float("nan")
    x[0, 1] = float("-inf")
    x[0, 2] = 1e-9 * torch.arange(d)
    x[0, 3] = 7.25
    x[0, 4] = (torch.arange(d) % 31) * 0.5          # scale 1: odd multiples are halves
    x[0, 5] = 1000 + (torch.arange(d) % 7) * 0.125   # the offset's fp16 step is of the range's size
    x[0, 6] = torch.tensor([65504.0, -65504.0]).repeat(d // 2)
    x[0, 7] = 3e38 if dt != torch.float16 else 6e4
    x = x.to(dt)
    cache = cs.QCache.empty(1, H, n, d)
    ws = cs.QCacheWorkspace(cache)
    cs.cs_qcache_append(cache, x.cuda(), (-x).cuda(), ws, start=ints([0]), pos=ints([0]))
    for got, gs, r in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, -x)):
        c, s = ref.quantise(r.transpose(1, 2))
        assert torch.equal(got.cpu(), c) and torch.equal(gs.cpu(), s)
        assert torch.isfinite(gs.float()).all()


@pytest.mark.parametrize("shift", [0, 1, 8])
def test_append_and_read_of_strided_rows(shift):
    """k and v as slices of one projection's output, on 16-byte boundaries or not; the cache a slice of a larger one."""
    B, n, H, d, S = 2, 5, 3, 64, 11
    g = gen(shift)
    qkv = torch.randn(B, n, 4 + 2 * H + 1, d, generator=g).half()
    flat = torch.zeros(qkv.numel() + 8, dtype=torch.float16, device="cuda")
    dev = flat[shift:shift + qkv.numel()].view(qkv.shape)
    dev.copy_(qkv)
    big, _ = filled(B + 2, H + 2, S, d, g)
    cut = lambda t: t[1:1 + B, 2:]  # noqa: E731
    all_before = [t.clone() for t in (big.k, big.v, big.k_scale, big.v_scale, big.weight, big.pos)]
    cache = cs.QCache(cut(big.k), cut(big.v), cut(big.k_scale), cut(big.v_scale), weight=cut(big.weight), pos=cut(big.pos))
    ws = cs.QCacheWorkspace(cache)
    cs.cs_qcache_append(cache, dev[:, :, 4:4 + H], dev[:, :, 4 + H:4 + 2 * H], ws, start=ints([0, 6]), pos=ints([3, 4]))
    for i, sl in enumerate((slice(4, 4 + H), slice(4 + H, 4 + 2 * H))):
        c, s = ref.quantise(qkv[:, :, sl].transpose(1, 2))
        want, swant = all_before[i], all_before[2 + i]
        for b, st in ((0, 0), (1, 6)):
            want[1 + b, 2:, st:st + n] = c[b].cuda()
            swant[1 + b, 2:, st:st + n] = s[b].cuda()
    assert torch.equal(big.k, all_before[0]) and torch.equal(big.v, all_before[1])
    assert torch.equal(big.k_scale, all_before[2]) and torch.equal(big.v_scale, all_before[3])
    out = torch.zeros(B, n, 2 * H * d + shift, dtype=torch.float32, device="cuda")
    ko = out[..., shift:shift + H * d].unflatten(-1, (H, d))
    vo = out[..., shift + H * d:].unflatten(-1, (H, d))
    cs.cs_qcache_read(cache, ko, vo, ws, start=ints([0, 6]))
    for got, sl in ((ko, slice(4, 4 + H)), (vo, slice(4 + H, 4 + 2 * H))):
        val = ref.values(*ref.quantise(qkv[:, :, sl]))
        assert ((got.cpu().double() - val).abs() <= 2.0 ** -24 * val.abs()).all()


def test_append_skips_what_has_no_slot():
    B, n, H, d, S = 2, 4, 2, 64, 6
    g = gen(5)
    cache, before = filled(B, H, S, d, g)
    x = new_rows(B, n, H, d, torch.float16, g)
    ws = cs.QCacheWorkspace(cache)
    slots = torch.tensor([[[0, -1, 3, 5], [-1, -1, -1, -1]], [[5, 4, 3, 2], [1, 2, 3, -1]]], dtype=torch.int32)
    cs.cs_qcache_append(cache, x.cuda(), x.cuda(), ws, slots=slots.cuda(), n_new=ints([3, 0]), pos=ints([10, 20]))
    assert cs.cs_get_device_error(ws) == 0
    want = before[0].clone()
    c = ref.quantise(x.transpose(1, 2))[0]
    want[0, 0, 0], want[0, 0, 3] = c[0, 0, 0], c[0, 0, 2]
    assert torch.equal(cache.k.cpu(), want) and int(cache.pos[0, 0, 3]) == 12
    # past the end, before the start, and more tokens than there are
    cs.cs_qcache_append(cache, x.cuda(), x.cuda(), ws, start=ints([4, -3]), pos=ints([0, 0]))
    want[0, :, 4:], want[1, :, :1] = c[0, :, :2], c[1, :, 3:]
    assert torch.equal(cache.k.cpu(), want)
    assert cs.cs_get_device_error(ws, clear=True) == cs.CS_DEVERR_INDEX
    cs.cs_qcache_append(cache, x.cuda(), x.cuda(), ws, start=ints([0, 0]), n_new=ints([-1, 9]), pos=ints([0, 0]))
    want[1, :, :4] = c[1]
    assert torch.equal(cache.k.cpu(), want)
    assert cs.cs_get_device_error(ws, clear=True) == cs.CS_DEVERR_COUNT
    k, v = (torch.ones(B, 2, H, d, device="cuda") for _ in range(2))
    cs.cs_qcache_read(cache, k, v, ws, slots=ints([[[-1, -1]] * H] * B))
    assert not k.any() and not v.any() and cs.cs_get_device_error(ws) == 0
    cs.cs_qcache_read(cache, k, v, ws, start=ints([5, 0]))
    assert k[0, 0].any() and not k[0, 1].any() and cs.cs_get_device_error(ws, clear=True) == cs.CS_DEVERR_INDEX


# -------------------------------------------------------------------------------------------------------------- attention

def attend(cache, cpu, q, length, q_pos=None, on=None, scale=0.0, decay=1.0, weight=None, ws=None, out=None):
    """Runs the call and compares it with the plain form, returns (out, weight)."""
    H = q.shape[2]
    mask = None
    if on is not None:
        bits = torch.zeros(on.shape[0], -(-H // 32), dtype=torch.int64)
        for j in range(H):
            bits[:, j // 32] |= on[:, j].long() << (j % 32)
        mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int().cuda()
    ws = ws or cs.QCacheWorkspace(cache, n_heads=H, n_q=q.shape[1])
    out = torch.full_like(q, float("nan"), device="cuda") if out is None else out
    w = torch.full(cache.weight.shape, -1.0, device="cuda") if weight is None else weight
    untouched = w.clone()
    cs.cs_qcache_attention(cache, q.cuda(), ints(length), out, ws, q_pos=None if q_pos is None else ints(q_pos), mask=mask, scale=scale,
                           weight=w, decay=decay)
    k, ks, v, vs, old, pos = cpu
    ro, re, rw, rwe = ref.attention(k, ks, v, vs, pos, q, length, q_pos, on, scale, old, decay)
    err = (out.cpu().double() - ro).abs()
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps
    assert (err <= re + ref.half_step(q.dtype) * (ro.abs() + re) + tiny).all(), (err - re).max()
    for b, n in enumerate(length):
        n = min(max(int(n), 0), cache.capacity)
        assert ((w[b, :, :n].cpu().double() - rw[b, :, :n]).abs() <= rwe[b, :, :n]).all()
        assert torch.equal(w[b, :, n:], untouched[b, :, n:])
    return out, w


def some_q(B, n_q, H, d, dt, g, size=1.0):
    return (torch.randn(B, n_q, H, d, generator=g) * size).to(dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("group,n_q", [(1, 1), (2, 1), (4, 1), (3, 2), (8, 1), (5, 1), (16, 1), (17, 1), (8, 4)])
def test_attention_heads_and_types(d, group, n_q, dt):
    B, kv, S = 2, 2, 150
    g = gen(d, group, n_q)
    cache, cpu = filled(B, kv, S, d, g)
    attend(cache, cpu, some_q(B, n_q, kv * group, d, dt, g), [S, 77], decay=0.5)


@pytest.mark.parametrize("group", [1, 8, 12])
@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 500, 2049])
def test_attention_lengths(S, group):
    kv, d = 2, 128
    g = gen(S, group)
    cache, cpu = filled(3, kv, S, d, g)
    attend(cache, cpu, some_q(3, 1, kv * group, d, torch.float32, g, 2.0), [S, max(0, S - 1), 0])


def test_attention_many_ragged_sequences():
    g = gen(77)
    B, kv, S, d = 70, 3, 201, 64
    cache, cpu = filled(B, kv, S, d, g)
    length = torch.randint(0, S + 1, (B,), generator=g).tolist()
    attend(cache, cpu, some_q(B, 1, kv * 4, d, torch.bfloat16, g), length, decay=0.0)


def test_attention_long_rows_split():
    g = gen(78)
    cache, cpu = filled(1, 1, 20011, 64, g)
    attend(cache, cpu, some_q(1, 1, 4, 64, torch.float32, g, 1.5), [20011])
    attend(cache, cpu, some_q(1, 2, 5, 64, torch.float16, g, 0.0), [19990])   # flat: every slot weighs the same


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("group,n_q", [(1, 5), (4, 3), (2, 1), (8, 7)])
def test_attention_by_position(group, n_q, dt):
    """Each query token sees the slots up to its position; empty slots are passed over whatever they hold."""
    B, kv, S, d = 3, 2, 90, 128
    g = gen(group, n_q)
    cache, cpu = filled(B, kv, S, d, g)
    gone = torch.rand(B, kv, S, generator=g) < 0.3
    gone[2, 1] = True
    k, ks, v, vs, w, pos = cpu
    pos = pos.masked_fill(gone, -1)
    cache.pos.copy_(pos)
    cache.k_scale[gone.cuda()] = float("nan")
    cache.v_scale[gone.cuda()] = float("inf")
    # positions 0 .. S - 1: sequence 0's queries are the newest, 1's see about half, 2's first ones see nothing
    attend(cache, (k, ks, v, vs, w, pos), some_q(B, n_q, kv * group, d, dt, g), [S, 60, S], q_pos=[S - n_q, 40, -2])


def test_attention_reads_nothing_past_the_length():
    B, kv, S, d = 2, 2, 100, 128
    g = gen(9)
    cache, cpu = filled(B, kv, S, d, g)
    cache.k_scale[:, :, 41:] = float("nan")
    cache.v_scale[:, :, 41:] = float("nan")
    cache.k[:, :, 41:] = 255
    attend(cache, cpu, some_q(B, 1, 8, d, torch.float32, g), [41, 3])


@pytest.mark.parametrize("group", [1, 4, 16])
def test_attention_of_chosen_heads(group):
    B, kv, S, d = 3, 5, 70, 64
    g = gen(group, 3)
    cache, cpu = filled(B, kv, S, d, g)
    on = torch.rand(B, kv * group, generator=g) < 0.3
    on[1] = False
    on[2] = True
    out, w = attend(cache, cpu, some_q(B, 2, kv * group, d, torch.float32, g), [S, S, 33], on=on)
    assert not out[1].any() and torch.equal(w[1].cpu(), cpu[4][1])


@pytest.mark.parametrize("B,kv,group", [(3, 40, 1), (40, 5, 3), (34, 33, 2)])
def test_attention_of_few_chosen_heads_of_many(B, kv, group):
    """More cache heads and more sequences than a warp has lanes; most heads are not read, some sequences are empty."""
    S, d = 37, 64
    g = gen(B, kv, group)
    cache, cpu = filled(B, kv, S, d, g)
    on = torch.rand(B, kv * group, generator=g) < 0.1
    on[1] = False
    length = torch.randint(0, S + 1, (B,), generator=g)
    length[2] = 0
    attend(cache, cpu, some_q(B, 1, kv * group, d, torch.float32, g), length.tolist(), on=on, decay=0.5)


@pytest.mark.parametrize("scale", [0.3, -0.2, 1e-6])
def test_attention_scale(scale):
    g = gen(19)
    cache, cpu = filled(2, 2, 130, 64, g)
    attend(cache, cpu, some_q(2, 1, 6, 64, torch.float32, g), [130, 66], scale=scale)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("group", [2, 8, 12])
def test_attention_rising_and_falling_logits(d, group):
    """Slots in the order of their logits, up for one sequence and down for the other, steep enough that the running
    maxima move in every unit, or never after the first."""
    S = 700
    g = gen(d, group, 20)
    cache, cpu = filled(2, 1, S, d, g)
    ramp = torch.linspace(-30, 30, S)[:, None] * torch.ones(d) / d
    k, ks = ref.quantise(torch.stack([ramp, ramp.flip(0)])[:, None] + 0.01 * torch.randn(2, 1, S, d, generator=g))
    cache.k.copy_(k)
    cache.k_scale.copy_(ks)
    q = 1.0 + 0.1 * torch.rand(2, 1, group, d, generator=g)
    attend(cache, (k, ks) + tuple(cpu[2:]), q, [S, S], scale=1.0)


def test_attention_length_out_of_range_is_clamped_and_flagged():
    g = gen(10)
    cache, cpu = filled(2, 1, 20, 64, g)
    ws = cs.QCacheWorkspace(cache)
    attend(cache, cpu, some_q(2, 1, 1, 64, torch.float32, g), [25, -4], ws=ws)
    assert cs.cs_get_device_error(ws) == cs.CS_DEVERR_COUNT


@pytest.mark.parametrize("group", [1, 6])
def test_attention_gathers_weight_in_place(group):
    g = gen(11, group)
    B, kv, S, d = 2, 2, 300, 128
    cache, cpu = filled(B, kv, S, d, g)
    cpu = list(cpu)
    ws = cs.QCacheWorkspace(cache, n_heads=kv * group)
    for decay in (1.0, 0.75, 0.0):
        _, w = attend(cache, cpu, some_q(B, 1, kv * group, d, torch.float16, g), [S, 211], decay=decay, weight=cache.weight, ws=ws)
        cpu[4] = w.cpu()
    # with no old weights a head's weights sum to its group's size
    assert torch.allclose(cache.weight[0].sum(-1), torch.full((kv,), float(group), device="cuda"), rtol=1e-5)


def test_attention_without_weights_writes_none():
    g = gen(12)
    cache, cpu = filled(1, 2, 50, 64, g)
    before = cache.weight.clone()
    q = some_q(1, 1, 4, 64, torch.float32, g).cuda()
    out = torch.empty_like(q)
    cs.cs_qcache_attention(cache, q, ints([50]), out, cs.QCacheWorkspace(cache, n_heads=4))
    ro, re, _, _ = ref.attention(*cpu[:4], cpu[5], q.cpu(), [50])
    assert ((out.cpu().double() - ro).abs() <= re + 2.0 ** -24 * ro.abs()).all() and torch.equal(cache.weight, before)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e30])
def test_attention_queries_of_any_size(size):
    """Tiny and huge queries: a flat softmax, and one slot that takes all."""
    g = gen(13)
    cache, cpu = filled(1, 1, 64, 64, g)
    q = some_q(1, 1, 2, 64, torch.float32, g, size)
    if size < 1:
        attend(cache, cpu, q, [64])
        return
    out = torch.empty_like(q, device="cuda")
    cs.cs_qcache_attention(cache, q.cuda(), ints([64]), out, cs.QCacheWorkspace(cache, n_heads=2))
    k, v = ref.values(cpu[0], cpu[1])[0, 0], ref.values(cpu[2], cpu[3])[0, 0]
    for j in range(2):
        best = (k @ q[0, 0, j].double()).argmax()
        # the first slot leads by more than 2^10 in the logits; its value in one rounding of three terms
        assert ((out[0, 0, j].cpu().double() - v[best]).abs() <= 2.0 ** -18 * (v[best].abs() + 8)).all()


@pytest.mark.parametrize("vsize", [1e-4, 3e3])
def test_attention_values_of_any_size(vsize):
    g = gen(14)
    x = torch.randn(1, 1, 200, 64, generator=g)
    cache, cpu = filled(1, 1, 200, 64, g)
    v, vs = ref.quantise(x * vsize)
    cache.v.copy_(v)
    cache.v_scale.copy_(vs)
    attend(cache, (cpu[0], cpu[1], v, vs, cpu[4], cpu[5]), some_q(1, 1, 3, 64, torch.float32, g), [200])


def test_attention_nan_query_stays_in_its_row():
    g = gen(15)
    cache, cpu = filled(1, 2, 100, 128, g)
    q = some_q(1, 1, 8, 128, torch.float32, g)
    q[0, 0, 2, 5] = float("nan")
    q[0, 0, 5, 7] = float("inf")
    out = torch.empty_like(q, device="cuda")
    cs.cs_qcache_attention(cache, q.cuda(), ints([100]), out, cs.QCacheWorkspace(cache, n_heads=8))
    good = [0, 1, 3, 4, 6, 7]
    ro, re, _, _ = ref.attention(*cpu[:4], cpu[5], q, [100], on=torch.tensor([[j in good for j in range(8)]]))
    assert torch.isnan(out[0, 0, 2]).all() and torch.isnan(out[0, 0, 5]).all()
    assert ((out.cpu().double() - ro).abs() <= re + 2.0 ** -24 * ro.abs())[:, :, good].all()


@pytest.mark.parametrize("shift", [0, 1])
def test_attention_strided(shift):
    """q from a packed projection, out into a wider buffer, the cache and the weights views of larger ones."""
    B, kv, G, S, d = 2, 2, 4, 45, 64
    g = gen(16, shift)
    big, cpu = filled(B + 1, kv + 1, S, d, g)
    cut = lambda t: t[1:, :kv]  # noqa: E731
    cache = cs.QCache(cut(big.k), cut(big.v), cut(big.k_scale), cut(big.v_scale), weight=cut(big.weight), pos=cut(big.pos))
    buf = torch.zeros(B * 3 * (kv * G + 4) * d + 8, device="cuda")
    q = buf[shift:shift + B * 3 * (kv * G + 4) * d].view(B, 3, kv * G + 4, d)[:, :, 2:-2]
    q.copy_(some_q(B, 3, kv * G, d, torch.float32, g))
    out = torch.zeros(B, 3, kv * G * d + 3, device="cuda")[..., 3:].unflatten(-1, (kv * G, d))
    cpu = [cut(t) for t in cpu]
    attend(cache, cpu, q.cpu(), [S, 20], weight=cut(big.weight), out=out)
    # the cache as [batch, slots, heads, ...] memory has no contiguous slots: refused
    with pytest.raises(ValueError):
        cs.QCache(*(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def test_attention_is_reproducible_and_follows_its_stream():
    g = gen(17)
    B, kv, S, d = 4, 4, 1111, 128
    cache, cpu = filled(B, kv, S, d, g)
    q = some_q(B, 1, 32, d, torch.float32, g)
    length = ints([S, 5, 700, 0])
    first = None
    side = torch.cuda.Stream()
    ws = cs.QCacheWorkspace(cache, n_heads=32)
    for i in range(4):
        s = side if i % 2 else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            qd = torch.zeros(q.shape, device="cuda")
            torch.cuda._sleep(2000000)
            qd.copy_(q, non_blocking=True)
            out, w = torch.empty_like(qd), torch.zeros_like(cache.weight)
            cs.cs_qcache_attention(cache, qd, length, out, ws, weight=w)
            got = (out.cpu(), w.cpu())
        torch.cuda.current_stream().wait_stream(s)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_attention_offsets_past_32_bits():
    """A cache whose last head starts beyond 2^31 codes and ends beyond 2^32 bytes; few of its slots hold a token."""
    H, S, d = 2, 9_000_001, 256
    cache = cs.QCache(torch.zeros(1, H, S, d // 2, dtype=torch.uint8, device="cuda"), torch.zeros(1, H, S, d // 2, dtype=torch.uint8, device="cuda"),
                      torch.zeros(1, H, S, d // 64, 2, dtype=torch.float16, device="cuda"),
                      torch.zeros(1, H, S, d // 64, 2, dtype=torch.float16, device="cuda"),
                      weight=torch.zeros(1, H, S, device="cuda"), pos=torch.full((1, H, S), -1, dtype=torch.int32, device="cuda"))
    g = gen(18)
    n = 50
    x, y = (torch.randn(1, n, H, d, generator=g) for _ in range(2))
    slots = torch.cat([torch.randint(0, S - 60, (n - 3,), generator=g).unique(), torch.arange(S - 60, S)])[-n:].int()
    slots = slots.expand(1, H, n).contiguous()
    ws = cs.QCacheWorkspace(cache, n_heads=2 * H)
    cs.cs_qcache_append(cache, x.cuda(), y.cuda(), ws, slots=slots.cuda(), pos=ints([0]))
    q = some_q(1, 1, 2 * H, d, torch.float32, g)
    out = torch.empty_like(q, device="cuda")
    cs.cs_qcache_attention(cache, q.cuda(), ints([S]), out, ws, q_pos=ints([n]), weight=cache.weight)
    (k, ks), (v, vs) = ref.quantise(x.transpose(1, 2)), ref.quantise(y.transpose(1, 2))
    ro, re, rw, rwe = ref.attention(k, ks, v, vs, None, q, [n], old=torch.zeros(1, H, n))
    assert ((out.cpu().double() - ro).abs() <= re + 2.0 ** -24 * ro.abs()).all()
    got = torch.stack([cache.weight[0, h, slots[0, h].long().cuda()] for h in range(H)]).cpu()
    assert ((got[None].double() - rw).abs() <= rwe).all()
    cache.weight.add_(1.0)
    cache.weight[0, :, S - 2] = 0.25
    cache.pos.fill_(5)
    one = torch.empty(1, H, 1, dtype=torch.int32, device="cuda")
    cs.cs_qcache_evict(cache, ints([S]), S, one, ws)
    assert one.flatten().tolist() == [S - 2] * H


# ------------------------------------------------------------------------------------------------------------ evict, trim

def strange_weights(B, H, S, g, kind):
    w = torch.randn(B, H, S, generator=g).exp()
    if kind == "ties":
        w = torch.randint(0, 3, (B, H, S), generator=g).float()
    elif kind == "same":
        w = torch.full((B, H, S), 0.5)
    elif kind == "specials":
        w = torch.randn(B, H, S, generator=g)
        for x in (float("nan"), float("inf"), float("-inf"), 0.0, -0.0):
            w[torch.rand(B, H, S, generator=g) < 0.1] = x
    elif kind == "close":
        w = 1.0 + torch.randint(0, 200, (B, H, S), generator=g) * 2.0 ** -23
    return w


def weight_cache(w, pos):
    return cs.QCache(None, None, None, None, weight=w.cuda(), pos=None if pos is None else pos.cuda())


@pytest.mark.parametrize("kind", ["plain", "ties", "same", "specials", "close"])
@pytest.mark.parametrize("S,limit,n", [(1, 1, 1), (7, 7, 1), (40, 33, 5), (64, 64, 64), (1000, 1000, 1), (1025, 1020, 37), (5000, 5000, 700)])
def test_evict(S, limit, n, kind):
    B, H = 4, 2
    g = gen(S, limit, n, len(kind))
    w = strange_weights(B, H, S, g, kind)
    length = [limit, max(0, limit - n // 2), max(0, limit - n), 0]
    pos = torch.stack([torch.randperm(2 * S, generator=g)[:S] for _ in range(B * H)]).view(B, H, S).int()
    pos[torch.rand(B, H, S, generator=g) < 0.05] = -1
    for p, sinks, recent in ((None, 0, 0), (pos, 0, 0), (pos, 3, 0), (pos, 3, S // 2), (pos, 0, 4 * S)):
        cache = weight_cache(w, p)
        ws = cs.QCacheWorkspace(cache)
        slots = torch.full((B, H, n), -7, dtype=torch.int32, device="cuda")
        nxt = [2 * S, 2 * S, S, 1]
        cs.cs_qcache_evict(cache, ints(length), limit, slots, ws, next_pos=ints(nxt), sinks=sinks, recent=recent)
        assert torch.equal(slots.cpu(), ref.evict(w, p, length, limit, n, sinks, recent, nxt))
        assert cs.cs_get_device_error(ws) == 0


@pytest.mark.parametrize("S", [20000, 70001])
def test_evict_long(S):
    g = gen(S)
    w = strange_weights(2, 1, S, g, "plain")
    w[1] = (w[1] * 8).round()
    cache = weight_cache(w, None)
    for n in (1, 3, S // 3):
        slots = torch.empty(2, 1, n, dtype=torch.int32, device="cuda")
        cs.cs_qcache_evict(cache, ints([S, S - 1]), S, slots, cs.QCacheWorkspace(cache))
        assert torch.equal(slots.cpu(), ref.evict(w, None, [S, S - 1], S, n))


def test_evict_length_above_the_limit_is_flagged():
    g = gen(21)
    w = strange_weights(1, 2, 30, g, "plain")
    cache = weight_cache(w, None)
    ws = cs.QCacheWorkspace(cache)
    slots = torch.empty(1, 2, 4, dtype=torch.int32, device="cuda")
    cs.cs_qcache_evict(cache, ints([25]), 20, slots, ws)
    assert torch.equal(slots.cpu(), ref.evict(w, None, [20], 20, 4)) and cs.cs_get_device_error(ws) == cs.CS_DEVERR_COUNT


@pytest.mark.parametrize("kind", ["plain", "ties", "specials"])
@pytest.mark.parametrize("S,keep,cap,d", [(1, 1, 1, 64), (50, 17, 20, 64), (300, 299, 300, 128), (513, 100, 100, 192), (700, 700, 701, 256), (30, 200, 200, 128)])
def test_trim(S, keep, cap, d, kind):
    B, H = 3, 2
    g = gen(S, keep, d, len(kind))
    src, cpu = filled(B, H, S, d, g)
    w = strange_weights(B, H, S, g, kind)
    src.weight.copy_(w)
    pos = cpu[5]
    length, nxt = [S, S // 2, 0], [S, S, 5]
    dst, old = filled(B, H, cap, d, g)
    ws = cs.QCacheWorkspace(src)
    cs.cs_qcache_trim(src, ints(length), keep, dst, ws, next_pos=ints(nxt), sinks=2, recent=5)
    left = ref.stays(w, pos, length, keep, 2, 5, nxt)
    for name, i in (("k", 0), ("k_scale", 1), ("v", 2), ("v_scale", 3), ("weight", 4), ("pos", 5)):
        want, have = old[i].clone(), (w if name == "weight" else cpu[i])
        for b in range(B):
            for h in range(H):
                want[b, h, :len(left[b][h])] = have[b, h, left[b][h]]
        got = getattr(dst, name).cpu()
        assert np.array_equal(got.numpy(), want.numpy(), equal_nan=name == "weight"), name


# ------------------------------------------------------------------------------------------------------------ all together

def test_steps_in_a_captured_graph():
    """Evict, append and attend as one captured step, replayed with new tokens and grown lengths, against the plain forms."""
    B, H, G, S, d, steps = 2, 2, 2, 8, 64, 14
    g = gen(33)
    cache = cs.QCache.empty(B, H, S, d)
    ws = cs.QCacheWorkspace(cache, n_heads=H * G)
    length, nxt = ints([0, 3]), ints([0, 3])
    x0 = torch.randn(B, 3, H, d, generator=g)
    cs.cs_qcache_append(cache, x0.cuda(), x0.cuda(), ws, start=ints([0, 0]), n_new=ints([0, 3]), pos=ints([0, 0]))
    q, k, v = (torch.zeros(B, 1, n, d, device="cuda") for n in (H * G, H, H))
    out, slots = torch.zeros_like(q), torch.zeros(B, H, 1, dtype=torch.int32, device="cuda")

    def step():
        cs.cs_qcache_evict(cache, length, S, slots, ws, next_pos=nxt, sinks=1, recent=2)
        cs.cs_qcache_append(cache, k, v, ws, slots=slots, pos=nxt)
        length.add_(1).clamp_(max=S)
        cs.cs_qcache_attention(cache, q, length, out, ws, q_pos=nxt, weight=cache.weight, decay=0.9)
        nxt.add_(1)

    state = [t.clone() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos, length, nxt)]
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((cache.k, cache.k_scale, cache.v, cache.v_scale, cache.weight, cache.pos, length, nxt), state):
        t.copy_(s)
    ck, cks, cv, cvs, cw, cp = (t.cpu() for t in state[:6])
    n, at = [0, 3], [0, 3]
    for i in range(steps):
        qi, ki, vi = (torch.randn(B, 1, m, d, generator=g) for m in (H * G, H, H))
        q.copy_(qi), k.copy_(ki), v.copy_(vi)
        graph.replay()
        want = ref.evict(cw, cp, n, S, 1, 1, 2, at)
        assert torch.equal(slots.cpu(), want)
        ix = (torch.arange(B)[:, None, None], torch.arange(H)[None, :, None], want.long())
        (ck[ix], cks[ix]), (cv[ix], cvs[ix]) = ref.quantise(ki.transpose(1, 2)), ref.quantise(vi.transpose(1, 2))
        cw[ix] = 0.0
        cp[ix] = torch.tensor(at, dtype=torch.int32)[:, None, None].expand(B, H, 1)
        n = [min(x + 1, S) for x in n]
        ro, re, rw, rwe = ref.attention(ck, cks, cv, cvs, cp, qi, n, q_pos=at, old=cw, decay=0.9)
        at = [x + 1 for x in at]
        assert ((out.cpu().double() - ro).abs() <= re + 2.0 ** -24 * (ro.abs() + re)).all()
        got = cache.weight.cpu()
        assert ((got.double() - rw).abs() <= rwe).all()
        cw = got    # the next step's choice goes by the weights that the GPU holds
    assert torch.equal(cache.k.cpu(), ck) and torch.equal(cache.v_scale.cpu(), cvs) and torch.equal(cache.pos.cpu(), cp)
    assert cs.cs_get_device_error(ws) == 0
