"""How near attention over the 4-bit cache comes to its 64-bit form, where slots, groups and rows differ widely in size.

Caches are made of codes and scales outright.  All keys have scale 1/4 and offset -2; channel 0 steers a slot's logit (code
8 is 0, so the slots that matter have small logits and no rounding of theirs hides the values').  Values have offset 0 and
positive scales, so that nothing cancels in an output, and an error may be measured against it.

The fp32 tolerance, relative to the norm of one row's 64 channels of a group: the exponential 2^-22, p s as an operand 2^-22,
a unit's products (six sums cut off after 24 bits, 2^-24 each on average) and the sums of p and of units 2^-23 each, which is
2^-21 with the roundings of the join; and for logits of size X two roundings, 2^-23 X.  A 16-bit output is rounded once, and its
products carry 2^-16 (two parts of 8 bits) and logits 2^-20 of the sum of their terms' sizes (cut off after 24 bits, 16 at a time).
"""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _qcache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def steered(B, kv, S, d, group, dt, g, lead):
    """codes, scales of keys and values, and queries for which a slot's logit is lead (code - 8) / 8 beside small terms."""
    G = d // 64
    kn = torch.randint(4, 13, (B, kv, S, d), generator=g)
    kn[..., 0] = 8
    ks = torch.tensor([0.25, -2.0]).half().expand(B, kv, S, G, 2).clone()
    vn = torch.randint(0, 16, (B, kv, S, d), generator=g)
    vs = torch.zeros(B, kv, S, G, 2, dtype=torch.float16)
    vs[..., 0] = (0.02 * (1 + 0.5 * torch.rand(B, kv, S, G, generator=g))).half()
    q = 0.2 * torch.randn(B, 1, kv * group, d, generator=g)
    q[..., 0] = lead / 2 * d ** 0.5
    return kn, ks, vn, vs, q.to(dt)


def packed(n):
    return (n[..., 0::2] + 16 * n[..., 1::2]).to(torch.uint8)


def check(kn, ks, vn, vs, q, dt):
    """Runs the call; each row's and group's error against the 64-bit form."""
    B, kv, S, d = kn.shape
    group = q.shape[2] // kv
    cache = cs.QCache(packed(kn).cuda(), packed(vn).cuda(), ks.cuda(), vs.cuda())
    out = torch.empty_like(q, device="cuda")
    ws = cs.QCacheWorkspace(cache, n_heads=q.shape[2])
    cs.cs_qcache_attention(cache, q.cuda(), torch.full((B,), S, dtype=torch.int32, device="cuda"), out, ws)
    got = out.cpu().double().view(B, kv, group, d)
    for b in range(B):
        for h in range(kv):
            k, v = ref.values(packed(kn[b, h]), ks[b, h]), ref.values(packed(vn[b, h]), vs[b, h])
            x = q[b, 0].double().view(kv, group, d)[h]
            s = x @ k.T * d ** -0.5
            p = s.softmax(-1)
            want = p @ v
            err = got[b, h] - want
            if dt == torch.float32:
                most = (p * s.abs()).sum(-1, keepdim=True)   # the size of the logits that matter
                rel = err.view(group, -1, 64).norm(dim=-1) / want.view(group, -1, 64).norm(dim=-1)
                assert (rel <= 2.0 ** -21 + 2.0 ** -23 * most).all(), rel
            else:
                a = (x.abs() @ k.abs().T * d ** -0.5 + 4 * x.abs().sum(-1, keepdim=True) * d ** -0.5).max()
                wide = p @ (15 * vs[b, h, :, :, 0].double()).repeat_interleave(64, -1)
                bound = (2.0 ** -16 + 2.0 ** -20 * a) * wide
                half = ref.half_step(dt)
                assert (err.abs() <= bound + half * (want.abs() + bound)).all()


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 104729 * int(k) for i, k in enumerate(key)) + 3)


DTS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8, 16])
@pytest.mark.parametrize("S", [31, 2000])
def test_alike(S, group, d, dt):
    g = gen(S, group, d)
    check(*steered(1, 2, S, d, group, dt, g, 0.0), dt)


@pytest.mark.parametrize("group", [1, 8])
def test_long(group):
    g = gen(group)
    check(*steered(1, 1, 60001, 128, group, torch.float32, g, 0.0), torch.float32)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("wide", [12, 17])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_a_wide_slot_without_weight(group, d, wide, dt):
    """One slot in ten has value scales 2^wide of the others' and e^-60 of their weight."""
    S = 250
    g = gen(group, d, wide)
    kn, ks, vn, vs, q = steered(1, 2, S, d, group, dt, g, 60.0)
    kn[:, :, 5::10, 0] = 0
    vs[:, :, 5::10, :, 0] *= 2.0 ** wide
    check(kn, ks, vn, vs, q, dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("wide", [12, 17])
@pytest.mark.parametrize("d", [128, 192, 256])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_a_wide_group(group, d, wide, dt):
    """The first 64 channels' scales are 2^wide of the others'."""
    g = gen(group, d, wide, 1)
    kn, ks, vn, vs, q = steered(1, 2, 250, d, group, dt, g, 0.0)
    vs[..., 0, 0] *= 2.0 ** wide
    check(kn, ks, vn, vs, q, dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("group", [2, 8, 16])
def test_a_wide_slot_for_one_row(group, dt):
    """One query head looks at the wide slot alone, the others at all but it."""
    g = gen(group, 2)
    kn, ks, vn, vs, q = steered(1, 2, 250, 128, group, dt, g, 60.0)
    kn[:, :, 77, 0] = 0
    vs[:, :, 77, :, 0] *= 2.0 ** 17
    q[:, :, ::group, 0] *= -1
    check(kn, ks, vn, vs, q, dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_wide_slots_first(group, d, dt):
    """The first half of the slots is wide and has e^-30 of the weight; with this many heads a warp goes over both halves."""
    S = 512
    g = gen(group, d, 3)
    kn, ks, vn, vs, q = steered(16, 16, S, d, group, dt, g, 60.0)
    kn[:, :, :S // 2, 0] = 4
    vs[:, :, :S // 2, :, 0] *= 2.0 ** 17
    check(kn, ks, vn, vs, q, dt)


@pytest.mark.parametrize("group", [1, 8])
def test_long_heads_of_16_bits_do_not_drift(group):
    """304 heads of 400,000 slots: a CTA has a whole head or more to itself, and a warp of it sums up 50,000 slots.  All slots
    weigh the same and a channel's code is the same in all of them (12 to 15), so the output is a mean that is easily told.
    A rounding to fp16 is off by 2^-11 / sqrt(3) at the most in the mean square, and over 304 x 4 values that is 2^-11 / 60 =
    8e-6 of the mean; four times that are allowed."""
    B, kv, S, d = 38, 8, 400_000, 64
    g = torch.Generator("cuda").manual_seed(group)
    k = torch.zeros(B, kv, S, d // 2, dtype=torch.uint8, device="cuda")
    v = torch.tensor([0xdc, 0xfe], dtype=torch.uint8, device="cuda").repeat(d // 4).expand(B, kv, S, d // 2).contiguous()
    ks = torch.zeros(B, kv, S, 1, 2, dtype=torch.float16, device="cuda")
    vs = torch.rand(B, kv, S, 1, 2, generator=g, device="cuda").add_(0.5).half()
    cache = cs.QCache(k, v, ks, vs)
    q = torch.zeros(B, 1, kv * group, d, dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    ws = cs.QCacheWorkspace(cache, n_heads=kv * group, weights=False)
    cs.cs_qcache_attention(cache, q, torch.full((B,), S, dtype=torch.int32, device="cuda"), out, ws)
    code = torch.tensor([12, 13, 14, 15], dtype=torch.float64, device="cuda").repeat(d // 4)
    s, z = (vs[..., 0, i].double().mean(-1)[..., None] for i in (0, 1))
    want = (z + s * code).view(B, 1, kv, 1, d)
    rel = out.double().view(B, 1, kv, group, d) / want - 1
    assert rel.mean().abs() <= 4 * 2.0 ** -11 / 60 and rel.abs().max() <= 2.0 ** -11 + 1e-5
