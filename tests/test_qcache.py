"""The 4-bit KV cache's host side: refusals before any CUDA call, and the plain
forms that the GPU tests compare with."""
import ctypes as C

import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs
from contextual_sparsity_sparse_gb300 import build as cb

import _qcache_ref as ref

INVALID, UNSUPPORTED, WORKSPACE = 1, 3, 5
P = 4096   # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    cb.build()
    return cs.lib()


def cache(batch=2, n_heads=4, d_head=128, capacity=100, ldb=0, ldh=0, k=P, v=P, ks=P, vs=P, weight=P, pos=P):
    return cs._QCache(batch, n_heads, d_head, capacity, ldb, ldh, k, v, ks, vs, weight, pos)


def rows(data=P, dtype=0, ldb=512, ldt=512, ldh=128):
    return cs._Rows(data, dtype, ldb, ldt, ldh)


def ref_(x):
    return C.byref(x) if x is not None else None


BAD_CACHES = [(dict(batch=0), INVALID), (dict(n_heads=0), INVALID), (dict(capacity=0), INVALID), (dict(batch=4097), UNSUPPORTED),
              (dict(capacity=(1 << 24) + 1), UNSUPPORTED), (dict(n_heads=1025), UNSUPPORTED), (dict(ldh=99), INVALID),
              (dict(ldb=99), INVALID), (dict(weight=P + 2), INVALID), (dict(pos=P + 1), INVALID)]
BAD_CODES = [(dict(d_head=32), UNSUPPORTED), (dict(d_head=96), UNSUPPORTED), (dict(d_head=320), UNSUPPORTED), (dict(k=None), INVALID),
             (dict(vs=None), INVALID), (dict(k=P + 8), INVALID), (dict(ks=P + 2), INVALID)]


@pytest.mark.parametrize("bad,status", BAD_CACHES + BAD_CODES)
def test_bad_caches_are_refused(lib, bad, status):
    c, r = cache(**bad), rows()
    assert lib.cs_qcache_append(ref_(c), ref_(r), ref_(r), 1, P, None, None, P, P, 1 << 20, None) == status
    assert lib.cs_qcache_read(ref_(c), ref_(r), ref_(r), 1, P, None, P, 1 << 20, None) == status
    assert lib.cs_qcache_attention(ref_(c), ref_(r), 4, 1, P, None, None, 0.0, 1.0, None, ref_(rows(2 * P)), P, 1 << 30, None) == status
    assert lib.cs_qcache_trim(ref_(c), P, 10, P, 0, 0, ref_(cache(k=9 * P, v=9 * P)), P, 1 << 20, None) == status
    if (bad, status) in BAD_CACHES:
        assert lib.cs_qcache_evict(ref_(c), P, 50, 1, P, 0, 0, P, P, 1 << 20, None) == status
    assert lib.cs_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(k=rows(None)), INVALID), (dict(v=None), INVALID), (dict(k=rows(dtype=3)), INVALID), (dict(k=rows(P + 2)), INVALID),
    (dict(k=rows(dtype=1)), INVALID), (dict(k=rows(ldt=-1)), INVALID), (dict(n=-1), INVALID), (dict(start=None), INVALID),
    (dict(slots=P), INVALID), (dict(pos=None), INVALID), (dict(pos=P + 2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=P + 16), WORKSPACE), (dict(wsb=128), WORKSPACE)])
def test_append_and_read_refusals(lib, change, status):
    a = dict(k=rows(), v=rows(), n=1, start=P, slots=None, pos=P, ws=P, wsb=1 << 20, **{})
    a.update(change)
    assert lib.cs_qcache_append(ref_(cache()), ref_(a["k"]), ref_(a["v"]), a["n"], a["start"], a["slots"], None, a["pos"], a["ws"],
                                a["wsb"], None) == status
    if "pos" not in change:
        assert lib.cs_qcache_read(ref_(cache()), ref_(a["k"]), ref_(a["v"]), a["n"], a["start"], a["slots"], a["ws"], a["wsb"],
                                  None) == status


def test_calls_without_tokens_do_nothing(lib):
    none = rows(None)
    assert lib.cs_qcache_append(ref_(cache()), ref_(none), ref_(none), 0, P, None, None, P, P, 1 << 20, None) == 0
    assert lib.cs_qcache_read(ref_(cache()), ref_(none), ref_(none), 0, None, P, P, 1 << 20, None) == 0
    assert lib.cs_qcache_attention(ref_(cache()), ref_(none), 8, 0, P, None, None, 0.0, 1.0, None, ref_(none), P, 1 << 30, None) == 0


@pytest.mark.parametrize("groups,good,bad", [(1, 4, 2), (2, 8, 4), (3, 4, 2), (4, 16, 8)])
def test_scales_are_aligned_to_what_is_copied_of_a_slot(lib, groups, good, bad):
    for at, status in ((good, 0), (bad, INVALID)):
        c = cache(d_head=64 * groups, ks=P + at)
        r = rows(None)
        assert lib.cs_qcache_read(ref_(c), ref_(r), ref_(r), 0, P, None, P, 1 << 20, None) == status


def test_append_wants_positions_exactly_when_the_cache_has_them(lib):
    r = rows()
    assert lib.cs_qcache_append(ref_(cache(pos=None)), ref_(r), ref_(r), 1, P, None, None, P, P, 1 << 20, None) == INVALID
    assert b"positions" in lib.cs_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(q=rows(dtype=1)), INVALID), (dict(out=rows(P)), INVALID), (dict(heads=6), INVALID), (dict(heads=0), INVALID),
    (dict(n_q=-1), INVALID), (dict(n_q=1025), UNSUPPORTED), (dict(length=None), INVALID), (dict(length=P + 1), INVALID),
    (dict(q_pos=P, c=cache(pos=None)), INVALID), (dict(mask=P + 2), INVALID), (dict(weight=P + 2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(decay=float("nan")), INVALID),
    (dict(weight=P, c=cache(weight=None)), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=256), WORKSPACE)])
def test_attention_refusals(lib, change, status):
    a = dict(c=cache(), q=rows(), heads=8, n_q=1, length=P, q_pos=None, mask=None, scale=0.0, decay=1.0, weight=None,
             out=rows(2 * P), ws=P, wsb=1 << 30)
    a.update(change)
    assert lib.cs_qcache_attention(ref_(a["c"]), ref_(a["q"]), a["heads"], a["n_q"], a["length"], a["q_pos"], a["mask"], a["scale"],
                                   a["decay"], a["weight"], ref_(a["out"]), a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(c=cache(weight=None)), INVALID), (dict(length=None), INVALID), (dict(limit=101), INVALID), (dict(n=0), INVALID),
    (dict(n=51, limit=50), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(recent=4, next_pos=None), INVALID),
    (dict(sinks=4, c=cache(pos=None)), INVALID), (dict(slots=None), INVALID), (dict(ws=None), WORKSPACE)])
def test_evict_refusals(lib, change, status):
    a = dict(c=cache(k=None, v=None, ks=None, vs=None, d_head=0), length=P, limit=100, n=1, next_pos=P, sinks=0, recent=0, slots=P,
             ws=P, wsb=1 << 20)
    a.update(change)
    assert lib.cs_qcache_evict(ref_(a["c"]), a["length"], a["limit"], a["n"], a["next_pos"], a["sinks"], a["recent"], a["slots"],
                               a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(dst=cache(n_heads=3)), INVALID), (dict(dst=cache(d_head=64)), INVALID), (dict(keep=0), INVALID), (dict(keep=101), INVALID),
    (dict(dst=cache()), INVALID), (dict(dst=cache(k=8 * P, v=9 * P, ks=10 * P, vs=11 * P, weight=None, pos=13 * P)), INVALID),
    (dict(dst=cache(k=8 * P, v=9 * P, ks=10 * P, vs=11 * P, weight=12 * P, pos=None)), INVALID), (dict(wsb=512), WORKSPACE)])
def test_trim_refusals(lib, change, status):
    a = dict(c=cache(), dst=cache(k=8 * P, v=9 * P, ks=10 * P, vs=11 * P, weight=12 * P, pos=13 * P), keep=100, wsb=1 << 20)
    a.update(change)
    assert lib.cs_qcache_trim(ref_(a["c"]), P, a["keep"], P, 0, 0, ref_(a["dst"]), P, a["wsb"], None) == status


@pytest.mark.parametrize("sizes", [(0, 1, 1, 64, 1, 1), (1, 0, 1, 64, 1, 1), (1, 1, 0, 64, 1, 1), (1, 1, 1, 80, 1, 1),
                                   (1, 2, 1, 64, 3, 1), (1, 1, 1, 64, 1, 0), (1, 1, 1, 64, 64, 17), (4097, 1, 1, 64, 1, 1)])
def test_workspace_size_of_sizes_that_no_call_takes(lib, sizes):
    assert lib.cs_qcache_workspace_size(*sizes) == 0


def test_qcache_tensors_must_step_alike():
    k = torch.zeros(2, 3, 10, 32, dtype=torch.uint8)
    s = torch.zeros(2, 3, 10, 1, 2, dtype=torch.float16)
    for bad in (dict(v=k[..., :16]), dict(v=k.float()), dict(k_scale=s[:, :2]), dict(v_scale=None), dict(weight=torch.zeros(2, 3, 9)),
                dict(weight=torch.zeros(2, 3, 20)[..., :10]), dict(weight=torch.zeros(2, 3, 10, 2)[..., 0])):
        a = dict(k=k, v=k, k_scale=s, v_scale=s, weight=None, pos=None)
        a.update(bad)
        with pytest.raises(ValueError):
            cs.QCache(**a)
    with pytest.raises(ValueError):
        cs.QCache(None, None, None, None)


def test_plain_quantiser():
    """Worked by hand: a ramp is held exactly, a constant group by its offset, and a half goes to the even code."""
    x = torch.arange(64).float() % 16
    codes, sc = ref.quantise(x)
    assert sc.tolist() == [[1.0, 0.0]] and torch.equal(ref.values(codes, sc), x.double())
    codes, sc = ref.quantise(torch.full((64,), 2.5))
    assert sc.tolist() == [[0.0, 2.5]] and not codes.any()
    x = torch.zeros(64)
    x[:4] = torch.tensor([15.0, 0.5, 1.5, 2.5])
    assert ref.values(*ref.quantise(x))[:4].tolist() == [15.0, 0.0, 2.0, 2.0]
    x[:3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    v = ref.values(*ref.quantise(x))
    assert torch.isfinite(v).all() and v[0] > 65000 and v[1] == -65504


def test_plain_quantiser_error_is_half_a_step():
    """Every value is within half a step of what it is held as: s / 2, and what rounding the scale and the offset to fp16 moves
    (the largest code's end by 15 s 2^-11, the offset by 2^-11 of itself)."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 256, generator=g) * 3
    codes, sc = ref.quantise(x)
    s = sc[..., 0].double().repeat_interleave(64, -1)
    z = sc[..., 1].double().abs().repeat_interleave(64, -1)
    assert ((ref.values(codes, sc) - x.double()).abs() <= s / 2 + (15 * s + z) * 2.0 ** -11).all()


def test_plain_order():
    w = torch.tensor([3.0, float("nan"), 1.0, 1.0, float("-inf"), -0.0, 0.0])
    assert ref.order(w, None, 0, 0, None) == [1, 4, 5, 6, 2, 3, 0]
    pos = torch.tensor([0, 9, 5, -1, 8, 4, 3])
    assert ref.order(w, pos, 1, 2, 10) == [3, 5, 6, 2, 1, 4, 0]
