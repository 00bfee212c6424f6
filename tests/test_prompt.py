"""Host side of the prompt's, the tree's, append_rows' and fork's calls: refusals before any CUDA call, and the plain forms."""
import ctypes as C

import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs
from contextual_sparsity_sparse_gb300 import build as cb

import _prompt_ref as ref
from test_qcache import BAD_CACHES, BAD_CODES, INVALID, P, UNSUPPORTED, WORKSPACE, cache, ref_, rows

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    cb.build()
    return cs.lib()


def r16(data=P, dtype=F16, ldb=512, ldt=512, ldh=128):
    return rows(data, dtype, ldb, ldt, ldh)


PROMPT = dict(q=r16(), k=r16(2 * P), v=r16(3 * P), heads=4, kv=2, d=128, batch=2, qs=P, tq=10, ks=P, tk=20, causal=1, scale=0.0,
              out=r16(4 * P), ws=P, wsb=1 << 30)


def prompt(lib, **change):
    a = dict(PROMPT, **change)
    return lib.cs_prompt_attention(ref_(a["q"]), ref_(a["k"]), ref_(a["v"]), a["heads"], a["kv"], a["d"], a["batch"], a["qs"], a["tq"],
                                   a["ks"], a["tk"], a["causal"], a["scale"], ref_(a["out"]), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=rows(None)), INVALID), (dict(v=r16(dtype=BF16)), INVALID), (dict(out=r16(4 * P, dtype=3)), INVALID),
    (dict(q=r16(P + 8)), INVALID), (dict(k=r16(ldt=508)), INVALID), (dict(v=r16(ldh=4)), INVALID), (dict(out=r16(4 * P + 2)), INVALID),
    (dict(q=r16(ldt=-512)), INVALID), (dict(batch=0), INVALID), (dict(batch=4097), UNSUPPORTED), (dict(heads=3), INVALID),
    (dict(kv=0), INVALID), (dict(heads=258), UNSUPPORTED), (dict(heads=1026, kv=513), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(tq=-1), INVALID), (dict(tk=-1), INVALID), (dict(qs=None), INVALID), (dict(qs=P + 2), INVALID),
    (dict(ks=P + 1), INVALID), (dict(ks=None), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(out=r16(2 * P)), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=P + 8), WORKSPACE), (dict(wsb=16), WORKSPACE),
    (dict(tq=1 << 25), UNSUPPORTED),
    (dict(q=rows(dtype=F32), k=rows(2 * P, F32), v=rows(3 * P, F32), out=rows(4 * P, F32)), UNSUPPORTED)])
def test_prompt_refusals(lib, change, status):
    assert prompt(lib, **change) == status
    assert lib.cs_last_error()


def test_a_prompt_without_query_tokens_is_nothing(lib):
    assert prompt(lib, tq=0, q=r16(None), out=r16(None)) == 0


def test_prompt_workspace_sizes(lib):
    size = lib.cs_prompt_workspace_size
    assert size(1, 1, 1, 64, 0, 0) > 0 and size(4096, 1024, 8, 128, 100000, 100000) > 0
    for bad in ((0, 1, 1, 64, 1, 1), (4097, 1, 1, 64, 1, 1), (1, 3, 2, 64, 1, 1), (1, 129, 1, 64, 1, 1), (1, 1, 1, 96, 1, 1),
                (1, 1, 1, 64, -1, 1), (1, 0, 1, 64, 1, 1)):
        assert size(*bad) == 0


TREE = dict(q=r16(), k=r16(2 * P), v=r16(3 * P), heads=8, n=5, length=P, parent=P, n_new=P, scale=0.0, out=r16(4 * P), ws=P, wsb=1 << 30)


def tree(lib, c, **change):
    a = dict(TREE, **change)
    return lib.cs_qcache_tree_attention(ref_(c), ref_(a["q"]), ref_(a["k"]), ref_(a["v"]), a["heads"], a["n"], a["length"], a["parent"],
                                        a["n_new"], a["scale"], ref_(a["out"]), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=r16(dtype=BF16)), INVALID), (dict(out=r16(P)), INVALID),
    (dict(out=r16(3 * P)), INVALID), (dict(heads=7), INVALID), (dict(heads=0), INVALID), (dict(n=0), INVALID), (dict(n=129), UNSUPPORTED),
    (dict(heads=64, n=65), UNSUPPORTED), (dict(length=None), INVALID), (dict(length=P + 1), INVALID), (dict(parent=P + 2), INVALID),
    (dict(n_new=P + 2), INVALID), (dict(scale=float("inf")), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE),
    (dict(q=rows(), k=rows(2 * P), v=rows(3 * P), out=rows(4 * P)), UNSUPPORTED)])
def test_tree_refusals(lib, change, status):
    assert tree(lib, cache(), **change) == status
    assert lib.cs_last_error()


@pytest.mark.parametrize("bad,status", BAD_CACHES + BAD_CODES + [(dict(d_head=192), UNSUPPORTED)])
def test_bad_caches_are_refused(lib, bad, status):
    assert tree(lib, cache(**bad)) == status
    if bad != dict(d_head=192):
        assert lib.cs_qcache_append_rows(ref_(cache(**bad)), ref_(rows()), ref_(rows()), 9, P, 1, P, None, P, P, 1 << 20, None) == status
        assert lib.cs_qcache_fork(ref_(cache(**bad)), P, P, None, P, 1 << 20, None) == status
        assert lib.cs_qcache_fork(ref_(cache(k=9 * P, v=9 * P, ks=9 * P, vs=9 * P, weight=9 * P, pos=9 * P)), P, P, ref_(cache(**bad)), P,
                                  1 << 20, None) == status


def test_tree_workspace_sizes(lib):
    size = lib.cs_qcache_tree_workspace_size
    assert size(1, 1, 1, 64, 1, 1) > 0 and size(64, 8, 131072, 128, 64, 64) > 0
    for bad in ((0, 1, 1, 64, 1, 1), (1, 1, 1, 192, 1, 1), (1, 2, 1, 64, 3, 1), (1, 1, 1, 64, 1, 0), (1, 1, 1, 64, 1, 129),
                (1, 1, 1, 64, 16, 65), (1, 2, 1, 64, 1, 1)):
        assert size(*bad) == 0


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID), (dict(v=rows(dtype=F16)), INVALID), (dict(k=rows(P + 2)), INVALID), (dict(n_rows=-1), INVALID), (dict(n=-1), INVALID),
    (dict(rows=None), INVALID), (dict(rows=P + 2), INVALID), (dict(start=None), INVALID), (dict(slots=P), INVALID), (dict(pos=None), INVALID),
    (dict(pos=P + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE), (dict(n_rows=1 << 25), INVALID)])
def test_append_rows_refusals(lib, change, status):
    a = dict(k=rows(), v=rows(), n_rows=7, rows=P, n=2, start=P, slots=None, pos=P, ws=P, wsb=1 << 20, **{})
    a.update(change)
    assert lib.cs_qcache_append_rows(ref_(cache()), ref_(a["k"]), ref_(a["v"]), a["n_rows"], a["rows"], a["n"], a["start"], a["slots"],
                                     a["pos"], a["ws"], a["wsb"], None) == status


def other(**change):
    return cache(**dict(dict(k=9 * P, v=10 * P, ks=11 * P, vs=12 * P, weight=13 * P, pos=14 * P), **change))


@pytest.mark.parametrize("dst,source,length,ws,status", [
    (None, None, P, P, INVALID), (None, P, None, P, INVALID), (None, P + 2, P, P, INVALID), (None, P, P, None, WORKSPACE),
    (other(n_heads=3), P, P, P, INVALID), (other(d_head=64), P, P, P, INVALID), (other(weight=None), P, P, P, INVALID),
    (other(pos=None), P, P, P, INVALID), (other(k=P), P, P, P, INVALID), (other(pos=P), P, P, P, INVALID),
    (cache(batch=1), P, P, P, INVALID), (cache(ldh=101), P, P, P, INVALID)])
def test_fork_refusals(lib, dst, source, length, ws, status):
    assert lib.cs_qcache_fork(ref_(cache()), source, length, ref_(dst), ws, 1 << 20, None) == status


def test_python_refusals():
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="no call takes"):
        cs.PromptWorkspace(1, 3, 2, 64, 10)
    ws = type("W", (), dict(ptr=256, nbytes=1 << 20))()
    with pytest.raises(ValueError, match="CUDA"):
        cs.cs_prompt_attention(q, q, q, q.clone(), torch.zeros(2, dtype=torch.int32), ws, stream=0)
    with pytest.raises(ValueError, match="contiguous rows"):
        cs.cs_prompt_attention(q.transpose(1, 2), q, q, q, torch.zeros(2, dtype=torch.int32), ws, stream=0)


# ------------------------------------------------------------------------------------------------------- the plain forms

def test_plain_prompt_is_softmax_attention():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(7, h, 64, generator=g).half() for h in (4, 2, 2))
    out, bound = ref.prompt(q, k, v, [3, 0, 4], [3, 0, 4])
    want = torch.nn.functional.scaled_dot_product_attention(*(t[3:].double().transpose(0, 1) for t in (q, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1))),
                                                            is_causal=True)
    assert torch.allclose(out[3:].transpose(0, 1), want) and (bound > 0).all()
    out, _ = ref.prompt(q[:3], k[:1], v[:1], [3], [1])
    assert (out[:2] == 0).all() and torch.equal(out[2, 0], v[0, 0].double())


def test_plain_paths():
    p = ref.paths(torch.tensor([-1, 0, 0, 2, -1]), 5)
    assert [set(torch.nonzero(r).flatten().tolist()) for r in p] == [{0}, {0, 1}, {0, 2}, {0, 2, 3}, {4}]
    assert torch.equal(ref.paths(None, 4), torch.ones(4, 4, dtype=torch.bool).tril())


def test_workspaces_of_larger_sizes_have_room_for_smaller_calls():
    """Fewer key/value heads make larger groups, and so more works: sizes do not fall with any argument."""
    lib_ = cs.lib()
    heads = [(h, k) for k in (1, 2, 8, 64) for h in (1, 2, 8, 16, 64, 128) if h % k == 0 and h >= k]
    sizes = {(b, h, k, d, t): lib_.cs_prompt_workspace_size(b, h, k, d, t, t)
             for b in (1, 300) for h, k in heads for d in (64, 128) for t in (1, 500, 1025, 100000)}
    trees = {(b, h, k, d, s, n): lib_.cs_qcache_tree_workspace_size(b, k, s, d, h, n)
             for b in (1, 300) for h, k in heads for d in (64, 128) for s in (100, 5000) for n in (1, 3, 8)}
    for table in (sizes, trees):
        assert all(table.values())
        for small, x in table.items():
            for large, y in table.items():
                if all(a <= b for a, b in zip(small, large)):
                    assert x <= y, (small, large)


def test_more_than_can_change_places_is_refused(lib):
    for batch, d in ((1793, 256), (3585, 128)):
        c = cache(batch=batch, d_head=d, n_heads=1)
        assert lib.cs_qcache_fork(ref_(c), P, P, None, P, 1 << 20, None) == UNSUPPORTED and lib.cs_last_error()


def test_strides_that_no_row_is_reached_by_may_be_anything(lib):
    """Between sequences, where rows are packed; between tokens or heads, where there is one."""
    odd = dict(ldb=-5, ldt=512, ldh=128)
    none = dict(tq=0, q=r16(None, **odd), out=r16(None, **odd))     # so that nothing is launched
    assert prompt(lib, k=r16(2 * P, **odd), v=r16(3 * P, ldb=3, ldt=512, ldh=128), **none) == 0
    one = dict(ldb=1, ldt=129, ldh=-3)
    assert prompt(lib, heads=1, kv=1, tk=1, k=r16(2 * P, **one), v=r16(3 * P, **one), **none) == 0
    assert prompt(lib, heads=1, kv=1, tk=2, k=r16(2 * P, **one), v=r16(3 * P, **one), **none) == INVALID
    assert prompt(lib, heads=4, kv=2, tk=1, k=r16(2 * P, **one), v=r16(3 * P, **one), **none) == INVALID
    append = lambda r: lib.cs_qcache_append_rows(ref_(cache()), ref_(r), ref_(r), 7, P, 0, P, None, P, P, 1 << 20, None)  # noqa: E731
    assert append(rows(ldb=-1)) == 0 and append(rows(ldt=-1)) == INVALID
