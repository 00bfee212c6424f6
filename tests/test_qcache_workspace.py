"""How much workspace the 4-bit cache's calls ask for."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs
from contextual_sparsity_sparse_gb300 import build as cb

MB = 1 << 20


@pytest.fixture(scope="module")
def size():
    cb.build()
    return cs.lib().cs_qcache_workspace_size


# batch, cache heads, slots, channels, query heads, query tokens
SHAPES = [(256, 8, 4096, 64, 128, 1), (32, 8, 4096, 64, 128, 1), (64, 8, 8192, 128, 64, 1), (1, 8, 131001, 128, 64, 1),
          (64, 8, 8192, 256, 128, 4), (4, 304, 1000, 64, 304, 1), (4, 114, 1000, 128, 114, 1), (1, 1, 1, 64, 1, 1), (4096, 1, 1, 64, 16, 1)]


def columns(rows):
    return 4 if rows <= 4 else 8 if rows <= 8 else 16


def slots_and(b, kv, cap, heads, n_q, more):
    return b * kv * cap * 4 * columns(heads // kv * n_q) + more


@pytest.mark.parametrize("shape", SHAPES)
def test_logits_take_no_more_than_a_word_per_slot_and_column(size, shape):
    b, kv, cap, d, heads, n_q = shape
    # beside the logits: the records, at most 304 CTAs x 2 x 16 columns x 259 floats, and a trim's list
    assert 0 < size(*shape) <= slots_and(b, kv, cap, heads, n_q, 15 * MB + 11 * MB) or size(*shape) <= b * kv * cap * 4 + MB


def test_many_sequences_of_a_few_ctas_heads(size):
    """A CTA keeps the logits of two heads at the most, however many sequences there are."""
    small, large = size(64, 8, 4096, 64, 128, 1), size(1024, 8, 4096, 64, 128, 1)
    trim = 4 * 8 * 4096 * 1024
    assert large <= max(2 * small, 2 * trim)


def test_calls_without_attention(size):
    assert size(64, 8, 8192, 128, 0, 1) == 256 + 4 * 64 * 8 * 8192
    assert size(64, 8, 8192, 128, 0, 0) == size(64, 8, 8192, 128, 0, 1)
    assert size(64, 8, 8192, 128, 64, 0) == 0 and size(64, 8, 0, 128, 0, 1) == 0 and size(64, 8, 9, 96, 0, 1) == 0


def test_attention_without_weights_asks_for_no_logits(size, monkeypatch):
    """Refused for its workspace, or not: n_q 0 comes after the check and launches nothing."""
    import ctypes as C
    P = 4096
    c = cs._QCache(64, 8, 128, 1 << 20, 0, 0, P, P, P, P, P, P)
    r = cs._Rows(None, 0, 0, 0, 0)
    few = size(64, 8, 1, 128, 64, 1)
    assert few < 12 * MB

    def call(weight, n_bytes):
        return cs.lib().cs_qcache_attention(C.byref(c), C.byref(r), 64, 0, P, None, None, 0.0, 1.0, weight, C.byref(r), P, n_bytes, None)
    assert call(None, few) == 0
    assert call(P, few) == 5   # CS_ERR_WORKSPACE


def test_python_workspaces(size, monkeypatch):
    asked = []
    monkeypatch.setattr(cs, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(cs, "_stream", lambda s: 0)

    class Lib:
        def cs_qcache_workspace_size(self, *a):
            asked.append(a)
            return size(*a)

        def cs_workspace_init(self, *a):
            return 0
    monkeypatch.setattr(cs, "lib", Lib)
    lead = (2, 3, 5000)
    w = torch.zeros(lead)
    assert cs.QCacheWorkspace(cs.QCache(None, None, None, None, weight=w), n_heads=3).nbytes <= 1024
    k, s = torch.zeros(lead + (32,), dtype=torch.uint8), torch.zeros(lead + (1, 2), dtype=torch.float16)
    full = cs.QCache(k, k.clone(), s, s.clone(), weight=w)
    assert cs.QCacheWorkspace(full).nbytes == size(*lead, 64, 3, 1)
    assert cs.QCacheWorkspace(full, n_heads=0).nbytes == size(*lead, 64, 0, 1)
    lean = cs.QCacheWorkspace(full, n_heads=6, n_q=4, weights=False)
    assert max(size(2, 3, 1, 64, 6, 4), size(*lead, 64, 0, 1)) == lean.nbytes < size(*lead, 64, 6, 4)
    with pytest.raises(ValueError):
        cs.QCacheWorkspace(full, n_heads=4)
    with pytest.raises(ValueError):
        cs.QCacheWorkspace(full, n_heads=4, weights=False)
