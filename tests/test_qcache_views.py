"""Which views a 4-bit cache takes: its tensors step by whole slots, and no two of its slots share memory."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

B, H, S, D = 4, 3, 10, 128


@pytest.fixture
def on_cpu(monkeypatch):
    """Addresses of CPU tensors are as good as any where nothing is launched."""
    monkeypatch.setattr(cs, "_ptr", lambda t: None if t is None else t.data_ptr())


def tensors(b=B, h=H):
    z = lambda dt, *tail: torch.zeros((b, h, S) + tail, dtype=dt)  # noqa: E731
    return dict(k=z(torch.uint8, D // 2), v=z(torch.uint8, D // 2), k_scale=z(torch.float16, D // 64, 2),
                v_scale=z(torch.float16, D // 64, 2), weight=z(torch.float32), pos=z(torch.int32))


@pytest.mark.parametrize("b,h", [(1, H), (B, 1), (1, 1)])
def test_expanded_caches_are_refused(on_cpu, b, h):
    """One sequence's (or head's) slots shared by several: a step of 0 would mean a dense cache, far past the memory."""
    views = {n: t.expand((B, H) + t.shape[2:]) for n, t in tensors(b, h).items()}
    with pytest.raises(ValueError, match="expanded"):
        cs.QCache(**views)
    with pytest.raises(ValueError, match="expanded"):
        cs.QCache(None, None, None, None, weight=views["weight"], pos=views["pos"])


@pytest.mark.parametrize("b,h", [(1, H), (B, 1)])
def test_expanded_weights_of_the_attention_are_refused(on_cpu, b, h):
    cache = cs.QCache(**tensors())
    q = torch.zeros(B, 1, H, D)
    with pytest.raises(ValueError, match="expanded"):
        cs.cs_qcache_attention(cache, q, torch.zeros(B, dtype=torch.int32), torch.zeros_like(q), None,
                               weight=torch.zeros(b, h, S).expand(B, H, S))


def test_what_is_not_expanded_is_taken(on_cpu):
    dense = cs.QCache(**tensors())
    assert (dense.ld_batch, dense.ld_head) == (H * S, S)
    # sequences and heads cut out of a larger cache, and heads before sequences
    part = cs.QCache(**{n: t[1:3, 1:] for n, t in tensors().items()})
    assert (part.ld_batch, part.ld_head) == (H * S, S)
    turned = cs.QCache(**{n: t.transpose(0, 1) for n, t in tensors().items()})
    assert (turned.ld_batch, turned.ld_head) == (S, H * S)
    # a size of 1 steps nowhere, so its stride says nothing
    one = cs.QCache(**{n: t[:1].as_strided((1,) + t.shape[1:], (0,) + t.stride()[1:]) for n, t in tensors().items()})
    assert one.ld_head == S and one.ld_batch >= S
