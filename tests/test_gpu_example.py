"""The bounded-cache example runs as it stands, and with a budget that holds every token its only error is the
quantisation's."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build()
    spec = importlib.util.spec_from_file_location("bounded_cache", os.path.join(ROOT, "examples", "bounded_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_bounded(example):
    cache, at, worst = example.main(steps=6, prompt=300, budget=64, sinks=3, recent=10)
    # every head still has the first tokens and the latest ones, and no token twice (100 more steps were timed)
    for row in cache.pos.flatten(0, 1).tolist():
        assert len(set(row)) == 64 and min(row) >= 0
    now = int(at[0])
    kept = set(cache.pos[0, 0].tolist())
    assert {0, 1, 2} <= kept and set(range(now - 10, now)) <= kept
    assert worst < 1.0


def test_with_room_for_all_tokens(example):
    """300 prompt tokens fit the budget's slots, and two new ones take the places of the lightest.  4 bits are 15 steps
    over the about 5 standard deviations that 64 values span, so a value is off by 5 / 15 / sqrt(12) = 0.1 of its size,
    and a logit of 128 channels of a query of length 14 by 14 x 0.1 / sqrt(128) x sqrt(128 / 128) = 0.12: together below
    a quarter of the output."""
    _, _, worst = example.main(steps=2, prompt=300, budget=300, sinks=3, recent=10)
    assert worst < 0.25
