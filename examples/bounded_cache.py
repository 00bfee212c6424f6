"""Decoding with a bounded cache in 4 bits, and with few heads per token.

One attention layer serves a batch of sequences whose KV cache has a fixed
budget of slots.  A prompt's keys and values are quantised into a cache of
their own, its last tokens' attention shows which of them matter, and the
heaviest are taken over into the decode cache.  Then every step, captured once
as a CUDA graph and replayed,

  1. chooses the heads to compute (a low-rank predictor and top-k, as for FFN neurons),
  2. gives up the slots that gathered the least attention, if the budget is used up,
  3. quantises the new token into them, and
  4. attends with the chosen heads, adding each slot's weight to its account.

    python examples/bounded_cache.py [--steps 64]

Tokens are synthetic: one in twenty is one that queries look for, the others
get little attention each.  The printed difference is against attention in 64
bits over every token's unquantised keys and values: what the budget and the 4
bits cost together.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import contextual_sparsity_sparse_gb300 as cs  # noqa: E402


def full_attention(q, k, v, on):
    """q [B, H, d] over all of k, v [B, n, G, d] in 64 bits; heads that are not on give zeros."""
    B, H, d = q.shape
    rows = q.double().view(B, k.shape[2], -1, d)
    s = torch.einsum("bgrd,bngd->bgrn", rows, k.double()) * d ** -0.5
    out = torch.einsum("bgrn,bngd->bgrd", s.softmax(-1), v.double()).reshape(B, H, d)
    return torch.where(on[..., None], out, 0.0)


def main(steps=64, batch=4, heads=32, kv_heads=8, d_head=128, prompt=1500, budget=512, sinks=4, recent=64, rank=64,
         active=24, device="cuda"):
    g = torch.Generator(device).manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    d = heads * d_head
    dtype = torch.bfloat16

    # what the queries of a cache head look for, and one key in twenty has
    sought = torch.nn.functional.normalize(rand(kv_heads, d_head), dim=-1)

    def keys(n):
        found = (torch.rand((batch, n, kv_heads, 1), generator=g, device=device) < 0.05).float()
        return (rand(batch, n, kv_heads, d_head) + 9 * found * sought).to(dtype)

    def queries(n):
        return (rand(batch, n, heads, d_head) + 9 * sought.repeat_interleave(heads // kv_heads, 0)).to(dtype)

    # ---- the prompt: quantise it, let its last tokens attend, keep what they looked at
    length = torch.full((batch,), prompt, dtype=torch.int32, device=device)
    zero = torch.zeros_like(length)
    whole = cs.QCache.empty(batch, kv_heads, prompt, d_head, device=device)
    ws = cs.QCacheWorkspace(whole, n_heads=heads, n_q=4)
    pk, pv = keys(prompt), rand(batch, prompt, kv_heads, d_head).to(dtype)
    cs.cs_qcache_append(whole, pk, pv, ws, start=zero, pos=zero)
    pq = queries(4)
    cs.cs_qcache_attention(whole, pq, length, torch.empty_like(pq), ws, q_pos=length - 4, weight=whole.weight)
    cache = cs.QCache.empty(batch, kv_heads, budget, d_head, device=device)
    cs.cs_qcache_trim(whole, length, budget, cache, ws, next_pos=length, sinks=sinks, recent=recent)

    # ---- one decode step on fixed buffers
    pred = cs.Predictor(rand(rank, d).half() * d ** -0.5, rand(heads, rank).half() * rank ** -0.5)
    pws = cs.Workspace(d, heads, rank, B=batch, device=device)
    x = torch.zeros(batch, d, device=device)
    scores = torch.zeros(batch, heads, device=device)
    idx = torch.zeros(batch, heads, dtype=torch.int32, device=device)
    count = torch.zeros(batch, dtype=torch.int32, device=device)
    mask = torch.zeros(batch, -(-heads // 32), dtype=torch.int32, device=device)
    q, k, v = (torch.zeros(batch, 1, n, d_head, dtype=dtype, device=device) for n in (heads, kv_heads, kv_heads))
    out = torch.zeros_like(q)
    slots = torch.zeros(batch, kv_heads, 1, dtype=torch.int32, device=device)
    used, at = torch.full_like(length, budget), length.clone()
    params = cs.select_params(cs.CS_SEL_TOPK, active)

    def step():
        cs.cs_predict(pred, x, scores, pws)
        cs.cs_select(scores, params, idx, count, mask=mask, ws=pws)
        cs.cs_qcache_evict(cache, used, budget, slots, ws, next_pos=at, sinks=sinks, recent=recent)
        cs.cs_qcache_append(cache, k, v, ws, slots=slots, pos=at)
        used.add_(1).clamp_(max=budget)
        cs.cs_qcache_attention(cache, q, used, out, ws, mask=mask, weight=cache.weight)
        at.add_(1)

    kept = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.weight, cache.pos, used, at)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, cache.weight, cache.pos, used, at), kept):
        t.copy_(was)

    # ---- decode, and compare with attention over everything
    all_k, all_v, worst = [pk], [pv], 0.0
    for _ in range(steps):
        x.copy_(rand(batch, d))
        q.copy_(queries(1))
        k.copy_(keys(1))
        v.copy_(rand(batch, 1, kv_heads, d_head))
        graph.replay()
        all_k.append(k.clone())
        all_v.append(v.clone())
        on = torch.zeros(batch, heads, dtype=torch.bool, device=device)
        on.scatter_(1, idx[:, :active].long(), True)
        ref = full_attention(q[:, 0], torch.cat(all_k, 1), torch.cat(all_v, 1), on)
        worst = max(worst, ((out[:, 0].double() - ref).norm() / ref.norm()).item())
        assert not out[:, 0][~on].any()
    torch.cuda.synchronize()
    assert cs.cs_get_device_error(ws) == 0 and cs.cs_get_device_error(pws) == 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    size = sum(t.numel() * t.element_size() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.weight, cache.pos))
    print(f"{steps} steps of {batch} sequences, {active} of {heads} heads, {budget} of {prompt + steps} tokens kept: "
          f"{size / 2**20:.2f} MiB of cache, {10 * start.elapsed_time(end):.1f} us a step, "
          f"relative difference from full attention at most {worst:.3f}")
    return cache, at, worst


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=64)
    main(steps=p.parse_args().steps)
