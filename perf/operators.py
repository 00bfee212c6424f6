"""The quantised KV cache's operators, as cases to measure: what a decode step does with a cache held in 4 bits.

A cache holds, for `batch` sequences, `kv_heads` heads and `capacity` slots, one key and one value row of `d` channels per
slot.  A row is cut into groups of 64 channels; a group keeps a scale and an offset in fp16 and 64 codes of 4 bits (byte i of
a row holds channel 2i in its low and channel 2i + 1 in its high half), which stand for offset + scale * code.  Beside each
slot stand its accumulated attention weight and the position of its token.

 append     quantises new tokens into given slots, and reads those slots back as the values they stand for
 attention  one to a few query tokens per sequence over the cache; the weight that each slot got is added to its account
 evict      the slots that the next tokens take: free ones first, then those of the least accumulated weight
 trim       a cache cut down to its `keep` heaviest slots, into another cache (read back as values)

`own` false: plain torch operations.  `own` true: the framework's calls.
"""
import random

import torch

own = False

GROUP = 64
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
F32_15TH = 1.0 / 15.0


# ------------------------------------------------------------------------------------------------------------------ cases

def _attention(name, batch, heads, kv_heads, d, capacity, dtype, n_q=1, ragged=True, causal=False, heads_on=0, weights=True):
    c = dict(op="attention", batch=batch, heads=heads, kv_heads=kv_heads, d=d, capacity=capacity, dtype=dtype, n_q=n_q,
             ragged=ragged, causal=causal, heads_on=heads_on, weights=weights)
    return dict(c, name=name) if name else c


def _append(name, batch, kv_heads, d, capacity, dtype, n, scattered):
    c = dict(op="append", batch=batch, kv_heads=kv_heads, d=d, capacity=capacity, dtype=dtype, n=n, scattered=scattered)
    return dict(c, name=name) if name else c


def _evict(name, batch, kv_heads, capacity, n, sinks, recent, ragged):
    c = dict(op="evict", batch=batch, kv_heads=kv_heads, capacity=capacity, n=n, sinks=sinks, recent=recent, ragged=ragged)
    return dict(c, name=name) if name else c


def _trim(name, batch, kv_heads, d, capacity, keep, sinks, recent, ragged):
    c = dict(op="trim", batch=batch, kv_heads=kv_heads, d=d, capacity=capacity, keep=keep, sinks=sinks, recent=recent,
             ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the first tokens of one short conversation with a small model: latency is all there is
        _attention("attention-short", 1, 8, 8, 64, 128, "fp32", ragged=False),
        # one decode token of the OPT-13B-shaped layer (40 heads of 128, 2,048 cached positions)
        _attention("attention-opt13b", 1, 40, 40, 128, 2048, "bf16", ragged=False),
        # one token over one very long document, LLaMA-70B-shaped heads (64 over 8 of 128); nothing is evicted, so no weights
        _attention("attention-long", 1, 64, 8, 128, 131001, "fp16", ragged=False, weights=False),
        # four tokens to verify per sequence (speculative decoding) with a quarter of the heads chosen
        _attention("attention-verify", 4, 32, 32, 128, 2049, "fp32", n_q=4, causal=True, heads_on=8),
        # a serving batch of Falcon-40B-shaped heads (128 over 8 of 64), lengths from one token to full
        _attention("attention-batch-d64", 32, 128, 8, 64, 4096, "bf16"),
        # a large serving batch of LLaMA-70B-shaped heads
        _attention("attention-batch", 64, 64, 8, 128, 8192, "bf16"),
        # a decode step's new tokens, each into the slot that eviction freed for its head
        _append("append-step", 64, 8, 128, 4096, "bf16", 1, True),
        # a prompt's tokens into an empty cache
        _append("append-prompt", 1, 8, 128, 8192, "bf16", 7999, False),
        # a full cache of one sequence gives up one slot per head for the next token (OPT-13B-shaped layer)
        _evict("evict-one", 1, 40, 2048, 1, 4, 64, False),
        # a batch of full and half-full caches makes room for a chunk of tokens
        _evict("evict-chunk", 64, 8, 8192, 37, 4, 256, True),
        # one long prompt's cache cut down to the budget of decoding
        _trim("trim-prompt", 1, 8, 128, 32768, 4096, 4, 512, False),
        # a batch of caches of many lengths cut down to half the longest
        _trim("trim-batch", 16, 8, 64, 4001, 2000, 4, 128, True),
    ]


MOST_ROWS = 64 * 8 * 8192 * 128   # channels in the largest listed cache
MOST_LOGITS = 64 * 64 * 8192      # query-key pairs of the largest listed case


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "evict", "trim"])
    kv = rng.choice([1, 2, 4, 5, 8, 8, 12, 40])
    d = rng.choice([64, 128, 128, 192, 256])
    batch = _log(rng, 1, 64)
    dtype = rng.choice(sorted(DTYPES))
    if op == "attention":
        group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 16])
        n_q = rng.choice([1, 1, 1, 1, 2, 3, 4])
        most = min(131072, MOST_ROWS // (batch * kv * d), MOST_LOGITS // (batch * kv * group * n_q))
        capacity = _log(rng, 1, max(1, most))
        causal = n_q > 1 or rng.random() < 0.3
        heads_on = rng.randint(1, kv * group) if rng.random() < 0.3 else 0
        return _attention(None, batch, kv * group, kv, d, capacity, dtype, n_q, rng.random() < 0.7, causal, heads_on,
                          rng.random() < 0.7)
    if op == "append":
        n = _log(rng, 1, max(1, min(8192, (7999 * 8 * 128) // (batch * kv * d))))
        capacity = n + _log(rng, 1, 2048)
        return _append(None, batch, kv, d, capacity, dtype, n, rng.random() < 0.5)
    if op == "evict":
        capacity = _log(rng, 2, min(131072, (64 * 8 * 8192) // (batch * kv)))
        n = _log(rng, 1, max(1, capacity // 4))
        sinks = rng.randint(0, min(8, capacity - n))
        recent = rng.randint(0, min(256, capacity - n - sinks))
        return _evict(None, batch, kv, capacity, n, sinks, recent, rng.random() < 0.5)
    capacity = _log(rng, 2, min(65536, (32768 * 8 * 128) // (batch * kv * d)))
    keep = _log(rng, 1, capacity)
    sinks = rng.randint(0, min(8, keep))
    recent = rng.randint(0, min(512, keep - sinks))
    return _trim(None, batch, kv, d, capacity, keep, sinks, recent, rng.random() < 0.5)


def _lengths(case):
    """The sequences' lengths, before they are shuffled: full, or evenly spread from one token to full."""
    b, s = case["batch"], case["capacity"]
    if not case["ragged"]:
        return [s] * b
    return [1 + int((i + 0.5) * (s - 1) / b) if b > 1 else s - s // 3 for i in range(b)]


def work(case):
    b = case["batch"]
    row = 0 if case["op"] == "evict" else 2 * (case["d"] // 2 + 4 * (case["d"] // GROUP))   # a slot's key and value rows
    if case["op"] == "attention":
        es = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        tokens = sum(_lengths(case))
        on = case["heads_on"] or case["heads"]
        # the fewest cache heads that so many chosen query heads can share
        kv = -(-on * case["kv_heads"] // case["heads"])
        per = row + (4 if case["causal"] else 0)
        ends = 2 * b * case["n_q"] * on * case["d"] * es
        mass = 8 * tokens * case["kv_heads"] if case["weights"] else 0
        return {"bytes": tokens * kv * per + ends + mass, "flops": 4 * tokens * on * case["n_q"] * case["d"]}
    if case["op"] == "append":
        es = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        rows = b * case["n"] * case["kv_heads"]
        # new rows in, codes, weight and position out; the codes back in, their values out
        return {"bytes": rows * (2 * 2 * case["d"] * es + 2 * row + 8), "flops": rows * 2 * case["d"] * 8}
    used = sum(_lengths(case)) * case["kv_heads"]
    if case["op"] == "evict":
        return {"bytes": used * 8 + 4 * b * case["kv_heads"] * case["n"], "flops": used}
    kept = sum(min(n, case["keep"]) for n in _lengths(case)) * case["kv_heads"]
    whole = b * case["kv_heads"] * case["keep"]
    # every weight and position, the kept rows in and out, then back in as fp16 values
    return {"bytes": used * 8 + kept * (2 * row + 8 + 8) + whole * (row + 2 * 2 * case["d"]), "flops": used + whole * 4 * case["d"]}


# ----------------------------------------------------------------------------------------------------------------- inputs

def _quantise(x):
    """Codes [..., d / 2] and (scale, offset) [..., d / 64, 2] of rows [..., d].

    scale = fp16((max - min) / 15), the quotient as a product with fp32(1 / 15); offset = fp16(min); code = the nearest of
    0..15 to (x - offset) / scale, halves to even (0 where the scale is 0).  The choice of a code is made in 64 bits."""
    g = torch.nan_to_num(x.float(), nan=0.0).clamp(-65504.0, 65504.0).unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    scale, offset = ((hi - lo) * F32_15TH).half(), lo.half()
    s = scale.double().unsqueeze(-1)
    code = ((g.double() - offset.double().unsqueeze(-1)) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15)
    code = torch.where(s > 0, code, 0.0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack([scale, offset], -1)


def _values(codes, scales):
    """The fp32 values [..., d] that codes and (scale, offset) stand for."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    s = scales.float()
    return (n * s[..., 0:1] + s[..., 1:2]).flatten(-2)


def _rows(shape, g, spread):
    """Rows as attention meets them: channels of different means and widths, a few of them outliers."""
    d = shape[-1]
    x = torch.randn(shape, generator=g, device="cuda")
    x.mul_(0.5 + torch.rand((shape[1], 1, d), generator=g, device="cuda"))
    return x.add_(spread * torch.randn((shape[1], 1, d), generator=g, device="cuda") ** 3)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = random.Random(seed)
    op, b, kv, cap = case["op"], case["batch"], case["kv_heads"], case["capacity"]
    st = {"case": case}
    if op == "append":
        d, n, dt = case["d"], case["n"], DTYPES[case["dtype"]]
        # the projection's output: one token's heads side by side
        new = _rows((b, 2 * kv, n, d), g, 0.3).to(dt).transpose(1, 2).contiguous()
        st["k"], st["v"] = new[:, :, :kv], new[:, :, kv:]
        st["at"] = torch.randint(0, cap, (b,), generator=g, device="cuda", dtype=torch.int32)   # the next position
        if case["scattered"]:
            # slots that eviction gave, another set in each head
            keys = torch.rand((b, kv, cap), generator=g, device="cuda")
            st["slots"] = keys.argsort(-1)[..., :n].sort(-1).values.to(torch.int32).contiguous()
            st["start"] = None
        else:
            st["slots"] = None
            st["start"] = torch.randint(0, cap - n + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        st["back"] = torch.empty((2, b, n, kv, d), device="cuda", dtype=dt)
        st.update(_buffers(b, kv, cap, d))
    elif op == "attention":
        d, n_q, dt = case["d"], case["n_q"], DTYPES[case["dtype"]]
        heads = case["heads"]
        lens = _lengths(case)
        r.shuffle(lens)
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kc, ks = _quantise(_rows((b, kv, cap, d), g, 0.3))
        vc, vs = _quantise(_rows((b, kv, cap, d), g, 0.1))
        q = torch.randn((b, n_q, heads, d), generator=g, device="cuda") * (0.5 + torch.rand((heads, 1), generator=g, device="cuda"))
        st["q"] = q.to(dt)
        st["out"] = torch.empty_like(st["q"])
        st.update(codes_k=kc, codes_v=vc, scales_k=ks, scales_v=vs)
        st["pos"] = None
        st["q_pos"] = None
        if case["causal"]:
            # slots hold their tokens in no order, as they do after evictions; some stand empty, and the newest tokens
            # are the queries' own
            p = torch.rand((b, kv, cap), generator=g, device="cuda")
            p = p.masked_fill(torch.arange(cap, device="cuda") >= st["len"][:, None, None], 2.0).argsort(-1).argsort(-1)
            empty = torch.rand((b, kv, cap), generator=g, device="cuda") < 0.03
            st["pos"] = p.masked_fill(empty, -1).to(torch.int32)
            st["q_pos"] = (st["len"] - n_q).to(torch.int32)
        st["mask"] = None
        if case["heads_on"]:
            on = torch.rand((b, heads), generator=g, device="cuda").argsort(-1).argsort(-1) < case["heads_on"]
            words = -(-heads // 32)
            bits = torch.nn.functional.pad(on, (0, 32 * words - heads)).view(b, words, 32).long()
            m = (bits << torch.arange(32, device="cuda")).sum(-1)
            st["mask"] = torch.where(m >= 2 ** 31, m - 2 ** 32, m).to(torch.int32)
        st["weight"] = st["weight_out"] = None
        if case["weights"]:
            st["weight"] = torch.rand((b, kv, cap), generator=g, device="cuda").pow_(4.0).mul_(8.0)
            st["weight_out"] = torch.zeros((b, kv, cap), device="cuda")
    else:
        lens = _lengths(case)
        r.shuffle(lens)
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # a few slots hold most of the weight, some newest ones hold none yet, and equal weights happen
        w = torch.randn((b, kv, cap), generator=g, device="cuda").mul_(2.0).exp_()
        w = torch.where(torch.rand((b, kv, cap), generator=g, device="cuda") < 0.2, (w * 4).round() / 4, w)
        used = torch.arange(cap, device="cuda") < st["len"][:, None, None]
        p = torch.rand((b, kv, cap), generator=g, device="cuda").masked_fill(~used, 2.0).argsort(-1).argsort(-1)
        st["next"] = st["len"] + torch.randint(0, 4096, (b,), generator=g, device="cuda", dtype=torch.int32)
        gone = (st["next"] - st["len"])[:, None, None]
        # the first tokens and the latest ones are still there, what lay between is thinned out
        st["pos"] = torch.where(p < 8, p, p + gone).to(torch.int32).masked_fill(~used, -1)
        st["weight"] = w
        if op == "evict":
            st["slots"] = torch.empty((b, kv, case["n"]), dtype=torch.int32, device="cuda")
        else:
            d, keep = case["d"], case["keep"]
            kc, ks = _quantise(_rows((b, kv, cap, d), g, 0.3))
            vc, vs = _quantise(_rows((b, kv, cap, d), g, 0.1))
            st.update(codes_k=kc, codes_v=vc, scales_k=ks, scales_v=vs, dst=_buffers(b, kv, keep, d))
            st["back"] = torch.empty((2, b, keep, kv, d), device="cuda", dtype=torch.float16)
            st["start"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    if own:
        _handles(st)
    return st


def _buffers(b, kv, cap, d):
    z = lambda *s, dt: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    return dict(codes_k=z(b, kv, cap, d // 2, dt=torch.uint8), codes_v=z(b, kv, cap, d // 2, dt=torch.uint8),
                scales_k=z(b, kv, cap, d // GROUP, 2, dt=torch.float16), scales_v=z(b, kv, cap, d // GROUP, 2, dt=torch.float16),
                weight=z(b, kv, cap, dt=torch.float32), pos=torch.full((b, kv, cap), -1, dtype=torch.int32, device="cuda"))


def _handles(st):
    """The framework's handles on the state's buffers: the cache's descriptor and the workspace."""
    import contextual_sparsity_sparse_gb300 as cs
    c = st["case"]
    if c["op"] == "evict":
        # eviction looks at weights and positions alone
        st["cache"] = cs.QCache(None, None, None, None, weight=st["weight"], pos=st["pos"])
    else:
        st["cache"] = cs.QCache(st["codes_k"], st["codes_v"], st["scales_k"], st["scales_v"], weight=st["weight"], pos=st["pos"])
    if c["op"] == "trim":
        t = st["dst"]
        st["to"] = cs.QCache(t["codes_k"], t["codes_v"], t["scales_k"], t["scales_v"], weight=t["weight"], pos=t["pos"])
    st["ws"] = cs.QCacheWorkspace(st["cache"], n_heads=c.get("heads", c["kv_heads"]), n_q=c.get("n_q", 1))


# -------------------------------------------------------------------------------------------------------------- operators

def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "evict": _own_evict, "trim": _own_trim}[op](st)
    return {"append": _plain_append, "attention": _plain_attention, "evict": _plain_evict, "trim": _plain_trim}[op](st)


def _own_append(st):
    import contextual_sparsity_sparse_gb300 as cs
    cs.cs_qcache_append(st["cache"], st["k"], st["v"], st["ws"], slots=st["slots"], start=st["start"], pos=st["at"])
    cs.cs_qcache_read(st["cache"], st["back"][0], st["back"][1], st["ws"], slots=st["slots"], start=st["start"])
    return {"k": st["back"][0], "v": st["back"][1], "pos": st["pos"], "weight": st["weight"]}


def _plain_append(st):
    b, n, kv = st["k"].shape[:3]
    if st["slots"] is not None:
        slots = st["slots"].long()
    else:
        slots = (st["start"].long()[:, None, None] + torch.arange(n, device="cuda")).expand(b, kv, n)
    at = (torch.arange(b, device="cuda")[:, None, None], torch.arange(kv, device="cuda")[None, :, None], slots)
    back = []
    for codes, scales, x in ((st["codes_k"], st["scales_k"], st["k"]), (st["codes_v"], st["scales_v"], st["v"])):
        c, s = _quantise(x.transpose(1, 2))
        codes[at], scales[at] = c, s
        back.append(_values(codes[at], scales[at]).transpose(1, 2).to(x.dtype))
    st["weight"][at] = 0.0
    st["pos"][at] = (st["at"][:, None, None] + torch.arange(n, device="cuda", dtype=torch.int32)).expand(b, kv, n)
    return {"k": back[0], "v": back[1], "pos": st["pos"], "weight": st["weight"]}


def _own_attention(st):
    import contextual_sparsity_sparse_gb300 as cs
    cs.cs_qcache_attention(st["cache"], st["q"], st["len"], st["out"], st["ws"], q_pos=st["q_pos"], mask=st["mask"],
                           weight=st["weight_out"], decay=0.875)
    return {"out": st["out"], "weight": st["weight_out"]} if st["weight_out"] is not None else {"out": st["out"]}


def _plain_attention(st):
    q = st["q"]
    b, n_q, heads, d = q.shape
    kv, cap = st["codes_k"].shape[1:3]
    k = _values(st["codes_k"], st["scales_k"])
    # rows of one cache head: its group of query heads, each with its tokens
    rows = q.float().view(b, n_q, kv, heads // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, d)
    s = (rows @ k.transpose(-1, -2)) * d ** -0.5
    s = s.view(b, kv, heads // kv, n_q, cap)
    seen = (torch.arange(cap, device="cuda") < st["len"][:, None])[:, None, None, None]
    if st["pos"] is not None:
        last = st["q_pos"][:, None] + torch.arange(n_q, device="cuda")
        p = st["pos"][:, :, None, None]
        seen = seen & (p >= 0) & (p <= last[:, None, None, :, None])
    if st["mask"] is not None:
        on = (st["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        seen = seen & (on.flatten(-2)[:, :heads] != 0).view(b, kv, -1, 1, 1)
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = (s - top.masked_fill(top == float("-inf"), 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total.masked_fill(total == 0, 1.0)
    v = _values(st["codes_v"], st["scales_v"])
    out = (p.view(b, kv, -1, cap) @ v).view(b, kv, heads // kv, n_q, d).permute(0, 3, 1, 2, 4).reshape(b, n_q, heads, d).to(q.dtype)
    if st["weight_out"] is None:
        return {"out": out}
    used = (torch.arange(cap, device="cuda") < st["len"][:, None])[:, None]
    st["weight_out"].copy_(torch.where(used, 0.875 * st["weight"] + p.sum((2, 3)), st["weight_out"]))
    return {"out": out, "weight": st["weight_out"]}


def _ranks(st, used):
    """Each slot's place in the order of eviction: empty slots, then by weight (equal ones by slot), protected ones last."""
    case, w, p = st["case"], st["weight"], st["pos"]
    kept = (p >= 0) & ((p < case["sinks"]) | (p >= (st["next"] - case["recent"])[:, None, None]))
    cls = torch.where(p < 0, 0, torch.where(kept, 2, 1)).masked_fill(~used, 3)
    order = w.sort(dim=-1, stable=True).indices
    order = order.gather(-1, cls.gather(-1, order).sort(dim=-1, stable=True).indices)
    return torch.empty_like(order).scatter_(-1, order, torch.arange(w.shape[-1], device="cuda").expand_as(order))


def _own_evict(st):
    import contextual_sparsity_sparse_gb300 as cs
    c = st["case"]
    cs.cs_qcache_evict(st["cache"], st["len"], c["capacity"], st["slots"], st["ws"], next_pos=st["next"], sinks=c["sinks"],
                       recent=c["recent"])
    return {"slots": st["slots"]}


def _plain_evict(st):
    c = st["case"]
    slot = torch.arange(c["capacity"], device="cuda")
    n_used = st["len"].long()[:, None, None]
    give = (c["n"] - (c["capacity"] - n_used)).clamp(min=0)
    chosen = _ranks(st, slot < n_used) < give
    # the given up slots in ascending order, then the free ones, which follow the last used slot
    first = torch.where(chosen | (slot >= n_used), slot, c["capacity"]).sort(-1).values[..., :c["n"]]
    return {"slots": first.to(torch.int32)}


def _own_trim(st):
    import contextual_sparsity_sparse_gb300 as cs
    c = st["case"]
    cs.cs_qcache_trim(st["cache"], st["len"], c["keep"], st["to"], st["ws"], next_pos=st["next"], sinks=c["sinks"], recent=c["recent"])
    cs.cs_qcache_read(st["to"], st["back"][0], st["back"][1], st["ws"], start=st["start"])
    return {"k": st["back"][0], "v": st["back"][1], "pos": st["dst"]["pos"], "weight": st["dst"]["weight"]}


def _plain_trim(st):
    c, dst = st["case"], st["dst"]
    slot = torch.arange(c["capacity"], device="cuda")
    n_used = st["len"].long()[:, None, None]
    stays = (slot < n_used) & (_ranks(st, slot < n_used) >= n_used - c["keep"])
    src = torch.where(stays, slot, c["capacity"]).sort(-1).values[..., :c["keep"]]
    there = src < c["capacity"]
    src = src.clamp(max=c["capacity"] - 1)
    for key in ("codes_k", "codes_v", "scales_k", "scales_v", "weight", "pos"):
        x = st[key]
        at = src.view(src.shape + (1,) * (x.dim() - 3))
        got = x.gather(2, at.expand(src.shape + x.shape[3:]))
        dst[key].copy_(torch.where(there.view(at.shape), got, dst[key]))
    k, v = (_values(dst["codes_" + x], dst["scales_" + x]).transpose(1, 2).half() for x in "kv")
    return {"k": k, "v": v, "pos": dst["pos"], "weight": dst["weight"]}


# ------------------------------------------------------------------------------------------------------ from the definition

def _decode64(codes, scales):
    """Values in 64 bits of one head's rows: offset + scale * code, channel by channel."""
    d = 2 * codes.shape[-1]
    ch = torch.arange(d, device=codes.device)
    nib = (codes[..., ch // 2].to(torch.int32) >> (4 * (ch % 2))) & 15
    return scales[..., ch // GROUP, 1].double() + scales[..., ch // GROUP, 0].double() * nib


def _exact_rows(x):
    """The values that new rows [..., d] come to stand for: the format's fp16 scales and offsets, the code in 64 bits."""
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[-1], GROUP):
        w = torch.nan_to_num(x[..., c:c + GROUP].float(), nan=0.0).clamp(-65504.0, 65504.0)
        lo = w.min(-1, keepdim=True).values
        s = ((w.max(-1, keepdim=True).values - lo) * F32_15TH).half().double()
        z = lo.half().double()
        n = torch.floor((w.double() - z) / s.clamp(min=2.0 ** -24) + 0.5)
        even = ((w.double() - z) / s.clamp(min=2.0 ** -24)) % 1.0 == 0.5
        n = torch.where(even, 2.0 * torch.round((w.double() - z) / s.clamp(min=2.0 ** -24) / 2.0), n)
        y[..., c:c + GROUP] = torch.where(s > 0, z + s * n.clamp(0.0, 15.0), z)
    return y


def exact(case, seed):
    if case["op"] == "evict":
        return None   # whole numbers alone
    st = prepare(case, seed)
    if case["op"] == "append":
        return {"k": _exact_rows(st["k"]), "v": _exact_rows(st["v"]), "pos": None, "weight": None}
    b, kv, cap, d = case["batch"], case["kv_heads"], case["capacity"], case["d"]
    if case["op"] == "trim":
        k = torch.zeros((b, case["keep"], kv, d), dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        w = torch.zeros((b, kv, case["keep"]), dtype=torch.float64, device="cuda")
        lens, after = st["len"].tolist(), st["next"].tolist()
        for i in range(b):
            for h in range(kv):
                n = lens[i]
                p, acc = st["pos"][i, h, :n], st["weight"][i, h, :n].double()
                safe = (p >= 0) & ((p < case["sinks"]) | (p >= after[i] - case["recent"]))
                low = torch.where(p < 0, float("-inf"), torch.where(safe, float("inf"), acc))
                best = torch.sort(low, stable=True).indices
                # among protected slots, too, the lightest go first
                best = torch.cat([best[low[best] != float("inf")], best[low[best] == float("inf")][torch.sort(acc[best[low[best] == float("inf")]], stable=True).indices]])
                left = torch.sort(best[max(0, n - case["keep"]):]).values
                k[i, :len(left), h] = _decode64(st["codes_k"][i, h, left], st["scales_k"][i, h, left])
                v[i, :len(left), h] = _decode64(st["codes_v"][i, h, left], st["scales_v"][i, h, left])
                w[i, h, :len(left)] = acc[left]
        return {"k": k, "v": v, "pos": None, "weight": w}
    heads, n_q = case["heads"], case["n_q"]
    out = torch.zeros((b, n_q, heads, d), dtype=torch.float64, device="cuda")
    wout = torch.zeros((b, kv, cap), dtype=torch.float64, device="cuda") if case["weights"] else None
    share = heads // kv
    for i, n in enumerate(st["len"].tolist()):
        for h in range(kv):
            k, v = (_decode64(st["codes_" + x][i, h, :n], st["scales_" + x][i, h, :n]) for x in "kv")
            # one row per query token and head of the group
            q = st["q"][i, :, h * share:(h + 1) * share].double().reshape(-1, d)
            s = q @ k.T / d ** 0.5
            ok = torch.ones((n_q, share, n), dtype=torch.bool, device="cuda")
            if case["causal"]:
                p = st["pos"][i, h, :n]
                ok &= ((p >= 0) & (p <= st["q_pos"][i] + torch.arange(n_q, device="cuda")[:, None]))[:, None]
            if st["mask"] is not None:
                head = h * share + torch.arange(share, device="cuda")
                ok &= ((st["mask"][i, head // 32] >> (head % 32).int()) & 1).bool()[:, None]
            ok = ok.reshape(-1, n)
            s = torch.where(ok, s, float("-inf"))
            e = torch.where(ok, torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300)), 0.0)
            t = e.sum(-1, keepdim=True)
            e = torch.where(t > 0, e / t, 0.0)
            out[i, :, h * share:(h + 1) * share] = (e @ v).reshape(n_q, share, d)
            if wout is not None:
                wout[i, h, :n] = 0.875 * st["weight"][i, h, :n].double() + e.sum(0)
    return {"out": out, "weight": wout} if case["weights"] else {"out": out}
