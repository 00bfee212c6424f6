"""Operators around the 4-bit KV cache, as cases to measure: prompts, trees of drafted tokens, forks of sequences.

A cache holds, for `batch` sequences, `kv_heads` heads and `capacity` slots, one key and one value row of `d` channels per
slot.  A row is cut into groups of 64 channels; a group keeps a scale and an offset in fp16 and 64 codes of 4 bits (byte i of
a row holds channel 2i in its low and channel 2i + 1 in its high half), which stand for offset + scale * code.  Beside each
slot stand its accumulated attention weight and the position of its token (negative: an empty slot).

 prompt     attention of whole prompts, packed one behind the other: causal or not, grouped heads, after a prefix or not
 tree       attention of a tree of drafted tokens over a cache's slots, the token itself and its ancestors in the tree
 rows       new tokens quantised into given slots, from rows that lie anywhere (packed prompts, a tree's accepted path),
            and those slots read back as the values they stand for
 fork       sequences of a cache taken over by other sequences, in the same cache or in another

`own` false: plain torch operations.  `own` true: the framework's calls.
"""
import random

import torch

own = False

GROUP = 64
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
F32_15TH = 1.0 / 15.0


# ------------------------------------------------------------------------------------------------------------------ cases

def _prompt(name, batch, heads, kv_heads, d, dtype, tokens, prefix=0, causal=True, ragged=True):
    c = dict(op="prompt", batch=batch, heads=heads, kv_heads=kv_heads, d=d, dtype=dtype, tokens=tokens, prefix=prefix,
             causal=causal, ragged=ragged)
    return dict(c, name=name) if name else c


def _tree(name, batch, heads, kv_heads, d, capacity, dtype, n, ragged=True, positions=True):
    c = dict(op="tree", batch=batch, heads=heads, kv_heads=kv_heads, d=d, capacity=capacity, dtype=dtype, n=n, ragged=ragged,
             positions=positions)
    return dict(c, name=name) if name else c


def _rows(name, batch, kv_heads, d, capacity, dtype, n, packed):
    c = dict(op="rows", batch=batch, kv_heads=kv_heads, d=d, capacity=capacity, dtype=dtype, n=n, packed=packed)
    return dict(c, name=name) if name else c


def _fork(name, batch, kv_heads, d, capacity, groups, in_place, ragged):
    c = dict(op="fork", batch=batch, kv_heads=kv_heads, d=d, capacity=capacity, groups=groups, in_place=in_place, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the first words of a conversation with a small model: latency is all there is
        _prompt("prompt-short", 1, 8, 8, 64, "fp16", 9),
        # one prompt that fills the context of the OPT-13B-shaped layer (40 heads of 128, 2,048 positions)
        _prompt("prompt-opt13b", 1, 40, 40, 128, "bf16", 2048, ragged=False),
        # a serving batch's prompts of one token to 5,000, packed, LLaMA-70B-shaped heads (64 over 8 of 128)
        _prompt("prompt-packed", 16, 64, 8, 128, "bf16", 5000),
        # the next 200 tokens or so of long conversations, whose earlier tokens are there already (Falcon-40B-shaped heads)
        _prompt("prompt-turns", 4, 128, 8, 64, "fp16", 201, prefix=32768),
        # a short conversation with a small model verifies five drafted tokens
        _tree("tree-short", 1, 8, 8, 64, 100, "fp16", 5, ragged=False),
        # sixteen drafted tokens over the OPT-13B-shaped layer's full cache
        _tree("tree-opt13b", 1, 40, 40, 128, 2048, "bf16", 16, ragged=False),
        # a tree over one very long document, LLaMA-70B-shaped heads
        _tree("tree-long", 1, 64, 8, 128, 131001, "fp16", 26, ragged=False, positions=False),
        # wide trees over a serving batch of many lengths
        _tree("tree-batch", 32, 64, 8, 128, 8192, "bf16", 64),
        # the paths that a serving batch's trees were accepted on, into the slots that eviction gave
        _rows("rows-accept", 64, 8, 128, 4096, "bf16", 6, False),
        # packed prompts of many lengths into empty caches
        _rows("rows-prompts", 16, 8, 128, 1500, "fp16", 999, True),
        # sixteen answers are sampled from one prompt: its slots go to all of them
        _fork("fork-samples", 16, 8, 128, 4096, 1, True, False),
        # beams of eight sentences change places, into the other one of two caches (Falcon-40B-shaped cache heads)
        _fork("fork-beams", 32, 8, 64, 2049, 8, False, True),
    ]


MOST_PAIRS = 64 * 16 * 5000 * 5000 // 6      # query-key pairs over all heads of the largest listed prompt
MOST_SLOTS = 32 * 8 * 8192 * 128             # channels in the largest listed tree's cache
MOST_LOGITS = 32 * 64 * 8192 * 64            # its query-key pairs
MOST_COPY = 16 * 8 * 4096 * 128              # channels of the largest listed fork


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "tree", "rows", "fork"])
    kv = rng.choice([1, 2, 4, 5, 8, 8, 12, 40])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(sorted(DTYPES))
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 16])
    if op == "prompt":
        batch = _log(rng, 1, 32)
        prefix = _log(rng, 1, 32768) if rng.random() < 0.35 else 0
        causal = rng.random() < 0.8
        per = MOST_PAIRS // (batch * kv * group)
        # without an earlier part a full-length square of pairs has to fit, half of it where it is causal
        most = int(per / prefix) if prefix else int((2 * per) ** 0.5 if causal else per ** 0.5)
        tokens = _log(rng, 1, max(1, min(most, 512 if prefix else 16384)))
        return _prompt(None, batch, kv * group, kv, d, dtype, tokens, prefix, causal, rng.random() < 0.7)
    if op == "tree":
        batch = _log(rng, 1, 32)
        n = _log(rng, 1, 64)
        most = min(131072, MOST_SLOTS // (batch * kv * d), MOST_LOGITS // (batch * kv * group * n))
        return _tree(None, batch, kv * group, kv, d, _log(rng, 1, max(1, most)), dtype, n, rng.random() < 0.7,
                     rng.random() < 0.6)
    batch = _log(rng, 1, 64)
    if op == "rows":
        packed = rng.random() < 0.5
        n = _log(rng, 1, max(1, min(4096 if packed else 16, (16 * 999 * 8 * 128) // (batch * kv * d))))
        return _rows(None, batch, kv, d, n + _log(rng, 1, 2048), dtype, n, packed)
    batch = max(2, batch)
    capacity = _log(rng, 1, max(1, min(32768, MOST_COPY // (batch * kv * d))))
    return _fork(None, batch, kv, d, capacity, rng.randint(1, batch), rng.random() < 0.5, rng.random() < 0.6)


def _spread(most, n, ragged):
    """n lengths, before they are shuffled: all the longest, or evenly spread from one to the longest."""
    if not ragged:
        return [most] * n
    return [1 + int((i + 0.5) * (most - 1) / n) if n > 1 else most - most // 3 for i in range(n)]


def _prompt_lengths(case):
    """(query tokens, keys) of every sequence, before they are shuffled: the keys are an earlier part's and the queries' own."""
    q = _spread(case["tokens"], case["batch"], case["ragged"])
    if not case["prefix"]:
        return [(n, n) for n in q]
    earlier = _spread(case["prefix"], case["batch"], case["ragged"])
    return [(n, n + earlier[-1 - i]) for i, n in enumerate(q)]


def _visible(n_q, n_k, causal):
    return n_q * n_k - n_q * (n_q - 1) // 2 if causal else n_q * n_k


def work(case):
    b, kv, d = case["batch"], case["kv_heads"], case["d"]
    row = 2 * (d // 2 + 4 * (d // GROUP))   # a slot's key and value rows in the cache
    if case["op"] == "prompt":
        lens = _prompt_lengths(case)
        n_q, n_k = sum(q for q, _ in lens), sum(k for _, k in lens)
        pairs = sum(_visible(q, k, case["causal"]) for q, k in lens)
        return {"bytes": 2 * 2 * d * (n_q * case["heads"] + n_k * kv), "flops": 4 * d * case["heads"] * pairs}
    if case["op"] == "tree":
        n = case["n"]
        lens = _spread(case["capacity"], b, case["ragged"])
        slot = kv * (row + (4 if case["positions"] else 0))
        # of the drafted tokens that one sees, itself alone is counted
        return {"bytes": sum(lens) * slot + 2 * 2 * b * n * d * (case["heads"] + kv) + 4 * b * n,
                "flops": 4 * d * case["heads"] * n * (sum(lens) + b)}
    if case["op"] == "rows":
        rows = sum(_spread(case["n"], b, True)) * kv
        # new rows in, codes, weight and position out; the codes back in, their values out
        return {"bytes": rows * (2 * 2 * d * 2 + 2 * row + 8), "flops": rows * 2 * d * 8}
    lens = _spread(case["capacity"], b, case["ragged"])
    # every source read once, every copy written once
    if case["in_place"]:
        copies, sources = b - case["groups"], case["groups"]
    else:
        copies, sources = b, case["groups"]
    mean = sum(lens) / len(lens)
    return {"bytes": int((copies + sources) * mean) * kv * (row + 8), "flops": 0}


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


def _channels(shape, g, spread):
    """Rows [..., heads, d] as attention meets them: channels of different means and widths, a few of them outliers."""
    x = torch.randn(shape, generator=g, device="cuda")
    x.mul_(0.5 + torch.rand(shape[-2:], generator=g, device="cuda"))
    return x.add_(spread * torch.randn(shape[-2:], generator=g, device="cuda") ** 3)


def _projected(lead, heads, kv, d, dtype, g):
    """q, k and v [*lead, heads, d] as slices of one projection's output."""
    x = torch.cat([torch.randn((*lead, heads, d), generator=g, device="cuda") *
                   (0.5 + torch.rand((heads, 1), generator=g, device="cuda")),
                   _channels((*lead, kv, d), g, 0.3), _channels((*lead, kv, d), g, 0.1)], -2).to(dtype)
    return x[..., :heads, :], x[..., heads:heads + kv, :], x[..., heads + kv:, :]


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _parents(n, r):
    """A drafted tree: a few first tokens, every other one a continuation of an earlier one, most often of a late one."""
    return [-1 if t == 0 or r.random() < 0.08 else max(r.randrange(t), r.randrange(t)) for t in range(n)]


def _buffers(b, kv, cap, d):
    z = lambda *s, dt: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    return dict(codes_k=z(b, kv, cap, d // 2, dt=torch.uint8), codes_v=z(b, kv, cap, d // 2, dt=torch.uint8),
                scales_k=z(b, kv, cap, d // GROUP, 2, dt=torch.float16), scales_v=z(b, kv, cap, d // GROUP, 2, dt=torch.float16),
                weight=z(b, kv, cap, dt=torch.float32), pos=torch.full((b, kv, cap), -1, dtype=torch.int32, device="cuda"))


CACHE = ("codes_k", "codes_v", "scales_k", "scales_v", "weight", "pos")


def _filled(b, kv, cap, d, g):
    kc, ks = _quantise(_channels((b, cap, kv, d), g, 0.3).transpose(1, 2))
    vc, vs = _quantise(_channels((b, cap, kv, d), g, 0.1).transpose(1, 2))
    return dict(codes_k=kc.contiguous(), codes_v=vc.contiguous(), scales_k=ks.contiguous(), scales_v=vs.contiguous())


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = random.Random(seed)
    op, b, kv, d = case["op"], case["batch"], case["kv_heads"], case["d"]
    st = {"case": case}
    if op == "prompt":
        lens = _prompt_lengths(case)
        r.shuffle(lens)
        st["lens"] = lens
        n_q, n_k = sum(q for q, _ in lens), sum(k for _, k in lens)
        dt = DTYPES[case["dtype"]]
        if case["prefix"]:
            st["q"] = _projected((n_q,), case["heads"], 0, d, dt, g)[0]
            _, st["k"], st["v"] = _projected((n_k,), 0, kv, d, dt, g)
        else:
            st["q"], st["k"], st["v"] = _projected((n_q,), case["heads"], kv, d, dt, g)
        st["q_start"] = _starts([q for q, _ in lens])
        st["k_start"] = _starts([k for _, k in lens]) if case["prefix"] else None
        st["out"] = torch.empty((n_q, case["heads"], d), dtype=dt, device="cuda")
    elif op == "tree":
        n, cap, dt = case["n"], case["capacity"], DTYPES[case["dtype"]]
        lens = _spread(cap, b, case["ragged"])
        r.shuffle(lens)
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st.update(_filled(b, kv, cap, d, g))
        st["pos"] = st["n_new"] = None
        if case["positions"]:
            # slots hold their tokens in no order, as they do after evictions, and some stand empty
            p = torch.rand((b, kv, cap), generator=g, device="cuda").argsort(-1)
            st["pos"] = p.masked_fill(torch.rand((b, kv, cap), generator=g, device="cuda") < 0.03, -1).to(torch.int32)
        st["weight"] = None
        st["q"], st["k"], st["v"] = _projected((b, n), case["heads"], kv, d, dt, g)
        st["parent"] = torch.tensor([_parents(n, r) for _ in range(b)], dtype=torch.int32, device="cuda")
        if case["ragged"]:
            # some trees were cut short
            st["n_new"] = torch.tensor([r.randint((n + 1) // 2, n) for _ in range(b)], dtype=torch.int32, device="cuda")
        st["out"] = torch.empty((b, n, case["heads"], d), dtype=dt, device="cuda")
    elif op == "rows":
        n, cap, dt = case["n"], case["capacity"], DTYPES[case["dtype"]]
        lens = _spread(n, b, True)
        r.shuffle(lens)
        per = None if case["packed"] else max(64, 2 * n)   # a tree's tokens
        total = sum(lens) if case["packed"] else b * per
        _, st["k"], st["v"] = _projected((total,), 1, kv, d, dt, g)
        at, first = [], 0
        for i, m in enumerate(lens):
            if case["packed"]:
                path = list(range(first, first + m))
                first += m
            else:
                path = [i * per + t for t in sorted(r.sample(range(per), m))]
            at.append(path + [-1] * (n - m))
        st["rows"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        st["at"] = torch.randint(0, cap, (b,), generator=g, device="cuda", dtype=torch.int32)   # the next position
        st["slots"] = st["start"] = None
        if case["packed"]:
            st["start"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        else:
            # slots that eviction gave, another set in each head
            keys = torch.rand((b, kv, cap), generator=g, device="cuda")
            st["slots"] = keys.argsort(-1)[..., :n].sort(-1).values.to(torch.int32).contiguous()
        st["back"] = torch.empty((2, b, n, kv, d), device="cuda", dtype=dt)
        st.update(_buffers(b, kv, cap, d))
    else:
        cap = case["capacity"]
        lens = _spread(cap, b, case["ragged"])
        r.shuffle(lens)
        first = r.sample(range(b), case["groups"])   # the sequences that others continue
        source = [first[i % len(first)] for i in range(b)]
        if case["in_place"]:
            for i in first:
                source[i] = i
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["source"] = torch.tensor(source, dtype=torch.int32, device="cuda")
        st.update({key: torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8) if t.dtype == torch.uint8
                   else torch.rand(t.shape, generator=g, device="cuda").mul_(9).to(t.dtype)
                   for key, t in _buffers(b, kv, cap, d).items()})
        st["pos"] = torch.randint(-1, 4 * cap, (b, kv, cap), generator=g, device="cuda", dtype=torch.int32)
        if not case["in_place"]:
            st["dst"] = _buffers(b, kv, cap, d)
    if own:
        _handles(st)
    return st


def _handles(st):
    """The framework's handles on the state's buffers: the cache's descriptor and the workspace."""
    import contextual_sparsity_sparse_gb300 as cs
    c = st["case"]
    if c["op"] == "prompt":
        st["ws"] = cs.PromptWorkspace(c["batch"], c["heads"], c["kv_heads"], c["d"], st["q"].shape[0], st["k"].shape[0])
        return
    st["cache"] = cs.QCache(st["codes_k"], st["codes_v"], st["scales_k"], st["scales_v"], weight=st["weight"], pos=st["pos"])
    if c["op"] == "tree":
        st["ws"] = cs.QCacheTreeWorkspace(st["cache"], c["heads"], c["n"])
        return
    st["ws"] = cs.QCacheWorkspace(st["cache"], n_heads=0)
    if c["op"] == "fork":
        t = st.get("dst")
        st["to"] = None if t is None else cs.QCache(t["codes_k"], t["codes_v"], t["scales_k"], t["scales_v"],
                                                    weight=t["weight"], pos=t["pos"])


# -------------------------------------------------------------------------------------------------------------- operators

def run(st):
    op = st["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "tree": _own_tree, "rows": _own_rows, "fork": _own_fork}[op](st)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "rows": _plain_rows, "fork": _plain_fork}[op](st)


def _own_prompt(st):
    import contextual_sparsity_sparse_gb300 as cs
    cs.cs_prompt_attention(st["q"], st["k"], st["v"], st["out"], st["q_start"], st["ws"], k_start=st["k_start"],
                           causal=st["case"]["causal"])
    return {"out": st["out"]}


def _plain_prompt(st):
    c = st["case"]
    kv, d = c["kv_heads"], c["d"]
    g = c["heads"] // kv
    out = torch.empty_like(st["out"])
    q0 = k0 = 0
    for n_q, n_k in st["lens"]:
        # [kv, ., d], a cache head's query heads one behind the other
        q = st["q"][q0:q0 + n_q].float().view(n_q, kv, g, d).permute(1, 2, 0, 3)
        k = st["k"][k0:k0 + n_k].float().permute(1, 2, 0)
        v = st["v"][k0:k0 + n_k].float().transpose(0, 1)
        for t in range(0, n_q, 512):
            m = min(512, n_q - t)
            end = n_k - n_q + t + m if c["causal"] else n_k
            s = (q[:, :, t:t + m].reshape(kv, g * m, d) @ k[..., :end]) * d ** -0.5
            if c["causal"]:
                late = torch.arange(end, device="cuda") > torch.arange(n_k - n_q + t, end, device="cuda")[:, None]
                s = s.view(kv, g, m, end).masked_fill_(late, float("-inf")).view(kv, g * m, end)
            p = s.sub_(s.amax(-1, keepdim=True)).exp_()
            o = (p @ v[:, :end]) / p.sum(-1, keepdim=True)
            out[q0 + t:q0 + t + m] = o.view(kv, g, m, d).permute(2, 0, 1, 3).reshape(m, kv * g, d).to(out.dtype)
        q0, k0 = q0 + n_q, k0 + n_k
    return {"out": out}


def _own_tree(st):
    import contextual_sparsity_sparse_gb300 as cs
    cs.cs_qcache_tree_attention(st["cache"], st["q"], st["k"], st["v"], st["len"], st["out"], st["ws"], parent=st["parent"],
                                n_new=st["n_new"])
    return {"out": st["out"]}


def _ancestors(parent):
    """[batch, n, n]: whether token j is token t or an ancestor of it."""
    n = parent.shape[1]
    tokens = torch.arange(n, device=parent.device)
    up = ((parent.unsqueeze(-1) == tokens) | (tokens == tokens[:, None])).float()   # one step up, or none
    for _ in range((n - 1).bit_length()):
        up = ((up @ up) > 0).float()                                                  # twice as many
    return up > 0


def _plain_tree(st):
    q = st["q"]
    b, n, heads, d = q.shape
    kv, cap = st["codes_k"].shape[1:3]
    g = heads // kv
    rows = q.float().view(b, n, kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, kv, g * n, d)
    keys = torch.cat([_values(st["codes_k"], st["scales_k"]), st["k"].float().transpose(1, 2)], 2)
    s = (rows @ keys.transpose(-1, -2)) * d ** -0.5
    used = (torch.arange(cap, device="cuda") < st["len"][:, None])[:, None]
    if st["pos"] is not None:
        used = used & (st["pos"] >= 0)
    seen = torch.cat([used[:, :, None, None].expand(b, kv, g, n, cap),
                      _ancestors(st["parent"])[:, None, None].expand(b, kv, g, n, n)], -1).reshape(b, kv, g * n, cap + n)
    s = s.masked_fill_(~seen, float("-inf"))
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    values = torch.cat([_values(st["codes_v"], st["scales_v"]), st["v"].float().transpose(1, 2)], 2)
    out = (p @ values) / p.sum(-1, keepdim=True)
    out = out.view(b, kv, g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, heads, d)
    if st["n_new"] is not None:
        out = out.masked_fill((torch.arange(n, device="cuda") >= st["n_new"][:, None])[..., None, None], 0.0)
    return {"out": out.to(q.dtype)}


def _own_rows(st):
    import contextual_sparsity_sparse_gb300 as cs
    cs.cs_qcache_append_rows(st["cache"], st["k"], st["v"], st["rows"], st["ws"], start=st["start"], slots=st["slots"],
                             pos=st["at"])
    cs.cs_qcache_read(st["cache"], st["back"][0], st["back"][1], st["ws"], slots=st["slots"], start=st["start"])
    return {"k": st["back"][0], "v": st["back"][1], "pos": st["pos"], "weight": st["weight"]}


def _plain_rows(st):
    b, n = st["rows"].shape
    kv = st["k"].shape[1]
    slots = torch.arange(n, device="cuda").expand(b, kv, n) if st["slots"] is None else st["slots"].long()
    if st["start"] is not None:
        slots = slots + st["start"].long()[:, None, None]
    there = (st["rows"] >= 0)[:, None].expand(b, kv, n)
    at = (torch.arange(b, device="cuda")[:, None, None].expand(b, kv, n), torch.arange(kv, device="cuda")[None, :, None].expand(b, kv, n),
          slots)
    back = []
    for codes, scales, x in ((st["codes_k"], st["scales_k"], st["k"]), (st["codes_v"], st["scales_v"], st["v"])):
        c, s = _quantise(x[st["rows"].long().clamp(min=0)].transpose(1, 2))
        codes[at] = torch.where(there[..., None], c, codes[at])
        scales[at] = torch.where(there[..., None, None], s, scales[at])
        back.append(_values(codes[at], scales[at]).transpose(1, 2).to(x.dtype))
    st["weight"][at] = torch.where(there, 0.0, st["weight"][at])
    new = (st["at"][:, None, None] + torch.arange(n, device="cuda", dtype=torch.int32)).expand(b, kv, n)
    st["pos"][at] = torch.where(there, new, st["pos"][at])
    return {"k": back[0], "v": back[1], "pos": st["pos"], "weight": st["weight"]}


def _own_fork(st):
    import contextual_sparsity_sparse_gb300 as cs
    cs.cs_qcache_fork(st["cache"], st["source"], st["len"], st["ws"], dst=st["to"])
    return {key: st.get("dst", st)[key] for key in CACHE}


def _plain_fork(st):
    dst = st.get("dst", st)
    source = st["source"].long()
    used = (torch.arange(st["case"]["capacity"], device="cuda") < st["len"].long()[source][:, None])[:, None]
    for key in CACHE:
        got = st[key][source]
        dst[key].copy_(torch.where(used.view(used.shape + (1,) * (got.dim() - 3)), got, dst[key]))
    return {key: dst[key] for key in CACHE}


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
        r = (w.double() - z) / s.clamp(min=2.0 ** -24)
        n = torch.where(r % 1.0 == 0.5, 2.0 * torch.round(r / 2.0), torch.floor(r + 0.5))   # halves to even
        y[..., c:c + GROUP] = torch.where(s > 0, z + s * n.clamp(0.0, 15.0), z)
    return y


def _softmax64(s, ok):
    """exp(s) / sum over what a row sees, zeros for a row that sees nothing."""
    top = torch.where(ok, s, -1e300).max(-1, keepdim=True).values
    e = torch.where(ok, torch.exp(s - top), 0.0)
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300)


def exact(case, seed):
    if case["op"] == "fork":
        return None   # copies alone
    st = prepare(case, seed)
    if case["op"] == "rows":
        out = {}
        for key in "kv":
            y = torch.zeros((*st["rows"].shape, *st[key].shape[1:]), dtype=torch.float64, device="cuda")
            for i, path in enumerate(st["rows"].tolist()):
                path = [p for p in path if p >= 0]
                y[i, :len(path)] = _exact_rows(st[key][path])
            out[key] = y
        return {**out, "pos": None, "weight": None}
    kv, d, heads = case["kv_heads"], case["d"], case["heads"]
    share = heads // kv
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prompt":
        if 2 * d * heads * sum(q * k for q, k in st["lens"]) * 2 > 1e13:
            return None
        ends_q = torch.tensor([q for q, _ in st["lens"]]).cumsum(0).tolist()
        ends_k = torch.tensor([k for _, k in st["lens"]]).cumsum(0).tolist()
        for (n_q, n_k), eq, ek in zip(st["lens"], ends_q, ends_k):
            for h in range(heads):
                k, v = st["k"][ek - n_k:ek, h // share].double(), st["v"][ek - n_k:ek, h // share].double()
                for t in range(0, n_q, 4096):
                    rows = torch.arange(t, min(n_q, t + 4096), device="cuda")
                    s = (st["q"][eq - n_q + rows, h].double() @ k.T) / d ** 0.5
                    # a query's own key is as far from the last one as the query is from the last query
                    ok = (n_k - 1 - torch.arange(n_k, device="cuda") >= n_q - 1 - rows[:, None]) if case["causal"] \
                        else torch.ones_like(s, dtype=torch.bool)
                    out[eq - n_q + rows, h] = _softmax64(s, ok) @ v
        return {"out": out}
    lens = st["len"].tolist()
    for i, n in enumerate(lens):
        m = case["n"] if st["n_new"] is None else int(st["n_new"][i])
        parent = st["parent"][i].tolist()
        path = torch.zeros((m, m), dtype=torch.bool)
        for t in range(m):
            a = t
            while a >= 0:
                path[t, a] = True
                a = parent[a]
        path = path.cuda()
        for h in range(kv):
            k = torch.cat([_decode64(st["codes_k"][i, h, :n], st["scales_k"][i, h, :n]), st["k"][i, :m, h].double()])
            v = torch.cat([_decode64(st["codes_v"][i, h, :n], st["scales_v"][i, h, :n]), st["v"][i, :m, h].double()])
            live = torch.ones(n, dtype=torch.bool, device="cuda") if st["pos"] is None else st["pos"][i, h, :n] >= 0
            ok = torch.cat([live.expand(m, n), path], 1)
            for j in range(h * share, (h + 1) * share):
                s = st["q"][i, :m, j].double() @ k.T / d ** 0.5
                out[i, :m, j] = _softmax64(s, ok) @ v
    return {"out": out}
