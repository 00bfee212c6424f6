"""Attention of packed prompts against its plain 64-bit form."""
import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

import _prompt_ref as ref

pytestmark = pytest.mark.gpu
DTS = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def starts(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).to(torch.int32)


def make(q_lens, k_lens, heads, kv, d, dt, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k, v = r(sum(q_lens), heads, d), r(sum(k_lens), kv, d) + r(kv, d), r(sum(k_lens), kv, d) + 0.5 * r(kv, d)
    return q.to(dt), k.to(dt), v.to(dt)


def call(q, k, v, q_lens, k_lens=None, out=None, ws=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    if ws is None:
        ws = cs.PromptWorkspace(len(q_lens), q.shape[1], k.shape[1], q.shape[2], q.shape[0], k.shape[0])
    cs.cs_prompt_attention(q, k, v, out, starts(q_lens), ws, k_start=None if k_lens is None else starts(k_lens), **kw)
    return out, ws


def check(q, k, v, q_lens, k_lens=None, causal=True, scale=0.0, out=None):
    out, ws = call(q, k, v, q_lens, k_lens, causal=causal, scale=scale, out=out)
    assert cs.cs_get_device_error(ws) == 0
    want, bound = ref.prompt(q, k, v, q_lens, q_lens if k_lens is None else k_lens, causal, scale)
    n = sum(q_lens)
    off = (out[:n].double() - want[:n]).abs()
    assert (off <= bound[:n]).all(), (off / bound[:n].clamp(min=1e-30)).max().item()
    return out


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads,kv,d", [(1, 1, 64), (8, 8, 64), (6, 2, 128), (5, 1, 128), (16, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("q_lens", [[1], [17], [128], [129, 1, 0, 64], [300, 257], [0, 0, 3]])
def test_causal(q_lens, heads, kv, d, dt):
    check(*make(q_lens, q_lens, heads, kv, d, dt), q_lens)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,k_lens", [([1], [1000]), ([5, 70], [131, 70]), ([200], [1]), ([130, 3], [0, 4]), ([64], [640]),
                                           ([1, 1, 1], [128, 129, 127]), ([0, 9], [50, 300])])
def test_other_keys(q_lens, k_lens, causal, dt):
    """Keys of an earlier part, none at all, or fewer than query tokens: causal rows that see nothing are zero."""
    check(*make(q_lens, k_lens, 8, 2, 128, dt), q_lens, k_lens, causal)


@pytest.mark.parametrize("heads,kv,d", [(128, 1, 64), (127, 1, 64), (7, 1, 128), (12, 4, 64), (40, 40, 128), (65, 1, 128)])
def test_groups(heads, kv, d):
    q_lens = [33, 5]
    check(*make(q_lens, q_lens, heads, kv, d, torch.bfloat16), q_lens)


@pytest.mark.parametrize("q_lens,k_lens,heads,kv,d,causal", [
    ([1], [20001], 8, 1, 128, True), ([3, 1], [9000, 12345], 8, 8, 64, True), ([100], [16384], 4, 4, 128, True),
    ([33], [30000], 16, 1, 64, False), ([2000], [2000], 2, 2, 128, True), ([1, 700], [5000, 2900], 2, 1, 128, True)])
def test_long_keys_and_few_rows(q_lens, k_lens, heads, kv, d, causal):
    check(*make(q_lens, k_lens, heads, kv, d, torch.float16), q_lens, k_lens, causal)


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    q_lens = torch.randint(0, 40, (150,), generator=g).tolist()
    check(*make(q_lens, q_lens, 4, 2, 64, torch.bfloat16), q_lens)


@pytest.mark.parametrize("scale", [0.3, -0.2, 1e-30, 30.0])
def test_scales(scale):
    check(*make([200], [200], 2, 1, 128, torch.float16), [200], scale=scale)


@pytest.mark.parametrize("dt", DTS)
def test_growing_logits(dt):
    """Every key beats the ones before it by a lot, so that the running maximum moves all the time; and the reverse."""
    for step in (1.0, -1.0):
        q, k, v = make([700], [700], 2, 2, 64, dt)
        k[..., 0] = (step * torch.arange(700, device="cuda")[:, None]).to(dt)
        q[..., 0] = 4.0
        check(q, k, v, [700])


def test_layouts():
    """Slices of one projection's output, heads before tokens, and rows that are not dense."""
    lens, heads, kv, d = [70, 131], 6, 2, 64
    q, k, v = make(lens, lens, heads, kv, d, torch.float16)
    want, _ = call(q, k, v, lens)
    both = torch.cat([q, k, v], 1)
    got, _ = call(both[:, :heads], both[:, heads:heads + kv], both[:, heads + kv:], lens, out=torch.empty_like(q))
    assert torch.equal(got, want)
    turned = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    got, _ = call(turned(q), turned(k), turned(v), lens, out=turned(torch.empty_like(q)))
    assert torch.equal(got, want)
    wide = torch.full((sum(lens), heads, d + 8), 3.0, dtype=torch.float16, device="cuda")
    got, _ = call(q, k, v, lens, out=wide[..., :d])
    assert torch.equal(got, want) and (wide[..., d:] == 3.0).all()


def test_what_lies_behind_the_last_sequence():
    """Rows in no sequence are neither read for a result nor written."""
    lens = [50, 20]
    q, k, v = make([100], [100], 4, 2, 64, torch.bfloat16)
    for t in (q, k, v):
        t[70:] = float("nan")
    out = check(q, k, v, lens)
    assert (out[70:] == 7.0).all()
    shifted = torch.full_like(q, 7.0)
    ws = cs.PromptWorkspace(1, 4, 2, 64, 100)
    cs.cs_prompt_attention(q, k, v, shifted, torch.tensor([50, 70], dtype=torch.int32, device="cuda"), ws)
    assert torch.equal(shifted[50:70], out[50:70]) and (shifted[:50] == 7.0).all() and (shifted[70:] == 7.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("lens", [[40], [200, 300]])
def test_what_is_not_seen_has_no_influence(bad, lens):
    """NaN and infinities in keys and values reach the rows that see them, and no others."""
    q, k, v = make(lens, lens, 4, 2, 64, torch.float16)
    clean, _ = call(q, k, v, lens)
    at = lens[0] - 11
    for t in (k, v):
        poisoned = t.clone()
        poisoned[at] = bad
        out, _ = call(q, poisoned if t is k else k, poisoned if t is v else v, lens)
        assert torch.isfinite(out[:at]).all() and torch.isfinite(out[lens[0]:]).all()
        d = torch.finfo(torch.float16).eps
        assert ((out[:at].double() - clean[:at].double()).abs() <= 4 * d * clean[:at].double().abs() + 4 * d).all()
        assert torch.equal(out[lens[0]:], clean[lens[0]:])
        if t is v:
            assert not torch.isfinite(out[at:lens[0]]).any()
    poisoned = q.clone()
    poisoned[at] = bad
    out, _ = call(poisoned, k, v, lens)
    keep = torch.arange(sum(lens)) != at
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[at]).all()


def test_keys_of_minus_infinity():
    """All of a row's logits -inf: it sees nothing that counts, and gives zeros."""
    q, k, v = make([5], [5], 1, 1, 64, torch.float16)
    q[:] = 1.0
    k[:] = 0.0
    k[..., 0] = float("-inf")
    out, _ = call(q, k, v, [5])
    assert (out == 0).all()


def test_wrong_starts_are_flagged_and_stay_in_bounds():
    q, k, v = make([64], [64], 2, 1, 64, torch.float16)
    for at in ([0, 40, 20, 64], [-5, 10, 20, 64], [0, 10, 20, 1000], [3, 2, 1, 0]):
        ws = cs.PromptWorkspace(3, 2, 1, 64, 64)
        out = torch.full_like(q, 7.0)
        cs.cs_prompt_attention(q, k, v, out, torch.tensor(at, dtype=torch.int32, device="cuda"), ws)
        assert cs.cs_get_device_error(ws) == cs.CS_DEVERR_COUNT
        assert torch.isfinite(out).all()


def test_same_bits_again_captured_and_on_another_stream():
    lens, k_lens = [130, 1, 77], [9000, 300, 77]
    q, k, v = make(lens, k_lens, 8, 2, 128, torch.bfloat16)
    first, ws = call(q, k, v, lens, k_lens)
    again, _ = call(q, k, v, lens, k_lens, ws=ws)
    assert torch.equal(first, again)
    side = torch.cuda.Stream()
    out, s, sk = torch.zeros_like(q), starts(lens), starts(k_lens)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cs.cs_prompt_attention(q, k, v, out, s, ws, k_start=sk)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cs.cs_prompt_attention(q, k, v, out, s, ws, k_start=sk)
        cs.cs_prompt_attention(q, k, v, out, s, ws, k_start=sk)
    # other inputs, other lengths: the graph reads them anew
    q2, k2, v2 = make(lens, k_lens, 8, 2, 128, torch.bfloat16, seed=5)
    lens2, k_lens2 = [8, 100, 100], [1, 9276, 100]
    for a, b in ((q, q2), (k, k2), (v, v2), (s, starts(lens2)), (sk, starts(k_lens2))):
        a.copy_(b)
    want, _ = call(q2, k2, v2, lens2, k_lens2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert cs.cs_get_device_error(ws) == 0


@pytest.mark.parametrize("dt", DTS)
def test_long_prompt(dt):
    check(*make([3001, 1500], [3001, 1500], 8, 1, 128, dt), [3001, 1500])


def test_what_is_not_seen_has_no_influence_where_keys_are_cut():
    """The same with records of pieces: few rows over many keys, NaN in the last values, which only the last row sees."""
    q_lens, k_lens = [5], [20000]
    q, k, v = make(q_lens, k_lens, 8, 1, 128, torch.bfloat16)
    clean, _ = call(q, k, v, q_lens, k_lens)
    v[-1] = float("nan")
    out, _ = call(q, k, v, q_lens, k_lens)
    want, bound = ref.prompt(q[:4], k[:-1], v[:-1], [4], [19999])
    assert ((out[:4].double() - want).abs() <= bound).all()
    assert torch.isnan(out[4]).all() and not torch.isnan(clean).any()


def test_more_starts_than_sequences_and_sizes_of_a_larger_workspace():
    """A workspace of larger sizes serves smaller calls; the same tensors, other sequences."""
    q, k, v = make([300], [300], 4, 2, 64, torch.float16)
    ws = cs.PromptWorkspace(9, 8, 2, 128, 1000, 5000)
    for lens in ([300], [0, 300], [1] * 7, [150, 150], [299, 1]):
        n = sum(lens)
        out, _ = call(q, k, v, lens, ws=ws)
        want, bound = ref.prompt(q, k, v, lens, lens)
        assert ((out[:n].double() - want[:n]).abs() <= bound[:n]).all() and (out[n:] == 7.0).all()
    assert cs.cs_get_device_error(ws) == 0


def test_no_query_tokens_and_no_keys():
    ws = cs.PromptWorkspace(2, 2, 1, 64, 10, 10)
    empty = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    cs.cs_prompt_attention(empty, empty[:, :1], empty[:, :1], empty.clone(), starts([0, 0]), ws)
    q = torch.randn(10, 2, 64, device="cuda").half()
    out = torch.full_like(q, 7.0)
    cs.cs_prompt_attention(q, empty[:, :1], empty[:, :1], out, starts([3, 7]), ws, k_start=starts([0, 0]))
    assert (out == 0).all() and cs.cs_get_device_error(ws) == 0


def test_heads_of_every_group_up_to_128():
    for group in (2, 3, 4, 6, 9, 10, 11, 13, 24, 31, 33, 43, 64, 100):
        check(*make([6, 70], [6, 70], group, 1, 64, torch.bfloat16, seed=group), [6, 70])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("q_lens,k_lens,d", [([300, 200], [300, 200], 64), ([400], [400], 128), ([6, 40], [20000, 200], 128),
                                             ([100], [9000], 64)])
def test_bad_values_of_some_channels(q_lens, k_lens, d, dt):
    """Channels whose values are bad throughout, from a key on, or at one key: the other channels keep their bits, and rows
    before a bad value theirs within the bound, whether the keys are cut or not."""
    q, k, v = make(q_lens, k_lens, 8, 2, d, dt)
    clean, _ = call(q, k, v, q_lens, k_lens)
    want, bound = ref.prompt(q, k, v, q_lens, k_lens)
    at = sum(k_lens) - 4      # a key of the last sequence that its last 4 rows see
    bad = v.clone()
    bad[..., 3] = float("inf")
    bad[at:, :, 10] = float("nan")
    bad[at, :, d - 1] = float("-inf")
    out, ws = call(q, k, bad, q_lens, k_lens)
    assert cs.cs_get_device_error(ws) == 0
    rows = sum(q_lens) - 4
    keep = [c for c in range(d) if c not in (3, 10, d - 1)]
    assert torch.equal(out[..., keep], clean[..., keep])
    assert not torch.isfinite(out[..., 3]).any()
    for c in (10, d - 1):
        off = (out[:rows, :, c].double() - want[:rows, :, c]).abs()
        assert (off <= bound[:rows, :, c]).all()
        assert not torch.isfinite(out[rows:, :, c]).any()


def test_all_values_and_all_keys_bad():
    """A prompt of NaN takes no longer than another: no wait runs out over it, and its neighbours are as they were."""
    lens = [6000, 300]
    q, k, v = make(lens, lens, 8, 2, 128, torch.bfloat16)
    clean, _ = call(q, k, v, lens)
    for t in (k, v):
        poisoned = t.clone()
        poisoned[:6000] = float("nan")
        out, ws = call(q, poisoned if t is k else k, poisoned if t is v else v, lens)
        assert cs.cs_get_device_error(ws) == 0
        assert torch.isnan(out[:6000]).all() and torch.equal(out[6000:], clean[6000:])


@pytest.mark.parametrize("q_lens,k_lens", [([500], [500]), ([3], [20000])])
def test_the_largest_values_of_bf16(q_lens, k_lens):
    """Sums over many keys stay in range where the values are of the largest there are."""
    q, k, v = make(q_lens, k_lens, 4, 1, 64, torch.bfloat16)
    v = (v.sign() * 3e38 * (0.5 + 0.5 * torch.rand(v.shape, device="cuda"))).to(torch.bfloat16)
    check(q, k, v, q_lens, k_lens)


@pytest.mark.parametrize("q_lens,k_lens", [
    ([5] * 31, None), ([5] * 32, None), ([0, 300, 0, 0, 1] * 6, None), ([2048], None), ([2049], None), ([1] * 20 + [0] * 11, None),
    ([1, 64, 65], [1000, 64, 984]), ([1, 64, 65], [1000, 64, 985]), ([0] * 30 + [129], [0] * 30 + [2048]), ([0, 0], [0, 0])])
def test_about_the_limits_of_short_lists(q_lens, k_lens):
    """As many sequences, works and keys as are listed without a kernel of their own, one less and one more."""
    for heads, kv, d in ((2, 2, 64), (16, 1, 128)):
        check(*make(q_lens, q_lens if k_lens is None else k_lens, heads, kv, d, torch.bfloat16), q_lens, k_lens)


def test_lists_of_both_kinds_in_turn():
    """Calls that share a workspace, with and without a kernel for the list, eager and captured."""
    q, k, v = make([3000], [3000], 8, 2, 64, torch.float16)
    ws = cs.PromptWorkspace(40, 8, 2, 64, 3000)
    cases = [[100, 50], [2900, 30], [70] * 40, [1, 2, 3], [2048]]
    views = [[t[:sum(lens)] for t in (q, k, v)] + [starts(lens)] for lens in cases]
    want = [call(*x[:3], lens)[0] for x, lens in zip(views, cases)]
    got = [torch.full_like(w, 7.0) for w in want]

    def all_of_them():
        for x, g in zip(views, got):
            cs.cs_prompt_attention(*x[:3], g, x[3], ws)
    all_of_them()
    assert all(torch.equal(w, g) for w, g in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_of_them()
    for g in got:
        g.fill_(7.0)
    graph.replay()
    graph.replay()
    assert all(torch.equal(w, g) for w, g in zip(want, got))
    assert cs.cs_get_device_error(ws) == 0


@pytest.mark.parametrize("batch", [3, 40])
@pytest.mark.parametrize("tq,tk", [(300, 100), (100, 300)])
def test_one_tensor_for_both_starts_of_different_totals(batch, tq, tk):
    """The same starts passed twice are cut to each total by itself, as two tensors of them are."""
    q, k, v = make([tq], [tk], 4, 2, 64, torch.bfloat16)
    at = starts([0] * (batch - 3) + [90, 110, 100])
    ws = cs.PromptWorkspace(batch, 4, 2, 64, tq, tk)
    out, other = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    cs.cs_prompt_attention(q, k, v, out, at, ws, k_start=at, causal=False)
    assert cs.cs_get_device_error(ws, clear=True) == cs.CS_DEVERR_COUNT
    cs.cs_prompt_attention(q, k, v, other, at, ws, k_start=at.clone(), causal=False)
    assert cs.cs_get_device_error(ws) == cs.CS_DEVERR_COUNT
    assert torch.equal(out, other)
    cut = lambda total: [min(x, total) for x in (0, 90, 200, 300)]  # noqa: E731
    q_lens, k_lens = ([b - a for a, b in zip(x, x[1:])] for x in (cut(tq), cut(tk)))
    want, bound = ref.prompt(q, k, v, q_lens, k_lens, False)
    assert ((out.double() - want).abs() <= bound).all()


def fastest(f, n=5):
    """The shortest of n runs, in ms."""
    best = float("inf")
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("causal,lens,heads,kv,d,dt,bad", [
    (False, [4090, 6], 8, 8, 128, torch.bfloat16, [4090]),           # the first value behind a sequence
    (False, [4090, 6], 32, 4, 64, torch.float16, list(range(4090, 4096))),
    (True, [4090, 6], 16, 2, 128, torch.bfloat16, [4091]),
    (True, [4096], 8, 8, 64, torch.float16, list(range(127, 4096, 128)))])
def test_values_that_are_not_seen_cost_no_more_than_the_works_again(causal, lens, heads, kv, d, dt, bad):
    """Rows beside values that are not finite keep their bits, and the call its time within a small factor, although every key
    that they see themselves is finite, or many are."""
    q, k, v = make(lens, lens, heads, kv, d, dt)
    clean, ws = call(q, k, v, lens, causal=causal)
    out, s = torch.empty_like(q), starts(lens)
    run = lambda: cs.cs_prompt_attention(q, k, v, out, s, ws, causal=causal)  # noqa: E731
    before = fastest(run)
    v[bad] = float("nan")
    out.fill_(7.0)
    after = fastest(run)
    first = bad[0] if causal else lens[0]
    assert torch.equal(out[:first], clean[:first])
    assert torch.isnan(out[first:]).all() if causal else torch.isnan(out[lens[0]:]).all()
    assert cs.cs_get_device_error(ws) == 0
    assert after < 10 * before + 0.1, (before, after)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d,group,keys", [(64, 1, 300), (128, 4, 300), (128, 1, 9000)])
def test_seen_infinities_keep_their_sign(d, group, keys, dt):
    """Infinities among the last keys, which some rows see and others do not: with their sign, and NaN where both are seen."""
    n = 300
    q, k, v = make([n], [keys], group, 1, d, dt)
    q *= 0.1        # no weight far from the others
    at = keys - n   # key at + i is query token i's own
    v[at + 200, 0, 3], v[at + 250, 0, 7], v[at + 270, 0, 7], v[at + 280, 0, 9] = (float(x) for x in ("inf", "-inf", "inf", "nan"))
    out, ws = call(q, k, v, [n], [keys])
    clean = v.clone()
    clean[~torch.isfinite(clean)] = 0.0
    want, _ = call(q, k, clean, [n], [keys])
    mended = out.clone()
    for c, first, what in ((3, 200, torch.isposinf), (7, 250, lambda x: ~torch.isfinite(x)), (9, 280, torch.isnan)):
        assert what(out[first:, :, c]).all() and torch.isfinite(out[:first, :, c]).all()
        mended[first:, :, c] = want[first:, :, c]
    assert torch.isneginf(out[250:270, :, 7]).all()
    keep = torch.ones(d, dtype=torch.bool)
    keep[[3, 7, 9]] = False
    assert torch.equal(mended[..., keep], want[..., keep]) and torch.equal(mended[:200], want[:200])
    assert cs.cs_get_device_error(ws) == 0


def test_spoilt_works_of_a_long_list():
    """More works to a CTA than have a mark of their own; sequences of one token, whose outputs are their values."""
    batch, heads, d = 4096, 64, 64
    lens = [1] * batch
    q, k, v = make(lens, lens, heads, heads, d, torch.float16)
    bad = torch.arange(batch, device="cuda") % 97 == 5
    v[bad] = float("nan")
    out, ws = call(q, k, v, lens)
    assert torch.equal(out[~bad], v[~bad]) and torch.isnan(out[bad]).all()
    assert cs.cs_get_device_error(ws) == 0


def test_a_captured_call_beside_bad_values():
    q, k, v = make([500, 200], [500, 200], 8, 2, 128, torch.bfloat16)
    s = starts([500, 200])
    clean, ws = call(q, k, v, [500, 200])
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cs.cs_prompt_attention(q, k, v, out, s, ws)
    good = v[500].clone()
    for _ in range(3):
        v[500] = float("inf")
        graph.replay()
        assert torch.equal(out[:500], clean[:500]) and not torch.isfinite(out[500:]).any()
        v[500] = good
        graph.replay()
        assert torch.equal(out, clean)
    assert cs.cs_get_device_error(ws) == 0


def test_a_workspace_serves_fewer_key_heads():
    """More works than a workspace for as many key/value heads as query heads would list: 12,000 tokens, two to a pair."""
    lens = [100] * 120
    q, k, v = make(lens, lens, 128, 4, 64, torch.float16)
    ws = cs.PromptWorkspace(120, 128, 128, 64, 12000)
    for kv in (1, 2, 4):
        out, _ = call(q, k[:, :kv], v[:, :kv], lens, ws=ws)
        want, _ = call(q, k[:, :kv], v[:, :kv], lens)
        assert torch.equal(out, want) and cs.cs_get_device_error(ws) == 0


@pytest.mark.parametrize("batch", [255, 256, 257, 700])
def test_more_sequences_than_listing_threads(batch):
    """Several sequences' starts to a thread of the list's kernel, empty ones and those with an earlier part among them."""
    g = torch.Generator().manual_seed(batch)
    q_lens = torch.randint(0, 6, (batch,), generator=g).tolist()
    k_lens = [n + int(x) for n, x in zip(q_lens, torch.randint(0, 20, (batch,), generator=g))]
    check(*make(q_lens, k_lens, 4, 2, 64, torch.bfloat16), q_lens, k_lens)


@pytest.mark.parametrize("d", [64, 128])
def test_one_token_and_one_head_of_any_stride(d):
    """The only row there is starts on a 16-byte boundary, whatever the strides that lead to others."""
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(4, 1, d + 1, generator=g, device="cuda").half()
    x = [torch.empty(d + 9, dtype=torch.float16, device="cuda")[:d + 1].copy_(t[0]).unsqueeze(0) for t in x]
    q, k, v, out = (t[:, :d].unsqueeze(1) for t in x)
    assert q.stride(0) % 8
    ws = cs.PromptWorkspace(1, 1, 1, d, 1)
    cs.cs_prompt_attention(q, k, v, out, starts([1]), ws)
    assert torch.equal(out, v) and cs.cs_get_device_error(ws) == 0


@pytest.mark.parametrize("q_lens,k_lens", [([300], [300]), ([5], [20000])])
def test_small_values_of_bf16(q_lens, k_lens):
    """Values near 2^-96: a key's p v is off by at most 2^-150 more, and the largest alone is 2^-128 (p of it 2^-32), of which
    300 keys' are 2^-14 at most; 20,000 with logits of a width of 1 to 2 have sums of 100 times that."""
    q, k, v = make(q_lens, k_lens, 4, 1, 64, torch.bfloat16)
    check(q, k, (v.double() * 2.0 ** -96).to(torch.bfloat16), q_lens, k_lens)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d,group,keys", [(64, 1, 300), (128, 4, 300), (128, 1, 9000)])
def test_infinities_of_both_signs_are_nan(d, group, keys, dt):
    """Both among the keys that not all rows of a work see; and NaN before an infinity."""
    n = 300
    q, k, v = make([n], [keys], group, 1, d, dt)
    q *= 0.1
    at = keys - n
    for i, c, x in ((258, 3, "-inf"), (264, 3, "inf"), (258, 5, "nan"), (264, 5, "inf"), (258, 6, "inf"), (264, 6, "inf")):
        v[at + i, 0, c] = float(x)
    out, ws = call(q, k, v, [n], [keys])
    assert torch.isfinite(out[:258]).all()
    assert torch.isneginf(out[258:264, :, 3]).all() and torch.isnan(out[264:, :, 3]).all()
    assert torch.isnan(out[258:, :, 5]).all() and torch.isposinf(out[258:, :, 6]).all()
    assert cs.cs_get_device_error(ws) == 0
