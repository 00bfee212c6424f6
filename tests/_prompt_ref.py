"""Plain 64-bit forms of the prompt's and the drafted tree's attention, written from their definitions in include/cs.h, with
bounds on what the kernels may be off by."""
import torch

import _qcache_ref as qref

half_step = qref.half_step


def rows(q, k, v, ok, scale, dt, delta, p_step, v_step=0.0):
    """(out, bound) of query rows q [R, d] over keys k, v [n, d], which a row sees where ok [R, n]; 64 bits.

    delta: per unit of A = |scale| sum |q| |k|, how far a logit may be off; p_step, v_step: relative steps of p's and v's
    roundings.  First-order effects on an output, of terms p |v|: 2 A delta (in p and in the sum), p_step + v_step, 2^-18 for
    the exponential, its argument and the division, and 2^-23 for each of the n / 16 cut off sums of a chain; p below the
    smallest normal value of its type, 2^-32 of the sum for each key; then the output's own rounding."""
    s = scale * (q @ k.T)
    top = torch.where(ok, s, -1e300).max(-1, keepdim=True).values
    e = torch.where(ok, torch.exp(s - top), 0.0)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total.clamp(min=1e-300), 0.0)
    v = torch.where(ok.any(0)[:, None], v, 0.0)       # what no row sees may be anything
    out = p @ v
    a = abs(scale) * (q.abs() @ k.abs().T)
    a = torch.where(ok, a, 0.0).max(-1, keepdim=True).values
    n = k.shape[0]
    terms = p @ v.abs()
    rel = 2 * delta * a + p_step + v_step + 2.0 ** -18 + n / 16 * 2.0 ** -23
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    bound = rel * terms + n * 2.0 ** -32 * v.abs().amax(0, keepdim=True).clamp(max=1e300) if n else torch.zeros_like(out)
    return out, bound + half_step(dt) * (out.abs() + bound) + tiny


def prompt(q, k, v, q_lens, k_lens, causal=True, scale=0.0):
    """(out, bound), [Tq, H, d] in 64 bits on the inputs' device."""
    dt, (tq, heads, d), kv = q.dtype, q.shape, k.shape[1]
    out = torch.zeros(tq, heads, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    q0 = k0 = 0
    for lq, lk in zip(q_lens, k_lens):
        for h in range(heads):
            if lq == 0:
                continue
            g = h // (heads // kv)
            ok = torch.ones(lq, lk, dtype=torch.bool, device=q.device)
            if causal:
                ok = ok.tril(lk - lq)
            out[q0:q0 + lq, h], bound[q0:q0 + lq, h] = rows(
                q[q0:q0 + lq, h].double(), k[k0:k0 + lk, g].double(), v[k0:k0 + lk, g].double(), ok, scale or d ** -0.5, dt,
                2.0 ** -18, half_step(dt)) if lk else (0.0, 0.0)
        q0, k0 = q0 + lq, k0 + lk
    return out, bound


def paths(parent, n):
    """[n, n] bool: token j is token t or one of its ancestors."""
    ok = torch.zeros(n, n, dtype=torch.bool)
    for t in range(n):
        a = t
        while a >= 0:
            ok[t, a] = True
            a = a - 1 if parent is None else (int(parent[a]) if -1 <= int(parent[a]) < a else -1)
    return ok


def drafted(x):
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=65504.0, neginf=-65504.0).clamp(-65504.0, 65504.0)
    return x.half().double()


def tree(k, ks, v, vs, pos, q, kn, vn, length, parent=None, n_new=None, scale=0.0):
    """(out, bound) [B, n, H, d]; k .. pos are the cache's arrays (CPU), pos or None."""
    B, n, H, d = q.shape
    kv, cap = k.shape[1:3]
    out = torch.zeros(B, n, H, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        m = n if n_new is None else min(max(int(n_new[b]), 0), n)
        L = min(max(int(length[b]), 0), cap)
        if m == 0:
            continue
        ok_new = paths(None if parent is None else parent[b], m)
        for h in range(H):
            g = h // (H // kv)
            live = torch.ones(L, dtype=torch.bool) if pos is None else pos[b, g, :L] >= 0
            kk, vv = qref.values(k[b, g, :L], ks[b, g, :L]), qref.values(v[b, g, :L], vs[b, g, :L])
            kk, vv = torch.where(live[:, None], kk, 0.0), torch.where(live[:, None], vv, 0.0)
            # keys and values in fp16: half a step each; q too, of the row's largest 2^-29 at the most
            out[b, :m, h], bound[b, :m, h] = rows(
                q[b, :m, h].double(), torch.cat([kk, drafted(kn[b, :m, g])]), torch.cat([vv, drafted(vn[b, :m, g])]),
                torch.cat([live.expand(m, L), ok_new], 1), scale or d ** -0.5, q.dtype, half_step(torch.float16) + 2.0 ** -18,
                half_step(torch.float16), half_step(torch.float16))
    return out, bound
