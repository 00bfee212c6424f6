"""Plain 64-bit forms of the 4-bit KV cache's operators (CPU tensors), written
from their definitions in include/cs.h."""
import numpy as np
import torch

GROUP = 64


def half_step(dt):
    """The largest relative error of one rounding to dt."""
    return torch.finfo(dt).eps / 2


def quantise(x):
    """codes [..., d/2] uint8 and scales [..., d/64, 2] fp16 of rows x [..., d]."""
    g = torch.nan_to_num(x.float(), nan=0.0, posinf=65504.0, neginf=-65504.0).clamp(-65504.0, 65504.0)
    g = g.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1).values, g.max(-1).values
    s = torch.from_numpy(((hi - lo).numpy() * np.float32(1.0 / 15.0)).astype(np.float32)).half()
    z = lo.half()
    sd = s.double()[..., None]
    q = (g.double() - z.double()[..., None]) / torch.where(sd > 0, sd, torch.ones_like(sd))
    n = torch.where(sd > 0, torch.from_numpy(np.rint(q.numpy())).clamp(0, 15), torch.zeros_like(q))
    n = n.to(torch.uint8).reshape(x.shape)
    return n[..., 0::2] + 16 * n[..., 1::2], torch.stack([s, z], -1)


def values(codes, scales, spread=False):
    """What the codes stand for, in 64 bits; spread: |offset| + scale * code instead (for error bounds)."""
    d = 2 * codes.shape[-1]
    n = torch.stack([codes % 16, codes // 16], -1).reshape(*codes.shape[:-1], d // GROUP, GROUP).double()
    s, z = scales[..., 0:1].double(), scales[..., 1:2].double()
    return (n * s + (z.abs() if spread else z)).reshape(*codes.shape[:-1], d)


def attention(k, ks, v, vs, pos, q, length, q_pos=None, on=None, scale=0.0, old=None, decay=1.0):
    """(out, its error bound per unit step, weight, its error bound).  k..pos are the cache's arrays, q [B, n_q, H, d];
    on: bool [B, H].  The bounds add, for every row, the first-order effect of

      - a logit error of at most 2^-18 A, A = |scale| sum |q| (|offset| + s code): q in two fp16 parts (2^-22), products exact,
        sums of 16 channels whose partial sums may be cut off (2^-22 of their size, 4 chains of 4), a handful of fp32
        roundings, the exponent's argument in fp32;
      - 2^-18 for p, its two fp16 parts, the exponential and the division;
      - sums over N slots in chains of N / 16 products with 2^-23 each.
    """
    B, n_q, H, d = q.shape
    kv, cap = k.shape[1:3]
    G = H // kv
    sc = scale or d ** -0.5
    out = torch.zeros(B, n_q, H, d, dtype=torch.float64)
    err = torch.zeros_like(out)
    w = torch.zeros(B, kv, cap, dtype=torch.float64) if old is None else old.double().clone()
    werr = torch.zeros(B, kv, cap, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(length[b]), 0), cap)
        for h in range(kv):
            kk, vv = values(k[b, h, :n], ks[b, h, :n]), values(v[b, h, :n], vs[b, h, :n])
            ka, va = values(k[b, h, :n], ks[b, h, :n], True), values(v[b, h, :n], vs[b, h, :n], True)
            mass = torch.zeros(n, dtype=torch.float64)
            merr = torch.zeros(n, dtype=torch.float64)
            for t in range(n_q):
                ok = torch.ones(n, dtype=torch.bool)
                if q_pos is not None:
                    p = pos[b, h, :n]
                    ok = (p >= 0) & (p <= int(q_pos[b]) + t)
                for j in range(h * G, (h + 1) * G):
                    if (on is not None and not on[b, j]) or not ok.any():
                        continue
                    x = q[b, t, j].double()
                    s = sc * (kk[ok] @ x)
                    delta = 2.0 ** -18 * (abs(sc) * (ka[ok] @ x.abs())).max()
                    e = torch.exp(s - s.max())
                    p = e / e.sum()
                    rel = 2 * delta + 2.0 ** -18 + n / 16 * 2.0 ** -23
                    out[b, t, j] = p @ vv[ok]
                    err[b, t, j] = rel * (p @ va[ok])
                    mass[ok] += p
                    merr[ok] += rel * p
            w[b, h, :n] = (decay * old[b, h, :n].double() if decay and old is not None else 0.0) + mass
            werr[b, h, :n] = merr + 2.0 ** -22 * w[b, h, :n].abs() + 1e-30
    return out, err, w, werr


def order(weight, pos, sinks, recent, next_pos):
    """The order in which one head's slots are given up."""
    def cls(i):
        if pos is None:
            return 1
        p = int(pos[i])
        return 0 if p < 0 else 2 if p < sinks or (recent > 0 and p >= next_pos - recent) else 1
    w = np.asarray(weight, dtype=np.float64)
    rank = [(cls(i), not np.isnan(w[i]), 0.0 if np.isnan(w[i]) else w[i] + 0.0, i) for i in range(len(w))]
    return [r[3] for r in sorted(rank)]


def evict(weight, pos, length, limit, n, sinks=0, recent=0, next_pos=None):
    B, kv = weight.shape[:2]
    out = torch.empty(B, kv, n, dtype=torch.int32)
    for b in range(B):
        used = min(int(length[b]), limit)
        give = max(0, n - (limit - used))
        for h in range(kv):
            o = order(weight[b, h, :used], None if pos is None else pos[b, h, :used], sinks, recent,
                      None if next_pos is None else int(next_pos[b]))
            out[b, h] = torch.tensor(sorted(o[:give]) + list(range(used, used + n - give)), dtype=torch.int32)
    return out


def stays(weight, pos, length, keep, sinks=0, recent=0, next_pos=None):
    """[b][h] -> the slots that a trim leaves, ascending."""
    got = []
    for b in range(weight.shape[0]):
        used = int(length[b])
        got.append([sorted(order(weight[b, h, :used], None if pos is None else pos[b, h, :used], sinks, recent,
                                 None if next_pos is None else int(next_pos[b]))[max(0, used - keep):])
                    for h in range(weight.shape[1])])
    return got
