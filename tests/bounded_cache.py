"""Plain 64-bit references of the calls between a projection and a bounded
cache: norms, rotation and append, gathered attention weight, eviction."""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def offsets(lens):
    return ints([0] + np.cumsum(lens).tolist() if len(lens) else [0])


def table_of(seed, slots, bs, extra=3):
    """(table, num_blocks): shuffled pages for rows of these slot counts, -1 behind them."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-s // bs) for s in slots]
    nb = sum(used) + extra
    perm = torch.randperm(nb, generator=g).tolist()
    table = torch.full((len(slots), max(used + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), nb


def rope_reference(qkv, Hq, Hkv, rot, pairing, freq, position, q_norm, k_norm, eps):
    """([T][Hq + Hkv][D] turned heads, tolerance) in 64 bits; position: [T][rot / 2]
    whole numbers.  An output is off by half a step of its type; in 32 bits by the
    norm (D products and sums under a root, D / 2 units; divisions and products,
    8), the angle (half a turn rounded, pi units, and the 64-bit turns, 1) and its
    sine and cosine (4), and the rotation's three operations, all relative to the
    pair's length."""
    D = qkv.shape[-1]
    x = qkv[:, :Hq + Hkv].double()
    for heads, norm in ((slice(0, Hq), q_norm), (slice(Hq, Hq + Hkv), k_norm)):
        if norm is not None:
            y = x[:, heads]
            x[:, heads] = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * norm.double()
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if pairing else (i, i + rot // 2)
    angle = position.double() * freq.double()[None] if rot else position.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    out, size = x.clone(), x.abs()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = torch.hypot(x[..., a], x[..., b])
    units = D / 2 + 20
    return out, (U[qkv.dtype] * out.abs() + units * 2.0 ** -24 * size) * 1.01


def weight_reference(d, before, decay, path=None, accept=None, window=0):
    """([B][Hkv][stride] weights with NaN where nothing is written, tolerance).
    A probability is off, relatively, by the D products and sums of its score and
    of the scores its row's sum holds (D 2^-24 of sum |q k|, twice), the scaled
    difference and the exponentials (2^-21 + 2^-22 of that size, twice) and N sums
    (N 2^-24); a slot's sum over R rows by R + 2 units more; one below 2^-120 may
    be lost."""
    Hkv, g, D, bs = d["Hkv"], d["Hq"] // d["Hkv"], d["D"], d["bs"]
    off, prefix = d["seq_off"].tolist(), d["prefix"].tolist()
    B = len(prefix)
    stride = before.shape[-1] if before is not None else d["stride"]
    out = torch.full((B, Hkv, stride), math.nan, dtype=torch.float64, device=d["q"].device)
    tol = torch.zeros_like(out)
    for b in range(B):
        P = prefix[b]
        m = off[b + 1] - off[b] if path is None else int(accept[b])
        rows = list(range(m))
        first = max(0, m - window) if window else 0
        ids = d["table"][b, :-(-(P + m) // bs)].long()
        for h in range(Hkv):
            total = torch.zeros(P + m, dtype=torch.float64, device=out.device)
            if before is not None:
                total[:P] = decay * before[b, h, :P].double()
            err = total.abs() * 2.0 ** -23
            k = d["k"][ids, h].reshape(-1, D)[:P + m].double()
            if first < m:
                at = torch.tensor([off[b] + (i if path is None else int(path[b][i])) for i in rows[first:]], device=out.device)
                q = d["q"][at, h * g:(h + 1) * g].double()
                seen = P + torch.arange(first, m, device=out.device)
                z = torch.einsum("mgd,kd->mgk", q, k) * d["scale"]
                hidden = torch.arange(P + m, device=out.device)[None] > seen[:, None]
                p = torch.softmax(z.masked_fill(hidden[:, None], -math.inf), -1)
                size = torch.einsum("mgd,kd->mgk", q.abs(), k.abs()).masked_fill(hidden[:, None], 0.0).amax(-1, keepdim=True) * d["scale"]
                rel = 2 * (D * 2.0 ** -24 * size + 2.0 ** -21 + 2.0 ** -22 * size) + (P + m) * 2.0 ** -24
                added = p.sum((0, 1))
                err += (p * rel).sum((0, 1)) + ((m - first) * g + 2) * 2.0 ** -24 * (added + total) + (m - first) * g * 2.0 ** -120
                total = total + added
            out[b, h, :P + m] = total
            tol[b, h, :P + m] = err * 1.01
    return out, tol


def keep_reference(w, length, keep, first, last):
    """The slots that stay (plain Python): w a list of weights or None."""
    kept = min(keep, length)
    first = min(first, kept)
    last = min(last, kept - first)
    mid = list(range(first, length - last))

    def order(s):
        x = 0.0 if w is None else w[s]
        return (x != x, 0.0 if x != x else -x, s)
    heavy = sorted(mid, key=order)[:kept - first - last]
    return list(range(first)) + sorted(heavy) + list(range(length - last, length))
