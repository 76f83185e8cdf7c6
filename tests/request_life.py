"""Plain 64-bit references of the calls around the verification pass: prompt
attention, log probabilities, and the page calls (plain Python on lists)."""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def paged_batch(seed, lens, prefix, Hq, Hkv, D, bs, dtype, spread=1.0, extra_rows=0, device="cuda"):
    """Random inputs of one prompt-attention call.  Everything that is not a
    request's own slot holds NaN: the pages' ends, the unused pages, and
    extra_rows rows of q behind the last request."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-(n + p) // bs) for n, p in zip(lens, prefix)]
    nb = sum(used) + 3
    width = max(used + [1]) + 1
    perm = torch.randperm(nb, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    k = torch.full((nb, Hkv, bs, D), math.nan)
    v = k.clone()
    at = 0
    for b, (n, p) in enumerate(zip(lens, prefix)):
        ids = perm[at:at + used[b]]
        at += used[b]
        table[b, :used[b]] = torch.tensor(ids, dtype=torch.int32)
        for j, page in enumerate(ids):
            m = min(bs, n + p - j * bs)
            k[page, :, :m] = torch.randn((Hkv, m, D), generator=g) * spread
            v[page, :, :m] = torch.randn((Hkv, m, D), generator=g)
    T = sum(lens)
    q = torch.full((T + extra_rows, Hq, D), math.nan)
    q[:T] = torch.randn((T, Hq, D), generator=g)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    d = dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), table=table, seq_off=torch.from_numpy(off),
             prefix=torch.tensor(prefix, dtype=torch.int32))
    d = {n: t.to(device) for n, t in d.items()}
    d.update(B=len(lens), T=T + extra_rows, n_max=max(lens), max_prefix=max(prefix), Hq=Hq, Hkv=Hkv, D=D, bs=bs, nb=nb,
             scale=1.0 / math.sqrt(D))
    return d


def prompt_reference(d):
    """(out, tolerance) in 64 bits.  With w_k the softmax weights and A = sum
    w_k |v_k|, an output is off by at most half a step of its type, plus, for
    bf16, half a step on every weight (A * 2^-8: the probabilities are rounded
    before the product with V); plus, in 32 bits, the relative error of a
    weight: D products and sums of a score (D 2^-24 on sum |q k|), the scaled
    difference and the exponential (2^-21 and 2^-22 |score|), and N sums."""
    Hkv, g, D, bs = d["Hkv"], d["Hq"] // d["Hkv"], d["D"], d["bs"]
    off, prefix = d["seq_off"].tolist(), d["prefix"].tolist()
    out = torch.full(d["q"].shape, math.nan, dtype=torch.float64, device=d["q"].device)
    tol = out.clone()
    half = U[d["q"].dtype]
    for b in range(d["B"]):
        n, P = off[b + 1] - off[b], prefix[b]
        if n == 0:
            continue
        ids = d["table"][b, :-(-(P + n) // bs)].long()
        for h in range(Hkv):
            k = d["k"][ids, h].reshape(-1, D)[:P + n].double()
            v = d["v"][ids, h].reshape(-1, D)[:P + n].double()
            q = d["q"][off[b]:off[b] + n, h * g:(h + 1) * g].double()
            s = torch.einsum("ngd,kd->ngk", q, k) * d["scale"]
            unseen = torch.arange(P + n, device=q.device)[None] > (P + torch.arange(n, device=q.device))[:, None]
            w = torch.softmax(s.masked_fill(unseen[:, None], -math.inf), -1)
            o, A = torch.einsum("ngk,kd->ngd", w, v), torch.einsum("ngk,kd->ngd", w, v.abs())
            size = torch.einsum("ngd,kd->ngk", q.abs(), k.abs()).amax(-1) * d["scale"]
            rel = D * 2.0 ** -24 * size + 2.0 ** -21 + 2.0 ** -22 * size + (P + n) * 2.0 ** -24
            t = half * o.abs() + 2 * rel[..., None] * A
            if half > 2.0 ** -20:
                t += half * A
            out[off[b]:off[b] + n, h * g:(h + 1) * g] = o
            tol[off[b]:off[b] + n, h * g:(h + 1) * g] = t * 1.01
    return out, tol


def rank_order(x):
    """Indices of x (1-D, 64 bits) in rank order: larger first, equal by lower
    index, NaN last."""
    key = np.where(np.isnan(x), np.inf, -x) + 0.0
    return np.lexsort((np.arange(len(x)), key, np.isnan(x)))


def logprob_reference(x, token, tau, k):
    """(logprob, entropy, rank, top ids, top logprobs) of one row in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        z = (x - x.max()) * tau
        e = np.exp(z)
        lse = np.log(e.sum())
        logp = z - lse
        p = np.exp(logp)
        ent = -np.where(p > 0, p * logp, 0.0).sum() if not np.isnan(lse) else math.nan
    order = rank_order(x)
    rank = -1 if token < 0 else int(np.where(order == token)[0][0])
    top = order[:k]
    return (logp[token] if token >= 0 else math.nan), ent, rank, top, logp[top]


class Pages:
    """The page calls on Python lists: a table, a pool and (layers, 2) caches
    as numpy arrays [num_blocks][Hkv][bs][D]."""

    def __init__(self, table, pool, count, num_blocks, bs, caches=()):
        self.table = [list(map(int, r)) for r in table]
        self.pool, self.count = list(map(int, pool)), int(count)
        self.nb, self.bs, self.caches = num_blocks, bs, caches

    def fork(self, src, dst, length, room):
        B, mb, bs = len(self.table), len(self.table[0]), self.bs
        N = len(src)
        status, plan = [0] * N, [None] * N
        for i in range(N):
            s, d, n, r = src[i], dst[i], length[i], room[i]
            if not (-1 <= s < B and 0 <= d < B and n >= 0 and r >= 0 and (s >= 0 or n == 0)):
                status[i] = 128
            elif dst.count(d) > 1 or (s >= 0 and s != d and s in dst):
                status[i] = 128
            elif n + r > mb * bs:
                status[i] = 4
            else:
                full, held, need = n // bs, -(-n // bs), -(-(n + r) // bs)
                source = self.table[s][:held] if s >= 0 else []
                if any(not 0 <= p < self.nb for p in source):
                    status[i] |= 16
                if s == d:
                    fresh = [j for j in range(held, need) if self.table[d][j] < 0]
                    if any(p >= self.nb for p in self.table[d][held:need]):
                        status[i] |= 16
                else:
                    fresh = list(range(full, need))
                    if any(p >= 0 for p in self.table[d][:need]):
                        status[i] |= 128
                plan[i] = (full, source, fresh)
        total = sum(len(plan[i][2]) for i in range(N) if not status[i])
        bad = 0
        if total and not total <= self.count <= len(self.pool):
            bad = 4
        elif any(not 0 <= p < self.nb for p in self.pool[self.count - total:self.count]):
            bad = 16
        for i in range(N):
            if status[i]:
                continue
            full, source, fresh = plan[i]
            if fresh and bad:
                status[i] = bad
                continue
            row = self.table[dst[i]]
            if src[i] != dst[i]:
                row[:full] = source[:full]
            for j in fresh:
                self.count -= 1
                row[j] = self.pool[self.count]
            tail = length[i] - full * self.bs
            if src[i] != dst[i] and tail:
                for c in self.caches:
                    c[row[full], :, :tail] = c[source[full], :, :tail]
        return status

    def free(self, rows, keep):
        B, bs = len(self.table), self.bs
        status, drop = [], []
        for i, r in enumerate(rows):
            st = 0
            if not 0 <= r < B or keep[i] < 0 or rows.count(r) > 1:
                st = 128
            else:
                j0 = min(len(self.table[0]), -(-keep[i] // bs))
                if any(p >= self.nb for p in self.table[r][j0:]):
                    st = 16
                else:
                    drop.append((i, r, j0))
            status.append(st)
        kept = [list(r) for r in self.table]
        for _, r, j0 in drop:
            kept[r][j0:] = [-1] * (len(kept[r]) - j0)
        held = {p for r in kept for p in r}
        released, owner = [], []
        for i, r, j0 in drop:
            for p in self.table[r][j0:]:
                if p >= 0 and p not in held and p not in released:
                    released.append(p)
                    owner.append(i)
        if released and not 0 <= self.count <= len(self.pool) - len(released):
            for i in set(owner):
                status[i] |= 4
            return status
        self.table = kept
        self.pool[self.count:self.count + len(released)] = released
        self.count += len(released)
        return status

    def compact(self):
        free = self.pool[:self.count] if 0 <= self.count <= len(self.pool) else None
        held = {p for r in self.table for p in r if p >= 0}
        if free is None or len(set(free)) < len(free) or any(not 0 <= p < self.nb for p in free) or held & set(free) or \
                any(p >= self.nb for p in held):
            return 16, list(range(self.nb)), 0
        both = sorted(held | set(free))
        n = len(held)
        new = [p for p in both[:n] if p not in held]
        old = [p for p in both[n:] if p in held]
        to = list(range(self.nb))
        for a, b in zip(old, new):
            to[a] = b
            for c in self.caches:
                c[b] = c[a]
        self.table = [[to[p] if p >= 0 else p for p in r] for r in self.table]
        self.pool[:self.count] = both[n:][::-1]
        return 0, to, len(old)
