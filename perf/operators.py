"""The operators of a request's life around the verification pass, as cases to
measure: prompt attention over the paged cache, log probabilities of tokens,
and the page calls (fork, free, compact).

Each case runs either in its plain form (elementary torch operations in 32
bits) or, with `own` set, through the library's entry points."""
import math
import random

import torch

own = False

DEV = "cuda"
ATTENTION, SCORES, PATH, FORK, FREE, COMPACT = "attention", "token scores", "path scores", "fork", "free", "compact"


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # sixteen prompts admitted together into a server's 16-token pages, 128 to 4096 tokens each
        attention("16 prompts packed", 16, 128, 4096, 0, 0, 32, 8, 128, 16, "bf16", 11),
        # one long document from its first token
        attention("one prompt of 16384", 1, 16384, 16384, 0, 0, 32, 8, 128, 256, "bf16", 12),
        # the next chunk of four long prompts whose first 8192 tokens are already cached, wide groups
        attention("chunks after 8192", 4, 512, 512, 8192, 8192, 64, 8, 128, 256, "bf16", 13),
        # a batch of single tokens over ragged prefixes: the decode step without a draft
        attention("64 single tokens", 64, 1, 1, 256, 16384, 32, 8, 128, 16, "bf16", 14),
        # the smallest model of the tests: fp32, no grouping, an odd length
        attention("small fp32", 2, 97, 129, 0, 128, 4, 4, 64, 16, "fp32", 15),
        # prompt scoring: every token of 2048 positions with its entropy and 20 alternatives, large vocabulary
        scores("2048 positions", 8, 2048, 128256, 20, "fp32", 21),
        # one sampled token of one request
        scores("one position", 1, 1, 32000, 5, "fp32", 22),
        # the emitted tokens of a batched verification step
        path_scores("64 accepted paths", 64, 64, 32000, 5, "bf16", 23),
        # parallel sampling: 64 continuations of four prompts, large pages, every layer's partial page copied
        pages("fork 64 rows", FORK, 32, 128, 8, 128, 256, "bf16", rows=72, max_blocks=16, n=64, sources=4, room=64, seed=31),
        # one more beam of a short request, and room for its next tree
        pages("fork 2 rows", FORK, 2, 256, 8, 128, 16, "bf16", rows=8, max_blocks=64, n=2, sources=2, room=64, seed=32),
        # 64 finished requests of 256, half of their pages shared with others
        pages("free 64 rows", FREE, 1, 262144, 1, 64, 16, "bf16", rows=256, max_blocks=1024, n=64, sources=32, room=0, seed=33),
        # a fragmented pool brought together before the cache is shrunk
        pages("compact 600 pages", COMPACT, 32, 2048, 8, 128, 16, "bf16", rows=64, max_blocks=64, n=600, sources=0, room=0, seed=34),
    ]


def attention(name, B, n_lo, n_hi, p_lo, p_hi, Hq, Hkv, D, bs, dtype, seed):
    return dict(name=name, op=ATTENTION, B=B, n_lo=n_lo, n_hi=n_hi, p_lo=p_lo, p_hi=p_hi, Hq=Hq, Hkv=Hkv, D=D, bs=bs, dtype=dtype, lens=seed)


def scores(name, B, T, V, k, dtype, seed):
    return dict(name=name, op=SCORES, B=B, T=T, V=V, k=k, dtype=dtype, lens=seed)


def path_scores(name, B, n_max, V, k, dtype, seed):
    return dict(name=name, op=PATH, B=B, n_max=n_max, V=V, k=k, dtype=dtype, lens=seed)


def pages(name, op, layers, blocks, Hkv, D, bs, dtype, rows, max_blocks, n, sources, room, seed):
    return dict(name=name, op=op, layers=layers, blocks=blocks, Hkv=Hkv, D=D, bs=bs, dtype=dtype, rows=rows, max_blocks=max_blocks, n=n, sources=sources,
                room=room, lens=seed)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice((ATTENTION, ATTENTION, ATTENTION, SCORES, SCORES, PATH, FORK, FREE, COMPACT))
    seed = rng.randrange(1 << 30)
    if op == ATTENTION:
        Hq, Hkv, D = rng.choice(((32, 8, 128), (64, 8, 128), (16, 4, 128), (8, 2, 64), (16, 2, 64), (4, 4, 64), (6, 2, 64), (20, 4, 128), (5, 1, 64)))
        dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
        B, n_hi, p_hi = _log(rng, 1, 64), _log(rng, 1, 12000), rng.choice((0, _log(rng, 1, 16384)))
        if dtype == "fp32":
            n_hi, p_hi = min(n_hi, 1 + n_hi % 1500), min(p_hi, 1 + p_hi % 4000)
        while B > 1 and B * Hq * n_hi * (n_hi + p_hi) > 16 * 16384 * 16384:
            B = (B + 1) // 2
        while B * Hq * n_hi * (n_hi + p_hi) > 16 * 16384 * 16384:
            n_hi = n_hi * 2 // 3
        c = attention("", B, rng.choice((0, 1, n_hi, (n_hi + 1) // 2)), n_hi, rng.choice((0, p_hi // 2, p_hi)), p_hi, Hq, Hkv, D, rng.choice((8, 16, 64, 256)), dtype, seed)
    elif op == SCORES:
        V = rng.choice((_log(rng, 50, 131072), 32000, 128256))
        T = _log(rng, 1, max(1, min(4096, 2000 * 128256 // V)))
        c = scores("", rng.randint(1, min(T, 16)), T, V, min(V, rng.choice((0, 1, 5, 20, 32))), rng.choice(("fp32", "bf16")), seed)
    elif op == PATH:
        V = rng.choice((_log(rng, 50, 131072), 32000))
        c = path_scores("", _log(rng, 1, 64), rng.randint(2, 64), V, min(V, rng.choice((0, 1, 5, 20, 32))), rng.choice(("fp32", "bf16")), seed)
    elif op == FREE:
        rows, max_blocks = _log(rng, 2, 300), _log(rng, 4, 1024)
        n = rng.randint(1, rows)
        c = pages("", FREE, 1, rows * max_blocks, 1, 64, rng.choice((8, 16, 64)), "bf16", rows, max_blocks, n, max(1, rows // rng.choice((2, 8))), 0, seed)
    else:
        layers, Hkv, D = rng.choice((1, 2, 7, 32)), rng.choice((1, 2, 8)), rng.choice((64, 128))
        bs, dtype = rng.choice((8, 16, 64)), rng.choice(("bf16", "fp32"))
        if op == COMPACT:
            blocks = _log(rng, 16, min(2048, 6 * 10 ** 8 // (layers * Hkv * D * bs)))
            c = pages("", COMPACT, layers, blocks, Hkv, D, bs, dtype, _log(rng, 8, 64), 64, rng.randint(1, max(1, blocks // 4)), 0, 0, seed)
        else:
            rows, max_blocks, room = _log(rng, 3, 64), rng.randint(8, 24), rng.randint(0, 60)
            sources = rng.randint(1, (rows + 1) // 2)
            c = pages("", FORK, layers, rows * max_blocks + 8, Hkv, D, bs, dtype, rows, max_blocks, rng.randint(1, rows - sources), sources, room, seed)
    del c["name"]
    return c


# ------------------------------------------------------- sizes of one case ----

def _lengths(c):
    """New tokens and cached tokens of each request of an attention case."""
    r = random.Random(c["lens"])
    n = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    n[r.randrange(c["B"])] = c["n_hi"]
    p = [r.randint(c["p_lo"], c["p_hi"]) for _ in range(c["B"])]
    return n, p


def _rows(c):
    """Logits rows of each request: (sizes, accepted lengths or None)."""
    r = random.Random(c["lens"])
    if c["op"] == PATH:
        n = [r.randint(1, c["n_max"]) for _ in range(c["B"])]
        n[r.randrange(c["B"])] = c["n_max"]
        return n, [r.randint(1, min(8, x)) for x in n]
    cut = sorted(r.randint(0, c["T"]) for _ in range(c["B"] - 1))
    return [b - a for a, b in zip([0] + cut, cut + [c["T"]])], None


def _fork_lens(c):
    """Slots held by each source row, and (source, length) of each fork."""
    r = random.Random(c["lens"])
    top = c["max_blocks"] * c["bs"] - c["room"] if c["max_blocks"] * c["bs"] > c["room"] else 1
    held = [r.randint(max(1, top // 2), top) for _ in range(c["sources"])]
    src = [r.randrange(c["sources"]) for _ in range(c["n"])]
    return held, src, [held[s] - r.randint(0, held[s] // 4) for s in src]


def _bytes(dtype):
    return 4 if dtype == "fp32" else 2


def _dtype(dtype):
    return torch.float32 if dtype == "fp32" else torch.bfloat16


def work(c):
    if c["op"] == ATTENTION:
        n, p = _lengths(c)
        e = _bytes(c["dtype"])
        seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, p))
        kv = sum(a + b for a, b in zip(n, p))
        return {"bytes": 2 * e * c["D"] * (sum(n) * c["Hq"] + kv * c["Hkv"]), "flops": 4 * c["D"] * c["Hq"] * seen}
    if c["op"] in (SCORES, PATH):
        n, acc = _rows(c)
        rows = sum(acc) if acc else sum(n)
        out = c["B"] * c["n_max"] if acc else rows
        return {"bytes": rows * c["V"] * _bytes(c["dtype"]) + out * (12 + 8 * c["k"]), "flops": 6 * rows * c["V"]}
    if c["op"] == FREE:
        return {"bytes": 4 * c["rows"] * c["max_blocks"] + 8 * c["n"] * c["max_blocks"], "flops": 0}
    row = 2 * c["layers"] * c["Hkv"] * c["D"] * _bytes(c["dtype"])  # one slot's K and V in every layer
    if c["op"] == FORK:
        _, _, lens = _fork_lens(c)
        return {"bytes": 2 * row * sum(x % c["bs"] for x in lens) + 8 * c["n"] * c["max_blocks"], "flops": 0}
    return {"bytes": 2 * row * c["bs"] * c["n"] + 8 * c["rows"] * c["max_blocks"] + 8 * c["blocks"], "flops": 0}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(n):
    off = [0]
    for x in n:
        off.append(off[-1] + x)
    return _ints(off)


def prepare(c, seed):
    g = _gen(seed)
    s = dict(c, kept={})
    if c["op"] == ATTENTION:
        n, p = _lengths(c)
        used = [(a + b + c["bs"] - 1) // c["bs"] for a, b in zip(n, p)]
        blocks, width, dt = sum(used) + 3, max(used), _dtype(c["dtype"])
        order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
        first = _offsets(used)[:-1]
        j = torch.arange(width, device=DEV, dtype=torch.int32)
        own_page = j[None] < _ints(used)[:, None]
        table = torch.where(own_page, order[(first[:, None] + j[None]).clamp(max=blocks - 1).long()], -1)
        kv = [torch.randn((blocks, c["Hkv"], c["bs"], c["D"]), generator=g, device=DEV, dtype=dt) for _ in range(2)]
        q = torch.randn((sum(n), c["Hq"], c["D"]), generator=g, device=DEV, dtype=dt)
        s.update(T=sum(n), n_top=max(n), p_top=max(p), blocks=blocks, width=width, table=table.contiguous(), k=kv[0], v=kv[1], q=q,
                 seq_off=_offsets(n), prefix=_ints(p), scale=1.0 / math.sqrt(c["D"]))
    elif c["op"] in (SCORES, PATH):
        n, acc = _rows(c)
        T = sum(n)
        # logits of variance 3 with one likely token a row, as the verifier's workloads have them
        x = torch.randn((T, c["V"]), generator=g, device=DEV) * math.sqrt(3.0)
        spike = torch.randint(0, c["V"], (T, 1), generator=g, device=DEV)
        x.scatter_add_(1, spike, torch.full((T, 1), 8.0, device=DEV))
        tau = 0.5 + torch.rand((c["B"],), generator=g, device=DEV)
        any_token = torch.randint(0, c["V"], (T,), generator=g, device=DEV)
        likely = torch.rand((T,), generator=g, device=DEV) < 0.7
        token = torch.where(likely, spike[:, 0], any_token).to(torch.int32)
        s.update(T=T, x=x.to(_dtype(c["dtype"])), tau=tau, off=_offsets(n), n_top=max(n))
        if acc is None:
            s.update(token=token)
        else:
            # an increasing path from the root of each tree, and the tokens emitted along it
            steps = torch.rand((c["B"], c["n_max"]), generator=g, device=DEV)
            steps[:, 0] = -1.0
            steps[torch.arange(c["n_max"], device=DEV)[None] >= _ints(n)[:, None]] = 2.0
            order = steps.argsort(1)
            a = _ints(acc)
            j = torch.arange(c["n_max"], device=DEV)[None]
            path = torch.where(j < a[:, None], order, 1 << 20).sort(1).values
            path = torch.where(j < a[:, None], path, -1).to(torch.int32)
            at = (s["off"][:-1, None] + path).clamp(min=0).long()
            s.update(path=path, accept=a, emitted=torch.where(path >= 0, token[at], -1))
    else:
        _prepare_pages(c, s, g)
    return s


def _prepare_pages(c, s, g):
    rows, mb, nb, bs = c["rows"], c["max_blocks"], c["blocks"], c["bs"]
    # table, pool and count lie in one buffer: a scheduler hands them over in one copy
    meta = torch.full((rows * mb + nb + 1,), -1, dtype=torch.int32, device=DEV)
    table, pool, count = meta[: rows * mb].view(rows, mb), meta[rows * mb:-1], meta[-1:]
    order = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(mb, device=DEV)
    if c["op"] == FORK:
        held, src, lens = _fork_lens(c)
        used = [(x + bs - 1) // bs for x in held]
        first = _offsets(used)[:-1]
        own_page = j[None] < _ints(used)[:, None]
        table[: c["sources"]] = torch.where(own_page, order[(first[:, None] + j[None]).clamp(max=nb - 1).long()], -1)
        taken = sum(used)
        s.update(src=_ints(src), dst=_ints([c["sources"] + i for i in range(c["n"])]), len=_ints(lens), room_of=_ints([c["room"]] * c["n"]))
    elif c["op"] == FREE:
        # the first rows hold pages of their own, the others share the first half of one of these and go on alone
        filled = j[None] < mb - mb // 4
        ids = order.view(rows, mb)
        table[:] = torch.where(filled, ids, -1)
        shared = torch.arange(rows, device=DEV) % c["sources"]
        half = (j[None] < mb // 2) & (torch.arange(rows, device=DEV)[:, None] >= c["sources"])
        table[:] = torch.where(half, ids[shared], table)
        gone = torch.randperm(rows, generator=g, device=DEV)[: c["n"]].to(torch.int32)
        s.update(gone=gone, keep=torch.zeros_like(gone))
        named = torch.zeros(nb, dtype=torch.bool, device=DEV)
        named[table[table >= 0].long()] = True
        rest = (~named).nonzero()[:, 0].to(torch.int32)
        pool[: rest.numel()] = rest
        count.fill_(rest.numel())
    else:
        live = min(nb // 2, rows * mb)
        live, moved = max(live, c["n"]), c["n"]
        low = torch.randperm(live, generator=g, device=DEV)
        high = live + torch.randperm(nb - live, generator=g, device=DEV)
        ids = torch.cat((low[moved:], high[:moved])).to(torch.int32)
        ids = ids[torch.randperm(live, generator=g, device=DEV)]
        rest = torch.cat((low[:moved], high[moved:])).to(torch.int32)
        table.view(-1)[:live] = ids
        pool[: rest.numel()] = rest
        count.fill_(rest.numel())
    if c["op"] == FORK:
        rest = order[taken:]
        pool[: rest.numel()] = rest
        count.fill_(rest.numel())
    s.update(meta=meta, start=meta.clone(), table=table, pool=pool, count=count)
    if c["op"] != FREE:
        cache = torch.randn((c["layers"], 2, nb, c["Hkv"], bs, c["D"]), generator=g, device=DEV, dtype=_dtype(c["dtype"]))
        s.update(cache=cache, k_ptrs=torch.tensor([cache[i, 0].data_ptr() for i in range(c["layers"])], dtype=torch.int64, device=DEV),
                 v_ptrs=torch.tensor([cache[i, 1].data_ptr() for i in range(c["layers"])], dtype=torch.int64, device=DEV))


def run(s):
    if s["op"] == ATTENTION:
        return _own_attention(s) if own else _plain_attention(s)
    if s["op"] == SCORES:
        return _own_scores(s) if own else _plain_scores(s["x"], s["token"], _request_of(s), s["tau"], s["k"])
    if s["op"] == PATH:
        return _own_path(s) if own else _plain_path(s)
    s["meta"].copy_(s["start"])
    if s["op"] == FORK:
        return _own_fork(s) if own else _plain_fork(s)
    if s["op"] == FREE:
        return _own_free(s) if own else _plain_free(s)
    return _own_compact(s) if own else _plain_compact(s)


# ------------------------------------------------------------ plain forms ----

def _request_of(s):
    off = s["seq_off"] if "seq_off" in s else s["off"]
    return torch.searchsorted(off[1:].contiguous(), torch.arange(s["T"], device=DEV, dtype=torch.int32), right=True)


def _plain_attention(s):
    """Scores of every (row, key) pair of the padded batch, a softmax over the
    keys that the row may see, and the product with the values."""
    B, Hkv, g, D, bs = s["B"], s["Hkv"], s["Hq"] // s["Hkv"], s["D"], s["bs"]
    b = _request_of(s)
    i = torch.arange(s["T"], device=DEV) - s["seq_off"][b]
    q = torch.zeros((B, s["n_top"], Hkv, g, D), device=DEV)
    q[b, i] = s["q"].float().view(-1, Hkv, g, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * s["n_top"], D)
    at = s["table"].clamp(min=0).long()

    def gather(cache):  # [B][Hkv][keys][D]
        return cache[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, s["width"] * bs, D).float()

    x = torch.matmul(q, gather(s["k"]).transpose(2, 3)).mul_(s["scale"])
    last = s["prefix"][:, None] + torch.arange(s["n_top"], device=DEV)[None]
    unseen = torch.arange(s["width"] * bs, device=DEV)[None, None] > last[:, :, None]
    x = x.view(B, Hkv, g, s["n_top"], s["width"] * bs)
    x.masked_fill_(unseen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    v = gather(s["v"])
    own_slot = torch.arange(s["width"] * bs, device=DEV)[None] < (s["prefix"] + s["seq_off"][1:] - s["seq_off"][:-1])[:, None]
    v.masked_fill_(~own_slot[:, None, :, None], 0.0)
    o = torch.matmul(x.view(B, Hkv, g * s["n_top"], -1), v).view(B, Hkv, g, s["n_top"], D) / total
    return o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, s["Hq"], D).to(s["q"].dtype)


def _order_key(x):
    """Whole numbers in the order of the floats (and -0 equal to +0)."""
    bits = (x + 0.0).view(torch.int32)
    return torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF)


def _plain_scores(x, token, request, tau, k):
    x, V = x.float(), x.shape[1]
    d = (x - x.amax(1, keepdim=True)) * tau[request][:, None]
    e = d.exp()
    total = e.sum(1)
    log_total = total.log()
    entropy = log_total - (e * d.clamp(min=-3e38)).sum(1) / total
    del e
    t = token.long()[:, None]
    logprob = d.gather(1, t)[:, 0] - log_total
    ids = torch.arange(V, device=DEV)[None]
    xt = x.gather(1, t)
    rank = ((x > xt) | ((x == xt) & (ids < t))).sum(1).to(torch.int32)
    key = _order_key(x).long() * (1 << 20) + (V - 1 - ids)
    top = key.topk(k, dim=1).indices if k else t[:, :0]
    return logprob, entropy, rank, top.to(torch.int32), d.gather(1, top) - log_total[:, None]


def _plain_path(s):
    B, m = s["path"].shape
    there = torch.arange(m, device=DEV)[None] < s["accept"][:, None]
    row = (s["off"][:-1, None] + s["path"])[there].long()
    b = torch.arange(B, device=DEV)[:, None].expand(B, m)[there]
    got = _plain_scores(s["x"][row], s["emitted"][there], b, s["tau"], s["k"])
    out = []
    for v in got:  # five results, laid out [B][n_max]
        whole = torch.full((B, m) + v.shape[1:], -1 if v.dtype == torch.int32 else math.nan, dtype=v.dtype, device=DEV)
        whole[there] = v
        out.append(whole)
    return tuple(out)


def _bits(cache):
    return cache.view(torch.int16 if cache.dtype == torch.bfloat16 else torch.int32)


def _plain_fork(s):
    bs, table = s["bs"], s["table"]
    j = torch.arange(s["max_blocks"], device=DEV)[None]
    full = (s["len"] // bs)[:, None]
    need = ((s["len"] + s["room_of"] + bs - 1) // bs)[:, None]
    source = table[s["src"].long()]
    fresh = (j >= full) & (j < need)
    nth = fresh.view(-1).cumsum(0).view(fresh.shape)
    page = s["pool"][(s["count"].long() - nth).clamp(min=0)]
    row = torch.where(j < full, source, torch.where(fresh, page, table[s["dst"].long()]))
    table[s["dst"].long()] = row
    s["count"].sub_(nth[-1, -1].to(torch.int32))
    tail = (s["len"] % bs > 0).nonzero()[:, 0]
    at = full[tail].long()
    old, new = source[tail].gather(1, at)[:, 0].long(), row[tail].gather(1, at)[:, 0].long()
    kept = torch.arange(bs, device=DEV)[None] < (s["len"] % bs)[tail][:, None]
    cache = s["cache"]
    cache[:, :, new] = torch.where(kept[None, None, :, None, :, None], cache[:, :, old], cache[:, :, new])
    return {"table": table, "pool": s["pool"], "count": s["count"], "cache": _bits(cache)}


def _plain_free(s):
    bs, table, nb = s["bs"], s["table"], s["blocks"]
    rows = s["gone"].long()
    j = torch.arange(s["max_blocks"], device=DEV)[None]
    mine = table[rows]
    dropped = (j >= ((s["keep"] + bs - 1) // bs)[:, None]) & (mine >= 0)
    table[rows] = torch.where(dropped, -1, mine)
    held = torch.zeros(nb + 1, dtype=torch.bool, device=DEV)
    held[torch.where(table >= 0, table, nb).view(-1).long()] = True
    ids = torch.where(dropped, mine, nb).view(-1).long()
    at = torch.arange(ids.numel(), device=DEV)
    first = torch.full((nb + 1,), ids.numel(), device=DEV).scatter_reduce(0, ids, at, "amin")
    released = dropped.view(-1) & ~held[ids] & (first[ids] == at)
    to = s["count"].long() + released.cumsum(0) - 1
    s["pool"][to[released]] = ids[released].to(torch.int32)
    s["count"].add_(released.sum().to(torch.int32))
    return {"table": table, "pool": s["pool"], "count": s["count"]}


def _plain_compact(s):
    table, nb, cache = s["table"], s["blocks"], s["cache"]
    ids = torch.arange(nb, device=DEV, dtype=torch.int32)
    live = torch.zeros(nb + 1, dtype=torch.bool, device=DEV)
    live[torch.where(table >= 0, table, nb).view(-1).long()] = True
    free = torch.zeros(nb + 1, dtype=torch.bool, device=DEV)
    free[torch.where(ids < s["count"], s["pool"], nb).long()] = True
    live, free = live[:nb], free[:nb]
    place = (live | free).cumsum(0) - 1
    n = live.sum()
    old, new = (live & (place >= n)).nonzero()[:, 0], (free & (place < n)).nonzero()[:, 0]
    cache[:, :, new] = cache[:, :, old]
    to = ids.clone()
    to[old] = new.to(torch.int32)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    rest = ((live | free) & (place >= n)).nonzero()[:, 0].flip(0).to(torch.int32)
    s["pool"][: rest.numel()] = rest
    return {"table": table, "pool": s["pool"], "count": s["count"], "map": to, "moved": (to != ids).sum(dtype=torch.int32).view(1), "cache": _bits(cache)}


# ------------------------------------------------------- the library's calls ----

def _kept(s, name, make):
    """Outputs and workspaces that a user's program keeps from call to call."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _own_attention(s):
    import tree_speculative_verification_spec_gb300 as S
    size = (s["B"], s["T"], s["n_top"], s["p_top"], s["Hq"], s["Hkv"], s["D"])
    ws = _kept(s, "ws", lambda: torch.empty(S.spec_prompt_workspace_size(*size), dtype=torch.uint8, device=DEV))
    out = _kept(s, "out", lambda: torch.empty_like(s["q"]))
    status = _kept(s, "status", lambda: torch.zeros(s["B"], dtype=torch.int32, device=DEV))
    S.spec_prompt_attention(s["q"], s["k"], s["v"], s["table"], s["width"], s["bs"], s["blocks"], s["prefix"], s["seq_off"], *size, s["scale"], out, ws, status)
    return out


def _score_outputs(s, shape):
    f, i = dict(device=DEV), dict(dtype=torch.int32, device=DEV)
    return (torch.empty(shape, **f), torch.empty(shape, **f), torch.empty(shape, **i), torch.empty(shape + (s["k"],), **i), torch.empty(shape + (s["k"],), **f))


def _own_scores(s):
    import tree_speculative_verification_spec_gb300 as S
    out = _kept(s, "out", lambda: _score_outputs(s, (s["T"],)))
    status = _kept(s, "status", lambda: torch.zeros(s["B"], dtype=torch.int32, device=DEV))
    S.spec_token_logprobs(s["x"], s["token"], s["off"], s["tau"], s["B"], s["T"], s["V"], s["k"], *out, status)
    return out


def _own_path(s):
    import tree_speculative_verification_spec_gb300 as S
    out = _kept(s, "out", lambda: _score_outputs(s, (s["B"], s["n_max"])))
    status = _kept(s, "status", lambda: torch.zeros(s["B"], dtype=torch.int32, device=DEV))
    S.spec_path_logprobs(s["x"], s["off"], s["path"], s["accept"], s["emitted"], s["tau"], s["B"], s["T"], s["n_max"], s["V"], s["k"], *out, status)
    return out


def _page_scratch(s, S, n):
    return _kept(s, "ws", lambda: torch.empty(S.spec_pages_workspace_size(s["rows"], s["max_blocks"], s["blocks"], n), dtype=torch.uint8, device=DEV))


def _own_fork(s):
    import tree_speculative_verification_spec_gb300 as S
    ws = _page_scratch(s, S, s["n"])
    status = _kept(s, "status", lambda: torch.zeros(s["n"], dtype=torch.int32, device=DEV))
    S.spec_pages_fork(s["k_ptrs"], s["v_ptrs"], s["layers"], s["table"], s["rows"], s["max_blocks"], s["bs"], s["blocks"], s["src"], s["dst"], s["len"], s["room_of"],
                      s["n"], s["Hkv"], s["D"], S.SPEC_F32 if s["dtype"] == "fp32" else S.SPEC_BF16, s["pool"], s["count"], ws, status)
    return {"table": s["table"], "pool": s["pool"], "count": s["count"], "cache": _bits(s["cache"])}


def _own_free(s):
    import tree_speculative_verification_spec_gb300 as S
    ws = _page_scratch(s, S, s["n"])
    status = _kept(s, "status", lambda: torch.zeros(s["n"], dtype=torch.int32, device=DEV))
    S.spec_pages_free(s["table"], s["rows"], s["max_blocks"], s["bs"], s["blocks"], s["gone"], s["keep"], s["n"], s["pool"], s["count"], ws, status)
    return {"table": s["table"], "pool": s["pool"], "count": s["count"]}


def _own_compact(s):
    import tree_speculative_verification_spec_gb300 as S
    ws = _page_scratch(s, S, 0)
    page_map = _kept(s, "map", lambda: torch.empty(s["blocks"], dtype=torch.int32, device=DEV))
    moved = _kept(s, "moved", lambda: torch.empty(1, dtype=torch.int32, device=DEV))
    status = _kept(s, "status", lambda: torch.zeros(1, dtype=torch.int32, device=DEV))
    S.spec_pages_compact(s["k_ptrs"], s["v_ptrs"], s["layers"], s["table"], s["rows"], s["max_blocks"], s["bs"], s["blocks"], s["Hkv"], s["D"],
                         S.SPEC_F32 if s["dtype"] == "fp32" else S.SPEC_BF16, s["pool"], s["count"], page_map, moved, ws, status)
    return {"table": s["table"], "pool": s["pool"], "count": s["count"], "map": page_map, "moved": moved, "cache": _bits(s["cache"])}


# ------------------------------------------------- definitions in 64 bits ----

def exact(c, seed):
    if c["op"] == ATTENTION:
        return _exact_attention(prepare(c, seed))
    if c["op"] in (SCORES, PATH):
        s = prepare(c, seed)
        if c["op"] == SCORES:
            return _exact_scores(s, list(range(s["T"])), s["token"].tolist(), _row_owner(s))
        path, emitted, off, acc = (s[k].tolist() for k in ("path", "emitted", "off", "accept"))
        entries = [(b, i) for b in range(c["B"]) for i in range(acc[b])]
        got = _exact_scores(s, [off[b] + path[b][i] for b, i in entries], [emitted[b][i] for b, i in entries], [b for b, _ in entries])
        at = torch.tensor([b * c["n_max"] + i for b, i in entries], device=DEV)
        out = []
        for v in got:
            if v is None:
                out.append(None)
                continue
            whole = torch.full((c["B"] * c["n_max"],) + v.shape[1:], math.nan, dtype=torch.float64, device=DEV)
            whole[at] = v
            out.append(whole.view((c["B"], c["n_max"]) + v.shape[1:]))
        return tuple(out)
    return None  # pages are copied and numbered, nothing is computed


def _row_owner(s):
    off = s["off"].tolist()
    return [b for b in range(s["B"]) for _ in range(off[b], off[b + 1])]


def _exact_scores(s, rows, tokens, owner):
    tau = s["tau"].double()
    lp, ent, top = [], [], []
    for a in range(0, len(rows), 256):
        r = torch.tensor(rows[a:a + 256], device=DEV)
        z = s["x"][r].double() * tau[torch.tensor(owner[a:a + 256], device=DEV)][:, None]
        norm = torch.logsumexp(z, 1)
        logp = z - norm[:, None]
        p = logp.exp()
        ent.append(-torch.where(p > 0, p * logp, 0.0).sum(1))
        lp.append(logp.gather(1, torch.tensor(tokens[a:a + 256], device=DEV)[:, None])[:, 0])
        top.append(logp.topk(s["k"], dim=1).values)
    return torch.cat(lp), torch.cat(ent), None, None, torch.cat(top)


def _exact_attention(s):
    Hkv, g, D, bs = s["Hkv"], s["Hq"] // s["Hkv"], s["D"], s["bs"]
    off, prefix = s["seq_off"].tolist(), s["prefix"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(s["B"]):
        n, P = off[b + 1] - off[b], prefix[b]
        ids = s["table"][b, : (P + n + bs - 1) // bs].long()
        for h in range(Hkv):
            k = s["k"][ids, h].reshape(-1, D)[: P + n].double()
            v = s["v"][ids, h].reshape(-1, D)[: P + n].double()
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                q = s["q"][off[b] + i: off[b] + i + m, h * g: (h + 1) * g].double()
                seen = P + i + m
                z = torch.einsum("mgd,kd->mgk", q, k[:seen]) * s["scale"]
                late = torch.arange(seen, device=DEV)[None] > (P + i + torch.arange(m, device=DEV))[:, None]
                w = torch.softmax(z.masked_fill(late[:, None], -math.inf), -1)
                out[off[b] + i: off[b] + i + m, h * g: (h + 1) * g] = torch.einsum("mgk,kd->mgd", w, v[:seen])
    return out
