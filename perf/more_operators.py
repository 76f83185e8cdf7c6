"""The operators between a projection and a bounded cache, as cases to measure:
head norms and rotary positions on the way into the paged cache, the attention
weight that cached slots gather, and the eviction of the light ones.

Each case runs either in its plain form (elementary torch operations in 32
bits) or, with `own` set, through the library's entry points."""
import math
import random

import torch

own = False

DEV = "cuda"
ROPE, WEIGHT, EVICT = "rope append", "attention weight", "evict"
ROWS, LAST, PATH = "every row", "last rows", "accepted path"  # whose attention counts


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # the trees of a batched verification step: positions are the prefix plus each node's depth
        rope("64 trees", 64, 8, 64, 0, 1024, 32, 8, 128, 16, "bf16", 11, pos="tree"),
        # one long document's first pass, large pages
        rope("prompt of 16384", 1, 16384, 16384, 0, 0, 32, 8, 128, 256, "bf16", 12),
        # prompts of an image and text: time, height and width have pairs of their own
        rope("image and text", 4, 1500, 2048, 0, 64, 64, 8, 128, 256, "bf16", 13, pos="image", axes=3),
        # the smallest model of the tests after evictions: fp32, neighbouring pairs, half of the head rotated, no norms
        rope("small fp32", 2, 1, 5, 0, 128, 4, 4, 64, 16, "fp32", 14, pos="far", rot=32, pairs=1, norms=False),
        # a batched step's accepted paths over ragged prefixes
        weight("64 accepted paths", 64, 8, 64, 256, 16384, 32, 8, 128, 16, "bf16", 21, rows=PATH),
        # one token of one long request, the decode step without a draft
        weight("one token", 1, 1, 1, 16384, 16384, 32, 8, 128, 16, "bf16", 22),
        # the last 32 tokens of four long prompts, wide groups: what a prompt's cache is cut by
        weight("last rows of prompts", 4, 512, 512, 8192, 8192, 64, 8, 128, 256, "bf16", 23, rows=LAST, window=32),
        # every token of one prompt
        weight("prompt of 8192", 1, 8192, 8192, 0, 0, 32, 8, 128, 256, "bf16", 24),
        # fp32, no grouping, odd lengths
        weight("small fp32 weight", 2, 7, 33, 0, 128, 4, 4, 64, 16, "fp32", 25),
        # four long prompts cut to a draft's cache in every layer
        evict("four prompts to 1024", 32, 4, 6000, 8192, 1024, 4, 64, 8, 128, 16, "bf16", 31),
        # a batch of short requests held to its budget, large pages
        evict("64 requests to 256", 2, 64, 200, 1024, 256, 4, 32, 8, 128, 256, "bf16", 32),
        # one layer's cache of one request, fp32
        evict("one row fp32", 1, 1, 700, 700, 129, 0, 17, 2, 64, 16, "fp32", 33),
    ]


def rope(name, B, n_lo, n_hi, p_lo, p_hi, Hq, Hkv, D, bs, dtype, seed, pos="slots", axes=1, rot=0, pairs=0, norms=True):
    return dict(name=name, op=ROPE, B=B, n_lo=n_lo, n_hi=n_hi, p_lo=p_lo, p_hi=p_hi, Hq=Hq, Hkv=Hkv, D=D, bs=bs, dtype=dtype, lens=seed, pos=pos,
                axes=axes, rot=rot or D, pairs=pairs, norms=norms)


def weight(name, B, n_lo, n_hi, p_lo, p_hi, Hq, Hkv, D, bs, dtype, seed, rows=ROWS, window=0):
    return dict(name=name, op=WEIGHT, B=B, n_lo=n_lo, n_hi=n_hi, p_lo=p_lo, p_hi=p_hi, Hq=Hq, Hkv=Hkv, D=D, bs=bs, dtype=dtype, lens=seed, rows=rows,
                window=window)


def evict(name, layers, N, len_lo, len_hi, keep, first, last, Hkv, D, bs, dtype, seed):
    return dict(name=name, op=EVICT, layers=layers, N=N, len_lo=len_lo, len_hi=len_hi, keep=keep, first=first, last=last, Hkv=Hkv, D=D, bs=bs,
                dtype=dtype, lens=seed)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 2, 64), (4, 4, 64), (6, 2, 64), (20, 4, 128), (5, 1, 64))


def draw(rng):
    op = rng.choice((ROPE, WEIGHT, EVICT))
    seed = rng.randrange(1 << 30)
    dtype, bs = rng.choice(("bf16", "bf16", "bf16", "fp32")), rng.choice((8, 16, 64, 256))
    if op == EVICT:
        layers, Hkv, D = rng.choice((1, 2, 7, 32)), rng.choice((1, 2, 8)), rng.choice((64, 128))
        N, top = _log(rng, 1, 64), _log(rng, 2, 40000)
        while layers * N * Hkv * D * top * _bytes(dtype) > 32 * 4 * 8 * 128 * 8192 * 2:
            N, top = (N + 1) // 2, top * 2 // 3
        keep = _log(rng, 1, max(1, top // 4))
        while layers * N * Hkv * D * keep * _bytes(dtype) > 32 * 4 * 8 * 128 * 1024 * 2:
            keep = keep // 2
        c = evict("", layers, N, rng.choice((top, (top + 1) // 2, 1)), top, keep, rng.choice((0, 4, 64)), rng.choice((0, 1, keep // 2, 32)), Hkv, D, bs,
                  dtype, seed)
        del c["name"]
        return c
    Hq, Hkv, D = rng.choice(HEADS)
    if op == ROPE:
        pos = rng.choice(("slots", "tree", "image", "far"))
        n_hi = _log(rng, 1, 1024 if pos == "tree" else 12000)
        n_hi = min(n_hi, 16384 * 48 * 128 // ((Hq + 2 * Hkv) * D * _bytes(dtype) // 2))
        B = _log(rng, 1, max(1, min(64, 16384 * 48 * 128 // (n_hi * (Hq + 2 * Hkv) * D * _bytes(dtype) // 2))))
        rot = rng.choice((D, D, D // 2, 6))
        c = rope("", B, rng.choice((1, n_hi, (n_hi + 1) // 2)), n_hi, 0, rng.choice((0, 700)), Hq, Hkv, D, bs, dtype, seed, pos,
                 rng.choice((2, 3)) if pos == "image" else 1, rot, rng.randrange(2), rng.random() < 0.7)
    else:
        rows = rng.choice((ROWS, LAST, PATH))
        n_hi, p_hi = _log(rng, 1, {ROWS: 6000, LAST: 6000, PATH: 64}[rows]), rng.choice((0, _log(rng, 1, 20000)))
        window = _log(rng, 1, 128) if rows == LAST else 0
        if dtype == "fp32":
            n_hi, p_hi = 1 + n_hi % 1000, 1 + p_hi % 4000
        B = _log(rng, 1, 64)
        while rows == ROWS and Hq * n_hi * (n_hi + p_hi) > 2 ** 30:
            n_hi = n_hi * 2 // 3
        most = {ROWS: n_hi, LAST: min(n_hi, window), PATH: min(8, n_hi)}[rows]
        while B > 1 and (B * Hq * most * (n_hi + p_hi) > 2 ** 30 or B * (n_hi + p_hi) * Hkv > 64 * 16384 * 8):
            B = (B + 1) // 2
        c = weight("", B, rng.choice((0, 1, n_hi, (n_hi + 1) // 2)), n_hi, rng.choice((0, p_hi // 2, p_hi)), p_hi, Hq, Hkv, D, bs, dtype, seed, rows, window)
    del c["name"]
    return c


# ------------------------------------------------------- sizes of one case ----

def _lengths(c):
    """New tokens (or tree nodes), cached tokens and accepted nodes of each request."""
    r = random.Random(c["lens"])
    n = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    n[r.randrange(c["B"])] = c["n_hi"]
    p = [r.randint(c["p_lo"], c["p_hi"]) for _ in range(c["B"])]
    return n, p, [r.randint(min(1, x), min(8, x)) for x in n]


def _counted(c):
    """For each request: the rows whose attention counts, and the slot of its first token."""
    n, p, acc = _lengths(c)
    m = acc if c["rows"] == PATH else n
    first = [max(0, x - c["window"]) if c["rows"] == LAST else 0 for x in m]
    return m, p, first


def _held(c):
    r = random.Random(c["lens"])
    length = [r.randint(min(c["len_lo"], c["len_hi"]), c["len_hi"]) for _ in range(c["N"])]
    length[r.randrange(c["N"])] = c["len_hi"]
    return length


def _bytes(dtype):
    return 4 if dtype == "fp32" else 2


def _dtype(dtype):
    return torch.float32 if dtype == "fp32" else torch.bfloat16


def work(c):
    e = _bytes(c["dtype"])
    if c["op"] == ROPE:
        n, _, _ = _lengths(c)
        heads = sum(n) * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * e * sum(n) * (c["Hq"] + 2 * c["Hkv"]) * c["D"], "flops": heads * (7 if c["norms"] else 3)}
    if c["op"] == WEIGHT:
        m, p, first = _counted(c)
        slots, rows = sum(a + b for a, b in zip(m, p)), sum(a - f for a, f in zip(m, first))
        seen = sum((a - f) * b + (a * (a + 1) - f * (f + 1)) // 2 for a, b, f in zip(m, p, first))
        return {"bytes": e * c["D"] * (slots * c["Hkv"] + rows * c["Hq"]) + 4 * c["Hkv"] * (slots + sum(p)), "flops": (2 * c["D"] + 4) * c["Hq"] * seen}
    length = _held(c)
    kept = sum(min(c["keep"], x) for x in length)
    unit = c["layers"] * c["Hkv"]
    return {"bytes": unit * (4 * sum(length) + kept * (4 * c["D"] * e + 8)), "flops": 0}


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


def _table(g, used, spare, width):
    """Rows of shuffled pages, -1 behind each row's own."""
    blocks = sum(used) + spare
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    first = _offsets(used)[:-1]
    j = torch.arange(width, device=DEV, dtype=torch.int32)
    return torch.where(j[None] < _ints(used)[:, None], order[(first[:, None] + j[None]).clamp(max=blocks - 1).long()], -1).contiguous(), blocks


def prepare(c, seed):
    g = _gen(seed)
    s = dict(c, kept={})
    if c["op"] == EVICT:
        _prepare_evict(c, s, g)
        return s
    n, p, acc = _lengths(c)
    used = [(a + b + c["bs"] - 1) // c["bs"] for a, b in zip(n, p)]
    width, dt, T = max(max(used), 1), _dtype(c["dtype"]), sum(n)
    table, blocks = _table(g, used, 3, width)
    s.update(T=T, n_top=max(n), p_top=max(p), blocks=blocks, width=width, table=table, seq_off=_offsets(n), prefix=_ints(p))
    cache = (blocks, c["Hkv"], c["bs"], c["D"])
    if c["op"] == ROPE:
        x = torch.randn((T, c["Hq"] + 2 * c["Hkv"], c["D"]), generator=g, device=DEV)
        pairs = c["rot"] // 2
        # frequencies of base 500000 as long-context models have them, one axis after another over the pairs
        freq = 500000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) * 2 / c["rot"])
        axis = torch.arange(pairs, device=DEV, dtype=torch.int32) * c["axes"] // pairs
        pos, base = _positions(c, n, p, T)
        norm = [(1.0 + 0.2 * torch.randn(c["D"], generator=g, device=DEV)).to(dt) if c["norms"] else None for _ in range(2)]
        s.update(qkv=(x * 1.5).to(dt), freq=freq.float(), axis=axis if c["axes"] > 1 else None, positions=pos, base=base, q_norm=norm[0], k_norm=norm[1],
                 eps=1e-6, k=torch.zeros(cache, device=DEV, dtype=dt), v=torch.zeros(cache, device=DEV, dtype=dt))
        return s
    q = torch.randn((T, c["Hq"], c["D"]), generator=g, device=DEV)
    k = torch.randn(cache, generator=g, device=DEV, dtype=dt)
    before = torch.rand((c["B"], c["Hkv"], width * c["bs"]), generator=g, device=DEV).pow_(4)
    s.update(q=(q * 1.5).to(dt), k=k, before=before, scale=1.0 / math.sqrt(c["D"]), decay=0.9375, stride=width * c["bs"], path=None, accept=None)
    if c["rows"] == PATH:
        # an increasing path from the root of each tree
        steps = torch.rand((c["B"], s["n_top"]), generator=g, device=DEV)
        steps[:, 0] = -1.0
        steps[torch.arange(s["n_top"], device=DEV)[None] >= _ints(n)[:, None]] = 2.0
        a, j = _ints(acc), torch.arange(s["n_top"], device=DEV)[None]
        path = torch.where(j < a[:, None], steps.argsort(1), 1 << 20).sort(1).values
        s.update(path=torch.where(j < a[:, None], path, -1).to(torch.int32), accept=a)
    return s


def _positions(c, n, p, T):
    """Offsets [axes][T] (None: the row's index) and bases [B] (None: the prefix)."""
    r = random.Random(c["lens"] + 1)
    if c["pos"] == "slots":
        return None, None
    if c["pos"] == "far":  # slots were given up: the text is much longer than the cache
        return None, _ints([x + r.randint(100000, 1000000) for x in p])
    if c["pos"] == "tree":
        depth = []
        for x in n:
            own_depth = [0]
            for i in range(1, x):
                own_depth.append(own_depth[r.randint(max(0, i - 8), i - 1)] + 1)
            depth += own_depth[:x]
        return _ints([depth]), None
    out = [[] for _ in range(c["axes"])]  # some text, an image of rows and columns, text again
    for x in n:
        head, side = min(x, r.randint(0, 40)), max(1, math.isqrt(x * 3 // 4))
        image = min(x - head, side * side)
        for a in range(c["axes"]):
            at = list(range(head))
            at += [head + (0, i // side, i % side)[a + 3 - c["axes"]] for i in range(image)]
            out[a] += at + [head + side + i for i in range(x - head - image)]
    return _ints(out), _ints([r.randint(0, 3000) for _ in p])


def _prepare_evict(c, s, g):
    length = _held(c)
    bs, N, dt = c["bs"], c["N"], _dtype(c["dtype"])
    used = [(x + bs - 1) // bs for x in length]
    room = (min(c["keep"], max(length)) + bs - 1) // bs
    width = max(max(used), room)
    # rows 0 .. N-1 hold the requests, rows N .. 2N-1 have pages for what is kept
    table, blocks = _table(g, used + [room] * N, 2, width)
    # weights span many sizes; a short mantissa makes some equal, and slots that nothing looked at weigh nothing
    w = torch.randn((c["layers"], 2 * N, c["Hkv"], width * bs), generator=g, device=DEV).mul_(2.0).exp_().bfloat16().float()
    w[torch.rand(w.shape, generator=g, device=DEV) < 0.1] = 0.0
    cache = torch.empty((c["layers"], 2, blocks, c["Hkv"], bs, c["D"]), device=DEV, dtype=dt)
    for layer in cache:
        layer.copy_(torch.randn(layer.shape, generator=g, device=DEV, dtype=dt))
    s.update(table=table, width=width, blocks=blocks, weight=w, stride=width * bs, cache=cache, src=_ints(list(range(N))),
             dst=_ints(list(range(N, 2 * N))), length=_ints(length), budget=_ints([c["keep"]] * N), lengths=length,
             k_ptrs=torch.tensor([x[0].data_ptr() for x in cache], dtype=torch.int64, device=DEV),
             v_ptrs=torch.tensor([x[1].data_ptr() for x in cache], dtype=torch.int64, device=DEV))


def run(s):
    if s["op"] == ROPE:
        return _own_rope(s) if own else _plain_rope(s)
    if s["op"] == WEIGHT:
        return _own_weight(s) if own else _plain_weight(s)
    return _own_evict(s) if own else _plain_evict(s)


# ------------------------------------------------------------ plain forms ----

def _request_of(s):
    return torch.searchsorted(s["seq_off"][1:].contiguous(), torch.arange(s["T"], device=DEV, dtype=torch.int32), right=True)


def _plain_rope(s):
    D, Hq, Hkv, rot, bs = s["D"], s["Hq"], s["Hkv"], s["rot"], s["bs"]
    b = _request_of(s)
    u = torch.arange(s["T"], device=DEV) - s["seq_off"][b]
    base = (s["prefix"] if s["base"] is None else s["base"])[b]
    pos = base[None] + (u[None] if s["positions"] is None else s["positions"])
    if s["axis"] is not None:
        pos = pos[s["axis"].long()]
    angle = pos.double().t() * s["freq"].double()  # [T][pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x, norm):
        x = x.float()
        if norm is not None:
            x = x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * norm.float()
        lo, hi = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["pairs"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        both = (lo * cos - hi * sin, hi * cos + lo * sin)
        turned = torch.stack(both, -1).flatten(-2) if s["pairs"] else torch.cat(both, -1)
        return torch.cat((turned, x[..., rot:]), -1).to(s["qkv"].dtype)

    q = turn(s["qkv"][:, :Hq], s["q_norm"])
    slot = s["prefix"][b] + u
    page = s["table"][b, slot // bs].long()
    s["k"][page, :, slot % bs] = turn(s["qkv"][:, Hq:Hq + Hkv], s["k_norm"])
    s["v"][page, :, slot % bs] = s["qkv"][:, Hq + Hkv:]
    return q, s["k"], s["v"]


def _plain_weight(s):
    """Softmax weights of every counted row of the padded batch, summed over the
    rows and the heads of a group."""
    B, Hkv, g, D, bs = s["B"], s["Hkv"], s["Hq"] // s["Hkv"], s["D"], s["bs"]
    n = s["seq_off"][1:] - s["seq_off"][:-1]
    count = s["accept"] if s["path"] is not None else n
    first = (count - s["window"]).clamp(min=0) if s["rows"] == LAST else torch.zeros_like(count)
    most = {ROWS: s["n_top"], LAST: min(s["n_top"], s["window"]), PATH: min(8, s["n_top"])}[s["rows"]]
    i = first[:, None] + torch.arange(most, device=DEV)[None]  # the row's index in its request
    there = i < count[:, None]
    at = s["path"][:, :most].clamp(min=0) if s["path"] is not None else i
    row = (s["seq_off"][:-1, None] + at).clamp(max=max(s["T"] - 1, 0)).long()
    q = s["q"][row].float().view(B, most, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * most, D)
    keys = s["k"][s["table"].clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(B, Hkv, s["width"] * bs, D).float()
    x = torch.matmul(q, keys.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, g, most, -1)
    slot = torch.arange(s["width"] * bs, device=DEV)
    unseen = (slot[None, None] > (s["prefix"][:, None] + i)[:, :, None]) | ~there[:, :, None]
    x.masked_fill_(unseen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    x.div_(x.sum(-1, keepdim=True).clamp(min=1e-30))
    added = x.sum((2, 3))
    old = torch.where(slot[None] < s["prefix"][:, None], 0.0, 1.0).bool()[:, None]
    total = torch.where(old, 0.0, s["decay"] * s["before"]) + added
    held = slot[None] < (s["prefix"] + count)[:, None]
    return torch.where(held[:, None], total, 0.0)


def _order_key(x):
    """Whole numbers in the order of the floats (and -0 equal to +0)."""
    bits = (x + 0.0).view(torch.int32)
    return torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF)


def _plain_evict(s):
    layers, Hkv, bs, N = s["layers"], s["Hkv"], s["bs"], s["N"]
    most = s["keep"]
    slots = torch.full((layers, N, Hkv, most), -1, dtype=torch.int32, device=DEV)
    weight, cache = s["weight"], s["cache"]
    l, h = torch.arange(layers, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    for i, length in enumerate(s["lengths"]):
        kept = min(most, length)
        first = min(s["first"], kept)
        last = min(s["last"], kept - first)
        w = weight[:, i, :, first:length - last]
        key = _order_key(w).long() * (1 << 20) + ((1 << 20) - 1 - torch.arange(w.shape[2], device=DEV))
        heavy = key.topk(kept - first - last, dim=2).indices.sort(2).values + first
        ends = [torch.arange(a, b, device=DEV).expand(layers, Hkv, -1) for a, b in ((0, first), (length - last, length))]
        old = torch.cat((ends[0], heavy, ends[1]), 2)
        slots[:, i, :, :kept] = old.to(torch.int32)
        new = torch.arange(kept, device=DEV)
        page_old, page_new = s["table"][i][old // bs].long(), s["table"][N + i][new // bs].long()
        for kv in range(2):
            cache[l, kv, page_new[None, None], h, (new % bs)[None, None]] = cache[l, kv, page_old, h, old % bs]
        weight[:, N + i, :, :kept] = weight[:, i].gather(2, old)
    return {"slots": slots, "new_len": s["length"].clamp(max=most), "weight": weight, "cache": _bits(cache)}


def _bits(cache):
    return cache.view(torch.int16 if cache.dtype == torch.bfloat16 else torch.int32)


# ------------------------------------------------------- the library's calls ----

def _kept(s, name, make):
    """Outputs and workspaces that a user's program keeps from call to call."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _status(s, n):
    return _kept(s, "status", lambda: torch.zeros(n, dtype=torch.int32, device=DEV))


def _own_rope(s):
    import tree_speculative_verification_spec_gb300 as S
    q = _kept(s, "q", lambda: torch.empty((s["T"], s["Hq"], s["D"]), dtype=s["qkv"].dtype, device=DEV))
    S.spec_rope_append(s["qkv"], s["q_norm"], s["k_norm"], s["eps"], s["freq"], s["axis"], s["rot"], s["pairs"], s["base"], s["positions"], s["axes"], q,
                       s["k"], s["v"], s["table"], s["width"], s["bs"], s["blocks"], s["prefix"], s["seq_off"], s["B"], s["T"], s["n_top"], s["Hq"], s["Hkv"],
                       s["D"], _status(s, s["B"]))
    return q, s["k"], s["v"]


def _own_weight(s):
    import tree_speculative_verification_spec_gb300 as S
    size = (s["B"], s["T"], s["n_top"], s["p_top"], s["Hq"], s["Hkv"], s["D"])
    ws = _kept(s, "ws", lambda: torch.empty(S.spec_weight_workspace_size(*size), dtype=torch.uint8, device=DEV))
    out = _kept(s, "out", lambda: torch.zeros_like(s["before"]))
    S.spec_attention_weight(s["q"], s["k"], s["table"], s["width"], s["bs"], s["blocks"], s["prefix"], s["seq_off"], s["path"], s["accept"], s["window"], *size,
                            s["scale"], s["decay"], s["before"], out, s["stride"], ws, _status(s, s["B"]))
    return out


def _own_evict(s):
    import tree_speculative_verification_spec_gb300 as S
    slots = _kept(s, "slots", lambda: torch.empty((s["layers"], s["N"], s["Hkv"], s["keep"]), dtype=torch.int32, device=DEV))
    new_len = _kept(s, "new_len", lambda: torch.empty(s["N"], dtype=torch.int32, device=DEV))
    S.spec_kv_evict(s["k_ptrs"], s["v_ptrs"], s["layers"], s["table"], 2 * s["N"], s["width"], s["bs"], s["blocks"], s["src"], s["dst"], s["length"],
                    s["budget"], s["N"], s["keep"], s["first"], s["last"], s["weight"], s["stride"], s["Hkv"], s["D"],
                    S.SPEC_F32 if s["dtype"] == "fp32" else S.SPEC_BF16, slots, new_len, _status(s, s["N"]))
    return {"slots": slots, "new_len": new_len, "weight": s["weight"], "cache": _bits(s["cache"])}


# ------------------------------------------------- definitions in 64 bits ----

def exact(c, seed):
    if c["op"] == EVICT:
        return None  # weights are compared and rows are copied, nothing is computed
    s = prepare(c, seed)
    return _exact_rope(s) if c["op"] == ROPE else _exact_weight(s)


def _exact_rope(s):
    """Pairs as complex numbers, turned by exp(i position frequency)."""
    Hq, Hkv, rot, bs = s["Hq"], s["Hkv"], s["rot"], s["bs"]
    off, prefix = s["seq_off"].tolist(), s["prefix"].tolist()
    base = prefix if s["base"] is None else s["base"].tolist()
    axis = [0] * (rot // 2) if s["axis"] is None else s["axis"].tolist()
    q = torch.empty((s["T"], Hq, s["D"]), dtype=torch.float64, device=DEV)
    k, v = s["k"].double(), s["v"].double()
    first = torch.arange(rot // 2, device=DEV) * (2 if s["pairs"] else 1)
    second = first + (1 if s["pairs"] else rot // 2)

    def head(x, norm, turn):
        x = x.double()
        if norm is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + s["eps"]) * norm.double()
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    for b in range(s["B"]):
        for at in range(off[b], off[b + 1], 4096):
            end = min(at + 4096, off[b + 1])
            u = torch.arange(at - off[b], end - off[b], device=DEV)
            rows = [(u if s["positions"] is None else s["positions"][a, at:end].long()) + base[b] for a in range(s["axes"])]
            place = torch.stack([rows[a] for a in axis], 1).double()
            turn = torch.polar(torch.ones_like(place), place * s["freq"].double())
            q[at:end] = head(s["qkv"][at:end, :Hq], s["q_norm"], turn)
            slot = prefix[b] + u
            page = s["table"][b][slot // bs].long()
            k[page, :, slot % bs] = head(s["qkv"][at:end, Hq:Hq + Hkv], s["k_norm"], turn)
            v[page, :, slot % bs] = s["qkv"][at:end, Hq + Hkv:].double()
    return q, k, v


def _exact_weight(s):
    Hkv, g, D, bs = s["Hkv"], s["Hq"] // s["Hkv"], s["D"], s["bs"]
    off, prefix = s["seq_off"].tolist(), s["prefix"].tolist()
    m, _, first = _counted(s)
    out = torch.zeros(s["before"].shape, dtype=torch.float64, device=DEV)
    for b in range(s["B"]):
        P, end = prefix[b], prefix[b] + m[b]
        ids = s["table"][b, : (end + bs - 1) // bs].long()
        for h in range(Hkv):
            out[b, h, :P] = s["decay"] * s["before"][b, h, :P].double()
            k = s["k"][ids, h].reshape(-1, D)[:end].double()
            for i in range(first[b], m[b], 1024):
                j = torch.arange(i, min(i + 1024, m[b]), device=DEV)
                row = off[b] + (j if s["path"] is None else s["path"][b, j].long())
                seen = P + min(i + 1024, m[b])
                z = torch.einsum("mgd,kd->mgk", s["q"][row, h * g:(h + 1) * g].double(), k[:seen]) * s["scale"]
                late = torch.arange(seen, device=DEV)[None] > (P + j)[:, None]
                out[b, h, :seen] += torch.softmax(z.masked_fill(late[:, None], -math.inf), -1).sum((0, 1))
    return out
