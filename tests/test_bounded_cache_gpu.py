"""Norms, rotation and append; gathered attention weight; eviction: against
plain implementations in 64 bits, at the sizes, masks and bad arguments where
they can go wrong."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from bounded_cache import ints, keep_reference, offsets, rope_reference, table_of, weight_reference
from request_life import paged_batch

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


# ------------------------------------------------------------- rope append ----

class Rope:
    """One call's inputs; everything that must stay holds 7."""

    def __init__(self, seed, lens, prefix, Hq, Hkv, D, bs, dtype, rot=None, pairing=0, axes=1, norms=(True, True), pos=None, base=None, gap=0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.prefix, self.Hq, self.Hkv, self.D, self.bs, self.dtype = lens, prefix, Hq, Hkv, D, bs, dtype
        self.rot, self.pairing, self.axes = D if rot is None else rot, pairing, axes
        self.T = sum(lens) + extra
        wide = Hq + 2 * Hkv
        self.buffer = torch.randn((self.T, wide * D + gap), generator=g).mul(1.7).to(dtype).cuda()
        self.qkv = self.buffer[:, :wide * D]
        self.norm = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() if n else None for n in norms]
        self.freq = (10000.0 ** (-torch.arange(0, self.rot, 2, dtype=torch.float64) / max(self.rot, 1))).float().cuda() if self.rot else None
        self.axis = (torch.randint(0, axes, (self.rot // 2,), generator=g).to(torch.int32).cuda()) if axes > 1 else None
        self.pos = None if pos is None else pos.to(torch.int32).cuda()
        self.base = None if base is None else ints(base)
        self.table, self.nb = table_of(seed, [p + n for p, n in zip(prefix, lens)], bs)
        self.off = offsets(lens)
        self.status = ints([0] * len(lens))

    def call(self, n_max=None, status=None, stream=None, outs=None):
        q, k, v = outs or (torch.full((self.T, self.Hq, self.D), 7.0, dtype=self.dtype, device="cuda"),
                           *(torch.full((self.nb, self.Hkv, self.bs, self.D), 7.0, dtype=self.dtype, device="cuda") for _ in range(2)))
        S.spec_rope_append(self.qkv, *self.norm, 1e-5, self.freq, self.axis, self.rot, self.pairing, self.base, self.pos, self.axes, q, k, v, self.table,
                           self.table.shape[1], self.bs, self.nb, ints(self.prefix), self.off, len(self.lens), self.T,
                           max(self.lens) if n_max is None else n_max, self.Hq, self.Hkv, self.D, self.status if status is None else status, stream)
        return q, k, v

    def check(self, got, skip_rows=()):
        q, k, v = got
        first = self.off.tolist()
        where = []  # (row, request, index)
        for b, n in enumerate(self.lens):
            where += [(first[b] + u, b, u) for u in range(n) if first[b] + u not in skip_rows]
        rows = torch.tensor([w[0] for w in where], device="cuda", dtype=torch.long)
        base = [0 if self.base is None else int(self.base[b]) for b in range(len(self.lens))]
        place = torch.zeros((len(where), self.rot // 2), dtype=torch.float64, device="cuda")
        u = torch.tensor([w[2] for w in where], device="cuda", dtype=torch.long)
        start = torch.tensor([self.prefix[w[1]] if self.base is None else base[w[1]] for w in where], device="cuda", dtype=torch.long)
        for i in range(self.rot // 2):
            ax = 0 if self.axis is None else min(int(self.axis[i]), self.axes - 1)
            place[:, i] = (start + (u if self.pos is None else self.pos[ax][rows].long())).double()
        x = self.qkv.reshape(self.T, -1, self.D)[rows]
        ref, tol = rope_reference(x, self.Hq, self.Hkv, self.rot, self.pairing, self.freq, place, *self.norm, 1e-5)
        slot = torch.tensor([self.prefix[w[1]] + w[2] for w in where], device="cuda", dtype=torch.long)
        owner = torch.tensor([w[1] for w in where], device="cuda", dtype=torch.long)
        page = self.table[owner, slot // self.bs].long()
        for part, want, t in ((q[rows], ref[:, :self.Hq], tol[:, :self.Hq]), (k[page, :, slot % self.bs], ref[:, self.Hq:], tol[:, self.Hq:])):
            worst = ((part.double() - want).abs() - t).max() if part.numel() else 0.0
            assert worst <= 0, float(worst)
        assert torch.equal(v[page, :, slot % self.bs], x[:, self.Hq + self.Hkv:])
        # nothing else changed
        rest = torch.ones(self.T, dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert (q[rest] == 7.0).all()
        for c in (k, v):
            mark = torch.ones(c.shape[:3], dtype=torch.bool, device="cuda")
            mark[page, :, slot % self.bs] = False
            assert (c[mark] == 7.0).all()


@DTYPES
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (4, 4, 64), (5, 1, 64), (20, 4, 128), (3, 3, 128), (1, 1, 64)])
@pytest.mark.parametrize("pairing", [S.SPEC_ROPE_HALVES, S.SPEC_ROPE_NEIGHBOURS], ids=["halves", "neighbours"])
def test_rope_heads_and_pairs(Hq, Hkv, D, pairing, dtype):
    r = Rope(3, [7, 0, 1, 33], [0, 5, 130, 15], Hq, Hkv, D, 16, dtype, pairing=pairing, extra=3)
    r.check(r.call())
    assert r.status.tolist() == [0] * 4


@DTYPES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot", [0, 2, 6, 16, 30, 32, 62, 64])
@pytest.mark.parametrize("pairing", [0, 1], ids=["halves", "neighbours"])
def test_rope_part_of_a_head(rot, pairing, D, dtype):
    r = Rope(5, [5, 9], [3, 40], 6, 2, D, 8, dtype, rot=rot, pairing=pairing, norms=(True, False))
    r.check(r.call())
    r = Rope(6, [5, 9], [3, 40], 6, 2, D, 8, dtype, rot=rot, pairing=pairing, norms=(False, rot % 4 == 0))
    r.check(r.call())


@DTYPES
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_rope_axes(axes, dtype):
    pos = torch.randint(0, 4000, (axes, 45), generator=torch.Generator().manual_seed(axes))
    r = Rope(7, [20, 25], [0, 700], 8, 2, 128, 256, dtype, axes=axes, pos=pos, base=[11, 0], pairing=axes % 2)
    r.check(r.call())
    assert r.status.tolist() == [0, 0]


@DTYPES
def test_rope_far_positions_and_tree_depths(dtype):
    depth = torch.tensor([[0, 1, 1, 2, 3, 0, 1, 2, 2, 2]])
    r = Rope(9, [5, 5], [64, 2], 8, 2, 128, 16, dtype, pos=depth, base=[(1 << 24) - 4, 1000003])
    r.check(r.call())
    assert r.status.tolist() == [0, 0]
    r = Rope(9, [5, 5], [64, 2], 8, 2, 128, 16, dtype, pos=depth)  # behind the prefix
    r.check(r.call())


@DTYPES
def test_rope_many_tokens_and_a_wider_projection(dtype):
    """Four tokens a CTA; rows that lie apart; more requests than a CTA has threads."""
    r = Rope(11, [3000, 0, 1, 777], [0, 9, 333, 16], 8, 2, 64, 64, dtype, gap=32, extra=5)
    r.check(r.call())
    lens = [(i * 7) % 5 for i in range(700)]
    r = Rope(12, lens, [(i * 13) % 40 for i in range(700)], 4, 2, 64, 8, dtype, extra=1)
    r.check(r.call())
    assert not r.status.any()


def test_rope_bad_requests_are_left_alone():
    ok = dict(Hq=8, Hkv=2, D=64, bs=16, dtype=torch.bfloat16)

    def run(change):
        r = Rope(13, [6, 6, 6], [0, 20, 4], **ok)
        change(r)
        got = r.call(n_max=6)
        return r, got, r.status.tolist()

    def page(r):
        r.table[1, 1] = r.nb
    r, got, st = run(page)
    assert st == [0, S.SPEC_DEV_BAD_BLOCK, 0]
    r.check(got, skip_rows=range(6, 12))

    def prefix(r):
        r.prefix[1] = r.table.shape[1] * 16 - 5
    r, got, st = run(prefix)
    assert st == [0, S.SPEC_DEV_CAPACITY, 0]
    r.check(got, skip_rows=range(6, 12))

    def negative(r):
        r.prefix[2] = -1
    r, got, st = run(negative)
    assert st == [0, 0, S.SPEC_DEV_CAPACITY]
    r.check(got, skip_rows=range(12, 18))

    r = Rope(13, [6, 9, 6], [0, 20, 4], **ok)
    got = r.call(n_max=8)
    assert r.status.tolist() == [0, S.SPEC_DEV_BAD_TREE, 0]
    r.check(got, skip_rows=range(6, 15))

    # rows behind T
    r = Rope(13, [6, 6, 6], [0, 20, 4], **ok)
    r.T = 17
    q = torch.full((18, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.full((r.nb, 2, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    r.call(outs=(q, k, v))
    assert r.status.tolist() == [0, 0, S.SPEC_DEV_BAD_TREE] and (q[12:] == 7.0).all()


def test_rope_bad_positions_leave_their_rows_alone():
    pos = torch.arange(12)[None].repeat(2, 1)
    pos[1, 3], pos[0, 7], pos[1, 9] = -30, (1 << 24), (1 << 31) - 1
    r = Rope(15, [6, 6], [0, 20], 8, 2, 64, 16, torch.bfloat16, axes=2, pos=pos, base=[5, 39])
    r.axis[:2] = ints([0, 1])
    got = r.call()
    assert r.status.tolist() == [S.SPEC_DEV_BAD_POSITION] * 2
    r.check(got, skip_rows=(3, 7, 9))
    # a pair's axis that does not exist stops every row
    r = Rope(15, [6, 6], [0, 20], 8, 2, 64, 16, torch.bfloat16, axes=2, pos=torch.zeros((2, 12)))
    r.axis[5] = 2
    got = r.call()
    assert r.status.tolist() == [S.SPEC_DEV_BAD_POSITION] * 2
    r.check(got, skip_rows=range(12))


def test_rope_incoming_status_is_kept_and_not_read():
    r = Rope(17, [6, 6], [0, 20], 8, 2, 64, 16, torch.float32)
    r.status = ints([S.SPEC_DEV_TIMEOUT, 0])
    r.check(r.call())
    assert r.status.tolist() == [S.SPEC_DEV_TIMEOUT, 0]


def test_rope_on_a_side_stream_and_in_a_graph():
    r = Rope(19, [40, 3], [0, 20], 8, 2, 128, 16, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = tuple(torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in ((43, 8, 128), (r.nb, 2, 16, 128), (r.nb, 2, 16, 128)))
    side.wait_stream(torch.cuda.current_stream())
    r.call(outs=outs, stream=side)
    side.synchronize()
    r.check(outs)
    prefix, status = ints(r.prefix), ints([0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.spec_rope_append(r.qkv, *r.norm, 1e-5, r.freq, None, 128, 0, None, None, 1, *outs, r.table, r.table.shape[1], 16, r.nb, prefix, r.off, 2, 43, 40, 8,
                           2, 128, status)
    r.buffer.mul_(0.5)
    for o in outs:
        o.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    r.check(outs)


@DTYPES
def test_rope_pages_beyond_32_bit_offsets(dtype):
    r = Rope(21, [70, 1], [30, 600], 4, 2, 128, 256, dtype)
    nb = (1 << 31) // (2 * 256 * 128) + 3
    r.table = torch.where(r.table >= 0, r.table + (nb - r.nb), -1).to(torch.int32)
    small, r.nb = r.nb, nb
    q = torch.full((71, 4, 128), 7.0, dtype=dtype, device="cuda")
    k, v = (torch.empty((nb, 2, 256, 128), dtype=dtype, device="cuda") for _ in range(2))
    for c in (k, v):
        c[-small:] = 7.0
    r.call(outs=(q, k, v))
    r.table = torch.where(r.table >= 0, r.table - (nb - small), -1).to(torch.int32)
    r.check((q, k[-small:], v[-small:]))


# --------------------------------------------------------- attention weight ----

def _weight(d, before, path=None, accept=None, window=0, decay=0.75, out=None, status=None, stream=None, n_max=None, ws_fill=None):
    stride = before.shape[-1] if before is not None else d["stride"]
    size = (d["B"], d["T"], d["n_max"] if n_max is None else n_max, d["max_prefix"], d["Hq"], d["Hkv"], d["D"])
    ws = torch.full((S.spec_weight_workspace_size(*size),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((d["B"], d["Hkv"], stride), 7.0, device="cuda") if out is None else out
    status = ints([0] * d["B"]) if status is None else status
    S.spec_attention_weight(d["q"], d["k"], d["table"], d["table"].shape[1], d["bs"], d["nb"], d["prefix"], d["seq_off"], path, accept, window, *size,
                            d["scale"], decay, before, out, stride, ws, status, stream)
    return out, status


def _before(d, seed=1):
    stride = d["table"].shape[1] * d["bs"] + 5
    b = torch.full((d["B"], d["Hkv"], stride), math.nan)
    g = torch.Generator().manual_seed(seed)
    for i, p in enumerate(d["prefix"].tolist()):
        b[i, :, :p] = torch.rand((d["Hkv"], p), generator=g) * 3
    return b.cuda()


def _weight_holds(d, got, before, decay=0.75, skip=(), **kw):
    ref, tol = weight_reference(d, before, decay, **kw)
    for b in range(d["B"]):
        if b in skip:
            assert (got[b] == 7.0).all()
            continue
        mine = ~ref[b].isnan()
        assert (got[b][~mine] == 7.0).all()
        over = ((got[b].double() - ref[b]).abs() - tol[b])[mine]
        assert over.numel() == 0 or over.max() <= 0, (b, float(over.max()), float((got[b].double() - ref[b]).abs()[mine].max()))


SIZES = [([1], [0]), ([1], [1]), ([1], [127]), ([1], [128]), ([3, 0, 1], [0, 17, 700]), ([130, 5], [3, 260]), ([64, 64, 64], [64, 0, 1]),
         ([300, 1, 0, 9], [0, 2000, 40, 511])]


@DTYPES
@pytest.mark.parametrize("lens,prefix", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(32, 8, 128, 16), (4, 4, 64, 8), (10, 2, 64, 64), (64, 8, 128, 256), (5, 1, 128, 16)])
def test_weight_of_packed_rows(lens, prefix, Hq, Hkv, D, bs, dtype):
    d = paged_batch(31, lens, prefix, Hq, Hkv, D, bs, dtype, extra_rows=2)
    before = _before(d)
    got, st = _weight(d, before)
    assert st.tolist() == [0] * len(lens)
    _weight_holds(d, got, before)


@DTYPES
@pytest.mark.parametrize("window", [1, 4, 40, 1000])
def test_weight_of_the_last_rows(window, dtype):
    d = paged_batch(33, [200, 3, 0, 41], [0, 900, 10, 64], 16, 2, 128, 16, dtype)
    before = _before(d)
    got, st = _weight(d, before, window=window)
    assert not st.any()
    _weight_holds(d, got, before, window=window)


def _path(seed, lens, accept):
    g = np.random.default_rng(seed)
    top = max(lens)
    path = np.full((len(lens), top), -1, np.int32)
    for b, (n, a) in enumerate(zip(lens, accept)):
        if a:
            path[b, :a] = np.sort(np.concatenate([[0], g.choice(np.arange(1, n), a - 1, replace=False)]) if n > 1 else [0])
    return path


@DTYPES
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (4, 4, 64), (6, 2, 64)])
@pytest.mark.parametrize("window", [0, 3])
def test_weight_of_accepted_paths(Hq, Hkv, D, window, dtype):
    lens, accept = [20, 1, 64, 40, 7], [5, 1, 8, 0, 7]
    d = paged_batch(35, lens, [100, 2000, 0, 33, 15], Hq, Hkv, D, 16, dtype)
    path = _path(1, lens, accept)
    before = _before(d)
    got, st = _weight(d, before, ints(path.tolist()), ints(accept), window)
    assert not st.any()
    _weight_holds(d, got, before, path=path, accept=accept, window=window)


@DTYPES
def test_weight_of_a_long_accepted_path(dtype):
    """More rows than one tile holds, gathered."""
    lens, accept = [700, 90], [513, 90]
    d = paged_batch(36, lens, [300, 1000], 8, 2, 64, 16, dtype)
    path = _path(2, lens, accept)
    before = _before(d)
    got, st = _weight(d, before, ints(path.tolist()), ints(accept))
    assert not st.any()
    _weight_holds(d, got, before, path=path, accept=accept)


@DTYPES
@pytest.mark.parametrize("spread", [0.0, 1.0, 6.0])
def test_weight_in_place_from_zeros_and_with_steep_scores(spread, dtype):
    d = paged_batch(37, [9, 70], [50, 700], 8, 2, 64, 16, dtype, spread=spread)
    before = _before(d)
    want, tol = weight_reference(d, before, 1.0)
    buf = before.clone()
    _weight(d, buf, out=buf, decay=1.0)
    mine = ~want.isnan()
    assert ((buf.double() - want).abs()[mine] <= tol[mine]).all()
    assert buf[~mine].isnan().all()
    d["stride"] = before.shape[-1]
    got, _ = _weight(d, None)
    ref, tol = weight_reference(d, None, 0.0)
    mine = ~ref.isnan()
    assert ((got.double() - ref).abs()[mine] <= tol[mine]).all() and (got[~mine] == 7.0).all()
    # every row's probabilities sum to one
    assert abs(float(got[0, 0, :59].double().sum()) - 9 * 4) < 1e-3


@DTYPES
@pytest.mark.parametrize("lens,prefix", [([2, 1], [40000, 5000]), ([1] * 70, [3 * i for i in range(70)]), ([2500], [0])], ids=["long", "many", "prompt"])
def test_weight_long_and_wide_batches(lens, prefix, dtype):
    d = paged_batch(39, lens, prefix, 8, 2, 128, 64, dtype)
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)
    again, _ = _weight(d, before)
    assert torch.equal(got, again)  # the same bits every time


@DTYPES
@pytest.mark.parametrize("spread", [0.0, 6.0, 40.0])
@pytest.mark.parametrize("lens,prefix", [([1, 2], [2000, 300]), ([3], [9000]), ([8, 1, 4], [100, 30, 20000])], ids=["short", "one", "long"])
def test_weight_few_rows_with_steep_scores(lens, prefix, spread, dtype):
    d = paged_batch(42, lens, prefix, 8, 2, 64, 16, dtype, spread=spread)
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)


@DTYPES
def test_weight_of_a_mixed_batch(dtype):
    """Rows for every way through the kernels in one call: none, one, a few, a
    tile, many; keys from none to more than a cluster holds."""
    lens = [0, 1, 8, 9, 33, 64, 65, 300, 1, 0, 2]
    prefix = [700, 0, 2500, 2500, 100, 0, 900, 50, 36000, 0, 12]
    d = paged_batch(44, lens, prefix, 8, 2, 64, 16, dtype, extra_rows=3)
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)
    got, st = _weight(d, before, window=5)
    assert not st.any()
    _weight_holds(d, got, before, window=5)


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,window", [([3000], [0], 8, 1, 0), ([700, 64, 900], [300, 2000, 0], 6, 2, 0), ([2000, 10], [5, 90], 5, 1, 1500),
                                                       ([600], [4000], 4, 2, 0)])
def test_weight_in_parts_of_the_rows(lens, prefix, Hq, Hkv, window):
    """So few key tiles that the rows of a request are summed in parts."""
    d = paged_batch(49, lens, prefix, Hq, Hkv, 64, 16, torch.bfloat16)
    before = _before(d)
    got, st = _weight(d, before, window=window)
    assert not st.any()
    _weight_holds(d, got, before, window=window)
    st = ints([S.SPEC_DEV_TIMEOUT] + [0] * (len(lens) - 1))
    got, st = _weight(d, before, window=window, status=st)
    _weight_holds(d, got, before, window=window, skip=(0,))


@DTYPES
def test_weight_at_a_scale_of_zero(dtype):
    d = paged_batch(46, [3, 50], [20, 300], 8, 2, 64, 16, dtype)
    d["scale"] = 0.0
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)


@DTYPES
@pytest.mark.parametrize("n", [1, 20], ids=["few", "rows"])
def test_weight_bad_blocks_do_not_touch_other_requests(n, dtype):
    """More requests than are numbered at a time, with bad pages among the last:
    what one CTA flags, another may see before it numbers its items."""
    B = 300
    d = paged_batch(48, [n] * B, [(i * 37) % 900 for i in range(B)], 8, 2, 64, 16, dtype)
    bad = [3, 255, 256, 270, 299]
    for b in bad:
        d["table"][b, 0] = d["nb"] + 5
    before = _before(d)
    for _ in range(3):
        got, st = _weight(d, before)
        assert st.tolist() == [S.SPEC_DEV_BAD_BLOCK if b in bad else 0 for b in range(B)]
        table = d["table"].clone()
        d["table"][bad, 0] = 0
        ref, tol = weight_reference(d, before, 0.75)
        d["table"] = table
        for b in range(B):
            if b not in bad:
                mine = ~ref[b].isnan()
                assert ((got[b].double() - ref[b]).abs()[mine] <= tol[b][mine]).all() and (got[b][~mine] == 7.0).all()


@DTYPES
def test_weight_two_calls_at_once(dtype):
    """Two streams, a workspace each."""
    ds = [paged_batch(s, [2, 40], [3000, 200], 8, 2, 64, 16, dtype) for s in (50, 51)]
    befores, outs, streams = [_before(d) for d in ds], [], [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for d, before, stream in zip(ds, befores, streams):
            with torch.cuda.stream(stream):
                outs.append(_weight(d, before, stream=stream))
    torch.cuda.synchronize()
    for d, before, (got, st) in zip(ds, befores, outs):
        assert not st.any()
        _weight_holds(d, got, before)


@DTYPES
@pytest.mark.parametrize("Hq,Hkv", [(256, 2), (96, 1), (200, 1)], ids=["128", "96", "200"])
def test_weight_wide_groups(Hq, Hkv, dtype):
    d = paged_batch(40, [5, 1, 2], [0, 700, 33], Hq, Hkv, 64, 16, dtype)
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)


@DTYPES
def test_weight_bad_requests_are_left_as_they_were(dtype):
    def batch():
        return paged_batch(41, [6, 6, 6], [30, 20, 40], 8, 2, 64, 16, dtype)
    d = batch()
    before = _before(d)
    st = ints([0, S.SPEC_DEV_BAD_TREE, 0])
    got, st = _weight(d, before, status=st)
    assert st.tolist() == [0, S.SPEC_DEV_BAD_TREE, 0]
    _weight_holds(d, got, before, skip=(1,))
    got, st = _weight(d, before, n_max=5)
    assert st.tolist() == [S.SPEC_DEV_BAD_TREE] * 3 and (got == 7.0).all()
    d = batch()
    d["prefix"][1] = 41  # above max_prefix
    got, st = _weight(d, before)
    assert st.tolist() == [0, S.SPEC_DEV_CAPACITY, 0]
    d["prefix"][1] = 20
    _weight_holds(d, got, before, skip=(1,))
    short = before[:, :, :45].contiguous()  # 40 + 6 slots do not fit
    got, st = _weight(d, short)
    assert st.tolist() == [0, 0, S.SPEC_DEV_CAPACITY]
    assert (got[2] == 7.0).all()
    d = batch()
    d["table"][0, 1] = d["nb"]
    got, st = _weight(d, before)
    assert st.tolist() == [S.SPEC_DEV_BAD_BLOCK, 0, 0]
    d["table"][0, 1] = 0
    ref, tol = weight_reference(d, before, 0.75)
    for b in (1, 2):
        mine = ~ref[b].isnan()
        assert ((got[b].double() - ref[b]).abs()[mine] <= tol[b][mine]).all()


def test_weight_bad_paths():
    d = paged_batch(43, [6, 6, 6, 6], [30, 20, 40, 3], 8, 2, 64, 16, torch.bfloat16)
    before = _before(d)
    path = [[0, 2, 5, -1, -1, -1], [0, 6, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5], [0, -1, 3, 4, -1, -1]]
    got, st = _weight(d, before, ints(path), ints([3, 2, 7, -1]))
    assert st.tolist() == [0, S.SPEC_DEV_BAD_PATH, S.SPEC_DEV_BAD_PATH, S.SPEC_DEV_BAD_PATH]
    _weight_holds(d, got, before, skip=(1, 2, 3), path=path, accept=[3, 0, 0, 0])
    got, st = _weight(d, before, ints(path), ints([3, 0, 6, 4]), window=2)  # the bad entry of the last one is not counted
    assert not st.any()
    _weight_holds(d, got, before, path=path, accept=[3, 0, 6, 4], window=2)


def test_weight_in_a_graph_with_other_data():
    d = paged_batch(45, [4, 200], [3000, 0], 8, 2, 128, 16, torch.bfloat16)
    before = _before(d)
    buf = before.clone()
    size = (2, 204, 200, 3000, 8, 2, 128)
    ws = torch.empty(S.spec_weight_workspace_size(*size), dtype=torch.uint8, device="cuda")
    st = ints([0, 0])

    def call():
        S.spec_attention_weight(d["q"], d["k"], d["table"], d["table"].shape[1], 16, d["nb"], d["prefix"], d["seq_off"], None, None, 0, *size, d["scale"], 1.0,
                                buf, buf, buf.shape[-1], ws, st)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for scale in (0.5, 1.5):
        d["q"].mul_(scale)
        buf.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = weight_reference(d, before, 1.0)
        mine = ~ref.isnan()
        assert ((buf.double() - ref).abs()[mine] <= tol[mine]).all()
    assert not st.any()


@DTYPES
def test_weight_cache_beyond_32_bit_offsets(dtype):
    d = paged_batch(47, [70, 1], [30, 600], 4, 2, 128, 256, dtype)
    nb = (1 << 31) // (2 * 256 * 128) + 3
    big = torch.empty((nb, 2, 256, 128), dtype=dtype, device="cuda")
    big[-d["nb"]:] = d["k"]
    d["k"], d["table"] = big, torch.where(d["table"] >= 0, d["table"] + (nb - d["nb"]), -1).to(torch.int32)
    d["nb"] = nb
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)


# ------------------------------------------------------------------ evict ----

class Evict:
    def __init__(self, seed, lens, keep, first, last, layers=2, Hkv=2, D=64, bs=16, dtype=torch.bfloat16, ties=True, spare=1):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.keep, self.first, self.last, self.layers, self.Hkv, self.D, self.bs, self.dtype = lens, keep, first, last, layers, Hkv, D, bs, dtype
        N = len(lens)
        self.N, self.keep_max = N, max(keep)
        kept = [min(k, n) for k, n in zip(keep, lens)]
        self.table, self.nb = table_of(seed, lens + kept, bs)
        self.B = 2 * N
        self.stride = self.table.shape[1] * bs
        w = torch.randn((layers, self.B, Hkv, self.stride), generator=g).mul(3)
        if ties:
            w = w.round() / 4 * (torch.rand(w.shape, generator=g) > 0.2)  # many equal, zeros of both signs
        self.weight = w.cuda()
        self.cache = torch.randn((layers, 2, self.nb, Hkv, bs, D), generator=g).to(dtype).cuda()
        self.src, self.dst = list(range(N)), list(range(N, 2 * N))

    def call(self, weight="own", status=None, keep="own", keep_max=None, stream=None):
        w = self.weight if isinstance(weight, str) else weight
        km = self.keep_max if keep_max is None else keep_max
        n = len(self.src)
        slots, new_len = torch.full((self.layers, n, self.Hkv, km), 77, dtype=torch.int32, device="cuda"), ints([77] * n)
        status = ints([77] * n)
        ptrs = [torch.tensor([c[i].data_ptr() for c in self.cache], dtype=torch.int64, device="cuda") for i in range(2)]
        S.spec_kv_evict(*ptrs, self.layers, self.table, self.B, self.table.shape[1], self.bs, self.nb, ints(self.src), ints(self.dst), ints(self.lens),
                        ints(self.keep) if isinstance(keep, str) else keep, n, km, self.first, self.last, w, self.stride, self.Hkv, self.D,
                        S.SPEC_F32 if self.dtype == torch.float32 else S.SPEC_BF16, slots, new_len, status, stream)
        return slots, new_len, status

    def run_and_check(self, flagged=None, weight="own", **kw):
        flagged = flagged or {}
        cache, weights = self.cache.clone(), self.weight.clone()
        slots, new_len, status = self.call(weight=weight, **kw)
        assert status.tolist() == [flagged.get(i, 0) for i in range(len(self.src))]
        want_slots = np.full(tuple(slots.shape), -1, np.int32)
        wl, table = weights.cpu().tolist(), self.table.cpu()
        for i in range(len(self.src)):
            if i in flagged:
                assert int(new_len[i]) == 0
                continue
            kept = min(self.keep[i], self.lens[i])
            assert int(new_len[i]) == kept
            for layer in range(self.layers):
                for h in range(self.Hkv):
                    w = wl[layer][self.src[i]][h] if isinstance(weight, str) else None
                    stay = keep_reference(w, self.lens[i], self.keep[i], self.first, self.last)
                    assert len(stay) == kept
                    want_slots[layer, i, h, :kept] = stay
                    old, new = torch.tensor(stay, dtype=torch.long), torch.arange(kept)
                    p_old, p_new = table[self.src[i]][old // self.bs].long(), table[self.dst[i]][new // self.bs].long()
                    cache[layer, :, p_new.cuda(), h, (new % self.bs).cuda()] = cache[layer, :, p_old.cuda(), h, (old % self.bs).cuda()]
                    if isinstance(weight, str):
                        weights[layer, self.dst[i], h, :kept] = weights[layer, self.src[i], h, old.cuda()]
        assert np.array_equal(slots.cpu().numpy(), want_slots)
        assert torch.equal(self.weight.view(torch.int32), weights.view(torch.int32))
        view = torch.int16 if self.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(self.cache.view(view), cache.view(view))


@DTYPES
@pytest.mark.parametrize("ties", [True, False], ids=["ties", "distinct"])
@pytest.mark.parametrize("lens,keep,first,last", [([1], [1], 0, 0), ([1], [0], 4, 4), ([5, 0, 40], [9, 3, 7], 1, 2), ([700, 3, 513, 512, 90], [129, 40, 512, 1, 90], 4, 17),
                                                  ([600], [100], 60, 60), ([600], [100], 0, 0), ([600], [599], 0, 1), ([2100, 1500], [64, 1000], 4, 0),
                                                  ([40], [20], 0, 100), ([40], [20], 100, 3)], ids=[str(i) for i in range(10)])
def test_evict_keeps_the_heavy_slots(lens, keep, first, last, ties, dtype):
    Evict(51, lens, keep, first, last, dtype=dtype, ties=ties).run_and_check()


@pytest.mark.parametrize("Hkv,D,bs,layers", [(8, 128, 256, 1), (1, 64, 8, 5), (3, 128, 64, 3)])
def test_evict_shapes(Hkv, D, bs, layers):
    Evict(53, [300, 77], [50, 33], 4, 8, layers=layers, Hkv=Hkv, D=D, bs=bs).run_and_check()


def test_evict_orders_nan_infinities_zeros_and_close_weights():
    e = Evict(55, [800], [799], 0, 0, ties=False)  # pages for the largest of the budgets below
    w = e.weight[:, 0]
    w[..., 0:200:3] = math.nan
    w[..., 1:200:3] = math.inf
    w[..., 2:200:3] = -math.inf
    w[..., 200:400] = torch.tensor([0.0, -0.0], device="cuda").repeat(100)
    w[..., 400:600] = 1.0 + torch.arange(200, device="cuda") * 2.0 ** -23  # they differ in the last bits
    w[..., 600:700] = 1e-42  # denormal
    w[..., 700:] = -1e-42
    e.run_and_check()
    for keep in (1, 67, 68, 267, 300, 268, 367, 368, 468, 568, 668, 733, 734, 799):
        e.keep = [keep]
        e.run_and_check(keep_max=799)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 16385, 49152, 49153, 70000])
def test_evict_long_rows(n):
    """Around the sizes where the selection changes its way."""
    e = Evict(56, [n, 100], [301, 50], 3, 5, layers=1, Hkv=1, bs=64)
    e.run_and_check()
    e.weight[:] = e.weight.abs() + 1.0  # one exponent and a few more
    e.run_and_check()


def test_evict_without_weights_is_a_window():
    e = Evict(57, [90, 400], [40, 40], 4, 36)
    e.run_and_check(weight=None)
    e.first, e.last = 0, 0
    e.run_and_check(weight=None)


def test_evict_one_budget_for_all_and_many_rows():
    e = Evict(59, [(i * 37) % 200 for i in range(40)], [25] * 40, 2, 5, layers=1)
    e.run_and_check(keep=None)


def test_evict_from_shared_pages():
    """Two rows evict from the same pages: the source is only read."""
    e = Evict(61, [200, 200], [30, 60], 2, 4)
    e.table[1] = e.table[0]
    e.run_and_check()
    e.src = [0, 0]
    e.run_and_check()


def test_evict_flags():
    def fresh():
        return Evict(63, [60, 61, 62, 63], [10, 11, 12, 13], 1, 2)
    bad_row, cap, block = S.SPEC_DEV_BAD_ROW, S.SPEC_DEV_CAPACITY, S.SPEC_DEV_BAD_BLOCK
    for name, value in (("src", -1), ("src", 8), ("dst", -1), ("dst", 8), ("lens", -1), ("keep", -1), ("keep", 14)):
        e = fresh()
        getattr(e, name)[1] = value
        e.run_and_check({1: bad_row}, keep_max=13)
    e = fresh()
    e.dst[1] = 1  # itself
    e.run_and_check({1: bad_row})
    e = fresh()
    e.dst[1] = 3  # another's source
    e.run_and_check({1: bad_row})
    e = fresh()
    e.dst[2] = e.dst[1]
    e.run_and_check({1: bad_row, 2: bad_row})
    e = fresh()
    e.lens[2] = e.table.shape[1] * 16 + 1
    e.run_and_check({2: cap})
    e = fresh()
    e.table[0, 3] = -1
    e.table[7, 0] = e.nb
    e.run_and_check({0: block, 3: block})
    e = fresh()  # pages behind what is held are not looked at
    e.table[0, 4:] = e.nb
    e.run_and_check()


def test_evict_in_a_graph_and_on_a_stream():
    e = Evict(65, [500, 300], [90, 80], 4, 8)
    ptrs = [torch.tensor([c[i].data_ptr() for c in e.cache], dtype=torch.int64, device="cuda") for i in range(2)]
    src, dst, lens, keep = ints(e.src), ints(e.dst), ints(e.lens), ints(e.keep)
    slots, new_len, status = torch.zeros((2, 2, 2, 90), dtype=torch.int32, device="cuda"), ints([0, 0]), ints([0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.spec_kv_evict(*ptrs, 2, e.table, e.B, e.table.shape[1], 16, e.nb, src, dst, lens, keep, 2, 90, 4, 8, e.weight, e.stride, 2, 64, S.SPEC_BF16, slots,
                        new_len, status)
    e.weight.neg_()
    graph.replay()
    torch.cuda.synchronize()
    got = e.cache.clone(), e.weight.clone(), slots.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, _, st = e.call()
    side.synchronize()
    assert torch.equal(again, got[2]) and torch.equal(e.cache, got[0]) and torch.equal(e.weight, got[1]) and not st.any()
    e.run_and_check()


def test_evict_caches_beyond_32_bit_offsets():
    e = Evict(67, [300], [70], 4, 8, layers=1, Hkv=2, D=128, bs=256)
    nb = (1 << 31) // (2 * 256 * 128) + 3
    big = torch.empty((1, 2, nb, 2, 256, 128), dtype=torch.bfloat16, device="cuda")
    big[:, :, -e.nb:] = e.cache
    small, e.table = e.nb, torch.where(e.table >= 0, e.table + (nb - e.nb), -1).to(torch.int32)
    want = keep_reference(e.weight[0, 0, 1].tolist(), 300, 70, 4, 8)
    e.cache, e.nb = big, nb
    slots, new_len, st = e.call()
    assert st.tolist() == [0] and new_len.tolist() == [70] and slots[0, 0, 1].tolist() == want
    old, new = torch.tensor(want, device="cuda"), torch.arange(70, device="cuda")
    for kv in range(2):
        got = big[0, kv, e.table[1][new // 256].long(), 1, new % 256]
        assert torch.equal(got, big[0, kv, e.table[0][old // 256].long(), 1, old % 256])
    assert small < 10


def test_evict_right_before_tree_attention():
    """Tree attention reads the prefix's rows before it waits for the kernel before
    it: both ways of copying have to be done by then."""
    for layers, N in ((1, 2), (20, 8)):  # a copy kernel of its own, and the selecting CTAs' copies
        e = Evict(71, [900] * N, [512] * N, 4, 64, layers=layers, Hkv=2, D=128, bs=16)
        T = N * 4
        # each row of the short ones has a page for a tree
        spare = torch.arange(e.nb - 3, e.nb, dtype=torch.int32, device="cuda")
        table = e.table[N:].clone()
        table[:, 32] = spare[torch.arange(N, device="cuda") % 3]
        parent, off = ints([-1, 0, 1, 1] * N), ints([4 * i for i in range(N + 1)])
        mask, depth, st = torch.zeros((T, 1), dtype=torch.int64, device="cuda"), ints([0] * T), ints([0] * N)
        S.spec_tree_mask_build(parent, off, N, 4, mask, depth, st)
        q = torch.randn((T, 8, 128), generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
        ws = torch.empty(S.spec_attention_workspace_size(N, T, 4, 512, 8, 2, 128), dtype=torch.uint8, device="cuda")
        prefix = ints([512] * N)
        ptrs = [torch.tensor([c[i].data_ptr() for c in e.cache], dtype=torch.int64, device="cuda") for i in range(2)]
        slots, new_len, status = torch.empty((layers, N, 2, 512), dtype=torch.int32, device="cuda"), ints([0] * N), ints([0] * N)
        src, dst, lens = ints(e.src), ints(e.dst), ints(e.lens)
        outs = []
        for again in (False, True, False, True, False):
            if not again:  # what the short rows held before
                e.cache[:, :, e.table[N:, :32].reshape(-1).long()] = 0
            torch.cuda.synchronize()
            out = torch.empty_like(q)
            if not again:
                S.spec_kv_evict(*ptrs, layers, e.table, e.B, e.table.shape[1], 16, e.nb, src, dst, lens, None, N, 512, 4, 64, e.weight, e.stride, 2, 128,
                                S.SPEC_BF16, slots, new_len, status)
            S.spec_tree_attention(q, e.cache[-1, 0], e.cache[-1, 1], table, table.shape[1], 16, e.nb, prefix, off, mask, N, T, 4, 512, 8, 2, 128, 0.1, out, ws, st)
            torch.cuda.synchronize()
            outs.append(out)
        assert not st.any() and all(torch.equal(o, outs[1]) for o in outs)


@DTYPES
def test_weight_of_requests_without_rows(dtype):
    """No new row at all: the weights decay."""
    d = paged_batch(72, [1, 1], [300, 5], 8, 2, 64, 16, dtype)
    before = _before(d)
    d.update(q=d["q"][:0], seq_off=ints([0, 0, 0]), T=0, n_max=0)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)
    got, st = _weight(d, None) if d.update(stride=before.shape[-1]) is None else None
    assert (got[0, :, :300] == 0).all() and (got[0, :, 300:] == 7.0).all() and (got[1, :, :5] == 0).all()
