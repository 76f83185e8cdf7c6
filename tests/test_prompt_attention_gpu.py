"""Prompt attention through the C ABI against 64-bit attention: lengths from
zero to several tiles, prefixes, group widths that do and do not divide a row
tile, page sizes, both types, split keys, refusals on the device."""
import math

import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from request_life import paged_batch, prompt_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


def _size(d):
    return (d["B"], d["T"], d["n_max"], d["max_prefix"], d["Hq"], d["Hkv"], d["D"])


def _call(d, out=None, status=None, ws=None, stream=None, table=None):
    out = torch.full_like(d["q"], 7.0) if out is None else out
    status = torch.zeros(d["B"], dtype=torch.int32, device="cuda") if status is None else status
    ws = torch.empty(S.spec_prompt_workspace_size(*_size(d)), dtype=torch.uint8, device="cuda") if ws is None else ws
    table = d["table"] if table is None else table
    S.spec_prompt_attention(d["q"], d["k"], d["v"], table, table.shape[1], d["bs"], d["nb"], d["prefix"], d["seq_off"],
                            *_size(d), d["scale"], out, ws, status, stream=stream)
    return out, status


def _holds(d, out, rows=None):
    ref, tol = prompt_reference(d)
    rows = torch.arange(int(d["seq_off"][-1]), device="cuda") if rows is None else rows
    err = (out.double() - ref).abs()[rows]
    assert torch.isfinite(out[rows].double()).all()
    worst = (err / tol[rows]).max().item() if rows.numel() else 0.0
    assert worst <= 1.0, worst


CASES = [
    # lens, prefix, Hq, Hkv, D, bs
    ([1], [0], 4, 4, 64, 16),
    ([128], [0], 4, 4, 64, 16),
    ([5, 0, 1, 64], [0, 7, 0, 3], 8, 2, 64, 8),
    ([0, 0, 3], [0, 0, 0], 8, 2, 128, 64),
    ([129, 127, 1, 255, 257], [0, 1, 128, 129, 500], 8, 2, 128, 16),
    ([300, 33], [0, 1000], 32, 8, 128, 16),
    ([64, 65, 63], [0, 64, 63], 64, 8, 128, 256),
    ([100, 43, 2], [13, 0, 200], 6, 2, 64, 64),       # g = 3: a token's heads straddle row tiles
    ([90, 17], [5, 300], 20, 4, 128, 32),             # g = 5
    ([70], [20], 5, 1, 64, 16),
    ([40, 1, 130], [0, 256, 3], 32, 1, 64, 128),      # one kv head
    ([600], [0], 16, 2, 128, 512),
    ([2, 1, 1, 3, 1, 1, 1], [900, 1500, 5, 0, 1, 2047, 2048], 16, 4, 128, 16),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}x{max(c[0])}-{c[2]}:{c[3]}-D{c[4]}-p{c[5]}" for c in CASES])
def test_prompt_attention_holds(case, dtype):
    lens, prefix, Hq, Hkv, D, bs = case
    d = paged_batch(sum(lens) + D, lens, prefix, Hq, Hkv, D, bs, dtype, extra_rows=3)
    out, status = _call(d)
    assert status.tolist() == [0] * d["B"]
    _holds(d, out)
    T = int(d["seq_off"][-1])
    assert (out[T:] == 7.0).all()  # rows behind the last request stay as they were


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_long_prefixes_split_over_the_gpu(dtype):
    d = paged_batch(5, [3, 1], [6000, 9000], 8, 2, 128, 64, dtype)
    assert S.spec_prompt_workspace_size(*_size(d)) > 256
    out, status = _call(d)
    assert status.tolist() == [0, 0]
    _holds(d, out)
    with pytest.raises(S.SpecError) as e:
        _call(d, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == S.SPEC_ERR_WORKSPACE


@pytest.mark.parametrize("spread", [0.0, 40.0, 300.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_scores_far_apart(dtype, spread):
    """Equal keys, and keys whose scores lie hundreds apart: the reference of
    the exponentials has to follow the maximum along the keys."""
    d = paged_batch(9, [200, 70], [0, 333], 8, 2, 128, 16, dtype, spread=spread)
    out, status = _call(d)
    assert status.tolist() == [0, 0]
    _holds(d, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_keys_that_grow_along_the_sequence(dtype):
    """Each later block of keys dwarfs the ones before, and the reverse."""
    for sign in (1.0, -1.0):
        d = paged_batch(11, [400], [0], 4, 2, 64, 16, dtype)
        ids = d["table"][0, :25].long()
        grow = torch.exp2(torch.arange(400, device="cuda") / 40.0 * sign).view(25, 1, 16, 1)
        d["k"][ids] = (d["k"][ids].float() * grow * (1.0 if sign > 0 else 64.0)).to(dtype)
        out, status = _call(d)
        _holds(d, out)


def test_many_requests():
    """More requests than one sorting pass takes, most of a few tokens."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 9, (700,), generator=g).tolist()
    prefix = torch.randint(0, 90, (700,), generator=g).tolist()
    d = paged_batch(13, lens, prefix, 8, 2, 64, 16, torch.bfloat16)
    out, status = _call(d)
    assert status.tolist() == [0] * 700
    _holds(d, out)


def test_larger_ragged_batch():
    d = paged_batch(17, [1024, 77, 2000, 513], [0, 1500, 100, 0], 32, 8, 128, 16, torch.bfloat16)
    out, status = _call(d)
    assert status.tolist() == [0] * 4
    _holds(d, out)


def test_refused_requests_leave_the_others_alone():
    d = paged_batch(19, [40, 30, 20, 10, 50], [10, 20, 0, 70, 5], 8, 2, 64, 16, torch.bfloat16)
    ref_out, _ = _call(d)
    table = d["table"].clone()
    table[2, 0] = d["nb"]           # an id past the pool
    d["prefix"] = d["prefix"].clone()
    d["prefix"][3] = d["max_prefix"] + 1
    status = torch.zeros(5, dtype=torch.int32, device="cuda")
    status[1] = S.SPEC_DEV_BAD_TREE  # failed before this call
    out, status = _call(d, table=table, status=status)
    assert status.tolist() == [0, S.SPEC_DEV_BAD_TREE, S.SPEC_DEV_BAD_BLOCK, S.SPEC_DEV_CAPACITY, 0]
    off = d["seq_off"].tolist()
    for b in (0, 4):
        assert torch.equal(out[off[b]:off[b + 1]], ref_out[off[b]:off[b + 1]])
    for b in (1, 3):
        assert (out[off[b]:off[b + 1]] == 7.0).all()


def test_requests_outside_the_stated_bounds():
    d = paged_batch(23, [40, 30], [0, 0], 8, 2, 64, 16, torch.bfloat16)
    good, _ = _call(d)
    d["n_max"] = 35  # the first request is longer than the call allows
    out, status = _call(d)
    assert status.tolist() == [S.SPEC_DEV_BAD_TREE, 0]
    assert (out[:40] == 7.0).all() and torch.equal(out[40:], good[40:])
    d["n_max"], d["T"] = 40, 60  # rows beyond T
    out, status = _call(d)
    assert status.tolist() == [0, S.SPEC_DEV_BAD_TREE]
    assert torch.equal(out[:40], good[:40]) and (out[40:] == 7.0).all()


def test_runs_on_a_side_stream_and_replays_from_a_graph():
    d = paged_batch(29, [33, 150, 1], [400, 0, 3000], 8, 2, 128, 16, torch.bfloat16)
    ref, _ = _call(d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, status = torch.full_like(d["q"], 7.0), torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(S.spec_prompt_workspace_size(*_size(d)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _call(d, out, status, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(d, out, status, ws)
    for seed in (1, 2):
        d["q"].copy_(torch.randn(d["q"].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(d["q"].dtype))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        _holds(d, out)


def test_workspace_contents_do_not_matter(monkeypatch):
    d = paged_batch(31, [3], [5000], 8, 2, 128, 64, torch.bfloat16)
    ref, _ = _call(d)
    monkeypatch.setenv("SPECTREE_WORKSPACE_CANARY", "1")
    out, _ = _call(d)
    assert torch.equal(out, ref) and not math.isnan(out.float().sum().item())


def test_a_batch_without_any_token():
    d = paged_batch(37, [0, 0, 0], [0, 5, 40], 8, 2, 64, 16, torch.bfloat16, extra_rows=4)
    d["n_max"] = 3
    for dtype in (torch.bfloat16, torch.float32):
        for n in ("q", "k", "v"):
            d[n] = d[n].to(dtype)
        out, status = _call(d)
        assert status.tolist() == [0, 0, 0] and (out == 7.0).all()


def test_calls_on_two_streams_at_once_and_again():
    """Two batches on two streams, each with its own workspace, several times
    over: every call gives the same bits."""
    ds = [paged_batch(41, [500, 3, 129], [0, 4000, 77], 16, 4, 128, 16, torch.bfloat16),
          paged_batch(43, [1], [9000], 8, 1, 64, 32, torch.bfloat16)]
    ref = [_call(d)[0] for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    ws = [torch.empty(S.spec_prompt_workspace_size(*_size(d)), dtype=torch.uint8, device="cuda") for d in ds]
    outs = [[torch.full_like(d["q"], 7.0) for _ in range(4)] for d in ds]
    st = [torch.zeros(d["B"], dtype=torch.int32, device="cuda") for d in ds]
    torch.cuda.synchronize()
    for i in range(4):
        for d, s, w, o, t in zip(ds, streams, ws, outs, st):
            _call(d, o[i], t, w, stream=s)
    torch.cuda.synchronize()
    for r, o in zip(ref, outs):
        assert all(torch.equal(r, x) for x in o)


def test_infinities_and_nan_stay_in_their_own_rows():
    """A query row of NaN, and one whose scores are infinite, next to sound rows."""
    d = paged_batch(47, [40, 9], [0, 300], 8, 2, 64, 16, torch.bfloat16)
    ref, _ = _call(d)
    d["q"] = d["q"].clone()
    d["q"][7, 2] = math.nan
    d["q"][11, 5] = math.inf
    out, status = _call(d)
    assert status.tolist() == [0, 0] and torch.isnan(out[7, 2]).all()
    sound = torch.ones(49, 8, dtype=torch.bool, device="cuda")
    sound[7, 2] = sound[11, 5] = False
    d["q"][7, 2], d["q"][11, 5] = 0.0, 0.0  # the reference of the other rows
    want, tol = prompt_reference(d)
    assert ((out.double() - want).abs() <= tol)[sound].all()


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 2)], ids=["tma_q", "copied_q"])
@pytest.mark.parametrize("fill", [math.nan, math.inf, 3e4], ids=["nan", "inf", "large"])
def test_rows_beside_a_request_leave_its_bits_alone(fill, Hq, Hkv):
    """A row tile reaches past its request, into the next one's rows and the rows
    behind the last: what they hold does not show in a single bit."""
    d = paged_batch(53, [70, 21], [40, 300], Hq, Hkv, 128, 16, torch.bfloat16, extra_rows=5)
    d["q"][91:] = 0.0
    ref, _ = _call(d)
    d["q"][91:] = fill
    out, status = _call(d)
    assert status.tolist() == [0, 0] and torch.equal(out[:91], ref[:91])
    d["q"][70:91] = fill
    out, status = _call(d)
    assert status.tolist() == [0, 0] and torch.equal(out[:70], ref[:70])


@pytest.mark.parametrize("scale", [0.0, 1e-30])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_a_scale_of_zero_averages_what_a_row_sees(dtype, scale):
    """Every score 0: hidden keys weigh nothing all the same.  The second batch
    splits its keys."""
    for lens, prefix in (([200, 1, 70], [0, 333, 5]), ([3, 1], [6000, 9000])):
        d = paged_batch(59, lens, prefix, 8, 2, 128, 16, dtype)
        d["scale"] = scale
        out, status = _call(d)
        assert status.tolist() == [0] * len(lens)
        _holds(d, out)


def test_a_workspace_that_fits_one_batch_serves_smaller_ones():
    """A server's one buffer, sized for its largest batch: smaller batches, which
    would split their keys further, run in it too."""
    for dtype in (torch.bfloat16, torch.float32):
        for lens, prefix in (([1] * 3, [4000, 16000, 90]), ([200], [3000]), ([1], [9000])):
            d = paged_batch(71, lens, prefix, 8, 2, 128, 64, dtype)
            d["max_prefix"] = 16384
            need = S.spec_prompt_workspace_size(*_size(d))
            per = -(-4 * d["T"] * 8 * 130 // 256) * 256 + 256
            for room in sorted({256, 256 + 2 * per, 256 + 3 * per, need - 1, need}):
                out, status = _call(d, ws=torch.empty(room, dtype=torch.uint8, device="cuda"))
                assert status.tolist() == [0] * len(lens)
                _holds(d, out)
            with pytest.raises(S.SpecError) as e:
                _call(d, ws=torch.empty(255, dtype=torch.uint8, device="cuda"))
            assert e.value.code == S.SPEC_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_row_that_sees_one_key_returns_its_value(D, dtype):
    """The first token of a fresh prompt, and rows that one key's score leaves
    alone (it leads by more than 24 bits): V itself, every bit."""
    lens = [1] * 40 + [130, 300]
    d = paged_batch(67, lens, [0] * 42, 8, 2, D, 16, dtype, spread=2.0)
    lead = d["table"][41, 3].long()             # slots 48 .. 63 of the last request: slot 50 leads
    d["k"][lead, :, 2] = 400.0
    d["q"][170 + 51:470] = d["q"][170 + 51:470].abs() + 0.5
    out, status = _call(d)
    assert status.tolist() == [0] * 42
    for b, t in [(b, b) for b in range(40)] + [(40, 40), (41, 170)]:
        v = d["v"][d["table"][b, 0].long(), :, 0]
        assert torch.equal(out[t], v.repeat_interleave(4, 0)), b
    v = d["v"][lead, :, 2].repeat_interleave(4, 0)
    assert (out[170 + 51:470] == v).all()


@pytest.mark.parametrize("size", [-90, 90])
@pytest.mark.parametrize("score", [0.0, 35.0, -35.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_values_of_any_size(dtype, score, size):
    """Values of 2^-90 and 2^90 under scores about +-50 (log2): no accumulator
    overflows and no product is lost."""
    for lens, prefix in (([200, 70], [0, 333]), ([3], [6000])):
        d = paged_batch(61, lens, prefix, 8, 2, 128, 16, dtype, spread=0.5)
        d["v"] = (d["v"].float() * 2.0 ** size).to(dtype)
        d["q"] = (d["q"].float() * 0.5 + 1.0).to(dtype)
        d["k"] = (d["k"].float() + score / math.sqrt(128)).to(dtype)
        out, status = _call(d)
        assert status.tolist() == [0] * len(lens)
        _holds(d, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv", [(256, 2), (256, 1), (96, 1)], ids=["128", "256", "96"])
def test_wide_groups(Hq, Hkv, dtype):
    """Groups as wide as a row tile, wider, and such as share no factor with it."""
    d = paged_batch(73, [5, 1, 2], [0, 700, 33], Hq, Hkv, 64, 16, dtype)
    out, status = _call(d)
    assert status.tolist() == [0] * 3
    _holds(d, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("prefix", [[0, 5, 300], [0, 5, 9000]], ids=["whole", "split"])
def test_packing_that_starts_behind_row_zero(prefix, dtype):
    """Rows before the first request belong to nobody: NaN in q, left alone in out."""
    d = paged_batch(79, [40, 3, 77], prefix, 8, 2, 64, 16, dtype)
    gap = 37
    lead = torch.full((gap,) + d["q"].shape[1:], math.nan, device="cuda", dtype=dtype)
    d["q"], d["seq_off"], d["T"] = torch.cat([lead, d["q"]]), d["seq_off"] + gap, d["T"] + gap
    out, status = _call(d)
    assert status.tolist() == [0] * 3 and (out[:gap] == 7.0).all()
    _holds(d, out, torch.arange(gap, d["T"], device="cuda"))


@pytest.mark.parametrize("dtype,bs", [(torch.bfloat16, 16), (torch.bfloat16, 65536), (torch.float32, 256)], ids=["bf16", "one_page", "fp32"])
def test_caches_beyond_32_bit_offsets(dtype, bs):
    """Pages at the end of caches of more than 2^31 elements (2^32 bytes and more)."""
    Hkv, D = 2, 128
    nb = (1 << 31) // (Hkv * bs * D) + 3
    d = paged_batch(83, [70, 1], [30, 600], 4, Hkv, D, bs, dtype)
    for n in ("k", "v"):
        big = torch.empty((nb, Hkv, bs, D), dtype=dtype, device="cuda")
        big[-d["nb"]:] = d[n]
        d[n] = big
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (nb - d["nb"]), -1).to(torch.int32)
    d["nb"] = nb
    out, status = _call(d)
    assert status.tolist() == [0, 0]
    _holds(d, out)
    # the append reaches them too
    new = [torch.randn((71, Hkv, D), device="cuda").to(dtype) for _ in range(2)]
    S.spec_kv_append(*new, d["k"], d["v"], d["table"], d["table"].shape[1], bs, nb, d["prefix"], d["seq_off"], 2, 70, Hkv, D, status)
    assert status.tolist() == [0, 0]
    for c, x in zip((d["k"], d["v"]), new):
        for b, (o, n, p) in enumerate(((0, 70, 30), (70, 1, 600))):
            s = p + torch.arange(n, device="cuda")
            assert torch.equal(c[d["table"][b][s // bs].long(), :, s % bs], x[o:o + n])
    out, status = _call(d)
    _holds(d, out)
