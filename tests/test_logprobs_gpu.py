"""Log probabilities, entropy, rank and alternatives through the C ABI against
64-bit softmax rows."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from request_life import logprob_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


def _outputs(shape, k):
    f = dict(device="cuda")
    i = dict(dtype=torch.int32, device="cuda")
    return (torch.full(shape, 7.0, **f), torch.full(shape, 7.0, **f), torch.full(shape, 7, **i),
            torch.full(shape + (k,), 7, **i), torch.full(shape + (k,), 7.0, **f))


def _tokens_call(x, tokens, off, tau, k, status=None):
    T, V = x.shape
    B = len(off) - 1
    out = _outputs((T,), k)
    status = torch.zeros(B, dtype=torch.int32, device="cuda") if status is None else status
    S.spec_token_logprobs(x, torch.tensor(tokens, dtype=torch.int32, device="cuda"),
                          torch.tensor(off, dtype=torch.int32, device="cuda"),
                          None if tau is None else torch.tensor(tau, dtype=torch.float32, device="cuda"), B, T, V, k,
                          *out, status)
    return out, status.tolist()


def _tolerance(x, tau, ref_lp):
    """A weight e^(tau (x - m)) is off by 2^-22 (the exponential) and by 2^-22
    of its exponent (three roundings), which weighs at most e^-t t < 1 / e of
    the largest; a thread adds at most ceil(V / 256) + 64 of them and raises
    its reference at most once per 16, each raise 2^-21; the logarithm and the
    difference are off by 2^-23 of their size.  The entropy adds one more
    product per weight: the same, times the size of its terms."""
    n = -(-len(x) // 256) + 64
    rel = 2.0 ** -22 * 2 + n * 2.0 ** -24 + (n / 16) * 2.0 ** -21
    size = 0.0 if not np.isfinite(ref_lp) else abs(ref_lp)
    return rel + 2.0 ** -22 * (size + math.log(len(x)) + 1)


def _check(row, out, i, token, tau, k):
    lp, ent, rank, top, top_lp = logprob_reference(row, token, tau, k)
    got = [o[i].cpu() for o in out]
    for g, r in ((got[0].item(), lp), (got[1].item(), ent)):
        if math.isnan(r):
            assert math.isnan(g)
        elif math.isinf(r):
            assert g == r
        else:
            assert abs(g - r) <= _tolerance(row, tau, r) * (1 + math.log(len(row))), (g, r)
    assert got[2].item() == rank
    assert got[3].tolist() == list(top)
    for g, r in zip(got[4].tolist(), top_lp):
        assert (math.isnan(g) and math.isnan(r)) or g == r or abs(g - r) <= _tolerance(row, tau, r), (g, r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 2, 2), (2, 7, 5), (1, 31, 31), (4, 33, 32), (5, 1000, 20), (3, 4099, 32),
                                   (1, 32000, 5), (9, 32001, 1), (400, 513, 3), (2, 128256, 20), (1, 131072, 32),
                                   (7, 50257, 0)])
def test_token_logprobs(T, V, k, dtype):
    g = torch.Generator().manual_seed(T * V + k)
    x = (torch.randn((T, V), generator=g) * 2.5).to(dtype)
    tokens = torch.randint(0, V, (T,), generator=g).tolist()
    tokens[-1] = int(x[-1].float().argmax())
    cut = sorted(torch.randint(0, T + 1, (2,), generator=g).tolist())
    off = [0] + cut + [T]
    tau = [0.7, 1.0, 2.5]
    out, status = _tokens_call(x.cuda(), tokens, off, tau, k)
    assert status == [0, 0, 0]
    for i in list(range(min(T, 6))) + [T - 1]:
        b = sum(i >= c for c in cut)
        _check(x[i].double().numpy(), out, i, tokens[i], float(np.float32(tau[b])), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_ties_masks_and_rows_without_a_distribution(dtype):
    V, k = 5000, 32
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(4)
    rows, tokens = [], []

    def add(row, token):
        rows.append(row)
        tokens.append(token)
    add(torch.zeros(V), 4999)                                            # all equal
    add(torch.randint(-3, 4, (V,), generator=g).float(), 17)             # many ties
    x = torch.full((V,), -math.inf)
    x[[70, 4097, 12]] = torch.tensor([1.0, 2.0, 2.0])
    add(x, 70)                                                           # three tokens left
    add(x.clone(), 5)                                                    # a masked token: -inf
    x = torch.full((V,), low)
    x[4000] = 0.5
    add(x, 3)                                                            # masked by the type's lowest value
    add(torch.full((V,), -math.inf), 9)                                  # nothing left: no distribution
    add(torch.full((V,), low), 9)                                        # every entry the lowest value: uniform
    x = torch.randn(V, generator=g)
    x[[3, 44, 4500]] = math.nan
    add(x, 44)                                                           # NaN ranks last
    x = torch.randn(V, generator=g)
    x[[8, 9]] = math.inf
    add(x, 9)
    x = torch.zeros(V)
    x[100:200] = -0.0
    add(x, 150)                                                          # -0 equals +0
    add(torch.arange(V).float(), 0)                                      # ascending: every entry enters the list
    add(torch.randn(V, generator=g), -1)                                 # no token given
    xs = torch.stack(rows).to(dtype)
    out, status = _tokens_call(xs.cuda(), tokens, [0, len(rows)], None, k)
    assert status == [0]
    for i in range(len(rows)):
        _check(xs[i].double().numpy(), out, i, tokens[i], 1.0, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_ties_and_what_is_not_finite_far_from_the_token(dtype):
    """Ranks over whole stages of lower and of higher ids than the token's."""
    V, k = 20000, 7
    g = torch.Generator().manual_seed(8)
    zeros = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    mixed = torch.randn(V, generator=g)
    mixed[torch.randint(0, V, (300,), generator=g)] = math.nan
    some = torch.randn(V, generator=g)
    some[torch.randint(0, V, (9000,), generator=g)] = -math.inf
    some[17000:] = -math.inf
    tiny = torch.randint(-2, 3, (V,), generator=g).float() * 2.0 ** -149
    high = torch.randn(V, generator=g)
    high[[40, 9000, 19000]] = math.inf
    rows, tokens = [], []
    for row in (zeros, mixed, some, tiny, high):
        for t in (3, 12001, 19999):
            rows.append(row)
            tokens.append(t)
    rows.append(high)
    tokens.append(9000)
    xs = torch.stack(rows).to(dtype)
    out, status = _tokens_call(xs.cuda(), tokens, [0, len(rows)], None, k)
    assert status == [0]
    for i in range(len(rows)):
        _check(xs[i].double().numpy(), out, i, tokens[i], 1.0, k)


def test_bad_tokens_and_temperatures():
    x = torch.randn((6, 300), generator=torch.Generator().manual_seed(1))
    out, status = _tokens_call(x.cuda(), [1, 300, -2, 4, 5, 6], [0, 3, 4, 5], [1.0, 0.0, math.inf], 3)
    assert status == [S.SPEC_DEV_BAD_TOKEN, S.SPEC_DEV_BAD_TEMP, S.SPEC_DEV_BAD_TEMP]
    _check(x[0].double().numpy(), out, 0, 1, 1.0, 3)
    for i in (1, 2, 3, 4, 5):  # flagged entries, and row 5 that no request owns
        assert math.isnan(out[0][i].item()) and math.isnan(out[1][i].item()) and out[2][i].item() == -1
        assert out[3][i].tolist() == [-1] * 3 and all(map(math.isnan, out[4][i].tolist()))


@pytest.mark.parametrize("V", [40, 9000], ids=["one_warp", "many"])
@pytest.mark.parametrize("tau,low", [(1e-30, -1e31), (1e-30, -1e30), (1e-30, -3e38), (3.4e38, -1e9), (3.4e38, -math.inf)])
def test_temperatures_at_the_ends_of_their_range(tau, low, V):
    """Masked logits that still weigh at the smallest inverse temperature, before
    and behind the unmasked ones, and products that overflow at the largest."""
    x = torch.full((3, V), low)
    x[0, :2], x[1, V - 3:], x[2, V // 2] = 1.0, 2.0, -0.5
    tokens, k = [1, 0, V // 2], 5
    out, status = _tokens_call(x.cuda(), tokens, [0, 3], [tau], k)
    assert status == [0]
    for i, t in enumerate(tokens):
        row, f = x[i].double().numpy(), float(np.float32(tau))
        lp, ent, rank, top, top_lp = logprob_reference(row, t, f, k)
        if tau > 1.0:  # beyond fp32: minus infinity there
            lp, top_lp = (np.where(v < -3.4e38, -math.inf, v) for v in (lp, top_lp))
        got = [o[i].cpu() for o in out]
        for g, r in [(got[0].item(), lp), (got[1].item(), ent)] + list(zip(got[4].tolist(), top_lp)):
            assert g == r or abs(g - r) <= _tolerance(row, f, r) * (1 + math.log(V)), (g, r)
        assert got[2].item() == rank and got[3].tolist() == list(top)


def test_optional_outputs_and_alignment():
    """Rows that start anywhere, and calls that want the log probability alone."""
    for dtype in (torch.float32, torch.bfloat16):
        V = 1003
        base = torch.randn(5 * V + 1, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
        x = base[1:].view(5, V)
        out, status = _tokens_call(x, [0, 1002, 500, 501, 7], [0, 5], None, 4)
        for i, t in enumerate([0, 1002, 500, 501, 7]):
            _check(x[i].cpu().double().numpy(), out, i, t, 1.0, 4)
        lp = torch.zeros(5, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        S.spec_token_logprobs(x, torch.tensor([0, 1002, 500, 501, 7], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, 5], dtype=torch.int32, device="cuda"), None, 1, 5, V, 0, lp, None, None,
                              None, None, st)
        assert torch.equal(lp, out[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_path_logprobs(dtype):
    g = np.random.default_rng(6)
    sizes, V, k, n_max = [5, 1, 0, 40, 12, 7], 777, 6, 41
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    B, T = len(sizes), int(off[-1])
    x = torch.from_numpy(g.standard_normal((T, V)).astype(np.float32)).to(dtype)
    acc = np.array([3, 1, 0, 9, 12, 2], np.int32)
    path = np.full((B, n_max), -1, np.int32)
    emitted = np.full((B, n_max), -1, np.int32)
    for b in range(B):
        if acc[b]:
            rest = g.choice(np.arange(1, max(2, sizes[b])), acc[b] - 1, replace=False)
            path[b, :acc[b]] = [0] + sorted(rest.tolist())
        emitted[b, :acc[b]] = g.integers(0, V, acc[b])
    path[5, 1] = 7       # outside the request's tree
    emitted[3, 4] = V    # outside the vocabulary
    out = _outputs((B, n_max), k)
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    S.spec_path_logprobs(x.cuda(), c(off), c(path), c(acc), c(emitted), None, B, T, n_max, V, k, *out, status)
    assert status.tolist() == [0, 0, 0, S.SPEC_DEV_BAD_TOKEN, 0, S.SPEC_DEV_BAD_PATH]
    for b in range(B):
        for i in range(n_max):
            if i >= acc[b] or (b, i) in ((5, 1), (3, 4)):
                assert math.isnan(out[0][b, i].item()) and math.isnan(out[1][b, i].item()) and out[2][b, i].item() == -1
                assert out[3][b, i].tolist() == [-1] * k and all(map(math.isnan, out[4][b, i].tolist()))
            else:
                _check(x[off[b] + path[b, i]].double().numpy(), [o[b] for o in out], i, int(emitted[b, i]), 1.0, k)


def test_logprobs_repeat_and_replay():
    x = torch.randn((64, 32000), device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    tokens = list(range(64))
    a, _ = _tokens_call(x, tokens, [0, 64], None, 20)
    b, _ = _tokens_call(x, tokens, [0, 64], None, 20)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    out, st = _outputs((64,), 20), torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.spec_token_logprobs(x, tok, off, None, 1, 64, 32000, 20, *out, st)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _tokens_call(x, tokens, [0, 64], None, 20)
    assert all(torch.equal(p, q) for p, q in zip(out, want))


@pytest.mark.parametrize("B,V,k", [(1, 40000, 7), (1100, 60, 3), (30, 9000, 32)])
def test_path_logprobs_in_every_launch_shape(B, V, k):
    """One request spread over a cluster, more requests than a CTA numbers for
    itself, and rounds of several entries per CTA; each with entries that are
    left out in the middle."""
    g = np.random.default_rng(B)
    n_max = 6
    sizes = g.integers(1, n_max + 1, B)
    sizes[0] = n_max
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    T = int(off[-1])
    x = torch.from_numpy(g.standard_normal((T, V)).astype(np.float32) * 3)
    acc = np.array([int(g.integers(0, s + 1)) for s in sizes], np.int32)
    acc[0] = n_max
    path = np.full((B, n_max), -1, np.int32)
    emitted = np.full((B, n_max), -1, np.int32)
    for b in range(B):
        path[b, :acc[b]] = np.arange(acc[b])
        emitted[b, :acc[b]] = g.integers(0, V, acc[b])
    path[0, 2], emitted[0, 4] = sizes[0], -1   # a node outside the tree, and no token
    if B > 2:
        acc[B - 1] = n_max + 1                 # more accepted nodes than there can be
    tau = g.uniform(0.5, 2.0, B).astype(np.float32)
    out, status = _outputs((B, n_max), k), torch.zeros(B, dtype=torch.int32, device="cuda")
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    S.spec_path_logprobs(x.cuda(), c(off), c(path), c(acc), c(emitted), c(tau), B, T, n_max, V, k, *out, status)
    want = [0] * B
    want[0] = S.SPEC_DEV_BAD_PATH | S.SPEC_DEV_BAD_TOKEN
    if B > 2:
        want[B - 1] = S.SPEC_DEV_BAD_PATH
    assert status.tolist() == want
    host = [o.cpu() for o in out]
    for b in list(range(min(B, 25))) + [B - 1]:
        for i in range(n_max):
            if i >= acc[b] or acc[b] > n_max or (b == 0 and i in (2, 4)):
                assert math.isnan(host[0][b, i].item()) and host[2][b, i].item() == -1 and host[3][b, i].tolist() == [-1] * k
            else:
                _check(x[off[b] + path[b, i]].double().numpy(), [o[b] for o in host], i, int(emitted[b, i]), float(tau[b]), k)


def test_arguments_of_other_types_are_refused():
    x = torch.zeros((2, 8), device="cuda")
    off, st = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lp = torch.zeros(2, device="cuda")
    tok = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(tok=tok.long()), dict(lp=lp.double()), dict(x=x.half())):
        a = dict(x=x, tok=tok, lp=lp)
        a.update(bad)
        with pytest.raises(ValueError):
            S.spec_token_logprobs(a["x"], a["tok"], off, None, 1, 2, 8, 0, a["lp"], None, None, None, None, st)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V,nans,masked", [
    (7, [2], []), (7, [0], []), (1003, [100], []), (1003, [0], []), (1003, [1002], []), (4300, [5], []), (4300, [4200], []),
    (12288, [5], [(4096, 8192)]), (12288, [4095], [(4096, 12288)]), (12288, [12287], [(0, 12287)]),
    (131072, [5], [(4096, 8192)]), (131072, [131071], [(0, 131071)]), (131072, [16390], [(16391, 131072)]), (50, list(range(50)), [])])
def test_one_nan_among_masked_logits(V, nans, masked, dtype):
    """A NaN leaves the row without a distribution, whatever stands behind it: the
    row's tail, the end of a partly filled stage, entries of -inf; rows that
    start anywhere, and rows alone in their call (spread over a cluster when
    they are long) or among others."""
    g = torch.Generator().manual_seed(V + len(nans) + len(masked))
    rows = torch.randn((3, V), generator=g)
    for a, b in masked:
        rows[0, a:b] = rows[2, a:b] = -math.inf
    rows[0, nans] = rows[2, nans] = math.nan
    base = torch.zeros(3 * V + 8, dtype=dtype)
    k = min(V, 9)
    for shift in (0, 1, 3):
        base[shift:shift + 3 * V] = rows.to(dtype).flatten()
        x = base.cuda()[shift:shift + 3 * V].view(3, V)
        for first, n in ((0, 3), (0, 1), (2, 1)):
            tokens = [(nans[0] + i) % V for i in range(n)]
            out, status = _tokens_call(x[first:first + n], tokens, [0, n], None, k)
            assert status == [0]
            for i in range(n):
                row = x[first + i].cpu().double().numpy()
                _check(row, out, i, tokens[i], 1.0, k)
                assert math.isnan(out[0][i].item()) == (first + i != 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_logits_beyond_32_bit_offsets(dtype):
    """Rows behind the first 2^31 elements, of the packed call and of the path's."""
    V, k = 131071, 3
    T = (1 << 31) // V + 7
    x = torch.zeros((T, V), dtype=dtype, device="cuda")
    last = torch.randn((6, V), generator=torch.Generator().manual_seed(5)).to(dtype)
    x[-6:] = last.cuda()
    tokens = [0] * (T - 6) + [V - 1, 7, 0, 65536, 99, 100]
    out, status = _tokens_call(x, tokens, [0, 11, T], [1.0, 0.5], k)
    assert status == [0, 0]
    for i in range(6):
        _check(last[i].double().numpy(), out, T - 6 + i, tokens[T - 6 + i], 0.5, k)
    c = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out, status = _outputs((2, 4), k), c([0, 0])
    S.spec_path_logprobs(x, c([0, T - 6, T]), c([[0, 1, -1, -1], [0, 2, 3, 5]]), c([2, 4]), c([[4, 5, -1, -1], [8, 9, 10, V - 1]]), None, 2,
                         T, 4, V, k, *out, status)
    assert status.tolist() == [0, 0]
    for i, (r, t) in enumerate(((0, 8), (2, 9), (3, 10), (5, V - 1))):
        _check(last[r].double().numpy(), [o[1] for o in out], i, t, 1.0, k)
    _check(np.zeros(V), [o[0] for o in out], 1, 5, 1.0, k)


def test_packing_that_starts_behind_row_zero():
    x = torch.randn((9, 500), generator=torch.Generator().manual_seed(6))
    out, status = _tokens_call(x.cuda(), list(range(9)), [3, 3, 8], [9.0, 2.0], 4)
    assert status == [0, 0]
    for i in range(9):
        if 3 <= i < 8:
            _check(x[i].double().numpy(), out, i, i, 2.0, 4)
        else:
            assert math.isnan(out[0][i].item()) and out[2][i].item() == -1 and out[3][i].tolist() == [-1] * 4


def test_calls_on_two_streams_at_once():
    """A spread row and many rows side by side, several times over: the same bits."""
    xs = [torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(s[0])) for s in ((1, 131072), (300, 32000))]
    ref = [_tokens_call(x, list(range(len(x))), [0, len(x)], None, 20)[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    args = [(torch.arange(len(x), dtype=torch.int32, device="cuda"), torch.tensor([0, len(x)], dtype=torch.int32, device="cuda"),
             torch.zeros(1, dtype=torch.int32, device="cuda")) for x in xs]
    outs = [[_outputs((len(x),), 20) for _ in range(4)] for x in xs]
    torch.cuda.synchronize()
    for i in range(4):
        for x, s, (tok, off, st), o in zip(xs, streams, args, outs):
            S.spec_token_logprobs(x, tok, off, None, 1, len(x), x.shape[1], 20, *o[i], st, stream=s)
    torch.cuda.synchronize()
    for r, o in zip(ref, outs):
        assert all(torch.equal(p, q) for one in o for p, q in zip(r, one))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V,k,T", [(9013, 2, 300), (9013, 3, 450), (4096, 2, 400), (30000, 2, 150), (9013, 5, 222), (70000, 20, 60)])
def test_alternatives_while_every_warp_finds_better_ones(V, k, T, dtype):
    """Rows that rise towards their end, so that the bars move with every entry
    while other warps read them: the same list in each of many calls."""
    g = torch.Generator().manual_seed(V + k)
    ramp = torch.linspace(0, 8, V)[None] + torch.randn((T, V), generator=g) * torch.rand((T, 1), generator=g) * 4
    ramp[::5] = torch.linspace(0, 8, V)[None]
    x = ramp.to(dtype).cuda()
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)  # equal ones by lower id
    tok, off = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), _outputs((T,), k)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        out[3].fill_(-7)
        S.spec_token_logprobs(x, tok, off, None, 1, T, V, k, *out, st)
        wrong += (out[3] != order).any(1).sum()
    assert st.tolist() == [0] and wrong.item() == 0
