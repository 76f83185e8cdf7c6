"""Calls of a bounded cache at the edges of what their arguments may say:
against plain implementations in 64 bits."""
import threading

import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from bounded_cache import ints
from request_life import paged_batch
from test_bounded_cache_gpu import DTYPES, _before, _weight, _weight_holds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


@DTYPES
@pytest.mark.parametrize("T,n_max", [(0, 512), (0, 4000), (7, 0), (0, 0)])
def test_weight_decays_where_a_batch_cannot_have_rows(T, n_max, dtype):
    """Rows of q outside every request, or a fixed n_max without a row of q."""
    d = paged_batch(80, [1, 1, 1], [300, 5, 9000], 8, 2, 64, 16, dtype, extra_rows=9)
    before = _before(d)
    d.update(q=d["q"][:T], seq_off=ints([0] * 4), T=T)
    got, st = _weight(d, before, n_max=n_max)
    assert not st.any()
    _weight_holds(d, got, before)


@DTYPES
def test_weight_flags_rows_that_the_batch_cannot_have(dtype):
    d = paged_batch(81, [1, 1, 1], [300, 5, 900], 8, 2, 64, 16, dtype)
    before = _before(d)
    # without a row of q, the last request starts behind T
    for T, n_max, bad in ((0, 512, (1, 2)), (3, 0, (1,))):
        d.update(T=T, seq_off=ints([0, 0, 1, 1]))
        got, st = _weight(d, before, n_max=n_max)
        assert st.tolist() == [S.SPEC_DEV_BAD_TREE if b in bad else 0 for b in range(3)]
        _weight_holds({**d, "seq_off": ints([0, 0, 0, 0])}, got, before, skip=bad)


def test_evict_from_two_threads():
    """Tables of different widths want different amounts of shared memory: neither
    thread's may be taken for the other's."""
    def work(width, out):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                cache = torch.zeros((2, 4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
                k, v = (torch.tensor([c.data_ptr()], dtype=torch.int64, device="cuda") for c in cache)
                table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
                table[0, :2], table[1, 0] = ints([0, 1]), 2
                weight = torch.rand((1, 2, 1, width * 16), device="cuda")
                src, dst, length = ints([0]), ints([1]), ints([20])
                slots, new_len, status = torch.empty((1, 1, 1, 8), dtype=torch.int32, device="cuda"), ints([0]), ints([0])
                stream.synchronize()
                for _ in range(4000):
                    S.spec_kv_evict(k, v, 1, table, 2, width, 16, 4, src, dst, length, None, 1, 8, 1, 2, weight, width * 16, 1, 64, S.SPEC_BF16, slots, new_len,
                                    status)
                stream.synchronize()
                out.append((new_len.tolist(), status.tolist()))
        except Exception as e:
            out.append(repr(e))
    outs = [[], []]
    threads = [threading.Thread(target=work, args=a) for a in zip((3000, 600), outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert outs == [[([8], [0])]] * 2


@pytest.mark.parametrize("window", [0, 40])
def test_weight_under_a_wide_bound_of_rows(window):
    """n_max says what a request may have at most, not what a batch of a thousand has."""
    lens = [(i * 7) % 3 for i in range(1200)]
    lens[700], lens[1199] = 300, 41
    d = paged_batch(82, lens, [(i * 5) % 40 for i in range(1200)], 64, 8, 64, 16, torch.bfloat16, extra_rows=1)
    before = _before(d)
    got, st = _weight(d, before, n_max=1 << 20, window=window)
    assert not st.any()
    _weight_holds(d, got, before, window=window)


@DTYPES
@pytest.mark.parametrize("spread", [6.0, 40.0])
@pytest.mark.parametrize("Hq,lens,prefix", [(32, [1, 2], [2000, 300]), (16, [3, 8], [900, 3000]), (32, [8, 1, 4], [100, 30, 20000])], ids=["short", "rows", "long"])
def test_weight_few_wide_rows_with_steep_scores(Hq, lens, prefix, spread, dtype):
    """Heads of 128, sums that leave the middle of 32 bits: a second look at the rows."""
    d = paged_batch(83, lens, prefix, Hq, 4, 128, 16, dtype, spread=spread)
    before = _before(d)
    got, st = _weight(d, before)
    assert not st.any()
    _weight_holds(d, got, before)


def test_weight_two_graphs_with_a_workspace_each():
    """Captured passes of two streams replayed at once."""
    ds = [paged_batch(s, lens, prefix, 8, 2, 64, 16, torch.bfloat16) for s, lens, prefix in ((84, [2, 40], [3000, 200]), (85, [300], [50]))]
    befores, outs, graphs, keep = [_before(d) for d in ds], [], [], []
    for d, before in zip(ds, befores):
        size = (d["B"], d["T"], d["n_max"], d["max_prefix"], 8, 2, 64)
        ws = torch.empty(S.spec_weight_workspace_size(*size), dtype=torch.uint8, device="cuda")
        out, st = torch.full_like(before, 7.0), ints([0] * d["B"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            S.spec_attention_weight(d["q"], d["k"], d["table"], d["table"].shape[1], 16, d["nb"], d["prefix"], d["seq_off"], None, None, 0, *size, d["scale"], 0.75,
                                    before, out, out.shape[-1], ws, st)
        outs.append((out, st))
        graphs.append(graph)
        keep.append(ws)
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for d, before, (out, st) in zip(ds, befores, outs):
        assert not st.any()
        _weight_holds(d, out, before)
