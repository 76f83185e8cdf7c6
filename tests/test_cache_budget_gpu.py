"""A bounded cache through the pipeline, where its parts meet: rotaries of
several axes, streams, workspaces and table rows."""
import math

import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from bounded_cache import ints, offsets, rope_reference, weight_reference
from test_request_life_gpu import Pool
from tree_speculative_verification_spec_gb300.pipeline import CacheBudget, DeviceBatch, PromptPass, Rotary, VerifyPass

pytestmark = pytest.mark.gpu
Hq, Hkv, D, BS = 8, 2, 64, 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


def _randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("axes", [1, 3])
def test_a_tree_behind_a_prompt_of_several_axes(axes):
    """An image's prompt, then a verification of text: one rotary for both."""
    n, parent = 40, [-1, 0, 0, 2, 1]
    g = torch.Generator().manual_seed(3)
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    axis = torch.randint(0, axes, (D // 2,), generator=g).to(torch.int32).cuda() if axes > 1 else None
    rotary = Rotary(freq, D, axis=axis, axes=axes)
    pos = torch.randint(0, 500, (axes, n), generator=g).to(torch.int32).cuda()
    kc, vc = (torch.zeros((6, Hkv, BS, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, zero, scale = ints([[4, 1, 3]]), ints([0]), 1 / math.sqrt(D)

    def holds(qkv, q, place, first):
        ref, tol = rope_reference(qkv, Hq, Hkv, D, 0, freq, place, None, None, 0.0)
        assert ((q.double() - ref[:, :Hq]).abs() <= tol[:, :Hq]).all()
        for h in range(Hkv):
            k = kc[table[0].long(), h].reshape(-1, D)[first:first + len(qkv)]
            assert ((k.double() - ref[:, Hq + h]).abs() <= tol[:, Hq + h]).all()

    qkv = _randn((n, Hq + 2 * Hkv, D), 1)
    p = PromptPass(torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda"), kc, vc, table, offsets([n]), zero, n, 0, scale)
    p.run(prompt_qkv=qkv, rotary=rotary, pos_base=zero, pos=pos)
    assert p.status.tolist() == [0]
    holds(qkv, p.q, pos.t()[:, axis.long()] if axes > 1 else pos.t().expand(-1, D // 2), 0)

    T, qkv = len(parent), _randn((len(parent), Hq + 2 * Hkv, D), 2)
    v = VerifyPass(DeviceBatch(B=1, T=T, n_max=T, V=7, Hq=Hq, Hkv=Hkv, D=D, block_size=BS, num_blocks=6, max_prefix=n, parent=ints(parent),
                               tree_off=offsets([T]), tokens=ints([0] * T), prefix_len=ints([n]), block_table=table,
                               q=torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda"), k_cache=kc, v_cache=vc,
                               p_logits=torch.zeros((T, 7), device="cuda"), q_probs=None, uniforms=None, scale=scale))
    v.run("greedy", commit=False, tree_qkv=qkv, rotary=rotary, pos_base=ints([700]))
    assert v.status.tolist() == [0]
    depth = torch.tensor([0, 1, 1, 2, 2], device="cuda")
    holds(qkv, v.batch.q, (700 + depth)[:, None].expand(-1, D // 2), n)


def _observed(budget, lens, prefix, **kw):
    """A pass of rows in an empty cache, observed."""
    n = sum(lens)
    pages = -(-(max(lens) + max(prefix)) // BS)
    kc = torch.zeros((pages * len(lens), budget.Hkv, BS, D), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(pages * len(lens), dtype=torch.int32, device="cuda").view(len(lens), pages)
    p = PromptPass(torch.ones((n, Hq, D), dtype=torch.bfloat16, device="cuda"), kc, kc, table, offsets(lens), ints(prefix), max(lens), max(prefix), 0.125)
    if kw.get("stream") is not None:
        kw["stream"].wait_stream(torch.cuda.current_stream())
    budget.observe_prompt(0, p, **kw)
    return p


def test_a_reserved_workspace_serves_smaller_passes():
    """Captured with less rows and keys than were reserved: nothing is allocated."""
    budget = CacheBudget(1, 64, Hkv, 8192)
    budget.reserve(64, 512, 300, 4096, Hq, D)
    ws = budget._ws.data_ptr()
    for lens, prefix in (([1], [4096]), ([1] * 8, [4000] * 8), ([300], [0]), ([300], [4096]), ([8] * 64, [100] * 64), ([300, 200], [5, 3000])):
        p = _observed(budget, lens, prefix)
        _observed(budget, lens, prefix, window=1)
        assert budget._ws.data_ptr() == ws and not p.status.any()


def _stream_of_memory(t):
    """The stream whose pool a tensor's memory is from."""
    at = t.data_ptr()
    return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]


def test_a_workspace_is_the_observing_streams_own():
    """Memory of another stream may still be written by what was queued there."""
    budget, side = CacheBudget(1, 64, Hkv, 8192), torch.cuda.Stream()
    for lens, prefix in (([5], [0]), ([300], [4000])):
        p = _observed(budget, lens, prefix, stream=side)
        side.synchronize()
        assert not p.status.any()
        assert _stream_of_memory(budget._ws) == [side.cuda_stream]
    budget.reserve(64, 4096, 4000, 8000, Hq, D, stream=side)
    assert _stream_of_memory(budget._ws) == [side.cuda_stream]
    with torch.cuda.stream(side):
        again = CacheBudget(1, 64, Hkv, 8192)
        _observed(again, [5], [0])
        assert _stream_of_memory(again._ws) == [side.cuda_stream]
    side.synchronize()


@pytest.mark.parametrize("captured", [False, True])
def test_forked_rows_go_on_from_their_weights(captured):
    """A prompt, two forks of it and a flagged one, a chunk on both: what they
    gather decays what the prompt gave, not what the rows held before."""
    n, chunk = 50, [3, 7]
    budget = CacheBudget(1, 4, Hkv, 6 * BS, decay=0.5)
    pool = Pool(4, 6, 30, Hkv, BS, D, 1)
    kc, vc = pool.caches[0]
    pool.fork([-1], [0], [0], [n])
    p = PromptPass(_randn((n, Hq, D), 1), kc, vc, pool.table[:1], offsets([n]), ints([0]), n, 0, 0.125)
    p.run((_randn((n, Hkv, D), 2), _randn((n, Hkv, D), 3)))
    budget.weight.fill_(5.0)
    budget.observe_prompt(0, p)
    src, dst, length, room, st = ints([0, 0, 9]), ints([1, 2, 3]), ints([n, n, 0]), ints(chunk + [0]), ints([77] * 3)
    S.spec_pages_fork(pool.k, pool.v, 1, pool.table, *pool.shape, src, dst, length, room, 3, Hkv, D, S.SPEC_BF16, pool.pool, pool.count, pool.ws, st)
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            budget.fork(src, dst, st)
        graph.replay()
    else:
        budget.fork(src, dst, st)
    assert st.tolist() == [0, 0, S.SPEC_DEV_BAD_ROW]
    before = budget.weight[0, 0].clone()
    assert torch.equal(budget.weight[0, 1], before) and torch.equal(budget.weight[0, 2], before) and (budget.weight[0, 3] == 5.0).all()
    c = PromptPass(_randn((sum(chunk), Hq, D), 4), kc, vc, pool.table[1:3], offsets(chunk), ints([n, n]), max(chunk), n, 0.125)
    c.run((_randn((sum(chunk), Hkv, D), 5), _randn((sum(chunk), Hkv, D), 6)))
    budget.observe_prompt(0, c, row=1)
    assert c.status.tolist() == [0, 0] and torch.equal(budget.weight[0, 0], before)
    d = dict(q=c.q, k=kc, table=pool.table[1:3], seq_off=c.seq_off, prefix=c.prefix_len, Hq=Hq, Hkv=Hkv, D=D, bs=BS, scale=0.125)
    ref, tol = weight_reference(d, torch.stack([before] * 2), 0.5)
    mine = ~ref.isnan()
    assert ((budget.weight[0, 1:3].double() - ref).abs()[mine] <= tol[mine]).all()
