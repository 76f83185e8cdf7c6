"""What the pipeline hands to the C ABI, without a GPU: the calls are recorded
in place of the library's, and the buffers they would read are looked at."""
import pytest
import torch

from tree_speculative_verification_spec_gb300 import pipeline
from tree_speculative_verification_spec_gb300.pipeline import CacheBudget, DeviceBatch, Rotary, VerifyPass

Hq, Hkv, D, BS = 4, 2, 64, 16


def ints(v):
    return torch.tensor(v, dtype=torch.int32)


class Calls(list):
    """Stands for the binding: calls are recorded, sizes are one small number."""
    SPEC_ATTN_AUTO = SPEC_Q_PER_PARENT = SPEC_ROPE_HALVES = 0
    RETURNS = 256

    def __getattr__(self, name):
        def call(*args, **kw):
            self.append((name, args, kw))
            return self.RETURNS
        return call


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(pipeline, "S", c)
    return c


# places of spec_rope_append's arguments
AXIS, POS_BASE, POS, AXES, ROWS = 5, 8, 9, 10, 21


def _verify_pass(nodes=(3, 2), extra=0):
    T, cache = sum(nodes), torch.zeros((8, Hkv, BS, D))
    off = ints([0] + [sum(nodes[:i + 1]) for i in range(len(nodes))])
    return VerifyPass(DeviceBatch(B=len(nodes), T=T, n_max=max(nodes), V=7, Hq=Hq, Hkv=Hkv, D=D, block_size=BS, num_blocks=8, max_prefix=9,
                                  parent=ints([-1, 0, 1, -1, 0]), tree_off=off, tokens=ints([0] * T), prefix_len=ints([9, 4]), block_table=ints([[0, 1], [2, 3]]),
                                  q=torch.zeros((T + extra, Hq, D)), k_cache=cache, v_cache=cache, p_logits=torch.zeros((T, 7)), q_probs=None, uniforms=None, scale=0.1))


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_project_names_a_position_for_every_axis_it_asks_for(calls, axes):
    """A pair of axis a reads pos[a * T + row]: there has to be one, and it is the
    node's depth whatever the axis."""
    v = _verify_pass(extra=axes % 2)  # q may be longer than the batch
    v.depth[:] = ints([0, 1, 2, 0, 1])
    axis = ints([i % axes for i in range(D // 2)]) if axes > 1 else None
    rotary = Rotary(torch.ones(D // 2), D, axis=axis, axes=axes)
    base = ints([100, 200])
    v.project(torch.zeros((5, Hq + 2 * Hkv, D)), rotary, base)
    (args,) = [a for n, a, _ in calls if n == "spec_rope_append"]
    pos, T = args[POS].reshape(-1), v.batch.T
    assert pos.numel() >= args[AXES] * T
    assert args[ROWS] == T
    for a in set(range(1) if args[AXIS] is None else args[AXIS].tolist()):
        assert 0 <= a < args[AXES]
        assert pos[a * T:(a + 1) * T].tolist() == [0, 1, 2, 0, 1]
    assert args[POS_BASE] is base and rotary.axes == axes and rotary.axis is axis


def _append(calls, T=5, B=2, rot=D, **change):
    """Rotary.append over T rows, with one buffer changed."""
    kw = dict(qkv=torch.zeros((T, Hq + 2 * Hkv, D)), inv_freq=torch.ones(rot // 2), axis=None, axes=1, pos_base=None, pos=None, q_norm=None, k_norm=None)
    kw.update(change)
    cache = torch.zeros((8, Hkv, BS, D))
    rotary = Rotary(kw["inv_freq"], rot, axis=kw["axis"], axes=kw["axes"], q_norm=kw["q_norm"], k_norm=kw["k_norm"])
    rotary.append(kw["qkv"], torch.zeros((T, Hq, D)), cache, cache, ints([[0, 1]] * B), ints([0] * B), ints([0] * (B + 1)), T, ints([0] * B), kw["pos_base"],
                  kw["pos"])
    return calls[-1][1]


AXIS3 = dict(axis=ints([0, 1, 2] * 10 + [0, 1]), axes=3)


@pytest.mark.parametrize("change", [
    dict(pos=ints([[0] * 5] * 2), **AXIS3), dict(pos=ints([0] * 14), **AXIS3), dict(pos=ints([[0] * 6] * 3), **AXIS3),
    dict(pos=ints([[0] * 5] * 3), axis=ints([0] * 31), axes=3), dict(pos_base=ints([0])),
    dict(qkv=torch.zeros((4, Hq + 2 * Hkv, D)), pos=ints([[0] * 5] * 3), **AXIS3),
    dict(qkv=torch.zeros((5, Hq + Hkv, D))), dict(qkv=torch.zeros((5, 511))), dict(inv_freq=torch.ones(31)), dict(q_norm=torch.ones(63)), dict(k_norm=torch.ones(32))],
    ids=["pos of two axes", "flat pos", "pos of other rows", "axis", "pos_base", "qkv", "heads", "width", "inv_freq", "q_norm", "k_norm"])
def test_append_refuses_buffers_that_end_early(calls, change):
    with pytest.raises(ValueError):
        _append(calls, **change)
    assert not calls


@pytest.mark.parametrize("change", [
    dict(), dict(pos=ints([0] * 5)), dict(pos=ints([[0] * 5])), dict(pos=ints([0] * 9)), dict(pos=ints([[0] * 5] * 3), **AXIS3), dict(pos=ints([0] * 15), **AXIS3),
    dict(pos=ints([[0] * 5] * 4), **AXIS3), dict(pos_base=ints([0, 0])), dict(pos_base=ints([0] * 9)), dict(qkv=torch.zeros((9, (Hq + 2 * Hkv) * D))),
    dict(inv_freq=None, rot=0), dict(inv_freq=torch.ones(40)), dict(q_norm=torch.ones(64), k_norm=torch.ones(64))])
def test_append_takes_buffers_that_are_long_enough(calls, change):
    args = _append(calls, **change)
    assert args[POS] is change.get("pos") and args[POS_BASE] is change.get("pos_base") and args[ROWS] == 5


@pytest.mark.parametrize("change,rows", [(dict(qkv=torch.zeros((4, Hq + 2 * Hkv, D))), 4), (dict(pos=ints([0] * 3)), 3), (dict(pos=ints([0] * 3), qkv=torch.zeros((2, 512))), 2)])
def test_append_asks_for_the_rows_that_every_buffer_has(calls, change, rows):
    """A q longer than the batch is no error; requests behind the rows are flagged by the call."""
    assert _append(calls, **change)[ROWS] == rows


@pytest.mark.parametrize("rows", [1, 3])
def test_evict_refuses_a_part_of_the_table(calls, rows):
    """Rows are checked against the budget's number of them: a slice of the table
    would be read behind its end."""
    budget = CacheBudget(1, 4, Hkv, 64, device="cpu")
    with pytest.raises(ValueError, match="rows"):
        budget.evict(None, None, ints([[0, 1]] * rows), BS, 8, ints([0]), ints([3]), ints([20]), 8, 0, 0, D, 0)
    assert not calls
    for whole in (4, 5):  # the rows behind the budget's are not named
        budget.evict(None, None, ints([[0, 1]] * whole), BS, 8, ints([0]), ints([3]), ints([20]), 8, 0, 0, D, 0)
    assert [n for n, _, _ in calls] == ["spec_kv_evict"] * 2


@pytest.mark.parametrize("change", [dict(dst=ints([3])), dict(length=ints([20])), dict(keep=ints([8]))])
def test_evict_refuses_lists_that_end_early(calls, change):
    budget = CacheBudget(1, 4, Hkv, 64, device="cpu")
    kw = dict(src=ints([0, 1]), dst=ints([2, 3]), length=ints([20, 20]), keep=None)
    kw.update(change)
    with pytest.raises(ValueError):
        budget.evict(None, None, ints([[0, 1]] * 4), BS, 8, kw["src"], kw["dst"], kw["length"], 8, 0, 0, D, 0, keep=kw["keep"])
    assert not calls


def test_a_budget_that_grows_slot_by_slot_keeps_little(calls):
    """Outgrown workspaces stay (a captured graph may still use them), so their sum
    has to stay near the last one's size."""
    budget, need = CacheBudget(1, 1, Hkv, 64, device="cpu"), 0
    for step in range(4800):
        need = calls.RETURNS = 512 * (step + 1)
        budget.reserve(1, 1, 1, step, Hq, D)
        assert budget._ws.numel() >= need
    assert budget._ws.numel() + sum(t.numel() for t in budget._outgrown) <= 4 * need
    kept = [t.data_ptr() for t in budget._outgrown] + [budget._ws.data_ptr()]
    budget.reserve(1, 1, 1, 0, Hq, D)
    assert [t.data_ptr() for t in budget._outgrown] + [budget._ws.data_ptr()] == kept


def test_a_first_reservation_is_exact(calls):
    calls.RETURNS = 1000
    budget = CacheBudget(1, 1, Hkv, 64, device="cpu")
    budget.reserve(1, 1, 1, 0, Hq, D)
    assert budget._ws.numel() == 1000


@pytest.mark.parametrize("src,dst,status,moved", [
    ([0], [3], None, {3: 0}), ([0, 0, 1], [2, 3, 4], None, {2: 0, 3: 0, 4: 1}), ([-1, 2], [0, 1], None, {1: 2}), ([1, 1], [1, 4], None, {4: 1}),
    ([0, 1, 2], [3, 4, 5], [0, 128, 0], {3: 0, 5: 2}), ([6, -2, 0, 1], [3, 4, 6, -1], None, {}), ([0, 7, 5], [9, 2, 0], None, {0: 5}), ([], [], None, {}),
    ([0, 1], [4, 5], [4, 4], {})])
def test_a_fork_takes_its_weights_along(src, dst, status, moved):
    """Rows that are no fork's, or a flagged one's, stay as they were."""
    budget = CacheBudget(2, 6, Hkv, 8, device="cpu")
    budget.weight.copy_(torch.rand(budget.weight.shape, generator=torch.Generator().manual_seed(1)))
    want = budget.weight.clone()
    for d, s in moved.items():
        want[:, d] = budget.weight[:, s]
    budget.fork(ints(src), ints(dst), None if status is None else ints(status))
    assert torch.equal(budget.weight, want)


def _prompt_pass():
    cache = torch.zeros((8, Hkv, BS, D))
    return pipeline.PromptPass(torch.zeros((5, Hq, D)), cache, cache, ints([[0, 1]]), ints([0, 5]), ints([0]), 5, 0, 0.1)


@pytest.mark.parametrize("kind", ["prompt", "tree"])
def test_a_pass_takes_rows_once(calls, kind):
    """Ready rows or a projection's: never both, and a projection with its rotary."""
    kv, qkv, rotary = (torch.zeros((5, Hkv, D)),) * 2, torch.zeros((5, Hq + 2 * Hkv, D)), Rotary()
    p, first = (_prompt_pass(), ()) if kind == "prompt" else (_verify_pass(), ("greedy",))
    calls.clear()
    for kw in ({f"{kind}_kv": kv, f"{kind}_qkv": qkv, "rotary": rotary}, {f"{kind}_qkv": qkv}, {f"{kind}_kv": kv, f"{kind}_qkv": qkv}):
        with pytest.raises(ValueError, match="qkv"):
            p.run(*first, **kw)
        assert not calls
    p.run(*first, **{f"{kind}_kv": kv})
    assert "spec_kv_append" in [n for n, _, _ in calls]
    calls.clear()
    p.run(*first, **{f"{kind}_qkv": qkv, "rotary": rotary})
    names = [n for n, _, _ in calls]
    assert "spec_rope_append" in names and "spec_kv_append" not in names
    calls.clear()
    p.run(*first, rotary=rotary)  # rows that are in the cache already
    names = [n for n, _, _ in calls]
    assert "spec_rope_append" not in names and "spec_kv_append" not in names
