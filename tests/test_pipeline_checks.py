"""What the pipeline hands to the C ABI, without a GPU: the calls are recorded
in place of the library's, and the buffers they would read are looked at."""
import pytest
import torch

from tree_speculative_verification_spec_gb300 import pipeline
from tree_speculative_verification_spec_gb300.pipeline import DeviceBatch, Rotary, VerifyPass

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
AXIS, POS_BASE, POS, AXES = 5, 8, 9, 10


def _verify_pass(nodes=(3, 2)):
    T, cache = sum(nodes), torch.zeros((8, Hkv, BS, D))
    off = ints([0] + [sum(nodes[:i + 1]) for i in range(len(nodes))])
    return VerifyPass(DeviceBatch(B=len(nodes), T=T, n_max=max(nodes), V=7, Hq=Hq, Hkv=Hkv, D=D, block_size=BS, num_blocks=8, max_prefix=9,
                                  parent=ints([-1, 0, 1, -1, 0]), tree_off=off, tokens=ints([0] * T), prefix_len=ints([9, 4]), block_table=ints([[0, 1], [2, 3]]),
                                  q=torch.zeros((T, Hq, D)), k_cache=cache, v_cache=cache, p_logits=torch.zeros((T, 7)), q_probs=None, uniforms=None, scale=0.1))


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_project_names_a_position_for_every_axis_it_asks_for(calls, axes):
    """A pair of axis a reads pos[a * T + row]: there has to be one, and it is the
    node's depth whatever the axis."""
    v = _verify_pass()
    v.depth[:] = ints([0, 1, 2, 0, 1])
    axis = ints([i % axes for i in range(D // 2)]) if axes > 1 else None
    rotary = Rotary(torch.ones(D // 2), D, axis=axis, axes=axes)
    base = ints([100, 200])
    v.project(torch.zeros((5, Hq + 2 * Hkv, D)), rotary, base)
    (args,) = [a for n, a, _ in calls if n == "spec_rope_append"]
    pos, T = args[POS].reshape(-1), v.batch.T
    assert pos.numel() >= args[AXES] * T
    for a in set(range(1) if args[AXIS] is None else args[AXIS].tolist()):
        assert 0 <= a < args[AXES]
        assert pos[a * T:(a + 1) * T].tolist() == [0, 1, 2, 0, 1]
    assert args[POS_BASE] is base and rotary.axes == axes and rotary.axis is axis
