"""Workspace of spec_attention_weight against its query, without a GPU: a call
whose workspace is too small says so before it looks for a device, one whose
workspace is large enough fails for want of a device."""
import ctypes
import random

import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from tree_speculative_verification_spec_gb300 import build

P = ctypes.c_void_p(1 << 20)  # stands for a device pointer that no call may touch here
# with a device the calls would go on to run on those pointers
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made for machines without a GPU")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def _call(size, ws_bytes, dtype=S.SPEC_BF16, window=0, path=False):
    B, T, n_max, max_prefix, Hq, Hkv, D = size
    return S.lib().spec_attention_weight(P, P, P, 1 << 16, 16, 1 << 10, P, P, P if path else None, n_max if path else 0, P if path else None, window, *size, dtype,
                                         0.1, 1.0, None, P, 1 << 20, P if ws_bytes else None, ws_bytes, P, None)


def _suffices(size, ws_bytes, **kw):
    code = _call(size, ws_bytes, **kw)
    assert code in (S.SPEC_ERR_CUDA, S.SPEC_ERR_WORKSPACE), code
    return code == S.SPEC_ERR_CUDA


DTYPES = pytest.mark.parametrize("dtype", [S.SPEC_BF16, S.SPEC_F32], ids=["bf16", "fp32"])


@DTYPES
@pytest.mark.parametrize("size", [(1, 0, 512, 1000, 8, 2, 64), (2, 100, 0, 1000, 8, 2, 64), (3, 0, 0, 9, 8, 2, 64), (4, 0, 4000, 0, 32, 8, 128), (4, 70, 0, 20000, 4, 4, 128)])
def test_batches_without_rows_need_no_more_than_the_query_says(size, dtype):
    """No request can have a row: nothing is put into the workspace."""
    assert _suffices(size, S.spec_weight_workspace_size(*size), dtype=dtype)
    assert _suffices(size, 0, dtype=dtype)


def _sizes(rng):
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 2), (4, 4), (6, 2), (5, 1), (96, 1), (200, 1), (8, 1)])

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    return (log(1, 400), log(1, 40000), log(1, 20000), rng.choice((0, log(1, 200000))), Hq, Hkv, rng.choice((64, 128)))


@pytest.mark.parametrize("seed", range(4))
def test_a_workspace_serves_every_call_of_no_larger_sizes(seed):
    """Whatever the batch, its window and its type: smaller ones split further."""
    rng = random.Random(seed)
    for _ in range(400):
        size = _sizes(rng)
        have = S.spec_weight_workspace_size(*size)
        for _ in range(6):
            less = tuple(rng.choice((x, rng.randint(0, x), min(x, 1))) for x in size[:4])
            less = (max(less[0], 1),) + less[1:] + size[4:]
            if less[2] + less[3] == 0:
                continue
            assert S.spec_weight_workspace_size(*less) <= have, (size, less)
            kw = dict(dtype=rng.choice((S.SPEC_BF16, S.SPEC_F32)), window=rng.choice((0, 0, 1, rng.randint(1, 300))), path=less[2] > 0 and rng.random() < 0.3)
            assert _suffices(less, have, **kw), (size, less, kw)


def test_a_small_tree_after_a_wide_batch():
    """32/8 heads, D 128, prefix 4096: four trees of 8 nodes, and one of 8."""
    have = S.spec_weight_workspace_size(4, 32, 8, 4096, 32, 8, 128)
    assert S.spec_weight_workspace_size(1, 8, 8, 4096, 32, 8, 128) <= have
    assert have <= 1 << 20
