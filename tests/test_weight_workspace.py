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
