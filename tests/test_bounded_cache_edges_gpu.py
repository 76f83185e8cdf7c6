"""Calls of a bounded cache at the edges of what their arguments may say:
against plain implementations in 64 bits."""
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
