"""Host-side checks of the prompt, log-probability and page calls, without a
GPU: every refusal comes back as a code before any launch, empty calls are
accepted, and the workspace queries cover what the calls need."""
import ctypes

import pytest

import tree_speculative_verification_spec_gb300 as S
from tree_speculative_verification_spec_gb300 import build

P = ctypes.c_void_p(1 << 20)      # stands for a device pointer that no call may touch here
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def _prompt(q=P, k=P, v=P, table=P, max_blocks=4, bs=16, nb=8, prefix=P, off=P, B=1, T=4, n_max=4, max_prefix=10, Hq=4,
            Hkv=2, D=64, dtype=S.SPEC_BF16, out=P, ws=None, ws_bytes=0, status=P, scale=0.125):
    return S.lib().spec_prompt_attention(q, k, v, table, max_blocks, bs, nb, prefix, off, B, T, n_max, max_prefix, Hq, Hkv,
                                         D, dtype, scale, out, ws, ws_bytes, status, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), S.SPEC_ERR_INVALID_ARG), (dict(T=-1), S.SPEC_ERR_INVALID_ARG), (dict(n_max=-1), S.SPEC_ERR_INVALID_ARG),
    (dict(max_prefix=-1), S.SPEC_ERR_INVALID_ARG), (dict(Hq=5), S.SPEC_ERR_INVALID_ARG), (dict(Hkv=0), S.SPEC_ERR_INVALID_ARG),
    (dict(dtype=7), S.SPEC_ERR_INVALID_ARG), (dict(D=96), S.SPEC_ERR_UNSUPPORTED), (dict(bs=24), S.SPEC_ERR_UNSUPPORTED),
    (dict(bs=4), S.SPEC_ERR_UNSUPPORTED), (dict(n_max=1 << 30), S.SPEC_ERR_UNSUPPORTED),
    (dict(T=1 << 30, Hq=8, Hkv=8), S.SPEC_ERR_UNSUPPORTED), (dict(q=None), S.SPEC_ERR_INVALID_ARG),
    (dict(off=None), S.SPEC_ERR_INVALID_ARG), (dict(status=None), S.SPEC_ERR_INVALID_ARG), (dict(q=ODD), S.SPEC_ERR_INVALID_ARG),
    (dict(out=ODD), S.SPEC_ERR_INVALID_ARG), (dict(k=ODD), S.SPEC_ERR_INVALID_ARG), (dict(max_blocks=0), S.SPEC_ERR_INVALID_ARG),
    (dict(B=70000), S.SPEC_ERR_UNSUPPORTED), (dict(max_prefix=100000), S.SPEC_ERR_WORKSPACE),
    (dict(max_prefix=100000, ws=P, ws_bytes=64), S.SPEC_ERR_WORKSPACE),
    (dict(max_prefix=100000, ws=ODD, ws_bytes=1 << 30), S.SPEC_ERR_WORKSPACE),
    (dict(scale=-1.0), S.SPEC_ERR_INVALID_ARG), (dict(scale=float("nan")), S.SPEC_ERR_INVALID_ARG),
    (dict(scale=float("inf")), S.SPEC_ERR_INVALID_ARG),
    (dict(B=0, q=None), S.SPEC_OK), (dict(T=0, q=None), S.SPEC_OK), (dict(n_max=0, q=None), S.SPEC_OK)])
def test_prompt_attention_refusals(change, code):
    assert _prompt(**change) == code


def _tokens(logits=P, dtype=S.SPEC_F32, tokens=P, off=P, B=1, T=4, V=100, k=3, logprob=P, status=P):
    return S.lib().spec_token_logprobs(logits, dtype, tokens, off, None, B, T, V, k, logprob, P, P, P, P, status, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), S.SPEC_ERR_INVALID_ARG), (dict(T=-1), S.SPEC_ERR_INVALID_ARG), (dict(V=0), S.SPEC_ERR_INVALID_ARG),
    (dict(k=-1), S.SPEC_ERR_INVALID_ARG), (dict(V=2, k=3), S.SPEC_ERR_INVALID_ARG), (dict(k=33), S.SPEC_ERR_UNSUPPORTED),
    (dict(V=131073), S.SPEC_ERR_UNSUPPORTED), (dict(dtype=2), S.SPEC_ERR_INVALID_ARG), (dict(logits=None), S.SPEC_ERR_INVALID_ARG),
    (dict(logits=ctypes.c_void_p((1 << 20) + 2)), S.SPEC_ERR_INVALID_ARG), (dict(logprob=None), S.SPEC_ERR_INVALID_ARG),
    (dict(tokens=None), S.SPEC_ERR_INVALID_ARG), (dict(status=None), S.SPEC_ERR_INVALID_ARG), (dict(B=0, logits=None), S.SPEC_OK),
    (dict(T=0, logits=None), S.SPEC_OK)])
def test_token_logprobs_refusals(change, code):
    assert _tokens(**change) == code


def _path(n_max=4, path=P, accept=P, T=4, k=2):
    return S.lib().spec_path_logprobs(P, S.SPEC_F32, P, path, accept, P, None, 1, T, n_max, 100, k, P, P, P, P, P, P, None)


@pytest.mark.parametrize("change,code", [
    (dict(n_max=-1), S.SPEC_ERR_INVALID_ARG), (dict(n_max=1025), S.SPEC_ERR_UNSUPPORTED), (dict(path=None), S.SPEC_ERR_INVALID_ARG),
    (dict(accept=None), S.SPEC_ERR_INVALID_ARG), (dict(n_max=0, path=None), S.SPEC_OK), (dict(T=-1), S.SPEC_ERR_INVALID_ARG),
    (dict(k=40), S.SPEC_ERR_UNSUPPORTED)])
def test_path_logprobs_refusals(change, code):
    assert _path(**change) == code



def _fork(k=P, v=P, layers=1, table=P, B=2, mb=4, bs=16, nb=8, src=P, N=1, Hkv=2, D=64, dtype=S.SPEC_BF16, pool=P, cap=8, count=P,
          ws=P, ws_bytes=1 << 20, status=P):
    return S.lib().spec_pages_fork(k, v, layers, table, B, mb, bs, nb, src, P, P, None, N, Hkv, D, dtype, pool, cap, count, ws, ws_bytes,
                                   status, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), S.SPEC_ERR_INVALID_ARG), (dict(mb=0), S.SPEC_ERR_INVALID_ARG), (dict(nb=0), S.SPEC_ERR_INVALID_ARG),
    (dict(N=-1), S.SPEC_ERR_INVALID_ARG), (dict(layers=-1), S.SPEC_ERR_INVALID_ARG), (dict(k=None), S.SPEC_ERR_INVALID_ARG),
    (dict(Hkv=0), S.SPEC_ERR_INVALID_ARG), (dict(D=80), S.SPEC_ERR_UNSUPPORTED), (dict(bs=20), S.SPEC_ERR_UNSUPPORTED),
    (dict(dtype=3), S.SPEC_ERR_INVALID_ARG), (dict(cap=-1), S.SPEC_ERR_INVALID_ARG), (dict(src=None), S.SPEC_ERR_INVALID_ARG),
    (dict(pool=None), S.SPEC_ERR_INVALID_ARG), (dict(count=None), S.SPEC_ERR_INVALID_ARG), (dict(table=None), S.SPEC_ERR_INVALID_ARG),
    (dict(B=1 << 16, mb=1 << 15), S.SPEC_ERR_UNSUPPORTED), (dict(N=1 << 20, mb=1 << 11), S.SPEC_ERR_UNSUPPORTED),
    (dict(ws=None), S.SPEC_ERR_WORKSPACE), (dict(ws_bytes=8), S.SPEC_ERR_WORKSPACE), (dict(ws=ODD), S.SPEC_ERR_WORKSPACE),
    (dict(N=0, src=None), S.SPEC_OK)])
def test_pages_fork_refusals(change, code):
    assert _fork(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), S.SPEC_ERR_INVALID_ARG), (dict(rows=None), S.SPEC_ERR_INVALID_ARG), (dict(bs=9), S.SPEC_ERR_UNSUPPORTED),
    (dict(cap=-1), S.SPEC_ERR_INVALID_ARG), (dict(ws_bytes=8), S.SPEC_ERR_WORKSPACE), (dict(N=0, rows=None), S.SPEC_OK)])
def test_pages_free_refusals(change, code):
    a = dict(N=1, rows=P, bs=16, cap=8, ws=P, ws_bytes=1 << 20)
    a.update(change)
    assert S.lib().spec_pages_free(P, 2, 4, a["bs"], 8, a["rows"], None, a["N"], P, a["cap"], P, a["ws"], a["ws_bytes"], P, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(layers=-1), S.SPEC_ERR_INVALID_ARG), (dict(page_map=None), S.SPEC_ERR_INVALID_ARG), (dict(moved=None), S.SPEC_ERR_INVALID_ARG),
    (dict(table=None), S.SPEC_ERR_INVALID_ARG), (dict(D=32), S.SPEC_ERR_UNSUPPORTED), (dict(ws_bytes=8), S.SPEC_ERR_WORKSPACE),
    (dict(nb=(1 << 30) + 1), S.SPEC_ERR_UNSUPPORTED)])
def test_pages_compact_refusals(change, code):
    a = dict(layers=1, page_map=P, moved=P, table=P, D=64, ws_bytes=1 << 20, nb=8)
    a.update(change)
    assert S.lib().spec_pages_compact(P, P, a["layers"], a["table"], 2, 4, 16, a["nb"], 2, a["D"], S.SPEC_BF16, P, 8, P, a["page_map"],
                                      a["moved"], P, a["ws_bytes"], P, None) == code


def test_workspace_sizes_and_names():
    # key splits of a single row need its partial rows; a batch that fills the GPU needs none
    assert S.spec_prompt_workspace_size(1, 1, 1, 30000, 32, 8, 128) >= 2 * 32 * (128 + 2) * 4
    assert S.spec_prompt_workspace_size(64, 64 * 512, 512, 0, 32, 8, 128) == 256
    assert S.spec_prompt_workspace_size(0, 0, 0, 0, 32, 8, 128) == 256
    assert S.spec_pages_workspace_size(256, 1024, 262144, 64) >= 4 * 262144
    assert S.spec_pages_workspace_size(1, 1, 1, 1) == 256
    assert S.spec_dev_status_string(S.SPEC_DEV_BAD_ROW) == "bad table row"


def test_append_takes_more_rows_than_a_tree_has():
    """A prompt's rows reach the cache by the append of the tree's."""
    a = lambda n_max, B: S.lib().spec_kv_append(None, None, None, None, None, 4, 16, 4, None, None, B, n_max, 2, 64, S.SPEC_BF16, None, None)  # noqa: E731
    assert a(100000, 0) == S.SPEC_OK
    assert a(100000, 1) == S.SPEC_ERR_INVALID_ARG  # past the size checks, at the pointers


@pytest.mark.parametrize("B,max_blocks,N,code", [((1 << 30) + 1, 1, 1, S.SPEC_ERR_UNSUPPORTED), (4, 1 << 20, 1025, S.SPEC_ERR_UNSUPPORTED),
                                                 (4, 1 << 20, 1024, S.SPEC_ERR_WORKSPACE), (1025, 1 << 20, 1, S.SPEC_ERR_UNSUPPORTED),
                                                 (1 << 30, 1, 1, S.SPEC_ERR_WORKSPACE)])
def test_page_calls_keep_their_counters_in_32_bits(B, max_blocks, N, code):
    L = S.lib()
    assert L.spec_pages_free(P, B, max_blocks, 16, 8, P, None, N, P, 8, P, P, 8, P, None) == code
    assert L.spec_pages_fork(P, P, 1, P, B, max_blocks, 16, 8, P, P, P, None, N, 2, 64, S.SPEC_BF16, P, 8, P, P, 8, P, None) == code


def test_tables_of_cache_addresses_are_checked_before_a_call():
    import torch
    from tree_speculative_verification_spec_gb300 import _binding
    for table, layers in ((torch.zeros(2, dtype=torch.int32), 2), (torch.zeros(2), 2), (torch.zeros(1, dtype=torch.int64), 2)):
        with pytest.raises(ValueError, match="int64"):
            _binding._addresses(table, layers)
    assert _binding._addresses(None, 0) is None
