"""Host-side checks of the calls around a bounded cache, without a GPU: every
refusal comes back as a code before any launch, empty calls are accepted, and
the binding checks types."""
import ctypes

import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from tree_speculative_verification_spec_gb300 import build

P = ctypes.c_void_p(1 << 20)      # stands for a device pointer that no call may touch here
ODD = ctypes.c_void_p((1 << 20) + 8)
BAD, UNSUP, WS, OK = S.SPEC_ERR_INVALID_ARG, S.SPEC_ERR_UNSUPPORTED, S.SPEC_ERR_WORKSPACE, S.SPEC_OK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def _rope(qkv=P, stride=512, q_norm=P, k_norm=P, eps=1e-6, freq=P, axis=None, rot=64, pairing=0, base=None, pos=None, axes=1, q=P, k=P, v=P, table=P, mb=4,
          bs=16, nb=8, prefix=P, off=P, B=1, T=4, n_max=4, Hq=4, Hkv=2, D=64, dtype=S.SPEC_BF16, status=P):
    return S.lib().spec_rope_append(qkv, stride, q_norm, k_norm, eps, freq, axis, rot, pairing, base, pos, axes, q, k, v, table, mb, bs, nb, prefix, off, B, T,
                                    n_max, Hq, Hkv, D, dtype, status, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(n_max=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(mb=0), BAD), (dict(nb=0), BAD),
    (dict(dtype=2), BAD), (dict(D=96), UNSUP), (dict(bs=24), UNSUP), (dict(bs=4), UNSUP), (dict(rot=-2), BAD), (dict(rot=66), BAD), (dict(rot=7), BAD),
    (dict(pairing=2), BAD), (dict(axes=0), BAD), (dict(axes=5, axis=P, pos=P), BAD), (dict(axes=2, axis=P), BAD), (dict(axes=2, pos=P), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(stride=511), BAD), (dict(stride=516), BAD),
    (dict(stride=-512), BAD), (dict(B=70000), UNSUP), (dict(T=1 << 30), UNSUP), (dict(qkv=None), BAD), (dict(q=None), BAD), (dict(k=None), BAD),
    (dict(v=None), BAD), (dict(table=None), BAD), (dict(prefix=None), BAD), (dict(off=None), BAD), (dict(status=None), BAD), (dict(freq=None), BAD),
    (dict(qkv=ODD), BAD), (dict(q=ODD), BAD), (dict(k=ODD), BAD), (dict(v=ODD), BAD), (dict(q_norm=ODD), BAD), (dict(k_norm=ODD), BAD),
    (dict(B=0, qkv=None), OK), (dict(T=0, qkv=None), OK), (dict(n_max=0, qkv=None), OK)])
def test_rope_append_refusals(change, code):
    assert _rope(**change) == code


def _weight(q=P, k=P, table=P, mb=4, bs=16, nb=8, prefix=P, off=P, path=None, path_stride=0, accept=None, window=0, B=1, T=4, n_max=4, max_prefix=10, Hq=4,
            Hkv=2, D=64, dtype=S.SPEC_BF16, scale=0.125, decay=1.0, before=None, weight=P, stride=64, ws=P, ws_bytes=1 << 20, status=P):
    return S.lib().spec_attention_weight(q, k, table, mb, bs, nb, prefix, off, path, path_stride, accept, window, B, T, n_max, max_prefix, Hq, Hkv, D, dtype,
                                         scale, decay, before, weight, stride, ws, ws_bytes, status, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(n_max=-1), BAD), (dict(max_prefix=-1), BAD), (dict(Hq=5), BAD), (dict(Hkv=0), BAD), (dict(dtype=7), BAD),
    (dict(D=96), UNSUP), (dict(bs=24), UNSUP), (dict(n_max=1 << 30), UNSUP), (dict(T=1 << 30, Hq=8, Hkv=8), UNSUP), (dict(B=70000), UNSUP),
    (dict(window=-1), BAD), (dict(stride=-1), BAD), (dict(stride=(1 << 31) + 1), UNSUP), (dict(path=P, path_stride=4), BAD), (dict(accept=P), BAD),
    (dict(path=P, accept=P, path_stride=0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD), (dict(decay=-0.5), BAD),
    (dict(decay=float("inf")), BAD), (dict(q=None), BAD), (dict(k=None), BAD), (dict(table=None), BAD), (dict(prefix=None), BAD), (dict(off=None), BAD),
    (dict(weight=None), BAD), (dict(status=None), BAD), (dict(q=ODD), BAD), (dict(k=ODD), BAD), (dict(mb=0), BAD), (dict(nb=0), BAD), (dict(ws=None), WS),
    (dict(ws_bytes=64), WS), (dict(ws=ODD), WS), (dict(B=0, q=None), OK)])
def test_attention_weight_refusals(change, code):
    assert _weight(**change) == code


def _evict(k=P, v=P, layers=1, table=P, B=2, mb=4, bs=16, nb=8, src=P, dst=P, length=P, N=1, keep_max=8, first=0, last=0, stride=64, Hkv=2, D=64,
           dtype=S.SPEC_BF16, slots=P, new_len=P, status=P):
    return S.lib().spec_kv_evict(k, v, layers, table, B, mb, bs, nb, src, dst, length, None, N, keep_max, first, last, P, stride, Hkv, D, dtype, slots, new_len,
                                 status, None)


@pytest.mark.parametrize("change,code", [
    (dict(layers=0), BAD), (dict(B=-1), BAD), (dict(mb=0), BAD), (dict(nb=0), BAD), (dict(N=-1), BAD), (dict(keep_max=-1), BAD), (dict(first=-1), BAD),
    (dict(last=-1), BAD), (dict(Hkv=0), BAD), (dict(stride=-1), BAD), (dict(dtype=3), BAD), (dict(D=80), UNSUP), (dict(bs=20), UNSUP),
    (dict(layers=40000), UNSUP), (dict(N=70000), UNSUP), (dict(layers=30000, N=60000, Hkv=2), UNSUP), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(table=None), BAD), (dict(src=None), BAD), (dict(dst=None), BAD), (dict(length=None), BAD), (dict(slots=None), BAD), (dict(new_len=None), BAD),
    (dict(status=None), BAD), (dict(N=0, src=None), OK)])
def test_evict_refusals(change, code):
    assert _evict(**change) == code


def test_names_and_workspace():
    assert S.spec_dev_status_string(S.SPEC_DEV_BAD_POSITION) == "bad position"
    assert S.spec_weight_workspace_size(0, 0, 0, 0, 32, 8, 128) == 256
    # a (maximum, sum) for every row of q at least
    assert S.spec_weight_workspace_size(2, 1000, 600, 4000, 32, 8, 128) >= 8 * 1000 * 32


def test_binding_checks_types_before_a_call():
    t = torch.zeros
    with pytest.raises(ValueError, match="one dtype"):
        S.spec_rope_append(t(4, 512), None, None, 1e-6, t(32), None, 64, 0, None, None, 1, t(4, 4, 64).bfloat16(), t(8, 2, 16, 64), t(8, 2, 16, 64), None, 4, 16,
                           8, None, None, 1, 4, 4, 4, 2, 64, None)
    with pytest.raises(ValueError, match="contiguous rows"):
        S.spec_rope_append(t(4, 512), None, None, 1e-6, t(32), None, 64, 0, None, None, 1, t(4, 4, 64), t(8, 2, 16, 64), t(8, 2, 16, 64), None, 4, 16, 8, None,
                           None, 1, 4, 4, 4, 2, 64, None)
    with pytest.raises(ValueError, match="one dtype"):
        S.spec_attention_weight(t(4, 4, 64), t(8, 2, 16, 64).bfloat16(), None, 4, 16, 8, None, None, None, None, 0, 1, 4, 4, 10, 4, 2, 64, 0.1, 1.0, None, None,
                                64, None, None)
