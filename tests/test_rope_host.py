"""What the rotation and the norms refuse before anything is launched (no GPU needed: no pointer is followed)."""
import ctypes
import math

import pytest
import torch

import learned_kv_cache_gb300 as kvp
from learned_kv_cache_gb300 import _lib
from learned_kv_cache_gb300.rope import _Freqs


@pytest.fixture(scope="module")
def lib():
    from learned_kv_cache_gb300 import build
    build.build()
    return _lib.load()


P = 4096
FREQS = (ctypes.c_double * 64)(*[1.0] * 64)


def freqs(rotary_dim=128, interleaved=0, gain=1.0, inv=FREQS):
    return ctypes.byref(_Freqs(inv, rotary_dim, interleaved, gain))


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def rope(lib, x=P, out=P, dtype=1, b=2, h=4, s=8, d=128, xs=None, os=None, f=True, pos=None, pstride=0, start=0, inv=0):
    return lib.kvp_rope(x, out, dtype, b, h, s, d, xs, os, freqs() if f is True else f, pos, pstride, start, inv, None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(x=4100), -1), (dict(out=4104), -1), (dict(dtype=7), -2), (dict(b=0), -1),
    (dict(h=0), -1), (dict(s=0), -1), (dict(b=1 << 16, s=1 << 16), -1), (dict(d=96), -2), (dict(f=None), -1),
    (dict(d=64), -2), (dict(f=freqs(rotary_dim=24)), -2), (dict(f=freqs(rotary_dim=0)), -2), (dict(f=freqs(interleaved=2)), -1),
    (dict(f=freqs(gain=math.inf)), -1), (dict(f=freqs(gain=1e60)), -1), (dict(f=freqs(inv=None)), -1),
    (dict(f=freqs(inv=(ctypes.c_double * 64)(*[-1e-30] * 64))), -1), (dict(f=freqs(inv=(ctypes.c_double * 64)(*[math.nan] * 64))), -1),
    (dict(f=freqs(inv=(ctypes.c_double * 64)(*[1e7] * 64))), -1), (dict(inv=2), -1), (dict(pos=P, pstride=7), -1),
    (dict(start=2 ** 31 - 8 + 1), -1), (dict(xs=strides(4096, 1024, 132)), -1), (dict(xs=strides(-4096, 1024, 128)), -1),
    (dict(xs=strides(1 << 40, 1024, 128)), -1), (dict(os=strides(4096, 1024, 0)), -1), (dict(os=strides(4096, 1024, 64)), -1),
    (dict(os=strides(4096, 128, 128)), -1), (dict(os=strides(0, 1024, 128)), -1), (dict(os=strides(2048, 1024, 128)), -1),
])
def test_rope_refusals(lib, change, code):
    assert rope(lib, **change) == code
    assert lib.kvp_last_error() != b""


def norm(lib, q=P, k=P, qo=P, ko=P, dtype=1, b=2, hq=4, hkv=2, s=8, d=128, qos=None, qw=P, kw=P, wd=1, eps=1e-6, f=None):
    return lib.kvp_qk_norm_rope(q, k, qo, ko, dtype, b, hq, hkv, s, d, None, None, qos, None, qw, kw, wd, eps, f, None, 0, 0,
                                None)


def back(lib, dqo=P, dko=P, q=P, k=P, dq=P, dk=P, dtype=1, b=2, hq=4, hkv=2, s=8, d=128, dqs=None, qw=P, wd=1, eps=1e-6,
         f=None, ws=P, ws_bytes=1 << 40):
    return lib.kvp_qk_norm_rope_backward(dqo, dko, q, k, dq, dk, P, P, dtype, b, hq, hkv, s, d, None, None, None, None, dqs,
                                         None, qw, P, wd, eps, f, None, 0, 0, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(q=8), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(wd=2), -2),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(eps=1e60), -1), (dict(qw=4097), -1), (dict(dtype=3), -2),
    (dict(d=80), -2), (dict(f=freqs(rotary_dim=8)), -2),
])
def test_norm_refusals(lib, change, code):
    assert norm(lib, **change) == code
    assert back(lib, **change) == code


def test_norm_refusals_of_outputs(lib):
    assert norm(lib, qo=None) == -1 and norm(lib, ko=4100) == -1
    assert norm(lib, qos=strides(0, 1024, 128)) == -1
    assert back(lib, dq=None) == -1 and back(lib, dk=4100) == -1 and back(lib, dqo=None) == -1
    assert back(lib, dqs=strides(0, 1024, 128)) == -1
    assert back(lib, ws=None) == -5 and back(lib, ws_bytes=16) == -5 and back(lib, ws=P + 16) == -1
    size = lib.kvp_qk_norm_rope_backward_workspace_size
    assert size(1, 2, 4, 2, 8, 128) > 0
    assert size(9, 2, 4, 2, 8, 128) == 0 and size(1, 2, 0, 2, 8, 128) == 0 and size(1, 2, 4, 2, 8, 96) == 0


def test_cpu_tensors_are_refused():
    x = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError):
        kvp.kvp_rope(x, kvp.Rope(64))
    with pytest.raises(ValueError):
        kvp.kvp_qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        kvp.kvp_qk_norm_rope_backward(x, x, x, x)
