"""Entry points of the heads' norm and rotation without a GPU: phases, refusals
with the documented codes before the device is touched, and the binding's
checks."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from attention_attn_fwd_gb300 import build as cuda_build

OK, INVALID, UNSUPPORTED, ALIGN = (
    attn.ATTN_OK, attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED,
    attn.ATTN_ERR_ALIGNMENT)
MB = 1 << 20
BF16, E4M3 = attn.ATTN_BF16, attn.ATTN_E4M3
# 2 pi by its decimals.
TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751,
                      10 ** 49)


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return attn.load_library()


@pytest.mark.parametrize("f", [0.0, 1.0, 0.5, 1e-4, 10000.0 ** (-3 / 64), -0.7,
                               1e-12, -1e-9, 123456.789, 2.0 ** 32])
def test_phases_are_right_to_a_unit(lib, f):
    turn = Fraction(f) / TWO_PI * 2 ** 64
    off = (attn.attn_rope_phase([f])[0] - turn) % 2 ** 64
    assert min(off, 2 ** 64 - off) <= 1


def test_phase_refusals(lib):
    for f in (math.nan, math.inf, -math.inf, 2.0 ** 33):
        with pytest.raises(attn.AttnError):
            attn.attn_rope_phase([1.0, f])
    assert attn.attn_rope_phase([]) == []
    one = ctypes.c_ulonglong()
    assert lib.attn_rope_phase(None, 1, ctypes.byref(one)) == INVALID
    assert lib.attn_rope_phase(None, -1, None) == INVALID
    assert lib.attn_rope_phase(None, 0, None) == OK


def rope(**kw):
    a = dict(phase=MB, axis=None, D=64, rot=32, axes=1, interleaved=0)
    a.update(kw)
    return attn._RopeStruct(*[a[n] for n, _ in attn._RopeStruct._fields_])


def view(p, S, H, D=64, **kw):
    a = dict(p=p, stride_b=S * H * D, stride_s=H * D, stride_h=D)
    a.update(kw)
    return attn._heads(a["p"] or 0, a["stride_b"], a["stride_s"],
                       a["stride_h"])


def fwd(lib, r=None, q={}, k={}, v={}, wq=None, wk=None, f32=0, eps=1e-6,
        pos=None, lens=None, new=None, off=None, qo=64 * MB, ko=65 * MB,
        vo=66 * MB, B=2, S=4, Hq=4, Hkv=2, cap=4, dtype=BF16):
    r = rope() if r is None else r
    views = [x if x is None or isinstance(x, bytes) else
             view(**{**dict(p=p, S=S, H=H), **x}) for x, p, H in (
                 (q, 16 * MB, 4), (k, 17 * MB, 2), (v, 18 * MB, 2))]
    return lib.attn_qk_rope(ctypes.byref(r), *views, wq, wk, f32, eps, pos,
                            lens, new, off, qo, ko, vo, B, S, Hq, Hkv, cap,
                            dtype, None)


def bwd(lib, r=None, dq=16 * MB, dk=17 * MB, dv=18 * MB, q={}, k={}, wq=20 * MB,
        wk=21 * MB, f32=0, eps=1e-6, pos=None, off=None, dxq={}, dxk={},
        dxv={}, dwq=22 * MB, dwk=23 * MB, B=2, S=4, Hq=4, Hkv=2, dtype=BF16,
        ws=32 * MB, ws_bytes=16 * MB):
    r = rope() if r is None else r
    views = [x if x is None or isinstance(x, bytes) else
             view(**{**dict(p=p, S=S, H=H), **x}) for x, p, H in (
                 (q, 24 * MB, 4), (k, 25 * MB, 2), (dxq, 64 * MB, 4),
                 (dxk, 65 * MB, 2), (dxv, 66 * MB, 2))]
    return lib.attn_qk_rope_bwd(ctypes.byref(r), dq, dk, dv, views[0],
                                views[1], wq, wk, f32, eps, pos, off,
                                *views[2:], dwq, dwk, B, S, Hq, Hkv, dtype, ws,
                                ws_bytes, None)


BOTH = [
    (dict(r=dict(D=96)), UNSUPPORTED), (dict(r=dict(D=0)), INVALID),
    (dict(r=dict(rot=-8)), INVALID), (dict(r=dict(rot=72)), INVALID),
    (dict(r=dict(rot=12)), UNSUPPORTED), (dict(r=dict(phase=None)), INVALID),
    (dict(r=dict(phase=MB + 4)), ALIGN), (dict(r=dict(axes=0)), INVALID),
    (dict(r=dict(axes=256)), INVALID), (dict(r=dict(axes=2)), INVALID),
    (dict(B=-1), INVALID), (dict(S=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(dtype=E4M3), INVALID), (dict(dtype=9), INVALID),
    (dict(B=1 << 16, S=1 << 15), INVALID), (dict(Hq=1 << 21), INVALID),
    (dict(B=1 << 15, S=1 << 15, Hq=1 << 8), INVALID),
    (dict(wq=20 * MB, eps=0.0), INVALID),
    (dict(wq=20 * MB, eps=-1.0), INVALID),
    (dict(wq=20 * MB, eps=math.nan), INVALID),
    (dict(wq=20 * MB, eps=math.inf), INVALID),
    (dict(wq=20 * MB + 1), ALIGN), (dict(wk=20 * MB + 2, f32=1), ALIGN),
    (dict(pos=30 * MB, off=31 * MB), INVALID), (dict(pos=30 * MB + 2), ALIGN),
    (dict(off=31 * MB + 1), ALIGN),
]


def with_rope(kw):
    kw = dict(kw)
    if "r" in kw:
        kw["r"] = rope(**kw["r"])
    return kw


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(vo=None), INVALID), (dict(qo=None), INVALID),
    (dict(ko=None), INVALID), (dict(qo=64 * MB + 8), ALIGN),
    (dict(ko=65 * MB + 2), ALIGN), (dict(cap=3), INVALID),
    (dict(q=dict(p=None)), INVALID), (dict(q=dict(p=16 * MB + 8)), ALIGN),
    (dict(q=dict(stride_s=260)), ALIGN), (dict(q=dict(stride_h=68)), ALIGN),
    (dict(k=dict(stride_b=-512)), INVALID),
    (dict(k=dict(stride_b=1 << 62)), INVALID),
    (dict(lens=30 * MB + 2), ALIGN), (dict(new=30 * MB + 1), ALIGN),
    (dict(qo=16 * MB), INVALID),           # over an input
    (dict(ko=66 * MB), INVALID),           # over another output
    (dict(q=dict(stride_b=48 * MB)), INVALID),   # spans an output
])
def test_forward_refusals(lib, kw, code):
    assert fwd(lib, **with_rope(kw)) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dv=None), INVALID), (dict(dxv=None), INVALID),
    (dict(dq=16 * MB + 8), ALIGN), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(dxq=None), INVALID),
    (dict(dwq=None), INVALID), (dict(dwk=None), INVALID),
    (dict(wq=None), INVALID), (dict(dwq=22 * MB + 2), ALIGN),
    (dict(ws=None), ALIGN), (dict(ws=32 * MB + 16), ALIGN),
    (dict(ws_bytes=100), INVALID), (dict(ws=64 * MB), INVALID),
    (dict(dwk=22 * MB), INVALID),
    (dict(dxq=dict(stride_h=0)), INVALID),       # places share elements
    (dict(dxq=dict(stride_s=128)), INVALID),
    (dict(dxk=dict(p=64 * MB)), INVALID),        # over dq
    (dict(dxk=dict(p=64 * MB + 128)), INVALID),
    (dict(dxq=dict(p=24 * MB)), INVALID),        # over an input
    (dict(dxq=dict(stride_h=64, stride_s=512, stride_b=2048),
          dxk=dict(p=64 * MB + 3 * 128, stride_s=512, stride_b=2048)),
     INVALID),                                   # packed, but one head over
    (dict(dxq=dict(stride_s=512, stride_b=2048),
          dxk=dict(p=64 * MB + 512, stride_s=512, stride_b=4096)), INVALID),
    (dict(dxq=dict(stride_s=512, stride_b=2048),
          dxk=dict(p=64 * MB + 7 * 128, stride_s=512, stride_b=2048)),
     INVALID),                                   # reaches the next token's dq
])
def test_backward_refusals(lib, kw, code):
    assert bwd(lib, **with_rope(kw)) == code


def test_no_ops(lib):
    assert fwd(lib, B=0) == OK
    assert fwd(lib, S=0) == OK
    none = dict(wq=None, wk=None, dwq=None, dwk=None)
    assert bwd(lib, B=0, **none) == OK
    assert bwd(lib, S=0, **none) == OK


def test_null_rope(lib):
    q = view(16 * MB, 1, 1)
    assert lib.attn_qk_rope(None, q, q, None, None, None, 0, 1e-6, None, None,
                            None, None, 64 * MB, 65 * MB, None, 1, 1, 1, 1, 1,
                            BF16, None) == INVALID


def test_workspace_bytes(lib):
    f = attn.attn_qk_rope_bwd_workspace_bytes
    assert 0 < f(64) < f(128)
    assert f(0) == f(96) == f(-64) == 0


def test_binding_refusals(lib):
    with pytest.raises(attn.AttnError):
        attn.Rope([1.0] * 33, 64, device="cpu")      # more pairs than D / 2
    with pytest.raises(attn.AttnError):
        attn.Rope([1.0] * 6, 64, device="cpu")       # 12 elements
    with pytest.raises(attn.AttnError):
        attn.Rope([1.0] * 8, 96, device="cpu")
    with pytest.raises(attn.AttnError):
        attn.Rope([1.0] * 8, 64, axes=[0] * 7, device="cpu")
    with pytest.raises(attn.AttnError):
        attn.Rope([1.0] * 8, 64, axes=[-1] * 8, device="cpu")
    with pytest.raises(attn.AttnError):
        attn.Rope([1.0] * 8, 64, device="cpu")       # no host fallback
