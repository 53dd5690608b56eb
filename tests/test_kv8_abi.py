"""8-bit cache entry points without a GPU: refusals with the documented codes
before the device is touched, the workspace size, and the binding's checks."""
import ctypes

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from attention_attn_fwd_gb300 import build as cuda_build

OK, INVALID, UNSUPPORTED, ALIGN = (
    attn.ATTN_OK, attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED,
    attn.ATTN_ERR_ALIGNMENT)
MB = 1 << 20
BF16, E4M3 = attn.ATTN_BF16, attn.ATTN_E4M3


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return attn.load_library()


def cache(**kw):
    """A cache of addresses that are never dereferenced on these paths."""
    a = dict(k=16 * MB, v=32 * MB, k_scale=48 * MB, v_scale=49 * MB,
             lens=50 * MB, B=2, Hkv=2, capacity=100, D=64, block=32)
    a.update(kw)
    return attn._KV8(*[a[n] for n, _ in attn._KV8._fields_])


SIZES = [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(capacity=0), INVALID),
    (dict(D=0), INVALID), (dict(block=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED), (dict(block=8), UNSUPPORTED),
    (dict(block=48), UNSUPPORTED), (dict(block=256), UNSUPPORTED),
    (dict(B=1 << 23, Hkv=2), INVALID), (dict(capacity=0x7fffffff), INVALID),
]
POINTERS = [
    (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(lens=None), INVALID), (dict(k=16 * MB + 8), ALIGN),
    (dict(v=32 * MB + 4), ALIGN), (dict(k_scale=48 * MB + 2), ALIGN),
    (dict(lens=50 * MB + 1), ALIGN),
]


def append(lib, c, K=64 * MB, V=65 * MB, Sq=4, new=None, dtype=BF16):
    return lib.attn_kv8_append(ctypes.byref(c), K, V, Sq, new, dtype, None)


def fwd(lib, c, Q=64 * MB, O=65 * MB, LSE=66 * MB, w=None, Hq=4, Sq=1,
        new=None, scale=0.1, dtype=BF16, ws=67 * MB, ws_bytes=64 * MB):
    return lib.attn_kv8_fwd(ctypes.byref(c), Q, O, LSE, w, Hq, Sq, new, scale,
                            1, dtype, ws, ws_bytes, None)


def evict(lib, s, d, w=64 * MB, dw=65 * MB, keep=50, recent=5, idx=66 * MB):
    return lib.attn_kv8_evict(ctypes.byref(s), ctypes.byref(d), w, dw, keep,
                              recent, idx, None)


def other(**kw):
    a = dict(k=116 * MB, v=132 * MB, k_scale=148 * MB, v_scale=149 * MB,
             lens=150 * MB)
    a.update(kw)
    return cache(**a)


@pytest.mark.parametrize("change,code", SIZES + POINTERS)
def test_bad_caches_are_refused(lib, change, code):
    c = cache(**change)
    assert append(lib, c) == code
    assert fwd(lib, c) == code
    assert evict(lib, c, other()) == code
    assert evict(lib, cache(), other(**change)) == code


def test_capacities_near_int32_are_refused(lib):
    """Kernels count up to 16384 places past a length in 32 bits."""
    for over in (0, 1, 16384, 1 << 16):
        c = cache(B=1, Hkv=1, capacity=0x7fffffff - over)
        assert append(lib, c) == INVALID
        assert fwd(lib, c) == INVALID
        assert evict(lib, c, other(B=1, Hkv=1)) == INVALID


def test_null_cache(lib):
    assert lib.attn_kv8_append(None, 64 * MB, 65 * MB, 1, None, BF16,
                               None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(Sq=-1), INVALID),
    (dict(Sq=101), INVALID), (dict(dtype=E4M3), INVALID),
    (dict(dtype=7), INVALID), (dict(K=64 * MB + 2), ALIGN),
    (dict(new=70 * MB + 2), ALIGN), (dict(K=16 * MB), INVALID),
    (dict(V=32 * MB + 16), INVALID),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(O=None), INVALID), (dict(Hq=3), INVALID),
    (dict(Hq=0), INVALID), (dict(Sq=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(dtype=E4M3), INVALID), (dict(Q=64 * MB + 8), ALIGN),
    (dict(O=65 * MB + 8), ALIGN), (dict(LSE=66 * MB + 2), ALIGN),
    (dict(w=69 * MB + 1), ALIGN), (dict(ws=None), ALIGN),
    (dict(ws=67 * MB + 128), ALIGN), (dict(new=70 * MB + 3), ALIGN),
])
def test_fwd_refusals(lib, kw, code):
    assert fwd(lib, cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(keep=0), INVALID), (dict(keep=101), INVALID),
    (dict(recent=-1), INVALID), (dict(recent=51), INVALID),
    (dict(w=None), INVALID), (dict(dw=None), INVALID),
    (dict(idx=None), INVALID), (dict(w=64 * MB + 2), ALIGN),
    (dict(idx=66 * MB + 1), ALIGN), (dict(dw=64 * MB), INVALID),
    (dict(idx=65 * MB), INVALID),
])
def test_evict_refusals(lib, kw, code):
    assert evict(lib, cache(), other(), **kw) == code


@pytest.mark.parametrize("change", [
    dict(B=3), dict(Hkv=1), dict(D=128), dict(block=16),
    dict(k=16 * MB),                     # K's memory alone is the source's
    dict(k=16 * MB + 4096),              # or overlaps it
    dict(lens=50 * MB),                  # lens must be other memory
    dict(v=16 * MB + 256),
])
def test_evict_destination_refusals(lib, change):
    assert evict(lib, cache(), other(**change)) == INVALID


def test_evict_in_place_needs_the_same_capacity_and_its_own_lens(lib):
    assert evict(lib, cache(), cache()) == INVALID  # shares lens
    assert evict(lib, cache(), cache(lens=51 * MB, capacity=99)) == INVALID


def test_no_ops(lib):
    assert append(lib, cache(B=0)) == OK
    assert append(lib, cache(), Sq=0) == OK
    assert fwd(lib, cache(B=0)) == OK
    assert fwd(lib, cache(), Sq=0) == OK
    assert evict(lib, cache(B=0), other(B=0)) == OK


def test_workspace_bytes(lib):
    f = attn.attn_kv8_workspace_bytes
    one = f(8, 32, 8, 1, 4096, 128, False)
    assert 0 < one < f(8, 32, 8, 1, 4096, 128, True)
    # Without weights it does not grow with the capacity.
    assert f(8, 32, 8, 1, 131072, 128, False) == one
    assert f(8, 32, 8, 512, 4096, 128, False) > 0
    for bad in ((-1, 32, 8, 1, 64, 128), (8, 30, 8, 1, 64, 128),
                (8, 32, 0, 1, 64, 128), (8, 32, 8, -1, 64, 128),
                (8, 32, 8, 1, 0, 128), (8, 32, 8, 1, 64, 96)):
        assert f(*bad, False) == 0
    assert f(0, 32, 8, 1, 64, 128, False) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    k = torch.zeros(1, 1, 64, 64, dtype=torch.uint8)
    s, n = torch.zeros(1, 1, 2), torch.zeros(1, dtype=torch.int32)
    for bad in ((k, k, s, s, n, 33), (k[0], k, s, s, n, 32),
                (k, k[:, :, :63], s, s, n, 32), (k, k, s[..., :1], s, n, 32),
                (k.float(), k, s, s, n, 32), (k, k, s.half(), s, n, 32),
                (k, k, s, s, n.long(), 32), (k, k, s, s, n, 32)):
        with pytest.raises(attn.AttnError):
            attn.KV8Cache(*bad)
