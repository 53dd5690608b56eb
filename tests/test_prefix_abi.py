"""The entry point of attention behind a shared prefix without a GPU: refusals
with the documented codes before the device is touched, the workspace size, and
the binding's checks."""
import ctypes
import math

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
    a = dict(prefix_k=8 * MB, prefix_v=12 * MB, prefix_len=15 * MB, k=16 * MB,
             v=32 * MB, lens=50 * MB, B=2, Hkv=2, prefix_capacity=300,
             capacity=100, D=64)
    a.update(kw)
    return attn._Prefix(*[a[n] for n, _ in attn._Prefix._fields_])


def fwd(lib, c, Q=64 * MB, O=65 * MB, LSE=66 * MB, Hq=4, Sq=1, new=None,
        scale=0.1, dtype=BF16, ws=128 * MB, ws_bytes=256 * MB):
    return lib.attn_prefix_fwd(ctypes.byref(c), Q, O, LSE, Hq, Sq, new, scale,
                               1, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(capacity=0), INVALID),
    (dict(prefix_capacity=0), INVALID), (dict(D=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(B=1 << 23), INVALID), (dict(capacity=0x7fffffff), INVALID),
    (dict(prefix_capacity=0x7fffffff - (1 << 16)), INVALID),
    (dict(prefix_k=None), INVALID), (dict(prefix_v=None), INVALID),
    (dict(prefix_len=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(lens=None), INVALID),
    (dict(prefix_k=8 * MB + 8), ALIGN), (dict(prefix_v=12 * MB + 2), ALIGN),
    (dict(k=16 * MB + 8), ALIGN), (dict(v=32 * MB + 4), ALIGN),
    (dict(lens=50 * MB + 1), ALIGN), (dict(prefix_len=15 * MB + 2), ALIGN),
])
def test_bad_caches_are_refused(lib, change, code):
    for Sq in (1, 30, 300):
        assert fwd(lib, cache(**change), Sq=Sq) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(O=None), INVALID), (dict(Hq=3), INVALID),
    (dict(Hq=0), INVALID), (dict(Sq=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(dtype=E4M3), INVALID), (dict(dtype=7), INVALID),
    (dict(Q=64 * MB + 8), ALIGN), (dict(O=65 * MB + 8), ALIGN),
    (dict(LSE=66 * MB + 2), ALIGN), (dict(new=70 * MB + 3), ALIGN),
    (dict(ws=None), ALIGN), (dict(ws=128 * MB + 128), ALIGN),
    (dict(ws_bytes=1000), INVALID), (dict(O=64 * MB), INVALID),
    (dict(O=16 * MB), INVALID), (dict(O=8 * MB), INVALID),
    (dict(LSE=65 * MB), INVALID), (dict(LSE=50 * MB), INVALID),
    (dict(ws=64 * MB), INVALID), (dict(Sq=1 << 30), INVALID),
    (dict(Hq=258), UNSUPPORTED),
])
def test_refusals(lib, kw, code):
    assert fwd(lib, cache(), **kw) == code


def test_null_cache(lib):
    assert lib.attn_prefix_fwd(None, 64 * MB, 65 * MB, None, 4, 1, None, 0.1,
                               1, BF16, 128 * MB, 256 * MB, None) == INVALID


def test_counts_beyond_32_bits_are_refused(lib):
    """Places of the list of tiles are counted in 32 bits."""
    big = cache(B=1 << 20, Hkv=15, capacity=1 << 20)
    for Sq in (1, 30, 300):
        assert fwd(lib, big, Hq=30, Sq=Sq) == INVALID
        assert attn.attn_prefix_workspace_bytes(
            1 << 20, 30, 15, Sq, 300, 1 << 20, 64) == 0


def test_no_ops(lib):
    assert fwd(lib, cache(B=0)) == OK
    assert fwd(lib, cache(), Sq=0) == OK


def test_workspace_bytes(lib):
    f = attn.attn_prefix_workspace_bytes
    one = f(8, 32, 8, 1, 4096, 4096, 128)
    assert one > 0
    # It does not grow with the lengths.
    assert f(8, 32, 8, 1, 131072, 65536, 128) == one
    assert f(8, 32, 8, 30, 4096, 4096, 128) > 0
    assert f(8, 32, 8, 512, 4096, 4096, 128) > 0
    for bad in ((-1, 32, 8, 1, 64, 64, 128), (8, 30, 8, 1, 64, 64, 128),
                (8, 32, 0, 1, 64, 64, 128), (8, 32, 8, -1, 64, 64, 128),
                (8, 32, 8, 1, 0, 64, 128), (8, 32, 8, 1, 64, 0, 128),
                (8, 32, 8, 1, 64, 64, 96)):
        assert f(*bad) == 0
    assert f(0, 32, 8, 1, 64, 64, 128) == f(8, 32, 8, 0, 64, 64, 128) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    p = torch.zeros(1, 2, 8, 64, dtype=torch.float16)
    k = torch.zeros(3, 2, 5, 64, dtype=torch.float16)
    n, m = torch.zeros(1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in ((p, p, n, k, k, m), (p[0], p, n, k, k, m),
                (p, p, n, k, k[:, :, :4], m), (p, p, m, k, k, m),
                (p, p, n, k, k, n), (p, p, n, k.float(), k.float(), m),
                (p, p.bfloat16(), n, k, k, m), (k, k, n, k, k, m),
                (p, p, n.long(), k, k, m), (p, p, n, k.int(), k.int(), m)):
        with pytest.raises(attn.AttnError):
            attn.PrefixCache(*bad)
