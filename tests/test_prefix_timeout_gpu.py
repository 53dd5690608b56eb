"""Waits that run out behind a shared prefix, through the C ABI.

In ``attn_selftest_prefix_timeout`` one CTA waits in vain for its first key tile,
or its first query rows, with a 10 ms limit.  In shares of a key tile or two all
copies are under way before any wait, so that the copying warps have done
everything long before another role gives up.  The call has to return, the
status word to report it, the rows of other K/V heads to be right (what a CTA
that gave up left of the list in the workspace is not trusted: it begins as
ones, or large numbers), and the next calls to give the same bits as before.
"""
import time

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests.test_prefix_gpu import make, randn

pytestmark = pytest.mark.gpu

LIMIT_NS = 10_000_000  # 10 ms


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


# B, Hq, Hkv, D, Sq, prefix, own, and a CTA that has key tiles: the three ways of
# few, packed and many rows, with shares of one or two key tiles (the first four
# places of the list are empty) and of several units.
CASES = [
    (4, 8, 2, 128, 1, 450, 250, 4), (5, 6, 2, 64, 3, 200, 250, 5),
    (4, 8, 2, 128, 20, 450, 250, 4), (3, 4, 2, 64, 40, 333, 250, 4),
    (4, 8, 2, 128, 200, 450, 250, 2), (2, 4, 2, 64, 70, 0, 250, 4),
    (2, 4, 2, 128, 1, 60000, 250, 1), (40, 16, 16, 64, 70, 900, 300, 0),
    (1, 600, 300, 128, 60, 200, 300, 0),
]


@pytest.mark.parametrize("fill", [0xff, 0x70])
@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("case", CASES)
def test_a_wait_runs_out(case, rows, fill):
    B, Hq, Hkv, D, Sq, P, own, block = case
    dtype = "bf16" if rows else "f16"
    joint = Hq // Hkv * Sq > 128 or B == 1
    c = make(B, Hkv, D, P, max(P, 1), [own - 7 * (i % 9) for i in range(B)],
             own, dtype)
    q = randn(B, Hq, Sq, D, dtype=dtype, seed=3)
    want = attn.prefix_fwd(c, q)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == (0, 0)
    ws = attn.prefix_workspace(c, Hq, Sq)
    ws.fill_(fill)
    o, lse = torch.zeros_like(q), torch.zeros_like(want[1])
    t0 = time.perf_counter()
    st = attn.attn_selftest_prefix_timeout(
        c, q.data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, Sq, 0, D ** -0.5,
        True, attn.ATTN_BF16 if dtype == "bf16" else attn.ATTN_F16,
        ws.data_ptr(), ws.numel(), block, rows, LIMIT_NS,
        torch.cuda.current_stream().cuda_stream)
    assert st == attn.ATTN_OK
    st, code = attn.attn_device_status()
    assert time.perf_counter() - t0 < 5.0
    assert st == attn.ATTN_ERR_TIMEOUT and code & 0xff == 1, hex(code)
    assert (code >> 8) & 0xff != 0, hex(code)
    assert attn.attn_device_status() == (0, 0)
    if B <= 5 and Hkv == 2 and P < 1000:  # a CTA has no two units
        g = Hq // Hkv
        assert torch.equal(o[:, g:], want[0][:, g:])
        assert torch.equal(lse[:, g:], want[1][:, g:])
        if joint:  # units of one sequence
            assert torch.equal(o[1:], want[0][1:])
            assert torch.equal(lse[1:], want[1][1:])
    for _ in range(3):
        attn.prefix_fwd(c, q, out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == (0, 0)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_no_time_is_refused():
    c = make(2, 1, 64, 100, 100, [50, 50], 50, "f16")
    q = randn(2, 2, 1, 64, dtype="f16", seed=3)
    ws = attn.prefix_workspace(c, 2, 1)
    assert attn.attn_selftest_prefix_timeout(
        c, q.data_ptr(), torch.empty_like(q).data_ptr(), 0, 2, 1, 0, 0.1, True,
        attn.ATTN_F16, ws.data_ptr(), ws.numel(), 0, 0, 0, 0) == \
        attn.ATTN_ERR_INVALID_ARG
