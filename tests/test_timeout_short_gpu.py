"""A forward wait that runs out where the loading warp has asked for all it will
ever load long before: one or two key tiles, fewer than the ring holds.  The
call returns and reports it, other CTAs' rows are right, and the next call's
too."""
import pytest
import torch

import attention_attn_fwd_gb300 as attn
from attention_attn_fwd_gb300.inputs import Workload, make_qkv
from tests.gpu_parity import check_full
from tests.test_timeout_gpu import check_timeout_code, selftest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("Skv", [100, 128, 256])
def test_few_key_tiles(Skv):
    # Units of rows 0-255 and 256-511 of a K/V head's two query heads, or of
    # 256 rows of one: the first CTA's lie in query heads 0 and 1.
    w = Workload("timeout_short", 1, 4, 2, 512, Skv, 128, "bf16", False)
    assert attn.attn_device_status() == (0, 0)
    q, k, v = (x.cuda() for x in make_qkv(w, seed=63))
    want, z = attn.fwd(q, k, v, causal=False)
    o, lse = torch.zeros_like(q), torch.zeros_like(z)
    for _ in range(3):
        assert selftest(w, q, k, v, o, lse,
                        torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK
        check_timeout_code(*attn.attn_device_status())
        assert torch.equal(o[:, 2:], want[:, 2:])
        assert torch.equal(lse[:, 2:], z[:, 2:])
        again, _ = attn.fwd(q, k, v, causal=False)
        assert torch.equal(again, want)
    check_full(w, seed=63)
    assert attn.attn_device_status() == (0, 0)
