"""Gradients into one packed buffer whose heads lie ahead of its tokens, in
turn, or ahead of the batch: the bits of separate outputs."""
import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests.test_rope_gpu import DT, EPS, freqs, heads, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("order", [(0, 2, 1, 3), (2, 0, 1, 3), (1, 0, 2, 3),
                                   (0, 1, 2, 3), "in turn"])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
def test_parts_of_a_packed_buffer(order, D, dtype):
    """order: the dimensions (batch, token, head) as they lie in memory."""
    B, S, Hq, Hkv = 3, 37, 6, 2
    if order == "in turn":
        Hq = Hkv
    x = [heads(B, S, H, D, dtype, 5 + i).cuda()
         for i, H in enumerate((Hq, Hkv))]
    dy = [heads(B, S, H, D, dtype, 20 + i).transpose(1, 2).contiguous().cuda()
          for i, H in enumerate((Hq, Hkv, Hkv))]
    w = [weight(D, torch.float32, 30 + i).cuda() for i in range(2)]
    rope = attn.Rope(freqs(D), D)
    kw = dict(q_weight=w[0], k_weight=w[1], eps=EPS)
    want = attn.qk_rope_bwd(rope, dy[0], dy[1], *x, dv=dy[2], **kw)
    n = Hq + 2 * Hkv
    if order == "in turn":
        room = torch.full((B, S, Hkv, 3, D), 7.0, dtype=DT[dtype],
                          device="cuda")
        parts = room.unbind(3)
    else:
        shape = [(B, S, n, D)[i] for i in order]
        back = [order.index(i) for i in range(4)]
        room = torch.full(shape, 7.0, dtype=DT[dtype], device="cuda")
        parts = room.permute(back).split((Hq, Hkv, Hkv), 2)
    got = attn.qk_rope_bwd(rope, dy[0], dy[1], *x, dv=dy[2], dq_out=parts[0],
                           dk_out=parts[1], dv_out=parts[2], **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with pytest.raises(attn.AttnError):
        attn.qk_rope_bwd(rope, dy[0], dy[1], *x, dv=dy[2], dq_out=parts[0],
                         dk_out=parts[1], dv_out=parts[1], **kw)
