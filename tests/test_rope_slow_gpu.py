"""Pairs that turn slowly, at near positions: small angles to their own accuracy.

Of a pair (1, 0) the second number becomes sin t.  The angle is off by 2^-23 of
itself and by the phase's half unit, 2^-65 of a turn a position (below 2^-33 of
the smallest angle here); its sine and the product by 2^-22 together; and it is
rounded once, by half a bf16 step of it.
"""
import pytest
import torch

import attention_attn_fwd_gb300 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_small_angles(D, interleaved):
    n = D // 2
    freq = 10.0 ** torch.linspace(-9, -3, n, dtype=torch.float64)
    rope = attn.Rope(freq, D, interleaved=interleaved)
    pos = torch.tensor([[1, -1, 2, 5, -17, 100, 0]], dtype=torch.int32)
    S = pos.shape[1]
    x = torch.zeros(1, S, 1, D, dtype=torch.bfloat16)
    a = slice(0, D, 2) if interleaved else slice(0, n)
    b = slice(1, D, 2) if interleaved else slice(n, D)
    x[..., a] = 1.0
    t = pos[0].double()[:, None] * freq
    got = attn.qk_rope(rope, x.cuda(), x.cuda(), positions=pos.cuda())
    back = attn.qk_rope_bwd(rope, x.transpose(1, 2).contiguous().cuda(),
                            x.transpose(1, 2).contiguous().cuda(),
                            positions=pos.cuda())
    for y, sign in ((got[0][0, 0], 1), (got[1][0, 0], 1), (back[0][0, :, 0], -1)):
        y = y.double().cpu()
        want = sign * torch.sin(t)
        err = (y[:, b] - want).abs()
        # (bf16: half a step is eps / 2 = 2^-8 of a number at most.)
        half = torch.finfo(torch.bfloat16).eps / 2
        assert (err <= (half + 2.0 ** -21) * want.abs()).all(), \
            float((err / want.abs()).nan_to_num().max())
        assert (y[:, a] - torch.cos(t)).abs().max() <= half
