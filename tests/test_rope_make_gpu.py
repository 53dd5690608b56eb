"""Axes without pairs: positions may be given for all sections."""
import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests.test_rope_gpu import heads, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("sections", [(32, 0), (20, 12, 0), (0, 32, 0, 0),
                                      (8, 0, 24)])
def test_sections_of_no_pairs(sections):
    B, S, D = 2, 9, 64
    x = [heads(B, S, H, D, "bf16", H).cuda() for H in (4, 2)]
    pos = torch.randint(0, 4000, (len(sections), B, S), generator=rng(1),
                        dtype=torch.int32).cuda()
    rope = attn.Rope.make(D, sections=sections)
    got = attn.qk_rope(rope, *x, positions=pos)
    used = max(i for i, n in enumerate(sections) if n) + 1
    want = attn.qk_rope(rope, *x, positions=pos[:used])
    plain = attn.Rope.make(D, sections=sections[:used])
    other = attn.qk_rope(plain, *x, positions=pos[:used])
    dy = [torch.randn_like(y) for y in got[:2]]
    back = attn.qk_rope_bwd(rope, *dy, positions=pos)
    same = attn.qk_rope_bwd(plain, *dy, positions=pos[:used])
    for i in range(2):
        assert torch.equal(got[i], want[i]) and torch.equal(got[i], other[i])
        assert torch.equal(back[i], same[i])
    for bad in (len(sections) + 1, used - 1):
        if bad:
            with pytest.raises(attn.AttnError):
                attn.qk_rope(rope, *x, positions=pos[:1].expand(
                    bad, B, S).contiguous())
