"""Rope.make without a GPU: refusals that come before the device's."""
import pytest

import attention_attn_fwd_gb300 as attn
from attention_attn_fwd_gb300 import build as cuda_build


@pytest.mark.parametrize("rot", [1, 7, 9, 12, 63, 65, -8])
def test_elements_that_are_no_multiple_of_eight(rot):
    cuda_build.build()
    for sections in (None, (rot // 2,)):
        with pytest.raises(attn.AttnError) as e:
            attn.Rope.make(64, rot=rot, sections=sections, device="cpu")
        assert e.value.status == attn.ATTN_ERR_UNSUPPORTED
