"""Handles read the tensors that they were made of: these change in place, and
another one in the place of one is refused rather than not read."""
import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests.test_prefix_gpu import make, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def test_a_cache_s_tensors():
    c = make(2, 1, 64, 100, 100, [50, 49], 60, "f16", fill=0.0)
    q = randn(2, 2, 1, 64, dtype="f16", seed=3)
    first, _ = attn.prefix_fwd(c, q)
    for name in c.held:
        with pytest.raises(attn.AttnError):
            setattr(c, name, getattr(c, name) + 1)
        setattr(c, name, getattr(c, name))
    same, _ = attn.prefix_fwd(c, q)
    assert torch.equal(first, same)
    c.lens += 1
    got, _ = attn.prefix_fwd(c, q)
    again = attn.PrefixCache(c.prefix_k, c.prefix_v, c.prefix_len, c.k, c.v,
                             c.lens)
    want, _ = attn.prefix_fwd(again, q)
    assert torch.equal(got, want) and not torch.equal(got, first)


def test_a_rotation_s_tensors():
    rope = attn.Rope.make(64)
    for name in rope.held:
        with pytest.raises(attn.AttnError):
            setattr(rope, name, getattr(rope, name).clone())
