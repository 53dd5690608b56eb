"""Values at the ends of fp32's range behind a shared prefix, in many parts.

Tolerances as in test_prefix_gpu: O is rounded once (2^-8 of itself), the
weights once (2^-8 of sum p |v|), and a weight is off by 2^-11 of itself at most.
"""
import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests.test_prefix_gpu import exact, make, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def check(c, q):
    o, lse = attn.prefix_fwd(c, q)
    want, z, a = exact(c, q, [q.shape[2]] * c.B, True, c.D ** -0.5)
    assert o.isfinite().all()
    half = 2.0 ** -8
    assert ((o.double() - want).abs() <= half * want.abs() +
            (half + 2.0 ** -11) * a).all()
    assert (lse.double() - z).abs().max() <= 2.0 ** -12 + 2.0 ** -20 * 16


# Few rows (a row a warp, spread over warps, four rows a warp), packed rows, rows
# that fill units.
CASES = [(2, 1, 2, 1, 5000, 300), (2, 1, 2, 3, 90, 9000), (70, 8, 4, 2, 700, 50),
         (2, 1, 2, 20, 5000, 300), (9, 6, 2, 60, 300, 300),
         (2, 1, 2, 200, 5000, 300), (1, 2, 3, 20, 9000, 40)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_parts_of_the_largest_values(case, D):
    """An average of numbers near bf16's largest is one: parts' sums of them
    pass fp32's largest number, twice such a number does."""
    B, Hkv, g, Sq, P, own = case
    c = make(B, Hkv, D, P, P, [own - i % 7 for i in range(B)], own, "bf16")
    for x in (c.prefix_v, c.v):
        x.abs_().clamp_(max=1.0).mul_(0.5).add_(1.0).mul_(2.0 ** 127)
    check(c, randn(B, Hkv * g, Sq, D, dtype="bf16", seed=5))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("case", CASES)
def test_parts_of_one_large_value(case, sign):
    """Every value alike: O is that value."""
    B, Hkv, g, Sq, P, own = case
    c = make(B, Hkv, 64, P, P, [own] * B, own, "bf16")
    c.prefix_v.fill_(sign * 1.75 * 2.0 ** 127)
    c.v.fill_(sign * 1.75 * 2.0 ** 127)
    q = randn(B, Hkv * g, Sq, 64, dtype="bf16", seed=6)
    o, _ = attn.prefix_fwd(c, q)
    # (The weights are rounded apart from their sum.)
    assert ((o.double() / (sign * 1.75 * 2.0 ** 127) - 1).abs()
            <= 2.0 ** -7).all()
