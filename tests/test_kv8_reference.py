"""The CPU reference of the 8-bit cache operators against torch's own E4M3
conversion and hand-computed cases (no GPU)."""
import math

import pytest
import torch

from tests import kv8_reference as ref


def test_decode_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(ref.F8).double()
    got = ref.decode(codes)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


def test_encode_matches_torch_inside_the_range():
    x = torch.cat([torch.linspace(-448, 448, 20001),
                   torch.randn(20000, generator=ref.rng(0)) * 0.02,
                   ref._POS[:-1].float() / 2 + ref._POS[1:].float() / 2])
    want = x.to(ref.F8).view(torch.uint8)
    assert torch.equal(ref.encode(x.double()), want)


def test_encode_saturates():
    x = torch.tensor([449.0, 1e9, -math.inf, math.nan], dtype=torch.float64)
    assert ref.decode(ref.encode(x)).tolist()[:3] == [448.0, 448.0, -448.0]
    assert ref.encode(x)[3] == 127


@pytest.mark.parametrize("amax,want", [
    (448.0, 1.0), (448.0001, 2.0), (1.75, 2.0 ** -8), (1.0, 2.0 ** -8),
    (0.0, 2.0 ** -126), (1e-45, 2.0 ** -126), (3.38e38, 2.0 ** 120)])
def test_tight(amax, want):
    assert ref.tight(amax) == want


def test_append_grows_a_block():
    c = ref.Cache(1, 1, 16, 64, 16)
    x = torch.ones(1, 1, 1, 64)
    c.lens = [1]
    c.append(x, x)
    assert float(c.scale["k"][0, 0, 0]) == 2.0 ** -8
    c.lens = [2]
    c.append(1000 * x, 0.5 * x)
    assert float(c.scale["k"][0, 0, 0]) == 4.0  # 1000 <= 448 * 4
    assert float(c.scale["v"][0, 0, 0]) == 2.0 ** -8
    assert c.values("k", 0, 0)[0].tolist() == [1.0] * 64
    assert c.values("k", 0, 0)[1].tolist() == [1024.0] * 64  # nearest code
    assert c.values("v", 0, 0)[1].tolist() == [0.5] * 64


def test_attention_of_one_token_is_its_value():
    c = ref.filled(1, 2, 8, 64, 16, [1], 3)
    q = torch.randn(1, 4, 1, 64, generator=ref.rng(4)).half()
    o, lse, w, *_ = ref.attention(c, q, 0.125, True)
    for h in range(4):
        assert torch.allclose(o[0, h, 0], c.values("v", 0, h // 2)[0])
    assert w[0, :, 0].tolist() == pytest.approx([2.0, 2.0])


def test_evict_order_ties_and_nan():
    c = ref.filled(1, 1, 8, 64, 16, [6], 5)
    w = torch.tensor([[[0.5, math.nan, 0.5, 2.0, 0.5, 0.0, 9.0, 9.0]]])
    out, ow, idx = c.evict(w, 4, 1, 8)
    assert idx[0, 0].tolist() == [0, 2, 3, 5]
    assert out.lens == [4]
    assert ow[0, 0].tolist() == [0.5, 0.5, 2.0, 0.0, 0, 0, 0, 0]
    kept = c.values("k", 0, 0)[[0, 2, 3, 5]]
    assert torch.equal(out.values("k", 0, 0), kept)
