"""8-bit cache operators at the ends of their range, on the GPU against the
float64 reference."""
import math

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests import kv8_reference as ref
from tests.test_kv8_gpu import (  # noqa: F401
    built, check_fwd, clean_status, run_fwd, same_cache, upload)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ large scales

@pytest.mark.parametrize("D,block", [(64, 16), (128, 64)])
@pytest.mark.parametrize("scale", [
    2.0 ** 125, 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 126, 1.75 * 2.0 ** 127,
    1.25 * 2.0 ** -126])
def test_append_into_a_block_that_keeps_a_scale_at_the_end_of_the_range(
        scale, D, block):
    c = ref.filled(1, 2, 40, D, block, [5], 1)
    for n in "kv":
        c.scale[n][:, :, 0] = scale
    g = ref.rng(7)
    x = (torch.rand(1, 2, 9, D, generator=g) * 2 - 1).double()
    x = x * torch.exp2((-8 * torch.rand(1, 2, 9, 1, generator=g)).double())
    # Up to 2^127.99 or 440 scales, whichever is less.
    x = (x * min(2.0 ** 127.99, 440 * scale)).bfloat16()
    c.lens = [14]
    gpu = upload(c)
    attn.kv8_append(gpu, x.cuda(), x.cuda())
    c.append(x, x)
    if math.frexp(scale)[0] == 0.5:  # a power of two: exact
        same_cache(gpu, c)
        return
    # The quotient's fp32 rounding moves it across a tie at most: codes differ
    # by one step, and seldom.
    for n in "kv":
        a = getattr(gpu, n).view(torch.uint8).cpu()[:, :, :14].int()
        b = c.code[n][:, :, :14].int()
        assert int((a - b).abs().max()) <= 1
        assert float((a != b).float().mean()) < 0.01
        assert torch.equal(getattr(gpu, n + "_scale").cpu().double(),
                           c.scale[n])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("top", [120, 127])
def test_evict_of_numbers_past_the_largest_fp32(top, in_place):
    """A code times its scale may exceed 2^128 (bf16's largest numbers round
    up to it): the kept block's scale is still that of its largest number."""
    B, H, cap, D, block, keep = 1, 2, 256, 64, 16, 90
    c = ref.filled(B, H, cap, D, block, [cap], 75)
    g = ref.rng(76)
    for n in "kv":
        e = torch.randint(0, 9, c.scale[n].shape, generator=g)
        c.scale[n] = torch.exp2((top - e).double())
        # Blocks of zeros under every scale, and of the smallest ones.
        c.code[n][:, :, 32:48] = 0
        c.code[n][:, :, 0:16, 0] = 0x7E
        c.scale[n][:, :, 5] = 2.0 ** -126
        c.scale[n][:, :, 6] = 2.0 ** -120
    w = torch.rand(B, H, cap, generator=g)
    want, ow, idx = c.evict(w, keep, 10, cap)
    gpu = upload(c)
    out = None if in_place else upload(ref.Cache(B, H, cap, D, block))
    out, out_w, got = attn.kv8_evict(gpu, w.cuda(), keep, 10, out=out)
    assert torch.equal(got.cpu(), idx)
    assert torch.equal(out_w.cpu(), ow)
    if in_place:
        nb = -(-keep // block)
        for n in "kv":
            want.code[n][:, :, keep:] = c.code[n][:, :, keep:]
            want.scale[n][:, :, nb:] = c.scale[n][:, :, nb:]
    same_cache(out, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq", [2, 64, 150])
def test_fwd_weights_of_keys_near_the_largest_fp32(Sq, D):
    """Keys of 2^115 under queries of 2^-112: scores of ordinary size."""
    c = ref.filled(2, 2, 300, D, 32, [300, 170], 161)
    c.scale["k"] *= 2.0 ** 115
    q = torch.randn(2, 4, Sq, D, generator=ref.rng(162)) * 2.0 ** -112
    check_fwd(c, q.bfloat16(), scale=0.125 / math.sqrt(D))


# --------------------------------------------------- V scales far apart

def uneven(B, H, cap, D, block, gap, big):
    """A cache whose first `big` tokens have V scales `gap` times the others'
    and next to no weight under q = (1, 0, ..), followed by `big` tokens of
    weight 1 whose values are 0 in the first half of D; the rest share weights
    of 2^-11 to 2^-19 and values of one sign."""
    g = ref.rng(171)
    some = min(2, H)  # heads that differ
    k = torch.randn(1, some, cap, D, generator=g) * 0.5
    k[..., 0] = -7.5 - 5.5 * torch.rand(1, some, cap, generator=g)
    k[:, :, :big, 0] = -44.0
    k[:, :, big:2 * big, 0] = 0.0
    v = 0.5 + 0.5 * torch.rand(1, some, cap, D, generator=g)
    v[:, :, big:2 * big, :D // 2] = 0.0
    c = ref.Cache(1, some, cap, D, block)
    c.lens = [cap]
    c.append(k.half(), v.half())
    c.scale["v"][:, :, :big // block] *= gap
    for n in "kv":
        c.code[n] = c.code[n].repeat(B, H // some, 1, 1)
        c.scale[n] = c.scale[n].repeat(B, H // some, 1)
    c.B, c.H, c.lens = B, H, [cap] * B
    return c


UNEVEN = [
    # B, H, cap: segments by clusters, cut, one to a CTA or a few.
    (2, 2, 700), (1, 2, 3000), (1, 4, 6000),
    # As many segments as CTAs: each is walked by one.
    (10, 64, 1100),
]


@pytest.mark.parametrize("D,block", [(64, 32), (128, 16), (64, 128)])
@pytest.mark.parametrize("rows", [1, 3, 12, 40])
@pytest.mark.parametrize("gap", [12, 14, 15])
@pytest.mark.parametrize("case", UNEVEN)
def test_fwd_small_values_beside_a_block_of_a_large_scale(case, gap, rows, D,
                                                          block):
    """Up to 2^15 apart, block scales cost no precision: the output comes from
    blocks far below the largest scale and from weights far below 1."""
    B, H, cap = case
    c = uneven(B, H, cap, D, block, 2.0 ** gap, 128)
    q = torch.zeros(B, H, rows, D)
    q[..., 0] = 1.0
    check_fwd(c, q.half(), causal=False, scale=1.0, with_w=False,
              where="cuda")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [2, 64])  # units cut, whole
@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("gap", [16, 22, 24, 25, 26, 32, 33, 40])
def test_fwd_block_scales_further_apart(gap, rows, H, D):
    """Few rows hold any number exactly, many rows up to a distance of 2^22.
    Beyond, numbers are off by 2^-23 of the largest scale S at most: V's halves
    are held in units of S / 2^7, so a scale of S / 2^32 or less has a factor
    of 2^-25 or less, which fp16 rounds to 0, and loses numbers of up to
    448 * 2^-32 S = 2^-23.2 S; above that the halves are rounded to multiples
    of 2^-24 units, 2^-32 S off."""
    B, cap, block = 1, 700, 32
    c = uneven(B, H, cap, D, block, 2.0 ** gap, 128)
    q = torch.zeros(B, H, rows, D)
    q[..., 0] = 1.0
    q = q.bfloat16()
    out, lse, _, _ = run_fwd(c, q, False, scale=1.0, with_w=False)
    o_r, l_r, _, t_o, t_l, _ = ref.attention(c, q, 1.0, False)
    largest = float(c.scale["v"].max())
    extra = 2.0 ** -23 * largest if rows > 16 and gap > 22 else 0.0
    e = (out.double() - o_r).abs()
    assert bool((e <= t_o + extra).all()), float((e - t_o).max() / largest)
    assert bool(((lse.double() - l_r).abs() <= t_l).all())


# ------------------------------------------ values at the ends of the range

ENDS = [
    # Hq, Hkv, cap, len, Sq: clusters, cut, a long cut one, whole units, split
    # ones.
    (4, 2, 300, 300, 1), (4, 2, 2000, 1999, 2), (8, 1, 9000, 9000, 1),
    (2, 2, 200, 200, 40), (4, 2, 5000, 5000, 64), (2, 1, 3000, 2222, 300),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("exponent", [-126, -120, 110, 119])
@pytest.mark.parametrize("case", ENDS)
def test_fwd_values_at_the_ends_of_the_range(case, exponent, D):
    """V of one sign under flat weights: every output is an average of them,
    of their size, also where their sum leaves fp32."""
    Hq, Hkv, cap, n, Sq = case
    g = ref.rng(181)
    c = ref.filled(1, Hkv, cap, D, 64, [n], 182)
    # Codes 0x30 to 0x7E: 0.5 to 448.
    c.code["v"][:, :, :n] = torch.randint(
        0x30, 0x7F, (1, Hkv, n, D), generator=g, dtype=torch.uint8)
    c.scale["v"][c.scale["v"].isfinite()] = 2.0 ** exponent
    q = (torch.randn(1, Hq, Sq, D, generator=g) * 0.1).bfloat16()
    out, lse, _, _ = run_fwd(c, q, with_w=False)
    o_r, l_r, _, t_o, t_l, _ = ref.attention(c, q, D ** -0.5, True)
    # The bound without its absolute term; half of bf16's least step instead.
    t_o = t_o - 1e-30 + 2.0 ** -134
    e = (out.double() - o_r).abs()
    assert bool((e <= t_o).all()), float((e / o_r.abs()).max())
    assert bool(((lse.double() - l_r).abs() <= t_l).all())


# ------------------------------------------------- rows that see nothing

@pytest.mark.parametrize("cap", [100, 5000])
@pytest.mark.parametrize("Sq", [3, 40, 200])
def test_fwd_rows_that_see_nothing_beside_a_nan_value(Sq, cap):
    """Two tokens and Sq rows at positions 2 - Sq .. 1: all but the last two
    see none and get 0, though V's codes are NaN."""
    c = ref.filled(1, 2, cap, 64, 16, [2], 191)
    c.code["v"][:, :, :2] = 0x7F
    q = torch.randn(1, 4, Sq, 64, generator=ref.rng(192)).half()
    w = [None, torch.zeros(1, 2, cap).cuda()]
    for weights in w:
        out, lse = attn.kv8_fwd(upload(c), q.cuda(), weights=weights)
        out, lse = out.cpu(), lse.cpu()
        assert bool((out[:, :, :-2] == 0).all())
        assert bool((lse[:, :, :-2] == -math.inf).all())
        assert bool(out[:, :, -2:].isnan().all())
        assert bool(lse[:, :, -2:].isfinite().all())
