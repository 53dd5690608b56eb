"""Norm and rotation of heads on the GPU, and their gradients, against float64.

Tolerances.  A result is rounded once, off by half a step (finfo.eps / 2 of
itself, half of the smallest subnormal number at least), and computed in fp32:
squares summed over 8 numbers and a tree, one rsqrt and a product leave a and b
of a pair off by less than 2^-21 of themselves, cos and sin are off by less
than 2^-21, so a cos - b sin is off by less than 2^-20 (|a| + |b|).
"""
import math

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests import rope_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def clean_status():
    attn.attn_device_status()
    yield
    torch.cuda.synchronize()
    assert attn.attn_device_status() == (0, 0)


def rng(seed):
    return torch.Generator().manual_seed(seed)


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def heads(B, S, H, D, dtype, seed):
    x = torch.randn(B, S, H, D, generator=rng(seed), dtype=torch.float64)
    x *= torch.exp(torch.randn(B, S, H, 1, generator=rng(seed + 1),
                               dtype=torch.float64))
    return x.to(DT[dtype])


def weight(D, dtype, seed):
    return (1 + 0.3 * torch.randn(D, generator=rng(seed))).to(dtype)


def bound(want, pair, dtype):
    """Half a step of `want`, and 2^-20 of the pairs' magnitudes."""
    return (torch.finfo(DT[dtype]).eps / 2) * want.abs() + TINY[dtype] + \
        2.0 ** -20 * pair


def near(got, want, tol):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    bad &= ~(got.isnan() & want.isnan()) & (got != want)
    assert not bad.any(), (int(bad.sum()), float((got - want)[bad].abs().max()))


def forward(x, w, t, interleaved, dtype):
    """(definition, magnitude of each element's pair) in float64."""
    n = ref.norm(x.double(), None if w is None else w.double(), EPS)
    y = ref.rotate(n, t, interleaved)
    i, j = ref.places(2 * t.shape[-1], interleaved)
    pair = n.abs()
    both = n[..., i].abs() + n[..., j].abs()
    pair[..., i] = both
    pair[..., j] = both
    return y, pair


CASES = [
    # B, S, Hq, Hkv, D, rot, axes, interleaved, norm, w32, packed
    (1, 1, 1, 1, 64, 64, 1, False, True, False, False),
    (1, 1, 32, 8, 128, 128, 1, False, True, False, True),
    (3, 17, 4, 2, 64, 32, 1, True, True, True, True),
    (2, 33, 6, 3, 128, 96, 3, False, True, True, False),
    (2, 31, 5, 5, 64, 48, 2, True, False, False, True),
    (1, 130, 7, 1, 128, 8, 1, False, True, False, False),
    (4, 9, 3, 1, 64, 0, 1, False, True, False, True),
    (1, 1000, 12, 4, 128, 128, 1, True, False, False, True),
    (5, 67, 1, 1, 64, 16, 3, True, True, False, False),
]


def make(case, dtype, seed):
    B, S, Hq, Hkv, D, rot, axes, inter, norm, w32, packed = case
    if packed:
        qkv = heads(B, S, Hq + 2 * Hkv, D, dtype, seed).cuda()
        q, k, v = qkv.split((Hq, Hkv, Hkv), 2)
    else:
        q, k, v = (heads(B, S, H, D, dtype, seed + i).cuda()
                   for i, H in enumerate((Hq, Hkv, Hkv)))
    wt = torch.float32 if w32 else DT[dtype]
    w = [weight(D, wt, seed + 7 + i) if norm else None for i in range(2)]
    ax = [i * axes * 2 // rot for i in range(rot // 2)] if axes > 1 else None
    rope = attn.Rope(freqs(rot), D, axes=ax, interleaved=inter)
    pos = None
    if axes > 1:
        pos = torch.randint(-5, 4000, (axes, B, S), generator=rng(seed + 9),
                            dtype=torch.int32)
    count = torch.arange(S).expand(1, B, S) if pos is None else pos
    t = ref.angles(freqs(rot), ax or [0] * (rot // 2), count)
    return rope, (q, k, v), w, pos, t


def gpu(x):
    return None if x is None else x.cuda()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, dtype):
    inter = case[7]
    rope, (q, k, v), w, pos, t = make(case, dtype, 3)
    qo, ko, vo = attn.qk_rope(rope, q, k, v, gpu(w[0]), gpu(w[1]), EPS,
                              positions=gpu(pos))
    for x, wx, got in ((q, w[0], qo), (k, w[1], ko)):
        y, pair = forward(x.cpu(), wx, t, inter, dtype)
        near(got, y.transpose(1, 2),
             bound(y, pair, dtype).transpose(1, 2))
    assert torch.equal(vo, v.transpose(1, 2))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_into_a_cache(dtype):
    """Rows go to places lens - n .. lens - 1; all else keeps its bits."""
    B, S, Hq, Hkv, D, cap = 4, 9, 6, 2, 64, 40
    lens, new = [40, 9, 23, 5], [9, 9, 0, 4]
    rope = attn.Rope(freqs(D), D)
    q, k, v = (heads(B, S, H, D, dtype, 5 + H + i).cuda()
               for i, H in enumerate((Hq, Hkv, Hkv)))
    w = weight(D, torch.float32, 1)
    old = [heads(B, cap, Hkv, D, dtype, 9).transpose(1, 2).contiguous()
           for _ in range(2)]
    oldq = heads(B, S, Hq, D, dtype, 8).transpose(1, 2).contiguous()
    out = [x.clone().cuda() for x in (oldq, *old)]
    lens_t = torch.tensor(lens, dtype=torch.int32)
    offset = 3000
    attn.qk_rope(rope, q, k, v, w.cuda(), w.cuda(), EPS,
                 lens=lens_t.cuda(),
                 new_lens=torch.tensor(new, dtype=torch.int32).cuda(),
                 offset=torch.tensor([offset], dtype=torch.int32).cuda(),
                 q_out=out[0], k_out=out[1], v_out=out[2])
    first = lens_t - torch.tensor(new)
    pos = first[:, None] + torch.arange(S) + offset
    t = ref.angles(freqs(D), [0] * 32, pos[None])
    yq, pq = forward(q.cpu(), w, t, False, dtype)
    yk, pk = forward(k.cpu(), w, t, False, dtype)
    for b in range(B):
        n, f = new[b], int(first[b])
        near(out[0][b, :, :n], yq[b, :n].transpose(0, 1),
             bound(yq, pq, dtype)[b, :n].transpose(0, 1))
        near(out[1][b, :, f:f + n], yk[b, :n].transpose(0, 1),
             bound(yk, pk, dtype)[b, :n].transpose(0, 1))
        assert torch.equal(out[2][b, :, f:f + n].cpu(),
                           v[b, :n].transpose(0, 1).cpu())
        assert torch.equal(out[0][b, :, n:].cpu(), oldq[b, :, n:])
        for got, was in zip(out[1:], old):
            assert torch.equal(got[b, :, :f].cpu(), was[b, :, :f])
            assert torch.equal(got[b, :, f + n:].cpu(), was[b, :, f + n:])


def test_rows_without_a_cache_and_with_counts():
    rope = attn.Rope(freqs(64), 64)
    q, k = (heads(2, 5, H, 64, "bf16", H).cuda() for H in (2, 1))
    out = torch.full((2, 2, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((2, 1, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    new = torch.tensor([0, 3], dtype=torch.int32).cuda()
    got = attn.qk_rope(rope, q, k, new_lens=new, q_out=out, k_out=ko)
    assert got[2] is None
    whole = attn.qk_rope(rope, q, k)
    for a, b in ((out, whole[0]), (ko, whole[1])):
        assert torch.equal(a[1, :, :3], b[1, :, :3])
        assert (a[0] == 7).all() and (a[1, :, 3:] == 7).all()


@pytest.mark.parametrize("first", [0, 100000, 2 ** 24 - 3, 2 ** 31 - 6,
                                   -(2 ** 31)])
def test_far_positions(first):
    """Whole turns are dropped exactly: as exact at 2^31 as at 0."""
    D, S = 128, 5
    f = [1.0, 0.7310585786, 3.3e-5] + freqs(D)[3:]
    rope = attn.Rope(f, D)
    q = heads(1, S, 2, D, "f16", 1)
    pos = (first + torch.arange(S)).to(torch.int32).view(1, 1, S)
    got = attn.qk_rope(rope, q.cuda(), q.cuda(), positions=pos.cuda())[0]
    # The float64 angle of the reference is itself off by 2^31 * 2^-53.
    t = ref.angles(f, [0] * 64, pos.long())
    y, pair = forward(q, None, t, False, "f16")
    near(got, y.transpose(1, 2), bound(y, pair, "f16").transpose(1, 2))


def test_counting_passes_int32():
    """Counted positions are 64-bit sums of an offset and a place."""
    rope = attn.Rope([1.0] * 32, 64)
    q = heads(1, 8, 1, 64, "f16", 1)
    off = torch.tensor([2 ** 31 - 4], dtype=torch.int32)
    got = attn.qk_rope(rope, q.cuda(), q.cuda(), offset=off.cuda())[0]
    t = (2 ** 31 - 4 + torch.arange(8, dtype=torch.float64)).view(1, 8, 1)
    y, pair = forward(q, None, t.expand(1, 8, 32), False, "f16")
    near(got, y.transpose(1, 2), bound(y, pair, "f16").transpose(1, 2))


def test_large_numbers_are_normed():
    """Rows whose squares pass fp32, beside ordinary ones of the same warp."""
    D = 64
    x = heads(1, 6, 2, D, "bf16", 4)
    x[0, 1] *= 2.0 ** 90
    x[0, 2, 0] = torch.finfo(torch.bfloat16).max
    x[0, 4] *= 2.0 ** 64
    w = weight(D, torch.float32, 2)
    rope = attn.Rope(freqs(D), D)
    got = attn.qk_rope(rope, x.cuda(), x.cuda(), None, w.cuda(), w.cuda(),
                       EPS)[0]
    t = ref.angles(freqs(D), [0] * 32, torch.arange(6).view(1, 1, 6))
    y, pair = forward(x, w, t, False, "bf16")
    near(got, y.transpose(1, 2), bound(y, pair, "bf16").transpose(1, 2))


def test_infinities_and_nan_stay_in_their_rows():
    D = 64
    x = heads(1, 4, 3, D, "f16", 4)
    clean = attn.qk_rope(attn.Rope(freqs(D), D), x.cuda(), x.cuda())[0]
    y = x.clone()
    y[0, 1, 1, 5] = math.nan
    y[0, 2, 0, 60] = math.inf
    for w in (None, torch.ones(D).cuda()):
        base = attn.qk_rope(attn.Rope(freqs(D), D), x.cuda(), x.cuda(), None,
                            w, w)[0]
        got = attn.qk_rope(attn.Rope(freqs(D), D), y.cuda(), y.cuda(), None,
                           w, w)[0]
        hit = torch.zeros(1, 3, 4, dtype=torch.bool)
        hit[0, 1, 1] = hit[0, 0, 2] = True
        assert torch.equal(got.cpu()[~hit], base.cpu()[~hit])
        assert (~got.cpu()[hit].isfinite()).any(-1).all()
    # Elements that are not rotated do not touch each other.
    rope = attn.Rope(freqs(16), D)
    got = attn.qk_rope(rope, y.cuda(), y.cuda())[0].cpu()
    want = y.transpose(1, 2).clone()
    assert torch.equal(got[..., 16:].isnan(), want[..., 16:].isnan())
    assert torch.equal(got[0, 0, 2, 16:], want[0, 0, 2, 16:])
    assert clean.isfinite().all()


# --------------------------------------------------------------- backward

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, dtype):
    """dx = r (g - x^ mean(g x^)) is off by half a step and by less than 2^-19
    of its terms' magnitudes; a weight's gradient, a sum in chains of at most
    200, by less than 2^-16 of the sum of its terms' magnitudes."""
    B, S, Hq, Hkv, D, rot, axes, inter, norm, w32, packed = case
    rope, (q, k, v), w, pos, t = make(case, dtype, 3)
    dy = [heads(B, S, H, D, dtype, 50 + i).transpose(1, 2).contiguous()
          for i, H in enumerate((Hq, Hkv, Hkv))]
    kw = {}
    if packed:
        out = torch.full((B, S, Hq + 2 * Hkv, D), math.nan, device="cuda",
                         dtype=DT[dtype])
        kw = dict(zip(("dq_out", "dk_out", "dv_out"),
                      out.split((Hq, Hkv, Hkv), 2)))
    got = attn.qk_rope_bwd(rope, dy[0].cuda(), dy[1].cuda(), q, k,
                           dv=dy[2].cuda(), q_weight=gpu(w[0]),
                           k_weight=gpu(w[1]), eps=EPS, positions=gpu(pos),
                           **kw)
    for i, x in enumerate((q, k)):
        d = dy[i].double().transpose(1, 2)
        w64 = None if w[i] is None else w[i].double()
        dx, dw = ref.qk_rope_bwd(d, x.cpu().double(), w64, t, inter, EPS)
        dn, pair = forward(d, None, -t, inter, dtype)
        if w64 is None:
            near(got[i], dx, bound(dx, pair, dtype))
            assert got[3 + i] is None
            continue
        y = x.cpu().double()
        r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
        xhat = y * r
        g = pair * w64.abs()
        terms = r * (g + xhat.abs() * (g * xhat.abs()).mean(-1, keepdim=True))
        near(got[i], dx, (torch.finfo(DT[dtype]).eps / 2) * dx.abs() +
             TINY[dtype] + 2.0 ** -19 * terms)
        near(got[3 + i], dw,
             2.0 ** -16 * (pair * xhat.abs()).sum(dim=(0, 1, 2)))
    assert torch.equal(got[2], dy[2].cuda().transpose(1, 2))


def test_backward_against_differences():
    """The change of sum(y dy) along a direction, by central differences of
    the float64 forward of step 2^-14 (third-order terms below 2^-22)."""
    B, S, H, D = 2, 7, 3, 64
    rope = attn.Rope(freqs(D), D)
    x = heads(B, S, H, D, "f16", 1)
    dy = heads(B, S, H, D, "f16", 2).transpose(1, 2).contiguous()
    w = weight(D, torch.float32, 3)
    got = attn.qk_rope_bwd(rope, dy.cuda(), dy.cuda(), x.cuda(), x.cuda(),
                           q_weight=w.cuda(), k_weight=w.cuda(), eps=EPS)
    t = ref.angles(freqs(D), [0] * 32, torch.arange(S).expand(1, B, S))
    u = torch.randn(x.shape, generator=rng(4), dtype=torch.float64)
    uw = torch.randn(D, generator=rng(5), dtype=torch.float64)
    h = 2.0 ** -14

    def loss(xx, ww):
        return (ref.qk_rope(xx, ww, t, False, EPS) *
                dy.double().transpose(1, 2)).sum()

    X, W = x.double(), w.double()
    by_x = (loss(X + h * u, W) - loss(X - h * u, W)) / (2 * h)
    by_w = (loss(X, W + h * uw) - loss(X, W - h * uw)) / (2 * h)
    dx, dw = got[0].double().cpu(), got[3].double().cpu()
    # Each product is off by half an fp16 step of dx: 2^-11 of its size.
    assert abs((dx * u).sum() - by_x) <= 2.0 ** -11 * (dx * u).abs().sum()
    assert abs((dw * uw).sum() - by_w) <= 2.0 ** -14 * (dw * uw).abs().sum()


def test_backward_of_large_numbers():
    D = 64
    x = heads(1, 3, 1, D, "bf16", 4)
    x[0, 1] *= 2.0 ** 80
    dy = heads(1, 3, 1, D, "bf16", 5).transpose(1, 2).contiguous()
    w = torch.ones(D)
    got = attn.qk_rope_bwd(attn.Rope([], D), dy.cuda(), dy.cuda(), x.cuda(),
                           x.cuda(), q_weight=w.cuda(), k_weight=w.cuda(),
                           eps=EPS)
    t = torch.zeros(1, 3, 0)
    dx, dw = ref.qk_rope_bwd(dy.double().transpose(1, 2), x.double(),
                             w.double(), t, False, EPS)
    for i in (0, 2):
        near(got[0][:, i], dx[:, i], 2.0 ** -8 * dx[:, i].abs().max())
    near(got[0][:, 1], dx[:, 1], 2.0 ** -7 * dx[:, 1].abs().max())
    near(got[3], dw, 2.0 ** -16 * (3 * D + dw.abs()))


def test_empty_calls():
    rope = attn.Rope(freqs(64), 64)
    w = torch.ones(64, device="cuda")
    for B, S in ((0, 4), (2, 0)):
        x = torch.zeros(B, S, 2, 64, device="cuda", dtype=torch.float16)
        y = attn.qk_rope(rope, x, x, x, w, w)
        assert y[0].shape == (B, 2, S, 64)
        d = attn.qk_rope_bwd(rope, *y[:2], x, x, dv=y[2], q_weight=w,
                             k_weight=w, dq_weight=w + 1, dk_weight=w + 2)
        assert not d[3].any() and not d[4].any()


LAYOUTS = ["heads first", "part of a longer row", "one batch entry for all"]


def laid_out(x, layout):
    """The values of x [B, S, H, D] in memory of another layout."""
    B, S, H, D = x.shape
    if layout == "heads first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "part of a longer row":
        room = torch.full((B, S, H + 3, D + 8), math.nan, dtype=x.dtype,
                          device=x.device)
        room[:, :, 1:H + 1, 8:] = x
        return room[:, :, 1:H + 1, 8:]
    return x[:1].expand(B, S, H, D)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_strided_inputs(layout):
    B, S, D = 3, 21, 64
    rope = attn.Rope(freqs(D), D)
    w = weight(D, torch.float32, 1).cuda()
    x = [laid_out(heads(B, S, H, D, "f16", H).cuda(), layout)
         for H in (6, 2, 2)]
    got = attn.qk_rope(rope, *x, w, w, EPS)
    want = attn.qk_rope(rope, *[y.contiguous() for y in x], w, w, EPS)
    dy = [heads(B, S, H, D, "f16", 9).transpose(1, 2).contiguous().cuda()
          for H in (6, 2, 2)]
    back = attn.qk_rope_bwd(rope, *dy[:2], x[0], x[1], dv=dy[2], q_weight=w,
                            k_weight=w, eps=EPS)
    plain = attn.qk_rope_bwd(rope, *dy[:2], x[0].contiguous(),
                             x[1].contiguous(), dv=dy[2], q_weight=w,
                             k_weight=w, eps=EPS)
    for a, b in zip((*got, *back), (*want, *plain)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout", LAYOUTS[:2])
def test_strided_gradients(layout):
    B, S, D = 2, 19, 128
    rope = attn.Rope(freqs(D), D)
    dy = [heads(B, S, H, D, "bf16", 9).transpose(1, 2).contiguous().cuda()
          for H in (3, 1, 1)]
    want = attn.qk_rope_bwd(rope, *dy[:2], dv=dy[2])
    out = [laid_out(torch.zeros_like(x), layout) for x in want[:3]]
    got = attn.qk_rope_bwd(rope, *dy[:2], dv=dy[2], dq_out=out[0],
                           dk_out=out[1], dv_out=out[2])
    for a, b, c in zip(got, want, out):
        assert a is c and torch.equal(a, b)


def test_one_of_two_is_normed():
    B, S, D = 2, 9, 64
    rope = attn.Rope(freqs(D), D)
    w = weight(D, torch.float16, 1).cuda()
    q, k = (heads(B, S, H, D, "f16", H).cuda() for H in (4, 2))
    both, none = attn.qk_rope(rope, q, k, None, w, w, EPS), \
        attn.qk_rope(rope, q, k)
    got = attn.qk_rope(rope, q, k, None, w, None, EPS)
    assert torch.equal(got[0], both[0]) and torch.equal(got[1], none[1])
    got = attn.qk_rope(rope, q, k, None, None, w, EPS)
    assert torch.equal(got[0], none[0]) and torch.equal(got[1], both[1])
    dy = [heads(B, S, H, D, "f16", 9).transpose(1, 2).contiguous().cuda()
          for H in (4, 2)]
    both = attn.qk_rope_bwd(rope, *dy, q, k, q_weight=w, k_weight=w, eps=EPS)
    none = attn.qk_rope_bwd(rope, *dy)
    got = attn.qk_rope_bwd(rope, *dy, q, None, q_weight=w, eps=EPS)
    assert torch.equal(got[0], both[0]) and torch.equal(got[1], none[1])
    assert torch.equal(got[3], both[3]) and got[4] is None
    got = attn.qk_rope_bwd(rope, *dy, None, k, k_weight=w, eps=EPS)
    assert torch.equal(got[0], none[0]) and torch.equal(got[1], both[1])
    assert got[3] is None and torch.equal(got[4], both[4])


def test_many_heads_and_tokens():
    """Heads and tokens that fill and pass the launch's blocks; a backward whose
    blocks of heads are more than its thread blocks."""
    D = 64
    rope = attn.Rope(freqs(D), D)
    w = weight(D, torch.float32, 1).cuda()
    for B, S, Hq, Hkv in ((1, 1, 513, 27), (3, 683, 9, 7), (1, 3, 9000, 1)):
        q, k = (heads(B, S, H, D, "bf16", 2).cuda() for H in (Hq, Hkv))
        got = attn.qk_rope(rope, q, k, None, w, w, EPS)
        t = ref.angles(freqs(D), [0] * 32, torch.arange(S).expand(1, B, S))
        for x, y in ((q, got[0]), (k, got[1])):
            z, pair = forward(x.cpu(), w.cpu(), t, False, "bf16")
            near(y, z.transpose(1, 2), bound(z, pair, "bf16").transpose(1, 2))
        dy = [torch.randn_like(x) for x in got[:2]]
        back = attn.qk_rope_bwd(rope, *dy, q, k, q_weight=w, k_weight=w,
                                eps=EPS)
        again = attn.qk_rope_bwd(rope, *dy, q, k, q_weight=w, k_weight=w,
                                 eps=EPS)
        for a, b in zip(back, again):
            assert a is None or torch.equal(a, b)
        d = dy[0].double().cpu().transpose(1, 2)
        dx, dw = ref.qk_rope_bwd(d, q.cpu().double(), w.cpu().double(), t,
                                 False, EPS)
        terms = (forward(d, None, -t, False, "bf16")[1] *
                 ref.norm(q.cpu().double(), torch.ones(D), EPS).abs())
        near(back[3], dw, 2.0 ** -16 * terms.sum(dim=(0, 1, 2)))
        assert (back[0].double().cpu() - dx).abs().max() <= \
            2.0 ** -7 * dx.abs().max()


# ------------------------------------------------------ streams and graphs

def test_on_another_stream_and_in_a_graph():
    case = (2, 33, 6, 3, 128, 96, 3, False, True, True, True)
    rope, (q, k, v), w, pos, t = make(case, "bf16", 3)
    w = [x.cuda() for x in w]
    pos = pos.cuda()
    dy = [heads(2, 33, H, 128, "bf16", 50).transpose(1, 2).contiguous().cuda()
          for H in (6, 3, 3)]
    want = attn.qk_rope(rope, q, k, v, *w, EPS, positions=pos)
    back = attn.qk_rope_bwd(rope, *dy[:2], q, k, dv=dy[2], q_weight=w[0],
                            k_weight=w[1], eps=EPS, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = attn.qk_rope(rope, q, k, v, *w, EPS, positions=pos, stream=s)
    got2 = attn.qk_rope_bwd(rope, *dy[:2], q, k, dv=dy[2], q_weight=w[0],
                            k_weight=w[1], eps=EPS, positions=pos, stream=s)
    s.synchronize()
    for a, b in zip((*want, *back), (*got, *got2)):
        assert torch.equal(a, b)
    # Two graphs with workspaces of their own, replayed side by side.
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = attn.qk_rope(rope, q, k, v, *w, EPS, positions=pos)
            o += attn.qk_rope_bwd(rope, *dy[:2], q, k, dv=dy[2],
                                  q_weight=w[0], k_weight=w[1], eps=EPS,
                                  positions=pos)
        graphs.append(g)
        outs.append(o)
    for o in outs:
        for x in o:
            x.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip((*want, *back), o):
            assert torch.equal(a, b)


def test_lengths_out_of_range_are_clamped_and_reported():
    rope = attn.Rope(freqs(64), 64)
    q = heads(3, 4, 1, 64, "f16", 1).cuda()
    cache = torch.zeros(3, 1, 6, 64, device="cuda", dtype=torch.float16)
    lens = torch.tensor([9, -1, 2], dtype=torch.int32).cuda()
    attn.qk_rope(rope, q, q, lens=lens, k_out=cache)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == (attn.ATTN_ERR_INVALID_ARG, 2)
    used = cache.abs().sum(-1)[:, 0].cpu() > 0
    assert used.tolist() == [[False, False, True, True, True, True],
                             [False] * 6, [True, True] + [False] * 4]


# ------------------------------------------------- with the attention itself

def test_a_training_step_through_attention():
    """qk_rope, fwd, bwd and qk_rope_bwd in turn against autograd of the
    definition in float64.  Every stage rounds to bf16 (2^-8 of a value): the
    gradients of the step stay within 2^-5 of their largest, the bound of the
    backward's own parity tests (2e-2) and three more roundings."""
    B, S, Hq, Hkv, D = 2, 200, 4, 2, 64
    qkv = heads(B, S, Hq + 2 * Hkv, D, "bf16", 1)
    w = [weight(D, torch.float32, 2 + i) for i in range(2)]
    do = heads(B, S, Hq, D, "bf16", 6).transpose(1, 2).contiguous()
    rope = attn.Rope.make(D)
    q, k, v = qkv.cuda().split((Hq, Hkv, Hkv), 2)
    qr, kr, vr = attn.qk_rope(rope, q, k, v, w[0].cuda(), w[1].cuda(), EPS)
    o, lse = attn.fwd(qr, kr, vr, causal=True)
    dq, dk, dv = attn.bwd(qr, kr, vr, o, lse, do.cuda(), causal=True)
    back = torch.empty(B, S, Hq + 2 * Hkv, D, device="cuda",
                       dtype=torch.bfloat16)
    parts = back.split((Hq, Hkv, Hkv), 2)
    got = attn.qk_rope_bwd(rope, dq, dk, q, k, dv=dv, q_weight=w[0].cuda(),
                           k_weight=w[1].cuda(), eps=EPS, dq_out=parts[0],
                           dk_out=parts[1], dv_out=parts[2])
    x = qkv.double().requires_grad_()
    ws = [y.double().requires_grad_() for y in w]
    t = ref.angles(freqs(D), [0] * 32, torch.arange(S).expand(1, B, S))
    a, b, c = x.split((Hq, Hkv, Hkv), 2)
    a = ref.rotate_graph(ref.norm(a, ws[0], EPS), t, False).transpose(1, 2)
    b = ref.rotate_graph(ref.norm(b, ws[1], EPS), t, False).transpose(1, 2)
    b, c = (y.repeat_interleave(Hq // Hkv, 1) for y in (b, c.transpose(1, 2)))
    s = a @ b.transpose(2, 3) / math.sqrt(D)
    s = s.masked_fill(~torch.ones(S, S).tril().bool(), -math.inf)
    (torch.softmax(s, -1) @ c).backward(do.double())
    for g, want in ((back, x.grad), (got[3], ws[0].grad),
                    (got[4], ws[1].grad)):
        err = (g.double().cpu() - want).abs().max()
        assert err <= 2.0 ** -5 * want.abs().max(), float(err)


def test_a_decoding_step_into_an_8_bit_cache():
    """qk_rope, kv8_append and kv8_fwd in turn: the keys that the cache holds
    are qk_rope's, to E4M3's half step."""
    B, Hq, Hkv, D, cap, n = 2, 4, 2, 64, 100, 37
    rope = attn.Rope.make(D)
    w = weight(D, torch.float32, 1).cuda()
    cache = attn.KV8Cache.empty(B, Hkv, cap, D, block=32)
    x = heads(B, n + 1, Hq + 2 * Hkv, D, "bf16", 3).cuda()
    whole = attn.qk_rope(rope, *x.split((Hq, Hkv, Hkv), 2), w, w, EPS)
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    for part in (x[:, :n], x[:, n:]):
        q, k, v = part.split((Hq, Hkv, Hkv), 2)
        qr, kr, vr = attn.qk_rope(rope, q, k, v, w, w, EPS, offset=first)
        cache.lens += part.shape[1]
        attn.kv8_append(cache, kr, vr)
        o, lse = attn.kv8_fwd(cache, qr)
        first += part.shape[1]
    scale = cache.k_scale.repeat_interleave(32, 2)[:, :, :n + 1, None]
    held = cache.k[:, :, :n + 1].float() * scale
    off = (held - whole[1].float()).abs()
    assert (off <= 2.0 ** -4 * whole[1].float().abs() +
            2.0 ** -10 * scale).all()
    k, v = (y.repeat_interleave(Hq // Hkv, 1).double() for y in (
        held, cache.v[:, :, :n + 1].float() *
        cache.v_scale.repeat_interleave(32, 2)[:, :, :n + 1, None]))
    s = whole[0][:, :, n:].double() @ k.transpose(2, 3) / math.sqrt(D)
    want = torch.softmax(s, -1) @ v
    # (P is rounded to fp16, O to bf16.)
    assert ((o.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 *
            (torch.softmax(s, -1) @ v.abs())).all()
