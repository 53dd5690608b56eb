"""8-bit cache operators on the GPU against the float64 reference."""
import math

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests import kv8_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


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


def upload(c):
    """KV8Cache with the reference cache's contents."""
    return attn.KV8Cache(
        c.code["k"].cuda(), c.code["v"].cuda(), c.scale["k"].float().cuda(),
        c.scale["v"].float().cuda(),
        torch.tensor(c.lens, dtype=torch.int32).cuda(), c.block)


def counts(new):
    return None if new is None else torch.tensor(
        new, dtype=torch.int32).cuda()


def same_cache(gpu, c, lens=True):
    for n in "kv":
        code = getattr(gpu, n).view(torch.uint8).cpu()
        nan = ((code & 127) == 127) & ((c.code[n] & 127) == 127)
        assert torch.equal(torch.where(nan, 127, code),
                           torch.where(nan, 127, c.code[n])), n
        assert torch.equal(getattr(gpu, n + "_scale").cpu().double(),
                           c.scale[n]), n + "_scale"
    if lens:
        assert gpu.lens.cpu().tolist() == c.lens


# ------------------------------------------------------------------ append

APPENDS = [
    # B, H, cap, D, block, before, new rows given, counts (None: all)
    (1, 1, 1, 64, 16, [0], 1, None),
    (2, 3, 70, 128, 64, [0, 63], 1, None),
    (3, 2, 130, 64, 16, [15, 16, 17], 1, None),
    (2, 2, 300, 128, 128, [127, 100], 2, None),
    (4, 1, 257, 64, 32, [0, 5, 31, 64], 100, [100, 0, 1, 77]),
    (2, 5, 513, 128, 32, [1, 33], 480, [480, 333]),
    (1, 2, 1000, 128, 16, [0], 1000, None),
    (3, 3, 200, 64, 128, [199, 128, 0], 5, [1, 5, 0]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", APPENDS)
def test_append(case, dtype):
    B, H, cap, D, block, before, Sq, new = case
    c = ref.filled(B, H, cap, D, block, before, 1)
    x = [(torch.randn(B, H, Sq, D, generator=ref.rng(s)) *
          torch.exp(torch.randn(B, H, Sq, 1, generator=ref.rng(s + 9)))
          ).to(DT[dtype]) for s in (2, 3)]
    n = [Sq] * B if new is None else new
    c.lens = [a + i for a, i in zip(before, n)]
    gpu = upload(c)
    attn.kv8_append(gpu, x[0].cuda(), x[1].cuda(), new_lens=counts(new))
    c.append(x[0], x[1], new=n)
    same_cache(gpu, c)


def test_append_one_by_one_matches_the_reference_at_every_step():
    B, H, cap, D, block = 2, 2, 80, 64, 32
    c = ref.Cache(B, H, cap, D, block)
    gpu = upload(c)
    for t in range(70):
        x = [(torch.randn(B, H, 1, D, generator=ref.rng(100 * s + t)) *
              2.0 ** (t % 23 - 11)).bfloat16() for s in (1, 2)]
        c.lens = [t + 1] * B
        gpu.lens += 1
        attn.kv8_append(gpu, x[0].cuda(), x[1].cuda())
        c.append(x[0], x[1])
        same_cache(gpu, c)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_extremes(dtype):
    """Zeros, the type's largest and smallest numbers, infinities and NaN."""
    B, H, cap, D, block = 1, 1, 96, 64, 16
    info = torch.finfo(DT[dtype])
    x = torch.zeros(1, 1, 96, 64, dtype=torch.float64)
    x[0, 0, 16:32] = info.max * torch.linspace(-1, 1, 64).double()
    x[0, 0, 32:48] = info.tiny * torch.linspace(-1, 1, 64).double()
    x[0, 0, 48:64, 0] = math.inf
    x[0, 0, 48:64, 1] = -math.inf
    x[0, 0, 48:64, 2] = 3.0
    x[0, 0, 64:80, 3] = math.nan
    x[0, 0, 64:80, 4] = -5.0
    x[0, 0, 80:96] = math.inf
    x = x.to(DT[dtype])
    c = ref.Cache(B, H, cap, D, block)
    c.lens = [96]
    gpu = upload(c)
    attn.kv8_append(gpu, x.cuda(), x.cuda())
    c.append(x, x)
    same_cache(gpu, c)


def test_append_keeps_a_scale_of_other_origin():
    c = ref.filled(1, 1, 64, 64, 32, [5], 1)
    for n in "kv":
        c.scale[n][0, 0, 0] = float(torch.tensor(0.0123))
    x = torch.randn(1, 1, 3, 64, generator=ref.rng(7)).half()
    c.lens = [8]
    gpu = upload(c)
    attn.kv8_append(gpu, x.cuda(), x.cuda())
    c.append(x, x)
    # x / scale is rounded to fp32 before the rounding to E4M3, which moves a
    # quotient across a tie at most: codes differ by one step, and seldom.
    for n in "kv":
        a = getattr(gpu, n).view(torch.uint8).cpu()[0, 0, :8].int()
        b = c.code[n][0, 0, :8].int()
        assert int((a - b).abs().max()) <= 1
        assert float((a != b).float().mean()) < 0.01
        assert torch.equal(getattr(gpu, n + "_scale").cpu().double(),
                           c.scale[n])


# --------------------------------------------------------------- attention

def run_fwd(c, q, causal=True, new=None, scale=None, with_w=True, gpu=None,
            **kw):
    """GPU result on buffers of sentinels, checked to stay where they must."""
    B, Hq, Sq, D = q.shape
    gpu = gpu or upload(c)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.full(q.shape, 7.5, dtype=q.dtype).cuda()
    lse = torch.full((B, Hq, Sq), 3.25).cuda()
    w0 = torch.rand(B, c.H, c.cap, generator=ref.rng(77))
    w = w0.cuda() if with_w else None
    ws = attn.kv8_workspace(gpu, Hq, Sq, with_w)
    guard = torch.full((ws.numel() + 4096,), 0xA5, dtype=torch.uint8).cuda()
    attn.kv8_fwd(gpu, q.cuda(), scale=scale, causal=causal,
                 new_lens=counts(new), weights=w, out=out, lse=lse,
                 workspace=guard[:ws.numel()], **kw)
    torch.cuda.synchronize()
    assert bool((guard[ws.numel():] == 0xA5).all()), "workspace overrun"
    return (out.cpu(), lse.cpu(), w.cpu() if with_w else None, w0)


def check_fwd(c, q, causal=True, new=None, scale=None, with_w=True, gpu=None,
              where="cpu"):
    B, Hq, Sq, D = q.shape
    scale_ = 1.0 / math.sqrt(D) if scale is None else scale
    out, lse, w, w0 = run_fwd(c, q, causal, new, scale, with_w, gpu)
    o_r, l_r, w_r, t_o, t_l, t_w = (
        t.cpu() for t in ref.attention(c.to(where), q.to(where), scale_,
                                       causal, new))
    for b in range(B):
        n = Sq if new is None else new[b]
        assert bool((out[b, :, n:] == 7.5).all())
        assert bool((lse[b, :, n:] == 3.25).all())
        e = (out[b, :, :n].double() - o_r[b, :, :n]).abs()
        assert bool((e <= t_o[b, :, :n]).all()), (
            "O", b, float((e - t_o[b, :, :n]).max()))
        got, want = lse[b, :, :n].double(), l_r[b, :, :n]
        empty = want == -math.inf
        assert torch.equal(got == -math.inf, empty)
        e = torch.where(empty, 0.0, got - torch.where(empty, 0.0, want)).abs()
        assert bool((e <= t_l[b, :, :n]).all()), ("LSE", b, float(e.max()))
        assert bool((out[b, :, :n][empty] == 0).all())
        if with_w:
            L = c.lens[b]
            assert torch.equal(w[b, :, L:], w0[b, :, L:])
            e = (w[b].double() - w0[b].double() - w_r[b]).abs()
            # Adding to the accumulator rounds once more.
            tol = t_w[b] + 2.0 ** -23 * (w0[b] + w_r[b])
            assert bool((e <= tol).all()), ("w", b, float((e - tol).max()))


FWDS = [
    # B, Hq, Hkv, cap, D, block, lens, Sq, new
    (1, 1, 1, 1, 64, 16, [1], 1, None),
    (1, 8, 1, 40, 128, 16, [17], 1, None),
    (2, 4, 4, 64, 64, 64, [64, 1], 1, None),
    (3, 8, 2, 300, 128, 64, [0, 299, 300], 1, None),
    (4, 14, 2, 1000, 64, 32, [1000, 15, 16, 129], 1, None),
    (5, 6, 2, 515, 128, 128, [515, 0, 4, 200, 77], 5, [5, 5, 0, 3, 1]),
    (2, 16, 1, 333, 64, 16, [333, 100], 1, None),
    (2, 3, 3, 400, 64, 32, [3, 400], 9, [9, 7]),
    (1, 7, 1, 700, 128, 64, [700], 3, None),
    (2, 8, 2, 600, 64, 64, [600, 131], 40, [40, 17]),
    (2, 4, 2, 257, 128, 32, [257, 64], 130, None),
    (1, 6, 6, 150, 64, 16, [150], 150, None),
    (40, 2, 1, 90, 64, 16, [(7 * i) % 91 for i in range(40)], 1, None),
    (1, 4, 1, 9000, 128, 128, [8999], 1, None),
    (1, 32, 4, 2500, 128, 64, [2500], 64, None),
    (3, 4, 1, 520, 64, 64, [520, 0, 30], 64, [50, 64, 64]),
]


@pytest.mark.parametrize("with_w", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", FWDS)
def test_fwd(case, dtype, causal, with_w):
    B, Hq, Hkv, cap, D, block, lens, Sq, new = case
    c = ref.filled(B, Hkv, cap, D, block, lens, 11)
    q = torch.randn(B, Hq, Sq, D, generator=ref.rng(12)).to(DT[dtype])
    check_fwd(c, q, causal, new, with_w=with_w)


SHORT = [
    # Caches around the sizes up to which a CTA takes a whole segment (by
    # capacity, segments and whether weights are accumulated).
    (4, 8, 2, 256, 128, 64, [0, 256, 1, 100], 3, [3, 0, 2, 3]),
    (4, 8, 2, 257, 128, 64, [0, 257, 1, 100], 3, [3, 0, 2, 3]),
    (3, 6, 2, 512, 64, 32, [0, 511, 77], 5, [5, 5, 0]),
    (3, 6, 2, 513, 64, 32, [0, 511, 77], 5, [5, 5, 0]),
    (3, 4, 4, 200, 64, 16, [2, 200, 5], 13, [13, 13, 9]),
    (3, 32, 16, 512, 128, 128, [512, 0, 300], 1, None),
    (3, 32, 16, 513, 128, 128, [512, 0, 300], 1, None),
    (40, 16, 8, 1024, 64, 64, [(89 * i) % 1025 for i in range(40)], 2, None),
    (40, 4, 2, 1100, 64, 32, [(97 * i) % 1101 for i in range(40)], 1, None),
    (50, 4, 1, 600, 128, 16, [(41 * i) % 601 for i in range(50)], 3,
     [i % 4 for i in range(50)]),
    (2, 16, 16, 1, 128, 16, [1, 0], 1, None),
    # Clusters of up to 8, with fewer tiles than CTAs, and none.
    (3, 8, 2, 2000, 128, 64, [2000, 3, 0], 1, None),
    (3, 8, 2, 2000, 128, 64, [1999, 17, 700], 3, [3, 1, 0]),
    (2, 16, 2, 1500, 64, 32, [1500, 40], 2, None),
    (2, 16, 2, 4000, 64, 128, [4000, 2049], 2, [2, 1]),
    (5, 32, 8, 4000, 128, 128, [4000, 0, 1, 2222, 333], 1, None),
]


@pytest.mark.parametrize("with_w", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", SHORT)
def test_fwd_short(case, dtype, causal, with_w):
    B, Hq, Hkv, cap, D, block, lens, Sq, new = case
    c = ref.filled(B, Hkv, cap, D, block, lens, 15)
    q = torch.randn(B, Hq, Sq, D, generator=ref.rng(16)).to(DT[dtype])
    check_fwd(c, q, causal, new, with_w=with_w)


LONG = [
    # Many key tiles and units for every CTA.
    (4, 32, 8, 2100, 128, 64, [2100, 2077, 1500, 2099], 250, None),
    (3, 24, 8, 3001, 64, 32, [3001, 2000, 2999], 333, [333, 1, 300]),
    (8, 16, 16, 1030, 128, 16, [1030 - 7 * i for i in range(8)], 129, None),
    (16, 16, 8, 1500, 128, 128, [1500 - 90 * i for i in range(16)], 1, None),
    (16, 32, 4, 2049, 64, 64, [2049 - 120 * i for i in range(16)], 2, None),
    (70, 8, 8, 300, 128, 32, [(37 * i) % 301 for i in range(70)], 2, None),
    (2, 16, 4, 20000, 128, 128, [20000, 13001], 4, None),
    (40, 8, 8, 1100, 128, 64, [(97 * i) % 1101 for i in range(40)], 2, None),
    # Many rows, units cut.
    (2, 32, 8, 4100, 128, 64, [4100, 3001], 250, None),
    (4, 16, 16, 1500, 128, 16, [1500, 0, 1499, 700], 129, [129, 3, 0, 129]),
    (33, 1, 1, 4000, 64, 128, [121 * i for i in range(33)], 20, None),
    # Many rows, whole units, several to a CTA.
    (20, 16, 16, 300, 128, 32, [300 - 15 * i for i in range(20)], 129, None),
    (40, 4, 4, 300, 64, 16, [(37 * i) % 301 for i in range(40)], 70,
     [(11 * i) % 71 for i in range(40)]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", LONG)
def test_fwd_long(case, dtype, causal):
    """Against the float64 definition computed on the GPU, and again: the
    same bits every time."""
    B, Hq, Hkv, cap, D, block, lens, Sq, new = case
    g = ref.rng(13)
    c = ref.Cache(B, Hkv, cap, D, block)
    c.lens = list(lens)
    nblk = -(-cap // block)
    for n in "kv":  # codes at random (no NaN), scales over four octaves
        code = torch.randint(0, 256, (B, Hkv, cap, D), generator=g,
                             dtype=torch.uint8)
        c.code[n] = torch.where((code & 127) > 100, code & 0x9F, code)
        c.scale[n] = torch.exp2(torch.randint(
            -5, -1, (B, Hkv, nblk), generator=g).double())
    q = torch.randn(B, Hq, Sq, D, generator=g).to(DT[dtype])
    scale = 0.5 / math.sqrt(D)
    check_fwd(c, q, causal, new, scale=scale, where="cuda")
    gpu = upload(c)
    first = run_fwd(c, q, causal, new, scale, gpu=gpu)
    for _ in range(8):
        again = run_fwd(c, q, causal, new, scale, gpu=gpu)
        for a, b in zip(first[:3], again[:3]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("Sq", [1, 33])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
def test_fwd_scales(scale, Sq):
    c = ref.filled(2, 2, 200, 64, 32, [200, 45], 21)
    q = torch.randn(2, 8, Sq, 64, generator=ref.rng(22)).bfloat16()
    check_fwd(c, q, scale=scale)


@pytest.mark.parametrize("Sq", [1, 40])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_fwd_block_scales_of_unlike_size(dtype, Sq):
    """Any positive scales, 2^-10 to 2^10 apart; rows of unlike size."""
    c = ref.filled(2, 2, 500, 128, 16, [500, 123], 31)
    g = ref.rng(32)
    for n in "kv":
        f = torch.exp2(20 * torch.rand(c.scale[n].shape, generator=g) - 10)
        s = (c.scale[n] * f * (0.02 if n == "k" else 1)).float().double()
        c.scale[n] = torch.where(c.scale[n].isfinite(), s, c.scale[n])
    q = torch.randn(2, 4, Sq, 128, generator=g)
    q = (q * torch.exp2(8 * torch.rand(2, 4, Sq, 1, generator=g) - 8)
         ).to(DT[dtype])
    check_fwd(c, q, scale=0.02)


@pytest.mark.parametrize("Sq", [1, 30])
def test_fwd_tiny_and_huge_queries(Sq):
    c = ref.filled(1, 1, 100, 64, 16, [100], 41)
    q = torch.randn(1, 2, Sq, 64, generator=ref.rng(42))
    check_fwd(c, (q * 1e-30).bfloat16())
    check_fwd(c, (q * 1e30).bfloat16(), scale=1e-30)
    check_fwd(c, (q * 1e-5).half(), scale=100.0)


@pytest.mark.parametrize("Sq", [1, 30])
def test_fwd_nan_stays_in_its_row(Sq):
    c = ref.filled(1, 1, 100, 64, 16, [100], 41)
    q = torch.randn(1, 3, Sq, 64, generator=ref.rng(43)).half()
    clean, lse, _, _ = run_fwd(c, q, with_w=False)
    q[0, 1, Sq - 1, 5] = math.nan
    out, lse2, _, _ = run_fwd(c, q, with_w=False)
    assert bool(out[0, 1, Sq - 1].isnan().all())
    assert bool(lse2[0, 1, Sq - 1].isnan())
    keep = torch.ones(3, Sq, dtype=torch.bool)
    keep[1, Sq - 1] = False
    assert torch.equal(out[0][keep], clean[0][keep])
    assert torch.equal(lse2[0][keep], lse[0][keep])


@pytest.mark.parametrize("Sq", [1, 48])
def test_fwd_is_deterministic_and_replays_in_a_graph(Sq):
    c = ref.filled(3, 2, 700, 128, 64, [700, 3, 350], 51)
    q = torch.randn(3, 8, Sq, 128, generator=ref.rng(52)).bfloat16()
    first = run_fwd(c, q)
    again = run_fwd(c, q)
    for a, b in zip(first[:3], again[:3]):
        assert torch.equal(a, b)
    gpu, qd = upload(c), q.cuda()
    out, lse = torch.zeros_like(qd), torch.zeros(3, 8, Sq).cuda()
    w = first[3].cuda()
    ws = attn.kv8_workspace(gpu, 8, Sq, True)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        attn.kv8_fwd(gpu, qd, weights=w, out=out, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first[0])
    assert torch.equal(lse.cpu(), first[1])
    assert torch.equal(w.cpu(), first[2])
    # Other lengths and queries, the same graph.
    c.lens = [100, 0, 699]
    q2 = torch.randn(3, 8, Sq, 128, generator=ref.rng(53)).bfloat16()
    want = run_fwd(c, q2)
    gpu.lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    qd.copy_(q2)
    w.copy_(first[3])
    graph.replay()
    torch.cuda.synchronize()
    # The last sequence now reaches the NaN codes behind its tokens: bits.
    assert torch.equal(out.cpu().view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(w.cpu().view(torch.int32), want[2].view(torch.int32))


@pytest.mark.parametrize("cap", [200, 700, 1500, 5000])
@pytest.mark.parametrize("Sq", [1, 4, 30])
def test_fwd_results_do_not_depend_on_weights(Sq, cap):
    c = ref.filled(3, 4, cap, 64, 64, [cap, 3, cap // 2], 151)
    q = torch.randn(3, 16, Sq, 64, generator=ref.rng(152)).half()
    a = run_fwd(c, q, with_w=True)
    b = run_fwd(c, q, with_w=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_fwd_two_streams_at_once():
    c = ref.filled(2, 2, 900, 64, 32, [900, 450], 61)
    q = [torch.randn(2, 4, 3, 64, generator=ref.rng(s)).half()
         for s in (62, 63)]
    want = [run_fwd(c, x)[:2] for x in q]
    gpu, qd = upload(c), [x.cuda() for x in q]
    ws = [attn.kv8_workspace(gpu, 4, 3) for _ in q]
    got = [(torch.zeros_like(x), torch.zeros(2, 4, 3).cuda()) for x in qd]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, (o, l), s in zip(qd, ws, got, streams):
            attn.kv8_fwd(gpu, x, out=o, lse=l, workspace=w, stream=s)
    torch.cuda.synchronize()
    for (o, l), (a, b) in zip(got, want):
        assert torch.equal(o.cpu(), a) and torch.equal(l.cpu(), b)


@pytest.mark.parametrize("Sq", [1, 40])
def test_fwd_buffers_of_the_least_alignment(Sq):
    """Q and O 16 bytes, LSE, weights and scales 4 bytes aligned."""
    c = ref.filled(2, 2, 600, 64, 32, [600, 77], 121)
    q = torch.randn(2, 8, Sq, 64, generator=ref.rng(122)).bfloat16()
    want = run_fwd(c, q)
    gpu = upload(c)

    def shifted(t, by):
        """A contiguous copy `by` elements behind an aligned address."""
        flat = torch.empty(t.numel() + by, dtype=t.dtype).cuda()[by:]
        return flat.view(t.shape).copy_(t)

    odd = attn.KV8Cache(
        shifted(gpu.k.view(torch.uint8), 16),
        shifted(gpu.v.view(torch.uint8), 48), shifted(gpu.k_scale, 1),
        shifted(gpu.v_scale, 3), shifted(gpu.lens, 1), 32)
    out = shifted(torch.full(q.shape, 7.5, dtype=q.dtype), 8)
    assert out.data_ptr() % 32 == 16
    lse = shifted(torch.full((2, 8, Sq), 3.25), 1)
    w = shifted(want[3], 1)
    attn.kv8_fwd(odd, shifted(q, 24), weights=w, out=out, lse=lse)
    assert torch.equal(out.cpu(), want[0])
    assert torch.equal(lse.cpu(), want[1])
    assert torch.equal(w.cpu(), want[2])
    x = torch.randn(2, 2, 5, 64, generator=ref.rng(123)).half()
    gpu.lens.copy_(torch.tensor([600, 82]))
    odd.lens.copy_(gpu.lens)
    attn.kv8_append(gpu, x.cuda(), x.cuda())
    attn.kv8_append(odd, shifted(x, 8), shifted(x, 24))
    for a, b in ((gpu.k, odd.k), (gpu.v, odd.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(gpu.k_scale, odd.k_scale)
    w1, w2 = w.clone(), shifted(w, 3)
    a = attn.kv8_evict(gpu, w1, 100, 10)
    b = attn.kv8_evict(odd, w2, 100, 10)
    assert torch.equal(a[2], b[2]) and torch.equal(w1, w2)
    for n in ("k", "v"):
        assert torch.equal(getattr(gpu, n)[:, :, :100].view(torch.uint8),
                           getattr(odd, n)[:, :, :100].view(torch.uint8))


def test_many_rows_weights_and_eviction_on_two_streams_and_in_graphs():
    """Two runs of append, attention with weights and eviction at once, eager
    and as graphs that replay side by side, to the bits of one alone."""
    def start(seed):
        c = ref.filled(2, 2, 700, 128, 64, [650, 300], seed)
        x = torch.randn(2, 2, 50, 128, generator=ref.rng(seed + 1)).bfloat16()
        q = torch.randn(2, 8, 50, 128, generator=ref.rng(seed + 2)).bfloat16()
        gpu = upload(c)
        return dict(
            cache=gpu, k=gpu.k.view(torch.uint8).clone(),
            v=gpu.v.view(torch.uint8).clone(), ks=gpu.k_scale.clone(),
            vs=gpu.v_scale.clone(), lens=gpu.lens + 50, x=x.cuda(),
            q=q.cuda(), w=torch.zeros(2, 2, 700).cuda(),
            out=torch.zeros(2, 8, 50, 128, dtype=torch.bfloat16).cuda(),
            lse=torch.zeros(2, 8, 50).cuda(),
            ws=attn.kv8_workspace(gpu, 8, 50, True),
            dst=attn.KV8Cache.empty(2, 2, 256, 128, 64),
            dw=torch.zeros(2, 2, 256).cuda(),
            idx=torch.zeros(2, 2, 200, dtype=torch.int32).cuda())

    def run(s):
        g = s["cache"]
        g.k.view(torch.uint8).copy_(s["k"])
        g.v.view(torch.uint8).copy_(s["v"])
        g.k_scale.copy_(s["ks"])
        g.v_scale.copy_(s["vs"])
        g.lens.copy_(s["lens"])
        s["w"].zero_()
        attn.kv8_append(g, s["x"], s["x"])
        attn.kv8_fwd(g, s["q"], weights=s["w"], out=s["out"], lse=s["lse"],
                     workspace=s["ws"])
        attn.kv8_evict(g, s["w"], 200, 30, out=s["dst"], out_weights=s["dw"],
                       indices=s["idx"])

    def result(s):
        n = int(s["dst"].lens.max())
        return [t.clone() for t in (
            s["out"], s["lse"], s["w"], s["dw"], s["idx"], s["dst"].lens,
            s["dst"].k.view(torch.uint8)[:, :, :n],
            s["dst"].v_scale[:, :, :-(-n // 64)])]

    states = [start(131), start(141)]
    want = []
    for s in states:
        run(s)
        torch.cuda.synchronize()
        want.append(result(s))

    def same():
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            for a, b in zip(result(s), w):
                assert torch.equal(a.cpu(), b.cpu())

    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(10):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                run(s)
    same()
    graphs = []
    for s in states:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(s)
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    same()


# ---------------------------------------------------------------- eviction

EVICTS = [
    # B, H, cap, D, block, lens, keep, recent
    (1, 1, 20, 64, 16, [20], 1, 0),
    (1, 1, 20, 64, 16, [20], 1, 1),
    (2, 2, 100, 128, 16, [100, 40], 50, 10),
    (3, 2, 300, 64, 64, [0, 300, 299], 299, 5),
    (2, 3, 515, 128, 128, [515, 514], 129, 129),
    (2, 1, 1000, 64, 32, [1000, 33], 700, 0),
    (1, 2, 5000, 128, 64, [4999], 1234, 200),
    (4, 1, 64, 64, 16, [64, 1, 63, 32], 64, 3),
    # Several CTAs select together: their parts uneven, all or none recent.
    (1, 2, 9001, 64, 128, [9001], 4000, 700),
    (2, 1, 20000, 64, 32, [19999, 12345], 777, 0),
    (1, 1, 70000, 64, 64, [70000], 69999, 65000),
    (2, 1, 40000, 64, 128, [40000, 90], 100, 100),
    (1, 1, 300000, 64, 128, [299999], 1000, 10),
    (1, 1, 290000, 64, 64, [290000], 5000, 0),
    (2, 2, 4097, 64, 16, [4097, 4096], 4095, 1),
]


def some_weights(B, H, cap, seed):
    """Weights with many equal values, zeros of both signs and NaN."""
    g = ref.rng(seed)
    w = (torch.rand(B, H, cap, generator=g) * 8).floor() / 4
    w = torch.where(w == 0.25, -0.0, w)
    fine = torch.rand(B, H, cap, generator=g)
    w = torch.where(fine > 0.6, fine, w)
    return torch.where(fine < 0.02, math.nan, w)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICTS)
def test_evict(case, in_place):
    B, H, cap, D, block, lens, keep, recent = case
    c = ref.filled(B, H, cap, D, block, lens, 71)
    g = ref.rng(72)
    for n in "kv":  # blocks of unlike size, so that codes get requantised
        f = torch.exp2((12 * torch.rand(c.scale[n].shape, generator=g)).floor())
        c.scale[n] *= f
    w = some_weights(B, H, cap, 73)
    room = cap if in_place else keep + 7
    want, ow, idx = c.evict(w, keep, recent, room)
    gpu, wd = upload(c), w.cuda()
    if in_place:
        # What lies behind the kept tokens' last block stays.
        for n in "kv":
            for b in range(B):
                m = want.lens[b]
                nb = -(-m // block)
                want.code[n][b, :, m:] = c.code[n][b, :, m:]
                want.scale[n][b, :, nb:] = c.scale[n][b, :, nb:]
        out, out_w, got = attn.kv8_evict(gpu, wd, keep, recent)
        assert out_w is wd and out.k is gpu.k
    else:
        dst = upload(ref.Cache(B, H, room, D, block))
        before = upload(c)
        out, out_w, got = attn.kv8_evict(gpu, wd, keep, recent, out=dst)
        for n in ("k", "v"):  # the source stays
            assert torch.equal(getattr(gpu, n), getattr(before, n))
        assert torch.equal(wd.cpu().nan_to_num(9), w.nan_to_num(9))
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), idx)
    assert torch.equal(out_w.cpu().nan_to_num(9), ow.nan_to_num(9))
    same_cache(out, want)
    assert gpu.lens.cpu().tolist() == lens


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_of_blocks_that_lose_their_large_tokens(in_place):
    """Kept codes shift up by as much as 2^17, or down to nothing."""
    B, H, cap, D, block, keep = 1, 1, 128, 64, 32, 40
    g = ref.rng(75)
    x = torch.randn(1, 1, cap, D, generator=g).double()
    size = torch.exp2((24 * torch.rand(cap, generator=g) - 24).floor())
    size[::8] = 2.0 ** 12
    x = (x * size[None, None, :, None]).float().bfloat16()
    c = ref.Cache(B, H, cap, D, block)
    c.lens = [cap]
    c.append(x, x)
    w = torch.rand(B, H, cap, generator=g)
    w[0, 0, ::8] = 0.0       # the large ones leave,
    w[0, 0, 64::8] = 1.0     # but for those of the last blocks
    want, ow, idx = c.evict(w, keep, 0, cap)
    gpu = upload(c)
    out = None if in_place else upload(ref.Cache(B, H, cap, D, block))
    out, out_w, got = attn.kv8_evict(gpu, w.cuda(), keep, 0, out=out)
    assert torch.equal(got.cpu(), idx)
    if in_place:
        for n in "kv":
            want.code[n][:, :, keep:] = c.code[n][:, :, keep:]
            want.scale[n][:, :, 2:] = c.scale[n][:, :, 2:]
    same_cache(out, want)


# ------------------------------------------------------------- all together

def test_a_serving_run():
    """Prompt, weights, eviction, then decoding steps over the smaller cache,
    each against the reference on the same state."""
    B, H, g, D, block, cap = 2, 2, 4, 64, 32, 400
    c = ref.Cache(B, H, cap, D, block)
    gpu = upload(c)
    wd, w = torch.zeros(B, H, cap).cuda(), None
    prompt = [300, 170]
    x = [torch.randn(B, H, 300, D, generator=ref.rng(s)).bfloat16()
         for s in (81, 82)]
    q = torch.randn(B, H * g, 300, D, generator=ref.rng(83)).bfloat16()
    c.lens = list(prompt)
    gpu.lens.copy_(torch.tensor(prompt, dtype=torch.int32))
    attn.kv8_append(gpu, x[0].cuda(), x[1].cuda(), new_lens=counts(prompt))
    c.append(x[0], x[1], new=prompt)
    same_cache(gpu, c)
    check_fwd(c, q, new=prompt, gpu=gpu)
    attn.kv8_fwd(gpu, q.cuda(), new_lens=counts(prompt), weights=wd)
    w = wd.cpu()
    small = attn.KV8Cache.empty(B, H, 128, D, block)
    for t in ("k", "v"):
        getattr(small, t).view(torch.uint8).fill_(0x7F)
        getattr(small, t + "_scale").fill_(math.inf)
    small, sw, idx = attn.kv8_evict(gpu, wd, 100, recent=20, out=small)
    c, w_small, idx_r = c.evict(w, 100, 20, 128)
    assert torch.equal(idx.cpu(), idx_r)
    same_cache(small, c)
    for step in range(12):
        x = [torch.randn(B, H, 1, D, generator=ref.rng(90 + 2 * step + s))
             .bfloat16() for s in (0, 1)]
        q = torch.randn(B, H * g, 1, D, generator=ref.rng(200 + step)
                        ).bfloat16()
        small.lens += 1
        c.lens = [n + 1 for n in c.lens]
        attn.kv8_append(small, x[0].cuda(), x[1].cuda())
        c.append(x[0], x[1])
        same_cache(small, c)
        check_fwd(c, q, gpu=small)
        attn.kv8_fwd(small, q.cuda(), weights=sw)
        if step == 6:  # in place, between two steps
            ws = sw.cpu()
            small, sw, idx = attn.kv8_evict(small, sw, 60, recent=8)
            behind = c
            c, _, idx_r = c.evict(ws, 60, 8, 128)
            assert torch.equal(idx.cpu(), idx_r)
            for n in "kv":  # the freed places keep what they held
                for b in range(B):
                    nb = -(-c.lens[b] // block)
                    c.code[n][b, :, c.lens[b]:] = \
                        behind.code[n][b, :, c.lens[b]:]
                    c.scale[n][b, :, nb:] = behind.scale[n][b, :, nb:]
            same_cache(small, c)


# ---------------------------------------------------- lengths out of range

def test_lengths_out_of_range_are_clamped_and_reported():
    c = ref.filled(2, 1, 64, 64, 16, [64, 10], 91)
    q = torch.randn(2, 2, 1, 64, generator=ref.rng(92)).half()
    gpu = upload(c)
    want = attn.kv8_fwd(gpu, q.cuda())[0]
    gpu.lens.copy_(torch.tensor([70, 10], dtype=torch.int32))
    got = attn.kv8_fwd(gpu, q.cuda())[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert attn.attn_device_status() == (attn.ATTN_ERR_INVALID_ARG, 2)
    gpu.lens.copy_(torch.tensor([-3, 10], dtype=torch.int32))
    got = attn.kv8_fwd(gpu, q.cuda())[0]
    torch.cuda.synchronize()
    assert bool((got[0] == 0).all()) and torch.equal(got[1], want[1])
    assert attn.attn_device_status() == (attn.ATTN_ERR_INVALID_ARG, 2)
    assert attn.attn_device_status() == (0, 0)


def test_new_counts_out_of_range_are_clamped_and_reported():
    c = ref.filled(2, 1, 64, 64, 16, [64, 10], 93)
    q = torch.randn(2, 2, 3, 64, generator=ref.rng(94)).half()
    want = run_fwd(c, q, new=[3, 0], with_w=False)
    got = run_fwd(c, q, new=[9, -1], with_w=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert attn.attn_device_status() == (attn.ATTN_ERR_INVALID_ARG, 2)
    # Appending more tokens than the length counts: the length decides.
    x = torch.randn(2, 1, 3, 64, generator=ref.rng(95)).half()
    a, b = upload(c), upload(c)
    a.lens.copy_(torch.tensor([64, 2], dtype=torch.int32))
    b.lens.copy_(torch.tensor([64, 2], dtype=torch.int32))
    attn.kv8_append(a, x.cuda(), x.cuda(), new_lens=counts([3, 3]))
    torch.cuda.synchronize()
    assert attn.attn_stream_status() == (attn.ATTN_ERR_INVALID_ARG, 2)
    attn.kv8_append(b, x.cuda(), x.cuda(), new_lens=counts([3, 2]))
    for n in ("k", "v"):
        assert torch.equal(getattr(a, n).view(torch.uint8),
                           getattr(b, n).view(torch.uint8))


# ------------------------------------------------- graphs, streams, refusals

def test_a_decoding_step_in_a_graph():
    """lens += 1, append, attention with weights: captured once, replayed."""
    B, H, g, D, block, cap = 2, 2, 4, 128, 32, 96
    c = ref.filled(B, H, cap, D, block, [40, 7], 101)
    gpu = upload(c)
    k, v = (torch.empty(B, H, 1, D, dtype=torch.float16).cuda()
            for _ in range(2))
    q = torch.empty(B, H * g, 1, D, dtype=torch.float16).cuda()
    w = torch.zeros(B, H, cap).cuda()
    out, lse = torch.empty_like(q), torch.empty(B, H * g, 1).cuda()
    ws = attn.kv8_workspace(gpu, H * g, 1, True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu.lens += 1
        attn.kv8_append(gpu, k, v)
        attn.kv8_fwd(gpu, q, weights=w, out=out, lse=lse, workspace=ws)
    total = torch.zeros(B, H, cap, dtype=torch.float64)
    tol = torch.zeros_like(total)
    for step in range(40):
        x = [torch.randn(B, H, 1, D, generator=ref.rng(300 + 2 * step + s))
             .half() for s in (0, 1)]
        y = torch.randn(B, H * g, 1, D, generator=ref.rng(500 + step)).half()
        k.copy_(x[0])
        v.copy_(x[1])
        q.copy_(y)
        graph.replay()
        c.lens = [n + 1 for n in c.lens]
        c.append(x[0], x[1])
        o_r, l_r, w_r, t_o, t_l, t_w = ref.attention(c, y, D ** -0.5, True)
        assert bool(((out.cpu().double() - o_r).abs() <= t_o).all())
        assert bool(((lse.cpu().double() - l_r).abs() <= t_l).all())
        total += w_r
        tol += t_w + 2.0 ** -23 * total
    same_cache(gpu, c)
    assert bool(((w.cpu().double() - total).abs() <= tol).all())


def test_calls_take_the_given_stream_and_the_tensors_device():
    c = ref.filled(1, 2, 64, 64, 16, [50], 103)
    q = torch.randn(1, 4, 2, 64, generator=ref.rng(104)).half()
    want = run_fwd(c, q)
    side = torch.cuda.Stream()
    got = run_fwd(c, q, stream=side)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)


def test_a_call_on_another_stream_allocates_there():
    """Memory that the current stream still reads (its tensor is gone) must
    not be handed to a call that runs on another stream meanwhile."""
    c = ref.filled(1, 2, 64, 64, 16, [50], 107)
    q = torch.randn(1, 64, 64, 64, generator=ref.rng(108)).half().cuda()
    gpu = upload(c)
    want = run_fwd(c, q.cpu(), with_w=False)
    side = torch.cuda.Stream()
    w = torch.rand(1, 2, 64, generator=ref.rng(109)).cuda()
    small = attn.KV8Cache.empty(1, 2, 32, 64, 16)
    # Freed blocks of every size that the calls ask for, read late.
    old = [torch.full((n,), 3, dtype=torch.uint8).cuda()
           for n in (q.nbytes, 4 * 64 * 64,
                     attn.kv8_workspace(gpu, 64, 64).nbytes,
                     4 * 2 * 32, 4 * 2 * 20)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    late = [t.clone() for t in old]
    del old
    out, lse = attn.kv8_fwd(gpu, q, stream=side)
    attn.kv8_evict(gpu, w, 20, out=small, stream=side)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in late)
    assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("Sq", [1, 24])
def test_work_of_other_streams_is_awaited(Sq, captured):
    """The queries come late from a second stream, joined by an event between
    append and attention; then the next step's keys, read from the output."""
    B, H, g, D, block = 1, 2, 4, 64, 16
    c = ref.filled(B, H, 300, D, block, [250], 110)
    x = torch.randn(B, H, Sq, D, generator=ref.rng(111)).half()
    y = torch.randn(B, H * g, Sq, D, generator=ref.rng(112)).half()
    c.lens = [250 + Sq]
    gpu = upload(c)
    c.append(x, x)
    want = run_fwd(c, y, with_w=False)
    xd, yd = x.cuda(), y.cuda()
    ws = attn.kv8_workspace(gpu, H * g, Sq)
    q = torch.zeros_like(yd)
    out, lse = torch.zeros_like(yd), torch.zeros(B, H * g, Sq).cuda()
    copy = torch.zeros_like(out)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(4_000_000)  # about 2 ms
            q.copy_(yd)
        attn.kv8_append(gpu, xd, xd)
        main.wait_stream(side)
        attn.kv8_fwd(gpu, q, out=out, lse=lse, workspace=ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            copy.copy_(out)
        main.wait_stream(side)
        attn.kv8_append(gpu, xd, xd)  # (the same tokens again)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    else:
        run = step
    for _ in range(3):
        q.zero_()
        out.zero_()
        copy.zero_()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[0])
        assert torch.equal(lse.cpu(), want[1])
        assert torch.equal(copy, out)
    same_cache(gpu, c)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes of K codes: append, attention of few
    and many rows, weights and eviction at its end."""
    B, H, cap, D, block = 2, 2, 20_000_000, 64, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    gpu = attn.KV8Cache.empty(B, H, cap, D, block)
    assert gpu.k.numel() > 1 << 32
    for n in ("k", "v"):
        getattr(gpu, n).view(torch.uint8).zero_()
        getattr(gpu, n + "_scale").fill_(2.0 ** -126)  # blocks of zeros
    gpu.lens.copy_(torch.tensor([3, cap], dtype=torch.int32))
    x = torch.zeros(B, H, 2, D)
    x[:, :, 1] = torch.eye(D)[:H][None] * 16
    val = torch.randn(B, H, 2, D, generator=ref.rng(105))
    attn.kv8_append(gpu, x.half().cuda(), val.half().cuda())
    c = ref.Cache(1, H, 4, D, 16)  # the last four tokens of sequence 1
    c.lens = [4]
    pad = torch.zeros(1, H, 2, D)
    c.append(torch.cat([pad, x[1:].half().float()], 2),
             torch.cat([pad, val[1:].half().float()], 2))
    for n in "kv":
        got = ref.decode(getattr(gpu, n)[1, :, -4:].view(torch.uint8).cpu())
        scale = getattr(gpu, n + "_scale")[1, :, -1].cpu().double()
        for h in range(H):
            assert torch.equal(got[h] * scale[h], c.values(n, 0, h))
    for Sq in (2, 40):
        q = torch.zeros(B, H, Sq, D)
        q[:, :, :] = torch.eye(D)[:H][None, :, None] * 16
        new = torch.tensor([0, Sq], dtype=torch.int32)
        w = torch.zeros(B, H, cap).cuda()
        out, lse = attn.kv8_fwd(gpu, q.half().cuda(), scale=1.0,
                                new_lens=new.cuda(), weights=w)
        # Score 256 against zeros: the last token takes all of the last row.
        v = torch.stack([c.values("v", 0, h)[-1] for h in range(H)])
        assert torch.equal(out[1, :, -1].cpu(), v.half())
        assert torch.allclose(lse[1, :, -1].cpu(), torch.tensor(256.0))
        # The rows before see zeros only: every weight 1 / tokens seen.
        seen = cap - 1 - torch.arange(Sq - 1).flip(0)
        assert torch.allclose(lse[1, :, :-1].cpu().double(),
                              torch.log(seen.double()).expand(H, -1),
                              atol=1e-4, rtol=0)
        assert torch.allclose(w[1, :, -1].cpu(), torch.tensor(1.0))
        total = w[1].double().sum(1).cpu()
        assert torch.allclose(total, torch.full((H,), float(Sq)).double(),
                              rtol=1e-4)
        assert float(w[0].abs().sum()) == 0.0
        del w
    w = torch.zeros(B, H, cap).cuda()
    w[1, :, 5] = 2.0
    w[1, :, cap - 9] = 1.0
    small, sw, idx = attn.kv8_evict(
        gpu, w, 4, recent=2, out=attn.KV8Cache.empty(B, H, 4, D, block))
    assert idx[1].cpu().tolist() == [[5, cap - 9, cap - 2, cap - 1]] * H
    assert small.lens.cpu().tolist() == [3, 4]
    got = ref.decode(small.v[1, :, 2:].view(torch.uint8).cpu())
    for h in range(H):
        assert torch.equal(got[h] * float(small.v_scale[1, h, 0]),
                           c.values("v", 0, h)[-2:])


def test_refusals_on_the_device():
    c = ref.filled(1, 2, 64, 64, 16, [50], 106)
    gpu = upload(c)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.float16).cuda()
    k = torch.zeros(1, 2, 2, 64, dtype=torch.float16).cuda()
    ws = attn.kv8_workspace(gpu, 4, 2)
    bad = [
        lambda: attn.kv8_append(gpu, k.float(), k),
        lambda: attn.kv8_append(gpu, k, k.bfloat16()),
        lambda: attn.kv8_append(gpu, k[:, :1], k),
        lambda: attn.kv8_append(gpu, k.transpose(1, 2), k),
        lambda: attn.kv8_append(gpu, k.cpu(), k),
        lambda: attn.kv8_append(gpu, k, k, new_lens=gpu.lens.long()),
        lambda: attn.kv8_append(gpu, k, k, new_lens=gpu.lens.cpu()),
        lambda: attn.kv8_fwd(gpu, q[0]),
        lambda: attn.kv8_fwd(gpu, q[:, :3]),
        lambda: attn.kv8_fwd(gpu, q.transpose(2, 3).contiguous()),
        lambda: attn.kv8_fwd(gpu, q.transpose(1, 2).contiguous()
                             .transpose(1, 2)),
        lambda: attn.kv8_fwd(gpu, q, out=q),
        lambda: attn.kv8_fwd(gpu, q, scale=float("nan")),
        lambda: attn.kv8_fwd(gpu, q, workspace=ws[:-256]),
        lambda: attn.kv8_fwd(gpu, q, workspace=ws.cpu()),
        lambda: attn.kv8_fwd(gpu, q, workspace=ws[128:]),
        lambda: attn.kv8_fwd(gpu, q, workspace=ws[:1].expand(ws.numel())),
        lambda: attn.kv8_fwd(gpu, q, weights=torch.zeros(1, 2, 63).cuda()),
        lambda: attn.kv8_fwd(gpu, q, weights=torch.zeros(1, 2, 64)),
        lambda: attn.kv8_fwd(gpu, q, lse=torch.zeros(1, 4, 2)),
        lambda: attn.kv8_evict(gpu, torch.zeros(1, 2, 64).cuda(), 0),
        lambda: attn.kv8_evict(gpu, torch.zeros(1, 2, 64).cuda(), 65),
        lambda: attn.kv8_evict(gpu, torch.zeros(1, 2, 64).cuda(), 9, 10),
        lambda: attn.kv8_evict(gpu, torch.zeros(1, 2, 64).cuda(), 9, out=gpu),
        lambda: attn.kv8_evict(gpu, torch.zeros(1, 2, 64), 9),
        lambda: attn.kv8_evict(
            gpu, torch.zeros(1, 2, 64).cuda(), 9,
            out=attn.KV8Cache.empty(1, 2, 64, 64, block=32)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(attn.AttnError):
            f()
            pytest.fail("call %d was taken" % i)
    torch.cuda.synchronize()
    same_cache(gpu, c)
