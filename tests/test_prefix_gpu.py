"""Attention behind a shared prefix on the GPU against float64.

Tolerances.  With queries and keys of N(0, 1), sum |q k| * scale is below 2^5
for D <= 128, and a score, a sum in fp32, is off by less than D 2^-24 times
that, 2^-12: a weight by 2^-12 of itself, and O by 2^-11 of sum p |v| at most.
Weights are rounded to the inputs' type once (half a step, eps / 2 of sum p
|v|), and so is O (eps / 2 of itself).  The LSE is off by the scores' 2^-12 and
by fp32's own rounding.
"""
import math

import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests import rope_reference as ref

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


def randn(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(DT[dtype])


def make(B, Hkv, D, plen, pcap, lens, cap, dtype, seed=1, fill=math.nan):
    """A cache whose memory behind the lengths holds `fill`."""
    pk, pv = (randn(1, Hkv, pcap, D, dtype=dtype, seed=seed + i)
              for i in range(2))
    k, v = (randn(B, Hkv, cap, D, dtype=dtype, seed=seed + 2 + i)
            for i in range(2))
    lens = torch.tensor(lens, dtype=torch.int32).cuda()
    late = torch.arange(cap, device="cuda")[None] >= lens[:, None]
    for x in (k, v):
        x.masked_fill_(late[:, None, :, None], fill)
    for x in (pk, pv):
        x[:, :, plen:] = fill
    plen = torch.tensor([plen], dtype=torch.int32).cuda()
    return attn.PrefixCache(pk, pv, plen, k, v, lens)


def exact(c, q, new, causal, scale):
    """(O, LSE, sum p |v|) in float64, NaN behind new[b]."""
    B, Hq, Sq, D = q.shape
    g, P = Hq // c.Hkv, int(c.prefix_len)
    o = torch.full((B, Hq, Sq, D), math.nan, dtype=torch.float64,
                   device="cuda")
    a = torch.full_like(o, math.nan)
    lse = torch.full((B, Hq, Sq), math.nan, dtype=torch.float64,
                     device="cuda")
    for b, (L, n) in enumerate(zip(c.lens.tolist(), new)):
        if n == 0:
            continue
        end = torch.full((n,), P + L, device="cuda")
        if causal:
            end = P + (L - n + 1 + torch.arange(n, device="cuda")).clamp(min=0)
        seen = torch.arange(P + L, device="cuda") < end[:, None]
        for h in range(c.Hkv):
            k = torch.cat([c.prefix_k[0, h, :P], c.k[b, h, :L]]).double()
            v = torch.cat([c.prefix_v[0, h, :P], c.v[b, h, :L]]).double()
            x = q[b, h * g:(h + 1) * g, :n].double()
            s = (x @ k.T * scale).masked_fill(~seen, -math.inf)
            z = torch.logsumexp(s, -1) if P + L else \
                torch.full((g, n), -math.inf, device="cuda").double()
            p = torch.exp(s - z.masked_fill(z == -math.inf, 0)[..., None])
            lse[b, h * g:(h + 1) * g, :n] = z
            o[b, h * g:(h + 1) * g, :n] = p @ v
            a[b, h * g:(h + 1) * g, :n] = p @ v.abs()
    return o, lse, a


def compare(got_o, got_lse, want, dtype):
    o, lse, a = want
    rows = ~lse.isnan()
    half = torch.finfo(DT[dtype]).eps / 2
    err = (got_o.double() - o).abs()[rows]
    tol = (half * o.abs() + (half + 2.0 ** -11) * a + 2.0 ** -25)[rows]
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol)[bad].max()))
    if got_lse is None:
        return
    x, y = got_lse.double()[rows], lse[rows]
    none = y == -math.inf
    assert torch.equal(x == -math.inf, none)
    off = (x - y)[~none].abs()
    assert (off <= 2.0 ** -12 + 2.0 ** -20 * y[~none].abs()).all(), \
        float(off.max())


def check(c, Hq, Sq, dtype, new=None, causal=True, scale=None, seed=9):
    q = randn(c.B, Hq, Sq, c.D, dtype=dtype, seed=seed)
    counts = None if new is None else \
        torch.tensor(new, dtype=torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((c.B, Hq, Sq), 7.0, device="cuda")
    s = c.D ** -0.5 if scale is None else scale
    want = exact(c, q, [Sq] * c.B if new is None else new, causal, s)
    for _ in range(2):  # the same bits again
        got = attn.prefix_fwd(c, q, scale=scale, causal=causal,
                              new_lens=counts, out=out, lse=lse)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == (0, 0)
        first = out.clone() if _ == 0 else first
        assert torch.equal(out, first)
    assert got[0] is out and got[1] is lse
    compare(out, lse, want, dtype)
    if new is not None:
        late = torch.arange(Sq, device="cuda")[None] >= counts[:, None]
        late = late[:, None].expand(c.B, Hq, Sq)
        assert (out[late] == 7).all() and (lse[late] == 7).all()
    return q, out, lse


# One row to many: the rows of a K/V head (Hq / Hkv * Sq) decide the kernels.
CASES = [
    # B, Hq, Hkv, D, Sq, plen, prefix room, lens, capacity, new, causal
    (1, 1, 1, 64, 1, 1, 1, [1], 1, None, True),
    (2, 4, 1, 128, 1, 130, 131, [0, 5], 9, [0, 1], True),
    (3, 8, 2, 128, 1, 128, 128, [1, 128, 129], 200, None, True),
    (3, 8, 8, 64, 1, 127, 300, [300, 17, 64], 300, None, True),
    (70, 8, 2, 128, 1, 1000, 1000, [7 * i % 90 for i in range(70)], 90,
     [int(7 * i % 90 > 0) for i in range(70)], True),
    (300, 2, 2, 64, 1, 257, 260, [1 + i % 40 for i in range(300)], 64, None,
     True),
    (5, 12, 3, 64, 3, 77, 80, [3, 50, 700, 0, 2], 701, [3, 1, 2, 0, 2], True),
    (4, 16, 1, 128, 1, 513, 600, [33, 2, 0, 90], 100, [1, 1, 0, 1], True),
    (2, 6, 2, 64, 5, 333, 333, [5, 40], 40, None, False),
    (3, 8, 1, 128, 2, 0, 5, [2, 700, 30], 700, [2, 2, 1], True),
    # More rows than 16: packed with those of the other sequences.
    (3, 9, 1, 128, 2, 300, 300, [2, 150, 257], 260, None, True),
    (5, 8, 2, 64, 9, 129, 200, [9, 300, 0, 4, 128], 300, [9, 7, 0, 4, 9],
     True),
    (2, 4, 1, 128, 40, 64, 64, [40, 999], 1000, None, True),
    (7, 14, 2, 64, 13, 700, 700, [13, 14, 15, 16, 17, 18, 140], 141,
     [13, 0, 5, 13, 1, 2, 13], True),
    (4, 3, 3, 128, 140, 0, 1, [140, 300, 141, 0], 300, [140, 140, 3, 0],
     True),
    (3, 4, 2, 64, 30, 500, 512, [0, 77, 200], 200, None, False),
    # Rows that fill units: the prefix and the own keys in one list.
    (1, 4, 2, 128, 20, 100, 100, [60], 70, None, True),
    (2, 4, 1, 128, 64, 300, 301, [64, 500], 500, None, True),
    (3, 8, 2, 64, 60, 129, 129, [0, 61, 400], 400, [0, 60, 33], True),
    (2, 2, 2, 128, 513, 640, 700, [513, 900], 900, [513, 300], True),
    (2, 8, 4, 64, 500, 1, 64, [500, 777], 777, None, True),
    (2, 2, 1, 128, 250, 0, 1, [0, 300], 300, [0, 250], True),
    (2, 2, 1, 64, 125, 77, 77, [0, 300], 300, None, False),
    # Groups that do not divide a tile's rows, and the largest.
    (2, 5, 1, 64, 100, 140, 140, [100, 333], 333, None, True),
    (3, 21, 3, 128, 15, 300, 300, [15, 40, 129], 130, [15, 1, 14], True),
    (2, 127, 1, 64, 3, 200, 200, [3, 20], 20, None, True),
    (3, 128, 1, 128, 1, 200, 200, [1, 20, 0], 20, [1, 1, 0], True),
    (2, 256, 2, 64, 2, 130, 130, [2, 200], 200, None, True),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, dtype):
    B, Hq, Hkv, D, Sq, plen, pcap, lens, cap, new, causal = case
    check(make(B, Hkv, D, plen, pcap, lens, cap, dtype), Hq, Sq, dtype, new,
          causal)


# Nine to sixteen rows of more sequences and heads.
WIDE = [
    (20, 12, 3, 64, 3, 77, 80, [3, 50, 700, 0, 2] * 4, 701,
     [3, 1, 2, 0, 2] * 4, True),
    (45, 16, 1, 128, 1, 513, 600, [31 * i % 90 for i in range(45)], 100,
     [int(31 * i % 90 > 0) for i in range(45)], True),
    (21, 6, 2, 64, 5, 333, 333, [5 + 7 * i for i in range(21)], 150, None,
     False),
    (40, 8, 1, 128, 2, 0, 5, [2 + 113 * i % 700 for i in range(40)], 702,
     [1 + i % 2 for i in range(40)], True),
    (10, 80, 5, 128, 1, 128, 128, [128, 1, 129, 17] * 2 + [300, 16], 300, None,
     True),
    (3, 144, 16, 64, 1, 1000, 1001, [5, 900, 77], 900, None, True),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", WIDE)
def test_nine_to_sixteen_rows(case, dtype):
    B, Hq, Hkv, D, Sq, plen, pcap, lens, cap, new, causal = case
    check(make(B, Hkv, D, plen, pcap, lens, cap, dtype), Hq, Sq, dtype, new,
          causal)


@pytest.mark.parametrize("Sq,group", [(1, 4), (5, 7), (40, 2), (70, 3),
                                      (300, 1)])
def test_matches_the_loops_of_the_definition(Sq, group):
    """The reference above against one that takes every row by itself."""
    c = make(2, 2, 64, 20, 21, [Sq + 3, Sq], Sq + 3, "f16")
    new = [Sq, max(0, Sq - 2)]
    q = randn(2, 2 * group, Sq, 64, dtype="f16", seed=3)
    o, lse, _ = exact(c, q, new, True, 0.125)
    cpu = [x.cpu() for x in (q, c.prefix_k[0], c.prefix_v[0], c.k, c.v)]
    o2, lse2 = ref.prefix(cpu[0], *cpu[1:], 20, c.lens.tolist(), new, True,
                          0.125)
    rows = ~lse2.isnan()
    assert (o.cpu() - o2)[rows].abs().max() <= 1e-12
    assert (lse.cpu() - lse2)[rows].abs().max() <= 1e-12


@pytest.mark.parametrize("Sq", [1, 20, 200])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_scales(scale, Sq):
    c = make(3, 2, 64, 200, 200, [200, 300, 256], 300, "bf16")
    check(c, 4, Sq, "bf16", scale=scale)


@pytest.mark.parametrize("Sq", [1, 20, 200])
def test_rows_that_see_nothing(Sq):
    c = make(2, 1, 128, 0, 4, [0, 3], 300, "f16")
    q = randn(2, 2, Sq, 128, dtype="f16", seed=3)
    o, lse = attn.prefix_fwd(c, q, causal=False)
    assert not o[0].any() and (lse[0] == -math.inf).all()
    assert o[1].isfinite().all() and lse[1].isfinite().all()
    if Sq > 3:  # causal: only the last three rows of the second see a token
        new = torch.tensor([0, Sq], dtype=torch.int32).cuda()
        o, lse = attn.prefix_fwd(c, q, new_lens=new)
        assert not o[1, :, :-3].any()
        assert (lse[1, :, :-3] == -math.inf).all()
        assert lse[1, :, -3:].isfinite().all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Sq", [1, 3, 20, 200])
def test_scores_far_apart(Sq, dtype):
    """Large queries: weights of nearly one key, maxima that grow late."""
    c = make(2, 2, 64, 300, 300, [250, 400], 400, dtype)
    q = randn(2, 4, Sq, 64, dtype=dtype, seed=5) * 30
    o, lse = attn.prefix_fwd(c, q)
    want, z, a = exact(c, q, [Sq] * 2, True, 0.125)
    # Scores of up to 2^10 are off by 2^-12 * 30: weights by 2^-7.
    half = torch.finfo(DT[dtype]).eps / 2
    assert ((o.double() - want).abs() <= half * want.abs() +
            (half + 2.0 ** -6) * a + 2.0 ** -25).all()
    assert (lse.double() - z).abs().max() <= 2.0 ** -7


@pytest.mark.parametrize("Sq", [1, 20, 200])
def test_large_values(Sq):
    """V near bf16's largest number: sums of P V stay within fp32."""
    c = make(2, 1, 64, 5000, 5000, [300, 300], 300, "bf16")
    big = 2.0 ** 120
    c.prefix_v.mul_(big)
    c.v.mul_(big)
    q = randn(2, 2, Sq, 64, dtype="bf16", seed=5)
    o, lse = attn.prefix_fwd(c, q)
    want, z, a = exact(c, q, [Sq] * 2, True, 0.125)
    half = 2.0 ** -8
    assert ((o.double() - want).abs() <= half * want.abs() +
            (half + 2.0 ** -11) * a).all()


@pytest.mark.parametrize("Sq", [1, 20, 200])
def test_small_values(Sq):
    """V near 2^-100.  P is held times 2^-24, so sums of P V have steps of
    2^-149 at the least: each of the 700 is off by 2^-150 at most, which is
    2^-126 of O, together below 2^-116."""
    c = make(2, 1, 64, 400, 400, [300, 300], 300, "bf16")
    c.prefix_v.mul_(2.0 ** -100)
    c.v.mul_(2.0 ** -100)
    q = randn(2, 2, Sq, 64, dtype="bf16", seed=5)
    o, lse = attn.prefix_fwd(c, q)
    want, z, a = exact(c, q, [Sq] * 2, True, 0.125)
    half = 2.0 ** -8
    assert ((o.double() - want).abs() <= half * want.abs() +
            (half + 2.0 ** -11) * a + 2.0 ** -116).all()


@pytest.mark.parametrize("Sq", [1, 2, 20, 200])
def test_nan_stays_in_its_row(Sq):
    c = make(3, 2, 64, 140, 140, [200, 201, 256], 300, "f16")
    q = randn(3, 4, Sq, 64, dtype="f16", seed=5)
    clean, zc = attn.prefix_fwd(c, q)
    q[1, 2, Sq // 2, 3] = math.nan
    o, z = attn.prefix_fwd(c, q)
    hit = torch.zeros(3, 4, Sq, dtype=torch.bool, device="cuda")
    hit[1, 2, Sq // 2] = True
    assert o[hit].isnan().all() and z[hit].isnan().all()
    # (A NaN row may make its neighbours rescale at another time.)
    assert (o[~hit] - clean[~hit]).abs().max() <= 2.0 ** -9
    assert (z[~hit] - zc[~hit]).abs().max() <= 2.0 ** -12


@pytest.mark.parametrize("Sq", [1, 20, 200])
def test_nan_of_one_sequence_stays_there(Sq):
    c = make(3, 2, 64, 140, 140, [200, 201, 256], 300, "f16")
    q = randn(3, 4, Sq, 64, dtype="f16", seed=5)
    clean, _ = attn.prefix_fwd(c, q)
    c.v[1, :, 0] = math.nan
    c.k[1, :, 0] = math.inf
    o, _ = attn.prefix_fwd(c, q)
    assert torch.equal(o[0], clean[0]) and torch.equal(o[2], clean[2])
    assert o[1].isnan().any()


def test_long_prefix_and_long_own_keys():
    c = make(2, 2, 128, 100001, 100100, [70001, 3], 70001, "bf16")
    check(c, 8, 1, "bf16")
    check(c, 4, 12, "bf16", new=[12, 3])


def test_places_beyond_32_bits():
    """Own keys that begin 2^31 elements and more into their tensors."""
    cap = (1 << 22) + 5
    k, v = (torch.empty(2, 3, cap, 128, dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    lens = torch.tensor([10, 150], dtype=torch.int32).cuda()
    small = make(2, 3, 128, 40, 40, [10, 150], 150, "bf16")
    for x, y in ((k, small.k), (v, small.v)):
        x[:, :, :150] = y
    c = attn.PrefixCache(small.prefix_k, small.prefix_v, small.prefix_len, k,
                         v, lens)
    for Sq in (1, 5, 100):
        q = randn(2, 6, Sq, 128, dtype="bf16", seed=3)
        new = torch.tensor([min(Sq, 10), Sq], dtype=torch.int32).cuda()
        a = attn.prefix_fwd(c, q, new_lens=new)
        b = attn.prefix_fwd(small, q, new_lens=new)
        for i, n in enumerate(new.tolist()):
            for x, y in zip(a, b):
                assert torch.equal(x[i, :, :n], y[i, :, :n])


def test_lengths_out_of_range_are_clamped_and_reported():
    for Sq in (1, 20, 200):
        c = make(2, 1, 64, 30, 30, [300, 0], 300, "f16")
        q = randn(2, 2, Sq, 64, dtype="f16", seed=3)
        want = attn.prefix_fwd(c, q)
        c.lens.copy_(torch.tensor([301, -1]))
        c.prefix_len.fill_(31)
        got = attn.prefix_fwd(c, q)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == (attn.ATTN_ERR_INVALID_ARG, 2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_calls():
    c = make(2, 1, 64, 3, 3, [1, 1], 4, "f16")
    o, lse = attn.prefix_fwd(c, torch.zeros(2, 1, 0, 64, device="cuda",
                                            dtype=torch.float16))
    assert o.shape == (2, 1, 0, 64) and lse.shape == (2, 1, 0)


def test_without_lse():
    for Sq in (1, 20, 200):
        c = make(2, 1, 64, 300, 300, [200, 210], 300, "f16")
        q = randn(2, 2, Sq, 64, dtype="f16", seed=3)
        o, lse = attn.prefix_fwd(c, q)
        keep = torch.full_like(lse, 3.0)
        o2, none = attn.prefix_fwd(c, q, need_lse=False, lse=keep)
        assert none is None and torch.equal(o, o2) and (keep == 3).all()


def test_an_odd_output_address():
    """O 16-byte but not 32-byte aligned."""
    c = make(2, 1, 64, 300, 300, [256, 256], 300, "f16")
    q = randn(2, 1, 256, 64, dtype="f16", seed=3)
    want, _ = attn.prefix_fwd(c, q)
    room = torch.zeros(q.numel() + 8, dtype=torch.float16, device="cuda")
    out = room[8:].view(q.shape)
    attn.prefix_fwd(c, q, out=out)
    assert torch.equal(out, want) and not room[:8].any()


# ------------------------------------------------------ streams and graphs

def same_bits(a, b):
    """(The second lengths reach into memory that holds NaN.)"""
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("Sq", [1, 20, 200])
def test_streams_and_graphs(Sq):
    c = make(4, 2, 128, 700, 700, [200, 210, 300, 290], 300, "bf16")
    q = randn(4, 8, Sq, 128, dtype="bf16", seed=3)
    want = attn.prefix_fwd(c, q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = attn.prefix_fwd(c, q, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        ws = attn.prefix_workspace(c, 8, Sq)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attn.prefix_fwd(c, q, workspace=ws))
        graphs.append((g, ws))
    # Lengths are read when a graph runs.
    for lens in ([200, 210, 300, 290], [250, 201, 220, 299]):
        c.lens.copy_(torch.tensor(lens))
        c.prefix_len.fill_(700 - lens[0])
        want = attn.prefix_fwd(c, q)
        for o in outs:
            for x in o:
                x.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            for (g, ws), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(same_bits(a, b) for a, b in zip(want, o))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,D,Sq,plen", [
    (4, 8, 2, 128, 20, 450), (3, 4, 2, 64, 40, 333), (4, 8, 2, 128, 1, 450),
    (5, 6, 2, 128, 3, 200), (4, 8, 2, 128, 200, 450)])
def test_the_same_bits_side_by_side(B, Hq, Hkv, D, Sq, plen, dtype):
    """Calls on three streams at once, whatever shared memory held before."""
    c = make(B, Hkv, D, plen, plen, [250 - 7 * i for i in range(B)], 300,
             dtype)
    q = randn(B, Hq, Sq, D, dtype=dtype, seed=3)
    want = [x.clone() for x in attn.prefix_fwd(c, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [attn.prefix_workspace(c, Hq, Sq) for _ in streams]
    outs = [[torch.zeros_like(x) for x in want] for _ in streams]
    for _ in range(10):
        for _ in range(4):
            for s, w, o in zip(streams, spaces, outs):
                attn.prefix_fwd(c, q, out=o[0], lse=o[1], workspace=w,
                                stream=s)
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o))
            for x in o:
                x.zero_()
        # Another shape's numbers in shared memory.
        noise = make(B, Hkv, D, 100, 100, [90] * B, 90, dtype, seed=77)
        attn.prefix_fwd(noise, q * 50, causal=False)


def test_many_sequences():
    """More sequences than a warp's lanes, several times over."""
    B = 1500
    lens = [(37 * i) % 23 for i in range(B)]
    new = [min(1, n) for n in lens]
    c = make(B, 1, 64, 300, 300, lens, 23, "bf16")
    check(c, 2, 1, "bf16", new)
    check(make(B, 1, 64, 300, 300, [n + 9 for n in lens], 40, "f16"), 2, 9,
          "f16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,Hkv,group,Sq,D", [
    (60, 9, 4, 5, 128), (50, 10, 3, 40, 64), (1, 600, 2, 10, 128),
    (1, 500, 2, 60, 64), (3, 300, 1, 18, 128)])
def test_several_units_a_block(B, Hkv, group, Sq, D, dtype):
    """More (sequence, head) units of one Q tile than thread blocks, of one
    key tile to four, of lengths that end anywhere in a tile; causal and not."""
    lens = [Sq + 83 * i % 431 for i in range(B)]
    c = make(B, Hkv, D, 200, 201, lens, 480, dtype)
    check(c, Hkv * group, Sq, dtype)
    new = [(Sq - 5 * i) % (Sq + 1) for i in range(B)]
    check(c, Hkv * group, Sq, dtype, new, causal=False)


def test_calls_in_a_row_share_a_workspace():
    """Different shapes one behind the other on one stream and workspace."""
    c = make(4, 2, 64, 500, 500, [200, 210, 300, 290], 300, "f16")
    sizes = [(8, 1), (4, 20), (2, 300), (8, 2), (4, 200), (2, 1)]
    ws = torch.empty(max(attn.prefix_workspace(c, H, S).numel()
                         for H, S in sizes), dtype=torch.uint8, device="cuda")
    qs = [randn(4, H, S, 64, dtype="f16", seed=S) for H, S in sizes]
    want = [attn.prefix_fwd(c, q) for q in qs]
    torch.cuda.synchronize()
    got = [attn.prefix_fwd(c, q, workspace=ws) for _ in range(5) for q in qs]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(want[i % 6], g))


# ------------------------------------------------------ as a decoder uses them

def test_decoding_behind_a_prefix():
    """A prefix written by qk_rope, then steps of a batch: qk_rope into the
    cache, prefix_fwd over it.  Against attn.fwd over the whole of each
    sequence (whose own rounding is the other side's too: 2^-8 of sum p |v|
    each), and the float64 definition on the same cache."""
    B, Hq, Hkv, D, P, cap = 3, 8, 2, 128, 333, 16
    rope = attn.Rope.make(D)
    w = [torch.rand(D, device="cuda") + 0.5 for _ in range(2)]
    prompt = randn(1, P, Hq + 2 * Hkv, D, dtype="bf16", seed=1)
    q, k, v = prompt.split((Hq, Hkv, Hkv), 2)
    _, pk, pv = attn.qk_rope(rope, q, k, v, *w)
    cache = attn.PrefixCache.empty(pk, pv, B, cap)
    step = torch.zeros(B, dtype=torch.int32, device="cuda")
    tokens = []
    for t, (S, new) in enumerate([(4, [4, 2, 3]), (1, [1, 1, 1]),
                                  (1, [1, 0, 1])]):
        new = torch.tensor(new, dtype=torch.int32).cuda()
        x = randn(B, S, Hq + 2 * Hkv, D, dtype="bf16", seed=10 + t)
        tokens.append((x, new.tolist()))
        cache.lens += new
        q, k, v = x.split((Hq, Hkv, Hkv), 2)
        qr, _, _ = attn.qk_rope(rope, q, k, v, *w, lens=cache.lens,
                                new_lens=new, offset=cache.prefix_len,
                                k_out=cache.k, v_out=cache.v)
        o, lse = attn.prefix_fwd(cache, qr, new_lens=new)
        compare(o, lse, exact(cache, qr, new.tolist(), True, D ** -0.5),
                "bf16")
    for b in range(B):
        whole = torch.cat([prompt] + [x[b:b + 1, :n[b]] for x, n in tokens],
                          1)
        q, k, v = whole.split((Hq, Hkv, Hkv), 2)
        qr, kr, vr = attn.qk_rope(rope, q, k, v, *w)
        L = int(cache.lens[b])
        assert torch.equal(cache.k[b, :, :L], kr[0, :, P:])
        assert torch.equal(cache.v[b, :, :L], vr[0, :, P:])
        want, z = attn.fwd(qr[:, :, -1:].contiguous(), kr, vr, causal=True,
                           input_pos=P + L - 1)
        n = tokens[-1][1][b]
        if n:
            assert (o[b, :, n - 1] - want[0, :, 0]).abs().max() <= 2.0 ** -6
            assert (lse[b, :, n - 1] - z[0, :, 0]).abs().max() <= 2.0 ** -11
