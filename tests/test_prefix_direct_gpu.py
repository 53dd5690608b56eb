"""Units of two Q tiles over the prefix and a sequence's own keys whose key tiles
all fall to one thread block: their rows leave for O directly, several such
units a block.  Against float64; the cut of the list is made again here, so that
the shapes are known to have such units."""
import pytest
import torch

import attention_attn_fwd_gb300 as attn
from tests.test_prefix_gpu import check, make, randn

pytestmark = pytest.mark.gpu

TM, TN, OVER = 128, 128, 4  # rows of a Q tile, keys of a tile, empty places


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def up(x, y):
    return -(-x // y)


def units(B, Hkv, g, Sq, plen, lens, new, causal):
    """(key tiles of Q tile 0, of Q tile 1, of the unit) in the list's order."""
    tile_rows = TM // g * g
    rows, np = g * Sq, up(plen, TN)
    found = []
    for b in range(B):
        for u in range(up(up(rows, tile_rows), 2)):
            n = []
            for t in range(2):
                r0 = (2 * u + t) * tile_rows
                last = min(r0 + tile_rows, new[b] * g) - 1
                if last < r0:
                    n.append(0)
                    continue
                end = lens[b]
                if causal:
                    end = min(end, max(0, lens[b] - new[b] + last // g + 1))
                n.append(np + up(end, TN))
            found += [(n[0], n[1], max(n))] * Hkv
    return found


def whole_units(found):
    """Of each thread block, the units that are its own altogether."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    total = sum(s + OVER for *_, s in found if s)
    n = min(sms, total)
    cut = [i * (total // n) + min(i, total % n) for i in range(n + 1)]
    blocks = [[] for _ in range(n)]
    at, c = 0, 0
    for unit in found:
        if not unit[2]:
            continue
        first, at = at + OVER, at + OVER + unit[2]
        while cut[c + 1] <= first:
            c += 1
        if at <= cut[c + 1]:
            blocks[c].append(unit)
    return blocks


# B, Hkv, group, Sq, prefix, own, new tokens, causal
CASES = [
    (8, 64, 1, 256, 200, 400, [256, 256, 131, 100, 0, 255, 256, 1], True),
    (8, 64, 1, 256, 200, 400, None, True),
    (5, 60, 3, 100, 130, 300, [100, 99, 43, 42, 7], True),
    (6, 70, 2, 128, 0, 500, [128, 70, 65, 64, 63, 128], True),
    (4, 80, 2, 200, 128, 333, [200, 129, 128, 20], False),
    (40, 8, 4, 64, 300, 130, None, True),
]


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (128, "f16"),
                                     (64, "bf16")])
@pytest.mark.parametrize("case", CASES)
def test_whole_units(case, D, dtype):
    B, Hkv, g, Sq, plen, own, new, causal = case
    n = [Sq] * B if new is None else new
    lens = [max(n[b], own - 37 * b % 200) for b in range(B)]
    assert g * Sq > TM  # these rows' units have the prefix in their list
    blocks = whole_units(units(B, Hkv, g, Sq, plen, lens, n, causal))
    assert sum(len(x) for x in blocks) > 152
    assert sum(len(x) > 1 for x in blocks) > 20
    if causal:  # the tiles' key counts differ, or one has no rows
        assert any(a != b for x in blocks for a, b, _ in x)
    c = make(B, Hkv, D, plen, max(plen, 1), lens, own, dtype)
    q, out, lse = check(c, g * Hkv, Sq, dtype, new, causal)
    # O 16-byte but not 32-byte aligned: the same bits.
    counts = None if new is None else \
        torch.tensor(new, dtype=torch.int32).cuda()
    room = torch.full((q.numel() + 8,), 7.0, dtype=q.dtype, device="cuda")
    odd = room[8:].view(q.shape)
    assert odd.data_ptr() % 32 == 16
    attn.prefix_fwd(c, q, causal=causal, new_lens=counts, out=odd)
    assert torch.equal(odd, out) and (room[:8] == 7).all()


def test_rows_that_see_nothing_beside_whole_units():
    """Rows ahead of a sequence's tokens, and sequences without any."""
    B, Hkv, Sq = 6, 64, 256
    lens = [100, 0, 256, 3, 300, 130]
    blocks = whole_units(units(B, Hkv, 1, Sq, 0, lens, [Sq] * B, True))
    assert sum(len(x) for x in blocks) > 100
    c = make(B, Hkv, 64, 0, 1, lens, 300, "f16")
    q = randn(B, Hkv, Sq, 64, dtype="f16", seed=3)
    out = torch.full_like(q, 7.0)
    _, lse = attn.prefix_fwd(c, q, out=out)
    for b, n in enumerate(lens):
        blind = max(0, Sq - n)
        assert not out[b, :, :blind].any()
        assert (lse[b, :, :blind] == -float("inf")).all()
        assert lse[b, :, blind:].isfinite().all()
        # Row i sees i - blind + 1 tokens; the first of them is one token's V.
        if blind < Sq and n <= Sq:
            assert torch.equal(out[b, :, blind], c.v[b, :, 0])
