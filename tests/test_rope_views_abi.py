"""Which views of gradients attn_qk_rope_bwd takes as apart, without a GPU: a
view that is taken passes every check up to the device's."""
import itertools
import random

import pytest

import attention_attn_fwd_gb300 as attn
from attention_attn_fwd_gb300 import build as cuda_build
from tests.test_rope_abi import INVALID, MB, bwd

D = 64
P = 512 * MB  # elements' places are counted from here


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return attn.load_library()


def taken(lib, views, B, S, Hq, Hkv):
    """Whether these dq, dk and dv (offset, strides b, s, h in elements) get
    past the checks of their places: what comes behind them is the device's
    check of the addresses, which without a device has a code of its own."""
    kw = {n: dict(p=P + 2 * o, stride_b=b, stride_s=s, stride_h=h)
          for n, (o, b, s, h) in zip(("dxq", "dxk", "dxv"), views)}
    return bwd(lib, B=B, S=S, Hq=Hq, Hkv=Hkv, wq=None, wk=None, dwq=None,
               dwk=None, ws=None, **kw) != INVALID


def places(view, B, S, H):
    o, b, s, h = view
    return [o + i * b + j * s + k * h + d for i in range(B) for j in range(S)
            for k in range(H) for d in range(D)]


@pytest.fixture(scope="module", autouse=True)
def without_a_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the device's own check answers alike")


def test_heads_within_tokens_that_meet_across_the_batch(lib):
    """dk of the first sequence's second token is dq of the second's first."""
    views = [(0, 192, 128, D), (D, 192, 128, D), (4096, 192, 128, D)]
    assert not taken(lib, views, 2, 2, 1, 1)


@pytest.mark.parametrize("B,S,Hq,Hkv", [(2, 3, 4, 2), (3, 1, 2, 2), (1, 5, 2, 1),
                                        (2, 2, 1, 1), (4, 3, 1, 1)])
def test_packed_buffers_are_taken(lib, B, S, Hq, Hkv):
    n = Hq + 2 * Hkv
    first = (0, Hq, Hq + Hkv)
    # [B, S, heads, D], [B, heads, S, D], [S, B, heads, D], [heads, B, S, D]
    for b, s, h in ((S * n * D, n * D, D), (n * S * D, D, S * D),
                    (n * D, B * n * D, D), (S * D, D, B * S * D)):
        views = [(f * h, b, s, h) for f in first]
        assert taken(lib, views, B, S, Hq, Hkv)
        # In any order, and with room between.
        for x in itertools.permutations(views):
            if Hq == Hkv:
                assert taken(lib, list(x), B, S, Hq, Hkv)
        # One head over.
        views[1] = ((first[1] - 1) * h, b, s, h)
        assert not taken(lib, views, B, S, Hq, Hkv)
    # Heads of queries, keys and values in turn.
    if Hq == Hkv:
        views = [(i * D, S * n * D, n * D, 3 * D) for i in range(3)]
        assert taken(lib, views, B, S, Hq, Hkv)


def test_views_that_share_an_element_are_never_taken(lib):
    """Random strides against the sets of places; and of those that share none
    some are taken."""
    rng = random.Random(1)
    shared = apart = some = 0
    for _ in range(4000):
        B, S, Hq, Hkv = (rng.choice((1, 2, 3)) for _ in range(4))
        strides = lambda: [D * rng.choice((1, 2, 3, 4, 6, 8, 9, 12))
                           for _ in range(3)]
        st = strides()
        views = [(D * rng.randrange(0, 14),
                  *(st if rng.random() < 0.7 else strides()))
                 for _ in range(2)] + [(1 << 20, 4096, 512, D)]
        got = taken(lib, views, B, S, Hq, Hkv)
        q, k = (places(v, B, S, H) for v, H in zip(views, (Hq, Hkv)))
        if len(set(q)) < len(q) or len(set(k)) < len(k) or set(q) & set(k):
            shared += 1
            assert not got, (B, S, Hq, Hkv, views)
        else:
            apart += 1
            some += got
    assert shared > 500 and apart > 500 and some > 200
