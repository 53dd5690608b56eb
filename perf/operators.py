"""The 8-bit cache operators: their plain forms, their calls and the sizes they are timed at.

Three operators of a decoder's cache whose keys and values are held as E4M3
codes with one fp32 scale for each block of `block` tokens of a head:

  append   quantises the K and V of new tokens into the cache;
  fwd      attention of new query rows over it, with the row log-sum-exps and,
           on request, the attention weight each cached token received added
           to an accumulator;
  evict    keeps the tokens of most accumulated weight (and the latest ones)
           and writes them, requantised, to a smaller cache.

A length lens[b] counts the tokens of sequence b, the new ones included; the
new tokens are its last new[b] (at most the Sq rows given, left-aligned).
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step's K and V of a batch (the smallest call there is).
        dict(name="append_step", op="append", B=8, Hkv=8, cap=4096, D=128, block=64, Sq=1, dtype="bf16", spread=600, ragged=False),
        # A batch of prompts written at once into an empty cache.
        dict(name="append_prompt", op="append", B=8, Hkv=8, cap=4096, D=128, block=64, Sq=4096, dtype="bf16", spread=0, ragged=False),
        # A padded batch of continued prompts: odd lengths, blocks half full.
        dict(name="append_ragged", op="append", B=5, Hkv=3, cap=1501, D=64, block=32, Sq=301, dtype="f16", spread=700, ragged=True),
        # One decoding step over a 4096-token cache, weights accumulated.
        dict(name="fwd_step", op="fwd", B=8, Hq=32, Hkv=8, cap=4096, D=128, block=64, Sq=1, dtype="bf16", spread=64, ragged=False, causal=True, weights=True),
        # One decoding step of a single very long conversation.
        dict(name="fwd_step_long", op="fwd", B=1, Hq=32, Hkv=4, cap=131072, D=128, block=128, Sq=1, dtype="bf16", spread=99, ragged=False, causal=True, weights=False),
        # The same without shared heads, small heads, lengths from 0 up.
        dict(name="fwd_step_mha", op="fwd", B=16, Hq=16, Hkv=16, cap=2048, D=64, block=32, Sq=1, dtype="f16", spread=2048, ragged=False, causal=True, weights=True),
        # A few drafted tokens checked at once, padded batch, odd sizes.
        dict(name="fwd_draft", op="fwd", B=7, Hq=12, Hkv=4, cap=3001, D=64, block=16, Sq=5, dtype="f16", spread=3001, ragged=True, causal=True, weights=True),
        # A prompt's chunk of 512 tokens over the 4096 cached ones.
        dict(name="fwd_chunk", op="fwd", B=8, Hq=32, Hkv=8, cap=4096, D=128, block=64, Sq=512, dtype="bf16", spread=0, ragged=False, causal=True, weights=False),
        # The last 64 tokens of a prompt, whose weights choose what is kept.
        dict(name="fwd_observe", op="fwd", B=2, Hq=32, Hkv=8, cap=8192, D=128, block=64, Sq=64, dtype="bf16", spread=1000, ragged=False, causal=True, weights=True),
        # Cross attention to cached encoder states of ragged lengths.
        dict(name="fwd_cross", op="fwd", B=4, Hq=16, Hkv=16, cap=1500, D=64, block=32, Sq=200, dtype="f16", spread=1500, ragged=True, causal=False, weights=False),
        # A batch's caches halved between two decoding steps.
        dict(name="evict_batch", op="evict", B=8, Hkv=8, cap=4096, D=128, block=64, keep=2048, recent=256, spread=64),
        # A long prompt's cache compressed once to an eighth.
        dict(name="evict_long", op="evict", B=1, Hkv=4, cap=131072, D=128, block=128, keep=16384, recent=1024, spread=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "fwd", "fwd", "evict"])
    D = rng.choice([64, 128])
    block = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    B = _log_int(rng, 1, 32)
    cap = _log_int(rng, 65, 131072)
    most = 1 << 19  # tokens times heads of a drawn cache
    cap = max(65, min(cap, most // (B * Hkv)))
    spread = rng.choice([0, cap // 3, cap])
    if op == "evict":
        keep = rng.randint(1, cap)
        return dict(op=op, B=B, Hkv=Hkv, cap=cap, D=D, block=block, keep=keep, recent=rng.randint(0, min(keep, 1024)), spread=spread)
    Sq = rng.choice([1, 1, _log_int(rng, 2, 9), _log_int(rng, 10, 600)])
    Sq = min(Sq, cap)
    ragged = rng.random() < 0.5
    dtype = rng.choice(["bf16", "f16"])
    if op == "append":
        return dict(op=op, B=B, Hkv=Hkv, cap=cap, D=D, block=block, Sq=Sq, dtype=dtype, spread=spread, ragged=ragged)
    group = rng.choice([1, 2, 3, 4, 7, 8])
    scores = B * Hkv * group * cap  # fp32 scores of one row each: bounded
    Sq = max(1, min(Sq, (1 << 29) // scores, int(5e8) // scores))
    return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, cap=cap, D=D, block=block, Sq=Sq, dtype=dtype, spread=spread, ragged=ragged,
                causal=rng.random() < 0.8, weights=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _lens(case, gen):
    """Lengths of the sequences: the capacity less up to `spread`."""
    less = torch.randint(0, case["spread"] + 1, (case["B"],), generator=gen)
    if case["spread"]:
        less[0] = 0
    return (case["cap"] - less).to(torch.int32)


def _work_lens(case):
    """The lengths' mean, for work(): half of `spread` below the capacity."""
    return case["cap"] - case["spread"] / 2


def _tokens(B, H, S, D, gen):
    """Keys or values as projections give them: channels of unlike size, a
    few of them large, and tokens of unlike size."""
    x = torch.randn(B, H, S, D, generator=gen, device="cuda")
    channel = torch.exp(0.5 * torch.randn(1, H, 1, D, generator=gen, device="cuda"))
    token = torch.exp(0.3 * torch.randn(B, H, S, 1, generator=gen, device="cuda"))
    return x.mul_(channel).mul_(token)


def _blocks(case):
    return -(-case["cap"] // case["block"])


def _filled(case, lens, gen):
    """Codes and scales of a cache filled to `lens`; behind them lies what
    memory that was never written may hold."""
    B, H, S, D, n = case["B"], case["Hkv"], case["cap"], case["D"], case["block"]
    x = _tokens(B, H, S, D, gen)
    used = (torch.arange(S, device="cuda")[None] < lens[:, None])[:, None, :, None]
    x = torch.where(used, x, torch.zeros_like(x))
    pad = _blocks(case) * n - S
    xb = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, -1, n, D)
    scale = _scale_for(xb.abs().amax(dim=(3, 4)))
    code = (xb / scale[..., None, None]).to(torch.float8_e4m3fn).view(B, H, -1, D)[:, :, :S].contiguous()
    code.view(torch.uint8).masked_fill_(~used, 0x7F)  # NaN
    begun = torch.arange(_blocks(case), device="cuda")[None] * n < lens[:, None]
    scale = torch.where(begun[:, None], scale, torch.full_like(scale, float("inf")))
    return code, scale.contiguous()


def _scale_for(amax):
    """The smallest power of two that brings amax to 448 = 1.75 * 2^8 or less."""
    bits = amax.float().view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return ((e.clamp(min=-126) + 127) << 23).view(torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    B, H, S, D = case["B"], case["Hkv"], case["cap"], case["D"]
    lens = _lens(case, host)
    st = {"case": case}
    if case["op"] in ("append", "fwd"):
        # New tokens of each sequence: all Sq rows, or fewer in a padded batch.
        new = torch.full((B,), case["Sq"], dtype=torch.int32)
        if case["ragged"]:
            new = torch.randint(0, case["Sq"] + 1, (B,), generator=host).to(torch.int32)
            new[0] = case["Sq"]
        if case["op"] == "append" or case["causal"]:
            new = torch.minimum(new, lens)
        st["new"] = new.cuda() if case["ragged"] or case["spread"] else None
    lens = lens.cuda()
    if case["op"] == "append":
        before = lens - (st["new"] if st["new"] is not None else case["Sq"])
        st["k"], st["k_scale"] = _filled(case, before, gen)
        st["v"], st["v_scale"] = _filled(case, before, gen)
        st["k_new"] = _tokens(B, H, case["Sq"], D, gen).to(_dtype(case))
        st["v_new"] = _tokens(B, H, case["Sq"], D, gen).to(_dtype(case))
    else:
        st["k"], st["k_scale"] = _filled(case, lens, gen)
        st["v"], st["v_scale"] = _filled(case, lens, gen)
    st["lens"] = lens
    if case["op"] == "fwd":
        shape = (B, case["Hq"], case["Sq"])
        st["q"] = torch.randn(*shape, D, generator=gen, device="cuda").to(_dtype(case))
        st["o"] = torch.zeros(*shape, D, device="cuda", dtype=_dtype(case))
        st["lse"] = torch.zeros(*shape, device="cuda")
        st["weights"] = torch.rand(B, H, S, generator=gen, device="cuda") if case["weights"] else None
    if case["op"] == "evict":
        # Few tokens receive most of the weight, and some none at all.
        w = torch.rand(B, H, S, generator=gen, device="cuda").pow_(8)
        st["weights"] = torch.where(w < 1e-6, torch.zeros_like(w), w)
        room = case["keep"] + case["block"]  # for the tokens to come
        st["out_k"], st["out_v"] = torch.zeros(2, B, H, room, D, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).unbind()
        st["out_k_scale"] = torch.zeros(B, H, -(-room // case["block"]), device="cuda")
        st["out_v_scale"] = torch.zeros_like(st["out_k_scale"])
        st["out_lens"] = torch.zeros(B, device="cuda", dtype=torch.int32)
        st["out_weights"] = torch.zeros(B, H, room, device="cuda")
        st["indices"] = torch.zeros(B, H, case["keep"], device="cuda", dtype=torch.int32)
    if own:  # the handles that a serving program makes once
        import attention_attn_fwd_gb300 as attn
        st["cache"] = attn.KV8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"], lens, case["block"])
        if case["op"] == "fwd":
            st["workspace"] = attn.kv8_workspace(st["cache"], case["Hq"], case["Sq"], case["weights"])
        if case["op"] == "evict":
            st["out"] = attn.KV8Cache(st["out_k"], st["out_v"], st["out_k_scale"], st["out_v_scale"], st["out_lens"], case["block"])
    return st


# ------------------------------------------------------------------- passes

def run(st):
    case = st["case"]
    if case["op"] == "append":
        if own:
            import attention_attn_fwd_gb300 as attn
            attn.kv8_append(st["cache"], st["k_new"], st["v_new"], new_lens=st["new"])
        else:
            _plain_append(st)
        # E4M3 numbers and their blocks' factors, the whole cache.
        return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if case["op"] == "fwd":
        if own:
            import attention_attn_fwd_gb300 as attn
            attn.kv8_fwd(st["cache"], st["q"], causal=case["causal"], new_lens=st["new"], weights=st["weights"], out=st["o"], lse=st["lse"], workspace=st["workspace"])
        else:
            _plain_fwd(st)
        return {"o": st["o"], "lse": st["lse"], "weights": st["weights"]}
    if own:
        import attention_attn_fwd_gb300 as attn
        attn.kv8_evict(st["cache"], st["weights"], case["keep"], recent=case["recent"], out=st["out"], out_weights=st["out_weights"], indices=st["indices"])
    else:
        _plain_evict(st)
    return {k: st[k] for k in ("out_k", "out_v", "out_k_scale", "out_v_scale", "out_lens", "out_weights", "indices")}


def _plain_append(st):
    case = st["case"]
    n, D, S, Sq = case["block"], case["D"], case["cap"], case["Sq"]
    new = st["new"] if st["new"] is not None else torch.full_like(st["lens"], Sq)
    start = (st["lens"] - new).long()
    pos = torch.arange(S, device="cuda")[None] - start[:, None]  # [B, S]: which new token
    fresh = (pos >= 0) & (pos < new[:, None])
    old = pos < 0
    nb = _blocks(case)
    pad = nb * n - S
    begun = (torch.arange(nb, device="cuda")[None] * n) < start[:, None]  # holds earlier tokens
    touched = torch.nn.functional.pad(fresh, (0, pad)).view(-1, nb, n).any(2)
    for code, scale, x in ((st["k"], st["k_scale"], st["k_new"]), (st["v"], st["v_scale"], st["v_new"])):
        B, H = x.shape[:2]
        at = pos.clamp(0, Sq - 1)[:, None, :, None].expand(B, H, S, D)
        x = torch.where(fresh[:, None, :, None], torch.gather(x, 2, at).float(), 0.0)
        finite = torch.where(torch.isfinite(x), x.abs(), 0.0)
        amax = torch.nn.functional.pad(finite, (0, 0, 0, pad)).view(B, H, nb, n, D).amax(dim=(3, 4))
        tight = _scale_for(amax)
        keeps = begun[:, None] & (amax <= E4M3_MAX * scale)
        after = torch.where(touched[:, None], torch.where(keeps, scale, tight), scale)
        each = lambda s: s.repeat_interleave(n, 2)[:, :, :S, None]  # noqa: E731
        was = torch.where(old[:, None, :, None], code.float() * each(scale), 0.0)
        value = torch.where(fresh[:, None, :, None], x, was)
        q = (value / each(after)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        grown = (touched[:, None] & begun[:, None] & ~keeps).repeat_interleave(n, 2)[:, :, :S]
        write = fresh[:, None] | (old[:, None] & grown)
        code.view(torch.uint8).copy_(torch.where(write[..., None], q.view(torch.uint8), code.view(torch.uint8)))
        scale.copy_(after)


def _values(code, scale, n, lens):
    """The numbers a cache stands for, in 32 bits; zero behind the lengths."""
    S = code.shape[2]
    x = code.float() * scale.repeat_interleave(n, 2)[:, :, :S, None]
    used = torch.arange(S, device="cuda")[None] < lens[:, None]
    return torch.where(used[:, None, :, None], x, 0.0)


def _visible(case, lens, new):
    """[B, Sq, S]: the keys each new row sees."""
    j = torch.arange(case["cap"], device="cuda")
    i = torch.arange(case["Sq"], device="cuda")
    end = lens[:, None].expand(-1, case["Sq"])
    if case["causal"]:
        end = (lens - new)[:, None] + i + 1
    return (j < end[..., None]) & (i < new[:, None])[..., None]


def _plain_fwd(st):
    case, q = st["case"], st["q"]
    B, Hq, Sq, D = q.shape
    H = case["Hkv"]
    g = Hq // H
    new = st["new"] if st["new"] is not None else torch.full_like(st["lens"], Sq)
    k = _values(st["k"], st["k_scale"], case["block"], st["lens"])
    v = _values(st["v"], st["v_scale"], case["block"], st["lens"])
    s = q.float().view(B, H, g * Sq, D) @ k.transpose(2, 3) / math.sqrt(D)
    s = s.view(B, H, g, Sq, -1)
    s.masked_fill_(~_visible(case, st["lens"], new)[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(m == -math.inf, 0.0, m)))
    l = p.sum(-1, keepdim=True)
    p.mul_(torch.where(l > 0, 1.0 / l, 0.0))
    o = (p.view(B, H, g * Sq, -1) @ v).view(B, Hq, Sq, D)
    lse = (m + torch.log(l)).view(B, Hq, Sq)
    row = (torch.arange(Sq, device="cuda")[None] < new[:, None])[:, None]
    st["o"].copy_(torch.where(row[..., None], o, st["o"].float()))
    st["lse"].copy_(torch.where(row, lse, st["lse"]))
    if st["weights"] is not None:
        st["weights"].add_(p.sum(dim=(2, 3)))


def _plain_evict(st):
    case, lens = st["case"], st["lens"].long()
    B, H, S, D = st["k"].shape
    n, keep, recent = case["block"], case["keep"], case["recent"]
    j = torch.arange(S, device="cuda")[None]
    w = st["weights"].double()
    w = torch.where((j >= lens[:, None] - recent)[:, None], math.inf, w)
    w = torch.where((j < lens[:, None])[:, None], w, -math.inf)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :keep]
    kept = torch.arange(keep, device="cuda")[None] < lens[:, None]  # [B, keep]
    order = torch.sort(torch.where(kept[:, None], order, S), dim=2).values
    at = order.clamp(max=S - 1)
    st["indices"].copy_(torch.where(kept[:, None], order, -1))
    st["out_lens"].copy_(lens.clamp(max=keep))
    st["out_weights"].zero_()
    st["out_weights"][:, :, :keep] = torch.where(kept[:, None], torch.gather(st["weights"], 2, at), 0.0)
    nb = -(-keep // n)
    pad = nb * n - keep
    whole = (lens <= keep)[:, None, None]  # nothing leaves: copied as they are
    begun = (torch.arange(nb, device="cuda")[None] * n < lens[:, None])[:, None]
    for name in ("k", "v"):
        code, scale = st[name], st[name + "_scale"]
        at4 = at[..., None].expand(B, H, keep, D)
        old = torch.gather(code.view(torch.uint8), 2, at4)
        factor = torch.gather(scale, 2, at // n)
        value = torch.where(kept[:, None, :, None], old.view(torch.float8_e4m3fn).float() * factor[..., None], 0.0)
        amax = torch.nn.functional.pad(value, (0, 0, 0, pad)).view(B, H, nb, n, D).abs().amax(dim=(3, 4))
        tight = torch.where(whole, torch.nn.functional.pad(scale, (0, nb))[:, :, :nb], _scale_for(amax))
        q = (value / tight.repeat_interleave(n, 2)[:, :, :keep, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        q = torch.where(whole[..., None], old, q)
        out = st["out_" + name].view(torch.uint8)[:, :, :keep]
        out.copy_(torch.where(kept[:, None, :, None], q, out))
        out = st["out_" + name + "_scale"][:, :, :nb]
        out.copy_(torch.where(begun, tight, out))


# ------------------------------------------------------ what a pass has to do

def work(case):
    B, H, D, n = case["B"], case["Hkv"], case["D"], case["block"]
    tokens = _work_lens(case)
    rows = case.get("Sq", 1) * (0.5 if case.get("ragged") else 1.0)
    if case["op"] == "append":
        # Each new K and V element read (2 bytes) and its code written (1).
        t = B * H * min(rows, tokens)
        return {"bytes": 2 * t * (3 * D + 4 / n), "flops": 4 * t * D}
    if case["op"] == "fwd":
        seen = tokens - (rows - 1) / 2 if case["causal"] else tokens
        seen = max(seen, 1)
        b = 2 * B * H * tokens * (D + 4 / n) + B * case["Hq"] * rows * (4 * D + 4)
        if case["weights"]:
            b += 8 * B * H * tokens
        return {"bytes": b, "flops": 4 * B * case["Hq"] * rows * seen * D}
    kept = min(case["keep"], tokens)
    # Weights read; the kept tokens read and written, with their weights and places.
    return {"bytes": B * H * (4 * tokens + 2 * kept * 2 * (D + 4 / n) + 8 * kept), "flops": B * H * (2 * kept * 2 * D + tokens)}


# --------------------------------------------------------- 64-bit definition

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "fwd": _exact_fwd, "evict": _exact_evict}[case["op"]](case, st)


def _pow2(amax):
    """Smallest 2^e >= amax / 448 by its binary exponent, e >= -126."""
    frac, e = torch.frexp(amax.double() / 448.0)  # amax/448 = frac 2^e, frac in [0.5, 1)
    e = e - (frac == 0.5).int()
    return _two_to(torch.where(amax > 0, e, -126).clamp(min=-126))


def _two_to(e):
    """2^e in 64 bits, for whole numbers e of a double's normal range."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """x to 4 significant bits (spacing 2^-9 at least), half to even."""
    _, e = torch.frexp(x)
    step = _two_to((e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(case, st):
    n, Sq = case["block"], case["Sq"]
    lens = st["lens"].tolist()
    new = st["new"].tolist() if st["new"] is not None else [Sq] * case["B"]
    if sum(-(-c // n) + 1 for c in new) > 4000:
        return None
    out = {}
    for name in ("k", "v"):
        code = st[name].double()
        scale = st[name + "_scale"].double()
        for b in range(case["B"]):
            p0, t = lens[b] - new[b], 0
            while t < new[b]:
                blk = (p0 + t) // n
                c = min(new[b] - t, (blk + 1) * n - p0 - t)
                x = st[name + "_new"][b, :, t:t + c].double()
                amax = x.abs().amax(dim=(1, 2))
                s = _pow2(amax)
                first = blk * n
                if first < p0 + t and t == 0:  # a block begun earlier
                    was = scale[b, :, blk].clone()
                    s = torch.where(amax <= 448.0 * was, was, s)
                    held = code[b, :, first:p0] * was[:, None, None]
                    code[b, :, first:p0] = _round_e4m3(held / s[:, None, None])
                code[b, :, p0 + t:p0 + t + c] = _round_e4m3(x / s[:, None, None])
                scale[b, :, blk] = s
                t += c
        out[name], out[name + "_scale"] = code, scale
    return out


def _exact_fwd(case, st):
    B, Hq, Sq, D = st["q"].shape
    H, n = case["Hkv"], case["block"]
    lens = st["lens"].tolist()
    new = st["new"].tolist() if st["new"] is not None else [Sq] * B
    o, lse = st["o"].double(), st["lse"].double()
    w = st["weights"].double() if st["weights"] is not None else None
    for b in range(B):
        c, L = new[b], lens[b]
        if c == 0:
            continue
        for h in range(Hq):
            kv = h // (Hq // H)
            if L == 0:
                o[b, h, :c], lse[b, h, :c] = 0.0, -math.inf
                continue
            blk = torch.arange(L, device="cuda") // n
            k = st["k"][b, kv, :L].double() * st["k_scale"][b, kv].double()[blk][:, None]
            v = st["v"][b, kv, :L].double() * st["v_scale"][b, kv].double()[blk][:, None]
            s = (st["q"][b, h, :c].double() @ k.T) / math.sqrt(D)
            if case["causal"]:
                late = torch.arange(L, device="cuda")[None] > (L - c + torch.arange(c, device="cuda"))[:, None]
                s = s.masked_fill(late, -math.inf)
            lse[b, h, :c] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[b, h, :c, None])
            o[b, h, :c] = p @ v
            if w is not None:
                w[b, kv, :L] += p.sum(0)
    return {"o": o, "lse": lse, "weights": w}


def _exact_evict(case, st):
    n, keep, recent = case["block"], case["keep"], case["recent"]
    B, H = case["B"], case["Hkv"]
    out = {k: st[k].double() for k in ("out_k", "out_v", "out_k_scale", "out_v_scale", "out_weights")}
    for b in range(B):
        L = int(st["lens"][b])
        m = min(L, keep)
        nb = -(-m // n)
        for h in range(H):
            if L <= keep:
                idx = torch.arange(L, device="cuda")
            else:
                c = L - recent  # candidates: value down, then place up
                place = torch.arange(c, device="cuda")
                value, first = torch.sort(st["weights"][b, h, :c].double(), descending=True, stable=True)
                idx = torch.cat([place[first[:keep - recent]], torch.arange(c, L, device="cuda")]).sort().values
            out["out_weights"][b, h] = 0.0
            out["out_weights"][b, h, :m] = st["weights"][b, h, idx].double()
            for name in ("k", "v"):
                code = st[name][b, h, idx].double()
                scale = st[name + "_scale"][b, h].double()
                if L <= keep:
                    out["out_" + name][b, h, :m], out["out_%s_scale" % name][b, h, :nb] = code, scale[:nb]
                    continue
                x = torch.zeros(nb * n, case["D"], device="cuda", dtype=torch.float64)
                x[:m] = code * scale[idx // n][:, None]
                s = _pow2(x.view(nb, -1).abs().amax(1))
                out["out_" + name][b, h, :m] = _round_e4m3(x / s.repeat_interleave(n)[:, None])[:m]
                out["out_%s_scale" % name][b, h, :nb] = s
    return {**{k: out.get(k) for k in ("out_k", "out_v", "out_k_scale", "out_v_scale", "out_weights")}, "out_lens": None, "indices": None}
