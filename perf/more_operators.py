"""What a decoder layer does around its attention: the plain forms, the calls and the sizes they are timed at.

  rope      norms the queries and keys of each head and rotates them by their
            positions, on one or several axes, on the way from the projections'
            [B, S, H, D] to the attention's [B, H, S, D] or into a cache;
  rope_bwd  its backward pass: the projections' gradients and the norm weights';
  prefix    attention of a batch whose sequences share a long prefix: the
            prefix's keys and values are held once, each sequence's own behind.

A cache's length lens[b] counts the tokens of sequence b, the new ones
included; the new tokens are its last new[b] (at most the S rows given,
left-aligned).
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step of a batch into its cache (the smallest call there is).
        dict(name="rope_step", op="rope", B=8, S=1, Hq=32, Hkv=8, D=128, rot=128, axes=1, interleaved=False, norm=True, f32w=False, cap=4096, offset=8192, spread=600, ragged=False, packed=False, dtype="bf16"),
        # A prompt of 8192 tokens, shared heads, separate projections.
        dict(name="rope_prompt", op="rope", B=1, S=8192, Hq=32, Hkv=4, D=128, rot=128, axes=1, interleaved=False, norm=True, f32w=False, cap=0, offset=0, spread=0, ragged=False, packed=False, dtype="bf16"),
        # Clips of video tokens at (time, height, width), one packed projection, neighbouring pairs.
        dict(name="rope_video", op="rope", B=2, S=4051, Hq=16, Hkv=16, D=64, rot=64, axes=3, interleaved=True, norm=True, f32w=True, cap=0, offset=0, spread=0, ragged=False, packed=True, dtype="f16"),
        # A padded batch of continued prompts, odd sizes, half of each head rotated, no norm.
        dict(name="rope_ragged", op="rope", B=5, S=301, Hq=12, Hkv=3, D=64, rot=32, axes=1, interleaved=False, norm=False, f32w=False, cap=1501, offset=777, spread=700, ragged=True, packed=True, dtype="f16"),
        # A training step's backward over a batch of 4096-token sequences.
        dict(name="bwd_train", op="rope_bwd", B=4, S=4096, Hq=32, Hkv=8, D=128, rot=128, axes=1, interleaved=False, norm=True, f32w=False, packed=True, dtype="bf16"),
        # A small batch of images and text at three axes, odd sizes, three quarters rotated.
        dict(name="bwd_axes", op="rope_bwd", B=3, S=331, Hq=10, Hkv=5, D=64, rot=48, axes=3, interleaved=False, norm=True, f32w=True, packed=False, dtype="f16"),
        # A small batch's decoding step behind a system prompt.
        dict(name="prefix_step", op="prefix", B=8, Hq=32, Hkv=8, D=128, Sq=1, P=4096, cap=512, spread=400, ragged=False, causal=True, dtype="bf16"),
        # A large batch's decoding step behind a long shared document.
        dict(name="prefix_batch", op="prefix", B=64, Hq=32, Hkv=8, D=128, Sq=1, P=8192, cap=1024, spread=1000, ragged=False, causal=True, dtype="bf16"),
        # Many samples of one prompt, no shared heads, small heads.
        dict(name="prefix_samples", op="prefix", B=256, Hq=16, Hkv=16, D=64, Sq=1, P=2048, cap=300, spread=299, ragged=False, causal=True, dtype="f16"),
        # One very long prefix, short answers.
        dict(name="prefix_long", op="prefix", B=32, Hq=32, Hkv=4, D=128, Sq=1, P=65531, cap=256, spread=200, ragged=False, causal=True, dtype="bf16"),
        # Drafted tokens checked at once, padded batch, odd sizes.
        dict(name="prefix_draft", op="prefix", B=24, Hq=21, Hkv=3, D=64, Sq=5, P=5001, cap=901, spread=901, ragged=True, causal=True, dtype="f16"),
        # Prompts' chunks of 512 tokens behind 3584 shared ones.
        dict(name="prefix_chunk", op="prefix", B=8, Hq=32, Hkv=8, D=128, Sq=512, P=3584, cap=512, spread=0, ragged=False, causal=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "prefix", "prefix"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    dtype = rng.choice(["bf16", "f16"])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "prefix":
        B = _log_int(rng, 1, 256)
        P = _log_int(rng, 1, 65536)
        cap = _log_int(rng, 1, 2048)
        cap = max(1, min(cap, (1 << 18) // (B * Hkv)))
        Sq = min(cap, rng.choice([1, 1, 1, _log_int(rng, 2, 9), _log_int(rng, 10, 512)]))
        while B * Hkv * group * Sq * (P + cap) > 2.5e8:  # scores of a pass
            if Sq > 1:
                Sq = -(-Sq // 2)
            else:
                P = -(-P // 2)
        spread = rng.choice([0, cap // 3, cap])
        return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, Sq=Sq, P=P, cap=cap, spread=spread, ragged=rng.random() < 0.4, causal=rng.random() < 0.8, dtype=dtype)
    Hq = Hkv * group
    B = _log_int(rng, 1, 32)
    most = (1 << 26) // ((Hq + 2 * Hkv) * D * B)
    S = rng.choice([1, _log_int(rng, 2, 600), _log_int(rng, 600, 8192)])
    S = max(1, min(S, most))
    rot = rng.choice([D // 4, D // 2, 3 * D // 4, D, D])
    case = dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, rot=rot, axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, f32w=rng.random() < 0.4, packed=rng.random() < 0.5, dtype=dtype)
    if op == "rope_bwd":
        return case
    cached = S <= 600 and rng.random() < 0.6
    cap = S + _log_int(rng, 1, 2000) if cached else 0
    return dict(case, cap=cap, offset=_log_int(rng, 1, 100000) if cached else 0, spread=rng.choice([0, cap // 3, cap]) if cached else 0, ragged=cached and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _tokens(B, S, H, D, gen):
    """Projections' outputs: channels of unlike size, a few of them large,
    and tokens of unlike size."""
    x = torch.randn(B, S, H, D, generator=gen, device="cuda")
    channel = torch.exp(0.5 * torch.randn(1, 1, H, D, generator=gen, device="cuda"))
    token = torch.exp(0.3 * torch.randn(B, S, H, 1, generator=gen, device="cuda"))
    return x.mul_(channel).mul_(token)


def _lens(case, host):
    """Lengths of the sequences, the capacity less up to `spread`, and their new tokens."""
    less = torch.randint(0, case["spread"] + 1, (case["B"],), generator=host)
    if case["spread"]:
        less[0] = 0
    lens = (case["cap"] - less).to(torch.int32)
    rows = case["S"] if "S" in case else case["Sq"]
    new = torch.full((case["B"],), rows, dtype=torch.int32)
    if case["ragged"]:
        new = torch.randint(0, rows + 1, (case["B"],), generator=host).to(torch.int32)
        new[0] = rows
    if case.get("causal", True):
        new = torch.minimum(new, lens)
    return lens.cuda(), new.cuda() if case["ragged"] or case["spread"] else None


def _cache(case, filled, gen):
    """Keys or values of tokens up to `filled`; behind them lies what memory
    that was never written may hold."""
    x = _tokens(case["B"], case["cap"], case["Hkv"], case["D"], gen).transpose(1, 2).to(_dtype(case)).contiguous()
    late = torch.arange(case["cap"], device="cuda")[None] >= filled[:, None]
    return x.masked_fill_(late[:, None, :, None], math.nan)


def _grid(case):
    """Positions of B clips of S tokens on the axes, the last one fastest."""
    i = torch.arange(case["S"], device="cuda", dtype=torch.int32)
    i = i[None] + 5 * torch.arange(case["B"], device="cuda", dtype=torch.int32)[:, None]
    side = max(1, round(case["S"] ** (1 / case["axes"])))
    return torch.stack([i // side ** a if a == case["axes"] - 1 else i // side ** a % side for a in reversed(range(case["axes"]))]).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    st = {"case": case}
    if case["op"] == "prefix":
        _prepare_prefix(case, st, gen, host)
    else:
        _prepare_rope(case, st, gen, host)
    return st


def _prepare_rope(case, st, gen, host):
    B, S, Hq, Hkv, D, n = case["B"], case["S"], case["Hq"], case["Hkv"], case["D"], case["rot"] // 2
    dt = _dtype(case)
    # Frequencies and axes of the pairs, as a model's configuration gives them.
    st["freq"] = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    st["axis"] = torch.arange(n) * case["axes"] // n
    st["freq_gpu"], st["axis_gpu"] = st["freq"].cuda(), st["axis"].cuda()
    if case["packed"]:
        st["qkv"] = _tokens(B, S, Hq + 2 * Hkv, D, gen).to(dt)
    else:
        st["q"], st["k"], st["v"] = (_tokens(B, S, H, D, gen).to(dt) for H in (Hq, Hkv, Hkv))
    st["wq"] = st["wk"] = None
    if case["norm"]:
        wt = torch.float32 if case["f32w"] else dt
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(wt) for _ in range(2))
    # Positions: given where there are several axes, else counted.
    st["pos"] = _grid(case) if case["axes"] > 1 else None
    st["lens"] = st["new"] = st["offset"] = None
    if case["op"] == "rope_bwd":
        st["dq"], st["dk"], st["dv"] = (_tokens(B, S, H, D, gen).transpose(1, 2).to(dt).contiguous() for H in (Hq, Hkv, Hkv))
        if case["packed"]:
            st["dqkv"] = torch.zeros_like(st["qkv"])
        else:
            st["dx"] = [torch.zeros_like(st[x]) for x in "qkv"]
        if case["norm"]:
            st["dwq"], st["dwk"] = torch.zeros(2, D, device="cuda").unbind()
    else:
        st["q_out"] = torch.zeros(B, Hq, S, D, device="cuda", dtype=dt)
        if case["cap"]:
            st["lens"], st["new"] = _lens(case, host)
            before = st["lens"] - (st["new"] if st["new"] is not None else S)
            st["k_out"], st["v_out"] = _cache(case, before, gen), _cache(case, before, gen)
            if st["pos"] is None:
                st["offset"] = torch.tensor([case["offset"]], device="cuda", dtype=torch.int32)
        else:
            st["k_out"], st["v_out"] = (torch.zeros(B, Hkv, S, D, device="cuda", dtype=dt) for _ in range(2))
    if own:  # the handle that a model makes once
        import attention_attn_fwd_gb300 as attn
        st["rope"] = attn.Rope(st["freq"], D, axes=st["axis"], interleaved=case["interleaved"])
        if case["op"] == "rope_bwd":
            st["workspace"] = attn.qk_rope_bwd_workspace(st["rope"])


def _prepare_prefix(case, st, gen, host):
    B, Hq, Hkv, D, Sq, dt = case["B"], case["Hq"], case["Hkv"], case["D"], case["Sq"], _dtype(case)
    st["lens"], st["new"] = _lens(case, host)
    st["k"], st["v"] = _cache(case, st["lens"], gen), _cache(case, st["lens"], gen)
    # The prefix's memory has room for more than it holds.
    shared = dict(case, B=1, cap=case["P"] + 37)
    st["plen"] = torch.tensor([case["P"]], device="cuda", dtype=torch.int32)
    st["pk"], st["pv"] = _cache(shared, st["plen"], gen), _cache(shared, st["plen"], gen)
    st["q"] = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dt)
    st["o"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(B, Hq, Sq, device="cuda")
    if own:  # what a serving program makes once
        import attention_attn_fwd_gb300 as attn
        st["cache"] = attn.PrefixCache(st["pk"], st["pv"], st["plen"], st["k"], st["v"], st["lens"])
        st["workspace"] = attn.prefix_workspace(st["cache"], Hq, Sq)


# ------------------------------------------------------------------- passes

def _split(case, st, packed, apart):
    """The heads of queries, keys and values [B, S, H, D]."""
    if case["packed"]:
        return st[packed].split((case["Hq"], case["Hkv"], case["Hkv"]), 2)
    return apart


def run(st):
    case = st["case"]
    if case["op"] == "rope":
        q, k, v = _split(case, st, "qkv", (st.get("q"), st.get("k"), st.get("v")))
        if own:
            import attention_attn_fwd_gb300 as attn
            attn.qk_rope(st["rope"], q, k, v, q_weight=st["wq"], k_weight=st["wk"], eps=EPS, positions=st["pos"], lens=st["lens"], new_lens=st["new"], offset=st["offset"],
                         q_out=st["q_out"], k_out=st["k_out"], v_out=st["v_out"])
        else:
            _plain_rope(st, q, k, v)
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    if case["op"] == "rope_bwd":
        q, k, _ = _split(case, st, "qkv", (st.get("q"), st.get("k"), st.get("v")))
        dx = _split(case, st, "dqkv", st.get("dx"))
        dw = (st["dwq"], st["dwk"]) if case["norm"] else (None, None)
        if own:
            import attention_attn_fwd_gb300 as attn
            attn.qk_rope_bwd(st["rope"], st["dq"], st["dk"], q, k, dv=st["dv"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS, positions=st["pos"],
                             dq_out=dx[0], dk_out=dx[1], dv_out=dx[2], dq_weight=dw[0], dk_weight=dw[1], workspace=st["workspace"])
        else:
            _plain_rope_bwd(st, q, k, dx, dw)
        return {"dx": st["dqkv"] if case["packed"] else st["dx"], "dwq": dw[0], "dwk": dw[1]}
    if own:
        import attention_attn_fwd_gb300 as attn
        attn.prefix_fwd(st["cache"], st["q"], causal=case["causal"], new_lens=st["new"], out=st["o"], lse=st["lse"], workspace=st["workspace"])
    else:
        _plain_prefix(st)
    return {"o": st["o"], "lse": st["lse"]}


def _angles(st):
    """cos and sin of every token and pair, [B, S, 1, rot / 2]: the angles in 64 bits."""
    case = st["case"]
    B, S = case["B"], case["S"]
    if st["pos"] is not None:
        pos = st["pos"][st["axis_gpu"]].permute(1, 2, 0).double()
    else:
        pos = torch.arange(S, device="cuda", dtype=torch.float64)[None, :, None].expand(B, S, 1)
        if st["lens"] is not None:
            new = st["new"] if st["new"] is not None else S
            pos = pos + (st["lens"] - new + st["offset"]).double()[:, None, None]
    t = pos * st["freq_gpu"]
    return torch.cos(t).float()[:, :, None], torch.sin(t).float()[:, :, None]


def _halves(x, case):
    """The pairs' first and second numbers, and what is not rotated."""
    r = case["rot"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _joined(a, b, rest, case):
    if case["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _plain_rope(st, q, k, v):
    case = st["case"]
    cos, sin = _angles(st)
    done = []
    for x, w in ((q, st["wq"]), (k, st["wk"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b, rest = _halves(x, case)
        done.append(_joined(a * cos - b * sin, a * sin + b * cos, rest, case).transpose(1, 2))
    q, k = done
    v = v.transpose(1, 2)
    if not case["cap"]:
        st["q_out"].copy_(q)
        st["k_out"].copy_(k)
        st["v_out"].copy_(v)
        return
    S = case["S"]
    new = st["new"] if st["new"] is not None else torch.full_like(st["lens"], S)
    valid = (torch.arange(S, device="cuda")[None] < new[:, None])[:, None, :, None]
    st["q_out"].copy_(torch.where(valid, q, st["q_out"].float()))
    # The cache's place j takes the new token j - (lens - new).
    i = torch.arange(case["cap"], device="cuda")[None] - (st["lens"] - new)[:, None]
    fresh = ((i >= 0) & (i < new[:, None]))[:, None, :, None]
    at = i.clamp(0, S - 1)[:, None, :, None].expand(-1, case["Hkv"], -1, case["D"])
    for out, x in ((st["k_out"], k), (st["v_out"], v)):
        out.copy_(torch.where(fresh, torch.gather(x.to(out.dtype), 2, at), out))


def _plain_rope_bwd(st, q, k, dx, dw):
    case = st["case"]
    cos, sin = _angles(st)
    _plain_rope_bwd_one(case, st["dq"], q, st["wq"], cos, sin, dx[0], dw[0])
    _plain_rope_bwd_one(case, st["dk"], k, st["wk"], cos, sin, dx[1], dw[1])
    dx[2].copy_(st["dv"].transpose(1, 2))


def _plain_rope_bwd_one(case, dy, x, w, cos, sin, dx, dw):
    a, b, rest = _halves(dy.float().transpose(1, 2), case)
    dn = _joined(a * cos + b * sin, b * cos - a * sin, rest, case)
    if w is None:
        dx.copy_(dn)
        return
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * r
    dw.copy_((dn * xhat).sum(dim=(0, 1, 2)))
    g = dn * w.float()
    dx.copy_(r * (g - xhat * (g * xhat).mean(-1, keepdim=True)))


def _plain_prefix(st):
    case, q = st["case"], st["q"].float()
    B, Hq, Sq, D = q.shape
    H, P, S = case["Hkv"], case["P"], case["cap"]
    g = Hq // H
    new = st["new"] if st["new"] is not None else torch.full_like(st["lens"], Sq)
    used = (torch.arange(S, device="cuda")[None] < st["lens"][:, None])[:, None, :, None]
    k = torch.where(used, st["k"].float(), 0.0)
    v = torch.where(used, st["v"].float(), 0.0)
    q = (q / math.sqrt(D)).view(B, H, g * Sq, D)
    rows = q.transpose(0, 1).reshape(H, B * g * Sq, D)
    s0 = (rows @ st["pk"][0, :, :P].float().transpose(1, 2)).view(H, B, g * Sq, P).transpose(0, 1)
    s1 = q @ k.transpose(2, 3)
    end = st["lens"][:, None].expand(B, Sq)
    if case["causal"]:
        end = (st["lens"] - new)[:, None] + torch.arange(1, Sq + 1, device="cuda")
    seen = torch.arange(S, device="cuda") < end[..., None]
    s1.view(B, H, g, Sq, S).masked_fill_(~seen[:, None, None], -math.inf)
    m = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    p0, p1 = torch.exp(s0 - m), torch.exp(s1 - m)
    l = p0.sum(-1, keepdim=True) + p1.sum(-1, keepdim=True)
    o0 = p0.transpose(0, 1).reshape(H, B * g * Sq, P) @ st["pv"][0, :, :P].float()
    o = (o0.view(H, B, g * Sq, D).transpose(0, 1) + p1 @ v) / l
    row = (torch.arange(Sq, device="cuda")[None] < new[:, None])[:, None]
    st["o"].copy_(torch.where(row[..., None], o.reshape(B, Hq, Sq, D), st["o"].float()))
    st["lse"].copy_(torch.where(row, (m + torch.log(l)).reshape(B, Hq, Sq), st["lse"]))


# ------------------------------------------------------ what a pass has to do

def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    half = 0.5 if case.get("ragged") else 1.0
    if case["op"] != "prefix":
        t = B * case["S"] * half
        pos = 4 * case["axes"] * t if case["axes"] > 1 else 0
        if case["op"] == "rope":
            # Each element read and written; sums of squares, two products, four of the rotation.
            return {"bytes": 4 * t * (Hq + 2 * Hkv) * D + pos, "flops": 8 * t * (Hq + Hkv) * D}
        b = t * D * (6 * (Hq + Hkv) + 4 * Hkv) if case["norm"] else 4 * t * D * (Hq + 2 * Hkv)
        return {"bytes": b + pos, "flops": 16 * t * (Hq + Hkv) * D}
    rows = case["Sq"] * half
    tokens = case["cap"] - case["spread"] / 2
    seen = max(tokens - (rows - 1) / 2, 0) if case["causal"] else tokens
    b = 4 * Hkv * D * (case["P"] + B * tokens) + B * Hq * rows * (4 * D + 4)
    return {"bytes": b, "flops": 4 * B * Hq * rows * (case["P"] + seen) * D}


# --------------------------------------------------------- 64-bit definition

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(case, st)
    return _exact_rope(case, st) if case["op"] == "rope" else _exact_rope_bwd(case, st)


def _turns(case, st, b):
    """e^(i t) of every token of sequence b and pair, as complex numbers."""
    S = case["S"]
    pos = torch.arange(S, device="cuda", dtype=torch.float64)
    if st["lens"] is not None:
        new = int(st["new"][b]) if st["new"] is not None else S
        pos = pos + int(st["lens"][b]) - new + case["offset"]
    t = []
    for f, a in zip(st["freq"].tolist(), st["axis"].tolist()):
        p = pos if st["pos"] is None else st["pos"][a, b].double()
        t.append(p * f)
    t = torch.stack(t, 1)
    return torch.polar(torch.ones_like(t), t)


def _pairs(case):
    """Places of the pairs' first and second numbers."""
    i = torch.arange(case["rot"] // 2, device="cuda")
    return (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)


def _exact_rotated(case, x, turn):
    """x [S, D] with its pairs multiplied by turn [S, rot / 2]."""
    i, j = _pairs(case)
    z = torch.complex(x[:, i].contiguous(), x[:, j].contiguous()) * turn
    y = x.clone()
    y[:, i], y[:, j] = z.real, z.imag
    return y


def _parts(case, st):
    if case["packed"]:
        Hq, Hkv = case["Hq"], case["Hkv"]
        x = st["qkv"]
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    return st["q"], st["k"], st["v"]


def _exact_rope(case, st):
    out = {"q": st["q_out"].double(), "k": st["k_out"].double(), "v": st["v_out"].double()}
    x = dict(zip("qkv", _parts(case, st)))
    for b in range(case["B"]):
        turn = _turns(case, st, b)
        n = case["S"] if st["new"] is None else int(st["new"][b])
        at = 0 if st["lens"] is None else int(st["lens"][b]) - n
        for name, w, first in (("q", st["wq"], 0), ("k", st["wk"], at), ("v", None, at)):
            for h in range(x[name].shape[2]):
                y = x[name][b, :n, h].double()
                if w is not None:
                    y = y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS) * w.double()
                if name != "v":
                    y = _exact_rotated(case, y, turn[:n])
                out[name][b, h, first:first + n] = y
    return out


def _exact_rope_bwd(case, st):
    q, k, v = _parts(case, st)
    D = case["D"]
    back, dw = [], []
    for x, dy, w in ((q, st["dq"], st["wq"]), (k, st["dk"], st["wk"])):
        dx = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        total = torch.zeros(D, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            turn = _turns(case, st, b).conj()
            for h in range(x.shape[2]):
                dn = _exact_rotated(case, dy[b, h].double(), turn)
                if w is None:
                    dx[b, :, h] = dn
                    continue
                y = x[b, :, h].double()
                norm = torch.sqrt(y.square().sum(1, keepdim=True) / D + EPS)
                total += (dn * y / norm).sum(0)
                g = dn * w.double()
                # d(y / norm): the part along y is taken off.
                dx[b, :, h] = g / norm - y * (g * y).sum(1, keepdim=True) / (D * norm ** 3)
        back.append(dx)
        dw.append(total if w is not None else None)
    back.append(st["dv"].double().transpose(1, 2))
    return {"dx": torch.cat(back, 2) if case["packed"] else back, "dwq": dw[0], "dwk": dw[1]}


def _exact_prefix(case, st):
    B, Hq, Sq, D = st["q"].shape
    H, P = case["Hkv"], case["P"]
    g = Hq // H
    if B * H > 6000:
        return None
    lens = st["lens"].tolist()
    new = st["new"].tolist() if st["new"] is not None else [Sq] * B
    o, lse = st["o"].double(), st["lse"].double()
    for h in range(H):
        pk, pv = st["pk"][0, h, :P].double(), st["pv"][0, h, :P].double()
        for b in range(B):
            c, L = new[b], lens[b]
            if c == 0:
                continue
            k = torch.cat([pk, st["k"][b, h, :L].double()])
            v = torch.cat([pv, st["v"][b, h, :L].double()])
            x = st["q"][b, h * g:(h + 1) * g, :c].double().reshape(g * c, D)
            s = (x @ k.T / math.sqrt(D)).view(g, c, P + L)
            if case["causal"]:
                place = P + L - c + torch.arange(c, device="cuda")
                s = s.masked_fill((torch.arange(P + L, device="cuda") > place[:, None])[None], -math.inf)
            z = torch.logsumexp(s, -1)
            lse[b, h * g:(h + 1) * g, :c] = z
            p = torch.exp(s - z[..., None])
            o[b, h * g:(h + 1) * g, :c] = (p.view(g * c, -1) @ v).view(g, c, D)
    return {"o": o, "lse": lse}
