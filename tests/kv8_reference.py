"""The 8-bit cache operators in float64 on the CPU, from their definitions,
without the package's code; and the bounds their GPU results must keep."""
import math

import torch

F8 = torch.float8_e4m3fn


def rng(seed):
    return torch.Generator().manual_seed(seed)


def decode(codes):
    """E4M3 codes (uint8) as float64: sign, 4-bit exponent of bias 7, 3-bit
    mantissa; S.1111.111 is NaN."""
    c = codes.to(torch.int64)
    sign = 1.0 - 2.0 * (c >> 7).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, (e - 7).double()),
                    m / 8 * 2.0 ** -6)
    return torch.where((c & 127) == 127, torch.nan, sign * x)


_ALL = torch.arange(256, dtype=torch.uint8)
_VAL = decode(_ALL)
_POS = _VAL[:127]  # 0 .. 448, ascending


def encode(x):
    """float64 -> E4M3 codes: nearest, ties to the even code, saturating."""
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(_POS, a.nan_to_num(0.0).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = pick | (torch.signbit(x).long() << 7)
    return torch.where(x.isnan(), 127, code).to(torch.uint8)


def tight(amax):
    """Smallest 2^e >= amax / 448, e >= -126 (a python float)."""
    if amax == 0:
        return 2.0 ** -126
    m, e = math.frexp(amax / 448.0)
    return math.ldexp(1.0, max(e - (m == 0.5), -126))


class Cache:
    """Codes (uint8), scales (float64) and lengths on the CPU."""

    def __init__(self, B, H, cap, D, block):
        nblk = -(-cap // block)
        self.B, self.H, self.cap, self.D, self.block = B, H, cap, D, block
        self.code = {n: torch.full((B, H, cap, D), 0x7F, dtype=torch.uint8)
                     for n in "kv"}
        self.scale = {n: torch.full((B, H, nblk), math.inf,
                                    dtype=torch.float64) for n in "kv"}
        self.lens = [0] * B

    def to(self, device):
        c = Cache(self.B, self.H, 1, self.D, self.block)
        c.cap, c.lens = self.cap, list(self.lens)
        c.code = {n: t.to(device) for n, t in self.code.items()}
        c.scale = {n: t.to(device) for n, t in self.scale.items()}
        return c

    def clone(self):
        c = Cache(self.B, self.H, self.cap, self.D, self.block)
        c.code = {n: t.clone() for n, t in self.code.items()}
        c.scale = {n: t.clone() for n, t in self.scale.items()}
        c.lens = list(self.lens)
        return c

    def values(self, n, b, h):
        L = self.lens[b]
        s = self.scale[n][b, h].repeat_interleave(self.block)[:L]
        return decode(self.code[n][b, h, :L]) * s[:, None]

    def append(self, k, v, new=None):
        """k, v [B, H, Sq, D]; lens already counts the new tokens."""
        for n, x in (("k", k), ("v", v)):
            x = x.double()
            for b in range(self.B):
                cnt = x.shape[2] if new is None else new[b]
                start = self.lens[b] - cnt
                for h in range(self.H):
                    i = 0
                    while i < cnt:
                        blk = (start + i) // self.block
                        c = min(cnt - i, (blk + 1) * self.block - start - i)
                        part = x[b, h, i:i + c]
                        fin = part[part.isfinite()].abs()
                        amax = float(fin.max()) if fin.numel() else 0.0
                        s = tight(amax)
                        t0 = blk * self.block
                        if t0 < start:
                            old = float(self.scale[n][b, h, blk])
                            if amax <= 448.0 * old:
                                s = old
                            else:
                                held = self.code[n][b, h, t0:start]
                                self.code[n][b, h, t0:start] = encode(
                                    decode(held) * old / s)
                        self.scale[n][b, h, blk] = s
                        self.code[n][b, h, start + i:start + i + c] = encode(
                            part / s)
                        i += c

    def evict(self, weights, keep, recent, room):
        """(cache of capacity `room`, weights, indices)."""
        out = Cache(self.B, self.H, room, self.D, self.block)
        ow = torch.zeros(self.B, self.H, room)
        idx = torch.full((self.B, self.H, keep), -1, dtype=torch.int32)
        for b in range(self.B):
            L = self.lens[b]
            m = min(L, keep)
            out.lens[b] = m
            for h in range(self.H):
                if L <= keep:
                    places = list(range(L))
                else:
                    w = weights[b, h].tolist()
                    key = lambda j: (math.isnan(w[j]),  # noqa: E731
                                     0.0 if math.isnan(w[j]) else -w[j], j)
                    best = sorted(range(L - recent), key=key)[:keep - recent]
                    places = sorted(best) + list(range(L - recent, L))
                at = torch.tensor(places, dtype=torch.long)
                idx[b, h, :m] = at.int()
                ow[b, h, :m] = weights[b, h, at]
                for n in "kv":
                    if L <= keep:
                        nb = -(-L // self.block)
                        out.code[n][b, h, :L] = self.code[n][b, h, :L]
                        out.scale[n][b, h, :nb] = self.scale[n][b, h, :nb]
                        continue
                    x = self.values(n, b, h)[at]
                    for t in range(0, m, self.block):
                        part = x[t:t + self.block]
                        s = tight(float(part.abs().max()))
                        out.scale[n][b, h, t // self.block] = s
                        out.code[n][b, h, t:t + len(part)] = encode(part / s)
        return out, ow, idx


def attention(cache, q, scale, causal, new=None):
    """Lists over (b, h, row) results of the definition, float64: O, LSE,
    weights [B, H, cap], and bounds of the fp32 kernels' errors."""
    B, Hq, Sq, D = q.shape
    g = Hq // cache.H
    qd = q.double()
    new_ = dict(dtype=torch.float64, device=q.device)
    o = torch.zeros(B, Hq, Sq, D, **new_)
    lse = torch.full((B, Hq, Sq), -math.inf, **new_)
    w = torch.zeros(B, cache.H, cache.cap, **new_)
    tol_o, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    tol_w = torch.zeros_like(w)
    eps = torch.finfo(q.dtype).eps / 2
    for b in range(B):
        L = cache.lens[b]
        cnt = Sq if new is None else new[b]
        if L == 0 or cnt == 0:
            continue
        for h in range(Hq):
            k, v = (cache.values(n, b, h // g) for n in "kv")
            s = scale * (qd[b, h, :cnt] @ k.T)
            end = torch.full((cnt,), L, device=q.device)
            if causal:
                end = torch.arange(L - cnt + 1, L + 1, device=q.device)
            see = torch.arange(L, device=q.device)[None] < end[:, None]
            s = s.masked_fill(~see, -math.inf)
            lse[b, h, :cnt] = torch.logsumexp(s, 1)
            any_ = see.any(1)
            p = torch.where(any_[:, None], torch.exp(
                s - torch.where(any_, lse[b, h, :cnt], 0.0)[:, None]), 0.0)
            o[b, h, :cnt] = p @ v
            w[b, h // g, :L] += p.sum(0)
            # A score is a sum of D products and two or three factors, each
            # step off by one fp32 ulp (2^-23) at most, so off by
            # (D + 8) 2^-23 sum |q k| scale; 2^-18 covers exp2, log2 and the
            # sums over the keys (chains of a few hundred 2^-24 roundings).
            mag = abs(scale) * (qd[b, h, :cnt].abs() @ k.abs().T)
            mag = mag.masked_fill(~see, 0.0)
            rel = ((D + 8) * 2.0 ** -23 * mag).amax(1) + 2.0 ** -18
            tol_lse[b, h, :cnt] = rel + 2.0 ** -23 * torch.where(
                any_, lse[b, h, :cnt].abs(), 0.0)
            # Weights p carry twice that (their own score and the LSE); the
            # output also the fp16 rounding of p (2^-11), its fp32 sums over
            # the keys (2^-12) and its own rounding.
            spread = p @ v.abs()
            tol_o[b, h, :cnt] = (spread * (2 * rel[:, None] + 2.0 ** -11
                                           + 2.0 ** -12)
                                 + eps * o[b, h, :cnt].abs() + 1e-30)
            if q.dtype == torch.float16:  # subnormal outputs
                tol_o[b, h, :cnt] += 2.0 ** -25
            tol_w[b, h // g, :L] += (p * 2 * rel[:, None]).sum(0) + 2.0 ** -40
    return o, lse, w, tol_o, tol_lse, tol_w


def filled(B, H, cap, D, block, lens, seed, factor=1.0):
    """A cache of normal tokens appended at once; behind the lengths lie NaN
    codes and infinite scales."""
    g = rng(seed)
    c = Cache(B, H, cap, D, block)
    c.lens = list(lens)
    most = max(max(lens), 1)
    x = [torch.randn(B, H, most, D, generator=g)
         * torch.exp(0.5 * torch.randn(1, H, 1, D, generator=g)) * factor
         for _ in range(2)]
    c.append(x[0].half(), x[1].half(), new=list(lens))
    return c
