"""The norm and rotation of heads and their gradients in float64, and attention
behind a shared prefix: what the GPU operators are compared with."""
import math

import torch


def angles(freq, axes, positions):
    """[B, S, pairs] from positions [axes, B, S]."""
    f = torch.tensor([float(x) for x in freq], dtype=torch.float64)
    a = torch.tensor([int(x) for x in axes], dtype=torch.long)
    return positions[a].permute(1, 2, 0).double() * f


def places(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, t, interleaved):
    """x [B, S, H, D] with its pairs turned by t [B, S, pairs]."""
    i, j = places(2 * t.shape[-1], interleaved)
    c, s = torch.cos(t)[:, :, None], torch.sin(t)[:, :, None]
    y = x.clone()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def norm(x, w, eps):
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def qk_rope(x, w, t, interleaved, eps):
    """Normed and rotated [B, S, H, D], float64."""
    return rotate(norm(x, w, eps), t, interleaved)


def qk_rope_bwd(dy, x, w, t, interleaved, eps):
    """(dx [B, S, H, D], dw [D] or None) for dy [B, S, H, D], by autograd of
    the definition."""
    x = x.clone().requires_grad_()
    leaf = None if w is None else w.clone().requires_grad_()
    y = rotate_graph(norm(x, leaf, eps), t, interleaved)
    y.backward(dy)
    return x.grad, None if w is None else leaf.grad


def rotate_graph(x, t, interleaved):
    """rotate() without assignments in place."""
    r = 2 * t.shape[-1]
    i, j = places(r, interleaved)
    c, s = torch.cos(t)[:, :, None], torch.sin(t)[:, :, None]
    a = x[..., i] * c - x[..., j] * s
    b = x[..., i] * s + x[..., j] * c
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else \
        torch.cat([a, b], -1)
    return torch.cat([y, x[..., r:]], -1)


def prefix(q, pk, pv, k, v, plen, lens, new, causal, scale):
    """O [B, Hq, Sq, D] and LSE in float64 (0 and -inf where nothing is seen);
    rows at or behind new[b] are NaN."""
    B, Hq, Sq, D = q.shape
    Hkv = k.shape[1]
    o = torch.full((B, Hq, Sq, D), math.nan, dtype=torch.float64)
    lse = torch.full((B, Hq, Sq), math.nan, dtype=torch.float64)
    for b in range(B):
        n, L = new[b], lens[b]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            keys = torch.cat([pk[g, :plen], k[b, g, :L]]).double()
            vals = torch.cat([pv[g, :plen], v[b, g, :L]]).double()
            for i in range(n):
                end = plen + (max(0, L - n + i + 1) if causal else L)
                if end == 0:
                    o[b, h, i], lse[b, h, i] = 0.0, -math.inf
                    continue
                s = keys[:end] @ q[b, h, i].double() * scale
                lse[b, h, i] = torch.logsumexp(s, 0)
                o[b, h, i] = torch.exp(s - lse[b, h, i]) @ vals[:end]
    return o, lse
