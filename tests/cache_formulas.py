"""Rotary positions, the paged cache and its attention in 64 bits, for the tests."""
import math

import torch


def turn(x, positions, frequencies, interleaved=False, scale=1.0, inverse=False):
    """x [T, N, D] with the first 2 * len(frequencies) elements of every head rotated."""
    R = 2 * len(frequencies)
    x = x.double()
    p = positions.double()[:, None] * torch.as_tensor(frequencies, dtype=torch.float64, device=x.device)[None]
    c, s = scale * torch.cos(p)[:, None], scale * torch.sin(p)[:, None] * (-1 if inverse else 1)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2], y[..., R // 2: R] = a * c - b * s, a * s + b * c
    return y


def paged(pages, page, heads, dim, fp8, device, generator, order="page,row,head", scale=1.0):
    """A cache of random values: (k, v, k_scale, v_scale), [pages, page, heads, dim] of some order in memory."""
    def one(*shape):
        if order == "page,head,row":
            shape = (shape[0], shape[2], shape[1], *shape[3:])
        t = torch.randn(*shape, generator=generator, device=device) * scale
        return t.transpose(1, 2) if order == "page,head,row" else t
    out = []
    for _ in range(2):
        t = one(pages, page, heads, dim)
        if fp8:
            s = t.abs().amax(-1) / 448
            q = (t / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
            out.append((q, s))
        else:
            out.append((t.to(torch.bfloat16), None))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def values(cache, scale):
    """The cache's values in 64 bits, [pages, page, heads, dim]."""
    return cache.double() if scale is None else cache.double() * scale.double().unsqueeze(-1)


def attend(q, k, v, table, lengths, scale=None, window=0):
    """(o [B, QH, D], lse [B, QH]) over the rows k, v [pages, page, KH, D] (64 bits) of each sequence."""
    B, QH, D = q.shape
    page, KH = k.shape[1], k.shape[2]
    o = torch.zeros(B, QH, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, QH), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lengths.tolist()):
        if n <= 0:
            continue
        rows = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        at = table[b, rows // page].long()
        kk, vv = k[at, rows % page], v[at, rows % page]
        s = torch.einsum("hgd,thd->hgt", q[b].double().view(KH, QH // KH, D), kk) * (D ** -0.5 if scale is None else scale)
        o[b] = torch.einsum("hgt,thd->hgd", torch.softmax(s, 2), vv).reshape(QH, D)
        lse[b] = torch.logsumexp(s, 2).reshape(QH)
    return o, lse
