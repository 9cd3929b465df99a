"""Plain 64-bit form of the query/key norm with rotation and of its gradient
(torch, from the definition), shared by their tests."""
from __future__ import annotations

import torch


def turns(positions, freqs):
    """cos and sin [T, 1, rot / 2]."""
    a = positions.double()[:, None, None] * freqs.double()
    return torch.cos(a), torch.sin(a)


def pairs(dim: int, rot: int, neighbours: bool):
    """Columns of the pairs' first and second members."""
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)


def turn(v, cos, sin, neighbours: bool):
    """The rotation of the last dimension's first columns."""
    i, j = (t.to(v.device) for t in pairs(v.shape[-1], 2 * cos.shape[-1], neighbours))
    out = v.clone()
    out[..., i] = v[..., i] * cos - v[..., j] * sin
    out[..., j] = v[..., j] * cos + v[..., i] * sin
    return out


def other(v, rot: int, neighbours: bool):
    """The other member of each column's pair (0 where it has none)."""
    i, j = (t.to(v.device) for t in pairs(v.shape[-1], rot, neighbours))
    out = torch.zeros_like(v)
    out[..., i], out[..., j] = v[..., j], v[..., i]
    return out


def forward(x, w, positions, freqs, eps, neighbours):
    """x [T, heads, dim] in float64."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return turn(x * r * w, *turns(positions, freqs), neighbours)


def backward(x, w, positions, freqs, eps, neighbours, g):
    """(dx, dw)"""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    cos, sin = turns(positions, freqs)
    m = turn(g, cos, -sin, neighbours)
    gw, n = m * w, x * r
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (m * n).sum((0, 1))
