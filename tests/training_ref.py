"""Plain float64 implementations of the training operators, from their definitions in include/engram.h, with the
magnitudes that bound a float32 computation's error (no GPU work at import)."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24   # unit roundoff of float32
U16 = 2.0 ** -8    # twice bf16's unit roundoff: one rounding, and a neighbour where float32 error moves a tie


def embed_grad(ids, up, R, row_start, scale):
    """(sum [R, D], sum of magnitudes [R, D], the most positions on one row), float64."""
    ids = ids.reshape(-1).long() - row_start
    up = up.reshape(ids.numel(), up.shape[-1]).double()
    keep = torch.nonzero((ids >= 0) & (ids < R)).flatten()
    out = torch.zeros((R, up.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    out.index_add_(0, ids[keep], up[keep] * scale)
    mag.index_add_(0, ids[keep], (up[keep] * scale).abs())
    m = int(torch.bincount(ids[keep], minlength=1).max()) if keep.numel() else 0
    return out, mag, m


def sum_tolerance(ref, mag, m, bf16):
    """m float32 additions in any order and one product: (m + 2) U32 of the magnitudes; then one rounding."""
    return (m + 2) * U32 * mag + (U16 if bf16 else 2 * U32) * ref.abs() + 1e-40


def gate_backward(x, kv, q, k, eps, dot, dout, mask=None):
    """dict of dx, dkv, dq, dk and, per output, the magnitude its float32 error is measured against (dx_mag, ...)."""
    x, kv, q, k, d, up = (t.double() for t in (x, kv, q, k, dot, dout))
    T, hc, dim = x.shape
    kv = kv[:, :(hc + 1) * dim]
    if mask is not None:  # a masked token takes no part, whatever it holds
        m = mask.bool().reshape(T)
        x, kv, d = torch.where(m[:, None, None], x, 1.0), torch.where(m[:, None], kv, 1.0), torch.where(m[:, None], d, 1.0)
    else:
        m = torch.ones(T, dtype=torch.bool)
    live = m.double()[:, None]
    key, v = kv[:, :hc * dim].reshape(T, hc, dim), kv[:, hc * dim:]
    w = q * k
    rh = (x.square().mean(-1) + eps).rsqrt()
    rk = (key.square().mean(-1) + eps).rsqrt()
    s = rh * rk * dim ** -0.5
    z = d.abs().clamp(min=1e-6).sqrt()
    g = torch.sigmoid(torch.copysign(z, d)) * live
    slope = torch.where(dot.double().abs() < float(torch.tensor(1e-6, dtype=torch.float32)), 0.0, g * (1 - g) / (2 * z)) * live
    upl = torch.where(m[:, None, None], up, 0.0)
    dd = (upl * v[:, None]).sum(-1) * slope
    dd_mag = (upl * v[:, None]).abs().sum(-1) * slope
    e, em = dd[..., None], dd_mag[..., None]
    a, b = s[..., None] * w, (d * rh * rh / dim)[..., None]
    c = (d * rk * rk / dim)[..., None]
    dx = up + torch.where(m[:, None, None], e * (a * key - b * x), 0.0)
    dkey = torch.where(m[:, None, None], e * (a * x - c * key), 0.0)
    dv = (g[..., None] * upl).sum(1)
    both = e * s[..., None] * x * key
    both = torch.where(m[:, None, None], both, 0.0).sum(0)
    both_mag = torch.where(m[:, None, None], em * s[..., None] * (x * key).abs(), 0.0).sum(0)
    return dict(
        dx=dx, dx_mag=up.abs() + em * ((a * key).abs() + (b * x).abs()),
        dkv=torch.cat([dkey.reshape(T, hc * dim), dv], 1),
        dkv_mag=torch.cat([(em * ((a * x).abs() + (c * key).abs())).reshape(T, hc * dim), (g[..., None] * upl.abs()).sum(1)], 1),
        dq=both * k, dq_mag=both_mag * k.abs(), dk=both * q, dk_mag=both_mag * q.abs())


def gate_forward(x, kv, q, k, eps, mask=None):
    """(out, dot) of engram_gate_output in float64, no rounding of the result."""
    x, kv, q, k = (t.double() for t in (x, kv, q, k))
    T, hc, dim = x.shape
    key, v = kv[:, :hc * dim].reshape(T, hc, dim), kv[:, hc * dim:(hc + 1) * dim]
    rstd = (x.square().mean(-1) + eps).rsqrt() * (key.square().mean(-1) + eps).rsqrt()
    dot = (x * (q * k) * key).sum(-1) * rstd * dim ** -0.5
    gate = torch.sigmoid(torch.copysign(dot.abs().clamp(min=1e-6).sqrt(), dot))
    if mask is not None:
        gate = gate * mask.double()[:, None]
    return x + gate[..., None] * v[:, None], dot
