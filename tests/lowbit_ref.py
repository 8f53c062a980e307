"""Plain float64 implementations of the narrow formats, from their definitions in include/engram.h (no GPU work at import).
Rows are float64 tensors on the CPU holding bf16 values."""
from __future__ import annotations

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _blocks(x):
    """[..., D] as [..., ceil(D/32), 32], zeros past D."""
    return torch.nn.functional.pad(x.double(), (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))


def _codes(blocks, top):
    """Scale codes [..., blocks]: floor(log2 amax) - top + 127 in [0, 254], 0 for zeros, 255 where a value is not finite."""
    amax = blocks.abs().amax(-1)
    e = torch.frexp(torch.where(torch.isfinite(amax) & (amax > 0), amax, 1.0)).exponent - 1 - top
    code = torch.where(amax > 0, (e + 127).clamp(0, 254), 0)
    return torch.where(torch.isfinite(blocks).all(-1), code, 255)


def scale_of(code):
    code = code.double()
    return torch.where(code == 255, torch.nan, torch.exp2(code - 127))


def mx4_quant(x):
    """(codes of the elements uint8 [n, K], scale codes uint8 [n, K/32]) of rows [n, K]."""
    b = _blocks(x)
    s = _codes(b, 2)
    y = torch.where((s == 255)[..., None], 0.0, b / torch.exp2(s.double() - 127)[..., None])
    grid = torch.tensor(E2M1, dtype=torch.float64)
    d = (y.abs()[..., None] - grid).abs()
    best = d.amin(-1, keepdim=True)
    near = d == best  # one or two neighbours: of two, the even code
    code = torch.where(near.sum(-1) == 1, near.int().argmax(-1), (near & (torch.arange(8) % 2 == 0)).int().argmax(-1))
    code = code + 8 * torch.signbit(y).long()
    return code.flatten(-2).to(torch.uint8), s.to(torch.uint8)


def mx4_values(code, s):
    grid = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)
    return (grid[code.long()].unflatten(-1, (-1, 32)) * scale_of(s)[..., None]).flatten(-2)


def pairs(code):
    """Element codes [n, K] as bytes [n, K/2], the even column in the low half."""
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpair(q):
    return torch.stack([q & 15, q >> 4], -1).flatten(-2)


def scales_laid_out(s):
    """Scale codes [n, K/32] in the MX scale layout [K/128, n up to a multiple of 4, 4] (padding rows 0)."""
    n, nb = s.shape
    out = torch.zeros((nb // 4, (n + 3) // 4 * 4, 4), dtype=torch.uint8)
    for r in range(n):
        out[:, r] = s[r].view(nb // 4, 4)
    return out


def scales_rows(laid, n):
    return laid[:, :n].permute(1, 0, 2).reshape(n, -1)


def weight_laid_out(code, s):
    """Element codes [N, K] and scale codes [N, K/32] in the weight layout, byte by byte from its formula."""
    N, K = code.shape
    G, S = (N + 63) // 64, K // 128
    pad = torch.zeros((G * 64, K), dtype=torch.uint8)
    pad[:N] = code
    ps = torch.zeros((G * 64, K // 32), dtype=torch.uint8)
    ps[:N] = s
    out = torch.zeros((G, S, 4352), dtype=torch.uint8)
    rows = 64 * torch.arange(G)[:, None]
    for j in range(4):
        for r in range(16):
            n = (rows + 16 * j + r)[:, 0]
            for c in range(4):
                cols = 128 * torch.arange(S) + 32 * c
                for b in range(16):
                    lo = pad[n][:, cols + 2 * b]
                    out[:, :, 1024 * j + 256 * c + 16 * r + b] = lo | (pad[n][:, cols + 2 * b + 1] << 4)
                out[:, :, 4096 + 64 * c + 4 * r + j] = ps[n][:, cols // 32]
    return out


def mx8_values(q, s):
    """Values of E4M3FN bytes [n, K] with scale codes [n, K/32]."""
    return (q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) * scale_of(s)[..., None]).flatten(-2)


def int8_quant(x):
    """(int8 of x's shape, scale codes uint8 [..., ceil(D/32)]) of rows [..., D]."""
    b = _blocks(x)
    s = _codes(b, 0)
    y = torch.where((s == 255)[..., None], 0.0, b * torch.exp2(133 - s.double())[..., None])
    q = torch.round(y).clamp(-127, 127)
    return q.flatten(-2)[..., :x.shape[-1]].to(torch.int8), s.to(torch.uint8)


def int8_values(q, s):
    unit = scale_of(s) / 64
    return q.double() * unit.repeat_interleave(32, -1)[..., :q.shape[-1]]
