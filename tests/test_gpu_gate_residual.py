"""engram_gate_residual over its forms: a call's rows are those of calls on parts of them, bit for bit, wherever the long form
takes over, and out may be x."""
import pytest
import torch

import gram_hash_embedding_amd as g

pytestmark = pytest.mark.gpu


def _inputs(T, hc, dim, seed, ld=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, hc, dim), generator=gen, device="cuda").to(torch.bfloat16)
    value = torch.randn((T, ld or dim), generator=gen, device="cuda").to(torch.bfloat16)[:, :dim]
    dot = torch.randn((T, hc), generator=gen, device="cuda")
    mask = torch.rand((T,), generator=gen, device="cuda") > 0.3
    return x, value, dot, mask


# 2^22 pieces of 16 bytes are the last that the short form takes
@pytest.mark.parametrize("T,hc,dim,ld", [(4096, 4, 2048, None), (4097, 4, 2048, None), (70001, 3, 168, 176), (20011, 8, 256, None),
                                         (600000, 1, 56, None), (1100001, 4, 8, 24)])
def test_long_calls_match_their_parts(T, hc, dim, ld):
    x, value, dot, mask = _inputs(T, hc, dim, T, ld)
    out = g.engram_gate_residual(x, value, dot, mask)
    step = max(1, (1 << 21) // (hc * dim // 8) - 3)
    for a in range(0, T, step):
        b = min(T, a + step)
        assert torch.equal(out[a:b], g.engram_gate_residual(x[a:b], value[a:b], dot[a:b], mask[a:b])), (a, b)
    inplace = x.clone()
    assert torch.equal(g.engram_gate_residual(inplace, value, dot, mask, out=inplace), out)


def test_long_calls_against_the_formula():
    """x + gate * value in 64 bits: one bf16 rounding of the result, two float32 ones (of the product and the sum) and the
    float32 gate, whose relative error is below 2^-20."""
    T, hc, dim = 5000, 4, 1848
    x, value, dot, mask = _inputs(T, hc, dim, 5)
    out = g.engram_gate_residual(x, value, dot, mask).double()
    d = dot.double()
    gate = torch.sigmoid(torch.sign(d) * d.abs().clamp(min=1e-6).sqrt()) * mask[:, None]
    part = gate[..., None] * value.double()[:, None]
    want = x.double() + part
    assert ((out - want).abs() <= want.abs() * 2.0 ** -8 + (part.abs() + want.abs()) * 2.0 ** -19 + 1e-38).all()


def test_more_pieces_than_32_bits_count():
    """2^32 pieces and more: the rows at the start, on either side of the 2^32nd and at the end."""
    hc, dim = 64, 128
    T = (1 << 32) // (hc * dim // 8) + 5000
    if torch.cuda.mem_get_info()[0] < 5 * T * hc * dim // 2:
        pytest.skip("needs 90 GB of GPU memory")
    x = torch.zeros((T, hc, dim), dtype=torch.bfloat16, device="cuda")
    value = torch.zeros((T, dim), dtype=torch.bfloat16, device="cuda")
    dot = torch.zeros((T, hc), device="cuda")
    mask = torch.ones((T,), dtype=torch.bool, device="cuda")
    n, want = 300, {}
    for at in (0, (1 << 31) // 1024 - 150, (1 << 32) // 1024 - 150, T - n):
        rows = slice(at, at + n)
        x[rows], value[rows], dot[rows], mask[rows] = _inputs(n, hc, dim, at % 1000)
        want[at] = g.engram_gate_residual(x[rows].clone(), value[rows], dot[rows], mask[rows])
    g.engram_gate_residual(x, value, dot, mask, out=x)
    for at, w in want.items():
        assert torch.equal(x[at:at + n], w), at
    assert not x[n:2 * n].any()
