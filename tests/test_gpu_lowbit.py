"""The 4-bit weights and the 8-bit checkpoints on the GPU, against their plain implementations in 64 bits: quantised bytes and
products in whole numbers exactly, everything else within tolerances derived from the roundings of its float32 sums."""
import zlib

import pytest
import torch

import gram_hash_embedding_amd as g
from tests import lowbit_ref as ref
from tests import training_ref as tref

pytestmark = pytest.mark.gpu
U32, U16 = tref.U32, tref.U16
EPS = 1e-20


def _bf16(gen, shape, std=1.0, spread=0):
    x = torch.randn(shape, generator=gen) * std
    if spread:
        x = x * torch.exp2(torch.randint(-spread, spread, (*shape[:-1], 1), generator=gen).float())
    return x.to(torch.bfloat16)


def _gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _patterns(cols):
    """Every bf16 pattern, in rows of `cols`."""
    return torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(-1, cols)


# ---- quantisation ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("rows,K", [(1, 128), (5, 256), (257, 1536), (1000, 640), (3, 6144)])
def test_mx4_quant(gpu_device, rows, K):
    x = _bf16(_gen("q4", rows, K), (rows, K), spread=100)
    x[0, :32] = 0
    x[0, 5] = -0.0
    x[0, 32:64] = 7.75 * 2.0 ** -20  # saturates
    x[-1, 64:96] = 2.0 ** -133       # bf16's smallest subnormal: below the scales' range
    x[-1, 96:128] = torch.tensor([0.25 * k for k in range(32)]).to(torch.bfloat16)  # the ties
    x[rows // 2, 17] = 2.0 ** 127
    q, s = g.engram_mx4_quant(x.to(gpu_device))
    code, sc = ref.mx4_quant(x.double())
    assert torch.equal(ref.scales_rows(s.cpu(), rows), sc)
    assert torch.equal(q.cpu(), ref.pairs(code))


def test_mx4_quant_of_every_pattern(gpu_device):
    """Every bf16 value next to its like (a block's scale fits them), next to 1.0 (most round to zero or saturate), infinities
    and NaN among them."""
    x = _patterns(128)
    for y in (x, torch.where(torch.arange(128) % 32 == 0, torch.ones((), dtype=torch.bfloat16), x)):
        q, s = g.engram_mx4_quant(y.contiguous().to(gpu_device))
        code, sc = ref.mx4_quant(y.double())
        assert torch.equal(ref.scales_rows(s.cpu(), 512), sc)
        assert torch.equal(q.cpu(), ref.pairs(code))


@pytest.mark.parametrize("N,K", [(8, 128), (64, 128), (72, 256), (200, 640), (1280, 1536)])
def test_pack_weight(gpu_device, N, K):
    gen = _gen("pack", N, K)
    code = torch.randint(0, 16, (N, K), dtype=torch.uint8, generator=gen)
    s = torch.randint(0, 256, (N, K // 32), dtype=torch.uint8, generator=gen)
    w = g.engram_mx4_pack_weight(ref.pairs(code).to(gpu_device), ref.scales_laid_out(s).to(gpu_device))
    assert torch.equal(w.cpu(), ref.weight_laid_out(code, s))


@pytest.mark.parametrize("shape", [(1, 8), (3, 32), (7, 40), (33, 1000), (5, 3, 264), (257, 5120), (1, 65536)])
def test_ckpt(gpu_device, shape):
    x = _bf16(_gen("ck", shape), shape, spread=100)
    flat = x.view(-1, shape[-1])
    flat[0, :8] = 0
    flat[0, 3] = -0.0
    flat[-1, -8:] = 2.0 ** -133
    flat[0, -1] = 127.5
    q, s = g.engram_ckpt_save(x.to(gpu_device))
    qr, sr = ref.int8_quant(x.double())
    assert torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)
    back = g.engram_ckpt_load(q, s).cpu()
    assert back.shape == x.shape and torch.equal(back.double(), ref.int8_values(qr, sr))


def test_ckpt_of_every_pattern(gpu_device):
    x = _patterns(128)
    for y in (x, torch.where(torch.arange(128) % 32 == 0, torch.ones((), dtype=torch.bfloat16), x)):
        q, s = g.engram_ckpt_save(y.contiguous().to(gpu_device))
        qr, sr = ref.int8_quant(y.double())
        assert torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)
        assert torch.equal(g.engram_ckpt_load(q, s).cpu().double().nan_to_num(7e77), ref.int8_values(qr, sr).nan_to_num(7e77))


# ---- products -------------------------------------------------------------------------------------------------------
def _weights(gen, N, K, dev, whole=False):
    """(packed weights on the GPU, their values in 64 bits)."""
    code = torch.randint(0, 16, (N, K), dtype=torch.uint8, generator=gen)
    s = torch.randint(126, 129, (N, K // 32), dtype=torch.uint8, generator=gen) if whole else torch.randint(
        118, 124, (N, K // 32), dtype=torch.uint8, generator=gen)
    w = g.engram_mx4_pack_weight(ref.pairs(code).to(dev), ref.scales_laid_out(s).to(dev))
    return w, ref.mx4_values(code, s)


def _rows(gen, T, K, bits, dev, whole=False):
    """(rows on the GPU, their scales, their values in 64 bits)."""
    s = torch.randint(126, 129, (T, K // 32), dtype=torch.uint8, generator=gen) if whole else torch.randint(
        122, 130, (T, K // 32), dtype=torch.uint8, generator=gen)
    if bits == 4:
        code = torch.randint(0, 16, (T, K), dtype=torch.uint8, generator=gen)
        q, v = ref.pairs(code), ref.mx4_values(code, s)
    elif whole:  # -4 .. 4 in E4M3
        q = torch.randint(-4, 5, (T, K), generator=gen).float().to(torch.float8_e4m3fn).view(torch.uint8)
        v = ref.mx8_values(q, s)
    else:
        q = torch.randn((T, K), generator=gen).mul(40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = ref.mx8_values(q, s)
    return q.to(dev), ref.scales_laid_out(s).to(dev), v


# every count of tokens at which the forms of the kernels hand over, one off either side; steps of 128 columns from one on, odd
# counts; columns that end inside a record
PRODUCTS = [(1, 128, 8), (2, 256, 64), (15, 384, 72), (16, 640, 136), (17, 1536, 264), (31, 128, 520), (32, 1536, 64),
            (33, 256, 1280), (63, 896, 200), (64, 1536, 1280), (65, 128, 264), (100, 384, 2056), (127, 512, 136),
            (128, 1536, 640), (129, 640, 520), (255, 256, 264), (256, 1536, 5120), (257, 384, 1288), (300, 6144, 256),
            (511, 128, 1000), (700, 1536, 2560), (1025, 768, 1032), (2100, 256, 8200)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_product_in_whole_numbers(gpu_device, T, K, N, bits):
    """Elements that are multiples of a quarter up to 6 x 6 x 4 x 4 in magnitude: sums of up to 6,144 products stay below 2^22
    quarters, exact in float32 in any order, so the result is the exact sum rounded once."""
    gen = _gen("whole", T, K, N, bits)
    w, wv = _weights(gen, N, K, gpu_device, whole=True)
    a, s, av = _rows(gen, T, K, bits, gpu_device, whole=True)
    want = (av.to(gpu_device) @ wv.t().contiguous().to(gpu_device)).to(torch.float32).to(torch.bfloat16)
    got = g.engram_wkv_mx4(a, s, w, nout=N)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(1, 1536, 25600), (77, 1536, 2560), (400, 6144, 520), (1030, 1536, 5128)])
def test_product(gpu_device, T, K, N, bits):
    """One rounding to bf16 of half a step, and the matrix core's sums: it keeps its products less exactly than float32 sums
    would, by up to 2^-12 of the sum of their magnitudes (what the 8-bit projection is held to)."""
    gen = _gen("real", T, K, N, bits)
    w, wv = _weights(gen, N, K, gpu_device)
    a, s, av = _rows(gen, T, K, bits, gpu_device)
    av, wt = av.to(gpu_device), wv.t().contiguous().to(gpu_device)
    want, mag = av @ wt, av.abs() @ wt.abs()
    got = g.engram_wkv_mx4(a, s, w, nout=N).double()
    assert ((got - want).abs() <= U16 * want.abs() + 2.0 ** -12 * mag).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_do_not_depend_on_the_call(gpu_device, bits):
    """The same rows alone, in small calls and in a large one: the same bits from every form of the kernel."""
    gen = _gen("same", bits)
    T, K, N = 1100, 1536, 1416
    w, _ = _weights(gen, N, K, gpu_device)
    a, s, _ = _rows(gen, T, K, bits, gpu_device)
    whole = g.engram_wkv_mx4(a, s, w, nout=N)
    sr = ref.scales_rows(s.cpu(), T)
    for t0, n in ((0, 1), (5, 16), (100, 20), (7, 33), (64, 64), (300, 100), (1, 128), (500, 256), (40, 300), (3, 700)):
        part = g.engram_wkv_mx4(a[t0:t0 + n].contiguous(), ref.scales_laid_out(sr[t0:t0 + n]).to(gpu_device), w, nout=N)
        assert torch.equal(part, whole[t0:t0 + n]), (t0, n)


@pytest.mark.parametrize("T", [3, 300])
def test_extreme_scales(gpu_device, T):
    """Scales at both ends whose products are ordinary; a NaN scale reaches its own row, or its own column, and no other."""
    gen = _gen("extreme", T)
    K, N = 512, 264
    code = torch.randint(0, 16, (T, K), dtype=torch.uint8, generator=gen)
    wcode = torch.randint(0, 16, (N, K), dtype=torch.uint8, generator=gen)
    c = torch.randint(10, 245, (K // 32,), generator=gen)
    sa = c.expand(T, -1).to(torch.uint8).contiguous()
    sw = (254 - c + torch.randint(-1, 2, (N, K // 32), generator=gen)).to(torch.uint8)
    av, wv = ref.mx4_values(code, sa), ref.mx4_values(wcode, sw)
    want = (av @ wv.t()).to(torch.float32).to(torch.bfloat16)
    sa[T // 2, 5], sw[33, 9] = 255, 255
    w = g.engram_mx4_pack_weight(ref.pairs(wcode).to(gpu_device), ref.scales_laid_out(sw).to(gpu_device))
    got = g.engram_wkv_mx4(ref.pairs(code).to(gpu_device), ref.scales_laid_out(sa).to(gpu_device), w, nout=N).cpu()
    nan = torch.zeros((T, N), dtype=torch.bool)
    nan[T // 2], nan[:, 33] = True, True
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], want[~nan])


def _gate_inputs(gen, T, hc, dim, dev):
    x = _bf16(gen, (T, hc, dim)).to(dev)
    q, k = (1 + _bf16(gen, (hc, dim), 0.1)).to(dev), (1 + _bf16(gen, (hc, dim), 0.1)).to(dev)
    return x, q, k


def _dot_tolerance(x, key, q, k):
    """(dot, tolerance) in 64 bits: the sums of dim terms in float32, the two means' relative errors, and a few roundings."""
    x, key, w = x.double(), key.double(), q.double() * k.double()
    dim = x.shape[-1]
    scale = ((x.square().mean(-1) + EPS) * (key.square().mean(-1) + EPS) * dim).rsqrt()
    dot, mag = (x * w * key).sum(-1) * scale, (x * w * key).abs().sum(-1) * scale
    return dot, 2 * (dim + 16) * U32 * mag


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,hc,dim", [(1, 128, 1, 256), (16, 256, 4, 256), (37, 1536, 2, 512), (64, 384, 3, 256),
                                        (65, 640, 4, 768), (129, 128, 1, 1024), (256, 1536, 4, 512), (300, 384, 4, 5120),
                                        (1000, 1536, 2, 2560), (515, 6144, 1, 256)])
def test_gate(gpu_device, T, K, hc, dim, bits):
    gen = _gen("gate", T, K, hc, dim, bits)
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    a, s, _ = _rows(gen, T, K, bits, gpu_device)
    x, q, k = _gate_inputs(gen, T, hc, dim, gpu_device)
    kv = g.engram_wkv_mx4(a, s, w)
    value = torch.full((T, dim + 24), 3.0, dtype=torch.bfloat16, device=gpu_device)
    got, dot = g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS, value=value)
    assert got is value and torch.equal(value[:, :dim], kv[:, hc * dim:]) and (value[:, dim:] == 3).all()
    want, tol = _dot_tolerance(x, kv[:, :hc * dim].view(T, hc, dim), q, k)
    assert ((dot.double() - want).abs() <= tol).all()
    again, dot2 = g.engram_wkv_mx4_gate(a, s, w, x.view(T, 1, hc, dim), q, k, EPS)
    assert torch.equal(again, kv[:, hc * dim:]) and torch.equal(dot2, dot)


def test_empty_calls(gpu_device):
    gen = _gen("empty")
    w, _ = _weights(gen, 1280, 384, gpu_device)
    u8, bf = torch.uint8, torch.bfloat16
    mk = lambda shape, dt: torch.empty(shape, dtype=dt, device=gpu_device)  # noqa: E731
    assert g.engram_wkv_mx4(mk((0, 384), u8), mk((3, 0, 4), u8), w).shape == (0, 1280)
    x, q, k = _gate_inputs(gen, 0, 4, 256, gpu_device)
    value, dot = g.engram_wkv_mx4_gate(mk((0, 192), u8), mk((3, 0, 4), u8), w, x, q, k, EPS)
    assert value.shape == (0, 256) and dot.shape == (0, 4)
    qq, ss = g.engram_mx4_quant(mk((0, 384), bf))
    assert qq.shape == (0, 192) and ss.shape == (3, 0, 4)
    qq, ss = g.engram_ckpt_save(mk((0, 40), bf))
    assert g.engram_ckpt_load(qq, ss).shape == (0, 40)
    out, dot, c = g.engram_gate_output_ckpt(x, mk((0, 1280), bf), q, k, EPS)
    assert out.shape == x.shape
    dx, dkv, dq, dk = g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, x)
    assert dx.shape == x.shape and (dq == 0).all() and (dk == 0).all()


# ---- checkpoints in the gate's training step --------------------------------------------------------------------------
GATES = [(1, 1, 8), (7, 4, 256), (33, 3, 264), (20, 2, 40), (9, 64, 16), (300, 4, 1024), (65, 1, 5120), (40, 4, 5120),
         (30, 2, 6152), (21, 4, 8192), (600, 4, 2056), (5, 3, 2048), (300, 4, 512), (300, 2, 3080)]


def _gate_case(T, hc, dim, dev, extra=0, masked=True):
    gen = _gen("ckpt", T, hc, dim)
    x, q, k = _gate_inputs(gen, T, hc, dim, dev)
    kv = _bf16(gen, (T, (hc + 1) * dim + extra), 0.5).to(dev)
    mask = (torch.rand(T, generator=gen) < 0.7).to(dev) if masked else None
    dout = _bf16(gen, (T, hc, dim), 1e-2).to(dev)
    return x, kv, q, k, mask, dout


@pytest.mark.parametrize("T,hc,dim", GATES)
def test_gate_output_ckpt(gpu_device, T, hc, dim):
    x, kv, q, k, mask, _ = _gate_case(T, hc, dim, gpu_device, extra=16)
    out, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    rows = kv[:, :(hc + 1) * dim].contiguous().view(T, hc + 1, dim)
    for got, want in zip(c, (*g.engram_ckpt_save(x), *g.engram_ckpt_save(rows))):
        assert torch.equal(got, want)
    want, tol = _dot_tolerance(x, rows[:, :hc], q, k)
    assert ((dot.double() - want).abs() <= tol).all()
    # the output from the dot that was written: the gate in float32 (a few roundings of at most 1), the product, the sum, bf16
    gate = torch.sigmoid(torch.copysign(dot.double().abs().clamp(min=1e-6).sqrt(), dot.double()))[..., None]
    if mask is not None:
        gate = gate * mask[:, None, None]
    res = x.double() + gate * rows[:, hc:].double()
    tol = U16 * res.abs() + 16 * U32 * (x.double().abs() + rows[:, hc:].double().abs())
    assert ((out.double() - res).abs() <= tol).all()
    if mask is not None:
        assert torch.equal(out[~mask], x[~mask])


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,hc,dim", GATES)
def test_gate_backward_ckpt(gpu_device, T, hc, dim, masked):
    """The gradient from checkpoints is that of the values they stand for, bit for bit, and within the bound of the formula in 64
    bits on them."""
    x, kv, q, k, mask, dout = _gate_case(T, hc, dim, gpu_device, masked=masked)
    _, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    got = g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, mask)
    xl, kvl = g.engram_ckpt_load(c.x, c.x_scale), g.engram_ckpt_load(c.kv, c.kv_scale).view(T, -1)
    for a, b in zip(got, g.engram_gate_output_backward(xl, kvl, q, k, EPS, dot, dout, mask)):
        assert torch.equal(a, b)
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    want = tref.gate_backward(cpu(xl), cpu(kvl), cpu(q), cpu(k), EPS, cpu(dot), cpu(dout), cpu(mask))
    for name, t, terms in zip(("dx", "dkv", "dq", "dk"), got, (dim + 64, dim + 64, T + dim + 64, T + dim + 64)):
        # d rh^2 / dim in the formula and a dot that belongs to other rows: the norms enter as they are, so no more than sums
        tol = 2 * terms * U32 * want[name + "_mag"] + (U16 * want[name].abs() if t.dtype == torch.bfloat16 else 0)
        assert ((cpu(t).double() - want[name]).abs() <= tol + 1e-38).all(), name


def test_masked_rows_may_hold_anything(gpu_device):
    T, hc, dim = 40, 4, 264
    x, kv, q, k, mask, dout = _gate_case(T, hc, dim, gpu_device)
    xb, kvb = x.clone(), kv.clone()
    xb[~mask], kvb[~mask] = float("nan"), float("inf")
    out, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    out2, dot2, c2 = g.engram_gate_output_ckpt(xb, kvb, q, k, EPS, mask)
    assert torch.equal(out2[mask], out[mask]) and torch.equal(dot2[mask], dot[mask])
    for a, b in zip(g.engram_gate_output_backward_ckpt(c2, q, k, EPS, dot2, dout, mask),
                    g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, mask)):
        assert torch.equal(a, b)
    # unmasked, a NaN is read back as NaN and reaches its token's gradient
    c3 = g.engram_gate_output_ckpt(xb, kv, q, k, EPS)[2]
    assert g.engram_ckpt_load(c3.x, c3.x_scale)[~mask].isnan().all()
    assert not g.engram_ckpt_load(c3.x, c3.x_scale)[mask].isnan().any()


def test_gradient_in_place_and_all_masked(gpu_device):
    T, hc, dim = 50, 4, 512
    x, kv, q, k, _, dout = _gate_case(T, hc, dim, gpu_device)
    _, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS)
    dx, dkv, dq, dk = g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout)
    own = dout.clone()
    dx2, dkv2, *_ = g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, own, dx=own)
    assert dx2 is own and torch.equal(dx2, dx) and torch.equal(dkv2, dkv)
    none = torch.zeros(T, dtype=torch.bool, device=gpu_device)
    dx, dkv, dq, dk = g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, none)
    assert torch.equal(dx, dout) and not dkv.any() and not dq.any() and not dk.any()


def test_gradient_against_differences(gpu_device):
    """Along its own gradient the loss sum(out * dout), taken at the values kept, changes by the gradient's squared norm."""
    T, hc, dim = 12, 2, 64
    x, kv, q, k, mask, dout = _gate_case(T, hc, dim, gpu_device)
    _, _, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    at = [g.engram_ckpt_load(c.x, c.x_scale).cpu().double(), g.engram_ckpt_load(c.kv, c.kv_scale).cpu().double().view(T, -1),
          q.cpu().double(), k.cpu().double()]
    m, up = mask.cpu(), dout.cpu().double()

    def loss(v):
        out, d = tref.gate_forward(*v, EPS, m)
        return float((out * up).sum()), d

    dot = loss(at)[1].float().to(gpu_device)  # of the values kept, so that the formula's norms are the dot's
    grads = [t.cpu().double() for t in g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, mask)]
    for i, gr in enumerate(grads):
        norm = float(gr.norm())
        step = 1e-7 * float(at[i].norm()) / norm
        hi, d1 = loss([v + step * gr if i == n else v for n, v in enumerate(at)])
        lo, d0 = loss([v - step * gr if i == n else v for n, v in enumerate(at)])
        assert torch.equal(torch.sign(d1), torch.sign(d0))
        # bf16 roundings of the gradient: 2^-8 of it, here and in the norm
        assert abs((hi - lo) / (2 * step) / norm ** 2 - 1) < 2.0 ** -6, i


# ---- streams, graphs, arguments ---------------------------------------------------------------------------------------
def test_another_stream(gpu_device):
    gen = _gen("stream")
    T, K, hc, dim = 200, 384, 4, 256
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    a, s, _ = _rows(gen, T, K, 8, gpu_device)
    x, kv, q, k, mask, dout = _gate_case(T, hc, dim, gpu_device)
    rows = _bf16(gen, (T, K)).to(gpu_device)
    side = torch.cuda.Stream()

    def calls(stream):
        r = [*g.engram_mx4_quant(rows, stream=stream), g.engram_wkv_mx4(a, s, w, stream=stream),
             *g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS, stream=stream)]
        out, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask, stream=stream)
        return r + [out, dot, *c, *g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, mask, stream=stream),
                    g.engram_ckpt_load(c.x, c.x_scale, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(side)
    torch.cuda.current_stream().wait_stream(side)
    for p, r in zip(got, want):
        assert torch.equal(p.flatten(), r.flatten())


@pytest.mark.parametrize("T", [9, 300])
def test_captured(gpu_device, T):
    """A decode call and a training step captured into a graph each, replayed on changing inputs between eager calls."""
    gen = _gen("graph", T)
    K, hc, dim = 384, 4, 256
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    rows = _bf16(gen, (T, K)).to(gpu_device)
    x, kv, q, k, mask, dout = _gate_case(T, hc, dim, gpu_device)
    ws = torch.empty(max(16, g.engram_wkv_gate_workspace_bytes(T, hc, dim),
                         g.engram_gate_output_backward_workspace_bytes(T, hc, dim)), dtype=torch.uint8, device=gpu_device)

    def step():
        aq, asc = g.engram_mx4_quant(rows)
        value, dot = g.engram_wkv_mx4_gate(aq, asc, w, x, q, k, EPS, workspace=ws)
        out, d, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
        grads = g.engram_gate_output_backward_ckpt(c, q, k, EPS, d, dout, mask, workspace=ws)
        return [g.engram_wkv_mx4(aq, asc, w), value, dot, out, d, *c, *grads]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(4):
        rows.copy_(_bf16(gen, (T, K)).to(gpu_device))
        x.copy_(_bf16(gen, (T, hc, dim)).to(gpu_device))
        kv.copy_(_bf16(gen, (T, (hc + 1) * dim), 0.5).to(gpu_device))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), turn


def test_refusals(gpu_device):
    gen = _gen("refuse")
    dev = gpu_device
    w, _ = _weights(gen, 1280, 384, dev)
    a, s, _ = _rows(gen, 10, 384, 8, dev)
    x, kv, q, k, mask, dout = _gate_case(10, 4, 256, dev)
    _, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS)
    bf = torch.bfloat16
    for call in (lambda: g.engram_wkv_mx4(a[:, :256].contiguous(), s, w), lambda: g.engram_wkv_mx4(a, s[:2].contiguous(), w),
                 lambda: g.engram_wkv_mx4(a, s, w[..., :4096].contiguous()), lambda: g.engram_wkv_mx4(a, s, w, nout=1216),
                 lambda: g.engram_wkv_mx4(a, s, w, out=torch.empty((10, 1288), dtype=bf, device=dev)),
                 lambda: g.engram_wkv_mx4(a.t(), s, w), lambda: g.engram_wkv_mx4_gate(a, s, w, x[:9], q, k, EPS),
                 lambda: g.engram_wkv_mx4_gate(a, s, w, x, q[:3], k, EPS),
                 lambda: g.engram_wkv_mx4_gate(a, s, w[:16].contiguous(), x, q, k, EPS),
                 lambda: g.engram_mx4_quant(torch.zeros((4, 96), dtype=bf, device=dev)),
                 lambda: g.engram_mx4_pack_weight(a[:, :192].contiguous(), s[:, :8].contiguous()),
                 lambda: g.engram_ckpt_load(c.x, c.x_scale[:, :3]), lambda: g.engram_ckpt_load(c.x, c.kv_scale),
                 lambda: g.engram_gate_output_ckpt(x, kv[:, :1272], q, k, EPS),
                 lambda: g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask[:9]),
                 lambda: g.engram_gate_output_backward_ckpt(c._replace(kv=c.x), q, k, EPS, dot, dout),
                 lambda: g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot[:9], dout),
                 lambda: g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, dkv=kv[:9])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.engram_mx4_quant(x.view(10, -1).float()), lambda: g.engram_wkv_mx4(a.float(), s, w),
                 lambda: g.engram_gate_output_backward_ckpt(c._replace(x=c.x.view(torch.uint8)), q, k, EPS, dot, dout)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(g.EngramError, match="workspace"):
        g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    with pytest.raises(g.EngramError, match="D must"):
        g.engram_ckpt_save(torch.zeros((4, 12), dtype=bf, device=dev))
