"""The narrow formats' plain implementations against other statements of the same definitions, and the refusals of the entry
points (CPU: a refused call touches no device)."""
import ctypes
from fractions import Fraction

import pytest
import torch

import gram_hash_embedding_amd as g
from tests import lowbit_ref as ref

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100004)


def _err():
    return g.lib().engram_last_error().decode()


def _bf16(seed, shape, spread=20):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * torch.exp2(torch.randint(-spread, spread, (*shape[:-1], 1), generator=gen).float())
    return x.to(torch.bfloat16)


def test_mx4_quant_by_fractions():
    """Every element is the nearest of the sixteen values to x / 2^e in exact arithmetic, the even code of two."""
    x = _bf16(1, (6, 128))
    x[0, :32] = 0
    x[1, 3] = 5.0 * 2.0 ** 10   # a tie (4 and 6 are as near)
    x[2, 32:64] = torch.tensor([k * 0.25 for k in range(32)]).to(torch.bfloat16)  # every tie of the grid up to 7.75
    code, s = ref.mx4_quant(x.double())
    for n in range(x.shape[0]):
        for b in range(4):
            blk = [Fraction(float(v)) for v in x[n, 32 * b:32 * b + 32]]
            amax = max(abs(v) for v in blk)
            e = -127
            if amax:
                e = max(-127, (amax.numerator.bit_length() - amax.denominator.bit_length() - 3))
                while Fraction(2) ** (e + 3) <= amax:
                    e += 1
            assert int(s[n, b]) == e + 127
            for i, v in enumerate(blk):
                y = abs(v) / Fraction(2) ** e
                d = [abs(y - Fraction(m)) for m in ref.E2M1]
                best = [k for k in range(8) if d[k] == min(d)]
                want = best[0] if len(best) == 1 else [k for k in best if k % 2 == 0][0]
                assert int(code[n, 32 * b + i]) & 7 == want
                assert (int(code[n, 32 * b + i]) >> 3) == int(torch.signbit(x[n, 32 * b + i]))


def test_int8_values_are_within_half_a_unit_and_exact_in_bf16():
    x = _bf16(2, (50, 1000), 60)
    x[0] = 127.5
    x[1, 5] = 2.0 ** -133  # bf16's smallest subnormal
    x[1, :5] = 0
    x[1, 6:] = 0
    q, s = ref.int8_quant(x.double())
    v = ref.int8_values(q, s)
    assert torch.equal(v.to(torch.bfloat16).double(), v)
    unit = torch.exp2(s.double() - 133).repeat_interleave(32, -1)[:, :1000]
    assert ((v - x.double()).abs() <= unit / 2).all()
    q2, s2 = ref.int8_quant(v)
    assert torch.equal(ref.int8_values(q2, s2), v)  # what was kept is kept again unchanged


@pytest.mark.parametrize("quant", [ref.mx4_quant, ref.int8_quant])
def test_not_finite_blocks(quant):
    x = torch.ones((3, 128), dtype=torch.float64)
    x[0, 40], x[1, 127], x[2, 0] = float("inf"), float("nan"), -float("inf")
    code, s = quant(x)
    want = torch.full((3, 4), 125 if quant is ref.mx4_quant else 127, dtype=torch.uint8)
    want[0, 1] = want[1, 3] = want[2, 0] = 255
    assert torch.equal(s, want) and (code[0, 32:64] == 0).all()


def test_weight_layout_is_the_measured_cases():
    from perf import more_operators as m

    code = torch.randint(0, 16, (136, 384), dtype=torch.uint8)
    code[code == 8] = 9  # (values tell +0 from -0, the layout's helper there takes values)
    s = torch.randint(0, 255, (136, 12), dtype=torch.uint8)
    grid = torch.tensor(ref.E2M1 + [-v for v in ref.E2M1])
    m.DEVICE = "cpu"
    try:
        got = m._weight_laid_out(grid[code.long()].view(136, 12, 32), s.to(torch.int32))
    finally:
        m.DEVICE = "cuda"
    assert torch.equal(got, ref.weight_laid_out(code, s))


@pytest.mark.parametrize("args,status,msg", [
    (dict(rows=-1), 1, "rows < 0"), (dict(K=0), 1, "K=0"), (dict(K=96), 1, "K=96"), (dict(K=-128), 1, "K=-128"),
    (dict(x=None), 1, "null"), (dict(q=None), 1, "null"), (dict(scale=None), 1, "null"), (dict(x=ODD), 1, "misaligned"),
    (dict(q=ctypes.c_void_p(0x100002)), 1, "misaligned"), (dict(rows=0, x=None), 0, "")])
def test_mx4_quant_validation(args, status, msg):
    a = dict(x=FAKE, rows=5, K=128, q=FAKE, scale=FAKE)
    a.update(args)
    rc = g.lib().engram_mx4_quant(a["x"], a["rows"], a["K"], a["q"], a["scale"], None)
    assert rc == status and (status == 0 or msg in _err())


@pytest.mark.parametrize("args,msg", [
    (dict(K=100), "K must"), (dict(N=12), "columns"), (dict(N=0), "columns"), (dict(q=None), "null"), (dict(scale=None), "null"),
    (dict(packed=None), "null"), (dict(q=ODD), "misaligned"), (dict(packed=ODD), "misaligned")])
def test_pack_validation(args, msg):
    a = dict(q=FAKE, scale=FAKE, N=72, K=128, packed=FAKE)
    a.update(args)
    assert g.lib().engram_mx4_pack_weight(a["q"], a["scale"], a["N"], a["K"], a["packed"], None) == 1 and msg in _err()


def test_weight_bytes():
    assert g.engram_mx4_weight_bytes(25600, 1536) == 400 * 12 * 4352
    assert g.engram_mx4_weight_bytes(8, 128) == 4352
    for N, K in ((12, 128), (8, 64), (0, 128), (8, 1 << 21), (1 << 23, 128), (-8, 128)):
        assert g.lib().engram_mx4_weight_bytes(N, K) == -1
        with pytest.raises(ValueError):
            g.engram_mx4_weight_bytes(N, K)


@pytest.mark.parametrize("args,status,msg", [
    (dict(T=-1), 1, "T < 0"), (dict(bits=6), 1, "a_bits"), (dict(K=64), 1, "K must"), (dict(K=130), 1, "K must"),
    (dict(N=4), 1, "columns"), (dict(a=None), 1, "null"), (dict(a_scale=None), 1, "null"), (dict(w=None), 1, "null"),
    (dict(kv=None), 1, "null"), (dict(a=ODD), 1, "misaligned"), (dict(a_scale=ODD), 1, "misaligned"),
    (dict(w=ODD), 1, "misaligned"), (dict(kv=ODD), 1, "misaligned"), (dict(T=0, a=None), 0, ""),
    (dict(T=1 << 50), 1, "too many")])
def test_wkv_mx4_validation(args, status, msg):
    a = dict(a=FAKE, a_scale=FAKE, bits=8, w=FAKE, kv=FAKE, T=10, K=128, N=64)
    a.update(args)
    rc = g.lib().engram_wkv_mx4(a["a"], a["a_scale"], a["bits"], a["w"], a["kv"], a["T"], a["K"], a["N"], None)
    assert rc == status and (status == 0 or msg in _err())


@pytest.mark.parametrize("args,status,msg", [
    (dict(T=-1), 1, "T < 0"), (dict(bits=0), 1, "a_bits"), (dict(hc=0), 1, "hc=0"), (dict(hc=65), 1, "hc=65"),
    (dict(dim=128), 1, "dim=128"), (dict(dim=300), 1, "dim=300"), (dict(hc=64, dim=1 << 17), 1, "exceeds"),
    (dict(K=96), 1, "K must"), (dict(ld=248), 1, "ld_value"), (dict(ld=260), 1, "ld_value"), (dict(ld=(1 << 22) + 8), 1, "ld_value"), (dict(wn=16), 2, "workspace"),
    (dict(a=None), 1, "null"), (dict(x=None), 1, "null"), (dict(q=None), 1, "null"), (dict(value=None), 1, "null"),
    (dict(dot=None), 1, "null"), (dict(ws=None), 1, "null"), (dict(x=ODD), 1, "misaligned"), (dict(value=ODD), 1, "misaligned"),
    (dict(dot=ctypes.c_void_p(0x100001)), 1, "misaligned"), (dict(T=0, a=None), 0, "")])
def test_wkv_mx4_gate_validation(args, status, msg):
    a = dict(a=FAKE, a_scale=FAKE, bits=4, w=FAKE, x=FAKE, q=FAKE, k=FAKE, value=FAKE, ld=256, dot=FAKE, ws=FAKE, wn=1 << 30,
             T=10, K=128, hc=4, dim=256)
    a.update(args)
    rc = g.lib().engram_wkv_mx4_gate(a["a"], a["a_scale"], a["bits"], a["w"], a["x"], a["q"], a["k"], 1e-20, a["value"],
                                     a["ld"], a["dot"], a["ws"], a["wn"], a["T"], a["K"], a["hc"], a["dim"], None)
    assert rc == status and (status == 0 or msg in _err())


@pytest.mark.parametrize("args,status,msg", [
    (dict(rows=-1), 1, "rows < 0"), (dict(D=12), 1, "D must"), (dict(D=0), 1, "D must"), (dict(D=1 << 21), 1, "D must"),
    (dict(x=None), 1, "null"), (dict(q=None), 1, "null"), (dict(scale=None), 1, "null"), (dict(x=ODD), 1, "misaligned"),
    (dict(q=ODD), 1, "misaligned"), (dict(rows=0, x=None), 0, "")])
def test_ckpt_validation(args, status, msg):
    a = dict(x=FAKE, q=FAKE, scale=FAKE, rows=5, D=40)
    a.update(args)
    for rc in (g.lib().engram_ckpt_save(a["x"], a["rows"], a["D"], a["q"], a["scale"], None),
               g.lib().engram_ckpt_load(a["q"], a["scale"], a["rows"], a["D"], a["x"], None)):
        assert rc == status and (status == 0 or msg in _err())


@pytest.mark.parametrize("args,status,msg", [
    (dict(T=-1), 1, "T < 0"), (dict(hc=0), 1, "hc=0"), (dict(hc=65), 1, "hc=65"), (dict(dim=12), 1, "dim=12"),
    (dict(dim=8200), 1, "dim=8200"), (dict(ld=1272), 1, "ld_kv"), (dict(ld=1281), 1, "ld_kv"), (dict(x=None), 1, "null"),
    (dict(kv=None), 1, "null"), (dict(out=None), 1, "null"), (dict(dot=None), 1, "null"), (dict(xq=None), 1, "null"),
    (dict(xs=None), 1, "null"), (dict(kvq=None), 1, "null"), (dict(kvs=None), 1, "null"), (dict(x=ODD), 1, "misaligned"),
    (dict(xq=ODD), 1, "misaligned"), (dict(kvq=ODD), 1, "misaligned"), (dict(T=0, x=None), 0, "")])
def test_gate_output_ckpt_validation(args, status, msg):
    a = dict(x=FAKE, kv=FAKE, ld=1280, q=FAKE, k=FAKE, out=FAKE, dot=FAKE, xq=FAKE, xs=FAKE, kvq=FAKE, kvs=FAKE, T=10, hc=4,
             dim=256)
    a.update(args)
    rc = g.lib().engram_gate_output_ckpt(a["x"], a["kv"], a["ld"], a["q"], a["k"], 1e-20, None, a["out"], a["dot"], a["xq"],
                                         a["xs"], a["kvq"], a["kvs"], a["T"], a["hc"], a["dim"], None)
    assert rc == status and (status == 0 or msg in _err())


@pytest.mark.parametrize("args,status,msg", [
    (dict(T=-1), 1, "T < 0"), (dict(hc=0), 1, "hc=0"), (dict(dim=8200), 1, "dim=8200"), (dict(xq=None), 1, "null"),
    (dict(xs=None), 1, "null"), (dict(kvq=None), 1, "null"), (dict(kvs=None), 1, "null"), (dict(dout=None), 1, "null"),
    (dict(dq=None), 1, "null"), (dict(ws=None), 1, "null"), (dict(xq=ODD), 1, "misaligned"), (dict(kvq=ODD), 1, "misaligned"),
    (dict(dx=ODD), 1, "misaligned"), (dict(wn=16), 2, "workspace")])
def test_gate_backward_ckpt_validation(args, status, msg):
    a = dict(xq=FAKE, xs=FAKE, kvq=FAKE, kvs=FAKE, q=FAKE, k=FAKE, dot=FAKE, dout=FAKE, dx=FAKE, dkv=FAKE, dq=FAKE, dk=FAKE,
             ws=FAKE, wn=1 << 30, T=10, hc=4, dim=256)
    a.update(args)
    rc = g.lib().engram_gate_output_backward_ckpt(a["xq"], a["xs"], a["kvq"], a["kvs"], a["q"], a["k"], 1e-20, a["dot"],
                                                  a["dout"], None, a["dx"], a["dkv"], a["dq"], a["dk"], a["ws"], a["wn"],
                                                  a["T"], a["hc"], a["dim"], None)
    assert rc == status and msg in _err()


def test_cpu_tensors_are_refused():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    for call in (lambda: g.engram_mx4_quant(x), lambda: g.engram_ckpt_save(x), lambda: g.engram_mx4_quant([1.0])):
        with pytest.raises((ValueError, TypeError)):
            call()
