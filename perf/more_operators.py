"""The Engram module in narrow formats, as measured cases: its projection with 4-bit weights, and its training step with
8-bit checkpoints of the stream and of the keys and the value.

Every case names one operator (`op`) with its sizes.  `run` computes it in plain torch operations in 32 bits, or, where
`own` is set, through the entry points of gram_hash_embedding_amd.  `exact` computes it in 64 bits.

    wkv4       engram_wkv_mx4                    the projection with MXFP4 weights, of rows held in MXFP8 ("mx8"), or of bf16
               (engram_mx4_quant)                rows rounded to MXFP4 on the way ("mx4")
    gate4      engram_wkv_mx4_gate               the same projection with the gate's pre-activation in it, and the residual
               engram_gate_residual
    ckpt       engram_gate_output_ckpt           the gate and the residual, keeping the stream, the keys and the value in 8
               engram_ckpt_load                  bits (MXINT8), and reading them back
    ckpt_grad  engram_gate_output_backward_ckpt  the gradient of the gate and the residual from what was kept

Formats (OCP microscaling): 32 consecutive columns of a row share a scale 2^(s - 127), one byte; elements are E2M1 (MXFP4),
E4M3 (MXFP8) or integers in 64ths (MXINT8).
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-20


def listed():
    return [
        # one token of one sequence: what its projection costs is reading the weights
        dict(name="wkv4_token", op="wkv4", a="mx8", tokens=1, K=1536, nout=25600),
        # a decode step of 256 sequences
        dict(name="wkv4_decode", op="wkv4", a="mx8", tokens=256, K=1536, nout=25600),
        # a short sequence of odd length, its rows rounded to 4 bits too
        dict(name="wkv4_short", op="wkv4", a="mx4", tokens=251, K=1536, nout=25600),
        # 4 x 2,048 tokens
        dict(name="wkv4_mid", op="wkv4", a="mx4", tokens=8192, K=1536, nout=25600),
        # the same at the released row width (24 columns of 256)
        dict(name="wkv4_wide", op="wkv4", a="mx8", tokens=8192, K=6144, nout=25600),
        # the long prefill's 65,536 tokens
        dict(name="wkv4_long", op="wkv4", a="mx4", tokens=65536, K=1536, nout=25600),
        # a decode step of 256 sequences through the end of the module
        dict(name="gate4_decode", op="gate4", a="mx8", tokens=256, hc=4, dim=5120, K=1536, masked=0.0),
        # 4 x 2,048 tokens of which 10 % are masked
        dict(name="gate4_mid", op="gate4", a="mx4", tokens=8192, hc=4, dim=5120, K=1536, masked=0.1),
        # a training step of the tiny configuration: a launch-bound call
        dict(name="ckpt_tiny", op="ckpt", tokens=64, hc=4, dim=256, masked=0.0),
        # a training step of 4 x 2,048 tokens, 10 % masked
        dict(name="ckpt_mid", op="ckpt", tokens=8192, hc=4, dim=5120, masked=0.1),
        # their gradients
        dict(name="ckpt_grad_tiny", op="ckpt_grad", tokens=64, hc=4, dim=256, masked=0.0),
        dict(name="ckpt_grad_mid", op="ckpt_grad", tokens=8192, hc=4, dim=5120, masked=0.1),
    ]


def _log(rng, lo, hi):
    """A size in [lo, hi], evenly over its logarithm; round ones are left to the listed cases."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if v < 512 or v % 512 else v - 1


def draw(rng):
    op = rng.choice(["wkv4", "wkv4", "gate4", "ckpt", "ckpt_grad"])
    a = rng.choice(["mx4", "mx8"])
    K = 128 * (_log(rng, 3, 48) if op == "gate4" else _log(rng, 1, 48))
    if op == "wkv4":
        return dict(op=op, a=a, tokens=_log(rng, 1, 8192), K=K, nout=8 * _log(rng, 16, 3200))
    masked = rng.choice([0.0, 0.1])
    if op == "gate4":
        return dict(op=op, a=a, tokens=_log(rng, 1, 8192), hc=rng.choice([1, 2, 3, 4]), dim=256 * _log(rng, 1, 20), K=K,
                    masked=masked)
    return dict(op=op, tokens=_log(rng, 16, 8192), hc=rng.choice([1, 2, 3, 4, 4]), dim=8 * _log(rng, 32, 640),
                masked=masked)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _gen(seed, k=0):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) * 64 + k)


def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=torch.float32, device=DEVICE).normal_(0.0, std, generator=gen).to(dtype)


def _rows(gen, T, K):
    """Looked-up table rows: normal values, each run of 64 columns at a scale of its own in 2^-8 .. 2^-3."""
    s = torch.exp2(torch.randint(-8, -2, (T, K // 64, 1), device=DEVICE, generator=gen).float())
    return (_normal(gen, (T, K // 64, 64), 1.0, torch.float32) * s).to(torch.bfloat16).view(T, K)


def _scale_codes(x, top):
    """The shared scale's code of blocks [..., 32]: floor(log2 of the largest magnitude) - top, as E8M0."""
    amax = x.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - top
    return torch.where(amax > 0, (e + 127).clamp(0, 254), 0).to(torch.int32)


def _pow2(codes):
    return torch.exp2(codes.float() - 127)


def _round_e2m1(y):
    """|y| to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, with y's sign."""
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6), y)


def _mx4(x):
    """Rows [n, K] as MXFP4: (element values [n, K/32, 32], scale codes [n, K/32])."""
    b = x.float().view(x.shape[0], -1, 32)
    s = _scale_codes(b, 2)
    return _round_e2m1(b / _pow2(s)[..., None]), s


def _scales_laid_out(s):
    """Scale codes [n, K/32] as the library keeps a row operand's: uint8 [K/128, n up to a multiple of 4, 4]."""
    n, nb = s.shape
    out = torch.zeros((nb // 4, (n + 3) // 4 * 4, 4), dtype=torch.uint8, device=DEVICE)
    out[:, :n] = s.view(n, nb // 4, 4).permute(1, 0, 2).to(torch.uint8)
    return out


def _weight_laid_out(v, s):
    """MXFP4 weights as the library keeps them: uint8 [N / 64, K / 128, 4352], a record for 64 rows and 128 columns.  Row
    64 g + 16 j + r, column 128 t + 32 c + e: the element is half e % 2 of byte 1024 j + 256 c + 16 r + e / 2 of record
    [g, t], its scale byte 4096 + 64 c + 4 r + j.  Rows past N are zeros."""
    n, nb = s.shape
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEVICE)
    code = torch.searchsorted(grid, v.abs()).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.view(n, nb, 16, 2)
    G = (n + 63) // 64
    byte = torch.zeros((G * 64, nb, 16), dtype=torch.uint8, device=DEVICE)
    byte[:n] = code[..., 0] | (code[..., 1] << 4)
    sc = torch.zeros((G * 64, nb), dtype=torch.uint8, device=DEVICE)
    sc[:n] = s.to(torch.uint8)
    byte = byte.view(G, 4, 16, nb // 4, 4, 16).permute(0, 3, 1, 4, 2, 5).reshape(G, nb // 4, 4096)
    sc = sc.view(G, 4, 16, nb // 4, 4).permute(0, 3, 4, 2, 1).reshape(G, nb // 4, 256)
    return torch.cat([byte, sc], -1).contiguous()


def _int8(x):
    """Blocks of 32 columns (the last of a row may be shorter) as MXINT8: (int8 of x's shape, scale codes uint8)."""
    D = x.shape[-1]
    b = torch.nn.functional.pad(x.float(), (0, -D % 32)).unflatten(-1, (-1, 32))
    s = _scale_codes(b, 0)
    q = torch.round(b / _pow2(s)[..., None] * 64).clamp(-127, 127).to(torch.int8)
    return q.flatten(-2)[..., :D].contiguous(), s.to(torch.uint8)


def _int8_values(q, s):
    """What MXINT8 elements and scale codes stand for, in 32 bits."""
    return q.float() * (_pow2(s) / 64).repeat_interleave(32, -1)[..., :q.shape[-1]]


def prepare(case, seed):
    op, T = case["op"], case["tokens"]
    s = dict(case=case, op=op)
    g = _gen(seed)
    if op in ("wkv4", "gate4"):
        K = case["K"]
        N = case["nout"] if op == "wkv4" else (case["hc"] + 1) * case["dim"]
        rows = _rows(g, T, K)
        if case["a"] == "mx8":  # the gather wrote its rows as MXFP8
            b = rows.float().view(T, -1, 32)
            sc = _scale_codes(b, 8)
            q = (b / _pow2(sc)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["a"], s["a_scale"] = q.view(torch.uint8).view(T, K), _scales_laid_out(sc)
        else:
            s["a"] = rows
        s["w"] = _weight_laid_out(*_mx4(_normal(g, (N, K), 0.02)))
    if op == "wkv4":
        return s
    hc, dim = case["hc"], case["dim"]
    s["x"] = _normal(g, (T, hc, dim), 1.0)
    s["q"] = 1 + _normal(g, (hc, dim), 0.1)
    s["k"] = 1 + _normal(g, (hc, dim), 0.1)
    s["mask"] = torch.rand(T, device=DEVICE, generator=g) >= case["masked"] if case["masked"] else None
    if op == "gate4":
        return s
    kv = _normal(g, (T, hc + 1, dim), 0.5)
    if op == "ckpt":
        s["kv"] = kv.view(T, (hc + 1) * dim)
        return s
    # what the forward kept: the stream, the keys and the value in 8 bits and the gate's pre-activation
    s["xq"], s["xs"] = _int8(s["x"])
    s["kvq"], s["kvs"] = _int8(kv)
    h, key = s.pop("x").float(), kv[:, :hc].float()
    s["dot"] = _dot(h, key, s["q"].float() * s["k"].float())
    s["dout"] = _normal(g, (T, hc, dim), 1e-3)
    return s


def _dot(h, key, w):
    rstd = torch.rsqrt(h.square().mean(-1) + EPS) * torch.rsqrt(key.square().mean(-1) + EPS)
    return (h * w * key).sum(-1) * rstd * h.shape[-1] ** -0.5


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gram_hash_embedding_amd as eng

    op = s["op"]
    if op in ("wkv4", "gate4"):
        a, a_scale = (s["a"], s["a_scale"]) if "a_scale" in s else eng.engram_mx4_quant(s["a"])
        if op == "wkv4":
            return eng.engram_wkv_mx4(a, a_scale, s["w"], nout=s["case"]["nout"])
        value, dot = eng.engram_wkv_mx4_gate(a, a_scale, s["w"], s["x"], s["q"], s["k"], EPS)
        return dict(value=value, out=eng.engram_gate_residual(s["x"], value, dot, s["mask"]))
    if op == "ckpt":
        out, dot, ckpt = eng.engram_gate_output_ckpt(s["x"], s["kv"], s["q"], s["k"], EPS, s["mask"])
        return dict(out=out, dot=dot, x=eng.engram_ckpt_load(ckpt.x, ckpt.x_scale),
                    kv=eng.engram_ckpt_load(ckpt.kv, ckpt.kv_scale))
    ckpt = eng.GateCheckpoint(s["xq"], s["xs"], s["kvq"], s["kvs"])
    dx, dkv, dq, dk = eng.engram_gate_output_backward_ckpt(ckpt, s["q"], s["k"], EPS, s["dot"], s["dout"],
                                                           token_mask=s["mask"])
    return dict(dx=dx, dkv=dkv, dq=dq, dk=dk)


def _operands(s):
    """The projection's two operands, in 32 bits."""
    if "a_scale" in s:
        T, K = s["a"].shape
        codes = s["a_scale"][:, :T].permute(1, 0, 2).reshape(T, K // 32, 1)
        a = s["a"].view(torch.float8_e4m3fn).float().view(T, -1, 32) * _pow2(codes)
    else:
        v, codes = _mx4(s["a"])
        a = v * _pow2(codes)[..., None]
    G, S = s["w"].shape[:2]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEVICE)
    byte = s["w"][..., :4096].view(G, S, 4, 4, 16, 16).permute(0, 2, 4, 1, 3, 5)
    val = grid[torch.stack([byte & 15, byte >> 4], -1).int()].reshape(G * 64, S * 4, 32)
    codes = s["w"][..., 4096:].view(G, S, 4, 16, 4).permute(0, 4, 3, 1, 2).reshape(G * 64, S * 4, 1)
    return a.flatten(1), (val * _pow2(codes)).flatten(1)


def _gate(dot, mask):
    gate = torch.sigmoid(torch.copysign(torch.sqrt(dot.abs().clamp(min=1e-6)), dot))
    return gate if mask is None else torch.where(mask[:, None], gate, 0.0)


def _run_plain(s):
    op, case = s["op"], s["case"]
    if op == "wkv4":
        a, w = _operands(s)
        return (a @ w[:case["nout"]].t()).to(torch.bfloat16)
    hc, dim = case["hc"], case["dim"]
    w = s["q"].float() * s["k"].float()
    if op in ("gate4", "ckpt"):
        h = s["x"].float()
        if op == "gate4":
            a, wt = _operands(s)
            kv = (a @ wt.t()).view(-1, hc + 1, dim)
        else:
            kv = s["kv"].float().view(-1, hc + 1, dim)
        dot = _dot(h, kv[:, :hc], w)
        out = (h + _gate(dot, s["mask"])[..., None] * kv[:, hc:]).to(torch.bfloat16)
        if op == "gate4":
            return dict(value=kv[:, hc].to(torch.bfloat16), out=out)
        return dict(out=out, dot=dot, x=_int8_values(*_int8(h)).to(torch.bfloat16),
                    kv=_int8_values(*_int8(kv)).to(torch.bfloat16))
    x, kv, dout, d = _int8_values(s["xq"], s["xs"]), _int8_values(s["kvq"], s["kvs"]), s["dout"].float(), s["dot"]
    key, v = kv[:, :hc], kv[:, hc]
    rh = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    rk = torch.rsqrt(key.square().mean(-1, keepdim=True) + EPS)
    z = torch.sqrt(d.abs().clamp(min=1e-6))
    g = torch.sigmoid(torch.copysign(z, d))
    ddot = torch.where(d.abs() >= 1e-6, (dout * v[:, None, :]).sum(-1) * g * (1 - g) / (2 * z), 0.0)
    if s["mask"] is not None:
        ddot = torch.where(s["mask"][:, None], ddot, 0.0)
        g = torch.where(s["mask"][:, None], g, 0.0)
    ddot, g, d = ddot[..., None], g[..., None], d[..., None]
    c = rh * rk * dim ** -0.5
    dx = (dout + ddot * (c * w * key - d * rh * rh / dim * x)).to(torch.bfloat16)
    dkey = ddot * (c * w * x - d * rk * rk / dim * key)
    dkv = torch.cat([dkey, (g * dout).sum(1, keepdim=True)], 1).flatten(1).to(torch.bfloat16)
    dw = (ddot * c * x * key).sum(0)
    return dict(dx=dx, dkv=dkv, dq=dw * s["k"].float(), dk=dw * s["q"].float())


# ---------------------------------------------------------------------------------------------------------------------
# the bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    op, T = case["op"], case["tokens"]
    if op in ("wkv4", "gate4"):
        K = case["K"]
        N = case["nout"] if op == "wkv4" else (case["hc"] + 1) * case["dim"]
        b = N * K * 17 // 32 + T * (K * 2 if case["a"] == "mx4" else K * 33 // 32)
        if op == "wkv4":
            return dict(bytes=b + 2 * T * N, flops=2 * T * N * K)
        hc, dim = case["hc"], case["dim"]
        return dict(bytes=b + T * dim * (4 * hc + 2) + 4 * hc * dim, flops=2 * T * N * K + 10 * T * hc * dim)
    hc, dim = case["hc"], case["dim"]
    kept = (2 * hc + 1) * (dim + (dim + 31) // 32)  # a token's stream, keys and value in 8 bits with their scales
    if op == "ckpt":  # the rows in, the output, and the rows as they are read back
        return dict(bytes=T * (2 * dim * (5 * hc + 2) + 4 * hc) + 4 * hc * dim, flops=T * dim * (14 * hc + 4))
    return dict(bytes=T * (kept + 2 * dim * (3 * hc + 1) + 4 * hc) + 12 * hc * dim, flops=T * dim * (28 * hc + 3))


# ---------------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _exact_e8m0(blocks, top):
    """The block's scale 2^k, k = floor(log2 amax) - top kept in [-127, 127], from the exponent field of amax in 64 bits."""
    bits = blocks.abs().amax(-1, keepdim=True).view(torch.int64)
    k = torch.where(bits > 0, (bits >> 52) - 1023 - top, -127).clamp(-127, 127)
    return ((k + 1023) << 52).view(torch.float64)


def _exact_mx4(x):
    """The values of the nearest MXFP4 rows: the count of the midpoints below an element is its code."""
    b = x.double().view(x.shape[0], -1, 32)
    p = _exact_e8m0(b, 2)
    a = (b / p).abs()
    code = sum((a > m).long() for m in (0.25, 1.25, 2.5, 5.0)) + sum((a >= m).long() for m in (0.75, 1.75, 3.5))
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEVICE)
    return (torch.sign(b) * grid[code] * p).flatten(1)


def _exact_weight(packed):
    """The [rows, K] values of weights as the library keeps them, record by record position."""
    G, S = packed.shape[:2]
    out = torch.empty((G, 4, 16, S, 4, 32), dtype=torch.float64, device=DEVICE)  # [g, j, r, t, c, e]
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    lut = torch.tensor([m if c < 8 else -m for c, m in enumerate(mag + mag)], dtype=torch.float64, device=DEVICE)
    for j in range(4):
        for c in range(4):
            at = packed[..., 1024 * j + 256 * c:1024 * j + 256 * c + 256].reshape(G, S, 16, 16).long()
            code = packed[..., 4096 + 64 * c + j:4096 + 64 * c + 64:4].reshape(G, S, 16, 1).double()
            p = torch.exp2(code - 127)
            out[:, j, :, :, c, 0::2] = (lut[at % 16] * p).transpose(1, 2)
            out[:, j, :, :, c, 1::2] = (lut[at // 16] * p).transpose(1, 2)
    return out.reshape(G * 64, S * 128)


def _exact_int8(x):
    D = x.shape[-1]
    parts = []
    for c0 in range(0, D, 32):
        b = x[..., c0:c0 + 32].double()
        p = _exact_e8m0(b, 0) / 64
        parts.append(torch.clamp(torch.round(b / p), -127, 127) * p)
    return torch.cat(parts, -1)


def _exact_kept(q, s):
    """MXINT8 by their definition: integer / 64 times 2^(code - 127)."""
    idx = torch.arange(q.shape[-1], device=DEVICE) // 32
    return torch.ldexp(q.double() / 64, s.int()[..., idx] - 127)


def _exact_gate(d, live):
    root = torch.sqrt(torch.maximum(d.abs(), torch.full_like(d, 1e-6)))
    return live[:, None] / (1 + torch.exp(torch.where(torch.signbit(d), root, -root))), root


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["tokens"]
    if op in ("wkv4", "gate4"):
        if "a_scale" in s:
            a = s["a"].view(torch.float8_e4m3fn).double()
            for t in range(s["a_scale"].shape[0]):
                codes = s["a_scale"][t, :T].double()
                for b in range(4):
                    c0 = 128 * t + 32 * b
                    a[:, c0:c0 + 32] *= torch.exp2(codes[:, b:b + 1] - 127)
        else:
            a = _exact_mx4(s["a"])
        kv = torch.mm(a, _exact_weight(s["w"]).t())
        if op == "wkv4":
            return kv[:, :case["nout"]]
    hc, dim = case["hc"], case["dim"]
    live = torch.ones(T, dtype=torch.float64, device=DEVICE) if s["mask"] is None else s["mask"].double()
    q, k = s["q"].double(), s["k"].double()
    if op in ("gate4", "ckpt"):
        if op == "ckpt":
            kv = s["kv"].double()
        v = kv[:, hc * dim:]
        outs, dots = [], []
        for c in range(hc):
            h, key = s["x"][:, c].double(), kv[:, c * dim:(c + 1) * dim]
            d = (h * key * (q[c] * k[c])).sum(1) / torch.sqrt(
                ((h * h).mean(1) + EPS) * ((key * key).mean(1) + EPS) * dim)
            gate, _ = _exact_gate(d[:, None], live)
            outs.append(h + gate * v)
            dots.append(d)
        if op == "gate4":
            return dict(value=v, out=torch.stack(outs, 1))
        return dict(out=torch.stack(outs, 1), dot=torch.stack(dots, 1), x=_exact_int8(s["x"]),
                    kv=_exact_int8(s["kv"].view(T, hc + 1, dim)))
    x, kv = _exact_kept(s["xq"], s["xs"]), _exact_kept(s["kvq"], s["kvs"])
    v = kv[:, hc]
    dv = torch.zeros_like(v)
    dx, dkey, dq, dk = [], [], [], []
    for c in range(hc):  # copy by copy: the derivative of sum(out * dout) through the gate, the given dot and its two norms
        h, key, up, d = x[:, c], kv[:, c], s["dout"][:, c].double(), s["dot"][:, c:c + 1].double()
        gate, root = _exact_gate(d, live)
        dv += gate * up
        slope = torch.where(s["dot"][:, c:c + 1].abs() < 1e-6, 0.0, gate * (1 - gate) / (2 * root))
        e = (up * v).sum(1, keepdim=True) * slope
        mh, mk = (h * h).mean(1, keepdim=True) + EPS, (key * key).mean(1, keepdim=True) + EPS
        unit = 1 / torch.sqrt(mh * mk * dim)
        dx.append(up + e * (unit * (q[c] * k[c]) * key - d * h / (mh * dim)))
        dkey.append(e * (unit * (q[c] * k[c]) * h - d * key / (mk * dim)))
        both = (e * unit * h * key).sum(0)
        dq.append(both * k[c])
        dk.append(both * q[c])
    return dict(dx=torch.stack(dx, 1), dkv=torch.cat(dkey + [dv], 1), dq=torch.stack(dq), dk=torch.stack(dk))
