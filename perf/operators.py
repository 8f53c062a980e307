"""The operators that train the Engram module and its embeddings, as measured cases.

Every case names one operator (`op`) with its sizes.  `run` computes it in plain torch operations in 32 bits, or, where
`own` is set, through the entry points of gram_hash_embedding_amd.  `exact` computes it in 64 bits.

    embed       engram_embed                 table rows of token ids, scaled
    embed_grad  engram_embed_grad            its gradient, one row per table row
    embed_rows  engram_embed_grad_rows       its gradient as the distinct rows (hashed tables)
    gate        engram_gate_output_backward  the gradient of the gate and the residual
    wkv         engram_wkv_backward          the gradient of the wkv projection
    clip        engram_grad_norm + engram_clip_grads
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
EPS = 1e-20
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the token embedding of one decode step of 256 sequences, rows scaled by sqrt(dim)
        dict(name="embed_decode", op="embed", n=256, rows=129280, dim=5120, table="bf16", out="bf16", ids="i64",
             scale=71.5, outside=0.0),
        # the token embedding of a 65,536-token prefill
        dict(name="embed_long", op="embed", n=65536, rows=129280, dim=5120, table="bf16", out="bf16", ids="i64",
             scale=71.5, outside=0.0),
        # its gradient for a small training step of the tiny configuration: a launch-bound call
        dict(name="embed_grad_tiny", op="embed_grad", n=64, rows=1000, dim=256, grad="bf16", out="f32", ids="i64",
             scale=16.0, outside=0.0),
        # its gradient for 4 x 2,048 Zipf tokens over the whole vocabulary, fp32
        dict(name="embed_grad_mid", op="embed_grad", n=8192, rows=129280, dim=5120, grad="bf16", out="f32", ids="i64",
             scale=71.5, outside=0.0),
        # the hashed table's gradient: 8,192 tokens x 24 columns, a table of 3,988,006 rows of 64
        dict(name="embed_rows_mid", op="embed_rows", tokens=8192, cols=24, rows=3988006, dim=64, grad="bf16",
             out="f32", ids="i64", scale=1.0),
        # the same for 65,536 tokens and the released table's 384,006,168 rows
        dict(name="embed_rows_long", op="embed_rows", tokens=65536, cols=24, rows=384006168, dim=64, grad="bf16",
             out="f32", ids="i64", scale=1.0),
        # the gate's gradient at the tiny configuration: a launch-bound call
        dict(name="gate_tiny", op="gate", tokens=64, hc=4, dim=256, masked=0.0),
        # the gate's gradient for 4 x 2,048 tokens, 10 % masked
        dict(name="gate_mid", op="gate", tokens=8192, hc=4, dim=5120, masked=0.1),
        # the projection's gradient for a short sequence of odd length: bound by the weight's traffic
        dict(name="wkv_short", op="wkv", tokens=251, K=1536, nout=25600, dw="f32"),
        # the projection's gradient for 4 x 2,048 tokens
        dict(name="wkv_mid", op="wkv", tokens=8192, K=1536, nout=25600, dw="f32"),
        # the gradients of one tiny layer: a launch-bound call
        dict(name="clip_tiny", op="clip", layers=1, hc=4, dim=256, K=192, rows=384, width=32, vocab=1000, dw="f32",
             max_norm=1.0),
        # the gradients of two layers of 4 x 2,048 tokens and of the token embedding
        dict(name="clip_mid", op="clip", layers=2, hc=4, dim=5120, K=1536, rows=196608, width=64, vocab=129280,
             dw="f32", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    """A size in [lo, hi], evenly over its logarithm; round ones are left to the listed cases."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if v < 512 or v % 512 else v - 1


def _width(rng, lo, hi):
    """A row width in [lo, hi]: a configuration-like one, or an odd multiple of 8."""
    if rng.random() < 0.4:
        return rng.choice([v for v in (32, 64, 128, 256, 512, 1024, 1536, 2048, 4096, 5120, 10240, 20480, 25600)
                           if lo <= v <= hi])
    return min(hi, 8 * (_log(rng, lo // 8, hi // 8) | 1))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_rows", "gate", "wkv", "clip"])
    dt = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    ids = rng.choice(["i64", "i32"])
    if op == "embed":
        return dict(op=op, n=_log(rng, 16, 32768), rows=_log(rng, 1000, 129280), dim=_width(rng, 32, 5120), table=dt(),
                    out=dt(), ids=ids, scale=rng.choice([1.0, 71.5]), outside=rng.choice([0.0, 0.05]))
    if op == "embed_grad":
        return dict(op=op, n=_log(rng, 16, 8192), rows=_log(rng, 1000, 129280), dim=_width(rng, 32, 5120), grad=dt(),
                    out=dt(), ids=ids, scale=rng.choice([1.0, 71.5]), outside=rng.choice([0.0, 0.05]))
    if op == "embed_rows":
        return dict(op=op, tokens=_log(rng, 16, 32768), cols=rng.choice([6, 24]), rows=_log(rng, 9670, 384006168),
                    dim=rng.choice([32, 64, 64, 128]), grad=dt(), out=dt(), ids=ids, scale=1.0)
    if op == "gate":
        return dict(op=op, tokens=_log(rng, 16, 8192), hc=rng.choice([1, 2, 4, 4, 4]), dim=_width(rng, 256, 5120),
                    masked=rng.choice([0.0, 0.1]))
    if op == "wkv":
        return dict(op=op, tokens=_log(rng, 16, 8192), K=_width(rng, 192, 1536), nout=_width(rng, 1280, 25600), dw=dt())
    return dict(op=op, layers=rng.choice([1, 2]), hc=4, dim=_width(rng, 256, 5120), K=_width(rng, 192, 1536),
                rows=_log(rng, 384, 196608), width=rng.choice([32, 64]), vocab=_log(rng, 1000, 129280), dw=dt(),
                max_norm=rng.choice([1.0, 1.0, 1e6]))


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _gen(seed, k=0):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) * 64 + k)


def _normal(gen, shape, std, dtype):
    return torch.empty(shape, dtype=torch.float32, device=DEVICE).normal_(0.0, std, generator=gen).to(dtype)


def _zipf(gen, n, vocab):
    """Token ids with P(id) ~ (id + 1)^-1.1, as natural text's."""
    p = torch.arange(1, vocab + 1, dtype=torch.float64, device=DEVICE).pow(-1.1)
    cdf = torch.cumsum(p, 0)
    u = torch.rand(n, dtype=torch.float64, device=DEVICE, generator=gen) * cdf[-1]
    return torch.searchsorted(cdf, u).clamp_(max=vocab - 1)


def _token_ids(case, gen):
    ids = _zipf(gen, case["n"], case["rows"])
    if case["outside"]:  # positions that take no part carry an id outside the table
        ids = torch.where(torch.rand(case["n"], device=DEVICE, generator=gen) < case["outside"],
                          torch.full_like(ids, -1), ids)
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def _hash_ids(case, gen):
    """[tokens, cols] ids of 2-, 3- and 4-grams of Zipf tokens, each column in its own share of the table."""
    n, cols, rows = case["tokens"], case["cols"], case["rows"]
    tok = _zipf(gen, n + 3, 99092)
    mult = (torch.arange(1, 5, dtype=torch.int64, device=DEVICE) * 2654435761 * 97) | 1
    share = rows // cols
    prod = [tok[3 - s:n + 3 - s] * mult[s] for s in range(4)]
    out, r = [], prod[0]
    for g in range(1, 4):
        r = r ^ prod[g]
        for h in range(cols // 3):
            c = (g - 1) * (cols // 3) + h
            p = share - 2 * c if share - 2 * c > 1 else share
            out.append(torch.remainder(r, p) + c * share)
    return torch.stack(out, dim=1).contiguous().to(torch.int32 if case["ids"] == "i32" else torch.int64)


def _clip_shapes(case):
    """(shape, dtype) of every gradient: per layer the projection's, q's and k's and the table rows'; the embedding's."""
    got = []
    for _ in range(case["layers"]):
        got += [(((case["hc"] + 1) * case["dim"], case["K"]), case["dw"]), ((case["hc"], case["dim"]), "f32"),
                ((case["hc"], case["dim"]), "f32"), ((case["rows"], case["width"]), "f32")]
    return got + [((case["vocab"], case["dim"]), "bf16")]


def prepare(case, seed):
    op = case["op"]
    s = dict(case=case, op=op)
    g = _gen(seed)
    if op == "embed":
        s["ids"] = _token_ids(case, g)
        s["table"] = _normal(g, (case["rows"], case["dim"]), 0.02, _DT[case["table"]])
    elif op == "embed_grad":
        s["ids"] = _token_ids(case, g)
        s["grad"] = _normal(g, (case["n"], case["dim"]), 1e-3, _DT[case["grad"]])
    elif op == "embed_rows":
        s["ids"] = _hash_ids(case, g)
        s["grad"] = _normal(g, (case["tokens"], case["cols"], case["dim"]), 1e-3, _DT[case["grad"]])
    elif op == "gate":
        T, hc, dim = case["tokens"], case["hc"], case["dim"]
        s["x"] = _normal(g, (T, hc, dim), 1.0, torch.bfloat16)
        s["kv"] = _normal(g, (T, (hc + 1) * dim), 0.5, torch.bfloat16)
        s["q"] = (1 + _normal(g, (hc, dim), 0.1, torch.float32)).to(torch.bfloat16)
        s["k"] = (1 + _normal(g, (hc, dim), 0.1, torch.float32)).to(torch.bfloat16)
        s["dout"] = _normal(g, (T, hc, dim), 1e-3, torch.bfloat16)
        s["mask"] = torch.rand(T, device=DEVICE, generator=g) >= case["masked"] if case["masked"] else None
        # what the forward saved: the gate's pre-activation
        s["dot"] = _gate_dot(s["x"], s["kv"], s["q"], s["k"])
    elif op == "wkv":
        T, K, N = case["tokens"], case["K"], case["nout"]
        s["dkv"] = _normal(g, (T, N), 1e-3, torch.bfloat16)
        s["a"] = _normal(g, (T, K), 0.1, torch.bfloat16)
        s["w"] = _normal(g, (N, K), 0.02, torch.bfloat16)
    elif op == "clip":
        s["grads"] = [_normal(_gen(seed, 1 + i), shape, 1e-2, _DT[d]) for i, (shape, d) in
                      enumerate(_clip_shapes(case))]
    else:
        raise ValueError(op)
    return s


def _gate_dot(x, kv, q, k):
    T, hc, dim = x.shape
    out = torch.empty((T, hc), dtype=torch.float32, device=DEVICE)
    for t0 in range(0, T, 2048):
        h = x[t0:t0 + 2048].float()
        key = kv[t0:t0 + 2048, :hc * dim].reshape(-1, hc, dim).float()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS) * torch.rsqrt(key.square().mean(-1) + EPS)
        out[t0:t0 + 2048] = (h * (q.float() * k.float()) * key).sum(-1) * rstd * dim ** -0.5
    return out


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gram_hash_embedding_amd as eng

    case, op = s["case"], s["op"]
    if op == "embed":
        return eng.engram_embed(s["ids"], s["table"], scale=case["scale"], out_dtype=_DT[case["out"]])
    if op == "embed_grad":
        return eng.engram_embed_grad(s["ids"], s["grad"], case["rows"], scale=case["scale"],
                                     out_dtype=_DT[case["out"]])
    if op == "embed_rows":
        ids, rows, count = eng.engram_embed_grad_rows(s["ids"], s["grad"], case["rows"], scale=case["scale"],
                                                      out_dtype=_DT[case["out"]])
        return dict(ids=ids, rows=rows, count=count)
    if op == "gate":
        dx, dkv, dq, dk = eng.engram_gate_output_backward(s["x"], s["kv"], s["q"], s["k"], EPS, s["dot"], s["dout"],
                                                          token_mask=s["mask"])
        return dict(dx=dx, dkv=dkv, dq=dq, dk=dk)
    if op == "wkv":
        da, dw = eng.engram_wkv_backward(s["dkv"], s["a"], s["w"], dw_dtype=_DT[case["dw"]])
        return dict(da=da, dw=dw)
    norm = eng.engram_grad_norm(s["grads"])
    if "outs" not in s:  # the clipped gradients' buffers, kept from step to step
        s["outs"] = [torch.empty_like(g) for g in s["grads"]]
    eng.engram_clip_grads(s["grads"], norm, case["max_norm"], outs=s["outs"])
    return dict(norm=norm, grads=s["outs"])


def _run_plain(s):
    case, op = s["case"], s["op"]
    if op == "embed":
        ids = s["ids"].long()
        ok = (ids >= 0) & (ids < case["rows"])
        rows = s["table"][torch.where(ok, ids, 0)].float() * case["scale"]
        return torch.where(ok[:, None], rows, 0.0).to(_DT[case["out"]])
    if op == "embed_grad":
        ids = s["ids"].long()
        ok = (ids >= 0) & (ids < case["rows"])
        acc = torch.zeros((case["rows"], case["dim"]), dtype=torch.float32, device=DEVICE)
        acc.index_add_(0, torch.where(ok, ids, 0), torch.where(ok[:, None], s["grad"].float(), 0.0))
        return (acc * case["scale"]).to(_DT[case["out"]])
    if op == "embed_rows":
        ids, grad = s["ids"].reshape(-1).long(), s["grad"].reshape(-1, case["dim"])
        n = ids.numel()
        key, order = torch.sort(ids, stable=True)
        head = torch.ones(n, dtype=torch.bool, device=DEVICE)
        head[1:] = key[1:] != key[:-1]
        slot = torch.cumsum(head, 0) - 1
        unique = torch.full((n,), -1, dtype=torch.int64, device=DEVICE)
        unique[slot] = key
        acc = torch.zeros((n, case["dim"]), dtype=torch.float32, device=DEVICE)
        acc.index_add_(0, slot, grad[order].float())
        return dict(ids=unique, rows=(acc * case["scale"]).to(_DT[case["out"]]), count=(slot[-1:] + 1).to(torch.int32))
    if op == "gate":
        x, kv, dout, d = s["x"].float(), s["kv"].float(), s["dout"].float(), s["dot"]
        T, hc, dim = x.shape
        w = s["q"].float() * s["k"].float()
        key, v = kv[:, :hc * dim].view(T, hc, dim), kv[:, hc * dim:]
        rh = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        rk = torch.rsqrt(key.square().mean(-1, keepdim=True) + EPS)
        z = torch.sqrt(d.abs().clamp(min=1e-6))
        g = torch.sigmoid(torch.copysign(z, d))
        dg = (dout * v[:, None, :]).sum(-1)
        ddot = torch.where(d.abs() >= 1e-6, dg * g * (1 - g) / (2 * z), 0.0)
        if s["mask"] is not None:
            ddot = torch.where(s["mask"][:, None], ddot, 0.0)
            g = torch.where(s["mask"][:, None], g, 0.0)
        ddot, g, d = ddot[..., None], g[..., None], d[..., None]
        c = rh * rk * dim ** -0.5
        dx = (dout + ddot * (c * w * key - d * rh * rh / dim * x)).to(torch.bfloat16)
        dkey = ddot * (c * w * x - d * rk * rk / dim * key)
        dkv = torch.cat([dkey.reshape(T, hc * dim), (g * dout).sum(1)], dim=1).to(torch.bfloat16)
        dw = (ddot * c * x * key).sum(0)
        return dict(dx=dx, dkv=dkv, dq=dw * s["k"].float(), dk=dw * s["q"].float())
    if op == "wkv":
        dkv = s["dkv"].float()
        return dict(da=(dkv @ s["w"].float()).to(torch.bfloat16), dw=(dkv.t() @ s["a"].float()).to(_DT[case["dw"]]))
    total = torch.stack([g.float().square().sum() for g in s["grads"]]).sum()
    norm = torch.sqrt(total).reshape(1)
    coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
    return dict(norm=norm, grads=[(g.float() * coef).to(g.dtype) for g in s["grads"]])


# ---------------------------------------------------------------------------------------------------------------------
# the bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def _distinct(n, vocab):
    """How many of n Zipf ids are distinct, on average."""
    p = np.arange(1, vocab + 1, dtype=np.float64) ** -1.1
    return float(np.sum(-np.expm1(n * np.log1p(-p / p.sum()))))


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, D = case["n"], case["dim"]
        idb = n * (4 if case["ids"] == "i32" else 8)
        if op == "embed":
            return dict(bytes=idb + _distinct(n, case["rows"]) * D * _SIZE[case["table"]] + n * D * _SIZE[case["out"]],
                        flops=n * D)
        return dict(bytes=idb + n * D * _SIZE[case["grad"]] + case["rows"] * D * _SIZE[case["out"]], flops=2 * n * D)
    if op == "embed_rows":
        n, D = case["tokens"] * case["cols"], case["dim"]
        return dict(bytes=n * ((4 if case["ids"] == "i32" else 8) + 8 + D * (_SIZE[case["grad"]] + _SIZE[case["out"]])),
                    flops=2 * n * D)
    if op == "gate":
        T, hc, dim = case["tokens"], case["hc"], case["dim"]
        return dict(bytes=T * ((5 * hc + 2) * dim * 2 + 4 * hc) + hc * dim * 12, flops=T * dim * (24 * hc + 2))
    if op == "wkv":
        T, K, N = case["tokens"], case["K"], case["nout"]
        return dict(bytes=2 * (T * N + 2 * T * K + N * K) + _SIZE[case["dw"]] * N * K, flops=4 * T * K * N)
    b = sum(2 * math.prod(shape) * _SIZE[d] for shape, d in _clip_shapes(case))
    return dict(bytes=b, flops=sum(3 * math.prod(shape) for shape, _ in _clip_shapes(case)))


# ---------------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        ids = s["ids"].long()
        table = torch.cat([s["table"], torch.zeros((1, case["dim"]), dtype=s["table"].dtype, device=DEVICE)])
        ids = torch.where((ids < 0) | (ids >= case["rows"]), case["rows"], ids)
        return torch.index_select(table, 0, ids).double().mul_(case["scale"])
    if op == "embed_grad":
        ids = s["ids"].long()
        keep = torch.nonzero((ids >= 0) & (ids < case["rows"])).flatten()
        out = torch.zeros((case["rows"], case["dim"]), dtype=torch.float64, device=DEVICE)
        out.index_put_((ids[keep],), s["grad"][keep].double() * case["scale"], accumulate=True)
        return out
    if op == "embed_rows":
        flat = s["ids"].reshape(-1).long()
        unique, slot = torch.unique(flat, sorted=True, return_inverse=True)
        out = torch.zeros((flat.numel(), case["dim"]), dtype=torch.float64, device=DEVICE)
        out.index_put_((slot,), s["grad"].reshape(-1, case["dim"]).double() * case["scale"], accumulate=True)
        return dict(ids=None, rows=out, count=None)
    if op == "gate":
        return _exact_gate(s)
    if op == "wkv":
        dkv, a, w = s["dkv"].double(), s["a"].double(), s["w"].double()
        return dict(da=torch.mm(dkv, w), dw=torch.mm(dkv.t(), a))
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return dict(norm=torch.tensor([norm], dtype=torch.float64), grads=[g.double() * coef for g in s["grads"]])


def _exact_gate(s):
    """Copy by copy: the derivative of sum(out * dout) through sigmoid(signed sqrt of the given dot), the dot and its
    two norms."""
    T, hc, dim = s["x"].shape
    live = torch.ones(T, dtype=torch.float64, device=DEVICE) if s["mask"] is None else s["mask"].double()
    v = s["kv"][:, hc * dim:].double()
    dv = torch.zeros_like(v)
    dx, dkey, dq, dk = [], [], [], []
    for c in range(hc):
        h, key, up = s["x"][:, c].double(), s["kv"][:, c * dim:(c + 1) * dim].double(), s["dout"][:, c].double()
        q, k = s["q"][c].double(), s["k"][c].double()
        d = s["dot"][:, c].double()
        root = torch.sqrt(torch.maximum(d.abs(), torch.full_like(d, 1e-6)))
        gate = live / (1 + torch.exp(torch.where(torch.signbit(d), root, -root)))
        dv += gate[:, None] * up
        slope = torch.where(s["dot"][:, c].abs() < 1e-6, 0.0, gate * (1 - gate) / (2 * root))
        e = ((up * v).sum(1) * slope)[:, None]
        mh, mk = (h * h).mean(1, keepdim=True) + EPS, (key * key).mean(1, keepdim=True) + EPS
        unit = 1 / torch.sqrt(mh * mk * dim)
        dx.append(up + e * (unit * (q * k) * key - d[:, None] * h / (mh * dim)))
        dkey.append(e * (unit * (q * k) * h - d[:, None] * key / (mk * dim)))
        both = (e * unit * h * key).sum(0)
        dq.append(both * k)
        dk.append(both * q)
    return dict(dx=torch.stack(dx, 1), dkv=torch.cat(dkey + [dv], 1), dq=torch.stack(dq), dk=torch.stack(dk))
