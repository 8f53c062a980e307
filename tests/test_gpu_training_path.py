"""A training step of the module on the tiny workload: forward, EngramForward.backward, clip_grads.  Every stage against
its float64 reference on the stage's own inputs, and the whole against the forward's differences."""
import math

import numpy as np
import pytest
import torch

import synth
import synth.workload as sw
from tests import training_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
def test_training_step(gpu_device, masked):
    from gram_hash_embedding_amd.forward import clip_grads

    cfg = synth.CONFIGS[1]
    wl = sw.build(cfg, device=gpu_device)
    fwd, x, T = wl.fwd, wl.x[0], cfg.tokens
    lw = fwd.layers[0]
    hc, dim = x.shape[-2], x.shape[-1]
    gen = torch.Generator().manual_seed(1)
    mask = (torch.rand(wl.input_ids.shape, generator=gen) < 0.7).to(gpu_device) if masked else None
    dout = (torch.randn(x.shape, generator=gen) * 0.01).to(torch.bfloat16).to(gpu_device)
    ids = fwd.hash(wl.input_ids, 0, mask)
    a, kv, dot, _ = fwd.layer(0, ids, x, token_mask=mask, output=True)
    got = fwd.backward(0, ids, x, a, kv, dot, dout, token_mask=mask)

    cpu = lambda t: t.detach().cpu()  # noqa: E731
    x3, up = cpu(x).view(T, hc, dim), cpu(dout).view(T, hc, dim)
    m = None if mask is None else cpu(mask).view(T)
    want = ref.gate_backward(x3, cpu(kv), cpu(lw.q_weight), cpu(lw.k_weight), fwd.eps, cpu(dot), up, m)
    dkv, da = cpu(fwd._bufs["dkv"]).view(T, -1), cpu(fwd._bufs["da"]).view(T, -1)
    for name, t, terms in (("dx", got.dx.view(T, hc, dim), dim + 64), ("dkv", dkv, dim + 64),
                           ("dq", got.dq, T + dim + 64), ("dk", got.dk, T + dim + 64)):
        tol = 2 * terms * ref.U32 * want[name + "_mag"] + (ref.U16 * want[name].abs() if t.dtype == torch.bfloat16 else 0)
        assert ((cpu(t).double() - want[name]).abs() <= tol + 1e-38).all(), name
    a2, w = cpu(a).view(T, -1).double(), cpu(lw.wkv).double()
    p = dkv.double()
    assert ((da.double() - p @ w).abs() <= 2 * w.shape[0] * ref.U32 * (p.abs() @ w.abs()) + ref.U16 * (p @ w).abs()).all()
    dw = p.t() @ a2
    assert ((cpu(got.dwkv).double() - dw).abs() <= 2 * T * ref.U32 * (p.abs().t() @ a2.abs()) + 2 * ref.U32 * dw.abs()).all()
    R, D = lw.weight.shape
    flat = cpu(ids).reshape(-1)
    rows, mag, n = ref.embed_grad(flat, da.reshape(-1, D), R, 0, 1.0)
    u, c = torch.unique(flat), int(got.row_count)
    assert c == u.numel() and torch.equal(cpu(got.row_ids)[:c], u) and (cpu(got.row_ids)[c:] == -1).all()
    assert ((cpu(got.rows)[:c].double() - rows[u]).abs() <= ref.sum_tolerance(rows[u], mag[u], n, False)).all()

    # the whole: along its own gradient g the loss changes by |g|^2 per unit step.  What is rounded to bf16 on the way
    # (dkv, da, dx) is off by 2^-9 of itself, so the product of the computed gradient with itself stays within a few 2^-8
    # of the true derivative along it; 2^-6 is asked for.
    g = [cpu(got.dx).view(T, hc, dim).double(), da.double(), cpu(got.dwkv).double(), cpu(got.dq).double(), cpu(got.dk).double()]
    at = [x3.double(), a2, w, cpu(lw.q_weight).double(), cpu(lw.k_weight).double()]

    def loss(vals):
        out, d = ref.gate_forward(vals[0], vals[1] @ vals[2].t(), vals[3], vals[4], fwd.eps, m)
        return float((out * up.double()).sum()), d

    for i in range(len(g)):
        norm = float(g[i].norm())
        step = 1e-7 * float(at[i].norm()) / norm  # (a step of 1e-4 carries some pre-activations over the corner at 0)
        hi, d1 = loss([v + step * g[i] if k == i else v for k, v in enumerate(at)])
        lo, d0 = loss([v - step * g[i] if k == i else v for k, v in enumerate(at)])
        assert torch.equal(torch.sign(d1), torch.sign(d0))  # no gate crosses its corner on the way
        assert abs((hi - lo) / (2 * step) / norm ** 2 - 1) < 2.0 ** -6, i

    # clipping the layer's gradients together
    tensors = got.tensors()
    before = [cpu(t).double() for t in tensors]
    total = math.sqrt(sum(float(t.square().sum()) for t in before))
    norm = clip_grads(tensors, total / 3)
    assert abs(float(norm) / total - 1) < 4 * ref.U32
    for t, b in zip(tensors, before):
        assert np.allclose(cpu(t).numpy(), b.numpy() / 3, rtol=1e-5, atol=0)
