"""The narrow formats through the module's own path: EngramForward.step on 4-bit weights, and a training step of a layer whose
backward reads 8-bit checkpoints."""
import dataclasses

import pytest
import torch

import gram_hash_embedding_amd as g
import synth
import synth.workload as sw

pytestmark = pytest.mark.gpu

# the tiny workload with rows of 64, so that a token's row is 6 x 64 = 384 columns (whole steps of 128), and two layers of it
CFG = dataclasses.replace(synth.CONFIGS[1], head_dim=64)


def _workload(dev):
    wl = sw.build(CFG, device=dev, packed=True)
    for lw in wl.fwd.layers:
        lw.wkv_mx4 = g.engram_mx4_pack_weight(*g.engram_mx4_quant(lw.wkv))
    return wl


def _copy(ts):
    return [t.clone() for t in ts]


@pytest.mark.parametrize("a_bits", [8, 4])
def test_step_on_4_bit_weights(gpu_device, a_bits):
    """Each form of the step is the entry points called one after the other; the forms agree on the value columns bit for bit."""
    wl = _workload(gpu_device)
    fwd, x, ids0 = wl.fwd, wl.x[0], wl.input_ids
    T, hc, dim = CFG.tokens, CFG.hc_mult, CFG.dim
    lw = fwd.layers[0]
    ids = fwd.hash(ids0, 0, wl.token_mask)
    rows = g.engram_gather_dequant(ids, lw.weight, lw.scale, lw.block_size, layer=0).view(T, -1)
    aq, asc = (g.engram_mx_quant if a_bits == 8 else g.engram_mx4_quant)(rows)
    kv = g.engram_wkv_mx4(aq, asc, lw.wkv_mx4)
    x3 = x.reshape(T, hc, dim)
    want_dot = g.engram_gate_dot(x3, kv, lw.q_weight, lw.k_weight, fwd.eps)
    want_out = g.engram_gate_output(x, kv, lw.q_weight, lw.k_weight, fwd.eps, wl.token_mask)
    plain = _copy(fwd.step(ids0, 0, x, wl.token_mask, fp4=True, a_bits=a_bits))
    assert torch.equal(plain[0], want_dot)
    out = _copy(fwd.step(ids0, 0, x, wl.token_mask, fp4=True, a_bits=a_bits, output=True))
    assert torch.equal(out[0], want_out)
    value, dot = g.engram_wkv_mx4_gate(aq, asc, lw.wkv_mx4, x3, lw.q_weight, lw.k_weight, fwd.eps)
    assert torch.equal(value, kv[:, hc * dim:])
    for kw in (dict(), dict(hash_gather=True), dict(packed=True)) + ((dict(gather_mx=True, packed=True), dict(gather_mx=True))
                                                                     if a_bits == 8 else ()):
        got = _copy(fwd.step(ids0, 0, x, wl.token_mask, fp4=True, a_bits=a_bits, fused=True, **kw))
        assert torch.equal(got[0], dot), kw
        got = _copy(fwd.step(ids0, 0, x, wl.token_mask, fp4=True, a_bits=a_bits, fused=True, output=True, **kw))
        assert torch.equal(got[0], g.engram_gate_residual(x, value, dot, wl.token_mask)), kw


def test_step_refusals(gpu_device):
    wl = _workload(gpu_device)
    fwd, x = wl.fwd, wl.x[0]
    for kw in (dict(fp8=True), dict(all_layers=True, fused=True), dict(a_bits=4, gather_mx=True), dict(a_bits=6)):
        with pytest.raises(ValueError):
            fwd.step(wl.input_ids, 0, x, wl.token_mask, fp4=True, **kw)
    fwd.layers[0].wkv_mx4 = None
    with pytest.raises(ValueError, match="4-bit"):
        fwd.step(wl.input_ids, 0, x, wl.token_mask, fp4=True)
    ids = fwd.hash(wl.input_ids, 0, wl.token_mask)
    for kw in (dict(), dict(output=True, fused=True)):
        with pytest.raises(ValueError, match="checkpoint"):
            fwd.layer(0, ids, x, checkpoint=True, **kw)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_training_step_with_checkpoints(gpu_device, masked, packed):
    """Two micro-batches, both forwards before either backward: every gradient is that of the ordinary path on the values that
    the checkpoints stand for."""
    wl = _workload(gpu_device)
    fwd, T, hc, dim = wl.fwd, CFG.tokens, CFG.hc_mult, CFG.dim
    gen = torch.Generator().manual_seed(3)
    lw = fwd.layers[0]
    held = []
    for step in range(2):
        x = torch.randn((*wl.input_ids.shape, hc, dim), generator=gen).to(torch.bfloat16).to(gpu_device)
        tokens = torch.randint(0, CFG.vocab_size, wl.input_ids.shape, generator=gen).to(gpu_device)
        mask = (torch.rand(wl.input_ids.shape, generator=gen) < 0.7).to(gpu_device) if masked else None
        ids = fwd.hash(tokens, 0, mask).clone()
        a, kv, dot, out = _copy(fwd.layer(0, ids, x, token_mask=mask, output=True))
        ck, got = fwd.layer(0, ids, x, token_mask=mask, output=True, checkpoint=True, packed=packed)
        # the dot's sums are in another order: the outputs may be a step of bf16 apart, and no more
        assert ((got.double() - out.double()).abs() <= 2.0 ** -7 * out.double().abs() + 2.0 ** -9 * kv.double().abs().max()).all()
        held.append((x, ids, mask, a, ck, (torch.randn(x.shape, generator=gen) * 0.01).to(torch.bfloat16).to(gpu_device)))
    for x, ids, mask, a, ck, dout in held:
        grads = fwd.backward(0, ids, dout=dout, token_mask=mask, checkpoint=ck, packed=packed)
        got = _copy([grads.dx, *grads.tensors(), grads.row_ids, grads.row_count])
        xl = g.engram_ckpt_load(ck.rows.x, ck.rows.x_scale).view(x.shape)
        kvl = g.engram_ckpt_load(ck.rows.kv, ck.rows.kv_scale).view(T, -1)
        want = fwd.backward(0, ids, xl, a, kvl, ck.dot, dout, token_mask=mask)
        for p, r in zip(got, [want.dx, *want.tensors(), want.row_ids, want.row_count]):
            assert torch.equal(p, r)
    with pytest.raises(ValueError, match="dout"):
        fwd.backward(0, held[0][1], checkpoint=held[0][4])
