"""Training steps with 8-bit checkpoints as a loop runs them: the ids as `hash` and `hash_gather` return them, several
micro-batches between their forwards and their backwards, and batches without tokens."""
import dataclasses

import pytest
import torch

import gram_hash_embedding_amd as g
import synth
import synth.workload as sw
from tests.test_gpu_lowbit_path import _copy

pytestmark = pytest.mark.gpu

CFG = dataclasses.replace(synth.CONFIGS[1], n_layers=2, rows_alloc=(9670, 10000))


@pytest.mark.parametrize("gathered", [False, True])
def test_micro_batches_with_the_ids_of_hash(gpu_device, gathered):
    """Three micro-batches, every forward before any backward, in every layer: the ids lie in a buffer that the next `hash` fills,
    and each gradient is still that of its own ids, as from copies of them."""
    wl = sw.build(CFG, device=gpu_device, packed=True)
    fwd, hc, dim = wl.fwd, CFG.hc_mult, CFG.dim
    gen = torch.Generator().manual_seed(5)
    held = []
    for _ in range(3):
        tokens = torch.randint(0, CFG.vocab_size, wl.input_ids.shape, generator=gen).to(gpu_device)
        x = torch.randn((*tokens.shape, hc, dim), generator=gen).to(torch.bfloat16).to(gpu_device)
        dout = (torch.randn(x.shape, generator=gen) * 0.01).to(torch.bfloat16).to(gpu_device)
        if gathered:
            ids, rows = fwd.hash_gather(tokens, 0)
        else:
            ids, rows = fwd.hash(tokens, 0), [None] * fwd.E
        own = ids.clone()
        ck = [fwd.layer(e, ids, x, output=True, a=rows[e], checkpoint=True)[0] for e in range(fwd.E)]
        held.append((ids, own, dout, ck))
    assert CFG.n_layers == 2 and not torch.equal(held[0][1], held[1][1])
    for ids, own, dout, ck in reversed(held):
        for e in range(fwd.E):
            got = fwd.backward(e, ids, dout=dout, checkpoint=ck[e])
            got = _copy([got.dx, *got.tensors(), got.row_ids, got.row_count])
            a = fwd.gather(e, own).clone()
            kvl = g.engram_ckpt_load(ck[e].rows.kv, ck[e].rows.kv_scale).view(dout.shape[0] * dout.shape[1], -1)
            xl = g.engram_ckpt_load(ck[e].rows.x, ck[e].rows.x_scale).view(dout.shape)
            want = fwd.backward(e, own, xl, a, kvl, ck[e].dot, dout)
            for p, r in zip(got, [want.dx, *want.tensors(), want.row_ids, want.row_count]):
                assert torch.equal(p, r), e


@pytest.mark.parametrize("shape", [(1, 0), (0, 7)])
def test_a_batch_without_tokens(gpu_device, shape):
    """Every form of the path takes one: nothing is kept, the weights' gradients are zeros and no row is reached."""
    cfg = dataclasses.replace(CFG, head_dim=64)
    wl = sw.build(cfg, device=gpu_device, packed=True)
    fwd, hc, dim = wl.fwd, cfg.hc_mult, cfg.dim
    for lw in fwd.layers:
        lw.wkv_mx4 = g.engram_mx4_pack_weight(*g.engram_mx4_quant(lw.wkv))
    tokens = torch.empty(shape, dtype=torch.int64, device=gpu_device)
    x = torch.empty((*shape, hc, dim), dtype=torch.bfloat16, device=gpu_device)
    for kw in (dict(), dict(fused=True), dict(hash_gather=True), dict(fused=True, all_layers=True), dict(fp4=True),
               dict(fp4=True, fused=True), dict(fp4=True, a_bits=4), dict(fp4=True, fused=True, gather_mx=True)):
        for t in fwd.step(tokens, 0, x, output=True, **kw):
            assert t.shape == x.shape, kw
    ids = fwd.hash(tokens, 0)
    a, kv, dot, out = fwd.layer(0, ids, x, output=True)
    ck, got = fwd.layer(0, ids, x, output=True, checkpoint=True)
    assert out.shape == got.shape == x.shape and ck.rows.x.shape == (0, hc, dim) and ck.rows.kv.shape == (0, hc + 1, dim)
    for grads in (fwd.backward(0, ids, x, a, kv, dot, x), fwd.backward(0, None, dout=x, checkpoint=ck)):
        assert grads.dx.shape == x.shape and int(grads.row_count) == 0 and grads.row_ids.numel() == grads.rows.numel() == 0
        assert not grads.dwkv.any() and not grads.dq.any() and not grads.dk.any()
