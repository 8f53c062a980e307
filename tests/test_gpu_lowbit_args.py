"""Arguments of the narrow formats' entry points that may be left out in part."""
import pytest
import torch

import gram_hash_embedding_amd as g
from tests.test_gpu_lowbit import EPS, _gate_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [(), ("x", "x_scale"), ("kv",), ("x_scale", "kv_scale"), ("x", "x_scale", "kv", "kv_scale")])
def test_a_checkpoint_given_in_part(gpu_device, given):
    """The tensors that are not given are allocated and returned, and the gradient takes what was returned."""
    x, kv, q, k, mask, dout = _gate_case(37, 3, 264, gpu_device)
    _, dot, want = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    held = g.GateCheckpoint(*[torch.empty_like(t) if name in given else None for name, t in zip(want._fields, want)])
    for checkpoint in (held, tuple(held)):
        c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask, checkpoint=checkpoint)[2]
        assert isinstance(c, g.GateCheckpoint)
        for name, t, own, r in zip(want._fields, c, held, want):
            assert torch.equal(t, r) and (name not in given or t is own), name
        for a, b in zip(g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout, mask),
                        g.engram_gate_output_backward_ckpt(want, q, k, EPS, dot, dout, mask)):
            assert torch.equal(a, b)
    with pytest.raises(ValueError, match="checkpoint"):
        g.engram_gate_output_backward_ckpt(want._replace(kv=None), q, k, EPS, dot, dout, mask)
