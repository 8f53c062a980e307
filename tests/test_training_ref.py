"""The float64 reference of the gate's gradient against central differences of the forward, and the host-side refusals
of the training entry points (statuses come back before anything is enqueued, so no device is touched)."""
import ctypes

import pytest
import torch

import gram_hash_embedding_amd as g
from tests import training_ref as ref

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x100002)


@pytest.mark.parametrize("hc,dim,masked", [(1, 8, False), (4, 16, True), (3, 24, False)])
def test_gate_gradient_against_differences(hc, dim, masked):
    """Central differences with step 1e-6 in float64: truncation ~1e-12 of the third derivative, rounding ~1e-16 / 1e-6
    of a sum of about a hundred terms of order one -- together well under 1e-7 against gradients of order 0.01 to 1."""
    gen = torch.Generator().manual_seed(hc * 100 + dim)
    T, eps = 5, 1e-3
    r = lambda *s: torch.randn(*s, dtype=torch.float64, generator=gen)  # noqa: E731
    x, kv, q, k, up = r(T, hc, dim), r(T, (hc + 1) * dim), 1 + 0.1 * r(hc, dim), 1 + 0.1 * r(hc, dim), r(T, hc, dim)
    mask = torch.tensor([1, 0, 1, 1, 0]) if masked else None
    loss = lambda *a: float((ref.gate_forward(*a, eps, mask)[0] * up).sum())  # noqa: E731
    dot = ref.gate_forward(x, kv, q, k, eps, mask)[1]
    assert float(dot.abs().min()) > 1e-4  # away from the clamp, where the function has a corner
    got = ref.gate_backward(x, kv, q, k, eps, dot, up, mask)
    args = [x, kv, q, k]
    for which, name in enumerate(("dx", "dkv", "dq", "dk")):
        flat = args[which].reshape(-1)
        for i in torch.randperm(flat.numel(), generator=gen)[:40].tolist():
            keep = float(flat[i])
            flat[i] = keep + 1e-6
            hi = loss(*args)
            flat[i] = keep - 1e-6
            lo = loss(*args)
            flat[i] = keep
            assert abs((hi - lo) / 2e-6 - float(got[name].reshape(-1)[i])) < 1e-7 + 1e-7 * abs(float(got[name].reshape(-1)[i]))


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    """sum(up * table[ids] * scale) is linear in the table: its derivative against the reference, entry by entry."""
    gen = torch.Generator().manual_seed(3)
    ids = torch.randint(-2, 9, (40,), generator=gen)
    up = torch.randn(40, 8, dtype=torch.float64, generator=gen)
    got, _, _ = ref.embed_grad(ids, up, 7, 0, 2.5)
    for r in range(7):
        want = 2.5 * up[ids == r].sum(0)
        assert torch.allclose(got[r], want, rtol=1e-13, atol=1e-13)


def _err():
    return g.lib().engram_last_error().decode()


@pytest.mark.parametrize("args,status,msg", [
    (dict(D=12), 1, "multiple of 8"), (dict(D=0), 1, "multiple of 8"), (dict(D=65544), 1, "multiple of 8"),
    (dict(n=-1), 1, "n < 0"), (dict(R=0), 1, "R < 1"), (dict(id_bytes=2), 1, "id_bytes"),
    (dict(td=2), 1, "dtype"), (dict(od=-1), 1, "dtype"), (dict(ids=None), 1, "null"), (dict(table=None), 1, "null"),
    (dict(out=None), 1, "null"), (dict(table=ODD), 1, "misaligned"), (dict(out=ODD), 1, "misaligned"),
    (dict(ids=ODD), 1, "misaligned"), (dict(n=0, ids=None, table=None, out=None), 0, None),
])
def test_embed_validation(args, status, msg):
    a = dict(ids=FAKE, id_bytes=8, n=4, table=FAKE, td=0, R=10, D=64, out=FAKE, od=0)
    a.update(args)
    rc = g.lib().engram_embed(a["ids"], a["id_bytes"], a["n"], a["table"], a["td"], a["R"], 0, a["D"], 1.0, a["out"],
                              a["od"], None)
    assert rc == status
    assert msg is None or msg in _err()


@pytest.mark.parametrize("rows_form", [False, True])
@pytest.mark.parametrize("args,status,msg", [
    (dict(D=12), 1, "multiple of 8"), (dict(T=-1), 1, "T < 0"), (dict(C=0), 1, "C=0"), (dict(C=1025, stride=1025), 1, "C=1025"),
    (dict(stride=5), 1, "stride"), (dict(T=1 << 28), 1, "2^30"), (dict(R=0), 1, "R=0"), (dict(R=1 << 31), 1, "R="),
    (dict(id_bytes=3), 1, "id_bytes"), (dict(gd=7), 1, "dtype"), (dict(od=2), 1, "dtype"), (dict(ids=None), 1, "null"),
    (dict(up=None), 1, "null"), (dict(out=None), 1, "null"), (dict(ws=None), 1, "workspace"), (dict(up=ODD), 1, "misaligned"),
    (dict(out=ODD), 1, "misaligned"), (dict(ws=ODD), 1, "misaligned"), (dict(wn=100), 2, "workspace"),
])
def test_embed_grad_validation(args, status, msg, rows_form):
    a = dict(ids=FAKE, id_bytes=8, T=1000, stride=6, C=6, up=FAKE, gd=0, R=1000, D=64, out=FAKE, od=1, ws=FAKE, wn=1 << 30)
    a.update(args)
    head = (a["ids"], a["id_bytes"], a["T"], a["stride"], a["C"], a["up"], a["gd"], a["R"], 0, a["D"], 1.0)
    if rows_form:
        rc = g.lib().engram_embed_grad_rows(*head, FAKE, a["out"], a["od"], FAKE, a["ws"], a["wn"], None)
    else:
        rc = g.lib().engram_embed_grad(*head, a["out"], a["od"], 0, a["ws"], a["wn"], None)
    assert rc == status and msg in _err()


def test_workspace_sizes_outside_the_limits():
    L = g.lib()
    assert L.engram_embed_grad_workspace_bytes(0, 64, 10) == 0
    for n, D, R in ((-1, 64, 10), (1 << 31, 64, 10), (10, 4, 10), (10, 64, 0), (10, 64, 1 << 31)):
        assert L.engram_embed_grad_workspace_bytes(n, D, R) == -1
    assert L.engram_gate_output_backward_workspace_bytes(0, 4, 64) == 0
    for T, hc, dim in ((-1, 4, 64), (1, 0, 64), (1, 65, 64), (1, 4, 4), (1, 4, 8200)):
        assert L.engram_gate_output_backward_workspace_bytes(T, hc, dim) == -1
    for T, K, N in ((-1, 8, 8), (1, 4, 8), (1, 8, 12), (1, 8, 1 << 22)):
        assert L.engram_wkv_backward_workspace_bytes(T, K, N) == -1


@pytest.mark.parametrize("args,status,msg", [
    (dict(T=-1), 1, "T < 0"), (dict(hc=0), 1, "hc=0"), (dict(hc=65), 1, "hc=65"), (dict(dim=12), 1, "dim=12"),
    (dict(dim=8200), 1, "dim=8200"), (dict(ld=1272), 1, "ld_kv"), (dict(ld=1281), 1, "ld_kv"), (dict(x=None), 1, "null"),
    (dict(kv=None), 1, "null"), (dict(q=None), 1, "null"), (dict(dot=None), 1, "null"), (dict(dout=None), 1, "null"),
    (dict(dx=None), 1, "null"), (dict(dkv=None), 1, "null"), (dict(dq=None), 1, "null"), (dict(ws=None), 1, "null"),
    (dict(x=ODD), 1, "misaligned"), (dict(dx=ODD), 1, "misaligned"), (dict(dq=ODD), 1, "misaligned"), (dict(wn=16), 2, "workspace"),
])
def test_gate_backward_validation(args, status, msg):
    a = dict(x=FAKE, kv=FAKE, ld=1280, q=FAKE, k=FAKE, dot=FAKE, dout=FAKE, dx=FAKE, dkv=FAKE, dq=FAKE, dk=FAKE, ws=FAKE,
             wn=1 << 30, T=10, hc=4, dim=256)
    a.update(args)
    rc = g.lib().engram_gate_output_backward(a["x"], a["kv"], a["ld"], a["q"], a["k"], 1e-20, a["dot"], a["dout"], None,
                                             a["dx"], a["dkv"], a["dq"], a["dk"], a["ws"], a["wn"], a["T"], a["hc"], a["dim"],
                                             None)
    assert rc == status and msg in _err()


@pytest.mark.parametrize("args,status,msg", [
    (dict(T=-1), 1, "T outside"), (dict(K=12), 1, "K=12"), (dict(N=12), 1, "Nout=12"), (dict(dt=3), 1, "dtype"),
    (dict(da=None, dw=None), 1, "neither"), (dict(dkv=None), 1, "null"), (dict(a=None), 1, "null"), (dict(w=None), 1, "null"),
    (dict(dkv=ODD), 1, "misaligned"), (dict(dw=ODD), 1, "misaligned"), (dict(da=ODD), 1, "misaligned"),
    (dict(ws=None), 1, "workspace"), (dict(wn=16), 2, "workspace"),
])
def test_wkv_backward_validation(args, status, msg):
    a = dict(dkv=FAKE, a=FAKE, w=FAKE, da=FAKE, dw=FAKE, dt=1, ws=FAKE, wn=1 << 40, T=64, K=64, N=25600)
    a.update(args)
    rc = g.lib().engram_wkv_backward(a["dkv"], a["a"], a["w"], a["da"], a["dw"], a["dt"], 0, a["ws"], a["wn"], a["T"], a["K"],
                                     a["N"], None)
    assert rc == status and msg in _err()


def _list(n=2, ptr=0x100000, size=100, dtype=1):
    return ((ctypes.c_void_p * n)(*[ptr] * n), (ctypes.c_int64 * n)(*[size] * n), (ctypes.c_int32 * n)(*[dtype] * n))


def test_norm_and_clip_validation():
    L = g.lib()
    p, n, d = _list()
    assert L.engram_grad_norm_workspace_bytes(2, n, d) == 16
    assert L.engram_grad_norm(-1, p, n, d, FAKE, FAKE, 16, None) == 1 and "tensors < 0" in _err()
    assert L.engram_grad_norm(2, None, n, d, FAKE, FAKE, 16, None) == 1 and "null list" in _err()
    assert L.engram_grad_norm(2, p, n, d, None, FAKE, 16, None) == 1 and "norm" in _err()
    assert L.engram_grad_norm(2, p, n, d, FAKE, None, 16, None) == 1 and "workspace" in _err()
    assert L.engram_grad_norm(2, p, n, d, FAKE, FAKE, 8, None) == 2 and "workspace" in _err()
    for bad, msg in ((_list(dtype=4), "dtype"), (_list(size=-1), "size"), (_list(ptr=0), "null pointer"),
                     (_list(ptr=0x100002), "misaligned")):
        assert L.engram_grad_norm(2, *bad, FAKE, FAKE, 16, None) == 1 and msg in _err()
        assert L.engram_clip_grads(2, bad[0], bad[0], bad[1], bad[2], FAKE, 1.0, None) == 1 and msg in _err()
    assert L.engram_clip_grads(2, p, p, n, d, None, 1.0, None) == 1 and "norm" in _err()
    assert L.engram_clip_grads(2, p, None, n, d, FAKE, 1.0, None) == 1 and "null list" in _err()
    assert L.engram_clip_grads(2, p, p, n, d, FAKE, -1.0, None) == 1 and "max_norm" in _err()
    assert L.engram_clip_grads(2, p, p, n, d, FAKE, float("nan"), None) == 1 and "max_norm" in _err()
    assert L.engram_clip_grads(2, p, _list(ptr=0)[0], n, d, FAKE, 1.0, None) == 1 and "output 0" in _err()
    assert L.engram_clip_grads(0, None, None, None, None, None, 1.0, None) == 0


class _Addresses:
    """Stands in for a call's device: takes any ids."""

    def ids(self, ids):
        return ids.data_ptr(), ids.element_size()


@pytest.mark.parametrize("tokens", [(0, 7), (3, 0), (2, 7)])
@pytest.mark.parametrize("C,D", [(6, 32), (24, 64), (1, 8)])
def test_rows_of_a_layers_gradient(tokens, C, D):
    """[B*L, C, D], [B, L, C, D] and [B*L, C*D] are all rows of D, for an empty batch too."""
    from gram_hash_embedding_amd import training

    training._load()
    (B, L), E = tokens, 3
    T = B * L
    ids = torch.zeros((B, L, E, C), dtype=torch.int64)
    for shape in ((T, C, D), (B, L, C, D), (T, C * D)):
        ip, ib, t, stride, c, n, d = training._lookup(_Addresses(), ids, torch.zeros(shape), 1)
        assert (t, stride, c, n, d) == (T, E * C, C, T * C, D), shape
        assert ip == ids.data_ptr() + 8 * C and ib == 8


def test_rows_of_a_layers_gradient_that_do_not_divide():
    from gram_hash_embedding_amd import training

    training._load()
    ids = torch.zeros((2, 7, 1, 6), dtype=torch.int64)
    with pytest.raises(ValueError, match="row of D elements"):
        training._lookup(_Addresses(), ids, torch.zeros((14, 6 * 32 + 8)), 0)
