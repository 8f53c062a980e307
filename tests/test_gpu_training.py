"""The training entry points against float64 references (tests/training_ref.py).  Tolerances are worst-case bounds of
float32 sums of the case's length, plus one rounding to the output's type."""
import math

import numpy as np
import pytest
import torch

from tests import training_ref as ref
from tests.gpu_util import bits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def _eng():
    import gram_hash_embedding_amd as g

    return g


def _within(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = (got - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max()):.3g} over"


def _randn(gen, shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


# ---------------------------------------------------------------------------------------------------------------------
# lookup
# ---------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("tdt,odt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("n,R,D,idt,row_start", [
    (1, 1, 8, torch.int64, 0), (7, 50, 24, torch.int32, 0), (257, 33, 72, torch.int64, 1000), (65, 100, 136, torch.int32, -3),
    (300, 40, 520, torch.int64, 0), (5, 9, 5120, torch.int64, 2)])
def test_embed(gpu_device, tdt, odt, n, R, D, idt, row_start):
    gen = torch.Generator().manual_seed(n + D)
    table = _randn(gen, (R, D), tdt)
    table[0, 0] = math.inf
    table[R - 1, D - 1] = NAN
    ids = torch.randint(-2, R + 2, (n,), generator=gen) + row_start
    ids[0] = row_start + R - 1
    if n > 2:
        ids[1], ids[2] = row_start + R, torch.iinfo(idt).min
    out = _eng().engram_embed(ids.to(idt).to(gpu_device), table.to(gpu_device), scale=1.7, row_start=row_start, out_dtype=odt)
    r = ids - row_start
    ok = (r >= 0) & (r < R)
    want = torch.where(ok[:, None], table[torch.where(ok, r, 0)].float() * torch.tensor(1.7, dtype=F32), 0.0).to(odt)
    assert out.dtype == odt
    assert torch.equal(out.cpu().isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(out.cpu().float()), torch.nan_to_num(want.float()))


# (n, D) of at least 2^24 elements, from where a thread takes four rows; odd counts, every width's kernel; the last of each
# width over 256 MB of output, which passes the caches
@pytest.mark.parametrize("tdt,odt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("n,D", [
    (699051, 24), (262145, 64), (2100003, 64), (233017, 72), (1048579, 128), (131073, 136), (550001, 256), (32767, 512),
    (32768, 512), (63551, 264), (290003, 520), (3283, 5120), (30001, 5120), (2047, 8200), (17001, 8200)])
def test_embed_of_many_rows(gpu_device, n, D, tdt, odt):
    g, R = _eng(), 1003
    gen = torch.Generator(device=gpu_device).manual_seed(n)
    table = torch.empty((R, D), device=gpu_device).normal_(generator=gen).to(tdt)
    ids = torch.randint(-1, R + 1, (n,), generator=gen, device=gpu_device)
    out = torch.full((n + 7, D), NAN, dtype=odt, device=gpu_device)
    g.engram_embed(ids, table, scale=1.7, out=out[:n])
    assert out[n:].isnan().all()
    want = (torch.cat([table, torch.zeros((1, D), dtype=tdt, device=gpu_device)]).float() * torch.tensor(1.7)).to(odt)
    r = torch.where((ids < 0) | (ids >= R), R, ids)
    for i in range(0, n, 1 << 18):
        assert torch.equal(out[:n][i:i + (1 << 18)], want[r[i:i + (1 << 18)]]), i


def test_embed_shapes_and_refusals(gpu_device):
    g = _eng()
    table = torch.ones((4, 16), dtype=BF, device=gpu_device)
    ids = torch.zeros((2, 3), dtype=torch.int64, device=gpu_device)
    assert g.engram_embed(ids, table).shape == (2, 3, 16)
    assert g.engram_embed(ids[:0], table).shape == (0, 3, 16)
    with pytest.raises(TypeError):
        g.engram_embed(ids.float(), table)
    with pytest.raises(TypeError):
        g.engram_embed(ids, table.half())
    with pytest.raises(ValueError):
        g.engram_embed(ids, table.t())
    with pytest.raises(ValueError):
        g.engram_embed(ids.cpu(), table)
    with pytest.raises(ValueError):
        g.engram_embed(ids, table, out=torch.empty((2, 3, 8), dtype=BF, device=gpu_device))
    with pytest.raises(g.EngramError):
        g.engram_embed(ids, torch.ones((4, 12), dtype=BF, device=gpu_device))


# ---------------------------------------------------------------------------------------------------------------------
# its gradient
# ---------------------------------------------------------------------------------------------------------------------
def _ids_of(kind, n, R, gen):
    if kind == "one":
        return torch.full((n,), R // 2)
    if kind == "distinct":
        return torch.randperm(max(R, n), generator=gen)[:n]
    if kind == "runs":  # runs of 1 to 40 positions of one row, shuffled
        out = torch.repeat_interleave(torch.randperm(n, generator=gen) % R, torch.randint(1, 41, (n,), generator=gen))[:n]
        return out[torch.randperm(n, generator=gen)]
    if kind == "outside":
        return torch.where(torch.rand(n, generator=gen) < 0.5, -1 - torch.arange(n), R + torch.arange(n))
    ids = (R * torch.rand(n, generator=gen).double() ** 3).long()
    ids[torch.rand(n, generator=gen) < 0.1] = R
    return ids


def _both_forms(g, ids, up, R, D, dev, gdt, odt, row_start=0, scale=1.0):
    dense = g.engram_embed_grad(ids, up, R, scale=scale, row_start=row_start, out_dtype=odt)
    unique, rows, count = g.engram_embed_grad_rows(ids, up, R, scale=scale, row_start=row_start, out_dtype=odt)
    return dense, unique, rows, count


def _check_grad(g, ids, up, R, D, dev, odt, row_start=0, scale=1.0, what=""):
    n = ids.numel()
    idd, upd = ids.to(dev), up.to(dev)
    want, mag, m = ref.embed_grad(ids, up, R, row_start, scale)
    tol = ref.sum_tolerance(want, mag, m, odt == BF)
    dense, unique, rows, count = _both_forms(g, idd, upd, R, D, dev, up.dtype, odt, row_start, scale)
    _within(dense, want, tol, what + " dense")
    r = ids.long() - row_start
    u = torch.unique(r[(r >= 0) & (r < R)])
    c = int(count)
    assert c == u.numel(), (what, c, u.numel())
    assert torch.equal(unique.cpu()[:c], u + row_start) and (unique.cpu()[c:] == -1).all(), what
    # the two forms give the same bits
    assert torch.equal(rows.cpu()[:c], dense.cpu()[u]), what
    assert not rows.cpu()[c:].any(), what
    again = g.engram_embed_grad(idd, upd, R, scale=scale, row_start=row_start, out_dtype=odt)
    assert torch.equal(again, dense), what


@pytest.mark.parametrize("kind", ["one", "distinct", "runs", "outside", "zipf"])
@pytest.mark.parametrize("n,R,D,gdt,odt", [
    (1, 1, 8, BF, F32), (15, 40, 24, F32, F32), (16, 16, 32, BF, BF), (17, 300, 64, F32, BF), (511, 700, 72, BF, F32),
    (1025, 1100, 136, BF, F32), (4095, 5000, 8, F32, F32), (4096, 70000, 16, BF, F32), (4097, 1030, 264, BF, BF),
    (9001, 9001, 520, BF, F32)])
def test_embed_grad(gpu_device, kind, n, R, D, gdt, odt):
    gen = torch.Generator().manual_seed(n * 7 + D)
    ids = _ids_of(kind, n, R, gen)
    _check_grad(_eng(), ids, _randn(gen, (n, D), gdt), R, D, gpu_device, odt, scale=3.0, what=f"{kind} {n}")


@pytest.mark.parametrize("kind", ["one", "runs", "zipf"])
@pytest.mark.parametrize("n", [1024, 2047, 2049, 8191, 8192, 8193])
def test_embed_grad_at_the_sorts_edges(gpu_device, n, kind):
    """Where one launch, one sorting workgroup and the sort over tiles hand over."""
    gen = torch.Generator().manual_seed(n)
    for R in (3, 300, 70000):
        _check_grad(_eng(), _ids_of(kind, n, R, gen), _randn(gen, (n, 16), BF), R, 16, gpu_device, F32, what=f"{kind} {R}")


@pytest.mark.parametrize("n,R,D,kind", [(270000, 3988006, 8, "zipf"), (300001, 129280, 8, "runs"), (262144, 513, 8, "one")])
def test_embed_grad_many_tiles(gpu_device, n, R, D, kind):
    gen = torch.Generator().manual_seed(n)
    _check_grad(_eng(), _ids_of(kind, n, R, gen), _randn(gen, (n, D), BF), R, D, gpu_device, F32, what=kind)


@pytest.mark.parametrize("kind", ["one", "distinct", "runs", "zipf"])
@pytest.mark.parametrize("n,R,D", [
    (512, 90, 16), (513, 90, 16), (512, 3988006, 8), (513, 3988006, 8), (524288, 60000, 8), (524289, 60000, 8),
    (600001, 3988006, 8), (786433, 700, 8)])
def test_embed_grad_where_its_forms_hand_over(gpu_device, n, R, D, kind):
    """512 ids: one launch; 524,288: tiles of four ids a thread, past that eight."""
    gen = torch.Generator().manual_seed(n + 1)
    ids = _ids_of(kind, n, R, gen)
    _check_grad(_eng(), ids, _randn(gen, (n, D), BF), R, D, gpu_device, F32, what=kind)


@pytest.mark.parametrize("gdt,odt", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("n,R,D", [(1400003, 50001, 32), (700001, 30001, 64), (355003, 90001, 128), (131101, 20001, 256),
                                   (131101, 20001, 264)])
def test_embed_grad_past_the_caches(gpu_device, n, R, D, gdt, odt):
    """More than 256 MB moved: upstream and finished rows pass the caches, in both forms, for every count of lanes a row has.
    References on the GPU, in 64 bits."""
    g = _eng()
    gen = torch.Generator(device=gpu_device).manual_seed(n)
    ids = (R * torch.rand(n, generator=gen, device=gpu_device).double() ** 3).long()
    ids[::17] = R
    up = torch.empty((n, D), device=gpu_device).normal_(generator=gen).to(gdt)
    want = torch.zeros((R + 1, D), dtype=torch.float64, device=gpu_device)
    mag = torch.zeros_like(want)
    want.index_add_(0, ids, up.double())
    mag.index_add_(0, ids, up.double().abs())
    want, mag = want[:R], mag[:R]
    tol = ref.sum_tolerance(want, mag, int(torch.bincount(ids)[:R].max()), odt == BF)
    dense = g.engram_embed_grad(ids, up, R, out_dtype=odt)
    assert ((dense.double() - want).abs() <= tol).all()
    unique, rows, count = g.engram_embed_grad_rows(ids, up, R, out_dtype=odt)
    u, c = torch.unique(ids[ids < R]), int(count)
    assert c == u.numel() and torch.equal(unique[:c], u) and (unique[c:] == -1).all()
    assert torch.equal(rows[:c], dense[u]) and not rows[c:].any()


@pytest.mark.parametrize("n", [100, 3000, 9000])
def test_embed_grad_of_more_zeros_than_a_grid_holds(gpu_device, n):
    """34.6 GB of gradient: what is past 32 GiB has a launch of its own, in each of the three forms."""
    g, R, D = _eng(), 135000003, 64
    pick = torch.tensor([0, 1, 134217727, 134217728, 134217729, R - 2, R - 1], device=gpu_device)
    ids = pick.repeat(n)[:n]
    up = torch.ones((n, D), dtype=BF, device=gpu_device)
    grad = torch.full((R, D), NAN, device=gpu_device)
    g.engram_embed_grad(ids, up, R, out=grad)
    assert torch.equal(grad[pick, 0], torch.bincount(ids)[pick].float())
    assert (grad[pick] == grad[pick, :1]).all()
    grad[pick] = 0
    for i in range(0, R, 1 << 24):
        assert not grad[i:i + (1 << 24)].any(), i


@pytest.mark.parametrize("n", [3, 900, 5000, 280000])
@pytest.mark.parametrize("R", [(1 << 31) - 1, 384006168])
def test_embed_grad_rows_of_a_huge_table(gpu_device, n, R):
    gen = torch.Generator().manual_seed(n)
    ids = (R * torch.rand(n, generator=gen).double() ** 8).long().clamp_(max=R - 1)
    ids[0], ids[-1] = R - 1, 0
    up = _randn(gen, (n, 32), BF)
    u, slot = torch.unique(ids, return_inverse=True)
    want, mag, m = ref.embed_grad(slot, up, u.numel(), 0, 1.0)
    unique, rows, count = _eng().engram_embed_grad_rows(ids.to(torch.int32).to(gpu_device), up.to(gpu_device), R)
    c = int(count)
    assert c == u.numel() and torch.equal(unique.cpu()[:c], u) and (unique.cpu()[c:] == -1).all()
    _within(rows[:c], want, ref.sum_tolerance(want, mag, m, False), "rows")
    assert not rows[c:].any()


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("row_start", [0, 12345, -7])
def test_embed_grad_row_start_and_id_types(gpu_device, idt, row_start):
    gen = torch.Generator().manual_seed(5)
    ids = (_ids_of("zipf", 777, 90, gen) - 3 + row_start).to(idt)
    _check_grad(_eng(), ids, _randn(gen, (777, 40), BF), 90, 40, gpu_device, F32, row_start=row_start, what="row_start")


@pytest.mark.parametrize("B,L", [(2, 9), (3, 400)])
def test_embed_grad_of_one_layer(gpu_device, B, L):
    g, E, C, D, R = _eng(), 3, 6, 32, 500
    gen = torch.Generator().manual_seed(L)
    ids = torch.randint(0, R, (B, L, E, C), generator=gen)
    up = _randn(gen, (B * L, C, D), BF)
    for e in range(E):
        flat = ids[:, :, e].reshape(-1)
        want, mag, m = ref.embed_grad(flat, up, R, 0, 1.0)
        for shape in ((B * L, C, D), (B * L, C * D)):
            got = g.engram_embed_grad(ids.to(gpu_device), up.to(gpu_device).view(shape), R, layer=e)
            _within(got, want, ref.sum_tolerance(want, mag, m, False), "layer")


@pytest.mark.parametrize("n", [0, 5, 700, 6000])
@pytest.mark.parametrize("odt", [BF, F32])
def test_embed_grad_accumulate(gpu_device, n, odt):
    gen = torch.Generator().manual_seed(n)
    R, D = 60, 48
    ids, up = _ids_of("zipf", n, R, gen), _randn(gen, (n, D), BF)
    ids[ids == 7] = 8
    base = _randn(gen, (R, D), odt)
    base[7] = NAN  # a row no id points at is not touched
    want, mag, m = ref.embed_grad(ids, up, R, 0, 0.5)
    want += base.double()
    mag += base.double().abs()
    out = base.to(gpu_device)
    got = _eng().engram_embed_grad(ids.to(gpu_device), up.to(gpu_device), R, scale=0.5, out=out, accumulate=True)
    assert got.data_ptr() == out.data_ptr()
    keep = torch.arange(R) != 7
    _within(got[keep.to(gpu_device)], want[keep], ref.sum_tolerance(want, mag, m + 1, odt == BF)[keep], "accumulate")
    assert got[7].isnan().all()


def test_ids_at_the_ends_of_64_bits(gpu_device):
    """Ids and first rows whose difference does not fit 64 bits are outside the table like any other."""
    g = _eng()
    lo, hi = -(1 << 63), (1 << 63) - 1
    for row_start, inside in ((hi - 3, (hi - 3, hi)), (lo, (lo, lo + 3)), (5, (5, 8)), (-5, (-5, -2))):
        ids = torch.tensor([lo, lo + 1, lo + 3, -6, -5, -2, -1, 0, 4, 5, 8, 9, hi - 4, hi - 3, hi], device=gpu_device)
        ok = ((ids >= inside[0]) & (ids <= inside[1])).cpu()
        out = g.engram_embed(ids, torch.ones((4, 8), device=gpu_device), row_start=row_start).cpu()
        assert torch.equal(out[:, 0] == 1, ok) and torch.equal(out[:, 0] == 0, ~ok)
        got = g.engram_embed_grad(ids, torch.ones((ids.numel(), 8), device=gpu_device), 4, row_start=row_start)
        assert float(got[:, 0].sum()) == int(ok.sum())
        unique, _, count = g.engram_embed_grad_rows(ids, torch.ones((ids.numel(), 8), device=gpu_device), 4,
                                                    row_start=row_start)
        assert int(count) == int(ok.sum()) and torch.equal(unique[:int(count)].cpu(), torch.unique(ids.cpu()[ok]))


def test_offsets_past_32_bits(gpu_device):
    """A table and its gradient of 2.5 G elements: rows on both sides of 2^31 elements and 2^32 bytes."""
    g, R, D = _eng(), 610000, 4096
    table = torch.zeros((R, D), dtype=BF, device=gpu_device)
    pick = torch.tensor([0, 1, 262143, 262144, 524287, 524288, 524289, R - 1], device=gpu_device)
    rows = torch.randn((pick.numel(), D), device=gpu_device).to(BF)
    table[pick] = rows
    for reps in (1, 300):  # one launch, and the sorted path
        ids = pick.repeat(reps)
        assert torch.equal(g.engram_embed(ids, table), rows.repeat(reps, 1))
        up = torch.zeros((ids.numel(), D), dtype=BF, device=gpu_device)
        up[:pick.numel()] = rows
        grad = g.engram_embed_grad(ids, up, R, out=torch.full((R, D), NAN, dtype=BF, device=gpu_device))
        assert torch.equal(grad[pick], rows)
        grad[pick] = 0
        assert not grad.any()
        del grad


def test_embed_grad_no_ids_and_non_finite(gpu_device):
    g = _eng()
    none = torch.empty((0,), dtype=torch.int64, device=gpu_device)
    out = g.engram_embed_grad(none, torch.empty((0, 16), dtype=BF, device=gpu_device), 5,
                              out=torch.full((5, 16), NAN, device=gpu_device))
    assert not out.any()
    unique, rows, count = g.engram_embed_grad_rows(none, torch.empty((0, 16), dtype=BF, device=gpu_device), 5)
    assert unique.numel() == 0 and rows.shape == (0, 16) and int(count) == 0
    # NaN and infinity stay in their rows and columns, and out-of-table positions leak nothing
    ids = torch.tensor([3, -1, 3, 9, 2, 0], device=gpu_device)
    up = torch.ones((6, 16), dtype=BF)
    up[1], up[3], up[0, 5], up[4, 2] = NAN, NAN, NAN, math.inf
    got = g.engram_embed_grad(ids, up.to(gpu_device), 5).cpu()
    want = torch.zeros((5, 16))
    want[3], want[2], want[0] = 2, 1, 1
    want[2, 2] = math.inf
    assert got[3, 5].isnan()
    got[3, 5] = want[3, 5]
    assert torch.equal(got, want)


def test_embed_grad_of_one_layer_of_no_tokens(gpu_device):
    g, E, C, D, R = _eng(), 3, 6, 32, 50
    for B, L in ((0, 9), (2, 0)):
        ids = torch.zeros((B, L, E, C), dtype=torch.int64, device=gpu_device)
        for shape in ((0, C, D), (B, L, C, D), (0, C * D)):
            up = torch.zeros(shape, dtype=BF, device=gpu_device)
            out = g.engram_embed_grad(ids, up, R, layer=1)
            assert out.shape == (R, D) and not out.any(), shape
            unique, rows, count = g.engram_embed_grad_rows(ids, up, R, layer=1)
            assert unique.shape == (0,) and rows.shape == (0, D) and int(count) == 0, shape


def test_embed_grad_refusals(gpu_device):
    g = _eng()
    ids = torch.zeros(6, dtype=torch.int64, device=gpu_device)
    up = torch.zeros((6, 16), dtype=BF, device=gpu_device)
    with pytest.raises(ValueError):
        g.engram_embed_grad(ids, up[:5], 4)
    with pytest.raises(ValueError):
        g.engram_embed_grad(ids, up, 4, accumulate=True)
    with pytest.raises(ValueError):
        g.engram_embed_grad(ids, up, 4, out=torch.zeros((5, 16), device=gpu_device))
    with pytest.raises(ValueError):
        g.engram_embed_grad(ids, up, 0)
    with pytest.raises(ValueError):
        g.engram_embed_grad(ids, up, 4, layer=0)
    with pytest.raises(TypeError):
        g.engram_embed_grad(ids, up.half(), 4)
    with pytest.raises(g.EngramError) as e:  # (the first sizes need none)
        g.engram_embed_grad(ids.repeat(300), up.repeat(300, 1), 4,
                            workspace=torch.zeros(16, dtype=torch.uint8, device=gpu_device))
    assert e.value.status == g.ENGRAM_ERANGE
    with pytest.raises(ValueError):
        g.engram_embed_grad_rows(ids, up, 4, rows=torch.zeros((5, 16), device=gpu_device))


# ---------------------------------------------------------------------------------------------------------------------
# the gate's gradient
# ---------------------------------------------------------------------------------------------------------------------
def _gate_inputs(T, hc, dim, seed, ld=None):
    gen = torch.Generator().manual_seed(seed)
    kv = _randn(gen, (T, ld or (hc + 1) * dim), BF, 0.5)
    x, dout = _randn(gen, (T, hc, dim), BF), _randn(gen, (T, hc, dim), BF, 1e-2)
    q, k = (1 + _randn(gen, (hc, dim), F32, 0.1)).to(BF), (1 + _randn(gen, (hc, dim), F32, 0.1)).to(BF)
    dot = ref.gate_forward(x, kv, q, k, 1e-20)[1].float()
    return x, kv, q, k, dot, dout


def _check_gate(got, want, T, dim, what):
    """The sums over dim and over tokens are float32: (dim + 64) U32 and (T + dim + 64) U32 of the magnitudes."""
    for name, t in zip(("dx", "dkv", "dq", "dk"), got):
        terms = dim + 64 + (T if name in ("dq", "dk") else 0)
        tol = 2 * terms * ref.U32 * want[name + "_mag"] + (ref.U16 if t.dtype == BF else 0) * want[name].abs() + 1e-38
        _within(t, want[name], tol, f"{what} {name}")


@pytest.mark.parametrize("T,hc,dim", [
    (1, 4, 8), (5, 4, 256), (64, 4, 264), (700, 4, 1024), (33, 4, 5120), (9, 4, 5128), (7, 4, 8192), (40, 1, 512), (40, 2, 1032),
    (40, 3, 64), (21, 5, 520), (3, 64, 16), (11, 1, 8192), (6000, 4, 8), (6000, 3, 8)])
@pytest.mark.parametrize("masked", [False, True])
def test_gate_backward(gpu_device, T, hc, dim, masked):
    g = _eng()
    x, kv, q, k, dot, dout = _gate_inputs(T, hc, dim, T + dim)
    mask = None
    if masked:
        mask = torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.6
        x[~mask], kv[~mask], dot[~mask] = NAN, NAN, NAN  # what a masked token holds does not matter
    d = lambda t: None if t is None else t.to(gpu_device)  # noqa: E731
    args = [d(t) for t in (x, kv, q, k)] + [1e-20, d(dot), d(dout)]
    got = g.engram_gate_output_backward(*args, token_mask=d(mask))
    _check_gate(got, ref.gate_backward(x, kv, q, k, 1e-20, dot, dout, mask), T, dim, f"{T} {hc} {dim}")
    if masked:
        off = ~mask
        assert np.array_equal(bits(got[0])[off.numpy()], bits(dout)[off.numpy()])
        assert not bits(got[1])[off.numpy()].any()
    again = g.engram_gate_output_backward(*args, token_mask=d(mask), dx=args[6])  # dx over dout
    assert again[0].data_ptr() == args[6].data_ptr()
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("hc", [1, 2, 4])
@pytest.mark.parametrize("dim", [504, 1016, 2040, 2056, 2568, 5112, 5120, 5128, 8192])
def test_gate_backward_at_every_width(gpu_device, hc, dim):
    """Every count of copies that has a kernel of its own at every count of threads; some workgroups take two tokens."""
    g, T = _eng(), 290
    x, kv, q, k, dot, dout = _gate_inputs(T, hc, dim, dim + hc)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(dim)) < 0.8
    mask[0], mask[256] = True, True  # (the first workgroup's two)
    x[~mask], kv[~mask], dot[~mask] = NAN, NAN, NAN
    d = lambda t: t.to(gpu_device)  # noqa: E731
    got = g.engram_gate_output_backward(*[d(t) for t in (x, kv, q, k)], 1e-20, d(dot), d(dout), token_mask=d(mask))
    _check_gate(got, ref.gate_backward(x, kv, q, k, 1e-20, dot, dout, mask), T, dim, f"{hc} {dim}")


def test_gate_backward_all_masked_and_no_tokens(gpu_device):
    g = _eng()
    x, kv, q, k, dot, dout = [t.to(gpu_device) for t in _gate_inputs(6, 4, 64, 1)]
    dx, dkv, dq, dk = g.engram_gate_output_backward(x, kv, q, k, 1e-20, dot, dout,
                                                    token_mask=torch.zeros(6, dtype=torch.uint8, device=gpu_device))
    assert torch.equal(dx, dout) and not dkv.any() and not dq.any() and not dk.any()
    dx, dkv, dq, dk = g.engram_gate_output_backward(x[:0], kv[:0], q, k, 1e-20, dot[:0], dout[:0],
                                                    dq=torch.full_like(dq, NAN), dk=torch.full_like(dk, NAN))
    assert dx.shape == (0, 4, 64) and dkv.shape == (0, 320) and not dq.any() and not dk.any()


@pytest.mark.parametrize("hc", [4, 3])
def test_gate_backward_edges_of_the_dot(gpu_device, hc):
    """Pre-activations at and around the clamp, signed zeros, large ones; zero rows of the stream and of the keys."""
    g, dim = _eng(), 64
    x, kv, q, k, dot, dout = _gate_inputs(12, hc, dim, 9, ld=(hc + 1) * dim + 24)
    tiny = float(np.float32(1e-6))
    below = float(np.nextafter(np.float32(1e-6), np.float32(0)))
    for i, v in enumerate((0.0, -0.0, tiny, -tiny, below, -below, 3e-6, -1e-3, 60.0, -60.0)):
        dot[i] = v
    x[10], kv[11] = 0, 0
    dot[10], dot[11] = 0, 0
    got = g.engram_gate_output_backward(*[t.to(gpu_device) for t in (x, kv, q, k)], 1e-20, dot.to(gpu_device),
                                        dout.to(gpu_device))
    _check_gate(got, ref.gate_backward(x, kv, q, k, 1e-20, dot, dout), 12, dim, "edges")
    for i in (0, 1, 4, 5, 10, 11):  # the clamp is flat: only the residual passes
        assert torch.equal(got[0][i].cpu(), dout[i]), i


@pytest.mark.parametrize("hc", [1, 2, 4, 3])
@pytest.mark.parametrize("d", [20.0, 72.0, 300.0, 400.0, -72.0, -400.0, -1000.0])
def test_gate_backward_far_from_the_corner(gpu_device, hc, d):
    """Every pre-activation large: the sigmoid's slope is small and keeps its digits (dq and dk are float32).  A rounding of
    sqrt(|d|) moves the slope by up to sqrt(1000) U32, well inside the sums' (dim + 64) U32.  (Past 400 the float64
    reference's own 1 - g has fewer digits than that.)"""
    g, dim = _eng(), 64
    x, kv, q, k, dot, dout = _gate_inputs(12, hc, dim, 11)
    dot = torch.full_like(dot, d)
    got = g.engram_gate_output_backward(*[t.to(gpu_device) for t in (x, kv, q, k)], 1e-20, dot.to(gpu_device),
                                        dout.to(gpu_device))
    want = ref.gate_backward(x, kv, q, k, 1e-20, dot, dout)
    assert want["dq"].abs().max() > 1e-20
    _check_gate(got, want, 12, dim, f"{d}")


def test_gate_backward_past_32_bits(gpu_device):
    """108,000 tokens: the stream holds 2.2 G elements, kv 2.8 G; sampled tokens, and the rest must be finite."""
    g, T, hc, dim = _eng(), 108000, 4, 5120
    gen = torch.Generator(device=gpu_device).manual_seed(3)
    r = lambda *s: torch.empty(s, dtype=BF, device=gpu_device).normal_(generator=gen)  # noqa: E731
    x, kv, dout = r(T, hc, dim), r(T, (hc + 1) * dim), r(T, hc, dim)
    q, k = 1 + 0.1 * r(hc, dim), 1 + 0.1 * r(hc, dim)
    dot = torch.empty((T, hc), device=gpu_device).normal_(generator=gen)
    dx, dkv, dq, dk = g.engram_gate_output_backward(x, kv, q, k, 1e-20, dot, dout)
    at = torch.tensor([0, 1, 53687, 52428, 83886, 104857, 104858, T - 2, T - 1])
    c = lambda t: t[at.to(gpu_device)].cpu()  # noqa: E731
    want = ref.gate_backward(c(x), c(kv), q.cpu(), k.cpu(), 1e-20, c(dot), c(dout))
    for name, t in (("dx", c(dx)), ("dkv", c(dkv))):
        _within(t, want[name], 2 * (dim + 64) * ref.U32 * want[name + "_mag"] + ref.U16 * want[name].abs(), name)
    assert torch.isfinite(dq).all() and torch.isfinite(dk).all()


def test_gate_backward_refusals(gpu_device):
    g = _eng()
    x, kv, q, k, dot, dout = [t.to(gpu_device) for t in _gate_inputs(6, 4, 64, 1)]
    ok = dict(x=x, kv=kv, q_weight=q, k_weight=k, eps=1e-20, dot=dot, dout=dout)
    for bad in (dict(kv=kv[:, :256].contiguous()), dict(kv=kv[:5]), dict(dot=dot[:, :3].contiguous()), dict(dout=dout[:5]),
                dict(q_weight=q[:3]), dict(token_mask=torch.ones(5, dtype=torch.bool, device=gpu_device)),
                dict(dkv=torch.empty((6, 256), dtype=BF, device=gpu_device)), dict(x=x.transpose(0, 1).contiguous())):
        with pytest.raises(ValueError):
            g.engram_gate_output_backward(**{**ok, **bad})
    with pytest.raises(TypeError):
        g.engram_gate_output_backward(**{**ok, "dout": dout.float()})
    with pytest.raises(g.EngramError):
        g.engram_gate_output_backward(**ok, workspace=torch.empty(16, dtype=torch.uint8, device=gpu_device))


# ---------------------------------------------------------------------------------------------------------------------
# the projection's gradient
# ---------------------------------------------------------------------------------------------------------------------
def _guarded(t, device):
    """`t` on the GPU at the front of a buffer whose next elements are NaN: what a tile reads past its operand shows."""
    buf = torch.full((t.numel() + 65536,), NAN, dtype=t.dtype, device=device)
    buf[:t.numel()] = t.reshape(-1).to(device)
    return buf[:t.numel()].view(t.shape)


@pytest.mark.parametrize("dwt", [F32, BF])
@pytest.mark.parametrize("T,K,N", [
    (1, 8, 8), (3, 72, 200), (64, 192, 1280), (63, 64, 264), (65, 264, 72), (257, 264, 520), (300, 1536, 512), (251, 128, 2056),
    (1000, 40, 1304), (2049, 256, 256), (5000, 64, 64),
    (700, 1032, 12552), (1003, 1544, 10616)])  # the larger tiles: both products in a launch, and alone too
def test_wkv_backward(gpu_device, T, K, N, dwt):
    g = _eng()
    gen = torch.Generator().manual_seed(T + K + N)
    dkv, a, w = _randn(gen, (T, N), BF, 0.1), _randn(gen, (T, K), BF), _randn(gen, (N, K), BF, 0.1)
    dd, ad, wd = (_guarded(t, gpu_device) for t in (dkv, a, w))
    da, dw = g.engram_wkv_backward(dd, ad, wd, dw_dtype=dwt)
    p, q, r = dkv.double(), a.double(), w.double()
    _within(da, p @ r, 2 * N * ref.U32 * (p.abs() @ r.abs()) + ref.U16 * (p @ r).abs(), "da")
    tol = 2 * T * ref.U32 * (p.abs().t() @ q.abs()) + (ref.U16 if dwt == BF else 2 * ref.U32) * (p.t() @ q).abs()
    _within(dw, p.t() @ q, tol, "dw")
    again = g.engram_wkv_backward(dd, ad, wd, dw_dtype=dwt)
    assert torch.equal(again[0], da) and torch.equal(again[1], dw)
    # each product alone (its sum may be cut into other parts); accumulation adds to what is there
    tol_da = 2 * N * ref.U32 * (p.abs() @ r.abs()) + ref.U16 * (p @ r).abs()
    only_da, none = g.engram_wkv_backward(dd, None, wd, need_dw=False)
    assert none is None
    _within(only_da, p @ r, tol_da, "da alone")
    none, only_dw = g.engram_wkv_backward(dd, ad, None, need_da=False, dw_dtype=dwt)
    assert none is None
    _within(only_dw, p.t() @ q, tol, "dw alone")
    base = _randn(gen, (N, K), dwt)
    _, acc = g.engram_wkv_backward(dd, ad, wd, dw=base.to(gpu_device), accumulate=True)
    want = p.t() @ q + base.double()
    tol = 2 * (T + 1) * ref.U32 * (p.abs().t() @ q.abs() + base.double().abs())
    _within(acc, want, tol + (ref.U16 if dwt == BF else 2 * ref.U32) * want.abs(), "accumulated dw")


@pytest.mark.parametrize("T,K,N", [
    (64, 1536, 25600), (251, 1536, 25600), (2048, 1536, 25600), (4000, 1536, 5120), (5984, 344, 9624), (5687, 584, 5416),
    (8000, 456, 2000), (8192, 256, 1320), (300, 320, 600), (700, 1032, 12552), (1, 8, 8)])
def test_wkv_backward_alone_gives_the_same_bits(gpu_device, T, K, N):
    """Whether the other product is asked for changes neither's sum (the large shapes' splits differ between the two)."""
    g = _eng()
    gen = torch.Generator(device=gpu_device).manual_seed(T + K)
    r = lambda *s: torch.empty(s, device=gpu_device).normal_(generator=gen).to(BF)  # noqa: E731
    dkv, a, w = r(T, N), r(T, K), r(N, K)
    da, dw = g.engram_wkv_backward(dkv, a, w)
    assert torch.equal(g.engram_wkv_backward(dkv, None, w, need_dw=False)[0], da)
    assert torch.equal(g.engram_wkv_backward(dkv, a, None, need_da=False)[1], dw)


@pytest.mark.parametrize("dwt", [F32, BF])
@pytest.mark.parametrize("T,K,N", [
    (251, 1536, 25600), (2049, 1544, 25608), (521, 1544, 25608),     # 256 x 256 tiles, da's sum split
    (33001, 1032, 5128), (30011, 520, 8200), (70001, 1544, 1288),    # the same, dW's sum split, alone too
    (60013, 248, 2056), (40003, 264, 5128),                          # 128 x 128 ones for dW alone and for both
    (261, 6144, 25600), (131, 6152, 2568), (3001, 6144, 1288)])      # the released head_dim's reduction
def test_wkv_backward_of_whole_numbers(gpu_device, T, K, N, dwt):
    """Entries of -2 to 2: every sum (280,004 at most) is exact in float32 in any order, so one lost, doubled or misplaced
    term of any tile, slab or part shows."""
    g = _eng()
    gen = torch.Generator(device=gpu_device).manual_seed(T + K)

    def whole(*shape):
        buf = torch.full((math.prod(shape) + 65536,), NAN, dtype=BF, device=gpu_device)  # what is read past it shows
        buf[:-65536] = torch.randint(-2, 3, (math.prod(shape),), generator=gen, device=gpu_device).to(BF)
        return buf[:-65536].view(shape)

    dkv, a, w = whole(T, N), whole(T, K), whole(N, K)
    da = torch.mm(dkv.double(), w.double())
    dw = torch.mm(dkv.double().t().contiguous(), a.double())
    assert da.abs().max() < 2 ** 24 and dw.abs().max() < 2 ** 24
    got = g.engram_wkv_backward(dkv, a, w, dw_dtype=dwt)
    assert torch.equal(got[0], da.to(BF)) and torch.equal(got[1], dw.to(dwt))
    assert torch.equal(g.engram_wkv_backward(dkv, None, w, need_dw=False)[0], da.to(BF))
    assert torch.equal(g.engram_wkv_backward(dkv, a, None, need_da=False, dw_dtype=dwt)[1], dw.to(dwt))
    base = torch.randint(-9, 10, (N, K), generator=gen, device=gpu_device).to(dwt)
    want = (dw + base.double()).to(dwt)
    assert torch.equal(g.engram_wkv_backward(dkv, a, w, dw=base, accumulate=True)[1], want)


def test_wkv_backward_selects_rows(gpu_device):
    """One-hot operands: da picks a row of w, dw a row of a, exactly, at every tile and k-step position."""
    g, T, K, N = _eng(), 300, 320, 600
    gen = torch.Generator().manual_seed(1)
    w, a = _randn(gen, (N, K), BF), _randn(gen, (T, K), BF)
    pick = torch.randperm(N, generator=gen)[:T]
    dkv = torch.zeros((T, N), dtype=BF)
    dkv[torch.arange(T), pick] = 1
    da, dw = g.engram_wkv_backward(*[t.to(gpu_device) for t in (dkv, a, w)])
    assert torch.equal(da.cpu(), w[pick])
    want = torch.zeros((N, K))
    want[pick] = a.float()
    assert torch.equal(dw.cpu(), want)


def test_wkv_backward_no_tokens_and_non_finite(gpu_device):
    g, N, K = _eng(), 264, 72
    empty = torch.empty((0, N), dtype=BF, device=gpu_device)
    w = torch.ones((N, K), dtype=BF, device=gpu_device)
    da, dw = g.engram_wkv_backward(empty, torch.empty((0, K), dtype=BF, device=gpu_device), w,
                                   dw=torch.full((N, K), NAN, device=gpu_device))
    assert da.shape == (0, K) and not dw.any()
    keep = torch.full((N, K), 3.0, device=gpu_device)
    g.engram_wkv_backward(empty, torch.empty((0, K), dtype=BF, device=gpu_device), w, dw=keep, accumulate=True)
    assert (keep == 3).all()
    # a NaN token spoils its own row of da and every dw; an infinite weight its column
    dkv, a = torch.ones((70, N), dtype=BF, device=gpu_device), torch.ones((70, K), dtype=BF, device=gpu_device)
    w[5, 3] = math.inf
    dkv[66, 10] = NAN
    da, dw = g.engram_wkv_backward(dkv, a, w)
    assert da[66].isnan().all() and da[:66, 3].isinf().all() and torch.isfinite(da[:66, 4:]).all()
    assert dw[10].isnan().all() and torch.isfinite(dw[:10]).all() and torch.isfinite(dw[11:]).all()


def test_wkv_backward_past_32_bits(gpu_device):
    """dkv of 2.4 G elements: one-hot tokens pick rows of w and rows of a, exactly, on both sides of 2^31 elements."""
    g, T, K, N = _eng(), 95000, 64, 25600
    gen = torch.Generator().manual_seed(4)
    w, a = _randn(gen, (N, K), BF).to(gpu_device), _randn(gen, (T, K), BF).to(gpu_device)
    dkv = torch.zeros((T, N), dtype=BF, device=gpu_device)
    tok = torch.tensor([0, 5, 41943, 83885, 83886, 83887, 94999], device=gpu_device)
    col = torch.tensor([0, 25599, 12800, 255, 256, 77, 20000], device=gpu_device)
    dkv[tok, col] = 1
    da, dw = g.engram_wkv_backward(dkv, a, w)
    assert torch.equal(da[tok], w[col]) and torch.equal(dw[col], a[tok].float())
    da[tok], dw[col] = 0, 0
    assert not da.any() and not dw.any()


def test_wkv_backward_refusals(gpu_device):
    g = _eng()
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device=gpu_device)  # noqa: E731
    for bad in ((z(8, 64), z(7, 32), z(64, 32)), (z(8, 64), z(8, 32), z(56, 32)), (z(8, 64), z(8, 32), z(64, 40)),
                (z(8, 64), None, z(64, 32)), (z(8, 64), z(8, 32), None)):
        with pytest.raises(ValueError):
            g.engram_wkv_backward(*bad)
    with pytest.raises(ValueError):
        g.engram_wkv_backward(z(8, 64), z(8, 32), z(64, 32), accumulate=True)
    with pytest.raises(ValueError):
        g.engram_wkv_backward(z(8, 64), z(8, 32), z(64, 32), need_da=False, need_dw=False)
    with pytest.raises(TypeError):
        g.engram_wkv_backward(z(8, 64, dt=F32), z(8, 32), z(64, 32))
    with pytest.raises(ValueError):
        g.engram_wkv_backward(z(8, 60), z(8, 32), z(60, 32))


# ---------------------------------------------------------------------------------------------------------------------
# norm and clipping
# ---------------------------------------------------------------------------------------------------------------------
def _norm_of(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def _tensors(sizes, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [_randn(gen, (n,), BF if i % 2 else F32, std) for i, n in enumerate(sizes)]


@pytest.mark.parametrize("sizes", [(1,), (0, 3, 0), (7, 8, 9), (16383, 16384, 16385, 32767, 32769), (100000, 1, 70001),
                                   tuple(range(1, 230))])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e6])
def test_norm_and_clip(gpu_device, sizes, max_norm):
    """The sum is kept in float64 and rounded once at the end (2 U32 of the root, as the reference's own rounding); the
    factor takes an addition, a division and a product more: 6 U32 in all, then the type's rounding."""
    g = _eng()
    ts = _tensors(sizes, len(sizes))
    dev = [t.to(gpu_device) for t in ts]
    norm = g.engram_grad_norm(dev)
    want = _norm_of(ts)
    assert abs(float(norm) - want) <= 2 * ref.U32 * want
    assert torch.equal(g.engram_grad_norm(dev), norm)
    coef = min(1.0, max_norm / (want + 1e-6))
    outs = [torch.full_like(t, NAN) for t in dev]
    got = g.engram_clip_grads(dev, norm, max_norm, outs=outs)
    assert all(a is b for a, b in zip(got, outs))
    for o, t in zip(outs, ts):
        r = t.double() * coef
        _within(o, r, (8 * ref.U32 + (ref.U16 if t.dtype == BF else 0)) * r.abs() + 1e-38, "clipped")
    for d, t in zip(dev, ts):
        assert torch.equal(d.cpu(), t)
    same = g.engram_clip_grads(dev, norm, max_norm)  # in place
    for s, o in zip(same, outs):
        assert torch.equal(s, o)


def test_norm_of_unaligned_views(gpu_device):
    g = _eng()
    ts = _tensors((4099, 4099), 2)
    for off in (1, 2, 3, 5):
        views = [t.to(gpu_device)[off:] for t in ts]
        norm = g.engram_grad_norm(views)
        want = _norm_of([t[off:] for t in ts])
        assert abs(float(norm) - want) <= 2 * ref.U32 * want
        outs = [torch.zeros_like(t.to(gpu_device))[1:][:t.numel() - off] if off > 1 else torch.zeros_like(v)
                for t, v in zip(ts, views)]
        g.engram_clip_grads(views, norm, 1.0, outs=outs)
        for o, t in zip(outs, ts):
            r = t[off:].double() * (1 / (want + 1e-6))
            _within(o, r, (8 * ref.U32 + (ref.U16 if t.dtype == BF else 0)) * r.abs() + 1e-38, "unaligned")


def test_norm_extremes(gpu_device):
    g = _eng()
    assert float(g.engram_grad_norm([])) == 0
    assert float(g.engram_grad_norm([torch.zeros(9, device=gpu_device)])) == 0
    z = g.engram_clip_grads([torch.zeros(9, device=gpu_device)], torch.zeros(1, device=gpu_device), 1.0)
    assert not z[0].any()
    big = [torch.full((1000,), 1e30, device=gpu_device)]  # the squares are past float32
    assert abs(float(g.engram_grad_norm(big)) / (1e30 * math.sqrt(1000)) - 1) <= 4 * ref.U32
    small = [torch.full((1000,), 1e-30, device=gpu_device)]
    assert abs(float(g.engram_grad_norm(small)) / (1e-30 * math.sqrt(1000)) - 1) <= 4 * ref.U32
    for bad, is_bad in ((math.inf, math.isinf), (NAN, math.isnan)):
        t = torch.ones(5000, device=gpu_device)
        t[4321] = bad
        norm = g.engram_grad_norm([t])
        assert is_bad(float(norm))
        out = g.engram_clip_grads([t], norm, 1.0, outs=[torch.empty_like(t)])[0]
        if math.isinf(bad):  # the factor is 0: the finite ones vanish, infinity times 0 is NaN
            assert out[4321].isnan() and int((out == 0).sum()) == 4999
        else:
            assert out.isnan().all()


def test_norm_and_clip_past_a_launch(gpu_device):
    """64 GiB in one tensor, more than a launch's grid holds: every element, on both sides of each cut, and the tensors
    around it."""
    g, n = _eng(), (1 << 35) + 2053
    first, last = torch.full((1025,), 0.5, device=gpu_device), torch.full((77,), -0.25, dtype=BF, device=gpu_device)
    big = torch.full((n,), 2.0 ** -10, dtype=BF, device=gpu_device)
    at = torch.tensor([0, (1 << 34) - 1, 1 << 34, (1 << 35) - 1, 1 << 35, n - 1], device=gpu_device)
    big[at] = 3.0
    want = math.sqrt(1025 * 0.25 + 77 * 0.0625 + (n - 6) * 2.0 ** -20 + 6 * 9)
    norm = g.engram_grad_norm([first, big, last])
    assert abs(float(norm) - want) <= 2 * ref.U32 * want
    g.engram_clip_grads([first, big, last], torch.full((1,), 4.0, device=gpu_device), 2.0)
    # the factor is 2 / (4 + 1e-6): a half less 1.25e-7, and both values round to their halves in bf16
    assert (big[at] == 1.5).all()
    big[at] = 2.0 ** -11
    for i in range(0, n, 1 << 32):
        assert bool((big[i:i + (1 << 32)] == 2.0 ** -11).all()), i
    assert (last == -0.125).all() and (first - 0.25).abs().max() <= 2.0 ** -23


def test_norm_and_clip_refusals(gpu_device):
    g = _eng()
    t = torch.ones(8, device=gpu_device)
    n = torch.ones(1, device=gpu_device)
    for call in (lambda: g.engram_grad_norm([t.half()]), lambda: g.engram_clip_grads([t], n.double(), 1.0)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.engram_grad_norm([t[::2]]), lambda: g.engram_clip_grads([t], n, 1.0, outs=[t, t]),
                 lambda: g.engram_clip_grads([t], n, 1.0, outs=[t[:4]]), lambda: g.engram_clip_grads([t], t, 1.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(g.EngramError):
        g.engram_clip_grads([t], n, -1.0)


# ---------------------------------------------------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------------------------------------------------
def _all_ops(g, s, stream=None):
    e = g.engram_embed(s["tok"], s["table"], scale=4.0, stream=stream)
    dx, dkv, dq, dk = g.engram_gate_output_backward(s["x"], s["kv"], s["q"], s["k"], 1e-20, s["dot"], s["dout"], stream=stream)
    da, dw = g.engram_wkv_backward(dkv, s["a"], s["w"], stream=stream)
    u, r, c = g.engram_embed_grad_rows(s["ids"], da.view(-1, 32), 5000, stream=stream)
    de = g.engram_embed_grad(s["tok"], e, 300, stream=stream)
    grads = [dq, dk, dw, r, de]
    norm = g.engram_grad_norm(grads, stream=stream)
    outs = [torch.empty_like(t) for t in grads]
    g.engram_clip_grads(grads, norm, 0.5, outs=outs, stream=stream)
    return [e, dx, dkv, dq, dk, da, dw, u, r, c, de, norm, *outs]


def _state(dev, seed, T=200):
    x, kv, q, k, dot, dout = [t.to(dev) for t in _gate_inputs(T, 4, 64, seed)]
    gen = torch.Generator().manual_seed(seed)
    return dict(x=x, kv=kv, q=q, k=k, dot=dot, dout=dout, a=_randn(gen, (T, 192), BF).to(dev),
                w=_randn(gen, (320, 192), BF, 0.1).to(dev), ids=torch.randint(0, 5000, (T * 6,), generator=gen).to(dev),
                tok=torch.randint(0, 300, (T,), generator=gen).to(dev), table=_randn(gen, (300, 64), BF).to(dev))


def test_on_another_stream(gpu_device):
    g = _eng()
    s = _state(gpu_device, 1)
    want = _all_ops(g, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all_ops(g, s)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # one call handed a stream, its temporaries and outputs made there
    side.wait_stream(torch.cuda.current_stream())
    dw = [g.engram_wkv_backward(s["kv"], s["a"], s["w"], stream=side)[1] for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    ref_dw = g.engram_wkv_backward(s["kv"], s["a"], s["w"])[1]
    assert all(torch.equal(d, ref_dw) for d in dw)


def test_graph_replays(gpu_device):
    g = _eng()
    s = _state(gpu_device, 2)
    _all_ops(g, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _all_ops(g, s)
    for seed in (3, 4, 5):
        for name, t in _state(gpu_device, seed).items():
            s[name].copy_(t)
        want = [t.clone() for t in _all_ops(g, s)]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
