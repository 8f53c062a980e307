"""The 4-bit projection's tiles where there are many, and calls that no small size reaches: every tile against whole numbers and
against the others, arrays of more than 2^32 elements, calls in flight at once and graphs of their own."""
import pytest
import torch

import gram_hash_embedding_amd as g
from tests import lowbit_ref as ref
from tests.test_gpu_lowbit import EPS, _bf16, _dot_tolerance, _gate_case, _gate_inputs, _gen, _rows, _weights

pytestmark = pytest.mark.gpu

# 128 tokens a tile from 384 of 256 columns, 64 and 32 from 128, 16: a count either side, and steps of every remainder
WIDE = [(500, 128, 25600), (385, 256, 25592), (513, 384, 25544), (400, 640, 25600), (2305, 896, 5400), (12300, 128, 1000),
        (384, 384, 25600), (65, 128, 25600), (129, 640, 25544), (250, 1536, 25600), (700, 256, 8200), (64, 256, 25600),
        (40, 896, 25592), (33, 128, 32776), (200, 384, 9000), (17, 1536, 25600), (32, 640, 25544), (1, 384, 25600)]
# an eighth of the columns along all rows, rather than eight tile rows along the columns
ALONG_ROWS = [(3000, 384, 25544), (4100, 128, 8200), (2200, 640, 25592), (9001, 256, 6400), (2050, 1536, 25600), (20000, 128, 2312)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", WIDE + ALONG_ROWS)
def test_tiles_in_whole_numbers(gpu_device, T, K, N, bits):
    """Exact sums, as of the small products: multiples of a quarter whose sums stay below 2^22 quarters."""
    gen = _gen("wide", T, K, N, bits)
    w, wv = _weights(gen, N, K, gpu_device, whole=True)
    a, s, av = _rows(gen, T, K, bits, gpu_device, whole=True)
    want = (av.float().to(gpu_device) @ wv.float().t().contiguous().to(gpu_device)).to(torch.bfloat16)  # exact in float32 too
    out = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=gpu_device)
    g.engram_wkv_mx4(a, s, w, out=out[1:-1])
    assert torch.equal(out[1:-1], want) and (out[0] == 7).all() and (out[-1] == 7).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("K,hc,dim", [(384, 4, 5120), (1536, 4, 2304)])
def test_every_tile_gives_the_same_rows(gpu_device, K, hc, dim, bits):
    """The rows of a call of 128 tokens a tile, in calls of 64, 32 and 16: the same bits, of the product and of its value
    columns, and the dot that the stored keys give within its bound; a call's own results again, the same."""
    gen = _gen("tiles", K, hc, dim, bits)
    T = 1400
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    a, s, _ = _rows(gen, T, K, bits, gpu_device)
    x, q, k = _gate_inputs(gen, T, hc, dim, gpu_device)
    kv = g.engram_wkv_mx4(a, s, w)
    value, dot = g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS)
    assert torch.equal(value, kv[:, hc * dim:])
    want, tol = _dot_tolerance(x, kv[:, :hc * dim].view(T, hc, dim), q, k)
    assert ((dot.double() - want).abs() <= tol).all()
    for _ in range(3):
        v2, d2 = g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS)
        assert torch.equal(v2, value) and torch.equal(d2, dot)
    sr = ref.scales_rows(s.cpu(), T)
    for t0, n in ((0, 1), (9, 16), (400, 17), (77, 32), (200, 33), (1000, 64), (3, 65), (128, 128), (131, 256), (400, 400), (1, 700)):
        rows = slice(t0, t0 + n)
        part = (a[rows].contiguous(), ref.scales_laid_out(sr[rows]).to(gpu_device), w)
        assert torch.equal(g.engram_wkv_mx4(*part), kv[rows]), (t0, n)
        v, d = g.engram_wkv_mx4_gate(*part, x[rows].contiguous(), q, k, EPS)
        assert torch.equal(v, value[rows]), (t0, n)
        assert ((d.double() - want[rows]).abs() <= tol[rows]).all(), (t0, n)


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def _sample(T, n=40):
    """Rows at the start, around every 2^32nd element that the caller names, and at the end."""
    return lambda *marks: [slice(max(0, min(m, T - n)), max(0, min(m, T - n)) + n) for m in (0, *marks, T - n)]


@pytest.mark.parametrize("bits", [4, 8])
def test_product_past_32_bits(gpu_device, bits):
    """kv of more than 2^32 elements: sampled rows are those of calls of their own."""
    _room(40)
    T, K, N = 170001, 128, 25600
    gen = _gen("long", bits)
    w, _ = _weights(gen, N, K, gpu_device)
    a, s, _ = _rows(gen, T, K, bits, gpu_device)
    kv = g.engram_wkv_mx4(a, s, w)
    sr = ref.scales_rows(s.cpu(), T)
    for r in _sample(T)((1 << 31) // N - 20, (1 << 32) // N - 20):
        assert torch.equal(kv[r], g.engram_wkv_mx4(a[r].contiguous(), ref.scales_laid_out(sr[r]).to(gpu_device), w)), r


def test_fused_product_past_32_bits(gpu_device):
    """A stream of more than 2^32 elements, and rows of more than 2^32 bytes."""
    _room(60)
    T, K, hc, dim = 4200007, 1024, 4, 256
    gen = _gen("longgate")
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    dg = torch.Generator(device=gpu_device).manual_seed(3)
    a = torch.randint(0, 120, (T, K), dtype=torch.uint8, generator=dg, device=gpu_device)
    s = torch.full(((K // 128), (T + 3) // 4 * 4, 4), 122, dtype=torch.uint8, device=gpu_device)
    x = torch.randn((T, hc, dim), generator=dg, device=gpu_device, dtype=torch.bfloat16)
    _, q, k = _gate_inputs(gen, 1, hc, dim, gpu_device)
    value, dot = g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS)
    for r in _sample(T)((1 << 31) // 1024 - 20, (1 << 32) // 1024 - 20):
        part = a[r].contiguous(), s[:, :40].contiguous(), w
        kv = g.engram_wkv_mx4(*part)
        assert torch.equal(value[r], kv[:, hc * dim:]), r
        want, tol = _dot_tolerance(x[r], kv[:, :hc * dim].view(-1, hc, dim), q, k)
        assert ((dot[r].double() - want).abs() <= tol).all(), r


def test_quantisation_past_32_bits(gpu_device):
    _room(40)
    T, K = 4200003, 1024
    x = torch.randn((T, K), dtype=torch.bfloat16, device=gpu_device)
    q, s = g.engram_mx4_quant(x)
    for r in _sample(T)((1 << 31) // K - 20, (1 << 32) // K - 20):
        pq, ps = g.engram_mx4_quant(x[r])
        assert torch.equal(q[r], pq) and torch.equal(s[:, r], ps), r


def test_checkpoints_past_32_bits(gpu_device):
    """Through the module's step as well: the kept rows, the output and the gradient."""
    _room(110)
    T, hc, dim = 1100000, 4, 1024
    dg = torch.Generator(device=gpu_device).manual_seed(4)
    x = torch.randn((T, hc, dim), generator=dg, device=gpu_device, dtype=torch.bfloat16)
    kv = torch.randn((T, (hc + 1) * dim), generator=dg, device=gpu_device, dtype=torch.bfloat16)
    dout = torch.randn((T, hc, dim), generator=dg, device=gpu_device, dtype=torch.bfloat16)
    _, q, k = _gate_inputs(_gen("longckpt"), 1, hc, dim, gpu_device)
    out, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS)
    back = g.engram_ckpt_load(c.kv, c.kv_scale)
    dx, dkv, _, _ = g.engram_gate_output_backward_ckpt(c, q, k, EPS, dot, dout)
    saved = g.engram_ckpt_save(x)
    for r in _sample(T)((1 << 31) // 5120 - 20, (1 << 31) // 4096 - 20, (1 << 32) // 5120 - 20, (1 << 32) // 4096 - 20):
        po, pd, pc = g.engram_gate_output_ckpt(x[r], kv[r], q, k, EPS)
        assert torch.equal(out[r], po) and torch.equal(dot[r], pd), r
        assert all(torch.equal(t[r], p) for t, p in zip(c, pc)), r
        assert torch.equal(saved[0][r], pc.x) and torch.equal(saved[1][r], pc.x_scale), r
        assert torch.equal(back[r], g.engram_ckpt_load(pc.kv, pc.kv_scale)), r
        gx, gkv, _, _ = g.engram_gate_output_backward_ckpt(pc, q, k, EPS, pd, dout[r])
        assert torch.equal(dx[r], gx) and torch.equal(dkv[r], gkv), r


def test_calls_in_flight_at_once(gpu_device):
    """The same calls on two streams, each with a workspace of its own: the results of either alone."""
    gen = _gen("two")
    K, hc, dim = 1536, 4, 1024
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    sides = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for T in (700, 333):
        x, kv, q, k, mask, dout = _gate_case(T, hc, dim, gpu_device)
        ws = [torch.empty(n, dtype=torch.uint8, device=gpu_device) for n in (
            g.engram_wkv_gate_workspace_bytes(T, hc, dim), g.engram_gate_output_backward_workspace_bytes(T, hc, dim))]
        sets.append((_bf16(gen, (T, K)).to(gpu_device), x, kv, q, k, mask, dout, ws))

    def calls(stream, rows, x, kv, q, k, mask, dout, ws):
        a, s = g.engram_mx4_quant(rows, stream=stream)
        out, d, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask, stream=stream)
        return [g.engram_wkv_mx4(a, s, w, stream=stream), *g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS, workspace=ws[0], stream=stream),
                out, d, *c, *g.engram_gate_output_backward_ckpt(c, q, k, EPS, d, dout, mask, workspace=ws[1], stream=stream)]

    want = [calls(None, *p) for p in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [calls(side, *p) for side, p in zip(sides, sets)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, r) for p, r in zip(a, b))


def test_two_graphs_one_workspace(gpu_device):
    """Two captured steps of different sizes that share a workspace, replayed in turn on one stream."""
    gen = _gen("graphs")
    K, hc, dim = 384, 4, 512
    w, _ = _weights(gen, (hc + 1) * dim, K, gpu_device)
    cases = [_gate_case(T, hc, dim, gpu_device) for T in (50, 260)]
    rows = [_bf16(gen, (c[0].shape[0], K)).to(gpu_device) for c in cases]
    ws = torch.empty(max(f(260, hc, dim) for f in (g.engram_wkv_gate_workspace_bytes, g.engram_gate_output_backward_workspace_bytes)),
                     dtype=torch.uint8, device=gpu_device)

    def step(i):
        x, kv, q, k, mask, dout = cases[i]
        a, s = g.engram_mx4_quant(rows[i])
        value, dot = g.engram_wkv_mx4_gate(a, s, w, x, q, k, EPS, workspace=ws)
        res = g.engram_gate_residual(x, value, dot, mask)
        out, d, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
        return [value, dot, res, out, d, *c, *g.engram_gate_output_backward_ckpt(c, q, k, EPS, d, dout, mask, workspace=ws)]

    graphs, held = [], []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(step(i))
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1) if turn % 2 else (1, 0):
            rows[i].copy_(_bf16(gen, rows[i].shape).to(gpu_device))
            cases[i][0].copy_(_bf16(gen, cases[i][0].shape).to(gpu_device))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            got = [t.clone() for t in held[i]]
            for p, r in zip(got, step(i)):
                assert torch.equal(p, r), (turn, i)


@pytest.mark.parametrize("T,hc,dim", [(50, 4, 512), (33, 3, 264), (9, 1, 8192), (700, 4, 5120)])
def test_output_with_checkpoints_in_place(gpu_device, T, hc, dim):
    """out may be x: the stream kept is the one that came in; given tensors are filled and nothing beside them."""
    x, kv, q, k, mask, _ = _gate_case(T, hc, dim, gpu_device, extra=8)
    out, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    nb = (dim + 31) // 32
    held = [torch.full((T + 1, n, w), 9, dtype=t, device=gpu_device) for n, w, t in (
        (hc, dim, torch.int8), (hc, nb, torch.uint8), (hc + 1, dim, torch.int8), (hc + 1, nb, torch.uint8))]
    stream = x.clone()
    o2, d2, c2 = g.engram_gate_output_ckpt(stream, kv, q, k, EPS, mask, out=stream, dot=torch.empty_like(dot),
                                           checkpoint=g.GateCheckpoint(*[t[:T] for t in held]))
    assert o2 is stream and torch.equal(o2, out) and torch.equal(d2, dot)
    for t, a, b in zip(held, c, c2):
        assert torch.equal(a, b) and (t[T] == 9).all()


@pytest.mark.parametrize("dim", [8, 24, 120, 128, 136, 248, 256, 264, 512, 520, 1016, 1024, 1032, 2048, 2056, 4096, 4104, 6144, 6152,
                                 8192])
@pytest.mark.parametrize("T,hc", [(1, 1), (3, 3), (67, 2), (130, 5)])
def test_output_with_checkpoints_at_every_width(gpu_device, T, hc, dim):
    """A group of lanes, a wave or a workgroup a row: what is kept bit for bit, the dot within its bound, the output as the
    residual gives it from that dot."""
    x, kv, q, k, mask, _ = _gate_case(T, hc, dim, gpu_device, extra=16)
    out, dot, c = g.engram_gate_output_ckpt(x, kv, q, k, EPS, mask)
    rows = kv[:, :(hc + 1) * dim].contiguous().view(T, hc + 1, dim)
    for got, want in zip(c, (*g.engram_ckpt_save(x), *g.engram_ckpt_save(rows))):
        assert torch.equal(got, want)
    want, tol = _dot_tolerance(x, rows[:, :hc], q, k)
    assert ((dot.double() - want).abs() <= tol).all()
    assert torch.equal(out, g.engram_gate_residual(x, kv[:, hc * dim:(hc + 1) * dim], dot, mask))
