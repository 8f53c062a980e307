"""The launches of the 4-bit projection and of the 8-bit checkpoints at sizes that no test allocates: every grid within the
runtime's limits, all of the work covered, every launch's failure reported."""
import shutil

import pytest

from tests.launches import Library

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not installed")
AT = 1 << 40  # a device address; nothing follows it
EHIP = 3
CARD = 288 << 30


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    with Library(tmp_path_factory.mktemp("launches")) as lib:
        yield lib


P = ("p", AT)
END = ("p", None)


def _quant(lib, rows, K, f=None):
    return lib.call("engram_mx4_quant", [P, ("i64", rows), ("i32", K), P, P, END], f)


def _pack(lib, N, K, f=None):
    return lib.call("engram_mx4_pack_weight", [P, P, ("i32", N), ("i32", K), P, END], f)


def _wkv(lib, bits, T, K, N, f=None):
    return lib.call("engram_wkv_mx4", [P, P, ("i32", bits), P, P, ("i64", T), ("i32", K), ("i32", N), END], f)


def _gate(lib, bits, T, K, hc, dim, f=None):
    return lib.call("engram_wkv_mx4_gate", [P, P, ("i32", bits), P, P, P, P, ("f32", 1e-20), P, ("i64", dim), P, P, ("i64", 1 << 60),
                                            ("i64", T), ("i32", K), ("i32", hc), ("i32", dim), END], f)


def _save(lib, rows, D, f=None):
    return lib.call("engram_ckpt_save", [P, ("i64", rows), ("i32", D), P, P, END], f)


def _load(lib, rows, D, f=None):
    return lib.call("engram_ckpt_load", [P, P, ("i64", rows), ("i32", D), P, END], f)


def _output(lib, T, hc, dim, f=None):
    return lib.call("engram_gate_output_ckpt", [P, P, ("i64", (hc + 1) * dim), P, P, ("f32", 1e-20), END, *[P] * 6, ("i64", T),
                                                ("i32", hc), ("i32", dim), END], f)


def _grad(lib, T, hc, dim, f=None):
    return lib.call("engram_gate_output_backward_ckpt", [*[P] * 6, ("f32", 1e-20), P, P, END, *[P] * 5, ("i64", 1 << 60),
                                                         ("i64", T), ("i32", hc), ("i32", dim), END], f)


def _fits(launches):
    return all(x * bx < 1 << 32 and y < 1 << 16 and z == 1 for x, y, z, bx, _, _ in launches)


def _threads(launch):
    x, y, _, bx, _, _ = launch
    return x * y * bx


ROWS = [1, 5, 1000, (1 << 26) + 1, 1 << 31, (1 << 33) + 7]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("K", [128, 1536, 1 << 20])
def test_quantisation_of_any_size(library, rows, K):
    """A thread has 8 columns."""
    status, launches = _quant(library, rows, K)
    if rows * K > 1 << 48:
        assert status == 1 and not launches
        return
    assert status == 0 and len(launches) == 1 and _fits(launches)
    assert _threads(launches[0]) >= rows * K // 8


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D", [8, 40, 5120, 1 << 20])
def test_checkpoints_of_any_size(library, rows, D):
    """A thread has 8 columns; the saving one's rows are padded to whole blocks."""
    for call, cols in ((_save, -(-D // 32) * 32), (_load, D)):
        status, launches = call(library, rows, D)
        if rows * (-(-D // 32) * 32) > 1 << 48:
            assert status == 1 and not launches
            continue
        assert status == 0 and len(launches) == 1 and _fits(launches)
        assert _threads(launches[0]) >= rows * cols // 8


@pytest.mark.parametrize("N,K", [(8, 128), (25600, 1536), (1 << 22, 128), (8, 1 << 20), (1 << 22, 1 << 20)])
def test_packing_of_any_size(library, N, K):
    """A workgroup has a record."""
    status, launches = _pack(library, N, K)
    assert status == 0 and len(launches) == 1 and _fits(launches)
    assert _threads(launches[0]) >= -(-N // 64) * (K // 128) * 256


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(1, 128, 8), (16, 1536, 25600), (17, 1536, 25600), (64, 1536, 25600), (65, 1536, 25600),
                                   (256, 1536, 25600), (257, 1536, 25600), (1 << 20, 1536, 25600), (1 << 30, 128, 8),
                                   (1 << 30, 128, 256), (1 << 32, 128, 1 << 22), (1, 1 << 20, 1 << 22), (100, 128, 512)])
def test_products_of_any_size(library, bits, T, K, N):
    """A wave has 64 columns of a tile's 16 to 128 tokens; what a grid does not hold is more than the card does."""
    status, launches = _wkv(library, bits, T, K, N)
    if status == 1:
        assert not launches and 2 * T * N + T * K * bits // 8 > CARD
        return
    assert status == 0 and len(launches) == 1 and _fits(launches)
    x, y, _, bx, _, _ = launches[0]
    assert any(0 <= x * y - -(-T // m) * -(-N // bx) < x for m in (16, 32, 64, 128))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,hc,dim", [(1, 128, 1, 256), (251, 1536, 4, 5120), (65536, 1536, 4, 5120), (1 << 25, 128, 4, 256),
                                        (1 << 20, 128, 64, 256), (1 << 33, 128, 4, 256), (7, 128, 1, 1 << 21)])
def test_fused_products_of_any_size(library, bits, T, K, hc, dim):
    status, launches = _gate(library, bits, T, K, hc, dim)
    if status == 1:
        assert not launches and 2 * T * hc * dim > CARD
        return
    assert status == 0 and len(launches) == 2 and _fits(launches)
    x, _, _, bx, _, _ = launches[0]
    assert x in [-(-T // m) * ((hc + 1) * dim // bx) for m in (16, 32, 64, 128)] and (hc + 1) * dim % bx == 0


@pytest.mark.parametrize("T,hc,dim", [(1, 1, 8), (8192, 4, 5120), (1 << 22, 4, 1024), (1 << 31, 1, 8), (1 << 30, 3, 8),
                                      (1 << 24, 64, 8), (7, 64, 8192)])
def test_outputs_and_gradients_of_any_size(library, T, hc, dim):
    """A token's copy of the output has 16, 32 or 64 threads up to 1,024 columns, then a workgroup."""
    status, launches = _output(library, T, hc, dim)
    assert status == 0 and len(launches) == 1 and _fits(launches)
    x, y, _, bx, _, _ = launches[0]
    a_row = 16 if dim <= 128 else 32 if dim <= 256 else 64 if dim <= 1024 else bx
    assert x * y >= -(-T * hc // (bx // a_row))
    status, launches = _grad(library, T, hc, dim)
    assert status == 0 and len(launches) == 2 and _fits(launches)


@pytest.mark.parametrize("dim", [8, 256, 1024, 1032, 6144, 6152, 8192])
@pytest.mark.parametrize("T,hc", [(1 << 22, 1), ((1 << 22) + 1, 1), (1 << 23, 1), ((1 << 23) + 3, 3), (1 << 31, 64)])
def test_outputs_of_workgroups_of_any_width(library, T, hc, dim):
    """Past 6,144 columns a workgroup has 512 threads: its rows of the grid are half as long.  The limit itself: as many rows as
    no memory holds."""
    status, launches = _output(library, T, hc, dim)
    assert status == 0 and len(launches) == 1 and _fits(launches)
    x, y, _, bx, _, _ = launches[0]
    a_row = 16 if dim <= 128 else 32 if dim <= 256 else 64 if dim <= 1024 else bx
    assert 0 <= x * y - -(-T * hc // (bx // a_row)) < x
    assert _output(library, (1 << 37) // hc + 1, hc, dim) == (1, [])


CALLS = {
    "quantisation": lambda lib, f: _quant(lib, 251, 1536, f),
    "packing": lambda lib, f: _pack(lib, 25600, 1536, f),
    **{f"product of {T} tokens, {b}": lambda lib, f, T=T, b=b: _wkv(lib, b, T, 1536, 25600, f)
       for T in (1, 33, 200, 8192) for b in (4, 8)},
    **{f"fused product of {T} tokens, {b}": lambda lib, f, T=T, b=b: _gate(lib, b, T, 1536, 4, 5120, f)
       for T in (1, 33, 200, 8192) for b in (4, 8)},
    "saving": lambda lib, f: _save(lib, 1000, 40, f),
    "loading": lambda lib, f: _load(lib, 1000, 40, f),
    **{f"output of {d}": lambda lib, f, d=d: _output(lib, 100, 4, d, f) for d in (256, 4096, 5120, 8192)},
    **{f"gradient of {h} copies": lambda lib, f, h=h: _grad(lib, 100, h, 256, f) for h in (1, 2, 3, 4)},
    "gradient of no tokens": lambda lib, f: _grad(lib, 0, 4, 256, f),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_failed_launch_is_reported(library, name):
    status, launches = CALLS[name](library, None)
    assert status == 0 and launches
    for i in range(len(launches)):
        assert CALLS[name](library, i)[0] == EHIP, f"launch {i} of {len(launches)}: {launches[i]}"
