"""The launches of the training entry points at sizes that no test allocates: every grid within the runtime's limit, all of
the work covered, every launch's failure reported."""
import shutil

import pytest

from tests.launches import Library

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not installed")
AT = 1 << 40  # a device address; nothing follows it
EHIP = 3


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    with Library(tmp_path_factory.mktemp("launches")) as lib:
        yield lib


def _lists(sizes, kinds):
    n = len(sizes)
    return [("i32", n), ("p[]", [AT] * n)], [("i64[]", sizes), ("i32[]", kinds)]


def _clip(library, sizes, kinds, fail_at=None):
    head, tail = _lists(sizes, kinds)
    return library.call("engram_clip_grads", [*head, ("p[]", [AT] * len(sizes)), *tail, ("p", AT), ("f32", 1.0), ("p", None)],
                        fail_at)


@pytest.mark.parametrize("sizes,kinds", [
    ([384006168 * 64], [1]),                       # the dense float32 gradient of the released table: 98 GB
    ([384006168 * 64], [0]),
    ([1 << 40], [1]),                              # the documented limit
    ([1 << 33] * 9, [0] * 9),                      # a list of 144 GB of smaller tensors
    ([5, (1 << 34) + 3, 0, 7, (1 << 34) - 1024], [1, 1, 0, 0, 1]),
    ([1 << 24] * 3000, [1] * 3000),
    ([1000, 3000], [0, 1]),
])
def test_clip_of_any_size(library, sizes, kinds):
    """A workgroup clips 256 pieces of 16 bytes: together the launches have one for every such run of every tensor."""
    status, launches = _clip(library, sizes, kinds)
    assert status == 0
    runs = sum(-(-n * (4 if k else 2) // 4096) for n, k in zip(sizes, kinds))
    assert all(x * bx < 1 << 32 for x, _, _, bx, _, _ in launches)
    assert sum(x for x, *_ in launches) == runs


def test_clip_stops_at_a_launch_that_fails(library):
    """In place, gradients behind a failed launch are left as they were."""
    for fail_at in range(3):
        status, launches = _clip(library, [1 << 20] * 250, [1] * 250, fail_at)  # 96 tensors a launch
        assert status == EHIP and len(launches) == fail_at + 1


@pytest.mark.parametrize("sizes,kinds", [([1 << 40], [1]), ([1 << 38] * 3, [0] * 3), ([7, 100000], [0, 1])])
def test_norm_of_any_size(library, sizes, kinds):
    head, tail = _lists(sizes, kinds)
    status, launches = library.call("engram_grad_norm", [*head, *tail, ("p", AT), ("p", AT), ("i64", 1 << 50), ("p", None)])
    assert status == 0
    assert sum(x for x, *_ in launches[:-1]) == sum(-(-n * (4 if k else 2) // 65536) for n, k in zip(sizes, kinds))


def _dense(library, n, R, D, fail_at=None, C=1, kind=1):
    return library.call("engram_embed_grad", [
        ("p", AT), ("i32", 8), ("i64", n // C), ("i64", C), ("i32", C), ("p", AT), ("i32", 0), ("i64", R), ("i64", 0), ("i32", D),
        ("f32", 1.0), ("p", AT), ("i32", kind), ("i32", 0), ("p", AT), ("i64", 1 << 60), ("p", None)], fail_at)


def _rows(library, n, R, D, fail_at=None):
    return library.call("engram_embed_grad_rows", [
        ("p", AT), ("i32", 8), ("i64", n), ("i64", 1), ("i32", 1), ("p", AT), ("i32", 0), ("i64", R), ("i64", 0), ("i32", D),
        ("f32", 1.0), ("p", AT), ("p", AT), ("i32", 1), ("p", AT), ("p", AT), ("i64", 1 << 60), ("p", None)], fail_at)


def _embed(library, n, D, fail_at=None):
    return library.call("engram_embed", [("p", AT), ("i32", 8), ("i64", n), ("p", AT), ("i32", 0), ("i64", 1000), ("i64", 0),
                                         ("i32", D), ("f32", 1.0), ("p", AT), ("i32", 0), ("p", None)], fail_at)


def _gate(library, T, hc, dim, fail_at=None):
    return library.call("engram_gate_output_backward", [
        ("p", AT), ("p", AT), ("i64", (hc + 1) * dim), ("p", AT), ("p", AT), ("f32", 1e-20), ("p", AT), ("p", AT), ("p", None),
        *[("p", AT)] * 5, ("i64", 1 << 60), ("i64", T), ("i32", hc), ("i32", dim), ("p", None)], fail_at)


def _wkv(library, T, K, N, fail_at=None, da=AT, dw=AT):
    return library.call("engram_wkv_backward", [
        ("p", AT), ("p", AT), ("p", AT), ("p", da), ("p", dw), ("i32", 1), ("i32", 0), ("p", AT), ("i64", 1 << 60), ("i64", T),
        ("i32", K), ("i32", N), ("p", None)], fail_at)


def _norm(library, sizes, fail_at=None):
    head, tail = _lists(sizes, [1] * len(sizes))
    return library.call("engram_grad_norm", [*head, *tail, ("p", AT), ("p", AT), ("i64", 1 << 60), ("p", None)], fail_at)


BIG = 384006168  # the released table's rows: 98 GB of float32 zeros, more than a launch of the sort writes beside it
CALLS = {
    "lookup": lambda lib, f: _embed(lib, 1000, 64, f),
    "dense, no ids": lambda lib, f: _dense(lib, 0, 100, 64, f),
    "dense, few ids": lambda lib, f: _dense(lib, 100, 100, 64, f),
    "dense, one workgroup's sort": lambda lib, f: _dense(lib, 3000, 100, 64, f),
    "dense, one workgroup's sort, big": lambda lib, f: _dense(lib, 3000, BIG, 64, f),
    "dense, sort over tiles": lambda lib, f: _dense(lib, 300000, 100, 64, f),
    "dense, sort over tiles, big": lambda lib, f: _dense(lib, 30000, BIG, 64, f),
    "rows, no ids": lambda lib, f: _rows(lib, 0, 100, 64, f),
    "rows, few ids": lambda lib, f: _rows(lib, 100, 100, 64, f),
    "rows, one workgroup's sort": lambda lib, f: _rows(lib, 3000, 100, 64, f),
    "rows, sort over tiles": lambda lib, f: _rows(lib, 600000, BIG, 64, f),
    "gate": lambda lib, f: _gate(lib, 100, 4, 256, f),
    "gate, any copies": lambda lib, f: _gate(lib, 100, 3, 256, f),
    "gate, no tokens": lambda lib, f: _gate(lib, 0, 4, 256, f),
    "projection": lambda lib, f: _wkv(lib, 251, 1536, 25600, f),
    "projection, no tokens": lambda lib, f: _wkv(lib, 0, 64, 64, f),
    "norm": lambda lib, f: _norm(lib, [1000] * 200, f),
    "clip": lambda lib, f: _clip(lib, [1000] * 200, [1] * 200, f),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_failed_launch_is_reported(library, name):
    status, launches = CALLS[name](library, None)
    assert status == 0 and launches
    for i in range(len(launches)):
        assert CALLS[name](library, i)[0] == EHIP, f"launch {i} of {len(launches)}: {launches[i]}"


@pytest.mark.parametrize("n", [600, 9000, 1 << 20, (1 << 28) + 1, 1 << 30])
@pytest.mark.parametrize("D", [8, 32, 64, 128, 256, 264, 512, 520, 4096, 5120, 65536])
def test_embedding_gradients_of_any_size(library, n, D):
    """All ids that 288 GB can hold rows of are taken; what a grid does not hold is refused before anything is launched."""
    for call in (lambda: _dense(library, n, 1000, D), lambda: _rows(library, n, 1000, D)):
        status, launches = call()
        assert status in (0, 1)
        assert status == 0 or (not launches and n * D * 2 > 288 << 30), (n, D)
    for m in (n, 16 * n):
        status, launches = _embed(library, m, D)
        assert status == 0 or (status == 1 and not launches and m * D * 2 > 288 << 30), (m, D)


@pytest.mark.parametrize("T,K,N", [
    (1, 8, 8), (251, 1536, 25600), (1 << 30, 8, 8), (1 << 30, 64, 64), (1 << 30, 264, 264), (1 << 27, 1536, 256),
    (1 << 30, 1 << 20, 8), (1 << 30, 8, 1 << 21), (1, 1 << 20, 1 << 21), (1 << 30, 1 << 20, 1 << 21)])
@pytest.mark.parametrize("da,dw", [(AT, AT), (AT, None), (None, AT)])
def test_projection_gradients_of_any_size(library, T, K, N, da, dw):
    status, launches = _wkv(library, T, K, N, da=da, dw=dw)
    held = 2 * (T * N + (T * K if da else 0) + (T * K if dw else 0) + (N * K if da else 0)) + (4 * N * K if dw else 0)
    assert status == 0 or (status == 1 and not launches and held > 288 << 30)


@pytest.mark.parametrize("T,hc,dim", [(1 << 20, 4, 8192), (1 << 31, 1, 8), (1 << 30, 3, 8), (1 << 24, 64, 8), (7, 64, 8192)])
def test_gate_gradients_of_any_size(library, T, hc, dim):
    assert _gate(library, T, hc, dim)[0] == 0
