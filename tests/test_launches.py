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
