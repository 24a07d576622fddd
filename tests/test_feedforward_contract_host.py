"""What the feed-forward operators promise about their workspaces and check
about their arguments, without a GPU."""

import itertools

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_optimizer_gb300 as mp
from mixed_precision_optimizer_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()


ROWS = [0, 1, 100, 256, 257, 2048, 8192, 16384, 16385, 100000]
ALIGNED = [16, 512, 1024, 2560, 4096, 5120, 9728, 14336, 19456, 77808, 77824, 128256]
ANY = [1, 7, 63, 777, 1023, 4097, 9727, 38911, 77823, 77825]


@pytest.mark.parametrize("any_layout", [False, True])
def test_linear_workspace_serves_smaller_sizes(any_layout):
    """A size is at least that of every call whose m, n and k are none larger:
    with any_layout for all widths, without it for those that need no copy."""
    widths = sorted(ALIGNED + ANY) if any_layout else ALIGNED
    size = {s: mp.linear_workspace_size(*s, any_layout=any_layout) for s in itertools.product(ROWS, widths, widths)}
    for axis in range(3):
        for s in size:
            values = (ROWS, widths, widths)[axis]
            i = values.index(s[axis])
            if i:                                    # one step down each axis: the rest follows
                smaller = s[:axis] + (values[i - 1],) + s[axis + 1:]
                assert size[smaller] <= size[s], (smaller, s)


def test_linear_workspace_of_every_width():
    """The same in steps of one column past each change of the slices, where
    the bias gradient's partial sums go up and down."""
    for m in (512, 8192, 16384):
        sizes = [mp.linear_workspace_size(m, n, 16, any_layout=True) for n in range(1, 20000, 7)]
        assert sizes == sorted(sizes)
    # aligned widths, and the two orders of a block's products
    assert mp.linear_workspace_size(8192, 128256, 4096) >= mp.linear_workspace_size(8192, 4096, 4096)
    assert mp.linear_workspace_size(8192, 9728, 2560) >= mp.linear_workspace_size(8192, 2560, 9728)
    assert mp.linear_workspace_size(128, 4096, 4096, any_layout=True) >= mp.linear_workspace_size(128, 4096, 1023)
