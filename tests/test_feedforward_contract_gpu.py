"""What the feed-forward operators promise about workspaces, on the GPU."""

import pytest

from gpu_helpers import require_gpu, torch
import mixed_precision_optimizer_gb300 as mp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def layer(m, n, k, ws):
    """Forward and backward of one layer in this workspace; its outputs."""
    x, w, dz = normal(1, m, k), normal(2, n, k, std=0.1), normal(3, m, n)
    y, dx = torch.empty_like(dz), torch.empty_like(x)
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    mp.linear(x, w, y, act="silu", workspace=ws)
    mp.linear_backward(dz, x, w, dx=dx, dw=dw, dbias=db, accumulate=False, workspace=ws)
    assert mp.device_status(ws) == mp.OPT_OK
    return y, dx, dw, db


@pytest.mark.parametrize("size,any_layout,calls", [
    ((8192, 9728, 2560), False, [(8192, 2560, 2560), (8192, 2048, 512), (4096, 9728, 512), (300, 512, 64), (8192, 9728, 2560)]),
    ((1024, 4096, 4096), True, [(100, 777, 1001), (1024, 4095, 1023), (1023, 1, 4095), (1, 4093, 3), (1000, 1023, 4095),
                                (700, 1024, 1024)])])
def test_one_workspace_for_smaller_sizes(size, any_layout, calls):
    """Each call has the bits that it has in a workspace of its own."""
    shared = mp.linear_workspace(*size, any_layout=any_layout)
    shared[mp.feedforward.LINEAR_HEADER_BYTES:].fill_(0xFF)
    for c in calls:
        for a, b in zip(layer(*c, shared), layer(*c, mp.linear_workspace(*c))):
            assert torch.equal(a, b), c


def test_the_two_products_of_a_block_share_the_larger_workspace():
    tokens, hidden, width = 8192, 9728, 2560
    ws = max(mp.linear_workspace(tokens, hidden, width), mp.linear_workspace(tokens, width, hidden), key=torch.numel)
    layer(tokens, hidden, width, ws)
    layer(tokens, width, hidden, ws)


# words of the header: the tile counter, the CTAs that have finished, the tiles claimed
@pytest.mark.parametrize("words", [{32: 5}, {32: 0x7FFFFFFF}, {32: -2 ** 31}, {32: -1}, {33: 3}, {33: -1}, {34: 7},
                                   {32: -16, 33: 151, 34: -1}])
@pytest.mark.parametrize("shape", [(2100, 2300, 100), (4096, 2560, 264)])
def test_a_header_that_is_not_zero_is_reported(shape, words):
    """A large product in such a workspace ends, writes nothing outside its
    output, and opt_device_status reports the workspace; zeroed, it works again.
    (A counter of -1 costs one CTA pair its share; the others compute every tile.)"""
    m, n, k = shape
    x, w = normal(1, m, k), normal(2, n, k, std=0.1)
    want, ws = torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), mp.linear_workspace(m, n, k)
    mp.linear(x, w, want, workspace=ws)
    assert mp.device_status(ws) == mp.OPT_OK and not ws[:256].any()
    header = ws[:256].view(torch.int32)
    for i, v in words.items():
        header[i] = v
    wide = torch.full((m + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
    y = wide[1:-1]
    mp.linear(x, w, y, workspace=ws)
    status = mp.device_status(ws)
    assert status == mp.OPT_ERR_WORKSPACE or (words == {32: -1} and status == mp.OPT_OK and torch.equal(y, want))
    assert ((y == want) | (y == 7)).all() and (wide[0] == 7).all() and (wide[-1] == 7).all()
    header.zero_()
    mp.linear(x, w, y, workspace=ws)
    assert mp.device_status(ws) == mp.OPT_OK and torch.equal(y, want)
