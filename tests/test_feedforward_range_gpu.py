"""Feed-forward operators on values far from one, against the fp64 oracle.

Tolerances are those of the formats and of the order of operations (the same
as for values of order one): a bf16 output is within 2^-8 of its magnitude, an
fp32 chain of a few roundings within 2^-20 of its terms' magnitudes.
"""

import numpy as np
import pytest

from gpu_helpers import require_gpu, torch
import mixed_precision_optimizer_gb300 as mp
from oracle import feedforward as O

pytestmark = pytest.mark.gpu

BF16, REL32 = 2.0 ** -8, 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, shape, dtype=torch.bfloat16, std=1.0, off=0):
    """Normal values; `off`: a slice that starts so many elements into rows 8 wider."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    wide = tuple(shape[:-1]) + (shape[-1] + (8 if off else 0),)
    t = (torch.randn(wide, generator=g, device="cuda", dtype=torch.float64) * std).to(dtype)
    return t[..., off:off + shape[-1]]


def np64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what=""):
    got = np64(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) / np.maximum(bound, 1e-300)
    assert (over <= 1).all(), f"{what}: {int((over > 1).sum())} of {over.size} beyond the bound, worst {over.max():.3g} times"


# a width for every kernel of the gradient: a warp's row of one, two and four groups,
# rows of 128 to 512 threads (bf16 ones through the ring), and rows in shared memory; odd
# widths and slices that share a shift, and slices that do not
@pytest.mark.parametrize("rows,cols,dy_off,h_off", [
    (40, 64, 0, 0), (40, 512, 0, 0), (40, 1024, 0, 0), (700, 2048, 0, 0), (9, 4096, 0, 0), (9, 8192, 0, 0), (5, 14336, 0, 0),
    (40, 251, 0, 0), (40, 505, 0, 0), (40, 1017, 0, 0), (40, 2545, 3, 3), (9, 8187, 0, 0),
    (40, 250, 1, 2), (40, 1023, 1, 2), (9, 4089, 1, 2), (3, 16391, 0, 0), (3, 20000, 0, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e-14, 1e14, 1e16])
def test_norm_gradient_of_rows_of_any_magnitude(rows, cols, dy_off, h_off, dtype, size):
    """dx = rstd (g - n mean(g n)): n = h rstd is of order one whatever h's
    magnitude, so a row of 1e-14 (eps = 0), 1e14 or 1e16 keeps its projection."""
    dy, h, gamma = normal(1, (rows, cols), off=dy_off), normal(2, (rows, cols), dtype, size, h_off), normal(3, (cols,)) + 1
    y, rstd = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, device="cuda")
    mp.rmsnorm(h, gamma, 0.0, y=y, rstd=rstd)
    wr = 1 / np.sqrt(np.mean(np64(h) ** 2, 1))
    within(rstd, wr, REL32 * wr, "rstd")
    within(y, O.rmsnorm(np64(h), np64(gamma), 0.0)[1], (BF16 + REL32) * np.abs(O.rmsnorm(np64(h), np64(gamma), 0.0)[1]), "y")
    dx, dgamma = torch.full((rows, cols), float("nan"), dtype=dtype, device="cuda"), torch.empty(cols, device="cuda")
    mp.rmsnorm_backward(dy, h, gamma, rstd, dx, dgamma=dgamma, accumulate=False, workspace=mp.rmsnorm_workspace(rows, cols))
    wx, wg = O.rmsnorm_backward(np64(dy), np64(h), np64(gamma), np64(rstd))
    n, g = np64(h) * np64(rstd)[:, None], np64(dy) * np64(gamma)
    mag = np64(rstd)[:, None] * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), 1, keepdims=True))
    within(dx, wx, (BF16 if dtype == torch.bfloat16 else 0) * np.abs(wx) + 2 * REL32 * mag, "dx")
    within(dgamma, wg, (rows + 8) * 2.0 ** -23 * np.sum(np.abs(np64(dy) * n), 0), "dgamma")


# the split kernel with the lanes on columns (16, 32 and 64 rows) and on rows, the pair
# kernel, and clusters of pairs; rows that move in 16-byte pieces and others
@pytest.mark.parametrize("m,n,k", [(5, 64, 200), (30, 64, 200), (60, 1024, 200), (130, 128, 264), (2100, 100, 2300),
                                   (1000, 2200, 1500), (40, 64, 201)])
@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_activation_gradient_of_large_values(m, n, k, kind):
    """The derivative of gelu and silu is 1 or 0 far from zero, up to the
    largest finite pre-activation."""
    dz, w = normal(1, (m, n)), normal(2, (n, k), std=0.1)
    far = torch.tensor([-3e38, -1e20, -3e19, -1e13, -60.0, 60.0, 1e13, 3e19, 1e20, 3e38], device="cuda")
    z = far[torch.arange(m * k, device="cuda") % 10].to(torch.bfloat16).view(m, k)
    dx = torch.full((m, k), float("nan"), dtype=torch.bfloat16, device="cuda")
    mp.linear_backward(dz, None, w, dx=dx, z_prev=z, act_prev=kind, workspace=mp.linear_workspace(m, n, k))
    plain = np64(dz) @ np64(w)
    want = plain * O.act_grad(np64(z), kind)
    err = (n + 8) * 2.0 ** -23 * (np.abs(np64(dz)) @ np.abs(np64(w)))
    within(dx, want, BF16 * (np.abs(want) + err) + err, "dx")


# dw of 16384 tokens by each kernel: pairs with a last wave of clusters, clusters alone, pairs with tiles
# of 128 columns, and the split kernel with one and with two CTAs to a tile
@pytest.mark.parametrize("n,k", [(2560, 2560), (1280, 1280), (19456, 100), (128, 10240), (128, 8192)])
def test_weight_gradient_is_summed_in_segments(n, k):
    """The tensor cores truncate each addition to the accumulator, 16 tokens at
    a time.  Of positive terms an addition loses half a unit (2^-24 of the
    partial sum) on average and the partial sum is half of the final one: 1024
    additions in a row come out low by 1.5e-5 or more.  A segment of 768 tokens
    is 48 additions, at most 48 * 2^-25 = 1.4e-6, and the rounding additions of
    the segments do not add up; twice that is the bound."""
    m = 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dz = torch.rand((m, n), generator=g, device="cuda").add_(0.5).to(torch.bfloat16)
    x = torch.rand((m, k), generator=g, device="cuda").add_(0.5).to(torch.bfloat16)
    dw = torch.full((n, k), float("nan"), device="cuda")
    mp.linear_backward(dz, x, None, dw=dw, accumulate=False, workspace=mp.linear_workspace(m, n, k))
    rows = torch.arange(0, n, max(1, n // 500), device="cuda")          # rows of every tile
    want = dz[:, rows].double().t() @ x.double()
    rel = float((dw[rows].double() - want).norm() / want.norm())
    assert rel < 2 * 48 * 2.0 ** -25, rel
