"""Feed-forward operators on the GPU against the fp64 oracle.

Tolerances, from the formats and the order of operations:

* a bf16 output is one rounding of an fp32 value: half a unit in the last
  place is at most 2^-8 of its magnitude (BF16);
* an fp32 sum of k products differs from the exact one by at most
  (k + 8) 2^-23 sum |a b| (ACC: additions that round or truncate);
* an activation changes by at most 1.13 times its argument's error and its own
  evaluation (exp and a division, 2 units each) adds 2^-19 of the value;
* a norm's fp32 chain of four roundings and one square root of a mean is
  within 2^-20 of the value;
* an e4m3 code is the nearest one to a quotient that is within 2^-20 of the
  oracle's, so it may differ by one step where the quotient lies that close to
  a midpoint; the step is at most 1/8 of the value (2^-9 below 2^-6), and all
  other codes are equal.
"""

import numpy as np
import pytest

from gpu_helpers import host, require_gpu, torch
import mixed_precision_optimizer_gb300 as mp
from oracle import feedforward as O

pytestmark = pytest.mark.gpu

BF16, REL32, ACT = 2.0 ** -8, 2.0 ** -20, 2.0 ** -19


def ACC(k):
    return (k + 8) * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(seed, shape, dtype=torch.bfloat16, std=1.0, pad=0, off=0):
    """Normal values; pad / off: a slice that starts `off` elements into rows
    `pad` elements wider."""
    wide = tuple(shape[:-1]) + (shape[-1] + pad,)
    t = (torch.randn(wide, generator=gen(seed), device="cuda") * std).to(dtype)
    return t[..., off:off + shape[-1]]


def np64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what=""):
    got, want = np64(got) if torch.is_tensor(got) else got, np.asarray(want)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound, worst by {over.max():.3g}"


def empty(shape, dtype=torch.bfloat16):
    """Output buffers start as NaN: an element that is not written shows."""
    if dtype == torch.float8_e4m3fn:
        return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(dtype)
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def check_codes(q, scale, y, what=""):
    """e4m3 codes and scales of rows y (fp64)."""
    want_scale = O.row_scale(y)
    within(scale, want_scale, 4 * REL32 * want_scale, what + " scale")
    v = y / want_scale[:, None]
    got = np64(q.float())
    lo, hi = O.e4m3_rne(v * (1 - 4 * REL32)), O.e4m3_rne(v * (1 + 4 * REL32))
    ok = (got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi))
    assert ok.all(), f"{what}: {int((~ok).sum())} codes are not the nearest one"


# ------------------------------------------------------------------- norm --

NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 128), (2, 1023), (33, 1024), (7, 1111), (1, 4096), (300, 4096), (2, 4104),
               (1031, 136), (2, 14336), (3, 16384), (1, 16391), (2, 49152), (700, 64)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["dense", "aligned slice", "odd slice"])
def test_rmsnorm(rows, cols, dtype, layout):
    pad, off = {"dense": (0, 0), "aligned slice": (24, 8), "odd slice": (5, 3)}[layout]
    x = normal(1, (rows, cols), dtype, 1.0, pad, off)
    r = normal(2, (rows, cols), dtype, 2.0, pad, off) if layout != "aligned slice" else None
    gamma = normal(3, (cols,), torch.bfloat16 if cols % 2 else torch.float32) + 1
    h, y = empty((rows, cols + pad), dtype)[:, off:off + cols], empty((rows, cols + pad))[:, off:off + cols]
    q, s, rstd = empty((rows, cols), torch.float8_e4m3fn), empty((rows,), torch.float32), empty((rows,), torch.float32)
    mp.rmsnorm(x, gamma, 1e-5, residual=r, h=h, y=y, q=q, q_scale=s, rstd=rstd)
    wh, wy, wr = O.rmsnorm(np64(x), np64(gamma), 1e-5, None if r is None else np64(r))
    within(rstd, wr, REL32 * wr, "rstd")
    within(h, wh, (BF16 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(wh), "h")
    within(y, wy, (BF16 + REL32) * np.abs(wy), "y")
    # the codes: y's relative error is REL32 plus that of h (2^-24 of |x| + |r| where the sum cancels)
    if r is None:
        check_codes(q, s, wy, "q")
    else:
        v = wy / O.row_scale(wy)[:, None]
        cancel = 2.0 ** -23 * (np.abs(np64(x)) + np.abs(np64(r))) / np.maximum(np.abs(wh), 1e-30)
        d = np.abs(v) * (4 * REL32 + cancel)
        got = np64(q.float())
        assert ((got >= O.e4m3_rne(v - d)) & (got <= O.e4m3_rne(v + d))).all()


@pytest.mark.parametrize("rows,cols", [(1, 4096), (9, 1000), (2, 49152)])
def test_rmsnorm_outputs_do_not_depend_on_each_other(rows, cols):
    """Each output alone has the bits that it has beside the others, and h may
    be x or the residual in place."""
    x, r, gamma = normal(1, (rows, cols)), normal(2, (rows, cols)), normal(3, (cols,))
    h, y, q = empty((rows, cols)), empty((rows, cols)), empty((rows, cols), torch.float8_e4m3fn)
    s, rstd = empty((rows,), torch.float32), empty((rows,), torch.float32)
    mp.rmsnorm(x, gamma, residual=r, h=h, y=y, q=q, q_scale=s, rstd=rstd)
    y1, q1, s1, r1 = empty((rows, cols)), empty((rows, cols), torch.float8_e4m3fn), s.clone().zero_(), rstd.clone().zero_()
    mp.rmsnorm(x, gamma, residual=r, y=y1)
    mp.rmsnorm(x, gamma, residual=r, q=q1, q_scale=s1)
    mp.rmsnorm(x, gamma, residual=r, rstd=r1)
    for a, b in ((y, y1), (q, q1), (s, s1), (rstd, r1)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for k in range(2):
        xc, rc = x.clone(), r.clone()
        mp.rmsnorm(xc, gamma, residual=rc, h=(xc, rc)[k], y=y1)
        assert torch.equal((xc, rc)[k].view(torch.uint8), h.view(torch.uint8))
        assert torch.equal(y1.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal((rc, xc)[k].view(torch.uint8), (r, x)[k].view(torch.uint8))


def test_rmsnorm_special_rows():
    """Zeros with eps = 0 are 0 * inf = NaN and with eps > 0 zeros (scale at
    the floor); a NaN or an infinity stays in its row."""
    cols = 1000
    x = normal(1, (5, cols))
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 5] = float("inf")
    gamma = torch.ones(cols, device="cuda")
    y, q, s = empty((5, cols)), empty((5, cols), torch.float8_e4m3fn), empty((5,), torch.float32)
    mp.rmsnorm(x, gamma, 1e-6, y=y, q=q, q_scale=s)
    yh = np64(y)
    assert np.isfinite(yh[[0, 1, 4]]).all() and (yh[1] == 0).all() and (np64(q.float())[1] == 0).all()
    assert float(s[1]) == pytest.approx(1e-30 / 448, rel=1e-6)
    assert np.isnan(yh[2]).all() and np.isnan(np64(q.float())[2]).all()
    assert np.isnan(yh[3, 5]) and (np.delete(yh[3], 5) == 0).all()
    mp.rmsnorm(x, gamma, 0.0, y=y)
    assert np.isnan(np64(y)[1]).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (64, 128), (1, 4096), (700, 1023), (1031, 136), (2, 14336),
                                       (330, 2048), (3, 24576), (2, 16391), (4000, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["dense", "odd slice"])
def test_rmsnorm_backward(rows, cols, dtype, layout):
    pad, off = {"dense": (0, 0), "odd slice": (5, 3)}[layout]
    dy, h = normal(1, (rows, cols), torch.bfloat16, 1, pad, off), normal(2, (rows, cols), dtype, 3, pad, off)
    dh = normal(3, (rows, cols), dtype, 1, pad, off) if layout == "dense" else None
    gamma = normal(4, (cols,)) + 1
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    dx, dgamma = empty((rows, cols + pad), dtype)[:, off:off + cols], empty((cols,), torch.float32)
    ws = mp.rmsnorm_workspace(rows, cols)
    mp.rmsnorm_backward(dy, h, gamma, rstd, dx, dh=dh, dgamma=dgamma, accumulate=False, workspace=ws)
    wx, wg = O.rmsnorm_backward(np64(dy), np64(h), np64(gamma), np64(rstd), None if dh is None else np64(dh))
    n, g = np64(h) * np64(rstd)[:, None], np64(dy) * np64(gamma)
    # the terms g and n c may cancel: their own magnitudes bound the fp32 error
    mag = np64(rstd)[:, None] * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), 1, keepdims=True))
    mag = mag + (0 if dh is None else np.abs(np64(dh)))
    out = (BF16 if dtype == torch.bfloat16 else 0) * np.abs(wx)
    within(dx, wx, out + 2 * REL32 * mag, "dx")
    gmag = np.sum(np.abs(np64(dy) * n), 0)
    within(dgamma, wg, ACC(rows) * gmag, "dgamma")
    old = normal(5, (cols,), torch.float32)
    acc = old.clone()
    mp.rmsnorm_backward(dy, h, gamma, rstd, None, dgamma=acc, workspace=ws)
    within(acc, wg + np64(old), ACC(rows) * gmag + 2.0 ** -23 * (np.abs(wg) + np.abs(np64(old))), "dgamma +=")
    dx2 = dx.clone().fill_(float("nan"))
    mp.rmsnorm_backward(dy, h, gamma, rstd, dx2, dh=dh)
    assert torch.equal(dx2, dx)


def test_rmsnorm_backward_in_place_and_no_rows():
    dy, h, dh, gamma = normal(1, (40, 512)), normal(2, (40, 512)), normal(3, (40, 512)), normal(4, (512,))
    rstd = torch.rsqrt(h.float().square().mean(1))
    dx = empty((40, 512))
    mp.rmsnorm_backward(dy, h, gamma, rstd, dx, dh=dh)
    inplace = dh.clone()
    mp.rmsnorm_backward(dy, h, gamma, rstd, inplace, dh=inplace)
    assert torch.equal(inplace, dx)
    g = torch.full((512,), 3.0, device="cuda")
    none = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    mp.rmsnorm_backward(none, none, gamma, rstd[:0], none, dgamma=g)
    assert (g == 3).all()
    mp.rmsnorm_backward(none, none, gamma, rstd[:0], none, dgamma=g, accumulate=False)
    assert (g == 0).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 16), (777, 1111), (64, 4096), (2, 14336), (3, 49152), (1000, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["dense", "odd slice"])
def test_quantize_rows(rows, cols, dtype, layout):
    pad, off = {"dense": (0, 0), "odd slice": (5, 3)}[layout]
    x = normal(7, (rows, cols), dtype, 0.02, pad, off)
    if rows > 2:
        x[1] = 0
    q, s = empty((rows, cols), torch.float8_e4m3fn), empty((rows,), torch.float32)
    mp.quantize_rows(x, q, s)
    check_codes(q, s, np64(x))


# widths on both sides of each kernel's span, where 7 more columns take the next one
ODD_ROWS = [(1, 9), (9, 15), (700, 249), (20, 250), (5000, 251), (17, 505), (3, 506), (1300, 1017), (9, 1018), (40, 2041),
            (9, 2042), (900, 2545), (5, 4089), (9, 4090), (9, 8185), (700, 8187), (9, 16377), (9, 16378)]


def framed(rows, cols, dtype, off=3, pad=8):
    """A buffer of ones around rows of NaN that start `off` elements into it."""
    wide = torch.ones((rows, cols + pad), dtype=torch.float32, device="cuda").to(dtype)
    t = wide[:, off:off + cols]
    t.copy_(torch.full((rows, cols), float("nan"), device="cuda").to(dtype))
    return wide, t


def frame_intact(wide, cols, off=3):
    w = wide.float()
    return bool((w[:, :off] == 1).all()) and bool((w[:, off + cols:] == 1).all())


@pytest.mark.parametrize("rows,cols", ODD_ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("framing", [False, True])
def test_rmsnorm_rows_with_one_shift(rows, cols, dtype, framing):
    """All rows of a row index start equally far past a multiple of 8 elements:
    every value is right and nothing beside the rows is written."""
    pad, off = (8, 3) if framing else (0, 0)
    x, r = normal(1, (rows, cols), dtype, 1.0, pad, off), normal(2, (rows, cols), dtype, 2.0, pad, off)
    gamma = normal(3, (cols,), torch.bfloat16 if cols % 2 else torch.float32) + 1
    (hw, h), (yw, y), (qw, q) = (framed(rows, cols, t, off, pad) for t in (dtype, torch.bfloat16, torch.float8_e4m3fn))
    s, rstd = empty((rows,), torch.float32), empty((rows,), torch.float32)
    mp.rmsnorm(x, gamma, 1e-5, residual=r, h=h, y=y, rstd=rstd)
    wh, wy, wr = O.rmsnorm(np64(x), np64(gamma), 1e-5, np64(r))
    within(rstd, wr, REL32 * wr, "rstd")
    within(h, wh, (BF16 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(wh), "h")
    within(y, wy, (BF16 + REL32) * np.abs(wy), "y")
    mp.rmsnorm(x, gamma, 1e-5, q=q, q_scale=s)
    check_codes(q, s, O.rmsnorm(np64(x), np64(gamma), 1e-5, None)[1], "q")
    mp.quantize_rows(x, q, s)
    check_codes(q, s, np64(x), "rows")
    assert frame_intact(hw, cols, off) and frame_intact(yw, cols, off) and frame_intact(qw, cols, off)


@pytest.mark.parametrize("rows,cols", ODD_ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("framing", [False, True])
def test_rmsnorm_backward_rows_with_one_shift(rows, cols, dtype, framing):
    pad, off = (8, 3) if framing else (0, 0)
    dy, h = normal(1, (rows, cols), torch.bfloat16, 1, pad, off), normal(2, (rows, cols), dtype, 3, pad, off)
    dh = normal(3, (rows, cols), dtype, 1, pad, off)
    gamma = normal(4, (cols,)) + 1
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    (xw, dx), dgamma = framed(rows, cols, dtype, off, pad), empty((cols,), torch.float32)
    ws = mp.rmsnorm_workspace(rows, cols)
    mp.rmsnorm_backward(dy, h, gamma, rstd, dx, dh=dh, dgamma=dgamma, accumulate=False, workspace=ws)
    wx, wg = O.rmsnorm_backward(np64(dy), np64(h), np64(gamma), np64(rstd), np64(dh))
    n, g = np64(h) * np64(rstd)[:, None], np64(dy) * np64(gamma)
    mag = np64(rstd)[:, None] * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), 1, keepdims=True)) + np.abs(np64(dh))
    within(dx, wx, (BF16 if dtype == torch.bfloat16 else 0) * np.abs(wx) + 2 * REL32 * mag, "dx")
    within(dgamma, wg, ACC(rows) * np.sum(np.abs(np64(dy) * n), 0), "dgamma")
    assert frame_intact(xw, cols, off)
    inplace = dh.clone()
    if not framing:                                  # dx in dh's place
        mp.rmsnorm_backward(dy, h, gamma, rstd, inplace, dh=inplace)
        assert torch.equal(inplace, dx)


@pytest.mark.parametrize("rows,cols", [(9, 505), (700, 1023), (40, 2545), (9, 8187)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_gradient_does_not_depend_on_where_dx_lies(rows, cols, dtype):
    x, r, dy, gamma = normal(1, (rows, cols), dtype), normal(2, (rows, cols), dtype), normal(3, (rows, cols)), normal(4, (cols,))
    rstd = torch.rsqrt(x.float().square().mean(1))
    runs = []
    for pad, off in ((0, 0), (5, 3), (8, 1)):
        (wide, dx), dgamma = framed(rows, cols, dtype, off, pad), empty((cols,), torch.float32)
        mp.rmsnorm_backward(dy, x, gamma, rstd, dx, dh=r, dgamma=dgamma, accumulate=False,
                            workspace=mp.rmsnorm_workspace(rows, cols))
        assert frame_intact(wide, cols, off)
        runs.append((dx.float(), dgamma))
    for dx, dgamma in runs[1:]:
        assert torch.equal(dx, runs[0][0]) and torch.equal(dgamma, runs[0][1])


@pytest.mark.parametrize("rows,cols", [(9, 505), (700, 1023), (40, 2545), (9, 8187)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rmsnorm_outputs_that_lie_differently(rows, cols, dtype):
    """Rows of an odd width whose outputs do not share the inputs' alignment."""
    x, gamma = normal(1, (rows, cols), dtype), normal(4, (cols,))
    (hw, h), (yw, y) = framed(rows, cols, dtype, 3, 5), framed(rows, cols, torch.bfloat16, 1, 8)
    mp.rmsnorm(x, gamma, 1e-5, residual=x, h=h, y=y)
    wh, wy, _ = O.rmsnorm(np64(x), np64(gamma), 1e-5, np64(x))
    within(h, wh, (BF16 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(wh), "h")
    within(y, wy, (BF16 + REL32) * np.abs(wy), "y")
    assert frame_intact(hw, cols, 3) and frame_intact(yw, cols, 1)


# ----------------------------------------------------------------- linear --

LINEAR_SHAPES = [(1, 1, 1), (1, 8, 16), (2, 129, 65), (17, 64, 1023), (130, 257, 33), (64, 512, 256), (129, 128, 4096),
                 (300, 1000, 777), (5, 300, 8200), (512, 768, 128), (1, 4096, 1024), (257, 513, 64), (31, 2049, 136),
                 (3, 128, 2100), (40, 640, 4000), (200, 384, 1500)]


def linear_case(m, n, k, e4m3, layout, seed=0):
    pad, off = {"dense": (0, 0), "aligned slice": (32, 16), "odd slice": (5, 3)}[layout]
    x, w = normal(seed + 1, (m, k), std=1.0, pad=pad, off=off), normal(seed + 2, (n, k), std=0.1, pad=pad, off=off)
    if not e4m3:
        return x, w, None, None
    def q8(t):
        s = t.float().abs().amax(1).clamp_min(1e-30) / 448
        wide = torch.zeros(t.shape[0], k + pad, dtype=torch.float8_e4m3fn, device="cuda")
        wide[:, off:off + k] = (t.float() / s[:, None]).to(torch.float8_e4m3fn)
        return wide[:, off:off + k], s
    (xq, xs), (wq, wsc) = q8(x), q8(w)
    return xq, wq, xs, wsc


@pytest.mark.parametrize("m,n,k", LINEAR_SHAPES)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["dense", "aligned slice", "odd slice"])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_linear(m, n, k, e4m3, layout, kind):
    check_linear(m, n, k, e4m3, layout, kind)


# enough tiles of 256 x 128 or 256 x 256 for one of the three products to take the
# persistent kernel: ragged last tiles, several tiles per CTA pair, few or many k-blocks
LARGE_SHAPES = [(2100, 2300, 100), (2100, 100, 2300), (100, 2300, 2100), (4096, 2560, 264), (2305, 2311, 2333),
                (700, 4096, 2560), (4099, 2557, 261)]


@pytest.mark.parametrize("m,n,k", LARGE_SHAPES)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kind,layout", [("silu", "dense"), ("gelu", "aligned slice"), ("relu", "odd slice")])
def test_linear_large(m, n, k, e4m3, layout, kind):
    check_linear(m, n, k, e4m3, layout, kind)


@pytest.mark.parametrize("m,n,k", LARGE_SHAPES)
@pytest.mark.parametrize("kind,layout", [("silu", "dense"), ("none", "aligned slice"), ("gelu", "odd slice")])
def test_linear_backward_large(m, n, k, layout, kind):
    check_linear_backward(m, n, k, layout, kind)


# 24 to 38 tiles of 256 x 256 with 32 k-blocks or more: clusters of two CTA pairs
# (of which the last may have a short share); 80 tiles with 88: 76 by pairs and a
# last wave of 4 by clusters
SPLIT_TILES = [(1000, 1500, 2200), (1500, 1530, 2060), (2000, 2500, 5600)]


@pytest.mark.parametrize("m,n,k", SPLIT_TILES)
@pytest.mark.parametrize("kind,layout,e4m3", [("silu", "dense", False), ("gelu", "odd slice", False),
                                              ("none", "aligned slice", True)])
def test_linear_tiles_shared_by_pairs(m, n, k, kind, layout, e4m3):
    check_linear(m, n, k if not e4m3 else 2 * k, e4m3, layout, kind)


@pytest.mark.parametrize("m,n,k", SPLIT_TILES)
@pytest.mark.parametrize("kind,layout", [("gelu", "dense"), ("relu", "odd slice")])
def test_linear_backward_tiles_shared_by_pairs(m, n, k, kind, layout):
    check_linear_backward(m, k, n, layout, kind)        # dx: k in n's place
    check_linear_backward(k, m, n, layout, kind)        # dw: k tokens


def check_linear(m, n, k, e4m3, layout, kind):
    x, w, xs, wsc = linear_case(m, n, k, e4m3, layout)
    bias = normal(3, (n,), torch.bfloat16 if kind == "relu" else torch.float32) if kind != "gelu" else None
    pad = 0 if layout == "dense" else 3
    res = normal(4, (m, n), std=2.0, pad=pad) if kind in ("none", "silu") else None
    y, z = empty((m, n + pad))[:, pad:], empty((m, n + pad))[:, :n]
    ws = mp.linear_workspace(m, n, k, any_layout=True)
    mp.linear(x, w, y, bias=bias, act=kind, residual=res, z=z, x_scale=xs, w_scale=wsc, workspace=ws)
    xd, wd = np64(x.float()), np64(w.float())
    f = lambda t: None if t is None else np64(t)
    wy, wz = O.linear(xd, wd, f(bias), kind, f(res), f(xs), f(wsc))
    mag = np.abs(xd) @ np.abs(wd).T
    if e4m3:
        mag = mag * np64(xs)[:, None] * np64(wsc)[None, :]
    mag = mag + (0 if bias is None else np.abs(f(bias)))
    err = ACC(k) * mag
    within(z, wz, BF16 * (np.abs(wz) + err) + err, "z")
    err = 1.13 * err + ACT * np.abs(wy if res is None else wy - f(res)) + 1e-30
    if res is not None:
        err = err + 2.0 ** -23 * np.abs(wy)
    within(y, wy, BF16 * (np.abs(wy) + err) + err, "y")
    assert mp.device_status(ws) == mp.OPT_OK
    alone = empty((m, n))
    mp.linear(x, w, alone, bias=bias, act=kind, residual=res, x_scale=xs, w_scale=wsc, workspace=ws)
    assert torch.equal(alone, y)             # the same without z, and the same bits again
    if res is not None:                       # y over the residual itself
        buf = res.contiguous().clone()
        mp.linear(x, w, buf, bias=bias, act=kind, residual=buf, x_scale=xs, w_scale=wsc, workspace=ws)
        assert torch.equal(buf, y)


@pytest.mark.parametrize("m,n,k", LINEAR_SHAPES + [(2048, 136, 64), (4099, 64, 72)])
@pytest.mark.parametrize("layout", ["dense", "aligned slice", "odd slice"])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_linear_backward(m, n, k, layout, kind):
    check_linear_backward(m, n, k, layout, kind)


def check_linear_backward(m, n, k, layout, kind):
    pad, off = {"dense": (0, 0), "aligned slice": (24, 8), "odd slice": (5, 3)}[layout]
    dz, x = normal(1, (m, n), pad=pad, off=off), normal(2, (m, k), pad=pad, off=off)
    w = normal(3, (n, k), std=0.1, pad=pad, off=off)
    zp = normal(4, (m, k), std=2.0, pad=pad) if kind != "none" else None
    dx = empty((m, k + pad))[:, pad:]
    dw, db = empty((n, k), torch.float32), empty((n,), torch.float32)
    ws = mp.linear_workspace(m, n, k, any_layout=True)
    mp.linear_backward(dz, x, w, dx=dx, z_prev=zp, act_prev=kind, dw=dw, dbias=db, accumulate=False, workspace=ws)
    dzd, xd, wd = np64(dz), np64(x), np64(w)
    wx, ww, wb = O.linear_backward(dzd, xd, wd, None if zp is None else np64(zp), kind)
    mag = np.abs(dzd) @ np.abs(wd)
    err = 1.13 * ACC(n) * mag
    if zp is not None:
        # the derivative itself: 2^-19 of the sizes of its terms, |z| p (1 - p) c (1 + 3 b z^2) < 2
        err = err + 2 * ACT * 2 * np.abs(dzd @ wd)
    within(dx, wx, BF16 * (np.abs(wx) + err) + err, "dx")
    wmag, bmag = np.abs(dzd).T @ np.abs(xd), np.abs(dzd).sum(0)
    within(dw, ww, ACC(m) * wmag, "dw")
    within(db, wb, ACC(m) * bmag, "dbias")
    assert mp.device_status(ws) == mp.OPT_OK
    odw, odb = normal(5, (n, k), torch.float32), normal(6, (n,), torch.float32)
    adw, adb = odw.clone(), odb.clone()
    mp.linear_backward(dz, x, None, dw=adw, dbias=adb, workspace=ws)
    within(adw, ww + np64(odw), ACC(m) * wmag + 2.0 ** -23 * (np.abs(ww) + np.abs(np64(odw))), "dw +=")
    within(adb, wb + np64(odb), ACC(m) * bmag + 2.0 ** -23 * (np.abs(wb) + np.abs(np64(odb))), "dbias +=")
    dx1, dw1, db1 = empty((m, k)), empty((n, k), torch.float32), empty((n,), torch.float32)
    mp.linear_backward(dz, None, w, dx=dx1, z_prev=zp, act_prev=kind, workspace=ws)
    mp.linear_backward(dz, x, None, dw=dw1, dbias=db1, accumulate=False, workspace=ws)
    assert torch.equal(dx1, dx) and torch.equal(dw1, dw) and torch.equal(db1, db)


def test_weight_gradient_of_many_tokens_keeps_fp32():
    """16384 tokens: the sum's error stays that of fp32 additions that round
    (sqrt(m) 2^-24 in the 2-norm, with a factor of 4), not the m 2^-24 of
    additions that truncate."""
    m, n, k = 16384, 128, 256
    dz, x = normal(1, (m, n)), normal(2, (m, k)) + 0.25     # sums that grow as well as wander
    dz = (dz.float() + 0.25).to(torch.bfloat16)
    dw = empty((n, k), torch.float32)
    mp.linear_backward(dz, x, None, dw=dw, accumulate=False, workspace=mp.linear_workspace(m, n, k))
    want = np64(dz).T @ np64(x)
    rel = np.linalg.norm(np64(dw) - want) / np.linalg.norm(want)
    assert rel < 4 * np.sqrt(m) * 2.0 ** -24, rel


def test_linear_nonfinite_values_stay_in_their_rows():
    m, n, k = 70, 200, 100
    x, w = normal(1, (m, k)), normal(2, (n, k))
    x[3, 5], x[64, 99] = float("inf"), float("nan")
    y, ws = empty((m, n)), mp.linear_workspace(m, n, k)
    mp.linear(x, w, y, workspace=ws)
    yh = np64(y)
    assert np.isinf(yh[3]).all() and np.array_equal(np.sign(yh[3]), np.sign(np64(w)[:, 5]))
    assert np.isnan(yh[64]).all()
    assert np.isfinite(np.delete(yh, [3, 64], 0)).all()
    dz = normal(3, (m, n))
    dz[69, 199] = float("nan")
    dx, dw, db = empty((m, k)), empty((n, k), torch.float32), empty((n,), torch.float32)
    mp.linear_backward(dz, normal(4, (m, k)), w, dx=dx, dw=dw, dbias=db, accumulate=False, workspace=ws)
    assert np.isnan(np64(dx)[69]).all() and np.isfinite(np64(dx)[:69]).all()
    assert np.isnan(np64(dw)[199]).all() and np.isfinite(np64(dw)[:199]).all()
    assert np.isnan(np64(db)[199]) and np.isfinite(np64(db)[:199]).all()


def test_linear_no_rows():
    none, w = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), normal(1, (16, 32))
    out = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    mp.linear(none, w, out)
    dw, db = torch.full((16, 32), 2.0, device="cuda"), torch.full((16,), 2.0, device="cuda")
    mp.linear_backward(out, none, w, dx=none, dw=dw, dbias=db)
    assert (dw == 2).all() and (db == 2).all()
    mp.linear_backward(out, none, w, dx=none, dw=dw, dbias=db, accumulate=False)
    assert (dw == 0).all() and (db == 0).all()


def test_gradients_against_differences():
    """norm -> linear(gelu) -> linear against central differences of the fp64
    oracle's loss.  The chain rounds u, dz and dy to bf16 on the way, each at
    most 2^-8 of its values: 2e-2 in the 2-norm bounds their sum over three
    layers with a factor of 1.7."""
    m, c, f = 6, 24, 40
    r = np.random.default_rng(5)
    bf = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()
    x, gamma = bf(r.normal(size=(m, c))), bf(1 + 0.1 * r.normal(size=c))
    w1, b1, w2 = bf(0.3 * r.normal(size=(f, c))), bf(0.1 * r.normal(size=f)), bf(0.3 * r.normal(size=(c, f)))
    dy = bf(r.normal(size=(m, c)))
    ws, nws = mp.linear_workspace(m, f, c), mp.rmsnorm_workspace(m, c)
    y, rstd = empty((m, c)), empty((m,), torch.float32)
    u, z, out = empty((m, f)), empty((m, f)), empty((m, c))
    mp.rmsnorm(x, gamma, 1e-6, y=y, rstd=rstd)
    mp.linear(y, w1, u, bias=b1, act="gelu", z=z, workspace=ws)
    mp.linear(u, w2, out, workspace=ws)
    dz1, dw2, dw1 = empty((m, f)), empty((c, f), torch.float32), empty((f, c), torch.float32)
    db1, dn, dx, dg = empty((f,), torch.float32), empty((m, c)), empty((m, c)), empty((c,), torch.float32)
    mp.linear_backward(dy, u, w2, dx=dz1, z_prev=z, act_prev="gelu", dw=dw2, accumulate=False, workspace=ws)
    mp.linear_backward(dz1, y, w1, dx=dn, dw=dw1, dbias=db1, accumulate=False, workspace=ws)
    mp.rmsnorm_backward(dn, x, gamma, rstd, dx, dgamma=dg, accumulate=False, workspace=nws)
    P = dict(x=np64(x), gamma=np64(gamma), w1=np64(w1), b1=np64(b1), w2=np64(w2))

    def loss(p):
        _, n_, _ = O.rmsnorm(p["x"], p["gamma"], 1e-6)
        return float((O.linear(O.linear(n_, p["w1"], p["b1"], "gelu")[0], p["w2"])[0] * np64(dy)).sum())
    for name, got in (("x", dx), ("gamma", dg), ("w1", dw1), ("b1", db1), ("w2", dw2)):
        want = np.zeros_like(P[name])
        for i in np.ndindex(want.shape):
            a, b = {**P, name: P[name].copy()}, {**P, name: P[name].copy()}
            a[name][i] += 1e-4
            b[name][i] -= 1e-4
            want[i] = (loss(a) - loss(b)) / 2e-4
        rel = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
        assert rel < 2e-2, (name, rel)


def test_rows_far_apart():
    """Row distances and offsets past 32 bits (elements and bytes)."""
    ld = (1 << 31) + 64
    buf = torch.empty(2 * ld + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, 256), (ld, 1))
    x.copy_(normal(1, (3, 256)))
    w, gamma = normal(2, (128, 256), std=0.1), normal(3, (256,))
    near = x.contiguous()
    ya, yb, ws = empty((3, 128)), empty((3, 128)), mp.linear_workspace(3, 128, 256)
    mp.linear(x, w, ya, workspace=ws)
    mp.linear(near, w, yb, workspace=ws)
    assert torch.equal(ya, yb)
    na, nb = empty((3, 256)), empty((3, 256))
    mp.rmsnorm(x, gamma, y=na)
    mp.rmsnorm(near, gamma, y=nb)
    assert torch.equal(na, nb)
    far = torch.as_strided(buf, (3, 128), (ld, 1), 1024)
    mp.linear(near, w, far, residual=yb, workspace=ws)
    mp.linear(near, w, ya, residual=yb, workspace=ws)
    assert torch.equal(far.contiguous(), ya)
    dz = torch.as_strided(buf, (3, 128), (ld, 1), 2048)
    dz.copy_(normal(4, (3, 128)))
    dwa, dwb = empty((128, 256), torch.float32), empty((128, 256), torch.float32)
    mp.linear_backward(dz, x, None, dw=dwa, accumulate=False, workspace=ws)
    mp.linear_backward(dz.contiguous(), near, None, dw=dwb, accumulate=False, workspace=ws)
    assert torch.equal(dwa, dwb)


def test_other_stream_and_graph():
    """A call enqueues on the stream it is given, and a captured step replays
    with the inputs of the moment."""
    m, n, k = 64, 320, 192
    x, w, gamma = normal(1, (m, k)), normal(2, (n, k), std=0.1), normal(3, (k,))
    y, norm, rstd = empty((m, n)), empty((m, k)), empty((m,), torch.float32)
    dx, dw, db = empty((m, k)), empty((n, k), torch.float32), empty((n,), torch.float32)
    ws = mp.linear_workspace(m, n, k)

    def step(stream=None):
        mp.rmsnorm(x, gamma, y=norm, rstd=rstd, stream=stream)
        mp.linear(norm, w, y, act="silu", workspace=ws, stream=stream)
        mp.linear_backward(y, norm, w, dx=dx, dw=dw, dbias=db, accumulate=False, workspace=ws, stream=stream)
    outs = (norm, y, dx, dw, db)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    for t, v in zip(outs, want):
        assert torch.equal(t, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2 = normal(9, (m, k))
    keep = x.clone()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    second = [t.clone() for t in outs]
    step()
    torch.cuda.synchronize()
    for t, v in zip(outs, second):
        assert torch.equal(t, v)
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    for t, v in zip(outs, want):
        assert torch.equal(t, v)


def test_launches_are_named():
    with mp.LaunchProfiler(64) as prof:
        x, w = normal(1, (40, 63)), normal(2, (48, 63))
        y, ws = empty((40, 48)), mp.linear_workspace(40, 48, 63)
        mp.linear(x, w, y, workspace=ws)
        dx, dw, db = empty((40, 63)), empty((48, 63), torch.float32), empty((48,), torch.float32)
        mp.linear_backward(y, x, w, dx=dx, dw=dw, dbias=db, workspace=ws)
        q, s = empty((48, 63), torch.float8_e4m3fn), empty((48,), torch.float32)
        mp.quantize_rows(w, q, s)
        mp.rmsnorm(x, normal(3, (63,)), y=dx)
    torch.cuda.synchronize()
    names = {r["kernel"] for r in prof.records()}
    assert {"linear", "linear_repack", "linear_grad", "quantize_rows", "rmsnorm"} <= names


def test_python_argument_checks():
    """Shapes, layouts and types that do not fit raise before the library is
    called; leading dimensions and vectors count as rows."""
    x, w, ws = normal(1, (4, 6, 64)), normal(2, (32, 64)), mp.linear_workspace(24, 32, 64)
    y = empty((4, 6, 32))
    mp.linear(x, w, y, workspace=ws)
    flat = empty((24, 32))
    mp.linear(x.view(24, 64), w, flat, workspace=ws)
    assert torch.equal(y.view(24, 32), flat)
    one = empty((32,))
    mp.linear(x[0, 0], w, one, workspace=ws)
    assert torch.equal(one, flat[0])
    with pytest.raises(ValueError, match="y has shape"):
        mp.linear(x, w, empty((24, 31)), workspace=ws)
    with pytest.raises(ValueError, match="contiguous rows"):
        mp.linear(x.view(24, 64), normal(3, (64, 32)).t(), flat, workspace=ws)
    with pytest.raises(TypeError, match="w must be"):
        mp.linear(x, w.float(), y, workspace=ws)
    with pytest.raises(ValueError, match="x_scale"):
        mp.linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), y, x_scale=torch.ones(3, device="cuda"),
                  w_scale=torch.ones(32, device="cuda"), workspace=ws)
    with pytest.raises(RuntimeError):
        mp.linear(x.transpose(0, 1), w, y, workspace=ws)          # rows that are not evenly spaced
    with pytest.raises(mp.MpoptError, match="WORKSPACE"):
        mp.linear(x, w, y)
    with pytest.raises(mp.MpoptError, match="INVALID"):
        mp.rmsnorm(x, torch.ones(64, device="cuda"), -1.0, y=empty((4, 6, 64)))
    with pytest.raises(ValueError, match="dw has shape"):
        mp.linear_backward(flat, x.view(24, 64), None, dw=empty((64, 32), torch.float32), workspace=ws)
