"""Feed-forward operators without a GPU: the fp64 oracle's gradients against
central differences and its e4m3 rounding against torch's, and every refusal
of the C entry points and of the Python checks.  Pointers passed to the
library are fake aligned addresses: each call returns before a CUDA call."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_optimizer_gb300 as mp
from mixed_precision_optimizer_gb300 import build_lib, feedforward as ff
from oracle import feedforward as O

INV, UNSUP, MIS, WS = 1, 2, 3, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return mp.lib()


def differences(f, x, h):
    """d f / d x for a scalar f by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


# Central differences in fp64 with step h: truncation h^2 |f'''| / 6 and
# rounding 1e-16 |f| / h; h = 1e-4 on values of order one leaves both near 1e-8
# and 1e-11, so 1e-6 separates a wrong formula from the method's error.
H, TOL = 1e-4, 1e-6


@pytest.mark.parametrize("kind", ["none", "gelu", "silu"])
def test_oracle_activation_gradient(kind):
    u = np.linspace(-6, 6, 97)
    d = (O.act(u + H, kind) - O.act(u - H, kind)) / (2 * H)
    assert np.max(np.abs(d - O.act_grad(u, kind))) < TOL


def test_oracle_rmsnorm_gradient():
    r = np.random.default_rng(0)
    x, res, gamma = r.normal(size=(3, 7)), r.normal(size=(3, 7)), r.normal(size=7)
    dy, dh = r.normal(size=(3, 7)), r.normal(size=(3, 7))

    def loss(x_, res_, gamma_):
        h, y, _ = O.rmsnorm(x_, gamma_, 1e-3, res_)
        return float((y * dy).sum() + (h * dh).sum())
    h, _, rstd = O.rmsnorm(x, gamma, 1e-3, res)
    dx, dgamma = O.rmsnorm_backward(dy, h, gamma, rstd, dh)
    assert np.max(np.abs(differences(lambda t: loss(t, res, gamma), x, H) - dx)) < TOL
    assert np.max(np.abs(differences(lambda t: loss(x, t, gamma), res, H) - dx)) < TOL
    assert np.max(np.abs(differences(lambda t: loss(x, res, t), gamma, H) - dgamma)) < TOL


@pytest.mark.parametrize("kind", ["none", "gelu", "silu"])
def test_oracle_linear_gradient(kind):
    """Two layers: the second's dx, taken through the first's activation, is
    the first's dz."""
    r = np.random.default_rng(1)
    x, w1, b1, w2 = r.normal(size=(4, 5)), r.normal(size=(6, 5)), r.normal(size=6), r.normal(size=(3, 6))
    dy = r.normal(size=(4, 3))

    def loss(w1_, b1_, w2_):
        u, _ = O.linear(x, w1_, b1_, kind)
        return float((O.linear(u, w2_)[0] * dy).sum())
    u, z1 = O.linear(x, w1, b1, kind)
    dz1, dw2, _ = O.linear_backward(dy, u, w2, z1, kind)
    _, dw1, db1 = O.linear_backward(dz1, x, w1)
    assert np.max(np.abs(differences(lambda t: loss(t, b1, w2), w1, H) - dw1)) < TOL
    assert np.max(np.abs(differences(lambda t: loss(w1, t, w2), b1, H) - db1)) < TOL
    assert np.max(np.abs(differences(lambda t: loss(w1, b1, t), w2, H) - dw2)) < TOL


def test_oracle_e4m3_rounding_matches_torch():
    """Every e4m3 value, the midpoints between neighbours (ties) and values
    either side of them."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    vals = np.unique(codes[np.isfinite(codes)])
    mid = (vals[1:] + vals[:-1]) / 2
    v = np.concatenate([vals, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3_rne(v), want.astype(np.float64))


# ------------------------------------------------------------- refusals --

def norm_args(**kw):
    a = ff.OptRmsnormArgs(FAKE, None, FAKE, None, FAKE, None, None, FAKE, 4, 64, 64, 0, 0, 64, 0, 1, 1, 1e-6, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(gamma=None), INV), (dict(rows=-1), INV), (dict(cols=0), INV), (dict(dtype=2), INV),
    (dict(gamma_dtype=7), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(x_ld=63), INV),
    (dict(y_ld=63), INV), (dict(q=FAKE), INV), (dict(q_scale=FAKE), INV), (dict(residual=FAKE), INV),
    (dict(x=FAKE + 1), MIS), (dict(gamma=FAKE + 1), MIS), (dict(rstd=FAKE + 2), MIS), (dict(y=FAKE + 1), MIS),
    (dict(cols=49153, x_ld=49153, y_ld=49153), UNSUP), (dict(rows=(1 << 30) + 1), INV)])
def test_rmsnorm_refusals(L, kw, want):
    assert L.opt_rmsnorm_forward(ctypes.byref(norm_args(**kw)), None) == want


def test_nothing_to_do_is_ok(L):
    assert L.opt_rmsnorm_forward(ctypes.byref(norm_args(rows=0, x=None, y=None)), None) == mp.OPT_OK
    assert L.opt_quantize_rows(None, 0, 1, 0, 8, None, 0, None, None) == mp.OPT_OK
    a = ff.OptLinearArgs(m=0, n=4, k=4, dtype=1)
    assert L.opt_linear_forward(ctypes.byref(a), None, 0, None) == mp.OPT_OK
    a = ff.OptLinearGradArgs(m=0, n=4, k=4, accumulate=1, dw=FAKE)
    assert L.opt_linear_backward(ctypes.byref(a), None, 0, None) == mp.OPT_OK
    a = ff.OptLinearGradArgs(dz=FAKE, m=2, n=4, k=4, dz_ld=4)
    assert L.opt_linear_backward(ctypes.byref(a), None, 0, None) == mp.OPT_OK


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INV), (dict(h=None), INV), (dict(rstd=None), INV), (dict(gamma=None), INV), (dict(dy_ld=63), INV),
    (dict(dtype=2), INV), (dict(dgamma=FAKE + 1), MIS), (dict(dx=FAKE + 1), MIS), (dict(rows=-2), INV),
    (dict(cols=24577, dy_ld=24577, h_ld=24577, dx_ld=24577), UNSUP)])
def test_rmsnorm_backward_refusals(L, kw, want):
    a = ff.OptRmsnormGradArgs(FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, 4, 64, 64, 64, 0, 64, 1, 1, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    assert L.opt_rmsnorm_backward(ctypes.byref(a), FAKE, 1 << 30, None) == want


def test_rmsnorm_backward_workspace_refusals(L):
    a = ff.OptRmsnormGradArgs(FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, 4, 64, 64, 64, 0, 64, 1, 1, 0, 0)
    need = mp.rmsnorm_workspace_size(4, 64)
    assert need >= 4 * 64 * 4
    for ws, nb in ((None, 1 << 20), (FAKE, need - 1), (FAKE + 64, 1 << 20)):
        assert L.opt_rmsnorm_backward(ctypes.byref(a), ws, nb, None) == WS


@pytest.mark.parametrize("args,want", [
    ((None, 8, 1, 2, 8, FAKE, 8, FAKE, None), INV), ((FAKE, 8, 1, 2, 8, None, 8, FAKE, None), INV),
    ((FAKE, 8, 1, 2, 8, FAKE, 8, None, None), INV), ((FAKE, 7, 1, 2, 8, FAKE, 8, FAKE, None), INV),
    ((FAKE, 8, 2, 2, 8, FAKE, 8, FAKE, None), INV), ((FAKE + 2, 8, 0, 2, 8, FAKE, 8, FAKE, None), MIS),
    ((FAKE, 50000, 1, 2, 50000, FAKE, 50000, FAKE, None), UNSUP)])
def test_quantize_refusals(L, args, want):
    assert L.opt_quantize_rows(*args) == want


def linear_args(**kw):
    a = ff.OptLinearArgs(FAKE, FAKE, None, None, None, None, FAKE, None, 4, 64, 32, 32, 32, 0, 64, 0, 1, 1, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BIG = 1 << 30


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(m=-1), INV), (dict(n=0), INV),
    (dict(k=0), INV), (dict(dtype=0), INV), (dict(act=4), INV), (dict(act=-1), INV), (dict(x_ld=31), INV),
    (dict(w_ld=31), INV), (dict(y_ld=63), INV), (dict(z=FAKE, z_ld=10), INV), (dict(residual=FAKE), INV),
    (dict(bias=FAKE, bias_dtype=2), INV), (dict(x_scale=FAKE), INV), (dict(dtype=2), INV),
    (dict(dtype=2, x_scale=FAKE), INV), (dict(dtype=2, x_scale=FAKE, w_scale=FAKE + 1), MIS), (dict(x=FAKE + 1), MIS),
    (dict(bias=FAKE + 2, bias_dtype=0), MIS), (dict(k=BIG + 1, x_ld=BIG + 1, w_ld=BIG + 1), INV)])
def test_linear_refusals(L, kw, want):
    assert L.opt_linear_forward(ctypes.byref(linear_args(**kw)), FAKE, 1 << 30, None) == want


def test_linear_workspace_refusals(L):
    a = linear_args()
    for ws, nb in ((None, 1 << 20), (FAKE, 255), (FAKE + 128, 1 << 20)):
        assert L.opt_linear_forward(ctypes.byref(a), ws, nb, None) == WS
    # rows of 31 elements do not start on 16 bytes: room for the copies is part of the size
    a = linear_args(k=31, x_ld=31, w_ld=31)
    need = mp.linear_workspace_size(4, 64, 31)
    assert need > mp.linear_workspace_size(4, 64, 32)
    assert L.opt_linear_forward(ctypes.byref(a), FAKE, 256 + 255, None) == WS
    # a slice of wider rows that starts off 16 bytes: only with any_layout
    a = linear_args(x=FAKE + 2, x_ld=40)
    assert mp.linear_workspace_size(4, 64, 32, any_layout=True) > mp.linear_workspace_size(4, 64, 32)
    assert L.opt_linear_forward(ctypes.byref(a), FAKE, mp.linear_workspace_size(4, 64, 32), None) == WS
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, 0)):
        assert mp.linear_workspace_size(*bad) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dz=None), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(act_prev=9), INV), (dict(n=0), INV),
    (dict(dz_ld=63), INV), (dict(dx_ld=31), INV), (dict(z_prev=FAKE, z_prev_ld=31), INV), (dict(dw=FAKE + 2), MIS),
    (dict(dbias=FAKE + 1), MIS), (dict(dz=FAKE + 1), MIS)])
def test_linear_backward_refusals(L, kw, want):
    a = ff.OptLinearGradArgs(FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, 4, 64, 32, 64, 32, 32, 0, 32, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    assert L.opt_linear_backward(ctypes.byref(a), FAKE, 1 << 30, None) == want


def test_null_arguments(L):
    for f in (L.opt_rmsnorm_forward,):
        assert f(None, None) == INV
    for f in (L.opt_rmsnorm_backward, L.opt_linear_forward, L.opt_linear_backward):
        assert f(None, None, 0, None) == INV


def test_python_checks():
    """CPU tensors, wrong types and shapes are refused before the library is called."""
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(s)
    with pytest.raises(ValueError, match="CUDA"):
        mp.rmsnorm(b(2, 8), b(8), y=b(2, 8))
    with pytest.raises(TypeError):
        mp.rmsnorm(b(2, 8).half(), b(8), y=b(2, 8))
    with pytest.raises(ValueError, match="activation"):
        mp.linear(b(2, 8), b(4, 8), b(2, 4), act="tanh")
    with pytest.raises(TypeError):
        mp.linear(f(2, 8), b(4, 8), b(2, 4))
    with pytest.raises(ValueError, match="nothing"):
        mp.linear_backward(b(2, 4), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        mp.quantize_rows(f(2, 8), torch.zeros(2, 8, dtype=torch.float8_e4m3fn), f(2))


def test_packed_arguments_match_the_structs():
    """The functions pack their argument structs by format string: field by
    field the same bytes as the ctypes structs of the header."""
    for pack, cls in ((ff._PACK_NORM, ff.OptRmsnormArgs), (ff._PACK_NORM_GRAD, ff.OptRmsnormGradArgs),
                      (ff._PACK_LINEAR, ff.OptLinearArgs), (ff._PACK_LINEAR_GRAD, ff.OptLinearGradArgs)):
        vals = [0.5 if t is ctypes.c_float else 1 + i for i, (_, t) in enumerate(cls._fields_)]
        assert pack(*vals) == bytes(cls(*vals))
