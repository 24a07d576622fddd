"""The gated recurrence and its gradient entry by entry, for gates that are nearly
open or nearly closed, where either c or 1 - c is far below a rounding of one.

With u = 2^-24 and s = min(c, 1 - c) = e / (1 + e), e = exp(-|gate|), |gate| <= 24:
the constant log2 e and its product with the gate are rounded (2 u |gate| <= 48 u of e),
two instructions of 2 units of 2^-23 (4 u each), a sum and a product (2 u): s is
within 64 u = 2^-18 of itself (S).  So, Hm a bound on |h|, that is the same recurrence on
|x| and |h0|:
  h = h + c (x - h), taken from the smaller of c and 1 - c, is off by
  s (|x| + Hm) (S + 2 u) and a rounding of the result;  a product of 1 - c by S + u of
  itself where that is s, by c S + u beyond;  joining pieces adds 2 roundings for each
  level (warps, CTAs), 8 u Hm in all:
    e_t = (1 - c) e_{t-1} + s (|x_t| + Hm_{t-1}) (S + 2 u) + 8 u Hm_t
  and the same backwards for l, with Lm_t = |dy_t| + (1 - c_{t+1}) Lm_{t+1}.  These bounds
  shrink with the values: nothing is measured against a column's largest one.
"""

import numpy as np
import pytest

from gpu_helpers import dev, require_gpu, torch
import mixed_precision_optimizer_gb300 as mp
from oracle import feedforward as F

pytestmark = pytest.mark.gpu

U, S = 2.0 ** -24, 2.0 ** -18
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: U}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def np64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    got = np64(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    worst = np.unravel_index(np.argmax(over), over.shape)
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound, at {worst}: {got[worst]} for {want[worst]}"


def check(rows, cols, starts, gate, dtype, dy_size, seed=0):
    """x and dy far smaller than the states and gradients that come in."""
    r = np.random.default_rng(seed)
    sequences = len(starts) - 1
    cast = lambda a: dev(a.astype(np.float32)).to(dtype)
    x, gate, dy = cast(r.normal(size=(rows, cols)) * 1e-3), cast(gate), cast(r.normal(size=(rows, cols)) * dy_size)
    h0, dhT = (dev((r.normal(size=(sequences, cols)) * 1e3).astype(np.float32)) for _ in range(2))
    equal = len(set(np.diff(starts))) == 1 and starts[0] == 0 and starts[-1] == rows
    call = dict(sequences=sequences) if equal else dict(starts=dev(np.asarray(starts, np.int32)))
    y, dx, dg = (torch.zeros((rows, cols), dtype=dtype, device="cuda") for _ in range(3))
    hT, dh0, states = torch.zeros_like(h0), torch.zeros_like(h0), mp.recurrence_states(rows, cols, dtype)
    mp.gated_recurrence(x, gate, y, h0=h0, hT=hT, states=states, **call)
    mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, h0=h0, dhT=dhT, dh0=dh0, **call)

    X, G, DY, H0, DHT = np64(x), np64(gate), np64(dy), np64(h0), np64(dhT)
    c, a = F.sigmoid(G), F.sigmoid(-G)
    s = np.minimum(c, a)
    h, e, Hm, before, eb, Hb = (np.zeros((rows, cols)) for _ in range(6))
    lam, el, Lm = (np.zeros((rows, cols)) for _ in range(3))
    whT, eT, wd0, e0 = (np.zeros((sequences, cols)) for _ in range(4))
    for q in range(sequences):
        v, ev, m = H0[q], np.zeros(cols), np.abs(H0[q])
        for t in range(starts[q], starts[q + 1]):
            before[t], eb[t], Hb[t] = v, ev, m
            v = a[t] * v + c[t] * X[t]
            ev = a[t] * ev + s[t] * (np.abs(X[t]) + m) * (S + 2 * U)
            m = a[t] * m + c[t] * np.abs(X[t])
            ev = ev + 8 * U * m
            h[t], e[t], Hm[t] = v, ev, m
        whT[q], eT[q] = v, ev
        v, ev, m = DHT[q], np.zeros(cols), np.abs(DHT[q])
        for t in range(starts[q + 1] - 1, starts[q] - 1, -1):
            lam[t], Lm[t] = DY[t] + v, np.abs(DY[t]) + m
            el[t] = ev + 4 * U * Lm[t]
            v, m = a[t] * lam[t], a[t] * Lm[t]
            ev = a[t] * el[t] + s[t] * Lm[t] * (S + 2 * U) + 8 * U * m
        wd0[q], e0[q] = v, ev
    half = HALF[dtype] * 1.01
    within(hT, whT, eT, "hT")
    within(y, h, e + half * np.abs(h), "y")
    within(dh0, wd0, e0, "dh0")
    within(dx, c * lam, c * (el + (S + 4 * U) * Lm) + half * np.abs(c * lam), "dx")
    wg = c * a * lam * (X - before)
    d = np.abs(X - before) + eb
    within(dg, wg, c * a * ((el + (2 * S + 8 * U) * Lm) * d + Lm * (eb + 2 * U * (np.abs(X) + Hb))) + half * np.abs(wg), "dgate")


@pytest.mark.parametrize("length", [1, 2, 3])
@pytest.mark.parametrize("cols", [63, 64, 2056, 4096])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dy_size", [0.0, 1e-3])
def test_nearly_open_gates(length, cols, dtype, dy_size):
    """Few rows, each gate from 8 to 24: what is left of a state is e^-8 to e^-72 of it."""
    rows = 12 * length
    gate = np.random.default_rng(length).uniform(8, 24, (rows, cols))
    check(rows, cols, np.arange(13) * length, gate, dtype, dy_size)


@pytest.mark.parametrize("rows,cols", [(40, 72), (700, 65), (2100, 64), (300, 2056), (300, 4104)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("packed", [False, True])
def test_long_memories_with_open_gates_between(rows, cols, dtype, packed):
    """Gates of -24 to -10, which keep nearly everything, and in each column three that
    are nearly open: the state that goes on is told from a rounding of the one before."""
    r = np.random.default_rng(rows)
    gate = r.uniform(-24, -10, (rows, cols))
    for k in range(3):
        gate[r.integers(0, rows, cols), np.arange(cols)] = r.uniform(8, 20, cols)
    starts = np.array([0, 7, 7, rows // 2 + 3, rows - 2]) if packed else np.array([0, rows])
    check(rows, cols, starts, gate, dtype, 1e-6)


@pytest.mark.parametrize("sequences", [1, 3])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gates_of_any_size(sequences, dtype):
    gate = np.random.default_rng(5).uniform(-24, 24, (24, 200))
    check(24, 200, np.arange(sequences + 1) * (24 // sequences), gate, dtype, 1.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", [0, 7, 60, 99, 100, 103, 199])
def test_a_gate_that_is_no_number_stays_in_its_sequence(bad, where):
    """And an infinite one is open or closed: nothing else in its sequence is lost."""
    starts = [0, 60, 60, 100, 200]
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    r = np.random.default_rng(1)
    x, gate, dy = (dev(r.normal(size=(200, 72)).astype(np.float32)) for _ in range(3))
    outs = []
    for hit in (False, True):
        if hit:
            gate[where, 5] = bad
        y, dx, dg = (torch.zeros_like(x) for _ in range(3))
        states, hT, dh0 = mp.recurrence_states(200, 72, FP32), torch.zeros(4, 72, device="cuda"), torch.zeros(4, 72, device="cuda")
        mp.gated_recurrence(x, gate, y, starts=st, hT=hT, states=states)
        mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, starts=st, dh0=dh0)
        outs.append((y, dx, dg, hT, dh0))
    seq = max(i for i in range(4) if starts[i] <= where)
    for a, b in zip(*outs):
        own = torch.zeros(len(a), 72, dtype=torch.bool, device="cuda")
        own[(slice(starts[seq], starts[seq + 1]) if len(a) == 200 else seq), 5] = True
        assert torch.equal(a[~own], b[~own])
        if bad == bad:
            assert torch.isfinite(b).all()
    if bad != bad:
        assert torch.isnan(outs[1][0][where:starts[seq + 1], 5]).all() and torch.isnan(outs[1][1][starts[seq]:where + 1, 5]).all()


def test_open_gate_takes_x_itself():
    """Beyond 87 nothing of h is left, whatever its size."""
    x, h0 = torch.full((2, 64), 1e-3, device="cuda"), torch.full((2, 64), 1e30, device="cuda")
    y = torch.zeros_like(x)
    for g in (88.0, float("inf")):
        mp.gated_recurrence(x, torch.full_like(x, g), y, sequences=2, h0=h0)
        assert torch.equal(y, x)
        mp.gated_recurrence(x, torch.full_like(x, g), y, h0=h0[:1].contiguous())
        assert torch.equal(y, x)
