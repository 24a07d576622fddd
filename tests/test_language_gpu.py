"""Language-model operators on the GPU against the fp64 oracle.

Tolerances, from the formats and the order of operations:

* a rounding is off by at most half a step: 2^-24 of the value in fp32 (R32),
  2^-8 in bf16 (HALF);
* a sum of n fp32 terms, in any order, is within n 2^-24 sum |terms|;
* c = 1 / (1 + exp(-g)) for |g| <= 8: the rounding of g log2 e (2^-24 |g| of the
  value), two instructions of 2 units of 2^-23 each and one addition, within
  2^-20 (GATE);
* the recurrence: with M the largest |x|, |h0| of a column (so |h| <= M), a row
  adds its own rounding and that of x - h (2^-23 M), c's error times |x - h|, and,
  every 8 rows, the joining of pieces (2 roundings, and the error of the product
  of 1 - c: a rounding a row and that of its c's); twice the first and four times
  the second cover both:
    e_t = (1 - c_t) e_{t-1} + M (2^-22 + 4 c_t GATE)
  and the same backwards for l with M the largest |l|;
* an activation is within 2^-16 of itself (sigmoid(t), 2^-24 |t| of the value for
  |t| <= 87, and two instructions), its derivative within 2^-16: z p (1 - p) k is
  formed from a p that is off by 2^-23 at most where it is near one, and |z| k
  is below 45 where p (1 - p) is not 0;
* exp(d) of a logit, d = x - max: (2^-22 + 2^-23 |d|) exp(d), so a sum of n of
  them, n / 256 or fewer (a row of up to 1024: n / 32) to a thread, is within
  (n / 256 + 64) 2^-24 + 2^-20 of itself.
"""

import numpy as np
import pytest

from gpu_helpers import require_gpu, torch
import mixed_precision_optimizer_gb300 as mp
from oracle import feedforward as F
from oracle import language as O

pytestmark = pytest.mark.gpu

R32, HALF, GATE, ACT = 2.0 ** -24, 2.0 ** -8, 2.0 ** -20, 2.0 ** -16
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
STEP = {BF16: HALF, FP32: R32}
LAYOUTS = {"dense": (0, 0), "aligned slice": (24, 8), "odd slice": (5, 3)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(seed, shape, dtype=BF16, std=1.0, layout="dense"):
    pad, off = LAYOUTS[layout]
    wide = tuple(shape[:-1]) + (shape[-1] + pad,)
    return (torch.randn(wide, generator=gen(seed), device="cuda") * std).to(dtype)[..., off:off + shape[-1]]


def output(shape, dtype=BF16, layout="dense"):
    """NaN throughout (e4m3 and bytes: 0x7F), in the given layout."""
    pad, off = LAYOUTS[layout]
    wide = tuple(shape[:-1]) + (shape[-1] + pad,)
    if dtype in (E4M3, torch.uint8):
        return torch.full(wide, 0x7F, dtype=torch.uint8, device="cuda").view(dtype)[..., off:off + shape[-1]]
    return torch.full(wide, float("nan"), dtype=dtype, device="cuda")[..., off:off + shape[-1]]


def assert_frame_untouched(t, layout):
    """The columns around a slice from output() are as they were."""
    pad, off = LAYOUTS[layout]
    rows, cols = t.shape
    wide = torch.as_strided(t, (rows, cols + pad), (cols + pad, 1), t.storage_offset() - off)
    wide = wide.view(torch.uint8) if t.element_size() == 1 else wide
    frame = torch.cat([wide[:, :off], wide[:, off + cols:]], dim=1)
    assert bool((frame == 0x7F).all() if frame.dtype == torch.uint8 else torch.isnan(frame.float()).all())


def np64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what=""):
    got, want = np64(got) if torch.is_tensor(got) else got, np.asarray(want)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} not finite"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound, worst by {over.max():.3g}"


# -------------------------------------------------------------- embedding --

@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (1, 50, 4096), (3, 7, 8), (33, 100, 63), (257, 1000, 136), (40, 9, 2049),
                                             (700, 333, 1024)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_embedding(rows, vocab, cols, dtype, out, layout):
    table = normal(1, (vocab, cols), dtype, layout=layout)
    index = torch.int32 if rows % 2 else torch.int64
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=gen(2), device="cuda").to(index)
    y = output((rows, cols), out, layout)
    mp.embedding(tokens, table, y, scale=1.7)
    want = O.embedding(tokens.cpu().numpy(), np64(table), float(np.float32(1.7)))
    within(y, want, np.abs(want) * (STEP[out] * 1.01 + R32))
    assert_frame_untouched(y, layout)
    mp.embedding(tokens, table, y)                     # without a scale the rows themselves
    known = ((tokens >= 0) & (tokens < vocab))[:, None]
    assert torch.equal(y, torch.where(known, table[tokens.clamp(0, vocab - 1).long()].to(out), torch.zeros((), dtype=out, device="cuda")))


def test_embedding_tokens_of_any_value():
    """Tokens far outside the table are padding too."""
    table = normal(1, (10, 64))
    tokens = torch.tensor([-2 ** 63, 2 ** 63 - 1, 2 ** 32, -2 ** 32 + 3, 3, 10], device="cuda")
    y, g = output((6, 64)), torch.zeros(10, 64, device="cuda")
    mp.embedding(tokens, table, y)
    assert torch.equal(y[4], table[3]) and not y[[0, 1, 2, 3, 5]].any()
    dy = normal(2, (6, 64))
    dy[[0, 1, 2, 3, 5]] = float("nan")
    mp.embedding_backward(tokens, dy, g, workspace=mp.embedding_workspace(6, 10, 64))
    want = torch.zeros_like(g)
    want[3] = dy[4].float()
    assert torch.equal(g, want)


def check_embedding_backward(tokens, dy, vocab, scale, accumulate, what=""):
    rows, cols = dy.shape
    old = normal(7, (vocab, cols), FP32)
    g = old.clone()
    ws = mp.embedding_workspace(rows, vocab, cols)
    ws.fill_(0xFF)
    mp.embedding_backward(tokens, dy, g, scale=scale, accumulate=accumulate, workspace=ws)
    t = tokens.cpu().numpy()
    s = float(np.float32(scale))
    d = np64(dy)
    want = O.embedding_backward(t, d, vocab, s)
    size = O.embedding_backward(t, np.abs(d), vocab, abs(s))
    n = np.bincount(t[(t >= 0) & (t < vocab)], minlength=vocab)[:, None]
    base = np64(old) if accumulate else np.zeros_like(want)
    within(g, want + base, (n + 1) * R32 * size + 2 * R32 * (np.abs(want) + np.abs(base)), what)
    untouched = torch.from_numpy(n[:, 0] == 0).cuda()
    assert torch.equal(g[untouched], old[untouched] if accumulate else torch.zeros_like(old[untouched])), what
    again = old.clone()
    mp.embedding_backward(tokens, dy, again, scale=scale, accumulate=accumulate, workspace=ws)
    assert torch.equal(g, again), what


@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (2, 5, 64), (63, 1000, 8), (64, 2, 136), (65, 1, 1111), (200, 40, 2056),
                                             (1031, 300, 72), (4500, 1100, 64), (5000, 70000, 24), (9000, 1 << 20, 8),
                                             (33000, 3, 16), (4096, 4096, 9)])
@pytest.mark.parametrize("dtype,layout", [(BF16, "dense"), (FP32, "dense"), (BF16, "aligned slice"), (FP32, "odd slice")])
def test_embedding_backward(rows, vocab, cols, dtype, layout):
    index = torch.int32 if cols % 2 else torch.int64
    tokens = (torch.rand(rows, generator=gen(3), device="cuda") ** 3 * (vocab + 1)).long() - (1 if vocab > 1 else 0)
    check_embedding_backward(tokens.to(index), normal(4, (rows, cols), dtype, layout=layout), vocab, 0.3, rows % 2 == 0)


@pytest.mark.parametrize("pattern", ["one token", "all padding", "all different", "runs of 16", "runs of 17", "runs of 64",
                                     "runs of 65", "padding first", "two halves"])
@pytest.mark.parametrize("rows", [16, 32, 33, 1000, 8200])
def test_embedding_backward_runs(pattern, rows):
    """Runs of equal tokens that start, end and go on at every place of a piece."""
    i = torch.arange(rows, device="cuda")
    tokens = {"one token": i * 0 + 5, "all padding": i * 0 - 1, "all different": (i * 7919) % rows, "runs of 16": i // 16,
              "runs of 17": i // 17, "runs of 64": i // 64, "runs of 65": i // 65, "padding first": torch.where(i < rows // 2, -1, i % 3), "two halves": i * 2 // rows}[pattern]
    check_embedding_backward(tokens, normal(5, (rows, 40)), max(rows, 6), 1.0, True, pattern)


@pytest.mark.parametrize("rows", [8191, 8192, 8193])
@pytest.mark.parametrize("vocab", [3, 1024, 300000])
def test_embedding_backward_sorts_few_and_many_rows_alike(rows, vocab):
    """The two ways to sort, at the number of rows where one takes over."""
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=gen(6), device="cuda")
    check_embedding_backward(tokens, normal(5, (rows, 8)), vocab, 1.0, True)


def test_embedding_backward_no_rows():
    g = normal(1, (5, 8), FP32)
    old = g.clone()
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    mp.embedding_backward(none, torch.zeros(0, 8, dtype=BF16, device="cuda"), g)
    assert torch.equal(g, old)
    mp.embedding_backward(none, torch.zeros(0, 8, dtype=BF16, device="cuda"), g, accumulate=False)
    assert not g.any()
    mp.embedding(none, normal(2, (5, 8)), torch.zeros(0, 8, dtype=BF16, device="cuda"))


def test_embedding_workspace_of_a_larger_call():
    ws = mp.embedding_workspace(3000, 5000, 256)
    for rows, vocab, cols in ((3000, 5000, 256), (2999, 10, 255), (1, 5000, 256), (64, 1, 1)):
        tokens = torch.randint(0, vocab, (rows,), generator=gen(1), device="cuda")
        dy = normal(2, (rows, cols))
        a, b = torch.zeros(vocab, cols, device="cuda"), torch.zeros(vocab, cols, device="cuda")
        mp.embedding_backward(tokens, dy, a, workspace=ws)
        mp.embedding_backward(tokens, dy, b, workspace=mp.embedding_workspace(rows, vocab, cols))
        assert torch.equal(a, b)


# ------------------------------------------------------------- recurrence --

def gate_values(seed, shape, dtype, layout="dense"):
    """Gates in [-8, 8], a column's slow or fast."""
    g = normal(seed, shape, FP32, 1.5) + (torch.rand(shape[-1], generator=gen(seed + 1), device="cuda") * 8 - 6)
    out = output(shape, dtype, layout)
    out.copy_(g.clamp(-8, 8))
    return out


def ragged(rows, sequences, seed, tail=3):
    """Starts of random sequences, some empty; with a tail, rows before the first and behind the last."""
    r = np.random.default_rng(seed)
    first, end = (min(2, rows), max(rows - tail, min(2, rows))) if tail else (0, rows)
    return np.concatenate([[first], np.sort(r.integers(first, end + 1, sequences - 1)), [end]])


def error_of(c, m):
    """e_t of the header for one sequence's rows: c [rows][cols], m [cols]."""
    e, out = np.zeros_like(m), np.empty_like(c)
    for t in range(len(c)):
        e = (1 - c[t]) * e + m * (2.0 ** -22 + 4 * c[t] * GATE)
        out[t] = e
    return out


def check_recurrence(rows, cols, starts, sequences, dtype, layout="dense", with_h0=True, seed=0, what=""):
    """Forward and backward against the oracle."""
    x, gate = normal(seed, (rows, cols), dtype, layout=layout), gate_values(seed + 1, (rows, cols), dtype, layout)
    dy = normal(seed + 3, (rows, cols), dtype, layout=layout)
    h0 = normal(seed + 4, (sequences, cols), FP32) if with_h0 else None
    dhT = normal(seed + 5, (sequences, cols), FP32) if with_h0 else None
    cuts = O.equal_starts(rows, sequences) if starts is None else starts
    st = None if starts is None else torch.from_numpy(np.asarray(starts, np.int32)).cuda()
    y, hT, states = output((rows, cols), dtype, layout), output((sequences, cols), FP32), mp.recurrence_states(rows, cols, dtype)
    states.fill_(float("nan"))
    mp.gated_recurrence(x, gate, y, starts=st, sequences=sequences, h0=h0, hT=hT, states=states)
    dx, dg, dh0 = output((rows, cols), dtype, layout), output((rows, cols), dtype, layout), output((sequences, cols), FP32)
    mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, starts=st, sequences=sequences, h0=h0, dhT=dhT, dh0=dh0)
    n = lambda t: None if t is None else np64(t)
    wy, whT, before = O.recurrence(n(x), n(gate), cuts, n(h0))
    wdx, wdg, wdh0, lam = O.recurrence_backward(n(dy), n(x), n(gate), cuts, n(h0), n(dhT))
    inside = np.zeros(rows, bool)
    c = F.sigmoid(n(gate))
    M = np.maximum(np.abs(n(x)).max(0), 0 if h0 is None else np.abs(n(h0)).max(0))
    ML = np.maximum(np.nan_to_num(np.abs(lam)).max(0), 0 if dhT is None else np.abs(n(dhT)).max(0))
    e, el, eb = (np.zeros((rows, cols)) for _ in range(3))       # of h, of l, of the h before a row
    eT, e0 = np.zeros((sequences, cols)), np.zeros((sequences, cols))
    for s in range(sequences):
        part = slice(cuts[s], cuts[s + 1])
        inside[part] = True
        if cuts[s + 1] > cuts[s]:
            e[part] = error_of(c[part], M)
            eb[part] = np.concatenate([np.zeros((1, cols)), e[part][:-1]])
            el[part] = error_of(c[part][::-1], ML)[::-1]
            eT[s], e0[s] = e[part][-1], el[part][0] + 4 * GATE * ML
    for t in (y, dx, dg):
        assert np.isnan(np64(t)[~inside]).all(), f"{what}: rows outside of the sequences were written"
        assert_frame_untouched(t, layout)
    if not inside.any():
        return
    half = STEP[dtype] * 1.01
    i = inside
    within(np64(y)[i], wy[i], (e + half * np.abs(wy))[i], what + " y")
    d = np.abs(n(x) - before)
    within(np64(dx)[i], wdx[i], (c * (el + 4 * GATE * np.abs(lam)) + half * np.abs(wdx))[i], what + " dx")
    bound = c * (1 - c) * (el * (d + eb) + np.abs(lam) * (eb + d * 8 * GATE + M * R32)) + half * np.abs(wdg)
    within(np64(dg)[i], wdg[i], bound[i], what + " dgate")
    within(hT, whT, eT + R32 * np.abs(whT), what + " hT")
    within(dh0, wdh0, e0 + R32 * np.abs(wdh0), what + " dh0")


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 8), (15, 64), (16, 63), (17, 72), (128, 64), (129, 200), (300, 1), (700, 136),
                                       (2100, 65), (4500, 8)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_recurrence(rows, cols, dtype, layout):
    check_recurrence(rows, cols, None, 1, dtype, layout)


@pytest.mark.parametrize("rows,cols,sequences", [(6, 64, 6), (64, 4096, 64), (12, 5, 4), (96, 72, 3), (340, 64, 20), (1000, 40, 500),
                                                 (2048, 264, 8), (4096, 64, 2)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_recurrence_equal_sequences(rows, cols, sequences, dtype):
    check_recurrence(rows, cols, None, sequences, dtype)


@pytest.mark.parametrize("rows,cols,sequences", [(1, 8, 1), (5, 64, 9), (40, 64, 3), (200, 9, 7), (700, 136, 40), (2100, 64, 5),
                                                 (900, 72, 900), (300, 8, 2000), (3000, 520, 2)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tail", [0, 3])
def test_recurrence_ragged(rows, cols, sequences, dtype, tail):
    check_recurrence(rows, cols, ragged(rows, sequences, rows + sequences, tail), sequences, dtype)


@pytest.mark.parametrize("starts", [[0, 0, 0, 0], [4, 4, 4], [0, 0, 16, 16, 32, 40, 40], [0, 40, 40], [0, 1, 2, 3, 40], [3, 19, 20, 37],
                                    [0, 15, 16, 17, 32, 33]])
@pytest.mark.parametrize("with_h0", [False, True])
def test_recurrence_borders(starts, with_h0):
    """Empty sequences everywhere, borders on and beside the groups of rows."""
    for dtype in (BF16, FP32):
        for layout in ("dense", "odd slice"):
            check_recurrence(40, 24, np.array(starts), len(starts) - 1, dtype, layout, with_h0, what=str(starts))


@pytest.mark.parametrize("cols", [2048, 2056, 4088, 4096, 4104, 4107, 4224])
@pytest.mark.parametrize("layout", ["dense", "aligned slice"])
def test_recurrence_wide(cols, layout):
    """Where the warps of a CTA and the columns of a lane change."""
    check_recurrence(700, cols, None, 1, BF16, layout)
    check_recurrence(140, cols, None, 7, BF16, layout)
    check_recurrence(300, cols, np.array([3, 3, 19, 20, 100, 100, 297]), 6, BF16, layout)
    check_recurrence(40, cols, np.array([0, 15, 16, 17, 32, 33]), 5, BF16, layout, False)


@pytest.mark.parametrize("sequences,rows,cols", [(3000, 9000, 8), (70, 9000, 16), (5, 9000, 640)])
def test_recurrence_many_shares(sequences, rows, cols):
    """Sequences shared out among CTAs, each boundary where the rows say."""
    check_recurrence(rows, cols, ragged(rows, sequences, 5), sequences, BF16)
    check_recurrence(sequences * 3, cols, None, sequences, BF16)


def test_recurrence_without_states_and_in_place():
    x, gate, h0 = normal(1, (300, 72)), gate_values(2, (300, 72), BF16), normal(3, (3, 72), FP32)
    y, hT = output((300, 72)), output((3, 72), FP32)
    mp.gated_recurrence(x, gate, y, sequences=3, h0=h0, hT=hT)
    for over in (0, 1):
        t = [x.clone(), gate.clone()]
        mp.gated_recurrence(t[0], t[1], t[over], sequences=3, h0=h0)
        assert torch.equal(t[over], y) and torch.equal(t[1 - over], (x, gate)[1 - over])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("starts", [None, [0, 7, 150, 150, 300]])
def test_recurrence_backward_in_place(dtype, starts):
    x, gate, dy = normal(1, (300, 72), dtype), gate_values(2, (300, 72), dtype), normal(3, (300, 72), dtype)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    states, y = mp.recurrence_states(300, 72, dtype), output((300, 72), dtype)
    mp.gated_recurrence(x, gate, y, starts=st, states=states)
    want = output((300, 72), dtype), output((300, 72), dtype)
    mp.gated_recurrence_backward(dy, x, gate, states, *want, starts=st)
    for i, j in ((0, 1), (1, 2), (2, 0), (1, 0)):
        t = [dy.clone(), x.clone(), gate.clone()]
        mp.gated_recurrence_backward(*t, states, t[i], t[j], starts=st)
        assert torch.equal(t[i], want[0]) and torch.equal(t[j], want[1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [64, 1000, 13])
def test_recurrence_token_by_token(dtype, cols):
    """Steps of one row to each sequence, the state updated in place, give what one
    call over all rows gives, each within the bound, and as y exactly the
    rounding of the state."""
    b, steps = 5, 40
    x, gate = normal(1, (b, steps, cols), dtype), gate_values(2, (b * steps, cols), dtype).view(b, steps, cols)
    y, hT = output((b * steps, cols), dtype), output((b, cols), FP32)
    h0 = normal(3, (b, cols), FP32)
    mp.gated_recurrence(x.view(-1, cols), gate.view(-1, cols), y, sequences=b, h0=h0, hT=hT)
    h = h0.clone()
    M = np.maximum(np.abs(np64(x)).max((0, 1)), np.abs(np64(h0)).max(0))
    for t in range(steps):
        out = output((b, cols), dtype)
        mp.gated_recurrence(x[:, t], gate[:, t], out, sequences=b, h0=h, hT=h)
        assert torch.equal(out, h.to(dtype))
    e = np.stack([error_of(F.sigmoid(np64(gate[i])), M)[-1] for i in range(b)])
    within(h, np64(hT), 2 * e, "state")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("starts", [[0, 100, 200, 300], [0, 100, 100, 250, 300]])
def test_recurrence_nonfinite_values_stay_in_their_sequence(bad, starts):
    """Nor do they reach another column."""
    n, cuts = len(starts) - 1, np.array(starts)
    st = None if n == 3 else torch.tensor(starts, dtype=torch.int32, device="cuda")
    x, gate, dy = normal(1, (300, 72)), gate_values(2, (300, 72), BF16), normal(3, (300, 72))
    outs = []
    for hit in (False, True):
        if hit:
            x[120, 5] = bad
            dy[130, 6] = bad
        states, y, hT = mp.recurrence_states(300, 72, BF16), output((300, 72)), output((n, 72), FP32)
        dx, dg, dh0 = output((300, 72)), output((300, 72)), output((n, 72), FP32)
        mp.gated_recurrence(x, gate, y, starts=st, sequences=n, hT=hT, states=states)
        mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, starts=st, sequences=n, dh0=dh0)
        outs.append((y, dx, dg, hT, dh0))
    seq = int(np.searchsorted(cuts, 120, side="right") - 1)
    rows, states_ = torch.ones(300, 72, dtype=torch.bool, device="cuda"), torch.ones(n, 72, dtype=torch.bool, device="cuda")
    rows[cuts[seq]:cuts[seq + 1], 5:7] = False
    states_[seq, 5:7] = False
    for a, b in zip(*outs):
        same = rows if len(a) == 300 else states_
        assert torch.equal(a[same], b[same])
    y, dx = outs[1][0], outs[1][1]
    assert not torch.isfinite(y[120:cuts[seq + 1], 5].float()).any()
    assert not torch.isfinite(dx[cuts[seq]:131, 6].float()).any()


@pytest.mark.parametrize("g,c", [(float("inf"), 1.0), (300.0, 1.0), (-float("inf"), 0.0), (-300.0, 0.0)])
def test_recurrence_saturated_gates(g, c):
    """Gates of either infinity and of any size: h is x or stays; nothing is NaN."""
    x, dy, h0 = normal(1, (64, 64), FP32), normal(3, (64, 64), FP32), normal(2, (1, 64), FP32)
    gate = torch.full_like(x, g)
    y, dx, dg = (output((64, 64), FP32) for _ in range(3))
    states, dh0 = mp.recurrence_states(64, 64, FP32), output((1, 64), FP32)
    mp.gated_recurrence(x, gate, y, h0=h0, states=states)
    mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, h0=h0, dh0=dh0)
    if c:                                                # h + (x - h): two roundings, of values below 10
        within(y, np64(x), 20 * R32)
        assert torch.equal(dx, dy) and not dh0.any()
    else:
        assert torch.equal(y, h0.expand(64, 64)) and not dx.any()
    assert not dg.any()


@pytest.mark.parametrize("starts", [[5, 3, 300, -7, 20], [1000, 1000, 1000, 1000, 1000], [-9, -8, -7, -6, -5], [40, 30, 20, 10, 0],
                                    [2 ** 31 - 1, -2 ** 31, 100, 50, 2 ** 31 - 1]])
def test_recurrence_starts_that_break_the_rules(starts):
    """Wrong results, but nothing outside of the outputs is written and the call ends."""
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    x, gate, dy = normal(1, (300, 72)), gate_values(2, (300, 72), BF16), normal(3, (300, 72))
    y, dx, dg = (output((300, 72), BF16, "aligned slice") for _ in range(3))
    states, hT, dh0 = mp.recurrence_states(300, 72, BF16), output((4, 72), FP32), output((4, 72), FP32)
    states.zero_()
    mp.gated_recurrence(x, gate, y, starts=st, hT=hT, states=states)
    mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, starts=st, dh0=dh0)
    torch.cuda.synchronize()
    for t in (y, dx, dg):
        assert_frame_untouched(t, "aligned slice")


def test_recurrence_long_and_slow():
    """A sequence of 20000 rows whose gate is so small that 1 - c keeps a tenth of
    its digits in fp32: the state follows the sum of c (x - h)."""
    rows = 20000
    x = torch.ones(rows, 64, device="cuda")
    gate = torch.full((rows, 64), -16.0, device="cuda")
    y, hT = output((rows, 64), FP32), output((1, 64), FP32)
    mp.gated_recurrence(x, gate, y, hT=hT)
    c = 1 / (1 + np.exp(16.0))
    want = 1 - (1 - c) ** rows                          # 2.2e-3
    # c to 2^-24 * 16 + 2^-21 of itself, and 20000 roundings of h <= want, half a step each, in one direction at worst
    within(hT, np.full((1, 64), want), want * (2.0 ** -19 + rows * R32))


# ------------------------------------------------------------ checkpoints --

@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (2, 31), (5, 32), (9, 33), (4, 40), (33, 136), (257, 1023), (100, 4096),
                                       (2, 14336)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_checkpoint(rows, cols, dtype, layout):
    blocks = -(-cols // 32)
    x = normal(1, (rows, cols), dtype, layout=layout)
    x *= torch.exp2(torch.randint(-20, 20, (rows, 1), generator=gen(2), device="cuda").float()).to(dtype)
    q, scale = output((rows, cols), E4M3, layout), output((rows, blocks), torch.uint8, layout)
    mp.checkpoint_save(x, q, scale)
    wq, we = O.checkpoint_save(np64(x))
    assert np.array_equal(scale.cpu().numpy().astype(int) - 127, we)
    assert np.array_equal(np64(q.float()), wq)
    assert_frame_untouched(q, layout)
    assert_frame_untouched(scale, layout)
    wz = O.checkpoint_restore(wq, we)
    dy = normal(3, (rows, cols), layout=layout)
    for act in ("none", "relu", "gelu", "silu"):
        z, y, dz = (output((rows, cols), BF16, layout) for _ in range(3))
        mp.checkpoint_restore(q, scale, z=z, y=y, act=act, dy=dy, dz=dz)
        assert np.array_equal(np64(z), wz)
        wy, wd = F.act(wz, act), F.act_grad(wz, act) * np64(dy)
        # where the factor counts as 0; and the oracle's own 1 + tanh, rounded in fp64 to 2^-53 beside a result of 1e-16 and less
        tiny = (2.0 ** -126 + 2.0 ** -52) * np.maximum(1, np.abs(wz))
        within(y, wy, np.abs(wy) * (HALF + ACT) + tiny, act)
        within(dz, wd, HALF * 1.01 * np.abs(wd) + ACT * np.abs(np64(dy)) + tiny, act + " dz")
        for t in (z, y, dz):
            assert_frame_untouched(t, layout)
        only, over = output((rows, cols), BF16, layout), dy.clone()
        mp.checkpoint_restore(q, scale, y=only, act=act)
        mp.checkpoint_restore(q, scale, act=act, dy=over, dz=over)
        assert torch.equal(only, y) and torch.equal(over, dz)


@pytest.mark.parametrize("other", [0.0, 1.0, 3e38])
def test_checkpoint_of_every_bf16_value(other):
    """Each value beside a smaller, a middling and a large neighbour."""
    v = torch.arange(0, 1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16)
    x = torch.zeros(1 << 16, 32, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = v, other
    q, scale, z = output(x.shape, E4M3), output((1 << 16, 1), torch.uint8), output(x.shape)
    mp.checkpoint_save(x, q, scale)
    wq, we = O.checkpoint_save(np64(x))
    assert np.array_equal(np64(q.float()), wq, equal_nan=True) and np.array_equal(scale.cpu().numpy().astype(int) - 127, we)
    mp.checkpoint_restore(q, scale, z=z)
    assert np.array_equal(np64(z), O.checkpoint_restore(wq, we), equal_nan=True)
    finite = torch.isfinite(x.float())
    assert torch.isfinite(z.float())[finite].all()


@pytest.mark.parametrize("cols", [96, 95])
def test_checkpoint_nonfinite_values_leave_their_block_alone(cols):
    x = normal(1, (4, cols))
    clean = x.clone()
    x[1, 40], x[2, cols - 1], x[3, 0] = float("nan"), float("inf"), -float("inf")
    clean[1, 40], clean[2, cols - 1], clean[3, 0] = 0, 0, 0
    outs = []
    for t in (x, clean):
        q, s, z = output((4, cols), E4M3), output((4, 3), torch.uint8), output((4, cols))
        mp.checkpoint_save(t, q, s)
        mp.checkpoint_restore(q, s, z=z)
        outs.append((s, z))
    assert torch.equal(outs[0][0], outs[1][0])
    bad = ~torch.isfinite(x.float())
    assert torch.isnan(outs[0][1][bad].float()).all() and torch.equal(outs[0][1][~bad], outs[1][1][~bad])


# ---------------------------------------------------------- cross-entropy --

def check_cross_entropy(x, labels, scale=1.0, weight=None, grad=True, layout="dense", what=""):
    rows, cols = x.shape
    loss, lse = output((rows,), FP32), output((rows,), FP32)
    g = output((rows, cols), x.dtype, layout) if grad else None
    mp.cross_entropy(x, labels, loss, lse=lse, dlogits=g, scale=scale, weight=weight)
    w = np.ones(rows) if weight is None else np64(weight)
    s = float(np.float32(scale))
    v, lab = np64(x), labels.cpu().numpy()
    wl, wlse, wg = O.cross_entropy(v, lab, s, w)
    total = (cols / 256 + 64) * R32 + 2.0 ** -20
    within(lse, wlse, total + 4 * R32 * np.abs(wlse), what + " lse")
    at = np.abs(v[np.arange(rows), np.clip(lab, 0, cols - 1)])
    within(loss, wl, total + 4 * R32 * (np.abs(wl) + at), what + " loss")
    if grad:
        d = np.abs(v - v.max(1, keepdims=True))
        p = np.exp(v - wlse[:, None])
        bound = np.abs(s * w)[:, None] * (p * (total + 2.0 ** -20 + 2 * R32 * d) + 4 * R32 * (np.abs(wg) > 0))
        within(g, wg, bound + STEP[x.dtype] * 1.01 * np.abs(wg) + 2.0 ** -126, what + " dlogits")
        assert_frame_untouched(g, layout)
    return loss, lse, g


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2), (3, 7), (9, 64), (33, 1000), (5, 1024), (4, 1025), (7, 4099), (64, 8192),
                                       (3, 32003), (2, 128256), (1, 300001)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_cross_entropy(rows, cols, dtype, layout):
    x = normal(1, (rows, cols), dtype, 3.0, layout)
    index = torch.int32 if cols % 2 else torch.int64
    labels = torch.randint(0, cols, (rows,), generator=gen(2), device="cuda")
    if rows > 1:
        labels[rows // 2] = -100
    labels = labels.to(index)
    weight = torch.rand(rows, generator=gen(3), device="cuda") if rows % 2 else None
    loss, lse, g = check_cross_entropy(x, labels, 0.37, weight, True, layout)
    only, _, _ = check_cross_entropy(x, labels, 0.37, weight, False)
    assert torch.equal(only, loss)
    over = output((rows, cols), dtype, layout)
    over.copy_(x)
    mp.cross_entropy(over, labels, dlogits=over, scale=0.37, weight=weight)
    assert torch.equal(over, g)
    if layout != "dense":                                       # outputs that lie differently from the logits
        dense = output((rows, cols), dtype)
        mp.cross_entropy(x, labels, dlogits=dense, scale=0.37, weight=weight)
        assert torch.equal(dense, g)


@pytest.mark.parametrize("cols", [4096, 4097, 8193, 16384, 16385, 16391, 32769, 65543, 131072, 131079])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_cross_entropy_shares(cols, dtype):
    """Widths where a row's threads or CTAs become more; the label first, last and
    beside every border; more rows than the GPU holds at once in the narrow ones."""
    rows = 700 if cols < 20000 else 9
    x = normal(1, (rows, cols), dtype, 3.0)
    labels = torch.randint(0, cols, (rows,), generator=gen(2), device="cuda")
    edges = [0, cols - 1, 1, cols - 2, 7, 8, cols // 2, 4095, cols - 9]
    labels[:len(edges)] = torch.tensor(edges, device="cuda")
    check_cross_entropy(x, labels, 0.37)
    over = x.clone()
    g = output((rows, cols), dtype)
    mp.cross_entropy(x, labels, dlogits=g)
    mp.cross_entropy(over, labels, dlogits=over)
    assert torch.equal(over, g)


@pytest.mark.parametrize("cols", [5, 64, 1500, 40000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_cross_entropy_masks(cols, dtype):
    """Columns ruled out by -inf or by the type's lowest value; rows of which
    nothing is left; a label that is ruled out."""
    inf, low = float("inf"), torch.finfo(dtype).min
    x = normal(1, (7, cols), dtype, 2.0)
    x[0, cols // 2:] = -inf
    x[1, 1:] = -inf                                             # one column left: the label's
    x[2] = -inf                                                 # none
    x[3, : cols // 2] = low
    x[4] = low                                                  # all equal
    x[5, 3] = -inf                                              # the label's
    x[6] = -inf
    labels = torch.tensor([0, 0, 1, cols - 1, 2, 3, -1], device="cuda")
    loss, lse, g = output((7,), FP32), output((7,), FP32), output((7, cols), dtype)
    mp.cross_entropy(x, labels, loss, lse=lse, dlogits=g)
    wl, wlse, wg = O.cross_entropy(np64(x), labels.cpu().numpy())
    total = (cols / 256 + 64) * R32 + 2.0 ** -20
    # a row of lowest values alone has loss log(cols), but a label's distance from lse is lost in 3e38
    wl[4] = np.log(cols)
    fine = np.array([1, 1, 0, 1, 1, 0, 1], bool)
    assert np.array_equal(np64(loss)[~fine], wl[~fine]) and np.isinf(wl[~fine]).all()
    within(np64(loss)[fine], wl[fine], total + 4 * R32 * np.array([20, 20, 20, 20, 20])[: fine.sum()])
    fine = np.array([1, 1, 0, 1, 1, 1, 0], bool)
    assert np.array_equal(np64(lse)[~fine], [-inf, -inf])
    within(np64(lse)[fine], wlse[fine], total + 4 * R32 * np.abs(wlse[fine]))
    within(g, wg, STEP[dtype] * 1.01 * np.abs(wg) + 4 * total + 2.0 ** -20)
    assert not g[2].any() and not g[6].any() and not g[0, cols // 2:].any()


@pytest.mark.parametrize("cols", [9, 2000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_cross_entropy_nonfinite_rows(cols, bad):
    """A NaN or +inf fills its own row, unless the label is to be ignored."""
    x = normal(1, (4, cols))
    x[1, 3] = x[2, 3] = bad
    labels = torch.tensor([0, 1, -100, 2], device="cuda")
    loss, lse, g = output((4,), FP32), output((4,), FP32), output((4, cols))
    mp.cross_entropy(x, labels, loss, lse=lse, dlogits=g)
    assert torch.isnan(loss[1]) and torch.isnan(lse[1:3]).all() and torch.isnan(g[1].float()).all()
    assert float(loss[2]) == 0 and not g[2].any()
    for r in (0, 3):
        one = output((1, cols))
        mp.cross_entropy(x[r:r + 1], labels[r:r + 1], dlogits=one)
        assert torch.equal(one[0], g[r]) and torch.isfinite(loss[r])
    mp.cross_entropy(x, labels, loss)                            # without lse the row is not looked at
    assert float(loss[2]) == 0


def test_cross_entropy_large_logits():
    """The sum is taken from the maximum: offsets of any size change nothing else."""
    x = torch.randint(-8, 8, (6, 3000), generator=gen(1), device="cuda").float()
    labels = torch.randint(0, 3000, (6,), generator=gen(2), device="cuda")
    base, g = output((6,), FP32), output((6, 3000), FP32)
    mp.cross_entropy(x, labels, base, dlogits=g)
    for off in (1e4, -1e4, 2.0 ** 20):
        far, h = output((6,), FP32), output((6, 3000), FP32)
        mp.cross_entropy(x + off, labels, far, dlogits=h)
        assert torch.equal(far, base) and torch.equal(h, g)


# ------------------------------------------------------------------- all --

def test_no_rows():
    e = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
    mp.checkpoint_save(e(0, 40), e(0, 40, dtype=E4M3), e(0, 2, dtype=torch.uint8))
    mp.checkpoint_restore(e(0, 40, dtype=E4M3), e(0, 2, dtype=torch.uint8), y=e(0, 40))
    mp.cross_entropy(e(0, 40), e(0, dtype=torch.int64), e(0, dtype=FP32), dlogits=e(0, 40))
    h0, hT = normal(1, (3, 40), FP32), output((3, 40), FP32)
    mp.gated_recurrence(e(0, 40), e(0, 40), e(0, 40), sequences=3, h0=h0, hT=hT)
    assert torch.equal(hT, h0)
    mp.gated_recurrence(e(0, 40), e(0, 40), e(0, 40), sequences=3, hT=hT)
    assert not hT.any()
    dh0 = output((3, 40), FP32)
    mp.gated_recurrence_backward(e(0, 40), e(0, 40), e(0, 40), None, e(0, 40), e(0, 40), sequences=3, dhT=h0, dh0=dh0)
    assert torch.equal(dh0, h0)


def test_rows_far_apart():
    """Row distances and offsets past 32 bits (elements and bytes)."""
    ld = (1 << 31) + 64
    buf = torch.zeros(2 * ld + 4096, dtype=BF16, device="cuda")
    far = lambda n, off: torch.as_strided(buf, (3, n), (ld, 1), off)
    x, gate, y, dx, dg = (far(256, k * 256) for k in range(5))
    x.copy_(normal(1, (3, 256)))
    gate.copy_(normal(2, (3, 256)))
    near, ng = x.contiguous(), gate.contiguous()
    a, states, states2 = output((3, 256)), mp.recurrence_states(3, 256, BF16), mp.recurrence_states(3, 256, BF16)
    mp.gated_recurrence(x, gate, y, states=states)
    mp.gated_recurrence(near, ng, a, states=states2)
    assert torch.equal(y.contiguous(), a)
    b = output((3, 256)), output((3, 256))
    mp.gated_recurrence_backward(x, x, gate, states, dx, dg)
    mp.gated_recurrence_backward(near, near, ng, states2, *b)
    assert torch.equal(dx.contiguous(), b[0]) and torch.equal(dg.contiguous(), b[1])
    tokens = torch.tensor([2, 0, 1, 2, 3], device="cuda")
    e = output((5, 256))
    mp.embedding(tokens, x, e)
    assert torch.equal(e, torch.cat([near[tokens[:4]], torch.zeros_like(near[:1])]))
    mp.embedding(tokens[:3], near, y)
    assert torch.equal(y.contiguous(), near[tokens[:3]])
    t1, t2, ws = torch.zeros(4, 256, device="cuda"), torch.zeros(4, 256, device="cuda"), mp.embedding_workspace(3, 4, 256)
    mp.embedding_backward(tokens[:3], x, t1, workspace=ws)
    mp.embedding_backward(tokens[:3], near, t2, workspace=ws)
    assert torch.equal(t1, t2)
    q, s, q2, s2 = output((3, 256), E4M3), output((3, 8), torch.uint8), output((3, 256), E4M3), output((3, 8), torch.uint8)
    mp.checkpoint_save(x, q, s)
    mp.checkpoint_save(near, q2, s2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    mp.checkpoint_restore(q, s, y=y, act="silu", dy=x, dz=dx)
    mp.checkpoint_restore(q, s, y=a, act="silu", dy=near, dz=b[0])
    assert torch.equal(y.contiguous(), a) and torch.equal(dx.contiguous(), b[0])
    mp.cross_entropy(x, tokens[:3], dlogits=y)
    mp.cross_entropy(near, tokens[:3], dlogits=a)
    assert torch.equal(y.contiguous(), a)


def chain(tokens, labels, table, starts, bufs, ws, stream=None):
    """Embedding, checkpoint, recurrence, loss, and back."""
    x, gate, y, dx, dg, states, q, s, loss, g, dtable = bufs
    mp.embedding(tokens, table, x, scale=4.0, stream=stream)
    mp.checkpoint_save(x, q, s, stream=stream)
    mp.checkpoint_restore(q, s, y=gate, act="silu", stream=stream)
    mp.gated_recurrence(x, gate, y, starts=starts, states=states, stream=stream)
    mp.cross_entropy(y, labels, loss, dlogits=g, scale=0.1, stream=stream)
    mp.gated_recurrence_backward(g, x, gate, states, dx, dg, starts=starts, stream=stream)
    mp.embedding_backward(tokens, dx, dtable, scale=4.0, accumulate=False, workspace=ws, stream=stream)


def test_other_stream_and_graph():
    """A run of them enqueues on the stream it is given, and a captured one
    replays with the inputs of the moment."""
    rows, cols, vocab = 500, 200, 300
    tokens = torch.randint(-1, vocab, (rows,), generator=gen(1), device="cuda")
    labels, table = torch.randint(0, cols, (rows,), generator=gen(2), device="cuda"), normal(3, (vocab, cols))
    starts = torch.tensor([0, 100, 333, 333, 490], dtype=torch.int32, device="cuda")
    new = lambda dtype=BF16: torch.zeros(rows, cols, dtype=dtype, device="cuda")
    bufs = (new(), new(), new(), new(), new(), torch.zeros_like(mp.recurrence_states(rows, cols, BF16)),
            torch.zeros(rows, cols, dtype=torch.uint8, device="cuda").view(E4M3),
            torch.zeros(rows, 7, dtype=torch.uint8, device="cuda"), torch.zeros(rows, device="cuda"), new(),
            torch.zeros(vocab, cols, device="cuda"))
    ws = mp.embedding_workspace(rows, vocab, cols)
    outs = [t for t in bufs if t.dtype != E4M3]

    def clear():
        for t in outs:
            t.zero_()
    chain(tokens, labels, table, starts, bufs, ws)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    clear()
    side.wait_stream(torch.cuda.current_stream())
    chain(tokens, labels, table, starts, bufs, ws, stream=side)
    side.synchronize()
    for t, v in zip(outs, want):
        assert torch.equal(t, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(tokens, labels, table, starts, bufs, ws)
    keep, cuts = tokens.clone(), starts.clone()
    tokens.copy_(torch.randint(0, vocab, (rows,), generator=gen(9), device="cuda"))
    starts.copy_(torch.tensor([3, 3, 200, 400, 500], dtype=torch.int32))
    clear()
    graph.replay()
    torch.cuda.synchronize()
    second = [t.clone() for t in outs]
    clear()
    chain(tokens, labels, table, starts, bufs, ws)
    torch.cuda.synchronize()
    for t, v in zip(outs, second):
        assert torch.equal(t, v)
    tokens.copy_(keep)
    starts.copy_(cuts)
    clear()
    graph.replay()
    torch.cuda.synchronize()
    for t, v in zip(outs, want):
        assert torch.equal(t, v)


FIRST_CALLS_CAPTURED = """
import torch, mixed_precision_optimizer_gb300 as mp
x, gate, dy = (torch.randn(500, 2048, device="cuda").to(torch.bfloat16) for _ in range(3))
labels, tokens = torch.arange(500, device="cuda"), torch.arange(500, device="cuda") % 7
y, g, dx, dg = (torch.zeros_like(x) for _ in range(4))
wide = torch.randn(40, 40000, device="cuda")
states, table = mp.recurrence_states(500, 2048, x.dtype), torch.zeros(9, 2048, device="cuda")
loss, ws, dwide = torch.zeros(40, device="cuda"), mp.embedding_workspace(9000, 9, 2048), torch.zeros_like(wide)
many = torch.arange(9000, device="cuda") % 9
rows = torch.randn(9000, 2048, device="cuda")
def step():
    mp.gated_recurrence(x, gate, y, states=states)
    mp.cross_entropy(y, labels, dlogits=g)
    mp.cross_entropy(wide, labels[:40], loss, dlogits=dwide)
    mp.gated_recurrence_backward(dy, x, gate, states, dx, dg)
    mp.embedding_backward(many, rows, table, accumulate=False, workspace=ws)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
outs = [t.clone() for t in (y, g, loss, dwide, dx, dg, table)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, (y, g, loss, dwide, dx, dg, table))) and y.any() and table.any()
print("same")
"""


def test_first_calls_of_a_process_are_captured():
    """What a kernel asks once (its shared memory, the clusters that fit) may be asked
    while a stream is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_calls_on_two_streams_at_once():
    """Calls that share inputs, each with outputs and a workspace of its own."""
    rows, cols, vocab = 3000, 512, 700
    tokens, dy = torch.randint(0, vocab, (rows,), generator=gen(1), device="cuda"), normal(2, (rows, cols))
    gate = normal(3, (rows, cols))
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.zeros(vocab, cols, device="cuda"), output((rows, cols)), mp.embedding_workspace(rows, vocab, cols)) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (t, y, ws) in zip(sides, outs):
            mp.embedding_backward(tokens, dy, t, accumulate=False, workspace=ws, stream=s)
            mp.gated_recurrence(dy, gate, y, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(outs[0][:2], outs[1][:2]):
        assert torch.equal(a, b)
    y = output((rows, cols))
    mp.gated_recurrence(dy, gate, y)
    assert torch.equal(y, outs[0][1])


def test_gradients_against_differences():
    """The kernels' gradient of a small fp32 chain against central differences of
    the oracle's loss in fp64: truncation and rounding of the differences are
    below 1e-6, the kernels' errors (fp32) below 1e-5 of values of order one."""
    r = np.random.default_rng(0)
    rows, cols, vocab, starts = 12, 5, 4, np.array([0, 5, 5, 11])
    tokens, labels = r.integers(-1, vocab, rows), r.integers(0, cols, rows)
    table, gate, h0 = (r.normal(size=s).astype(np.float32) for s in ((vocab, cols), (rows, cols), (3, cols)))

    def loss(table_, gate_, h0_):
        y, _, _ = O.recurrence(O.embedding(tokens, table_, 1.5), gate_, starts, h0_)
        return float(O.cross_entropy(y[:11], labels[:11])[0].sum())
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    st = d(starts.astype(np.int32))
    x, y, g, dx, dg = (torch.zeros(rows, cols, device="cuda") for _ in range(5))
    states, dh0, dtable = mp.recurrence_states(rows, cols, FP32), output((3, cols), FP32), torch.zeros(vocab, cols, device="cuda")
    mp.embedding(d(tokens), d(table), x, scale=1.5)
    mp.gated_recurrence(x, d(gate), y, starts=st, h0=d(h0), states=states)
    lab = labels.copy()
    lab[11:] = -1
    mp.cross_entropy(y, d(lab), dlogits=g)
    mp.gated_recurrence_backward(g, x, d(gate), states, dx, dg, starts=st, h0=d(h0), dh0=dh0)
    mp.embedding_backward(d(tokens), dx, dtable, scale=1.5, workspace=mp.embedding_workspace(rows, vocab, cols))

    def differences(f, a):
        out = np.zeros(a.shape)
        for i in np.ndindex(a.shape):
            p, m = a.astype(np.float64), a.astype(np.float64)
            p[i] += 1e-4
            m[i] -= 1e-4
            out[i] = (f(p) - f(m)) / 2e-4
        return out
    within(dtable, differences(lambda t: loss(t, gate, h0), table), 1e-5)
    within(dg[:11], differences(lambda t: loss(table, t, h0), gate)[:11], 1e-5)
    within(dh0, differences(lambda t: loss(table, gate, t), h0), 1e-5)


def test_launches_are_named():
    with mp.LaunchProfiler(64) as prof:
        tokens, table = torch.randint(0, 9, (200,), generator=gen(1), device="cuda"), normal(1, (9, 64))
        x, y, states, g = output((200, 64)), output((200, 64)), mp.recurrence_states(200, 64, BF16), output((200, 64))
        mp.embedding(tokens, table, x)
        mp.gated_recurrence(x, x, y, states=states)
        mp.cross_entropy(y, tokens, dlogits=g)
        mp.gated_recurrence_backward(g, x, x, states, y, g)
        q, s = output((200, 64), E4M3), output((200, 2), torch.uint8)
        mp.checkpoint_save(x, q, s)
        mp.checkpoint_restore(q, s, y=y, act="gelu")
        mp.embedding_backward(tokens, x, torch.zeros(9, 64, device="cuda"), workspace=mp.embedding_workspace(200, 9, 64))
    torch.cuda.synchronize()
    names = {r["kernel"] for r in prof.records()}
    assert {"embedding", "embedding_grad", "recurrence", "recurrence_grad", "checkpoint_save", "checkpoint_restore",
            "cross_entropy"} <= names


def test_python_argument_checks():
    t = torch.randint(0, 9, (24,), generator=gen(1), device="cuda")
    x, table = normal(1, (4, 6, 64)), normal(2, (9, 64))
    y = output((4, 6, 64))
    mp.embedding(t.view(4, 6), table, y)
    assert torch.equal(y.view(24, 64), table[t])
    with pytest.raises(ValueError, match="y has shape"):
        mp.embedding(t, table, output((23, 64)))
    with pytest.raises(TypeError, match="int32 or int64"):
        mp.embedding(t.short(), table, y)
    with pytest.raises(ValueError, match="tokens must be"):
        mp.embedding(t.repeat(2)[::2], table, y)
    with pytest.raises(ValueError, match="CUDA"):
        mp.embedding(t.cpu(), table, y)
    with pytest.raises(ValueError, match="dtable has shape"):
        mp.embedding_backward(t, x, torch.zeros(9, 63, device="cuda"))
    with pytest.raises(ValueError, match="tokens must be"):
        mp.embedding_backward(t[:23], x, torch.zeros(9, 64, device="cuda"))
    with pytest.raises(mp.MpoptError, match="WORKSPACE"):
        mp.embedding_backward(t, x, torch.zeros(9, 64, device="cuda"))
    with pytest.raises(TypeError, match="gate must be"):
        mp.gated_recurrence(x, x.float(), y)
    with pytest.raises(ValueError, match="h0 has shape"):
        mp.gated_recurrence(x, x, y, sequences=2, h0=torch.zeros(1, 64, device="cuda"))
    with pytest.raises(ValueError, match="states has shape"):
        mp.gated_recurrence(x, x, y, states=torch.zeros(1, 64, device="cuda"))
    with pytest.raises(TypeError, match="starts must be"):
        mp.gated_recurrence(x, x, y, starts=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="starts has 3"):
        mp.gated_recurrence(x, x, y, starts=torch.zeros(3, dtype=torch.int32, device="cuda"), sequences=3)
    with pytest.raises(mp.MpoptError, match="INVALID"):
        mp.gated_recurrence(x, x, y, sequences=5)
    with pytest.raises(mp.MpoptError, match="INVALID"):
        mp.gated_recurrence_backward(x, x, x, None, y, output((4, 6, 64)))
    with pytest.raises(ValueError, match="scale has shape"):
        mp.checkpoint_save(x, output((4, 6, 64), E4M3), output((24, 1), torch.uint8))
    with pytest.raises(TypeError, match="scale must be"):
        mp.checkpoint_save(x, output((4, 6, 64), E4M3), torch.zeros(24, 2, device="cuda"))
    with pytest.raises(mp.MpoptError, match="INVALID"):
        mp.checkpoint_restore(output((24, 64), E4M3), output((24, 2), torch.uint8), dz=output((24, 64)))
    with pytest.raises(ValueError, match="labels must be"):
        mp.cross_entropy(x, t[:5], torch.zeros(24, device="cuda"))
    with pytest.raises(TypeError, match="dlogits must be"):
        mp.cross_entropy(x, t, dlogits=torch.zeros(24, 64, device="cuda"))
    with pytest.raises(ValueError, match="loss must be"):
        mp.cross_entropy(x, t, torch.zeros(23, device="cuda"))
    with pytest.raises(RuntimeError):
        mp.cross_entropy(x.transpose(0, 1), t, torch.zeros(24, device="cuda"))
