"""Language-model operators without a GPU: the fp64 oracle's gradients against
central differences, its checkpoints against the definition, and every refusal
of the C entry points and of the Python checks.  Pointers passed to the library
are fake aligned addresses: each call returns before a CUDA call."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_optimizer_gb300 as mp
from mixed_precision_optimizer_gb300 import build_lib, language as lm
from oracle import language as O

INV, UNSUP, MIS, WS = 1, 2, 3, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return mp.lib()


# ---------------------------------------------------------------- oracle --

# Central differences in fp64 with step 1e-4 on values of order one: truncation
# near 1e-8, rounding near 1e-11, so 1e-6 separates a wrong formula from them.
H, TOL = 1e-4, 1e-6


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += H
        b[i] -= H
        g[i] = (f(a) - f(b)) / (2 * H)
    return g


def test_oracle_recurrence_gradient():
    r = np.random.default_rng(0)
    rows, cols, starts = 9, 3, np.array([0, 4, 4, 5, 8])           # one empty, one of one row, one row behind the last
    x, gate, dy = r.normal(size=(rows, cols)), r.normal(size=(rows, cols)), r.normal(size=(rows, cols))
    h0, dhT = r.normal(size=(4, cols)), r.normal(size=(4, cols))

    def loss(x_, gate_, h0_):
        y, hT, _ = O.recurrence(x_, gate_, starts, h0_)
        return float((y[:8] * dy[:8]).sum() + (hT * dhT).sum())
    dx, dgate, dh0, _ = O.recurrence_backward(dy, x, gate, starts, h0, dhT)
    for got, want in ((differences(lambda t: loss(t, gate, h0), x), dx), (differences(lambda t: loss(x, t, h0), gate), dgate)):
        assert np.max(np.abs(got[:8] - want[:8])) < TOL and np.isnan(want[8]).all()
    assert np.max(np.abs(differences(lambda t: loss(x, gate, t), h0) - dh0)) < TOL


def test_oracle_cross_entropy_gradient():
    r = np.random.default_rng(1)
    x, labels, w = r.normal(size=(4, 6)) * 2, np.array([0, 5, -1, 3]), r.random(4)
    _, lse, g = O.cross_entropy(x, labels, 0.5, w)
    got = differences(lambda t: float((O.cross_entropy(t, labels)[0] * w * 0.5).sum()), x)
    assert np.max(np.abs(got - g)) < TOL
    assert np.allclose(lse, np.log(np.exp(x).sum(axis=1)), rtol=1e-14)


def test_oracle_cross_entropy_masks():
    inf = np.inf
    x = np.array([[-inf, -inf, -inf], [-inf, 1.0, -inf], [0.0, -inf, 0.0]])
    loss, lse, g = O.cross_entropy(x, np.array([1, 1, 1]))
    assert loss[0] == inf and lse[0] == -inf and not g[0].any()
    assert loss[1] == 0 and lse[1] == 1 and not g[1].any()
    assert loss[2] == inf and np.array_equal(g[2], [0.5, -1, 0.5])


def test_oracle_embedding_gradient():
    r = np.random.default_rng(2)
    table, tokens, dy = r.normal(size=(5, 3)), np.array([4, 0, 4, -1, 5, 4]), r.normal(size=(6, 3))
    got = differences(lambda t: float((O.embedding(tokens, t, 1.5) * dy).sum()), table)
    assert np.max(np.abs(got - O.embedding_backward(tokens, dy, 5, 1.5))) < TOL


def test_oracle_checkpoint():
    """The exponent is the smallest that takes the block to 448, and a value is
    off by no more than half a step of its code."""
    r = np.random.default_rng(3)
    x = r.normal(size=(40, 75)) * 2.0 ** r.integers(-30, 30, size=(40, 1))
    x[0, :32] = 448.0
    x[1, :32] = np.nextafter(448.0, 1e3)
    x[2, :32] = 0.0
    x[3, 3], x[3, 4] = np.nan, -np.inf
    q, e = O.checkpoint_save(x)
    assert e[0, 0] == 0 and e[1, 0] == 1 and e[2, 0] == O.MIN_EXP
    assert np.isnan(q[3, 3]) and np.isnan(q[3, 4]) and np.isfinite(np.delete(q[3], [3, 4])).all()
    z = O.checkpoint_restore(q, e)
    ok = np.isfinite(x)
    scale = np.exp2(np.repeat(e, 32, axis=1)[:, :75].astype(float))
    assert (np.abs(q[ok]) <= 448).all()
    assert (np.abs(z - x)[ok] <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)[ok]).all()


# ------------------------------------------------------------- refusals --

def call(L, name, cls, values, kw, *more):
    a = cls(**values)
    for k, v in kw.items():
        setattr(a, k, v)
    return getattr(L, name)(ctypes.byref(a), *more)


EMBEDDING = dict(tokens=FAKE, table=FAKE, y=FAKE, rows=4, vocab=10, cols=64, table_ld=64, y_ld=64, index_dtype=1, dtype=1,
                 y_dtype=1, scale=1.0)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=None), INV), (dict(table=None), INV), (dict(y=None), INV), (dict(rows=-1), INV), (dict(vocab=0), INV),
    (dict(cols=0), INV), (dict(table_ld=63), INV), (dict(y_ld=63), INV), (dict(index_dtype=2), INV), (dict(dtype=2), INV),
    (dict(y_dtype=2), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(tokens=FAKE + 4), MIS),
    (dict(tokens=FAKE + 2, index_dtype=0), MIS), (dict(table=FAKE + 1), MIS), (dict(y=FAKE + 2, y_dtype=0), MIS),
    (dict(rows=(1 << 30) + 1), INV), (dict(rows=0, tokens=None, y=None), 0)])
def test_embedding_refusals(L, kw, want):
    assert call(L, "opt_embedding_forward", lm.OptEmbeddingArgs, EMBEDDING, kw, None) == want


EMBEDDING_GRAD = dict(tokens=FAKE, dy=FAKE, dtable=FAKE, rows=4, vocab=10, cols=64, dy_ld=64, index_dtype=1, dtype=1,
                      accumulate=1, scale=1.0)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=None), INV), (dict(dy=None), INV), (dict(dtable=None), INV), (dict(dy_ld=63), INV), (dict(vocab=0), INV),
    (dict(vocab=(1 << 30) + 1), INV), (dict(dtype=2), INV), (dict(index_dtype=-1), INV), (dict(dtable=FAKE + 2), MIS),
    (dict(dy=FAKE + 1), MIS), (dict(scale=float("nan")), INV), (dict(rows=0, tokens=None, dy=None), 0)])
def test_embedding_backward_refusals(L, kw, want):
    assert call(L, "opt_embedding_backward", lm.OptEmbeddingGradArgs, EMBEDDING_GRAD, kw, FAKE, 1 << 30, None) == want


def test_embedding_workspace(L):
    need = mp.embedding_workspace_size(1000, 500, 64)
    assert need >= 4 * 4 * 1000
    for rows, vocab, cols in ((999, 500, 64), (1000, 1, 64), (1, 500, 63), (64, 3, 1)):
        assert mp.embedding_workspace_size(rows, vocab, cols) <= need
    assert mp.embedding_workspace_size(0, 500, 64) == mp.embedding_workspace_size(4, 0, 64) == 0
    for rows in (8193, 20000, 40000):               # fewer rows in shorter pieces
        assert mp.embedding_workspace_size(rows, 10, 64) >= mp.embedding_workspace_size(8192, 10, 64)
    need = mp.embedding_workspace_size(4, 10, 64)
    for ws, nb in ((None, 1 << 20), (FAKE, need - 1), (FAKE + 64, 1 << 20)):
        assert call(L, "opt_embedding_backward", lm.OptEmbeddingGradArgs, EMBEDDING_GRAD, {}, ws, nb, None) == WS


RECURRENCE = dict(x=FAKE, gate=FAKE * 2, starts=None, h0=FAKE * 3, y=FAKE * 4, hT=FAKE * 5, states=FAKE * 6, rows=8, cols=64,
                  sequences=2, x_ld=64, gate_ld=64, y_ld=64, dtype=1)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(gate=None), INV), (dict(y=None), INV), (dict(rows=9), INV), (dict(sequences=0), INV),
    (dict(cols=0), INV), (dict(dtype=2), INV), (dict(x_ld=63), INV), (dict(gate_ld=63), INV), (dict(y_ld=63), INV),
    (dict(x=FAKE + 1), MIS), (dict(starts=FAKE + 2), MIS), (dict(h0=FAKE * 3 + 2), MIS), (dict(hT=FAKE * 5 + 1), MIS),
    (dict(states=FAKE * 6 + 2), MIS), (dict(hT=FAKE * 3), INV), (dict(hT=FAKE * 3 + 256), INV),
    (dict(hT=FAKE * 3, starts=FAKE, sequences=8), INV), (dict(hT=FAKE * 3 + 4, sequences=8), INV),
    (dict(y=FAKE, y_ld=72), INV), (dict(y=FAKE * 2, y_ld=72), INV), (dict(rows=(1 << 30) + 2), INV),
    (dict(rows=0, hT=None, x=None, gate=None, y=None), 0), (dict(rows=0, hT=FAKE * 3), 0)])
def test_recurrence_refusals(L, kw, want):
    assert call(L, "opt_recurrence_forward", lm.OptRecurrenceArgs, RECURRENCE, kw, None) == want


RECURRENCE_GRAD = dict(dy=FAKE, x=FAKE * 2, gate=FAKE * 3, starts=None, h0=FAKE * 4, states=FAKE * 5, dhT=FAKE * 6, dx=FAKE * 7,
                       dgate=FAKE * 8, dh0=FAKE * 9, rows=8, cols=64, sequences=2, dy_ld=64, x_ld=64, gate_ld=64, dx_ld=64,
                       dgate_ld=64, dtype=1)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INV), (dict(x=None), INV), (dict(gate=None), INV), (dict(states=None), INV), (dict(dx=None), INV),
    (dict(dgate=None), INV), (dict(rows=9), INV), (dict(sequences=0), INV), (dict(dtype=2), INV), (dict(dy_ld=63), INV),
    (dict(dx_ld=63), INV), (dict(dgate_ld=63), INV), (dict(dh0=FAKE * 6), INV), (dict(dh0=FAKE * 4), INV),
    (dict(dgate=FAKE * 7), INV), (dict(dx=FAKE, dx_ld=72), INV), (dict(dgate=FAKE * 3, dgate_ld=72), INV),
    (dict(states=FAKE * 5 + 2), MIS), (dict(dhT=FAKE * 6 + 2), MIS), (dict(dx=FAKE * 7 + 1), MIS),
    (dict(rows=0, dh0=None, dy=None, x=None, gate=None, states=None, dx=None, dgate=None), 0)])
def test_recurrence_backward_refusals(L, kw, want):
    assert call(L, "opt_recurrence_backward", lm.OptRecurrenceGradArgs, RECURRENCE_GRAD, kw, None) == want


def test_state_rows(L):
    assert [L.opt_recurrence_state_rows(d) for d in (0, 1, 2, -1)] == [lm.STATE_ROWS, lm.STATE_ROWS, 0, 0]


@pytest.mark.parametrize("args,want", [
    ((None, 64, 1, 2, 64, FAKE, 64, FAKE, 2, None), INV), ((FAKE, 64, 1, 2, 64, None, 64, FAKE, 2, None), INV),
    ((FAKE, 64, 1, 2, 64, FAKE, 64, None, 2, None), INV), ((FAKE, 63, 1, 2, 64, FAKE, 64, FAKE, 2, None), INV),
    ((FAKE, 64, 1, 2, 64, FAKE, 63, FAKE, 2, None), INV), ((FAKE, 64, 1, 2, 64, FAKE, 64, FAKE, 1, None), INV),
    ((FAKE, 64, 2, 2, 64, FAKE, 64, FAKE, 2, None), INV), ((FAKE + 1, 64, 1, 2, 64, FAKE, 64, FAKE, 2, None), MIS),
    ((FAKE, 64, 1, -2, 64, FAKE, 64, FAKE, 2, None), INV), ((FAKE, 64, 1, 2, 0, FAKE, 64, FAKE, 2, None), INV),
    ((None, 64, 1, 0, 64, None, 64, None, 2, None), 0)])
def test_checkpoint_save_refusals(L, args, want):
    assert L.opt_checkpoint_save(*args) == want


CHECKPOINT = dict(q=FAKE, scale=FAKE, dy=FAKE, z=FAKE, y=FAKE, dz=FAKE, rows=4, cols=64, q_ld=64, scale_ld=2, dy_ld=64, z_ld=64,
                  y_ld=64, dz_ld=64, act=2)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(scale=None), INV), (dict(dy=None), INV), (dict(dz=None), INV), (dict(act=4), INV),
    (dict(act=-1), INV), (dict(q_ld=63), INV), (dict(scale_ld=1), INV), (dict(z_ld=63), INV), (dict(y_ld=63), INV),
    (dict(dz_ld=72), INV), (dict(z=FAKE + 1), MIS), (dict(dy=FAKE + 1), MIS), (dict(cols=0), INV), (dict(rows=-1), INV),
    (dict(rows=0, q=None), 0), (dict(dy=None, z=None, y=None, dz=None), 0)])
def test_checkpoint_restore_refusals(L, kw, want):
    assert call(L, "opt_checkpoint_restore", lm.OptCheckpointArgs, CHECKPOINT, kw, None) == want


CROSS_ENTROPY = dict(logits=FAKE, labels=FAKE, weight=None, loss=FAKE, lse=FAKE, dlogits=FAKE * 2, rows=4, cols=64, logits_ld=64,
                     dlogits_ld=64, dtype=1, index_dtype=1, scale=1.0)


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), INV), (dict(labels=None), INV), (dict(logits_ld=63), INV), (dict(dlogits_ld=63), INV),
    (dict(dtype=2), INV), (dict(index_dtype=3), INV), (dict(scale=float("inf")), INV), (dict(cols=0), INV),
    (dict(dlogits=FAKE, dlogits_ld=72), INV), (dict(logits=FAKE + 1), MIS), (dict(labels=FAKE + 4), MIS),
    (dict(loss=FAKE + 2), MIS), (dict(lse=FAKE + 2), MIS), (dict(weight=FAKE + 2), MIS), (dict(rows=0, logits=None), 0),
    (dict(loss=None, lse=None, dlogits=None), 0)])
def test_cross_entropy_refusals(L, kw, want):
    assert call(L, "opt_cross_entropy", lm.OptCrossEntropyArgs, CROSS_ENTROPY, kw, None) == want


def test_null_arguments(L):
    for name in ("opt_embedding_forward", "opt_recurrence_forward", "opt_recurrence_backward", "opt_checkpoint_restore",
                 "opt_cross_entropy"):
        assert getattr(L, name)(None, None) == INV
    assert L.opt_embedding_backward(None, FAKE, 1 << 20, None) == INV


def test_cpu_tensors_are_refused():
    f, b = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        mp.embedding(i, b(8, 16), b(4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        mp.embedding_backward(i, b(4, 16), f(8, 16))
    with pytest.raises(ValueError, match="CUDA"):
        mp.gated_recurrence(b(4, 16), b(4, 16), b(4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        mp.gated_recurrence_backward(b(4, 16), b(4, 16), b(4, 16), f(1, 16), b(4, 16), b(4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        mp.checkpoint_save(b(4, 16), torch.zeros(4, 16, dtype=torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        mp.cross_entropy(b(4, 16), i, f(4))
    with pytest.raises(TypeError, match="unsupported type"):
        mp.cross_entropy(i, i)
    with pytest.raises(TypeError, match="unsupported type"):
        mp.recurrence_states(4, 16, torch.float16)
    with pytest.raises(ValueError, match="activation"):
        mp.checkpoint_restore(torch.zeros(4, 16, dtype=torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8), act="tanh")


def test_packed_arguments_match_the_structs():
    """Field by field the same bytes as the ctypes structs of the header."""
    for pack, cls in ((lm._PACK_EMBEDDING, lm.OptEmbeddingArgs), (lm._PACK_EMBEDDING_GRAD, lm.OptEmbeddingGradArgs),
                      (lm._PACK_RECURRENCE, lm.OptRecurrenceArgs), (lm._PACK_RECURRENCE_GRAD, lm.OptRecurrenceGradArgs),
                      (lm._PACK_CHECKPOINT, lm.OptCheckpointArgs), (lm._PACK_CROSS_ENTROPY, lm.OptCrossEntropyArgs)):
        vals = [0.5 if t is ctypes.c_float else 1 + i for i, (_, t) in enumerate(cls._fields_)]
        assert pack(*vals) == bytes(cls(*vals))
