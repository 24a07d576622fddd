"""The language-model operators where a call takes several turns, passes or kernels that
smaller ones do not: wide recurrences in fp32, more rows of logits than the GPU
holds at once for every width, the radix sort's second look at rows beyond those
that it keeps, and states whose places the forward pass leaves.  Checks and tolerances are
those of test_language_gpu.py."""

import numpy as np
import pytest

from gpu_helpers import require_gpu, torch
import mixed_precision_optimizer_gb300 as mp
from test_language_gpu import (BF16, FP32, check_cross_entropy, check_embedding_backward, check_recurrence, gate_values, gen, normal,
                               output, ragged)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("cols", [2056, 4096, 4104, 4107])
@pytest.mark.parametrize("layout", ["dense", "odd slice"])
def test_wide_fp32_recurrences(cols, layout):
    """fp32 beyond the columns where warps and CTAs are shared out differently, one
    sequence, equal ones and packed ones, from one turn to several."""
    check_recurrence(700, cols, None, 1, FP32, layout)
    check_recurrence(140, cols, None, 7, FP32, layout)
    check_recurrence(300, cols, np.array([3, 3, 19, 20, 100, 100, 297]), 6, FP32, layout)
    check_recurrence(1100, cols, ragged(1100, 3, 1), 3, FP32, layout)


# Columns, and how many rows of them the GPU has room for at once: CTAs of 512 threads
# in all to an SM, a cluster of them to a row.
WIDTHS = [(1025, 64, 1), (4096, 64, 1), (4097, 128, 1), (8192, 128, 1), (16384, 256, 1), (32768, 256, 2), (32771, 256, 4),
          (65543, 256, 8), (131072, 256, 8)]


@pytest.mark.parametrize("cols,threads,ctas", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_cross_entropy_of_more_rows_than_the_gpu_holds(cols, threads, ctas, dtype):
    """Every cluster takes four rows or more: a place of the ring, of the statistics and of
    the mail is used again."""
    held = torch.cuda.get_device_properties(0).multi_processor_count * (512 // threads) // ctas
    rows = 3 * held + 5
    x = normal(1, (rows, cols), dtype, 3.0)
    labels = torch.randint(-1, cols, (rows,), generator=gen(2), device="cuda")
    labels[:2], labels[-2:] = torch.tensor([0, cols - 1], device="cuda"), torch.tensor([cols - 1, 0], device="cuda")
    for lo in range(0, rows, 1024):                      # what the oracle in 64 bits takes at a time
        hi = min(rows, lo + 1024)
        if lo == 0:
            loss, lse, g = output((rows,), FP32), output((rows,), FP32), output((rows, cols), dtype)
            mp.cross_entropy(x, labels, loss, lse=lse, dlogits=g, scale=0.37)
        part = check_cross_entropy(x[lo:hi], labels[lo:hi], 0.37)
        for a, b in zip(part, (loss, lse, g)):
            assert torch.equal(a, b[lo:hi])


@pytest.mark.parametrize("rows,vocab", [(40000, 128256), (70000, 1 << 20), (66000, 900)])
def test_embedding_backward_sorts_more_rows_than_it_keeps(rows, vocab):
    """Two, three passes and one over rows that a lane reads again in each."""
    tokens = (torch.rand(rows, generator=gen(3), device="cuda") ** 3 * (vocab + 1)).long() - 1
    check_embedding_backward(tokens, normal(4, (rows, 8)), vocab, 0.3, True)


@pytest.mark.parametrize("sequences,starts", [(40, None), (5, None), (3, [3, 11, 19, 30]), (4, [0, 8, 8, 24, 37])])
def test_states_are_needed_only_where_they_are_written(sequences, starts):
    x, gate, dy = normal(1, (40, 72)), gate_values(2, (40, 72), BF16), normal(3, (40, 72))
    h0, st = normal(4, (sequences, 72), FP32), None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    outs = []
    for before in (0.0, float("nan"), 1e30):
        states, y = mp.recurrence_states(40, 72, BF16).fill_(before), torch.zeros(40, 72, dtype=BF16, device="cuda")
        mp.gated_recurrence(x, gate, y, starts=st, sequences=sequences, h0=h0, states=states)
        dx, dg, dh0 = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(h0)
        mp.gated_recurrence_backward(dy, x, gate, states, dx, dg, starts=st, sequences=sequences, h0=h0, dh0=dh0)
        outs.append((y, dx, dg, dh0))
        assert all(torch.isfinite(t.float()).all() for t in outs[-1])
    for t in zip(*outs):
        assert torch.equal(t[0], t[1]) and torch.equal(t[0], t[2])
