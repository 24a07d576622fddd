"""What calls of the language-model operators leave: places of the recurrence's states."""

import pytest

from gpu_helpers import require_gpu, torch
import mixed_precision_optimizer_gb300 as mp
from test_language_gpu import BF16, FP32, gate_values, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


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
